"""The library's host side without a GPU: a child process loads libkda.so behind
a few HIP entry points of its own, which count the launches, refuse one of them
on demand and treat device memory as host memory.  No kernel runs."""
import json
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STUB = r"""
#include <string.h>
#include <stdlib.h>
typedef struct { unsigned x, y, z; } dim3_;
static int launches, refused_at, syncs, error;
int stub_launches(void) { return launches; }
int stub_syncs(void) { return syncs; }
void stub_reset(int refuse) { launches = syncs = error = 0; refused_at = refuse; }
int __hipPushCallConfiguration(dim3_ g, dim3_ b, size_t m, void *s) { return 0; }
int __hipPopCallConfiguration(dim3_ *g, dim3_ *b, size_t *m, void **s) {
    g->x = g->y = g->z = b->x = b->y = b->z = 1; *m = 0; *s = 0; return 0;
}
int hipLaunchKernel(const void *f, dim3_ g, dim3_ b, void **a, size_t m, void *s) {
    if (++launches == refused_at) error = 9;   /* hipErrorInvalidConfiguration */
    return error;
}
int hipGetLastError(void) { int e = error; error = 0; return e; }
int hipStreamSynchronize(void *s) { ++syncs; return 0; }
int hipMemcpyAsync(void *d, const void *s, size_t n, int k, void *q) { memcpy(d, s, n); return 0; }
int hipMallocAsync(void **p, size_t n, void *s) { *p = aligned_alloc(256, n); return *p ? 0 : 2; }
int hipFreeAsync(void *p, void *s) { free(p); return 0; }
const char *hipGetErrorString(int e) { return "refused"; }
"""

CHILD = r"""
import ctypes, json, struct, sys
stub = ctypes.CDLL(sys.argv[1], mode=ctypes.RTLD_GLOBAL)
sys.path.insert(0, sys.argv[2])
from gated_delta_rule_prefill_amd import kda
lib = kda.lib()
A = 1 << 20  # a device address that nothing reads

def offsets(*values):
    return (ctypes.c_int32 * len(values))(*values)

def address(x):
    return ctypes.addressof(x) if x is not None else 0

def inputs(cu_q=None, cu_k=None, bf16=True, T=300, H=4, dr=64):
    return kda._INPUTS.pack(A, A, A, A if dr else 0, H * (128 + dr), 128 + dr, H * 256, 256, H * 256, 256, dr,
                            address(cu_q), address(cu_k), T, T, 2, H, 128, dr, 128, 1 if bf16 else 0, 1, 0.1)

def forward(**kw):
    return lib.kda_latent_attention(inputs(**kw), A, A, None)

def backward(**kw):
    dr = kw.get("dr", 64)
    return lib.kda_latent_attention_backward(inputs(**kw), A, A, A, A, A, 4 * 256, 256, A, 4 * 256, 256,
                                             A if dr else 0, A, 1 << 40, None)

def decode(cu=None, T=2, H=4, bf16=True, ws=A):
    return lib.kda_latent_decode(A, H * 576, 576, A, 10, 64, A, 4, A, address(cu), T, 2, H, 512, 64, int(bf16), 0.1,
                                 A, A, ws, (1 << 40) if ws else 0, None)

def append(cu=None):
    return lib.kda_latent_append(A, 10, 64, A, 4, A, address(cu), 2, 2, 512, 64, 1, A, 576, A, 576, A, 1e-6, A, 1.0,
                                 0, A, A, None)

def rotary():
    return lib.kda_rotary(A, 256, 64, 2 * A, 256, 64, A, A, 10, 4, 64, 0, 64, 1, 1.0, 0, None)

def call(f, refuse=0, **kw):
    stub.stub_reset(refuse)
    status = f(**kw)
    return dict(status=status, launches=stub.stub_launches(), syncs=stub.stub_syncs(),
                text=kda.last_error() if status else "")

result = {}
exec(sys.stdin.read())
print("RESULT|" + json.dumps(result))
"""


def run(tmp_path, code, **env):
    """`code` in the child, after CHILD; what it puts into `result`."""
    src, so = tmp_path / "stub.c", tmp_path / "libstub.so"
    src.write_text(STUB)
    subprocess.run(["gcc", "-shared", "-fPIC", "-O1", "-o", str(so), str(src)], check=True, capture_output=True)
    r = subprocess.run([sys.executable, "-c", CHILD, str(so), ROOT], input=code, env=dict(os.environ, **env),
                       capture_output=True, text=True, timeout=300)
    line = [ln for ln in r.stdout.splitlines() if ln.startswith("RESULT|")]
    assert r.returncode == 0 and line, (r.returncode, r.stdout[-2000:], r.stderr[-2000:])
    return json.loads(line[0][7:])
