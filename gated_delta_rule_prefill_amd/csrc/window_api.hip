// window_api.hip -- C entry points of the window-attention operators: argument
// checks, workspace and launches (host code only).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/kda.h"
#include "api_checks.h"
#include "latent_launch.h"
#include "window_launch.h"

namespace {

using namespace kda::api;

// Heads, sizes and options that all calls share.
kda_status check_heads(int32_t H, int32_t Hk, int32_t d, int32_t dtype) {
    if (!dtype_ok(dtype)) return fail(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_DTYPE_F32 or KDA_DTYPE_BF16");
    if (H <= 0 || H > 65535 || Hk <= 0 || H % Hk != 0)
        return fail(KDA_ERR_INVALID_ARGUMENT, "H must be in [1, 65535] and a multiple of Hk >= 1");
    if (d != 64 && d != 128) return fail(KDA_ERR_UNSUPPORTED, "d must be 64 or 128");
    return KDA_OK;
}
kda_status check_window(int32_t window, int32_t sinks, float scale) {
    if (window < 1) return fail(KDA_ERR_INVALID_ARGUMENT, "window must be >= 1");
    if (sinks < 0 || sinks > kda::WINDOW_MAX_SINKS) return fail(KDA_ERR_INVALID_ARGUMENT, "sinks must be in [0, 64]");
    if (!(scale > 0.f) || !std::isfinite(scale)) return fail(KDA_ERR_INVALID_ARGUMENT, "scale must be finite and > 0");
    return KDA_OK;
}
kda_status check_alignment(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARGUMENT, "every pointer must be 16-byte aligned");
    return KDA_OK;
}
kda_status check_strides(std::initializer_list<int64_t> strides, int32_t dtype) {
    for (int64_t s : strides)
        if (!stride_ok(s, dtype)) return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be >= 0 and multiples of 16 bytes");
    return KDA_OK;
}

kda_status check_inputs(const kda_window_inputs* in) {
    if (!in) return fail(KDA_ERR_INVALID_ARGUMENT, "inputs must be non-NULL");
    if (kda_status st = check_heads(in->H, in->Hk, in->d, in->dtype)) return st;
    if (kda_status st = check_window(in->window, in->sinks, in->scale)) return st;
    if (in->num_seqs <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs must be >= 1");
    if (in->total_q < 0 || in->total_k < 0 || in->total_q > kMaxRows || in->total_k > kMaxRows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "total_q and total_k must be in [0, 2^31 - 4096]");
    const int64_t rows = in->total_q * (in->H / in->Hk);
    if (rows > kMaxRows) return fail(KDA_ERR_INVALID_ARGUMENT, "total_q * H / Hk must be <= 2^31 - 4096");
    if (!in->cu_seqlens_q) {
        if (in->cu_seqlens_k) return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_k needs cu_seqlens_q");
        if (in->total_q % in->num_seqs != 0 || in->total_k % in->num_seqs != 0)
            return fail(KDA_ERR_INVALID_ARGUMENT, "without cu_seqlens, the totals must be multiples of num_seqs");
    } else if (!in->cu_seqlens_k && in->total_k != in->total_q) {
        return fail(KDA_ERR_INVALID_ARGUMENT, "without cu_seqlens_k, total_k must equal total_q");
    }
    if (in->total_q > 0 && !in->q) return fail(KDA_ERR_INVALID_ARGUMENT, "q must be non-NULL");
    if (in->total_k > 0 && (!in->k || !in->v)) return fail(KDA_ERR_INVALID_ARGUMENT, "k and v must be non-NULL");
    if (kda_status st = check_alignment({in->q, in->k, in->v})) return st;
    if (kda_status st = check_strides({in->q_token_stride, in->q_head_stride, in->k_token_stride, in->k_head_stride,
                                       in->v_token_stride, in->v_head_stride}, in->dtype))
        return st;
    for (int64_t s : {in->q_token_stride, in->k_token_stride, in->v_token_stride, (int64_t)in->H * in->d})
        if (s >= (int64_t)1 << 23)   // a tile's 64 rows are addressed with 32-bit offsets
            return fail(KDA_ERR_INVALID_ARGUMENT, "token strides and H * d must be below 2^23 elements");
    // every kernel's grid: tiles (at least 64 rows each, and one more per sequence) times key heads
    if ((std::max(rows, in->total_k) / 64 + in->num_seqs) * in->Hk >= (int64_t)1 << 24)
        return fail(KDA_ERR_INVALID_ARGUMENT, "too many tiles ((rows / 64 + num_seqs) * Hk must be below 2^24)");
    return KDA_OK;
}

// KDA_DEBUG_SYNC: both sets of offsets.  Sequences need not be all of the rows.
kda_status check_offsets(const kda_window_inputs* in, hipStream_t stream) {
    if (kda_status st = kda::debug_check_offsets(in->cu_seqlens_q, in->num_seqs, in->total_q, false, stream)) return st;
    return kda::debug_check_offsets(in->cu_seqlens_k, in->num_seqs, in->total_k, false, stream);
}

// The paged cache and the packed new tokens over it.
kda_status check_cache(const kda_kv_cache* c, const int32_t* cu_seqlens, int64_t total_tokens, int32_t num_seqs,
                       int32_t dtype) {
    if (!c) return fail(KDA_ERR_INVALID_ARGUMENT, "cache must be non-NULL");
    if (num_seqs <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs must be >= 1");
    if (total_tokens < 0 || total_tokens > kMaxRows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens must be in [0, 2^31 - 4096]");
    if (!cu_seqlens && total_tokens % num_seqs != 0)
        return fail(KDA_ERR_INVALID_ARGUMENT, "without cu_seqlens, total_tokens must be a multiple of num_seqs");
    if (c->num_pages <= 0 || c->page_size <= 0 || c->max_pages <= 0)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_pages, page_size and max_pages must be >= 1");
    if ((int64_t)c->num_pages * c->page_size > kMaxRows || (int64_t)c->max_pages * c->page_size > kMaxRows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_pages and max_pages times page_size must be <= 2^31 - 4096");
    if (!c->k || !c->v || !c->block_table || !c->seq_lens)
        return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's k, v, block_table and seq_lens must be non-NULL");
    if (kda_status st = check_alignment({c->k, c->v})) return st;
    return check_strides({c->page_stride, c->token_stride, c->head_stride}, dtype);
}

kda_status check_workspace(const void* workspace, size_t workspace_bytes, size_t need) {
    if (!aligned16(workspace)) return fail(KDA_ERR_INVALID_ARGUMENT, "every pointer must be 16-byte aligned");
    if (!workspace && workspace_bytes != 0)
        return fail(KDA_ERR_INVALID_ARGUMENT, "workspace_bytes given without a workspace");
    if (workspace && workspace_bytes < need) {
        kda::set_last_error("workspace too small: need " + std::to_string(need) + " bytes");
        return KDA_ERR_WORKSPACE;
    }
    return KDA_OK;
}

// Calls go(workspace) with the caller's workspace, or with one allocated and freed
// on the stream.
template <typename F>
kda_status with_workspace(void* workspace, size_t need, hipStream_t stream, const char* what, F go) {
    void* ws = workspace;
    if (!ws)
        if (kda_status st = launched(hipMallocAsync(&ws, need, stream), "hipMallocAsync")) return st;
    kda_status st = launched(go(static_cast<unsigned char*>(ws)), what);
    if (!workspace) {
        const kda_status fr = launched(hipFreeAsync(ws, stream), "hipFreeAsync");
        if (st == KDA_OK) st = fr;
    }
    return st;
}

// Byte offset of the sinks' partial gradients in the backward pass's workspace, and its size.
struct BackwardSpace {
    size_t part, bytes;
    BackwardSpace(int64_t total_q, int32_t num_seqs, int32_t H, int32_t Hk, int32_t d, int32_t sinks) {
        part = align256((size_t)total_q * H * 8);
        bytes = part + align256((size_t)kda::window_slots(total_q, num_seqs) * Hk * sinks * 2 * d * 4) + 256;
    }
};

kda_status check_norm(const kda_norm_heads* q, const kda_norm_heads* k, const int32_t* positions,
                      const float* inv_freq, int64_t total_tokens, int32_t d, int32_t start, int32_t dr,
                      kda_dtype dtype, float eps, float amplitude, uint32_t flags, bool backward) {
    if (!q) return fail(KDA_ERR_INVALID_ARGUMENT, "q must be non-NULL");
    if (!dtype_ok(dtype)) return fail(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_DTYPE_F32 or KDA_DTYPE_BF16");
    if (flags & ~(uint32_t)KDA_ROTARY_INTERLEAVED) return fail(KDA_ERR_INVALID_ARGUMENT, "unknown flag bits");
    if (total_tokens < 0 || total_tokens > kMaxRows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens must be in [0, 2^31 - 4096]");
    if (d < 2 || d > 256 || d % 2 != 0) return fail(KDA_ERR_UNSUPPORTED, "d must be even and in [2, 256]");
    if (dr < 0 || dr % 2 != 0 || start < 0 || start > d || dr > d - start)
        return fail(KDA_ERR_INVALID_ARGUMENT, "dr must be even and >= 0, with 0 <= start and start + dr <= d");
    if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(KDA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
    if (!std::isfinite(amplitude)) return fail(KDA_ERR_INVALID_ARGUMENT, "amplitude must be finite");
    if (dr == 0 && (positions || inv_freq))
        return fail(KDA_ERR_INVALID_ARGUMENT, "positions and inv_freq need dr > 0");
    if (dr > 0 && total_tokens > 0 && (!positions || !inv_freq))
        return fail(KDA_ERR_INVALID_ARGUMENT, "dr > 0 needs positions and inv_freq");
    if (kda_status st = check_alignment({positions, inv_freq})) return st;
    const uintptr_t unit = elem_size(dtype) - 1;
    for (const kda_norm_heads* s : {q, k}) {
        if (!s) continue;
        if (s->H <= 0 || s->H > 65535) return fail(KDA_ERR_INVALID_ARGUMENT, "H must be in [1, 65535]");
        if (total_tokens > 0 && (!s->x || (backward ? !s->dy || !s->dx : !s->y)))
            return fail(KDA_ERR_INVALID_ARGUMENT, "the heads' tensors must be non-NULL");
        if (kda_status st = check_alignment({s->weight, backward ? s->dweight : nullptr})) return st;
        const void* ptrs[] = {s->x, backward ? s->dy : s->y, backward ? s->dx : nullptr};
        for (const void* p : ptrs)
            if (reinterpret_cast<uintptr_t>(p) & unit)
                return fail(KDA_ERR_INVALID_ARGUMENT, "the heads' tensors must be aligned to one element");
        const int64_t in[] = {s->x_token_stride, s->x_head_stride, backward ? s->dy_token_stride : 0,
                              backward ? s->dy_head_stride : 0};
        for (int64_t x : in)
            if (x < 0 || x >= ((int64_t)1 << 40)) return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be in [0, 2^40)");
        const void* to = backward ? s->dx : s->y;
        const int64_t ts = backward ? s->dx_token_stride : s->y_token_stride;
        const int64_t hs = backward ? s->dx_head_stride : s->y_head_stride;
        if (ts < 0 || hs < 0 || ts >= ((int64_t)1 << 40) || hs >= ((int64_t)1 << 40))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be in [0, 2^40)");
        if ((s->H > 1 && hs < d) || (total_tokens > 1 && ts < d))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides of a written tensor must be at least d");
        auto in_place = [&](const void* p, int64_t pt, int64_t ph) {
            return p != to || ((total_tokens <= 1 || pt == ts) && (s->H <= 1 || ph == hs));
        };
        if (total_tokens > 0 && (!in_place(s->x, s->x_token_stride, s->x_head_stride) ||
                                 (backward && !in_place(s->dy, s->dy_token_stride, s->dy_head_stride))))
            return fail(KDA_ERR_INVALID_ARGUMENT, "in place, both tensors must have the same strides");
    }
    return KDA_OK;
}

kda::QkNorm norm_args(const kda_norm_heads* q, const kda_norm_heads* k, const int32_t* positions, const float* inv_freq,
                      int64_t total_tokens, int32_t d, int32_t start, int32_t dr, float eps, float amplitude,
                      uint32_t flags) {
    kda::QkNorm a{};
    a.q = *q;
    if (k) a.k = *k;
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.total_tokens = total_tokens;
    a.d = d;
    a.start = start;
    a.dr = dr;
    a.eps = eps;
    a.amplitude = amplitude;
    a.flags = flags;
    return a;
}

}  // namespace

extern "C" {

kda_status kda_window_attention(const kda_window_inputs* in, void* o, float* lse, void* stream) {
    try {
        if (kda_status st = check_inputs(in)) return st;
        if (in->total_q == 0) return KDA_OK;
        if (!o) return fail(KDA_ERR_INVALID_ARGUMENT, "o must be non-NULL");
        if (kda_status st = check_alignment({o, lse})) return st;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        if (kda_status st = check_offsets(in, s)) return st;
        const kda::WindowArgs a{*in, kda_kv_cache{}, o, lse};
        return launched(kda::launch_window_attention(a, false, s), "window attention kernel");
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_window_attention");
    }
}

size_t kda_window_attention_backward_workspace_bytes(int64_t total_q, int32_t num_seqs, int32_t H, int32_t Hk,
                                                     int32_t d, int32_t sinks) {
    if (total_q < 0 || total_q > kMaxRows || num_seqs <= 0 || H <= 0 || H > 65535 || Hk <= 0 || H % Hk != 0 ||
        (d != 64 && d != 128) || sinks < 0 || sinks > kda::WINDOW_MAX_SINKS)
        return 0;
    return BackwardSpace(total_q, num_seqs, H, Hk, d, sinks).bytes;
}

kda_status kda_window_attention_backward(const kda_window_inputs* in, const void* o, const float* lse, const void* d_o,
                                         void* dq, void* dk, int64_t dk_token_stride, int64_t dk_head_stride, void* dv,
                                         int64_t dv_token_stride, int64_t dv_head_stride, void* workspace,
                                         size_t workspace_bytes, void* stream_ptr) {
    try {
        if (kda_status st = check_inputs(in)) return st;
        if (in->total_q > 0 && (!o || !lse || !d_o || !dq))
            return fail(KDA_ERR_INVALID_ARGUMENT, "o, lse, d_o and dq must be non-NULL");
        if (in->total_k > 0 && (!dk || !dv)) return fail(KDA_ERR_INVALID_ARGUMENT, "dk and dv must be non-NULL");
        if (kda_status st = check_alignment({o, lse, d_o, dq, dk, dv})) return st;
        if (kda_status st = check_strides({dk_token_stride, dk_head_stride, dv_token_stride, dv_head_stride}, in->dtype))
            return st;
        // written rows must not overlap
        if ((in->Hk > 1 && (dk_head_stride < in->d || dv_head_stride < in->d)) ||
            (in->total_k > 1 && (dk_token_stride < in->d || dv_token_stride < in->d)))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides of dk and dv must be at least d");
        // the second kernel's grid: key tiles and pieces of the sinks
        if ((in->total_k / 64 + in->total_q / kda::WINDOW_PIECE + 2 * (int64_t)in->num_seqs) * in->Hk >= (int64_t)1 << 24)
            return fail(KDA_ERR_INVALID_ARGUMENT,
                        "too many tiles ((total_k / 64 + total_q / 256 + 2 num_seqs) * Hk must be below 2^24)");
        const BackwardSpace s(in->total_q, in->num_seqs, in->H, in->Hk, in->d, in->sinks);
        if (kda_status st = check_workspace(workspace, workspace_bytes, s.bytes)) return st;
        if (in->total_q == 0 && in->total_k == 0) return KDA_OK;
        hipStream_t stream = reinterpret_cast<hipStream_t>(stream_ptr);
        if (kda_status st = check_offsets(in, stream)) return st;
        return with_workspace(workspace, s.bytes, stream, "window backward kernels", [&](unsigned char* ws) {
            const kda::WindowGrads g{o, lse, d_o, dq, dk, dk_token_stride, dk_head_stride, dv, dv_token_stride,
                                     dv_head_stride, reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + s.part)};
            return kda::launch_window_attention_backward(*in, g, stream);
        });
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_window_attention_backward");
    }
}

size_t kda_window_decode_workspace_bytes(int32_t d) {
    return d == 64 || d == 128 ? align256(kda::window_decode_workspace(d)) : 0;
}

kda_status kda_window_decode(const kda_kv_cache* cache, const void* q, int64_t q_token_stride, int64_t q_head_stride,
                             const int32_t* cu_seqlens, int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t Hk,
                             int32_t d, kda_dtype dtype, int32_t window, int32_t sinks, float scale, void* o,
                             float* lse, void* workspace, size_t workspace_bytes, void* stream_ptr) {
    try {
        if (kda_status st = check_heads(H, Hk, d, dtype)) return st;
        if (kda_status st = check_window(window, sinks, scale)) return st;
        if (kda_status st = check_cache(cache, cu_seqlens, total_tokens, num_seqs, dtype)) return st;
        if (total_tokens * H > kMaxRows)
            return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens * H must be <= 2^31 - 4096");
        if ((total_tokens * (H / Hk) / 16 + num_seqs) * Hk >= (int64_t)1 << 24)   // workgroups of 256 threads
            return fail(KDA_ERR_INVALID_ARGUMENT,
                        "too many tiles ((total_tokens * H / Hk / 16 + num_seqs) * Hk must be below 2^24)");
        if (total_tokens > 0 && (!q || !o)) return fail(KDA_ERR_INVALID_ARGUMENT, "q and o must be non-NULL");
        if (kda_status st = check_alignment({q, o, lse})) return st;
        if (kda_status st = check_strides({q_token_stride, q_head_stride}, dtype)) return st;
        const size_t need = kda_window_decode_workspace_bytes(d);
        if (kda_status st = check_workspace(workspace, workspace_bytes, need)) return st;
        if (total_tokens == 0) return KDA_OK;
        hipStream_t stream = reinterpret_cast<hipStream_t>(stream_ptr);
        if (kda_status st = kda::debug_check_offsets(cu_seqlens, num_seqs, total_tokens, false, stream)) return st;
        kda::WindowArgs a{kda_window_inputs{}, *cache, o, lse};
        a.in.q = q;
        a.in.q_token_stride = q_token_stride;
        a.in.q_head_stride = q_head_stride;
        a.in.cu_seqlens_q = cu_seqlens;
        a.in.total_q = total_tokens;
        a.in.num_seqs = num_seqs;
        a.in.H = H;
        a.in.Hk = Hk;
        a.in.d = d;
        a.in.dtype = dtype;
        a.in.window = window;
        a.in.sinks = sinks;
        a.in.scale = scale;
        return with_workspace(workspace, need, stream, "window decode kernels",
                              [&](unsigned char* ws) { return kda::launch_window_decode(a, ws, stream); });
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_window_decode");
    }
}

kda_status kda_kv_append(const kda_kv_cache* cache, const void* k, int64_t k_token_stride, int64_t k_head_stride,
                         const void* v, int64_t v_token_stride, int64_t v_head_stride, const int32_t* cu_seqlens,
                         int64_t total_tokens, int32_t num_seqs, int32_t Hk, int32_t d, kda_dtype dtype,
                         const float* norm_weight, float eps, const float* inv_freq, int32_t start, int32_t dr,
                         float amplitude, uint32_t flags, void* k_out, void* stream_ptr) {
    try {
        if (kda_status st = check_heads(Hk, Hk, d, dtype)) return st;
        if (kda_status st = check_cache(cache, cu_seqlens, total_tokens, num_seqs, dtype)) return st;
        if (flags & ~(uint32_t)KDA_ROTARY_INTERLEAVED) return fail(KDA_ERR_INVALID_ARGUMENT, "unknown flag bits");
        if (dr < 0 || dr % 2 != 0 || start < 0 || start > d || dr > d - start)
            return fail(KDA_ERR_INVALID_ARGUMENT, "dr must be even and >= 0, with 0 <= start and start + dr <= d");
        if ((dr > 0) != (inv_freq != nullptr)) return fail(KDA_ERR_INVALID_ARGUMENT, "inv_freq goes with dr > 0");
        if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(KDA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
        if (!std::isfinite(amplitude)) return fail(KDA_ERR_INVALID_ARGUMENT, "amplitude must be finite");
        if (total_tokens > 0 && (!k || !v)) return fail(KDA_ERR_INVALID_ARGUMENT, "k and v must be non-NULL");
        if (kda_status st = check_alignment({k, v, norm_weight, inv_freq, k_out})) return st;
        if (kda_status st = check_strides({k_token_stride, k_head_stride, v_token_stride, v_head_stride}, dtype)) return st;
        // written rows must not overlap
        if ((Hk > 1 && cache->head_stride < d) || (cache->page_size > 1 && cache->token_stride < d) ||
            (cache->num_pages > 1 && cache->page_stride < d))
            return fail(KDA_ERR_INVALID_ARGUMENT, "the cache's strides must be at least d");
        if (total_tokens == 0) return KDA_OK;
        hipStream_t stream = reinterpret_cast<hipStream_t>(stream_ptr);
        if (kda_status st = kda::debug_check_offsets(cu_seqlens, num_seqs, total_tokens, false, stream)) return st;
        const kda::KvAppend a{*cache, k, k_token_stride, k_head_stride, v, v_token_stride, v_head_stride, cu_seqlens,
                              total_tokens, num_seqs, Hk, d, norm_weight, eps, inv_freq, start, dr, amplitude, flags,
                              k_out};
        return launched(kda::launch_kv_append(a, dtype == KDA_DTYPE_BF16, stream), "kv append kernel");
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_kv_append");
    }
}

kda_status kda_qk_norm_rotary(const kda_norm_heads* q, const kda_norm_heads* k, const int32_t* positions,
                              const float* inv_freq, int64_t total_tokens, int32_t d, int32_t start, int32_t dr,
                              kda_dtype dtype, float eps, float amplitude, uint32_t flags, void* stream) {
    try {
        if (kda_status st = check_norm(q, k, positions, inv_freq, total_tokens, d, start, dr, dtype, eps, amplitude, flags,
                                       false))
            return st;
        if (total_tokens == 0) return KDA_OK;
        const kda::QkNorm a = norm_args(q, k, positions, inv_freq, total_tokens, d, start, dr, eps, amplitude, flags);
        return launched(kda::launch_qk_norm_rotary(a, dtype == KDA_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)),
                        "qk norm kernel");
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_qk_norm_rotary");
    }
}

size_t kda_qk_norm_rotary_backward_workspace_bytes(int32_t d) {
    return d < 2 || d > 256 || d % 2 != 0 ? 0 : align256(kda::qk_norm_workspace(d));
}

kda_status kda_qk_norm_rotary_backward(const kda_norm_heads* q, const kda_norm_heads* k, const int32_t* positions,
                                       const float* inv_freq, int64_t total_tokens, int32_t d, int32_t start,
                                       int32_t dr, kda_dtype dtype, float eps, float amplitude, uint32_t flags,
                                       void* workspace, size_t workspace_bytes, void* stream_ptr) {
    try {
        if (kda_status st = check_norm(q, k, positions, inv_freq, total_tokens, d, start, dr, dtype, eps, amplitude, flags,
                                       true))
            return st;
        const size_t need = kda_qk_norm_rotary_backward_workspace_bytes(d);
        if (kda_status st = check_workspace(workspace, workspace_bytes, need)) return st;
        if (total_tokens == 0 && !q->dweight && !(k && k->dweight)) return KDA_OK;
        hipStream_t stream = reinterpret_cast<hipStream_t>(stream_ptr);
        kda::QkNorm a = norm_args(q, k, positions, inv_freq, total_tokens, d, start, dr, eps, amplitude, flags);
        return with_workspace(workspace, need, stream, "qk norm backward kernels", [&](unsigned char* ws) {
            a.part = reinterpret_cast<float*>(ws);
            return kda::launch_qk_norm_rotary_backward(a, dtype == KDA_DTYPE_BF16, stream);
        });
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_qk_norm_rotary_backward");
    }
}

}  // extern "C"
