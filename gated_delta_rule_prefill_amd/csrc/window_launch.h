// window_launch.h -- host-visible launchers of the window-attention kernels and
// the argument blocks they share (no device code).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

constexpr int WINDOW_MAX_SINKS = 64;   // one key tile of the backward pass

// How many of the positions from `from` >= key on have a key in their window.  key + window
// may pass 32 bits; key - from cannot and is not above 0.
__host__ __device__ inline int positions_in_window(int key, int window, int from) {
    const int n = key - from + window;
    return n > 0 ? n : 0;
}

// The packed form and the paged one.  Paged: k and v come from the cache, and
// total_k, cu_seqlens_k and their strides are not looked at.
struct WindowArgs {
    kda_window_inputs in;
    kda_kv_cache pages;
    void* o;
    float* lse;
};
hipError_t launch_window_attention(const WindowArgs& a, bool paged, hipStream_t stream);

// row_stats: [H, total_q, 2] fp32 (lse in powers of two, delta); part: the sinks'
// partial gradients, [slots, Hk, sinks, 2 d] fp32 (window_backward.hip)
struct WindowGrads {
    const void* o;
    const float* lse;
    const void* d_o;
    void* dq;
    void* dk;
    int64_t dk_token_stride, dk_head_stride;
    void* dv;
    int64_t dv_token_stride, dv_head_stride;
    float* row_stats;
    float* part;
};
// Tokens of a piece of the sinks' gradients, and the slots that a batch's pieces take.  Short
// pieces, as with a small window they are the longest walks: 4,096 tokens, 32/8 heads of
// 128, window 128, dk and dv in us with 1,024, 512 and 256 tokens: 169, 105, 72; window
// 1,024: 224, 181, 167.
constexpr int WINDOW_PIECE = 256;
inline int64_t window_slots(int64_t total_q, int32_t num_seqs) { return total_q / WINDOW_PIECE + 2 * (int64_t)num_seqs; }
hipError_t launch_window_attention_backward(const kda_window_inputs& in, const WindowGrads& g, hipStream_t stream);

size_t window_decode_workspace(int32_t d);
hipError_t launch_window_decode(const WindowArgs& a, void* workspace, hipStream_t stream);

struct KvAppend {
    kda_kv_cache pages;
    const void* k;
    int64_t k_token_stride, k_head_stride;
    const void* v;
    int64_t v_token_stride, v_head_stride;
    const int32_t* cu_seqlens;
    int64_t total_tokens;
    int32_t num_seqs, Hk, d;
    const float* norm_weight;
    float eps;
    const float* inv_freq;
    int32_t start, dr;
    float amplitude;
    uint32_t flags;
    void* k_out;
};
hipError_t launch_kv_append(const KvAppend& a, bool bf16_io, hipStream_t stream);

struct QkNorm {
    kda_norm_heads q, k;   // k.H = 0 without keys
    const int32_t* positions;
    const float* inv_freq;
    int64_t total_tokens;
    int32_t d, start, dr;
    float eps, amplitude;
    uint32_t flags;
    float* part;           // backward: [workgroups, 2, d] fp32
};
size_t qk_norm_workspace(int32_t d);
hipError_t launch_qk_norm_rotary(const QkNorm& a, bool bf16_io, hipStream_t stream);
hipError_t launch_qk_norm_rotary_backward(const QkNorm& a, bool bf16_io, hipStream_t stream);

}  // namespace kda
