// latent_launch.h -- host-visible launchers of the latent-attention kernels
// and the argument blocks they share (no device code).
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/kda.h"

namespace kda {

// To be called behind every kernel's launch: its error, or under KDA_DEBUG_SYNC
// that of its execution.
hipError_t launch_result(hipStream_t stream);

hipError_t launch_latent_attention(const kda_latent_inputs& in, void* o, float* lse,
                                   hipStream_t stream);

// row_stats: [H, total_q, 2] fp32 (lse in powers of two, delta); pe_part: [total_k, H, dr] fp32
struct LatentGrads {
    const void* o;
    const float* lse;
    const void* d_o;
    void* dq;
    void* dk;
    int64_t dk_token_stride, dk_head_stride;
    void* dv;
    int64_t dv_token_stride, dv_head_stride;
    void* dk_pe;
    float* row_stats;
    float* pe_part;
    float* part_k;   // [splits, total_k, H, dn + dr + dv], [splits, total_q, H, dn + dr]
    float* part_q;
};
// Workgroups that share an fp32 tile of a batch of so many rows.
int latent_splits(int64_t rows, int32_t H);
hipError_t launch_latent_attention_backward(const kda_latent_inputs& in, const LatentGrads& g,
                                            hipStream_t stream);

struct LatentDecode {
    const void* q;
    int64_t q_token_stride, q_head_stride;
    const void* cache;
    int32_t num_pages, page_size;
    const int32_t* block_table;
    int32_t max_pages;
    const int32_t* seq_lens;
    const int32_t* cu_seqlens;
    int64_t total_tokens;
    int32_t num_seqs, H, dl, dr;
    float scale;
    void* o;
    float* lse;
    void* workspace;
};
size_t latent_decode_workspace(int32_t dl);
hipError_t launch_latent_decode(const LatentDecode& a, bool bf16_io, hipStream_t stream);

struct LatentAppend {
    void* cache;
    int32_t num_pages, page_size;
    const int32_t* block_table;
    int32_t max_pages;
    const int32_t* seq_lens;
    const int32_t* cu_seqlens;
    int64_t total_tokens;
    int32_t num_seqs, dl, dr;
    const void* c;
    int64_t c_token_stride;
    const void* k_pe;
    int64_t k_pe_token_stride;
    const float* norm_weight;
    float eps;
    const float* inv_freq;
    float amplitude;
    uint32_t flags;
    void* c_out;
    void* k_pe_out;
};
hipError_t launch_latent_append(const LatentAppend& a, bool bf16_io, hipStream_t stream);

struct Rotary {
    const void* x;
    int64_t x_token_stride, x_head_stride;
    void* y;
    int64_t y_token_stride, y_head_stride;
    const int32_t* positions;
    const float* inv_freq;
    int64_t total_tokens;
    int32_t H, d, start, dr;
    float amplitude;
    uint32_t flags;
};
hipError_t launch_rotary(const Rotary& a, bool bf16_io, hipStream_t stream);

}  // namespace kda
