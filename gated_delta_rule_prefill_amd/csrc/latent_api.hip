// latent_api.hip -- C entry points of the latent-attention operators: argument
// checks, workspace and launches (host code only).
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdint>
#include <string>

#include "../../include/kda.h"
#include "api_checks.h"
#include "latent_launch.h"

namespace {

using namespace kda::api;

kda_status check_inputs(const kda_latent_inputs* in) {
    if (!in) return fail(KDA_ERR_INVALID_ARGUMENT, "inputs must be non-NULL");
    if (!dtype_ok(in->dtype)) return fail(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_DTYPE_F32 or KDA_DTYPE_BF16");
    if (in->num_seqs <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs must be >= 1");
    if (in->H <= 0 || in->H > 65535) return fail(KDA_ERR_INVALID_ARGUMENT, "H must be in [1, 65535]");
    if (in->total_q < 0 || in->total_k < 0 || in->total_q > kMaxRows || in->total_k > kMaxRows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "total_q and total_k must be in [0, 2^31 - 4096]");
    if (in->dn != in->dv || (in->dn != 64 && in->dn != 128) || (in->dr != 0 && in->dr != 64))
        return fail(KDA_ERR_UNSUPPORTED, "dn = dv must be 64 or 128, dr 0 or 64");
    if (!(in->scale > 0.f) || !std::isfinite(in->scale))
        return fail(KDA_ERR_INVALID_ARGUMENT, "scale must be finite and > 0");
    if (!in->cu_seqlens_q) {
        if (in->cu_seqlens_k)
            return fail(KDA_ERR_INVALID_ARGUMENT, "cu_seqlens_k needs cu_seqlens_q");
        if (in->total_q % in->num_seqs != 0 || in->total_k % in->num_seqs != 0)
            return fail(KDA_ERR_INVALID_ARGUMENT, "without cu_seqlens, the totals must be multiples of num_seqs");
    } else if (!in->cu_seqlens_k && in->total_k != in->total_q) {
        return fail(KDA_ERR_INVALID_ARGUMENT, "without cu_seqlens_k, total_k must equal total_q");
    }
    if (in->total_q > 0 && !in->q) return fail(KDA_ERR_INVALID_ARGUMENT, "q must be non-NULL");
    if (in->total_k > 0 && (!in->k || !in->v || (in->dr && !in->k_pe)))
        return fail(KDA_ERR_INVALID_ARGUMENT, "k, v (and k_pe with dr > 0) must be non-NULL");
    const void* ptrs[] = {in->q, in->k, in->v, in->k_pe};
    for (const void* p : ptrs)
        if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARGUMENT, "every pointer must be 16-byte aligned");
    const int64_t strides[] = {in->q_token_stride, in->q_head_stride, in->k_token_stride, in->k_head_stride,
                               in->v_token_stride, in->v_head_stride, in->k_pe_token_stride};
    for (int64_t s : strides)
        if (!stride_ok(s, in->dtype))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be >= 0 and multiples of 16 bytes");
    const int64_t rows[] = {in->q_token_stride, in->k_token_stride, in->v_token_stride, in->k_pe_token_stride,
                            (int64_t)in->H * in->dv};
    for (int64_t s : rows)   // a tile's 64 rows are addressed with 32-bit offsets
        if (s >= (int64_t)1 << 23) return fail(KDA_ERR_INVALID_ARGUMENT, "token strides must be below 2^23 elements");
    // every kernel's grid: tiles (at least 64 rows each, and one more per sequence) times heads
    const int64_t most = (in->total_q > in->total_k ? in->total_q : in->total_k) / 64 + in->num_seqs;
    if (most * in->H >= (int64_t)1 << 24)   // of 256 threads each, in one dimension
        return fail(KDA_ERR_INVALID_ARGUMENT, "too many tiles ((rows / 64 + num_seqs) * H must be below 2^24)");
    return KDA_OK;
}

// KDA_DEBUG_SYNC: both sets of offsets.  Sequences need not be all of the rows.
kda_status check_offsets(const kda_latent_inputs* in, hipStream_t stream) {
    if (kda_status st = kda::debug_check_offsets(in->cu_seqlens_q, in->num_seqs, in->total_q, false, stream)) return st;
    return kda::debug_check_offsets(in->cu_seqlens_k, in->num_seqs, in->total_k, false, stream);
}

// The paged cache's arguments, shared by decode and append.
kda_status check_pages(const void* cache, int32_t num_pages, int32_t page_size, const int32_t* block_table,
                       int32_t max_pages, const int32_t* seq_lens, const int32_t* cu_seqlens, int64_t total_tokens,
                       int32_t num_seqs) {
    if (num_seqs <= 0) return fail(KDA_ERR_INVALID_ARGUMENT, "num_seqs must be >= 1");
    if (total_tokens < 0 || total_tokens > kMaxRows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens must be in [0, 2^31 - 4096]");
    if (num_pages <= 0 || page_size <= 0 || max_pages <= 0)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_pages, page_size and max_pages must be >= 1");
    if ((int64_t)num_pages * page_size > kMaxRows || (int64_t)max_pages * page_size > kMaxRows)
        return fail(KDA_ERR_INVALID_ARGUMENT, "num_pages and max_pages times page_size must be <= 2^31 - 4096");
    if (!cu_seqlens && total_tokens % num_seqs != 0)
        return fail(KDA_ERR_INVALID_ARGUMENT, "without cu_seqlens, total_tokens must be a multiple of num_seqs");
    if (!cache || !block_table || !seq_lens)
        return fail(KDA_ERR_INVALID_ARGUMENT, "cache, block_table and seq_lens must be non-NULL");
    return KDA_OK;
}

// Byte offsets of the backward pass's workspace.  The splits' sums (fp32 only) are
// sized for 128 channels and for any number of rows up to these: a tile of 64
// rows is shared by at most 8 workgroups, and all shared tiles by at most 256.
// So a workspace for a large batch also serves a small one, which is split.
struct BackwardSpace {
    size_t pe, part_k, part_q, bytes;
    static size_t split_rows(int64_t rows, int32_t H) { return std::min<size_t>(8 * (size_t)rows * H, 256 * 64); }
    BackwardSpace(int64_t total_q, int64_t total_k, int32_t H, int32_t dr, bool fp32) {
        pe = align256((size_t)total_q * H * 8);
        part_k = pe + align256((size_t)total_k * H * dr * 4);
        part_q = part_k + (fp32 ? align256(split_rows(total_k, H) * (256 + dr) * 4) : 0);
        bytes = part_q + (fp32 ? align256(split_rows(total_q, H) * (128 + dr) * 4) : 0) + 256;
    }
};

}  // namespace

namespace kda {

hipError_t launch_result(hipStream_t stream) {
    const hipError_t e = hipGetLastError();
    return e == hipSuccess && debug_sync() ? hipStreamSynchronize(stream) : e;
}

}  // namespace kda

extern "C" {

kda_status kda_latent_attention(const kda_latent_inputs* in, void* o, float* lse, void* stream) {
    try {
        if (kda_status st = check_inputs(in)) return st;
        if (in->total_q == 0) return KDA_OK;
        if (!o) return fail(KDA_ERR_INVALID_ARGUMENT, "o must be non-NULL");
        if (!aligned16(o) || !aligned16(lse)) return fail(KDA_ERR_INVALID_ARGUMENT, "every pointer must be 16-byte aligned");
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        if (kda_status st = check_offsets(in, s)) return st;
        return launched(kda::launch_latent_attention(*in, o, lse, s), "latent attention kernel");
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_latent_attention");
    }
}

size_t kda_latent_attention_backward_workspace_bytes(int64_t total_q, int64_t total_k, int32_t H, int32_t dr) {
    if (total_q < 0 || total_k < 0 || total_q > kMaxRows || total_k > kMaxRows || H <= 0 || H > 65535 ||
        (dr != 0 && dr != 64))
        return 0;
    return BackwardSpace(total_q, total_k, H, dr, true).bytes;
}

kda_status kda_latent_attention_backward(const kda_latent_inputs* in, const void* o, const float* lse,
                                         const void* d_o, void* dq, void* dk, int64_t dk_token_stride,
                                         int64_t dk_head_stride, void* dv, int64_t dv_token_stride,
                                         int64_t dv_head_stride, void* dk_pe, void* workspace,
                                         size_t workspace_bytes, void* stream_ptr) {
    try {
        if (kda_status st = check_inputs(in)) return st;
        if (in->total_q > 0 && (!o || !lse || !d_o || !dq))
            return fail(KDA_ERR_INVALID_ARGUMENT, "o, lse, d_o and dq must be non-NULL");
        if (in->total_k > 0 && (!dk || !dv || (in->dr && !dk_pe)))
            return fail(KDA_ERR_INVALID_ARGUMENT, "dk, dv (and dk_pe with dr > 0) must be non-NULL");
        const void* ptrs[] = {o, lse, d_o, dq, dk, dv, dk_pe, workspace};
        for (const void* p : ptrs)
            if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARGUMENT, "every pointer must be 16-byte aligned");
        const int64_t strides[] = {dk_token_stride, dk_head_stride, dv_token_stride, dv_head_stride};
        for (int64_t s : strides)
            if (!stride_ok(s, in->dtype))
                return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be >= 0 and multiples of 16 bytes");
        // written rows must not overlap
        if ((in->H > 1 && (dk_head_stride < in->dn || dv_head_stride < in->dv)) ||
            (in->total_k > 1 && (dk_token_stride < in->dn || dv_token_stride < in->dv)))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides of dk and dv must be at least dn and dv");
        if (!workspace && workspace_bytes != 0)
            return fail(KDA_ERR_INVALID_ARGUMENT, "workspace_bytes given without a workspace");
        const BackwardSpace s(in->total_q, in->total_k, in->H, in->dr, in->dtype == KDA_DTYPE_F32);
        const size_t need = s.bytes;
        if (workspace && workspace_bytes < need) {
            kda::set_last_error("workspace too small: need " + std::to_string(need) + " bytes");
            return KDA_ERR_WORKSPACE;
        }
        if (in->total_q == 0 && in->total_k == 0) return KDA_OK;
        hipStream_t stream = reinterpret_cast<hipStream_t>(stream_ptr);
        if (kda_status st = check_offsets(in, stream)) return st;
        unsigned char* ws = static_cast<unsigned char*>(workspace);
        if (!ws)
            if (kda_status st = launched(hipMallocAsync(reinterpret_cast<void**>(&ws), need, stream), "hipMallocAsync"))
                return st;
        kda::LatentGrads g{o, lse, d_o, dq, dk, dk_token_stride, dk_head_stride, dv, dv_token_stride, dv_head_stride,
                           dk_pe, reinterpret_cast<float*>(ws), reinterpret_cast<float*>(ws + s.pe),
                           reinterpret_cast<float*>(ws + s.part_k), reinterpret_cast<float*>(ws + s.part_q)};
        kda_status st = launched(kda::launch_latent_attention_backward(*in, g, stream), "latent backward kernels");
        if (!workspace) {
            const kda_status fr = launched(hipFreeAsync(ws, stream), "hipFreeAsync");
            if (st == KDA_OK) st = fr;
        }
        return st;
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_latent_attention_backward");
    }
}

size_t kda_latent_decode_workspace_bytes(int64_t total_tokens, int32_t num_seqs, int32_t H, int32_t dl, int32_t dr,
                                         kda_dtype dtype) {
    if (total_tokens < 0 || total_tokens > kMaxRows || num_seqs <= 0 || H <= 0 || H > 65535 ||
        (dl != 256 && dl != 512) || (dr != 0 && dr != 64) || !dtype_ok(dtype))
        return 0;
    return align256(kda::latent_decode_workspace(dl));
}

kda_status kda_latent_decode(const void* q, int64_t q_token_stride, int64_t q_head_stride, const void* cache,
                             int32_t num_pages, int32_t page_size, const int32_t* block_table, int32_t max_pages,
                             const int32_t* seq_lens, const int32_t* cu_seqlens, int64_t total_tokens,
                             int32_t num_seqs, int32_t H, int32_t dl, int32_t dr, kda_dtype dtype, float scale,
                             void* o, float* lse, void* workspace, size_t workspace_bytes, void* stream_ptr) {
    try {
        if (!dtype_ok(dtype)) return fail(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_DTYPE_F32 or KDA_DTYPE_BF16");
        if (kda_status st = check_pages(cache, num_pages, page_size, block_table, max_pages, seq_lens, cu_seqlens,
                                        total_tokens, num_seqs))
            return st;
        if (H <= 0 || H > 65535) return fail(KDA_ERR_INVALID_ARGUMENT, "H must be in [1, 65535]");
        if (total_tokens * H > kMaxRows)   // a sequence's row tiles are counted in 32 bits
            return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens * H must be <= 2^31 - 4096");
        if ((dl != 256 && dl != 512) || (dr != 0 && dr != 64))
            return fail(KDA_ERR_UNSUPPORTED, "dl must be 256 or 512, dr 0 or 64");
        if (!(scale > 0.f) || !std::isfinite(scale)) return fail(KDA_ERR_INVALID_ARGUMENT, "scale must be finite and > 0");
        if (total_tokens > 0 && (!q || !o)) return fail(KDA_ERR_INVALID_ARGUMENT, "q and o must be non-NULL");
        const void* ptrs[] = {q, cache, o, lse, workspace};
        for (const void* p : ptrs)
            if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARGUMENT, "every pointer must be 16-byte aligned");
        if (!stride_ok(q_token_stride, dtype) || !stride_ok(q_head_stride, dtype))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be >= 0 and multiples of 16 bytes");
        if (!workspace && workspace_bytes != 0)
            return fail(KDA_ERR_INVALID_ARGUMENT, "workspace_bytes given without a workspace");
        const size_t need = kda_latent_decode_workspace_bytes(total_tokens, num_seqs, H, dl, dr, dtype);
        if (workspace && workspace_bytes < need) {
            kda::set_last_error("workspace too small: need " + std::to_string(need) + " bytes");
            return KDA_ERR_WORKSPACE;
        }
        if (total_tokens == 0) return KDA_OK;
        hipStream_t stream = reinterpret_cast<hipStream_t>(stream_ptr);
        if (kda_status st = kda::debug_check_offsets(cu_seqlens, num_seqs, total_tokens, false, stream)) return st;
        void* ws = workspace;
        if (!ws)
            if (kda_status st = launched(hipMallocAsync(&ws, need, stream), "hipMallocAsync")) return st;
        const kda::LatentDecode a{q, q_token_stride, q_head_stride, cache, num_pages, page_size, block_table,
                                  max_pages, seq_lens, cu_seqlens, total_tokens, num_seqs, H, dl, dr, scale, o, lse, ws};
        kda_status st = launched(kda::launch_latent_decode(a, dtype == KDA_DTYPE_BF16, stream), "latent decode kernels");
        if (!workspace) {
            const kda_status fr = launched(hipFreeAsync(ws, stream), "hipFreeAsync");
            if (st == KDA_OK) st = fr;
        }
        return st;
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_latent_decode");
    }
}

kda_status kda_latent_append(void* cache, int32_t num_pages, int32_t page_size, const int32_t* block_table,
                             int32_t max_pages, const int32_t* seq_lens, const int32_t* cu_seqlens,
                             int64_t total_tokens, int32_t num_seqs, int32_t dl, int32_t dr, kda_dtype dtype,
                             const void* c, int64_t c_token_stride, const void* k_pe, int64_t k_pe_token_stride,
                             const float* norm_weight, float eps, const float* inv_freq, float amplitude,
                             uint32_t flags, void* c_out, void* k_pe_out, void* stream) {
    try {
        if (!dtype_ok(dtype)) return fail(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_DTYPE_F32 or KDA_DTYPE_BF16");
        if (flags & ~(uint32_t)KDA_ROTARY_INTERLEAVED) return fail(KDA_ERR_INVALID_ARGUMENT, "unknown flag bits");
        if (kda_status st = check_pages(cache, num_pages, page_size, block_table, max_pages, seq_lens, cu_seqlens,
                                        total_tokens, num_seqs))
            return st;
        if (dl <= 0 || dl % 64 != 0 || dl > 1024)
            return fail(KDA_ERR_UNSUPPORTED, "dl must be a multiple of 64 up to 1024");
        if (dr < 0 || dr > 256 || dr * elem_size(dtype) % 16 != 0)
            return fail(KDA_ERR_UNSUPPORTED, "dr must be a multiple of 16 bytes up to 256");
        if (total_tokens > 0 && (!c || (dr > 0 && !k_pe)))
            return fail(KDA_ERR_INVALID_ARGUMENT, "c (and k_pe with dr > 0) must be non-NULL");
        if (dr == 0 && (k_pe_out || inv_freq))
            return fail(KDA_ERR_INVALID_ARGUMENT, "k_pe_out and inv_freq need dr > 0");
        if (!(eps >= 0.f) || !std::isfinite(eps)) return fail(KDA_ERR_INVALID_ARGUMENT, "eps must be finite and >= 0");
        if (!std::isfinite(amplitude)) return fail(KDA_ERR_INVALID_ARGUMENT, "amplitude must be finite");
        const void* ptrs[] = {cache, c, k_pe, norm_weight, c_out, k_pe_out};
        for (const void* p : ptrs)
            if (!aligned16(p)) return fail(KDA_ERR_INVALID_ARGUMENT, "every pointer must be 16-byte aligned");
        if (!stride_ok(c_token_stride, dtype) || !stride_ok(k_pe_token_stride, dtype))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be >= 0 and multiples of 16 bytes");
        if (total_tokens == 0) return KDA_OK;
        hipStream_t s = reinterpret_cast<hipStream_t>(stream);
        if (kda_status st = kda::debug_check_offsets(cu_seqlens, num_seqs, total_tokens, false, s)) return st;
        const kda::LatentAppend a{cache, num_pages, page_size, block_table, max_pages, seq_lens, cu_seqlens,
                                  total_tokens, num_seqs, dl, dr, c, c_token_stride, k_pe, k_pe_token_stride,
                                  norm_weight, eps, inv_freq, amplitude, flags, c_out, k_pe_out};
        return launched(kda::launch_latent_append(a, dtype == KDA_DTYPE_BF16, s), "latent append kernel");
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_latent_append");
    }
}

kda_status kda_rotary(const void* x, int64_t x_token_stride, int64_t x_head_stride, void* y, int64_t y_token_stride,
                      int64_t y_head_stride, const int32_t* positions, const float* inv_freq, int64_t total_tokens,
                      int32_t H, int32_t d, int32_t start, int32_t dr, kda_dtype dtype, float amplitude,
                      uint32_t flags, void* stream) {
    try {
        if (!dtype_ok(dtype)) return fail(KDA_ERR_INVALID_ARGUMENT, "dtype must be KDA_DTYPE_F32 or KDA_DTYPE_BF16");
        if (flags & ~(uint32_t)(KDA_ROTARY_INTERLEAVED | KDA_ROTARY_INVERSE))
            return fail(KDA_ERR_INVALID_ARGUMENT, "unknown flag bits");
        if (H <= 0 || H > 65535) return fail(KDA_ERR_INVALID_ARGUMENT, "H must be in [1, 65535]");
        if (total_tokens < 0 || total_tokens > kMaxRows)
            return fail(KDA_ERR_INVALID_ARGUMENT, "total_tokens must be in [0, 2^31 - 4096]");
        if (d <= 0 || d > 4096) return fail(KDA_ERR_UNSUPPORTED, "d must be in [1, 4096]");
        if (dr < 2 || dr % 2 != 0 || start < 0 || start > d || dr > d - start)
            return fail(KDA_ERR_INVALID_ARGUMENT, "dr must be even and >= 2, with 0 <= start and start + dr <= d");
        if (!std::isfinite(amplitude)) return fail(KDA_ERR_INVALID_ARGUMENT, "amplitude must be finite");
        if (total_tokens > 0 && (!x || !y || !positions || !inv_freq))
            return fail(KDA_ERR_INVALID_ARGUMENT, "x, y, positions and inv_freq must be non-NULL");
        const uintptr_t unit = dtype == KDA_DTYPE_BF16 ? 1 : 3;
        if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & unit)
            return fail(KDA_ERR_INVALID_ARGUMENT, "x and y must be aligned to one element");
        const int64_t strides[] = {x_token_stride, x_head_stride, y_token_stride, y_head_stride};
        for (int64_t s : strides)
            if (s < 0 || s >= ((int64_t)1 << 40)) return fail(KDA_ERR_INVALID_ARGUMENT, "strides must be in [0, 2^40)");
        if ((H > 1 && y_head_stride < d) || (total_tokens > 1 && y_token_stride < d))
            return fail(KDA_ERR_INVALID_ARGUMENT, "strides of y must be at least d");
        if (total_tokens == 0) return KDA_OK;
        if (x == y && ((total_tokens > 1 && x_token_stride != y_token_stride) || (H > 1 && x_head_stride != y_head_stride)))
            return fail(KDA_ERR_INVALID_ARGUMENT, "in place, x and y must have the same strides");
        const kda::Rotary a{x, x_token_stride, x_head_stride, y, y_token_stride, y_head_stride, positions, inv_freq,
                            total_tokens, H, d, start, dr, amplitude, flags};
        return launched(kda::launch_rotary(a, dtype == KDA_DTYPE_BF16, reinterpret_cast<hipStream_t>(stream)),
                        "rotary kernel");
    } catch (...) {
        return fail(KDA_ERR_HIP, "unexpected C++ exception inside kda_rotary");
    }
}

kda_status kda_rotary_frequencies(int32_t dr, double base, double factor, int64_t original_context, float* inv_freq,
                                  float* amplitude) {
    if (dr < 2 || dr % 2 != 0 || dr > 4096) return fail(KDA_ERR_INVALID_ARGUMENT, "dr must be even and in [2, 4096]");
    if (!(base > 1.0) || !std::isfinite(base)) return fail(KDA_ERR_INVALID_ARGUMENT, "base must be finite and > 1");
    if (!(factor >= 1.0) || !std::isfinite(factor)) return fail(KDA_ERR_INVALID_ARGUMENT, "factor must be finite and >= 1");
    if (original_context < 0) return fail(KDA_ERR_INVALID_ARGUMENT, "original_context must be >= 0");
    if (!inv_freq) return fail(KDA_ERR_INVALID_ARGUMENT, "inv_freq must be non-NULL");
    const bool by_parts = original_context > 0;
    for (int32_t i = 0; i < dr / 2; ++i) {
        const double f = std::pow(base, -2.0 * i / dr);
        double keep = factor > 1.0 ? 0.0 : 1.0;   // share of the unscaled frequency
        if (by_parts) {
            const double turns = (double)original_context * f / (2.0 * 3.14159265358979323846);
            const double x = (turns - 1.0) / (32.0 - 1.0);
            keep = x < 0.0 ? 0.0 : x > 1.0 ? 1.0 : x;
        }
        inv_freq[i] = (float)(f * keep + f / factor * (1.0 - keep));
    }
    if (amplitude) *amplitude = by_parts && factor > 1.0 ? (float)(0.1 * std::log(factor) + 1.0) : 1.f;
    return KDA_OK;
}

}  // extern "C"
