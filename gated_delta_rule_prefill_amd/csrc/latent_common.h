// latent_common.h -- device helpers of the latent-attention kernels: tiles in
// LDS, their matrix operands, and the search for a workgroup's sequence.
#pragma once

#include "kda_common.h"
#include "latent_launch.h"

namespace kda {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// -- row-major tiles in LDS ------------------------------------------------------
// W elements per row, in 16-byte chunks; chunk c of row r is stored at chunk
// position c ^ swizzle(r).  The swizzle takes 8 values over 8 consecutive rows
// (operands read by rows: 16 rows at one chunk column) and 4 different pairs
// over 4 consecutive rows (operands read by columns: two neighbouring chunks
// of 4 rows), so both kinds of read spread over the banks.
template <typename E> constexpr int CHUNK_ELEMS = 16 / (int)sizeof(E);
__device__ __forceinline__ int swizzle(int r) { return ((r & 3) << 1) | ((r >> 2) & 1); }

template <typename E, int W>
__device__ __forceinline__ int tile_at(int row, int chunk) {
    return row * W + ((chunk ^ swizzle(row)) * CHUNK_ELEMS<E>);
}

// Operand by rows: lane l supplies row row0 + (l & 15), slots 8g .. 8g + 7 of
// the 32-wide block ks (g = l >> 4).
template <int W>
__device__ __forceinline__ bf16x8 row_frag(const bf16* t, int row0, int ks, int lane) {
    return *reinterpret_cast<const bf16x8*>(t + tile_at<bf16, W>(row0 + (lane & 15), 4 * ks + (lane >> 4)));
}
template <int W>
__device__ __forceinline__ f32x8 row_frag(const float* t, int row0, int ks, int lane) {
    const int r = row0 + (lane & 15), c = 8 * ks + 2 * (lane >> 4);
    const f32x4 a = *reinterpret_cast<const f32x4*>(t + tile_at<float, W>(r, c));
    const f32x4 b = *reinterpret_cast<const f32x4*>(t + tile_at<float, W>(r, c + 1));
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Operand by columns: lane l supplies column c0 + (l & 15), slots 0..3 from
// rows ra + 4g .. +3 and slots 4..7 from rows rb + 4g .. +3.  The rows 4g + i
// of two 16-row blocks are what an accumulator tile leaves in lane group g, so
// the other operand of the product stays in registers.  (bf16: the transposing
// LDS read, a lane group's 16 lanes fetching 4 rows of 16 columns.)
template <int W>
__device__ __forceinline__ bf16x8 col_frag(const bf16* t, int ra, int rb, int c0, int lane) {
    typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
    const int r = 4 * (lane >> 4) + ((lane & 15) >> 2), c = c0 + 4 * (lane & 3);
    const bf16* pa = t + tile_at<bf16, W>(ra + r, c >> 3) + (c & 4);
    const bf16* pb = t + tile_at<bf16, W>(rb + r, c >> 3) + (c & 4);
    const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)pa);
    const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)pb);
    typedef short s16x8 __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
}
template <int W>
__device__ __forceinline__ f32x8 col_frag(const float* t, int ra, int rb, int c0, int lane) {
    const int g4 = 4 * (lane >> 4), c = c0 + (lane & 15);
    f32x8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[i] = t[tile_at<float, W>(ra + g4 + i, c >> 2) + (c & 3)];
        v[4 + i] = t[tile_at<float, W>(rb + g4 + i, c >> 2) + (c & 3)];
    }
    return v;
}

// Two accumulator tiles (rows 4g + i of two 16-row blocks) as the 8 slots of
// an operand.  To bf16 each value is rounded to nearest: the products take
// bf16 operands, and a relative error of at most 2^-9 per weight is that of
// the inputs themselves.
__device__ __forceinline__ bf16x8 acc_frag(f32x4 a, f32x4 b, bf16) {
    return bf16x8{(bf16)a[0], (bf16)a[1], (bf16)a[2], (bf16)a[3], (bf16)b[0], (bf16)b[1], (bf16)b[2], (bf16)b[3]};
}
__device__ __forceinline__ f32x8 acc_frag(f32x4 a, f32x4 b, float) {
    return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
}

// Operand by rows straight from global memory (rows kept in registers).
__device__ __forceinline__ bf16x8 row_frag_global(const bf16* row, int ks, int lane) {
    return *reinterpret_cast<const bf16x8*>(row + 32 * ks + 8 * (lane >> 4));
}
__device__ __forceinline__ f32x8 row_frag_global(const float* row, int ks, int lane) {
    return load_vec<f32x8, float>(row + 32 * ks + 8 * (lane >> 4));
}

// -- staging: global -> registers -> LDS ---------------------------------------
// ROWS x W elements moved by NT threads; src(row, chunk) returns the chunk's
// address, or NULL for zeros.  The loads are issued by load() and waited for
// by store(), a tile of work later.
template <typename E, int W, int ROWS, int NT>
struct Stage {
    static constexpr int CPR = W / CHUNK_ELEMS<E>, N = ROWS * CPR / NT;
    static_assert(ROWS * CPR % NT == 0 && CPR % 8 == 0, "whole chunks per thread, 8 per swizzle group");
    u32x4 r[N];
    template <typename F>
    __device__ __forceinline__ void load(int tid, F src) {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int id = tid + NT * k;
            const E* p = src(id / CPR, id % CPR);
            r[k] = p ? *reinterpret_cast<const u32x4*>(p) : u32x4{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ void store(int tid, E* t) const {
#pragma unroll
        for (int k = 0; k < N; ++k) {
            const int id = tid + NT * k;
            *reinterpret_cast<u32x4*>(t + tile_at<E, W>(id / CPR, id % CPR)) = r[k];
        }
    }
};

// -- a workgroup's tile of a packed batch ----------------------------------------
__device__ __forceinline__ int clamp_offset(int x, int total) { return min(max(x, 0), total); }

// Rows [a, b) of sequence s.
__device__ __forceinline__ void sequence_rows(const int32_t* cu, int rows, int total, int s, int& a, int& b) {
    if (cu) {
        a = clamp_offset(cu[s], total);
        b = max(a, clamp_offset(cu[s + 1], total));
    } else {
        a = s * rows;
        b = a + rows;
    }
}

// Sequence and tile within it of the batch's tile number `want` (tiles of B
// rows, counted through the sequences in order); false behind the last tile.
// Packed batches: one pass over the offsets, NT of them at a time (a scan per
// wave, the waves' sums through scratch).  Called by all NT threads.
template <int B, int NT>
__device__ __forceinline__ bool find_tile(const int32_t* cu, int N, int rows, int total, int want,
                                          int* scratch /* [NT / 64 + 2] in LDS */, int& seq, int& tile) {
    if (!cu) {
        const int per = (rows + B - 1) / B;
        if (per == 0 || want >= per * N) return false;
        seq = want / per;
        tile = want - seq * per;
        return true;
    }
    constexpr int NW = NT / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int before = 0;
    for (int base = 0; base < N; base += NT) {
        const int s = base + tid;
        int n = 0;
        if (s < N) {
            int a, b;
            sequence_rows(cu, rows, total, s, a, b);
            n = (b - a + B - 1) / B;
        }
        int incl = n;
#pragma unroll
        for (int d = 1; d < 64; d <<= 1) {
            const int up = __shfl_up(incl, d);
            if (lane >= d) incl += up;
        }
        if (lane == 63) scratch[wave] = incl;
        if (tid == 0) scratch[NW] = -1;
        __syncthreads();
        int excl = before + incl - n, all = before;
#pragma unroll
        for (int w = 0; w < NW; ++w) {
            if (w < wave) excl += scratch[w];
            all += scratch[w];
        }
        if (want >= excl && want < excl + n) {
            scratch[NW] = s;
            scratch[NW + 1] = want - excl;
        }
        __syncthreads();
        seq = scratch[NW];
        tile = scratch[NW + 1];
        __syncthreads();
        if (seq >= 0) return true;
        before = all;
    }
    return false;
}

// Workgroup -> (head, tile): the heads go round robin over the 8 XCDs (as the
// workgroups do), and an XCD takes one head's tiles after another's, so that
// the workgroups running on it read the same keys through its L2.
__device__ __forceinline__ void head_tile_of_block(int H, int tiles, int& h, int& tile) {
    const int L = blockIdx.x;
    if ((H & 7) == 0) {
        const int j = L >> 3;
        h = (L & 7) + 8 * (j / tiles);
        tile = j % tiles;
    } else {
        h = L / tiles;
        tile = L % tiles;
    }
}

// max and sum over the lanes that share l & 15 (the 4 lane groups)
__device__ __forceinline__ float group_max(float x) {
    x = fmaxf(x, lane_xor<16>(x));
    return fmaxf(x, lane_xor<32>(x));
}
__device__ __forceinline__ float group_sum(float x) {
    x += lane_xor<16>(x);
    return x + lane_xor<32>(x);
}

}  // namespace kda
