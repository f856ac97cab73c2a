// window_common.h -- device helpers of the window-attention kernels: which keys a
// tile of query rows sees, and where they lie.
//
// The query heads that share a key head are rows beside each other: row r of a
// (sequence, key head) is query head r % G of token r / G, G = H / Hk.  A tile of
// rows is then few tokens wide, and the keys that only some of its rows see, at
// both ends of the window, are few: with 128 rows, G = 4 and a window of 128 the
// walk is 159 keys long where 128 tokens of one head would take 255.
#pragma once

#include "latent_common.h"
#include "window_launch.h"

namespace kda {

// The keys of a tile of rows, tokens i0 to i1 of a sequence with nk keys whose
// query i stands at position i + off: the first ns (sinks) and a run up to the
// last one's own position, numbered through without the gap between them.  Key
// number n is position n < ns ? n : n + shift; a row at position p sees number
// n <= p - shift with n < ns or n >= p - W + 1 - shift.  (shift is 0 where there is
// no gap, and positive only where every row stands behind the sinks.)
struct KeyRange {
    int W, ns, shift, total;
    int last_min, first_max;   // all rows see the numbers up to last_min that are sinks or not below first_max
    __device__ __forceinline__ KeyRange(int i0, int i1, int off, int window, int sinks, int nk) {
        W = min(window, nk);
        const int end = max(0, min(nk, i1 + off + 1));
        ns = min(sinks, end);
        shift = max(0, i0 + off - W + 1 - ns);
        total = max(0, end - shift);
        last_min = i0 + off - shift;
        first_max = i1 + off - W + 1 - shift;
    }
    // Of a row at position p: the last key number it sees, and the first behind the sinks.
    __device__ __forceinline__ int last(int p) const { return p - shift; }
    __device__ __forceinline__ int first(int p) const { return p - W + 1 - shift; }
    __device__ __forceinline__ int position(int n) const { return n < ns ? n : n + shift; }
    // Whether the row whose first key number is `first` does not see number n: one
    // comparison for the window, where there are no sinks (some: n may be one).
    __device__ __forceinline__ bool hides(int n, int first, bool some) const {
        const bool outside = (unsigned)(n - first) >= (unsigned)W;
        return some ? outside && (n >= ns || n > first + W - 1) : outside;
    }
    // The tiles [a, b) of n keys that all rows see whole and whose keys lie in one run.
    __device__ __forceinline__ void whole_tiles(int n, int& a, int& b) const {
        a = shift == 0 && first_max <= ns ? 0 : (max(first_max, ns) + n - 1) / n;
        b = (last_min + 1) / n;
    }
    // Whether rows between these two see all of the numbers [a, b).
    __device__ __forceinline__ bool whole(int a, int b, int last_of_first, int first_of_last) const {
        return b - 1 <= last_of_first && (a >= first_of_last || b <= ns);
    }
};

// Tiles of rows from global memory straight into LDS, as Direct (every wave writes 1
// KB of the tile in a row, its lanes fetch the chunks that belong there), also where some of
// a tile's rows are not there (`left` of them are; the last one is repeated behind)
// or do not follow on the others (the first `split` rows lie where `first` says).
// The loads are buffer loads: behind loads of the global kind the compiler waits for
// every LDS read in flight before it uses one, as if they came back out of order.
template <typename E, int W, int ROWS, int NT>
struct Tiles {
    static constexpr int CE = CHUNK_ELEMS<E>, CH = W / CE, N = ROWS * CH / NT, STEP = NT / CH;
    static_assert(ROWS * CH % NT == 0 && 64 % CH == 0 && STEP % 8 == 0, "whole rows in a wave, chunks in place from step to step");
    int row0;          // the row of this thread's chunk i is row0 + i STEP
    uint32_t stride;   // in bytes
    uint32_t at;       // of chunk 0 from the tile's base
    __device__ __forceinline__ Tiles(int tid, int64_t stride_) : row0(tid / CH), stride((uint32_t)(stride_ * sizeof(E))) {
        at = row0 * stride + 16u * ((tile_at<E, W>(row0, tid % CH) - row0 * W) / CE);
    }
    __device__ __forceinline__ int row(int i) const { return row0 + i * STEP; }
    // 16 bytes a lane from `at` bytes behind the wave's base to 1 KB of LDS.
    static __device__ __forceinline__ void fetch_chunks(const E* base, uint32_t at, uint32_t more, E* to) {
#ifdef __HIP_DEVICE_COMPILE__   // the host compiler does not know the type of a buffer
        typedef __attribute__((address_space(3))) void lds_void;
        __builtin_amdgcn_raw_ptr_buffer_load_lds(__builtin_amdgcn_make_buffer_rsrc(const_cast<E*>(base), 0, -1, 0x00020000),
                                                 (lds_void*)to, 16, at, more, 0, 0);   // raw: an offset of 32 bits
#endif
    }
    __device__ __forceinline__ void fetch(int wave, const E* base, E* t) const {
#pragma unroll
        for (int i = 0; i < N; ++i) fetch_chunks(base, at, i * STEP * stride, t + (i * NT + 64 * wave) * CE);
    }
    __device__ __forceinline__ void fetch_part(int wave, const E* base, const E* first, int split, int left, E* t) const {
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int there = min(row(i), left - 1);
            const uint32_t x = at + (uint32_t)(there - row0) * stride;
            E* to = t + (i * NT + 64 * wave) * CE;
            if (there >= split) fetch_chunks(base, x, 0, to);
            else fetch_chunks(first, x, 0, to);
        }
    }
    // Rows in any order, row(r) being the address of row r (strides are 0).
    template <typename F>
    __device__ __forceinline__ void fetch_rows(int wave, F row_at, E* t) const {
        typedef __attribute__((address_space(1))) const void global_void;
        typedef __attribute__((address_space(3))) void lds_void;
#pragma unroll
        for (int i = 0; i < N; ++i)
            __builtin_amdgcn_global_load_lds((global_void*)(reinterpret_cast<const char*>(row_at(row(i))) + at),
                                             (lds_void*)(t + (i * NT + 64 * wave) * CE), 16, 0, 0);
    }
    // Whether chunk i of a fetched tile in LDS, which this thread has fetched, belongs
    // to a row with values that are not finite.
    __device__ __forceinline__ bool bad_row(int tid, const E* t, int i) const {
        const u32x4 x = *reinterpret_cast<const u32x4*>(t + (i * NT + tid) * CE);
        bool bad = false;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            bad |= (x[e] & 0x7f800000u) == 0x7f800000u;
            if (sizeof(E) == 2) bad |= (x[e] & 0x7f80u) == 0x7f80u;
        }
        const unsigned long long any = __ballot(bad);
        return (any >> (tid & 63 & ~(CH - 1)) & (CH == 64 ? ~0ull : (1ull << CH) - 1)) != 0;
    }
    // Such rows of the tile `product` cleared, and those of `weights` set to NaN (see move_bad_rows).
    __device__ __forceinline__ void move_bad(int tid, E* product, E* weights) const {
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (bad_row(tid, product, i)) {
                *reinterpret_cast<u32x4*>(product + (i * NT + tid) * CE) = u32x4{0, 0, 0, 0};
                *reinterpret_cast<u32x4*>(weights + (i * NT + tid) * CE) = u32x4{QUIET, QUIET, QUIET, QUIET};
            }
    }
};

// Operands by columns of RT row tiles (RT 1: fp32, whose slots 4 to 7 stay empty), and
// their products.
template <int RT, typename Reader, typename E>
__device__ __forceinline__ auto cols(const Reader& read, const E* t, int row0, int ct) {
    if constexpr (RT == 2) return read(t, row0, row0 + 16, ct);
    else return read.half(t, row0, ct);
}
template <int RT, typename V>
__device__ __forceinline__ f32x4 mma_rows(const V& a, const V& b, f32x4 c) {
    if constexpr (RT == 2) {
        return mma32(a, b, c);
    } else {
#pragma unroll
        for (int m = 0; m < 4; ++m) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[m], b[m], c, 0, 0, 0);
        return c;
    }
}

// The sums of four waves, each of 16 rows (lane & 15) and D channels as accumulator
// tiles, added up in order: wave w is left with channel tiles [w D/64, (w + 1) D/64) in
// the first D/64 of acc.  lds: 64 D floats that no wave reads any more.
template <typename E, int D>
__device__ __forceinline__ void join_waves(E* lds, int wave, int col, int g, f32x4 (&acc)[D / 16]) {
    auto at = [&](int w, int c) { return reinterpret_cast<f32x4*>(lds) + (w * 16 + col) * (D / 4) + ((4 * c + g) ^ col); };
#pragma unroll
    for (int c = 0; c < D / 16; ++c) *at(wave, c) = acc[c];
    __syncthreads();
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        acc[c] = *at(0, wave * (D / 64) + c);
#pragma unroll
        for (int w = 1; w < 4; ++w) acc[c] += *at(w, wave * (D / 64) + c);
    }
}

// Query rows of a workgroup of the forward and dq kernels, and the batch's tiles of
// so many.
template <typename E, bool SPLIT> constexpr int WINDOW_ROWS = SPLIT ? 16 : 64 * LATENT_NQ<E>;
static inline int64_t row_tiles(const kda_window_inputs& in, int rows) {
    const int64_t G = in.H / in.Hk;
    return in.cu_seqlens_q ? in.total_q * G / rows + in.num_seqs : (in.total_q / in.num_seqs * G + rows - 1) / rows * in.num_seqs;
}
// Whether a workgroup's waves share 16 rows and split their keys rather than own rows
// each.  The split form has a walk of a quarter of the length and four times (bf16:
// eight times) the workgroups; it is taken as long as all of them run at once (128 KB of
// LDS each with d = 128, 64 KB with 64).  us, split against whole:
//   fp32, forward   d 128, 495 tokens x 4 heads, window 100    13 and 22
//                   d 64 (128), 1,024 tokens x 8, window 256   16.6 and 20.1 (36 and 32)
//   bf16, forward   d 128, 1,000 tokens x 4 on 1 key head, window 1,024 (128)   17 and 29 (13 and 15)
//   bf16, dq        the same                                                    18 and 41 (14 and 19)
// Where it takes more rounds it loses: fp32, d 128, 2,048 tokens x 8 70 and 35; bf16,
// 2,000 tokens x 8 on 2, window 1,024, 61 and 33, d 64 25 and 25.
static inline bool split_waves(const kda_window_inputs& in) {
    return row_tiles(in, 64) * in.Hk * 4 <= 256 * (128 / in.d);
}

// Cached tokens of a sequence.
__device__ __forceinline__ int cached_tokens(const kda_kv_cache& c, int seq) {
    return (int)max((int64_t)0, min((int64_t)c.seq_lens[seq], (int64_t)c.max_pages * c.page_size));
}
// The page and the row in it of key number n of a range, or row -1 behind its last.
// The page is loaded without a branch and looked at only when the row's offset from the
// cache's k and v (head 0; -1 where it is absent) is asked for, which lets a loop look
// rows up ahead: a wait for a page is one for all loads before it.
struct CachedRow {
    int page = 0, row = -1;
    __device__ __forceinline__ CachedRow() {}
    __device__ __forceinline__ CachedRow(const kda_kv_cache& c, int seq, const KeyRange& kr, int n, bool there = true) {
        const int j = kr.total > 0 ? kr.position(min(n, kr.total - 1)) : 0;
        const int pg = (int)((unsigned)j / (unsigned)c.page_size);
        page = c.block_table[(int64_t)seq * c.max_pages + pg];
        row = there && n < kr.total ? j - pg * c.page_size : -1;
    }
    __device__ __forceinline__ int64_t offset(const kda_kv_cache& c) const {
        return row >= 0 && page >= 0 && page < c.num_pages ? page * c.page_stride + row * c.token_stride : -1;
    }
};
// Offset of position j of a sequence, or -1 where its page is absent.
__device__ __forceinline__ int64_t cached_row(const kda_kv_cache& c, int seq, int j) {
    const int pg = (int)((unsigned)j / (unsigned)c.page_size);
    const int page = c.block_table[(int64_t)seq * c.max_pages + pg];
    if (page < 0 || page >= c.num_pages) return -1;
    return page * c.page_stride + (j - pg * c.page_size) * c.token_stride;
}

// Workgroup -> (key head, tile).  With a multiple of 8 heads as head_tile_of_block;
// otherwise the heads take turns, so that an XCD's workgroups share few of them
// where their number divides 8.
__device__ __forceinline__ void key_head_of_block(int Hk, int tiles, int L, int& h, int& tile) {
    if ((Hk & 7) == 0) {
        const int j = L >> 3;
        h = (L & 7) + 8 * (j / tiles);
        tile = j % tiles;
    } else {
        h = L % Hk;
        tile = L / Hk;
    }
}

}  // namespace kda
