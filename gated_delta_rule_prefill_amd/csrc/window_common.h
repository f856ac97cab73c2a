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

// Tile t of the keys (rows `stride` elements apart from base, the sequence's first)
// into registers: sinks, then the run behind them, zeros behind the last key.  An
// offset within the tile fits in 32 bits, as strides are below 2^23.
template <typename S, typename E>
__device__ __forceinline__ void load_keys(S& st, int tid, const KeyRange& kr, int n0, const E* base, int64_t stride) {
    const E *sinks = base + n0 * stride, *run = base + ((int64_t)n0 + kr.shift) * stride;
    const int left = kr.total - n0, split = kr.ns - n0;
#pragma unroll
    for (int p = 0; p < S::P; ++p) {
        const int r = tid / S::TPR + S::PASS * p;
        const uint32_t at = (uint32_t)min(r, left - 1) * (uint32_t)(stride * sizeof(E)) + 16 * (tid % S::TPR);
        const char* row = reinterpret_cast<const char*>(min(r, left - 1) < split ? sinks : run);
#pragma unroll
        for (int s = 0; s < S::S; ++s) {
            st.r[p][s] = *reinterpret_cast<const u32x4*>(row + at + 16 * S::TPR * s);
            if (r >= left) st.r[p][s] = u32x4{0, 0, 0, 0};
        }
    }
}

// Cached tokens of a sequence.
__device__ __forceinline__ int cached_tokens(const kda_kv_cache& c, int seq) {
    return (int)max((int64_t)0, min((int64_t)c.seq_lens[seq], (int64_t)c.max_pages * c.page_size));
}
// Offset of position j of a sequence from the cache's k and v (head 0), or -1
// where its page is absent.
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
