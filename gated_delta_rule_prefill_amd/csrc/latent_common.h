// latent_common.h -- device helpers of the latent-attention kernels: tiles in
// LDS, their matrix operands, and the search for a workgroup's sequence.
#pragma once

#include <type_traits>
#include <utility>

#include "kda_common.h"
#include "latent_launch.h"

namespace kda {

typedef unsigned u32x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

// Query rows of a wave in 16-row tiles (forward, dq).  bf16: two tiles, so that an operand read from LDS serves two
// products.  fp32: one; its products take sixteen times as long, LDS is no bound,
// and the smaller tiles spread a short batch over more CUs (130 tokens x 4
// heads: 22 us with two tiles).
template <typename E> constexpr int LATENT_NQ = sizeof(E) == 2 ? 2 : 1;

constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }
// A value that is the same in every lane, held in scalar registers.
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int64_t uniform(int64_t x) {
    return (int64_t)(((uint64_t)(uint32_t)uniform((int)(x >> 32)) << 32) | (uint32_t)uniform((int)x));
}
__device__ __forceinline__ float neg_inf() { return -__builtin_inff(); }

// -- row-major tiles in LDS ------------------------------------------------------
// W elements per row, in 16-byte chunks; chunk c of row r is stored at chunk
// position c ^ swizzle(r).  LDS serves 256 bytes (64 banks) a cycle, 16 lanes of
// 16 bytes; a read by rows is served 8 rows of one chunk column together with
// the 8 other rows of its neighbour, a read by columns 8 rows of one column
// pair.  Both are free of conflicts (counted: 4 and 2 cycles an instruction)
// when 8 neighbouring rows lie at 8 different pairs of positions in 256 bytes.
// A row of an odd number of 128 bytes alternates between the halves by itself,
// and the swizzle permutes groups of 8 chunks; a row of whole 256 bytes takes
// the half from the row's lowest bit, and the swizzle permutes groups of 16.
template <typename E> constexpr int CHUNK_ELEMS = 16 / (int)sizeof(E);
template <typename E, int W> constexpr bool WHOLE_ROWS = W * (int)sizeof(E) % 256 == 0;

template <typename E, int W>
__device__ __forceinline__ int tile_at(int row, int chunk) {
    static_assert(W * sizeof(E) % 128 == 0, "rows of whole 128 bytes");
    int f = ((row >> 1) & 3) << 1;
    if (WHOLE_ROWS<E, W>) f |= (row & 1) << 3;
    return row * W + ((chunk ^ f) * CHUNK_ELEMS<E>);
}

// Element at chunk c + c1 of the row whose chunk c is at `at`, for a constant c1
// that is a multiple of 8 and a c below 8.
template <typename E, int W>
__device__ __forceinline__ int later_chunk(int at, int c1) {
    constexpr int CE = CHUNK_ELEMS<E>;
    return WHOLE_ROWS<E, W> ? (at ^ ((c1 & 8) * CE)) + (c1 & ~15) * CE : at + c1 * CE;
}

// Operands by rows of a tile: lane l supplies row row0 + (l & 15), slots
// 8g .. 8g + 7 of the 32-wide block ks (g = l >> 4).  A lane's addresses come
// from two bases and constants; row0 is a multiple of 16.
// keep() in a loop's body makes the compiler derive the addresses there again
// rather than hold all of them in registers, which the largest kernels lack: an
// operand that is spilled costs far more than its read, as the wait for it also
// waits for the next tile's loads (dq 2.36 ms with three spilled operands in the
// loop, 1.67 without).
template <typename E, int W> struct RowReader;
template <int W> struct RowReader<bf16, W> {
    int at;   // in bytes
    __device__ __forceinline__ explicit RowReader(int lane) : at(2 * tile_at<bf16, W>(lane & 15, lane >> 4)) {}
    __device__ __forceinline__ void keep() { asm volatile("" : "+v"(at)); }
    __device__ __forceinline__ bf16x8 operator()(const bf16* t, int row0, int ks) const {
        constexpr int HALF = WHOLE_ROWS<bf16, W> ? 128 : 0;
        const int flip = 64 * (ks & 1) + (HALF && (ks >> 1 & 1) ? 128 : 0);
        const int on = HALF ? 256 * (ks >> 2) : 128 * (ks >> 1);
        return *reinterpret_cast<const bf16x8*>(reinterpret_cast<const char*>(t) + (at ^ flip) + on + 2 * row0 * W);
    }
};
template <int W> struct RowReader<float, W> {
    int at[2];
    __device__ __forceinline__ explicit RowReader(int lane) {
        at[0] = tile_at<float, W>(lane & 15, 2 * (lane >> 4));
        at[1] = tile_at<float, W>(lane & 15, 2 * (lane >> 4) + 1);
    }
    __device__ __forceinline__ void keep() {}
    __device__ __forceinline__ f32x8 operator()(const float* t, int row0, int ks) const {
        const f32x4 a = *reinterpret_cast<const f32x4*>(t + later_chunk<float, W>(at[0], 8 * ks) + row0 * W);
        const f32x4 b = *reinterpret_cast<const f32x4*>(t + later_chunk<float, W>(at[1], 8 * ks) + row0 * W);
        return f32x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    }
};

// Operands by columns: lane l supplies column 16 (ct0 + ct) + (l & 15), slots
// 0..3 from rows ra + 4g .. +3 and slots 4..7 from rows rb + 4g .. +3 (ra, rb
// multiples of 16).  The rows 4g + i of two 16-row blocks are what an
// accumulator tile leaves in lane group g, so the other operand of the product
// stays in registers.  (bf16: the transposing LDS read, a lane group's 16 lanes
// fetching 4 rows of 16 columns.)  CT column tiles, ct0 a multiple of CT, and of
// 4 where CT is more.
template <typename E, int W, int CT> struct ColReader;
template <int W, int CT> struct ColReader<bf16, W, CT> {
    int at, from;   // at in bytes
    __device__ __forceinline__ explicit ColReader(int lane, int ct0 = 0) : from(ct0) {
        const int r = 4 * (lane >> 4) + ((lane & 15) >> 2), c = 4 * (lane & 3);
        const int chunk = 2 * ct0 + (c >> 3);
        at = 2 * (tile_at<bf16, W>(r, CT <= 4 ? chunk : chunk & 7) + (c & 4));
    }
    __device__ __forceinline__ void keep() { asm volatile("" : "+v"(at)); }
    __device__ __forceinline__ bf16x8 operator()(const bf16* t, int ra, int rb, int ct) const {
        typedef __attribute__((address_space(3))) s16x4 lds_s16x4;
        typedef short s16x8 __attribute__((ext_vector_type(8)));
        const int far = CT <= 4 ? 0 : (from + ct) >> 2;   // 128-byte groups behind the first
        const int flip = 32 * (ct & 3) + (WHOLE_ROWS<bf16, W> ? 128 * (far & 1) : 0);
        const int on = WHOLE_ROWS<bf16, W> ? 256 * (far >> 1) : 128 * far;
        const char* p = reinterpret_cast<const char*>(t) + (at ^ flip) + on;
        const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 2 * ra * W));
        const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4*)(p + 2 * rb * W));
        return __builtin_bit_cast(bf16x8, s16x8{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]});
    }
};
template <int W, int CT> struct ColReader<float, W, CT> {
    int lane, ct0;
    __device__ __forceinline__ explicit ColReader(int lane, int ct0 = 0) : lane(lane), ct0(ct0) {}
    __device__ __forceinline__ void keep() {}
    __device__ __forceinline__ f32x8 operator()(const float* t, int ra, int rb, int ct) const {
        const int g4 = 4 * (lane >> 4), c = 16 * (ct0 + ct) + (lane & 15);
        f32x8 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[i] = t[tile_at<float, W>(ra + g4 + i, c >> 2) + (c & 3)];
            v[4 + i] = t[tile_at<float, W>(rb + g4 + i, c >> 2) + (c & 3)];
        }
        return v;
    }
    // Slots 0 to 3 alone.
    __device__ __forceinline__ f32x8 half(const float* t, int ra, int ct) const {
        const int g4 = 4 * (lane >> 4), c = 16 * (ct0 + ct) + (lane & 15);
        f32x8 v = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = t[tile_at<float, W>(ra + g4 + i, c >> 2) + (c & 3)];
        return v;
    }
};

// Two accumulator tiles (rows 4g + i of two 16-row blocks) as the 8 slots of
// an operand.  To bf16 each value is rounded to nearest: the products take
// bf16 operands, and a relative error of at most 2^-8 per weight is that of
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

// Called between the load of operands that a loop keeps in registers and the
// loop: the wait for them then stands here.  The compiler otherwise puts it where
// the loop first uses them, in every pass, where it also waits for the loads
// that the pass has just issued for the next tile (forward of the packed training
// step 1.24 ms with these waits in the loop, 1.17 without).
template <typename T> __device__ __forceinline__ void arrived(T& x) { asm volatile("" : "+v"(x)); }

// N steps use(e), each with an operand that fetch(e) reads from LDS D steps
// ahead into a ring of D + 1: the compiler, short of registers, otherwise puts
// every read right before its use and waits for it.
template <int I> using Int = std::integral_constant<int, I>;
template <int N, int D, int E, typename F, typename U>
__device__ __forceinline__ void ahead_step(F& fetch, U& use) {
    if constexpr (E + D < N) fetch(Int<E + D>());
    __builtin_amdgcn_sched_barrier(0);
    use(Int<E>());
    __builtin_amdgcn_sched_barrier(0);
}
template <int N, int D, typename F, typename U, int... E, int... S>
__device__ __forceinline__ void ahead_all(F& fetch, U& use, std::integer_sequence<int, E...>, std::integer_sequence<int, S...>) {
    (fetch(Int<S>()), ...);
    (ahead_step<N, D, E>(fetch, use), ...);
}
// fetch and use take the step as an Int<e>, so that what they index is known
// when they are compiled.
template <int N, int D, typename F, typename U>
__device__ __forceinline__ void ahead(F fetch, U use) {
    ahead_all<N, D>(fetch, use, std::make_integer_sequence<int, N>(), std::make_integer_sequence<int, (D < N ? D : N)>());
}

// -- staging: global -> registers -> LDS ---------------------------------------
// ROWS x W elements moved by NT threads, 8 or more threads to a row (128-byte
// lines), so that a thread's chunks lie at constant offsets from one address
// per row it serves.  The loads are issued by load() and waited for by store(),
// a tile of work later.
static __device__ const u32x4 kZeros[144] = {};   // a row of up to 576 fp32 channels
template <typename E> __device__ __forceinline__ const E* zero_row() { return reinterpret_cast<const E*>(kZeros); }

template <typename E, int W, int ROWS, int NT>
struct Stage {
    static constexpr int CE = CHUNK_ELEMS<E>, TPR = ROWS * 8 >= NT ? 8 : NT / ROWS;   // threads per row
    static constexpr int PASS = NT / TPR, P = ROWS / PASS, S = W / CE / TPR;
    static_assert(ROWS % PASS == 0 && PASS % 16 == 0 && W % (TPR * CE) == 0, "whole passes and steps");
    u32x4 r[P][S];
    // rows in any order: row(r) returns the row's address (zero_row() for a row
    // that is not there, so that no load is conditional).  ONCE: rows that no other
    // workgroup reads, which the caches need not keep.
    template <bool ONCE>
    static __device__ __forceinline__ u32x4 chunk(const E* a) {
        return ONCE ? __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(a)) : *reinterpret_cast<const u32x4*>(a);
    }
    template <bool ONCE, typename F>
    __device__ __forceinline__ void load(int tid, F row) {
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const E* a = row(tid / TPR + PASS * p) + CE * (tid % TPR);
#pragma unroll
            for (int s = 0; s < S; ++s) r[p][s] = chunk<ONCE>(a + TPR * CE * s);
        }
    }
    // Rows `stride` elements apart from a base that is the same for all threads,
    // the first `left` of them there and zeros behind: channels [0, W - W1) from
    // base, the last W1 from base1.  A thread's offset within the tile fits in
    // 32 bits and stays the same from tile to tile (strides are below 2^23).
    template <int W1>
    __device__ __forceinline__ void load_rows(int tid, const E* base, int64_t stride, const E* base1, int64_t stride1,
                                              int left) {
        constexpr int S0 = (W - W1) / CE / TPR;
        static_assert(W1 % (TPR * CE) == 0, "whole steps");
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const uint32_t there = min(tid / TPR + PASS * p, left - 1), chunk = 16 * (tid % TPR);
            const uint32_t at = there * (uint32_t)(stride * sizeof(E)) + chunk;
            const uint32_t at1 = there * (uint32_t)(stride1 * sizeof(E)) + chunk;
#pragma unroll
            for (int s = 0; s < S; ++s)
                r[p][s] = *reinterpret_cast<const u32x4*>(
                    s < S0 ? reinterpret_cast<const char*>(base + TPR * CE * s) + at
                           : reinterpret_cast<const char*>(base1 + TPR * CE * (s - S0)) + at1);
        }
        if (left < ROWS) {
#pragma unroll
            for (int p = 0; p < P; ++p)
                if (tid / TPR + PASS * p >= left)
#pragma unroll
                    for (int s = 0; s < S; ++s) r[p][s] = u32x4{0, 0, 0, 0};
        }
    }
    __device__ __forceinline__ void load_rows(int tid, const E* base, int64_t stride, int left) {
        load_rows<0>(tid, base, stride, base, stride, left);
    }
    // Whether row tid / TPR + PASS p of the loaded tile has a value that is not
    // finite, the last W1 channels aside: the same answer in the row's TPR threads.
    template <int W1 = 0>
    __device__ __forceinline__ bool bad_row(int tid, int p, bool bad = false) const {
        static_assert(W1 % (TPR * CE) == 0, "whole steps");
#pragma unroll
        for (int s = 0; s < (W - W1) / CE / TPR; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const unsigned x = r[p][s][i];
                bad |= (x & 0x7f800000u) == 0x7f800000u;
                if (sizeof(E) == 2) bad |= (x & 0x7f80u) == 0x7f80u;
            }
        const unsigned long long any = __ballot(bad) >> (tid & 63 & ~(TPR - 1));
        return (any & ((1ull << TPR) - 1)) != 0;
    }
    // The row's values that are not finite, and only those, set to 0.
    __device__ __forceinline__ void clear_bad(int p) {
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                unsigned x = r[p][s][i];
                if (sizeof(E) == 2) {
                    if ((x & 0x7f80u) == 0x7f80u) x &= 0xffff0000u;
                    if ((x & 0x7f800000u) == 0x7f800000u) x &= 0xffffu;
                } else if ((x & 0x7f800000u) == 0x7f800000u) {
                    x = 0u;
                }
                r[p][s][i] = x;
            }
    }
    __device__ __forceinline__ void fill_row(int p, unsigned x) {
#pragma unroll
        for (int s = 0; s < S; ++s) r[p][s] = u32x4{x, x, x, x};
    }
    // store(), each chunk's register refilled at once with the tile after next,
    // so that a tile's worth of loads stays in flight
    template <bool ONCE, typename F>
    __device__ __forceinline__ void store_load(int tid, E* t, F row) {
        const int at = tile_at<E, W>(tid / TPR, tid % TPR);
#pragma unroll
        for (int p = 0; p < P; ++p) {
            const E* a = row(tid / TPR + PASS * p) + CE * (tid % TPR);
#pragma unroll
            for (int s = 0; s < S; ++s) {
                *reinterpret_cast<u32x4*>(t + later_chunk<E, W>(at, TPR * s) + PASS * p * W) = r[p][s];
                r[p][s] = chunk<ONCE>(a + TPR * CE * s);
            }
        }
    }
    __device__ __forceinline__ void store(int tid, E* t) const {
        const int at = tile_at<E, W>(tid / TPR, tid % TPR);
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
            for (int s = 0; s < S; ++s)
                *reinterpret_cast<u32x4*>(t + later_chunk<E, W>(at, TPR * s) + PASS * p * W) = r[p][s];
    }
};

// The same from global memory straight into LDS, without registers between: for
// tiles whose rows need no look.  Every wave writes 1 KB of the tile in a row, its
// lanes fetch the chunks that belong there; channels [0, W - W1) come from one
// base, the last W1 from another.  The rows up to `last` are there, and that one
// is repeated behind it.  fetch() issues the loads; landed() and a barrier end them.
template <typename E, int W, int ROWS, int NT, int W1 = 0>
struct Direct {
    static constexpr int CE = CHUNK_ELEMS<E>, CH = W / CE, N = ROWS * CH / NT;
    static_assert(ROWS * CH % NT == 0, "whole waves");
    uint32_t at[N], second;   // byte offsets; a bit for each chunk of the second base
    __device__ __forceinline__ void rows(int tid, int64_t stride, int64_t stride1, int last) {
        second = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const int n = i * NT + tid, r = n / CH;
            const int chunk = (tile_at<E, W>(r, n % CH) - r * W) / CE;
            const bool from1 = W1 > 0 && chunk >= (W - W1) / CE;
            second |= from1 ? 1u << i : 0u;
            at[i] = (uint32_t)min(r, last) * (uint32_t)((from1 ? stride1 : stride) * sizeof(E)) +
                    16u * (from1 ? chunk - (W - W1) / CE : chunk);
        }
    }
    __device__ __forceinline__ void rows(int tid, int64_t stride, int last) { rows(tid, stride, 0, last); }
    __device__ __forceinline__ void fetch(int wave, const E* base, const E* base1, E* t) const {
        typedef __attribute__((address_space(1))) const void global_void;
        typedef __attribute__((address_space(3))) void lds_void;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const E* from = W1 > 0 && (second >> i & 1) ? base1 : base;
            __builtin_amdgcn_global_load_lds((global_void*)(reinterpret_cast<const char*>(from) + at[i]),
                                             (lds_void*)(t + (i * NT + 64 * wave) * CE), 16, 0, 0);
        }
    }
    __device__ __forceinline__ void fetch(int wave, const E* base, E* t) const { fetch(wave, base, base, t); }
};
__device__ __forceinline__ void landed() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A product over keys that some rows do not see multiplies their weights, 0, with
// what such a key holds, and 0 times NaN or Inf is NaN.  In the tiles where that
// can happen a row with values that are not finite is therefore cleared from the
// operand of that product, and put as NaN (QUIET: in bf16 as in fp32) into the
// operand or statistic that the weights come from: there the rows that do not see
// the key are masked, and those that do get NaN.
constexpr unsigned QUIET = 0x7fff7fffu;

template <typename A, typename B>
__device__ __forceinline__ void move_bad_rows(int tid, A& product, B& weights) {
    static_assert(A::P == B::P && A::TPR == B::TPR, "the same rows in the same threads");
#pragma unroll
    for (int p = 0; p < A::P; ++p)
        if (product.bad_row(tid, p)) {
            product.fill_row(p, 0u);
            weights.fill_row(p, QUIET);
        }
}

// A grid has fewer than 2^32 threads a dimension: workgroups in rows of 65,536.
// The last row may be longer than the work; the kernels test what they are given.
static inline dim3 grid_of(int64_t blocks) {
    return blocks <= 65536 ? dim3((unsigned)blocks) : dim3(65536, (unsigned)((blocks + 65535) / 65536));
}
__device__ __forceinline__ int64_t block_of_grid() { return (int64_t)blockIdx.y * gridDim.x + blockIdx.x; }

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

// Sequence and item within it of the batch's item number `want`, where sequence
// s has count(s) of them; false behind the last.  One pass over the sequences, NT
// at a time (a scan per wave, the waves' sums through scratch).  Called by all NT
// threads.
template <int NT, typename F>
__device__ __forceinline__ bool find_item(int N, int want, int* scratch /* [NT / 64 + 2] in LDS */, int& seq, int& item,
                                          F count) {
    constexpr int NW = NT / 64;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int before = 0;
    for (int base = 0; base < N; base += NT) {
        const int s = base + tid;
        const int n = s < N ? count(s) : 0;
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
        seq = uniform(scratch[NW]);
        item = uniform(scratch[NW + 1]);
        __syncthreads();
        if (seq >= 0) return true;
        before = all;
    }
    return false;
}

// Sequence and tile within it of the batch's tile number `want` (tiles of B
// rows, counted through the sequences in order); false behind the last tile.
// A token counts as `each` rows.
// Called by all NT threads.
template <int B, int NT>
__device__ __forceinline__ bool find_tile(const int32_t* cu, int N, int rows, int total, int want,
                                          int* scratch /* [NT / 64 + 2] in LDS */, int& seq, int& tile, int each = 1) {
    if (!cu) {
        const int per = (rows * each + B - 1) / B;
        if (per == 0 || want >= per * N) return false;
        seq = want / per;
        tile = want - seq * per;
        return true;
    }
    return find_item<NT>(N, want, scratch, seq, tile, [&](int s) {
        int a, b;
        sequence_rows(cu, rows, total, s, a, b);
        return ((b - a) * each + B - 1) / B;
    });
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

// -- tokens and positions ---------------------------------------------------------
// cos and sin of position * frequency (radians).  The product and its
// reduction to a fraction of a turn are in 64 bits: at position 10^6 a product
// in 32 bits is off by 0.06 radians.
__device__ __forceinline__ void rotation(int position, float inv_freq, bool inverse, float& c, float& s) {
    const double turns = (double)position * (double)inv_freq * 0.15915494309189535;
    const float r = (float)(turns - rint(turns));
    sincospif(2.f * r, &s, &c);
    if (inverse) s = -s;
}

// Sequence of packed token t: the first s with cu[s + 1] > t, or -1 for a row
// outside the sequences.  A 64-way search, one probe per lane and step.
__device__ __forceinline__ int sequence_of(const int32_t* cu, int N, int64_t t, int lane) {
    int lo = 0, hi = N;   // the answer is in [lo, hi]
    while (lo < hi) {
        const int step = (hi - lo + 63) / 64, at = lo + lane * step + step - 1;
        const bool past = at >= hi || cu[at + 1] > t;
        const unsigned long long b = __ballot(past);
        const int first = b ? __builtin_ctzll(b) : 64;
        const int nlo = lo + first * step;
        hi = min(hi, nlo + step - 1);
        lo = min(nlo, hi);
    }
    return lo < N && t >= cu[0] ? lo : -1;
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
