// window_decode.hip -- window attention of new tokens over a paged cache.
//
// A (token, query head of the group) pair is one query row; the rows of a sequence
// and key head meet the same cached keys and values:
//   z_rj = scale q_r . k_j,  o_r = sum_j softmax(z_r)_j v_j
// over the sinks and the window (KeyRange).  With one new token the G rows of a
// group share every cached row that is read, G flops per byte: the bytes of the
// window bound the kernel.  Many rows (chunks of several prompts) go to the forward
// kernel in its paged form.
//
// bf16, d = 128, 32 heads over 8, window 1,024: 256 sequences take 190 us, 5.4 TB/s of
// cached rows (reads alone reach 6.25; loads past the caches 2 % faster, at the expense
// of pages that sequences share; three workgroups a CU spill: 230).  One sequence with
// a window of 4,096: 9.0 us, 256 workgroups with one block of 32 keys a wave, and 4.2 for
// the join; latency.  (A join by the last workgroup to end needs a fence that writes an
// XCD's L2 back: 117 us.)
#include <algorithm>

#include "window_common.h"

namespace kda {

constexpr int DECODE_SLOTS = 512;   // partial results of 16 rows each
constexpr int DECODE_KEYS = 32;      // keys of a wave's step

// Where the rows of a row tile whose keys are split belong, for the join: row r is
// query head r % G of token first + r / G, and r runs from `row` over `rows` (0: there
// is no such tile).
struct DecodeTile {
    int32_t first, row, rows, pad;
};
// Workspace: a DecodeTile for each row tile, then its partial results, a split after
// another, 16 rows of o, m and l each.

// A workgroup takes 16 query rows of a sequence and key head and a run of its
// blocks of 32 keys; its 4 waves take the blocks in turns, each with its own running
// maximum, sum and output, and are joined in LDS.  No barrier inside the walk: keys go
// from memory into the matrix operands, values through a tile in LDS of the wave's
// own (to be read by columns), and the next block's loads are in flight during a
// block's products.
template <typename E, int D>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void window_decode_kernel(const WindowArgs a,
                                                                                   DecodeTile* __restrict__ where,
                                                                                   float* __restrict__ part, int splits)
{
    constexpr int KS = D / 32, BN = DECODE_KEYS, CE = CHUNK_ELEMS<E>, CH = D / CE;   // 16-byte chunks of a row
    constexpr int RPI = 64 / CH, VI = BN / RPI;   // rows of a wave's load, loads of a block's values
    constexpr int OS = D + 4;                     // row stride of the waves' outputs in LDS
    typedef typename Vec<E>::v8 v8;
    typedef typename Vec<E>::v4 v4;
    constexpr int TILE = BN * D * (int)sizeof(E), OUT = 16 * OS * 4;
    __shared__ __attribute__((aligned(16))) char buffer[4][TILE > OUT ? TILE : OUT];
    __shared__ int64_t place[4][2][BN];
    __shared__ float stat[4][2][16];
    __shared__ int found[3], scratch[6];

    const kda_window_inputs& in = a.in;
    const int unit = blockIdx.x / splits, split = blockIdx.x - unit * splits;
    const int h = unit % in.Hk, want = unit / in.Hk;
    const int rows_q = (int)(in.total_q / in.num_seqs), G = in.H / in.Hk;
    // the sequence, its rows and its cached tokens, looked up at once
    int seq = -1, tile = 0, q0 = 0, q1 = 0, nk = 0;
    if (in.cu_seqlens_q) {
        int a0 = 0, a1 = 0, n = 0, mine = -1;
        if (find_item<256>(in.num_seqs, want, scratch, seq, tile, [&](int s) {
                sequence_rows(in.cu_seqlens_q, rows_q, (int)in.total_q, s, a0, a1);
                n = cached_tokens(a.pages, s);
                mine = s;
                return ((a1 - a0) * G + 15) / 16;
            })) {
            if (mine == seq) found[0] = a0, found[1] = a1, found[2] = n;
            __syncthreads();
            q0 = uniform(found[0]), q1 = uniform(found[1]), nk = uniform(found[2]);
        }
    } else {
        const int per = (rows_q * G + 15) / 16;
        if (per > 0 && want < per * in.num_seqs) {
            seq = want / per;
            tile = want - seq * per;
            sequence_rows(nullptr, rows_q, (int)in.total_q, seq, q0, q1);
            nk = uniform(cached_tokens(a.pages, seq));
        }
    }
    const int nq = q1 - q0, off = nk - nq, rows = nq * G;
    // Row tiles are counted by a bound: behind the last one there is no sequence, and
    // `tile` says nothing.
    if (splits > 1 && split == 0 && threadIdx.x == 0)
        where[unit] = seq < 0 ? DecodeTile{0, 0, 0, 0} : DecodeTile{q0, tile * 16, min(16, rows - tile * 16), 0};
    if (seq < 0) return;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const float sc = in.scale * LOG2E;
    auto token = [&](int row) { return (int)((unsigned)min(row, rows - 1) / (unsigned)G); };
    const int i0 = uniform(token(tile * 16)), i1 = uniform(token(tile * 16 + 15));
    const KeyRange kr(i0, i1, off, in.window, in.sinks, nk);
    const int blocks = (kr.total + BN - 1) / BN;
    const int b0 = (int)((int64_t)blocks * split / splits), b1 = (int)((int64_t)blocks * (split + 1) / splits);
    const E* kp = (const E*)a.pages.k + h * a.pages.head_stride;
    const E* vp = (const E*)a.pages.v + h * a.pages.head_stride;

    // the cache row of key `lane` (below BN) of block b
    auto look_up = [&](int b) { return CachedRow(a.pages, seq, kr, b * BN + lane, lane < BN && b < b1); };
    CachedRow next_place = look_up(b0 + wave);

    const int r = min(tile * 16 + col, rows - 1), i = token(r);
    v8 q[KS];
    {
        const E* row = (const E*)in.q + (int64_t)(q0 + i) * in.q_token_stride + (h * G + r - i * G) * in.q_head_stride;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[ks] = row_frag_global(row, ks, lane);
    }
    const int first = kr.first(i + off);

    v8 k[2][KS];
    u32x4 v[VI];
    unsigned there = 0, next_there = 0;   // a bit for each key of the block that has a row
    auto load = [&](int b) {              // block b, whose rows next_place holds; then those of the wave's next
        int64_t* at = place[wave][b >> 2 & 1];
        const int64_t mine = next_place.offset(a.pages);
        next_there = (unsigned)__ballot(mine >= 0);
        if (lane < BN) at[lane] = mine;
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            const int64_t x = at[16 * tt + col];
            const E* row = x < 0 ? zero_row<E>() : kp + x;
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) k[tt][ks] = row_frag_global(row, ks, lane);
        }
#pragma unroll
        for (int n = 0; n < VI; ++n) {
            const int64_t x = at[n * RPI + lane / CH];
            const E* row = x < 0 ? zero_row<E>() : vp + x;
            v[n] = *reinterpret_cast<const u32x4*>(row + CE * (lane % CH));
        }
        next_place = look_up(b + 4);
    };
    E* vt = reinterpret_cast<E*>(buffer[wave]);
    const ColReader<E, D, D / 16> v_cols(lane);
    f32x4 acc[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) acc[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    float m = neg_inf(), l = 0.f;
    if (b0 + wave < b1) load(b0 + wave);
    for (int b = b0 + wave; b < b1; b += 4) {
        const int n0 = b * BN;
        there = next_there;
        const bool whole = kr.whole(n0, n0 + BN, kr.last_min, kr.first_max) && there == 0xffffffffu;
        // Rows of different tokens: a hidden key's weight is 0, and 0 times NaN or
        // Inf is NaN.  Its value row is cleared, and its score NaN where it is seen.
        unsigned bad = 0;
        if (i0 != i1 && !whole) {
#pragma unroll
            for (int n = 0; n < VI; ++n) {
                bool x = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    x |= (v[n][e] & 0x7f800000u) == 0x7f800000u;
                    if (sizeof(E) == 2) x |= (v[n][e] & 0x7f80u) == 0x7f80u;
                }
                const unsigned long long any = __ballot(x);
#pragma unroll
                for (int s = 0; s < RPI; ++s) {
                    const bool row_bad = (any >> (s * CH) & (CH == 64 ? ~0ull : (1ull << CH) - 1)) != 0;
                    if (row_bad) bad |= 1u << (n * RPI + s);
                    if (row_bad && lane / CH == s) v[n] = u32x4{0, 0, 0, 0};
                }
            }
        }
#pragma unroll
        for (int n = 0; n < VI; ++n)
            *reinterpret_cast<u32x4*>(vt + tile_at<E, D>(n * RPI + lane / CH, lane % CH)) = v[n];
        f32x4 s[2];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            s[tt] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) s[tt] = mma32(k[tt][ks], q[ks], s[tt]);
        }
        if (b + 4 < b1) load(b + 4);
        if (!whole) {
#pragma unroll
            for (int tt = 0; tt < 2; ++tt)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int x = 16 * tt + 4 * g + e, n = n0 + x;
                    if (bad >> x & 1) s[tt][e] = __builtin_nanf("");
                    if (kr.hides(n, first, n0 < kr.ns) || !(there >> x & 1)) s[tt][e] = neg_inf();
                }
        }
        float top = neg_inf();
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int e = 0; e < 4; ++e) top = fmaxf(top, s[tt][e]);
        top = group_max(top) * sc;
        // the maximum is raised only where it grew by more than 8, in powers of two
        if (__any(top > m + 8.f)) {
            const float mn = fmaxf(m, top), f = mn == neg_inf() ? 1.f : exp2_fast(m - mn);
            m = mn;
            l *= f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[c] *= f;
        }
        const float base = m == neg_inf() ? 0.f : m;
#pragma unroll
        for (int tt = 0; tt < 2; ++tt)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                s[tt][e] = exp2_fast(__builtin_fmaf(s[tt][e], sc, -base));
                l += s[tt][e];   // the sum takes the weights before their rounding
            }
        const v8 p = acc_frag(s[0], s[1], E());
        asm volatile("" ::: "memory");   // the wave's own stores of the values, then its reads
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[c] = mma32(v_cols(vt, 0, 16, c), p, acc[c]);
        asm volatile("" ::: "memory");
    }
    // the waves' results, joined: 16 threads to a row
    __syncthreads();
    float* wo = reinterpret_cast<float*>(buffer[wave]);
    l = group_sum(l);
    if (g == 0) stat[wave][0][col] = m, stat[wave][1][col] = l;
#pragma unroll
    for (int c = 0; c < D / 16; ++c) store_vec(wo + col * OS + 16 * c + 4 * g, acc[c]);
    __syncthreads();
    const int row = tid >> 4, c0 = tid & 15;
    float top = neg_inf(), sum = 0.f, f[4];
#pragma unroll
    for (int w = 0; w < 4; ++w) top = fmaxf(top, stat[w][0][row]);
    const float from = top == neg_inf() ? 0.f : top;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
        f[w] = exp2_fast(stat[w][0][row] - from);
        sum += f[w] * stat[w][1][row];
    }
    const int64_t slot = (int64_t)unit * splits + split;
    const int out_r = tile * 16 + row;
    if (out_r >= rows) return;
    const int out_i = token(out_r);
    const int64_t out = (int64_t)(q0 + out_i) * in.H + h * G + out_r - out_i * G;
    const float inv = splits > 1 ? 1.f : sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        f32x4 x = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < 4; ++w)
            x += f[w] * *reinterpret_cast<const f32x4*>(reinterpret_cast<const float*>(buffer[w]) + row * OS + 64 * c + 4 * c0);
        if (splits > 1) {
            store_vec(part + (slot * 16 + row) * (D + 4) + 64 * c + 4 * c0, x);
        } else {
            v4 y;
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] = from_f32<E>(x[e] * inv);
            store_vec((E*)a.o + out * D + 64 * c + 4 * c0, y);
        }
    }
    if (c0 == 0) {
        if (splits > 1) {
            float* ml = part + (slot * 16 + row) * (D + 4) + D;
            ml[0] = top;
            ml[1] = sum;
        } else if (a.lse) {
            a.lse[out] = sum == 0.f ? neg_inf() : (top + __log2f(sum)) * LN2;
        }
    }
}

// Joins the splits' results of a row tile: with M = max_s m_s,
//   o = sum_s 2^(m_s - M) o_s / sum_s 2^(m_s - M) l_s,  in order.
// 16 threads to a row; where there are few rows, several such groups share its splits,
// whose sums are added in LDS.
template <typename E, int D>
__global__ __launch_bounds__(256) void window_join_kernel(const WindowArgs a, const DecodeTile* __restrict__ where,
                                                          const float* __restrict__ part, int splits)
{
    constexpr int PS = D + 4;
    __shared__ __attribute__((aligned(16))) float joined[16][PS];
    const kda_window_inputs& in = a.in;
    const int unit = blockIdx.x, h = unit % in.Hk, G = in.H / in.Hk;
    const DecodeTile x = where[unit];
    if (x.rows <= 0) return;
    const int shift = x.rows > 8 ? 4 : x.rows > 4 ? 3 : x.rows > 2 ? 2 : x.rows > 1 ? 1 : 0;
    const int c0 = threadIdx.x & 15, at = threadIdx.x >> 4, row = at & ((1 << shift) - 1), group = at >> shift,
              groups = 16 >> shift;
    const bool there = row < x.rows;
    f32x4 y[D / 64];
    float top = neg_inf(), sum = 0.f;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) y[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (there) {
        const float* from = part + ((int64_t)unit * splits * 16 + row) * PS;
#pragma unroll 8
        for (int s = group; s < splits; s += groups) top = fmaxf(top, from[s * 16 * PS + D]);
        const float base = top == neg_inf() ? 0.f : top;
#pragma unroll 8
        for (int s = group; s < splits; s += groups) {
            const float* p = from + s * 16 * PS;
            const float f = exp2_fast(p[D] - base);
            sum += f * p[D + 1];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) y[c] += f * *reinterpret_cast<const f32x4*>(p + 64 * c + 4 * c0);
        }
    }
    if (groups > 1) {
#pragma unroll
        for (int c = 0; c < D / 64; ++c) store_vec(&joined[at][64 * c + 4 * c0], y[c]);
        if (c0 == 0) joined[at][D] = top, joined[at][D + 1] = sum;
        __syncthreads();
        if (group > 0) return;
        for (int i = 1; i < groups; ++i) top = fmaxf(top, joined[(i << shift) + row][D]);
        const float base = top == neg_inf() ? 0.f : top;
        sum = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) y[c] = f32x4{0.f, 0.f, 0.f, 0.f};
        for (int i = 0; i < groups; ++i) {
            const float* p = joined[(i << shift) + row];
            const float f = exp2_fast(p[D] - base);
            sum += f * p[D + 1];
#pragma unroll
            for (int c = 0; c < D / 64; ++c) y[c] += f * *reinterpret_cast<const f32x4*>(p + 64 * c + 4 * c0);
        }
    }
    if (!there) return;
    const int r = x.row + row, i = (int)((unsigned)r / (unsigned)G);
    const int64_t out = (int64_t)(x.first + i) * in.H + h * G + r - i * G;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
        typename Vec<E>::v4 v;
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = from_f32<E>(y[c][e] * inv);
        store_vec((E*)a.o + out * D + 64 * c + 4 * c0, v);
    }
    if (a.lse && c0 == 0) a.lse[out] = sum == 0.f ? neg_inf() : (top + __log2f(sum)) * LN2;
}

size_t window_decode_workspace(int32_t d) { return (size_t)DECODE_SLOTS * (sizeof(DecodeTile) + 16 * (d + 4) * 4); }

// Row tiles of all key heads.
static int64_t decode_units(const kda_window_inputs& in) { return row_tiles(in, 16) * in.Hk; }

template <typename E, int D>
static hipError_t launch(const WindowArgs& a, void* workspace, hipStream_t stream) {
    const kda_window_inputs& in = a.in;
    const int64_t N = in.num_seqs, units = decode_units(in);
    // Few row tiles have their keys split over workgroups, 128 keys or more each, as long
    // as all of them run at once, two a CU.  bf16, window 1,024, 32/8 heads, 512 workgroups
    // against 1,024 in us without the join: 8 sequences 12.0 and 14.5, 16 16.8 and 20.2,
    // 32 24.9 and 28.0; one, window 16,384, with the join: 21.9 and 28.  One, window 1,024,
    // with 64 keys or more: 6.2 + 4.7 for 6.8 + 3.6; with 256: 8.1 + 3.2.
    const int64_t most = std::min((int64_t)in.window + in.sinks + (in.total_q + N - 1) / N,
                                  (int64_t)a.pages.max_pages * a.pages.page_size);
    const int64_t splits = std::max<int64_t>(1, std::min((most + 127) / 128, DECODE_SLOTS / units));
    DecodeTile* where = (DecodeTile*)workspace;
    float* part = (float*)(where + DECODE_SLOTS);
    hipLaunchKernelGGL((window_decode_kernel<E, D>), dim3((unsigned)(units * splits)), dim3(256), 0, stream, a, where, part,
                       (int)splits);
    if (const hipError_t e = launch_result(stream)) return e;
    if (splits == 1) return hipSuccess;
    hipLaunchKernelGGL((window_join_kernel<E, D>), dim3((unsigned)units), dim3(256), 0, stream, a, where, part, (int)splits);
    return launch_result(stream);
}

hipError_t launch_window_decode(const WindowArgs& a, void* workspace, hipStream_t stream) {
    // The forward kernel shares a cached row among 128 rows (fp32: 64, or 16), but its
    // walk is not split: it takes batches of many row tiles, more than one of 16 rows a
    // sequence on average.  bf16, window 1,024, 32/8 heads, decode against forward in us: 1
    // sequence of 128 new tokens 21 and 38, 4 of 64 31 and 40, 16 of 16 31 and 38, of 32 57
    // and 41, 128 of 4 108 and 113, of 8 142 and 114.  fp32, window 512, 16/4 heads: 8 of 4 19
    // and 27, of 8 28 and 27, of 16 38 and 27, of 32 52 and 57, 64 of 4 52 and 57, of 8 67 and 60.
    // Batches of single tokens and one chunk go as a whole: 255 and a chunk of 128 209 and
    // 231, of 512 244 and 232, of 900 278 and 239, of 2,000 375 and 266; 63 and 2,000 241 and
    // 117; 31 and 128 37 and 50, 31 and 512 74 and 52.  The rule takes the other kernel for
    // 255 and 512, 31 and 128.
    const int64_t G = a.in.H / a.in.Hk;
    if (a.in.total_q * G > 16 * (int64_t)a.in.num_seqs &&
        decode_units(a.in) > (a.in.dtype == KDA_DTYPE_BF16 ? 512 : 64))
        return launch_window_attention(a, true, stream);
    if (a.in.dtype == KDA_DTYPE_BF16)
        return a.in.d == 128 ? launch<bf16, 128>(a, workspace, stream) : launch<bf16, 64>(a, workspace, stream);
    return a.in.d == 128 ? launch<float, 128>(a, workspace, stream) : launch<float, 64>(a, workspace, stream);
}

}  // namespace kda
