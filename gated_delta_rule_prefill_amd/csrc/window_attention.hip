// window_attention.hip -- window attention, forward: over packed keys, and over a
// paged cache for chunks of new tokens.
//
// Per query head, row i at position p:
//   z_ij = scale q_i . k_j  for j <= p with p - j < W or j < sinks
//   o_i  = sum_j exp(z_ij - z_max) v_j / sum_j exp(z_ij - z_max)
// in one pass over the keys of a tile of rows (KeyRange: the sinks, then the run
// that the window covers) with the running maximum and sum.  The scores of a tile
// are formed transposed, S^T = K Q^T (rows = keys), so that a lane holds 4
// neighbouring keys of one query row: as they stand, exponentiated, they are the
// operand of O^T += V^T P^T, whose other operand is V read by columns.  Scores and
// weights never leave the registers, and a row's maximum, sum and rescale factor
// are one value per lane.
//
// Bound by the products and, next to them, the exponentials (a step of 64 keys is 64
// matrix instructions and 176 others for a wave, 32 of them exponentials), at the power
// that the card grants: bf16, d = 128, 32 heads over 8, window 4,096, 32,768 tokens take
// 2.0 ms, 1.03 PFLOP/s over the pairs that see each other (a library product of 8192^3:
// 1.15 to 1.31), and 1.69 ms on inputs of zeros.  16 documents, 36,755 tokens, window
// 1,024: 0.64 ms, 0.77 PFLOP/s: of a workgroup's 36 us 13.5 tiles take 28, as many a tile as
// in the long prompt, its start and end the rest.  16 chunks of 128 tokens over a cache, window
// 1,024: 55 us in a run of a hundred, 61 as one of a program's first.  Without effect:
// more operands read ahead, the next tile's scores between the exponentials, priorities
// of the waves; 8 waves and twice the rows spill (2.25 ms).
#include "window_common.h"

namespace kda {

// A workgroup of 4 waves, one key head.  A wave has 32 (fp32: 16) query rows, whose
// operands q and o stay in registers, and walks all keys.  SPLIT (few rows; see split_waves):
// the workgroup has 16 rows, a wave walks a quarter of each tile's keys
// with a maximum and sum of its own, and the four are joined behind the last.  Key and
// value tiles of BN rows are double-buffered in LDS: the next tile's loads, straight
// into LDS, are issued before a tile's products.
template <typename E, int D, bool PAGED, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(E) == 2 && !SPLIT ? 2 : 1) void window_attention_kernel(const WindowArgs a, int tiles)
{
    constexpr int BN = (sizeof(E) == 2 ? 64 : 32) * (SPLIT ? 2 : 1), NQ = SPLIT ? 1 : LATENT_NQ<E>;
    constexpr int BQ = WINDOW_ROWS<E, SPLIT>, KS = D / 32, PD = sizeof(E) == 2 ? 3 : 1;
    constexpr int TT = BN / (SPLIT ? 64 : 16), PAIR = TT > 1 ? 2 : 1;   // a wave's key tiles, and those by turns
    typedef typename Vec<E>::v8 v8;
    // two arrays, so that a read of one is seen not to wait for loads into the other
    __shared__ __attribute__((aligned(16))) E even[BN * 2 * D];
    __shared__ __attribute__((aligned(16))) E odd[BN * 2 * D];
    __shared__ int64_t place[4][PAGED ? BN : 1];   // cache rows of the tiles' keys, -1: none
    __shared__ int gaps[4];                        // whether a tile has keys without a row

    const kda_window_inputs& in = a.in;
    int h, want, seq, tile;
    if (block_of_grid() >= (int64_t)tiles * in.Hk) return;
    key_head_of_block(in.Hk, tiles, (int)block_of_grid(), h, want);
    const int rows_q = (int)(in.total_q / in.num_seqs), G = in.H / in.Hk;
    if (!find_tile<BQ, 256>(in.cu_seqlens_q, in.num_seqs, rows_q, (int)in.total_q, tiles - 1 - want,
                            reinterpret_cast<int*>(even), seq, tile, G))
        return;
    int q0, q1, k0 = 0, nk;
    sequence_rows(in.cu_seqlens_q, rows_q, (int)in.total_q, seq, q0, q1);
    if constexpr (PAGED) {
        nk = uniform(cached_tokens(a.pages, seq));
    } else {
        int k1;
        sequence_rows(in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q, (int)(in.total_k / in.num_seqs),
                      (int)in.total_k, seq, k0, k1);
        nk = k1 - k0;
    }
    const int nq = q1 - q0, off = nk - nq, rows = nq * G;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int wrow = SPLIT ? tile * BQ : tile * BQ + 16 * NQ * wave;   // the wave's first row
    const float sc = in.scale * LOG2E;
    auto token = [&](int row) { return (int)((unsigned)min(row, rows - 1) / (unsigned)G); };
    const KeyRange kr(uniform(token(tile * BQ)), uniform(token(tile * BQ + BQ - 1)), off, in.window, in.sinks, nk);
    const int nt = (kr.total + BN - 1) / BN;
    int td, te;   // the tiles [td, te) are seen whole by all rows
    kr.whole_tiles(BN, td, te);

    const E *kp, *vp;
    if constexpr (PAGED) {
        kp = (const E*)a.pages.k + h * a.pages.head_stride;
        vp = (const E*)a.pages.v + h * a.pages.head_stride;
    } else {
        kp = (const E*)in.k + (int64_t)k0 * in.k_token_stride + h * in.k_head_stride;
        vp = (const E*)in.v + (int64_t)k0 * in.v_token_stride + h * in.v_head_stride;
    }

    // this lane's query rows
    v8 q[NQ][KS];
    int first[NQ];   // the first key number behind the sinks that the row sees
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = min(wrow + 16 * j + col, rows - 1), i = token(r);
        const E* row = (const E*)in.q + (int64_t)(q0 + i) * in.q_token_stride + (h * G + r - i * G) * in.q_head_stride;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[j][ks] = row_frag_global(row, ks, lane);
        first[j] = kr.first(i + off);
    }
    // of the wave's rows
    const int w0 = uniform(token(wrow)) + off, w1 = uniform(token(wrow + 16 * NQ - 1)) + off;
    const int last_lo = kr.last(w0), last_hi = kr.last(w1), first_lo = kr.first(w0), first_hi = kr.first(w1);

    // Keys that some row does not see weigh 0, and 0 times NaN or Inf is NaN: in the
    // tiles that are not seen whole such rows are found and taken out.
    const Tiles<E, D, BN, 256> k_tiles(tid, in.k_token_stride), v_tiles(tid, in.v_token_stride);   // PAGED: strides of 0
    auto load = [&](int t, E* to) {
        if constexpr (PAGED) {
            auto row = [&](const E* base) {
                return [&, base](int r) {
                    const int64_t at = place[t & 3][r];
                    return at < 0 ? zero_row<E>() : base + at;
                };
            };
            k_tiles.fetch_rows(wave, row(kp), to);
            v_tiles.fetch_rows(wave, row(vp), to + BN * D);
        } else {
            const int64_t n0 = (int64_t)t * BN, key = n0 + kr.shift;
            const E *kt = kp + key * in.k_token_stride, *vt = vp + key * in.v_token_stride;
            if (t >= td && t < te) {
                k_tiles.fetch(wave, kt, to);
                v_tiles.fetch(wave, vt, to + BN * D);
            } else {
                const int split = kr.ns - (int)n0, left = kr.total - (int)n0;
                k_tiles.fetch_part(wave, kt, kp + n0 * in.k_token_stride, split, left, to);
                v_tiles.fetch_part(wave, vt, vp + n0 * in.v_token_stride, split, left, to + BN * D);
            }
        }
    };
    auto store = [&](int t, E* to) {
        landed();
        if (t < td || t >= te) v_tiles.move_bad(tid, to + BN * D, to);
    };
    // PAGED: the cache row of key tid of tile t (tid < BN)
    auto look_up = [&](int t) { return CachedRow(a.pages, seq, kr, t * BN + tid); };
    auto keep = [&](int t, const CachedRow& found) {
        const int64_t at = found.offset(a.pages);
        place[t & 3][tid] = at;
        const bool gap = __any(at < 0);
        if (tid == 0) gaps[t & 3] = gap;
    };
    CachedRow next_place;   // of tile t + 2 in step t
    if constexpr (PAGED) {
        static_assert(BN <= 64, "one wave looks the rows up");
        if (tid < BN) {
            const CachedRow p0 = look_up(0), p1 = look_up(1);
            keep(0, p0);
            keep(1, p1);
            next_place = look_up(2);
        }
        __syncthreads();
    }
    RowReader<E, D> k_rows(lane);
    ColReader<E, D, D / 16> v_cols(lane);

    f32x4 acc[NQ][D / 16];
    float m[NQ], l[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        m[j] = neg_inf();
        l[j] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[j][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (nt > 0) {
        load(0, even);
        store(0, even);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) arrived(q[j][ks]);
    auto step = [&](int t, const E* K, E* next) __attribute__((always_inline)) {
        k_rows.keep(), v_cols.keep();
        const E* V = K + BN * D;
        const int r0 = SPLIT ? 16 * TT * wave : 0, n0 = t * BN + r0;   // the wave's first key of the tile
        if (t + 1 < nt) load(t + 1, next);
        if constexpr (PAGED)
            if (tid < BN) {
                keep(t + 2, next_place);
                next_place = look_up(t + 3);
            }
        if (wrow < rows && n0 <= last_hi && (n0 < kr.ns || n0 + 16 * TT > first_lo)) {
            f32x4 s[NQ][TT];
            v8 x[PD + 1];
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int j = 0; j < NQ; ++j) s[j][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
            // One sequence of operands, read ahead across its parts: the scores,
            // two key tiles by turns so that products in a row do not wait for
            // each other; and, after the weights, the product with the values.
            constexpr int E0 = TT * KS;
            v8 p[NQ][TT / PAIR];
            auto take_weights = [&]() {
                if (!kr.whole(n0, n0 + 16 * TT, last_lo, first_hi)) {
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (kr.hides(n0 + 16 * tt + 4 * g + i, first[j], n0 < kr.ns)) s[j][tt][i] = neg_inf();
                }
                if constexpr (PAGED)
                    if (uniform(gaps[t & 3])) {
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (place[t & 3][r0 + 16 * tt + 4 * g + i] < 0)
#pragma unroll
                                    for (int j = 0; j < NQ; ++j) s[j][tt][i] = neg_inf();
                    }
                // The running maximum is raised only when a row's grew by more than
                // 8 (in powers of two): until then the weights stay below 2^8 and
                // nothing needs rescaling.
                float top[NQ];
                bool grew = false;
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    float x = neg_inf();
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x = fmaxf(x, s[j][tt][i]);
                    top[j] = group_max(x) * sc;
                    grew |= top[j] > m[j] + 8.f;
                }
                if (__any(grew)) {
#pragma unroll
                    for (int j = 0; j < NQ; ++j) {
                        const float mn = fmaxf(m[j], top[j]);
                        const float f = mn == neg_inf() ? 1.f : exp2_fast(m[j] - mn);
                        m[j] = mn;
                        l[j] *= f;
#pragma unroll
                        for (int c = 0; c < D / 16; ++c) acc[j][c] *= f;
                    }
                }
#pragma unroll
                for (int j = 0; j < NQ; ++j) {
                    const float base = m[j] == neg_inf() ? 0.f : m[j];   // a row that has seen no key yet
#pragma unroll
                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            s[j][tt][i] = exp2_fast(__builtin_fmaf(s[j][tt][i], sc, -base));
                            l[j] += s[j][tt][i];   // the sum takes the weights before their rounding
                        }
#pragma unroll
                    for (int b = 0; b < TT / PAIR; ++b)
                        p[j][b] = acc_frag(s[j][PAIR * b], s[j][PAIR * b + PAIR - 1], E());
                }
            };
            auto tt_of = [](int e) constexpr { return e / (PAIR * KS) * PAIR + e % PAIR; };
            ahead<E0 + D / 16 * (TT / PAIR), PD>(
                [&](auto n) {
                    constexpr int e = n, f = e - E0;
                    if constexpr (e < E0) x[e % (PD + 1)] = k_rows(K, r0 + 16 * tt_of(e), e / PAIR % KS);
                    else x[e % (PD + 1)] = cols<PAIR>(v_cols, V, r0 + 16 * PAIR * (f / (D / 16)), f % (D / 16));
                },
                [&](auto n) {
                    constexpr int e = n, f = e - E0;
                    if constexpr (e < E0) {
                        constexpr int tt = tt_of(e);
#pragma unroll
                        for (int j = 0; j < NQ; ++j) s[j][tt] = mma32(x[e % (PD + 1)], q[j][e / PAIR % KS], s[j][tt]);
                    } else {
                        if constexpr (f == 0) take_weights();
#pragma unroll
                        for (int j = 0; j < NQ; ++j)
                            acc[j][f % (D / 16)] =
                                mma_rows<PAIR>(x[e % (PD + 1)], p[j][f / (D / 16)], acc[j][f % (D / 16)]);
                    }
                });
        }
        if (t + 1 < nt) store(t + 1, next);
        __syncthreads();
    };
    int t = 0;
    for (; t + 1 < nt; t += 2) {
        step(t, even, odd);
        step(t + 1, odd, even);
    }
    if (t < nt) step(t, even, odd);
    // SPLIT: the four waves' parts brought to the largest maximum and added up in order, a
    // quarter of the channels each
    constexpr int OWN = SPLIT ? D / 64 : D / 16;
    const int own = SPLIT ? wave * OWN : 0;
    if constexpr (SPLIT) {
        float* stat = reinterpret_cast<float*>(odd);
        stat[tid] = m[0];
        __syncthreads();
        float top = neg_inf();
#pragma unroll
        for (int w = 0; w < 4; ++w) top = fmaxf(top, stat[64 * w + lane]);
        const float f = m[0] == neg_inf() ? 0.f : exp2_fast(m[0] - top);   // no key: its sums are 0
        m[0] = top;
#pragma unroll
        for (int c = 0; c < D / 16; ++c) acc[0][c] *= f;
        stat[256 + tid] = l[0] * f;
        join_waves<E, D>(even, wave, col, g, acc[0]);
        l[0] = stat[256 + lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) l[0] += stat[256 + 64 * w + lane];
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = wrow + 16 * j + col;
        const float sum = group_sum(l[j]);
        if (r >= rows) continue;
        const int i = token(r);
        const int64_t out = (int64_t)(q0 + i) * in.H + h * G + r - i * G;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        E* row = (E*)a.o + out * D + 16 * own;
#pragma unroll
        for (int c = 0; c < OWN; ++c) {
            typename Vec<E>::v4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = from_f32<E>(acc[j][c][i] * inv);
            store_vec(row + 16 * c + 4 * g, x);
        }
        if (a.lse && g == 0 && own == 0) a.lse[out] = sum == 0.f ? neg_inf() : (m[j] + __log2f(sum)) * LN2;
    }
}

template <typename E, int D, bool PAGED, bool SPLIT>
static hipError_t launch_as(const WindowArgs& a, hipStream_t stream) {
    const int64_t tiles = row_tiles(a.in, WINDOW_ROWS<E, SPLIT>);
    hipLaunchKernelGGL((window_attention_kernel<E, D, PAGED, SPLIT>), grid_of(tiles * a.in.Hk), dim3(256), 0, stream, a,
                       (int)tiles);
    return launch_result(stream);
}
template <typename E, int D, bool PAGED>
static hipError_t launch(const WindowArgs& a, hipStream_t stream) {
    if constexpr (sizeof(E) == 4 || !PAGED)   // few rows over a cache: window_decode.hip
        if (split_waves(a.in)) return launch_as<E, D, PAGED, true>(a, stream);
    return launch_as<E, D, PAGED, false>(a, stream);
}

hipError_t launch_window_attention(const WindowArgs& a, bool paged, hipStream_t stream) {
    if (a.in.dtype == KDA_DTYPE_BF16) {
        if (a.in.d == 128) return paged ? launch<bf16, 128, true>(a, stream) : launch<bf16, 128, false>(a, stream);
        return paged ? launch<bf16, 64, true>(a, stream) : launch<bf16, 64, false>(a, stream);
    }
    if (a.in.d == 128) return paged ? launch<float, 128, true>(a, stream) : launch<float, 128, false>(a, stream);
    return paged ? launch<float, 64, true>(a, stream) : launch<float, 64, false>(a, stream);
}

}  // namespace kda
