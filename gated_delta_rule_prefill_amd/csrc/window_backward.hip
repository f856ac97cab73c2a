// window_backward.hip -- gradients of the window attention.
//
// With the forward's weights w_ij = exp(z_ij - lse_i), z = scale q k^T, the output
// gradient g_i = dL/do_i and delta_i = g_i . o_i, over the pairs that see each other:
//   dv_j = sum_i w_ij g_i
//   dz_ij = w_ij (g_i . v_j - delta_i)
//   dq_i = scale sum_j dz_ij k_j,   dk_j = scale sum_i dz_ij q_i
// where i runs over the rows of all query heads that share the key head.  Two
// kernels, so that every sum stays in one workgroup's registers and the result does
// not depend on an order of atomics: one walks the keys for a tile of query rows
// (dq, and delta on the way), one walks the query rows for a tile of keys (dk, dv).
// Each forms z and g v^T: two of the seven products are repeated.
//
// The sinks are seen by every later row of their sequence: their walk is cut into
// pieces of WINDOW_PIECE tokens behind the window of the first key tile, whose parts
// of dk and dv a third kernel adds up in order, with the first tile's own.
//
// bf16, d = 128, 32 heads over 8, window 1,024, 16 documents (36,755 tokens): dq 0.98 to 1.02 ms
// (four products of 0.24 TFLOP over the visible pairs, as it takes dz twice: 0.99 PFLOP/s),
// dk and dv 1.13 to 1.20 (four: 0.85, LDS: a wave reads every operand for its 16 keys
// alone).  One kernel for all would have to add a part of dq for each tile of 64 keys.
#include <algorithm>

#include "window_common.h"

namespace kda {

// What the rounding of two accumulator tiles to an operand (acc_frag) left of them.
// bf16: dq takes dz in two parts, 16 bits in all.  With one it was off by 1.5 times
// what the rounding of dq itself costs (2.5e-3 against 1.65e-3 in the norm, packed
// documents, window 1,024): by the rounding of dz and by delta, which comes from the
// rounded o; with two by 1.1 times.  The second part costs 0.16 ms of dq's 1.00.
__device__ __forceinline__ bf16x8 rest_frag(f32x4 a, f32x4 b, bf16x8 x) {
    bf16x8 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = (bf16)(a[i] - (float)x[i]), y[4 + i] = (bf16)(b[i] - (float)x[4 + i]);
    return y;
}

__device__ __forceinline__ f32x8 rest_frag(f32x4, f32x4, f32x8) { return f32x8{}; }   // nothing, and never asked for

// bf16: dq of a row that sees few keys is a difference of few terms, which the error of
// delta (that of the rounded o) moves by more than dq's own rounding: with a window of 3,
// dq is off by 2.8e-3 in the norm, rounded once by 1.65e-3.  Such rows take the exact
// delta, which their weights give: a wave whose rows see no key behind the first step of
// 32 has it before it needs it (the first 32 tokens of a sequence, but for those whose
// wave has the 33rd too); where window and sinks together are no more than FEW_KEYS,
// every row walks its keys twice.  The lengths of the sequences beside do not matter.
constexpr int FEW_KEYS = 16;

// dq and delta.  As in the forward kernel the scores are formed transposed (rows =
// keys), so that dz^T is the operand of dq^T += K^T dz^T as it stands.  dq itself
// takes delta from the rounded o, as its own sum is complete only behind the last
// key (but see FEW_KEYS); the second kernel takes that sum.
// A wave owns 32 rows (fp32: 16) and walks all keys, 32 at a time.  SPLIT (few rows;
// see split_waves): the workgroup has 16 rows, a wave walks a quarter of each
// tile's keys, and the waves' sums are added up in order.
template <typename E, int D, bool SPLIT, bool TWICE>
__global__ __launch_bounds__(256, sizeof(E) == 2 && !SPLIT ? 2 : 1) void window_dq_kernel(
    const kda_window_inputs in, const E* __restrict__ o, const float* __restrict__ lse,
    const E* __restrict__ d_o, E* __restrict__ dq, float* __restrict__ row_stats, int tiles)
{
    constexpr int BN = (sizeof(E) == 2 ? 64 : 32) * (SPLIT ? 2 : 1), NQ = SPLIT ? 1 : LATENT_NQ<E>;
    constexpr int BQ = WINDOW_ROWS<E, SPLIT>, KS = D / 32, PD = sizeof(E) == 2 ? 3 : 1;
    // key tiles worked on at a time, and how often
    constexpr int TT = BN == 64 && SPLIT ? 1 : 2, SUBS = SPLIT ? 1 : BN / 32;
    typedef typename Vec<E>::v8 v8;
    // two arrays, so that a read of one is seen not to wait for loads into the other
    __shared__ __attribute__((aligned(16))) E even[BN * 2 * D];
    __shared__ __attribute__((aligned(16))) E odd[BN * 2 * D];

    int h, want, seq, tile;
    if (block_of_grid() >= (int64_t)tiles * in.Hk) return;
    key_head_of_block(in.Hk, tiles, (int)block_of_grid(), h, want);
    const int rows_q = (int)(in.total_q / in.num_seqs), G = in.H / in.Hk;
    if (!find_tile<BQ, 256>(in.cu_seqlens_q, in.num_seqs, rows_q, (int)in.total_q, tiles - 1 - want,
                            reinterpret_cast<int*>(even), seq, tile, G))
        return;
    int q0, q1, k0, k1;
    sequence_rows(in.cu_seqlens_q, rows_q, (int)in.total_q, seq, q0, q1);
    sequence_rows(in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q, (int)(in.total_k / in.num_seqs),
                  (int)in.total_k, seq, k0, k1);
    const int nq = q1 - q0, nk = k1 - k0, off = nk - nq, rows = nq * G;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int wrow = SPLIT ? tile * BQ : tile * BQ + 16 * NQ * wave;
    const float sc = in.scale * LOG2E;
    auto token = [&](int row) { return (int)((unsigned)min(row, rows - 1) / (unsigned)G); };
    const KeyRange kr(uniform(token(tile * BQ)), uniform(token(tile * BQ + BQ - 1)), off, in.window, in.sinks, nk);
    const int nt = (kr.total + BN - 1) / BN;
    int td, te;   // the tiles [td, te) are seen whole by all rows
    kr.whole_tiles(BN, td, te);

    const E* kp = (const E*)in.k + (int64_t)k0 * in.k_token_stride + h * in.k_head_stride;
    const E* vp = (const E*)in.v + (int64_t)k0 * in.v_token_stride + h * in.v_head_stride;

    v8 q[NQ][KS], go[NQ][KS];   // the rows and their output gradients
    int first[NQ];   // the first key number behind the sinks that the row sees
    float lse2[NQ], dl[NQ], exact[NQ];   // delta from the rounded o, and from this kernel's own weights
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = min(wrow + 16 * j + col, rows - 1), i = token(r), head = h * G + r - i * G;
        const E* row = (const E*)in.q + (int64_t)(q0 + i) * in.q_token_stride + head * in.q_head_stride;
        const int64_t at = (int64_t)(q0 + i) * in.H + head;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[j][ks] = row_frag_global(row, ks, lane);
        float sum = 0.f;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
            go[j][ks] = row_frag_global(d_o + at * D, ks, lane);
            const v8 ov = row_frag_global(o + at * D, ks, lane);
#pragma unroll
            for (int e = 0; e < 8; ++e) sum += to_f32(go[j][ks][e]) * to_f32(ov[e]);
        }
        lse2[j] = lse[at] * LOG2E;
        // a row that sees no key has o = 0, and 0 times a d_o of NaN or Inf is NaN
        dl[j] = group_sum(sum);
        if (lse2[j] == neg_inf()) dl[j] = 0.f;
        exact[j] = 0.f;
        first[j] = kr.first(i + off);
    }
    const int w0 = uniform(token(wrow)) + off, w1 = uniform(token(wrow + 16 * NQ - 1)) + off;
    const int last_lo = kr.last(w0), last_hi = kr.last(w1), first_lo = kr.first(w0), first_hi = kr.first(w1);

    const Tiles<E, D, BN, 256> k_tiles(tid, in.k_token_stride), v_tiles(tid, in.v_token_stride);
    auto load = [&](int t, E* to) {
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
    };
    // Keys that some row does not see weigh 0, and 0 times NaN or Inf is NaN: in the
    // tiles that are not seen whole such rows are found and taken out.
    auto store = [&](int t, E* to) {
        landed();
        if (t < td || t >= te) k_tiles.move_bad(tid, to, to + BN * D);
    };
    RowReader<E, D> rows_of(lane);
    ColReader<E, D, D / 16> k_cols(lane);

    f32x4 acc[NQ][D / 16];
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) arrived(q[j][ks]), arrived(go[j][ks]);
    auto step = [&](int t, const E* K, E* next) __attribute__((always_inline)) {
        rows_of.keep(), k_cols.keep();
        const E* V = K + BN * D;
        if (t + 1 < nt) load(t + 1, next);
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
            const int r0 = SPLIT ? 16 * TT * wave : 32 * sub, n0 = t * BN + r0;
            if (wrow >= rows || n0 > last_hi || (n0 >= kr.ns && n0 + 16 * TT <= first_lo)) continue;
            f32x4 s[NQ][TT], dp[NQ][TT];
            v8 x[PD + 1];
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int j = 0; j < NQ; ++j) s[j][tt] = dp[j][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
            // One sequence of operands, read ahead across its parts: z = q k^T;
            // g v^T, between whose products the weights' exponentials run; and,
            // after dz, dq^T += K^T dz.
            constexpr int E0 = TT * KS, E1 = 2 * E0, NS = NQ * TT * 4;
            v8 dz[NQ], rest[NQ];
            ahead<E1 + D / 16, PD>(
                [&](auto n) {
                    constexpr int e = n;
                    x[e % (PD + 1)] = e < E0   ? rows_of(K, r0 + 16 * (e % TT), e / TT)
                                      : e < E1 ? rows_of(V, r0 + 16 * ((e - E0) % TT), (e - E0) / TT)
                                               : cols<TT>(k_cols, K, r0, e - E1);
                },
                [&](auto n) {
                    constexpr int e = n;
                    if constexpr (e < E0) {
#pragma unroll
                        for (int j = 0; j < NQ; ++j) s[j][e % TT] = mma32(x[e % (PD + 1)], q[j][e / TT], s[j][e % TT]);
                    } else if constexpr (e < E1) {
                        constexpr int f = e - E0;
#pragma unroll
                        for (int j = 0; j < NQ; ++j) dp[j][f % TT] = mma32(x[e % (PD + 1)], go[j][f / TT], dp[j][f % TT]);
#pragma unroll
                        for (int m = NS * f / E0; m < NS * (f + 1) / E0; ++m) {
                            const int j = m / (TT * 4), tt = m / 4 % TT, i = m % 4;
                            s[j][tt][i] = exp2_fast(__builtin_fmaf(s[j][tt][i], sc, -lse2[j]));
                        }
                    } else {
                        if (e == E1) {
                            if (!kr.whole(n0, n0 + 16 * TT, last_lo, first_hi)) {   // weights of hidden keys
#pragma unroll
                                for (int j = 0; j < NQ; ++j)
#pragma unroll
                                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            if (kr.hides(n0 + 16 * tt + 4 * g + i, first[j], n0 < kr.ns))
                                                s[j][tt][i] = 0.f, dp[j][tt][i] = 0.f;
                            }
#pragma unroll
                            for (int j = 0; j < NQ; ++j) {
#pragma unroll
                                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) exact[j] += s[j][tt][i] * dp[j][tt][i];
                                if (sizeof(E) == 2 && last_hi < 16 * TT) dl[j] = group_sum(exact[j]);   // see FEW_KEYS
#pragma unroll
                                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) s[j][tt][i] *= dp[j][tt][i] - dl[j];
                                dz[j] = acc_frag(s[j][0], s[j][TT - 1], E());
                                if constexpr (sizeof(E) == 2) rest[j] = rest_frag(s[j][0], s[j][1], dz[j]);
                            }
                        }
                        constexpr int c = e - E1;
#pragma unroll
                        for (int j = 0; j < NQ; ++j) acc[j][c] = mma_rows<TT>(x[e % (PD + 1)], dz[j], acc[j][c]);
                        if constexpr (sizeof(E) == 2)
#pragma unroll
                            for (int j = 0; j < NQ; ++j) acc[j][c] = mma32(x[e % (PD + 1)], rest[j], acc[j][c]);
                    }
                });
        }
        if (t + 1 < nt) store(t + 1, next);
        __syncthreads();
    };
    // TWICE: the second walk has the first one's exact delta.
    constexpr int passes = TWICE ? 2 : 1;
    for (int pass = 0; pass < passes; ++pass) {
        if (pass > 0) {
            float* sums = reinterpret_cast<float*>(odd);
            if constexpr (SPLIT) {
                sums[tid] = exact[0];
                __syncthreads();
                exact[0] = sums[lane];
#pragma unroll
                for (int w = 1; w < 4; ++w) exact[0] += sums[64 * w + lane];
                __syncthreads();
            }
#pragma unroll
            for (int j = 0; j < NQ; ++j) dl[j] = group_sum(exact[j]);
        }
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            exact[j] = 0.f;
#pragma unroll
            for (int c = 0; c < D / 16; ++c) acc[j][c] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        if (nt > 0) {
            load(0, even);
            store(0, even);
        }
        __syncthreads();
        int t = 0;
        for (; t + 1 < nt; t += 2) {
            step(t, even, odd);
            step(t + 1, odd, even);
        }
        if (t < nt) step(t, even, odd);
    }
    // SPLIT: the waves' sums, a quarter of the channels each
    constexpr int OWN = SPLIT ? D / 64 : D / 16;
    const int own = SPLIT ? wave * OWN : 0;
    if constexpr (SPLIT) {
        join_waves<E, D>(even, wave, col, g, acc[0]);
        float* sums = reinterpret_cast<float*>(odd);
        sums[tid] = exact[0];
        __syncthreads();
        exact[0] = sums[lane];
#pragma unroll
        for (int w = 1; w < 4; ++w) exact[0] += sums[64 * w + lane];
    }
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = wrow + 16 * j + col;
        const float sum = group_sum(exact[j]);
        if (r >= rows) continue;
        const int i = token(r), head = h * G + r - i * G;
        if (g == 0 && own == 0) {
            float* stats = row_stats + 2 * ((int64_t)head * in.total_q + q0 + i);
            stats[0] = lse2[j];
            stats[1] = sum;
        }
        E* row = dq + ((int64_t)(q0 + i) * in.H + head) * D + 16 * own;
#pragma unroll
        for (int c = 0; c < OWN; ++c) {
            typename Vec<E>::v4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = from_f32<E>(acc[j][c][i] * in.scale);
            store_vec(row + 16 * c + 4 * g, x);
        }
    }
}

// Work of a sequence in the second kernel: its key tiles, and behind them the
// pieces of the sinks' walk, as many items each as there are tiles with sinks.  Those
// tiles walk the tokens before `behind`, piece c those from behind + c WINDOW_PIECE
// on: no key before WINDOW_MAX_SINKS has them in its window.
template <bool SPLIT> constexpr int DKV_KEYS = SPLIT ? 16 : 64;   // of a tile
template <int KEYS>
struct KeyWork {
    int q0, nq, k0, nk, behind, tiles, pieces, sink_tiles;
    __device__ __forceinline__ KeyWork(const kda_window_inputs& in, int s) {
        int q1, k1;
        sequence_rows(in.cu_seqlens_q, (int)(in.total_q / in.num_seqs), (int)in.total_q, s, q0, q1);
        sequence_rows(in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q, (int)(in.total_k / in.num_seqs),
                      (int)in.total_k, s, k0, k1);
        nq = q1 - q0;
        nk = k1 - k0;
        tiles = (nk + KEYS - 1) / KEYS;
        behind = in.sinks > 0 ? min(nq, max(0, min(in.window, nk) + WINDOW_MAX_SINKS - 1 - (nk - nq))) : nq;
        pieces = nk > 0 ? (nq - behind + WINDOW_PIECE - 1) / WINDOW_PIECE : 0;
        sink_tiles = (min(in.sinks, nk) + KEYS - 1) / KEYS;
    }
    // The first slot of its partial gradients: one for the tiles with sinks, then one
    // for each piece (see window_slots).
    __device__ __forceinline__ int64_t slot(int s) const { return q0 / WINDOW_PIECE + 2 * (int64_t)s; }
};

// bf16: walks of no more than so many tokens take the weights and dz in two parts as well:
// where a few of them make the gradients of all keys their rounding shows (21 documents of
// 1 to 9 tokens: error of dk 2.6e-3, with two parts 1.7e-3).  In code of its own: a branch
// at the products cost the long walks 15 % (packed step 1,204 -> 1,440 us).
constexpr int FEW_ROWS = 32;

// dk and dv.  A wave owns 16 keys, whose k and v operands and gradients stay in
// registers; the query rows come 64 tokens of one head at a time (fp32: 32), head after
// head of the group, and are worked on 32 at a time (32 tokens a time, with twice the
// barriers: 1.32 ms against 1.20).  SPLIT (few keys): the workgroup has 16
// keys, a wave walks a quarter of each 128 rows (fp32: 64), and the waves' sums are added
// up in order behind the last.  The scores are formed with rows = queries, so that
// the weights and dz are the operands of dv^T += g^T w and dk^T += q^T dz as they stand.
template <typename E, int D, bool SPLIT>
__global__ __launch_bounds__(256, sizeof(E) == 2 && !SPLIT ? 2 : 1) void window_dkv_kernel(
    const kda_window_inputs in, const E* __restrict__ d_o, const float* __restrict__ row_stats,
    E* __restrict__ dk, int64_t dk_token_stride, int64_t dk_head_stride,
    E* __restrict__ dv, int64_t dv_token_stride, int64_t dv_head_stride, float* __restrict__ part, int items)
{
    constexpr int BQ = (sizeof(E) == 2 ? 64 : 32) * (SPLIT ? 2 : 1), BK = DKV_KEYS<SPLIT>;
    constexpr int KS = D / 32, PD = sizeof(E) == 2 ? 3 : 1;
    constexpr int RT = BQ == 64 && SPLIT ? 1 : 2, SUBS = SPLIT ? 1 : BQ / 32;   // row tiles worked on at a time, and how often
    typedef typename Vec<E>::v8 v8;
    // two arrays, so that a read of one is seen not to wait for loads into the other
    __shared__ __attribute__((aligned(16))) E even[BQ * 2 * D];
    __shared__ __attribute__((aligned(16))) E odd[BQ * 2 * D];
    __shared__ __attribute__((aligned(16))) float srow[2][2 * BQ];   // lse (base 2), then delta
    __shared__ unsigned long long bad_rows[2][(BQ + 63) / 64];       // a bit for each row to be taken out

    int h, want, seq, item;
    if (block_of_grid() >= (int64_t)items * in.Hk) return;
    key_head_of_block(in.Hk, items, (int)block_of_grid(), h, want);
    typedef KeyWork<BK> Work;
    if (!find_item<256>(in.num_seqs, want, reinterpret_cast<int*>(even), seq, item, [&](int s) {
            const Work w(in, s);
            return w.tiles + w.pieces * w.sink_tiles;
        }))
        return;
    const Work work(in, seq);
    const int nq = work.nq, nk = work.nk, off = nk - nq, G = in.H / in.Hk;
    const int piece = item < work.tiles ? -1 : (item - work.tiles) / work.sink_tiles;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int key0 = BK * (piece < 0 ? item : item - work.tiles - piece * work.sink_tiles);
    const int wkey = SPLIT ? key0 : key0 + 16 * wave, key = wkey + col;
    const int W = min(in.window, nk);
    const float sc = in.scale * LOG2E;
    // the tokens [ta, te) to walk
    const int ta = piece < 0 ? min(nq, max(0, key0 - off)) : work.behind + piece * WINDOW_PIECE;
    const int te = piece >= 0          ? min(nq, ta + WINDOW_PIECE)
                   : key0 < in.sinks ? max(ta, work.behind)
                                     : max(ta, (int)min((int64_t)nq, (int64_t)key0 + BK - 1 + W - off));
    const int per = (te - ta + BQ - 1) / BQ, nu = per * G;   // tiles of a head, and all

    v8 k[KS], v[KS];
    {
        const int64_t row = work.k0 + min(key, nk - 1);
        const E* kp = (const E*)in.k + row * in.k_token_stride + h * in.k_head_stride;
        const E* vp = (const E*)in.v + row * in.v_token_stride + h * in.v_head_stride;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) k[ks] = row_frag_global(kp, ks, lane), v[ks] = row_frag_global(vp, ks, lane);
    }
    const E* qp = (const E*)in.q + (int64_t)(work.q0 + ta) * in.q_token_stride + h * G * in.q_head_stride;
    const E* gp = d_o + ((int64_t)(work.q0 + ta) * in.H + h * G) * D;
    const float* sp = row_stats + 2 * ((int64_t)h * G * in.total_q + work.q0 + ta);

    // A head's tiles [td, tw): rows that all see all of the workgroup's keys.
    const int td = max(0, key0 + BK - 1 - (ta + off) + BQ - 1) / BQ;
    const int tw = min((te - ta) / BQ, positions_in_window(key0, W, ta + off) / BQ);
    // lse and delta of a row travel with one of the first BQ threads.
    float next_lse = 0.f, next_delta = 0.f;
    const Tiles<E, D, BQ, 256> q_tiles(tid, in.q_token_stride), g_tiles(tid, (int64_t)in.H * D);
    auto load = [&](int head, int t, E* to) {
        const int left = te - ta - t * BQ;
        const E* qt = qp + head * in.q_head_stride + (int64_t)t * BQ * in.q_token_stride;
        const E* gt = gp + (int64_t)head * D + (int64_t)t * BQ * in.H * D;
        if (tid < BQ) {   // behind the last row those of its copies, which are not kept
            const float* at = sp + 2 * ((int64_t)head * in.total_q + t * BQ + min(tid, left - 1));
            next_lse = at[0];
            next_delta = at[1];
        }
        if (left >= BQ) {
            q_tiles.fetch(wave, qt, to);
            g_tiles.fetch(wave, gt, to + BQ * D);
        } else {
            q_tiles.fetch_part(wave, qt, qt, 0, left, to);
            g_tiles.fetch_part(wave, gt, gt, 0, left, to + BQ * D);
        }
    };
    // A row with q that is not finite has no finite lse, one with g that is not finite
    // no finite delta (each enters every product of the row's sum, with a factor that
    // is not finite or a zero that makes NaN of it).  In tiles whose rows do not all
    // see all keys such rows are taken out, and their lse is NaN: the keys that see
    // them get NaN, the others a weight of 0 times finite values.  The copies of the
    // last row behind it are taken out with it; they weigh nothing: lse = inf.
    auto store = [&](int u, int t) {
        if (tid < BQ) {
            const bool there = tid < te - ta - t * BQ;
            const bool bad = !(__builtin_fabsf(next_lse) < __builtin_inff()) ||
                             !(__builtin_fabsf(next_delta) < __builtin_inff());
            const unsigned long long rows = __ballot(bad);
            srow[u & 1][tid] = !there ? __builtin_inff() : bad ? __builtin_nanf("") : next_lse;
            srow[u & 1][BQ + tid] = bad || !there ? 0.f : next_delta;
            if (lane == 0) bad_rows[u & 1][wave] = rows;
        }
        landed();
    };
    RowReader<E, D> rows_of(lane);
    ColReader<E, D, D / 16> cols_of(lane);
    f32x4 ak[D / 16], av[D / 16];
#pragma unroll
    for (int c = 0; c < D / 16; ++c) ak[c] = av[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (nu > 0) {
        load(0, 0, even);
        store(0, 0);
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) arrived(k[ks]), arrived(v[ks]);
    // Tile t of a head's tokens, number u of all; the next one is nt of nhead.
    auto step = [&](int u, int t, int nhead, int nt, E* Q, E* next, auto few) __attribute__((always_inline)) {
        constexpr bool FEW = decltype(few)::value != 0;
        rows_of.keep(), cols_of.keep();
        E* Gt = Q + BQ * D;
        if (u + 1 < nu) load(nhead, nt, next);
        if (t < td || t >= tw) {
            unsigned long long any = 0, bad[(BQ + 63) / 64];
#pragma unroll
            for (int w = 0; w < (BQ + 63) / 64; ++w) any |= bad[w] = (unsigned long long)uniform((int64_t)bad_rows[u & 1][w]);
            if (any) {
#pragma unroll
                for (int i = 0; i < q_tiles.N; ++i)
                    if (bad[i * q_tiles.STEP / 64] >> (q_tiles.row(i) & 63) & 1) {
                        *reinterpret_cast<u32x4*>(Q + (i * 256 + tid) * q_tiles.CE) = u32x4{0, 0, 0, 0};
                        *reinterpret_cast<u32x4*>(Gt + (i * 256 + tid) * q_tiles.CE) = u32x4{0, 0, 0, 0};
                    }
                __syncthreads();
            }
        }
#pragma unroll
        for (int sub = 0; sub < SUBS; ++sub) {
            const int r0 = SPLIT ? 16 * RT * wave : 32 * sub;   // the first of the tile's rows worked on
            const float* R = srow[u & 1] + r0;
            // positions of these rows
            const int p0 = ta + t * BQ + r0 + off, p1 = min(p0 + 16 * RT, te + off) - 1;
            if (p1 < max(p0, wkey) || (p0 - (wkey + 15) >= W && wkey >= in.sinks)) continue;
            f32x4 s[RT], dp[RT], ls[RT], de[RT];
            v8 x[PD + 1];
#pragma unroll
            for (int a = 0; a < RT; ++a) {
                s[a] = dp[a] = f32x4{0.f, 0.f, 0.f, 0.f};
                ls[a] = *reinterpret_cast<const f32x4*>(R + 16 * a + 4 * g);
                de[a] = *reinterpret_cast<const f32x4*>(R + BQ + 16 * a + 4 * g);
            }
            // One sequence of operands, read ahead across its parts: z = q k^T;
            // g v^T, between whose products the weights' exponentials run;
            // dv^T += g^T w, between whose products dz is formed; dk^T += q^T dz.
            constexpr int E0 = RT * KS, E1 = 2 * E0, E2 = E1 + D / 16, NS = 4 * RT;
            v8 wf, zf, rest;
            ahead<E2 + D / 16, PD>(
                [&](auto n) {
                    constexpr int e = n;
                    x[e % (PD + 1)] = e < E0   ? rows_of(Q, r0 + 16 * (e % RT), e / RT)
                                      : e < E1 ? rows_of(Gt, r0 + 16 * ((e - E0) % RT), (e - E0) / RT)
                                      : e < E2 ? cols<RT>(cols_of, Gt, r0, e - E1)
                                               : cols<RT>(cols_of, Q, r0, e - E2);
                },
                [&](auto n) {
                    constexpr int e = n;
                    const v8& a = x[e % (PD + 1)];
                    if constexpr (e < E0) {
                        s[e % RT] = mma32(a, k[e / RT], s[e % RT]);
                    } else if constexpr (e < E1) {
                        constexpr int f = e - E0;
                        dp[f % RT] = mma32(a, v[f / RT], dp[f % RT]);
#pragma unroll
                        for (int i = NS * f / E0; i < NS * (f + 1) / E0; ++i)
                            s[i / 4][i % 4] = exp2_fast(__builtin_fmaf(s[i / 4][i % 4], sc, -ls[i / 4][i % 4]));
                    } else if constexpr (e < E2) {
                        constexpr int c = e - E1;
                        if (c == 0) {
                            // weights of hidden keys
                            if (p0 < wkey + 15 || (p1 - wkey >= W && wkey + 15 >= in.sinks)) {
#pragma unroll
                                for (int i = 0; i < NS; ++i) {
                                    const int p = p0 + 16 * (i / 4) + 4 * g + i % 4;
                                    if (key > p || (p - key >= W && key >= in.sinks))
                                        s[i / 4][i % 4] = 0.f, dp[i / 4][i % 4] = 0.f;
                                }
                            }
                            wf = acc_frag(s[0], s[RT - 1], E());
                            if constexpr (FEW) rest = rest_frag(s[0], s[1], wf);
                        }
                        av[c] = mma_rows<RT>(a, wf, av[c]);
                        if constexpr (FEW) av[c] = mma32(a, rest, av[c]);
#pragma unroll
                        for (int i = NS * c / (D / 16); i < NS * (c + 1) / (D / 16); ++i)
                            dp[i / 4][i % 4] = s[i / 4][i % 4] * (dp[i / 4][i % 4] - de[i / 4][i % 4]);
                    } else {
                        constexpr int c = e - E2;
                        if (c == 0) {
                            zf = acc_frag(dp[0], dp[RT - 1], E());
                            if constexpr (FEW) rest = rest_frag(dp[0], dp[1], zf);
                        }
                        ak[c] = mma_rows<RT>(a, zf, ak[c]);
                        if constexpr (FEW) ak[c] = mma32(a, rest, ak[c]);
                    }
                });
        }
        if (u + 1 < nu) store(u + 1, nt);
        __syncthreads();
    };
    auto walk = [&](auto few) __attribute__((always_inline)) {
        int head = 0, t = 0;
        auto next = [&](int u, E* Q, E* to) __attribute__((always_inline)) {
            const int nt = t + 1 < per ? t + 1 : 0, nhead = nt ? head : head + 1;
            step(u, t, nhead, nt, Q, to, few);
            t = nt;
            head = nhead;
        };
        int u = 0;
        for (; u + 1 < nu; u += 2) {
            next(u, even, odd);
            next(u + 1, odd, even);
        }
        if (u < nu) next(u, even, odd);
    };
    if (sizeof(E) == 2 && te - ta <= FEW_ROWS) walk(Int<sizeof(E) == 2>());
    else walk(Int<0>());
    // SPLIT: the waves' sums, a quarter of the channels each
    constexpr int OWN = SPLIT ? D / 64 : D / 16;
    const int own = SPLIT ? wave * OWN : 0;
    if constexpr (SPLIT) {
        join_waves<E, D>(even, wave, col, g, ak);
        join_waves<E, D>(odd, wave, col, g, av);
    }
    if (key >= nk) return;
    const bool sink = key < in.sinks && work.pieces > 0;
    if (piece >= 0 && !sink) return;
    if (sink) {
        float* to = part + (((work.slot(seq) + piece + 1) * in.Hk + h) * in.sinks + key) * 2 * D + 16 * own + 4 * g;
#pragma unroll
        for (int c = 0; c < OWN; ++c) {
            store_vec(to + 16 * c, ak[c] * in.scale);
            store_vec(to + D + 16 * c, av[c]);
        }
        return;
    }
    const int64_t row = work.k0 + key;
    E* kr = dk + row * dk_token_stride + h * dk_head_stride + 16 * own;
    E* vr = dv + row * dv_token_stride + h * dv_head_stride + 16 * own;
#pragma unroll
    for (int c = 0; c < OWN; ++c) {
        typename Vec<E>::v4 kx, vx;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kx[i] = from_f32<E>(ak[c][i] * in.scale);
            vx[i] = from_f32<E>(av[c][i]);
        }
        store_vec(kr + 16 * c + 4 * g, kx);
        store_vec(vr + 16 * c + 4 * g, vx);
    }
}

// The sinks' gradients: the parts of the key tiles and of the pieces, in order,
// rounded once.  A workgroup per sequence and key head, a thread per 4 channels.
template <typename E, int D>
__global__ __launch_bounds__(256) void window_sinks_kernel(
    const kda_window_inputs in, const float* __restrict__ part, E* __restrict__ dk, int64_t dk_token_stride,
    int64_t dk_head_stride, E* __restrict__ dv, int64_t dv_token_stride, int64_t dv_head_stride)
{
    const int seq = (int)(block_of_grid() / in.Hk), h = (int)(block_of_grid() % in.Hk);
    if (seq >= in.num_seqs) return;
    const KeyWork<DKV_KEYS<false>> work(in, seq);
    if (work.pieces == 0) return;
    const int64_t stride = (int64_t)in.Hk * in.sinks * 2 * D;   // from slot to slot
    const float* from = part + (work.slot(seq) * in.Hk + h) * in.sinks * 2 * D;
    for (int id = threadIdx.x; id < min(in.sinks, work.nk) * (D / 2); id += 256) {
        const int key = id / (D / 2), c = 4 * (id % (D / 2));
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
        for (int p = 0; p <= work.pieces; ++p)
            sum += *reinterpret_cast<const f32x4*>(from + p * stride + key * 2 * D + c);
        typename Vec<E>::v4 x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = from_f32<E>(sum[i]);
        const int64_t row = work.k0 + key;
        store_vec(c < D ? dk + row * dk_token_stride + h * dk_head_stride + c
                        : dv + row * dv_token_stride + h * dv_head_stride + c - D, x);
    }
}

template <typename E, int D, bool SPLIT, bool TWICE>
static hipError_t launch_dq(const kda_window_inputs& in, const WindowGrads& a, hipStream_t stream) {
    const int64_t tiles = row_tiles(in, WINDOW_ROWS<E, SPLIT>);
    hipLaunchKernelGGL((window_dq_kernel<E, D, SPLIT, TWICE>), grid_of(tiles * in.Hk), dim3(256), 0, stream, in, (const E*)a.o,
                       a.lse, (const E*)a.d_o, (E*)a.dq, a.row_stats, (int)tiles);
    return launch_result(stream);
}

// Key tiles and pieces of the second kernel; pieces exist only where a token stands
// behind the windows of all keys that may be sinks.
static bool has_pieces(const kda_window_inputs& in) {
    return in.sinks > 0 && in.total_k > (int64_t)in.window + WINDOW_MAX_SINKS - 1;
}
static int64_t key_items(const kda_window_inputs& in, int keys) {
    return in.total_k / keys + in.num_seqs +
           (has_pieces(in) ? (in.total_q / WINDOW_PIECE + in.num_seqs) * ((in.sinks + keys - 1) / keys) : 0);
}
template <typename E, int D, bool SPLIT>
static hipError_t launch_dkv(const kda_window_inputs& in, const WindowGrads& a, hipStream_t stream) {
    const int64_t items = key_items(in, DKV_KEYS<SPLIT>);
    hipLaunchKernelGGL((window_dkv_kernel<E, D, SPLIT>), grid_of(items * in.Hk), dim3(256), 0, stream, in,
                       (const E*)a.d_o, a.row_stats, (E*)a.dk, a.dk_token_stride, a.dk_head_stride, (E*)a.dv,
                       a.dv_token_stride, a.dv_head_stride, a.part, (int)items);
    return launch_result(stream);
}

template <typename E, int D>
static hipError_t launch(const kda_window_inputs& in, const WindowGrads& a, hipStream_t stream) {
    if (in.total_q > 0) {
        constexpr bool BF16 = sizeof(E) == 2;
        const bool split = split_waves(in);
        hipError_t e;
        if (BF16 && (int64_t)in.window + in.sinks <= FEW_KEYS)
            e = split ? launch_dq<E, D, true, BF16>(in, a, stream) : launch_dq<E, D, false, BF16>(in, a, stream);
        else
            e = split ? launch_dq<E, D, true, false>(in, a, stream) : launch_dq<E, D, false, false>(in, a, stream);
        if (e) return e;
    }
    if (in.total_k == 0) return hipSuccess;
    hipError_t e;
    // fp32: the split form as long as the whole one has two workgroups a CU or fewer (four
    // with d = 64, half the LDS).  d 128, window 256, 1,024 tokens x 2 key heads: 142
    // against 428 us; 16 documents of 256: 104 against 154; 17,600 tokens x 8: 4.14 against
    // 3.65 ms.  d 64, window 512, 12,192 tokens x 4: 651 against 855.  bf16, whose products
    // are not what a short walk waits for: as long as the split form's workgroups take
    // little more than one round.  d 128, 4 query heads a key head, 1,000 tokens x 1 key
    // head, window 128 and 1,024: 20 against 38 us, 47 against 97; 2,000 x 2: 38 and 38, 56
    // against 107; 2,000 x 4, window 256: 56 against 41, d 64 28 against 31; 4,000 x 4: 50
    // against 39.
    const int64_t whole = key_items(in, DKV_KEYS<false>) * in.Hk;
    const int64_t most = (sizeof(E) == 4 ? 512 : 96) * (128 / D);
    e = whole <= most ? launch_dkv<E, D, true>(in, a, stream) : launch_dkv<E, D, false>(in, a, stream);
    if (e || !has_pieces(in)) return e;
    hipLaunchKernelGGL((window_sinks_kernel<E, D>), grid_of((int64_t)in.num_seqs * in.Hk), dim3(256), 0, stream, in,
                       a.part, (E*)a.dk, a.dk_token_stride, a.dk_head_stride, (E*)a.dv, a.dv_token_stride, a.dv_head_stride);
    return launch_result(stream);
}

hipError_t launch_window_attention_backward(const kda_window_inputs& in, const WindowGrads& a, hipStream_t stream) {
    if (in.dtype == KDA_DTYPE_BF16)
        return in.d == 128 ? launch<bf16, 128>(in, a, stream) : launch<bf16, 64>(in, a, stream);
    return in.d == 128 ? launch<float, 128>(in, a, stream) : launch<float, 64>(in, a, stream);
}

}  // namespace kda
