// latent_backward.hip -- gradients of the expanded latent attention.
//
// With the forward's weights w_ij = exp(z_ij - lse_i), z = scale q [k, k_pe]^T,
// the output gradient g_i = dL/do_i and delta_i = g_i . o_i:
//   dv_j = sum_i w_ij g_i
//   dz_ij = w_ij (g_i . v_j - delta_i)
//   dq_i = scale sum_j dz_ij [k_j, k_pe_j]
//   [dk_j, dk_pe_j] = scale sum_i dz_ij q_i,  dk_pe summed over the heads
// Two kernels, so that every sum stays in one workgroup's registers and the
// result does not depend on an order of atomics: one walks the keys for a tile
// of query rows (dq, and delta on the way), one walks the query rows for a
// tile of keys (dk, dv and the head's part of dk_pe).  Each forms z and g v^T: two
// of the seven products are repeated, 38 % more work at 128 + 64 channels than a
// single kernel's five.  That one would add a part of dq for every tile of 64
// keys, 20 GB in fp32 for the batch below, and in an order to be the same every
// time.  A third kernel sums dk_pe over the heads.
#include <algorithm>

#include "latent_common.h"

namespace kda {

// fp32: a batch of few tiles has each one's walk split over workgroups (the grid's
// second dimension), whose sums latent_sum_kernel adds in order.  One row tile's
// products fill a CU's matrix units for 5 us a step, on 40 CUs of 256 for 495
// tokens x 4 heads: 55 + 68 us without, 26 + 30 and the sum's 9 with.  Delta then comes from o, which in
// fp32 is as exact as the sum.
template <typename E> constexpr bool SPLIT = sizeof(E) == 4;
int latent_splits(int64_t rows, int32_t H) {
    const int64_t tiles = (rows + 63) / 64 * H;
    return tiles >= 128 || tiles == 0 ? 1 : (int)std::min<int64_t>(8, 256 / tiles);
}

// dq and delta.  As in the forward kernel the scores are formed transposed
// (rows = keys), so that dz^T is the operand of dq^T += K^T dz^T as it stands.
// dq itself takes delta from the rounded o, as its own sum is complete only
// behind the last key; the second kernel takes that sum.  Bound by the matrix
// products: 36,755 tokens in 16 documents x 32 heads, bf16: 1.69 ms, 1.07 PFLOP/s.
template <typename E, int DN, int DR>
__global__ __launch_bounds__(256, 2) void latent_dq_kernel(
    const kda_latent_inputs in, const E* __restrict__ o, const float* __restrict__ lse,
    const E* __restrict__ d_o, E* __restrict__ dq, float* __restrict__ row_stats, float* __restrict__ part, int tiles)
{
    constexpr int DQK = DN + DR, DV = DN, BN = 32, NQ = LATENT_NQ<E>, BQ = 64 * NQ;
    constexpr int KS = DQK / 32, VS = DV / 32, TT = BN / 16, PD = sizeof(E) == 2 ? 3 : 1;
    typedef typename Vec<E>::v8 v8;
    // two arrays, so that a read of one is seen not to wait for loads into the other
    __shared__ __attribute__((aligned(16))) E even[BN * (DQK + DV)];
    __shared__ __attribute__((aligned(16))) E odd[BN * (DQK + DV)];
    // the rows' output gradients and, where registers are short, the last block
    // of q: each wave's own, in operand order
    constexpr int QL = sizeof(E) == 2 && KS > 4 ? 1 : 0, QR = KS - QL;
    __shared__ __attribute__((aligned(16))) E sgo[4][NQ][VS + QL][64 * 8];

    int h, want, seq, tile;
    head_tile_of_block(in.H, tiles, h, want);
    const int rows_q = (int)(in.total_q / in.num_seqs);
    if (!find_tile<BQ, 256>(in.cu_seqlens_q, in.num_seqs, rows_q, (int)in.total_q, tiles - 1 - want,
                            reinterpret_cast<int*>(even), seq, tile))
        return;
    int q0, q1, k0, k1;
    sequence_rows(in.cu_seqlens_q, rows_q, (int)in.total_q, seq, q0, q1);
    sequence_rows(in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q, (int)(in.total_k / in.num_seqs),
                  (int)in.total_k, seq, k0, k1);
    const int nq = q1 - q0, nk = k1 - k0, off = nk - nq;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int wrow = tile * BQ + 16 * NQ * wave;
    const float sc = in.scale * LOG2E;

    const E* kp = (const E*)in.k + (int64_t)k0 * in.k_token_stride + h * in.k_head_stride;
    const E* vp = (const E*)in.v + (int64_t)k0 * in.v_token_stride + h * in.v_head_stride;
    const E* pp = DR ? (const E*)in.k_pe + (int64_t)k0 * in.k_pe_token_stride : nullptr;

    v8 q[NQ][QR];
    float lse2[NQ], dl[NQ], exact[NQ];   // delta from the rounded o, and from this kernel's own weights
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = wrow + 16 * j + col, rr = min(r, nq - 1);
        const E* row = (const E*)in.q + (int64_t)(q0 + rr) * in.q_token_stride + h * in.q_head_stride;
        const int64_t at = (int64_t)(q0 + rr) * in.H + h;
#pragma unroll
        for (int ks = 0; ks < QR; ++ks) q[j][ks] = row_frag_global(row, ks, lane);
        if (QL) store_frag(sgo[wave][j][VS], lane, row_frag_global(row, KS - 1, lane));
        float sum = 0.f;
#pragma unroll
        for (int vs = 0; vs < VS; ++vs) {
            const v8 gv = row_frag_global(d_o + at * DV, vs, lane), ov = row_frag_global(o + at * DV, vs, lane);
            store_frag(sgo[wave][j][vs], lane, gv);
#pragma unroll
            for (int i = 0; i < 8; ++i) sum += to_f32(gv[i]) * to_f32(ov[i]);
        }
        dl[j] = group_sum(sum);
        lse2[j] = lse[at] * LOG2E;
        exact[j] = 0.f;
    }
    const int end = in.causal ? min(nk, min(nq, (tile + 1) * BQ) + off) : nk;
    const int all = end > 0 ? (end + BN - 1) / BN : 0;
    // the key tiles of this split (fp32)
    const int tb = SPLIT<E> ? (int)((int64_t)all * blockIdx.y / gridDim.y) : 0;
    const int nt = SPLIT<E> ? (int)((int64_t)all * (blockIdx.y + 1) / gridDim.y) : all;
    const int wave_end = in.causal ? min(nk, min(nq, wrow + 16 * NQ) + off) : nk;
    const int wave_full = in.causal ? min(nk, wrow + off + 1) : nk;

    Stage<E, DQK, BN, 256> sk;
    Stage<E, DV, BN, 256> sv;
    // Tiles that all rows see whole go straight to LDS (64 + 0 channels, 8,192
    // tokens x 8 heads: both kernels 394 -> 312 us; 128 + 64: the same); the others
    // through registers, where rows that are not finite are found and taken out.
    Direct<E, DQK, BN, 256, DR> direct_k;
    Direct<E, DV, BN, 256> direct_v;
    auto load = [&](int t, auto hides, E* to) {
        const int64_t key = (int64_t)t * BN;
        const E* kt = kp + key * in.k_token_stride;
        const E* pt = DR ? pp + key * in.k_pe_token_stride : kt;
        const E* vt = vp + key * in.v_token_stride;
        if constexpr (hides) {
            sk.template load_rows<DR>(tid, kt, in.k_token_stride, pt, in.k_pe_token_stride, nk - t * BN);
            sv.load_rows(tid, vt, in.v_token_stride, nk - t * BN);
        } else {
            direct_k.fetch(wave, kt, pt, to);
            direct_v.fetch(wave, vt, to + BN * DQK);
        }
    };
    auto store = [&](auto hides, E* to) {
        if constexpr (hides) {
            move_bad_rows(tid, sk, sv);
            sk.store(tid, to);
            sv.store(tid, to + BN * DQK);
        } else {
            landed();
        }
    };
    RowReader<E, DQK> k_rows(lane);
    RowReader<E, DV> v_rows(lane);
    ColReader<E, DQK, DQK / 16> k_cols(lane);

    f32x4 acc[NQ][DQK / 16];
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int c = 0; c < DQK / 16; ++c) acc[j][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (tb < nt) {
        load(tb, Int<1>(), even);
        store(Int<1>(), even);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int ks = 0; ks < QR; ++ks) arrived(q[j][ks]);
    // A row that sees no key has o = 0, and 0 times a d_o of NaN or Inf is NaN.
    // (Where delta is summed the test costs two spilled registers, 2 % of the
    // packed training step.)
    if (wave_full <= 0)
#pragma unroll
        for (int j = 0; j < NQ; ++j)
            if (lse2[j] == neg_inf()) dl[j] = 0.f;
    // Tile t of the keys; hides: some row does not see all of the keys of it or
    // of the next one.
    auto step = [&](int t, auto hides, const E* K, E* next) {
        k_rows.keep(), v_rows.keep(), k_cols.keep();
        const E* V = K + BN * DQK;
        if (t + 1 < nt) load(t + 1, hides, next);
        if (t * BN < wave_end) {
            f32x4 s[NQ][TT], dp[NQ][TT];
            v8 x[PD + 1];
#pragma unroll
            for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                for (int j = 0; j < NQ; ++j) s[j][tt] = dp[j][tt] = f32x4{0.f, 0.f, 0.f, 0.f};
            // One sequence of operands, read ahead across its parts: z = q k^T;
            // g v^T, between whose products the weights' exponentials run; and,
            // after dz, dq^T += K^T dz.
            constexpr int E0 = TT * KS, E1 = E0 + TT * VS, NS = NQ * TT * 4;
            v8 y[2][NQ], dz[NQ];
            auto row_grads = [&](int vs) {   // (or q's last block, into y[1])
#pragma unroll
                for (int j = 0; j < NQ; ++j) y[vs == VS ? 1 : vs & 1][j] = load_frag(sgo[wave][j][vs], lane);
            };
            ahead<E1 + DQK / 16, PD>(
                [&](auto n) {
                    constexpr int e = n;
                    x[e % (PD + 1)] = e < E0   ? k_rows(K, 16 * (e % TT), e / TT)
                                      : e < E1 ? v_rows(V, 16 * ((e - E0) % TT), (e - E0) / TT)
                                               : k_cols(K, 0, 16, e - E1);
                },
                [&](auto n) {
                    constexpr int e = n;
                    if constexpr (e < E0) {
                        constexpr int ks = e / TT;
                        if (QL && e == E0 - 2 * TT) row_grads(VS);
                        if (e == E0 - TT) row_grads(0);
#pragma unroll
                        for (int j = 0; j < NQ; ++j) {
                            if constexpr (ks < QR) s[j][e % TT] = mma32(x[e % (PD + 1)], q[j][ks], s[j][e % TT]);
                            else s[j][e % TT] = mma32(x[e % (PD + 1)], y[1][j], s[j][e % TT]);
                        }
                    } else if constexpr (e < E1) {
                        constexpr int f = e - E0;
                        if (f % TT == 0 && f / TT + 1 < VS) row_grads(f / TT + 1);
#pragma unroll
                        for (int j = 0; j < NQ; ++j) dp[j][f % TT] = mma32(x[e % (PD + 1)], y[f / TT & 1][j], dp[j][f % TT]);
#pragma unroll
                        for (int m = NS * f / (TT * VS); m < NS * (f + 1) / (TT * VS); ++m) {
                            const int j = m / (TT * 4), tt = m / 4 % TT, i = m % 4;
                            s[j][tt][i] = exp2_fast(__builtin_fmaf(s[j][tt][i], sc, -lse2[j]));
                        }
                    } else {
                        if (e == E1) {
                            if (hides && (t + 1) * BN > wave_full) {   // weights of hidden keys
#pragma unroll
                                for (int j = 0; j < NQ; ++j) {
                                    const int last = in.causal ? min(nk - 1, wrow + 16 * j + col + off) : nk - 1;
#pragma unroll
                                    for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                                        for (int i = 0; i < 4; ++i)
                                            if (t * BN + 16 * tt + 4 * g + i > last) s[j][tt][i] = 0.f, dp[j][tt][i] = 0.f;
                                }
                            }
#pragma unroll
                            for (int j = 0; j < NQ; ++j) {
#pragma unroll
                                for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                                    for (int i = 0; i < 4; ++i) {
                                        exact[j] += s[j][tt][i] * dp[j][tt][i];
                                        s[j][tt][i] *= dp[j][tt][i] - dl[j];
                                    }
                                dz[j] = acc_frag(s[j][0], s[j][1], E());
                            }
                        }
                        constexpr int c = e - E1;
#pragma unroll
                        for (int j = 0; j < NQ; ++j) acc[j][c] = mma32(x[e % (PD + 1)], dz[j], acc[j][c]);
                    }
                });
        }
        if (t + 1 < nt) store(hides, next);
        __syncthreads();
    };
    const int full = in.causal ? min(nk, tile * BQ + off + 1) : nk;   // keys all the workgroup's rows see
    const int td = min(full / BN - 1, nt);                             // tiles up to here are seen whole
    direct_k.rows(tid, in.k_token_stride, in.k_pe_token_stride, BN);
    direct_v.rows(tid, in.v_token_stride, BN);
    int t = tb;
    for (; t + 1 < td; t += 2) {
        step(t, Int<0>(), even, odd);
        step(t + 1, Int<0>(), odd, even);
    }
    if (t < td) step(t++, Int<0>(), even, odd);
    for (; t < nt; ++t) step(t, Int<1>(), (t - tb) & 1 ? odd : even, (t - tb) & 1 ? even : odd);
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = wrow + 16 * j + col;
        const float sum = group_sum(exact[j]);
        if (r >= nq) continue;
        if (g == 0) {
            float* stats = row_stats + 2 * ((int64_t)h * in.total_q + q0 + r);
            stats[0] = lse2[j];
            stats[1] = SPLIT<E> && gridDim.y > 1 ? dl[j] : sum;
        }
        if (SPLIT<E> && gridDim.y > 1) {
            float* to = part + (((int64_t)blockIdx.y * in.total_q + q0 + r) * in.H + h) * DQK + 4 * g;
#pragma unroll
            for (int c = 0; c < DQK / 16; ++c) store_vec(to + 16 * c, acc[j][c] * in.scale);
            continue;
        }
        E* row = dq + ((int64_t)(q0 + r) * in.H + h) * DQK;
#pragma unroll
        for (int c = 0; c < DQK / 16; ++c) {
            typename Vec<E>::v4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = from_f32<E>(acc[j][c][i] * in.scale);
            store_vec(row + 16 * c + 4 * g, x);
        }
    }
}

// dk, dv and the head's part of dk_pe.  A wave owns 16 keys, whose k and v
// operands and gradients stay in registers; the query rows come 32 at a time.
// The scores are formed with rows = queries, so that the weights and dz are the
// operands of dv^T += g^T w and dk^T += q^T dz as they stand.  The same batch:
// 2.42 ms, 0.90 PFLOP/s.  Without its loads 2.1 ms, without LDS reads as well 1.9:
// the rest is the products.  Also measured: 32 keys a wave with one wave a SIMD
// 3.5 ms; 32 keys to two waves that share the channels, which halves the LDS
// reads, the same time; 128 keys a workgroup of 8 waves 2.84 (against 2.86).
template <typename E, int DN, int DR>
__global__ __launch_bounds__(256, sizeof(E) == 2 ? 2 : 1) void latent_dkv_kernel(
    const kda_latent_inputs in, const E* __restrict__ d_o, const float* __restrict__ row_stats,
    E* __restrict__ dk, int64_t dk_token_stride, int64_t dk_head_stride,
    E* __restrict__ dv, int64_t dv_token_stride, int64_t dv_head_stride, float* __restrict__ pe_part,
    float* __restrict__ part, int tiles)
{
    constexpr int DQK = DN + DR, DV = DN, BQ = 32, BK = 64;
    constexpr int KS = DQK / 32, VS = DV / 32, PD = sizeof(E) == 2 ? 3 : 1;
    typedef typename Vec<E>::v8 v8;
    // two arrays, so that a read of one is seen not to wait for loads into the other
    __shared__ __attribute__((aligned(16))) E even[BQ * (DQK + DV)];
    __shared__ __attribute__((aligned(16))) E odd[BQ * (DQK + DV)];
    __shared__ __attribute__((aligned(16))) float srow[2][2 * BQ];   // lse (base 2), then delta

    int h, want, seq, tile;
    head_tile_of_block(in.H, tiles, h, want);
    const int32_t* cu_k = in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q;
    const int rows_k = (int)(in.total_k / in.num_seqs);
    if (!find_tile<BK, 256>(cu_k, in.num_seqs, rows_k, (int)in.total_k, want, reinterpret_cast<int*>(even), seq,
                            tile))
        return;
    int q0, q1, k0, k1;
    sequence_rows(in.cu_seqlens_q, (int)(in.total_q / in.num_seqs), (int)in.total_q, seq, q0, q1);
    sequence_rows(cu_k, rows_k, (int)in.total_k, seq, k0, k1);
    const int nq = q1 - q0, nk = k1 - k0, off = nk - nq;
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int key0 = tile * BK, wkey = key0 + 16 * wave;
    const float sc = in.scale * LOG2E;

    v8 k[KS], v[VS];
    {
        const int64_t row = k0 + min(wkey + col, nk - 1);
        const E* kp = (const E*)in.k + row * in.k_token_stride + h * in.k_head_stride;
        const E* vp = (const E*)in.v + row * in.v_token_stride + h * in.v_head_stride;
        const E* pp = DR ? (const E*)in.k_pe + row * in.k_pe_token_stride : nullptr;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks)
            k[ks] = 32 * ks < DN ? row_frag_global(kp, ks, lane) : row_frag_global(pp, ks - DN / 32, lane);
#pragma unroll
        for (int vs = 0; vs < VS; ++vs) v[vs] = row_frag_global(vp, vs, lane);
    }
    const int all = (nq + BQ - 1) / BQ;
    const int first = in.causal ? min(all, max(0, key0 - off) / BQ) : 0;   // rows before it see none of the keys
    // the row tiles of this split (fp32)
    const int t0 = SPLIT<E> ? first + (int)((int64_t)(all - first) * blockIdx.y / gridDim.y) : first;
    const int nt = SPLIT<E> ? first + (int)((int64_t)(all - first) * (blockIdx.y + 1) / gridDim.y) : all;
    // first row tile whose rows see all of the workgroup's keys
    const int th = in.causal ? max(t0, min(nt, (key0 + BK - 1 - off + BQ - 1) / BQ)) : t0;
    // tile t lies in even or odd by its distance from th
    auto parity = [&](int t) { return (t - th) & 1; };

    const E* qp = (const E*)in.q + (int64_t)q0 * in.q_token_stride + h * in.q_head_stride;
    const E* gp = d_o + ((int64_t)q0 * in.H + h) * DV;
    typedef Stage<E, DQK, BQ, 256> SQ;
    SQ sq;
    Stage<E, DV, BQ, 256> sg;
    static_assert(SQ::P == 1 && SQ::TPR == 8, "a row per 8 threads");
    // lse and delta of a row travel with one thread: where all keys are seen the
    // first BQ threads (few and whole lines to load), else the row's own first
    // thread, which knows whether the row is finite.
    const float* stats = row_stats + 2 * ((int64_t)h * in.total_q + q0);
    float next_lse = 0.f, next_delta = 0.f;
    auto carried = [&](bool hides) { return !hides ? tid : tid % SQ::TPR == 0 ? tid / SQ::TPR : BQ; };
    auto load_stats = [&](int t, bool hides) {
        if (carried(hides) < BQ) {   // rows behind the last weigh nothing: lse = inf
            const int i = t * BQ + carried(hides);
            const float* at = stats + 2 * (int64_t)min(i, nq - 1);
            next_lse = i < nq ? at[0] : __builtin_inff();
            next_delta = i < nq ? at[1] : 0.f;
        }
    };
    auto store_stats = [&](int t, bool hides) {
        if (carried(hides) < BQ) {
            srow[parity(t)][carried(hides)] = next_lse;
            srow[parity(t)][BQ + carried(hides)] = next_delta;
        }
    };
    // Tiles of rows that all see all of the keys go straight to LDS (2.84 -> 2.42
    // ms); the others through registers, where rows that are not finite are found
    // and taken out.
    Direct<E, DQK, BQ, 256> direct_q;
    Direct<E, DV, BQ, 256> direct_g;
    auto load = [&](int t, auto hides, E* to) {
        const E* qt = qp + (int64_t)t * BQ * in.q_token_stride;
        const E* gt = gp + (int64_t)t * BQ * in.H * DV;
        load_stats(t, hides);
        if constexpr (hides) {
            sq.load_rows(tid, qt, in.q_token_stride, nq - t * BQ);
            sg.load_rows(tid, gt, (int64_t)in.H * DV, nq - t * BQ);
        } else {
            if (nq - t * BQ < BQ) {
                direct_q.rows(tid, in.q_token_stride, nq - t * BQ - 1);
                direct_g.rows(tid, (int64_t)in.H * DV, nq - t * BQ - 1);
            }
            direct_q.fetch(wave, qt, to);
            direct_g.fetch(wave, gt, to + BQ * DQK);
        }
    };
    auto store = [&](int t, auto hides, E* to) {
        if constexpr (hides) {
            const bool bad_delta = carried(hides) < BQ && !(__builtin_fabsf(next_delta) < __builtin_inff());
            if (sq.bad_row(tid, 0) | sg.bad_row(tid, 0, bad_delta)) {   // as move_bad_rows: lse becomes NaN
                sq.fill_row(0, 0u);
                sg.fill_row(0, 0u);
                next_lse = __builtin_nanf("");
                next_delta = 0.f;
            }
            sq.store(tid, to);
            sg.store(tid, to + BQ * DQK);
            store_stats(t, hides);
        } else {
            store_stats(t, hides);
            landed();
        }
    };

    RowReader<E, DQK> q_rows(lane);
    RowReader<E, DV> g_rows(lane);
    ColReader<E, DQK, DQK / 16> q_cols(lane);
    ColReader<E, DV, DV / 16> g_cols(lane);
    f32x4 ak[DQK / 16], av[DV / 16];
#pragma unroll
    for (int c = 0; c < DQK / 16; ++c) ak[c] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < DV / 16; ++c) av[c] = f32x4{0.f, 0.f, 0.f, 0.f};
    if (t0 < nt) {
        E* to = parity(t0) ? odd : even;
        load(t0, Int<1>(), to);
        store(t0, Int<1>(), to);
    }
    __syncthreads();
#pragma unroll
    for (int ks = 0; ks < KS; ++ks) arrived(k[ks]);
#pragma unroll
    for (int vs = 0; vs < VS; ++vs) arrived(v[vs]);
    // Tile t of the rows; hides: some row of it does not see all of the keys.
    auto step = [&](int t, auto hides, const E* Q, E* next) {
        q_rows.keep(), g_rows.keep(), q_cols.keep(), g_cols.keep();
        const E* G = Q + BQ * DQK;
        const float* R = srow[parity(t)];
        const int row0 = t * BQ;
        if (t + 1 < nt) load(t + 1, hides, next);
        if (!hides || row0 + BQ - 1 + off >= wkey) {
            f32x4 s[2], dp[2];
            v8 x[PD + 1];
#pragma unroll
            for (int a = 0; a < 2; ++a) s[a] = dp[a] = f32x4{0.f, 0.f, 0.f, 0.f};
            const f32x4 ls[2] = {*reinterpret_cast<const f32x4*>(R + 4 * g), *reinterpret_cast<const f32x4*>(R + 16 + 4 * g)};
            const f32x4 de[2] = {*reinterpret_cast<const f32x4*>(R + BQ + 4 * g),
                                 *reinterpret_cast<const f32x4*>(R + BQ + 16 + 4 * g)};
            // One sequence of operands, read ahead across its parts: z = q k^T;
            // g v^T, between whose products the weights' exponentials run;
            // dv^T += g^T w, between whose products dz is formed; dk^T += q^T dz.
            constexpr int E0 = 2 * KS, E1 = E0 + 2 * VS, E2 = E1 + DV / 16, NS = 8;
            v8 wf, zf;
            ahead<E2 + DQK / 16, PD>(
                [&](auto n) {
                    constexpr int e = n;
                    x[e % (PD + 1)] = e < E0   ? q_rows(Q, 16 * (e % 2), e / 2)
                                      : e < E1 ? g_rows(G, 16 * ((e - E0) % 2), (e - E0) / 2)
                                      : e < E2 ? g_cols(G, 0, 16, e - E1)
                                               : q_cols(Q, 0, 16, e - E2);
                },
                [&](auto n) {
                    constexpr int e = n;
                    const v8& a = x[e % (PD + 1)];
                    if constexpr (e < E0) {
                        s[e % 2] = mma32(a, k[e / 2], s[e % 2]);
                    } else if constexpr (e < E1) {
                        constexpr int f = e - E0;
                        dp[f % 2] = mma32(a, v[f / 2], dp[f % 2]);
#pragma unroll
                        for (int i = NS * f / (2 * VS); i < NS * (f + 1) / (2 * VS); ++i)
                            s[i / 4][i % 4] = exp2_fast(__builtin_fmaf(s[i / 4][i % 4], sc, -ls[i / 4][i % 4]));
                    } else if constexpr (e < E2) {
                        constexpr int c = e - E1;
                        if (c == 0) {
                            if (hides && row0 + off < wkey + 15) {   // weights of hidden keys
#pragma unroll
                                for (int i = 0; i < 8; ++i)
                                    if (wkey + col > row0 + 16 * (i / 4) + 4 * g + i % 4 + off)
                                        s[i / 4][i % 4] = 0.f, dp[i / 4][i % 4] = 0.f;
                            }
                            wf = acc_frag(s[0], s[1], E());
                        }
                        av[c] = mma32(a, wf, av[c]);
#pragma unroll
                        for (int i = NS * c / (DV / 16); i < NS * (c + 1) / (DV / 16); ++i)
                            dp[i / 4][i % 4] = s[i / 4][i % 4] * (dp[i / 4][i % 4] - de[i / 4][i % 4]);
                    } else {
                        constexpr int c = e - E2;
                        if (c == 0) zf = acc_frag(dp[0], dp[1], E());
                        ak[c] = mma32(a, zf, ak[c]);
                    }
                });
        }
        if (t + 1 < nt) store(t + 1, hides, next);
        __syncthreads();
    };
    int t = t0;
    for (; t < th; ++t) step(t, Int<1>(), parity(t) ? odd : even, parity(t) ? even : odd);
    direct_q.rows(tid, in.q_token_stride, BQ);
    direct_g.rows(tid, (int64_t)in.H * DV, BQ);
    for (; t + 1 < nt; t += 2) {
        step(t, Int<0>(), even, odd);
        step(t + 1, Int<0>(), odd, even);
    }
    if (t < nt) step(t, Int<0>(), even, odd);
    const int key = wkey + col;
    if (key >= nk) return;
    const int64_t row = k0 + key;
    if (SPLIT<E> && gridDim.y > 1) {
        float* to = part + (((int64_t)blockIdx.y * in.total_k + row) * in.H + h) * (DQK + DV) + 4 * g;
#pragma unroll
        for (int c = 0; c < DQK / 16; ++c) store_vec(to + 16 * c, ak[c] * in.scale);
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) store_vec(to + DQK + 16 * c, av[c]);
        return;
    }
    E* kr = dk + row * dk_token_stride + h * dk_head_stride;
    E* vr = dv + row * dv_token_stride + h * dv_head_stride;
#pragma unroll
    for (int c = 0; c < DN / 16; ++c) {
        typename Vec<E>::v4 kx, vx;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            kx[i] = from_f32<E>(ak[c][i] * in.scale);
            vx[i] = from_f32<E>(av[c][i]);
        }
        store_vec(kr + 16 * c + 4 * g, kx);
        store_vec(vr + 16 * c + 4 * g, vx);
    }
    if constexpr (DR > 0) {
        float* pr = pe_part + (row * in.H + h) * DR;
#pragma unroll
        for (int c = 0; c < DR / 16; ++c) store_vec(pr + 16 * c + 4 * g, ak[DN / 16 + c] * in.scale);
    }
}

// dk_pe = sum over the heads in order, fp32, rounded once.  A thread per 4
// channels of a key; rows behind the last sequence are left alone.
template <typename E, int DR>
__global__ __launch_bounds__(256) void latent_dkpe_kernel(const float* __restrict__ part, E* __restrict__ dk_pe,
                                                          const int32_t* __restrict__ cu, int N, int total, int H)
{
    const int64_t id = block_of_grid() * 256 + threadIdx.x;
    const int64_t row = id / (DR / 4);
    const int c = 4 * (int)(id % (DR / 4));
    const int first = cu ? clamp_offset(cu[0], total) : 0, last = cu ? clamp_offset(cu[N], total) : total;
    if (row < first || row >= last) return;
    const float* p = part + row * H * DR + c;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int h = 0; h < H; ++h) sum += *reinterpret_cast<const f32x4*>(p + (int64_t)h * DR);
    typename Vec<E>::v4 x;
#pragma unroll
    for (int i = 0; i < 4; ++i) x[i] = from_f32<E>(sum[i]);
    store_vec(dk_pe + row * DR + c, x);
}

// The splits' sums: dk, dv and dk_pe (over the heads too) of a key, dq of a query.
// A thread per 4 channels.
template <typename E, int DN, int DR>
__global__ __launch_bounds__(256) void latent_sum_kernel(const kda_latent_inputs in, const LatentGrads a, int splits_k,
                                                         int splits_q)
{
    constexpr int DQK = DN + DR, DV = DN, KC = (DN + DV) / 4, QC = DQK / 4;
    int64_t id = block_of_grid() * 256 + threadIdx.x;
    const int64_t per_key = splits_k > 1 ? in.H * KC + DR / 4 : 0, keys = in.total_k * per_key;
    const bool key = id < keys;
    if (!key) id -= keys;
    const int64_t per = key ? per_key : in.H * QC, total = key ? in.total_k : in.total_q, row = id / per;
    if (!key && (splits_q == 1 || row >= total)) return;
    const int j = (int)(id - row * per), splits = key ? splits_k : splits_q;
    const int32_t* cu = key && in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q;
    if (cu && (row < clamp_offset(cu[0], (int)total) || row >= clamp_offset(cu[in.num_seqs], (int)total))) return;
    f32x4 sum = {0.f, 0.f, 0.f, 0.f};
    E* to;
    if (!key || j < in.H * KC) {
        const int h = j / (key ? KC : QC), c = 4 * (j - h * (key ? KC : QC)), W = key ? DQK + DV : DQK;
        const float* from = (key ? a.part_k : a.part_q) + (row * in.H + h) * W + (key && c >= DN ? DR + c : c);
#pragma unroll 8
        for (int s = 0; s < splits; ++s) sum += *reinterpret_cast<const f32x4*>(from + s * total * in.H * W);
        to = !key     ? (E*)a.dq + (row * in.H + h) * DQK + c
             : c < DN ? (E*)a.dk + row * a.dk_token_stride + h * a.dk_head_stride + c
                      : (E*)a.dv + row * a.dv_token_stride + h * a.dv_head_stride + c - DN;
    } else {
        const int c = 4 * (j - in.H * KC);
        const float* from = a.part_k + row * in.H * (DQK + DV) + DN + c;
#pragma unroll 16
        for (int i = 0; i < splits * in.H; ++i)
            sum += *reinterpret_cast<const f32x4*>(from + (i / in.H * total * in.H + i % in.H) * (DQK + DV));
        to = (E*)a.dk_pe + row * DR + c;
    }
    store_vec(to, sum);
}

static int64_t tile_count(const int32_t* cu, int64_t total, int32_t N, int B) {
    return cu ? total / B + N : (total / N + B - 1) / B * N;
}

template <typename E, int DN, int DR>
static hipError_t launch(const kda_latent_inputs& in, const LatentGrads& a, hipStream_t stream) {
    const int64_t tq = tile_count(in.cu_seqlens_q, in.total_q, in.num_seqs, 64 * LATENT_NQ<E>);
    const int32_t* cu_k = in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q;
    const int64_t tk = tile_count(cu_k, in.total_k, in.num_seqs, 64);
    const int sq = SPLIT<E> ? latent_splits(in.total_q, in.H) : 1, sk = SPLIT<E> ? latent_splits(in.total_k, in.H) : 1;
    if (tq > 0)
        hipLaunchKernelGGL((latent_dq_kernel<E, DN, DR>), dim3((unsigned)(tq * in.H), sq), dim3(256), 0, stream, in,
                           (const E*)a.o, a.lse, (const E*)a.d_o, (E*)a.dq, a.row_stats, a.part_q, (int)tq);
    if (const hipError_t e = launch_result(stream)) return e;
    if (tk > 0)
        hipLaunchKernelGGL((latent_dkv_kernel<E, DN, DR>), dim3((unsigned)(tk * in.H), sk), dim3(256), 0, stream, in,
                           (const E*)a.d_o, a.row_stats, (E*)a.dk, a.dk_token_stride, a.dk_head_stride, (E*)a.dv,
                           a.dv_token_stride, a.dv_head_stride, a.pe_part, a.part_k, (int)tk);
    if (const hipError_t e = launch_result(stream)) return e;
    if constexpr (SPLIT<E>)
        if (sk > 1 || sq > 1) {
            const int64_t items = (sk > 1 ? in.total_k * (in.H * (2 * DN) / 4 + DR / 4) : 0) +
                                  (sq > 1 ? in.total_q * in.H * (DN + DR) / 4 : 0);
            hipLaunchKernelGGL((latent_sum_kernel<E, DN, DR>), grid_of((items + 255) / 256), dim3(256), 0, stream, in, a, sk, sq);
            if (const hipError_t e = launch_result(stream)) return e;
        }
    if constexpr (DR > 0)
        if (in.total_k > 0 && sk == 1) {
            hipLaunchKernelGGL((latent_dkpe_kernel<E, DR>), grid_of((in.total_k * (DR / 4) + 255) / 256), dim3(256), 0,
                               stream, a.pe_part, (E*)a.dk_pe, cu_k, in.num_seqs, (int)in.total_k, in.H);
            return launch_result(stream);
        }
    return hipSuccess;
}

hipError_t launch_latent_attention_backward(const kda_latent_inputs& in, const LatentGrads& a, hipStream_t stream) {
    if (in.dtype == KDA_DTYPE_BF16) {
        if (in.dn == 128) return in.dr ? launch<bf16, 128, 64>(in, a, stream) : launch<bf16, 128, 0>(in, a, stream);
        return in.dr ? launch<bf16, 64, 64>(in, a, stream) : launch<bf16, 64, 0>(in, a, stream);
    }
    if (in.dn == 128) return in.dr ? launch<float, 128, 64>(in, a, stream) : launch<float, 128, 0>(in, a, stream);
    return in.dr ? launch<float, 64, 64>(in, a, stream) : launch<float, 64, 0>(in, a, stream);
}

}  // namespace kda
