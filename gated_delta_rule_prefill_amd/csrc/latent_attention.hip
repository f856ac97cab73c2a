// latent_attention.hip -- expanded latent attention, forward.
//
// For a sequence with n queries and m keys, per head (scale > 0):
//   z_ij = scale (q_i . [k_j, k_pe_j]), j <= i + (m - n) when causal
//   o_i  = sum_j exp(z_ij - z_max) v_j / sum_j exp(z_ij - z_max)
// in one pass over the keys with the running maximum and sum.  The scores of a
// tile are formed transposed, S^T = K Q^T (rows = keys), so that a lane holds
// 4 neighbouring keys of one query row: as they stand, exponentiated, they are
// the operand of O^T += V^T P^T, whose other operand is V read by columns.
// Scores and weights never leave the registers, and the row's maximum, sum and
// rescale factor are one value per lane.
#include "latent_common.h"

namespace kda {

// The values that the kernel below took out of tile 0 and of those that some row
// of the workgroup does not see whole, found again: per channel the first key
// with Inf or NaN and the first with -Inf or NaN.  Weights of keys that a row sees
// are above 0, so it takes the one, the other or NaN, whatever its other keys add
// and thus behind the output's rounding.  It reads the values of those tiles once
// more: 8 rows of 2,048 tokens x 32 heads, 128 + 64 channels, padded with NaN from
// 1,500 on 456 us (436 with finite padding), from 1 on 505; 64 rows of 256 padded
// from 100 on 265 (166).  (With each key's weight worked out as well: 10.7 ms,
// 48 ms and 28 ms.)
template <typename E, int DN, int DR>
__device__ __forceinline__ void put_taken(E* o, int h, int seq, int tile, int* first /* [2][DN] in LDS */)
{
    constexpr int DV = DN, BN = 128 / (int)sizeof(E), NQ = LATENT_NQ<E>, BQ = 64 * NQ;
    constexpr int CE = CHUNK_ELEMS<E>, CH = DV / CE, PASS = 256 / CH, NONE = 0x7fffffff;
    typedef E vec __attribute__((ext_vector_type(CE)));
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    // The inputs are read from the kernel's first argument again, and nothing of this
    // is worked out ahead of the walk, whose registers are short.
    int tid = threadIdx.x;
    auto args = (const __attribute__((address_space(4))) kda_latent_inputs*)__builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+v"(tid), "+s"(args));
    const auto& in = *args;
    int q0, q1, k0, k1;
    sequence_rows(in.cu_seqlens_q, (int)(in.total_q / in.num_seqs), (int)in.total_q, seq, q0, q1);
    sequence_rows(in.cu_seqlens_k ? in.cu_seqlens_k : in.cu_seqlens_q, (int)(in.total_k / in.num_seqs),
                  (int)in.total_k, seq, k0, k1);
    const int nq = q1 - q0, nk = k1 - k0, off = nk - nq;
    const int full = in.causal ? min(nk, tile * BQ + off + 1) : nk;   // as in the kernel
    const int end = in.causal ? min(nk, min(nq, (tile + 1) * BQ) + off) : nk;

    for (int i = tid; i < 2 * DV; i += 256) first[i] = NONE;
    __syncthreads();
    int up[CE], down[CE];
#pragma unroll
    for (int e = 0; e < CE; ++e) up[e] = down[e] = NONE;
    const int behind = max(BN, full / BN * BN);   // first key behind the tiles that are seen whole
    const E* v = (const E*)in.v + (int64_t)k0 * in.v_token_stride + h * in.v_head_stride + tid % CH * CE;
    const int count = min(end, BN) + max(0, end - behind);
    for (int i = tid / CH; i < count; i += 4 * PASS) {
        vec x[4];
        int key[4];
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            const int at = min(i + n * PASS, count - 1);
            key[n] = at < BN ? at : at - BN + behind;
            x[n] = *reinterpret_cast<const vec*>(v + (int64_t)key[n] * in.v_token_stride);
        }
#pragma unroll
        for (int n = 0; n < 4; ++n)
#pragma unroll
            for (int e = 0; e < CE; ++e) {
                if (!(to_f32(x[n][e]) < __builtin_inff())) up[e] = min(up[e], key[n]);
                if (!(to_f32(x[n][e]) > neg_inf())) down[e] = min(down[e], key[n]);
            }
    }
#pragma unroll
    for (int e = 0; e < CE; ++e) {
        if (up[e] != NONE) atomicMin(first + tid % CH * CE + e, up[e]);
        if (down[e] != NONE) atomicMin(first + DV + tid % CH * CE + e, down[e]);
    }
    __syncthreads();
    const int col = tid & 15, g = tid >> 4 & 3;
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = tile * BQ + 16 * (NQ * (tid >> 6) + j) + col;
        const int last = in.causal ? min(nk - 1, r + off) : nk - 1;
        if (r >= nq) continue;
        E* row = o + ((int64_t)(q0 + r) * in.H + h) * DV;
#pragma unroll
        for (int c = 4 * g; c < DV; c += 16) {   // the channels that this lane has written
            const i32x4 u = *reinterpret_cast<const i32x4*>(first + c), d = *reinterpret_cast<const i32x4*>(first + DV + c);
            if (min(min(min(u[0], u[1]), min(u[2], u[3])), min(min(d[0], d[1]), min(d[2], d[3]))) > last) continue;
            typename Vec<E>::v4 x = load_vec<typename Vec<E>::v4>(row + c);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float y = to_f32(x[i]);
                if (u[i] <= last) y += __builtin_inff();
                if (d[i] <= last) y += neg_inf();
                x[i] = from_f32<E>(y);
            }
            store_vec(row + c, x);
        }
    }
}

// A workgroup: 4 waves of 32 (bf16) or 16 (fp32) query rows, whose operands q
// and o stay in registers, one head.  Key and value tiles of BN rows are
// double-buffered in LDS (80 KB, two workgroups a CU): the next tile's global
// loads are issued before a tile's products and stored to LDS behind them.
// Bound by the matrix products: 16,384 causal tokens x 32 heads, 128 + 64
// channels, bf16: 2.44 to 2.62 ms from card to card, 1.13 to 1.05 PFLOP/s, where a large
// library product reaches 1.15; documents of 256 to 4,096 tokens (36,755 in all) 1.16 ms.  fp32,
// 6 sequences of 1 to 130 tokens x 4 heads: 15 us, one row tile's walk over its keys.
template <typename E, int DN, int DR>
__global__ __launch_bounds__(256, 2) void latent_attention_kernel(
    const kda_latent_inputs in, E* __restrict__ o, float* __restrict__ lse, int tiles)
{
    constexpr int DQK = DN + DR, DV = DN, BN = 128 / (int)sizeof(E), NQ = LATENT_NQ<E>, BQ = 64 * NQ;
    constexpr int KS = DQK / 32, TT = BN / 16, PD = sizeof(E) == 2 ? 3 : 1;
    typedef typename Vec<E>::v8 v8;
    // two arrays, so that a read of one is seen not to wait for loads into the other
    __shared__ __attribute__((aligned(16))) E even[BN * (DQK + DV)];
    __shared__ __attribute__((aligned(16))) E odd[BN * (DQK + DV)];

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
    const int wrow = tile * BQ + 16 * NQ * wave;   // the wave's first row in the sequence
    const float sc = in.scale * LOG2E;

    const E* kp = (const E*)in.k + (int64_t)k0 * in.k_token_stride + h * in.k_head_stride;
    const E* vp = (const E*)in.v + (int64_t)k0 * in.v_token_stride + h * in.v_head_stride;
    const E* pp = DR ? (const E*)in.k_pe + (int64_t)k0 * in.k_pe_token_stride : nullptr;

    // this lane's query rows, and the last key each sees
    v8 q[NQ][KS];
    int last[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = wrow + 16 * j + col;
        const E* row = (const E*)in.q + (int64_t)(q0 + min(r, nq - 1)) * in.q_token_stride + h * in.q_head_stride;
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) q[j][ks] = row_frag_global(row, ks, lane);
        last[j] = in.causal ? min(nk - 1, r + off) : nk - 1;
    }
    const int end = in.causal ? min(nk, min(nq, (tile + 1) * BQ) + off) : nk;   // keys of the workgroup
    const int nt = end > 0 ? (end + BN - 1) / BN : 0;
    const int wave_end = in.causal ? min(nk, min(nq, wrow + 16 * NQ) + off) : nk;           // of the wave
    const int wave_full = in.causal ? min(nk, wrow + off + 1) : nk;                    // keys all its rows see

    Stage<E, DQK, BN, 256> sk;
    Stage<E, DV, BN, 256> sv;
    // Tiles that all rows see whole go straight to LDS (2.48 -> 2.38 ms for 16,384
    // tokens); the others through registers, where values that are not finite are
    // taken out: a hidden key's weight is 0, and 0 times NaN or Inf is NaN.  What
    // they give the rows that see them follows the outputs (put_taken).
    unsigned long long taken = 0;
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
#pragma unroll
            for (int p = 0; p < decltype(sv)::P; ++p) {
                const bool bad = sv.bad_row(tid, p);
                if (bad) sv.clear_bad(p);
                taken |= __ballot(bad);
            }
            sk.store(tid, to);
            sv.store(tid, to + BN * DQK);
        } else {
            landed();
        }
    };
    RowReader<E, DQK> k_rows(lane);
    ColReader<E, DV, DV / 16> v_cols(lane);

    f32x4 acc[NQ][DV / 16];
    float m[NQ], l[NQ];
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        m[j] = neg_inf();
        l[j] = 0.f;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) acc[j][c] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if (nt > 0) {
        load(0, Int<1>(), even);
        store(Int<1>(), even);
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < NQ; ++j)
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) arrived(q[j][ks]);
    // Tile t of the keys; hides: some row does not see all of the keys of it or
    // of the next one.
    auto step = [&](int t, auto hides, const E* K, E* next) {
        k_rows.keep(), v_cols.keep();
        const E* V = K + BN * DQK;
        if (t + 1 < nt) load(t + 1, hides, next);
        if (t * BN < wave_end) {
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
            v8 p[NQ][TT / 2];
            auto take_weights = [&]() {
                if (hides && (t + 1) * BN > wave_full) {
#pragma unroll
                    for (int j = 0; j < NQ; ++j)
#pragma unroll
                        for (int tt = 0; tt < TT; ++tt)
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (t * BN + 16 * tt + 4 * g + i > last[j]) s[j][tt][i] = neg_inf();
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
                        for (int c = 0; c < DV / 16; ++c) acc[j][c] *= f;
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
                    for (int b = 0; b < TT / 2; ++b) p[j][b] = acc_frag(s[j][2 * b], s[j][2 * b + 1], E());
                }
            };
            ahead<E0 + DV / 16 * (TT / 2), PD>(
                [&](auto n) {
                    constexpr int e = n, f = e - E0;
                    if constexpr (e < E0) x[e % (PD + 1)] = k_rows(K, 16 * (e / (2 * KS) * 2 + e % 2), e / 2 % KS);
                    else x[e % (PD + 1)] = v_cols(V, 32 * (f / (DV / 16)), 32 * (f / (DV / 16)) + 16, f % (DV / 16));
                },
                [&](auto n) {
                    constexpr int e = n, f = e - E0;
                    if constexpr (e < E0) {
#pragma unroll
                        for (int j = 0; j < NQ; ++j)
                            s[j][e / (2 * KS) * 2 + e % 2] =
                                mma32(x[e % (PD + 1)], q[j][e / 2 % KS], s[j][e / (2 * KS) * 2 + e % 2]);
                    } else {
                        if constexpr (f == 0) take_weights();
#pragma unroll
                        for (int j = 0; j < NQ; ++j)
                            acc[j][f % (DV / 16)] = mma32(x[e % (PD + 1)], p[j][f / (DV / 16)], acc[j][f % (DV / 16)]);
                    }
                });
        }
        if (t + 1 < nt) store(hides, next);
        __syncthreads();
    };
    const int full = in.causal ? min(nk, tile * BQ + off + 1) : nk;   // keys all the workgroup's rows see
    const int td = full / BN - 1;                                      // tiles up to here are seen whole
    direct_k.rows(tid, in.k_token_stride, in.k_pe_token_stride, BN);
    direct_v.rows(tid, in.v_token_stride, BN);
    int t = 0;
    for (; t + 1 < td; t += 2) {
        step(t, Int<0>(), even, odd);
        step(t + 1, Int<0>(), odd, even);
    }
    if (t < td) step(t++, Int<0>(), even, odd);
    for (; t < nt; ++t) step(t, Int<1>(), t & 1 ? odd : even, t & 1 ? even : odd);
#pragma unroll
    for (int j = 0; j < NQ; ++j) {
        const int r = wrow + 16 * j + col;
        const float sum = group_sum(l[j]);
        if (r >= nq) continue;
        const float inv = sum == 0.f ? 0.f : 1.f / sum;
        E* row = o + ((int64_t)(q0 + r) * in.H + h) * DV;
#pragma unroll
        for (int c = 0; c < DV / 16; ++c) {
            typename Vec<E>::v4 x;
#pragma unroll
            for (int i = 0; i < 4; ++i) x[i] = from_f32<E>(acc[j][c][i] * inv);
            store_vec(row + 16 * c + 4 * g, x);
        }
        if (lse && g == 0)
            lse[(int64_t)(q0 + r) * in.H + h] = sum == 0.f ? neg_inf() : (m[j] + __log2f(sum)) * LN2;
    }
    int* any = reinterpret_cast<int*>(even);
    if (lane == 0) any[wave] = taken != 0;
    __syncthreads();
    if (uniform(any[0] | any[1] | any[2] | any[3])) put_taken<E, DN, DR>(o, h, seq, tile, reinterpret_cast<int*>(odd));
}

template <typename E, int DN, int DR>
static hipError_t launch(const kda_latent_inputs& in, void* o, float* lse, hipStream_t stream) {
    constexpr int BQ = 64 * LATENT_NQ<E>;
    const int64_t tiles = in.cu_seqlens_q ? in.total_q / BQ + in.num_seqs
                                          : (in.total_q / in.num_seqs + BQ - 1) / BQ * in.num_seqs;
    hipLaunchKernelGGL((latent_attention_kernel<E, DN, DR>), dim3((unsigned)(tiles * in.H)), dim3(256), 0, stream,
                       in, (E*)o, lse, (int)tiles);
    return launch_result(stream);
}

hipError_t launch_latent_attention(const kda_latent_inputs& in, void* o, float* lse, hipStream_t stream) {
    if (in.dtype == KDA_DTYPE_BF16) {
        if (in.dn == 128) return in.dr ? launch<bf16, 128, 64>(in, o, lse, stream) : launch<bf16, 128, 0>(in, o, lse, stream);
        return in.dr ? launch<bf16, 64, 64>(in, o, lse, stream) : launch<bf16, 64, 0>(in, o, lse, stream);
    }
    if (in.dn == 128) return in.dr ? launch<float, 128, 64>(in, o, lse, stream) : launch<float, 128, 0>(in, o, lse, stream);
    return in.dr ? launch<float, 64, 64>(in, o, lse, stream) : launch<float, 64, 0>(in, o, lse, stream);
}

}  // namespace kda
