// latent_decode.hip -- absorbed latent attention over a paged cache.
//
// Every head reads the same cached row [c_j, k_pe_j]; a (token, head) pair is
// one query row:
//   z_rj = scale (q_r . [c_j, k_pe_j]),  o_r = sum_j softmax(z_r)_j c_j
// so a sequence's n new tokens with H heads are n H rows against one matrix of
// keys whose first dl columns are also the values.  A cached row is fetched
// once per 16 RT query rows; with 32 rows and 576 channels that is 60 flop per
// byte and the cache's bytes bound the kernel, with 64 rows and more the
// matrix products do.
//
// A workgroup takes 16 RT query rows of one sequence and walks key tiles of BN
// rows through LDS.  The scores of a tile are formed transposed (rows = keys)
// and split over the waves by row tiles and keys; each wave puts its weights
// into LDS, and the product with the values is split over the waves by value
// columns, so that the output (16 RT x dl, fp32) is spread over the waves'
// registers.
//
// The work of a batch (row tiles x key tiles of every sequence, in order) is
// cut into equal runs, one for each workgroup, whatever the lengths: a run may
// end inside a row tile, whose partial results a second kernel joins.  The cut
// depends on the lengths only, so results are reproducible.
#include "latent_common.h"

namespace kda {

constexpr int DEC_RUNS = 256;   // one workgroup per CU (its LDS tiles take the CU)
constexpr int DEC_WAVES = 8;

// Shape of a workgroup: RT row tiles of 16, BN keys a tile.  Where a sequence
// has up to 32 rows the cache's bytes are the bound and 32 rows are taken (two
// workgroups a CU with 4 waves and 32 keys each read as fast but leave twice the
// partial results: 260 against 256 us for 256 sequences, 39 against 34 for one);
// with more rows 64, so that a cached row is fetched half as often.
template <int RT_, int BN_> struct DecodeShape {
    static constexpr int RT = RT_, BN = BN_, BM = 16 * RT_;
};
template <typename E> using DecodeFew = DecodeShape<2, 128 / (int)sizeof(E)>;
template <typename E> using DecodeMany = DecodeShape<4, 128 / (int)sizeof(E)>;

// A row tile whose keys several workgroups share: its output rows and the
// runs [first, last] that hold its partial results.
struct DecodeSplit {
    int64_t row;       // first output row (token * H + head)
    int32_t rows;      // 0: nothing to join
    int32_t first, last, pad;
};

// Workspace: splits, then the partials' (m, l) pairs, then their outputs; run b
// has two slots of partials: 2b for a row tile begun in an earlier run, 2b + 1
// for one that a later run goes on with.
struct DecodeSpace {
    DecodeSplit* split;   // [DEC_RUNS]
    float* ml;            // [2 DEC_RUNS][BM][2]
    float* o;             // [2 DEC_RUNS][BM][dl]
};
template <typename S> static size_t space_bytes(int dl) {
    return sizeof(DecodeSplit) * DEC_RUNS + (size_t)2 * DEC_RUNS * S::BM * (2 + dl) * 4;
}
template <typename S> static DecodeSpace space_of(void* ws) {
    DecodeSpace s;
    s.split = reinterpret_cast<DecodeSplit*>(ws);
    s.ml = reinterpret_cast<float*>(s.split + DEC_RUNS);
    s.o = s.ml + (size_t)2 * DEC_RUNS * S::BM * 2;
    return s;
}

// Work of sequence s: row tiles x key tiles (a sequence without keys counts
// one, so that its output rows are written).
template <int BM, int BN>
__device__ __forceinline__ void sequence_work(const LatentDecode& a, int rows_q, int s, int& q0, int& n, int& len,
                                              int& row_tiles, int& key_tiles) {
    int q1;
    sequence_rows(a.cu_seqlens, rows_q, (int)a.total_tokens, s, q0, q1);
    n = q1 - q0;
    const int64_t room = (int64_t)a.max_pages * a.page_size;
    len = max(0, (int)min((int64_t)a.seq_lens[s], room));
    row_tiles = (int)(((int64_t)n * a.H + BM - 1) / BM);
    key_tiles = max(1, (len + BN - 1) / BN);
}

// by_tile: split entries are indexed by row tile (their number is at most
// DEC_RUNS), otherwise by the run that begins the row tile.
template <typename E, int DL, int DR, typename Shape>
__global__ __launch_bounds__(64 * DEC_WAVES, 2) void latent_decode_kernel(const LatentDecode a, DecodeSpace ws,
                                                                          int by_tile, int entries)
{
    constexpr int RT = Shape::RT, NW = DEC_WAVES, BN = Shape::BN, BM = Shape::BM;
    constexpr int W = DL + DR, NT = 64 * NW, TT = BN / 16, KS = W / 32;
    constexpr int TG = NW / RT < TT ? NW / RT : TT;    // a wave's scores: one row tile and
    constexpr int TW = TT / TG;                        // TW key tiles (key group of TG)
    constexpr int CT = DL / 16 / NW;                   // 16-column value tiles of a wave
    constexpr int PS = BN + 16 / (int)sizeof(E);       // row stride of the weights
    // With 32 rows a cached row is read by one workgroup, mostly: kept out of the
    // caches 240 us for 256 sequences, else 258.  (With 64, where several row tiles
    // share them, 599 against 541 for a chunk.)  Measured on a cache of 1.2 GB: one
    // that the last-level cache holds, or pages that sequences share, are not.
    constexpr bool ONCE = RT == 2;
    constexpr bool QREG = sizeof(E) == 2;              // query rows in registers; fp32 rows would fill them
    typedef typename Vec<E>::v8 v8;
    typedef typename Vec<E>::v4 v4;
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    __shared__ __attribute__((aligned(16))) E tilebuf[2][BN * W];
    __shared__ __attribute__((aligned(16))) E sp[BM * PS];
    __shared__ __attribute__((aligned(16))) float stat[TG][BM];
    __shared__ __attribute__((aligned(16))) int ridx[4][BN];   // cache rows of the tiles' keys, -1: none
    __shared__ int gaps[4];                                    // whether a tile has keys without a row
    __shared__ int grown[4];                                   // whether a tile raised a row's maximum
    __shared__ int64_t found[4];
    __shared__ int64_t wsum[NW][2];

    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6), col = lane & 15, g = lane >> 4;
    const int rows_q = (int)(a.total_tokens / a.num_seqs);
    const float sc = a.scale * LOG2E;
    // Workgroups go round robin over the 8 XCDs: neighbouring runs, which read
    // the same sequence's keys, go to one XCD and its L2.
    const int run = (blockIdx.x & 7) * (DEC_RUNS / 8) + (blockIdx.x >> 3);

    // this workgroup's run of the batch's work: the sum over the sequences,
    // then the sequence its run begins in
    int64_t total = 0, units = 0;
    for (int s = tid; s < a.num_seqs; s += NT) {
        int q0, n, len, rt, kt;
        sequence_work<BM, BN>(a, rows_q, s, q0, n, len, rt, kt);
        total += (int64_t)rt * kt;
        units += rt;
    }
    const int64_t mine = total, my_units = units;
    int64_t incl = total, uincl = units;   // inclusive over the lanes; NT sequences or fewer: the prefix itself
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t up = __shfl_up(incl, d), uup = __shfl_up(uincl, d);
        if (lane >= d) incl += up, uincl += uup;
    }
    if (lane == 63) wsum[wave][0] = incl, wsum[wave][1] = uincl;
    if (tid == 0) found[0] = -1;
    __syncthreads();
    int64_t base = 0, ubase = 0;
    total = units = 0;
#pragma unroll
    for (int w = 0; w < NW; ++w) {
        if (w < wave) base += wsum[w][0], ubase += wsum[w][1];
        total += wsum[w][0], units += wsum[w][1];
    }
    total = uniform(total);
    const int64_t per = (total + DEC_RUNS - 1) / DEC_RUNS;
    const int64_t begin = per * run, stop = min(total, begin + per);
    if (!by_tile) {
        if (tid == 0) ws.split[run].rows = 0;
    } else if (run == 0) {
        for (int64_t i = units + tid; i < entries; i += NT) ws.split[i].rows = 0;
    }
    if (begin >= stop) return;
    if (a.num_seqs <= NT) {
        const int64_t excl = base + incl - mine;
        if (begin >= excl && begin < excl + mine) found[0] = tid, found[1] = excl, found[2] = ubase + uincl - my_units;
        __syncthreads();
    } else {
        int64_t before = 0, ubefore = 0;
        for (int s0 = 0; s0 < a.num_seqs; s0 += NT) {
            const int s = s0 + tid;
            int64_t x = 0, u = 0;
            if (s < a.num_seqs) {
                int q0, n, len, rt, kt;
                sequence_work<BM, BN>(a, rows_q, s, q0, n, len, rt, kt);
                x = (int64_t)rt * kt;
                u = rt;
            }
            int64_t xi = x, ui = u;
#pragma unroll
            for (int d = 1; d < 64; d <<= 1) {
                const int64_t up = __shfl_up(xi, d), uup = __shfl_up(ui, d);
                if (lane >= d) xi += up, ui += uup;
            }
            __syncthreads();
            if (lane == 63) wsum[wave][0] = xi, wsum[wave][1] = ui;
            __syncthreads();
            int64_t b = before, ub = ubefore;
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                if (w < wave) b += wsum[w][0], ub += wsum[w][1];
                before += wsum[w][0], ubefore += wsum[w][1];
            }
            const int64_t excl = b + xi - x;
            if (begin >= excl && begin < excl + x) found[0] = s, found[1] = excl, found[2] = ub + ui - u;
            __syncthreads();
            if (uniform(found[0]) >= 0) break;
        }
    }
    int seq = (int)uniform(found[0]);
    int64_t seq_base = uniform(found[1]), unit_base = uniform(found[2]);

    const int rt = wave % RT, tg = wave / RT;      // row tile and key group of this wave's scores
    const bool scores = tg < TG;
    const E* cache = (const E*)a.cache;
    Stage<E, W, BN, NT> st;
    const RowReader<E, W> k_rows(lane);
    const ColReader<E, W, CT> c_cols(lane, wave * CT);

    for (int64_t pos = begin; pos < stop;) {
        int q0, n, len, row_tiles, key_tiles;
        sequence_work<BM, BN>(a, rows_q, seq, q0, n, len, row_tiles, key_tiles);
        if (pos >= seq_base + (int64_t)row_tiles * key_tiles) {   // behind this sequence (or it has no rows)
            seq_base += (int64_t)row_tiles * key_tiles;
            unit_base += row_tiles;
            ++seq;
            continue;
        }
        const int unit = (int)((pos - seq_base) / key_tiles), t0 = (int)((pos - seq_base) - (int64_t)unit * key_tiles);
        const int t1 = (int)min((int64_t)key_tiles, t0 + (stop - pos));
        const int64_t rows_all = (int64_t)n * a.H;
        const int64_t row0 = (int64_t)unit * BM;                     // first query row within the sequence
        const int nrows = (int)min((int64_t)BM, rows_all - row0);
        // keys that the tile's last row sees; key tiles behind them weigh nothing
        const int end = max(0, min(len, len - n + (int)((row0 + nrows - 1) / a.H) + 1));
        const int te = min(t1, (end + BN - 1) / BN);
        const int32_t* table = a.block_table + (int64_t)seq * a.max_pages;

        // Whole row tiles take their keys in a rotation that starts where the
        // run stands, so that workgroups of an XCD that work on different rows
        // of one sequence read the same keys at the same time, through its L2.
        const bool whole = t0 == 0 && t1 == key_tiles;
        const int count = max(0, te - t0), turn = whole && count > 0 ? (int)((pos - begin) % count) : 0;
        auto tile_of = [&](int k) { return t0 + (turn + k < count ? turn + k : turn + k - count); };   // k < count

        auto cache_row = [&](int k) -> int {                         // of the piece's tile k, key tid < BN
            if (k >= count) return -1;
            const int j = tile_of(k) * BN + tid;
            if (j >= len) return -1;
            const int pg = (int)((unsigned)j / (unsigned)a.page_size);
            const int page = table[pg];
            return page < 0 || page >= a.num_pages ? -1 : page * a.page_size + (j - pg * a.page_size);
        };
        auto row_of = [&](int k) {                                   // of the piece's tile k
            return [&, k](int r) {
                const int row = ridx[k & 3][r];
                return row < 0 ? zero_row<E>() : cache + (int64_t)row * W;
            };
        };
        auto keep_row = [&](int k, int row) {                        // tid < BN
            ridx[k & 3][tid] = row;
            const bool gap = __any(row < 0);
            if (tid == 0) gaps[k & 3] = gap;
        };
        if (tid < BN) {
            const int r0 = cache_row(0), r1 = cache_row(1), r2 = cache_row(2);
            keep_row(0, r0);
            keep_row(1, r1);
            keep_row(2, r2);
        }
        if (tid < 4) grown[tid] = 0;
        __syncthreads();
        int next_row = -1;
        // Rows with latents that are not finite, in tiles that hold keys some query
        // rows do not see: cleared, and marked -2 for those that do (their weight
        // becomes NaN; a weight of 0 would make 0 * NaN of a hidden key).  The key
        // part is in no product with weights: it gives the scores that it gives.
        const int first_last = len - n + (int)(row0 / a.H);          // last key that the tile's first row sees
        auto hides = [&](int k) { return (tile_of(k) + 1) * BN - 1 > first_last; };
        auto mark_bad_rows = [&](Stage<E, W, BN, NT>& rows, int k) {
            typedef Stage<E, W, BN, NT> S;
#pragma unroll
            for (int p = 0; p < S::P; ++p)
                if (rows.template bad_row<DR>(tid, p)) {
                    rows.fill_row(p, 0u);
                    if (tid % S::TPR == 0) ridx[k & 3][tid / S::TPR + S::PASS * p] = -2;
                }
        };
        if (count > 0) {
            Stage<E, W, BN, NT> first;
            first.template load<ONCE>(tid, row_of(0));
            st.template load<ONCE>(tid, row_of(1));
            if (tid < BN) next_row = cache_row(3);
            if (hides(0)) mark_bad_rows(first, 0);
            first.store(tid, tilebuf[0]);
        }
        v8 q[QREG ? KS : 1];
        const E* qp;
        int last;                                                    // last key this lane's row sees
        {
            const int64_t row = row0 + min(nrows - 1, 16 * rt + col);
            const int i = (int)(row / a.H), h = (int)(row - (int64_t)i * a.H);
            qp = (const E*)a.q + (int64_t)(q0 + i) * a.q_token_stride + h * a.q_head_stride;
            last = len - n + i;
            if (QREG)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) q[ks] = row_frag_global(qp, ks, lane);
        }
        f32x4 acc[RT][CT];
        float m[RT], own = neg_inf(), l = 0.f;                       // own: the maxima of this wave's row tile
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            m[r] = neg_inf();
#pragma unroll
            for (int c = 0; c < CT; ++c) acc[r][c] = f32x4{0.f, 0.f, 0.f, 0.f};
        }
        __syncthreads();
        // (256 sequences 240 us with this wait here, 255 without; chunks, whose pieces
        // have more tiles, 535 with and 520 without)
        if (QREG && RT == 2)
#pragma unroll
            for (int ks = 0; ks < KS; ++ks) arrived(q[ks]);
        for (int k = 0; k < count; ++k) {
            const int t = tile_of(k);
            const E* tile = tilebuf[k & 1];
            f32x4 s[TW];
            v4 p[TW];
            float part = 0.f;
            auto weigh = [&]() {
                const float from = own == neg_inf() ? 0.f : own;     // a row that has seen no key yet
                part = 0.f;
#pragma unroll
                for (int w = 0; w < TW; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float x = exp2_fast(__builtin_fmaf(s[w][i], sc, -from));
                        part += x;                // the sum takes the weights before their rounding
                        p[w][i] = from_f32<E>(x); // bf16: the product's operand type
                    }
            };
            auto put_weights = [&]() {
#pragma unroll
                for (int w = 0; w < TW; ++w) store_vec(sp + (16 * rt + col) * PS + 16 * (tg * TW + w) + 4 * g, p[w]);
            };
            if (scores) {
                const E* qt = qp;
                if (!QREG) asm volatile("" : "+v"(qt));              // fetched again for every tile
#pragma unroll
                for (int w = 0; w < TW; ++w) s[w] = f32x4{0.f, 0.f, 0.f, 0.f};
                constexpr int PD = QREG ? 4 : 1;
                // fp32: each score is summed in four parts, whose rounding errors
                // stay smaller than one sum's over 576 channels and whose products
                // do not wait for each other
                constexpr int NA = sizeof(E) == 4 ? 4 : 1;
                f32x4 more[NA][TW];
#pragma unroll
                for (int i = 1; i < NA; ++i)
#pragma unroll
                    for (int w = 0; w < TW; ++w) more[i][w] = f32x4{0.f, 0.f, 0.f, 0.f};
                v8 x[PD + 1], y[2];
                ahead<KS * TW, PD>(
                    [&](auto step) {
                        constexpr int e = step;
                        if constexpr (!QREG && e % TW == 0) y[e / TW & 1] = row_frag_global(qt, e / TW, lane);
                        x[e % (PD + 1)] = k_rows(tile, 16 * (TW * tg + e % TW), e / TW);
                    },
                    [&](auto step) {
                        constexpr int e = step;
                        if constexpr (QREG) s[e % TW] = mma32(x[e % (PD + 1)], q[e / TW], s[e % TW]);
                        else {
                            f32x4& sum = e / TW % NA ? more[e / TW % NA][e % TW] : s[e % TW];
                            sum = mma32(x[e % (PD + 1)], y[e / TW & 1], sum);
                        }
                    });
#pragma unroll
                for (int w = 0; w < TW; ++w)
                    if constexpr (NA == 4) s[w] = (s[w] + more[1][w]) + (more[2][w] + more[3][w]);
                if (uniform(gaps[k & 3]) || (t + 1) * BN - 1 > first_last) {
#pragma unroll
                    for (int w = 0; w < TW; ++w) {
                        const int k0 = 16 * (tg * TW + w) + 4 * g;
                        const i32x4 there = *reinterpret_cast<const i32x4*>(ridx[k & 3] + k0);
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if (there[i] == -2) s[w][i] = __builtin_nanf("");
                            if (there[i] == -1 || t * BN + k0 + i > last) s[w][i] = neg_inf();
                        }
                    }
                }
                float top = neg_inf();
#pragma unroll
                for (int w = 0; w < TW; ++w)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top = fmaxf(top, s[w][i]);
                top = group_max(top) * sc;
                if (g == 0) stat[tg][16 * rt + col] = top;
                if (__any(top > own + 8.f) && lane == 0) grown[k & 3] = 1;
                weigh();
            }
            __syncthreads();   // maxima are there; the other buffer's and the weights' last readers are done
            if (scores) put_weights();
            if (tid < BN) {
                keep_row(k + 3, next_row);
                next_row = cache_row(k + 4);
            }
            if (tid == 0) grown[(k + 2) & 3] = 0;
            if (k + 1 < count) {
                if (hides(k + 1)) mark_bad_rows(st, k + 1);
                st.template store_load<ONCE>(tid, tilebuf[(k + 1) & 1], row_of(k + 2));
            }
            // The weights are taken against the rows' running maxima as they
            // stand.  Only when a row's grew by more than 8 (in powers of two;
            // the first tile always) are the maxima raised, by every wave alike,
            // the sums rescaled and this tile's weights taken again.
            if (uniform(grown[k & 3])) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    float top = stat[0][16 * r + col];
#pragma unroll
                    for (int w = 1; w < TG; ++w) top = fmaxf(top, stat[w][16 * r + col]);
                    const bool grew = top > m[r] + 8.f;
                    const float f = grew ? exp2_fast(m[r] - top) : 1.f;
                    m[r] = grew ? top : m[r];
#pragma unroll
                    for (int c = 0; c < CT; ++c) acc[r][c] *= f;
                    if (r == rt) l *= f, own = m[r];
                }
                if (scores) {
                    weigh();
                    put_weights();
                }
            }
            l += part;
            __syncthreads();   // weights and the next tile are there
            constexpr int PD = 2, NE = TT / 2 * CT;
            v8 pw[2][RT], x[PD + 1];
            auto weights = [&](int b) {
#pragma unroll
                for (int r = 0; r < RT; ++r) {
                    const E* at = sp + (16 * r + col) * PS + 32 * b + 4 * g;
                    const v4 lo = load_vec<v4>(at), hi = load_vec<v4>(at + 16);
                    pw[b & 1][r] = v8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
                }
            };
            weights(0);
            ahead<NE, PD>(
                [&](auto step) {
                    constexpr int e = step;
                    x[e % (PD + 1)] = c_cols(tile, 32 * (e / CT), 32 * (e / CT) + 16, e % CT);
                },
                [&](auto step) {
                    constexpr int e = step, b = e / CT, c = e % CT;
                    if constexpr (c == CT - 1 && b + 1 < TT / 2) weights(b + 1);
#pragma unroll
                    for (int r = 0; r < RT; ++r) acc[r][c] = mma32(x[e % (PD + 1)], pw[b & 1][r], acc[r][c]);
                });
        }
        // the rows' sums over the waves
        __syncthreads();
        if (scores) {
            const float x = group_sum(l);
            if (g == 0) stat[tg][16 * rt + col] = x;
        }
        __syncthreads();
        const int64_t out0 = (int64_t)q0 * a.H + row0;
        const int slot = 2 * run + (t0 == 0 ? 1 : 0);
#pragma unroll
        for (int r = 0; r < RT; ++r) {
            float sum = stat[0][16 * r + col];
#pragma unroll
            for (int w = 1; w < TG; ++w) sum += stat[w][16 * r + col];
            const int row = 16 * r + col;
            if (row >= nrows) continue;
            if (whole) {
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                E* op = (E*)a.o + (out0 + row) * DL + 16 * wave * CT + 4 * g;
#pragma unroll
                for (int c = 0; c < CT; ++c) {
                    v4 x;
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[i] = from_f32<E>(acc[r][c][i] * inv);
                    store_vec(op + 16 * c, x);
                }
                if (a.lse && wave == 0 && g == 0)
                    a.lse[out0 + row] = sum == 0.f ? neg_inf() : (m[r] + __log2f(sum)) * LN2;
            } else {
                float* op = ws.o + ((int64_t)slot * BM + row) * DL + 16 * wave * CT + 4 * g;
#pragma unroll
                for (int c = 0; c < CT; ++c) store_vec(op + 16 * c, acc[r][c]);
                if (wave == 0 && g == 0) {
                    float* ml = ws.ml + ((int64_t)slot * BM + row) * 2;
                    ml[0] = m[r];
                    ml[1] = sum;
                }
            }
        }
        if (tid == 0) {   // the workgroup that begins a row tile says who holds its parts
            if (t0 == 0) {
                const int64_t first_work = seq_base + (int64_t)unit * key_tiles;
                DecodeSplit x;
                x.row = out0;
                x.rows = whole ? 0 : nrows;
                x.first = run;
                x.last = (int)((first_work + key_tiles - 1) / per);
                x.pad = 0;
                if (by_tile) {
                    if (unit_base + unit < entries) ws.split[unit_base + unit] = x;
                } else if (!whole) ws.split[run] = x;
            }
        }
        __syncthreads();   // statistics and tiles are free for the next piece
        pos += t1 - t0;
    }
}

// Joins the partial results of split row tiles: with M = max_p m_p,
//   o = sum_p 2^(m_p - M) o_p / sum_p 2^(m_p - M) l_p,
// the parts in order.  Many row tiles have few parts each: a wave per row.
template <typename E, int DL>
__global__ __launch_bounds__(256) void latent_join_rows_kernel(const DecodeSpace ws, E* __restrict__ o,
                                                               float* __restrict__ lse, int BM)
{
    constexpr int EPL = DL / 64;   // columns of a lane
    const DecodeSplit x = ws.split[blockIdx.x];
    const int lane = threadIdx.x & 63, row = blockIdx.y * 4 + (threadIdx.x >> 6);
    if (row >= x.rows) return;
    const int parts = x.last - x.first + 1;
    auto slot = [&](int p) { return (int64_t)(p == 0 ? 2 * x.first + 1 : 2 * (x.first + p)) * BM + row; };
    float top = neg_inf();
    for (int p = lane; p < parts; p += 64) top = fmaxf(top, ws.ml[slot(p) * 2]);
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    const float from = top == neg_inf() ? 0.f : top;
    f32x4 acc[EPL / 4];
    float sum = 0.f;
#pragma unroll
    for (int e = 0; e < EPL / 4; ++e) acc[e] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
    for (int p = 0; p < parts; ++p) {
        const float* ml = ws.ml + slot(p) * 2;
        const float f = exp2_fast(ml[0] - from);
        const float* src = ws.o + slot(p) * DL + 4 * lane;
        sum += f * ml[1];
#pragma unroll
        for (int e = 0; e < EPL / 4; ++e) acc[e] += f * *reinterpret_cast<const f32x4*>(src + 256 * e);
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
#pragma unroll
    for (int e = 0; e < EPL / 4; ++e) {
        typename Vec<E>::v4 y;
#pragma unroll
        for (int i = 0; i < 4; ++i) y[i] = from_f32<E>(acc[e][i] * inv);
        store_vec(o + (x.row + row) * DL + 256 * e + 4 * lane, y);
    }
    if (lse && lane == 0) lse[x.row + row] = sum == 0.f ? neg_inf() : (top + __log2f(sum)) * LN2;
}

// Few row tiles may have a part from every workgroup: a workgroup joins 64
// columns of a row, 16 threads side by side and the parts over 16 of them, the
// parts' factors worked out once in LDS.
template <typename E, int DL>
__global__ __launch_bounds__(256) void latent_join_parts_kernel(const DecodeSpace ws, E* __restrict__ o,
                                                                float* __restrict__ lse, int BM)
{
    __shared__ float factor[DEC_RUNS];
    __shared__ float red[4][2];
    __shared__ __attribute__((aligned(16))) f32x4 part[16][16];
    const DecodeSplit x = ws.split[blockIdx.x];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, row = blockIdx.y;
    if (row >= x.rows) return;
    const int parts = x.last - x.first + 1;   // at most one per run
    auto slot = [&](int p) { return (int64_t)(p == 0 ? 2 * x.first + 1 : 2 * (x.first + p)) * BM + row; };
    float m = neg_inf(), l = 0.f;
    if (tid < parts) {
        m = ws.ml[slot(tid) * 2];
        l = ws.ml[slot(tid) * 2 + 1];
    }
    float top = m;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (lane == 0) red[wave][0] = top;
    __syncthreads();
    top = fmaxf(fmaxf(red[0][0], red[1][0]), fmaxf(red[2][0], red[3][0]));
    const float f = m == neg_inf() ? 0.f : exp2_fast(m - top);
    factor[tid] = f;
    float sum = f * l;
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
    if (lane == 0) red[wave][1] = sum;
    __syncthreads();
    sum = (red[0][1] + red[1][1]) + (red[2][1] + red[3][1]);
    const int c = 64 * blockIdx.z + 4 * (tid & 15), first = tid >> 4;
    f32x4 acc = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int p = first; p < parts; p += 16) acc += factor[p] * *reinterpret_cast<const f32x4*>(ws.o + slot(p) * DL + c);
    part[first][tid & 15] = acc;
    __syncthreads();
    if (first != 0) return;
#pragma unroll
    for (int i = 1; i < 16; ++i) acc += part[i][tid];
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    typename Vec<E>::v4 y;
#pragma unroll
    for (int i = 0; i < 4; ++i) y[i] = from_f32<E>(acc[i] * inv);
    store_vec(o + (x.row + row) * DL + c, y);
    if (lse && tid == 0 && blockIdx.z == 0) lse[x.row + row] = sum == 0.f ? neg_inf() : (top + __log2f(sum)) * LN2;
}
static_assert(DEC_RUNS <= 256, "a thread per part");

// Whether the rows of a sequence fit in a tile of 32 (in one of 64 more than
// half would be empty).  By the average, which the host knows: with one sequence of
// two tokens (or of 128) among 256 of 32 heads all take tiles of 64, 279 us (312)
// against 240 for single tokens and 306 for two tokens each.
static bool few_rows(int64_t total_tokens, int32_t N, int32_t H) { return (total_tokens + N - 1) / N * H <= 32; }

size_t latent_decode_workspace(int32_t dl) {
    // Partial results are fp32 for either type, and a tile has as many rows.  Sized
    // for the larger shape whatever the batch, as a batch with more tokens may
    // take the smaller one.
    return space_bytes<DecodeMany<float>>(dl);
}

template <typename E, int DL, int DR, typename S>
static hipError_t launch(const LatentDecode& a, hipStream_t stream) {
    const DecodeSpace ws = space_of<S>(a.workspace);
    const int64_t rows = a.total_tokens * a.H;
    const int64_t bound = a.cu_seqlens ? rows / S::BM + a.num_seqs
                                       : (a.total_tokens / a.num_seqs * a.H + S::BM - 1) / S::BM * a.num_seqs;
    const bool by_tile = bound <= DEC_RUNS;
    const int entries = by_tile ? (int)bound : DEC_RUNS;
    hipLaunchKernelGGL((latent_decode_kernel<E, DL, DR, S>), dim3(DEC_RUNS), dim3(64 * DEC_WAVES), 0, stream, a, ws,
                       by_tile ? 1 : 0, entries);
    // the join goes where the decode kernel's entries point
    if (const hipError_t e = launch_result(stream)) return e;
    if (entries <= 32)   // 8 parts a row tile and more
        hipLaunchKernelGGL((latent_join_parts_kernel<E, DL>), dim3(entries, S::BM, DL / 64), dim3(256), 0, stream, ws,
                           (E*)a.o, a.lse, S::BM);
    else
        hipLaunchKernelGGL((latent_join_rows_kernel<E, DL>), dim3(entries, S::BM / 4), dim3(256), 0, stream, ws,
                           (E*)a.o, a.lse, S::BM);
    return launch_result(stream);
}

template <typename E, int DL, int DR>
static hipError_t launch_rows(const LatentDecode& a, hipStream_t stream) {
    const bool few = few_rows(a.total_tokens, a.num_seqs, a.H);
    return few ? launch<E, DL, DR, DecodeFew<E>>(a, stream) : launch<E, DL, DR, DecodeMany<E>>(a, stream);
}

hipError_t launch_latent_decode(const LatentDecode& a, bool bf16_io, hipStream_t stream) {
    if (bf16_io) {
        if (a.dl == 512) return a.dr ? launch_rows<bf16, 512, 64>(a, stream) : launch_rows<bf16, 512, 0>(a, stream);
        return a.dr ? launch_rows<bf16, 256, 64>(a, stream) : launch_rows<bf16, 256, 0>(a, stream);
    }
    if (a.dl == 512) return a.dr ? launch_rows<float, 512, 64>(a, stream) : launch_rows<float, 512, 0>(a, stream);
    return a.dr ? launch_rows<float, 256, 64>(a, stream) : launch_rows<float, 256, 0>(a, stream);
}

}  // namespace kda
