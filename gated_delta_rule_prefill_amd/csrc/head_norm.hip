// head_norm.hip -- RMS norm of every head with rotary positions in one pass,
// forwards and back, and the write of keys (normalised and turned alike) and values
// to a paged cache.  All move every byte once and are bound by that: bf16, d = 128,
// 36,755 tokens, 32 query and 8 key heads: forwards 148 us, 5.1 TB/s; back 212, 5.3 TB/s
// (a large copy: 4.9 to 5.2); keys and values of as many tokens to the cache and a dense
// copy of the keys 77 us, 4.9 TB/s.  256 tokens: 6.4 us, latency, and 5.2 for the append.
//
//   r = 1 / sqrt(mean(x^2) + eps),  n = r x,  y = R(p f) (n * w)
//   g = R(p f)^T dy,  h = g w,  dx = r (h - n mean(h n)),  dw = sum g n
//
// A row (token, head) belongs to LPR neighbouring lanes, one 16-byte chunk (VE
// elements) each, or with VE = 1 (strides or sizes that do not allow wide accesses) to
// a wave, NK elements a lane.  The pair of a channel may lie in another lane's chunk:
// it is read a second time, from the cache nearest by, rather than exchanged.  A
// row's loads come before its stores, so that rows can be replaced in place.
#include <algorithm>

#include "window_common.h"

namespace kda {

constexpr int NORM_PAIRS = 2048;    // angles of a workgroup
constexpr int NORM_PARTS = 1024;    // workgroups of the backward kernel, at most

// What lane `sub` of a row's lanes does: its elements and where their pairs are.
template <typename E, int VE, int LPR, int NK>
struct HeadRow {
    typedef E vec __attribute__((ext_vector_type(VE)));
    int d, start, half;
    bool inter;
    int at[NK];       // first element of chunk k, or -1
    int kind[NK];     // 0: not turned; 1, 2: first, second of the pairs; 3: pairs within the chunk
    __device__ __forceinline__ HeadRow(int sub, int d, int start, int dr, bool inter)
        : d(d), start(start), half(dr / 2), inter(inter) {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            const int e = VE * (sub + LPR * k), i = e - start;
            at[k] = e < d ? e : -1;
            kind[k] = i < 0 || i >= dr ? 0 : inter ? (VE > 1 ? 3 : 1 + (i & 1)) : i < half ? 1 : 2;
        }
    }
    // The pairs' other elements (kinds 1 and 2).
    __device__ __forceinline__ int other(int k) const {
        const int apart = inter ? 1 : half;
        return at[k] + (kind[k] == 1 ? apart : -apart);
    }
    // The first of the chunk's angles among the token's dr / 2.
    __device__ __forceinline__ int angle(int k) const {
        const int i = at[k] - start;
        return inter ? i / 2 : i < half ? i : i - half;
    }
    static __device__ __forceinline__ void get_weight(const float* w, int at, float* v) {
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = w ? w[at + i] : 1.f;
    }
    // A lane's chunks as they lie in memory; of(): as numbers, 0 where there are none.
    struct Raw {
        vec x[NK];
        __device__ __forceinline__ void of(float (&v)[NK][VE]) const {
#pragma unroll
            for (int k = 0; k < NK; ++k)
#pragma unroll
                for (int i = 0; i < VE; ++i) v[k][i] = to_f32(x[k][i]);
        }
    };
    // A row's chunks, and the chunks with their pairs' other elements.
    __device__ __forceinline__ void load(const E* row, Raw& own) const {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            own.x[k] = vec{};
            if (at[k] >= 0) own.x[k] = *reinterpret_cast<const vec*>(row + at[k]);
        }
    }
    __device__ __forceinline__ void load_pairs(const E* row, Raw& pairs) const {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            pairs.x[k] = vec{};
            if (at[k] >= 0 && (kind[k] == 1 || kind[k] == 2)) pairs.x[k] = *reinterpret_cast<const vec*>(row + other(k));
        }
    }
    template <bool FAR>
    static __device__ __forceinline__ void put(E* p, const float* v) {
        vec x;
#pragma unroll
        for (int i = 0; i < VE; ++i) x[i] = from_f32<E>(v[i]);
        if constexpr (FAR) __builtin_nontemporal_store(x, reinterpret_cast<vec*>(p));
        else *reinterpret_cast<vec*>(p) = x;
    }
    // Chunk k turned by its angles (way 1), or back (way -1); p: the other elements.
    __device__ __forceinline__ void turn(int k, float (&v)[VE], const float (&p)[VE], const float2* cs, float way) const {
        if (kind[k] == 0) return;
        const float2* w = cs + angle(k);
        if (kind[k] == 3) {
            if constexpr (VE > 1)
#pragma unroll
                for (int i = 0; i < VE / 2; ++i) {
                    const float2 r = w[i];
                    const float a = v[2 * i], b = v[2 * i + 1], sn = way * r.y;
                    v[2 * i] = a * r.x - b * sn;
                    v[2 * i + 1] = b * r.x + a * sn;
                }
            return;
        }
        const float sign = kind[k] == 1 ? -way : way;
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = v[i] * w[i].x + sign * w[i].y * p[i];
    }
    // Sum over the row's lanes.
    static __device__ __forceinline__ float sum(float x) {
        if constexpr (LPR > 1) x += lane_xor<1>(x);
        if constexpr (LPR > 2) x += lane_xor<2>(x);
        if constexpr (LPR > 4) x += lane_xor<4>(x);
        if constexpr (LPR > 8) x += lane_xor<8>(x);
        if constexpr (LPR > 16) x += lane_xor<16>(x);
        if constexpr (LPR > 32) x += lane_xor<32>(x);
        return x;
    }
    // 1 / sqrt(mean(v^2) + eps) of the row
    __device__ __forceinline__ float scale(const float (&v)[NK][VE], float eps) const {
        float x = 0.f;
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i) x += v[k][i] * v[k][i];
        return 1.f / sqrtf(sum(x) / (float)d + eps);
    }
};

// The angles of tokens [t0, t0 + nt) into LDS, times the amplitude.
template <typename F>
__device__ __forceinline__ void put_angles(float2* cs, int nt, int half, const float* inv_freq, float amplitude, F position) {
    for (int i = threadIdx.x; i < nt * half; i += 256) {
        float c, s;
        rotation(position(i / half), inv_freq[i % half], false, c, s);
        cs[i] = float2{c * amplitude, s * amplitude};
    }
}

// Walks rows first, first + step, ... of nt tokens with H heads each: (token, head)
// without a division a row.
struct RowWalk {
    int t, h;
    __device__ __forceinline__ RowWalk(int first, int H) : t(first / H), h(first - first / H * H) {}
    __device__ __forceinline__ void on(int step, int H) {
        h += step;
        while (h >= H) h -= H, ++t;
    }
};

// -- queries and keys ------------------------------------------------------------
// A workgroup takes a few tokens: their angles, then the rows of their query heads and
// those of their key heads, each row loaded while the one before is worked on.
template <typename E, int VE, int LPR, int NK, bool FAR>
__global__ __launch_bounds__(256) void qk_norm_kernel(const QkNorm a, int tokens)
{
    __shared__ float2 cs[NORM_PAIRS];
    constexpr int STEP = 256 / LPR;
    const int half = a.dr / 2;
    const int64_t t0 = block_of_grid() * tokens;
    const int nt = (int)max((int64_t)0, min((int64_t)tokens, a.total_tokens - t0));
    typedef HeadRow<E, VE, LPR, NK> Row;
    const Row row(threadIdx.x % LPR, a.d, a.start, a.dr, a.flags & KDA_ROTARY_INTERLEAVED);
    auto rows = [&](const kda_norm_heads& s, auto first) __attribute__((always_inline)) {
        const int H = s.H;
        if (H == 0) return;
        float w[NK][VE], wp[NK][VE];   // the weights of the lane's elements, and of their pairs' others
#pragma unroll
        for (int k = 0; k < NK; ++k)
            if (row.at[k] >= 0) {
                row.get_weight(s.weight, row.at[k], w[k]);
                if (row.kind[k] == 1 || row.kind[k] == 2) row.get_weight(s.weight, row.other(k), wp[k]);
            }
        typename Row::Raw own, pairs;
        auto load = [&](const RowWalk& at) {
            if (at.t >= nt) return;
            const E* x = (const E*)s.x + (t0 + at.t) * s.x_token_stride + at.h * s.x_head_stride;
            row.load(x, own);
            row.load_pairs(x, pairs);
        };
        RowWalk at(threadIdx.x / LPR, H);
        load(at);
        if constexpr (first) {   // the first rows are on their way
            if (half > 0) put_angles(cs, nt, half, a.inv_freq, a.amplitude, [&](int t) { return a.positions[t0 + t]; });
            __syncthreads();
        }
        while (at.t < nt) {
            float v[NK][VE], p[NK][VE];
            own.of(v);
            pairs.of(p);
            E* y = (E*)s.y + (t0 + at.t) * s.y_token_stride + at.h * s.y_head_stride;
            const float2* angles = cs + at.t * half;
            at.on(STEP, H);
            load(at);
            const float r = row.scale(v, a.eps);
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if (row.at[k] < 0) continue;
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    v[k][i] *= r * w[k][i];
                    p[k][i] *= r * wp[k][i];
                }
                row.turn(k, v[k], p[k], angles, 1.f);
                row.template put<FAR>(y + row.at[k], v[k]);
            }
        }
    };
    rows(a.q, Int<1>());
    rows(a.k, Int<0>());
}

// Gradients.  A lane's rows all have its channels: it adds up g n of its own rows, and
// the workgroup's sums go to part[workgroup][queries, keys][d].
template <typename E, int VE, int LPR, int NK, bool FAR>
__global__ __launch_bounds__(256) void qk_norm_backward_kernel(const QkNorm a, int tokens)
{
    __shared__ float2 cs[NORM_PAIRS];
    constexpr int STEP = 256 / LPR;
    __shared__ float sums[STEP][LPR * NK * VE];
    const int sub = threadIdx.x % LPR, mine = threadIdx.x / LPR, half = a.dr / 2;
    typedef HeadRow<E, VE, LPR, NK> Row;
    const Row row(sub, a.d, a.start, a.dr, a.flags & KDA_ROTARY_INTERLEAVED);
    float dw[2][NK][VE];
#pragma unroll
    for (int k = 0; k < NK; ++k)
#pragma unroll
        for (int i = 0; i < VE; ++i) dw[0][k][i] = dw[1][k][i] = 0.f;
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.total_tokens; t0 += (int64_t)gridDim.x * tokens) {
        const int nt = (int)min((int64_t)tokens, a.total_tokens - t0);
        auto rows = [&](const kda_norm_heads& s, float (&sum)[NK][VE], auto first) __attribute__((always_inline)) {
            const int H = s.H;
            if (H == 0) return;
            float w[NK][VE];
#pragma unroll
            for (int k = 0; k < NK; ++k)
                if (row.at[k] >= 0) row.get_weight(s.weight, row.at[k], w[k]);
            typename Row::Raw own, grad, pairs;
            auto load = [&](const RowWalk& at) {
                if (at.t >= nt) return;
                const E* dy = (const E*)s.dy + (t0 + at.t) * s.dy_token_stride + at.h * s.dy_head_stride;
                row.load((const E*)s.x + (t0 + at.t) * s.x_token_stride + at.h * s.x_head_stride, own);
                row.load(dy, grad);
                row.load_pairs(dy, pairs);
            };
            RowWalk at(mine, H);
            load(at);
            if constexpr (first)
                if (half > 0) {
                    __syncthreads();   // the last tokens' angles are read
                    put_angles(cs, nt, half, a.inv_freq, a.amplitude, [&](int t) { return a.positions[t0 + t]; });
                    __syncthreads();
                }
            while (at.t < nt) {
                float v[NK][VE], gr[NK][VE], p[NK][VE];
                own.of(v);
                grad.of(gr);
                pairs.of(p);
                E* dx = (E*)s.dx + (t0 + at.t) * s.dx_token_stride + at.h * s.dx_head_stride;
                const float2* angles = cs + at.t * half;
                at.on(STEP, H);
                load(at);
                const float r = row.scale(v, a.eps);
                float dot = 0.f;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    if (row.at[k] < 0) continue;
                    row.turn(k, gr[k], p[k], angles, -1.f);
#pragma unroll
                    for (int i = 0; i < VE; ++i) {
                        v[k][i] *= r;
                        const float gn = gr[k][i] * v[k][i];
                        sum[k][i] += gn;
                        dot += gn * w[k][i];
                        gr[k][i] *= w[k][i];
                    }
                }
                dot = row.sum(dot) / (float)a.d;
#pragma unroll
                for (int k = 0; k < NK; ++k) {
                    if (row.at[k] < 0) continue;
#pragma unroll
                    for (int i = 0; i < VE; ++i) gr[k][i] = r * (gr[k][i] - v[k][i] * dot);
                    row.template put<FAR>(dx + row.at[k], gr[k]);
                }
            }
        };
        rows(a.q, dw[0], Int<1>());
        rows(a.k, dw[1], Int<0>());
    }
#pragma unroll
    for (int kind = 0; kind < 2; ++kind) {
        __syncthreads();
#pragma unroll
        for (int k = 0; k < NK; ++k)
#pragma unroll
            for (int i = 0; i < VE; ++i) sums[mine][VE * (sub + LPR * k) + i] = dw[kind][k][i];
        __syncthreads();
        for (int c = threadIdx.x; c < a.d; c += 256) {
            float x = 0.f;
#pragma unroll 8
            for (int n = 0; n < STEP; ++n) x += sums[n][c];
            a.part[((int64_t)blockIdx.x * 2 + kind) * a.d + c] = x;
        }
    }
}

// The weights' gradients from the workgroups' parts: 16 channels a workgroup, the
// parts over 16 threads each, their sums in order.
__global__ __launch_bounds__(256) void qk_norm_weight_kernel(const QkNorm a, int parts)
{
    __shared__ float sums[16][17];
    const int c = 16 * blockIdx.x + (threadIdx.x & 15), n = threadIdx.x >> 4, kind = blockIdx.y;
    float* to = kind ? a.k.dweight : a.q.dweight;
    if (!to) return;
    float x = 0.f;
    if (c < a.d)
#pragma unroll 8
        for (int p = n; p < parts; p += 16) x += a.part[((int64_t)p * 2 + kind) * a.d + c];
    sums[n][threadIdx.x & 15] = x;
    __syncthreads();
    if (n != 0 || c >= a.d) return;
#pragma unroll
    for (int p = 1; p < 16; ++p) x += sums[p][threadIdx.x];
    to[c] = x;
}

static bool wide(const void* p, int64_t token_stride, int64_t head_stride, int es) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && token_stride * es % 16 == 0 && head_stride * es % 16 == 0;
}
static bool wide_sizes(int d, int start, int dr, uint32_t flags, int es) {
    const int ce = 16 / es;
    return d % ce == 0 && (dr == 0 || (start % ce == 0 && (flags & KDA_ROTARY_INTERLEAVED ? dr : dr / 2) % ce == 0));
}

// Calls go(chunk elements, lanes per row, chunks per lane) for rows of d channels.
template <typename E, typename F>
static void by_shape(bool wide, int d, F go) {
    constexpr int CE = CHUNK_ELEMS<E>;
    const int chunks = d / CE;
    if (!wide) go(Int<1>(), Int<64>(), Int<4>());
    else if (chunks <= 8) go(Int<CE>(), Int<8>(), Int<1>());
    else if (chunks <= 16) go(Int<CE>(), Int<16>(), Int<1>());
    else if (chunks <= 32) go(Int<CE>(), Int<32>(), Int<1>());
    else go(Int<CE>(), Int<64>(), Int<1>());
}

// Tokens of a workgroup: a few rows for each of its groups of lanes, its angles in
// LDS, and at least 512 workgroups.
static int norm_tokens(int64_t total, int heads, int lanes, int half, int each) {
    int64_t n = std::max<int64_t>(1, (int64_t)each * (256 / lanes) / heads);
    n = std::min(n, std::max<int64_t>(1, total / 512));
    return (int)std::min<int64_t>(n, half > 0 ? NORM_PAIRS / half : n);
}

// More than the 256 MB of the last-level cache is stored past the caches: 36,755 tokens,
// 40 heads of 128, bf16, forwards then back: 149 + 212 us.  With the forward's outputs
// through the caches 137 + 237, as what they hold back is written during the next kernel;
// with the gradients too 144 + 228.
static bool far(const QkNorm& a, int es) {
    return a.total_tokens * (a.q.H + a.k.H) * (int64_t)a.d * es > (int64_t)256 << 20;
}

template <typename E>
static hipError_t launch_norm(const QkNorm& a, hipStream_t stream) {
    bool w = wide_sizes(a.d, a.start, a.dr, a.flags, sizeof(E));
    for (const kda_norm_heads* s : {&a.q, &a.k})
        if (s->H > 0)
            w = w && wide(s->x, s->x_token_stride, s->x_head_stride, sizeof(E)) &&
                wide(s->y, s->y_token_stride, s->y_head_stride, sizeof(E));
    by_shape<E>(w, a.d, [&](auto ve, auto lpr, auto nk) {
        const int tokens = norm_tokens(a.total_tokens, a.q.H + a.k.H, lpr, a.dr / 2, 16);
        auto go = [&](auto kernel) {
            hipLaunchKernelGGL(kernel, grid_of((a.total_tokens + tokens - 1) / tokens), dim3(256), 0, stream, a, tokens);
        };
        if (far(a, sizeof(E)) && ve > 1) go(qk_norm_kernel<E, ve, lpr, nk, (ve > 1)>);
        else go(qk_norm_kernel<E, ve, lpr, nk, false>);
    });
    return launch_result(stream);
}

hipError_t launch_qk_norm_rotary(const QkNorm& a, bool bf16_io, hipStream_t stream) {
    return bf16_io ? launch_norm<bf16>(a, stream) : launch_norm<float>(a, stream);
}

size_t qk_norm_workspace(int32_t d) { return (size_t)NORM_PARTS * 2 * d * 4; }

template <typename E>
static hipError_t launch_norm_backward(const QkNorm& a, hipStream_t stream) {
    bool w = wide_sizes(a.d, a.start, a.dr, a.flags, sizeof(E));
    for (const kda_norm_heads* s : {&a.q, &a.k})
        if (s->H > 0)
            w = w && wide(s->x, s->x_token_stride, s->x_head_stride, sizeof(E)) &&
                wide(s->dy, s->dy_token_stride, s->dy_head_stride, sizeof(E)) &&
                wide(s->dx, s->dx_token_stride, s->dx_head_stride, sizeof(E));
    int parts = 0;
    if (a.total_tokens > 0) {
        by_shape<E>(w, a.d, [&](auto ve, auto lpr, auto nk) {
            const int tokens = norm_tokens(a.total_tokens, a.q.H + a.k.H, lpr, a.dr / 2, 20);
            parts = (int)std::min<int64_t>(NORM_PARTS, (a.total_tokens + tokens - 1) / tokens);
            auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, dim3(parts), dim3(256), 0, stream, a, tokens); };
            if (far(a, sizeof(E)) && ve > 1) go(qk_norm_backward_kernel<E, ve, lpr, nk, (ve > 1)>);
            else go(qk_norm_backward_kernel<E, ve, lpr, nk, false>);
        });
        if (const hipError_t e = launch_result(stream)) return e;
    }
    if (!a.q.dweight && !a.k.dweight) return hipSuccess;
    hipLaunchKernelGGL(qk_norm_weight_kernel, dim3((a.d + 15) / 16, 2), dim3(256), 0, stream, a, parts);
    return launch_result(stream);
}

hipError_t launch_qk_norm_rotary_backward(const QkNorm& a, bool bf16_io, hipStream_t stream) {
    return bf16_io ? launch_norm_backward<bf16>(a, stream) : launch_norm_backward<float>(a, stream);
}

// -- cache rows --------------------------------------------------------------------
constexpr int APPEND_TOKENS = 32;   // of a workgroup, at most

template <typename E, int VE, int LPR, int NK>
__global__ __launch_bounds__(256) void kv_append_kernel(const KvAppend a, int tokens)
{
    __shared__ float2 cs[NORM_PAIRS];
    __shared__ int where[APPEND_TOKENS];       // position, or the least integer outside the sequences
    __shared__ int64_t place[APPEND_TOKENS];   // cache row, -1: none
    constexpr int OUTSIDE = -2147483647 - 1;
    const int lane = threadIdx.x & 63, half = a.dr / 2;
    const int64_t t0 = block_of_grid() * tokens;
    const int nt = (int)max((int64_t)0, min((int64_t)tokens, a.total_tokens - t0));
    for (int x = threadIdx.x >> 6; x < nt; x += 4) {   // a wave per token
        const int64_t t = t0 + x;
        int seq, n, i;
        if (a.cu_seqlens) {
            seq = sequence_of(a.cu_seqlens, a.num_seqs, t, lane);
            const int first = seq < 0 ? 0 : a.cu_seqlens[seq];
            n = seq < 0 ? 0 : (int)min((int64_t)a.cu_seqlens[seq + 1], a.total_tokens) - first;   // as decode counts them
            i = (int)(t - first);
        } else {
            n = (int)(a.total_tokens / a.num_seqs);
            seq = (int)(t / n);
            i = (int)(t - (int64_t)seq * n);
        }
        if (lane == 0) {
            const int position = seq < 0 ? OUTSIDE : cached_tokens(a.pages, seq) - n + i;
            where[x] = position;
            place[x] = position < 0 ? -1 : cached_row(a.pages, seq, position);
        }
    }
    constexpr int STEP = 256 / LPR;
    typedef HeadRow<E, VE, LPR, NK> Row;
    const Row row(threadIdx.x % LPR, a.d, a.start, a.dr, a.flags & KDA_ROTARY_INTERLEAVED);
    float w[NK][VE], wp[NK][VE];
#pragma unroll
    for (int k = 0; k < NK; ++k)
        if (row.at[k] >= 0) {
            row.get_weight(a.norm_weight, row.at[k], w[k]);
            if (row.kind[k] == 1 || row.kind[k] == 2) row.get_weight(a.norm_weight, row.other(k), wp[k]);
        }
    __syncthreads();
    if (half > 0) {
        put_angles(cs, nt, half, a.inv_freq, a.amplitude, [&](int t) { return where[t]; });
        __syncthreads();
    }
    // key rows, then value rows
    typename Row::Raw own, pairs;
    const int mine = threadIdx.x / LPR;
    auto cached = [&](void* cache, const RowWalk& at) {
        return place[at.t] < 0 ? nullptr : (E*)cache + place[at.t] + at.h * a.pages.head_stride;
    };
    {
        auto load = [&](const RowWalk& at) {
            if (at.t >= nt) return;
            const E* k = (const E*)a.k + (t0 + at.t) * a.k_token_stride + at.h * a.k_head_stride;
            row.load(k, own);
            row.load_pairs(k, pairs);
        };
        RowWalk at(mine, a.Hk);
        load(at);
        while (at.t < nt) {
            float v[NK][VE], p[NK][VE];
            own.of(v);
            pairs.of(p);
            E* to = cached(a.pages.k, at);
            E* dense = a.k_out && where[at.t] != OUTSIDE ? (E*)a.k_out + ((t0 + at.t) * a.Hk + at.h) * a.d : nullptr;
            const float2* angles = cs + at.t * half;
            at.on(STEP, a.Hk);
            load(at);
            const float r = a.norm_weight ? row.scale(v, a.eps) : 1.f;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if (row.at[k] < 0) continue;
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    v[k][i] *= r * w[k][i];
                    p[k][i] *= r * wp[k][i];
                }
                row.turn(k, v[k], p[k], angles, 1.f);
                if (to) row.template put<false>(to + row.at[k], v[k]);
                if (dense) row.template put<false>(dense + row.at[k], v[k]);
            }
        }
    }
    for (RowWalk at(mine, a.Hk); at.t < nt; at.on(STEP, a.Hk)) {
        E* to = cached(a.pages.v, at);
        if (!to) continue;
        row.load((const E*)a.v + (t0 + at.t) * a.v_token_stride + at.h * a.v_head_stride, own);
#pragma unroll
        for (int k = 0; k < NK; ++k)
            if (row.at[k] >= 0) *reinterpret_cast<typename Row::vec*>(to + row.at[k]) = own.x[k];
    }
}

template <typename E>
static hipError_t launch_append(const KvAppend& a, hipStream_t stream) {
    const bool w = wide_sizes(a.d, a.start, a.dr, a.flags, sizeof(E));
    by_shape<E>(w, a.d, [&](auto ve, auto lpr, auto nk) {
        const int tokens = std::min(APPEND_TOKENS, norm_tokens(a.total_tokens, 2 * a.Hk, lpr, a.dr / 2, 4));
        hipLaunchKernelGGL((kv_append_kernel<E, ve, lpr, nk>), grid_of((a.total_tokens + tokens - 1) / tokens), dim3(256),
                           0, stream, a, tokens);
    });
    return launch_result(stream);
}

hipError_t launch_kv_append(const KvAppend& a, bool bf16_io, hipStream_t stream) {
    return bf16_io ? launch_append<bf16>(a, stream) : launch_append<float>(a, stream);
}

}  // namespace kda
