// head_norm.hip -- RMS norm of every head with rotary positions in one pass,
// forwards and back, and the write of keys (normalised and turned alike) and values
// to a paged cache.  All move every byte once and are bound by that.
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
    static __device__ __forceinline__ void get(const E* p, float* v) {
        if constexpr (VE == 1) v[0] = to_f32(p[0]);
        else {
            const vec x = *reinterpret_cast<const vec*>(p);
#pragma unroll
            for (int i = 0; i < VE; ++i) v[i] = to_f32(x[i]);
        }
    }
    static __device__ __forceinline__ void put(E* p, const float* v) {
        if constexpr (VE == 1) p[0] = from_f32<E>(v[0]);
        else {
            vec x;
#pragma unroll
            for (int i = 0; i < VE; ++i) x[i] = from_f32<E>(v[i]);
            *reinterpret_cast<vec*>(p) = x;
        }
    }
    static __device__ __forceinline__ void get_weight(const float* w, int at, float* v) {
#pragma unroll
        for (int i = 0; i < VE; ++i) v[i] = w ? w[at + i] : 1.f;
    }
    // Chunk k of a row, and the chunk with its pairs' other elements.
    __device__ __forceinline__ void load(const E* row, float (&v)[NK][VE], float (&p)[NK][VE]) const {
#pragma unroll
        for (int k = 0; k < NK; ++k) {
#pragma unroll
            for (int i = 0; i < VE; ++i) v[k][i] = p[k][i] = 0.f;
            if (at[k] < 0) continue;
            get(row + at[k], v[k]);
            if (kind[k] == 1 || kind[k] == 2) get(row + other(k), p[k]);
        }
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

// -- queries and keys ------------------------------------------------------------
template <typename E, int VE, int LPR, int NK>
__global__ __launch_bounds__(256) void qk_norm_kernel(const QkNorm a, int tokens)
{
    __shared__ float2 cs[NORM_PAIRS];
    const int sub = threadIdx.x % LPR, half = a.dr / 2, heads = a.q.H + a.k.H;
    const int64_t t0 = block_of_grid() * tokens;
    const int nt = (int)max((int64_t)0, min((int64_t)tokens, a.total_tokens - t0));
    const HeadRow<E, VE, LPR, NK> row(sub, a.d, a.start, a.dr, a.flags & KDA_ROTARY_INTERLEAVED);
    float w[2][NK][VE], wp[2][NK][VE];   // the weights of the lane's elements, and of their pairs' others
#pragma unroll
    for (int k = 0; k < NK; ++k)
        if (row.at[k] >= 0) {
            row.get_weight(a.q.weight, row.at[k], w[0][k]);
            row.get_weight(a.k.weight, row.at[k], w[1][k]);
            if (row.kind[k] == 1 || row.kind[k] == 2) {
                row.get_weight(a.q.weight, row.other(k), wp[0][k]);
                row.get_weight(a.k.weight, row.other(k), wp[1][k]);
            }
        }
    if (half > 0) put_angles(cs, nt, half, a.inv_freq, a.amplitude, [&](int t) { return a.positions[t0 + t]; });
    __syncthreads();
    for (int id = threadIdx.x / LPR; id < nt * heads; id += 256 / LPR) {
        const int t = id / heads, hh = id - t * heads;
        const bool key = hh >= a.q.H;
        const int h = key ? hh - a.q.H : hh;
        const E* x = (const E*)(key ? a.k.x : a.q.x) + (t0 + t) * (key ? a.k.x_token_stride : a.q.x_token_stride) +
                     h * (key ? a.k.x_head_stride : a.q.x_head_stride);
        E* y = (E*)(key ? a.k.y : a.q.y) + (t0 + t) * (key ? a.k.y_token_stride : a.q.y_token_stride) +
               h * (key ? a.k.y_head_stride : a.q.y_head_stride);
        float v[NK][VE], p[NK][VE];
        row.load(x, v, p);
        const float r = row.scale(v, a.eps);
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            if (row.at[k] < 0) continue;
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                v[k][i] *= r * (key ? w[1][k][i] : w[0][k][i]);
                p[k][i] *= r * (key ? wp[1][k][i] : wp[0][k][i]);
            }
            row.turn(k, v[k], p[k], cs + t * half, 1.f);
        }
#pragma unroll
        for (int k = 0; k < NK; ++k)
            if (row.at[k] >= 0) row.put(y + row.at[k], v[k]);
    }
}

// Gradients.  A lane's rows all have its channels: it adds up g n of its own rows, and
// the workgroup's sums go to part[workgroup][queries, keys][d].
template <typename E, int VE, int LPR, int NK>
__global__ __launch_bounds__(256) void qk_norm_backward_kernel(const QkNorm a, int tokens)
{
    __shared__ float2 cs[NORM_PAIRS];
    __shared__ float sums[256 / LPR][LPR * NK * VE];
    const int sub = threadIdx.x % LPR, mine = threadIdx.x / LPR, half = a.dr / 2, heads = a.q.H + a.k.H;
    const HeadRow<E, VE, LPR, NK> row(sub, a.d, a.start, a.dr, a.flags & KDA_ROTARY_INTERLEAVED);
    float w[2][NK][VE], dw[2][NK][VE];
#pragma unroll
    for (int k = 0; k < NK; ++k) {
#pragma unroll
        for (int i = 0; i < VE; ++i) dw[0][k][i] = dw[1][k][i] = 0.f;
        if (row.at[k] >= 0) {
            row.get_weight(a.q.weight, row.at[k], w[0][k]);
            row.get_weight(a.k.weight, row.at[k], w[1][k]);
        }
    }
    for (int64_t t0 = (int64_t)blockIdx.x * tokens; t0 < a.total_tokens; t0 += (int64_t)gridDim.x * tokens) {
        const int nt = (int)min((int64_t)tokens, a.total_tokens - t0);
        if (half > 0) {
            __syncthreads();   // the last tokens' angles are read
            put_angles(cs, nt, half, a.inv_freq, a.amplitude, [&](int t) { return a.positions[t0 + t]; });
            __syncthreads();
        }
        for (int id = mine; id < nt * heads; id += 256 / LPR) {
            const int t = id / heads, hh = id - t * heads;
            const bool key = hh >= a.q.H;
            const int h = key ? hh - a.q.H : hh;
            const E* x = (const E*)(key ? a.k.x : a.q.x) + (t0 + t) * (key ? a.k.x_token_stride : a.q.x_token_stride) +
                         h * (key ? a.k.x_head_stride : a.q.x_head_stride);
            const E* dy = (const E*)(key ? a.k.dy : a.q.dy) + (t0 + t) * (key ? a.k.dy_token_stride : a.q.dy_token_stride) +
                          h * (key ? a.k.dy_head_stride : a.q.dy_head_stride);
            E* dx = (E*)(key ? a.k.dx : a.q.dx) + (t0 + t) * (key ? a.k.dx_token_stride : a.q.dx_token_stride) +
                    h * (key ? a.k.dx_head_stride : a.q.dx_head_stride);
            float v[NK][VE], gr[NK][VE], p[NK][VE];
#pragma unroll
            for (int k = 0; k < NK; ++k) {
#pragma unroll
                for (int i = 0; i < VE; ++i) v[k][i] = 0.f;
                if (row.at[k] >= 0) row.get(x + row.at[k], v[k]);
            }
            row.load(dy, gr, p);
            const float r = row.scale(v, a.eps);
            float dot = 0.f;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if (row.at[k] < 0) continue;
                row.turn(k, gr[k], p[k], cs + t * half, -1.f);
#pragma unroll
                for (int i = 0; i < VE; ++i) {
                    v[k][i] *= r;
                    const float gn = gr[k][i] * v[k][i];
                    dw[0][k][i] += key ? 0.f : gn;
                    dw[1][k][i] += key ? gn : 0.f;
                    const float wi = key ? w[1][k][i] : w[0][k][i];
                    dot += gn * wi;
                    gr[k][i] *= wi;
                }
            }
            dot = row.sum(dot) / (float)a.d;
#pragma unroll
            for (int k = 0; k < NK; ++k) {
                if (row.at[k] < 0) continue;
#pragma unroll
                for (int i = 0; i < VE; ++i) gr[k][i] = r * (gr[k][i] - v[k][i] * dot);
                row.put(dx + row.at[k], gr[k]);
            }
        }
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
            for (int n = 0; n < 256 / LPR; ++n) x += sums[n][c];
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

template <typename E>
static hipError_t launch_norm(const QkNorm& a, hipStream_t stream) {
    bool w = wide_sizes(a.d, a.start, a.dr, a.flags, sizeof(E));
    for (const kda_norm_heads* s : {&a.q, &a.k})
        if (s->H > 0)
            w = w && wide(s->x, s->x_token_stride, s->x_head_stride, sizeof(E)) &&
                wide(s->y, s->y_token_stride, s->y_head_stride, sizeof(E));
    by_shape<E>(w, a.d, [&](auto ve, auto lpr, auto nk) {
        const int tokens = norm_tokens(a.total_tokens, a.q.H + a.k.H, lpr, a.dr / 2, 5);
        hipLaunchKernelGGL((qk_norm_kernel<E, ve, lpr, nk>), grid_of((a.total_tokens + tokens - 1) / tokens), dim3(256), 0,
                           stream, a, tokens);
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
            const int tokens = norm_tokens(a.total_tokens, a.q.H + a.k.H, lpr, a.dr / 2, 5);
            parts = (int)std::min<int64_t>(NORM_PARTS, (a.total_tokens + tokens - 1) / tokens);
            hipLaunchKernelGGL((qk_norm_backward_kernel<E, ve, lpr, nk>), dim3(parts), dim3(256), 0, stream, a, tokens);
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
    const int sub = threadIdx.x % LPR, lane = threadIdx.x & 63, half = a.dr / 2;
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
    const HeadRow<E, VE, LPR, NK> row(sub, a.d, a.start, a.dr, a.flags & KDA_ROTARY_INTERLEAVED);
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
    // key rows, then value rows of each token
    for (int id = threadIdx.x / LPR; id < nt * 2 * a.Hk; id += 256 / LPR) {
        const int t = id / (2 * a.Hk), hh = id - t * 2 * a.Hk;
        const bool value = hh >= a.Hk;
        const int h = value ? hh - a.Hk : hh;
        const int64_t at = place[t];
        E* cached = at < 0 ? nullptr : (E*)(value ? a.pages.v : a.pages.k) + at + h * a.pages.head_stride;
        if (value) {
            if (!cached) continue;
            const E* v = (const E*)a.v + (t0 + t) * a.v_token_stride + h * a.v_head_stride;
#pragma unroll
            for (int k = 0; k < NK; ++k)
                if (row.at[k] >= 0) {
                    typedef typename HeadRow<E, VE, LPR, NK>::vec vec;
                    *reinterpret_cast<vec*>(cached + row.at[k]) = *reinterpret_cast<const vec*>(v + row.at[k]);
                }
            continue;
        }
        E* dense = a.k_out && where[t] != OUTSIDE ? (E*)a.k_out + ((t0 + t) * a.Hk + h) * a.d : nullptr;
        if (!cached && !dense) continue;
        float v[NK][VE], p[NK][VE];
        row.load((const E*)a.k + (t0 + t) * a.k_token_stride + h * a.k_head_stride, v, p);
        const float r = a.norm_weight ? row.scale(v, a.eps) : 1.f;
#pragma unroll
        for (int k = 0; k < NK; ++k) {
            if (row.at[k] < 0) continue;
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                v[k][i] *= r * w[k][i];
                p[k][i] *= r * wp[k][i];
            }
            row.turn(k, v[k], p[k], cs + t * half, 1.f);
            if (cached) row.put(cached + row.at[k], v[k]);
            if (dense) row.put(dense + row.at[k], v[k]);
        }
    }
}

template <typename E>
static hipError_t launch_append(const KvAppend& a, hipStream_t stream) {
    const bool w = wide_sizes(a.d, a.start, a.dr, a.flags, sizeof(E));
    by_shape<E>(w, a.d, [&](auto ve, auto lpr, auto nk) {
        const int tokens = std::min(APPEND_TOKENS, norm_tokens(a.total_tokens, 2 * a.Hk, lpr, a.dr / 2, 8));
        hipLaunchKernelGGL((kv_append_kernel<E, ve, lpr, nk>), grid_of((a.total_tokens + tokens - 1) / tokens), dim3(256),
                           0, stream, a, tokens);
    });
    return launch_result(stream);
}

hipError_t launch_kv_append(const KvAppend& a, bool bf16_io, hipStream_t stream) {
    return bf16_io ? launch_append<bf16>(a, stream) : launch_append<float>(a, stream);
}

}  // namespace kda
