// latent_cache.hip -- what goes into the attention's cache and queries: rotary
// positions on part of a head, and the write of a token's normalised latent and
// rotated key part to its row of the paged cache.  Both move every byte once
// and are bound by that.
#include "latent_common.h"

namespace kda {

// cos and sin of position * frequency (radians).  The product and its
// reduction to a fraction of a turn are in 64 bits: at position 10^6 a product
// in 32 bits is off by 0.06 radians.
__device__ __forceinline__ void rotation(int position, float inv_freq, bool inverse, float& c, float& s) {
    const double turns = (double)position * (double)inv_freq * 0.15915494309189535;
    const float r = (float)(turns - rint(turns));
    sincospif(2.f * r, &s, &c);
    if (inverse) s = -s;
}

// -- rotary positions ---------------------------------------------------------------
// A workgroup takes `tokens` tokens: their dr / 2 angles go to LDS once for all
// heads, then its threads walk (token, head, item).  An item of the rotated
// part holds both elements of its pairs (VE pairs in the half layout), so a
// rotation in place reads nothing that another thread writes; the other items
// copy VE elements each and exist only when y is not x.  VE: elements of a
// 16-byte access, or 1 where alignment or sizes do not allow it.
constexpr int ROTARY_PAIRS = 2048;   // angles of a workgroup

template <typename E, int VE, bool INTERLEAVED, bool FAR>
__global__ __launch_bounds__(256) void rotary_kernel(const Rotary a, int tokens, int copies)
{
    __shared__ float2 cs[ROTARY_PAIRS];
    constexpr int IE = INTERLEAVED ? (VE == 1 ? 2 : VE) : 2 * VE;   // elements of a rotated item
    const int half = a.dr / 2;
    const int64_t t0 = block_of_grid() * tokens;
    const int nt = (int)min((int64_t)tokens, a.total_tokens - t0);
    for (int i = threadIdx.x; i < nt * half; i += 256) {
        float c, s;
        rotation(a.positions[t0 + i / half], a.inv_freq[i % half], a.flags & KDA_ROTARY_INVERSE, c, s);
        cs[i] = float2{c * a.amplitude, s * a.amplitude};
    }
    __syncthreads();
    typedef E vec __attribute__((ext_vector_type(VE)));
    auto get = [](const E* p, float* v) {
        if constexpr (VE == 1) v[0] = to_f32(p[0]);
        else {
            const vec x = *reinterpret_cast<const vec*>(p);
#pragma unroll
            for (int i = 0; i < VE; ++i) v[i] = to_f32(x[i]);
        }
    };
    auto store = [](E* p, vec x) {
        if constexpr (FAR) __builtin_nontemporal_store(__builtin_bit_cast(u32x4, x), reinterpret_cast<u32x4*>(p));
        else *reinterpret_cast<vec*>(p) = x;
    };
    auto put = [store](E* p, const float* v) {
        if constexpr (VE == 1) p[0] = from_f32<E>(v[0]);
        else {
            vec x;
#pragma unroll
            for (int i = 0; i < VE; ++i) x[i] = from_f32<E>(v[i]);
            store(p, x);
        }
    };
    const int turned = a.dr / IE, items = turned + copies, rows = nt * a.H;
    const int all = rows * items;
    for (int id = threadIdx.x; id < all; id += 256) {
        const int row = id / items, item = id - row * items;
        const int t = row / a.H, h = row - t * a.H;
        const E* x = (const E*)a.x + (t0 + t) * a.x_token_stride + h * a.x_head_stride;
        E* y = (E*)a.y + (t0 + t) * a.y_token_stride + h * a.y_head_stride;
        if (item >= turned) {
            int at = (item - turned) * VE;
            if (at >= a.start) at += a.dr;
            if constexpr (VE == 1) y[at] = x[at];
            else store(y + at, *reinterpret_cast<const vec*>(x + at));
            continue;
        }
        const float2* w = cs + t * half;
        if constexpr (INTERLEAVED && VE > 1) {
            const int at = a.start + item * VE;
            float v[VE], u[VE];
            get(x + at, v);
#pragma unroll
            for (int i = 0; i < VE / 2; ++i) {
                const float2 r = w[item * (VE / 2) + i];
                u[2 * i] = v[2 * i] * r.x - v[2 * i + 1] * r.y;
                u[2 * i + 1] = v[2 * i + 1] * r.x + v[2 * i] * r.y;
            }
            put(y + at, u);
        } else {   // VE pairs, their two elements `apart`
            const int apart = INTERLEAVED ? 1 : half;
            const int at = a.start + (INTERLEAVED ? 2 * item : item * VE);
            float v0[VE], v1[VE], u0[VE], u1[VE];
            get(x + at, v0);
            get(x + at + apart, v1);
#pragma unroll
            for (int i = 0; i < VE; ++i) {
                const float2 r = w[item * VE + i];
                u0[i] = v0[i] * r.x - v1[i] * r.y;
                u1[i] = v1[i] * r.x + v0[i] * r.y;
            }
            put(y + at, u0);
            put(y + at + apart, u1);
        }
    }
}

template <typename E>
static hipError_t launch_rotary_t(const Rotary& a, hipStream_t stream) {
    constexpr int CE = CHUNK_ELEMS<E>;
    const bool inter = a.flags & KDA_ROTARY_INTERLEAVED;
    const bool in_place = a.x == a.y;
    auto even = [&](int64_t n) { return n % CE == 0; };
    const bool wide = ((uintptr_t)a.x | (uintptr_t)a.y) % 16 == 0 && even(a.x_token_stride) && even(a.x_head_stride) &&
                      even(a.y_token_stride) && even(a.y_head_stride) && even(a.start) && even(a.d) &&
                      even(inter ? a.dr : a.dr / 2);
    const int copies = in_place ? 0 : (a.d - a.dr) / (wide ? CE : 1);
    const int items = a.dr / (wide ? (inter ? CE : 2 * CE) : 2) + copies;
    // Tokens of a workgroup: about three items a thread (a prompt of 65,536 x 32
    // x 192 in bf16, one token each: 275 us, 5.85 TB/s, where a copy of as many
    // bytes takes 306; with runs of four rows per thread, 346), with its angles
    // in LDS and at least 512 workgroups.
    int64_t tokens = 768 / ((int64_t)a.H * items);
    if (tokens > a.total_tokens / 512) tokens = a.total_tokens / 512;
    if (tokens > ROTARY_PAIRS / (a.dr / 2)) tokens = ROTARY_PAIRS / (a.dr / 2);
    if (tokens < 1) tokens = 1;
    const dim3 grid = grid_of((a.total_tokens + tokens - 1) / tokens);
    // More than the 256 MB of the last-level cache is stored past the caches (that
    // prompt 284 us without; what fits may stay there for its reader).
    const bool far = a.total_tokens * a.H * (int64_t)(in_place ? a.dr : a.d) * (int64_t)sizeof(E) > (int64_t)256 << 20;
    auto go = [&](auto kernel) { hipLaunchKernelGGL(kernel, grid, dim3(256), 0, stream, a, (int)tokens, copies); };
    if (wide && far) inter ? go(rotary_kernel<E, CE, true, true>) : go(rotary_kernel<E, CE, false, true>);
    else if (wide) inter ? go(rotary_kernel<E, CE, true, false>) : go(rotary_kernel<E, CE, false, false>);
    else inter ? go(rotary_kernel<E, 1, true, false>) : go(rotary_kernel<E, 1, false, false>);
    return launch_result(stream);
}

hipError_t launch_rotary(const Rotary& a, bool bf16_io, hipStream_t stream) {
    return bf16_io ? launch_rotary_t<bf16>(a, stream) : launch_rotary_t<float>(a, stream);
}

// -- cache rows ---------------------------------------------------------------------
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

// One wave per token: the latent stays in registers between its sum of squares
// and its write.
template <typename E>
__global__ __launch_bounds__(256) void latent_append_kernel(const LatentAppend a)
{
    constexpr int CE = CHUNK_ELEMS<E>, NC = 1024 / CE / 64;   // 16-byte chunks of a lane
    typedef E vec __attribute__((ext_vector_type(CE)));
    const int lane = threadIdx.x & 63;
    const int64_t t = block_of_grid() * 4 + (threadIdx.x >> 6);
    if (t >= a.total_tokens) return;
    const int chunks = a.dl / CE;
    // the token's own loads do not wait for its place
    vec x[NC];
    const E* c = (const E*)a.c + t * a.c_token_stride;
#pragma unroll
    for (int k = 0; k < NC; ++k)
        if (lane + 64 * k < chunks) x[k] = *reinterpret_cast<const vec*>(c + (lane + 64 * k) * CE);

    int seq, n, i;
    if (a.cu_seqlens) {
        seq = sequence_of(a.cu_seqlens, a.num_seqs, t, lane);
        if (seq < 0) return;
        const int first = a.cu_seqlens[seq];
        n = (int)min((int64_t)a.cu_seqlens[seq + 1], a.total_tokens) - first;   // as decode counts them
        i = (int)(t - first);
    } else {
        n = (int)(a.total_tokens / a.num_seqs);
        seq = (int)(t / n);
        i = (int)(t - (int64_t)seq * n);
    }
    const int len = (int)max((int64_t)0, min((int64_t)a.seq_lens[seq], (int64_t)a.max_pages * a.page_size));
    const int position = len - n + i;
    int64_t row = -1;
    if (position >= 0) {
        const int pg = (int)((unsigned)position / (unsigned)a.page_size);
        const int page = a.block_table[(int64_t)seq * a.max_pages + pg];
        if (page >= 0 && page < a.num_pages) row = (int64_t)page * a.page_size + (position - pg * a.page_size);
    }
    E* dst = row < 0 ? nullptr : (E*)a.cache + row * (a.dl + a.dr);

    if (a.norm_weight) {
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if (lane + 64 * k < chunks)
#pragma unroll
                for (int e = 0; e < CE; ++e) sum += to_f32(x[k][e]) * to_f32(x[k][e]);
#pragma unroll
        for (int d = 32; d >= 1; d >>= 1) sum += __shfl_xor(sum, d);
        const float scale = 1.f / sqrtf(sum / (float)a.dl + a.eps);
#pragma unroll
        for (int k = 0; k < NC; ++k)
            if (lane + 64 * k < chunks)
#pragma unroll
                for (int e = 0; e < CE; ++e)
                    x[k][e] = from_f32<E>(to_f32(x[k][e]) * scale * a.norm_weight[(lane + 64 * k) * CE + e]);
    }
#pragma unroll
    for (int k = 0; k < NC; ++k)
        if (lane + 64 * k < chunks) {
            const int at = (lane + 64 * k) * CE;
            if (dst) *reinterpret_cast<vec*>(dst + at) = x[k];
            if (a.c_out) *reinterpret_cast<vec*>((E*)a.c_out + t * a.dl + at) = x[k];
        }
    if (a.dr == 0) return;
    const E* p = (const E*)a.k_pe + t * a.k_pe_token_stride;
    const int half = a.dr / 2;
    for (int j = lane; j < half; j += 64) {
        const bool inter = a.flags & KDA_ROTARY_INTERLEAVED;
        const int i0 = inter ? 2 * j : j, i1 = inter ? 2 * j + 1 : j + half;
        float u = to_f32(p[i0]), w = to_f32(p[i1]);
        if (a.inv_freq) {
            float cs, sn;
            rotation(position, a.inv_freq[j], false, cs, sn);
            const float y = (u * cs - w * sn) * a.amplitude;
            w = (w * cs + u * sn) * a.amplitude;
            u = y;
        }
        const E eu = from_f32<E>(u), ew = from_f32<E>(w);
        if (dst) dst[a.dl + i0] = eu, dst[a.dl + i1] = ew;
        if (a.k_pe_out) {
            E* q = (E*)a.k_pe_out + t * a.dr;
            q[i0] = eu;
            q[i1] = ew;
        }
    }
}

hipError_t launch_latent_append(const LatentAppend& a, bool bf16_io, hipStream_t stream) {
    const dim3 grid = grid_of((a.total_tokens + 3) / 4);
    if (bf16_io) hipLaunchKernelGGL(latent_append_kernel<bf16>, grid, dim3(256), 0, stream, a);
    else hipLaunchKernelGGL(latent_append_kernel<float>, grid, dim3(256), 0, stream, a);
    return launch_result(stream);
}

}  // namespace kda
