// pi_kv.cu -- the cache write (norm of each head, rotation, quantisation) and
// the cache read of the attention half of a decode layer.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pi_attn.h"

namespace pi {
namespace {

__device__ __forceinline__ void raise(int *err) { atomicExch(err, int(kDevCheck)); }

// Row number of (sequence, position) for head 0, or -1 (an empty place, or out
// of range: reported).
__device__ long long row_of(const CacheView &c, int seq, int pos, int *err)
{
    if (pos < 0) return -1;
    const int col = pos >> c.page_shift;
    if (seq < 0 || seq >= c.n_seqs || col >= c.width) {
        raise(err);
        return -1;
    }
    const int page = c.table[seq * c.tstride + col];
    if (page < 0 || page >= c.n_pages) {
        raise(err);
        return -1;
    }
    return (long long)page * c.page_rows + (long long)(pos & (c.page_size - 1)) * c.slot_rows;
}

// E consecutive values (2 or 4) as floats.
template <int E>
__device__ __forceinline__ void load_vals(const uint8_t *base, long long i, int dt, float (&v)[E])
{
    if (dt == kF32) {
        const float *p = reinterpret_cast<const float *>(base) + i;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const float2 f = *reinterpret_cast<const float2 *>(p + e);
            v[e] = f.x;
            v[e + 1] = f.y;
        }
    } else {
        const uint16_t *p = reinterpret_cast<const uint16_t *>(base) + i;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
            const uint32_t w = *reinterpret_cast<const uint32_t *>(p + e);
            const float2 f = dt == kF16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w))
                                        : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w));
            v[e] = f.x;
            v[e + 1] = f.y;
        }
    }
}

__device__ __forceinline__ uint32_t pack2(float a, float b, int dt)
{
    if (dt == kF16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

template <int E>
__device__ __forceinline__ void store_vals(uint8_t *base, long long i, int dt, const float (&v)[E])
{
#pragma unroll
    for (int e = 0; e < E; e += 2) {
        if (dt == kF32)
            *reinterpret_cast<float2 *>(reinterpret_cast<float *>(base) + i + e) = make_float2(v[e], v[e + 1]);
        else
            *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(base) + i + e) = pack2(v[e], v[e + 1], dt);
    }
}

// The larger of two, NaN if either is.
__device__ __forceinline__ double max_nan(double a, double b) { return (a > b || a != a) ? a : b; }

// One vector into its cache row; lane l of the warp holds elements [l E, l E + E).
// Scale and codes in 64 bits: the codes are the definition's for the given values.
template <int E>
__device__ void store_row(const CacheView &c, uint8_t *codes, uint8_t *scales, long long row, int lane, const double (&x)[E])
{
    constexpr int D = 32 * E;
    if (c.fmt == kF16 || c.fmt == kBF16) {
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = float(x[e]);
        store_vals<E>(codes, row * D + lane * E, c.fmt, f);
        return;
    }
    double m = fabs(x[0]);
#pragma unroll
    for (int e = 1; e < E; ++e) m = max_nan(m, fabs(x[e]));
    const int span = c.fmt == kI8 ? 32 : 32 / E;   // lanes that share a scale
    for (int o = 1; o < span; o <<= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
    int q[E];
    if (c.fmt == kI8) {
        const float s = float(m / 127.0);
        const bool live = s > 0.f && !isinf(s);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = live ? max(-127, min(127, int(rint(x[e] / double(s))))) : 0;
        if (lane == 0) reinterpret_cast<float *>(scales)[row] = s;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) w |= uint32_t(q[e] & 255) << (8 * e);
        if (E == 4) reinterpret_cast<uint32_t *>(codes)[row * 32 + lane] = w;
        else reinterpret_cast<uint16_t *>(codes)[row * 32 + lane] = uint16_t(w);
    } else {
        const __half h = __double2half(m / 7.0);
        const float s = __half2float(h);
        const bool live = s > 0.f && !isinf(s);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = live ? max(-8, min(7, int(rint(x[e] / double(s))))) : 0;
        if (lane % span == 0) reinterpret_cast<__half *>(scales)[row * (D / 32) + lane / span] = h;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) w |= uint32_t((q[e] + 8) & 15) << (4 * e);
        if (E == 4) reinterpret_cast<uint16_t *>(codes)[row * 32 + lane] = uint16_t(w);
        else codes[row * 32 + lane] = uint8_t(w);
    }
}

__device__ __forceinline__ float root_inv(float x) { return 1.f / sqrtf(x); }
__device__ __forceinline__ double root_inv(double x) { return 1.0 / sqrt(x); }

// Norm and rotation of one head's vector in type T (float for queries, double
// for keys); `buf` is the warp's own row of shared memory.
template <int E, typename T>
__device__ void norm_rotate(const AppendParams &p, const float *weight, const double2 *turn, T *buf, int lane, T (&x)[E])
{
    if (p.eps > 0.f) {
        T ss = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) ss += x[e] * x[e];
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        const T r = root_inv(ss / T(32 * E) + T(p.eps));
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = x[e] * r * (weight ? T(weight[lane * E + e]) : T(1));
    }
    if (!p.rotary) return;
#pragma unroll
    for (int e = 0; e < E; ++e) buf[lane * E + e] = x[e];
    __syncwarp();
    const int half = p.rotary / 2;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        const int i = lane * E + e;
        if (i >= p.rotary) continue;
        const int pair = p.pairs ? i >> 1 : (i < half ? i : i - half);
        const bool first = p.pairs ? !(i & 1) : i < half;
        const T other = buf[p.pairs ? i ^ 1 : (first ? i + half : i - half)];
        const T co = T(turn[pair].x), si = T(turn[pair].y);
        x[e] = first ? x[e] * co - other * si : x[e] * co + other * si;
    }
    __syncwarp();
}

constexpr int kAppendWarps = 4;

template <int E>
__global__ void __launch_bounds__(32 * kAppendWarps) k_append(AppendParams p)
{
    constexpr int D = 32 * E;
    __shared__ double2 turn[64];
    __shared__ double rows[kAppendWarps][D];
    const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int pos = p.pos[t], seq = p.seq ? p.seq[t] : t;
    if (pos < 0) return;
    const long long row0 = row_of(p.c, seq, pos, p.err);
    if (row0 < 0) return;
    for (int i = threadIdx.x; i < p.rotary / 2; i += blockDim.x) {
        double s, c;
        sincos(double(pos) * p.freq[i], &s, &c);
        turn[i] = make_double2(c, s);
    }
    __syncthreads();
    const int total = p.heads + 2 * p.kv_heads;
    for (int h = blockIdx.y * kAppendWarps + warp; h < total; h += gridDim.y * kAppendWarps) {
        float f[E];
        if (h < p.heads) {
            load_vals<E>(p.q, t * p.qs + (long long)h * D + lane * E, p.dt, f);
            norm_rotate<E, float>(p, p.qn, turn, reinterpret_cast<float *>(rows[warp]), lane, f);
            store_vals<E>(p.q_out, t * p.os + (long long)h * D + lane * E, p.dt, f);
            continue;
        }
        const bool is_k = h < p.heads + p.kv_heads;
        const int head = h - p.heads - (is_k ? 0 : p.kv_heads);
        const long long row = row0 + (long long)head * p.c.head_rows;
        double x[E];
        load_vals<E>(is_k ? p.k : p.v, t * (is_k ? p.kstr : p.vstr) + (long long)head * D + lane * E, p.dt, f);
#pragma unroll
        for (int e = 0; e < E; ++e) x[e] = f[e];
        if (is_k) norm_rotate<E, double>(p, p.kn, turn, rows[warp], lane, x);
        store_row<E>(p.c, is_k ? p.c.k : p.c.v, is_k ? p.c.ks : p.c.vs, row, lane, x);
    }
}

// Eight consecutive elements of a cache row as floats; `i` counts elements from
// the start of the cache.
__device__ __forceinline__ void read8(const CacheView &c, const uint8_t *codes, const uint8_t *scales, long long row, int D,
                                      int at, float (&v)[8])
{
    const long long i = row * D + at;
    if (c.fmt == kI8) {
        const uint2 w = *reinterpret_cast<const uint2 *>(codes + i);
        const float s = reinterpret_cast<const float *>(scales)[row];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s * float(int8_t((e < 4 ? w.x : w.y) >> (8 * (e & 3))));
    } else if (c.fmt == kI4) {
        const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + i / 2);
        const float s = __half2float(reinterpret_cast<const __half *>(scales)[i / 32]);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = s * float(int((w >> (4 * e)) & 15) - 8);
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(codes + 2 * i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = c.fmt == kF16 ? __half22float2(*reinterpret_cast<const __half2 *>(&u[e]))
                                           : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e]));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
}

__global__ void __launch_bounds__(256) k_read(ReadParams p)
{
    const int per = p.kv_heads * p.dim / 8;   // pieces of 8 elements of one token
    const long long n = (long long)p.tokens * per;
    const bool is_v = blockIdx.y;
    for (long long j = blockIdx.x * 256LL + threadIdx.x; j < n; j += gridDim.x * 256LL) {
        const int t = int(j / per), piece = int(j - (long long)t * per);
        const int head = piece / (p.dim / 8), at = piece % (p.dim / 8) * 8;
        const long long row0 = row_of(p.c, p.seq ? p.seq[t] : t, p.pos[t], p.err);
        if (row0 < 0) continue;
        float v[8];
        read8(p.c, is_v ? p.c.v : p.c.k, is_v ? p.c.vs : p.c.ks, row0 + (long long)head * p.c.head_rows, p.dim, at, v);
        uint8_t *dst = is_v ? p.v : p.k;
        if (p.dt == kF32) {
            float4 *o = reinterpret_cast<float4 *>(reinterpret_cast<float *>(dst) + j * 8);
            o[0] = make_float4(v[0], v[1], v[2], v[3]);
            o[1] = make_float4(v[4], v[5], v[6], v[7]);
        } else {
            *reinterpret_cast<uint4 *>(dst + j * 16) =
                make_uint4(pack2(v[0], v[1], p.dt), pack2(v[2], v[3], p.dt), pack2(v[4], v[5], p.dt), pack2(v[6], v[7], p.dt));
        }
    }
}

}  // namespace

cudaError_t kv_append(const AppendParams &p, cudaStream_t st)
{
    const int total = p.heads + 2 * p.kv_heads;
    // a token's heads over several CTAs while there are few tokens
    int split = (2 * p.n_sm + p.tokens - 1) / p.tokens;
    const int most = (total + kAppendWarps - 1) / kAppendWarps;
    if (split > most) split = most;
    const dim3 grid(p.tokens, split);
    if (p.dim == 128) k_append<4><<<grid, 32 * kAppendWarps, 0, st>>>(p);
    else k_append<2><<<grid, 32 * kAppendWarps, 0, st>>>(p);
    return cudaGetLastError();
}

cudaError_t kv_read(const ReadParams &p, cudaStream_t st)
{
    const long long n = (long long)p.tokens * p.kv_heads * p.dim / 8;
    long long blocks = (n + 255) / 256;
    if (blocks > 8LL * p.n_sm) blocks = 8LL * p.n_sm;
    k_read<<<dim3(unsigned(blocks), 2), 256, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace pi
