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
template <typename T>
__device__ __forceinline__ T max_nan(T a, T b) { return (a > b || a != a) ? a : b; }

__device__ __forceinline__ float round_even(float x) { return rintf(x); }
__device__ __forceinline__ double round_even(double x) { return rint(x); }
__device__ __forceinline__ float mul_add(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double mul_add(double a, double b, double c) { return fma(a, b, c); }

// x / s rounded to a whole number, ties to even, by way of inv = 1 / s.  What
// the product's rounding may have made of a quotient next to a border is put
// right by the remainder x - q s, which is exact: of numbers of 24 bits for
// float x (s has 24), of 53 and 24 for double x.
template <typename T>
__device__ __forceinline__ int quantise(T x, T s, T inv, int lo, int hi)
{
    T q = round_even(x * inv);
    const T r = mul_add(-q, s, x), twice = r + r;
    const bool up = twice > s, down = twice < -s, tie = twice == s || twice == -s;
    if (up || down || tie) {
        const T step = twice > T(0) ? T(1) : T(-1);
        if (!tie || (int(q) & 1)) q += step;
    }
    return max(lo, min(hi, int(q)));
}

// One vector into its cache row; lane l of the warp holds elements [l E, l E + E).
// The codes are the definition's for the given values, float or double.
template <int E, typename T>
__device__ void store_row(const CacheView &c, uint8_t *codes, uint8_t *scales, long long row, int lane, const T (&x)[E])
{
    constexpr int D = 32 * E;
    if (c.fmt == kF16 || c.fmt == kBF16) {
        float f[E];
#pragma unroll
        for (int e = 0; e < E; ++e) f[e] = float(x[e]);
        store_vals<E>(codes, row * D + lane * E, c.fmt, f);
        return;
    }
    T m = fabs(x[0]);
#pragma unroll
    for (int e = 1; e < E; ++e) m = max_nan(m, T(fabs(x[e])));
    const int span = c.fmt == kI8 ? 32 : 32 / E;   // lanes that share a scale
    for (int o = 1; o < span; o <<= 1) m = max_nan(m, __shfl_xor_sync(~0u, m, o));
    int q[E];
    if (c.fmt == kI8) {
        const float s = float(double(m) / 127.0);
        const bool live = s > 0.f && !isinf(s);
        const T inv = T(1) / T(s);   // (infinite for the least of s: then the long way)
#pragma unroll
        for (int e = 0; e < E; ++e)
            q[e] = !live ? 0 : !isinf(inv) ? quantise<T>(x[e], T(s), inv, -127, 127)
                                           : max(-127, min(127, int(rint(double(x[e]) / double(s)))));
        if (lane == 0) reinterpret_cast<float *>(scales)[row] = s;
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) w |= uint32_t(q[e] & 255) << (8 * e);
        if (E == 4) reinterpret_cast<uint32_t *>(codes)[row * 32 + lane] = w;
        else reinterpret_cast<uint16_t *>(codes)[row * 32 + lane] = uint16_t(w);
    } else {
        const __half h = __double2half(double(m) / 7.0);
        const float s = __half2float(h);
        const bool live = s > 0.f && !isinf(s);
        const T inv = T(1) / T(s);
#pragma unroll
        for (int e = 0; e < E; ++e) q[e] = live ? quantise<T>(x[e], T(s), inv, -8, 7) : 0;
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
// for keys); `turn` the cosines and sines in that type, `buf` the warp's own row
// of shared memory.
template <int E, typename T, typename T2>
__device__ void norm_rotate(const AppendParams &p, const float *weight, const T2 *turn, T *buf, int lane, T (&x)[E])
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
        const T co = turn[pair].x, si = turn[pair].y;
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
    __shared__ float2 turn_f[64];
    __shared__ double rows[kAppendWarps][D];
    after_previous();
    const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const int pos = p.pos[t], seq = p.seq ? p.seq[t] : t;
    if (pos < 0) return;
    const long long row0 = row_of(p.c, seq, pos, p.err);
    if (row0 < 0) return;
    for (int i = threadIdx.x; i < p.rotary / 2; i += blockDim.x) {
        double s, c;
        sincos(double(pos) * p.freq[i], &s, &c);
        turn[i] = make_double2(c, s);
        turn_f[i] = make_float2(float(c), float(s));
    }
    __syncthreads();
    const int total = p.heads + 2 * p.kv_heads;
    for (int h = blockIdx.y * kAppendWarps + warp; h < total; h += gridDim.y * kAppendWarps) {
        float f[E];
        if (h < p.heads) {
            load_vals<E>(p.q, t * p.qs + (long long)h * D + lane * E, p.dt, f);
            norm_rotate<E, float>(p, p.qn, turn_f, reinterpret_cast<float *>(rows[warp]), lane, f);
            store_vals<E>(p.q_out, t * p.os + (long long)h * D + lane * E, p.dt, f);
            continue;
        }
        const bool is_k = h < p.heads + p.kv_heads;
        const int head = h - p.heads - (is_k ? 0 : p.kv_heads);
        const long long row = row0 + (long long)head * p.c.head_rows;
        load_vals<E>(is_k ? p.k : p.v, t * (is_k ? p.kstr : p.vstr) + (long long)head * D + lane * E, p.dt, f);
        if (is_k && (p.rotary || p.eps > 0.f)) {
            double x[E];
#pragma unroll
            for (int e = 0; e < E; ++e) x[e] = f[e];
            norm_rotate<E, double>(p, p.kn, turn, rows[warp], lane, x);
            store_row<E>(p.c, p.c.k, p.c.ks, row, lane, x);
        } else {
            store_row<E>(p.c, is_k ? p.c.k : p.c.v, is_k ? p.c.ks : p.c.vs, row, lane, f);
        }
    }
}

// Eight elements of a cache row: what is loaded, and as floats.
template <int FMT>
struct Eight {
    uint4 w;
    float s;
    __device__ __forceinline__ void load(const uint8_t *codes, const uint8_t *scales, long long row, int D, int at)
    {
        const long long i = row * D + at;
        if (FMT == kI8) {
            const uint2 v = *reinterpret_cast<const uint2 *>(codes + i);
            w.x = v.x, w.y = v.y;
            s = reinterpret_cast<const float *>(scales)[row];
        } else if (FMT == kI4) {
            w.x = *reinterpret_cast<const uint32_t *>(codes + i / 2);
            s = __half2float(reinterpret_cast<const __half *>(scales)[i / 32]);
        } else {
            w = *reinterpret_cast<const uint4 *>(codes + 2 * i);
        }
    }
    __device__ __forceinline__ void values(float (&v)[8]) const
    {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if (FMT == kI8) v[e] = s * float(int8_t(u[e / 4] >> (8 * (e & 3))));
            else if (FMT == kI4) v[e] = s * float(int((u[0] >> (4 * e)) & 15) - 8);
            else {
                const float2 f = FMT == kF16 ? __half22float2(*reinterpret_cast<const __half2 *>(&u[e / 2]))
                                             : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e / 2]));
                v[e] = e & 1 ? f.y : f.x;
            }
        }
    }
};

// Bound by the bytes written (for 4 bits to bf16, 8 of 10.25).  A warp takes up
// to 32 tokens, whose places its lanes look up at once, and moves a token's heads
// in pieces of 8 elements for each lane, four of K and four of V under way.
constexpr int kReadWarps = 8;
template <int FMT, int D>
__global__ void __launch_bounds__(32 * kReadWarps) k_read(ReadParams p, int block)
{
    after_previous();
    const int lane = threadIdx.x % 32, per = p.kv_heads * (D / 8);   // pieces of a token
    const int base = (blockIdx.x * kReadWarps + threadIdx.x / 32) * block;
    long long my_row = -1;
    if (lane < block && base + lane < p.tokens)
        my_row = row_of(p.c, p.seq ? p.seq[base + lane] : base + lane, p.pos[base + lane], p.err);
    for (int b = 0; b < block; ++b) {
        const long long row0 = __shfl_sync(~0u, my_row, b);
        if (row0 < 0) continue;
        const long long out = (long long)(base + b) * per;
        for (int c0 = lane; c0 < per; c0 += 128) {
            Eight<FMT> x[2][4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int c = c0 + 32 * i;
                if (c >= per) break;
                const long long row = row0 + (long long)(c / (D / 8)) * p.c.head_rows;
                x[0][i].load(p.c.k, p.c.ks, row, D, c % (D / 8) * 8);
                x[1][i].load(p.c.v, p.c.vs, row, D, c % (D / 8) * 8);
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c0 + 32 * i >= per) break;
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    float v[8];
                    x[kv][i].values(v);
                    uint8_t *dst = kv ? p.v : p.k;
                    const long long j = out + c0 + 32 * i;
                    if (p.dt == kF32) {
                        float4 *o = reinterpret_cast<float4 *>(reinterpret_cast<float *>(dst) + j * 8);
                        o[0] = make_float4(v[0], v[1], v[2], v[3]);
                        o[1] = make_float4(v[4], v[5], v[6], v[7]);
                    } else {
                        *reinterpret_cast<uint4 *>(dst + j * 16) = make_uint4(pack2(v[0], v[1], p.dt), pack2(v[2], v[3], p.dt),
                                                                              pack2(v[4], v[5], p.dt), pack2(v[6], v[7], p.dt));
                    }
                }
            }
        }
    }
}

template <int FMT>
cudaError_t read_launch(const ReadParams &p, cudaStream_t st)
{
    // tokens of a warp: so many that each SM has 32 warps of them, 32 at most
    int block = (p.tokens + 32 * p.n_sm - 1) / (32 * p.n_sm);
    if (block > 32) block = 32;
    const int grid = (p.tokens + block * kReadWarps - 1) / (block * kReadWarps);
    return launch_close(p.dim == 128 ? k_read<FMT, 128> : k_read<FMT, 64>, dim3(grid), 32 * kReadWarps, 0, st, 1, p, block);
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
    return launch_close(p.dim == 128 ? k_append<4> : k_append<2>, grid, 32 * kAppendWarps, 0, st, 1, p);
}

cudaError_t kv_read(const ReadParams &p, cudaStream_t st)
{
    switch (p.c.fmt) {
    case kF16: return read_launch<kF16>(p, st);
    case kBF16: return read_launch<kBF16>(p, st);
    case kI8: return read_launch<kI8>(p, st);
    default: return read_launch<kI4>(p, st);
    }
}

}  // namespace pi
