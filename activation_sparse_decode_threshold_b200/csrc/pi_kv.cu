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

__device__ __forceinline__ uint32_t pack2(float a, float b, int dt)
{
    if (dt == kF16) {
        const __half2 h = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<const uint32_t *>(&h);
}

// N consecutive values (2, 4 or 8), aligned to their size.
template <int DT, int N>
__device__ __forceinline__ void load_vals(const uint8_t *base, long long i, float (&v)[N])
{
    if (DT == kF32) {
        const float *p = reinterpret_cast<const float *>(base) + i;
        if (N == 2) {
            const float2 a = *reinterpret_cast<const float2 *>(p);
            v[0] = a.x, v[1] = a.y;
        } else {
#pragma unroll
            for (int e = 0; e < N / 4; ++e) {
                const float4 a = reinterpret_cast<const float4 *>(p)[e];
                v[4 * e] = a.x, v[4 * e + 1] = a.y, v[(4 * e + 2) % N] = a.z, v[(4 * e + 3) % N] = a.w;
            }
        }
    } else {
        uint32_t u[N / 2];
        if (N == 8) {
            const uint4 w = *reinterpret_cast<const uint4 *>(base + 2 * i);
            u[0] = w.x, u[1 % (N / 2)] = w.y, u[2 % (N / 2)] = w.z, u[3 % (N / 2)] = w.w;
        } else if (N == 4) {
            const uint2 w = *reinterpret_cast<const uint2 *>(base + 2 * i);
            u[0] = w.x, u[1 % (N / 2)] = w.y;
        } else {
            u[0] = *reinterpret_cast<const uint32_t *>(base + 2 * i);
        }
#pragma unroll
        for (int e = 0; e < N / 2; ++e) {
            const float2 f = DT == kF16 ? __half22float2(*reinterpret_cast<const __half2 *>(&u[e]))
                                        : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e]));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
}
template <int N>
__device__ __forceinline__ void store_vals(uint8_t *base, long long i, int dt, const float (&v)[N])
{
    if (dt == kF32) {
        float *p = reinterpret_cast<float *>(base) + i;
        if (N == 2) *reinterpret_cast<float2 *>(p) = make_float2(v[0], v[1]);
        else
#pragma unroll
            for (int e = 0; e < N / 4; ++e)
                reinterpret_cast<float4 *>(p)[e] = make_float4(v[4 * e], v[4 * e + 1], v[(4 * e + 2) % N], v[(4 * e + 3) % N]);
    } else {
        uint32_t u[N / 2];
#pragma unroll
        for (int e = 0; e < N / 2; ++e) u[e] = pack2(v[2 * e], v[2 * e + 1], dt);
        if (N == 8) *reinterpret_cast<uint4 *>(base + 2 * i) = make_uint4(u[0], u[1 % (N / 2)], u[2 % (N / 2)], u[3 % (N / 2)]);
        else if (N == 4) *reinterpret_cast<uint2 *>(base + 2 * i) = make_uint2(u[0], u[1 % (N / 2)]);
        else *reinterpret_cast<uint32_t *>(base + 2 * i) = u[0];
    }
}

// Magnitudes as whole numbers, in whose order infinity and NaN come last.
__device__ __forceinline__ unsigned magnitude(float x) { return __float_as_uint(x) & 0x7fffffffu; }
__device__ __forceinline__ unsigned long long magnitude(double x) { return (unsigned long long)__double_as_longlong(x) & 0x7fffffffffffffffull; }
__device__ __forceinline__ double value(unsigned m) { return double(__uint_as_float(m)); }
__device__ __forceinline__ double value(unsigned long long m) { return __longlong_as_double((long long)m); }

// m / n, rounded correctly: the product with 1 / n and one step by the remainder.
template <int N>
__device__ __forceinline__ double over(double m)
{
    const double q = m * (1.0 / N), r = fma(-double(N), q, m);
    return isfinite(q) ? fma(r, 1.0 / N, q) : q;
}

__device__ __forceinline__ float round_even(float x) { return rintf(x); }
__device__ __forceinline__ double round_even(double x) { return rint(x); }
__device__ __forceinline__ float mul_add(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ double mul_add(double a, double b, double c) { return fma(a, b, c); }

// x / s rounded to a whole number, ties to even, by way of inv, about 1 / s.
// What inv has made of a quotient next to a border is put right by the remainder
// x - q s, which is exact: of numbers of 24 bits for float x (s has 24), of 53
// and 24 for double x.
template <typename T>
__device__ __forceinline__ int quantise(T x, T s, T inv, int lo, int hi)
{
    const T q = round_even(x * inv), r = mul_add(-q, s, x), twice = r < T(0) ? -(r + r) : r + r;
    int n = int(q);
    if (twice > s || (twice == s && (n & 1))) n += r > T(0) ? 1 : -1;
    return max(lo, min(hi, n));
}

// Elements [at, at + N) of a vector into its cache row; the D / N lanes side by
// side that hold it are all here (`live` false: without a row to write).  The codes
// are the definition's for the given values, float or double.
template <int D, int N, typename T>
__device__ __forceinline__ void store_row(const CacheView &c, uint8_t *codes, uint8_t *scales, long long row, int at, bool live,
                                          const T (&x)[N])
{
    const long long i = row * D + at;
    if (c.fmt == kF16 || c.fmt == kBF16) {
        float f[N];
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = float(x[e]);
        if (live) store_vals<N>(codes, i, c.fmt, f);
        return;
    }
    auto m = magnitude(x[0]);
#pragma unroll
    for (int e = 1; e < N; ++e) m = max(m, magnitude(x[e]));
#pragma unroll
    for (int o = 1; o < 32 / N; o <<= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
    if (c.fmt == kI8) {
#pragma unroll
        for (int o = 32 / N; o < D / N; o <<= 1) m = max(m, __shfl_xor_sync(~0u, m, o));
        const float s = float(over<127>(value(m)));
        const bool some = s > 0.f && !isinf(s);
        const float inv = 1.f / s;   // (infinite for the least of s: then the long way)
        uint32_t w[2] = {0, 0};
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int q = !some ? 0 : inv < 1e38f ? quantise<T>(x[e], T(s), T(inv), -127, 127)
                                                  : max(-127, min(127, int(rint(double(x[e]) / double(s)))));
            w[e / 4] |= uint32_t(q & 255) << (8 * (e & 3));
        }
        if (live) {
            if (N == 8) *reinterpret_cast<uint2 *>(codes + i) = make_uint2(w[0], w[1]);
            else if (N == 4) *reinterpret_cast<uint32_t *>(codes + i) = w[0];
            else *reinterpret_cast<uint16_t *>(codes + i) = uint16_t(w[0]);
            if (at == 0) reinterpret_cast<float *>(scales)[row] = s;
        }
    } else {
        const __half h = __double2half(over<7>(value(m)));
        const float s = __half2float(h);
        const bool some = s > 0.f && !isinf(s);
        const T inv = T(1.f / s);
        uint32_t w = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) w |= uint32_t(((some ? quantise<T>(x[e], T(s), inv, -8, 7) : 0) + 8) & 15) << (4 * e);
        if (live) {
            if (N == 8) *reinterpret_cast<uint32_t *>(codes + i / 2) = w;
            else if (N == 4) *reinterpret_cast<uint16_t *>(codes + i / 2) = uint16_t(w);
            else codes[i / 2] = uint8_t(w);
            if (at % 32 == 0) reinterpret_cast<__half *>(scales)[i / 32] = h;
        }
    }
}

__device__ __forceinline__ float root_inv(float x) { return rsqrtf(x); }   // (off by 2 units of 2^-23 at most)
__device__ __forceinline__ double root_inv(double x) { return rsqrt(x); }

// Places in a vector's row of shared memory: more after each 8, so that lanes with
// 8 elements each meet no bank twice (512 tokens into 4 bits: 9.8 us, without 12.2).
__device__ __forceinline__ int spread(int i) { return i + (i >> 3); }
// The same for cosines and sines: whole 16 bytes.
__device__ __forceinline__ int spread(int i, float2) { return i + 2 * (i >> 3); }
__device__ __forceinline__ int spread(int i, double2) { return i + (i >> 3); }

// Norm and rotation of elements [at, at + N) of a vector, its other lanes side by
// side; float for queries, double for keys.  turn: cosine and sine of each
// element, the sine negative for the first of a pair; other: places of their
// partners in `buf`.
template <int D, int N, typename T, typename T2>
__device__ __forceinline__ void norm_rotate(const AppendParams &p, const float (&w)[N], const T2 *turn, const int (&other)[N], T *buf,
                                            int at, T (&x)[N])
{
    if (p.eps > 0.f) {
        T ss = 0;
#pragma unroll
        for (int e = 0; e < N; ++e) ss += x[e] * x[e];
#pragma unroll
        for (int o = D / N / 2; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
        T r = root_inv(ss * T(1.0 / D) + T(p.eps));
        // fp32 squares end at numbers of some 1e19: the heads that have larger ones are normed at 2^-80 of their size
        if (sizeof(T) == 4 && __any_sync(~0u, !(ss < T(0x1p120f)))) {
            const T down = ss < T(0x1p120f) ? T(1) : T(0x1p-80f);
            ss = 0;
#pragma unroll
            for (int e = 0; e < N; ++e) {
                x[e] *= down;
                ss += x[e] * x[e];
            }
#pragma unroll
            for (int o = D / N / 2; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
            r = root_inv(ss * T(1.0 / D) + T(p.eps) * down * down);
        }
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] = x[e] * r * T(w[e]);
    }
    if (!p.rotary) return;
#pragma unroll
    for (int e = 0; e < N; ++e) buf[spread(at + e)] = x[e];
    __syncwarp();
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const T2 a = turn[spread(at + e, T2())];
        const T y = x[e] * a.x + buf[other[e]] * a.y;
        x[e] = at + e < p.rotary ? y : x[e];
    }
    __syncwarp();
}

constexpr int kAppendWarps = 4;

// A CTA computes its token's angles once, for its part of the heads; a warp takes
// 32 N / D vectors (of V, K or Q) at a time, N elements to a lane.  Bound by the way from the position to the store where there are few
// tokens, and by instructions (a vector of 128 keys, in 64 bits, takes a warp
// some 300) where there are many; loads are under way before the angles, and each
// later one before its turn.  32 + 2 x 8 heads of 128 into 4 bits: one token 3.5
// us, 512 tokens 9.8 us.
template <int D, int N, int DT>
__global__ void __launch_bounds__(32 * kAppendWarps) k_append(AppendParams p)
{
    constexpr int L = D / N, V = 32 / L, W = kAppendWarps;   // lanes of a vector, vectors of a warp
    __shared__ double2 turn[D + D / 8];
    __shared__ __align__(16) float2 turn_f[D + D / 4];
    __shared__ double rows[W][V][D + D / 8];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, at = lane % L * N, mine = lane / L;
    after_previous();
    const int t = blockIdx.x, pos = p.pos[t];
    if (pos < 0) return;
    const int kv_tasks = (p.kv_heads + V - 1) / V, tasks = 2 * kv_tasks + (p.heads + V - 1) / V, step = gridDim.y * W;
    // task j: vectors V j' + mine of V, K or Q
    auto head_of = [&](int j) { return (j < kv_tasks ? j : j < 2 * kv_tasks ? j - kv_tasks : j - 2 * kv_tasks) * V + mine; };
    auto load = [&](int j, float (&f)[N]) {
        const int h = head_of(j), heads = j < 2 * kv_tasks ? p.kv_heads : p.heads;
        const uint8_t *src = j < kv_tasks ? p.v : j < 2 * kv_tasks ? p.k : p.q;
        const long long row = t * (j < kv_tasks ? p.vstr : j < 2 * kv_tasks ? p.kstr : p.qs);
        if (h < heads) load_vals<DT, N>(src, row + h * D + at, f);
    };
    int j = blockIdx.y * W + warp;
    float f[N] = {}, qw[N], kw[N];
    if (j < tasks) load(j, f);
#pragma unroll
    for (int e = 0; e < N; ++e) {
        qw[e] = p.qn ? p.qn[at + e] : 1.f;
        kw[e] = p.kn ? p.kn[at + e] : 1.f;
    }
    const long long row0 = row_of(p.c, p.seq ? p.seq[t] : t, pos, p.err);
    const int half = p.rotary / 2;
    for (int i = threadIdx.x; i < half; i += 32 * W) {
        double s, c;
        sincos(double(pos) * p.freq[i], &s, &c);
        const int a = p.pairs ? 2 * i : i, b = p.pairs ? 2 * i + 1 : i + half;
        turn[spread(a, double2())] = make_double2(c, -s);
        turn[spread(b, double2())] = make_double2(c, s);
        turn_f[spread(a, float2())] = make_float2(float(c), float(-s));
        turn_f[spread(b, float2())] = make_float2(float(c), float(s));
    }
    // V needs no angles
#pragma unroll 1
    for (; j < kv_tasks && row0 >= 0; j += step) {
        float next[N] = {};
        if (j + step < tasks) load(j + step, next);
        const int h = head_of(j);
        store_row<D, N>(p.c, p.c.v, p.c.vs, row0 + (long long)h * p.c.head_rows, at, h < p.kv_heads, f);
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = next[e];
    }
    __syncthreads();
    if (row0 < 0) return;
    int other[N];
#pragma unroll
    for (int e = 0; e < N; ++e) {
        const int i = at + e;
        other[e] = spread(i >= p.rotary ? i : p.pairs ? i ^ 1 : i < half ? i + half : i - half);
    }
#pragma unroll 1
    for (; j < tasks; j += step) {
        float next[N] = {};
        if (j + step < tasks) load(j + step, next);
        const int h = head_of(j);
        if (j >= 2 * kv_tasks) {
            norm_rotate<D, N, float>(p, qw, turn_f, other, reinterpret_cast<float *>(rows[warp][mine]), at, f);
            if (h < p.heads) store_vals<N>(p.q_out, t * p.os + h * D + at, DT, f);
        } else {
            const long long row = row0 + (long long)h * p.c.head_rows;
            if (p.rotary || p.eps > 0.f) {
                double x[N];
#pragma unroll
                for (int e = 0; e < N; ++e) x[e] = f[e];
                norm_rotate<D, N, double>(p, kw, turn, other, rows[warp][mine], at, x);
                store_row<D, N>(p.c, p.c.k, p.c.ks, row, at, h < p.kv_heads, x);
            } else {
                store_row<D, N>(p.c, p.c.k, p.c.ks, row, at, h < p.kv_heads, f);
            }
        }
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = next[e];
    }
}

template <int D, int N>
cudaError_t append_launch(const AppendParams &p, cudaStream_t st, int ctas)
{
    constexpr int V = 32 * N / D;
    const int tasks = 2 * ((p.kv_heads + V - 1) / V) + (p.heads + V - 1) / V, most = (tasks + kAppendWarps - 1) / kAppendWarps;
    // a token's vectors over as many CTAs as can all run at once
    int split = ctas * p.n_sm / p.tokens;
    split = split < 1 ? 1 : split > most ? most : split;
    return launch_close(p.dt == kF32 ? k_append<D, N, kF32> : p.dt == kF16 ? k_append<D, N, kF16> : k_append<D, N, kBF16>,
                        dim3(p.tokens, split), 32 * kAppendWarps, 0, st, 1, p);
}

// Few tokens: 4 elements to a lane, the shorter way (one token of 32 + 2 x 8 heads of 128 into 4 bits: 3.5 us, with 8
// elements 4.3).  Many: 8, in fewer instructions (512 tokens 9.8 us, with 4 elements 13).  Both are even at 64 to 130.
template <int D>
cudaError_t append_by_tokens(const AppendParams &p, cudaStream_t st)
{
    return p.tokens > p.n_sm ? append_launch<D, 8>(p, st, 5) : append_launch<D, 4>(p, st, 4);
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

// Bound by the bytes written (for 4 bits to bf16, 8 of 10.25): 8 x 4096 rows of 8
// heads of 128 take 33 us, 5.2 TB/s in all.  A warp takes up
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
    // tokens of a warp: so many that there are 128 warps for each SM, in turns (8 x 4096 rows of 4 bits: 2 tokens, 32.9 us;
    // one 38.9, four 35.7, seven, at once, 35.2), 32 at most
    int block = (p.tokens + 128 * p.n_sm - 1) / (128 * p.n_sm);
    if (block > 32) block = 32;
    const int grid = (p.tokens + block * kReadWarps - 1) / (block * kReadWarps);
    return launch_close(p.dim == 128 ? k_read<FMT, 128> : k_read<FMT, 64>, dim3(grid), 32 * kReadWarps, 0, st, 1, p, block);
}

}  // namespace

cudaError_t kv_append(const AppendParams &p, cudaStream_t st)
{
    return p.dim == 128 ? append_by_tokens<128>(p, st) : append_by_tokens<64>(p, st);
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
