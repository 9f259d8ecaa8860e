// pi_int4.cu -- products of an INT4 group-32 matrix with a few tokens.
//
// y[t][i] = sum over groups j of s[i][j] * sum over the group's 32 columns of
// (n - 8) x.  The inner sums run on the tensor cores (mma.sync m16n8k16, rows of
// W as A, tokens as the columns of B): n - 8 is exact in 16 bits and x is given
// in 16-bit parts that hold all of it, so the products are exact and only the
// fp32 sums round.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pi_attn.h"

namespace pi {
namespace {

constexpr int kWarps = 8;
constexpr int kThreadsMv = 32 * kWarps;
constexpr int kXBytes = 112 * 1024;    // shared memory for a chunk of x: 512 columns of 96 parts at least

// Unit (row tile, 64 columns): lane (g = lane / 4, t = lane % 4) finds at 16 lane
// the eight columns 8t .. 8t+7 of rows g and g + 8, first of the unit's first
// group, then of its second.  A word's nibbles 0, 4, 1, 5, 2, 6, 3, 7 are its
// columns in order, so that masking with 0x000f000f after shifts by 0, 4, 8, 12
// gives the 16-bit pairs of the matrix fragments.  Scales: 8 bytes for each g.
__global__ void k_pack(const uint8_t *q, const uint16_t *s, uint8_t *dst, int n, int k, int ku, long long units)
{
    const int lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const long long u = blockIdx.x * 8LL + threadIdx.x / 32;
    if (u >= units) return;
    const long long tile = u / ku;
    const int col = int(u - tile * ku) * 64;
    uint32_t w[4];
    for (int i = 0; i < 4; ++i) {   // group i / 2, row g + 8 (i % 2)
        const long long row = tile * 16 + g + 8 * (i & 1);
        const int c = col + 32 * (i >> 1);
        uint32_t v = 0x88888888u;
        if (row < n && c < k) v = *reinterpret_cast<const uint32_t *>(q + row * (k / 2) + c / 2 + 4 * t);
        uint32_t r = 0;
        for (int e = 0; e < 8; ++e) r |= ((v >> (4 * e)) & 15u) << (4 * ((e & 1) * 4 + (e >> 1)));
        w[i] = r;
    }
    uint8_t *out = dst + u * kInt4Unit;
    *reinterpret_cast<uint4 *>(out + 16 * lane) = make_uint4(w[0], w[1], w[2], w[3]);
    const long long row = tile * 16 + g + 8 * (t & 1);
    const int c = col + 32 * (t >> 1);
    reinterpret_cast<uint16_t *>(out + 512)[g * 4 + t] = row < n && c < k ? s[row * (k / 32) + c / 32] : uint16_t(0);
}

template <bool BF>
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Eight nibbles to four 16-bit pairs n - 8: a nibble under the exponent bits of
// 1024 (fp16) or 128 (bf16) is that number plus n.
template <bool BF>
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&r)[4])
{
    constexpr uint32_t magic = BF ? 0x43004300u : 0x64006400u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t v = ((w >> (4 * i)) & 0x000f000fu) | magic;
        if (BF) {
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), __floats2bfloat162_rn(136.f, 136.f));
            r[i] = *reinterpret_cast<const uint32_t *>(&d);
        } else {
            const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), __floats2half2_rn(1032.f, 1032.f));
            r[i] = *reinterpret_cast<const uint32_t *>(&d);
        }
    }
}

__device__ __forceinline__ void load8(const uint8_t *x, long long i, int xt, float (&v)[8])
{
    if (xt == kF32) {
        const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(x) + i);
        const float4 a = p[0], b = p[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(x + 2 * i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = xt == kF16 ? __half22float2(*reinterpret_cast<const __half2 *>(&u[e]))
                                        : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e]));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
        }
    }
}

// Parts of x: F16 and BF16 are their own 16-bit numbers; an F32 is three bf16
// numbers, each the leading 8 bits of what is left (cut off, so that no part
// overflows; 24 bits in all).  An infinity or NaN stays in the first part.
__device__ __forceinline__ float cut(float v) { return __uint_as_float(__float_as_uint(v) & 0xffff0000u); }

__device__ __forceinline__ float value_of(const uint8_t *p, long long i, int dt)
{
    if (dt == kF32) return reinterpret_cast<const float *>(p)[i];
    if (dt == kF16) return __half2float(reinterpret_cast<const __half *>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
}

// One CTA per tile of 16 rows; the warps share the columns of each chunk of x.
// PARTS: 3 for F32 x, else 1.  NT: tiles of 8 columns of B (tokens * PARTS).
template <bool BF, int PARTS, int NT>
__global__ void __launch_bounds__(kThreadsMv) k_matvec(Int4Params p, int chunk)
{
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float ssq[kInt4MaxTokens][kWarps];
    uint16_t *xs = reinterpret_cast<uint16_t *>(smem);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t4 = lane % 4;
    const int cols = p.tokens * PARTS;
    const int stride = chunk + 32;   // 64 bytes past a multiple of 128: no bank conflicts
    const long long tile = blockIdx.x;
    float acc[NT][4] = {};
    if (p.eps > 0.f) {
        for (int t = 0; t < p.tokens; ++t) {
            float ss = 0.f;
            for (int i = threadIdx.x * 8; i < p.k; i += kThreadsMv * 8) {
                float v[8];
                load8(p.x, t * p.xs + i, p.xt, v);
#pragma unroll
                for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
            }
            for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
            if (lane == 0) ssq[t][warp] = ss;
        }
    }
    for (int k0 = 0; k0 < p.ku * 64; k0 += chunk) {
        const int here = min(chunk, p.ku * 64 - k0);
        __syncthreads();
        for (int i = threadIdx.x; i < p.tokens * (here / 8); i += kThreadsMv) {
            const int t = i / (here / 8), at = i % (here / 8) * 8;
            uint16_t *dst = xs + t * stride + at;
            uint4 w = make_uint4(0, 0, 0, 0);
            if (PARTS == 1) {
                if (k0 + at < p.k) w = *reinterpret_cast<const uint4 *>(p.x + 2 * (t * p.xs + k0 + at));
                *reinterpret_cast<uint4 *>(dst) = w;
            } else {
                float v[8] = {};
                if (k0 + at < p.k) load8(p.x, t * p.xs + k0 + at, p.xt, v);
#pragma unroll
                for (int part = 0; part < PARTS; ++part) {
                    uint32_t u[4];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float c = cut(v[e]);
                        const uint32_t b = isnan(v[e]) ? 0x7fc0u : __float_as_uint(v[e]) >> 16;
                        u[e / 2] = e & 1 ? u[e / 2] | (b << 16) : b;
                        v[e] = isfinite(v[e]) ? v[e] - c : 0.f;
                    }
                    *reinterpret_cast<uint4 *>(dst + part * p.tokens * stride) = make_uint4(u[0], u[1], u[2], u[3]);
                }
            }
        }
        __syncthreads();
        for (int u = warp; u < here / 64; u += kWarps) {
            const uint8_t *w = p.w + (tile * p.ku + k0 / 64 + u) * kInt4Unit;
            const uint4 q = *reinterpret_cast<const uint4 *>(w + 16 * lane);
            const uint2 s = *reinterpret_cast<const uint2 *>(w + 512 + 8 * g);
            const uint32_t qq[4] = {q.x, q.y, q.z, q.w}, sp[2] = {s.x, s.y};
#pragma unroll
            for (int grp = 0; grp < 2; ++grp) {
                uint32_t lo[4], hi[4];
                nibbles<BF>(qq[2 * grp], lo);
                nibbles<BF>(qq[2 * grp + 1], hi);
                const float2 sc = __half22float2(*reinterpret_cast<const __half2 *>(&sp[grp]));
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) {
                    const int col = min(nt * 8 + g, cols - 1);
                    const uint4 b = *reinterpret_cast<const uint4 *>(xs + col * stride + u * 64 + grp * 32 + t4 * 8);
                    float c[4] = {};
                    mma16816<BF>(c, lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                    mma16816<BF>(c, lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                    acc[nt][0] += sc.x * c[0];
                    acc[nt][1] += sc.x * c[1];
                    acc[nt][2] += sc.y * c[2];
                    acc[nt][3] += sc.y * c[3];
                }
            }
        }
    }
    __syncthreads();
    // sums of the warps, in order
    float *red = reinterpret_cast<float *>(smem);   // [warp][16 rows][8 NT]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e)
            red[(warp * 16 + g + 8 * (e >> 1)) * (8 * NT) + nt * 8 + 2 * t4 + (e & 1)] = acc[nt][e];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * p.tokens; i += kThreadsMv) {
        const int r = i % 16, t = i / 16;
        const long long row = tile * 16 + r;
        if (row >= p.n) continue;
        float y = 0.f;
        for (int part = PARTS - 1; part >= 0; --part)
            for (int w = 0; w < kWarps; ++w) y += red[(w * 16 + r) * (8 * NT) + part * p.tokens + t];
        if (p.eps > 0.f) {
            float ss = 0.f;
            for (int w = 0; w < kWarps; ++w) ss += ssq[t][w];
            y *= 1.f / sqrtf(ss / float(p.k) + p.eps);
        }
        const long long at = t * p.ys + row;
        if (p.add) y += value_of(p.add, at, p.yt);
        if (p.yt == kF32) reinterpret_cast<float *>(p.y)[at] = y;
        else if (p.yt == kF16) reinterpret_cast<__half *>(p.y)[at] = __float2half(y);
        else reinterpret_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16(y);
    }
}

static_assert((kXBytes / (3 * kInt4MaxTokens) - 64) / 2 >= 64 * kWarps, "a chunk of x is never empty");
constexpr int smem_bytes(int nt) { return max(kXBytes, 8 * nt * 16 * kWarps * 4); }

template <bool BF, int PARTS, int NT>
cudaError_t launch(const Int4Params &p, cudaStream_t st, bool set)
{
    if (set)
        return cudaFuncSetAttribute(k_matvec<BF, PARTS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem_bytes(NT));
    // columns of x that fit, a multiple of 64 for each warp
    const int cols = p.tokens * PARTS;
    int chunk = (kXBytes / cols - 64) / 2 / (64 * kWarps) * (64 * kWarps);
    if (chunk > p.ku * 64) chunk = (p.ku * 64 + 511) / 512 * 512;
    const int bytes = max(cols * (chunk + 32) * 2, 8 * NT * 16 * kWarps * 4);
    k_matvec<BF, PARTS, NT><<<(p.n + 15) / 16, kThreadsMv, bytes, st>>>(p, chunk);
    return cudaGetLastError();
}

template <bool BF, int PARTS>
cudaError_t by_columns(int nt, const Int4Params &p, cudaStream_t st, bool set)
{
    switch (nt) {
    case 1: return launch<BF, PARTS, 1>(p, st, set);
    case 2: return launch<BF, PARTS, 2>(p, st, set);
    case 3: return launch<BF, PARTS, 3>(p, st, set);
    case 4: return launch<BF, PARTS, 4>(p, st, set);
    case 6: return launch<BF, PARTS, PARTS == 3 ? 6 : 1>(p, st, set);
    case 9: return launch<BF, PARTS, PARTS == 3 ? 9 : 1>(p, st, set);
    default: return launch<BF, PARTS, PARTS == 3 ? 12 : 1>(p, st, set);
    }
}

cudaError_t dispatch(const Int4Params &p, cudaStream_t st, bool set)
{
    if (p.xt == kF32) {
        const int cols = 3 * p.tokens;
        const int nt = cols <= 8 ? 1 : cols <= 16 ? 2 : cols <= 24 ? 3 : cols <= 32 ? 4 : cols <= 48 ? 6 : cols <= 72 ? 9 : 12;
        return by_columns<true, 3>(nt, p, st, set);
    }
    const int nt = (p.tokens + 7) / 8;
    return p.xt == kF16 ? by_columns<false, 1>(nt, p, st, set) : by_columns<true, 1>(nt, p, st, set);
}

}  // namespace

cudaError_t int4_setup()
{
    Int4Params p{};
    for (int xt : {int(kF32), int(kF16), int(kBF16)})
        for (p.tokens = 1; p.tokens <= kInt4MaxTokens; ++p.tokens) {
            p.xt = xt;
            const cudaError_t e = dispatch(p, nullptr, true);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t int4_pack(const uint8_t *q, const uint16_t *s, uint8_t *dst, int n, int k, cudaStream_t st)
{
    const int ku = (k + 63) / 64;
    const long long units = (long long)((n + 15) / 16) * ku;
    k_pack<<<unsigned((units + 7) / 8), 256, 0, st>>>(q, s, dst, n, k, ku, units);
    return cudaGetLastError();
}

cudaError_t int4_matvec(const Int4Params &p, cudaStream_t st) { return dispatch(p, st, false); }

}  // namespace pi
