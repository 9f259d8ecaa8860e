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

constexpr int kXBytes = 104 * 1024;    // shared memory for a chunk of x: 512 columns of 96 parts at least
constexpr int kMaxCluster = 8;
constexpr int kShareX = 64 * 1024;     // a CTA's part of x above this: the columns are split over more CTAs

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

// The matrix is read once: past L1, and first to leave L2.
__device__ __forceinline__ uint4 ldg_stream(const uint4 *p)
{
    uint4 v;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}
__device__ __forceinline__ uint2 ldg_stream(const uint2 *p)
{
    uint2 v;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.aligned;\nbarrier.cluster.wait.aligned;" ::: "memory");
}
// A number in the shared memory of the cluster's CTA `rank`.
__device__ __forceinline__ float peer(const float *p, int rank)
{
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(uint32_t(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
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

// A product's shape in shared memory.  W: warps of a CTA.
template <int NT>
struct MvCfg {
    static constexpr int kWarps = NT <= 4 ? 16 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kAhead = 4;                                // units in flight for each warp
    static constexpr int kSlot = 16 * 8 * NT;                       // sums of a warp for one row tile
    static constexpr int kSums = kWarps * 16 * kInt4MaxTokens;      // of a CTA's row tiles: [tile][token][row]
    static constexpr int kFixed = (2 * kWarps * kSlot + kSums) * 4; // bytes before the chunk of x
};

// A cluster takes row tiles (of 16), up to kWarps at a time; its CTAs share the
// columns.  A CTA's part, tiles x units of 64 columns, is laid end to end and
// shared out evenly over its warps, so that a warp has parts of two tiles at
// most: the sums of these go to two slots in shared memory, from there in order
// to the tile's sums, and from the CTAs, in order, to y.  Bound by the matrix's
// bytes: each warp keeps kAhead units of 576 bytes under way in registers, and x
// is brought to each CTA once (for 13 tokens of 8192 columns it is 213 KB, more
// than the CTA's share of the matrix: hence the clusters).
// PARTS: 3 for F32 x, else 1.  NT: tiles of 8 columns of B (tokens * PARTS).
template <bool BF, int PARTS, int NT>
__global__ void __launch_bounds__(MvCfg<NT>::kThreads, 1) k_matvec(Int4Params p, int log_cs, int clusters, int chunk)
{
    using C = MvCfg<NT>;
    constexpr int W = C::kWarps, T = C::kThreads, U = C::kAhead;
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float ssq[kInt4MaxTokens * W];
    __shared__ float total_sq[kInt4MaxTokens];
    __shared__ int from_warp[W], to_warp[W];   // of a tile: the slot of its first warp, its last warp
    float *slots = reinterpret_cast<float *>(smem), *sums = slots + 2 * W * C::kSlot;
    uint16_t *xs = reinterpret_cast<uint16_t *>(smem + C::kFixed);
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t4 = lane % 4;
    const int cols = p.tokens * PARTS, stride = chunk * 64 + 32;   // 64 bytes past a multiple of 128: no bank conflicts
    const int cs = 1 << log_cs, rank = blockIdx.x & (cs - 1), cluster = blockIdx.x >> log_cs;
    const int tiles = (p.n + 15) / 16;
    const unsigned each = unsigned(tiles) / unsigned(clusters), more = tiles - each * clusters;
    const int t_begin = cluster * each + min(unsigned(cluster), more), t_end = t_begin + each + (unsigned(cluster) < more);
    const int k_begin = p.ku * rank >> log_cs, k_end = p.ku * (rank + 1) >> log_cs;   // units
    const bool one_pass = k_end - k_begin <= chunk;

    for (int t0 = t_begin; t0 < t_end; t0 += W) {
        const int nt = min(W, t_end - t0);
        for (int k0 = k_begin; k0 < k_end; k0 += chunk) {
            const int ks = min(chunk, k_end - k0);
            const int busy = min(W, nt * ks), share = unsigned(nt * ks) / unsigned(busy), rest = nt * ks - share * busy;
            const int first = min(warp, busy) * share + min(warp, rest), end = first + (warp < busy ? share + (warp < rest) : 0);
            // the first units are under way before x is
            const int tile = first / ks;
            int k = first - tile * ks;
            const uint8_t *next = p.w + ((long long)(t0 + tile) * p.ku + k0 + k) * kInt4Unit;
            const long long jump = (long long)(p.ku - ks) * kInt4Unit;
            int next_k = k, ahead = first;
            uint4 wq[U];
            uint2 ws[U];
            auto load = [&](int i) {
                if (ahead >= end) return;
                wq[i] = ldg_stream(reinterpret_cast<const uint4 *>(next + 16 * lane));
                ws[i] = ldg_stream(reinterpret_cast<const uint2 *>(next + 512 + 8 * g));
                ++ahead;
                next += kInt4Unit;
                if (++next_k == ks) {
                    next_k = 0;
                    next += jump;
                }
            };
#pragma unroll
            for (int i = 0; i < U; ++i) load(i);
            // a tile belongs to the warps from the one with its first unit on
            if (lane == 0 && first < end) {
                const int last = (end - 1 - first + k) / ks;   // 1: the warp goes on into a second tile
                if (k == 0) from_warp[tile] = 2 * warp;
                if (last) from_warp[tile + 1] = 2 * warp + 1;
                if (first + ks - k <= end) to_warp[tile] = warp;
                if (last && first + 2 * ks - k <= end) to_warp[tile + 1] = warp;
            }
            if (t0 == t_begin || !one_pass) {
                const int pieces = ks * 8;   // of 8 columns
#pragma unroll 2
                for (int i = threadIdx.x; i < p.tokens * pieces; i += T) {
                    const int t = i / pieces, at = (i - t * pieces) * 8, col = k0 * 64 + at;
                    uint16_t *dst = xs + t * stride + at;
                    if (PARTS == 1) {
                        uint4 w = make_uint4(0, 0, 0, 0);
                        if (col < p.k) w = *reinterpret_cast<const uint4 *>(p.x + 2 * (t * p.xs + col));
                        *reinterpret_cast<uint4 *>(dst) = w;
                    } else {
                        float v[8] = {};
                        if (col < p.k) load8(p.x, t * p.xs + col, p.xt, v);
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
                if (p.eps > 0.f && t0 == t_begin) {
                    // sums of squares: one warp for each token, or for each of several pieces of it
                    const int split = max(1, W / p.tokens);
                    for (int i = warp; i < p.tokens * split; i += W) {
                        const int t = i / split, piece = i - t * split;
                        float ss = 0.f;
#pragma unroll 2
                        for (int c = piece * 32 + lane; c < pieces; c += 32 * split) {
                            const int col = k0 * 64 + 8 * c;
                            if (col >= p.k) break;
                            float v[8];
                            load8(p.x, t * p.xs + col, p.xt, v);
#pragma unroll
                            for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
                        }
#pragma unroll
                        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                        if (lane == 0) ssq[i] = ss;
                    }
                }
                __syncthreads();
                if (p.eps > 0.f && t0 == t_begin && threadIdx.x < p.tokens) {
                    const int split = max(1, W / p.tokens);
                    float ss = k0 == k_begin ? 0.f : total_sq[threadIdx.x];
                    for (int i = 0; i < split; ++i) ss += ssq[threadIdx.x * split + i];
                    total_sq[threadIdx.x] = ss;
                }
            }

            // ---- the warp's units
            float acc[NT][4] = {};
            float *slot = slots + 2 * warp * C::kSlot;
            auto flush = [&]() {
#pragma unroll
                for (int nt2 = 0; nt2 < NT; ++nt2) {
                    *reinterpret_cast<float2 *>(slot + g * 8 * NT + nt2 * 8 + 2 * t4) = make_float2(acc[nt2][0], acc[nt2][1]);
                    *reinterpret_cast<float2 *>(slot + (g + 8) * 8 * NT + nt2 * 8 + 2 * t4) = make_float2(acc[nt2][2], acc[nt2][3]);
                    acc[nt2][0] = acc[nt2][1] = acc[nt2][2] = acc[nt2][3] = 0.f;
                }
                slot += C::kSlot;
            };
            for (int u = first; u < end;) {
#pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (u >= end) break;
                    const uint32_t qq[4] = {wq[i].x, wq[i].y, wq[i].z, wq[i].w}, sp[2] = {ws[i].x, ws[i].y};
                    load(i);
#pragma unroll
                    for (int grp = 0; grp < 2; ++grp) {
                        uint32_t lo[4], hi[4];
                        nibbles<BF>(qq[2 * grp], lo);
                        nibbles<BF>(qq[2 * grp + 1], hi);
                        const float2 sc = __half22float2(*reinterpret_cast<const __half2 *>(&sp[grp]));
#pragma unroll
                        for (int n8 = 0; n8 < NT; ++n8) {
                            const int col = min(n8 * 8 + g, cols - 1);
                            const uint4 b = *reinterpret_cast<const uint4 *>(xs + col * stride + k * 64 + grp * 32 + t4 * 8);
                            float c[4] = {};
                            mma16816<BF>(c, lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                            mma16816<BF>(c, lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                            acc[n8][0] += sc.x * c[0];
                            acc[n8][1] += sc.x * c[1];
                            acc[n8][2] += sc.y * c[2];
                            acc[n8][3] += sc.y * c[3];
                        }
                    }
                    ++u;
                    if (++k == ks) {
                        k = 0;
                        flush();
                    }
                }
            }
            if (k != 0 && first < end) flush();
            __syncthreads();
            // ---- the tiles' sums: warps in order, parts from the least
            for (int i = threadIdx.x; i < nt * 16 * p.tokens; i += T) {
                const int r = i % 16, j = i / 16 % nt, t = i / 16 / nt;
                float y = k0 == k_begin ? 0.f : sums[(j * p.tokens + t) * 16 + r];
                const int s0 = from_warp[j], s1 = 2 * to_warp[j];
                const float *src = slots + s0 * C::kSlot + r * 8 * NT + t;
#pragma unroll
                for (int part = PARTS - 1; part >= 0; --part) y += src[part * p.tokens];
                src = slots + (s0 / 2 + 1) * 2 * C::kSlot + r * 8 * NT + t;
#pragma unroll 4
                for (int w = s0 / 2 + 1; w <= s1 / 2; ++w, src += 2 * C::kSlot) {
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part) y += src[part * p.tokens];
                }
                sums[(j * p.tokens + t) * 16 + r] = y;
            }
            if (cs == 1 || k0 + chunk < k_end) __syncthreads();
        }
        // ---- over the cluster's CTAs, in order, to y
        if (cs > 1) cluster_sync();
        const int all = nt * 16 * p.tokens;
        for (int i = (all * rank >> log_cs) + threadIdx.x; i < all * (rank + 1) >> log_cs; i += T) {
            const int r = i % 16, t = i / 16 % p.tokens, j = i / 16 / p.tokens;
            const long long row = (long long)(t0 + j) * 16 + r;
            if (row >= p.n) continue;
            float y = 0.f, ss = 0.f;
            if (cs == 1) {
                y = sums[i];
                if (p.eps > 0.f) ss = total_sq[t];
            } else {
                for (int c = 0; c < cs; ++c) {
                    y += peer(sums + i, c);
                    if (p.eps > 0.f) ss += peer(total_sq + t, c);
                }
            }
            if (p.eps > 0.f) y *= 1.f / sqrtf(ss / float(p.k) + p.eps);
            const long long at = t * p.ys + row;
            if (p.add) y += value_of(p.add, at, p.yt);
            if (p.yt == kF32) reinterpret_cast<float *>(p.y)[at] = y;
            else if (p.yt == kF16) reinterpret_cast<__half *>(p.y)[at] = __float2half(y);
            else reinterpret_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16(y);
        }
        if (cs > 1) cluster_sync();   // the others have read this CTA's sums
    }
}

static_assert((kXBytes / (3 * kInt4MaxTokens) - 64) / 128 >= 8, "a chunk of x is never empty");

template <bool BF, int PARTS, int NT>
cudaError_t launch(const Int4Params &p, cudaStream_t st, bool set)
{
    using C = MvCfg<NT>;
    static_assert(C::kFixed + kXBytes + 4096 <= 227 * 1024, "");
    if (set)
        return cudaFuncSetAttribute(k_matvec<BF, PARTS, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kFixed + kXBytes);
    const int cols = p.tokens * PARTS, tiles = (p.n + 15) / 16;
    int cs = 1;
    while (cs < kMaxCluster && cols * (p.ku / cs) * 128 > kShareX && p.ku / cs >= 2) cs *= 2;
    int chunk = (kXBytes / cols - 64) / 128;   // units of 64 columns that fit
    if (chunk > (p.ku + cs - 1) / cs) chunk = (p.ku + cs - 1) / cs;
    int clusters = cs == 1 ? p.n_sm : p.clusters[cs == 2 ? 0 : cs == 4 ? 1 : 2];
    if (clusters > tiles) clusters = tiles;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(clusters * cs);
    cfg.blockDim = dim3(C::kThreads);
    cfg.dynamicSmemBytes = C::kFixed + cols * (chunk * 64 + 32) * 2;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = cs;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = cs > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, k_matvec<BF, PARTS, NT>, p, cs == 1 ? 0 : cs == 2 ? 1 : cs == 4 ? 2 : 3, clusters, chunk);
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

cudaError_t int4_clusters(int (&clusters)[3])
{
    for (int i = 0; i < 3; ++i) {
        cudaLaunchAttribute attr{};
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 2 << i;
        attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(2 << i);
        cfg.blockDim = dim3(MvCfg<4>::kThreads);
        cfg.dynamicSmemBytes = MvCfg<4>::kFixed + kXBytes;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters[i], k_matvec<true, 3, 4>, &cfg);
        if (e != cudaSuccess) return e;
        if (clusters[i] < 1) clusters[i] = 1;
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
