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

constexpr int kMaxCluster = 8;

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

// d = A B + d, or (ADD false) A B.
template <bool BF, bool ADD>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1)
{
    const float c0 = ADD ? d[0] : 0.f, c1 = ADD ? d[1] : 0.f, c2 = ADD ? d[2] : 0.f, c3 = ADD ? d[3] : 0.f;
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%10, %11, %12, %13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%10, %11, %12, %13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

// (v & mask) | bits, in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
    return r;
}

// Eight nibbles to four 16-bit pairs: n - 8 in fp16, (n - 8) / 256 in bf16.  Under
// the exponent bits of 1024 (fp16) a nibble is that number plus n, and one four
// bits further up 1024 + 16 n, which a product and a sum bring to n - 8 without a
// shift; under those of 1/2 (bf16) it is 1/2 + n / 256.  All of it is exact.  The
// 256 keeps a group's 32 products of x up to bf16's or fp32's largest number in
// range, since their sum is at most max |x|; y gets it back at the end (kUnit).
template <bool BF>
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&r)[4])
{
    if (BF) {
        const uint32_t bias = 0x3f083f08u;   // 136 / 256
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t v = and_or(w >> (4 * i), 0x000f000fu, 0x3f003f00u);
            const __nv_bfloat162 d = __hsub2(*reinterpret_cast<const __nv_bfloat162 *>(&v), *reinterpret_cast<const __nv_bfloat162 *>(&bias));
            r[i] = *reinterpret_cast<const uint32_t *>(&d);
        }
    } else {
        const uint32_t bias = 0x64086408u, part = 0x2c002c00u, bias2 = 0xd480d480u;   // 1032; 1/16, -72
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t z = w >> (8 * i), v = and_or(z, 0x000f000fu, 0x64006400u), u = and_or(z, 0x00f000f0u, 0x64006400u);
            const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&bias));
            const __half2 e = __hfma2(*reinterpret_cast<const __half2 *>(&u), *reinterpret_cast<const __half2 *>(&part),
                                      *reinterpret_cast<const __half2 *>(&bias2));
            r[2 * i] = *reinterpret_cast<const uint32_t *>(&d);
            r[2 * i + 1] = *reinterpret_cast<const uint32_t *>(&e);
        }
    }
}

__device__ __forceinline__ void load8(const uint8_t *x, long long i, float (&v)[8])
{
    const float4 *p = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(x) + i);
    const float4 a = p[0], b = p[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
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
// Of eight numbers, some not finite: their leading parts (part 0; a NaN's digits
// may all be among the others), or what is left of the finite ones.
__device__ __forceinline__ void first_part_only(const float (&v)[8], int part, uint32_t (&u)[4])
{
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        // (inf - inf and NaN - NaN leave NaN: nothing is left of these)
        const uint32_t b = isnan(v[e]) ? (part == 0 ? 0x7fc0u : 0u) : __float_as_uint(v[e]) >> 16;
        u[e / 2] = e & 1 ? u[e / 2] | (b << 16) : b;
    }
}

__device__ __forceinline__ float value_of(const uint8_t *p, long long i, int dt)
{
    if (dt == kF32) return reinterpret_cast<const float *>(p)[i];
    if (dt == kF16) return __half2float(reinterpret_cast<const __half *>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
}

// unit / sqrt(mean x^2 + eps) for a token whose squares' sum leaves fp32 (numbers
// beyond some 1e18): summed again in 64 bits, by the half warp that needs it.
__device__ __noinline__ float root_inv_in_64(const uint8_t *x, long long at, int dt, int k, float eps, float unit)
{
    double ss = 0;
#pragma unroll 1
    for (int c = threadIdx.x % 16; c < k; c += 16) {
        const double v = value_of(x, at + c, dt);
        ss = fma(v, v, ss);
    }
#pragma unroll
    for (int o = 8; o; o >>= 1) ss += __shfl_xor_sync(0xffffu << (threadIdx.x & 16), ss, o);
    return float(unit * rsqrt(ss / k + eps));
}

// A product's shape in shared memory.  W: warps of a CTA.
template <int NT>
struct MvCfg {
    static constexpr int kWarps = NT <= 4 ? 16 : 8;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int kBatch = 4;                                // units that a warp takes from its ring at once
    static constexpr int kSlotRow = 8 * NT + 2;                     // (2: rows' same columns meet no bank twice)
    static constexpr int kSlot = 16 * kSlotRow;                     // sums of a warp for one row tile
    // Bytes: a slot for each warp's first tile (its second's takes the place of its ring); rings of `depth` batches; sums
    // of a CTA's row tiles, [tile][token][row]; behind them the chunk of x.
    static constexpr int kSlots = kWarps * kSlot * 4, kRing = kBatch * kInt4Unit, kSum = kWarps * 16 * 4;
    static constexpr int fixed(int depth, int tokens) { return kSlots + kWarps * kRing * depth + kSum * tokens; }
    static constexpr int kRoom = 222 * 1024;
    static constexpr int kLeastDepth = kSlot * 4 > 2 * kRing ? 3 : 2;
};

// A cluster takes row tiles (of 16), up to kWarps at a time; its CTAs share the
// columns.  A CTA's part, tiles x units of 64 columns, is laid end to end and
// shared out evenly over its warps, so that a warp has parts of two tiles at
// most: the sums of these go to two slots in shared memory, from there in order
// to the tile's sums, and from the CTAs, in order, to y.  Bound by the matrix's
// bytes, and before that, as it stands, by the instructions that unpack them (about
// 110 for a unit of 576 bytes with one tile of tokens): so each warp has few of
// them beside, keeps two or three batches of 4 units under way, and x is brought to
// each CTA once (for 13 tokens of 8192 columns it is 213 KB, about as much as the
// CTA's share of the matrix: hence the clusters).  6144x4096, one fp32 token with
// its norm: 6.8 us (2.1 TB/s); 8192x8192, 13 tokens: 17.0 us (2.3 TB/s).
// PARTS: 3 for F32 x, else 1.  NT: tiles of 8 columns of B (tokens * PARTS).  NORM:
// eps > 0; a kernel of its own, since what the norm needs costs the others registers
// (8192x8192, 13 tokens without a norm, by one kernel for both: 17.6 us).
template <bool BF, int PARTS, int NT, bool NORM>
__global__ void __launch_bounds__(MvCfg<NT>::kThreads, 1) k_matvec(Int4Params p, int log_cs, int clusters, int chunk, int depth, int split)
{
    using C = MvCfg<NT>;
    constexpr int W = C::kWarps, T = C::kThreads, U = C::kBatch;
    constexpr float kUnit = BF ? 256.f : 1.f;   // of the sums (nibbles())
    extern __shared__ __align__(16) uint8_t smem[];
    __shared__ float ssq[kInt4MaxTokens * W];
    __shared__ float total_sq[kInt4MaxTokens];
    __shared__ int from_warp[W], to_warp[W];   // of a tile: the slot of its first warp, its last warp
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t4 = lane % 4;
    float *slots = reinterpret_cast<float *>(smem);
    const uint32_t ring = uint32_t(__cvta_generic_to_shared(smem + C::kSlots)) + warp * depth * C::kRing;
    auto ring_slot = [&](int w) { return reinterpret_cast<float *>(smem + C::kSlots + w * depth * C::kRing); };
    float *sums = reinterpret_cast<float *>(smem + C::kSlots + W * C::kRing * depth);
    uint16_t *xs = reinterpret_cast<uint16_t *>(smem + C::fixed(depth, p.tokens));
    allow_next();
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
            const int k = first - tile * ks;
            // units not yet under way: `left` of this tile at `next`, then `later` of the one behind it
            const uint8_t *next = p.w + ((long long)(t0 + tile) * p.ku + k0 + k) * kInt4Unit;
            const uint8_t *behind = p.w + ((long long)(t0 + tile + 1) * p.ku + k0) * kInt4Unit;
            int left = min(end - first, ks - k), later = end - first - left, put = 0, get = 0;
            const int first_len = left, second_len = later;
            auto issue = [&]() {   // the next batch: U units, or the rest of a tile
                const int pieces = min(U, left) * (kInt4Unit / 16);
                const uint32_t dst = ring + put * (U * kInt4Unit);
#pragma unroll
                for (int i = 0; i < (U * kInt4Unit / 16 + 31) / 32; ++i)
                    if (lane + 32 * i < pieces) copy_async(dst + 16 * (lane + 32 * i), next + 16 * (lane + 32 * i));
                asm volatile("cp.async.commit_group;" ::: "memory");
                put = put + 1 == depth ? 0 : put + 1;
                next += U * kInt4Unit;
                left -= min(U, left);
                if (left == 0) {
                    next = behind;
                    left = later;
                    later = 0;
                }
            };
            for (int i = 1; i < depth; ++i) issue();
            // a tile belongs to the warps from the one with its first unit on
            if (lane == 0 && first < end) {
                const int last = (end - 1 - first + k) / ks;   // 1: the warp goes on into a second tile
                if (k == 0) from_warp[tile] = 2 * warp;
                if (last) from_warp[tile + 1] = 2 * warp + 1;
                if (first + ks - k <= end) to_warp[tile] = warp;
                if (last && first + 2 * ks - k <= end) to_warp[tile + 1] = warp;
            }
            after_previous();   // (the matrix is there since its creation; x and y may be the work of kernels before)
            if (t0 == t_begin || !one_pass) {
                // a warp for each token, or for each of `split` parts of it; the squares on the way
                const int pieces = ks * 8;   // of 8 columns
                for (int i = warp; i < p.tokens * split; i += W) {
                    const int t = i / split, part_of = i - t * split;
                    uint16_t *row = xs + t * stride;
                    float ss = 0.f;
                    const bool squares = NORM && t0 == t_begin;
#pragma unroll 4
                    for (int c = part_of * 32 + lane; c < pieces; c += 32 * split) {
                        const int col = k0 * 64 + 8 * c;
                        if (PARTS == 1) {
                            uint4 w = make_uint4(0, 0, 0, 0);
                            if (col < p.k) w = *reinterpret_cast<const uint4 *>(p.x + 2 * (t * p.xs + col));
                            *reinterpret_cast<uint4 *>(row + 8 * c) = w;
                            if (squares) {
                                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                                for (int e = 0; e < 4; ++e) {
                                    const float2 f = BF ? __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e]))
                                                        : __half22float2(*reinterpret_cast<const __half2 *>(&u[e]));
                                    ss += f.x * f.x;
                                    ss += f.y * f.y;
                                }
                            }
                        } else {
                            float v[8] = {};
                            if (col < p.k) load8(p.x, t * p.xs + col, v);
                            if (squares) {
#pragma unroll
                                for (int e = 0; e < 8; ++e) ss += v[e] * v[e];
                            }
                            float odd = 0.f;   // NaN if any is not finite
#pragma unroll
                            for (int e = 0; e < 8; ++e) odd = fmaf(v[e], 0.f, odd);
#pragma unroll
                            for (int part = 0; part < PARTS; ++part) {
                                uint32_t u[4];
#pragma unroll
                                for (int e = 0; e < 4; ++e)
                                    u[e] = __byte_perm(__float_as_uint(v[2 * e]), __float_as_uint(v[2 * e + 1]), 0x7632);
                                if (odd != 0.f) first_part_only(v, part, u);
                                *reinterpret_cast<uint4 *>(row + part * p.tokens * stride + 8 * c) = make_uint4(u[0], u[1], u[2], u[3]);
#pragma unroll
                                for (int e = 0; e < 8; ++e) v[e] -= cut(v[e]);
                            }
                        }
                    }
                    if (squares) {
#pragma unroll
                        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(~0u, ss, o);
                        if (lane == 0) ssq[i] = ss;
                    }
                }
                __syncthreads();
                if (NORM && t0 == t_begin && threadIdx.x < p.tokens) {
                    float ss = k0 == k_begin ? 0.f : total_sq[threadIdx.x];
                    for (int i = 0; i < split; ++i) ss += ssq[threadIdx.x * split + i];
                    total_sq[threadIdx.x] = ss;
                }
            }

            // ---- the warp's units
            float acc[NT][4] = {};
            const uint16_t *xb[NT];
#pragma unroll
            for (int n8 = 0; n8 < NT; ++n8) xb[n8] = xs + min(n8 * 8 + g, cols - 1) * stride + k * 64 + t4 * 8;
#pragma unroll 1
            for (int seg = 0; seg < 2; ++seg) {
                const int len = seg ? second_len : first_len;
                if (len == 0) break;
                for (int done = 0; done < len; done += U) {
                    issue();
                    if (depth == 4) asm volatile("cp.async.wait_group 3;" ::: "memory");
                    else if (depth == 3) asm volatile("cp.async.wait_group 2;" ::: "memory");
                    else asm volatile("cp.async.wait_group 1;" ::: "memory");
                    __syncwarp();
                    const uint32_t units = ring + get * (U * kInt4Unit);
                    const int have = min(U, len - done);
#pragma unroll
                    for (int i = 0; i < U; ++i) {
                        if (i >= have) break;
                        uint32_t qq[4], sp[2];
                        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                                     : "=r"(qq[0]), "=r"(qq[1]), "=r"(qq[2]), "=r"(qq[3]) : "r"(units + i * kInt4Unit + 16 * lane));
                        asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];"
                                     : "=r"(sp[0]), "=r"(sp[1]) : "r"(units + i * kInt4Unit + 512 + 8 * g));
#pragma unroll
                        for (int grp = 0; grp < 2; ++grp) {
                            uint32_t lo[4], hi[4];
                            nibbles<BF>(qq[2 * grp], lo);
                            nibbles<BF>(qq[2 * grp + 1], hi);
                            const float2 sc = __half22float2(*reinterpret_cast<const __half2 *>(&sp[grp]));
#pragma unroll
                            for (int n8 = 0; n8 < NT; ++n8) {
                                const uint4 b = *reinterpret_cast<const uint4 *>(xb[n8] + i * 64 + grp * 32);
                                float c[4];
                                mma16816<BF, false>(c, lo[0], hi[0], lo[1], hi[1], b.x, b.y);
                                mma16816<BF, true>(c, lo[2], hi[2], lo[3], hi[3], b.z, b.w);
                                acc[n8][0] += sc.x * c[0];
                                acc[n8][1] += sc.x * c[1];
                                acc[n8][2] += sc.y * c[2];
                                acc[n8][3] += sc.y * c[3];
                            }
                        }
                    }
                    __syncwarp();   // the batch has been read
                    get = get + 1 == depth ? 0 : get + 1;
#pragma unroll
                    for (int n8 = 0; n8 < NT; ++n8) xb[n8] += have * 64;
                }
                float *slot = seg ? ring_slot(warp) : slots + warp * C::kSlot;
#pragma unroll
                for (int n8 = 0; n8 < NT; ++n8) {
                    *reinterpret_cast<float2 *>(slot + g * C::kSlotRow + n8 * 8 + 2 * t4) = make_float2(acc[n8][0], acc[n8][1]);
                    *reinterpret_cast<float2 *>(slot + (g + 8) * C::kSlotRow + n8 * 8 + 2 * t4) = make_float2(acc[n8][2], acc[n8][3]);
                    acc[n8][0] = acc[n8][1] = acc[n8][2] = acc[n8][3] = 0.f;
                    xb[n8] -= ks * 64;   // (the second tile starts at the first column)
                }
            }
            __syncthreads();
            // ---- the tiles' sums: warps in order, parts from the least
            if (warp < nt) {   // a warp for each tile
                const int from = from_warp[warp], more = to_warp[warp] - from / 2, r = lane % 16;
                for (int t = lane / 16; t < p.tokens; t += 2) {
                    float *sum = sums + (warp * p.tokens + t) * 16 + r;
                    float y = k0 == k_begin ? 0.f : *sum;
                    const float *src = (from & 1 ? ring_slot(from / 2) : slots + from / 2 * C::kSlot) + r * C::kSlotRow + t;
#pragma unroll
                    for (int part = PARTS - 1; part >= 0; --part) y += src[part * p.tokens];
                    src = slots + (from / 2 + 1) * C::kSlot + r * C::kSlotRow + t;
#pragma unroll 4
                    for (int w = 0; w < more; ++w, src += C::kSlot) {
#pragma unroll
                        for (int part = PARTS - 1; part >= 0; --part) y += src[part * p.tokens];
                    }
                    *sum = y;
                }
            }
            if (cs == 1 || k0 + chunk < k_end) __syncthreads();
        }
        // ---- over the cluster's CTAs, in order, to y
        // each CTA has its part of the tiles; a half warp for 16 rows of a token
        const int j_begin = nt * rank >> log_cs, pairs = ((nt * (rank + 1) >> log_cs) - j_begin) * p.tokens;
        auto place = [&](int i, int &sum, int &t) {   // y's element (or -1), the sum's place, the token
            const int j = j_begin + i / p.tokens, row = (t0 + j) * 16 + lane % 16;
            t = i % p.tokens;
            sum = (j * p.tokens + t) * 16 + lane % 16;
            return i < pairs && row < p.n ? t * p.ys + row : -1;
        };
        int i = 2 * warp + lane / 16, sum, t;
        long long at = place(i, sum, t);
        float add = p.add && at >= 0 ? value_of(p.add, at, p.yt) : 0.f;   // under way while the CTAs wait for each other
        if (cs > 1) cluster_sync();
        for (; i < pairs; i += 2 * W) {
            float y = 0.f, ss = 0.f;
            if (cs == 1) {
                y = sums[sum];
                if (NORM) ss = total_sq[t];
            } else {
                for (int c = 0; c < cs; ++c) {
                    y += peer(sums + sum, c);
                    if (NORM) ss += peer(total_sq + t, c);
                }
            }
            float factor = kUnit;
            if (NORM) factor = kUnit / sqrtf(ss / float(p.k) + p.eps);
            // (a mean above 2^104, infinity included; fp16 numbers stay below, a NaN is one)
            if (BF && NORM && factor < 0x1p-44f) factor = root_inv_in_64(p.x, t * p.xs, p.xt, p.k, p.eps, kUnit);
            y *= factor;
            if (p.add) y += add;
            if (at >= 0) {
                if (p.yt == kF32) reinterpret_cast<float *>(p.y)[at] = y;
                else if (p.yt == kF16) reinterpret_cast<__half *>(p.y)[at] = __float2half(y);
                else reinterpret_cast<__nv_bfloat16 *>(p.y)[at] = __float2bfloat16(y);
            }
            at = place(i + 2 * W, sum, t);
            if (p.add && at >= 0) add = value_of(p.add, at, p.yt);
        }
        if (cs > 1) cluster_sync();   // the others have read this CTA's sums
    }
}

template <bool BF, int PARTS, int NT, bool NORM>
cudaError_t launch(const Int4Params &p, cudaStream_t st, bool set)
{
    using C = MvCfg<NT>;
    static_assert((C::kRoom - C::fixed(C::kLeastDepth, kInt4MaxTokens)) / (8 * NT) >= 64 + 4 * 128, "a chunk of x has 4 units at least");
    if (set) return cudaFuncSetAttribute(k_matvec<BF, PARTS, NT, NORM>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kRoom);
    const int cols = p.tokens * PARTS, tiles = (p.n + 15) / 16;
    // Over how many CTAs the columns are split: so many that x's part fits into shared memory at once (13 tokens of 8192
    // columns: two), beside rings as deep as then there is room for; for a CTA of its own three batches deep (8 tokens
    // of 8192 columns: one CTA with two batches takes 8% longer than two CTAs).
    auto fits = [&](int cs, int depth) { return C::fixed(depth, p.tokens) + cols * ((p.ku + cs - 1) / cs * 128 + 64) <= C::kRoom; };
    int cs = 1, depth = 4;
    while (cs < kMaxCluster && !fits(cs, cs == 1 ? 3 : C::kLeastDepth) && p.ku / cs >= 2) cs *= 2;
    while (depth > C::kLeastDepth && !fits(cs, depth)) --depth;
    const int units = (p.ku + cs - 1) / cs;
    int chunk = ((C::kRoom - C::fixed(depth, p.tokens)) / cols - 64) / 128;
    if (chunk > units) chunk = units;
    int clusters = cs == 1 ? p.n_sm : p.clusters[cs == 2 ? 0 : cs == 4 ? 1 : 2];
    if (clusters > tiles) clusters = tiles;
    return launch_close(k_matvec<BF, PARTS, NT, NORM>, dim3(clusters * cs), C::kThreads, C::fixed(depth, p.tokens) + cols * (chunk * 64 + 32) * 2,
                        st, cs, p, cs == 1 ? 0 : cs == 2 ? 1 : cs == 4 ? 2 : 3, clusters, chunk, depth,
                        p.tokens < C::kWarps ? C::kWarps / p.tokens : 1);
}

template <bool BF, int PARTS, bool NORM>
cudaError_t by_columns(int nt, const Int4Params &p, cudaStream_t st, bool set)
{
    switch (nt) {
    case 1: return launch<BF, PARTS, 1, NORM>(p, st, set);
    case 2: return launch<BF, PARTS, 2, NORM>(p, st, set);
    case 3: return launch<BF, PARTS, 3, NORM>(p, st, set);
    case 4: return launch<BF, PARTS, 4, NORM>(p, st, set);
    case 6: return launch<BF, PARTS, PARTS == 3 ? 6 : 1, NORM>(p, st, set);
    case 9: return launch<BF, PARTS, PARTS == 3 ? 9 : 1, NORM>(p, st, set);
    default: return launch<BF, PARTS, PARTS == 3 ? 12 : 1, NORM>(p, st, set);
    }
}

template <bool NORM>
cudaError_t by_type(const Int4Params &p, cudaStream_t st, bool set)
{
    if (p.xt == kF32) {
        const int cols = 3 * p.tokens;
        const int nt = cols <= 8 ? 1 : cols <= 16 ? 2 : cols <= 24 ? 3 : cols <= 32 ? 4 : cols <= 48 ? 6 : cols <= 72 ? 9 : 12;
        return by_columns<true, 3, NORM>(nt, p, st, set);
    }
    const int nt = (p.tokens + 7) / 8;
    return p.xt == kF16 ? by_columns<false, 1, NORM>(nt, p, st, set) : by_columns<true, 1, NORM>(nt, p, st, set);
}

cudaError_t dispatch(const Int4Params &p, cudaStream_t st, bool set)
{
    return p.eps > 0.f ? by_type<true>(p, st, set) : by_type<false>(p, st, set);
}

}  // namespace

cudaError_t int4_setup()
{
    Int4Params p{};
    for (int xt : {int(kF32), int(kF16), int(kBF16)})
        for (int tokens : {1, 3, 6, 9, 11, 17, 25})   // of each number of tiles
            for (float eps : {0.f, 1.f}) {
                p.xt = xt;
                p.tokens = tokens;
                p.eps = eps;
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
        cfg.dynamicSmemBytes = MvCfg<4>::kRoom;
        cfg.attrs = &attr;
        cfg.numAttrs = 1;
        const cudaError_t e = cudaOccupancyMaxActiveClusters(&clusters[i], k_matvec<true, 3, 4, true>, &cfg);
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
