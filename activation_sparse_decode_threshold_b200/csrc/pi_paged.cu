// pi_paged.cu -- attention of one new token per sequence over a paged cache.
//
// Mathematics: one pass over the positions with a running maximum m and sum l
// per query head: o = sum_j 2^(x_j - m) v_j, l = sum_j 2^(x_j - m), x_j the
// score times log2 e; o and l shrink by 2^(m - m') when the maximum grows to m'.
// Partial (m, l, o) of disjoint positions join the same way, in a fixed order.
//
// Bound: the cache's bytes (each is used for 2 products per query head).  So
// the work, all sequences' chunks of 16 positions for each cached head, is laid
// end to end and shared out evenly over all warps, whatever the lengths; a warp
// keeps its chunks coming by asynchronous copies several chunks ahead.  Products
// run on mma.sync m16n8k16, 8 query heads at a time as rows 0-7; rows 8-15 carry
// the low parts of the same 8 heads (queries and weights as two 16-bit parts,
// products with the 16-bit, 8-bit or 4-bit codes exact), which costs nothing:
// the rows would be empty.  Scales of quantised rows are applied in fp32 to the
// scores (K) and to the weights (V).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pi_attn.h"

namespace pi {
namespace {

constexpr int kChunk = 16;            // positions
constexpr int kMaxWarps = 12;
constexpr int kHeads = 8;             // query heads of an item

template <int FMT, int D>
struct Cfg {
    static constexpr bool kF = FMT == kF16 || FMT == kBF16;
    static constexpr int kRow = FMT == kI8 ? D : FMT == kI4 ? D / 2 : 2 * D;   // bytes of a cached row
    static constexpr int kScale = FMT == kI8 ? 4 : FMT == kI4 ? D / 16 : 0;    // bytes of its scales
    static constexpr int kCodes = kChunk * kRow;                              // bytes of a chunk's K (or V)
    static constexpr int kOffV = kCodes, kOffS = 2 * kCodes, kOffI = kOffS + (kScale ? 256 : 0);
    static constexpr int kStage = kOffI + 16;
    static constexpr int kWarps = 8;
    static constexpr int kStages = FMT == kI4 ? 8 : FMT == kI8 ? 6 : 3;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kPart = kHeads * D * 4 + 2 * kHeads * 4;             // bytes of a partial result
    static constexpr int kSmem = kWarps * kRing;
    static_assert(kRing >= kPart, "a warp's partial result takes the place of its ring");
    static_assert(kSmem <= 227 * 1024, "");
};

__device__ __forceinline__ uint32_t s2u(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }

// Copies of 16, 8 or 4 bytes; `live` false writes zeros and reads nothing.
template <int N>
__device__ __forceinline__ void copy_async(uint32_t dst, const uint8_t *src, bool live)
{
    const int n = live ? N : 0;
    if (N == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
    else asm volatile("cp.async.ca.shared.global [%0], [%1], %3, %2;" ::"r"(dst), "l"(src), "r"(n), "n"(N) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

__device__ __forceinline__ uint4 lds128(uint32_t a)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a)
{
    uint2 v;
    asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds32(uint32_t a)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}

__device__ __forceinline__ float exp2_(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

template <bool BF>
__device__ __forceinline__ void mma(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%0, %1, %2, %3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two numbers as 16-bit high parts and what is left of them as low parts.
template <bool BF>
__device__ __forceinline__ void split2(float a, float b, uint32_t &hi, uint32_t &lo)
{
    if (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(a - f.x, b - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    } else {
        const __half2 h = __floats2half2_rn(a, b);
        const float2 f = __half22float2(h);
        const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
        hi = *reinterpret_cast<const uint32_t *>(&h);
        lo = *reinterpret_cast<const uint32_t *>(&l);
    }
}

// A sum's high and low part as one number.  An infinite high part stands alone:
// its low part holds 0 times that infinity.
__device__ __forceinline__ float whole(float hi, float lo) { return isinf(hi) ? hi : hi + lo; }

__device__ __forceinline__ uint32_t hsub(uint32_t v, uint32_t m)
{
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&m));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// Eight 4-bit codes n to four fp16 pairs n - 8: nibbles (i, i + 4) to pair i.
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&r)[4])
{
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = hsub(((w >> (4 * i)) & 0x000f000fu) | 0x64006400u, 0x64086408u);
}
// Bytes (0, 1) and (2, 3) of w, signed bytes with the top bit flipped, to fp16 pairs.
__device__ __forceinline__ uint32_t bytes01(uint32_t w) { return hsub(__byte_perm(w, 0x64646464u, 0x4140), 0x64806480u); }
__device__ __forceinline__ uint32_t bytes23(uint32_t w) { return hsub(__byte_perm(w, 0x64646464u, 0x4342), 0x64806480u); }

// Eight consecutive inputs as floats.
__device__ __forceinline__ void load8(const uint8_t *p, long long i, int dt, float (&v)[8])
{
    if (dt == kF32) {
        const float4 *q = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p) + i);
        const float4 a = q[0], b = q[1];
        v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
        const uint4 w = *reinterpret_cast<const uint4 *>(p + 2 * i);
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const float2 f = dt == kF16 ? __half22float2(*reinterpret_cast<const __half2 *>(&u[e]))
                                        : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&u[e]));
            v[2 * e] = f.x;
            v[2 * e + 1] = f.y;
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
__device__ __forceinline__ void store8(uint8_t *p, long long i, int dt, const float (&v)[8])
{
    if (dt == kF32) {
        float4 *q = reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i);
        q[0] = make_float4(v[0], v[1], v[2], v[3]);
        q[1] = make_float4(v[4], v[5], v[6], v[7]);
    } else {
        *reinterpret_cast<uint4 *>(p + 2 * i) = make_uint4(pack2(v[0], v[1], dt), pack2(v[2], v[3], dt),
                                                           pack2(v[4], v[5], dt), pack2(v[6], v[7], dt));
    }
}

// Positions of one sequence that its query sees, and the chunks that hold them.
// A sequence with none has one chunk without positions, whose result is 0.
struct Span {
    int lo, hi, c0, c1;
};
__device__ __forceinline__ Span span_of(const AttnParams &p, int s, bool report)
{
    int len = p.len[s];
    const int room = p.c.width << p.c.page_shift;
    if (len < 0 || len > room) {
        if (report) atomicExch(p.err, int(kDevCheck));
        len = len < 0 ? 0 : room;
    }
    Span r;
    r.hi = len;
    r.lo = p.window && len > p.window ? len - p.window : 0;
    r.c0 = r.lo / kChunk;
    r.c1 = max((r.hi + kChunk - 1) / kChunk, r.c0 + 1);
    return r;
}

// Where a warp is in the row of all chunks: sequence s, item i of the
// sequence (cached head and block of 8 query heads), chunk c.
struct Cursor {
    int s, item, c;
    Span span;
};

enum { kFirst = 1, kLast = 2, kWhole = 4 };   // a chunk in its segment; a segment that is its whole item

// Weights times V scales s are taken relative to 2^(ref - 127), the largest s
// so far, and brought to fp16's range by 2^13.  The least ref keeps 2^(127 -
// ref + 13) finite, for rows of zeros (s = 0).
constexpr int kLeastRef = 16;

// Scale factor of scores and accumulators by power of two, from a number's exponent.
__device__ __forceinline__ float pow2_of(int biased) { return __int_as_float(biased << 23); }

template <int FMT, int D>
__global__ void __launch_bounds__(32 * Cfg<FMT, D>::kWarps, 1) k_paged(AttnParams p, int items, int blocks_per_head)
{
    using C = Cfg<FMT, D>;
    constexpr bool BF = FMT == kBF16;
    constexpr int W = C::kWarps, S = C::kStages, NT = D / 8;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long sums[W];
    __shared__ long long offs[32 * W];
    __shared__ int part_s[W][2], part_item[W][2];
    __shared__ int is_last;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int n = p.c.n_seqs;

    // ---- chunks before each thread's block of sequences --------------------
    const int per = (n + 32 * W - 1) / (32 * W);
    long long mine = 0;
    for (int s = threadIdx.x * per; s < min(n, (int(threadIdx.x) + 1) * per); ++s) {
        const Span r = span_of(p, s, blockIdx.x == 0);
        mine += (long long)(r.c1 - r.c0) * items;
    }
    long long scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane == 31) sums[warp] = scan;
    __syncthreads();
    long long total = 0, before = 0;
#pragma unroll
    for (int w = 0; w < W; ++w) {
        before += w < warp ? sums[w] : 0;
        total += sums[w];
    }
    offs[threadIdx.x] = before + scan - mine;
    __syncthreads();

    // ---- this warp's share ---------------------------------------------------
    const long long want = (total + W - 1) / W;
    const int ctas = int(want < gridDim.x ? want : gridDim.x);   // at least a chunk for each warp
    if (int(blockIdx.x) >= ctas) return;
    const long long shares = (long long)ctas * W, share = (long long)blockIdx.x * W + warp;
    const long long u0 = total * share / shares, u1 = total * (share + 1) / shares;
    const long long cta0 = total * blockIdx.x / ctas, cta1 = total * (blockIdx.x + 1LL) / ctas;
    uint8_t *ring = smem + warp * C::kRing;
    const uint32_t ring_u = s2u(ring);
    if (lane < 2) part_s[warp][lane] = -1;

    Cursor at{};
    if (u0 < u1) {
        int b = 0;   // the block that holds chunk u0: the last one that starts at or before it
        for (int step = 16 * W; step; step >>= 1)
            if (b + step < 32 * W && offs[b + step] <= u0) b += step;
        // (blocks without sequences start at the total, above u0)
        at.s = b * per;
        long long left = u0 - offs[b];
        for (;;) {
            at.span = span_of(p, at.s, false);
            const long long here = (long long)(at.span.c1 - at.span.c0) * items;
            if (left < here) break;
            left -= here;
            ++at.s;
        }
        const int nc = at.span.c1 - at.span.c0;
        at.item = int(left / nc);
        at.c = at.span.c0 + int(left - (long long)at.item * nc);
    }

    // ---- copies of one chunk into a stage --------------------------------------
    const long long slot_bytes = (long long)p.c.slot_rows * C::kRow, scale_slot = (long long)p.c.slot_rows * C::kScale;
    int page_a = -1, page_b = -1;
    auto look_up = [&]() {   // pages of the cursor's two halves of 8 positions
        const int a = at.c * kChunk, b = a + 8;
        const int32_t *row = p.c.table + at.s * p.c.tstride;
        page_a = a < at.span.hi && a + 8 > at.span.lo ? row[a >> p.c.page_shift] : -1;
        page_b = b < at.span.hi && b + 8 > at.span.lo ? row[b >> p.c.page_shift] : -1;
    };
    long long issued = u0;
    bool first = true, from_start = u0 < u1 && at.c == at.span.c0;
    if (u0 < u1) look_up();
    auto issue = [&](int stage) {
        if (issued >= u1) {
            copy_commit();
            return;
        }
        const int pos = at.c * kChunk;
        // positions seen, by bit
        unsigned mask = 0xffffu;
        if (pos + kChunk > at.span.hi) mask &= at.span.hi > pos ? (1u << (at.span.hi - pos)) - 1 : 0;
        if (pos < at.span.lo) mask &= ~((1u << (at.span.lo - pos)) - 1);
        if ((mask & 0x00ffu) && (unsigned)page_a >= (unsigned)p.c.n_pages) {
            if (lane == 0) atomicExch(p.err, int(kDevCheck));
            mask &= 0xff00u;
        }
        if ((mask & 0xff00u) && (unsigned)page_b >= (unsigned)p.c.n_pages) {
            if (lane == 0) atomicExch(p.err, int(kDevCheck));
            mask &= 0x00ffu;
        }
        const int hk = at.item / blocks_per_head;
        const long long head = (long long)hk * p.c.head_rows;
        const int sm = p.c.page_size - 1;
        const long long ra = (mask & 0x00ffu) ? (long long)page_a * p.c.page_rows + (long long)(pos & sm) * p.c.slot_rows + head : 0;
        const long long rb = (mask & 0xff00u) ? (long long)page_b * p.c.page_rows + (long long)((pos + 8) & sm) * p.c.slot_rows + head : 0;
        const uint32_t dst = ring_u + stage * C::kStage;
        // a row without a position is filled with zeros (its memory is not read)
        auto from = [&](const uint8_t *base, int key) {
            return base + (key < 8 ? ra : rb) * C::kRow + ((mask >> key) & 1 ? (key & 7) * slot_bytes : 0);
        };
        if (C::kF || FMT == kI8) {
            constexpr int JK = C::kRow / 64;   // 16-byte pieces of a K row for each lane of four
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int j = 0; j < JK; ++j)
                    copy_async<16>(dst + (h * JK + j) * 512 + lane * 16, from(p.c.k, g + 8 * h) + 16 * (t + 4 * j),
                                   (mask >> (g + 8 * h)) & 1);
            constexpr int JV = C::kRow >= 128 ? C::kRow / 128 : 1, NV = C::kRow >= 128 ? 16 : 8;
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const int key = 2 * t + (r & 1) + 8 * (r >> 1);
#pragma unroll
                for (int j = 0; j < JV; ++j)
                    copy_async<NV>(dst + C::kOffV + (r * JV + j) * 32 * NV + lane * NV,
                                   from(p.c.v, key) + NV * (g + 8 * j), (mask >> key) & 1);
            }
        } else {
            // rows whole, their 16-byte pieces permuted so that later reads of one piece of 8 rows meet no bank twice
            constexpr int P = C::kRow / 16;    // 4 or 2 pieces
#pragma unroll
            for (int i = 0; i < P / 2; ++i) {
                const int key = P == 4 ? g + 8 * i : lane / 2, piece = P == 4 ? t : lane % 2;
                const int put = key * C::kRow + 16 * (piece ^ ((key >> (P == 4 ? 1 : 2)) & (P - 1)));
                const bool live = (mask >> key) & 1;
                copy_async<16>(dst + put, from(p.c.k, key) + 16 * piece, live);
                copy_async<16>(dst + C::kOffV + put, from(p.c.v, key) + 16 * piece, live);
            }
        }
        if (C::kScale) {   // lanes 0-15: K of key lane, 16-31: V
            const int key = lane & 15;
            const bool live = (mask >> key) & 1;
            const uint8_t *base = (lane < 16 ? p.c.ks : p.c.vs) + (key < 8 ? ra : rb) * C::kScale +
                                  (live ? (key & 7) * scale_slot : 0);
            copy_async<C::kScale ? C::kScale : 4>(dst + C::kOffS + lane * 8, base, live);
        }
        copy_commit();
        // what the reader has to know
        const bool ends = at.c + 1 == at.span.c1, last = ends || issued + 1 == u1;
        if (lane == 0)
            *reinterpret_cast<int4 *>(ring + stage * C::kStage + C::kOffI) =
                make_int4(int(mask), (first ? kFirst : 0) | (last ? kLast : 0) | (ends && from_start ? kWhole : 0), at.s, at.item);
        first = last;
        ++issued;
        if (!ends) ++at.c;
        else if (issued < u1) {
            if (++at.item == items) {
                at.item = 0;
                ++at.s;
                at.span = span_of(p, at.s, false);
            }
            at.c = at.span.c0;
        }
        if (last) from_start = true;
        if (issued < u1) look_up();
    };
#pragma unroll
    for (int i = 0; i < S - 1; ++i) issue(i);

    // ---- one chunk after the other ---------------------------------------------
    uint32_t q[D / 16][4];
    float acc[NT][4] = {};
    float m = -INFINITY, l = 0.f, factor = 0.f;
    int ref = 0;   // exponent (biased) of the V scales that acc is relative to
    int parts = 0, cur_s = -1, cur_item = 0;
    bool open = false;   // acc holds a segment that is not its whole item and ends with the share
    // lane's value e of group i of 8 consecutive elements, and the group's first element
    auto value = [&](int i, int e) {
        if (FMT == kI4) return whole(acc[i * 4 + (e & 3)][e >> 2], acc[i * 4 + (e & 3)][2 + (e >> 2)]);
        if (FMT == kI8 && D == 128) return whole(acc[(i & 1) * 8 + e][i >> 1], acc[(i & 1) * 8 + e][2 + (i >> 1)]);
        return whole(acc[(i >> 1) * 8 + e][i & 1], acc[(i >> 1) * 8 + e][2 + (i & 1)]);
    };
    auto place = [&](int i) {
        if (FMT == kI4) return 32 * i + 8 * t;
        if (FMT == kI8 && D == 128) return 16 * (2 * t + (i >> 1)) + 8 * (i & 1);
        return 8 * (2 * t + (i & 1) + 8 * (i >> 1));
    };
    // (m, l, o) of this lane's part of head g, as the partial results are kept
    auto save = [&](float *dst) {
        const float unit = C::kScale ? pow2_of(ref) * 0x1p-13f : 1.f;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) {
            float4 *o = reinterpret_cast<float4 *>(dst + g * D + place(i));
            o[0] = make_float4(value(i, 0) * unit, value(i, 1) * unit, value(i, 2) * unit, value(i, 3) * unit);
            o[1] = make_float4(value(i, 4) * unit, value(i, 5) * unit, value(i, 6) * unit, value(i, 7) * unit);
        }
        if (t == 0) {
            dst[kHeads * D + g] = m;
            dst[kHeads * D + kHeads + g] = l;
        }
    };
    float *warp_part = p.part + (size_t)gridDim.x * 2 * (C::kPart / 4) + (size_t)(blockIdx.x * W + warp) * (C::kPart / 4);

    int stage = 0;
    for (long long u = u0; u < u1; ++u, stage = stage + 1 == S ? 0 : stage + 1) {
        copy_wait<S - 2>();
        __syncwarp();
        issue(stage ? stage - 1 : S - 1);
        const uint32_t base = ring_u + stage * C::kStage;
        const int4 info = *reinterpret_cast<const int4 *>(ring + stage * C::kStage + C::kOffI);
        const unsigned mask = unsigned(info.x);
        if (info.y & kFirst) {
            cur_s = info.z;
            cur_item = info.w;
            const int head = cur_item % blocks_per_head * kHeads + g;   // in its group
            const bool live = head < p.group;
            const long long row = cur_s * p.qs + (long long)(cur_item / blocks_per_head * p.group + head) * D;
            float v[D / 32][8], top = 0.f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
                const int d = FMT == kI4 ? 32 * i + 8 * t : FMT == kI8 ? 16 * (t + 4 * (i >> 1)) + 8 * (i & 1) : 8 * (t + 4 * i);
                if (live) load8(p.q, row + d, p.dt, v[i]);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (!live) v[i][e] = 0.f;
                    top = fmaxf(top, fabsf(v[i][e]));
                }
            }
            // the head's largest element is brought to [1, 2), so that no part leaves the range of 16 bits
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
            top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
            const int ex = min(max(__float_as_int(top) >> 23, 1), 253);
            const float down = pow2_of(254 - ex);
            factor = pow2_of(ex);
            factor *= p.softcap > 0.f ? p.scale : p.scale * 1.4426950408889634f;
#pragma unroll
            for (int i = 0; i < D / 32; ++i) {
#pragma unroll
                for (int e = 0; e < 8; ++e) v[i][e] *= down;
                constexpr int step = FMT == kI4 ? 4 : 1, next = FMT == kI4 ? 1 : 2;
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int e = FMT == kI4 ? 2 * h : 4 * h;
                    split2<BF>(v[i][e], v[i][e + step], q[2 * i + h][0], q[2 * i + h][1]);
                    split2<BF>(v[i][e + next], v[i][e + next + step], q[2 * i + h][2], q[2 * i + h][3]);
                }
            }
            m = -INFINITY;
            l = 0.f;
            ref = kLeastRef;
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[i][0] = acc[i][1] = acc[i][2] = acc[i][3] = 0.f;
        }

        // scores of head g at positions 2t, 2t + 1, 8 + 2t, 9 + 2t
        float x[4];
        float vs[4] = {};       // I8: V scales of these positions
        uint2 vs4[4];           // I4: four (two) fp16 scales of each
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            if (FMT == kI4) {
                x[2 * h] = x[2 * h + 1] = 0.f;
                uint2 ks[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    ks[e] = lds64(base + C::kOffS + (8 * h + 2 * t + e) * 8);
                    vs4[2 * h + e] = lds64(base + C::kOffS + (16 + 8 * h + 2 * t + e) * 8);
                }
#pragma unroll
                for (int j = 0; j < D / 32; ++j) {
                    const int key = g + 8 * h;
                    constexpr int P = C::kRow / 16;
                    const uint32_t w = lds32(base + key * C::kRow + 16 * (j ^ ((key >> (P == 4 ? 1 : 2)) & (P - 1))) + 4 * t);
                    uint32_t b[4];
                    nibbles(w, b);
                    float c[4] = {};
                    mma<false>(c, q[2 * j], b[0], b[1]);
                    mma<false>(c, q[2 * j + 1], b[2], b[3]);
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        const uint32_t u2 = j < 2 ? ks[e].x : ks[e].y;
                        const float2 sc = __half22float2(*reinterpret_cast<const __half2 *>(&u2));
                        x[2 * h + e] += (j & 1 ? sc.y : sc.x) * (c[e] + c[2 + e]);
                    }
                }
            } else {
                float c[4] = {};
                constexpr int JK = C::kRow / 64;
#pragma unroll
                for (int j = 0; j < JK; ++j) {
                    const uint4 w = lds128(base + (h * JK + j) * 512 + lane * 16);
                    if (FMT == kI8) {
                        const uint32_t u4[4] = {w.x ^ 0x80808080u, w.y ^ 0x80808080u, w.z ^ 0x80808080u, w.w ^ 0x80808080u};
#pragma unroll
                        for (int i = 0; i < 4; ++i) mma<false>(c, q[j * 4 + i], bytes01(u4[i]), bytes23(u4[i]));
                    } else {
                        mma<BF>(c, q[2 * j], w.x, w.y);
                        mma<BF>(c, q[2 * j + 1], w.z, w.w);
                    }
                }
                x[2 * h] = C::kF ? whole(c[0], c[2]) : c[0] + c[2];
                x[2 * h + 1] = C::kF ? whole(c[1], c[3]) : c[1] + c[3];
                if (FMT == kI8) {
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[2 * h + e] *= __uint_as_float(lds32(base + C::kOffS + (8 * h + 2 * t + e) * 8));
                        vs[2 * h + e] = __uint_as_float(lds32(base + C::kOffS + (16 + 8 * h + 2 * t + e) * 8));
                    }
                }
            }
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            x[e] *= factor;
            if (p.softcap > 0.f) {   // cap * tanh(x / cap) = cap - 2 cap / (1 + e^(2x / cap))
                const float z = exp2_(x[e] * (2.8853900817779268f / p.softcap));
                x[e] = (p.softcap - 2.f * p.softcap / (1.f + z)) * 1.4426950408889634f;
            }
        }
        if (mask != 0xffffu) {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (!((mask >> (2 * t + (e & 1) + 8 * (e >> 1))) & 1)) x[e] = -INFINITY;
        }
        // the running maximum (a NaN score is passed over here and makes l and o NaN below)
        float top = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
        top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
        top = fmaxf(top, m);
        int big = 0;   // exponent of the largest V scale
        if (FMT == kI8) {
            big = __float_as_int(fmaxf(fmaxf(vs[0], vs[1]), fmaxf(vs[2], vs[3]))) >> 23;
        } else if (FMT == kI4) {
            __half2 hm = *reinterpret_cast<const __half2 *>(&vs4[0].x);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                hm = __hmax2(hm, *reinterpret_cast<const __half2 *>(&vs4[e].x));
                if (D == 128) hm = __hmax2(hm, *reinterpret_cast<const __half2 *>(&vs4[e].y));
            }
            big = __float_as_int(__half2float(__hmax(__low2half(hm), __high2half(hm)))) >> 23;
        }
        const float zero = top == -INFINITY ? 0.f : top;
        if (__any_sync(~0u, top != m || big > ref)) {
            int grown = ref;
            if (C::kScale) {
                if (FMT == kI4 && big == 255) {   // an infinite scale spoils its own group only: the largest of the others
                    big = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e)
#pragma unroll
                        for (int i = 0; i < D / 64; ++i) {
                            const float2 sc = __half22float2(*reinterpret_cast<const __half2 *>(i ? &vs4[e].y : &vs4[e].x));
                            if (sc.x < INFINITY) big = max(big, __float_as_int(sc.x) >> 23);
                            if (sc.y < INFINITY) big = max(big, __float_as_int(sc.y) >> 23);
                        }
                }
                big = max(big, __shfl_xor_sync(~0u, big, 1));
                big = max(big, __shfl_xor_sync(~0u, big, 2));
                grown = max(ref, min(big, 253));
            }
            const float shrink = exp2_(m - zero);
            // 2^(ref - grown); a difference beyond the range of floats is 0
            const float both = shrink * (grown - ref > 126 ? 0.f : pow2_of(127 + ref - grown));
            l *= shrink;
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                acc[i][0] *= both;
                acc[i][1] *= both;
                acc[i][2] *= both;
                acc[i][3] *= both;
            }
            m = top;
            ref = grown;
        }
        float w[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            // F16: weights carry a factor 2^14, so that the low parts of small ones stay normal numbers
            w[e] = exp2_(FMT == kF16 ? x[e] - zero + 14.f : x[e] - zero);
            l += w[e];
        }
        if (C::kF) {
            uint32_t a[4];
            split2<BF>(w[0], w[1], a[0], a[1]);
            split2<BF>(w[2], w[3], a[2], a[3]);
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                uint4 r[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) r[i] = lds128(base + C::kOffV + (i * (D / 64) + j) * 512 + lane * 16);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t r0 = (&r[0].x)[i], r1 = (&r[1].x)[i], r2 = (&r[2].x)[i], r3 = (&r[3].x)[i];
                    mma<BF>(acc[j * 8 + 2 * i], a, __byte_perm(r0, r1, 0x5410), __byte_perm(r2, r3, 0x5410));
                    mma<BF>(acc[j * 8 + 2 * i + 1], a, __byte_perm(r0, r1, 0x7632), __byte_perm(r2, r3, 0x7632));
                }
            }
        } else if (FMT == kI8) {
            const float f = pow2_of(254 - ref) * 0x1p13f;
            uint32_t a[4];
            split2<false>(w[0] * (vs[0] * f), w[1] * (vs[1] * f), a[0], a[1]);
            split2<false>(w[2] * (vs[2] * f), w[3] * (vs[3] * f), a[2], a[3]);
            constexpr int WORDS = D / 32;   // 4 (16 bytes of a row for each lane) or 2
            uint32_t r[4][WORDS];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (WORDS == 4) {
                    const uint4 v = lds128(base + C::kOffV + i * 512 + lane * 16);
                    r[i][0] = v.x, r[i][1] = v.y, r[i][WORDS - 2] = v.z, r[i][WORDS - 1] = v.w;
                } else {
                    const uint2 v = lds64(base + C::kOffV + i * 256 + lane * 8);
                    r[i][0] = v.x, r[i][1] = v.y;
                }
            }
#pragma unroll
            for (int i = 0; i < WORDS; ++i) {
                const uint32_t r0 = r[0][i] ^ 0x80808080u, r1 = r[1][i] ^ 0x80808080u, r2 = r[2][i] ^ 0x80808080u,
                               r3 = r[3][i] ^ 0x80808080u;
                const uint32_t a01 = __byte_perm(r0, r1, 0x5140), a23 = __byte_perm(r0, r1, 0x7362);
                const uint32_t b01 = __byte_perm(r2, r3, 0x5140), b23 = __byte_perm(r2, r3, 0x7362);
                mma<false>(acc[4 * i], a, bytes01(a01), bytes01(b01));
                mma<false>(acc[4 * i + 1], a, bytes23(a01), bytes23(b01));
                mma<false>(acc[4 * i + 2], a, bytes01(a23), bytes01(b23));
                mma<false>(acc[4 * i + 3], a, bytes23(a23), bytes23(b23));
            }
        } else {
            const float f = pow2_of(254 - ref) * 0x1p13f;
            constexpr int P = C::kRow / 16;
            const uint32_t pick = g & 1 ? 0x7632 : 0x5410;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] *= f;
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {
                float v[4];
                uint32_t r[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = 2 * t + (e & 1) + 8 * (e >> 1);
                    const uint32_t u2 = j < 2 ? vs4[e].x : vs4[e].y;
                    const float2 sc = __half22float2(*reinterpret_cast<const __half2 *>(&u2));
                    v[e] = w[e] * (j & 1 ? sc.y : sc.x);
                    r[e] = lds32(base + C::kOffV + key * C::kRow + 16 * (j ^ ((key >> (P == 4 ? 1 : 2)) & (P - 1))) + 4 * (g >> 1));
                }
                uint32_t a[4], b0[4], b1[4];
                split2<false>(v[0], v[1], a[0], a[1]);
                split2<false>(v[2], v[3], a[2], a[3]);
                nibbles(__byte_perm(r[0], r[1], pick), b0);
                nibbles(__byte_perm(r[2], r[3], pick), b1);
#pragma unroll
                for (int i = 0; i < 4; ++i) mma<false>(acc[4 * j + i], a, b0[i], b1[i]);
            }
        }

        if (info.y & kLast) {
            l += __shfl_xor_sync(~0u, l, 1);
            l += __shfl_xor_sync(~0u, l, 2);
            if (FMT == kF16) l *= 0x1p-14f;
            if (FMT == kF16) {
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    acc[i][0] *= 0x1p-14f;
                    acc[i][1] *= 0x1p-14f;
                    acc[i][2] *= 0x1p-14f;
                    acc[i][3] *= 0x1p-14f;
                }
            }
            if (info.y & kWhole) {
                const int hb = cur_item % blocks_per_head * kHeads + g;
                if (hb < p.group) {
                    const int head = cur_item / blocks_per_head * p.group + hb;
                    const float unit = (l == 0.f ? 0.f : 1.f / l) * (C::kScale ? pow2_of(ref) * 0x1p-13f : 1.f);
#pragma unroll
                    for (int i = 0; i < D / 32; ++i) {
                        float o[8];
#pragma unroll
                        for (int e = 0; e < 8; ++e) o[e] = value(i, e) * unit;
                        store8(p.out, cur_s * p.os + (long long)head * D + place(i), p.dt, o);
                    }
                    if (p.lse && t == 0)
                        p.lse[(long long)cur_s * p.heads + head] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
                }
            } else {
                if (u + 1 < u1) save(warp_part);   // more follows: the first partial result leaves by way of L2
                else open = true;
                if (lane == 0) {
                    part_s[warp][open ? 1 : 0] = cur_s;
                    part_item[warp][open ? 1 : 0] = cur_item;
                }
                ++parts;
            }
        }
    }
    copy_wait<0>();
    __syncthreads();   // every ring is empty
    if (open) save(reinterpret_cast<float *>(ring));
    __syncthreads();

    // ---- partial results of the CTA's warps, item by item ---------------------------
    auto part_of = [&](int i) {   // contribution i: warp i / 2, its first or its last
        return i & 1 ? reinterpret_cast<const float *>(smem + (i / 2) * C::kRing)
                     : p.part + (size_t)gridDim.x * 2 * (C::kPart / 4) + (size_t)(blockIdx.x * W + i / 2) * (C::kPart / 4);
    };
    constexpr int EL = kHeads * D / (32 * W);          // consecutive elements of a thread
    static_assert(EL == 2 || EL == 4, "");
    const int e0 = threadIdx.x * EL, h = e0 / D;
    // joins (pm, pl, po) of one contribution to the thread's sums
    auto join = [&](float &jm, float &jl, float (&jo)[EL], const float *src, bool far) {
        const float pm = far ? __ldcg(src + kHeads * D + h) : src[kHeads * D + h];
        const float pl = far ? __ldcg(src + kHeads * D + kHeads + h) : src[kHeads * D + kHeads + h];
        float po[EL];
#pragma unroll
        for (int e = 0; e < EL; e += 2) {
            const float2 v = far ? __ldcg(reinterpret_cast<const float2 *>(src + e0 + e)) : *reinterpret_cast<const float2 *>(src + e0 + e);
            po[e] = v.x;
            po[e + 1] = v.y;
        }
        const float nm = fmaxf(jm, pm), zero = nm == -INFINITY ? 0.f : nm;
        const float a = exp2_(jm - zero), b = exp2_(pm - zero);
        jl = jl * a + pl * b;
#pragma unroll
        for (int e = 0; e < EL; ++e) jo[e] = jo[e] * a + po[e] * b;
        jm = nm;
    };
    auto finish = [&](int s, int item, float jm, float jl, const float (&jo)[EL]) {
        const int hb = item % blocks_per_head * kHeads + h;
        if (hb >= p.group) return;
        const int head = item / blocks_per_head * p.group + hb;
        const float unit = jl == 0.f ? 0.f : 1.f / jl;
        const long long i = s * p.os + (long long)head * D + e0 % D;
#pragma unroll
        for (int e = 0; e < EL; e += 2) {
            if (p.dt == kF32) *reinterpret_cast<float2 *>(reinterpret_cast<float *>(p.out) + i + e) = make_float2(jo[e] * unit, jo[e + 1] * unit);
            else *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(p.out) + i + e) = pack2(jo[e] * unit, jo[e + 1] * unit, p.dt);
        }
        if (p.lse && e0 % D == 0)
            p.lse[(long long)s * p.heads + head] = jl == 0.f ? -INFINITY : (jm + log2f(jl)) * 0.6931471805599453f;
    };
    for (int i = 0; i < 2 * W;) {
        const int s = part_s[i / 2][i & 1];
        if (s < 0) {
            ++i;
            continue;
        }
        const int item = part_item[i / 2][i & 1];
        float jm = -INFINITY, jl = 0.f, jo[EL] = {};
        int j = i;
        for (; j < 2 * W; ++j) {
            const int s2 = part_s[j / 2][j & 1];
            if (s2 < 0) continue;
            if (s2 != s || part_item[j / 2][j & 1] != item) break;
            join(jm, jl, jo, part_of(j), !(j & 1));
        }
        i = j;
        // the item's chunks, and whether they are all in this CTA
        long long start = offs[s / per];
        for (int r = s / per * per; r < s; ++r) {
            const Span sp = span_of(p, r, false);
            start += (long long)(sp.c1 - sp.c0) * items;
        }
        const Span sp = span_of(p, s, false);
        const int nc = sp.c1 - sp.c0;
        start += (long long)item * nc;
        const long long end = start + nc;
        if (start >= cta0 && end <= cta1) {
            finish(s, item, jm, jl, jo);
            continue;
        }
        const int a = int(((start + 1) * ctas - 1) / total), b = int((end * ctas - 1) / total);   // CTAs of its first and last chunk
        // slots: 2 CTA for an item that began before the CTA (or fills it), 2 CTA + 1 for one that begins in it
        float *dst = p.part + (size_t)(2 * blockIdx.x + (int(blockIdx.x) == a)) * (C::kPart / 4);
#pragma unroll
        for (int e = 0; e < EL; e += 2) *reinterpret_cast<float2 *>(dst + e0 + e) = make_float2(jo[e], jo[e + 1]);
        if (e0 % D == 0) {
            dst[kHeads * D + h] = jm;
            dst[kHeads * D + kHeads + h] = jl;
        }
        __threadfence();
        __syncthreads();
        if (threadIdx.x == 0) {
            const bool all = atomicAdd(p.tickets + a, 1u) == unsigned(b - a);
            if (all) p.tickets[a] = 0;   // zero again for the next call
            is_last = all;
        }
        __syncthreads();
        if (is_last) {
            __threadfence();
            jm = -INFINITY;
            jl = 0.f;
#pragma unroll
            for (int e = 0; e < EL; ++e) jo[e] = 0.f;
            for (int c = a; c <= b; ++c) join(jm, jl, jo, p.part + (size_t)(2 * c + (c == a)) * (C::kPart / 4), true);
            finish(s, item, jm, jl, jo);
        }
        __syncthreads();
    }
}

template <int FMT, int D>
cudaError_t launch(const AttnParams &p, cudaStream_t st, bool set)
{
    using C = Cfg<FMT, D>;
    if (set) return cudaFuncSetAttribute(k_paged<FMT, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    const int blocks = (p.group + kHeads - 1) / kHeads;
    k_paged<FMT, D><<<p.n_sm, 32 * C::kWarps, C::kSmem, st>>>(p, p.kv_heads * blocks, blocks);
    return cudaGetLastError();
}

template <int FMT>
cudaError_t by_dim(const AttnParams &p, cudaStream_t st, bool set)
{
    return p.dim == 128 ? launch<FMT, 128>(p, st, set) : launch<FMT, 64>(p, st, set);
}

cudaError_t dispatch(const AttnParams &p, cudaStream_t st, bool set)
{
    switch (p.c.fmt) {
    case kF16: return by_dim<kF16>(p, st, set);
    case kBF16: return by_dim<kBF16>(p, st, set);
    case kI8: return by_dim<kI8>(p, st, set);
    default: return by_dim<kI4>(p, st, set);
    }
}

}  // namespace

// 2 partial results for each CTA, then one for each warp
size_t attn_part_bytes(int n_sm) { return size_t(n_sm) * (2 + kMaxWarps) * Cfg<kF16, 128>::kPart; }
size_t attn_ticket_bytes(int n_sm) { return size_t(n_sm) * sizeof(unsigned); }

cudaError_t attn_setup()
{
    AttnParams p{};
    for (int fmt : {int(kF16), int(kBF16), int(kI8), int(kI4)})
        for (int dim : {64, 128}) {
            p.c.fmt = fmt;
            p.dim = dim;
            const cudaError_t e = dispatch(p, nullptr, true);
            if (e != cudaSuccess) return e;
        }
    return cudaSuccess;
}

cudaError_t paged_attention(const AttnParams &p, cudaStream_t st) { return dispatch(p, st, false); }

}  // namespace pi
