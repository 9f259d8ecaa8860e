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
// run on mma.sync m16n8k16 with the cache as the matrix of 16 rows (positions
// for the scores, elements of V for the sums) and 4 query heads as 8 columns:
// column 2h holds head h's queries or weights in 16 bits, column 2h + 1 what
// that rounding left, so that the products are those of 22 (bf16: 16) bits with
// the cache's 16-, 8- or 4-bit numbers, which are exact.  Over a bf16 cache 16 bits
// are all that F16 and BF16 callers' queries and results have; F32 callers get 24
// (WIDE): each product twice, with half the rounding in both first columns, and
// what is left in two parts (32 texts of 4096 positions, 4 queries to a cached head:
// 106.1 us instead of 103.5; 16 texts, 16 queries to a head of 64: 57.5, 50.0).  A
// head's two columns meet in one lane.  Scales of quantised rows are applied in
// fp32, to the scores (K) and to the weights (V).
//
// Measured: 32 ragged texts of bf16 (525 MB) 104 us, 5.0 TB/s; 32768 positions of
// 4 bits 24.0 us, of which 12 are its chunks' instructions and 10 the way to the
// first product and from the last to the result; 16 texts of 8 bits in a window,
// 16 queries to a cached head, 37.1 us, bound by instructions (taking 8 instead of
// 16 heads at a time, with 12 instead of 8 warps, makes it 6% longer).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cfloat>

#include "pi_attn.h"

namespace pi {
namespace {

// What the start of an item costs, in chunks (8-bit window of 16 ragged texts: with 1 18% longer, with 4 1% shorter; 200
// positions: 1% and 27% longer).
constexpr int kStart = 2;
constexpr int kSlots = 32;            // partial results of a CTA's warps, at most (2 for each)

// FMT: the cache's format.  NB: tiles of 4 query heads that share a cached head.
// WIDE: F32 queries and results over a bf16 cache.
template <int FMT, int D, int NB, bool WIDE = false>
struct Cfg {
    static_assert(!WIDE || FMT == kBF16, "");
    static constexpr bool kF = FMT == kF16 || FMT == kBF16;
    static constexpr int kRow = FMT == kI8 ? D : FMT == kI4 ? D / 2 : 2 * D;   // bytes of a cached row
    static constexpr int kScale = FMT == kI8 ? 4 : FMT == kI4 ? D / 16 : 0;    // bytes of its scales
    static constexpr int kPieces = kRow / 16;
    // Positions of a chunk: two times 16 where rows are small, for more independent work.
    static constexpr int kTiles = kRow <= 64 ? 2 : 1, kChunk = 16 * kTiles;
    static constexpr int kCodes = kChunk * kRow;                              // bytes of a chunk's K (or V)
    static constexpr int kOffV = kCodes, kOffS = 2 * kCodes, kOffI = kOffS + (kScale ? 16 * kChunk : 0);
    static constexpr int kStage = kOffI + 16;
    static constexpr int kHeads = 4 * NB;                                     // query heads of an item
    static constexpr int kStep = D / 16;                                      // products of 16 along the head
    static constexpr bool kQShared = WIDE || NB * D >= 512;                   // queries stay in shared memory
    static constexpr int kDP = D + 8;                                         // a head's distance in a partial result
    static constexpr int kPart = kHeads * (kDP + 2) * 4;                      // its bytes: o, then m and l
    static constexpr int kOffQ2 = kHeads * (kDP + 8) * 4;                     // WIDE: the queries' last parts
    static constexpr int kBuf = kOffQ2 + (WIDE ? 8 * D * NB : 0);             // a warp's: queries, later its result
    // Warps of a CTA: as many as registers and three stages each allow.
    static constexpr int kWarps = kF && D == 128 ? (NB == 4 ? 4 : NB == 2 ? 6 : 8) : NB * D == 64 && FMT != kI8 && !WIDE ? 16 : NB * D <= 128 ? 12 : 8;
    static constexpr int kRoom = 220 * 1024 / kWarps / 16 * 16;
    static constexpr int kStages = (kRoom - kBuf) / kStage < 8 ? (kRoom - kBuf) / kStage : 8;
    static constexpr int kRing = kStages * kStage;
    static constexpr int kSmem = kWarps * (kRing + kBuf);
    static_assert(kStages >= 3 && kBuf % 16 == 0 && kRing % 16 == 0 && kSmem + 7168 <= 227 * 1024, "");
    static_assert(kOffQ2 >= kHeads * kDP * 4 + kHeads * 4 && 16 * D * NB <= kHeads * kDP * 4, "");
};

__device__ __forceinline__ uint32_t s2u(const void *p) { return uint32_t(__cvta_generic_to_shared(p)); }

__device__ __forceinline__ float exp2_(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

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
// Four 8x8 matrices of 16-bit units, rows at the addresses of lanes 0-7, 8-15, ...
template <bool TRANS>
__device__ __forceinline__ void ldm4(uint32_t a, uint32_t (&r)[4])
{
    if (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ uint32_t transpose8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

constexpr float kLargeCap = 64.f;
// cap * tanh(y / cap) for x = 2 log2 e * y / cap.
__device__ __noinline__ float whole_cap(float x, float cap) { return cap * tanhf(0.34657359f * x); }

// 1 / x within 2^-23 of it.
__device__ __forceinline__ float reciprocal(float x)
{
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// d = A B + c
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint2 b, float c0, float c1, float c2, float c3)
{
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%10, %11, %12, %13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
                     "{%8, %9}, {%10, %11, %12, %13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b.x), "r"(b.y), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint2 b) { mma<BF>(d, a, b, d[0], d[1], d[2], d[3]); }
// The first product of a sum.
template <bool BF>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint2 b, bool first)
{
    if (first) mma<BF>(d, a, b, 0.f, 0.f, 0.f, 0.f);
    else mma<BF>(d, a, b);
}

// The two parts' sum.  An infinite high part stands alone: its low part holds 0
// times that infinity.
__device__ __forceinline__ float whole(float hi, float lo) { return isinf(hi) ? hi : hi + lo; }

__device__ __forceinline__ uint32_t hsub(uint32_t v, uint32_t m)
{
    const __half2 d = __hsub2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&m));
    return *reinterpret_cast<const uint32_t *>(&d);
}
__device__ __forceinline__ uint32_t hfma(uint32_t v, uint32_t a, uint32_t b)
{
    const __half2 d = __hfma2(*reinterpret_cast<const __half2 *>(&v), *reinterpret_cast<const __half2 *>(&a),
                              *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&d);
}
// (v & mask) | bits, in one instruction.
__device__ __forceinline__ uint32_t and_or(uint32_t v, uint32_t mask, uint32_t bits)
{
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(v), "r"(mask), "r"(bits));
    return r;
}

// Codes n of 4 bits (at bits 4 i of each half) as fp16 pairs n - 8: under the
// exponent of 1024 a code is 1024 + n, four bits further up 1024 + 16 n; what
// leads from there to n - 8 is exact.
__device__ __forceinline__ void nibbles(uint32_t w, uint32_t (&r)[4])
{
    const uint32_t z = w >> 8;
    r[0] = hsub(and_or(w, 0x000f000fu, 0x64006400u), 0x64086408u);
    r[1] = hfma(and_or(w, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
    r[2] = hsub(and_or(z, 0x000f000fu, 0x64006400u), 0x64086408u);
    r[3] = hfma(and_or(z, 0x00f000f0u, 0x64006400u), 0x2c002c00u, 0xd480d480u);
}
// Two bytes of w (signed, with the top bit flipped) as an fp16 pair: under the
// exponent of 1024 a byte b is 1024 + b.
template <uint32_t SEL>
__device__ __forceinline__ uint32_t bytes(uint32_t w) { return hsub(__byte_perm(w, 0x64646464u, SEL), 0x64806480u); }

// The j-th of four fp16 numbers.
__device__ __forceinline__ float half_of(uint2 v, int j)
{
    const uint32_t w = j < 2 ? v.x : v.y;
    const __half2 h = *reinterpret_cast<const __half2 *>(&w);
    return j & 1 ? __high2float(h) : __low2float(h);
}
// Two numbers' 16-bit roundings, and the roundings of what is left.
template <bool BF>
__device__ __forceinline__ uint2 split2(float a, float b)
{
    if (BF) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
        const float2 f = __bfloat1622float2(h);
        const __nv_bfloat162 l = __floats2bfloat162_rn(a - f.x, b - f.y);
        return make_uint2(*reinterpret_cast<const uint32_t *>(&h), *reinterpret_cast<const uint32_t *>(&l));
    }
    const __half2 h = __floats2half2_rn(a, b);
    const float2 f = __half22float2(h);
    const __half2 l = __floats2half2_rn(a - f.x, b - f.y);
    return make_uint2(*reinterpret_cast<const uint32_t *>(&h), *reinterpret_cast<const uint32_t *>(&l));
}

// Two numbers' words (rounding; what is left) as one word for each: its pair of columns.
__device__ __forceinline__ uint2 columns(uint2 w) { return make_uint2(__byte_perm(w.x, w.y, 0x5410), __byte_perm(w.x, w.y, 0x7632)); }
// Each number as its rounding (low half) and that of what is left (high half).
template <bool BF>
__device__ __forceinline__ uint2 parts(float a, float b)
{
    return columns(split2<BF>(a, b));
}

// Two numbers in 24 bits, for two products: half their rounding (twice, so that an
// infinity of the cache meets no zero there) with what is left, and with what that left.
__device__ __forceinline__ void split4(float a, float b, uint2 &first, uint2 &second)
{
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    const float2 f = __bfloat1622float2(h);
    const __nv_bfloat162 half = __floats2bfloat162_rn(0.5f * f.x, 0.5f * f.y);
    const uint2 rest = split2<true>(a - f.x, b - f.y);
    const uint32_t u = *reinterpret_cast<const uint32_t *>(&half);
    first = make_uint2(u, rest.x);
    second = make_uint2(u, rest.y);
}
// Eight consecutive results from shared memory.
__device__ __forceinline__ void output8(uint8_t *p, long long i, int dt, const float *v)
{
    const float4 a = *reinterpret_cast<const float4 *>(v), b = *reinterpret_cast<const float4 *>(v + 4);
    if (dt == kF32) {
        reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i)[0] = a;
        reinterpret_cast<float4 *>(reinterpret_cast<float *>(p) + i)[1] = b;
    } else if (dt == kF16) {
        const __half2 h[4] = {__floats2half2_rn(a.x, a.y), __floats2half2_rn(a.z, a.w), __floats2half2_rn(b.x, b.y), __floats2half2_rn(b.z, b.w)};
        *reinterpret_cast<uint4 *>(p + 2 * i) = *reinterpret_cast<const uint4 *>(h);
    } else {
        const __nv_bfloat162 h[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w), __floats2bfloat162_rn(b.x, b.y),
                                     __floats2bfloat162_rn(b.z, b.w)};
        *reinterpret_cast<uint4 *>(p + 2 * i) = *reinterpret_cast<const uint4 *>(h);
    }
}
// log of sum l at maximum m (a power of two's exponents); -infinity without any position.
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f; }

// Positions of one sequence that its query sees, and the chunks that hold them.
// A sequence with none has one chunk without positions, whose result is 0.
// (CH: positions of a chunk.)
struct Span {
    int lo, hi, c0, c1;
};
template <int CH>
__device__ __forceinline__ Span span_of(const AttnParams &p, int s, bool report)
{
    int len = __ldg(p.len + s);
    const int room = p.c.width << p.c.page_shift;   // at most 2^30
    if (len < 0 || len > room) {
        if (report) atomicExch(p.err, int(kDevCheck));
        len = len < 0 ? 0 : room;
    }
    Span r;
    r.hi = len;
    r.lo = p.window && len > p.window ? len - p.window : 0;
    r.c0 = r.lo / CH;
    r.c1 = max((r.hi + CH - 1) / CH, r.c0 + 1);
    return r;
}

// The work of a call in units: one for each chunk, and kStart before each item,
// for its start (queries, the result).  CTA c takes the units from first(c) up to
// first(c + 1): an even share, and item by item where all items are alike and
// the CTAs a multiple of them.
struct Shares {
    int total, ctas, each, more;
    __device__ Shares(int total_, int ctas_) : total(total_), ctas(ctas_), each(unsigned(total_) / unsigned(ctas_)), more(total_ - each * ctas_) {}
    __device__ int first(int c) const { return c * each + int(unsigned(c * more) / unsigned(ctas)); }
    __device__ int of(int unit) const
    {
        int c = int(float(unit) * (float(ctas) / float(total)));   // off by one at most
        if (first(c) > unit) --c;
        return first(c + 1) <= unit ? c + 1 : c;
    }
};

// Where a warp is in the row of all chunks: sequence s, item i of the
// sequence (cached head and block of its query heads), chunk c.
struct Cursor {
    int s, item, c;
    Span span;
};

// An item that has partial results in a CTA: their slots, and the CTAs that hold its first and last chunk.
struct Joint {
    int s, item, a, b;
    int begin, count;      // in the list of slots
};

enum { kFirst = 1, kLast = 2, kWhole = 4 };   // a chunk in its segment; a segment that is its whole item

// Weights times V scales s are taken relative to 2^(ref - 127), the largest s
// so far, and brought to fp16's range by 2^13.  The least ref keeps 2^(127 -
// ref + 13) finite, for rows of zeros (s = 0).
constexpr int kLeastRef = 16;

// A power of two from its exponent.
__device__ __forceinline__ float pow2_of(int biased) { return __int_as_float(biased << 23); }

template <int FMT, int D, int NB, bool WIDE>
__global__ void __launch_bounds__(32 * Cfg<FMT, D, NB, WIDE>::kWarps, 1) k_paged(AttnParams p, int items, int blocks_per_head)
{
    using C = Cfg<FMT, D, NB, WIDE>;
    constexpr bool BF = FMT == kBF16;
    constexpr int W = C::kWarps, S = C::kStages, T = 32 * W, KS = C::kStep, P = C::kPieces, DP = C::kDP, H = C::kHeads;
    constexpr int R = C::kTiles, CH = C::kChunk;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ int sums[W], offs[T];
    // partial results: slot 2 w of warp w's first segment (in global memory), 2 w + 1 of its last (in its buffer)
    __shared__ int part_s[kSlots], part_item[kSlots];
    __shared__ float part_m[2 * W][H], part_l[2 * W][H], part_f[2 * W][H];
    __shared__ Joint joints[2 * W];
    __shared__ int slot_list[kSlots];
    __shared__ const float *slot_at[kSlots];
    __shared__ int n_joints, last[2];
    __shared__ float2 joint_of[H];
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32, g = lane / 4, t = lane % 4;
    const int n = p.c.n_seqs;
    allow_next();
    after_previous();

    // ---- units before each sequence, or each thread's block of `per` sequences ---------
    const bool few = n <= 32;   // every warp counts for itself (and needs no barrier)
    const int per = few ? 1 : (n + T - 1) / T;
    int mine = 0, total = 0, scan;
#pragma unroll 1
    for (int i = few ? lane : threadIdx.x * per, end = min(n, i + per); i < end; ++i) {
        const Span r = span_of<CH>(p, i, blockIdx.x == 0 && (!few || warp == 0));
        mine += (r.c1 - r.c0 + kStart) * items;
    }
    scan = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(~0u, scan, o);
        if (lane >= o) scan += v;
    }
    if (lane < 2) part_s[2 * warp + lane] = -1;
    if (few) {
        total = __shfl_sync(~0u, scan, 31);
        if (warp == 0) offs[lane] = scan - mine;   // (for the joins)
    } else {
        if (lane == 31) sums[warp] = scan;
        __syncthreads();
        int before = 0;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            before += w < warp ? sums[w] : 0;
            total += sums[w];
        }
        offs[threadIdx.x] = before + scan - mine;   // (blocks without sequences: the total)
        __syncthreads();
    }

    // ---- this warp's share ---------------------------------------------------
    int ctas = min((total + W - 1) / W, int(gridDim.x));   // at least a unit for each warp
    // One text: no CTA with parts of two items, which saves joins (bf16, 32 cached heads of 128: 200 positions 8.6 us instead
    // of 10.9, 2000 15.0, 16.9, 8000 33.9, 34.4) and leaves SMs idle (128 of 148 work: 32768 positions 104.9 us, 100.0).
    if (n == 1 && 4 * items <= int(gridDim.x)) ctas = max(ctas / items, 1) * items;
    if (int(blockIdx.x) >= ctas) return;
    const Shares shares(total, ctas);
    const int cta0 = shares.first(blockIdx.x), units = shares.first(blockIdx.x + 1) - cta0;
    const int u0 = cta0 + units * warp / W;
    int left = cta0 + units * (warp + 1) / W - u0;   // units not yet taken
    uint8_t *ring = smem + warp * C::kRing;
    const uint32_t ring_u = s2u(ring);
    float *buf = reinterpret_cast<float *>(smem + W * C::kRing + warp * C::kBuf);

    Cursor at{};
    if (left > 0) {
        int b = 0;   // the block that holds unit u0: the last one that starts at or before it
        int rest;
        if (few) {
            b = __popc(__ballot_sync(~0u, lane < n && scan - mine <= u0)) - 1;
            rest = u0 - __shfl_sync(~0u, scan - mine, b);
        } else {
            for (int end = T; end - b > 1;) {
                const int mid = (b + end) / 2;
                if (offs[mid] <= u0) b = mid;
                else end = mid;
            }
            rest = u0 - offs[b];
        }
        at.s = b * per;
        for (;;) {
            at.span = span_of<CH>(p, at.s, false);
            const int here = (at.span.c1 - at.span.c0 + kStart) * items;
            if (rest < here) break;
            rest -= here;
            ++at.s;
        }
        const int nu = at.span.c1 - at.span.c0 + kStart;
        at.item = unsigned(rest) / unsigned(nu);
        const int unit = rest - at.item * nu;   // below kStart: the item's start
        left -= max(kStart - unit, 0);
        at.c = at.span.c0 + max(unit - kStart, 0);
    }

    // ---- copies of one chunk into a stage --------------------------------------
    // Row r's 16-byte piece i lies at piece place(r, i): 8 rows' same pieces meet all banks once.
    auto place = [](int r, int i) { return r * P + (i ^ (P >= 8 ? r & 7 : P == 4 ? (r >> 1) & 3 : (r >> 2) & 1)); };
    constexpr int RI = 32 / P;            // rows of one copy instruction
    const int my_row = lane / P, my_piece = lane % P;
    const unsigned slot_bytes = p.c.slot_rows * C::kRow;   // 2^18 at most
    // Pages of the 8 positions from 8 (page_g + lane) of sequence page_s.
    int page_s = -1, page_g = 0, my_page = -1;
    int issued = 0, head = at.item / blocks_per_head * p.c.head_rows;
    bool first = true, from_start = at.c == at.span.c0;
    auto issue = [&](int stage) {
        if (left <= 0) {
            copy_commit();
            return;
        }
        const int pos = at.c * CH, grp = pos / 8;
        if (at.s != page_s || unsigned(grp - page_g) >= 32u) {
            page_s = at.s;
            page_g = grp;
            const int a = pos + 8 * lane;   // (below 2^30 + 2^8)
            my_page = a < at.span.hi && a + 8 > at.span.lo
                          ? __ldg(p.c.table + at.s * p.c.tstride + (a >> p.c.page_shift)) : -1;
        }
        // positions seen, by bit
        unsigned mask = CH == 32 ? ~0u : 0xffffu;
        if (pos + CH > at.span.hi) mask = at.span.hi > pos ? (1u << (at.span.hi - pos)) - 1 : 0;
        if (pos < at.span.lo) mask &= ~((1u << (at.span.lo - pos)) - 1);
        // first rows of the groups of 8; a row without a position is filled with zeros (its memory is not read)
        long long first_row[2 * R], key_row = 0;   // key_row: of position key, whose scales this lane copies
        const int key = lane % CH;
        auto row_at = [&](int page, int position) -> long long {
            return unsigned(page) < unsigned(p.c.n_pages)
                       ? (long long)page * p.c.page_rows + ((position & (p.c.page_size - 1)) * p.c.slot_rows + head) : -1;
        };
        if (p.c.page_size >= CH) {   // one page holds them all
            const long long row = row_at(__shfl_sync(~0u, my_page, grp - page_g + ((__ffs(mask | 1u << (CH - 1)) - 1) >> 3)), pos);
            if (row < 0) {
                if (lane == 0 && mask) atomicExch(p.err, int(kDevCheck));
                mask = 0;
            }
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) first_row[i] = max(row, 0ll) + 8 * i * p.c.slot_rows;
            if (C::kScale) key_row = max(row, 0ll) + key * p.c.slot_rows;
        } else {
#pragma unroll
            for (int i = 0; i < 2 * R; ++i) {
                const long long row = row_at(__shfl_sync(~0u, my_page, grp - page_g + i), pos + 8 * i);
                if (row < 0) {
                    if (lane == 0 && (mask & 0xffu << (8 * i))) atomicExch(p.err, int(kDevCheck));
                    mask &= ~(0xffu << (8 * i));
                }
                first_row[i] = max(row, 0ll);
            }
            if (C::kScale) key_row = max(row_at(__shfl_sync(~0u, my_page, grp - page_g + key / 8), pos + key), 0ll);
        }
        const uint32_t dst = ring_u + stage * C::kStage;
        const bool all = mask == (CH == 32 ? ~0u : 0xffffu);
#pragma unroll
        for (int i = 0; i < CH / RI; ++i) {
            const int row = my_row + i * RI;
            const long long off = (RI == 16 && my_row >= 8 ? first_row[i * RI / 8 + 1] : first_row[i * RI / 8]) * C::kRow +
                                  ((row & 7) * slot_bytes + 16 * my_piece);
            const uint32_t to = dst + 16 * place(row, my_piece);
            const bool live = all || (mask >> row) & 1;
            copy_async<16>(to, p.c.k + off, live);
            copy_async<16>(to + C::kOffV, p.c.v + off, live);
        }
        if (C::kScale) {   // entries: K of all positions, then V
#pragma unroll
            for (int i = 0; i < R; ++i) {
                const int entry = lane + 32 * i;
                const uint8_t *base = (entry < CH ? p.c.ks : p.c.vs) + key_row * C::kScale;
                copy_async<C::kScale ? C::kScale : 4>(dst + C::kOffS + entry * 8, base, (mask >> key) & 1);
            }
        }
        copy_commit();
        // what the reader has to know
        const bool ends = at.c + 1 == at.span.c1, last = ends || left == 1;
        if (lane == 0)
            *reinterpret_cast<int4 *>(ring + stage * C::kStage + C::kOffI) =
                make_int4(int(mask), (first ? kFirst : 0) | (last ? kLast : 0) | (ends && from_start ? kWhole : 0), at.s, at.item);
        first = last;
        ++issued;
        --left;
        if (!ends) {
            ++at.c;
            return;
        }
        from_start = true;
        if ((left -= kStart) <= 0) return;   // (the next item's start)
        if (++at.item == items) {
            at.item = 0;
            ++at.s;
            at.span = span_of<CH>(p, at.s, false);
        }
        at.c = at.span.c0;
        head = at.item / blocks_per_head * p.c.head_rows;
    };
    // ---- one chunk after the other ---------------------------------------------
    uint2 q[C::kQShared ? 1 : KS][C::kQShared ? 1 : NB];
    float acc[NB][KS][4] = {};
    float m[NB], l[NB], factor[NB];            // of head 4 b + t; l of positions g and g + 8 only, until the segment's end
#pragma unroll
    for (int b = 0; b < NB; ++b) m[b] = -FLT_MAX, l[b] = factor[b] = 0.f;
    int ref = kLeastRef;
    int cur_s = -1, cur_item = 0;
    // elements of V in acc[.][i]: rows g and g + 8
    auto element = [&](int i, int second) {
        if (FMT == kI8) return 16 * i + 2 * g + second;
        if (FMT == kI4) return 32 * (i / 2) + 4 * g + 2 * (i & 1) + second;
        return 16 * i + 8 * second + g;
    };
    float *warp_part = p.part + (size_t)gridDim.x * 2 * (C::kPart / 4) + (size_t)(blockIdx.x * W + warp) * (C::kPart / 4);
    // this lane's row in loads of four matrices: rows 0-7 and 8-15 of piece 2 i, then of piece 2 i + 1 (K, and V of
    // 8 and 4 bits), or rows 0-7 of pieces 2 i and 2 i + 1, then rows 8-15 (V of 16 bits)
    const int mat_row = lane & 15, mat_piece = lane >> 4;
    const int mat_row_v = C::kF ? (lane & 7) + 8 * (lane >> 4) : mat_row, mat_piece_v = C::kF ? (lane >> 3) & 1 : mat_piece;

    int stage = 0, put = 0;
#pragma unroll 1
    for (int u = 1 - S; u < issued; ++u) {
        issue(put);
        put = put + 1 == S ? 0 : put + 1;
        if (u < 0) continue;
        __syncwarp();
        const uint32_t base = ring_u + stage * C::kStage;
        const int4 info = *reinterpret_cast<const int4 *>(ring + stage * C::kStage + C::kOffI);
        const unsigned mask = unsigned(info.x);
        if (info.y & kFirst) {
            cur_s = info.z;
            cur_item = info.w;
            // The queries' parts go to the buffer as the products take them: word (i, b, column 4 lanes, t) holds column
            // g's parts of places 2t, 2t + 1 and 2t + 8, 2t + 9 of product i.  Eight lanes share a head here.
            uint32_t *words = reinterpret_cast<uint32_t *>(buf);
            float *extra = buf + H * DP;   // factors
            const int hl = lane / 8, part = lane % 8;
            if (NB > 1) {   // all on their way to L1 at once
#pragma unroll
                for (int b = 0; b < NB; ++b) {
                    const int head = min(cur_item % blocks_per_head * H + 4 * b + hl, p.group - 1);
                    const long long at_q = cur_s * p.qs + (long long)(cur_item / blocks_per_head * p.group + head) * D + part * (D / 8);
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(p.q + at_q * (p.dt == kF32 ? 4 : 2)));
                }
            }
#pragma unroll 1
            for (int b = 0; b < NB; ++b) {
                constexpr int E = D / 8;   // elements of a lane: part E, ...
                const int head = cur_item % blocks_per_head * H + 4 * b + hl;   // in its group
                const bool live = head < p.group;
                const long long row = live ? cur_s * p.qs + (long long)(cur_item / blocks_per_head * p.group + head) * D : 0;
                float v[E], top = 0.f;
                if (p.dt == kF32) {
                    const float4 *src = reinterpret_cast<const float4 *>(reinterpret_cast<const float *>(p.q) + row + part * E);
#pragma unroll
                    for (int i = 0; i < E / 4; ++i) {
                        const float4 x = src[i];
                        v[4 * i] = x.x, v[4 * i + 1] = x.y, v[4 * i + 2] = x.z, v[4 * i + 3] = x.w;
                    }
                } else {
                    const uint4 *src = reinterpret_cast<const uint4 *>(reinterpret_cast<const uint16_t *>(p.q) + row + part * E);
#pragma unroll
                    for (int i = 0; i < E / 8; ++i) {
                        const uint4 x = src[i];
                        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float2 f = p.dt == kF16 ? __half22float2(*reinterpret_cast<const __half2 *>(&w[e]))
                                                          : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162 *>(&w[e]));
                            v[8 * i + 2 * e] = f.x;
                            v[8 * i + 2 * e + 1] = f.y;
                        }
                    }
                }
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    if (!live) v[e] = 0.f;
                    top = fmaxf(top, fabsf(v[e]));
                }
                // the head's largest element is brought to [1, 2), so that no part leaves the range of 16 bits
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 1));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 2));
                top = fmaxf(top, __shfl_xor_sync(~0u, top, 4));
                const int ex = min(max(__float_as_int(top) >> 23, 16), 253);
                const float down = pow2_of(254 - ex);
                if (part == 0)
                    extra[4 * b + hl] = pow2_of(ex) * (p.softcap > 0.f ? p.scale * (2.8853900817779268f / p.softcap) : p.scale * 1.4426950408889634f);
#pragma unroll
                for (int e = 0; e < E / 2; ++e) {   // a pair of elements, its product i, its place: word x or y of lanes 4 g + tt
                    const int d = part * E + 2 * e;
                    float x, y;
                    int i, tt, second;
                    if (FMT == kI4) {   // of 8 elements (0, 4), (1, 5), (2, 6), (3, 7)
                        const int at8 = 8 * (e / 4), k = e % 4;
                        x = v[at8 + k] * down;
                        y = v[at8 + k + 4] * down;
                        i = d / 32 * 2 + (k >> 1);
                        tt = d / 8 % 4;
                        second = k & 1;
                    } else {
                        x = v[2 * e] * down;
                        y = v[2 * e + 1] * down;
                        i = d / 16;
                        tt = FMT == kI8 ? d / 4 % 4 : d / 2 % 4;
                        second = FMT == kI8 ? d / 2 % 2 : d / 8 % 2;
                    }
                    uint32_t *to = words + (((i * NB + b) * 8 + 2 * hl) * 4 + tt) * 2 + second;
                    uint2 w, w2;
                    if (WIDE) {
                        split4(x, y, w, w2);
                        words[C::kOffQ2 / 4 + (((i * NB + b) * 4 + hl) * 4 + tt) * 2 + second] = w2.y;
                    } else {
                        w = split2<BF>(x, y);
                    }
                    to[0] = w.x;
                    to[8] = w.y;
                }
            }
            __syncwarp();
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                factor[b] = extra[4 * b + t];
                m[b] = -FLT_MAX;
                l[b] = 0.f;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    if (!C::kQShared) q[C::kQShared ? 0 : i][C::kQShared ? 0 : b] = reinterpret_cast<const uint2 *>(buf)[(i * NB + b) * 32 + lane];
                    acc[b][i][0] = acc[b][i][1] = acc[b][i][2] = acc[b][i][3] = 0.f;
                }
            }
            ref = kLeastRef;
        }
        copy_wait<S - 1>();
        __syncwarp();
        auto query = [&](int i, int b) {
            return C::kQShared ? reinterpret_cast<const uint2 *>(buf)[(i * NB + b) * 32 + lane] : q[C::kQShared ? 0 : i][C::kQShared ? 0 : b];
        };
        // (of the second products: the first columns are the first product's)
        auto query2 = [&](int i, int b) {
            return g & 1 ? reinterpret_cast<const uint2 *>(buf + C::kOffQ2 / 4)[(i * NB + b) * 16 + g / 2 * 4 + t] : query(i, b);
        };

        // ---- scores of head 4 b + t at positions 16 r + g and 16 r + g + 8
        float x[NB][2 * R];
        uint2 ks[2 * R], vs[2 * R];   // scales of these positions
        if (C::kScale) {
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) {
                if (FMT == kI8) {
                    ks[e].x = lds32(base + C::kOffS + (g + 8 * e) * 8);
                    vs[e].x = lds32(base + C::kOffS + 8 * CH + (g + 8 * e) * 8);
                } else {
                    ks[e] = lds64(base + C::kOffS + (g + 8 * e) * 8);
                    vs[e] = lds64(base + C::kOffS + 8 * CH + (g + 8 * e) * 8);
                }
            }
        }
        if (FMT == kI4) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2 * R; ++e) x[b][e] = 0.f;
#pragma unroll
            for (int i = 0; i < P / 2; ++i)
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    uint32_t r[4];
                    ldm4<false>(base + 16 * place(mat_row + 16 * rt, 2 * i + mat_piece), r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = 2 * i + h;
                        uint32_t p0[4], p1[4];   // elements (0, 4), (1, 5), (2, 6), (3, 7) of rows g and g + 8
                        nibbles(r[2 * h], p0);
                        nibbles(r[2 * h + 1], p1);
                        const uint32_t a0[4] = {p0[0], p1[0], p0[1], p1[1]}, a1[4] = {p0[2], p1[2], p0[3], p1[3]};
                        const float f0 = half_of(ks[2 * rt], j), f1 = half_of(ks[2 * rt + 1], j);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            float c[4];
                            mma<false>(c, a0, query(2 * j, b), true);
                            mma<false>(c, a1, query(2 * j + 1, b));
                            x[b][2 * rt] += f0 * (c[0] + c[1]);
                            x[b][2 * rt + 1] += f1 * (c[2] + c[3]);
                        }
                    }
                }
        } else {
            constexpr int CC = NB * R == 1 ? 2 : 1;   // independent sums, where there are few products to fill the pipe with
            float c[NB][R][CC][4];
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    if (FMT == kI8) {
                        if (i & 1) continue;
                        uint32_t r[4];
                        ldm4<false>(base + 16 * place(mat_row + 16 * rt, i + mat_piece), r);
#pragma unroll
                        for (int e = 0; e < 4; ++e) r[e] ^= 0x80808080u;
                        const uint32_t a0[4] = {bytes<0x4140>(r[0]), bytes<0x4140>(r[1]), bytes<0x4342>(r[0]), bytes<0x4342>(r[1])};
                        const uint32_t a1[4] = {bytes<0x4140>(r[2]), bytes<0x4140>(r[3]), bytes<0x4342>(r[2]), bytes<0x4342>(r[3])};
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            mma<false>(c[b][rt][0], a0, query(i, b), i == 0);
                            mma<false>(c[b][rt][CC - 1], a1, query(i + 1 < KS ? i + 1 : i, b), i == 0 && CC == 2);
                        }
                    } else {
                        uint32_t r[4];
                        ldm4<false>(base + 16 * place(mat_row + 16 * rt, 2 * i + mat_piece), r);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            mma<BF>(c[b][rt][i % CC], r, query(i, b), i < CC);
                            if (WIDE) mma<BF>(c[b][rt][i % CC], r, query2(i, b));
                        }
                    }
                }
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    float (&y)[4] = c[b][rt][0];
                    if (CC == 2) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) y[e] += c[b][rt][CC - 1][e];
                    }
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        x[b][2 * rt + e] = C::kF ? whole(y[2 * e], y[2 * e + 1]) : y[2 * e] + y[2 * e + 1];
                        if (FMT == kI8) x[b][2 * rt + e] *= __uint_as_float(ks[2 * rt + e].x);
                    }
                }
        }
        // what the mask leaves out is -infinity; cap * tanh(y / cap) = cap - 2 cap / (1 + e^(2y / cap)), which is off by
        // cap 2^-21 at most: for large caps, whose scores are small beside them, and for F32 callers tanh itself
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) x[b][e] *= factor[b];
        if (p.softcap > 0.f) {
            const float cap = p.softcap * 1.4426950408889634f;
            const bool itself = p.softcap > kLargeCap || p.dt == kF32;
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2 * R; ++e)
                    x[b][e] = itself ? whole_cap(x[b][e], cap) : fmaf(-2.f * cap, reciprocal(1.f + exp2_(x[b][e])), cap);
        }
        if (mask != (CH == 32 ? ~0u : 0xffffu)) {
#pragma unroll
            for (int e = 0; e < 2 * R; ++e)
                if (!((mask >> (g + 8 * e)) & 1)) {
#pragma unroll
                    for (int b = 0; b < NB; ++b) x[b][e] = -INFINITY;
                }
        }
        // (a NaN is passed over by the maxima and makes l and o NaN below)
        bool grows = false;
        float top[NB];
#pragma unroll
        for (int b = 0; b < NB; ++b) {
            top[b] = fmaxf(x[b][0], x[b][1]);
            if (R == 2) top[b] = fmaxf(top[b], fmaxf(x[b][2 * R - 2], x[b][2 * R - 1]));
            grows |= top[b] > m[b];
        }
        int big = 0;   // exponent of the largest V scale
        if (FMT == kI8) {
            float v = __uint_as_float(vs[0].x);
#pragma unroll
            for (int e = 1; e < 2 * R; ++e) v = fmaxf(v, __uint_as_float(vs[e].x));
            big = __float_as_int(v) >> 23;
        } else if (FMT == kI4) {
            __half2 hm = *reinterpret_cast<const __half2 *>(&vs[0].x);
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) {
                hm = __hmax2(hm, *reinterpret_cast<const __half2 *>(&vs[e].x));
                if (D == 128) hm = __hmax2(hm, *reinterpret_cast<const __half2 *>(&vs[e].y));
            }
            big = __float_as_int(__half2float(__hmax(__low2half(hm), __high2half(hm)))) >> 23;
        }
        if (__any_sync(~0u, grows || (C::kScale && big > ref))) {
            float both = 1.f;
            if (C::kScale) {
                if (FMT == kI4 && big == 255) {   // an infinite scale spoils its own group only: the largest of the others
                    big = 0;
#pragma unroll
                    for (int e = 0; e < 2 * R; ++e)
#pragma unroll
                        for (int j = 0; j < D / 32; ++j) {
                            const float sc = half_of(vs[e], j);
                            if (sc < INFINITY) big = max(big, __float_as_int(sc) >> 23);
                        }
                }
                const int grown = min(int(__reduce_max_sync(~0u, unsigned(max(ref, big)))), 253);
                both = grown - ref > 126 ? 0.f : pow2_of(127 + ref - grown);   // 2^(ref - grown); beyond floats' range 0
                ref = grown;
            }
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                float y = fmaxf(top[b], m[b]);
                y = fmaxf(y, __shfl_xor_sync(~0u, y, 4));
                y = fmaxf(y, __shfl_xor_sync(~0u, y, 8));
                y = fmaxf(y, __shfl_xor_sync(~0u, y, 16));
                const float shrink = exp2_(m[b] - y), f = shrink * both;
                l[b] *= shrink;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    acc[b][i][0] *= f;
                    acc[b][i][1] *= f;
                    acc[b][i][2] *= f;
                    acc[b][i][3] *= f;
                }
                m[b] = y;
            }
        }
        // ---- weights
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 2 * R; ++e) {
                // F16: weights carry a factor 2^14, so that the low parts of small ones stay normal numbers
                x[b][e] = exp2_(FMT == kF16 ? x[b][e] - m[b] + 14.f : x[b][e] - m[b]);
                l[b] += x[b][e];
            }
        // ---- sums of V
        const float f = pow2_of(254 - ref) * 0x1p13f;
        if (FMT == kI4) {
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int e = 0; e < 2 * R; ++e) x[b][e] *= f;
#pragma unroll
            for (int i = 0; i < P / 2; ++i)
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    uint32_t r[4];
                    ldm4<true>(base + C::kOffV + 16 * place(mat_row + 16 * rt, 2 * i + mat_piece), r);
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int j = 2 * i + h;
                        // element 4 g + e of positions 2t, 2t + 1 at bits 4 e
                        uint32_t p0[4], p1[4];
                        nibbles(r[2 * h], p0);
                        nibbles(r[2 * h + 1], p1);
                        const uint32_t a[2][4] = {{p0[0], p0[1], p1[0], p1[1]}, {p0[2], p0[3], p1[2], p1[3]}};
                        const float f0 = half_of(vs[2 * rt], j), f1 = half_of(vs[2 * rt + 1], j);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            const uint2 v = parts<false>(x[b][2 * rt] * f0, x[b][2 * rt + 1] * f1);
                            const uint2 w = make_uint2(transpose8(v.x), transpose8(v.y));
                            mma<false>(acc[b][2 * j], a[0], w);
                            mma<false>(acc[b][2 * j + 1], a[1], w);
                        }
                    }
                }
        } else {
            uint2 w[NB][R], w2[WIDE ? NB : 1][R];
#pragma unroll
            for (int b = 0; b < NB; ++b)
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    if (FMT == kI8) {
                        x[b][2 * rt] *= __uint_as_float(vs[2 * rt].x) * f;
                        x[b][2 * rt + 1] *= __uint_as_float(vs[2 * rt + 1].x) * f;
                    }
                    uint2 v;
                    if (WIDE) {
                        uint2 v2;
                        split4(x[b][2 * rt], x[b][2 * rt + 1], v, v2);
                        v = columns(v);
                        v2 = columns(v2);
                        w2[WIDE ? b : 0][rt] = make_uint2(transpose8(v2.x), transpose8(v2.y));
                    } else {
                        v = parts<BF>(x[b][2 * rt], x[b][2 * rt + 1]);
                    }
                    w[b][rt] = make_uint2(transpose8(v.x), transpose8(v.y));
                }
#pragma unroll
            for (int i = 0; i < KS; ++i)
#pragma unroll
                for (int rt = 0; rt < R; ++rt) {
                    uint32_t r[4];
                    if (FMT == kI8) {
                        if (i & 1) continue;
                        ldm4<true>(base + C::kOffV + 16 * place(mat_row_v + 16 * rt, i + mat_piece_v), r);
#pragma unroll
                        for (int e = 0; e < 4; ++e) r[e] ^= 0x80808080u;
                        // elements 2g and 2g + 1 of positions 2t, 2t + 1 in turn
                        const uint32_t a0[4] = {bytes<0x4240>(r[0]), bytes<0x4341>(r[0]), bytes<0x4240>(r[1]), bytes<0x4341>(r[1])};
                        const uint32_t a1[4] = {bytes<0x4240>(r[2]), bytes<0x4341>(r[2]), bytes<0x4240>(r[3]), bytes<0x4341>(r[3])};
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            mma<false>(acc[b][i], a0, w[b][rt]);
                            mma<false>(acc[b][i + 1 < KS ? i + 1 : i], a1, w[b][rt]);
                        }
                    } else {
                        ldm4<true>(base + C::kOffV + 16 * place(mat_row_v + 16 * rt, 2 * i + mat_piece_v), r);
#pragma unroll
                        for (int b = 0; b < NB; ++b) {
                            mma<BF>(acc[b][i], r, w[b][rt]);
                            if (WIDE) mma<BF>(acc[b][i], r, w2[WIDE ? b : 0][rt]);
                        }
                    }
                }
        }

        if (info.y & kLast) {   // o to the buffer, one row for each head
            if (C::kQShared) __syncwarp();
            const bool whole_item = info.y & kWhole, more = u + 1 < issued;
            const int slot = 2 * warp + !more;
#pragma unroll
            for (int b = 0; b < NB; ++b) {
                l[b] += __shfl_xor_sync(~0u, l[b], 4);
                l[b] += __shfl_xor_sync(~0u, l[b], 8);
                l[b] += __shfl_xor_sync(~0u, l[b], 16);
                float unit = C::kScale ? pow2_of(ref) * 0x1p-13f : FMT == kF16 ? 0x1p-14f : 1.f;
                if (FMT == kF16) l[b] *= 0x1p-14f;
                if (whole_item) unit = l[b] == 0.f ? 0.f : unit / l[b];
                float *o = buf + (4 * b + t) * DP;
#pragma unroll
                for (int i = 0; i < KS; ++i) {
                    o[element(i, 0)] = whole(acc[b][i][0], acc[b][i][1]) * unit;
                    o[element(i, 1)] = whole(acc[b][i][2], acc[b][i][3]) * unit;
                }
                if (g == 0 && !whole_item) {
                    part_m[slot][4 * b + t] = m[b];
                    part_l[slot][4 * b + t] = l[b];
                }
                if (g == 0 && whole_item && p.lse) {
                    const int hb = cur_item % blocks_per_head * H + 4 * b + t;
                    if (hb < p.group) p.lse[(long long)cur_s * p.heads + cur_item / blocks_per_head * p.group + hb] = lse_of(m[b], l[b]);
                }
            }
            __syncwarp();
            if (whole_item) {
                const int hb0 = cur_item % blocks_per_head * H;
                const long long row = cur_s * p.os + (long long)(cur_item / blocks_per_head * p.group + hb0) * D;
                const int end = min(p.group - hb0, H) * D;
#pragma unroll 1
                for (int e = 8 * lane; e < end; e += 256) output8(p.out, row + e, p.dt, buf + e / D * DP + e % D);
            } else {
                if (lane == 0) {
                    part_s[slot] = cur_s;
                    part_item[slot] = cur_item;
                }
                if (more) {   // the first partial result makes room by way of L2
#pragma unroll 1
                    for (int e = 4 * lane; e < H * DP; e += 128)
                        *reinterpret_cast<float4 *>(warp_part + e) = *reinterpret_cast<const float4 *>(buf + e);
                }
            }
        }
        __syncwarp();   // all have read the stage: the next copy may take it
        stage = stage + 1 == S ? 0 : stage + 1;
    }
    copy_wait<0>();
    __syncthreads();

    // ---- partial results of the CTA's warps, joined for each of their items ---------
    float *const cta_part = p.part + (size_t)gridDim.x * 2 * (C::kPart / 4) + (size_t)(blockIdx.x * W) * (C::kPart / 4);
    if (warp == 0) {   // one lane for each slot: the first slot of an item's run makes its entry
        const int s = lane < 2 * W ? part_s[lane] : -1, item = s >= 0 ? part_item[lane] : 0;
        const unsigned valid = __ballot_sync(~0u, s >= 0), before = valid & ((1u << lane) - 1);
        const int prev = before ? 31 - __clz(before) : lane;
        const int ps = __shfl_sync(~0u, s, prev), pi = __shfl_sync(~0u, item, prev);
        if (s >= 0) {
            slot_list[__popc(before)] = lane;
            slot_at[__popc(before)] = lane & 1 ? reinterpret_cast<const float *>(smem + W * C::kRing + (lane / 2) * C::kBuf)
                                               : cta_part + (size_t)(lane / 2) * (C::kPart / 4);
        }
        const bool head = s >= 0 && (!before || ps != s || pi != item);
        const unsigned heads = __ballot_sync(~0u, head);
        if (head) {
            Joint &j = joints[__popc(heads & ((1u << lane) - 1))];
            const unsigned later = heads & ~((2u << lane) - 1);
            j.s = s;
            j.item = item;
            j.begin = __popc(before);
            j.count = __popc(valid & ~((1u << lane) - 1) & (later ? (1u << (__ffs(later) - 1)) - 1 : ~0u));
            int start = offs[few ? s : s / per];
            for (int r = few ? s : s / per * per; r < s; ++r) {
                const Span sp = span_of<CH>(p, r, false);
                start += (sp.c1 - sp.c0 + kStart) * items;
            }
            const Span sp = span_of<CH>(p, s, false);
            const int nc = sp.c1 - sp.c0;
            start += item * (nc + kStart) + kStart;
            j.a = j.b = blockIdx.x;   // CTAs of its first and last chunk
            if (start < cta0) j.a = shares.of(start);
            if (start + nc > cta0 + units) j.b = shares.of(start + nc - 1);
        }
        if (lane == 0) n_joints = __popc(heads);
    }
    __syncthreads();
    const int nj = n_joints;
    // this CTA's partial results of items that others share: 2 CTA for one that began before it, 2 CTA + 1 for one
    // that begins in it
    auto far_of = [&](int cta, int a) { return p.part + (size_t)(2 * cta + (cta == a)) * (C::kPart / 4); };
    // four results of an item
    auto finish = [&](const Joint &j, int h, int d, float jm, float jl, float4 o) {
        const int hb = j.item % blocks_per_head * H + h;
        if (hb >= p.group) return;
        const int head = j.item / blocks_per_head * p.group + hb;
        const long long at4 = j.s * p.os + (long long)head * D + d;
        const float unit = jl == 0.f ? 0.f : 1.f / jl;
        o.x *= unit, o.y *= unit, o.z *= unit, o.w *= unit;
        if (p.dt == kF32) {
            *reinterpret_cast<float4 *>(reinterpret_cast<float *>(p.out) + at4) = o;
        } else if (p.dt == kF16) {
            const __half2 v[2] = {__floats2half2_rn(o.x, o.y), __floats2half2_rn(o.z, o.w)};
            *reinterpret_cast<uint2 *>(p.out + 2 * at4) = *reinterpret_cast<const uint2 *>(v);
        } else {
            const __nv_bfloat162 v[2] = {__floats2bfloat162_rn(o.x, o.y), __floats2bfloat162_rn(o.z, o.w)};
            *reinterpret_cast<uint2 *>(p.out + 2 * at4) = *reinterpret_cast<const uint2 *>(v);
        }
        if (p.lse && d == 0) p.lse[(long long)j.s * p.heads + head] = lse_of(jm, jl);
    };
    // weights of the slots by (item, head); the sums m and l in the rings, which are empty
    float *joint_m = reinterpret_cast<float *>(smem), *joint_l = joint_m + 2 * W * H;
    for (int e = threadIdx.x; e < nj * H; e += T) {
        const int h = e % H;
        const int k0 = joints[e / H].begin, k1 = k0 + joints[e / H].count;
        float jm = -FLT_MAX, jl = 0.f;
#pragma unroll 4
        for (int k = k0; k < k1; ++k) jm = fmaxf(jm, part_m[slot_list[k]][h]);
#pragma unroll 4
        for (int k = k0; k < k1; ++k) {
            const int i = slot_list[k];
            const float f = exp2_(part_m[i][h] - jm);
            part_f[k][h] = f;
            jl += f * part_l[i][h];
        }
        joint_m[e] = jm;
        joint_l[e] = jl;
    }
    __syncthreads();
#pragma unroll 1
    for (int e = threadIdx.x; e < nj * H * D / 4; e += T) {
        const Joint &j = joints[e / (H * D / 4)];
        const int h = e / (D / 4) % H, d = 4 * e % D, k1 = j.begin + j.count;
        float4 jo = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 1
        for (int k = j.begin; k < k1; k += 4) {   // four slots at a time
            float4 v[4];
            float f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int kk = min(k + i, k1 - 1);
                v[i] = *reinterpret_cast<const float4 *>(slot_at[kk] + h * DP + d);
                f[i] = part_f[kk][h];
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                if (k + i < k1) jo.x += f[i] * v[i].x, jo.y += f[i] * v[i].y, jo.z += f[i] * v[i].z, jo.w += f[i] * v[i].w;
        }
        const float jm = joint_m[e / (D / 4)], jl = joint_l[e / (D / 4)];
        if (j.a == j.b) {
            finish(j, h, d, jm, jl, jo);
        } else {
            float *dst = far_of(blockIdx.x, j.a);
            *reinterpret_cast<float4 *>(dst + h * DP + d) = jo;
            if (d == 0) {
                dst[H * DP + h] = jm;
                dst[H * (DP + 1) + h] = jl;
            }
        }
    }
    // ---- items that CTAs share: the CTA that is through last joins their results (its first and last item at most) ---
    if (nj == 0 || (joints[0].a == joints[0].b && joints[nj - 1].a == joints[nj - 1].b)) return;
    __threadfence();
    __syncthreads();
    if (threadIdx.x < 2) {
        const Joint &j = joints[threadIdx.x ? nj - 1 : 0];
        bool all = false;
        if (j.a != j.b && (threadIdx.x == 0 || nj > 1)) {
            all = atomicAdd(p.tickets + j.a, 1u) == unsigned(j.b - j.a);
            if (all) p.tickets[j.a] = 0;   // zero again for the next call
        }
        last[threadIdx.x] = all;
    }
    __syncthreads();
    // far_f: weights; far_o: sums of the thread groups
    float *far_f = reinterpret_cast<float *>(smem), *far_l = far_f + gridDim.x * H;
    constexpr int E4 = H * D / 4, G = T > E4 ? T / E4 : 1;   // threads of a result, groups of them
    float4 *far_o = reinterpret_cast<float4 *>(smem + 32 * 1024);
#pragma unroll 1
    for (int i = 0; i < 2; ++i) {
        if (!last[i]) continue;
        const Joint j = joints[i ? nj - 1 : 0];
        const int nc = j.b - j.a + 1;
        __threadfence();
        for (int e = threadIdx.x; e < nc * H; e += T) {
            const float *src = far_of(j.a + e / H, j.a) + H * DP + e % H;
            far_f[e] = __ldcg(src);
            far_l[e] = __ldcg(src + H);
        }
        __syncthreads();
        // a warp for each head: the maximum, the weights, the sum
        for (int h = warp; h < H; h += W) {
            float jm = -FLT_MAX, jl = 0.f;
            for (int c = lane; c < nc; c += 32) jm = fmaxf(jm, far_f[c * H + h]);
            for (int o = 16; o; o >>= 1) jm = fmaxf(jm, __shfl_xor_sync(~0u, jm, o));
            for (int c = lane; c < nc; c += 32) {
                const float f = exp2_(far_f[c * H + h] - jm);
                far_f[c * H + h] = f;
                jl += f * far_l[c * H + h];
            }
            for (int o = 16; o; o >>= 1) jl += __shfl_xor_sync(~0u, jl, o);
            if (lane == 0) joint_of[h] = make_float2(jm, jl);
        }
        __syncthreads();
        const int grp = G > 1 ? threadIdx.x / E4 : 0;
#pragma unroll 1
        for (int e = G > 1 ? threadIdx.x % E4 : threadIdx.x; e < E4; e += G > 1 ? E4 : T) {
            const int h = 4 * e / D, d = 4 * e % D;
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
            if (grp < G) {
#pragma unroll 4
                for (int c = grp; c < nc; c += G) {
                    const float4 v = __ldcg(reinterpret_cast<const float4 *>(far_of(j.a + c, j.a) + h * DP + d));
                    const float f = far_f[c * H + h];
                    o.x += f * v.x, o.y += f * v.y, o.z += f * v.z, o.w += f * v.w;
                }
                far_o[grp * E4 + e] = o;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int e = threadIdx.x; e < E4; e += T) {
            float4 jo = far_o[e];
#pragma unroll
            for (int k = 1; k < G; ++k) {
                const float4 v = far_o[k * E4 + e];
                jo.x += v.x, jo.y += v.y, jo.z += v.z, jo.w += v.w;
            }
            const float2 ml = joint_of[4 * e / D];
            finish(j, 4 * e / D, 4 * e % D, ml.x, ml.y, jo);
        }
        __syncthreads();
    }
}

// Query heads that share a cached head are taken 4, 8 or 16 at a time.
int tiles_of(int group) { return group <= 4 ? 1 : group <= 8 ? 2 : 4; }

template <int FMT, int D, int NB, bool WIDE>
cudaError_t launch(const AttnParams &p, cudaStream_t st, bool set)
{
    using C = Cfg<FMT, D, NB, WIDE>;
    if (set) return cudaFuncSetAttribute(k_paged<FMT, D, NB, WIDE>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
    const int blocks = (p.group + C::kHeads - 1) / C::kHeads;
    return launch_close(k_paged<FMT, D, NB, WIDE>, dim3(p.n_sm), 32 * C::kWarps, C::kSmem, st, 1, p, p.kv_heads * blocks, blocks);
}

template <int FMT, int D, bool WIDE>
cudaError_t by_group(const AttnParams &p, cudaStream_t st, bool set)
{
    switch (tiles_of(p.group)) {
    case 1: return launch<FMT, D, 1, WIDE>(p, st, set);
    case 2: return launch<FMT, D, 2, WIDE>(p, st, set);
    default: return launch<FMT, D, 4, WIDE>(p, st, set);
    }
}

template <int FMT, int D>
cudaError_t by_bits(const AttnParams &p, cudaStream_t st, bool set)
{
    return FMT == kBF16 && p.dt == kF32 ? by_group<FMT, D, FMT == kBF16>(p, st, set) : by_group<FMT, D, false>(p, st, set);
}

template <int FMT>
cudaError_t by_dim(const AttnParams &p, cudaStream_t st, bool set)
{
    return p.dim == 128 ? by_bits<FMT, 128>(p, st, set) : by_bits<FMT, 64>(p, st, set);
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

int attn_blocks(int group) { return (group + 4 * tiles_of(group) - 1) / (4 * tiles_of(group)); }

// 2 partial results for each CTA, then one for each of its warps (16 at most)
size_t attn_part_bytes(int n_sm, int group)
{
    const int nb = tiles_of(group);
    return size_t(n_sm) * 18 * (nb == 1 ? Cfg<kF16, 128, 1>::kPart : nb == 2 ? Cfg<kF16, 128, 2>::kPart : Cfg<kF16, 128, 4>::kPart);
}
size_t attn_ticket_bytes(int n_sm) { return size_t(n_sm) * sizeof(unsigned); }

cudaError_t attn_setup()
{
    AttnParams p{};
    for (int fmt : {int(kF16), int(kBF16), int(kI8), int(kI4)})
        for (int dim : {64, 128})
            for (int group : {4, 8, 16})
                for (int dt : {int(kF16), int(kF32)}) {
                    if (dt == kF32 && fmt != kBF16) continue;   // (other formats have one kernel for all callers)
                    p.c.fmt = fmt;
                    p.dim = dim;
                    p.group = group;
                    p.dt = dt;
                    const cudaError_t e = dispatch(p, nullptr, true);
                    if (e != cudaSuccess) return e;
                }
    return cudaSuccess;
}

cudaError_t paged_attention(const AttnParams &p, cudaStream_t st) { return dispatch(p, st, false); }

}  // namespace pi
