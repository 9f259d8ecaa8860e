// pi_paged.cu -- attention of one new token per sequence over a paged cache.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "pi_attn.h"

namespace pi {
namespace {

constexpr int kWarps = 8;

__device__ __forceinline__ float elem(const CacheView &c, const uint8_t *codes, const uint8_t *scales, long long row, int D,
                                      int at)
{
    const long long i = row * D + at;
    if (c.fmt == kF16) return __half2float(reinterpret_cast<const __half *>(codes)[i]);
    if (c.fmt == kBF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(codes)[i]);
    if (c.fmt == kI8) return reinterpret_cast<const float *>(scales)[row] * float(reinterpret_cast<const int8_t *>(codes)[i]);
    return __half2float(reinterpret_cast<const __half *>(scales)[i / 32]) *
           float(int((codes[i / 2] >> (4 * (i & 1))) & 15) - 8);
}

__device__ __forceinline__ float input(const uint8_t *p, long long i, int dt)
{
    if (dt == kF32) return reinterpret_cast<const float *>(p)[i];
    if (dt == kF16) return __half2float(reinterpret_cast<const __half *>(p)[i]);
    return __bfloat162float(reinterpret_cast<const __nv_bfloat16 *>(p)[i]);
}

__device__ __forceinline__ void output(uint8_t *p, long long i, int dt, float v)
{
    if (dt == kF32) reinterpret_cast<float *>(p)[i] = v;
    else if (dt == kF16) reinterpret_cast<__half *>(p)[i] = __float2half(v);
    else reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16(v);
}

// One CTA per query head and sequence; warp w takes positions w, w + 8, ...
// with a running maximum and sum, lane l elements l, l + 32, ...
template <int E>
__global__ void __launch_bounds__(32 * kWarps) k_attend(AttnParams p)
{
    constexpr int D = 32 * E;
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    const int h = blockIdx.x, s = blockIdx.y, warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    int len = p.len[s];
    const long long room = (long long)p.c.width * p.c.page_size;
    if (len < 0 || len > room) {
        if (threadIdx.x == 0) atomicExch(p.err, int(kDevCheck));
        len = len < 0 ? 0 : int(room);
    }
    const int first = p.window && len > p.window ? len - p.window : 0;
    float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) q[e] = input(p.q, s * p.qs + (long long)h * D + e * 32 + lane, p.dt);
    for (int j = first + warp; j < len; j += kWarps) {
        const int page = p.c.table[s * p.c.tstride + (j >> p.c.page_shift)];
        if (page < 0 || page >= p.c.n_pages) {
            if (lane == 0) atomicExch(p.err, int(kDevCheck));
            continue;
        }
        const long long row = (long long)page * p.c.page_rows + (long long)(j & (p.c.page_size - 1)) * p.c.slot_rows +
                              (long long)(h / p.group) * p.c.head_rows;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x += q[e] * elem(p.c, p.c.k, p.c.ks, row, D, e * 32 + lane);
        for (int k = 16; k; k >>= 1) x += __shfl_xor_sync(~0u, x, k);
        x *= p.scale;
        if (p.softcap > 0.f) x = p.softcap * tanhf(x / p.softcap);
        const float top = fmaxf(m, x), base = top == -INFINITY ? 0.f : top;
        const float keep = __expf(m - base), w = __expf(x - base);   // a NaN score makes the sums NaN
        l = l * keep + w;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = o[e] * keep + w * elem(p.c, p.c.v, p.c.vs, row, D, e * 32 + lane);
        m = top;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][e * 32 + lane] = o[e];
    if (lane == 0) {
        sm[warp] = m;
        sl[warp] = l;
    }
    __syncthreads();
    float top = -INFINITY, total = 0.f, w[kWarps];
    for (int i = 0; i < kWarps; ++i) top = fmaxf(top, sm[i]);
    for (int i = 0; i < kWarps; ++i) {
        w[i] = expf(sm[i] - (top == -INFINITY ? 0.f : top));
        total += w[i] * sl[i];
    }
    for (int i = threadIdx.x; i < D; i += 32 * kWarps) {
        float v = 0.f;
        for (int k = 0; k < kWarps; ++k) v += w[k] * so[k][i];
        output(p.out, s * p.os + (long long)h * D + i, p.dt, total > 0.f || total != total ? v / total : 0.f);
    }
    if (p.lse && threadIdx.x == 0) p.lse[(long long)s * p.heads + h] = total == 0.f ? -INFINITY : top + logf(total);
}

}  // namespace

size_t attn_part_bytes(int) { return 256; }
size_t attn_ticket_bytes(int) { return 256; }
cudaError_t attn_setup() { return cudaSuccess; }

cudaError_t paged_attention(const AttnParams &p, cudaStream_t st)
{
    const dim3 grid(p.heads, p.c.n_seqs);
    if (p.dim == 128) k_attend<4><<<grid, 32 * kWarps, 0, st>>>(p);
    else k_attend<2><<<grid, 32 * kWarps, 0, st>>>(p);
    return cudaGetLastError();
}

}  // namespace pi
