// pi_attn.h -- parameters shared by the host side (pi_attn.cu) and the kernels
// of the attention half of a decode layer.  Not part of the public interface.
#pragma once
#include <cstdint>
#include <cuda_runtime.h>

#include "pi_internal.h"

namespace pi {

#ifdef __CUDACC__
// The kernels of a layer follow each other closely: each is launched so that its
// CTAs may start while the kernel before it on the stream ends, allows the same
// to its own successor, and touches memory only after all before it is complete
// and visible (worth 1.3 us of a product of 1024x4096 with one token among others).
// allow_next() is for kernels whose CTAs all run at once: where
// they come in turns, waiting successors would take their places (8 x 4096 rows read:
// 39.8 us with it, 35.2 without).
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void allow_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
template <typename... P, typename... A>
cudaError_t launch_close(void (*kernel)(P...), dim3 grid, int threads, size_t smem, cudaStream_t st, int cluster, A... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, P(args)...);
}
#endif

constexpr int kInt4MaxTokens = 32;
// Packed INT4 matrix: units of 16 rows x 64 columns, unit (row tile, k) at
// (tile * units_per_row + k) * kInt4Unit.
constexpr int kInt4Unit = 512 + 64;   // nibbles, then 2 x 2 scales for each row pair

struct Int4Params {
    const uint8_t *w;
    int n, k;               // rows, columns
    int ku;                 // units along the columns
    int tokens;
    int xt, yt;             // Fmt of x, of y and add
    const uint8_t *x, *add;
    uint8_t *y;
    long long xs, ys;       // elements between tokens
    float eps;              // 0: no norm
    int n_sm, clusters[3];  // SMs; clusters of 2, 4, 8 CTAs that run at once
};
cudaError_t int4_clusters(int (&clusters)[3]);
cudaError_t int4_pack(const uint8_t *q, const uint16_t *s, uint8_t *dst, int n, int k, cudaStream_t st);
cudaError_t int4_setup();   // once per device, before any launch
cudaError_t int4_matvec(const Int4Params &p, cudaStream_t st);

// Rows of a cache.  A row number is page * page_rows + slot * slot_rows + head * head_rows.
struct CacheView {
    uint8_t *k, *v, *ks, *vs;
    int fmt;                // kF16, kBF16, kI8, kI4
    int n_pages, page_shift, page_size;
    int head_rows, slot_rows, page_rows;
    const int32_t *table;
    int n_seqs, width;
    long long tstride;
};

struct AppendParams {
    CacheView c;
    int heads, kv_heads, dim, rotary, pairs;
    float eps;
    int tokens, dt;
    const int32_t *seq, *pos;
    const uint8_t *q, *k, *v;
    uint8_t *q_out;
    long long qs, kstr, vstr, os;
    const float *qn, *kn;
    const double *freq;     // rotary / 2 angles per position
    int *err;
    int n_sm;
};
cudaError_t kv_append(const AppendParams &p, cudaStream_t st);

struct ReadParams {
    CacheView c;
    int kv_heads, dim, tokens, dt;
    const int32_t *seq, *pos;
    uint8_t *k, *v;
    int *err;
    int n_sm;
};
cudaError_t kv_read(const ReadParams &p, cudaStream_t st);

struct AttnParams {
    CacheView c;
    int heads, kv_heads, group, dim, dt;
    float scale, softcap;
    int window;
    const int32_t *len;
    const uint8_t *q;
    uint8_t *out;
    float *lse;
    long long qs, os;
    float *part;            // partial sums of sequences shared by CTAs
    unsigned *tickets;      // zero between calls
    int *err;
    int n_sm;
};
int attn_blocks(int group);   // blocks of query heads that share a cached head
size_t attn_part_bytes(int n_sm, int group);
size_t attn_ticket_bytes(int n_sm);
cudaError_t attn_setup();   // once per device, before any launch
cudaError_t paged_attention(const AttnParams &p, cudaStream_t st);

}  // namespace pi
