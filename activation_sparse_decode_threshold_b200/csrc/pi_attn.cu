// pi_attn.cu -- host side of the attention half of a decode layer
// (include/pi_ffn.h): validates every call before enqueuing work, owns the
// packed INT4 matrices and the attention handles' scratch, and launches the
// kernels of pi_int4.cu, pi_kv.cu and pi_paged.cu.
#include <cmath>
#include <cstdarg>
#include <cstdio>
#include <new>

#include "../../include/pi_ffn.h"
#include "pi_attn.h"

namespace {

pi_status fail(pi_status st, const char *fmt, ...)
{
    char msg[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(msg, sizeof msg, fmt, ap);
    va_end(ap);
    pi::set_last_error(msg);
    return st;
}

pi_status cuda_fail(cudaError_t e, const char *what)
{
    return fail(e == cudaErrorMemoryAllocation ? PI_ERR_OOM : PI_ERR_CUDA, "%s: %s (%s)", what,
                cudaGetErrorName(e), cudaGetErrorString(e));
}

#define PI_CUDA(call, what)                                   \
    do {                                                      \
        cudaError_t e_ = (call);                              \
        if (e_ != cudaSuccess) return cuda_fail(e_, what);    \
    } while (0)

// The handle's device for the length of a call.
struct OnDevice {
    int before = -1;
    cudaError_t status;
    explicit OnDevice(int device)
    {
        status = cudaGetDevice(&before);
        if (status == cudaSuccess && before != device) status = cudaSetDevice(device);
        else if (status == cudaSuccess) before = -1;
    }
    ~OnDevice()
    {
        if (before >= 0) cudaSetDevice(before);
    }
};

bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool is_float(pi_dtype t) { return t == PI_F32 || t == PI_F16 || t == PI_BF16; }
int bytes_of(pi_dtype t) { return t == PI_F32 ? 4 : 2; }
int fmt_of(pi_dtype t)
{
    return t == PI_F32 ? pi::kF32 : t == PI_F16 ? pi::kF16 : t == PI_BF16 ? pi::kBF16 : t == PI_I8 ? pi::kI8 : pi::kI4;
}

// Whether any of `rows` rows of a shares a byte with any of b (rows `as`, `bs`
// elements apart).  Rows of one buffer, side by side at the same distance, do not.
bool overlap(const void *a, long long as, int alen, int ab, const void *b, long long bs, int blen, int bb, int rows)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    const long long sa = as * ab, sb = bs * bb, la = (long long)alen * ab, lb = (long long)blen * bb;
    const uintptr_t a1 = a0 + (rows - 1) * sa + la, b1 = b0 + (rows - 1) * sb + lb;
    if (!(a0 < b1 && b0 < a1)) return false;
    if (rows > 1 && sa == sb) {
        const long long d = b0 >= a0 ? (long long)((b0 - a0) % sa) : (sa - (long long)((a0 - b0) % sa)) % sa;
        if (d >= la && d + lb <= sa) return false;
    }
    return true;
}

// Whether two buffers of na and nb bytes share one.
bool meet(const void *a, long long na, const void *b, long long nb)
{
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + nb && b0 < a0 + na;
}

pi_status check_device(int device, int *n_sm)
{
    int ndev = 0;
    PI_CUDA(cudaGetDeviceCount(&ndev), "cudaGetDeviceCount");
    if (device < 0 || device >= ndev) return fail(PI_ERR_INVALID_ARG, "bad device %d", device);
    int major = 0;
    PI_CUDA(cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, device), "cudaDeviceGetAttribute");
    if (major != 10)
        return fail(PI_ERR_UNSUPPORTED, "device %d is sm_%dx; this library is built for sm_100a", device, major);
    PI_CUDA(cudaDeviceGetAttribute(n_sm, cudaDevAttrMultiProcessorCount, device), "cudaDeviceGetAttribute");
    return PI_OK;
}

constexpr long long kMaxStride = 1LL << 40;

// A token row's address and distance: 16-byte aligned, rows apart.  One token's
// distance is not used.
pi_status check_rows(const char *name, const void *p, long long &stride, int len, int bytes, int tokens)
{
    if (!aligned16(p)) return fail(PI_ERR_INVALID_ARG, "%s must be 16-byte aligned", name);
    if (tokens == 1) stride = len;
    if (stride < len || stride > kMaxStride)
        return fail(PI_ERR_INVALID_ARG, "%s: row distance %lld is below the row length %d (or above 2^40)", name, stride,
                    len);
    if (tokens > 1 && stride * bytes % 16 != 0)
        return fail(PI_ERR_INVALID_ARG, "%s: row distance must be a multiple of 16 bytes", name);
    return PI_OK;
}

}  // namespace

struct pi_int4 {
    int n = 0, k = 0, ku = 0, device = 0, n_sm = 0, clusters[3] = {0, 0, 0};
    uint8_t *w = nullptr;
};

struct pi_attn {
    pi_attn_desc desc{};
    int n_sm = 0;
    uint8_t *scratch = nullptr;
    double *freq = nullptr;
    float *part = nullptr;
    unsigned *tickets = nullptr;
    int *err = nullptr;
};

extern "C" {

pi_status pi_int4_create(int n_rows, int n_cols, const void *q_dev, const void *s_dev, int device, void *stream,
                         pi_int4_t *out)
{
    if (!out) return fail(PI_ERR_INVALID_ARG, "pi_int4_create: null argument");
    *out = nullptr;
    if (!q_dev || !s_dev) return fail(PI_ERR_INVALID_ARG, "pi_int4_create: null argument");
    if (n_rows < 1 || n_rows > (1 << 20)) return fail(PI_ERR_INVALID_ARG, "n_rows must be in [1, 2^20]");
    if (n_cols < 32 || n_cols % 32 != 0 || n_cols > (1 << 17))
        return fail(PI_ERR_INVALID_ARG, "n_cols must be a multiple of 32 in [32, 2^17]");
    if (!aligned16(q_dev)) return fail(PI_ERR_INVALID_ARG, "q_dev must be 16-byte aligned");
    if (reinterpret_cast<uintptr_t>(s_dev) & 1u) return fail(PI_ERR_INVALID_ARG, "s_dev must be 2-byte aligned");
    int n_sm = 0;
    const pi_status st = check_device(device, &n_sm);
    if (st != PI_OK) return st;
    OnDevice on(device);
    PI_CUDA(on.status, "cudaSetDevice");
    pi_int4 *m = new (std::nothrow) pi_int4;
    if (!m) return fail(PI_ERR_OOM, "host allocation failed");
    m->n = n_rows;
    m->k = n_cols;
    m->ku = (n_cols + 63) / 64;
    m->device = device;
    m->n_sm = n_sm;
    const size_t bytes = size_t((n_rows + 15) / 16) * m->ku * pi::kInt4Unit;
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    cudaError_t e = pi::int4_setup();
    if (e == cudaSuccess) e = pi::int4_clusters(m->clusters);
    if (e == cudaSuccess) e = cudaMalloc(&m->w, bytes);
    if (e == cudaSuccess)
        e = pi::int4_pack(static_cast<const uint8_t *>(q_dev), static_cast<const uint16_t *>(s_dev), m->w, n_rows, n_cols,
                          cs);
    if (e == cudaSuccess) e = cudaStreamSynchronize(cs);
    if (e != cudaSuccess) {
        const pi_status bad = cuda_fail(e, "pi_int4_create");
        pi_int4_destroy(m);
        return bad;
    }
    *out = m;
    return PI_OK;
}

void pi_int4_destroy(pi_int4_t m)
{
    if (!m) return;
    OnDevice on(m->device);
    cudaFree(m->w);
    delete m;
}

pi_status pi_int4_matvec(pi_int4_t m, int n_tokens, pi_dtype x_dtype, const void *x_dev, int64_t x_stride,
                         const void *add_dev, pi_dtype y_dtype, void *y_dev, int64_t y_stride, float norm_eps, void *stream)
{
    if (!m || !x_dev || !y_dev) return fail(PI_ERR_INVALID_ARG, "pi_int4_matvec: null argument");
    if (n_tokens < 1 || n_tokens > pi::kInt4MaxTokens)
        return fail(PI_ERR_INVALID_ARG, "n_tokens must be in [1, %d]", pi::kInt4MaxTokens);
    if (!is_float(x_dtype) || !is_float(y_dtype))
        return fail(PI_ERR_INVALID_ARG, "x_dtype and y_dtype must be F32, F16 or BF16");
    if (!(norm_eps >= 0.f) || !std::isfinite(norm_eps)) return fail(PI_ERR_INVALID_ARG, "norm_eps must be >= 0");
    long long xs = x_stride, ys = n_tokens == 1 ? m->n : y_stride;
    const pi_status st = check_rows("x", x_dev, xs, m->k, bytes_of(x_dtype), n_tokens);
    if (st != PI_OK) return st;
    if (ys < m->n || ys > kMaxStride)
        return fail(PI_ERR_INVALID_ARG, "y: row distance %lld is below the row length %d (or above 2^40)", ys, m->n);
    const int yb = bytes_of(y_dtype);
    if ((reinterpret_cast<uintptr_t>(y_dev) | reinterpret_cast<uintptr_t>(add_dev)) & (yb - 1))
        return fail(PI_ERR_INVALID_ARG, "y and add must be aligned to their elements");
    if (overlap(x_dev, xs, m->k, bytes_of(x_dtype), y_dev, ys, m->n, yb, n_tokens))
        return fail(PI_ERR_INVALID_ARG, "x and y overlap");
    if (add_dev && add_dev != y_dev && overlap(add_dev, ys, m->n, yb, y_dev, ys, m->n, yb, n_tokens))
        return fail(PI_ERR_INVALID_ARG, "add and y overlap without being the same rows");
    OnDevice on(m->device);
    PI_CUDA(on.status, "cudaSetDevice");
    pi::Int4Params p{};
    p.w = m->w;
    p.n = m->n;
    p.k = m->k;
    p.ku = m->ku;
    p.tokens = n_tokens;
    p.xt = fmt_of(x_dtype);
    p.yt = fmt_of(y_dtype);
    p.x = static_cast<const uint8_t *>(x_dev);
    p.add = static_cast<const uint8_t *>(add_dev);
    p.y = static_cast<uint8_t *>(y_dev);
    p.xs = xs;
    p.ys = ys;
    p.eps = norm_eps;
    p.n_sm = m->n_sm;
    for (int i = 0; i < 3; ++i) p.clusters[i] = m->clusters[i];
    PI_CUDA(pi::int4_matvec(p, static_cast<cudaStream_t>(stream)), "pi_int4_matvec");
    return PI_OK;
}

pi_status pi_attn_create(const pi_attn_desc *desc, pi_attn_t *out)
{
    if (!desc || !out) return fail(PI_ERR_INVALID_ARG, "pi_attn_create: null argument");
    *out = nullptr;
    const pi_attn_desc &D = *desc;
    if (D.n_kv_heads < 1 || D.n_heads < 1 || D.n_heads > 1024 || D.n_heads % D.n_kv_heads != 0)
        return fail(PI_ERR_INVALID_ARG, "n_heads must be a multiple of n_kv_heads in [1, 1024]");
    if (D.head_dim != 64 && D.head_dim != 128) return fail(PI_ERR_UNSUPPORTED, "head_dim must be 64 or 128");
    if (D.cache_dtype != PI_F16 && D.cache_dtype != PI_BF16 && D.cache_dtype != PI_I8 && D.cache_dtype != PI_INT4G32)
        return fail(PI_ERR_UNSUPPORTED, "cache_dtype must be F16, BF16, I8 or INT4G32");
    if (D.page_size < 8 || D.page_size > 256 || (D.page_size & (D.page_size - 1)))
        return fail(PI_ERR_UNSUPPORTED, "page_size must be a power of two in [8, 256]");
    if (D.layout != PI_KV_HND && D.layout != PI_KV_NHD) return fail(PI_ERR_INVALID_ARG, "bad layout");
    if (D.rotary_dim < 0 || D.rotary_dim > D.head_dim || D.rotary_dim % 2 != 0)
        return fail(PI_ERR_INVALID_ARG, "rotary_dim must be even and in [0, head_dim]");
    if (D.rotary_pairs != 0 && D.rotary_pairs != 1) return fail(PI_ERR_INVALID_ARG, "rotary_pairs must be 0 or 1");
    if (D.rotary_dim > 0 && !(D.rope_theta > 0.f && std::isfinite(D.rope_theta)))
        return fail(PI_ERR_INVALID_ARG, "rope_theta must be > 0");
    if (!(D.norm_eps >= 0.f) || !std::isfinite(D.norm_eps)) return fail(PI_ERR_INVALID_ARG, "norm_eps must be >= 0");
    if (!std::isfinite(D.scale)) return fail(PI_ERR_INVALID_ARG, "scale must be finite");
    if (!(D.softcap == 0.f || (D.softcap >= 1e-6f && D.softcap <= 1e6f)))
        return fail(PI_ERR_INVALID_ARG, "softcap must be 0 or in [1e-6, 1e6]");
    if (D.window < 0) return fail(PI_ERR_INVALID_ARG, "window must be >= 0");
    int n_sm = 0;
    const pi_status st = check_device(D.device, &n_sm);
    if (st != PI_OK) return st;
    OnDevice on(D.device);
    PI_CUDA(on.status, "cudaSetDevice");
    pi_attn *a = new (std::nothrow) pi_attn;
    if (!a) return fail(PI_ERR_OOM, "host allocation failed");
    a->desc = D;
    if (D.scale == 0.f) a->desc.scale = 1.f / std::sqrt(float(D.head_dim));
    a->n_sm = n_sm;
    // scratch: freq [64] | err | tickets | partial sums
    double freq[64] = {0};
    for (int i = 0; i < D.rotary_dim / 2; ++i) freq[i] = std::pow(double(D.rope_theta), -2.0 * i / D.rotary_dim);
    const size_t o_err = sizeof freq, o_tick = o_err + 256;
    const size_t o_part = (o_tick + pi::attn_ticket_bytes(n_sm) + 255) & ~size_t(255);
    const size_t total = o_part + pi::attn_part_bytes(n_sm, D.n_heads / D.n_kv_heads);
    cudaError_t e = pi::attn_setup();
    if (e == cudaSuccess) e = cudaMalloc(&a->scratch, total);
    if (e == cudaSuccess) e = cudaMemset(a->scratch, 0, total);
    if (e == cudaSuccess) e = cudaMemcpy(a->scratch, freq, sizeof freq, cudaMemcpyHostToDevice);
    // (the fill runs on the default stream; a caller's first call may be on another)
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    if (e != cudaSuccess) {
        const pi_status bad = cuda_fail(e, "pi_attn_create");
        pi_attn_destroy(a);
        return bad;
    }
    a->freq = reinterpret_cast<double *>(a->scratch);
    a->err = reinterpret_cast<int *>(a->scratch + o_err);
    a->tickets = reinterpret_cast<unsigned *>(a->scratch + o_tick);
    a->part = reinterpret_cast<float *>(a->scratch + o_part);
    *out = a;
    return PI_OK;
}

void pi_attn_destroy(pi_attn_t a)
{
    if (!a) return;
    OnDevice on(a->desc.device);
    cudaFree(a->scratch);
    delete a;
}

pi_status pi_attn_sync(pi_attn_t a, void *stream)
{
    if (!a) return fail(PI_ERR_INVALID_ARG, "null handle");
    OnDevice on(a->desc.device);
    PI_CUDA(on.status, "cudaSetDevice");
    cudaStream_t cs = static_cast<cudaStream_t>(stream);
    int err = 0;
    PI_CUDA(cudaMemcpyAsync(&err, a->err, sizeof err, cudaMemcpyDeviceToHost, cs), "read error word");
    PI_CUDA(cudaStreamSynchronize(cs), "stream sync");
    if (err == pi::kDevOk) return PI_OK;
    PI_CUDA(cudaMemsetAsync(a->err, 0, sizeof err, cs), "clear error word");
    PI_CUDA(cudaStreamSynchronize(cs), "stream sync");
    return fail(PI_ERR_DEVICE_CHECK, "a sequence, position, length or page was out of range");
}

// Checks of the cache and its page table; fills the view.
static pi_status cache_view(pi_attn_t a, const pi_kv_cache *cache, const pi_kv_table *table, pi::CacheView &c)
{
    const pi_attn_desc &D = a->desc;
    if (!cache->k || !cache->v || !table->pages) return fail(PI_ERR_INVALID_ARG, "null cache or page table");
    const bool scaled = D.cache_dtype == PI_I8 || D.cache_dtype == PI_INT4G32;
    if (scaled != (cache->k_scale != nullptr) || scaled != (cache->v_scale != nullptr))
        return fail(PI_ERR_INVALID_ARG, "I8 and INT4G32 caches have k_scale and v_scale, others have none");
    if (!aligned16(cache->k) || !aligned16(cache->v) || !aligned16(cache->k_scale) || !aligned16(cache->v_scale))
        return fail(PI_ERR_INVALID_ARG, "cache pointers must be 16-byte aligned");
    if (cache->n_pages < 1) return fail(PI_ERR_INVALID_ARG, "n_pages must be >= 1");
    if (reinterpret_cast<uintptr_t>(table->pages) & 3u) return fail(PI_ERR_INVALID_ARG, "page table must be 4-byte aligned");
    if (table->n_seqs < 1 || table->n_seqs > 65536) return fail(PI_ERR_INVALID_ARG, "n_seqs must be in [1, 65536]");
    if (table->width < 1 || (long long)table->width * D.page_size > (1LL << 30))
        return fail(PI_ERR_INVALID_ARG, "width must be >= 1 and width * page_size at most 2^30");
    if (table->n_seqs > 1 && (table->stride < table->width || table->stride > kMaxStride))
        return fail(PI_ERR_INVALID_ARG, "page table: row distance below width (or above 2^40)");
    c.k = static_cast<uint8_t *>(cache->k);
    c.v = static_cast<uint8_t *>(cache->v);
    c.ks = static_cast<uint8_t *>(cache->k_scale);
    c.vs = static_cast<uint8_t *>(cache->v_scale);
    c.fmt = fmt_of(D.cache_dtype);
    c.n_pages = cache->n_pages;
    c.page_size = D.page_size;
    c.page_shift = 0;
    while ((1 << c.page_shift) < D.page_size) ++c.page_shift;
    c.page_rows = D.page_size * D.n_kv_heads;
    c.head_rows = D.layout == PI_KV_HND ? D.page_size : 1;
    c.slot_rows = D.layout == PI_KV_HND ? 1 : D.n_kv_heads;
    c.table = table->pages;
    c.n_seqs = table->n_seqs;
    c.width = table->width;
    c.tstride = table->stride;
    return PI_OK;
}

static pi_status check_tokens(const pi_kv_table *table, int n_tokens, const int32_t *seq, const int32_t *pos)
{
    if (n_tokens < 1 || n_tokens > (1 << 20)) return fail(PI_ERR_INVALID_ARG, "n_tokens must be in [1, 2^20]");
    if (!seq && n_tokens > table->n_seqs)
        return fail(PI_ERR_INVALID_ARG, "without seq_dev, n_tokens must not exceed n_seqs");
    if ((reinterpret_cast<uintptr_t>(seq) | reinterpret_cast<uintptr_t>(pos)) & 3u)
        return fail(PI_ERR_INVALID_ARG, "seq and pos must be 4-byte aligned");
    return PI_OK;
}

pi_status pi_kv_append(pi_attn_t a, const pi_kv_cache *cache, const pi_kv_table *table, int n_tokens,
                       const int32_t *seq_dev, const int32_t *pos_dev, pi_dtype dtype, const void *q_dev,
                       int64_t q_stride, const void *k_dev, int64_t k_stride, const void *v_dev, int64_t v_stride,
                       const float *q_norm_dev, const float *k_norm_dev, void *q_out_dev, int64_t q_out_stride,
                       void *stream)
{
    if (!a || !cache || !table || !pos_dev || !q_dev || !k_dev || !v_dev || !q_out_dev)
        return fail(PI_ERR_INVALID_ARG, "pi_kv_append: null argument");
    const pi_attn_desc &D = a->desc;
    if (!is_float(dtype)) return fail(PI_ERR_INVALID_ARG, "dtype must be F32, F16 or BF16");
    pi::AppendParams p{};
    pi_status st = cache_view(a, cache, table, p.c);
    if (st == PI_OK) st = check_tokens(table, n_tokens, seq_dev, pos_dev);
    const int b = bytes_of(dtype), qlen = D.n_heads * D.head_dim, klen = D.n_kv_heads * D.head_dim;
    p.qs = q_stride;
    p.kstr = k_stride;
    p.vstr = v_stride;
    p.os = q_out_stride;
    if (st == PI_OK) st = check_rows("q", q_dev, p.qs, qlen, b, n_tokens);
    if (st == PI_OK) st = check_rows("k", k_dev, p.kstr, klen, b, n_tokens);
    if (st == PI_OK) st = check_rows("v", v_dev, p.vstr, klen, b, n_tokens);
    if (st == PI_OK) st = check_rows("q_out", q_out_dev, p.os, qlen, b, n_tokens);
    if (st != PI_OK) return st;
    if (q_out_dev == q_dev ? p.os != p.qs : overlap(q_dev, p.qs, qlen, b, q_out_dev, p.os, qlen, b, n_tokens))
        return fail(PI_ERR_INVALID_ARG, "q and q_out overlap without being the same rows");
    if (overlap(k_dev, p.kstr, klen, b, q_out_dev, p.os, qlen, b, n_tokens) ||
        overlap(v_dev, p.vstr, klen, b, q_out_dev, p.os, qlen, b, n_tokens))
        return fail(PI_ERR_INVALID_ARG, "q_out overlaps k or v");
    if ((q_norm_dev || k_norm_dev) && D.norm_eps == 0.f)
        return fail(PI_ERR_INVALID_ARG, "norm weights without norm_eps");
    if ((reinterpret_cast<uintptr_t>(q_norm_dev) | reinterpret_cast<uintptr_t>(k_norm_dev)) & 3u)
        return fail(PI_ERR_INVALID_ARG, "norm weights must be 4-byte aligned");
    OnDevice on(D.device);
    PI_CUDA(on.status, "cudaSetDevice");
    p.heads = D.n_heads;
    p.kv_heads = D.n_kv_heads;
    p.dim = D.head_dim;
    p.rotary = D.rotary_dim;
    p.pairs = D.rotary_pairs;
    p.eps = D.norm_eps;
    p.tokens = n_tokens;
    p.dt = fmt_of(dtype);
    p.seq = seq_dev;
    p.pos = pos_dev;
    p.q = static_cast<const uint8_t *>(q_dev);
    p.k = static_cast<const uint8_t *>(k_dev);
    p.v = static_cast<const uint8_t *>(v_dev);
    p.q_out = static_cast<uint8_t *>(q_out_dev);
    p.qn = q_norm_dev;
    p.kn = k_norm_dev;
    p.freq = a->freq;
    p.err = a->err;
    p.n_sm = a->n_sm;
    PI_CUDA(pi::kv_append(p, static_cast<cudaStream_t>(stream)), "pi_kv_append");
    return PI_OK;
}

pi_status pi_kv_read(pi_attn_t a, const pi_kv_cache *cache, const pi_kv_table *table, int n_tokens,
                     const int32_t *seq_dev, const int32_t *pos_dev, pi_dtype dtype, void *k_dev, void *v_dev,
                     void *stream)
{
    if (!a || !cache || !table || !pos_dev || !k_dev || !v_dev)
        return fail(PI_ERR_INVALID_ARG, "pi_kv_read: null argument");
    if (!is_float(dtype)) return fail(PI_ERR_INVALID_ARG, "dtype must be F32, F16 or BF16");
    pi::ReadParams p{};
    pi_status st = cache_view(a, cache, table, p.c);
    if (st == PI_OK) st = check_tokens(table, n_tokens, seq_dev, pos_dev);
    if (st != PI_OK) return st;
    if (!aligned16(k_dev) || !aligned16(v_dev)) return fail(PI_ERR_INVALID_ARG, "k and v must be 16-byte aligned");
    const pi_attn_desc &D = a->desc;
    const long long bytes = (long long)n_tokens * D.n_kv_heads * D.head_dim * bytes_of(dtype), rows = (long long)cache->n_pages * p.c.page_rows;
    if (meet(k_dev, bytes, v_dev, bytes)) return fail(PI_ERR_INVALID_ARG, "k and v overlap");
    const long long row = D.cache_dtype == PI_I8 ? D.head_dim : D.cache_dtype == PI_INT4G32 ? D.head_dim / 2 : 2 * D.head_dim;
    const long long scale = D.cache_dtype == PI_I8 ? 4 : D.cache_dtype == PI_INT4G32 ? D.head_dim / 16 : 0;
    for (const void *out : {k_dev, v_dev})
        if (meet(out, bytes, cache->k, rows * row) || meet(out, bytes, cache->v, rows * row) ||
            (scale && (meet(out, bytes, cache->k_scale, rows * scale) || meet(out, bytes, cache->v_scale, rows * scale))))
            return fail(PI_ERR_INVALID_ARG, "k or v overlaps the cache");
    OnDevice on(D.device);
    PI_CUDA(on.status, "cudaSetDevice");
    p.kv_heads = D.n_kv_heads;
    p.dim = D.head_dim;
    p.tokens = n_tokens;
    p.dt = fmt_of(dtype);
    p.seq = seq_dev;
    p.pos = pos_dev;
    p.k = static_cast<uint8_t *>(k_dev);
    p.v = static_cast<uint8_t *>(v_dev);
    p.err = a->err;
    p.n_sm = a->n_sm;
    PI_CUDA(pi::kv_read(p, static_cast<cudaStream_t>(stream)), "pi_kv_read");
    return PI_OK;
}

pi_status pi_paged_attention(pi_attn_t a, const pi_kv_cache *cache, const pi_kv_table *table, const int32_t *len_dev,
                             pi_dtype dtype, const void *q_dev, int64_t q_stride, void *out_dev, int64_t out_stride,
                             float *lse_dev, void *stream)
{
    if (!a || !cache || !table || !len_dev || !q_dev || !out_dev)
        return fail(PI_ERR_INVALID_ARG, "pi_paged_attention: null argument");
    if (!is_float(dtype)) return fail(PI_ERR_INVALID_ARG, "dtype must be F32, F16 or BF16");
    const pi_attn_desc &D = a->desc;
    pi::AttnParams p{};
    pi_status st = cache_view(a, cache, table, p.c);
    if (st != PI_OK) return st;
    const int b = bytes_of(dtype), qlen = D.n_heads * D.head_dim, n = table->n_seqs;
    if ((long long)n * ((long long)table->width * D.page_size / 16 + 3) * D.n_kv_heads * pi::attn_blocks(D.n_heads / D.n_kv_heads) >
        (1LL << 30))
        return fail(PI_ERR_INVALID_ARG, "page table: n_seqs * width * page_size * n_kv_heads is above 2^34 (2^30 tiles of work)");
    p.qs = q_stride;
    p.os = out_stride;
    st = check_rows("q", q_dev, p.qs, qlen, b, n);
    if (st == PI_OK) st = check_rows("out", out_dev, p.os, qlen, b, n);
    if (st != PI_OK) return st;
    if (overlap(q_dev, p.qs, qlen, b, out_dev, p.os, qlen, b, n)) return fail(PI_ERR_INVALID_ARG, "q and out overlap");
    if ((reinterpret_cast<uintptr_t>(len_dev) | reinterpret_cast<uintptr_t>(lse_dev)) & 3u)
        return fail(PI_ERR_INVALID_ARG, "len and lse must be 4-byte aligned");
    OnDevice on(D.device);
    PI_CUDA(on.status, "cudaSetDevice");
    p.heads = D.n_heads;
    p.kv_heads = D.n_kv_heads;
    p.group = D.n_heads / D.n_kv_heads;
    p.dim = D.head_dim;
    p.dt = fmt_of(dtype);
    p.scale = D.scale;
    p.softcap = D.softcap;
    p.window = D.window;
    p.len = len_dev;
    p.q = static_cast<const uint8_t *>(q_dev);
    p.out = static_cast<uint8_t *>(out_dev);
    p.lse = lse_dev;
    p.part = a->part;
    p.tickets = a->tickets;
    p.err = a->err;
    p.n_sm = a->n_sm;
    PI_CUDA(pi::paged_attention(p, static_cast<cudaStream_t>(stream)), "pi_paged_attention");
    return PI_OK;
}

}  // extern "C"
