// kivi_paged_api.cu -- the C ABI of the paged cache (include/kivi.h): argument
// checks and launches.  The state of the sequences lives on the device, so the
// host checks what it is handed and the kernels check the rest.
#include <algorithm>
#include <climits>
#include <cmath>
#include <cstring>

#include <nvtx3/nvToolsExt.h>

#include "kivi_paged.cuh"

using namespace kivi;

namespace {

struct NvtxRange {
    explicit NvtxRange(const char *name) { nvtxRangePushA(name); }
    ~NvtxRange() { nvtxRangePop(); }
    NvtxRange(const NvtxRange &) = delete;
    NvtxRange &operator=(const NvtxRange &) = delete;
};

bool aligned(const void *p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1u)) == 0; }

int check_paged_params(const kivi_params *p)
{
    const int st = kivi_params_validate(p);
    if (st != KIVI_OK)
        return st;
    const int64_t pairs = (int64_t)p->batch * p->num_kv_heads;
    const int64_t columns = p->capacity_tokens / p->group;
    if (columns < 1 || p->capacity_tokens + p->sink_tokens + p->residual > INT_MAX - 4096 || columns * pairs > INT_MAX)
        return KIVI_ERR_UNSUPPORTED;
    return KIVI_OK;
}

int check_paged(const kivi_paged *c)
{
    if (!c)
        return KIVI_ERR_INVALID_ARG;
    const int st = check_paged_params(&c->p);
    if (st != KIVI_OK)
        return st;
    if (!c->pool || !c->k_fp16 || !c->v_fp16 || !c->table || !c->n_tokens || !c->n_evicted || !c->control ||
        !aligned(c->pool, 16) || !aligned(c->k_fp16, 16) || !aligned(c->v_fp16, 16) || !aligned(c->table, 4) ||
        !aligned(c->n_tokens, 4) || !aligned(c->n_evicted, 4) || !aligned(c->control, 4) || c->num_pages < 1 ||
        c->num_pages > INT_MAX)
        return KIVI_ERR_INVALID_ARG;
    return KIVI_OK;
}

PagedArgs paged_args(const kivi_params *p)
{
    PagedArgs a{};
    a.columns = (int)(p->capacity_tokens / p->group);
    a.rec_bytes = (int)kivi_history_record_bytes(p);
    a.bits = p->bits;
    a.fmt = p->fp8_format;
    a.meta = p->meta;
    a.G = p->group;
    a.flush_group = p->flush == KIVI_FLUSH_GROUP;
    a.R = p->residual;
    a.Ns = p->sink_tokens;
    a.rows = a.Ns + a.R;
    a.B = p->batch;
    a.Hkv = p->num_kv_heads;
    a.g = p->num_q_heads / p->num_kv_heads;
    a.fp8_k_scale = p->fp8_k_scale;
    a.fp8_v_scale = p->fp8_v_scale;
    return a;
}

PagedArgs paged_args(const kivi_paged *c)
{
    PagedArgs a = paged_args(&c->p);
    a.pool = static_cast<uint8_t *>(c->pool);
    a.k_fp16 = static_cast<__half *>(c->k_fp16);
    a.v_fp16 = static_cast<__half *>(c->v_fp16);
    a.table = c->table;
    a.n_tokens = c->n_tokens;
    a.n_evicted = c->n_evicted;
    a.control = c->control;
    a.num_pages = c->num_pages;
    return a;
}

constexpr float kLog2e = 1.4426950408889634f;

float softmax_scale(const kivi_paged *c, const kivi_chunk *x)
{
    return x->softmax_scale > 0.0f ? x->softmax_scale : 1.0f / std::sqrt((float)c->p.head_dim);
}

// What of a chunk a call reads.
enum Uses { kUseQ = 1, kUseK = 2, kUseV = 4, kNewOptional = 8 };

int check_chunk(const kivi_paged *c, const kivi_chunk *x, int uses)
{
    if (!x || x->reserved != 0 || !x->offsets || !aligned(x->offsets, 4) || x->num_tokens < 0 || x->max_new < 0 ||
        x->max_cached < 0 || (x->mask != KIVI_MASK_CAUSAL && x->mask != KIVI_MASK_FULL) ||
        std::isnan(x->softmax_scale) || std::isnan(x->softcap) || std::isinf(x->softmax_scale) ||
        std::isinf(x->softcap))
        return KIVI_ERR_INVALID_ARG;
    // scale and cap in log2 units, and their quotient, are fp32 numbers
    const float scale = softmax_scale(c, x);
    if (!std::isfinite(scale * kLog2e) || (x->softcap > 0.0f && (!std::isfinite(x->softcap * kLog2e) ||
                                                                 !std::isfinite(scale / x->softcap))))
        return KIVI_ERR_INVALID_ARG;
    if (x->num_tokens > INT_MAX / 2)
        return KIVI_ERR_UNSUPPORTED;
    // rows of query tiles are a grid dimension
    if ((int64_t)x->max_new * (c->p.num_q_heads / c->p.num_kv_heads) > (int64_t)65535 * 64)
        return KIVI_ERR_UNSUPPORTED;
    const int64_t d = c->p.head_dim;
    const bool some = x->max_new > 0 && x->num_tokens > 0;
    if ((uses & kUseQ) && some &&
        (!x->q || !aligned(x->q, 16) || x->q_stride % 8 != 0 || x->q_stride < c->p.num_q_heads * d))
        return KIVI_ERR_INVALID_ARG;
    const bool has_new = x->k != nullptr || ((uses & kUseV) && x->v != nullptr);
    if (some && (has_new || !(uses & kNewOptional))) {
        if (!x->k || !aligned(x->k, 16) || ((uses & kUseV) && (!x->v || !aligned(x->v, 16))) ||
            x->kv_stride % 8 != 0 || x->kv_stride < c->p.num_kv_heads * d)
            return KIVI_ERR_INVALID_ARG;
    }
    return KIVI_OK;
}

// The bound on cached tokens a call goes by: the caller's, or what the table holds.
int cached_bound(const PagedArgs &a, int max_cached)
{
    const int64_t most = (int64_t)a.columns * a.G + a.rows;
    return (int)(max_cached > 0 ? std::min<int64_t>(max_cached, most) : most);
}

ChunkArgs chunk_args(const kivi_paged *c, const kivi_chunk *x)
{
    ChunkArgs a{};
    a.q = static_cast<const __half *>(x->q);
    a.k = static_cast<const __half *>(x->k);
    a.v = static_cast<const __half *>(x->v);
    a.offsets = x->offsets;
    a.q_stride = x->q_stride;
    a.kv_stride = x->kv_stride;
    a.num_tokens = x->num_tokens;
    a.max_new = (int)std::min<int64_t>(x->max_new, x->num_tokens);
    a.max_cached = cached_bound(paged_args(&c->p), x->max_cached);
    const float scale = softmax_scale(c, x);
    a.scale_log2 = scale * kLog2e;
    // a cap above 2^64 scale changes no score that fp32 holds to 24 bits: |q.k| < 2^52, y = scale q.k / cap < 2^-12,
    // and tanh(y) = y (1 - y^2 / 3)
    if (x->softcap > 0.0f && scale / x->softcap >= 0x1p-64f) {
        a.cap_log2 = x->softcap * kLog2e;
        a.cap_inv = scale / x->softcap;
        a.cap_small = x->softcap < 64.0f;
    }
    a.full = x->mask == KIVI_MASK_FULL;
    a.v8 = aligned(x->k, 32) && aligned(x->v, 32) && x->kv_stride % 16 == 0 && aligned(c->k_fp16, 32) &&
           aligned(c->v_fp16, 32);
    return a;
}

size_t workspace_bytes(const PagedArgs &a, int max_new, int max_cached)
{
    size_t n = evict_bytes(a);
    if (max_new > 0) {
        const int most = cached_bound(a, max_cached);
        n = std::max(n, attention_bytes(a, max_new, most));
        n = std::max(n, weights_bytes(a, max_new, most));
    }
    return (n + 255) / 256 * 256;
}

int check_workspace(const PagedArgs &a, int max_new, int max_cached, const void *ws, size_t bytes)
{
    if (!ws || !aligned(ws, 16))
        return KIVI_ERR_INVALID_ARG;
    return bytes < workspace_bytes(a, max_new, max_cached) ? KIVI_ERR_WORKSPACE : KIVI_OK;
}

int done(kivi_paged *c, cudaError_t e, int launches)
{
    c->kernel_launches += launches;
    return e == cudaSuccess ? KIVI_OK : KIVI_ERR_CUDA;
}

}  // namespace

extern "C" {

int32_t kivi_paged_columns(const kivi_params *p)
{
    return check_paged_params(p) == KIVI_OK ? (int32_t)(p->capacity_tokens / p->group) : 0;
}

size_t kivi_paged_control_bytes(const kivi_params *p)
{
    return check_paged_params(p) == KIVI_OK ? (4 * (size_t)(1 + p->batch) + 255) / 256 * 256 : 0;
}

size_t kivi_paged_workspace_bytes(const kivi_params *p, int32_t max_new, int32_t max_cached)
{
    return check_paged_params(p) == KIVI_OK && max_new >= 0 && max_cached >= 0
               ? workspace_bytes(paged_args(p), max_new, max_cached) : 0;
}

int kivi_paged_init(kivi_paged *c, const kivi_params *p, void *pool, int64_t num_pages, void *k_fp16,
                    void *v_fp16, int32_t *table, int32_t *n_tokens, int32_t *n_evicted, uint32_t *control)
{
    if (!c || !p)
        return KIVI_ERR_INVALID_ARG;
    kivi_paged t;
    std::memset(&t, 0, sizeof(t));
    t.p = *p;
    t.pool = pool;
    t.k_fp16 = k_fp16;
    t.v_fp16 = v_fp16;
    t.table = table;
    t.n_tokens = n_tokens;
    t.n_evicted = n_evicted;
    t.control = control;
    t.num_pages = num_pages;
    const int st = check_paged(&t);
    if (st == KIVI_OK)
        *c = t;
    return st;
}

int kivi_paged_append(kivi_paged *c, const kivi_chunk *x, kivi_stream_t stream)
{
    NvtxRange nvtx_range("kivi_paged_append");
    int st = check_paged(c);
    if (st == KIVI_OK)
        st = check_chunk(c, x, kUseK | kUseV);
    if (st != KIVI_OK)
        return st;
    if (x->max_new == 0 || x->num_tokens == 0)
        return KIVI_OK;
    int launches = 0;
    const cudaError_t e = launch_paged_append(paged_args(c), chunk_args(c, x), reinterpret_cast<cudaStream_t>(stream),
                                              &launches);
    return done(c, e, launches);
}

int kivi_paged_attention(kivi_paged *c, const kivi_chunk *x, void *out, void *workspace, size_t ws_bytes,
                         kivi_stream_t stream)
{
    NvtxRange nvtx_range("kivi_paged_attention");
    int st = check_paged(c);
    if (st == KIVI_OK)
        st = check_chunk(c, x, kUseQ | kUseK | kUseV | kNewOptional);
    if (st != KIVI_OK)
        return st;
    if (x->max_new == 0 || x->num_tokens == 0)
        return KIVI_OK;
    if (!out || !aligned(out, 16))
        return KIVI_ERR_INVALID_ARG;
    const ChunkArgs a = chunk_args(c, x);
    const PagedArgs pa = paged_args(c);
    if (!long_attention_fits(pa, a.max_new, a.max_cached))
        return KIVI_ERR_UNSUPPORTED;
    st = check_workspace(pa, a.max_new, x->max_cached, workspace, ws_bytes);
    if (st != KIVI_OK)
        return st;
    int launches = 0;
    const cudaError_t e = launch_paged_attention(pa, a, static_cast<__half *>(out), workspace,
                                                 reinterpret_cast<cudaStream_t>(stream), &launches);
    return done(c, e, launches);
}

int kivi_paged_weights(kivi_paged *c, const kivi_chunk *x, float *weights, void *workspace, size_t ws_bytes,
                       kivi_stream_t stream)
{
    NvtxRange nvtx_range("kivi_paged_weights");
    int st = check_paged(c);
    if (st == KIVI_OK)
        st = check_chunk(c, x, kUseQ | kUseK | kNewOptional);
    if (st != KIVI_OK)
        return st;
    if (!weights || !aligned(weights, 4))
        return KIVI_ERR_INVALID_ARG;
    if (x->max_new == 0 || x->num_tokens == 0)
        return KIVI_OK;
    const ChunkArgs a = chunk_args(c, x);
    const PagedArgs pa = paged_args(c);
    st = check_workspace(pa, a.max_new, x->max_cached, workspace, ws_bytes);
    if (st != KIVI_OK)
        return st;
    int launches = 0;
    const cudaError_t e = launch_paged_weights(pa, a, weights, workspace, reinterpret_cast<cudaStream_t>(stream),
                                               &launches);
    return done(c, e, launches);
}

int kivi_paged_evict(kivi_paged *c, float *weights, int32_t budget_pages, int32_t recent_pages, void *workspace,
                     size_t ws_bytes, kivi_stream_t stream)
{
    NvtxRange nvtx_range("kivi_paged_evict");
    int st = check_paged(c);
    if (st != KIVI_OK)
        return st;
    if (!weights || !aligned(weights, 4) || budget_pages < 0 || recent_pages < 0)
        return KIVI_ERR_INVALID_ARG;
    const PagedArgs pa = paged_args(c);
    st = check_workspace(pa, 0, 0, workspace, ws_bytes);
    if (st != KIVI_OK)
        return st;
    int launches = 0;
    const cudaError_t e = launch_paged_evict(pa, weights, budget_pages, recent_pages, workspace,
                                             reinterpret_cast<cudaStream_t>(stream), &launches);
    return done(c, e, launches);
}

size_t kivi_sizeof_paged(void) { return sizeof(kivi_paged); }
size_t kivi_sizeof_chunk(void) { return sizeof(kivi_chunk); }

}  // extern "C"
