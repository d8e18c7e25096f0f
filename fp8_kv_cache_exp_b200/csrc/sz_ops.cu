// sz_ops.cu -- the extern "C" entry points of the operators on a paged cache
// (include/splitzip.h): host-side argument checks and dispatch.  No device
// memory is allocated here.
#include <cmath>
#include <cstdlib>

#include "sz_ops.cuh"

namespace {

using namespace sz;

bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

int num_sms() {
    static std::atomic<int> cache[kMaxDevices];
    int dev = 0, sms = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return 0;
    sms = cache[dev].load(std::memory_order_acquire);
    if (sms > 0) return sms;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    cache[dev].store(sms, std::memory_order_release);
    return sms;
}

sz_status check_cache(const sz_kv_cache_t *c) {
    if (!c) return SZ_ERR_INVALID_ARG;
    if (c->dtype != SZ_BF16 && c->dtype != SZ_FP8_E5M2) return SZ_ERR_UNSUPPORTED_DTYPE;
    if (!c->k_pool || !c->v_pool || !aligned(c->k_pool, 16) || !aligned(c->v_pool, 16) || !c->table ||
        !aligned(c->table, 4))
        return SZ_ERR_INVALID_ARG;
    if (c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16 != 0) return SZ_ERR_INVALID_ARG;
    if (c->kv_heads < 1 || c->kv_heads > 4096 || c->seqs < 1 || c->seqs > 65536 || c->page_tokens < 1 ||
        c->page_tokens > (1u << 20) || c->pool_pages < 1)
        return SZ_ERR_INVALID_ARG;
    if (c->table_pages < 1 || uint64_t(c->table_pages) * c->page_tokens >= (1ull << 31) ||
        (c->seqs > 1 && c->table_stride < c->table_pages))
        return SZ_ERR_INVALID_ARG;
    const uint64_t eb = c->dtype == SZ_BF16 ? 2 : 1;
    const uint64_t row = uint64_t(c->kv_heads) * c->head_dim * eb;
    if (c->page_bytes % 16 != 0 || c->page_bytes < row * c->page_tokens || c->page_bytes > (1ull << 40))
        return SZ_ERR_INVALID_ARG;
    return SZ_OK;
}

// A view of activations: alignment, and rows that do not overlap where it is written.
bool heads_ok(const sz_heads_t &h, uint64_t tokens, uint32_t dim, bool written) {
    if (h.heads < 1 || h.heads > 65536 || h.token_stride % 8 != 0 || h.head_stride % 8 != 0 ||
        h.token_stride > (1ull << 40) || h.head_stride > (1ull << 40))
        return false;
    if (tokens > 0 && (!h.data || !aligned(h.data, 16))) return false;
    if (written) {
        const uint64_t lo = h.token_stride < h.head_stride ? h.token_stride : h.head_stride;
        const bool by_head = h.head_stride <= h.token_stride;  // heads inside a token, or tokens inside a head
        const uint64_t inner = by_head ? h.heads : tokens, outer = by_head ? tokens : h.heads;
        const uint64_t hi = by_head ? h.token_stride : h.head_stride;
        if (inner > 1 && lo < dim) return false;
        if (outer > 1 && hi < (inner > 1 ? (inner - 1) * lo : 0) + dim) return false;
    }
    return true;
}

bool same_view(const sz_heads_t &a, const sz_heads_t &b) {
    return a.data == b.data && a.token_stride == b.token_stride && a.head_stride == b.head_stride;
}

// First and last byte of a view.
void extent(const sz_heads_t &h, uint64_t tokens, uint32_t dim, uintptr_t *a, uintptr_t *b) {
    *a = reinterpret_cast<uintptr_t>(h.data);
    *b = *a + 2 * ((tokens - 1) * h.token_stride + (uint64_t(h.heads) - 1) * h.head_stride + dim);
}

// Whether rows of two views of one layout meet, y's first being `gap` elements
// behind x's: for some difference of heads and of tokens they are less than a
// row apart.
bool rows_meet(int64_t gap, int64_t token_stride, int64_t head_stride, int64_t tokens, int64_t x_heads, int64_t y_heads,
               int64_t dim) {
    for (int64_t h = 1 - x_heads; h < y_heads; ++h) {
        const int64_t v = gap + h * head_stride;
        int64_t t = tokens > 1 && token_stride > 0 ? -(v / token_stride) : 0;  // brings v nearest to 0, or next to that
        t = t < 1 - tokens ? 1 - tokens : (t > tokens - 1 ? tokens - 1 : t);
        for (int64_t u = t - 1; u <= t + 1; ++u)
            if (u > -tokens && u < tokens && std::llabs(v + u * token_stride) < dim) return true;
    }
    return false;
}

// Whether two views' rows can meet: their extents do, and they are not the
// interleaved columns of one buffer (heads [a, b) and [b, c) of each token).
// Views of unlike layouts whose extents meet are taken to.
bool may_overlap(const sz_heads_t &x, const sz_heads_t &y, uint64_t tokens, uint32_t dim) {
    if (tokens == 0) return false;
    uintptr_t a, b, c, d;
    extent(x, tokens, dim, &a, &b);
    extent(y, tokens, dim, &c, &d);
    if (b <= c || d <= a) return false;
    if (x.token_stride == y.token_stride && x.token_stride > 0) {
        const uint64_t period = 2 * x.token_stride;  // bytes
        const uint64_t wx = 2 * ((uint64_t(x.heads) - 1) * x.head_stride + dim);
        const uint64_t wy = 2 * ((uint64_t(y.heads) - 1) * y.head_stride + dim);
        const uint64_t gap = a <= c ? (c - a) % period : (period - (a - c) % period) % period;  // of y behind x
        if (wx <= period && wy <= period && gap >= wx && gap + wy <= period) return false;
    }
    // (one token's or one head's stride is nothing)
    if ((tokens == 1 || x.token_stride == y.token_stride) &&
        (x.heads == 1 || y.heads == 1 || x.head_stride == y.head_stride))
        return rows_meet((int64_t(c) - int64_t(a)) / 2, int64_t(x.token_stride),
                         int64_t(x.heads > 1 ? x.head_stride : y.head_stride), int64_t(tokens), x.heads, y.heads, dim);
    return true;
}

bool norm_ok(const sz_head_norm_t &n) {
    if (!n.q_weight && !n.k_weight) return true;
    return aligned(n.q_weight, 16) && aligned(n.k_weight, 16) && n.eps >= 0.f && std::isfinite(n.eps);
}

bool rope_ok(const sz_rope_t &r, uint32_t dim) {
    if (!r.table) return true;
    return aligned(r.table, 16) && aligned(r.positions, 4) && r.rot >= 8 && r.rot % 8 == 0 && r.rot <= dim &&
           r.table_len >= 1 && r.table_len <= 0x7fffffffu;
}

CacheRef cache_ref(const sz_kv_cache_t &c) {
    CacheRef r;
    r.k = static_cast<uint8_t *>(c.k_pool);
    r.v = static_cast<uint8_t *>(c.v_pool);
    r.table = c.table;
    r.pool_pages = c.pool_pages;
    r.page_bytes = c.page_bytes;
    r.table_stride = c.table_stride;
    r.seqs = c.seqs;
    r.kv_heads = c.kv_heads;
    r.head_dim = c.head_dim;
    r.capacity = c.table_pages * c.page_tokens;
    r.row_bytes = c.kv_heads * c.head_dim * (c.dtype == SZ_BF16 ? 2 : 1);
    r.page_tokens = fast_div(c.page_tokens);
    return r;
}

HeadsRef heads_ref(const sz_heads_t &h) {
    return HeadsRef{static_cast<uint8_t *>(h.data), h.token_stride * 2, h.head_stride * 2, h.data ? h.heads : 0};
}

void rope_params(RopeParams &p, const sz_head_norm_t &n, const sz_rope_t &r) {
    p.q_weight = static_cast<const uint8_t *>(n.q_weight);
    p.k_weight = static_cast<const uint8_t *>(n.k_weight);
    p.eps = n.eps;
    p.rope = RopeRef{r.table, r.positions, r.table_len, r.table ? r.rot : 0, r.interleaved};
}

sz_status check_ws(const void *d_ws, size_t have, size_t need) {
    if (!d_ws || !aligned(d_ws, 8)) return SZ_ERR_INVALID_ARG;
    return have < need ? SZ_ERR_BUFFER_TOO_SMALL : SZ_OK;
}

}  // namespace

extern "C" {

size_t sz_ops_workspace_bytes(const sz_kv_cache_t *cache) {
    if (!cache) return size_t(kCtlWords) * 4;
    if (check_cache(cache) != SZ_OK) return 0;
    return size_t(kCtlWords) * 4 + kArrivedBytes + kDescBytes + attn_part_floats(cache->head_dim) * 4 + 16;
}

sz_status sz_kv_append_paged(const sz_kv_cache_t *cache, const sz_kv_append_t *a, void *d_ws, size_t ws_bytes,
                             cudaStream_t stream) {
    sz_status s = check_cache(cache);
    if (s != SZ_OK) return s;
    if (!a || a->tokens >= (1ull << 31)) return SZ_ERR_INVALID_ARG;
    s = check_ws(d_ws, ws_bytes, size_t(kCtlWords) * 4);
    if (s != SZ_OK) return s;
    const uint32_t dim = cache->head_dim;
    if (!heads_ok(a->k, a->tokens, dim, false) || !heads_ok(a->v, a->tokens, dim, false) ||
        a->k.heads != cache->kv_heads || a->v.heads != cache->kv_heads)
        return SZ_ERR_INVALID_ARG;
    if (!a->q.data != !a->q_out.data) return SZ_ERR_INVALID_ARG;
    if (a->q.data) {
        if (!heads_ok(a->q, a->tokens, dim, false) || !heads_ok(a->q_out, a->tokens, dim, true) ||
            a->q.heads != a->q_out.heads)
            return SZ_ERR_INVALID_ARG;
        if (!same_view(a->q, a->q_out) && may_overlap(a->q, a->q_out, a->tokens, dim)) return SZ_ERR_INVALID_ARG;
        if (may_overlap(a->k, a->q_out, a->tokens, dim) || may_overlap(a->v, a->q_out, a->tokens, dim))
            return SZ_ERR_INVALID_ARG;
    }
    if (!a->cu_q || !aligned(a->cu_q, 4) || !a->kv_len || !aligned(a->kv_len, 4)) return SZ_ERR_INVALID_ARG;
    if (!norm_ok(a->norm) || !rope_ok(a->rope, dim)) return SZ_ERR_INVALID_ARG;
    if (a->tokens == 0) return SZ_OK;
    RopeParams p{};
    p.ctl = static_cast<uint32_t *>(d_ws);
    p.cache = cache_ref(*cache);
    p.q = heads_ref(a->q);
    p.q_out = heads_ref(a->q_out);
    p.k = heads_ref(a->k);
    p.v = heads_ref(a->v);
    p.cu_q = a->cu_q;
    p.kv_len = a->kv_len;
    rope_params(p, a->norm, a->rope);
    p.tokens = uint32_t(a->tokens);
    p.head_dim = dim;
    p.inv_dim = 1.f / float(dim);
    const int sms = num_sms();
    if (sms <= 0) return SZ_ERR_CUDA;
    return launch_rope(p, true, int(cache->dtype), sms, stream);
}

sz_status sz_qk_norm_rope(const sz_qk_norm_rope_t *a, void *d_ws, size_t ws_bytes, cudaStream_t stream) {
    if (!a || a->tokens >= (1ull << 31)) return SZ_ERR_INVALID_ARG;
    const uint32_t dim = a->head_dim;
    if (dim < 16 || dim > 256 || dim % 16 != 0) return SZ_ERR_INVALID_ARG;
    const sz_status s = check_ws(d_ws, ws_bytes, size_t(kCtlWords) * 4);
    if (s != SZ_OK) return s;
    if (!a->q.data != !a->q_out.data || !a->k.data != !a->k_out.data) return SZ_ERR_INVALID_ARG;
    if (a->tokens > 0 && !a->q.data && !a->k.data) return SZ_ERR_INVALID_ARG;
    const sz_heads_t *in[2] = {&a->q, &a->k}, *out[2] = {&a->q_out, &a->k_out};
    for (int i = 0; i < 2; ++i) {
        if (!in[i]->data) continue;
        if (!heads_ok(*in[i], a->tokens, dim, false) || !heads_ok(*out[i], a->tokens, dim, true) ||
            in[i]->heads != out[i]->heads)
            return SZ_ERR_INVALID_ARG;
        for (int j = 0; j < 2; ++j)
            if (in[j]->data && !(i == j && same_view(*in[j], *out[i])) && may_overlap(*in[j], *out[i], a->tokens, dim))
                return SZ_ERR_INVALID_ARG;
    }
    if (a->q.data && a->k.data && may_overlap(a->q_out, a->k_out, a->tokens, dim)) return SZ_ERR_INVALID_ARG;
    if (!norm_ok(a->norm) || !rope_ok(a->rope, dim) || (a->rope.table && a->tokens > 0 && !a->rope.positions))
        return SZ_ERR_INVALID_ARG;
    if (a->tokens == 0) return SZ_OK;
    RopeParams p{};
    p.ctl = static_cast<uint32_t *>(d_ws);
    p.q = heads_ref(a->q);
    p.q_out = heads_ref(a->q_out);
    p.k = heads_ref(a->k);
    p.k_out = heads_ref(a->k_out);
    rope_params(p, a->norm, a->rope);
    p.tokens = uint32_t(a->tokens);
    p.head_dim = dim;
    p.inv_dim = 1.f / float(dim);
    const int sms = num_sms();
    if (sms <= 0) return SZ_ERR_CUDA;
    return launch_rope(p, false, SZ_BF16, sms, stream);
}

sz_status sz_attn_paged(const sz_kv_cache_t *cache, const sz_attn_t *a, void *d_ws, size_t ws_bytes,
                        cudaStream_t stream) {
    sz_status s = check_cache(cache);
    if (s != SZ_OK) return s;
    if (!a || a->tokens >= (1ull << 31)) return SZ_ERR_INVALID_ARG;
    s = check_ws(d_ws, ws_bytes, sz_ops_workspace_bytes(cache));
    if (s != SZ_OK) return s;
    const uint32_t dim = cache->head_dim;
    if (!heads_ok(a->q, a->tokens, dim, false) || !heads_ok(a->out, a->tokens, dim, true) ||
        a->q.heads != a->out.heads || a->q.heads % cache->kv_heads != 0)
        return SZ_ERR_INVALID_ARG;
    // a group's rows of all tokens are counted in 32 bits
    if (a->tokens * (a->q.heads / cache->kv_heads) >= (1ull << 31)) return SZ_ERR_INVALID_ARG;
    if (may_overlap(a->q, a->out, a->tokens, dim)) return SZ_ERR_INVALID_ARG;
    if (!a->cu_q || !aligned(a->cu_q, 4) || !a->kv_len || !aligned(a->kv_len, 4) || !aligned(a->lse, 4))
        return SZ_ERR_INVALID_ARG;
    if (!(a->scale > 0.f) || !std::isfinite(a->scale) || a->window > 0x7fffffffu) return SZ_ERR_INVALID_ARG;
    if (a->tokens == 0) return SZ_OK;
    AttnParams p{};
    uint8_t *ws = static_cast<uint8_t *>(d_ws);
    p.ctl = reinterpret_cast<uint32_t *>(ws);
    p.arrived = reinterpret_cast<uint32_t *>(ws + size_t(kCtlWords) * 4);
    p.desc = ws + size_t(kCtlWords) * 4 + kArrivedBytes;
    // the workspace is 8-byte aligned, partials are read and written 16 bytes at a time
    p.part = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(p.desc + kDescBytes) + 15) & ~uintptr_t(15));
    p.cache = cache_ref(*cache);
    p.q = heads_ref(a->q);
    p.out = heads_ref(a->out);
    p.cu_q = a->cu_q;
    p.kv_len = a->kv_len;
    p.lse = a->lse;
    p.scale_log2 = float(double(a->scale) * 1.4426950408889634);
    p.tokens = uint32_t(a->tokens);
    p.causal = a->causal;
    p.window = a->window;
    p.group = fast_div(a->q.heads / cache->kv_heads);
    const int sms = num_sms();
    if (sms <= 0) return SZ_ERR_CUDA;
    return launch_attn(p, int(cache->dtype), sms < int(kMaxSms) ? sms : int(kMaxSms), stream);
}

}  // extern "C"
