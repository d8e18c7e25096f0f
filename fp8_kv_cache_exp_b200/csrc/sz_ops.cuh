// sz_ops.cuh -- what the operators on a paged cache share: kernel parameter
// blocks, division by a launch constant, sequence lookup, page addresses and
// conversions.  The operators are declared in include/splitzip.h.
#pragma once

#include "sz_common.cuh"

namespace sz {

// n / d for n < 2^31 and a divisor fixed at launch: multiply by ceil(2^(31+s) / d)
// with s = ceil(log2 d), and shift (the error of the rounded-up reciprocal,
// below 2^s / 2^(31+s), stays under 1/n).
struct FastDiv {
    uint32_t d, mul, shift;
};
inline FastDiv fast_div(uint32_t d) {
    FastDiv f;
    f.d = d;
    uint32_t s = 0;
    while ((1ull << s) < d) ++s;
    f.shift = s;
    f.mul = uint32_t(((1ull << (31 + s)) + d - 1) / d);
    return f;
}
__device__ __forceinline__ uint32_t div_by(uint32_t n, const FastDiv &f) {
    return uint32_t((uint64_t(n) * f.mul) >> (31 + f.shift));
}

struct CacheRef {
    uint8_t *k, *v;
    const int32_t *table;
    uint64_t pool_pages, page_bytes;
    uint32_t table_stride, seqs, kv_heads, head_dim;
    uint32_t capacity;   // table_pages * page_tokens
    uint32_t row_bytes;  // kv_heads * head_dim * element bytes
    FastDiv page_tokens;
};

struct HeadsRef {
    uint8_t *p;
    uint64_t ts, hs;  // bytes from token to token and from head to head
    uint32_t heads;
};

struct RopeRef {
    const float *table;
    const int32_t *positions;
    uint32_t len, rot, interleaved;
};

struct RopeParams {
    uint32_t *ctl;
    CacheRef cache;  // append only
    HeadsRef q, q_out, k, k_out, v;
    const int32_t *cu_q, *kv_len;
    const uint8_t *q_weight, *k_weight;
    float eps, inv_dim;  // (1 / head_dim)
    RopeRef rope;
    uint32_t tokens, head_dim;
    FastDiv chunks;  // chunks of heads to a token
};

struct AttnParams {
    uint32_t *ctl;
    uint32_t *arrived;   // arrival counters, zero between calls
    uint8_t *desc;       // what a CTA of the tensor-memory kernel leaves for the joining one
    float *part;         // partial results, two slots for each CTA
    CacheRef cache;
    HeadsRef q, out;
    const int32_t *cu_q, *kv_len;
    float *lse;
    float scale_log2;    // scale * log2(e)
    uint32_t tokens, causal, window;
    FastDiv group;       // query heads to a KV head
    uint64_t wait_ns;    // limit of the tensor-memory kernel's waits
};

// ------------------------------------------------------------ device helpers

// Byte offset of place t of a sequence (its table row) in either pool, or
// kBadOffset, with the error recorded, when the page id is outside the pool.
__device__ __forceinline__ uint64_t place_offset(const CacheRef &c, uint32_t *ctl, const int32_t *row, uint32_t t) {
    const uint32_t page = div_by(t, c.page_tokens);
    const int64_t id = __ldg(row + page);
    if (id < 0 || uint64_t(id) >= c.pool_pages) {
        set_error(ctl, SZ_ERR_INVALID_ARG, page);
        return kBadOffset;
    }
    return uint64_t(id) * c.page_bytes + uint64_t(t - page * c.page_tokens.d) * c.row_bytes;
}

// The sequence of packed row t: the number of entries of cu_q[1..seqs] that
// are <= t (seqs for a row behind the last one).  All lanes of a warp ask for
// the same t; 32 entries are looked at in a round.
__device__ __forceinline__ uint32_t warp_find_seq(const int32_t *cu_q, uint32_t seqs, uint32_t t) {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t lo = 0, n = seqs;  // the answer is in [lo, lo + n]
    while (n > 0) {
        const uint32_t step = (n + 31) / 32;
        const uint32_t at = (lane + 1) * step;  // entries lo+1 .. lo+at: is the last of them <= t?
        const bool below = at <= n && __ldg(cu_q + lo + at) <= int32_t(t);
        const uint32_t c = __popc(__ballot_sync(0xffffffffu, below));
        lo += c * step;
        const uint32_t left = n - c * step;
        n = left < step ? left : step - 1;
    }
    return lo;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Two floats to E5M2, to nearest even.  The instruction saturates; values of
// at least 61440, half a step beyond the largest finite 57344, are infinity.
__device__ __forceinline__ uint32_t pack_e5m2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    uint32_t w = r;
    if (fabsf(lo) >= 61440.f) w = (w & 0xff80u) | 0x7cu;
    if (fabsf(hi) >= 61440.f) w = (w & 0x80ffu) | 0x7c00u;
    return w;
}

// Launchers (sz_rope.cu, sz_attn.cu, sz_attn_tc.cu).
sz_status launch_rope(const RopeParams &p, bool append, int dtype, int num_sms, cudaStream_t stream);
sz_status launch_attn(const AttnParams &p, int dtype, int num_sms, cudaStream_t stream);
sz_status launch_attn_tc(AttnParams p, int dtype, int num_sms, cudaStream_t stream);

// Workspace of sz_attn_paged behind the 256-byte control block: arrival
// counters, descriptors, then partial results.  A partial is kPartRows rows of a head's
// sums in float and two statistics a row.
constexpr uint32_t kMaxSms = 160;
constexpr uint32_t kAttnCtas = 3 * kMaxSms;  // most CTAs of any attention kernel
// counters: three for each CTA of the split kernel, or one for each warp of a tile
constexpr size_t kArrivedBytes = size_t(3) * kAttnCtas * 4;
static_assert(kMaxSms * 8 <= 3 * kAttnCtas, "arrival counters");
constexpr size_t kDescBytes = size_t(kMaxSms) * 192;
// floats of all partials: the largest (CTAs * rows) of the kernels is a
// persistent CTA for each SM with 256 rows, or kAttnCtas of 32
constexpr size_t attn_part_floats(uint32_t head_dim) { return size_t(2) * kMaxSms * 256 * (head_dim + 2); }

}  // namespace sz
