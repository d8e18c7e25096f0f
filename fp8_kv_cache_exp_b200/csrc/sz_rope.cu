// sz_rope.cu -- norm and rotation of query and key heads, to contiguous
// outputs (sz_qk_norm_rope) or, keys and values, into the pages of a cache
// (sz_kv_append_paged).
//
//   n_i = x_i * (1 / sqrt(mean(x^2) + eps)) * w_i
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first rot
//   elements, in 32 bits, rounded once to the output's type.  Each product and
//   sum of the rotation is rounded by itself: fused, some keys next to the border
//   of two 8-bit values would fall on its other side than the formula in 32 bits.
//
// One element is read, turned and written: the bytes are the bound, and for a
// few tokens the latency of the dependent loads (sequence, length, page id).
// Measured: 16,384 tokens of 40 heads of 128, normed: 67 us, 5.1 TB/s, 0.78 of a
// plain copy's rate (positions and their table rows are two loads in a row, and
// 24 warps an SM do not hide all of it; 64 registers a thread or other numbers of
// rows to a group are slower); chunks of 6 prompts into an E5M2 cache: 21 us; one
// token: 2.7 us, the call itself.
#include "sz_ops.cuh"

namespace sz {
namespace {

constexpr int kRopeThreads = 128;  // six CTAs an SM turn over more evenly than three of 256 (16,384 tokens: 67 us, 71)

// Plain loads: the rows may be those that the call writes (in place, each lane
// writes the elements that it read).
__device__ __forceinline__ void load8(float (&x)[8], const uint8_t *a, const uint8_t *b) {
    const uint2 u = *reinterpret_cast<const uint2 *>(a), w = *reinterpret_cast<const uint2 *>(b);
    x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(w.x), x[5] = bf16_hi(w.x), x[6] = bf16_lo(w.y), x[7] = bf16_hi(w.y);
}

// Sequences of a warp's groups, one warp-wide search for each token among them.
template <int LG>
__device__ __forceinline__ uint32_t group_seq(const RopeParams &p, uint32_t token) {
    const uint32_t lane = threadIdx.x & 31;
    uint32_t seq = 0, known = 0xffffffffu;
#pragma unroll
    for (int g = 0; g < 32 / LG; ++g) {
        const uint32_t t = __shfl_sync(0xffffffffu, token, g * LG);
        if (t != known) {
            const uint32_t s = warp_find_seq(p.cu_q, p.cache.seqs, t);
            if (lane / LG >= g) seq = s;
            known = t;
        }
    }
    return seq;
}

// The token's place in the cache and its position; false if it has none (which is recorded).
template <bool APPEND, int LG>
__device__ __forceinline__ bool locate(const RopeParams &p, uint32_t token, bool live, bool first, int64_t &pos,
                                       uint64_t &place) {
    bool ok = live;
    if constexpr (APPEND) {
        const uint32_t seq = group_seq<LG>(p, token);
        ok = ok && seq < p.cache.seqs && token >= uint32_t(__ldg(p.cu_q));
        if (ok) {
            pos = int64_t(__ldg(p.kv_len + seq)) - (int64_t(__ldg(p.cu_q + seq + 1)) - int64_t(token));
            if (pos < 0 || pos >= int64_t(p.cache.capacity)) {
                if (first) set_error(p.ctl, SZ_ERR_INVALID_ARG, token);
                ok = false;
            } else {
                place = place_offset(p.cache, p.ctl, p.cache.table + uint64_t(seq) * p.cache.table_stride, uint32_t(pos));
                ok = place != kBadOffset;
            }
        }
    }
    if (p.rope.rot > 0 && ok) {
        if (p.rope.positions) pos = __ldg(p.rope.positions + token);
        if (pos < 0 || pos >= int64_t(p.rope.len)) {
            if (first) set_error(p.ctl, SZ_ERR_INVALID_ARG, token);
            ok = false;
        }
    }
    return ok;
}

__device__ __forceinline__ void turn(float &a, float &b, float c, float s) {
    const float u = a, v = b;
    a = __fsub_rn(__fmul_rn(u, c), __fmul_rn(v, s));
    b = __fadd_rn(__fmul_rn(v, c), __fmul_rn(u, s));
}
__device__ __forceinline__ void unpack8(float *x, const uint4 &v) {
    x[0] = bf16_lo(v.x), x[1] = bf16_hi(v.x), x[2] = bf16_lo(v.y), x[3] = bf16_hi(v.y);
    x[4] = bf16_lo(v.z), x[5] = bf16_hi(v.z), x[6] = bf16_lo(v.w), x[7] = bf16_hi(v.w);
}
__device__ __forceinline__ uint4 pack8(const float *x) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

// A group of LG lanes has one token and N of its head rows; a lane holds two
// 16-byte runs of a row: of each half of the rotated part, or 16 elements in
// order (interleaved pairs, and what is not rotated).  All of a group's rows are
// on their way before anything that they wait for.  Runs of 8 bytes (below) took
// 109 us for 16,384 tokens of 40 heads of 128.
template <int LG, int N, bool APPEND, int DT>
__global__ void __launch_bounds__(kRopeThreads, 6) rope_wide_kernel(const __grid_constant__ RopeParams p) {
    constexpr uint32_t EB = DT == SZ_BF16 ? 2 : 1;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t l = threadIdx.x % LG;
    const uint32_t d = p.head_dim, rot = p.rope.rot, half = rot / 2;
    const uint64_t groups = uint64_t(p.tokens) * p.chunks.d;
    const uint64_t gid = (uint64_t(blockIdx.x) * kRopeThreads + threadIdx.x) / LG;
    const bool live = gid < groups;
    uint32_t token, chunk;
    if (groups < (1ull << 31)) {
        token = div_by(uint32_t(live ? gid : 0), p.chunks);
        chunk = uint32_t(live ? gid : 0) - token * p.chunks.d;
    } else {
        token = uint32_t((live ? gid : 0) / p.chunks.d);
        chunk = uint32_t((live ? gid : 0) % p.chunks.d);
    }
    // a group's rows are all queries, all keys or all values
    const uint32_t cq = (p.q.heads + N - 1) / N, ck = (p.k.heads + N - 1) / N;
    const bool is_q = chunk < cq, is_v = APPEND && chunk >= cq + ck;
    const uint32_t head0 = (is_q ? chunk : (is_v ? chunk - cq - ck : chunk - cq)) * N;
    const HeadsRef &in = is_q ? p.q : (is_v ? p.v : p.k);
    const uint32_t rows = live && l * 16 < d ? min(uint32_t(N), in.heads - head0) : 0;
    const bool turns = !is_v && l * 16 < rot, split = turns && !p.rope.interleaved;
    const uint32_t off_a = split ? 8 * l : 16 * l, off_b = split ? half + 8 * l : 16 * l + 8;

    // (plain loads: the rows may be those that the call writes; in place, each lane writes what it read)
    uint4 va[N], vb[N];
    {
        const uint8_t *row = in.p + token * in.ts + head0 * in.hs;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            if (i >= rows) continue;
            va[i] = *reinterpret_cast<const uint4 *>(row + i * in.hs + 2 * off_a);
            vb[i] = *reinterpret_cast<const uint4 *>(row + i * in.hs + 2 * off_b);
        }
    }
    const uint8_t *w = is_q ? p.q_weight : (is_v ? nullptr : p.k_weight);
    float g[16];
    if (w && rows > 0) {
        unpack8(g, __ldg(reinterpret_cast<const uint4 *>(w + 2 * off_a)));
        unpack8(g + 8, __ldg(reinterpret_cast<const uint4 *>(w + 2 * off_b)));
    }
    int64_t pos = 0;
    uint64_t place = kBadOffset;
    const bool ok = locate<APPEND, LG>(p, token, live, l == 0, pos, place);
    float cs[8], sn[8];
    if (ok && turns) {
        const float4 *t = reinterpret_cast<const float4 *>(p.rope.table + uint64_t(pos) * rot + 8 * l);
        const float4 *u = reinterpret_cast<const float4 *>(p.rope.table + uint64_t(pos) * rot + half + 8 * l);
        const float4 c0 = __ldg(t), c1 = __ldg(t + 1), s0 = __ldg(u), s1 = __ldg(u + 1);
        cs[0] = c0.x, cs[1] = c0.y, cs[2] = c0.z, cs[3] = c0.w, cs[4] = c1.x, cs[5] = c1.y, cs[6] = c1.z, cs[7] = c1.w;
        sn[0] = s0.x, sn[1] = s0.y, sn[2] = s0.z, sn[3] = s0.w, sn[4] = s1.x, sn[5] = s1.y, sn[6] = s1.z, sn[7] = s1.w;
    }
    const bool to_cache = APPEND && !is_q;
    uint8_t *to;
    uint64_t step;
    if (to_cache) {
        to = (is_v ? p.cache.v : p.cache.k) + place + uint64_t(head0) * d * EB;
        step = d * EB;
    } else {
        const HeadsRef &h = is_q ? p.q_out : p.k_out;
        to = h.p + token * h.ts + head0 * h.hs;
        step = h.hs;
    }

#pragma unroll
    for (int i = 0; i < N; ++i) {
        float x[16];
        unpack8(x, va[i]);
        unpack8(x + 8, vb[i]);
        if (p.q_weight || p.k_weight) {  // (some of the warp's groups may have none: all take part in the sum)
            float ss = 0.f;
            if (i < rows) {
#pragma unroll
                for (int j = 0; j < 16; ++j) ss = fmaf(x[j], x[j], ss);
            }
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (w) {
                const float rs = rsqrtf(ss * p.inv_dim + p.eps);
#pragma unroll
                for (int j = 0; j < 16; ++j) x[j] = x[j] * rs * g[j];
            }
        }
        if (i >= rows || !ok) continue;
        // half-split: element j of either run; interleaved: elements 2j and 2j + 1 of the sixteen
        if (split) {
#pragma unroll
            for (int j = 0; j < 8; ++j) turn(x[j], x[j + 8], cs[j], sn[j]);
        } else if (turns) {
#pragma unroll
            for (int j = 0; j < 8; ++j) turn(x[2 * j], x[2 * j + 1], cs[j], sn[j]);
        }
        if (DT == SZ_FP8_E5M2 && to_cache) {
            uint32_t y[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) y[j] = pack_e5m2(x[4 * j], x[4 * j + 1]) | pack_e5m2(x[4 * j + 2], x[4 * j + 3]) << 16;
            *reinterpret_cast<uint2 *>(to + i * step + off_a) = make_uint2(y[0], y[1]);
            *reinterpret_cast<uint2 *>(to + i * step + off_b) = make_uint2(y[2], y[3]);
        } else {
            *reinterpret_cast<uint4 *>(to + i * step + 2 * off_a) = pack8(x);
            *reinterpret_cast<uint4 *>(to + i * step + 2 * off_b) = pack8(x + 8);
        }
    }
}

// The same with eight elements to a lane, in two runs of 8 bytes: for halves of
// the rotated part that are not a multiple of 8 elements.
template <int LG, int N, bool APPEND, int DT>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams p) {
    constexpr uint32_t EB = DT == SZ_BF16 ? 2 : 1;
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t lane = threadIdx.x & 31, l = lane % LG;
    const uint32_t d = p.head_dim, rot = p.rope.rot, half = rot / 2;
    const uint64_t groups = uint64_t(p.tokens) * p.chunks.d;
    const uint64_t gid = (uint64_t(blockIdx.x) * kRopeThreads + threadIdx.x) / LG;
    const bool live = gid < groups;
    uint32_t token, chunk;
    if (groups < (1ull << 31)) {
        token = div_by(uint32_t(gid < groups ? gid : 0), p.chunks);
        chunk = uint32_t(gid) - token * p.chunks.d;
    } else {
        token = uint32_t(gid / p.chunks.d);
        chunk = uint32_t(gid % p.chunks.d);
    }

    const uint32_t hq = p.q.heads, hk = p.k.heads;
    const uint32_t rows = hq + hk + (APPEND ? p.v.heads : 0);
    const bool in_row = live && l * 8 < d;
    // element offsets of the lane's two runs of four
    const bool turns = l * 8 < rot;
    const bool split = turns && !p.rope.interleaved;
    const uint32_t off_a = split ? 4 * l : 8 * l, off_b = split ? half + 4 * l : 8 * l + 4;

    // all of the group's rows at once, before anything that they wait for
    float x[N][8];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t r = chunk * N + i;
        if (!in_row || r >= rows) continue;
        const HeadsRef &h = r < hq ? p.q : (r < hq + hk ? p.k : p.v);
        const uint32_t head = r < hq ? r : (r < hq + hk ? r - hq : r - hq - hk);
        const bool v = APPEND && r >= hq + hk;
        const uint8_t *row = h.p + token * h.ts + head * h.hs;
        load8(x[i], row + 2 * (v ? 8 * l : off_a), row + 2 * (v ? 8 * l + 4 : off_b));
    }

    int64_t pos = 0;        // position of the rotation
    uint64_t place = kBadOffset;
    const bool ok = locate<APPEND, LG>(p, token, live, l == 0, pos, place);
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (ok && turns) {
        const float4 c = __ldg(reinterpret_cast<const float4 *>(p.rope.table + uint64_t(pos) * rot + 4 * l));
        const float4 s = __ldg(reinterpret_cast<const float4 *>(p.rope.table + uint64_t(pos) * rot + half + 4 * l));
        cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
        sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
    }

#pragma unroll
    for (int i = 0; i < N; ++i) {
        const uint32_t r = chunk * N + i;
        if (__all_sync(0xffffffffu, !live || r >= rows)) continue;
        const bool is_q = r < hq, is_v = APPEND && r >= hq + hk;
        const uint8_t *w = is_q ? p.q_weight : (is_v ? nullptr : p.k_weight);
        const bool has = in_row && r < rows;
        if (p.q_weight || p.k_weight) {
            float ss = 0.f;
            if (has) {
#pragma unroll
                for (int j = 0; j < 8; ++j) ss = fmaf(x[i][j], x[i][j], ss);
            }
#pragma unroll
            for (int o = LG / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
            if (has && w) {
                const float rs = rsqrtf(ss * p.inv_dim + p.eps);
                float g[8];
                load8(g, w + 2 * off_a, w + 2 * off_b);
#pragma unroll
                for (int j = 0; j < 8; ++j) x[i][j] = __fmul_rn(__fmul_rn(x[i][j], rs), g[j]);
            }
        }
        if (!has || !ok) continue;
        if (turns && !is_v) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                // half-split: element j of either run; interleaved: elements 2j and 2j + 1 of the eight
                const int ia = j, ib = j + 4, ja = 2 * j, jb = 2 * j + 1;
                if (split) {
                    const float a = x[i][ia], b = x[i][ib];
                    x[i][ia] = __fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(b, sn[j]));
                    x[i][ib] = __fadd_rn(__fmul_rn(b, cs[j]), __fmul_rn(a, sn[j]));
                } else {
                    const float a = x[i][ja], b = x[i][jb];
                    x[i][ja] = __fsub_rn(__fmul_rn(a, cs[j]), __fmul_rn(b, sn[j]));
                    x[i][jb] = __fadd_rn(__fmul_rn(b, cs[j]), __fmul_rn(a, sn[j]));
                }
            }
        }
        const uint32_t wa = is_v ? 8 * l : off_a, wb = is_v ? 8 * l + 4 : off_b;
        if (APPEND && !is_q) {
            const uint32_t head = is_v ? r - hq - hk : r - hq;
            uint8_t *row = (is_v ? p.cache.v : p.cache.k) + place + uint64_t(head) * d * EB;
            if constexpr (DT == SZ_BF16) {
                *reinterpret_cast<uint2 *>(row + 2 * wa) = make_uint2(pack_bf16(x[i][0], x[i][1]), pack_bf16(x[i][2], x[i][3]));
                *reinterpret_cast<uint2 *>(row + 2 * wb) = make_uint2(pack_bf16(x[i][4], x[i][5]), pack_bf16(x[i][6], x[i][7]));
            } else {
                *reinterpret_cast<uint32_t *>(row + wa) = pack_e5m2(x[i][0], x[i][1]) | pack_e5m2(x[i][2], x[i][3]) << 16;
                *reinterpret_cast<uint32_t *>(row + wb) = pack_e5m2(x[i][4], x[i][5]) | pack_e5m2(x[i][6], x[i][7]) << 16;
            }
        } else {
            const HeadsRef &h = is_q ? p.q_out : p.k_out;
            uint8_t *row = h.p + token * h.ts + (is_q ? r : r - hq) * h.hs;
            *reinterpret_cast<uint2 *>(row + 2 * wa) = make_uint2(pack_bf16(x[i][0], x[i][1]), pack_bf16(x[i][2], x[i][3]));
            *reinterpret_cast<uint2 *>(row + 2 * wb) = make_uint2(pack_bf16(x[i][4], x[i][5]), pack_bf16(x[i][6], x[i][7]));
        }
    }
}

template <int LG, int N, bool APPEND, int DT, bool WIDE>
sz_status run(RopeParams p, cudaStream_t stream) {
    const uint32_t hq = p.q.heads, hk = p.k.heads, hv = APPEND ? p.v.heads : 0;
    p.chunks = fast_div(WIDE ? (hq + N - 1) / N + (hk + N - 1) / N + (hv + N - 1) / N : (hq + hk + hv + N - 1) / N);
    const uint64_t groups = uint64_t(p.tokens) * p.chunks.d;
    const uint64_t grid = cdiv(groups, kRopeThreads / LG);
    if (grid > 0x7fffffffull) return SZ_ERR_INVALID_ARG;
    cudaError_t e;
    if constexpr (WIDE) e = launch_pdl(rope_wide_kernel<LG, N, APPEND, DT>, unsigned(grid), kRopeThreads, 0, stream, p);
    else e = launch_pdl(rope_kernel<LG, N, APPEND, DT>, unsigned(grid), kRopeThreads, 0, stream, p);
    return e == cudaSuccess ? SZ_OK : SZ_ERR_CUDA;
}

// Lanes to a row, W elements to a lane.
template <bool APPEND, int DT, bool WIDE>
sz_status run_dim(const RopeParams &p, bool few, cudaStream_t stream) {
    constexpr int W = WIDE ? 16 : 8;
    if (p.head_dim <= 64) return few ? run<64 / W, 1, APPEND, DT, WIDE>(p, stream) : run<64 / W, 4, APPEND, DT, WIDE>(p, stream);
    if (p.head_dim <= 128)
        return few ? run<128 / W, 1, APPEND, DT, WIDE>(p, stream) : run<128 / W, 4, APPEND, DT, WIDE>(p, stream);
    return few ? run<256 / W, 1, APPEND, DT, WIDE>(p, stream) : run<256 / W, 4, APPEND, DT, WIDE>(p, stream);
}

template <bool WIDE>
sz_status run_kind(const RopeParams &p, bool append, int dtype, bool few, cudaStream_t stream) {
    if (!append) return run_dim<false, SZ_BF16, WIDE>(p, few, stream);
    return dtype == SZ_BF16 ? run_dim<true, SZ_BF16, WIDE>(p, few, stream) : run_dim<true, SZ_FP8_E5M2, WIDE>(p, few, stream);
}

}  // namespace

sz_status launch_rope(const RopeParams &p, bool append, int dtype, int num_sms, cudaStream_t stream) {
    // Few rows: one row to a group, so that they spread over the SMs; otherwise four, whose
    // loads are under way together and share a position's cosines and sines.
    const uint64_t rows = uint64_t(p.tokens) * (p.q.heads + p.k.heads + p.v.heads);
    const bool few = rows < uint64_t(num_sms) * 128;
    // halves of the rotated part in 16-byte runs, or (rot 8, 24, 40, ...) in runs of 8
    return p.rope.rot % 16 == 0 ? run_kind<true>(p, append, dtype, few, stream)
                                : run_kind<false>(p, append, dtype, few, stream);
}

}  // namespace sz
