// sz_rope.cu -- norm and rotation of query and key heads, to contiguous
// outputs (sz_qk_norm_rope) or, keys and values, into the pages of a cache
// (sz_kv_append_paged).
//
//   n_i = x_i * (1 / sqrt(mean(x^2) + eps)) * w_i
//   (a, b) -> (a cos - b sin, b cos + a sin) for the pairs of the first rot
//   elements; every product and sum is rounded to 32 bits by itself, and the
//   result once to the output's type.
//
// One element is read, turned and written: the bytes are the bound, and for a
// few tokens the latency of the dependent loads (sequence, length, page id).
#include "sz_ops.cuh"

namespace sz {
namespace {

constexpr int kRopeThreads = 256;

// Plain loads: the rows may be those that the call writes (in place, each lane
// writes the elements that it read).
__device__ __forceinline__ void load8(float (&x)[8], const uint8_t *a, const uint8_t *b) {
    const uint2 u = *reinterpret_cast<const uint2 *>(a), w = *reinterpret_cast<const uint2 *>(b);
    x[0] = bf16_lo(u.x), x[1] = bf16_hi(u.x), x[2] = bf16_lo(u.y), x[3] = bf16_hi(u.y);
    x[4] = bf16_lo(w.x), x[5] = bf16_hi(w.x), x[6] = bf16_lo(w.y), x[7] = bf16_hi(w.y);
}

// A group of LG lanes has one token and N of its head rows; a lane holds eight
// elements of a row: four of each half of the rotated part, or eight in order
// (interleaved pairs, and what is not rotated).
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

    bool ok = live;
    int64_t pos = 0;        // position of the rotation
    uint64_t place = kBadOffset;
    if constexpr (APPEND) {
        uint32_t seq = 0;
        for (int g = 0; g < 32 / LG; ++g) {  // one warp-wide search for each of its groups
            const uint32_t t = __shfl_sync(0xffffffffu, token, g * LG);
            const uint32_t s = warp_find_seq(p.cu_q, p.cache.seqs, t);
            if (lane / LG == g) seq = s;
        }
        ok = ok && seq < p.cache.seqs && token >= uint32_t(__ldg(p.cu_q));
        if (ok) {
            pos = int64_t(__ldg(p.kv_len + seq)) - (int64_t(__ldg(p.cu_q + seq + 1)) - int64_t(token));
            if (pos < 0 || pos >= int64_t(p.cache.capacity)) {
                if (l == 0) set_error(p.ctl, SZ_ERR_INVALID_ARG, token);
                ok = false;
            } else {
                place = place_offset(p.cache, p.ctl, p.cache.table + uint64_t(seq) * p.cache.table_stride,
                                     uint32_t(pos));
                ok = place != kBadOffset;
            }
        }
    }
    float cs[4] = {1.f, 1.f, 1.f, 1.f}, sn[4] = {0.f, 0.f, 0.f, 0.f};
    if (rot > 0 && ok) {
        if (p.rope.positions) pos = __ldg(p.rope.positions + token);
        if (pos < 0 || pos >= int64_t(p.rope.len)) {
            if (l == 0) set_error(p.ctl, SZ_ERR_INVALID_ARG, token);
            ok = false;
        } else if (turns) {
            const float4 c = __ldg(reinterpret_cast<const float4 *>(p.rope.table + uint64_t(pos) * rot + 4 * l));
            const float4 s = __ldg(reinterpret_cast<const float4 *>(p.rope.table + uint64_t(pos) * rot + half + 4 * l));
            cs[0] = c.x, cs[1] = c.y, cs[2] = c.z, cs[3] = c.w;
            sn[0] = s.x, sn[1] = s.y, sn[2] = s.z, sn[3] = s.w;
        }
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
                const float rs = rsqrtf(ss / float(d) + p.eps);
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

template <int LG, int N, bool APPEND, int DT>
sz_status run(RopeParams p, cudaStream_t stream) {
    const uint32_t rows = p.q.heads + p.k.heads + (APPEND ? p.v.heads : 0);
    p.chunks = fast_div((rows + N - 1) / N);
    const uint64_t groups = uint64_t(p.tokens) * p.chunks.d;
    const uint64_t grid = cdiv(groups, kRopeThreads / LG);
    if (grid > 0x7fffffffull) return SZ_ERR_INVALID_ARG;
    return launch_pdl(rope_kernel<LG, N, APPEND, DT>, unsigned(grid), kRopeThreads, 0, stream, p) == cudaSuccess
               ? SZ_OK
               : SZ_ERR_CUDA;
}

template <bool APPEND, int DT>
sz_status run_dim(const RopeParams &p, bool few, cudaStream_t stream) {
    if (p.head_dim <= 64) return few ? run<8, 1, APPEND, DT>(p, stream) : run<8, 4, APPEND, DT>(p, stream);
    if (p.head_dim <= 128) return few ? run<16, 1, APPEND, DT>(p, stream) : run<16, 4, APPEND, DT>(p, stream);
    return few ? run<32, 1, APPEND, DT>(p, stream) : run<32, 4, APPEND, DT>(p, stream);
}

}  // namespace

sz_status launch_rope(const RopeParams &p, bool append, int dtype, int num_sms, cudaStream_t stream) {
    // few rows: one row to a group, so that they spread over the SMs
    const uint64_t rows = uint64_t(p.tokens) * (p.q.heads + p.k.heads + p.v.heads);
    const bool few = rows < uint64_t(num_sms) * 128;
    if (!append) return run_dim<false, SZ_BF16>(p, few, stream);
    return dtype == SZ_BF16 ? run_dim<true, SZ_BF16>(p, few, stream) : run_dim<true, SZ_FP8_E5M2>(p, few, stream);
}

}  // namespace sz
