// sz_attn.cu -- attention of few rows over a paged cache (sz_attn_paged), and
// the choice between this kernel and the tensor-memory one (sz_attn_tc.cu).
//
//   x = scale * q . k,  m = max x,  p = exp(x - m),  o = sum p v / sum p
// in one pass: m and sum p are kept for what has been seen, and what has been
// summed is rescaled when m grows.  Scores, statistics and sums are floats; p
// is rounded to the type that v is multiplied in (bf16, or fp16 for an E5M2
// cache).
//
// Measured: 64 sequences of up to 8192 places, 32 heads on 8 of 128: 240 us, 5.5
// TB/s, 0.85 of a plain copy's rate; one sequence of 131,072 places, 32 heads on
// 4 in E5M2: 53 us, of which about 25 are fixed (the deal, the first pages' ids
// and rows, the joining of 111 parts a head); one token over 777 places: 10 us,
// all of it the latency of those steps.
//
// With few rows to a key the cache's bytes are the bound.  Each warp streams
// its own places, 16 at a time, through its own ring of asynchronous copies
// and waits for no other warp until its part of the tile is done; four warps
// of a CTA take turns over a tile's places, and CTAs split long tiles.
//
// E5M2 is the upper byte of fp16, so its keys and values become fp16 by a byte
// permute.  Queries are rounded to fp16 behind a power of two for each row
// that brings the row's largest below 2^14: three bits more than bf16 holds.
#include "sz_attn.cuh"

namespace sz {
namespace {

constexpr int kSplitThreads = 128;
constexpr int kSplitWarps = kSplitThreads / 32;
constexpr int kPlaces = 16;  // places of a warp's step
constexpr int kAhead = 4;
constexpr int kSplitBlock = 64;
constexpr int kSplitExtra = 0;

// Parts of a tile that a CTA joins at a time: up to kJoinMost at once, more of
// them in groups first.
constexpr int kJoinMost = 32;
__device__ __forceinline__ uint32_t join_group(uint32_t parts) { return parts <= 16 ? parts : (parts <= 144 ? 12 : 24); }
static_assert(kAttnCtas <= 24 * kJoinMost, "groups");

template <int DT, int DP, int MT>
struct SplitCfg {
    static constexpr int EB = DT == SZ_BF16 ? 2 : 1;
    static constexpr int TR = 16 * MT;
    static constexpr int PITCH = DP * EB + 16;             // odd in 16-byte units: rows fall on different banks
    static constexpr int STAGE = 2 * kPlaces * PITCH;      // keys, then values
    static constexpr int STAGES = DP > 128 ? 2 : (DP > 64 ? 3 : 5);
    static constexpr int RING = kSplitWarps * STAGES * STAGE;
    static constexpr int QPITCH = DP * 2 + 16;
    static constexpr int OPITCH = DP + 4;                  // floats
    static constexpr int JOIN = kSplitWarps * TR * OPITCH * 4;
    static constexpr int WEIGHTS = kJoinMost * TR * 4;
    static constexpr int MAIN = RING > JOIN ? (RING > WEIGHTS ? RING : WEIGHTS) : (JOIN > WEIGHTS ? JOIN : WEIGHTS);
    static constexpr int SMEM = MAIN + TR * QPITCH;
    // what the softmax's powers are multiplied by: small ones keep their bits in fp16
    static constexpr float RAISE = DT == SZ_BF16 ? 0.f : 8.f;
    // how far a row's largest score may grow, as a power of two, before its sums are rescaled
    static constexpr float SLACK = DT == SZ_BF16 ? 8.f : 6.f;
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t (&r)[4], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(a) : "memory");
}
__device__ __forceinline__ void ldsm2_t(uint32_t (&r)[2], uint32_t a) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0,%1}, [%2];"
                 : "=r"(r[0]), "=r"(r[1]) : "r"(a) : "memory");
}
template <int DT>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (DT == SZ_BF16)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
                     : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// Weights in the 16 bits that the tensor cores multiply: of at most 1 (or 2^SLACK
// behind a maximum that lags), each off by half a step, 2^-8 in bf16 and 2^-11 in
// fp16, of itself.  The tensor cores take no factors of 32 bits (tf32
// has fp16's 11, at half the rate), and the output is rounded to bf16.  Sums of
// weights are taken before the rounding.
template <int DT>
__device__ __forceinline__ uint32_t pack_p(float lo, float hi) {
    return DT == SZ_BF16 ? pack_bf16(lo, hi) : pack_f16(lo, hi);
}

template <int DT, int DP, int MT>
__global__ void __launch_bounds__(kSplitThreads) attn_split_kernel(const __grid_constant__ AttnParams p) {
    using C = SplitCfg<DT, DP, MT>;
    constexpr int TR = C::TR;
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ WorkScratch<kSplitThreads> s_work;
    __shared__ float s_m[kSplitWarps][TR], s_l[kSplitWarps][TR], s_rs[TR], s_M[TR], s_L[TR];
    __shared__ uint32_t s_edge, s_last;

    pdl_wait();
    pdl_launch_dependents();
    const uint32_t tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const uint32_t d = p.cache.head_dim, G = p.group.d;
    const uint32_t ksteps = d / 16;
    uint8_t *s_q = smem + C::MAIN;
    const uint32_t ring = smem_u32(smem) + warp * (C::STAGES * C::STAGE);
    const uint32_t qaddr = smem_u32(s_q);

    // copies: a group of lanes has a row, a lane one 16-byte piece of it
    constexpr uint32_t LPR = DP * C::EB / 16;             // 4, 8, 16 or 32 lanes to a row
    constexpr uint32_t ROWS = 32 / LPR;
    const uint32_t piece = lane % LPR, row0 = lane / LPR;
    const bool has_piece = piece * 16 < d * C::EB;
    const bool one_page = p.cache.page_tokens.d % kPlaces == 0;  // a step lies in one page
    if (tid == 0) s_edge = 0;  // whether an edge held a value that is not finite

    Work w;
    if (!work_begin<kSplitThreads, TR, kSplitBlock, kSplitExtra>(p, s_work, w)) return;
    for (;;) {
        const Part t = work_part<TR, kSplitBlock, kSplitExtra>(p, w, blockIdx.x);
        const int32_t *ids = p.cache.table + uint64_t(w.seq) * p.cache.table_stride;
        // places of this CTA's part, whole steps of 16 (lo down to a step's start)
        const uint32_t part_lo = max((t.block0 + t.from) * kSplitBlock, t.r.lo / kPlaces * kPlaces);
        const uint32_t part_hi = min((t.block0 + t.to) * kSplitBlock, t.r.hi);
        const uint32_t steps = part_hi > part_lo ? (part_hi - part_lo + kPlaces - 1) / kPlaces : 0;
        const uint64_t head_off = uint64_t(w.head) * d * C::EB + piece * 16;

        // The page id of the place that lane & 15 has in a step (-1: no place), and its offset.
        // Ids are asked for kAhead steps before their offsets are needed: a step that waited
        // for its own would take the load's latency.
        auto page_id = [&](uint32_t step) -> int32_t {
            if (one_page) return step < steps ? __ldg(ids + div_by(part_lo + step * kPlaces, p.cache.page_tokens)) : -1;
            const uint32_t at = part_lo + step * kPlaces + (lane & 15);
            return step < steps && at >= t.r.lo && at < part_hi ? __ldg(ids + div_by(at, p.cache.page_tokens)) : -1;
        };
        auto offset = [&](uint32_t step, int32_t id) -> uint64_t {
            const uint32_t at = part_lo + step * kPlaces + (lane & 15);
            if (step >= steps || at < t.r.lo || at >= part_hi) return kBadOffset;
            const uint32_t page = div_by(at, p.cache.page_tokens);
            if (id < 0 || uint64_t(id) >= p.cache.pool_pages) {
                set_error(p.ctl, SZ_ERR_INVALID_ARG, page);
                return kBadOffset;
            }
            return uint64_t(id) * p.cache.page_bytes + uint64_t(at - page * p.cache.page_tokens.d) * p.cache.row_bytes;
        };
        auto issue = [&](uint32_t slot, uint64_t off) {
            const uint32_t dst = ring + slot * C::STAGE + row0 * C::PITCH + piece * 16;
#pragma unroll
            for (uint32_t r = 0; r < kPlaces; r += ROWS) {
                const uint64_t o = __shfl_sync(0xffffffffu, off, int(r + row0));
                if (!has_piece) continue;
                const bool in = o != kBadOffset;
                const uint64_t a = in ? o + head_off : 0;
                cp_async16(dst + r * C::PITCH, p.cache.k + a, in);
                cp_async16(dst + (kPlaces + r) * C::PITCH, p.cache.v + a, in);
            }
        };

        // fill the ring
        // a step's copies: without a look at each place where all are seen and in one page
        auto issue_step = [&](uint32_t slot, uint32_t step, int32_t id) {
            const uint32_t at = part_lo + step * kPlaces;
            if (one_page && at >= t.r.lo && at + kPlaces <= part_hi && id >= 0 && uint64_t(id) < p.cache.pool_pages) {
                const uint32_t token = at - div_by(at, p.cache.page_tokens) * p.cache.page_tokens.d;
                const uint64_t from =
                    uint64_t(id) * p.cache.page_bytes + uint64_t(token + row0) * p.cache.row_bytes + head_off;
                const uint32_t dst = ring + slot * C::STAGE + row0 * C::PITCH + piece * 16;
                if (!has_piece) return;
                const uint8_t *k = p.cache.k + from, *v = p.cache.v + from;
#pragma unroll
                for (uint32_t r = 0; r < kPlaces; r += ROWS) {
                    cp_async16(dst + r * C::PITCH, k + r * p.cache.row_bytes, true);
                    cp_async16(dst + (kPlaces + r) * C::PITCH, v + r * p.cache.row_bytes, true);
                }
            } else {
                issue(slot, offset(step, id));
            }
        };
        int32_t id[kAhead];
        {
            int32_t first[C::STAGES - 1];
#pragma unroll
            for (int i = 0; i < C::STAGES - 1; ++i) first[i] = page_id(warp + i * kSplitWarps);
#pragma unroll
            for (int i = 0; i < kAhead; ++i) id[i] = page_id(warp + (C::STAGES - 1 + i) * kSplitWarps);
#pragma unroll
            for (int i = 0; i < C::STAGES - 1; ++i) {
                const uint32_t step = warp + i * kSplitWarps;
                if (step < steps) issue_step(i, step, first[i]);
                cp_commit();
            }
        }

        // queries of the tile's rows; rows behind the last are zeros
        constexpr uint32_t QP = DP / 8;                    // lanes to a row
        for (uint32_t r = tid / QP; r < TR; r += kSplitThreads / QP) {
            const uint32_t c = tid % QP;
            uint4 v = make_uint4(0, 0, 0, 0);
            if (r < t.rows && c * 8 < d) {
                const uint32_t i = div_by(t.r0 + r, p.group);
                v = *reinterpret_cast<const uint4 *>(p.q.p + uint64_t(t.s.q0 + i) * p.q.ts +
                                                     uint64_t(w.head * G + (t.r0 + r - i * G)) * p.q.hs + c * 16);
            }
            if constexpr (DT == SZ_FP8_E5M2) {
                uint32_t x[4] = {v.x, v.y, v.z, v.w};
                float top = 0.f;
#pragma unroll
                for (int j = 0; j < 4; ++j) top = fmaxf(top, fmaxf(fabsf(bf16_lo(x[j])), fabsf(bf16_hi(x[j]))));
#pragma unroll
                for (int o = QP / 2; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                int e = 0;
                if (top > 0.f && top < INFINITY) e = min(13 - (int(__float_as_uint(top) >> 23) - 127), 120);
                const float up = __uint_as_float(uint32_t(127 + e) << 23);
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = pack_f16(bf16_lo(x[j]) * up, bf16_hi(x[j]) * up);
                v = make_uint4(x[0], x[1], x[2], x[3]);
                if (c == 0) s_rs[r] = __uint_as_float(uint32_t(127 - e) << 23);
            }
            *reinterpret_cast<uint4 *>(s_q + r * C::QPITCH + c * 16) = v;
        }
        __syncthreads();

        // this lane's rows: lane / 4 and + 8 of each 16
        uint32_t lo[MT][2], hi[MT][2];
        float sc[MT][2], m[MT][2], l[MT][2], o[MT][DP / 8][4];
        const Range all = seen_by_all(p, t);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t r = i * 16 + h * 8 + lane / 4;
                Range rr{0, 0};
                if (r < t.rows) rr = token_range(p, t.s, div_by(t.r0 + r, p.group));
                lo[i][h] = rr.lo;
                hi[i][h] = rr.hi;
                sc[i][h] = p.scale_log2 * (DT == SZ_BF16 ? 1.f : s_rs[r]);
                m[i][h] = -INFINITY;
                l[i][h] = 0.f;
            }
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int n = 0; n < DP / 8; ++n) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;

        uint32_t slot = 0;
        for (uint32_t step = warp; step < steps; step += kSplitWarps) {
            // refill the slot that the last step freed, then wait for this one's
            {
                const uint32_t ahead = step + (C::STAGES - 1) * kSplitWarps;
                const uint32_t to = slot == 0 ? C::STAGES - 1 : slot - 1;
                if (ahead < steps) issue_step(to, ahead, id[0]);
                cp_commit();
#pragma unroll
                for (int i = 1; i < kAhead; ++i) id[i - 1] = id[i];
                id[kAhead - 1] = page_id(ahead + kAhead * kSplitWarps);
            }
            cp_wait<C::STAGES - 1>();
            __syncwarp();
            const uint32_t kb = ring + slot * C::STAGE, vb = kb + kPlaces * C::PITCH;
            float x[MT][2][4];
#pragma unroll
            for (int i = 0; i < MT; ++i)
#pragma unroll
                for (int n = 0; n < 2; ++n) x[i][n][0] = x[i][n][1] = x[i][n][2] = x[i][n][3] = 0.f;
            if constexpr (DT == SZ_BF16) {
                const uint32_t ka = kb + ((lane >> 4) * 8 + (lane & 7)) * C::PITCH + ((lane >> 3) & 1) * 16;
                const uint32_t qa = qaddr + ((lane >> 3 & 1) * 8 + (lane & 7)) * C::QPITCH + (lane >> 4) * 16;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    if (k >= ksteps) break;
                    uint32_t b[4];
                    ldsm4(b, ka + k * 32);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        uint32_t a[4];
                        ldsm4(a, qa + i * 16 * C::QPITCH + k * 32);
                        mma16<DT>(x[i][0], a, b[0], b[1]);
                        mma16<DT>(x[i][1], a, b[2], b[3]);
                    }
                }
            } else {
                // a lane's four bytes in a row are its two pairs of the step's 16: the same
                // order of the head's elements on both sides
                const uint32_t ka = kb + (lane >> 2) * C::PITCH + (lane & 3) * 4;
                const uint32_t qa = qaddr + (lane >> 2) * C::QPITCH + (lane & 3) * 8;
#pragma unroll
                for (int k = 0; k < DP / 16; ++k) {
                    if (k >= ksteps) break;
                    const uint32_t w0 = lds_u32(ka + k * 16), w1 = lds_u32(ka + 8 * C::PITCH + k * 16);
                    const uint32_t b00 = prmt(w0, 0, 0x1404), b01 = prmt(w0, 0, 0x3424);
                    const uint32_t b10 = prmt(w1, 0, 0x1404), b11 = prmt(w1, 0, 0x3424);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        const uint2 q0 = lds_u64(qa + i * 16 * C::QPITCH + k * 32);
                        const uint2 q1 = lds_u64(qa + (i * 16 + 8) * C::QPITCH + k * 32);
                        const uint32_t a[4] = {q0.x, q1.x, q0.y, q1.y};
                        mma16<DT>(x[i][0], a, b00, b01);
                        mma16<DT>(x[i][1], a, b10, b11);
                    }
                }
            }
            const uint32_t at = part_lo + step * kPlaces;
            const bool whole = at >= all.lo && at + kPlaces <= all.hi;
            if (has_edges(all, max(at, t.r.lo), min(at + kPlaces, part_hi))) {
#pragma unroll 1
                for (uint32_t r = row0; r < kPlaces; r += ROWS) {
                    const uint32_t c = at + r, a = vb + r * C::PITCH + piece * 16;
                    if (!has_piece || (c >= all.lo && c < all.hi)) continue;
                    uint4 v = lds_u128(a);
                    if (make_finite<DT>(v)) {
                        sts_u128(a, v);
                        s_edge = 1;
                    }
                }
                __syncwarp();
            }
            uint32_t pa[MT][4];
#pragma unroll
            for (int i = 0; i < MT; ++i) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    if (h == 1 && t.rows <= 8u + 16u * i) {  // no rows there
                        pa[i][1] = pa[i][3] = 0;
                        continue;
                    }
                    float e[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        e[j] = x[i][j >> 1][h * 2 + (j & 1)] * sc[i][h];
                        if (!whole) {
                            const uint32_t c = at + (j >> 1) * 8 + (lane & 3) * 2 + (j & 1);
                            if (c < lo[i][h] || c >= hi[i][h]) e[j] = -INFINITY;
                        }
                    }
                    float top = fmaxf(fmaxf(e[0], e[1]), fmaxf(e[2], e[3]));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                    top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                    const bool grows = top > m[i][h] + C::SLACK;
                    float c = 1.f;
                    if (__any_sync(0xffffffffu, grows)) {
                        if (grows) c = exp2_fast(m[i][h] - top), m[i][h] = top;
#pragma unroll
                        for (int n = 0; n < DP / 8; ++n) {
                            o[i][n][h * 2] *= c;
                            o[i][n][h * 2 + 1] *= c;
                        }
                    }
                    const float base = C::RAISE - (m[i][h] == -INFINITY ? 0.f : m[i][h]);
#pragma unroll
                    for (int j = 0; j < 4; ++j) e[j] = exp2_fast(e[j] + base);
                    l[i][h] = l[i][h] * c + ((e[0] + e[1]) + (e[2] + e[3]));
                    pa[i][h] = pack_p<DT>(e[0], e[1]);
                    pa[i][2 + h] = pack_p<DT>(e[2], e[3]);
                }
            }
            if constexpr (DT == SZ_BF16) {
                const uint32_t va = vb + ((lane >> 3 & 1) * 8 + (lane & 7)) * C::PITCH + (lane >> 4) * 16;
#pragma unroll
                for (int n = 0; n < DP / 16; ++n) {
                    if (n >= ksteps) break;
                    uint32_t b[4];
                    ldsm4_t(b, va + n * 32);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        mma16<DT>(o[i][2 * n], pa[i], b[0], b[1]);
                        mma16<DT>(o[i][2 * n + 1], pa[i], b[2], b[3]);
                    }
                }
            } else {
                // a transposed 16-bit unit is two neighbouring elements: the even ones make one
                // product's columns, the odd ones the next one's
                const uint32_t va = vb + (lane & 15) * C::PITCH;
#pragma unroll
                for (int n = 0; n < DP / 16; ++n) {
                    if (n >= ksteps) break;
                    uint32_t b[2];
                    ldsm2_t(b, va + n * 16);
                    const uint32_t e0 = prmt(b[0], 0, 0x2404), e1 = prmt(b[1], 0, 0x2404);
                    const uint32_t f0 = prmt(b[0], 0, 0x3414), f1 = prmt(b[1], 0, 0x3414);
#pragma unroll
                    for (int i = 0; i < MT; ++i) {
                        mma16<DT>(o[i][2 * n], pa[i], e0, e1);
                        mma16<DT>(o[i][2 * n + 1], pa[i], f0, f1);
                    }
                }
            }
            __syncwarp();
            slot = slot + 1 == C::STAGES ? 0 : slot + 1;
        }
        cp_wait<0>();

        // join the warps
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 1);
                l[i][h] += __shfl_xor_sync(0xffffffffu, l[i][h], 2);
                if ((lane & 3) == 0) {
                    s_m[warp][i * 16 + h * 8 + lane / 4] = m[i][h];
                    s_l[warp][i * 16 + h * 8 + lane / 4] = l[i][h];
                }
            }
        __syncthreads();
        if (tid < TR) {
            float M = -INFINITY, L = 0.f;
            for (int v = 0; v < kSplitWarps; ++v) M = fmaxf(M, s_m[v][tid]);
            const float safe = M == -INFINITY ? 0.f : M;
            for (int v = 0; v < kSplitWarps; ++v) L += s_l[v][tid] * exp2_fast(s_m[v][tid] - safe);
            s_M[tid] = M;
            s_L[tid] = L;
        }
        __syncthreads();
        float *s_o = reinterpret_cast<float *>(smem);
#pragma unroll
        for (int i = 0; i < MT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t r = i * 16 + h * 8 + lane / 4;
                const float M = s_M[r], f = M == -INFINITY ? 0.f : exp2_fast(m[i][h] - M);
                float *to = s_o + (warp * TR + r) * C::OPITCH;
                // a warp without places has nothing to add, and its factor may be 0 times nothing
#pragma unroll
                for (int n = 0; n < DP / 16; ++n) {
                    if (n >= ksteps) break;
                    const float a0 = o[i][2 * n][h * 2] * f, a1 = o[i][2 * n][h * 2 + 1] * f;
                    const float b0 = o[i][2 * n + 1][h * 2] * f, b1 = o[i][2 * n + 1][h * 2 + 1] * f;
                    if constexpr (DT == SZ_BF16) {
                        *reinterpret_cast<float2 *>(to + n * 16 + (lane & 3) * 2) = make_float2(a0, a1);
                        *reinterpret_cast<float2 *>(to + n * 16 + 8 + (lane & 3) * 2) = make_float2(b0, b1);
                    } else {
                        *reinterpret_cast<float4 *>(to + n * 16 + (lane & 3) * 4) = make_float4(a0, b0, a1, b1);
                    }
                }
            }
        __syncthreads();

        const bool whole_tile = t.c_first == t.c_last;
        const uint32_t quads = d / 4;
        float *part = p.part + uint64_t(part_slot(blockIdx.x, t)) * TR * (d + 2);
        auto finish = [&](uint32_t r, uint32_t c, float4 v, float M, float L) {
            const uint32_t i = div_by(t.r0 + r, p.group), head = w.head * G + (t.r0 + r - i * G);
            const float f = L == 0.f ? 0.f : 1.f / L;
            v.x *= f, v.y *= f, v.z *= f, v.w *= f;
            *reinterpret_cast<uint2 *>(p.out.p + uint64_t(t.s.q0 + i) * p.out.ts + uint64_t(head) * p.out.hs + c * 8) =
                make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            if (c == 0 && p.lse)
                p.lse[uint64_t(t.s.q0 + i) * p.q.heads + head] =
                    L == 0.f ? -INFINITY : kLn2 * (M - C::RAISE + log2f(L));
        };
        for (uint32_t e = tid; e < t.rows * quads; e += kSplitThreads) {
            const uint32_t r = e / quads, c = e - r * quads;
            float4 v = *reinterpret_cast<const float4 *>(s_o + r * C::OPITCH + c * 4);
#pragma unroll
            for (int k = 1; k < kSplitWarps; ++k) {
                const float4 a = *reinterpret_cast<const float4 *>(s_o + (k * TR + r) * C::OPITCH + c * 4);
                v.x += a.x, v.y += a.y, v.z += a.z, v.w += a.w;
            }
            if (s_edge) {
                float sum[4] = {v.x, v.y, v.z, v.w};
                add_not_finite<DT, 4>(p, w.seq, w.head, token_range(p, t.s, div_by(t.r0 + r, p.group)), all, part_lo,
                                      part_hi, c * 4, sum);
                v = make_float4(sum[0], sum[1], sum[2], sum[3]);
            }
            if (whole_tile) {
                finish(r, c, v, s_M[r], s_L[r]);
            } else {
                *reinterpret_cast<float4 *>(part + r * d + c * 4) = v;
                if (c == 0) {
                    part[TR * d + r] = s_M[r];
                    part[TR * d + TR + r] = s_L[r];
                }
            }
        }
        if (!whole_tile) {
            // Parts are joined by whoever comes last to them: of up to 16 at once, of more in
            // groups, and then the groups; one CTA that reads 111 parts takes 30 us.
            const uint32_t parts = t.c_last - t.c_first + 1, group = join_group(parts), mine = (blockIdx.x - t.c_first) / group;
            const uint32_t groups = (parts + group - 1) / group;
            // Whether this CTA is the last of n at a counter, which is then zero again.
            auto last_of = [&](uint32_t *counter, uint32_t n) {
                __threadfence();
                __syncthreads();
                if (tid == 0) {
                    s_last = atomicAdd(counter, 1u) == n - 1;
                    if (s_last) *counter = 0;
                }
                __syncthreads();
                __threadfence();
                return s_last != 0;
            };
            auto slot_of = [&](uint32_t k) { return p.part + uint64_t(part_slot(t.c_first + k, t)) * TR * (d + 2); };
            // Joins parts first, first + step, ... (n of them) to the result, or to the first one's place.
            auto join = [&](uint32_t first, uint32_t step, uint32_t n, bool result) {
                float *s_f = reinterpret_cast<float *>(smem);
                for (uint32_t r = warp; r < t.rows; r += kSplitWarps) {
                    const float *at = slot_of(first + min(lane, n - 1) * step) + TR * d + r;
                    const float m = lane < n ? __ldcg(at) : -INFINITY;
                    float M = m;
#pragma unroll
                    for (int v = 16; v > 0; v >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, v));
                    const float f = lane < n ? exp2_fast(m - (M == -INFINITY ? 0.f : M)) : 0.f;
                    float L = lane < n ? f * __ldcg(at + TR) : 0.f;
                    s_f[lane * TR + r] = f;
#pragma unroll
                    for (int v = 16; v > 0; v >>= 1) L += __shfl_xor_sync(0xffffffffu, L, v);
                    if (lane == 0) s_M[r] = M, s_L[r] = L;
                }
                __syncthreads();
                float *to = slot_of(first);
                for (uint32_t e = tid; e < t.rows * quads; e += kSplitThreads) {
                    const uint32_t r = e / quads, c = e - r * quads;
                    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 12
                    for (uint32_t k = 0; k < n; ++k) {
                        const float f = s_f[k * TR + r];
                        const float4 a = __ldcg(reinterpret_cast<const float4 *>(slot_of(first + k * step) + r * d + c * 4));
                        v.x = fmaf(f, a.x, v.x), v.y = fmaf(f, a.y, v.y);
                        v.z = fmaf(f, a.z, v.z), v.w = fmaf(f, a.w, v.w);
                    }
                    if (result) {
                        finish(r, c, v, s_M[r], s_L[r]);
                    } else {
                        *reinterpret_cast<float4 *>(to + r * d + c * 4) = v;
                        if (c == 0) to[TR * d + r] = s_M[r], to[TR * d + TR + r] = s_L[r];
                    }
                }
            };
            uint32_t *counter = mine == 0 ? p.arrived + t.c_first : p.arrived + kAttnCtas + t.c_first + mine * group;
            if (last_of(counter, min(group, parts - mine * group))) {
                join(mine * group, 1, min(group, parts - mine * group), groups == 1);
                if (groups > 1 && last_of(p.arrived + 2 * kAttnCtas + t.c_first, groups)) join(0, group, groups, true);
            }
        }
        __syncthreads();
        if (!work_next<TR, kSplitExtra>(p, w, t)) break;
    }
}

template <int DT, int DP, int MT>
sz_status run(const AttnParams &p, int num_sms, cudaStream_t stream) {
    using C = SplitCfg<DT, DP, MT>;
    static std::atomic<int> cache[kMaxDevices];
    auto kern = attn_split_kernel<DT, DP, MT>;
    const int per_sm = resident_per_sm(reinterpret_cast<const void *>(kern), kSplitThreads, C::SMEM, cache);
    if (per_sm <= 0) return SZ_ERR_CUDA;
    const unsigned grid = unsigned(num_sms) * unsigned(per_sm < 3 ? per_sm : 3);
    return launch_pdl(kern, grid, kSplitThreads, C::SMEM, stream, p) == cudaSuccess ? SZ_OK : SZ_ERR_CUDA;
}

template <int DT>
sz_status run_dim(const AttnParams &p, int num_sms, cudaStream_t stream) {
    const uint32_t d = p.cache.head_dim;
    const uint64_t rows = cdiv(p.tokens, p.cache.seqs) * p.group.d;
    // Rows of a sequence and KV head, on average.  20 (8 sequences of 5 tokens, groups of 4,
    // 8192 places): 58 us here, 74 in tensor memory; 64 (4 of 16 tokens, 4096 places): 68 and 44;
    // one sequence of 16 tokens over 65,536: 232 and 82.  Wider heads' sums do not fit there twice.
    // It is the average of the table's rows, all that the host knows: one long chunk among many
    // rows of none or of one token goes the slow way (512 tokens over 4096 places: 53 us alone, 70
    // in a table of 63 rows, 386 in one of 64).
    if (d <= 128 && rows > 32) return launch_attn_tc(p, DT, num_sms, stream);
    if (d <= 64) return rows <= 16 ? run<DT, 64, 1>(p, num_sms, stream) : run<DT, 64, 2>(p, num_sms, stream);
    if (d <= 128) return rows <= 16 ? run<DT, 128, 1>(p, num_sms, stream) : run<DT, 128, 2>(p, num_sms, stream);
    return run<DT, 256, 1>(p, num_sms, stream);
}

}  // namespace

sz_status launch_attn(const AttnParams &p, int dtype, int num_sms, cudaStream_t stream) {
    return dtype == SZ_BF16 ? run_dim<SZ_BF16>(p, num_sms, stream) : run_dim<SZ_FP8_E5M2>(p, num_sms, stream);
}

}  // namespace sz
