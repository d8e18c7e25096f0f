// sz_attn_tc.cu -- attention of many rows over a paged cache (sz_attn_paged) on
// the fifth-generation tensor cores.
//
//   x = scale * q . k,  p = exp(x - m),  o = sum p v / sum p
//
// A CTA takes 256 rows of one sequence and KV head, as two tiles of 128, and
// goes over their places in blocks of 128.  Scores, p and the sums of p v stay
// in tensor memory: per tile 128 columns of scores, which p overwrites in 16
// bits, and 128 columns of sums.  The roles:
//   warps 0-3, 4-7  softmax of the first and the second tile, a thread a row:
//                   a row's maximum and sum need no exchange between threads
//   warps 8-11      keys and values into shared memory
//   warps 12, 13    issue the products of a tile: p v, in two halves as p comes,
//                   then q k' of the next block; the other tile's products run
//                   while this one's softmax does
//   warps 14, 15    queries into shared memory: a tile's as soon as its last
//                   product with the ones before is done; values that are not
//                   finite out of the products (sz_attn.cuh)
// m is the largest score so far only to within 2^SLACK: the sums are rescaled
// (through registers) when a row's maximum has grown by more, so that most
// blocks leave them where they are.
//
// Measured, with other inputs from call to call: 2048 tokens over 8192 places, 32
// heads on 8 of 128: 260 us, 0.92 PFLOP/s; two 1024-token prompts of 32 heads of 80:
// 40 us; five ragged chunks of up to 700 tokens, window 1024, 32 heads on 4 in
// E5M2: 82 us.
//
// What bounds it: a block of 256 rows and heads of 128 is 2048 clocks of matrix
// products and 2048 clocks of ex2 (16 a clock), if each tile's chain (scores,
// softmax, products) takes no longer.  It does: about 3500 clocks, 230 for the
// scores to registers, 1700 for the softmax, 1000 for the products behind it and
// the rest for turns; the tensor and ex2 pipes are each busy half of the time.
// Short prompts pay for their tiles' starts and ends, 4 to 6 us for each part
// that a CTA has of a tile.  Blocks of 64 places with two buffers of
// scores have shorter chains, but q k' of 64 columns reads 6 KB of shared memory
// in what would be 32 clocks, and takes 48.
//
// Keys and values come by tensor copies of 8 to 128 rows of a page, where pages
// are a multiple of 8 tokens and all of the block is seen.  Other blocks, the
// ends of what is seen among them, are fetched row by row by 16-byte
// asynchronous copies, with zeros for places that nobody sees.  Both bring the
// swizzled layout that the products read.  (Row by row, the issue of a block's
// 64 KB takes four warps 1.2 us, as long as its products.)
//
// An E5M2 cache's rows come as they are and are spread to fp16 (E5M2 is fp16's
// upper byte) on their way to that layout; queries are then fp16 too, behind a
// power of two for each row that brings the row's largest below 2^14.
//
// A tile that a few CTAs share is joined by the last of them; one that many
// share (long contexts of few rows) by a second kernel, which starts as the first
// one ends and spreads the sums over all SMs.
#include <cuda.h>

#include "sz_attn.cuh"

namespace sz {
namespace {

// A wait's limit, 2 s, and how many polls lie between two looks at the clock and at
// whether another role has given up.  A copy of the library that tests giving up
// sets both otherwise (one poll: of the kind that does not suspend the thread).
#ifndef SZ_ATTN_WAIT_NS
#define SZ_ATTN_WAIT_NS 2000000000ull
#endif
#ifndef SZ_ATTN_POLLS
#define SZ_ATTN_POLLS 64
#endif
// What is under way when a CTA leaves is waited for, whether or not it has given up:
// microseconds, unless another warp's arrival at the same barrier never comes.
constexpr uint64_t kLandLimitNs = 5000000ull;  // 5 ms

constexpr int kTcThreads = 512;
constexpr int kTcRows = 256;
constexpr int kTcBlock = 128;
// A tile's fixed costs in blocks.  0, 1, 2, 3, 4 took, where tiles are cut: three
// 2000-token prompts, 32 heads on 8 of 128: 164, 151, 142, 143, 144 us; four of 1500:
// 136, 126, 123, 125, 126; 300 tokens over 4000 places: 61, 54, 53, 53, 53; 2048 over
// 8192: 231, 227, 228, 228, 231.
constexpr int kTcExtra = 2;
constexpr uint32_t kFewParts = 4;             // a tile of so many parts is joined by the last of them
constexpr uint32_t kQPanel = 128 * 128;       // bytes of 128 rows of 64 16-bit elements
constexpr uint32_t kPanel = kTcBlock * 128;   // of a block's rows
// registers of a softmax thread and of the others: 256 * 192 + 256 * 64 = 512 * 128,
// what the CTA is launched with
#define SZ_TC_REGS_SOFTMAX "192"
#define SZ_TC_REGS_OTHER "64"

template <int DT, int DP>
struct TcCfg {
    static constexpr uint32_t EB = DT == SZ_BF16 ? 2 : 1;
    static constexpr uint32_t PANELS = DP / 64;
    static constexpr uint32_t QTILE = PANELS * kQPanel;
    static constexpr uint32_t STAGE = PANELS * kPanel;       // a block's keys or values
    static constexpr uint32_t STAGES = (DT == SZ_BF16 ? 10 : 6) / PANELS;
    static constexpr uint32_t RAW = kTcBlock * DP;           // E5M2: as they come
    static constexpr uint32_t RAWS = (DT == SZ_BF16 ? 0 : 8) / PANELS;
    static constexpr uint32_t RING_AT = 2 * QTILE;           // behind the queries
    static constexpr uint32_t RAW_AT = RING_AT + STAGES * STAGE;
    static constexpr uint32_t AUX_AT = RAW_AT + RAWS * RAW;
    static constexpr uint32_t SMEM = AUX_AT + 1024 + 1024;   // barriers and exponents; slack to align the base
    static_assert(SMEM <= 232448, "shared memory");
    static_assert(sizeof(WorkScratch<kTcThreads>) <= STAGES * STAGE, "the scratch lies in the ring");
    // p's factor 2^RAISE keeps small weights among fp16's normal numbers; 2^(RAISE + SLACK) is in its range
    static constexpr float RAISE = DT == SZ_BF16 ? 0.f : 8.f;
    static constexpr float SLACK = DT == SZ_BF16 ? 8.f : 6.f;
};

struct TcAux {
    uint64_t full[10], empty[10];
    uint64_t edge_here[10];  // values of a block with edges have come, to be looked at before they are `full`
    uint64_t raw_full[8], raw_empty[8];
    uint64_t q_full[2], q_empty[2], q_here[2];  // (q_here: E5M2, queries as they come, for the softmax's threads to make fp16)
    uint64_t s_full[2], p_full[2][2];  // a tile's scores; the halves of its weights
    uint64_t o_full[2];                // a tile's sums, at the end of a part
    uint64_t turn[2];                  // a tile's turn at ex2
    uint64_t drain[2];
    uint32_t tmem, abort;
    uint32_t edge;  // an edge held a value that is not finite
    uint16_t order[kFewTiles];
};
static_assert(sizeof(TcAux) <= 1024, "aux");

// What a CTA leaves for the joining kernel: the tile that it shares with later
// CTAs only.
struct TcDesc {
    Work join;
    uint32_t joins;  // there is one
    uint32_t pad;
};
static_assert(sizeof(TcDesc) * kMaxSms <= kDescBytes, "descriptors");

__device__ __forceinline__ bool bar_poll(uint64_t *bar, uint32_t parity) {
    if constexpr (SZ_ATTN_POLLS > 1) return mbar_try_wait(bar, parity);
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\tmbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return ok != 0;
}

// Waits are bounded: after the limit the CTA gives up (every role then leaves
// its loop) and the error word says so.
__device__ __forceinline__ bool bar_wait(uint64_t *bar, uint32_t parity, TcAux *aux, uint32_t *ctl, uint64_t limit) {
    if (bar_poll(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t i = 1;; ++i) {
        if (bar_poll(bar, parity)) return true;
        if (i % SZ_ATTN_POLLS == 0) {
            if (*reinterpret_cast<volatile uint32_t *>(&aux->abort)) return false;
            if (global_ns() - t0 > limit) {
                *reinterpret_cast<volatile uint32_t *>(&aux->abort) = 1;
                set_error(ctl, SZ_ERR_TIMEOUT, blockIdx.x);
                return false;
            }
        }
    }
}
// All lanes wait, and go on together.
__device__ __forceinline__ bool warp_wait(uint64_t *bar, uint32_t parity, TcAux *aux, const AttnParams &p) {
    return __all_sync(0xffffffffu, bar_wait(bar, parity, aux, p.ctl, p.wait_ns));
}
__device__ __forceinline__ void bar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
// One box of a tensor copy: elements x.., a head, rows from `token` of a page.
__device__ __forceinline__ void tensor_g2s(uint32_t dst, const CUtensorMap *map, uint32_t x, uint32_t head, uint32_t token,
                                           uint32_t page, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(map), "r"(x), "r"(head), "r"(token), "r"(page), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void tensor3_g2s(uint32_t dst, const CUtensorMap *map, uint32_t x, uint32_t y, uint32_t z,
                                            uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(smem_u32(bar))
        : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ------------------------------------------------------------ tensor memory

__device__ __forceinline__ void tc_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t *bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}

__device__ __forceinline__ bool elect_one() {
    uint32_t yes;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
    return yes != 0;
}

#define SZ_R4(r, i) "=r"(r[i]), "=r"(r[i + 1]), "=r"(r[i + 2]), "=r"(r[i + 3])
#define SZ_R16(r, i) SZ_R4(r, i), SZ_R4(r, i + 4), SZ_R4(r, i + 8), SZ_R4(r, i + 12)
#define SZ_I4(r, i) "r"(r[i]), "r"(r[i + 1]), "r"(r[i + 2]), "r"(r[i + 3])
#define SZ_I16(r, i) SZ_I4(r, i), SZ_I4(r, i + 4), SZ_I4(r, i + 8), SZ_I4(r, i + 12)

// 16 or 32 neighbouring columns of the thread's row.
__device__ __forceinline__ void tc_ld16(uint32_t *r, uint32_t a) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
        : SZ_R16(r, 0) : "r"(a) : "memory");
}
__device__ __forceinline__ void tc_ld32(uint32_t *r, uint32_t a) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : SZ_R16(r, 0), SZ_R16(r, 16) : "r"(a) : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t a, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::
            SZ_I16(r, 0), "r"(a) : "memory");
}

// What a load brings is there only behind the wait: uses stay behind it too.
__device__ __forceinline__ void tc_arrived(uint32_t *r) {
    asm volatile("" : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                      "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]));
}

// Shared-memory descriptor of rows of 128 bytes, 8 rows to a swizzle atom:
// leading offset (from one 64-element panel to the next; only values, whose
// rows run along the result's columns, have a use for it), stride offset of
// 1024 bytes from 8 rows to the next.
__device__ __forceinline__ uint64_t smem_desc(uint32_t a) {
    return uint64_t((a >> 4) & 0x3fff) | uint64_t(kPanel >> 4) << 16 | uint64_t(1024 >> 4) << 32 | 1ull << 46 |
           2ull << 61;
}

// d += a b: both operands 16-bit (fp16, or bf16), sums in 32 bits, 128 rows.
__device__ __forceinline__ uint32_t instr_desc(int dt, uint32_t n, bool b_along_n) {
    const uint32_t t = dt == SZ_BF16 ? 1 : 0;
    return 1u << 4 | t << 7 | t << 10 | (b_along_n ? 1u << 16 : 0u) | (n >> 3) << 17 | (128u >> 4) << 24;
}
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(add)) : "memory");
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Two floats at a time.
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ void f2_split(uint64_t v, float &a, float &b) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ uint64_t f2_fma(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t f2_add(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 32 bytes of a row, a whole sector, where its address allows it.
__device__ __forceinline__ void store32(uint8_t *a, const uint32_t (&v)[8], bool aligned32) {
    if (aligned32) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]) : "memory");
    } else {
        reinterpret_cast<uint4 *>(a)[0] = make_uint4(v[0], v[1], v[2], v[3]);
        reinterpret_cast<uint4 *>(a)[1] = make_uint4(v[4], v[5], v[6], v[7]);
    }
}

// ------------------------------------------------------------------- roles

// Keys and values into shared memory (warps 8-11), in the order in which they
// are used: k0, v0, k1, v1, ...  `box`: rows of a tensor copy, 0 for none.
struct Maps {
    const CUtensorMap *k, *v;
    uint32_t box;
};

// E5M2: 16 values of a row of the block to fp16, in the layout of the products.
__device__ __forceinline__ void spread16(uint32_t block, uint32_t row, uint32_t piece, uint4 v) {
    const uint4 lo = make_uint4(prmt(v.x, 0, 0x1404), prmt(v.x, 0, 0x3424), prmt(v.y, 0, 0x1404), prmt(v.y, 0, 0x3424));
    const uint4 hi = make_uint4(prmt(v.z, 0, 0x1404), prmt(v.z, 0, 0x3424), prmt(v.w, 0, 0x1404), prmt(v.w, 0, 0x3424));
    const uint32_t a = block + (piece / 4) * kPanel + row * 128, ch = 2 * (piece % 4);
    // the lanes of the second panel go the other way round, off the first one's banks
    const bool odd = piece >= 4;
    sts_u128(a + (((ch + (odd ? 1 : 0)) ^ (row & 7)) << 4), odd ? hi : lo);
    sts_u128(a + (((ch + (odd ? 0 : 1)) ^ (row & 7)) << 4), odd ? lo : hi);
}

// `issued`: stages filled; `raws`: tiles fetched into the raw ring.
template <int DT, int DP>
__device__ __forceinline__ void load_parts(const AttnParams &p, const Maps &maps, Work w, uint32_t base, TcAux *aux,
                                           uint32_t &issued, uint32_t &raws) {
    using C = TcCfg<DT, DP>;
    constexpr uint32_t LPR = DP * C::EB / 16;  // lanes to a row of the cache
    constexpr uint32_t ROWS = 32 / LPR;        // rows to an instruction
    constexpr uint32_t N = 32 / ROWS;          // instructions to a warp's 32 rows of a block
    const uint32_t tid = threadIdx.x & 127, lane = tid & 31, warp = tid >> 5;
    const uint32_t d = p.cache.head_dim;
    const uint32_t piece = lane % LPR, row0 = warp * 32 + lane / LPR;
    const bool has_piece = piece * 16 < d * C::EB;
    uint32_t ready = 0;  // what is behind `ready` has been handed over
    auto hand_over = [&](uint32_t to) {
        if (ready == to) return;
        fence_proxy_async_smem();
        for (; ready < to; ++ready) bar_arrive(&aux->full[ready % C::STAGES]);
        __syncwarp();
    };
    auto stage_free = [&](uint32_t n) {
        if (n < C::STAGES) return true;
        return bool(__all_sync(0xffffffffu, mbar_try_wait(&aux->empty[n % C::STAGES], (n / C::STAGES - 1) & 1)));
    };
    auto wait_free = [&](uint32_t n) {
        return n < C::STAGES || warp_wait(&aux->empty[n % C::STAGES], (n / C::STAGES - 1) & 1, aux, p);
    };
    for (;;) {
        const Part t = work_part<kTcRows, kTcBlock, kTcExtra>(p, w, blockIdx.x);
        const int32_t *ids = p.cache.table + uint64_t(w.seq) * p.cache.table_stride;
        const uint32_t part_hi = min((t.block0 + t.to) * kTcBlock, t.r.hi);
        const uint64_t head_off = uint64_t(w.head) * d * C::EB + piece * 16;
        const EdgeBlocks edges = edge_blocks<kTcBlock>(p, t);
        // Values of edges among the pieces of block j that this thread has copied, `from(u)` their
        // addresses: those that are not finite become 0.
        auto look = [&](uint32_t j, auto &&from) {
            uint32_t c = 0;
#pragma unroll 4
            for (uint32_t u = 0; u < N; ++u) c |= carries<DT>(lds_u128(from(u)));
            if ((c & kNotFinite<DT>) == 0) return;
            const Range all = seen_by_all(p, t);
#pragma unroll 1
            for (uint32_t u = 0; u < N; ++u) {
                const uint32_t at = (t.block0 + j) * kTcBlock + row0 + u * ROWS;
                uint4 v = lds_u128(from(u));
                if ((at >= all.lo && at < all.hi) || !make_finite<DT>(v)) continue;
                sts_u128(from(u), v);
                *reinterpret_cast<volatile uint32_t *>(&aux->edge) = 1;
            }
            fence_proxy_async_smem();
        };

        // the place of this lane's row of a block, and its page's id
        auto place = [&](uint32_t j) { return (t.block0 + j) * kTcBlock + warp * 32 + lane; };
        auto page_id = [&](uint32_t j) -> int32_t {
            const uint32_t at = place(j);
            return j < t.to && at >= t.r.lo && at < part_hi ? __ldg(ids + div_by(at, p.cache.page_tokens)) : 0;
        };
        auto offset = [&](uint32_t j, int32_t id) -> uint64_t {
            const uint32_t at = place(j);
            if (at < t.r.lo || at >= part_hi) return kBadOffset;
            const uint32_t page = div_by(at, p.cache.page_tokens);
            if (id < 0 || uint64_t(id) >= p.cache.pool_pages) {
                set_error(p.ctl, SZ_ERR_INVALID_ARG, page);
                return kBadOffset;
            }
            return uint64_t(id) * p.cache.page_bytes + uint64_t(at - page * p.cache.page_tokens.d) * p.cache.row_bytes;
        };
        // Offsets of eight of a lane's rows first: one by one, the shuffles' latency
        // bounds the copies.
        auto copy = [&](const uint8_t *pool, uint64_t off, auto &&to) {
            constexpr uint32_t STEP = N < 8 ? N : 8;
#pragma unroll
            for (uint32_t u0 = 0; u0 < N; u0 += STEP) {
                uint64_t o[STEP];
#pragma unroll
                for (uint32_t u = 0; u < STEP; ++u)
                    o[u] = __shfl_sync(0xffffffffu, off, int((u0 + u) * ROWS + lane / LPR));
                if (has_piece) {
#pragma unroll
                    for (uint32_t u = 0; u < STEP; ++u) {
                        const bool in = o[u] != kBadOffset;
                        cp_async16(to(u0 + u), pool + (in ? o[u] + head_off : 0), in);
                    }
                }
            }
            cp_commit();
        };
        const uint32_t blocks = t.to - t.from, tiles = 2 * blocks;
        if (maps.box > 0) {
            // A lane's box of a block: its page's id, or -1 if any of the boxes' ids is
            // outside the pool or not all of the block is seen.
            constexpr uint32_t PARTS = DT == SZ_BF16 ? C::PANELS : 1;  // boxes to a row: one for each panel, or raw rows
            const uint32_t boxes = kTcBlock / maps.box * PARTS, mine = lane < boxes ? lane / PARTS : 0;
            auto box_place = [&](uint32_t j) { return (t.block0 + j) * kTcBlock + mine * maps.box; };
            auto box_id = [&](uint32_t j) -> int32_t {
                const uint32_t at = (t.block0 + j) * kTcBlock;
                if (j >= t.to || at < t.r.lo || at + kTcBlock > part_hi) return -1;
                return __ldg(ids + div_by(box_place(j), p.cache.page_tokens));
            };
            // both kinds of a tile end in 128 arrivals at `bar`
            auto fetch = [&](bool key, uint32_t j, int32_t id, uint32_t dst, uint32_t bytes, uint64_t *bar) {
                if (__all_sync(0xffffffffu, id >= 0 && uint64_t(uint32_t(id)) < p.cache.pool_pages)) {
                    if (tid == 0) mbar_arrive_expect_tx(bar, bytes);
                    else bar_arrive(bar);
                    __syncwarp();
                    if (warp == 0 && lane < boxes) {
                        const uint32_t at = box_place(j), panel = lane % PARTS;
                        const uint32_t token = at - div_by(at, p.cache.page_tokens) * p.cache.page_tokens.d;
                        const CUtensorMap *map = key ? maps.k : maps.v;
                        if constexpr (DT == SZ_BF16)
                            tensor_g2s(dst + panel * kPanel + mine * maps.box * 128, map, panel * 64, w.head, token, uint32_t(id), bar);
                        else
                            tensor_g2s(dst + mine * maps.box * DP, map, 0, w.head, token, uint32_t(id), bar);
                    }
                    __syncwarp();
                    return;
                }
                const uint64_t off = offset(j, page_id(j));
                copy(key ? p.cache.k : p.cache.v, off, [&](uint32_t u) {
                    const uint32_t row = row0 + u * ROWS;
                    return DT == SZ_BF16 ? dst + (piece / 8) * kPanel + row * 128 + (((piece % 8) ^ (row & 7)) << 4)
                                         : dst + row * DP + piece * 16;
                });
                cp_wait<0>();
                fence_proxy_async_smem();
                bar_arrive(bar);
                __syncwarp();
            };
            int32_t id = box_id(t.from), ahead = box_id(t.from + 1);
            auto next_fetch = [&](uint32_t n, uint32_t dst, uint32_t bytes, uint64_t *bar) {
                const uint32_t j = t.from + n / 2;
                if (n > 0 && (n & 1) == 0) {
                    id = ahead;
                    ahead = box_id(j + 1);  // under way while this block is fetched
                }
                fetch((n & 1) == 0, j, id, dst, bytes, bar);
            };
            if constexpr (DT == SZ_BF16) {
                for (uint32_t n = 0; n < tiles; ++n, ++issued) {
                    if (!wait_free(issued)) return;
                    // (the query warps look at edges)
                    const bool edge = (n & 1) && edges.has(t.from + n / 2);
                    next_fetch(n, base + C::RING_AT + (issued % C::STAGES) * C::STAGE, C::STAGE,
                               edge ? &aux->edge_here[issued % C::STAGES] : &aux->full[issued % C::STAGES]);
                }
                ready = issued;
            } else {
                const uint32_t raw0 = raws;
                for (uint32_t n = 0; n < tiles + C::RAWS - 1; ++n) {
                    if (n < tiles) {
                        const uint32_t slot = raws % C::RAWS;
                        if (raws >= C::RAWS && !warp_wait(&aux->raw_empty[slot], (raws / C::RAWS - 1) & 1, aux, p)) return;
                        next_fetch(n, base + C::RAW_AT + slot * C::RAW, C::RAW, &aux->raw_full[slot]);
                        ++raws;
                    }
                    if (n + 1 < C::RAWS || n + 1 - C::RAWS >= tiles) continue;
                    const uint32_t x = raw0 + n + 1 - C::RAWS, slot = x % C::RAWS;
                    if (!warp_wait(&aux->raw_full[slot], (x / C::RAWS) & 1, aux, p) || !wait_free(issued)) return;
                    if (has_piece) {
                        const uint32_t m = x - raw0, j = t.from + m / 2;
                        if ((m & 1) && edges.has(j))
                            look(j, [&](uint32_t u) {
                                return base + C::RAW_AT + slot * C::RAW + (row0 + u * ROWS) * DP + piece * 16;
                            });
#pragma unroll
                        for (uint32_t u0 = 0; u0 < N; u0 += 4) {
                            uint4 v[4];
#pragma unroll
                            for (uint32_t u = 0; u < 4; ++u)
                                v[u] = lds_u128(base + C::RAW_AT + slot * C::RAW + (row0 + (u0 + u) * ROWS) * DP + piece * 16);
#pragma unroll
                            for (uint32_t u = 0; u < 4; ++u)
                                spread16(base + C::RING_AT + (issued % C::STAGES) * C::STAGE, row0 + (u0 + u) * ROWS, piece, v[u]);
                        }
                    }
                    bar_arrive(&aux->raw_empty[slot]);
                    ++issued;
                    hand_over(issued);
                }
            }
            if (!work_next<kTcRows, kTcExtra>(p, w, t, aux->order)) return;
            continue;
        }
        int32_t id = page_id(t.from);
        uint64_t off = 0;
        auto next_copy = [&](uint32_t n, auto &&to) {
            if ((n & 1) == 0) {
                off = offset(t.from + n / 2, id);
                id = page_id(t.from + n / 2 + 1);
            }
            copy((n & 1) ? p.cache.v : p.cache.k, off, to);
        };
        if constexpr (DT == SZ_BF16) {
            const uint32_t first = issued;
            auto at = [&](uint32_t stage, uint32_t u) {
                const uint32_t row = row0 + u * ROWS;
                return base + C::RING_AT + (stage % C::STAGES) * C::STAGE + (piece / 8) * kPanel + row * 128 +
                       (((piece % 8) ^ (row & 7)) << 4);
            };
            auto arrived = [&](uint32_t to) {
                for (uint32_t x = ready; x < to; ++x) {
                    const uint32_t n = x - first;
                    if ((n & 1) && has_piece && edges.has(t.from + n / 2)) look(t.from + n / 2, [&](uint32_t u) { return at(x, u); });
                }
                hand_over(to);
            };
            for (uint32_t n = 0; n < tiles; ++n) {
                if (!stage_free(issued)) {
                    cp_wait<0>();
                    arrived(issued);
                    if (!wait_free(issued)) return;
                }
                next_copy(n, [&](uint32_t u) { return at(issued, u); });
                ++issued;
                cp_wait<2>();
                if (issued > ready + 2) arrived(issued - 2);
            }
            cp_wait<0>();
            arrived(issued);
        } else {
            const uint32_t raw = base + C::RAW_AT + tid * 16;
            constexpr uint32_t LAG = 2;  // tiles under way behind the one that is spread
            for (uint32_t n = 0; n < tiles + LAG; ++n) {
                if (n < tiles) next_copy(n, [&](uint32_t u) { return raw + (n % C::RAWS) * C::RAW + u * 2048; });
                else cp_commit();
                if (n < LAG) continue;
                const uint32_t m = n - LAG;  // the tile that has come
                cp_wait<LAG>();
                if (!wait_free(issued)) return;
                if (has_piece) {
                    if ((m & 1) && edges.has(t.from + m / 2))
                        look(t.from + m / 2, [&](uint32_t u) { return raw + (m % C::RAWS) * C::RAW + u * 2048; });
#pragma unroll
                    for (uint32_t u0 = 0; u0 < N; u0 += 4) {
                        uint4 v[4];
#pragma unroll
                        for (uint32_t u = 0; u < 4; ++u) v[u] = lds_u128(raw + (m % C::RAWS) * C::RAW + (u0 + u) * 2048);
#pragma unroll
                        for (uint32_t u = 0; u < 4; ++u)
                            spread16(base + C::RING_AT + (issued % C::STAGES) * C::STAGE, row0 + (u0 + u) * ROWS, piece, v[u]);
                    }
                }
                ++issued;
                hand_over(issued);
            }
            cp_wait<0>();
        }
        if (!work_next<kTcRows, kTcExtra>(p, w, t, aux->order)) return;
    }
}

template <int DT, int DP>
__device__ __forceinline__ void load_role(const AttnParams &p, const Maps &maps, const Work &w, uint32_t base, TcAux *aux) {
    using C = TcCfg<DT, DP>;
    uint32_t issued = 0, raws = 0;
    load_parts<DT, DP>(p, maps, w, base, aux, issued, raws);
    cp_wait<0>();
    // the tensor copies that are under way land (nobody else waits for them where the CTA gives up)
    if (maps.box == 0 || (threadIdx.x & 127) >= 32) return;
    uint64_t *bars = DT == SZ_BF16 ? aux->full : aux->raw_full;
    const uint32_t ring = DT == SZ_BF16 ? C::STAGES : C::RAWS, n = DT == SZ_BF16 ? issued : raws;
    for (uint32_t x = n > ring ? n - ring : 0; x < n; ++x) mbar_wait(&bars[x % ring], (x / ring) & 1, kLandLimitNs);
}

// Queries into shared memory (warps 14, 15): by tensor copies of 128 / G tokens
// of the group's G heads where G divides 128 (`map`; rows behind the sequence's
// last are then the next one's, and nobody's), or row by row.  Behind a part's
// queries the warps look at the values of its edges, where these come by tensor
// copies in the products' layout (`edges`): nobody has had those in registers.
// (Two 1024-token prompts of 32 heads of 80, and 2048 tokens over 8192 places:
// 39 and 224 us; by the load warps 43 and 265; by one warp beside the queries 47
// and 228; not at all 36 and 223.)
constexpr uint32_t kQueryWarps = 2;
template <int DT, int DP>
__device__ __forceinline__ void query_parts(const AttnParams &p, const CUtensorMap *map, bool edges, Work w, uint32_t base,
                                            TcAux *aux, uint32_t &seen, uint32_t &phases) {
    using C = TcCfg<DT, DP>;
    constexpr uint32_t QL = DP / 8, QR = 32 / QL;          // lanes to a row, rows to an instruction
    constexpr uint32_t BATCH = 8;
    const uint32_t lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) - 14, c = lane % QL;
    const uint32_t d = p.cache.head_dim, G = p.group.d;
    uint32_t kv = 0, edge_phases = 0;  // the part's first stage; bit i: the phase of edge_here[i]
    for (;;) {
        const Part t = work_part<kTcRows, kTcBlock, kTcExtra>(p, w, blockIdx.x);
        const uint8_t *q = p.q.p + uint64_t(t.s.q0) * p.q.ts + uint64_t(w.head * G) * p.q.hs;
        for (uint32_t i = 0; i * 128 < t.rows; ++i) {
            if (seen & (1u << i)) {
                if (!warp_wait(&aux->q_empty[i], (phases >> i) & 1, aux, p)) return;
                phases ^= 1u << i;
            }
            seen |= 1u << i;
            const uint32_t tile = base + i * C::QTILE + (c / 8) * kQPanel;
            uint64_t *bar = DT == SZ_BF16 ? &aux->q_full[i] : &aux->q_here[i];
            if (map) {
                if (warp == 0 && lane == 0) {
                    mbar_arrive_expect_tx(bar, C::QTILE);
                    const uint32_t token = t.s.q0 + div_by(t.r0 + i * 128, p.group);
                    for (uint32_t x = 0; x < C::PANELS; ++x)
                        tensor3_g2s(base + i * C::QTILE + x * kQPanel, map, x * 64, w.head * G, token, bar);
                } else {
                    bar_arrive(bar);
                }
                __syncwarp();
                continue;
            }
            {
                for (uint32_t r0 = warp * BATCH * QR; r0 < 128; r0 += kQueryWarps * BATCH * QR) {
                    // a lane finds one row; rows behind the last are zeros
                    const uint32_t mine = i * 128 + r0 + lane % (BATCH * QR);
                    uint64_t at = kBadOffset;
                    if (mine < t.rows) {
                        const uint32_t g = t.r0 + mine, tok = div_by(g, p.group);
                        at = uint64_t(tok) * p.q.ts + uint64_t(g - tok * G) * p.q.hs;
                    }
                    uint64_t o[BATCH];
#pragma unroll
                    for (uint32_t u = 0; u < BATCH; ++u) o[u] = __shfl_sync(0xffffffffu, at, int(u * QR + lane / QL));
                    if (c * 8 < d) {
#pragma unroll
                        for (uint32_t u = 0; u < BATCH; ++u) {
                            const uint32_t r = r0 + u * QR + lane / QL;
                            const bool in = o[u] != kBadOffset;
                            cp_async16(tile + r * 128 + (((c % 8) ^ (r & 7)) << 4), in ? q + o[u] + c * 16 : p.q.p, in);
                        }
                    }
                }
            }
            cp_commit();
            cp_wait<0>();
            fence_proxy_async_smem();
            bar_arrive(bar);
            __syncwarp();
        }
        if (DT == SZ_BF16 && edges) {
            const Range all = seen_by_all(p, t);
            const EdgeBlocks blocks = edge_blocks<kTcBlock>(p, t);
            for (uint32_t j = t.from; j < t.to; ++j) {
                if (!blocks.has(j)) {  // on to the ones at the other end
                    j = min(blocks.hi, t.to) - 1;
                    continue;
                }
                const uint32_t at = (t.block0 + j) * kTcBlock, lo = max(at, t.r.lo), hi = min(at + kTcBlock, t.r.hi);
                const uint32_t stage = (kv + 2 * (j - t.from) + 1) % C::STAGES;
                if (!warp_wait(&aux->edge_here[stage], (edge_phases >> stage) & 1, aux, p)) return;
                edge_phases ^= 1u << stage;
                const uint32_t block = base + C::RING_AT + stage * C::STAGE + (c / 8) * kPanel;
                auto look = [&](uint32_t from, uint32_t to) {
                    from += warp * QR + lane / QL;
                    auto address = [&](uint32_t x) { return block + (x - at) * 128 + (((c % 8) ^ (x & 7)) << 4); };
                    uint32_t found = 0;
#pragma unroll 8
                    for (uint32_t x = from; x < to; x += kQueryWarps * QR) found |= carries<DT>(lds_u128(address(x)));
                    if ((found & kNotFinite<DT>) == 0) return;
                    *reinterpret_cast<volatile uint32_t *>(&aux->edge) = 1;
                    for (uint32_t x = from; x < to; x += kQueryWarps * QR) {
                        uint4 v = lds_u128(address(x));
                        if (make_finite<DT>(v)) sts_u128(address(x), v);
                    }
                };
                look(lo, min(hi, all.lo));
                look(max(lo, all.hi), hi);
                fence_proxy_async_smem();
                // (`full` counts the 128 threads of the load warps)
                for (uint32_t x = 0; x < 128 / (32 * kQueryWarps); ++x) bar_arrive(&aux->full[stage]);
                __syncwarp();
            }
            kv += 2 * (t.to - t.from);
        }
        if (!work_next<kTcRows, kTcExtra>(p, w, t, aux->order)) return;
    }
}

template <int DT, int DP>
__device__ __forceinline__ void query_role(const AttnParams &p, const CUtensorMap *map, bool edges, const Work &w,
                                           uint32_t base, TcAux *aux) {
    uint32_t seen = 0, phases = 0;  // bit i: tile i has been there; the phase of q_empty[i], and of the last copy
    query_parts<DT, DP>(p, map, edges, w, base, aux, seen, phases);
    cp_wait<0>();
    if (!map || threadIdx.x / 32 != 14) return;
    uint64_t *here = DT == SZ_BF16 ? aux->q_full : aux->q_here;
    for (uint32_t i = 0; i < 2; ++i)
        if (seen >> i & 1) mbar_wait(&here[i], (phases >> i) & 1, kLandLimitNs);
}

// The products of tile i (warps 12 and 13).  A warp goes through the loop
// together and one elected lane issues: behind a test of the thread's own number
// the compiler does not see that one lane is left, and each product took twice
// as long.  All of tensor memory is this CTA's, so its addresses are constants.
template <int DT, int DP>
__device__ __forceinline__ void mma_role(const AttnParams &p, Work w, uint32_t base, TcAux *aux, uint32_t i, bool leader) {
    using C = TcCfg<DT, DP>;
    const uint32_t d = p.cache.head_dim, ksteps = d / 16;
    const uint32_t qk_desc = instr_desc(DT, kTcBlock, false), pv_desc = instr_desc(DT, d, true);
    uint32_t kv = 0;      // the part's first stage
    uint32_t phases = 0;  // bit 2: of q_full[i]; bit h: of p_full[i][h]
    const uint64_t qd = smem_desc(base + i * C::QTILE);
    auto wait = [&](uint64_t *bar, uint32_t bit) {
        const bool ok = warp_wait(bar, (phases >> bit) & 1, aux, p);
        phases ^= 1u << bit;
        tc_after();
        return ok;
    };
    auto full = [&](uint32_t n) {
        const bool ok = warp_wait(&aux->full[n % C::STAGES], (n / C::STAGES) & 1, aux, p);
        tc_after();
        return ok;
    };
    auto stage = [&](uint32_t n) { return smem_desc(base + C::RING_AT + (n % C::STAGES) * C::STAGE); };
    auto qk = [&](uint64_t kd) {
#pragma unroll
        for (uint32_t k = 0; k < DP / 16; ++k)
            if (k < ksteps)
                mma_ss(i * 128, qd + (((k / 4) * kQPanel + (k % 4) * 32) >> 4),
                       kd + (((k / 4) * kPanel + (k % 4) * 32) >> 4), qk_desc, k > 0);
    };
    auto pv = [&](uint32_t half, uint64_t vd, bool add) {
#pragma unroll
        for (uint32_t k = half * 4; k < half * 4 + 4; ++k)
            mma_ts(256 + i * 128, i * 128 + k * 8, vd + k * (2048 >> 4), pv_desc, add || k > 0);
    };
    Part t = work_part<kTcRows, kTcBlock, kTcExtra>(p, w, blockIdx.x);
    for (;;) {
        const uint32_t n = t.to - t.from;
        Part after = t;  // the next part, found while the first scores are on their way
        bool more = false;
        auto look_ahead = [&]() {
            more = work_next<kTcRows, kTcExtra>(p, w, t, aux->order);
            if (more) after = work_part<kTcRows, kTcBlock, kTcExtra>(p, w, blockIdx.x);
        };
        if (i * 128 < t.rows) {
            if (!full(kv)) return;
            if (!wait(&aux->q_full[i], 2)) return;
            if (leader) {
                qk(stage(kv));
                tc_commit(&aux->s_full[i]);
                tc_commit(&aux->empty[kv % C::STAGES]);
                if (n == 1) tc_commit(&aux->q_empty[i]);
            }
            __syncwarp();
            look_ahead();
            for (uint32_t j = 0; j < n; ++j) {
                const uint32_t v = kv + 2 * j + 1, k = v + 1;
                const uint64_t vd = stage(v), kd = stage(k);
                if (!full(v)) return;
                if (!wait(&aux->p_full[i][0], 0)) return;
                if (leader) pv(0, vd, j > 0);
                __syncwarp();
                // what the second half's way to the next scores does not depend on comes before it, or behind
                const bool more = j + 1 < n;
                if (more && !full(k)) return;
                if (!wait(&aux->p_full[i][1], 1)) return;
                if (leader) {
                    pv(1, vd, true);
                    if (more) {
                        qk(kd);
                        tc_commit(&aux->s_full[i]);
                        tc_commit(&aux->empty[v % C::STAGES]);
                        tc_commit(&aux->empty[k % C::STAGES]);
                        if (j + 2 == n) tc_commit(&aux->q_empty[i]);
                    } else {
                        tc_commit(&aux->o_full[i]);
                        tc_commit(&aux->empty[v % C::STAGES]);
                    }
                }
                __syncwarp();
            }
        } else {
            look_ahead();
            // the other tile's stages need this one's word too
            for (uint32_t j = 0; j < 2 * n; ++j) {
                if (!full(kv + j)) return;
                if (leader) bar_arrive(&aux->empty[(kv + j) % C::STAGES]);
                __syncwarp();
            }
        }
        kv += 2 * n;
        if (!more) return;
        t = after;
    }
}

// A warp's 32 rows of a tile with few parts: the warp that comes last to them
// adds them up, in the parts' order.
template <int DT>
__device__ __forceinline__ void join_few(const AttnParams &p, const Work &w, const Part &t, uint32_t r, uint32_t parts) {
    constexpr float RAISE = TcCfg<DT, 64>::RAISE;
    const uint32_t d = p.cache.head_dim, lane = threadIdx.x & 31;
    uint32_t *arrived = p.arrived + t.c_first * 8 + r / 32;
    __threadfence();
    __syncwarp();
    uint32_t n = 0;
    if (lane == 0) n = atomicAdd(arrived, 1u);
    if (__shfl_sync(0xffffffffu, n, 0) != parts - 1) return;
    __threadfence();
    if (lane == 0) *arrived = 0;
    const float *from[kFewParts];
    float f[kFewParts], M = -INFINITY, L = 0.f;
#pragma unroll
    for (uint32_t k = 0; k < kFewParts; ++k) {
        from[k] = p.part + uint64_t(part_slot(t.c_first + min(k, parts - 1), t)) * kTcRows * (d + 2);
        f[k] = k < parts ? __ldcg(from[k] + d * kTcRows + r) : -INFINITY;
        M = fmaxf(M, f[k]);
    }
#pragma unroll
    for (uint32_t k = 0; k < kFewParts; ++k) {
        f[k] = exp2_fast(f[k] - (M == -INFINITY ? 0.f : M));
        if (k < parts) L = fmaf(f[k], __ldcg(from[k] + (d + 1) * kTcRows + r), L);
    }
    const uint32_t g = t.r0 + r, tok = div_by(g, p.group), head = w.head * p.group.d + (g - tok * p.group.d);
    const float inv = L == 0.f ? 0.f : 1.f / L;
    uint8_t *out = p.out.p + uint64_t(t.s.q0 + tok) * p.out.ts + uint64_t(head) * p.out.hs;
    const bool aligned32 = ((reinterpret_cast<uintptr_t>(p.out.p) | p.out.ts | p.out.hs) & 31) == 0;
    for (uint32_t e = 0; e < d; e += 16) {
        float v[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) v[j] = 0.f;
#pragma unroll
        for (uint32_t k = 0; k < kFewParts; ++k) {
            if (k >= parts) break;
#pragma unroll
            for (int j = 0; j < 16; j += 4) {
                const float4 x = __ldcg(reinterpret_cast<const float4 *>(from[k]) + ((e + j) / 4 * kTcRows + r));
                v[j] = fmaf(f[k], x.x, v[j]), v[j + 1] = fmaf(f[k], x.y, v[j + 1]);
                v[j + 2] = fmaf(f[k], x.z, v[j + 2]), v[j + 3] = fmaf(f[k], x.w, v[j + 3]);
            }
        }
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            v[2 * j] *= inv, v[2 * j + 1] *= inv;
            pk[j] = pack_bf16(v[2 * j], v[2 * j + 1]);
        }
        if (r < t.rows) {
            store32(out + 2 * e, pk, aligned32);
        }
    }
    if (r < t.rows && p.lse)
        p.lse[uint64_t(t.s.q0 + tok) * p.q.heads + head] = L == 0.f ? -INFINITY : kLn2 * (M - RAISE + log2f(L));
}

// Softmax of one tile's rows, a thread a row, and what becomes of the sums.
template <int DT, int DP>
__device__ __forceinline__ void softmax_role(const AttnParams &p, Work w, uint32_t base, TcAux *aux, TcDesc *desc) {
    using C = TcCfg<DT, DP>;
    const uint32_t i = threadIdx.x / 128, row = threadIdx.x & 127;
    const uint32_t lanes = (threadIdx.x & 96) << 16;  // the warp's quarter of tensor memory
    const uint32_t s_at = lanes + i * 128, o_at = lanes + 256 + i * 128;
    const uint32_t d = p.cache.head_dim, G = p.group.d;
    uint32_t q_uses = 0, s_uses = 0, o_uses = 0, turns = 0;
    Part t = work_part<kTcRows, kTcBlock, kTcExtra>(p, w, blockIdx.x);
    for (;;) {
        const bool whole_tile = t.c_first == t.c_last;
        Work next = w;  // the part behind this one, found while this one's last product runs
        Part after = t;
        bool more = false;
        auto look_ahead = [&]() {
            more = work_next<kTcRows, kTcExtra>(p, next, t, aux->order);
            if (more) after = work_part<kTcRows, kTcBlock, kTcExtra>(p, next, blockIdx.x);
        };
        const uint32_t parts = t.c_last - t.c_first + 1;
        if (threadIdx.x == 0 && parts > kFewParts && t.c_first == blockIdx.x) {
            desc->join = w;
            desc->joins = 1;
        }
        if (i == 0 || t.rows > 128) {
            const uint32_t r = i * 128 + row;
            Range rr{0, 0};
            if (r < t.rows) rr = token_range(p, t.s, div_by(t.r0 + r, p.group));
            // every row of the 128 sees [full_lo, full_hi)
            const uint32_t full_hi = token_range(p, t.s, div_by(t.r0 + i * 128, p.group)).hi;
            const uint32_t full_lo = token_range(p, t.s, div_by(t.r0 + min(i * 128 + 128, t.rows) - 1, p.group)).lo;
            float sc = p.scale_log2;
            if constexpr (DT == SZ_FP8_E5M2) {
                // the row's queries to fp16, behind a power of two that its scores are divided by
                if (!warp_wait(&aux->q_here[i], q_uses++ & 1, aux, p)) return;
                const uint32_t at = base + i * C::QTILE + row * 128;
                const auto chunk = [&](uint32_t c) { return at + (c / 8) * kQPanel + (((c % 8) ^ (row & 7)) << 4); };
                uint32_t big = 0;  // of magnitudes as 16-bit integers, whose order is that of the numbers
                for (uint32_t c = 0; c < d / 8; c += 2) {
                    const uint4 u = lds_u128(chunk(c)), v = lds_u128(chunk(c + 1));
                    const uint32_t y = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu),
                                                __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
                    const uint32_t z = __vmaxu2(__vmaxu2(v.x & 0x7fff7fffu, v.y & 0x7fff7fffu),
                                                __vmaxu2(v.z & 0x7fff7fffu, v.w & 0x7fff7fffu));
                    big = __vmaxu2(big, __vmaxu2(y, z));
                }
                big = max(big >> 16, big & 0xffffu);
                // (no finite power for a row of zeros, or with infinities or NaN)
                const int e = big > 0 && big < 0x7f80u ? min(13 - (int(big >> 7) - 127), 120) : 0;
                const float up = __uint_as_float(uint32_t(127 + e) << 23);
                for (uint32_t c = 0; c < d / 8; c += 2) {
                    const uint4 u = lds_u128(chunk(c)), v = lds_u128(chunk(c + 1));
                    sts_u128(chunk(c), make_uint4(pack_f16(bf16_lo(u.x) * up, bf16_hi(u.x) * up), pack_f16(bf16_lo(u.y) * up, bf16_hi(u.y) * up),
                                                  pack_f16(bf16_lo(u.z) * up, bf16_hi(u.z) * up), pack_f16(bf16_lo(u.w) * up, bf16_hi(u.w) * up)));
                    sts_u128(chunk(c + 1), make_uint4(pack_f16(bf16_lo(v.x) * up, bf16_hi(v.x) * up), pack_f16(bf16_lo(v.y) * up, bf16_hi(v.y) * up),
                                                      pack_f16(bf16_lo(v.z) * up, bf16_hi(v.z) * up), pack_f16(bf16_lo(v.w) * up, bf16_hi(v.w) * up)));
                }
                // (not 0, which times a masked score's -infinity is NaN; scores times 2^-126 are below 2^-80, as they are times less)
                sc = fmaxf(sc * __uint_as_float(uint32_t(127 - e) << 23), 1.17549435e-38f);
                fence_proxy_async_smem();
                bar_arrive(&aux->q_full[i]);
            }
            float m = -INFINITY, l = 0.f;
            for (uint32_t j = t.from; j < t.to; ++j) {
                if (!warp_wait(&aux->s_full[i], s_uses++ & 1, aux, p)) return;
                tc_after();
                const uint32_t at = (t.block0 + j) * kTcBlock;
                const bool masked = at < full_lo || at + kTcBlock > full_hi;
                uint32_t x[128];
                tc_ld32(x, s_at);
                tc_ld32(x + 32, s_at + 32);
                tc_wait_ld();
                tc_ld32(x + 64, s_at + 64);
                tc_ld32(x + 96, s_at + 96);
#pragma unroll
                for (int c = 0; c < 64; c += 16) tc_arrived(x + c);
                if (masked) {
                    // columns [a, b) of the block are seen; the others' scores become -infinity
                    tc_wait_ld();
#pragma unroll
                    for (int c = 64; c < 128; c += 16) tc_arrived(x + c);
                    const uint32_t a = rr.lo > at ? rr.lo - at : 0, b = rr.hi > at ? rr.hi - at : 0;
#pragma unroll
                    for (uint32_t g = 0; g < 128; g += 32) {
                        const uint32_t ga = a > g ? min(a - g, 32u) : 0, gb = b > g ? min(b - g, 32u) : 0;
                        const uint32_t seen = uint32_t((1ull << gb) - 1) & uint32_t(~0ull << ga);
#pragma unroll
                        for (uint32_t c = 0; c < 32; ++c)
                            if (!(seen & (1u << c))) x[g + c] = 0xff800000u;
                    }
                }
                // (the first half's maximum while the second half comes)
                float tops[4];
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    tops[e] = max3(__uint_as_float(x[e]), __uint_as_float(x[e + 4]), __uint_as_float(x[e + 8]));
#pragma unroll
                for (int c = 12; c < 60; c += 8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], __uint_as_float(x[c + e]), __uint_as_float(x[c + e + 4]));
                }
                tc_wait_ld();
#pragma unroll
                for (int c = 64; c < 128; c += 16) tc_arrived(x + c);
#pragma unroll
                for (int c = 60; c < 124; c += 8) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) tops[e] = max3(tops[e], __uint_as_float(x[c + e]), __uint_as_float(x[c + e + 4]));
                }
#pragma unroll
                for (int e = 0; e < 4; ++e) tops[e] = fmaxf(tops[e], __uint_as_float(x[124 + e]));
                const float top = fmaxf(fmaxf(tops[0], tops[1]), fmaxf(tops[2], tops[3])) * sc;
                const bool grows = top > m + C::SLACK;
                if (__any_sync(0xffffffffu, grows)) {
                    const float c = grows ? exp2_fast(m - top) : 1.f;
                    if (grows) m = top;
                    l *= c;
                    if (j > t.from) {
                        // the scores came behind the last product: the sums are at rest
                        for (uint32_t k = 0; k < d; k += 16) {
                            uint32_t o[16];
                            tc_ld16(o, o_at + k);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * c);
                            tc_st16(o_at + k, o);
                        }
                    }
                }
                // The tiles take turns at ex2, three quarters of a block apart: side by
                // side they would both wait for it, and then both for their products
                // (2048 tokens over 8192 places, the same inputs again and again: 293 us, by
                // turns 229; with others each time, as at the top, the clocks are lower).  A polynomial in
                // place of a part of the ex2 took 13 us more: its multiply-adds, two to an
                // instruction or not, take the issue slots.
                if (t.rows > 128) {
                    if ((i == 1 || turns > 0) && !warp_wait(&aux->turn[i], (turns - 1 + i) & 1, aux, p)) return;
                    ++turns;
                }
                const float shift = C::RAISE - (m == -INFINITY ? 0.f : m);
                const uint64_t sc2 = f2(sc, sc), shift2 = f2(shift, shift);
                // (the weights are rounded to the 16 bits of the products, half a step, 2^-8 in bf16 and
                // 2^-11 in fp16; their sum is taken before, in 32: see pack_p in sz_attn.cu)
                uint64_t sum[2] = {0, 0};
#pragma unroll
                for (int c = 0; c < 128; c += 32) {
                    uint32_t pk[16];
#pragma unroll
                    for (int e = 0; e < 32; e += 2) {
                        float a, b;
                        f2_split(f2_fma(f2(__uint_as_float(x[c + e]), __uint_as_float(x[c + e + 1])), sc2, shift2), a, b);
                        a = exp2_fast(a);
                        b = exp2_fast(b);
                        sum[(e >> 1) & 1] = f2_add(sum[(e >> 1) & 1], f2(a, b));
                        pk[e / 2] = DT == SZ_BF16 ? pack_bf16(a, b) : pack_f16(a, b);
                    }
                    if (c == 64) {
                        // the first half has long been stored by now
                        tc_wait_st();
                        tc_before();
                        bar_arrive(&aux->p_full[i][0]);
                    }
                    tc_st16(s_at + c / 2, pk);
                    if (c == 64 && t.rows > 128) {
                        __syncwarp();
                        if ((threadIdx.x & 31) == 0) bar_arrive(&aux->turn[1 - i]);
                        __syncwarp();
                    }
                }
                tc_wait_st();
                tc_before();
                bar_arrive(&aux->p_full[i][1]);
                float a, b;
                f2_split(f2_add(sum[0], sum[1]), a, b);
                l += a + b;
            }
            look_ahead();
            if (!warp_wait(&aux->o_full[i], o_uses++ & 1, aux, p)) return;
            tc_after();
            if (__any_sync(0xffffffffu, *reinterpret_cast<volatile uint32_t *>(&aux->edge) != 0)) {
                // values that are not finite, which the products went without
                const Range all = seen_by_all(p, t);
                const uint32_t from = (t.block0 + t.from) * kTcBlock, to = min((t.block0 + t.to) * kTcBlock, t.r.hi);
#pragma unroll 1
                for (uint32_t k = 0; k < d; k += 16) {
                    uint32_t o[16];
                    float sum[16];
                    tc_ld16(o, o_at + k);
                    tc_wait_ld();
                    tc_arrived(o);
#pragma unroll
                    for (int e = 0; e < 16; ++e) sum[e] = __uint_as_float(o[e]);
                    add_not_finite<DT, 16>(p, w.seq, w.head, rr, all, from, to, k, sum);
#pragma unroll
                    for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(sum[e]);
                    __syncwarp();
                    tc_st16(o_at + k, o);
                }
                tc_wait_st();
            }
            if (whole_tile) {
                const uint32_t g = t.r0 + r, tok = div_by(g, p.group), head = w.head * G + (g - tok * G);
                const float f = l == 0.f ? 0.f : 1.f / l;
                uint8_t *out = p.out.p + uint64_t(t.s.q0 + tok) * p.out.ts + uint64_t(head) * p.out.hs;
                const bool aligned32 = ((reinterpret_cast<uintptr_t>(p.out.p) | p.out.ts | p.out.hs) & 31) == 0;
                for (uint32_t k = 0; k < d; k += 16) {
                    uint32_t o[16];
                    tc_ld16(o, o_at + k);
                    tc_wait_ld();
                    uint32_t pk[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float a = __uint_as_float(o[2 * e]) * f, b = __uint_as_float(o[2 * e + 1]) * f;
                        pk[e] = pack_bf16(a, b);
                    }
                    if (r < t.rows) {
                        store32(out + 2 * k, pk, aligned32);
                    }
                }
                if (r < t.rows && p.lse)
                    p.lse[uint64_t(t.s.q0 + tok) * p.q.heads + head] =
                        l == 0.f ? -INFINITY : kLn2 * (m - C::RAISE + log2f(l));
            } else {
                // four columns of 256 rows at a time, then the rows' m and l
                float *part = p.part + uint64_t(part_slot(blockIdx.x, t)) * kTcRows * (d + 2) + r;
                float4 *quad = reinterpret_cast<float4 *>(part - r) + r;
                for (uint32_t k = 0; k < d; k += 16) {
                    uint32_t o[16];
                    tc_ld16(o, o_at + k);
                    tc_wait_ld();
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        quad[(k / 4 + e) * kTcRows] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                                  __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                }
                part[d * kTcRows] = m;
                part[(d + 1) * kTcRows] = l;
                if (parts <= kFewParts) join_few<DT>(p, w, t, r, parts);
            }
            // the sums are read before the next part's first weights are announced
            tc_before();
        } else {
            look_ahead();
        }
        if (!more) return;
        w = next;
        t = after;
    }
}

template <int DT, int DP>
__global__ void __launch_bounds__(kTcThreads, 1)
    attn_tc_kernel(const __grid_constant__ AttnParams p, const __grid_constant__ CUtensorMap k_map,
                   const __grid_constant__ CUtensorMap v_map, const __grid_constant__ CUtensorMap q_map, uint32_t box,
                   uint32_t q_box) {
    using C = TcCfg<DT, DP>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    const uint32_t base = smem_u32(smem);
    TcAux *aux = reinterpret_cast<TcAux *>(smem + C::AUX_AT);
    const uint32_t tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
    TcDesc *desc = reinterpret_cast<TcDesc *>(p.desc) + blockIdx.x;

    if (tid == 0) {
        for (uint32_t i = 0; i < C::STAGES; ++i) {
            mbar_init(&aux->full[i], 128);
            mbar_init(&aux->empty[i], 2);
            mbar_init(&aux->edge_here[i], 128);
        }
        for (int i = 0; i < int(C::RAWS); ++i) {
            mbar_init(&aux->raw_full[i], 128);
            mbar_init(&aux->raw_empty[i], 128);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&aux->q_full[i], DT == SZ_BF16 ? 32 * kQueryWarps : 128);
            mbar_init(&aux->q_here[i], 32 * kQueryWarps);
            mbar_init(&aux->q_empty[i], 1);
            mbar_init(&aux->s_full[i], 1);
            for (int h = 0; h < 2; ++h) mbar_init(&aux->p_full[i][h], 128);
            mbar_init(&aux->o_full[i], 1);
            mbar_init(&aux->turn[i], 4);
        }
        mbar_init(&aux->drain[0], 1);
        mbar_init(&aux->drain[1], 1);
        fence_mbar_init();
        aux->abort = 0;
        aux->edge = 0;
    }
    pdl_wait();
    pdl_launch_dependents();
    Work w;
    const bool has = work_begin<kTcThreads, kTcRows, kTcBlock, kTcExtra>(
        p, *reinterpret_cast<WorkScratch<kTcThreads> *>(smem + C::RING_AT), w, aux->order);
    if (tid == 0) desc->joins = 0;
    if (!has) return;
    if (warp == 12) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(&aux->tmem))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
    }
    // the scratch's last reads are done before the copies write over it
    fence_proxy_async_smem();
    tc_before();
    __syncthreads();
    tc_after();
    const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(&aux->tmem);

    if (warp < 8) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 " SZ_TC_REGS_SOFTMAX ";");
        softmax_role<DT, DP>(p, w, base, aux, desc);
        __syncwarp();
        tc_wait_st();  // (where the CTA gives up, sums may be on their way back)
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 " SZ_TC_REGS_OTHER ";");
        if (warp < 12) {
            load_role<DT, DP>(p, Maps{&k_map, &v_map, box}, w, base, aux);
        } else if (warp < 14) {
            const bool leader = elect_one();
            mma_role<DT, DP>(p, w, base, aux, warp - 12, leader);
            // no product of this CTA's is under way when it gives its memory back, given up or not
            __syncwarp();
            if (leader) tc_commit(&aux->drain[warp - 12]);
            __syncwarp();
            mbar_wait(&aux->drain[warp - 12], 0, kLandLimitNs);
            __syncwarp();
        } else {
            query_role<DT, DP>(p, q_box ? &q_map : nullptr, box > 0, w, base, aux);
        }
    }
    __syncwarp();
    tc_before();
    __syncthreads();
    tc_after();
    if (warp == 12) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(tmem));
}

// ------------------------------------------------------------------ joining

constexpr int kJoinThreads = 256;
constexpr int kJoinRows = 32;
constexpr int kJoinSlices = kTcRows / kJoinRows;
constexpr uint32_t kJoinWarps = kJoinThreads / 32;
constexpr uint32_t kJoinSplit = 4;                        // groups of columns ...
constexpr uint32_t kJoinGroups = kJoinWarps / kJoinSplit; // ... and of parts
static_assert(kMaxSms <= kJoinThreads, "a thread looks at a CTA");

// Tiles of more than kFewParts parts; an item is 32 rows of one, a lane a row; a warp has a quarter of the columns of every second part.
template <int DT, int DP>
__global__ void __launch_bounds__(kJoinThreads) attn_join_kernel(const __grid_constant__ AttnParams p) {
    using C = TcCfg<DT, DP>;
    constexpr uint32_t COLS = DP / kJoinSplit;
    __shared__ float s_o[kJoinGroups - 1][DP][kJoinRows];
    __shared__ float s_m[kJoinWarps][kJoinRows], s_l[kJoinWarps][kJoinRows];
    pdl_wait();
    pdl_launch_dependents();
    __shared__ uint32_t s_list[kJoinWarps][33];
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t d = p.cache.head_dim, G = p.group.d;
    const TcDesc *descs = reinterpret_cast<const TcDesc *>(p.desc);
    // the tiles to join, listed by each warp for its 32 of the CTAs
    {
        const bool joins = threadIdx.x < gridDim.x && descs[threadIdx.x].joins;
        const uint32_t all = __ballot_sync(0xffffffffu, joins);
        if (joins) s_list[warp][1 + __popc(all & lanemask_lt())] = threadIdx.x;
        if (lane == 0) s_list[warp][0] = __popc(all);
    }
    __syncthreads();
    uint32_t tiles = 0;
#pragma unroll
    for (uint32_t k = 0; k < kJoinWarps; ++k) tiles += s_list[k][0];
    for (uint32_t item = blockIdx.x; item < tiles * kJoinSlices; item += gridDim.x) {
        const uint32_t slice = item % kJoinSlices;
        uint32_t k = 0, nth = item / kJoinSlices;
        while (nth >= s_list[k][0]) nth -= s_list[k++][0];
        const uint32_t c = s_list[k][1 + nth];
        const Work w = descs[c].join;
        const Part t = work_part<kTcRows, kTcBlock, kTcExtra>(p, w, c);
        if (slice * kJoinRows < t.rows) {
            __syncthreads();  // (the last item's sums are read)
            const uint32_t r = slice * kJoinRows + lane, parts = t.c_last - t.c_first + 1;
            auto slot = [&](uint32_t k) {
                return p.part + uint64_t(part_slot(t.c_first + k, t)) * kTcRows * (d + 2) + r;
            };
            // the largest m of all parts, and sum l against it
            float M = -INFINITY;
            for (uint32_t k = warp; k < parts; k += kJoinWarps) M = fmaxf(M, __ldcg(slot(k) + d * kTcRows));
            s_m[warp][lane] = M;
            __syncthreads();
#pragma unroll
            for (uint32_t k = 0; k < kJoinWarps; ++k) M = fmaxf(M, s_m[k][lane]);
            const float safe = M == -INFINITY ? 0.f : M;
            float L = 0.f;
            for (uint32_t k = warp; k < parts; k += kJoinWarps)
                L = fmaf(exp2_fast(__ldcg(slot(k) + d * kTcRows) - safe), __ldcg(slot(k) + (d + 1) * kTcRows), L);
            s_l[warp][lane] = L;
            const uint32_t col0 = (warp % kJoinSplit) * (d / kJoinSplit), kg = warp / kJoinSplit;
            float v[COLS];
#pragma unroll
            for (uint32_t e = 0; e < COLS; ++e) v[e] = 0.f;
            for (uint32_t k = kg; k < parts; k += kJoinGroups) {
                const float f = exp2_fast(__ldcg(slot(k) + d * kTcRows) - safe);
                const float4 *from = reinterpret_cast<const float4 *>(slot(k) - r) + col0 / 4 * kTcRows + r;
#pragma unroll
                for (uint32_t e = 0; e < COLS; e += 4)
                    if (e < d / kJoinSplit) {
                        const float4 x = __ldcg(from + e / 4 * kTcRows);
                        v[e] = fmaf(f, x.x, v[e]), v[e + 1] = fmaf(f, x.y, v[e + 1]);
                        v[e + 2] = fmaf(f, x.z, v[e + 2]), v[e + 3] = fmaf(f, x.w, v[e + 3]);
                    }
            }
            if (kg > 0) {
#pragma unroll
                for (uint32_t e = 0; e < COLS; ++e)
                    if (e < d / kJoinSplit) s_o[kg - 1][col0 + e][lane] = v[e];
            }
            __syncthreads();
            const uint32_t g = t.r0 + r, tok = div_by(g, p.group), head = w.head * G + (g - tok * G);
            if (kg == 0) {
                L = 0.f;
#pragma unroll
                for (uint32_t k = 0; k < kJoinWarps; ++k) L += s_l[k][lane];
                const float inv = L == 0.f ? 0.f : 1.f / L;
                uint8_t *out = p.out.p + uint64_t(t.s.q0 + tok) * p.out.ts + uint64_t(head) * p.out.hs + 2 * col0;
#pragma unroll
                for (uint32_t e = 0; e < COLS; e += 4) {
                    if (e >= d / kJoinSplit) break;
#pragma unroll
                    for (uint32_t j = e; j < e + 4; ++j) {
#pragma unroll
                        for (uint32_t k = 0; k < kJoinGroups - 1; ++k) v[j] += s_o[k][col0 + j][lane];
                        v[j] *= inv;
                    }
                    if (r < t.rows)
                        *reinterpret_cast<uint2 *>(out + 2 * e) =
                            make_uint2(pack_bf16(v[e], v[e + 1]), pack_bf16(v[e + 2], v[e + 3]));
                }
                if (warp == 0 && r < t.rows && p.lse)
                    p.lse[uint64_t(t.s.q0 + tok) * p.q.heads + head] =
                        L == 0.f ? -INFINITY : kLn2 * (M - C::RAISE + log2f(L));
            }
        }
    }
}

using EncodeTiled = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                 const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                 CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiled encode_tiled() {
    static std::atomic<void *> cache{nullptr};
    void *f = cache.load(std::memory_order_acquire);
    if (f) return reinterpret_cast<EncodeTiled>(f);
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
        return nullptr;
    cache.store(f, std::memory_order_release);
    return reinterpret_cast<EncodeTiled>(f);
}

// Pool as [pages, page_tokens, kv_heads, head_dim]; boxes of `box` rows of one
// head: 64 elements in the products' swizzle, or whole E5M2 rows as they are.
template <int DT, int DP>
bool pool_map(CUtensorMap *map, const AttnParams &p, uint8_t *pool, uint32_t box) {
    const CacheRef &c = p.cache;
    const EncodeTiled encode = encode_tiled();
    if (!encode || c.pool_pages >= (1ull << 31) || c.page_bytes >= (1ull << 40)) return false;
    constexpr uint64_t EB = TcCfg<DT, DP>::EB;
    const cuuint64_t dims[4] = {c.head_dim, c.kv_heads, c.page_tokens.d, c.pool_pages};
    const cuuint64_t strides[3] = {c.head_dim * EB, c.row_bytes, c.page_bytes};
    const cuuint32_t boxes[4] = {DT == SZ_BF16 ? 64u : uint32_t(DP), 1, box, 1}, one[4] = {1, 1, 1, 1};
    return encode(map, DT == SZ_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pool, dims,
                  strides, boxes, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  DT == SZ_BF16 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Queries as [tokens, heads, head_dim]; boxes of 128 / G tokens of G heads.
bool query_map(CUtensorMap *map, const AttnParams &p) {
    const EncodeTiled encode = encode_tiled();
    const uint32_t G = p.group.d;
    // (one token or one head: its stride is nothing that a map takes)
    const uint64_t hs = p.q.heads > 1 ? p.q.hs : uint64_t(p.cache.head_dim) * 2;
    const uint64_t ts = p.tokens > 1 ? p.q.ts : hs * p.q.heads;
    if (!encode || G > 128 || 128 % G != 0 || hs == 0 || ts == 0 || hs >= (1ull << 40) || ts >= (1ull << 40)) return false;
    const cuuint64_t dims[3] = {p.cache.head_dim, p.q.heads, p.tokens}, strides[2] = {hs, ts};
    const cuuint32_t boxes[3] = {64, G, 128 / G}, one[3] = {1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, p.q.p, dims, strides, boxes, one,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int DT, int DP>
sz_status run(const AttnParams &p, int num_sms, cudaStream_t stream) {
    using C = TcCfg<DT, DP>;
    static std::atomic<int> cache[kMaxDevices];
    auto kern = attn_tc_kernel<DT, DP>;
    if (resident_per_sm(reinterpret_cast<const void *>(kern), kTcThreads, C::SMEM, cache) <= 0) return SZ_ERR_CUDA;
    // rows of a box: the largest power of two that divides a page, from 8 (a swizzle atom) to a block
    CUtensorMap k_map{}, v_map{}, q_map{};
    uint32_t box = p.cache.page_tokens.d & (0u - p.cache.page_tokens.d);
    box = box < 8 ? 0 : (box < uint32_t(kTcBlock) ? box : uint32_t(kTcBlock));
    if (box && !(pool_map<DT, DP>(&k_map, p, p.cache.k, box) && pool_map<DT, DP>(&v_map, p, p.cache.v, box))) box = 0;
    const uint32_t q_box = query_map(&q_map, p) ? 1 : 0;
    if (launch_pdl(kern, unsigned(num_sms), kTcThreads, C::SMEM, stream, p, k_map, v_map, q_map, box, q_box) != cudaSuccess)
        return SZ_ERR_CUDA;
    return launch_pdl(attn_join_kernel<DT, DP>, unsigned(num_sms), kJoinThreads, 0, stream, p) ==
                   cudaSuccess
               ? SZ_OK
               : SZ_ERR_CUDA;
}

}  // namespace

sz_status launch_attn_tc(AttnParams p, int dtype, int num_sms, cudaStream_t stream) {
    p.wait_ns = SZ_ATTN_WAIT_NS;
    if (dtype == SZ_BF16)
        return p.cache.head_dim <= 64 ? run<SZ_BF16, 64>(p, num_sms, stream) : run<SZ_BF16, 128>(p, num_sms, stream);
    return p.cache.head_dim <= 64 ? run<SZ_FP8_E5M2, 64>(p, num_sms, stream)
                                  : run<SZ_FP8_E5M2, 128>(p, num_sms, stream);
}

}  // namespace sz
