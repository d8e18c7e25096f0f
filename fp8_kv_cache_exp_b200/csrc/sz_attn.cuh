// sz_attn.cuh -- what the attention kernels share: how the work is cut and
// shared out, how partial results are joined, and values that are not finite.
//
// A tile is TR rows of one sequence and one KV head: a row is a (token, query
// head of the group) pair, row r being token r / G, head r % G, so that one
// pass over keys and values serves all query heads that share them.  A tile's
// work is counted in blocks of BN places that any of its rows sees.  The
// blocks of all tiles, in the order (KV head, sequence, tile, block), are dealt
// out evenly and in runs: CTA c of C has floor(U / C) of them, and one more if
// c < U mod C.  A tile counts EXTRA blocks more than it has, in front, for what
// it costs besides them (queries to fetch, results to write).  A tile that
// falls to several CTAs is joined from their partial results, in the order of
// the CTAs, by the one that finishes last; so the result does not depend on
// which one that is.
#pragma once

#include <cuda_fp16.h>

#include "sz_ops.cuh"

namespace sz {

constexpr float kLn2 = 0.69314718055994531f;

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

struct SeqInfo {
    uint32_t q0, q_len, kv;
};

__device__ __forceinline__ SeqInfo seq_info(const AttnParams &p, uint32_t b) {
    const int32_t a = __ldg(p.cu_q + b), e = __ldg(p.cu_q + b + 1), n = __ldg(p.kv_len + b);
    SeqInfo s;
    const int32_t last = int32_t(p.tokens);
    const int32_t a1 = a < 0 ? 0 : (a > last ? last : a), e1 = e > last ? last : e;
    s.q0 = uint32_t(a1);
    s.q_len = e1 > a1 ? uint32_t(e1 - a1) : 0u;
    s.kv = n < 0 ? 0u : (uint32_t(n) > p.cache.capacity ? p.cache.capacity : uint32_t(n));
    return s;
}

// Places that a token sees: [lo, hi).
struct Range {
    uint32_t lo, hi;
};
__device__ __forceinline__ Range token_range(const AttnParams &p, const SeqInfo &s, uint32_t i) {
    const int64_t at = int64_t(s.kv) - int64_t(s.q_len) + int64_t(i);
    int64_t hi = p.causal ? at + 1 : int64_t(s.kv);
    if (hi < 0) hi = 0;
    int64_t lo = p.window ? at - int64_t(p.window) + 1 : 0;
    if (lo < 0) lo = 0;
    if (lo > hi) lo = hi;
    return Range{uint32_t(lo), uint32_t(hi)};
}

// Places that any row of a tile sees.  The first token's window reaches
// furthest back, the last token sees furthest.
template <int TR>
__device__ __forceinline__ Range tile_range(const AttnParams &p, const SeqInfo &s, uint32_t tile) {
    const uint32_t rows = s.q_len * p.group.d;
    const uint32_t r1 = min((tile + 1) * uint32_t(TR), rows) - 1;
    const Range a = token_range(p, s, div_by(tile * TR, p.group)), b = token_range(p, s, div_by(r1, p.group));
    return Range{a.lo < b.hi ? a.lo : b.hi, b.hi};
}

template <int BN>
__device__ __forceinline__ uint32_t range_blocks(const Range &r) {
    const uint32_t n = (r.hi + BN - 1) / BN - r.lo / BN;
    return n > 0 ? n : 1;  // a tile whose rows see nothing has its zeros to write
}

template <int TR>
__device__ __forceinline__ uint32_t seq_tiles(const AttnParams &p, const SeqInfo &s) {
    return (s.q_len * p.group.d + TR - 1) / TR;
}

// Quotient and remainder; nearly always of numbers that fit 32 bits.
__device__ __forceinline__ uint64_t quotient(uint64_t a, uint64_t b) {
    return ((a | b) >> 32) == 0 ? uint64_t(uint32_t(a) / uint32_t(b)) : a / b;
}

// Where a CTA stands in its share of the blocks.
struct Work {
    uint64_t at, end;       // next block of the share, its end (global numbers)
    uint64_t each;          // blocks of a share ...
    uint32_t more;          // ... and the number of CTAs, the first ones, that have one more
    uint32_t head, seq, tile;
    uint32_t from;          // the block of the tile at which `at` stands
    uint32_t whole;         // not 0: whole tiles, so many to a head; then `at` counts this CTA's
};
constexpr uint32_t kFewTiles = 32;  // of a head, for work_begin_few

template <int NT>
struct WorkScratch {
    uint64_t warp[NT / 32];
    uint64_t found_at;
    uint32_t tp[NT], q_len[NT], kv[NT];
    uint32_t found[3];
};

template <int NT>
__device__ __forceinline__ uint64_t block_scan64(uint64_t v, uint64_t *s_warp, uint64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint64_t x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    __syncthreads();
    if (lane == 31) s_warp[warp] = x;
    __syncthreads();
    uint64_t before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) {
        const uint64_t s = s_warp[w];
        before += (w < warp) ? s : 0u;
        all += s;
    }
    *total = all;
    return before + x - v;
}

// The share of CTA blockIdx.x of `per_head` blocks a head, up to the tile that it begins in.
__device__ __forceinline__ uint64_t work_share(const AttnParams &p, uint64_t per_head, Work &w) {
    const uint64_t total = per_head * p.cache.kv_heads;
    w.each = quotient(total, gridDim.x);
    w.more = uint32_t(total - w.each * gridDim.x);
    w.at = w.each * blockIdx.x + min(blockIdx.x, w.more);
    w.end = w.at + w.each + (blockIdx.x < w.more ? 1 : 0);
    w.head = per_head ? uint32_t(quotient(w.at, per_head)) : 0;
    return w.at - w.head * per_head;
}

// Whole tiles of a head in `order` (sequence << 8 | tile), the longest first: CTA
// c of C has every C-th of all heads' tiles, forwards and backwards in turn.
__device__ __forceinline__ bool work_whole(const AttnParams &p, Work &w, const uint16_t *order) {
    const uint64_t row = w.at * gridDim.x;
    const uint64_t x = row + ((w.at & 1) ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
    if (x >= uint64_t(w.whole) * p.cache.kv_heads) return false;
    const uint32_t rank = uint32_t(x) / p.cache.kv_heads;
    w.head = uint32_t(x) - rank * p.cache.kv_heads;
    w.seq = order[rank] >> 8;
    w.tile = order[rank] & 255;
    w.from = 0;
    return true;
}

// The same for at most 32 sequences with at most 32 tiles together, each warp by
// itself: the block's way (below) costs a call of one token 2 us.  Says whether
// it was possible; then `has` is whether the CTA has a share.
//
// With `order`, tiles of at most kWholeMost blocks that are at least as many as
// the CTAs are not cut: a part of a tile costs its queries, its results and their
// joining, as much as three to four blocks, and cutting saves half a tile.  Whole
// and cut, on 148 CTAs: two 1024-token prompts of 32 heads of 80 (tiles of 2 to 8
// blocks) 35 and 45 us; equal tiles of 8 blocks (64 tokens over 1024 places, 32
// heads on 8 of 128), 152 of them 49 and 47, 192: 52 and 57, 240: 53 and 66; 152 of
// 4 blocks 31 and 35.  A limit of 4 cuts the tiles of 8.  Longer tiles of prompts
// would gain too: two of 1152 tokens 43 us whole, 54 as they are, of 2048 87 and 96;
// of few equal long tiles a second round costs more than cutting them.  (All
// threads call it then, and each has `order` behind the next barrier.)
constexpr uint32_t kWholeMost = 8;
template <int TR, int BN, int EXTRA>
__device__ __forceinline__ bool work_begin_few(const AttnParams &p, Work &w, bool &has, uint16_t *order) {
    const uint32_t lane = threadIdx.x & 31, seqs = p.cache.seqs;
    if (seqs > 32) return false;
    SeqInfo si{0, 0, 0};
    if (lane < seqs) {
        si = seq_info(p, lane);
        if (blockIdx.x == 0 && threadIdx.x < 32 && __ldg(p.kv_len + lane) > int32_t(p.cache.capacity))
            set_error(p.ctl, SZ_ERR_INVALID_ARG, lane);
    }
    const uint32_t tiles = seq_tiles<TR>(p, si);
    if (__any_sync(0xffffffffu, tiles > 32)) return false;
    uint32_t ends = tiles;  // of this lane's sequence's tiles
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, ends, o);
        if (lane >= o) ends += y;
    }
    const uint32_t count = __shfl_sync(0xffffffffu, ends, 31);
    if (count > 32) return false;
    uint32_t seq = 0;  // of tile `lane`: the number of sequences that end at or before it
#pragma unroll
    for (int step = 16; step > 0; step >>= 1)
        if (__shfl_sync(0xffffffffu, ends, int(seq + step - 1)) <= lane) seq += step;
    seq = min(seq, 31u);
    const uint32_t q_len = __shfl_sync(0xffffffffu, si.q_len, int(seq)), kv = __shfl_sync(0xffffffffu, si.kv, int(seq));
    const uint32_t tile = lane - __shfl_sync(0xffffffffu, ends - tiles, int(seq));
    const uint32_t units =
        lane < count ? EXTRA + range_blocks<BN>(tile_range<TR>(p, SeqInfo{0, q_len, kv}, tile)) : 0;
    w.whole = 0;
    if (order && uint64_t(count) * p.cache.kv_heads >= gridDim.x &&
        !__any_sync(0xffffffffu, units > EXTRA + kWholeMost)) {
        uint32_t rank = 0;
#pragma unroll 8
        for (int j = 0; j < 32; ++j) {
            const uint32_t other = __shfl_sync(0xffffffffu, units, j);
            rank += other > units || (other == units && j < int(lane));
        }
        if (threadIdx.x < 32 && lane < count) order[rank] = uint16_t(seq << 8 | tile);
        w.whole = count;
        w.at = 0;
        __syncthreads();
        has = work_whole(p, w, order);
        return true;
    }
    uint64_t to = units;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint64_t y = __shfl_up_sync(0xffffffffu, to, o);
        if (lane >= o) to += y;
    }
    const uint64_t target = work_share(p, __shfl_sync(0xffffffffu, to, 31), w);
    has = w.at < w.end;
    if (!has) return true;
    const int src = __ffs(__ballot_sync(0xffffffffu, target < to && target >= to - units)) - 1;
    w.seq = __shfl_sync(0xffffffffu, seq, src);
    w.tile = __shfl_sync(0xffffffffu, tile, src);
    w.from = uint32_t(target - __shfl_sync(0xffffffffu, to - units, src));
    has = w.from + (w.end - w.at) > EXTRA;
    return true;
}

// The CTA's share; false if it has none.  All NT threads call it.
template <int NT, int TR, int BN, int EXTRA>
__device__ bool work_begin(const AttnParams &p, WorkScratch<NT> &s, Work &w, uint16_t *order = nullptr) {
    bool has;
    if (work_begin_few<TR, BN, EXTRA>(p, w, has, order)) return has;
    w.whole = 0;
    const uint32_t tid = threadIdx.x, seqs = p.cache.seqs;
    // this thread's tile of the chunk looked at last
    uint32_t seq = 0, tile = 0, units = 0, chunks = 0;
    uint64_t before = 0;
    auto note = [&](uint64_t target) {
        if (units > 0 && target >= before && target - before < units) {
            s.found[0] = seq;
            s.found[1] = tile;
            s.found[2] = uint32_t(target - before);
        }
    };
    // blocks of all tiles of one head; with `find`, notes the tile that block `target` falls in
    auto scan = [&](bool find, uint64_t target) {
        uint64_t run = 0;
        for (uint32_t sb = 0; sb < seqs; sb += NT) {
            const uint32_t b = sb + tid;
            uint32_t tiles = 0;
            if (b < seqs) {
                const SeqInfo si = seq_info(p, b);
                tiles = seq_tiles<TR>(p, si);
                s.q_len[tid] = si.q_len;
                s.kv[tid] = si.kv;
                if (!find && blockIdx.x == 0 && __ldg(p.kv_len + b) > int32_t(p.cache.capacity))
                    set_error(p.ctl, SZ_ERR_INVALID_ARG, b);
            }
            uint64_t count;
            s.tp[tid] = uint32_t(block_scan64<NT>(tiles, s.warp, &count));
            __syncthreads();
            for (uint32_t tb = 0; tb < uint32_t(count); tb += NT) {
                const uint32_t t = tb + tid;
                units = 0;
                if (t < uint32_t(count)) {
                    uint32_t j = 0, hi = min(seqs - sb, uint32_t(NT));  // tp[j] <= t < tp[hi]
                    while (hi - j > 1) {
                        const uint32_t mid = (j + hi) / 2;
                        if (s.tp[mid] <= t) j = mid; else hi = mid;
                    }
                    seq = sb + j;
                    tile = t - s.tp[j];
                    units = EXTRA + range_blocks<BN>(tile_range<TR>(p, SeqInfo{0, s.q_len[j], s.kv[j]}, tile));
                }
                uint64_t sum;
                before = run + block_scan64<NT>(units, s.warp, &sum);
                run += sum;
                ++chunks;
                if (find) note(target);
            }
            __syncthreads();
        }
        return run;
    };
    const uint64_t per_head = scan(false, 0);
    const uint64_t target = work_share(p, per_head, w);
    if (w.at == w.end) return false;
    if (chunks == 1) note(target);  // the one chunk is still at hand
    else scan(true, target);
    __syncthreads();
    w.seq = s.found[0];
    w.tile = s.found[1];
    w.from = s.found[2];
    __syncthreads();
    return w.from + (w.end - w.at) > EXTRA;
}

// The CTA that has a block.
__device__ __forceinline__ uint32_t work_owner(const Work &w, uint64_t block) {
    const uint64_t longer = (w.each + 1) * w.more;
    return block < longer ? uint32_t(quotient(block, w.each + 1))
                          : w.more + uint32_t(quotient(block - longer, w.each));
}

// A CTA's part of a tile: blocks [from, to) of its n.
struct Part {
    SeqInfo s;
    Range r;
    uint32_t rows, r0;      // rows of the tile, the first of them
    uint32_t block0;        // the tile's first block
    uint32_t from, to, n;
    uint32_t count;         // of the share's blocks, the extra ones among them
    uint32_t c_first, c_last;  // CTAs that share the tile
};

template <int TR, int BN, int EXTRA>
__device__ __forceinline__ Part work_part(const AttnParams &p, const Work &w, uint32_t cta) {
    Part t;
    t.s = seq_info(p, w.seq);
    t.r = tile_range<TR>(p, t.s, w.tile);
    t.r0 = w.tile * TR;
    t.rows = min(uint32_t(TR), t.s.q_len * p.group.d - t.r0);
    t.block0 = t.r.lo / BN;
    t.n = range_blocks<BN>(t.r);
    const uint32_t to = w.whole ? EXTRA + t.n : uint32_t(min(uint64_t(EXTRA + t.n), w.from + (w.end - w.at)));
    t.count = to - w.from;
    t.from = w.from > EXTRA ? w.from - EXTRA : 0;
    t.to = to - EXTRA;  // (work_begin and work_next leave no part without blocks of its own)
    if (t.from == 0 && t.to == t.n) {
        t.c_first = t.c_last = cta;
    } else {
        const uint64_t x0 = w.at - w.from + EXTRA;
        t.c_first = work_owner(w, x0);
        t.c_last = work_owner(w, x0 + t.n - 1);
    }
    return t;
}

// On to the next tile; false at the end of the share.
template <int TR, int EXTRA>
__device__ __forceinline__ bool work_next(const AttnParams &p, Work &w, const Part &t, const uint16_t *order = nullptr) {
    if (w.whole) {
        ++w.at;
        return work_whole(p, w, order);
    }
    w.at += t.count;
    if (w.at + EXTRA >= w.end) return false;
    w.from = 0;
    if (++w.tile < seq_tiles<TR>(p, t.s)) return true;
    w.tile = 0;
    do {
        if (++w.seq == p.cache.seqs) {
            w.seq = 0;
            if (++w.head >= p.cache.kv_heads) return false;  // only if cu_q changed under the call
        }
    } while (seq_info(p, w.seq).q_len == 0);
    return true;
}

// Slot of a CTA's partial result: the tile that it takes over from another
// CTA, or the one that it leaves to the next.
__device__ __forceinline__ uint32_t part_slot(uint32_t c, const Part &t) { return 2 * c + (c == t.c_first ? 1 : 0); }

// Values that are not finite.  In the products a place that a row does not see
// has the weight 0, and 0 times an infinity is NaN.  Only at a tile's edges, the
// places that some of its rows see and others do not, can a row meet such a
// place.  There values that are not finite go into the products as 0, and what
// they add to the rows that see them is added to those rows' sums by itself.  An
// edge is at most as long as the tile's tokens are many, so this costs little
// however long the context is (doing a row again, place by place, took 100 ms
// for 512 tokens over 16,384 places with one NaN among the tokens).

// Places that every row of a tile sees: part of what any of them sees, or, if
// there are none, [hi, hi) of that.
__device__ __forceinline__ Range seen_by_all(const AttnParams &p, const Part &t) {
    const uint32_t hi = token_range(p, t.s, div_by(t.r0, p.group)).hi;
    const uint32_t lo = token_range(p, t.s, div_by(t.r0 + t.rows - 1, p.group)).lo;
    return lo < hi ? Range{lo, hi} : Range{t.r.hi, t.r.hi};
}

// Blocks of a tile that hold edges: those before `lo` and from `hi` on.
struct EdgeBlocks {
    uint32_t lo, hi;
    __device__ __forceinline__ bool has(uint32_t j) const { return j < lo || j >= hi; }
};
template <int BN>
__device__ __forceinline__ EdgeBlocks edge_blocks(const AttnParams &p, const Part &t) {
    const Range all = seen_by_all(p, t);
    return EdgeBlocks{t.r.lo < all.lo ? (all.lo + BN - 1) / BN - t.block0 : 0,
                      t.r.hi > all.hi ? all.hi / BN - t.block0 : 0xffffffffu};
}

// Whether some of [lo, hi), places of the tile, are edges.
__device__ __forceinline__ bool has_edges(const Range &all, uint32_t lo, uint32_t hi) {
    return lo < hi && (lo < all.lo || hi > all.hi);
}

// Bits of kNotFinite are set for values with an exponent of ones only: one step of
// the exponent more carries to the sign's bit, and no further.
template <int DT>
constexpr uint32_t kNotFinite = DT == SZ_BF16 ? 0x80008000u : 0x80808080u;
template <int DT>
__device__ __forceinline__ uint32_t carries(uint32_t w) {
    return (w & ~kNotFinite<DT>) + (DT == SZ_BF16 ? 0x00800080u : 0x04040404u);
}
template <int DT>
__device__ __forceinline__ uint32_t carries(const uint4 &v) {
    return carries<DT>(v.x) | carries<DT>(v.y) | carries<DT>(v.z) | carries<DT>(v.w);
}
// 16 bytes of values, with 0 for those that are not finite; says whether there were any.
template <int DT>
__device__ __forceinline__ uint32_t finite_only(uint32_t w) {
    constexpr uint32_t shift = DT == SZ_BF16 ? 15 : 7;
    const uint32_t ones = (carries<DT>(w) & kNotFinite<DT>) >> shift;  // 1 in the lowest bit of each such value
    return w & ~(ones * (DT == SZ_BF16 ? 0xffffu : 0xffu));
}
template <int DT>
__device__ __forceinline__ bool make_finite(uint4 &v) {
    if ((carries<DT>(v) & kNotFinite<DT>) == 0) return false;
    v = make_uint4(finite_only<DT>(v.x), finite_only<DT>(v.y), finite_only<DT>(v.z), finite_only<DT>(v.w));
    return true;
}

// Adds to N of a row's sums, columns col.., the values that are not finite of the
// edges among places [from, to) that the row sees.
template <int DT, int N>
__device__ __forceinline__ void add_not_finite(const AttnParams &p, uint32_t seq, uint32_t kvh, const Range &row,
                                               const Range &all, uint32_t from, uint32_t to, uint32_t col, float *sum) {
    const int32_t *ids = p.cache.table + uint64_t(seq) * p.cache.table_stride;
    const uint64_t first = uint64_t(kvh) * p.cache.head_dim + col;
    to = min(to, row.hi);
#pragma unroll 1
    for (uint32_t t = max(from, row.lo); t < to; ++t) {
        if (t >= all.lo && t < all.hi) {
            t = all.hi - 1;
            continue;
        }
        const uint64_t off = place_offset(p.cache, p.ctl, ids, t);
        if (off == kBadOffset) continue;
        if constexpr (DT == SZ_BF16) {
            const uint2 *at = reinterpret_cast<const uint2 *>(p.cache.v + off + first * 2);
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                const uint2 w = __ldg(at + j / 4);
                const float v[4] = {bf16_lo(w.x), bf16_hi(w.x), bf16_lo(w.y), bf16_hi(w.y)};
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (!(fabsf(v[e]) < INFINITY)) sum[j + e] += v[e];
            }
        } else {
            const uint32_t *at = reinterpret_cast<const uint32_t *>(p.cache.v + off + first);
#pragma unroll
            for (int j = 0; j < N; j += 4) {
                const uint32_t w = __ldg(at + j / 4);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const float v = __half2float(__ushort_as_half(uint16_t((w >> (8 * e) & 0xff) << 8)));
                    if (!(fabsf(v) < INFINITY)) sum[j + e] += v;
                }
            }
        }
    }
}

}  // namespace sz
