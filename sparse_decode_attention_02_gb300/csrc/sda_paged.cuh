// Attention of the newest tokens of each request over its whole paged cache.
//
//     o = sum_t e^(s_t - m) v_t / sum_t e^(s_t - m),   s_t = scale q.k_t,
//     m = max_t s_t,  over the tokens t that the query token sees.
//
// One pass over the cache: a running maximum, sum and output per query row, in
// fp32; partial results over disjoint token ranges join exactly through their
// log-sum-exps.  A token-row of K|V (2D elements) meets at most 64 query rows,
// a few dozen flops a byte, so the bound is HBM and everything here serves an
// even, uninterrupted stream:
//   * Work split.  All (request, KV group) units' cache tiles form one line, in
//     that order, and CTA c of C takes tiles [cN/C, (c+1)N/C): every CTA streams
//     the same bytes whatever the lengths, found on the device from a prefix
//     sum over seq_lens.  A unit that crosses a CTA boundary leaves a partial
//     output and log-sum-exp per piece (at most two per CTA, so the workspace
//     does not grow with the batch); the join kernel merges them in order.
//   * Four warps, each its own producer and consumer: query rows (query_len x
//     heads) are the M dimension of mma.sync in MT tiles of 16, and the 4 / MT
//     warps of a tile take alternate stages of a shared ring, each with its own
//     running softmax, merged through shared memory when the unit's tiles are
//     done.  A warp that has used up a stage issues the TMA boxes of the stage
//     that comes into its place; it looks pages up a lane a piece, a batch
//     ahead, and runs ahead over unit boundaries.
// Two CTAs an SM: one's prologue and unit ends hide behind the other's stream,
// and eight warps leave each thread the registers for a whole output row tile
// (a producer warp apart would make it nine or ten, 168 registers, and spills).
#pragma once

#include "sda_common.cuh"

#include <algorithm>
#include <type_traits>

namespace sda {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 64;                    // query_len * heads
constexpr int kMaxCtas = 304;                   // two CTAs on each of 152 SMs
constexpr int kJoinThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kRescaleSlack = 8.0f;           // log2 units a running max may lag the true max
constexpr size_t kTaskBytes = kMaxCtas * sizeof(int4);

struct Params {
    const uint16_t *query;
    int64_t q_s0, q_s1;
    const int32_t *block_table;
    int64_t bt_s0;
    const int32_t *seq_lens;
    int64_t len_s;
    uint16_t *output;
    int64_t o_s0, o_s1;
    float *lse;
    int64_t l_s0, l_s1;
    const uint16_t *gate;
    int64_t g_s0, g_s1;
    const float *k_scale, *v_scale;
    unsigned int *flags;
    int4 *tasks;                                // (pieces, request, group, first CTA)
    float *partial;                             // [CTA][continued here / goes on][rows][D]
    float *part_lse;                            // [CTA][2][rows], log2 units
    long long pages;
    unsigned long long wait_ns;
    float scale;
    int requests, groups, heads, query_len, rows;   // rows: query_len * heads
    int table_cols, block, cap;                 // cap: tokens the table's width can hold
    int piece, tile;                            // tokens of a TMA box and of a stage
    int ctas, min_tiles, whole_units, by_unit;
    int q_vec, o_vec;                           // 8-byte loads of q and stores of the output
};

// Tokens of a stage for a cache row of `row_bytes`.
constexpr int stage_slots(int row_bytes)
{
    return row_bytes <= 128 ? 64 : row_bytes <= 384 ? 32 : 16;
}

template <bool FP8, int D, int MT>
struct Shape {
    static constexpr int kElt = FP8 ? 1 : 2;
    static constexpr int kRowBytes = 2 * D * kElt;
    static constexpr int kBands = kRowBytes / 128;
    // Tokens of a stage: 8 to 16 KB of cache; a warp takes a whole stage.
    static constexpr int kSlots = stage_slots(kRowBytes);
    static constexpr int kStageBytes = kSlots * kRowBytes;
    static constexpr int kSteps = D / 16;                       // QK k-steps
    static constexpr int kQBytes = kSteps * 32 * 16;            // a tile's Q fragments
    static constexpr int kChunk = D == 192 ? 48 : 32;           // output dims merged at a time
    static constexpr int kObufStride = kChunk + 4;
    static constexpr int kObufBytes = kWarps * 16 * kObufStride * 4;
    // Q fragments and the merge buffer share their place: Q is dead when a
    // unit's tiles are done.
    static constexpr int kSharedBytes = MT * kQBytes > kObufBytes ? MT * kQBytes : kObufBytes;
    static constexpr int kBudget = 113000;                      // two CTAs an SM
    static constexpr int kFit = (kBudget - kSharedBytes) / kStageBytes;
    static constexpr int kStages = kFit < 12 ? kFit : 12;
    static constexpr int kQOff = kStages * kStageBytes;
    static constexpr int kBarOff = kQOff + kSharedBytes;
    static constexpr int kHdrOff = kBarOff + 16 * kStages;
    static constexpr int kIssuedOff = kHdrOff + 8 * kStages;
    static constexpr int kMlOff = (kIssuedOff + 4 * kStages + 15) / 16 * 16;   // [warp][16][2]
    static constexpr int kRowOff = kMlOff + kWarps * 16 * 8;   // logit scale, gate per row
    static constexpr int kCtlOff = kRowOff + 2 * kMaxRows * 4;
    static constexpr int kBytes = kCtlOff + 128 + 1024;         // + the base's alignment
    static constexpr int kAlternate = kWarps / MT;      // warps of an M tile
    static_assert(kStageBytes % 1024 == 0 && kStages >= 3 && kBytes <= 115712, "ring");
    static_assert(kBarOff % 16 == 0 && kSharedBytes % 16 == 0, "alignment");
};

// The units' tiles in a line, and a CTA's part of it.
struct Segment {
    int request, group, first, last, tiles, len;   // tiles [first, last) of the unit's `tiles`
};

struct Walk {
    long long left;                             // tiles (whole_units: units) still to take
    int request, group, tile;

    static __device__ __forceinline__ int length(const Params &p, int q)
    {
        return min(p.seq_lens[q * p.len_s], p.cap);
    }

    static __device__ __forceinline__ int tiles_of(const Params &p, int len)
    {
        return len > 0 ? (len - 1) / p.tile + 1 : 0;
    }

    __device__ __forceinline__ bool next(const Params &p, Segment &s)
    {
        while (left > 0 && request < p.requests) {
            const int len = length(p, request), tiles = tiles_of(p, len);
            const int first = tile;
            const long long left_in_unit = tiles - first;
            s.request = request;
            s.group = group;
            s.first = first;
            s.tiles = tiles;
            s.len = len;
            const int take = static_cast<int>(p.whole_units ? left_in_unit : min(left, left_in_unit));
            s.last = first + take;
            left -= p.whole_units ? 1 : take;
            tile = first + take;
            if (tile == tiles) {
                tile = 0;
                // an empty request has no tiles in any group
                if (++group == p.groups || (tiles == 0 && !p.whole_units)) {
                    group = 0;
                    ++request;
                }
            }
            if (take > 0)
                return true;
        }
        return false;
    }
};

// ---------------------------------------------------------------------------
// PTX
// ---------------------------------------------------------------------------

__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap *map, int c0, int c1, int c2, int c3,
                                            int c4, uint32_t bar)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(c4), "r"(bar)
        : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr)
{
    uint4 v;
    asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(addr));
    return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
    return v;
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t (&r)[4])
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr));
}

template <bool FP8>
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    if constexpr (FP8) {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    } else {
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
            "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
            : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    }
}

// Two E4M3 bytes (low byte -> low half) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    const uint16_t v = static_cast<uint16_t>(two);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(a), "r"(sel));
    return r;
}

template <bool FP8>
__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    if constexpr (FP8) {
        uint32_t r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
        return r;
    } else {
        return pack_bf16(lo, hi);
    }
}

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// The headwise gate: sigmoid in fp32, rounded to bf16.
__device__ __forceinline__ float gate_factor(uint16_t bits)
{
    const float sig = __fdiv_rn(1.0f, 1.0f + expf(-bf16_bits_to_float(bits)));
    return __bfloat162float(__float2bfloat16_rn(sig));
}

// Token slot of column n (0..7) of an 8-slot score tile.  Columns (2p, 2p + 1)
// are slots (p, p + 4), so that the eight K rows of a shared-memory phase lie
// in eight different swizzled chunks.
__device__ __forceinline__ int slot_of(int n)
{
    return (n >> 1) | ((n & 1) << 2);
}

__device__ __forceinline__ uint64_t low_bits(int n)
{
    return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1ull;
}

// O[16 x D] += P[16 x 16 slots] V[16 slots x D].  `vrow`: this lane's V row for
// ldmatrix (k-slot (mi & 1) * 8 + lane % 8, of the chunk pair's chunk mi >> 1),
// `vsw` its swizzle phase.  bf16: P comes as a rounded part and the rest, so
// that its products carry 16 bits of it.  MASKED zeroes V of slots out of the
// mask (vm0: k-slots 2t, 2t + 1; vm1: 8 + 2t, 9 + 2t), whatever they hold.
template <bool FP8, int D, bool MASKED>
__device__ __forceinline__ void pv_accumulate(float (&o)[D / 8][4], const uint32_t (&pa)[4],
                                              const uint32_t (&pb)[4], uint32_t vrow, uint32_t bstride, int mi,
                                              int vsw, uint32_t vm0, uint32_t vm1)
{
    constexpr int kFirst = D * (FP8 ? 1 : 2) / 16;              // V's first 16-byte chunk of a row
#pragma unroll
    for (int c2 = 0; c2 < kFirst / 2; ++c2) {
        const int idx = kFirst + 2 * c2;
        const int ch = (idx & 7) + (mi >> 1);
        uint32_t r[4];
        ldsm_x4_trans(vrow + (idx >> 3) * bstride + ((ch ^ vsw) << 4), r);
        if constexpr (MASKED) {
            r[0] &= vm0;
            r[1] &= vm1;
            r[2] &= vm0;
            r[3] &= vm1;
        }
        if constexpr (FP8) {
            // a 16-dim chunk is two n8 tiles: its even dims and its odd ones
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const uint32_t x0 = prmt(r[2 * h], 0x3120u), x1 = prmt(r[2 * h + 1], 0x3120u);
                mma16816<true>(o[4 * c2 + 2 * h], pa, e4m3x2_to_f16x2(x0), e4m3x2_to_f16x2(x1));
                mma16816<true>(o[4 * c2 + 2 * h + 1], pa, e4m3x2_to_f16x2(x0 >> 16), e4m3x2_to_f16x2(x1 >> 16));
            }
        } else {
            mma16816<false>(o[2 * c2], pa, r[0], r[1]);
            mma16816<false>(o[2 * c2 + 1], pa, r[2], r[3]);
            mma16816<false>(o[2 * c2], pb, r[0], r[1]);
            mma16816<false>(o[2 * c2 + 1], pb, r[2], r[3]);
        }
    }
}

// ---------------------------------------------------------------------------
// Split kernel
// ---------------------------------------------------------------------------

// The line's length N and where this CTA's part begins; every thread of the
// block calls it.  Returns the tiles to take (0: none).
__device__ __forceinline__ void find_part(const Params &p, long long *scan, int *ctl, Walk &w, long long &x0,
                                          long long &total, int &used)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (p.whole_units) {
        const long long units = static_cast<long long>(p.requests) * p.groups;
        x0 = units * blockIdx.x / p.ctas;
        w.left = units * (blockIdx.x + 1) / p.ctas - x0;
        w.request = static_cast<int>(x0 / p.groups);
        w.group = static_cast<int>(x0 % p.groups);
        w.tile = 0;
        total = units;
        used = p.ctas;
        return;
    }
    const int per = (p.requests + kThreads - 1) / kThreads;
    const int q0 = min(p.requests, static_cast<int>(threadIdx.x) * per), q1 = min(p.requests, q0 + per);
    long long mine = 0;
    for (int q = q0; q < q1; ++q)
        mine += Walk::tiles_of(p, Walk::length(p, q));
    long long inc = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(~0u, inc, o);
        inc += lane >= o ? v : 0;
    }
    if (lane == 31)
        scan[warp] = inc;
    __syncthreads();
    long long before = 0, all = 0;
#pragma unroll
    for (int k = 0; k < kThreads / 32; ++k) {
        before += k < warp ? scan[k] : 0;
        all += scan[k];
    }
    long long at = (before + inc - mine) * p.groups;            // this thread's first tile in the line
    total = all * p.groups;
    used = static_cast<int>(min(static_cast<long long>(p.ctas), (total + p.min_tiles - 1) / p.min_tiles));
    const int c = static_cast<int>(blockIdx.x);
    if (c >= used) {
        w.left = 0;
        x0 = 0;
        return;
    }
    x0 = total * c / used;
    w.left = total * (c + 1) / used - x0;
    if (mine > 0 && x0 >= at && x0 < at + mine * p.groups) {    // one thread
        int q = q0, tiles = 0;
        for (;; ++q) {
            tiles = Walk::tiles_of(p, Walk::length(p, q));
            if (x0 < at + static_cast<long long>(tiles) * p.groups || q + 1 >= q1)
                break;
            at += static_cast<long long>(tiles) * p.groups;
        }
        ctl[0] = q;
        ctl[1] = static_cast<int>((x0 - at) / tiles);
        ctl[2] = static_cast<int>((x0 - at) % tiles);
    }
    __syncthreads();
    w.request = ctl[0];
    w.group = ctl[1];
    w.tile = ctl[2];
}

// A warp's share of the stream: the stages it issues (every kAlternate-th of
// the CTA's), a batch of their pieces looked up a lane a piece, and the next
// batch's table entries on their way.  A batch lies in one segment.
template <bool FP8, int D, int MT>
struct Feed {
    using S = Shape<FP8, D, MT>;
    Walk walk;
    Segment seg;
    int base;                                   // number of the segment's first stage
    int stage;                                  // the next stage to look up
    bool more;
    int per_stage, lane_stage, lane_piece;      // pieces of a stage; this lane's place in a batch
    int at, n, group, page, off, left;          // the batch: next stage to issue, stages, ...
    int n2, group2, page2, off2, left2;         // the one after

    __device__ __forceinline__ void advance(const Params &p)
    {
        while (more && stage >= base + (seg.last - seg.first)) {
            base += seg.last - seg.first;
            more = walk.next(p, seg);
        }
    }

    __device__ __forceinline__ void look_up(const Params &p)
    {
        n = n2;
        group = group2;
        page = page2;
        off = off2;
        left = left2;
        at = 0;
        n2 = 0;
        if (!more)
            return;
        const int P = p.piece, per_block = p.block / P;
        const int ahead = base + (seg.last - seg.first) - stage;       // > 0
        n2 = min(32 / per_stage, (ahead - 1) / S::kAlternate + 1);
        group2 = seg.group;
        const int f = (seg.first + stage - base + lane_stage * S::kAlternate) * per_stage + lane_piece;
        const int col = f / per_block;
        off2 = (f - col * per_block) * P;
        left2 = lane_stage < n2 ? seg.len - f * P : 0;  // tokens from the piece's first on
        // a column past the table is a length past it: cut off with a flag already
        page2 = left2 > 0 && col < p.table_cols ? p.block_table[seg.request * p.bt_s0 + col] : -1;
        stage += n2 * S::kAlternate;
        advance(p);
    }

    __device__ __forceinline__ void start(const Params &p, const Walk &from, int first, int lane)
    {
        walk = from;
        base = 0;
        stage = first;
        per_stage = p.tile / p.piece;
        lane_stage = lane / per_stage;
        lane_piece = lane - lane_stage * per_stage;
        more = walk.next(p, seg);
        advance(p);
        n2 = 0;
        look_up(p);
        look_up(p);
    }

    // Issues the next stage into place `slot`, if there is one.
    __device__ __forceinline__ void issue(const Params &p, const CUtensorMap *tmap, uint32_t ring, uint32_t full,
                                          uint64_t *hdr, int *issued, int slot, int lane)
    {
        if (n == 0)
            return;
        const uint32_t piece_bytes = static_cast<uint32_t>(p.piece) * S::kRowBytes;
        const bool mine = lane_stage == at && left > 0;
        const bool copy = mine && page >= 0 && page < p.pages;
        if (mine && !copy)
            atomicOr(p.flags, SDA_FLAG_BOUNDS);
        const unsigned cb = __ballot_sync(~0u, copy);
        const uint64_t bits = copy ? low_bits(min(p.piece, left)) << (lane_piece * p.piece) : 0ull;
        const unsigned lo = __reduce_or_sync(~0u, static_cast<unsigned>(bits));
        const unsigned hi = S::kSlots > 32 ? __reduce_or_sync(~0u, static_cast<unsigned>(bits >> 32)) : 0u;
        if (lane == 0) {
            hdr[slot] = (static_cast<uint64_t>(hi) << 32) | lo;
            issued[slot] += 1;
            if (cb)
                mbar_expect_tx(full + 8 * slot, __popc(cb) * piece_bytes);
        }
        __syncwarp();
        if (copy)
            tma_load_5d(ring + slot * S::kStageBytes + lane_piece * piece_bytes, tmap, 0, off, 0, group, page,
                        full + 8 * slot);
        if (lane == 0)
            mbar_arrive(full + 8 * slot);
        if (++at == n)
            look_up(p);
    }
};

template <bool FP8, int D, int MT>
__global__ void __launch_bounds__(kThreads, 2)
    sda_paged_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ Params p)
{
    using S = Shape<FP8, D, MT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const uint32_t sbase = smem_u32(smem);
    const uint32_t full_bar = sbase + S::kBarOff, empty_bar = full_bar + 8 * S::kStages;
    uint64_t *hdr = reinterpret_cast<uint64_t *>(smem + S::kHdrOff);
    int *issued = reinterpret_cast<int *>(smem + S::kIssuedOff);
    float *ml = reinterpret_cast<float *>(smem + S::kMlOff);
    float *row_scale = reinterpret_cast<float *>(smem + S::kRowOff);
    float *row_gate = row_scale + kMaxRows;
    int *ctl = reinterpret_cast<int *>(smem + S::kCtlOff);
    long long *scan = reinterpret_cast<long long *>(smem + S::kCtlOff + 16);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S::kStages; ++s) {
            mbar_init(full_bar + 8 * s, 1);
            mbar_init(empty_bar + 8 * s, MT > 1 ? MT - 1 : 1);   // the other warps that take a stage
            issued[s] = 0;
        }
        ctl[3] = 0;                             // a wait ran out
        mbar_init_fence();
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap)) : "memory");
    }
    pdl_launch_dependents();
    pdl_wait();
    __syncthreads();

    Walk walk;
    long long x0, total;
    int used;
    find_part(p, scan, ctl, walk, x0, total, used);

    const int mt = warp / S::kAlternate, turn = warp % S::kAlternate;
    Feed<FP8, D, MT> feed;
    if (mt == 0) {                              // the tile-0 warps issue
        feed.start(p, walk, turn, lane);
        for (int s = turn; s < S::kStages; s += S::kAlternate)
            feed.issue(p, &tmap, sbase, full_bar, hdr, issued, s, lane);
        if (S::kStages % S::kAlternate != 0)    // from now on a stage follows the one whose place it takes
            feed.start(p, walk, turn + S::kStages, lane);
    }

    const int ctid = threadIdx.x;               // 0..127
    const int g = lane >> 2, t = lane & 3;      // fragment row and column pair
    const int H = p.heads, R = p.rows;
    const float ks = FP8 ? __ldg(p.k_scale) : 1.0f, vs = FP8 ? __ldg(p.v_scale) : 1.0f;

    // Requests without tokens: zeros; and no join.
    for (int q = blockIdx.x; q < p.requests; q += gridDim.x) {
        const int len = Walk::length(p, q);
        if (ctid == 0 && p.seq_lens[q * p.len_s] > p.cap)
            atomicOr(p.flags, SDA_FLAG_BOUNDS);
        if (len > 0)
            continue;
        if (p.by_unit && !p.whole_units)
            for (int k = ctid; k < p.groups; k += kThreads)
                p.tasks[q * p.groups + k] = make_int4(0, 0, 0, 0);
        if (len < 0)
            continue;
        for (int e = ctid; e < p.groups * R * D; e += kThreads) {
            const int d = e % D, gr = e / D;    // gr: [token][group][head]
            const int h = gr % H;
            const int64_t row = static_cast<int64_t>(q) * p.query_len * p.groups + gr / H;
            p.output[row * p.o_s0 + h * p.o_s1 + d] = 0;
            if (d == 0 && p.lse)
                p.lse[row * p.l_s0 + h * p.l_s1] = -INFINITY;
        }
    }

    const uint32_t qfrag = sbase + S::kQOff + mt * S::kQBytes;
    float *obuf = reinterpret_cast<float *>(smem + S::kQOff);
    const int r0 = 16 * mt + g, r1 = r0 + 8;    // this thread's query rows
    // query token of each row; rows past R repeat the last token's limits
    const int j0 = min(r0 / H, p.query_len - 1), j1 = min(r1 / H, p.query_len - 1);

    // Shared-memory offsets of this lane's K rows and V rows in a stage.  A
    // stage holds its pieces one after another, each [band][token][128 bytes].
    const uint32_t bstride = static_cast<uint32_t>(p.piece) * 128u;
    const int mi = lane >> 3, vk = (mi & 1) * 8 + (lane & 7);
    const int ksw = slot_of(g), vsw = slot_of(vk & 7);
    auto tile_at = [&](int slot) -> uint32_t {  // byte offset of the 8-slot tile at `slot`
        const int k = slot / p.piece;
        return slot < p.tile ? k * bstride * S::kBands + (slot - k * p.piece) * 128u : 0u;
    };
    constexpr int NT = S::kSlots / 8, KS = S::kSlots / 16, NC = D * S::kElt / 64;
    constexpr uint64_t kAll = S::kSlots >= 64 ? ~0ull : (1ull << S::kSlots) - 1ull;
    uint32_t tile_off[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
        tile_off[i] = tile_at(8 * i);

    // this warp's next stage: its number, place in the ring and parity
    int stage = turn, ring = turn % S::kStages;
    uint32_t parity = static_cast<uint32_t>(turn / S::kStages) & 1u;
    int base = 0;                               // number of the segment's first stage
    bool dead = false;
    bool task_done = false;
    long long x = x0;

    Segment seg;
    while (walk.next(p, seg)) {
        const int len = seg.len;
        const int64_t out_row0 = static_cast<int64_t>(seg.request) * p.query_len * p.groups + seg.group;

        // ---- Query rows: logit scale, gate, fragments.
        auto q_row = [&](int r) -> const uint16_t * {
            const int j = r / H;
            return p.query + (out_row0 + static_cast<int64_t>(j) * p.groups) * p.q_s0 + (r - j * H) * p.q_s1;
        };
        // FP8: the fp16 product takes q scaled by a power of two that puts the
        // row's largest |q| in [2^14, 2^15), undone in the row's logit scale:
        // any bf16 row is exact down to 2^-31 of its largest value.
        constexpr int kPerRow = kThreads / (16 * MT);         // threads that look at a row
        {
            const int r = ctid / kPerRow, part = ctid % kPerRow;
            uint32_t mx = 0;
            if (FP8 && r < R) {
                const uint16_t *q = q_row(r);
                if (p.q_vec) {
                    for (int d = 4 * part; d < D; d += 4 * kPerRow) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(q + d);
                        mx = max(mx, max(max(v.x & 0x7FFFu, (v.x >> 16) & 0x7FFFu),
                                         max(v.y & 0x7FFFu, (v.y >> 16) & 0x7FFFu)));
                    }
                } else {
                    for (int d = part; d < D; d += kPerRow)
                        mx = max(mx, q[d] & 0x7FFFu);
                }
            }
#pragma unroll
            for (int o = 1; o < kPerRow; o <<= 1)
                mx = max(mx, __shfl_xor_sync(~0u, mx, o));
            if (part == 0) {
                const int e = FP8 && mx ? min(126, max(-126, 141 - max(1, static_cast<int>(mx >> 7)))) : 0;
                row_scale[r] = __int_as_float((127 + e) << 23);
                const int j = r / H;
                row_gate[r] = p.gate && r < R
                                  ? gate_factor(p.gate[(static_cast<int64_t>(seg.request) * p.query_len + j) * p.g_s0 +
                                                       static_cast<int64_t>(seg.group * H + r - j * H) * p.g_s1])
                                  : 1.0f;
            }
        }
        __syncthreads();
#pragma unroll 1
        for (int f = warp; f < MT * S::kSteps; f += kWarps) {
            const int m = f / S::kSteps, kk = f - m * S::kSteps;
            // the four dims of k-step kk that thread t's K words hold
            const int d = FP8 ? 64 * (kk >> 2) + 16 * t + 4 * (kk & 3) : 32 * (kk >> 1) + 8 * t + 4 * (kk & 1);
            uint32_t a[4];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 16 * m + g + 8 * k;
                uint32_t w0 = 0, w1 = 0;
                if (r < R) {
                    const uint16_t *q = q_row(r) + d;
                    if (p.q_vec) {
                        const uint2 v = *reinterpret_cast<const uint2 *>(q);
                        w0 = v.x;
                        w1 = v.y;
                    } else {
                        w0 = q[0] | (static_cast<uint32_t>(q[1]) << 16);
                        w1 = q[2] | (static_cast<uint32_t>(q[3]) << 16);
                    }
                }
                if constexpr (FP8) {
                    const float sc = row_scale[r];
                    w0 = pack2<true>(__uint_as_float(w0 << 16) * sc, __uint_as_float(w0 & 0xFFFF0000u) * sc);
                    w1 = pack2<true>(__uint_as_float(w1 << 16) * sc, __uint_as_float(w1 & 0xFFFF0000u) * sc);
                }
                a[k] = w0;
                a[2 + k] = w1;
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(sbase + S::kQOff + m * S::kQBytes +
                                                                          (kk * 32 + lane) * 16),
                         "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3])
                         : "memory");
        }
        __syncthreads();
        // logit scale in log2 units, the q prescale undone (a power of two: exact)
        const float sl0 = p.scale * kLog2e * ks / row_scale[r0], sl1 = p.scale * kLog2e * ks / row_scale[r1];

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};

        const int n_stages = seg.last - seg.first;
        for (; stage < base + n_stages; stage += S::kAlternate) {
            if (!dead) {
                const bool ok = mbar_wait(full_bar + 8 * ring, parity, p.wait_ns);
                if (!__all_sync(~0u, ok)) {
                    if (lane == 0) {
                        atomicOr(p.flags, SDA_FLAG_TIMEOUT);
                        ctl[3] = 1;
                    }
                    dead = true;
                }
            }
            const uint64_t loaded = dead ? 0ull : hdr[ring];
            const int tok0 = (seg.first + stage - base) * p.tile;
            // tokens of the stage that every row sees
            const int common = len - p.query_len + 1 - tok0;
            auto work = [&](auto plain) {
                constexpr bool kPlain = decltype(plain)::value;
                const uint32_t sb = sbase + ring * S::kStageBytes;

                // ---- S = Q K^T: tile i, column g is slot 8i + slot_of(g).
                float sc[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i)
                    sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.0f;
                const uint32_t krow = sb + ksw * 128u;
                constexpr int kGroup = NT < 4 ? NT : 4;   // score tiles, independent chains, at a time
                if constexpr (FP8) {
                    // thread t holds 16 dims a chunk: four k-steps
#pragma unroll
                    for (int i0 = 0; i0 < NT; i0 += kGroup) {
#pragma unroll
                        for (int c = 0; c < NC; ++c) {
                            const uint32_t off = (c >> 1) * bstride + ((((c & 1) * 4 + t) ^ ksw) << 4);
                            uint32_t w[kGroup][4];
#pragma unroll
                            for (int i = 0; i < kGroup; ++i) {
                                const uint4 v = lds128(krow + tile_off[i0 + i] + off);
                                w[i][0] = v.x;
                                w[i][1] = v.y;
                                w[i][2] = v.z;
                                w[i][3] = v.w;
                            }
#pragma unroll
                            for (int k = 0; k < 4; ++k) {
                                const uint4 qv = lds128(qfrag + ((4 * c + k) * 32 + lane) * 16);
                                const uint32_t qf[4] = {qv.x, qv.y, qv.z, qv.w};
#pragma unroll
                                for (int i = 0; i < kGroup; ++i)
                                    mma16816<true>(sc[i0 + i], qf, e4m3x2_to_f16x2(w[i][k]),
                                                   e4m3x2_to_f16x2(w[i][k] >> 16));
                            }
                        }
                    }
                } else {
                    // thread t holds 8 dims a chunk: two k-steps
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        const uint32_t off = (c >> 1) * bstride + ((((c & 1) * 4 + t) ^ ksw) << 4);
                        const uint4 qa = lds128(qfrag + ((2 * c) * 32 + lane) * 16);
                        const uint4 qb = lds128(qfrag + ((2 * c + 1) * 32 + lane) * 16);
                        const uint32_t fa[4] = {qa.x, qa.y, qa.z, qa.w}, fb[4] = {qb.x, qb.y, qb.z, qb.w};
#pragma unroll
                        for (int i0 = 0; i0 < NT; i0 += kGroup) {
                            uint4 kv[kGroup];
#pragma unroll
                            for (int i = 0; i < kGroup; ++i)
                                kv[i] = lds128(krow + tile_off[i0 + i] + off);
#pragma unroll
                            for (int i = 0; i < kGroup; ++i)
                                mma16816<false>(sc[i0 + i], fa, kv[i].x, kv[i].y);
#pragma unroll
                            for (int i = 0; i < kGroup; ++i)
                                mma16816<false>(sc[i0 + i], fb, kv[i].z, kv[i].w);
                        }
                    }
                }

                // ---- Mask; c0/c2 of tile i are slot 8i + t, c1/c3 slot 8i + t + 4.
                float mx0 = -INFINITY, mx1 = -INFINITY;
                if constexpr (kPlain) {
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
                        sc[i][0] *= sl0;
                        sc[i][1] *= sl0;
                        sc[i][2] *= sl1;
                        sc[i][3] *= sl1;
                        mx0 = fmaxf(mx0, fmaxf(sc[i][0], sc[i][1]));
                        mx1 = fmaxf(mx1, fmaxf(sc[i][2], sc[i][3]));
                    }
                } else {
                    const uint64_t s0 = loaded & low_bits(common + j0), s1 = loaded & low_bits(common + j1);
#pragma unroll
                    for (int i = 0; i < NT; ++i) {
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            const int slot = 8 * i + t + 4 * h;
                            sc[i][h] = (s0 >> slot) & 1ull ? sc[i][h] * sl0 : -INFINITY;
                            sc[i][2 + h] = (s1 >> slot) & 1ull ? sc[i][2 + h] * sl1 : -INFINITY;
                        }
                        mx0 = fmaxf(mx0, fmaxf(sc[i][0], sc[i][1]));
                        mx1 = fmaxf(mx1, fmaxf(sc[i][2], sc[i][3]));
                    }
                }

                // ---- Running maximum and sum.  The maximum may lag by
                // kRescaleSlack, so that outputs are seldom rescaled; p <= 2^8.
                mx0 = fmaxf(mx0, __shfl_xor_sync(~0u, mx0, 1));
                mx0 = fmaxf(mx0, __shfl_xor_sync(~0u, mx0, 2));
                mx1 = fmaxf(mx1, __shfl_xor_sync(~0u, mx1, 1));
                mx1 = fmaxf(mx1, __shfl_xor_sync(~0u, mx1, 2));
                if (__any_sync(~0u, mx0 > m_run[0] + kRescaleSlack || mx1 > m_run[1] + kRescaleSlack)) {
                    const float n0 = fmaxf(m_run[0], mx0), n1 = fmaxf(m_run[1], mx1);
                    const float a0 = n0 == -INFINITY ? 1.0f : fast_exp2(m_run[0] - n0);
                    const float a1 = n1 == -INFINITY ? 1.0f : fast_exp2(m_run[1] - n1);
                    m_run[0] = n0;
                    m_run[1] = n1;
                    l_run[0] *= a0;
                    l_run[1] *= a1;
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= a0;
                        o[n][1] *= a0;
                        o[n][2] *= a1;
                        o[n][3] *= a1;
                    }
                }
                const float ref0 = m_run[0] == -INFINITY ? 0.0f : m_run[0];
                const float ref1 = m_run[1] == -INFINITY ? 0.0f : m_run[1];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    sc[i][0] = fast_exp2(sc[i][0] - ref0);      // -inf gives 0
                    sc[i][1] = fast_exp2(sc[i][1] - ref0);
                    sc[i][2] = fast_exp2(sc[i][2] - ref1);
                    sc[i][3] = fast_exp2(sc[i][3] - ref1);
                    l_run[0] += sc[i][0] + sc[i][1];
                    l_run[1] += sc[i][2] + sc[i][3];
                }

                // ---- O += P V.  P in 11 bits (fp16, next to E4M3 values' 4), or
                // bf16 twice: rounded, and what the rounding left.
                const uint64_t seen = kPlain ? kAll : loaded & low_bits(common);
#pragma unroll
                for (int k2 = 0; k2 < KS; ++k2) {
                    const uint32_t km = static_cast<uint32_t>(seen >> (16 * k2)) & 0xFFFFu;
                    if (!kPlain && km == 0)
                        continue;
                    float pr[2][4];
#pragma unroll
                    for (int h = 0; h < 2; ++h)
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            // tokens that only some rows see come below
                            const bool in = kPlain || km == 0xFFFFu || ((km >> (8 * h + t + 4 * (k & 1))) & 1u);
                            pr[h][k] = in ? sc[2 * k2 + h][k] : 0.0f;
                        }
                    uint32_t pa[4], pb[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float lo = pr[k >> 1][2 * (k & 1)], hi = pr[k >> 1][2 * (k & 1) + 1];
                        pa[k] = pack2<FP8>(lo, hi);
                        if constexpr (!FP8)
                            pb[k] = pack2<FP8>(lo - __uint_as_float(pa[k] << 16),
                                               hi - __uint_as_float(pa[k] & 0xFFFF0000u));
                    }
                    const uint32_t vrow = sb + ((mi & 1) ? tile_off[2 * k2 + 1] : tile_off[2 * k2]) + vsw * 128u;
                    if (kPlain || km == 0xFFFFu) {
                        pv_accumulate<FP8, D, false>(o, pa, pb, vrow, bstride, mi, vsw, 0u, 0u);
                    } else {
                        auto both = [&](int s) {
                            return (((km >> s) & 1u) ? 0x0000FFFFu : 0u) | (((km >> (s + 4)) & 1u) ? 0xFFFF0000u : 0u);
                        };
                        pv_accumulate<FP8, D, true>(o, pa, pb, vrow, bstride, mi, vsw, both(t), both(t + 8));
                    }
                }
                // ---- The newest query_len - 1 tokens, which only some rows see:
                // one at a time in fp32, so that a value that is not a number
                // reaches the rows that see it alone.
                if constexpr (!kPlain) {
                for (uint64_t rest = loaded & ~seen & low_bits(common + p.query_len - 1); rest; rest &= rest - 1) {
                    const int s = __ffsll(static_cast<long long>(rest)) - 1;
                    float p0 = 0.0f, p1 = 0.0f;
                    uint32_t off = 0;
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        if ((s >> 3) == i) {
                            p0 = (s & 4) ? sc[i][1] : sc[i][0];
                            p1 = (s & 4) ? sc[i][3] : sc[i][2];
                            off = tile_off[i];
                        }
                    p0 = __shfl_sync(~0u, p0, (lane & ~3) | (s & 3));
                    p1 = __shfl_sync(~0u, p1, (lane & ~3) | (s & 3));
                    const bool see0 = s < common + j0, see1 = s < common + j1;
                    const uint32_t vrow = sb + off + (s & 7) * 128u + 4 * t;
                    constexpr int kFirst = D * S::kElt / 16;
#pragma unroll
                    for (int c = 0; c < kFirst; ++c) {
                        const int idx = kFirst + c;
                        const uint32_t w = lds32(vrow + (idx >> 3) * bstride + (((idx & 7) ^ (s & 7)) << 4));
                        if constexpr (FP8) {
                            const uint32_t a = e4m3x2_to_f16x2(w), b = e4m3x2_to_f16x2(w >> 16);
                            const float2 va = __half22float2(*reinterpret_cast<const __half2 *>(&a));
                            const float2 vb = __half22float2(*reinterpret_cast<const __half2 *>(&b));
                            if (see0) {
                                o[2 * c][0] += p0 * va.x;
                                o[2 * c + 1][0] += p0 * va.y;
                                o[2 * c][1] += p0 * vb.x;
                                o[2 * c + 1][1] += p0 * vb.y;
                            }
                            if (see1) {
                                o[2 * c][2] += p1 * va.x;
                                o[2 * c + 1][2] += p1 * va.y;
                                o[2 * c][3] += p1 * vb.x;
                                o[2 * c + 1][3] += p1 * vb.y;
                            }
                        } else {
                            const float va = __uint_as_float(w << 16), vb = __uint_as_float(w & 0xFFFF0000u);
                            if (see0) {
                                o[c][0] += p0 * va;
                                o[c][1] += p0 * vb;
                            }
                            if (see1) {
                                o[c][2] += p1 * va;
                                o[c][3] += p1 * vb;
                            }
                        }
                    }
                }
                }
            };
            if (loaded == kAll && common >= S::kSlots)
                work(std::true_type{});
            else if (loaded)
                work(std::false_type{});
            // ---- The place is free: the next stage for it.
            __syncwarp();
            if (MT > 1 && mt > 0) {
                if (lane == 0)
                    mbar_arrive(empty_bar + 8 * ring);
            } else if (!dead) {
                if (MT > 1 && !__all_sync(~0u, mbar_wait(empty_bar + 8 * ring, parity, p.wait_ns))) {
                    if (lane == 0) {
                        atomicOr(p.flags, SDA_FLAG_TIMEOUT);
                        ctl[3] = 1;
                    }
                    dead = true;
                } else {
                    feed.issue(p, &tmap, sbase, full_bar, hdr, issued, ring, lane);
                }
            }
            ring += S::kAlternate;
            while (ring >= S::kStages) {
                ring -= S::kStages;
                parity ^= 1u;
            }
        }
        base += n_stages;

        // ---- The unit's (or piece's) result: merge the tile's warps.
        const bool begins = seg.first == 0, ends = seg.last == seg.tiles;
        const bool whole = begins && ends;
        const int64_t piece = static_cast<int64_t>(blockIdx.x) * 2 + (begins ? 1 : 0);
        float l0 = l_run[0], l1 = l_run[1];
        l0 += __shfl_xor_sync(~0u, l0, 1);
        l0 += __shfl_xor_sync(~0u, l0, 2);
        l1 += __shfl_xor_sync(~0u, l1, 1);
        l1 += __shfl_xor_sync(~0u, l1, 2);
        if (t == 0) {
            float *mine = ml + (warp * 16 + g) * 2;
            mine[0] = m_run[0];
            mine[1] = l0;
            mine[16] = m_run[1];
            mine[17] = l1;
        }
        __syncthreads();                         // statistics are there; Q fragments are dead
        float fac[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = 16 * mt + g + 8 * k;
            const float *st = ml + (mt * S::kAlternate * 16 + g + 8 * k) * 2;
            float M = -INFINITY, L = 0.0f;
#pragma unroll
            for (int w = 0; w < S::kAlternate; ++w)
                M = fmaxf(M, st[32 * w]);
#pragma unroll
            for (int w = 0; w < S::kAlternate; ++w)
                L += st[32 * w + 1] * (st[32 * w] == -INFINITY ? 1.0f : fast_exp2(st[32 * w] - M));
            // only a row that saw nothing is empty: a sum that is not a number goes on
            const bool empty = M == -INFINITY && L == 0.0f;
            fac[k] = empty || m_run[k] == -INFINITY ? 0.0f : fast_exp2(m_run[k] - M) / L;
            if (turn == 0 && t == 0 && r < R) {
                const float lse2 = empty ? -INFINITY : M + log2f(L);
                if (!whole)
                    p.part_lse[piece * R + r] = lse2;
                else if (p.lse)
                    p.lse[(out_row0 + static_cast<int64_t>(r / H) * p.groups) * p.l_s0 + (r % H) * p.l_s1] = lse2 * kLn2;
            }
        }
        float *mine = obuf + (warp * 16 + g) * S::kObufStride;
#pragma unroll
        for (int ph = 0; ph < D / S::kChunk; ++ph) {
#pragma unroll
            for (int c = 0; c < S::kChunk / 16; ++c) {
                const int n = ph * (S::kChunk / 8) + 2 * c;     // n8 tiles n, n + 1: 16 dims
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    float *dst = mine + 8 * k * S::kObufStride + 16 * c;
                    const float f = fac[k];
                    if constexpr (FP8) {
                        *reinterpret_cast<float4 *>(dst + 4 * t) =
                            make_float4(o[n][2 * k] * f, o[n + 1][2 * k] * f, o[n][2 * k + 1] * f, o[n + 1][2 * k + 1] * f);
                    } else {
                        *reinterpret_cast<float2 *>(dst + 2 * t) = make_float2(o[n][2 * k] * f, o[n][2 * k + 1] * f);
                        *reinterpret_cast<float2 *>(dst + 8 + 2 * t) =
                            make_float2(o[n + 1][2 * k] * f, o[n + 1][2 * k + 1] * f);
                    }
                }
            }
            __syncthreads();
            constexpr int kVecs = S::kChunk / 4;
            for (int e = ctid; e < R * kVecs; e += kThreads) {
                const int r = e / kVecs, d = 4 * (e - r * kVecs);
                const float *src = obuf + ((r / 16) * S::kAlternate * 16 + r % 16) * S::kObufStride + d;
                float4 v = *reinterpret_cast<const float4 *>(src);
#pragma unroll
                for (int w = 1; w < S::kAlternate; ++w) {
                    const float4 u = *reinterpret_cast<const float4 *>(src + w * 16 * S::kObufStride);
                    v.x += u.x;
                    v.y += u.y;
                    v.z += u.z;
                    v.w += u.w;
                }
                const int dim = ph * S::kChunk + d;
                if (!whole) {
                    *reinterpret_cast<float4 *>(p.partial + (piece * R + r) * D + dim) = v;
                    continue;
                }
                const int j = r / H;
                uint16_t *dst = p.output + (out_row0 + static_cast<int64_t>(j) * p.groups) * p.o_s0 +
                                (r - j * H) * p.o_s1 + dim;
                const float f = vs * row_gate[r];
                const uint2 w = make_uint2(pack_bf16(v.x * f, v.y * f), pack_bf16(v.z * f, v.w * f));
                if (p.o_vec) {
                    *reinterpret_cast<uint2 *>(dst) = w;
                } else {
                    dst[0] = static_cast<uint16_t>(w.x);
                    dst[1] = static_cast<uint16_t>(w.x >> 16);
                    dst[2] = static_cast<uint16_t>(w.y);
                    dst[3] = static_cast<uint16_t>(w.y >> 16);
                }
            }
            __syncthreads();
        }
        // ---- Who joins the unit's pieces: the CTA that holds its first tile says.
        if (!p.whole_units && begins && ctid == 0) {
            int4 task = make_int4(0, 0, 0, 0);
            if (!ends) {
                const long long end = x + seg.tiles;            // past the unit's last tile
                const int last_cta = static_cast<int>((end * used - 1) / total);
                task = make_int4(last_cta - static_cast<int>(blockIdx.x) + 1, seg.request, seg.group, blockIdx.x);
            }
            if (p.by_unit)
                p.tasks[seg.request * p.groups + seg.group] = task;
            else if (!ends)
                p.tasks[blockIdx.x] = task;
        }
        task_done = task_done || (begins && !ends);
        x += n_stages;
    }
    if (!p.whole_units && !p.by_unit && !task_done && ctid == 0)
        p.tasks[blockIdx.x] = make_int4(0, 0, 0, 0);

    // After a wait that ran out, copies may be in flight: they land before the
    // block's memory can go to another.
    __syncthreads();
    if (ctl[3] && ctid < S::kStages && issued[ctid] > 0 &&
        !mbar_wait(full_bar + 8 * ctid, static_cast<uint32_t>(issued[ctid] - 1) & 1u, kDrainLimitNs))
        atomicOr(p.flags, SDA_FLAG_TIMEOUT);
}

template <bool FP8, int D, int MT>
sda_status launch_shape(const CUtensorMap &tmap, const Params &p, void *stream)
{
    using S = Shape<FP8, D, MT>;
    static size_t raised[64] = {};
    if (!raise_smem(sda_paged_kernel<FP8, D, MT>, S::kBytes, raised))
        return SDA_ERR_CUDA;
    return launch_pdl(sda_paged_kernel<FP8, D, MT>, dim3(static_cast<unsigned>(p.ctas)), dim3(kThreads), S::kBytes,
                      stream, tmap, p);
}

template <int D>
sda_status launch_dim(bool fp8, const CUtensorMap &tmap, const Params &p, void *stream)
{
    const int tiles = (p.rows + 15) / 16;       // of 16 query rows; three make four
    if (fp8)
        return tiles == 1   ? launch_shape<true, D, 1>(tmap, p, stream)
               : tiles == 2 ? launch_shape<true, D, 2>(tmap, p, stream)
                            : launch_shape<true, D, 4>(tmap, p, stream);
    return tiles == 1   ? launch_shape<false, D, 1>(tmap, p, stream)
           : tiles == 2 ? launch_shape<false, D, 2>(tmap, p, stream)
                        : launch_shape<false, D, 4>(tmap, p, stream);
}

// One translation unit per head size.
sda_status launch_64(bool fp8, const CUtensorMap &tmap, const Params &p, void *stream);
sda_status launch_128(bool fp8, const CUtensorMap &tmap, const Params &p, void *stream);
sda_status launch_192(bool fp8, const CUtensorMap &tmap, const Params &p, void *stream);
sda_status launch_256(bool fp8, const CUtensorMap &tmap, const Params &p, void *stream);

}  // namespace paged
}  // namespace sda
