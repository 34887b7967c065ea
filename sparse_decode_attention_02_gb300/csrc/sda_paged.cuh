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
//   * Workers.  Query rows (query_len x heads) are the M dimension of mma.sync
//     in MT tiles of 16; a worker is MT warps, one a tile, with a ring of
//     stages of its own.  Workers never wait for one another: a worker's Q
//     fragments and output live in registers, so the end of a short request
//     stalls one warp of an SM's eight and not a whole CTA.
//   * Work split.  All (request, KV group) units' cache tiles form one line, in
//     that order, each unit lengthened by what its end costs; worker v of V
//     takes the line from vN/V to (v+1)N/V: equal shares whatever the lengths,
//     found on the device from a prefix sum over seq_lens.  A unit that crosses
//     a boundary leaves a partial output and log-sum-exp per piece (at most two
//     per worker, so the workspace does not grow with the batch); the join
//     kernel merges them in order.
//   * A worker's first warp issues the TMA boxes of the stage that comes into
//     the place just used up; it looks pages up a lane a piece, a batch ahead,
//     and runs ahead over unit boundaries.
//   * Short units (a table of few tiles) are not put on the line: a worker takes
//     each whole, or where they are few a CTA does (ALONE), its workers a share of
//     the tiles each, and merges them itself; nothing is left for the join (46
//     requests of 211 tokens, E4M3: 16.7 us cut and joined, 8.4 alone).
// Two CTAs of four warps an SM: eight warps leave each thread the registers for
// a tile's whole Q and output (at 168 registers, with a producer warp, they spilled:
// the third case below 1296 us).
//
// Measured, with a copy at 6.68 TB/s: 64 chats of 8K to 32K tokens (bf16, 192 dims,
// 2 groups) 302 to 308 us, 6.6 TB/s; 12 requests of 64K to 128K with two new tokens (bf16,
// 192, 4 groups, 32 rows) 534 to 543 us, 6.9 TB/s; 16 documents of 128K to 256K (E4M3, 192,
// 4 groups) 713 to 724 us, 7.0 TB/s; one of 261,001 alone 76 us, 5.3 TB/s; 188 of up to 2500
// tokens over pages of 16 (E4M3, 128, 4 groups) 57 us, 4.5 TB/s, where the start and
// the join are a third; one of 40 tokens 5.0 to 5.6 us, latency.  E4M3 with 32 rows (192
// dims) reaches 0.6 of the copy rate, with 64 rows 0.34: there the bound is the chain
// of scores, softmax and products that two warps a scheduler overlap (tensor pipe
// 49 %).  Halving the conversions there, with weights exchanged between two warps,
// lengthened that chain (145 -> 160 us).
//
// Two more kinds of cache have elements of a byte and a scale for each block of tokens and
// head, one for keys, which multiplies logits, one for values, which multiplies weights;
// and of those a row's selected regions can be walked instead of a request's tokens.
// 16 documents of 64K to 128K tokens (192 dims, 4 groups): E4M3 377 to 380 us, 6.6 TB/s
// (one scale for all: 370 to 376), integers 414, 6.1 TB/s, bound by their conversions; 512 rows of
// 1024 regions of 8 tokens (E4M3, 192 dims) 284 us, 5.7 TB/s, in TMA boxes of 3 KB.
#pragma once

#include "sda_quant.cuh"

#include <algorithm>
#include <type_traits>

namespace sda {
namespace paged {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxRows = 64;                    // query_len * heads
constexpr int kMaxRegionHeads = 16;             // of a row that attends over regions
constexpr int kSms = 152;
constexpr int kMaxWorkers = kSms * 2 * kWarps;  // two CTAs of them on each SM (or three of two)
// Tiles that a unit's end is worth on the line (188 requests of up to 2500 tokens, then
// at 59 us with four: none 76, eight 61).  Of a quantised cache two: its tiles take
// longer, and few are cut finer (six rows of 2048 selected tokens, integers: 21.1 us
// with four, 16.4; 188 requests of up to 2500 77.2, 75.1).
constexpr int unit_cost(bool scaled)
{
    return scaled ? 2 : 4;
}
// A worker takes at least this many tiles before the line is cut finer (one request
// of 1198 tokens x 4 groups: 14.5 us, with two 14.9).
constexpr int kMinTiles = 1;
constexpr int kJoinThreads = 256;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kManyPieces = 32;                 // more and a row is joined by a whole block (up to it a lane a piece)
// Join items: eight rows of a unit, or a row of one in more than kManyPieces pieces.
constexpr int kMaxItems = kMaxWorkers * (kMaxRows / kJoinWarps);
constexpr int kItemWord = 16, kTicketWord = 17; // of the workspace header: items listed, join blocks done
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// What the cache holds: bf16; E4M3 with a scale for all keys and one for all values;
// E4M3 or integers with scales of their own for each block of tokens and head.  All
// one-byte kinds are multiplied in fp16, which holds them exactly.
enum Kind { kBf16, kE4m3, kScaledE4m3, kScaledInt8 };

// What a unit's tiles are: a request's tokens, or a row's selected regions, as many as
// its list has room for or as the extent kernel found (a run-time choice of the two in
// one kernel: 512 rows of 1024 regions 300 us, so 292).
enum Walked { kTokens, kRegions, kExtents };

// Who takes a unit: workers of the line, their pieces joined by another kernel (4 to 6 us of a
// small call); a CTA alone; or a cluster of CTAs, which merge through one another's shared
// memory in the same kernel.
enum Takers { kOnLine, kCta, kCluster };
constexpr int kMaxCluster = 8;

struct JoinItem {
    int pieces, request, group, first;          // the unit, and the worker with its first piece
    int row, rows, spare[2];                    // query rows of the item
};
constexpr size_t kItemBytes = kMaxItems * sizeof(JoinItem);

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
    const float *scales;                        // quantised caches: (key, value) pairs
    int64_t s_s0, s_s1, s_s2;
    // Regions: a unit is a row, p.requests rows of one group each.
    const int32_t *regions;
    int64_t reg_s0;
    const int32_t *positions;
    int64_t pos_s;
    const uint8_t *active;
    int64_t act_s;
    int32_t *extents;                           // NULL or, written by the extent kernel, Walk::length of each row
    unsigned int *flags;
    JoinItem *items;
    float *partial;                             // [worker][continued here / goes on][rows][D]
    float *part_lse;                            // [worker][2][rows], log2 units
    long long pages;
    unsigned long long wait_ns;
    float scale;
    int requests, groups, heads, query_len, rows;   // rows: query_len * heads
    int head_inv;                               // ceil(2^16 / heads): r * head_inv >> 16 is r / heads for r < 64
    int table_cols, block, cap;                 // cap: tokens the table's width can hold
    int piece, tile;                            // tokens of a TMA box and of a stage
    int ctas, workers, whole_units, cta_units;   // cta_units: ALONE
    int cluster;                                // CTAs of a unit: 1 or, a power of two, of a cluster
    unsigned long long per_block_inv, tile_inv, workers_inv;    // inverse_of the pieces of a page, tile, workers
    int q_vec, o_vec;                           // 8-byte loads of q and stores of the output
    unsigned long long span_inv, block_inv, per_region_inv, region_groups_inv, request_rows_inv;
    int per_region, region_tokens;              // pieces and tokens of a region
    int region_groups, request_rows;            // KV groups (0: no regions), rows that share a line of the table
    int listed;                                 // regions of a row's list
    int clear_inactive, one_scale;              // one_scale: a piece's tokens have one pair of scales
};

// Tokens of a stage for a cache row of `row_bytes`: 6 to 12 KB of cache where a
// worker is one warp (its ring is a quarter of the CTA's 96 KB), twice that for
// wider rows where warps share a worker's stages: more independent products a
// step, fewer hand-overs (two tiles of bf16, 192 dims: 571 us with 16 tokens, 542
// with 32).  Smaller stages leave more of them in flight, but the products less
// at a time: bf16, 192 dims, 306 us with 16 tokens, 322 with 8; E4M3, 128 dims,
// 59 with 32, 62 with 16.  Rows of 384 bytes lie between: 742 us with 32 tokens
// (two stages a worker), 713 with 16; a CTA alone with a unit has few of them
// (700 tokens 13.5 us with 32, 15.1 with 16).
constexpr int stage_slots(int row_bytes, int mt, bool alone)
{
    const int middle = alone ? 384 : 256;
    const int slots = row_bytes <= 128 ? 64 : row_bytes <= middle ? 32 : row_bytes <= 768 ? 16 : 8;
    return mt > 1 && row_bytes > middle ? 2 * slots : slots;
}

// CTAs that share an SM.  The products of several tiles of 64 dims gain from a
// third (32 rows, bf16: 207 -> 177 us for 1 GB of cache; 64 rows: 403 -> 326); one
// tile would lose its ring (165 -> 192), and from 128 dims on the registers are
// the second CTA's.
constexpr int ctas_per_sm(int dim, int mt)
{
    return dim <= 64 && mt > 1 ? 3 : 2;
}

// M tiles (of 16 query rows) of a worker; three make four.
constexpr int tiles_of_rows(int rows)
{
    return rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
}

// Value scales of up to 2^90 units, times weights below 2^15 and elements below 2^9, leave
// outputs room in fp32.
constexpr float kFarBelow = 0x1p-90f;

constexpr int kStateBytes = 136;                // WarpState

// FULL: a piece fills a stage (pages of at least a stage's tokens, in whole
// stages), so the offsets in a stage are constants: up to 16 % of the time for 32
// requests of 16K tokens (most with 32 and 64 query rows), 1 to 12 % for 60 of up to
// 500, at 64, 192 and 256 dims.  ALONE: each CTA has one unit, its workers a share of
// the unit's tiles each.
template <int KIND, int D, int MT, bool FULL, int ALONE = kOnLine, int WALKED = kTokens>
struct Shape {
    static constexpr int kWalked = WALKED;
    static constexpr bool kFull = FULL, kAlone = ALONE != kOnLine, kRegions = WALKED != kTokens, kScaled = KIND >= kScaledE4m3;
    static constexpr bool FP8 = KIND != kBf16;
    static constexpr int kUnitCost = unit_cost(kScaled);
    static constexpr int kElt = FP8 ? 1 : 2;
    static constexpr int kRowBytes = 2 * D * kElt;
    static constexpr int kBands = kRowBytes / 128;
    static constexpr int kSlots = stage_slots(kRowBytes, MT, kAlone);
    static constexpr int kStageBytes = kSlots * kRowBytes;
    static constexpr int kSteps = D / 16;                       // QK k-steps
    // Log2 units that the running maximum may lag behind the true one, and that the
    // weights are lifted by.  bf16 weights have fp32's range.  E4M3 caches take fp16
    // weights: lifted by 13 and at most four times the running maximum's they reach
    // 2^15 (fp16 ends at 2^16) and keep 11 bits down to 2^-27 of the largest, beyond
    // that 2^-38 of it.  Without the lift tokens 10 nats below one that takes nearly
    // all of the weight lost bits, and those 17 below it were lost, however many.
    static constexpr float kRescaleSlack = FP8 ? 2.0f : 8.0f, kLift = FP8 ? 13.0f : 0.0f;
    static constexpr int kWorkers = kWarps / MT;                // of a CTA
    // Q fragments stay in registers, beside the output's D / 2, but for 256 dims:
    // there they take a third of the ring's place (each lane its own words).
    static constexpr bool kQShared = D > 192;
    static constexpr int kQBytes = kQShared ? kSteps * 32 * 16 : 0;     // of a warp
    static constexpr int kPerSm = ctas_per_sm(D, MT);
    static constexpr int kRingBytes = (kPerSm == 2 ? 96 : 64) * 1024;
    static constexpr int kRing = (kRingBytes - kWarps * kQBytes) / kStageBytes / kWorkers;  // stages of a worker
    static constexpr int kStages = kRing * kWorkers;
    static constexpr int kQOff = kStages * kStageBytes;
    static constexpr int kBarOff = kQOff + kWarps * kQBytes;
    static constexpr int kHdrOff = kBarOff + 16 * kStages;
    static constexpr int kIssuedOff = kHdrOff + 8 * kStages;
    static constexpr int kCtlOff = (kIssuedOff + 4 * kStages + 15) / 16 * 16;
    static constexpr int kStatsOff = kCtlOff + 16 + 8 * (kThreads + kWarps);    // of a merge: maximum and sum of each row
    static constexpr int kStateOff = kStatsOff + kWarps * 16 * 8;
    static constexpr int kScaleOff = kStateOff + kWarps * kStateBytes;      // of each stage's eight-token tiles; of a merge
    static constexpr int kStageScales = kScaled ? kSlots / 8 * 8 : 0;
    static constexpr int kUnitsOff = kScaleOff + kStages * kStageScales;    // what the workers' outputs are in units of
    static constexpr int kBytes = kUnitsOff + (kScaled ? 4 * kWarps : 0) + 1024;     // + the base's alignment
    static_assert(kPerSm * kWorkers <= 2 * kWarps, "join list");
    static_assert(kStageBytes % 1024 == 0 && kRing >= 2 && kBytes <= 232448 / kPerSm - 1024, "ring");
};

// A worker's part of the line, unit by unit.
struct Segment {
    int request, group, first, last, tiles, len;   // tiles [first, last) of the unit's `tiles`
};

template <int WALKED, int COST>
struct Walk {
    long long left;                             // line from the unit's start to the part's end
    int request, group, tile;                   // (whole_units: units still to take)

    // Tokens of a unit; of an active row those of its list, up to the last region that it
    // sees or (without extents) all that there is room for.  0: a row of zeros, < 0: left
    // as it was.
    static __device__ __forceinline__ int length(const Params &p, int q)
    {
        if constexpr (WALKED == kExtents)
            return p.extents[q];
        else if constexpr (WALKED == kRegions)
            return p.active[q * p.act_s] ? p.cap : p.clear_inactive ? 0 : -1;
        else
            return min(p.seq_lens[q * p.len_s], p.cap);
    }

    static __device__ __forceinline__ int tiles_of(const Params &p, int len)
    {
        return len > 0 ? static_cast<int>(quotient(len - 1, p.tile_inv)) + 1 : 0;
    }

    __device__ __forceinline__ bool next(const Params &p, Segment &s)
    {
        while (left > 0 && request < p.requests) {
            const int len = length(p, request), tiles = tiles_of(p, len);
            s.request = request;
            s.group = group;
            s.first = tile;
            s.tiles = tiles;
            s.len = len;
            // a unit's cost comes before its tiles
            s.last = p.whole_units ? tiles
                                   : static_cast<int>(max(min(left - COST, static_cast<long long>(tiles)),
                                                          static_cast<long long>(tile)));
            const bool some = s.last > s.first;
            if (s.last == tiles) {
                left -= p.whole_units ? 1 : tiles > 0 ? tiles + COST : 0;
                tile = 0;
                if (++group == p.groups || (tiles == 0 && !p.whole_units)) {
                    group = 0;
                    ++request;
                }
            } else {
                left = 0;
            }
            if (some)
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

// A load that stays where it is written, long before its use.
__device__ __forceinline__ float load_now(const float *at)
{
    float v;
    asm volatile("ld.global.nc.f32 %0, [%1];" : "=f"(v) : "l"(at));
    return v;
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

__device__ __forceinline__ void mma1688(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t b)
{
    asm("mma.sync.aligned.m16n8k8.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5}, {%6}, {%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(b));
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t sel)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, 0, %2;" : "=r"(r) : "r"(a), "r"(sel));
    return r;
}

// Two fp32 values to packed fp16 (round to nearest even), `lo` in the low half.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// Two weights, >= 0, as the sum of two bf16 values each: the largest bf16 below the
// weight, and the rest, rounded (16 bits in all).  Both are above 0 unless the
// weight is 0, so that an infinite V keeps its sign in both products (a rest of 0 or
// of the other sign would make it NaN).
__device__ __forceinline__ void split_bf16(float lo, float hi, uint32_t &most, uint32_t &rest)
{
    const uint32_t a = max(__float_as_uint(lo), 1u) - 1u, b = max(__float_as_uint(hi), 1u) - 1u;
    asm("prmt.b32 %0, %1, %2, 0x7632;" : "=r"(most) : "r"(a), "r"(b));
    rest = pack_bf16(lo - __uint_as_float(a & 0xFFFF0000u), hi - __uint_as_float(b & 0xFFFF0000u));
}

// Keys of integers go into the products as fp16 numbers below the normal ones: the byte
// of x + 128 by itself stands for (x + 128) 2^-24, exactly.  Scores begin at -128 times
// the row's sum of q instead of 0, so that they round by the size of 255 |q|, not of
// |q k|: far below half a step of k.  (To take the 128 off each element takes two more
// instructions a word: 16 documents of 64K to 128K tokens 444 us, so 414.  Values have
// it taken off: where a token of nearly all weight is 0, outputs are as small as the
// rest of them, and would be off by the bias's rounding.)
constexpr float kKeyUnit = 0x1p-24f, kKeyBias = 128.0f;

// The four elements of a word of keys: two pairs of fp16 values, in order.
template <int KIND>
__device__ __forceinline__ uint2 key_pairs(uint32_t w)
{
    if constexpr (KIND == kScaledInt8) {
        const uint32_t x = w ^ 0x80808080u;
        return make_uint2(bytes_of<0x4140u>(x, 0u), bytes_of<0x4342u>(x, 0u));
    } else {
        return make_uint2(e4m3x2_to_f16x2(w), e4m3x2_to_f16x2(w >> 16));
    }
}

// The four elements of a word as fp32 values.
template <int KIND>
__device__ __forceinline__ float4 word_values(uint32_t w)
{
    uint32_t a, b;
    if constexpr (KIND == kScaledInt8) {
        const uint32_t x = w ^ 0x80808080u;
        a = int8x2_to_f16x2<0, 1>(x);
        b = int8x2_to_f16x2<2, 3>(x);
    } else {
        a = e4m3x2_to_f16x2(w);
        b = e4m3x2_to_f16x2(w >> 16);
    }
    const float2 u = __half22float2(*reinterpret_cast<const __half2 *>(&a));
    const float2 v = __half22float2(*reinterpret_cast<const __half2 *>(&b));
    return make_float4(u.x, u.y, v.x, v.y);
}

// A word of two tokens' values (two dims of one, two of the other): the pairs of the
// first dim and of the second.
template <int KIND>
__device__ __forceinline__ uint2 value_pairs(uint32_t w)
{
    if constexpr (KIND == kScaledInt8) {
        const uint32_t x = w ^ 0x80808080u;
        return make_uint2(int8x2_to_f16x2<0, 2>(x), int8x2_to_f16x2<1, 3>(x));
    } else {
        const uint32_t x = prmt(w, 0x3120u);
        return make_uint2(e4m3x2_to_f16x2(x), e4m3x2_to_f16x2(x >> 16));
    }
}

__device__ __forceinline__ float2 lds64(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr));
    return v;
}

// Eight bytes from global to shared memory, not waited for.
__device__ __forceinline__ void copy8(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(src) : "memory");
}

// The barrier's phase is not over before this thread's copies have landed.
__device__ __forceinline__ void copies_arrive(uint32_t bar)
{
    asm volatile("cp.async.mbarrier.arrive.shared::cta.b64 [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ float fast_exp2(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// 2^-k of 2^k, -126 <= k <= 126.
__device__ __forceinline__ float reciprocal_of_power(float x)
{
    return __uint_as_float((254u << 23) - __float_as_uint(x));
}

// The least power of two from x on, at most 2^126 (x > 0).
__device__ __forceinline__ float power_from(float x)
{
    return __uint_as_float(min((__float_as_uint(x) + 0x7FFFFFu) & 0x7F800000u, 253u << 23));
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
// `vsw` its swizzle phase.  bf16: P comes in two parts (split_bf16), so that its
// products carry 16 bits of it.  MASKED zeroes V of slots out of the
// mask (vm0: k-slots 2t, 2t + 1; vm1: 8 + 2t, 9 + 2t), whatever they hold.
template <int KIND, int D, bool MASKED>
__device__ __forceinline__ void pv_accumulate(float (&o)[D / 8][4], const uint32_t (&pa)[4],
                                              const uint32_t (&pb)[4], uint32_t vrow, uint32_t bstride, int mi,
                                              int vsw, uint32_t vm0, uint32_t vm1)
{
    constexpr bool FP8 = KIND != kBf16;
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
                const uint2 x0 = value_pairs<KIND>(r[2 * h]), x1 = value_pairs<KIND>(r[2 * h + 1]);
                mma16816<true>(o[4 * c2 + 2 * h], pa, x0.x, x1.x);
                mma16816<true>(o[4 * c2 + 2 * h + 1], pa, x0.y, x1.y);
            }
        } else {
            mma16816<false>(o[2 * c2], pa, r[0], r[1]);
            mma16816<false>(o[2 * c2 + 1], pa, r[2], r[3]);
            mma16816<false>(o[2 * c2], pb, r[0], r[1]);
            mma16816<false>(o[2 * c2 + 1], pb, r[2], r[3]);
        }
    }
}

// The same over eight slots of bf16, two chunk pairs at a time: O += P[16 x 8] V[8 x D].
template <int D, bool MASKED>
__device__ __forceinline__ void pv_accumulate8(float (&o)[D / 8][4], const uint32_t (&pa)[2], const uint32_t (&pb)[2],
                                               uint32_t vrow, uint32_t bstride, int mi, int vsw, uint32_t vm)
{
    constexpr int kFirst = D / 8;
#pragma unroll
    for (int c4 = 0; c4 < kFirst / 4; ++c4) {
        const int idx = kFirst + 4 * c4;
        uint32_t r[4];
        ldsm_x4_trans(vrow + (idx >> 3) * bstride + ((((idx & 7) + mi) ^ vsw) << 4), r);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if constexpr (MASKED)
                r[i] &= vm;
            mma1688(o[4 * c4 + i], pa[0], pa[1], r[i]);
            mma1688(o[4 * c4 + i], pb[0], pb[1], r[i]);
        }
    }
}

// ---------------------------------------------------------------------------
// Split kernel
// ---------------------------------------------------------------------------

// Where a worker's part begins, and how long it is.
struct Part {
    long long left, start;                      // as Walk::left; the unit's place on the line
    int request, group, tile;
};

// floor(total * i / workers) by the workers' inverse, which may fall one short.
__device__ __forceinline__ long long boundary(const Params &p, long long total, int i)
{
    const unsigned long long n = static_cast<unsigned long long>(total) * i;
    unsigned long long k = p.workers > 1 ? __umul64hi(n, p.workers_inv - 1) : n;
    k += n - k * p.workers >= static_cast<unsigned>(p.workers);
    return static_cast<long long>(k);
}

// The part of worker w of this CTA, the line's length, the workers that get a
// part of it (`used`) and the number v of the worker among them.  Where all
// workers get one, a CTA's are neighbours, so that their pieces of a long unit
// can be merged here; where there are fewer tiles, worker w of the CTA is number
// w * CTAs + CTA, which spreads them over the SMs.  Every thread of the block
// calls it; a worker's warps look for its part together.
// `sums`: kThreads + kWarps values of shared memory.
template <int WORKERS, class Line, int COST>
__device__ __forceinline__ Part find_part(const Params &p, long long *sums, int w, long long &total, int &used, int &v)
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int spread = w * static_cast<int>(gridDim.x) + static_cast<int>(blockIdx.x);
    if (p.whole_units) {
        total = static_cast<long long>(p.requests) * p.groups;
        used = p.workers;
        v = spread;
        const long long u0 = boundary(p, total, v);
        const unsigned q = static_cast<unsigned>(u0) / static_cast<unsigned>(p.groups);
        return {boundary(p, total, v + 1) - u0, 0, static_cast<int>(q), static_cast<int>(u0 - q * p.groups), 0};
    }
    // Spans of the requests on the line, of one group each; a thread sums a run of
    // them, or a lane has one where a warp has them all and needs no other.
    const bool few = p.requests <= 32;
    const int per = (p.requests + kThreads - 1) / kThreads;
    const int q0 = min(p.requests, static_cast<int>(threadIdx.x) * per), q1 = min(p.requests, q0 + per);
    auto span = [&](int q) -> long long {
        const int tiles = Line::tiles_of(p, Line::length(p, q));
        return tiles > 0 ? tiles + COST : 0;
    };
    auto scan = [&](long long x) {              // inclusive, over the warp
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(~0u, x, o);
            x += lane >= o ? y : 0;
        }
        return x;
    };
    long long mine = 0, inc, warp_sum[kWarps] = {}, all = 0;
    if (few) {
        mine = lane < p.requests ? span(lane) : 0;
        inc = scan(mine);
        all = __shfl_sync(~0u, inc, 31);
    } else {
        for (int q = q0; q < q1; ++q)
            mine += span(q);
        inc = scan(mine);
        sums[threadIdx.x] = inc - mine;         // before the thread's run, in its warp
        if (lane == 31)
            sums[kThreads + warp] = inc;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            warp_sum[k] = all;
            all += sums[kThreads + k];
        }
    }
    total = all * p.groups;
    constexpr int least = kMinTiles + COST;
    used = total >= static_cast<long long>(p.workers) * least ? p.workers
                                                               : (static_cast<int>(total) + least - 1) / least;
    v = used == p.workers ? static_cast<int>(blockIdx.x) * WORKERS + w : spread;
    if (v >= used)
        return {0, 0, 0, 0, 0};
    const unsigned shorter = static_cast<unsigned>(total);              // of a line with fewer workers
    const long long x = used == p.workers ? boundary(p, total, v) : shorter * static_cast<unsigned>(v) / used;
    const long long x1 = used == p.workers ? boundary(p, total, v + 1) : shorter * static_cast<unsigned>(v + 1) / used;

    int q = 0;
    long long at = 0, len = 0;
    if (few) {
        const int l = __ffs(__ballot_sync(~0u, inc * p.groups > x)) - 1;        // x is on the line
        len = __shfl_sync(~0u, mine, l);
        at = __shfl_sync(~0u, (inc - mine) * p.groups, l);
        q = l;
    } else {
        // The run that x lies in: the last that begins at or before it.
        int run = -1;
#pragma unroll
        for (int k = 0; k < kWarps; ++k)
            run += __popc(__ballot_sync(~0u, (warp_sum[k] + sums[32 * k + lane]) * p.groups <= x));
        // The request in the run, 32 at a time; requests without tokens span nothing.
        at = warp_sum[0];
#pragma unroll
        for (int k = 1; k < kWarps; ++k)
            at = run >= 32 * k ? warp_sum[k] : at;
        at = (at + sums[run]) * p.groups;
        q = run * per;
        for (;; q += 32) {
            const long long s = q + lane < p.requests ? span(q + lane) : 0;
            const long long to = scan(s) * p.groups;                        // past each request
            const unsigned past = __ballot_sync(~0u, at + to > x);
            if (past) {
                const int l = __ffs(past) - 1;
                len = __shfl_sync(~0u, s, l);
                at += __shfl_sync(~0u, to, l) - len * p.groups;
                q += l;
                break;
            }
            if (q + 32 >= p.requests)                                       // not reached: x is on the line
                return {0, 0, 0, 0, 0};
            at += __shfl_sync(~0u, to, 31);
        }
    }
    const unsigned long long in = x - at;
    const int g = static_cast<int>(in >> 32 || len >> 32 ? in / len : static_cast<unsigned>(in) / static_cast<unsigned>(len));
    const long long u0 = at + g * len;
    return {x1 - u0, u0, q, g, static_cast<int>(max(x - u0 - COST, 0ll))};
}

// Where a warp is on the line.  It lies in shared memory (all lanes write the
// same): between units it is not needed, and registers are short.
template <class Line>
struct Place {
    Line walk;
    Segment seg;
    long long unit;                             // where the segment's unit begins on the line

    // The next segment into seg; a copy of it in `s`.
    __device__ __forceinline__ bool next(const Params &p, long long part_end, Segment &s)
    {
        Line w = walk;
        __syncwarp();                           // every lane has read it
        unit = part_end - w.left;
        const bool some = w.next(p, s);
        walk = w;
        seg = s;
        __syncwarp();
        return some;
    }
};

template <class Line>
struct WarpState {
    Place<Line> here, ahead;                          // of the warp's products and of its feed
    long long part_end, total;                  // on the line; the line's length
    int used, number;                           // workers with a part; this one's number
};

static_assert(sizeof(WarpState<Walk<kTokens, 0>>) == kStateBytes, "shared memory of a warp");

// A worker's ring of stages: their places, barriers, headers (the slots that
// hold tokens) and how often each was issued.
struct Ring {
    uint32_t stages, full, scales;
    uint64_t *hdr;
    int *issued;
};

// A worker's stream: its stages in order, a batch of their pieces looked up a
// lane a piece, and the next batch's table entries on their way.  A batch lies
// in one segment.
template <class S>
struct Feed {
    Place<Walk<S::kWalked, S::kUnitCost>> *at_line;                // of the next segment to look up
    bool more;
    int tile;                                   // of the segment, the next to look up
    int per_stage, batch, lane_stage, lane_piece;   // pieces of a stage, stages of a batch; the lane's place in one
    int at, n, group, page, off, left;          // the batch: next stage to issue, stages, ...
    int n2, group2, page2, off2, left2;         // the one after
    // Quantised caches: the scales of the lane's piece of the batch and, of the stage that
    // begins at the lane, the slots that will hold tokens and the bytes to come.
    const float *scales;
    uint64_t bits;
    uint32_t bytes;
    int id3, pos3;                              // regions: of the batch after that, id and position, on their way

    __device__ __forceinline__ void look_up(const Params &p)
    {
        n = n2;
        group = group2;
        page = page2;
        off = off2;
        left = left2;
        at = 0;
        n2 = 0;
        // here, once for a batch, and not at each stage, where the products wait for it
        // (16 documents of 64K to 128K tokens, E4M3, 192 dims: 450 us there, 402 here)
        if constexpr (S::kScaled)
            prepare(p);
        if (!more)
            return;
        const int P = p.piece;
        Segment seg = at_line->seg;
        n2 = min(batch, seg.last - tile);
        group2 = seg.group;
        const int f = (tile + lane_stage) * per_stage + lane_piece;
        if constexpr (S::kRegions) {
            region_piece(p, seg.request, f);
        } else {
            const int col = static_cast<int>(quotient(f, p.per_block_inv));
            off2 = f * P - col * p.block;
            left2 = lane_stage < n2 ? seg.len - f * P : 0;          // tokens from the piece's first on
            page2 = left2 > 0 && col < p.table_cols ? p.block_table[seg.request * p.bt_s0 + col] : -1;
        }
        tile += n2;
        if (tile >= seg.last) {
            if constexpr (S::kAlone)
                more = false;
            else
                more = at_line->next(p, 0, seg);
            tile = seg.first;
        }
        if constexpr (S::kRegions)
            region_ids(p, seg);
    }

    // The feed's place is where the worker's part begins.
    __device__ __forceinline__ void start(const Params &p, Place<Walk<S::kWalked, S::kUnitCost>> *place, int lane)
    {
        at_line = place;
        per_stage = S::kFull ? 1 : p.tile / p.piece;
        batch = 32 / per_stage;
        lane_stage = lane / per_stage;
        lane_piece = lane - lane_stage * per_stage;
        Segment seg;
        if constexpr (S::kAlone) {              // the one that is there; it may be empty
            seg = at_line->seg;
            more = seg.last > seg.first;
        } else {
            more = at_line->next(p, 0, seg);
        }
        tile = seg.first;
        n2 = group2 = off2 = left2 = 0;         // no batch yet
        page2 = -1;
        if constexpr (S::kRegions)
            region_ids(p, seg);
        look_up(p);                             // the first batch's table entries are on their way
    }

    // Issues the batch's next stage, if there is one, into place `slot` of the
    // worker's ring.
    __device__ __forceinline__ void issue(const Params &p, const CUtensorMap *tmap, const Ring &r, int slot, int lane)
    {
        if (n > 0) {
            send(p, tmap, r, slot, 1, lane);
            if (at == n)
                look_up(p);
        }
    }

    // Fills the ring at the start: what the batch has at once, the rest one by one.
    __device__ __forceinline__ void fill(const Params &p, const CUtensorMap *tmap, const Ring &r, int lane)
    {
        look_up(p);
        int slot = 0;
        if (n > 0) {
            slot = min(n, S::kRing);
            send(p, tmap, r, 0, slot, lane);
            if (at == n)
                look_up(p);
        }
#pragma unroll 1
        for (; slot < S::kRing && n > 0; ++slot)
            issue(p, tmap, r, slot, lane);
    }

private:
    // The next batch's region ids, and its row's position, a batch before they are
    // needed: the table entries are looked up by them.
    __device__ __forceinline__ void region_ids(const Params &p, const Segment &seg)
    {
        const int f = (tile + lane_stage) * per_stage + lane_piece;
        const bool some = more && tile + lane_stage < seg.last && lane_stage < batch && f * p.piece < seg.len;
        const int64_t row = seg.request;
        id3 = some ? p.regions[row * p.reg_s0 + quotient(f, p.per_region_inv)] : -1;
        pos3 = some ? p.positions[row * p.pos_s] : -1;
    }

    // Piece f of a row's regions, of region id3: its request's table line, the row's group,
    // and how many of its tokens the row sees.
    __device__ __forceinline__ void region_piece(const Params &p, int request, int f)
    {
        const unsigned row = static_cast<unsigned>(request);
        const int in_region = f - static_cast<int>(quotient(f, p.per_region_inv)) * p.per_region;
        group2 = static_cast<int>(row - quotient(row, p.region_groups_inv) * p.region_groups);
        const int64_t token = static_cast<int64_t>(id3) * p.region_tokens + in_region * p.piece;
        const int64_t seen = id3 >= 0 ? static_cast<int64_t>(pos3) + 1 - token : 0;
        left2 = static_cast<int>(max(min(seen, static_cast<int64_t>(p.piece)), static_cast<int64_t>(0)));
        page2 = -1;
        if (id3 < -1)
            atomicOr(p.flags, SDA_FLAG_BOUNDS);
        if (left2 > 0) {                        // token <= position: 31 bits
            const int col = static_cast<int>(quotient(static_cast<uint32_t>(token), p.block_inv));
            off2 = static_cast<int>(token) - col * p.block;
            if (col < p.table_cols)
                page2 = p.block_table[static_cast<int64_t>(quotient(row, p.request_rows_inv)) * p.bt_s0 + col];
        }
    }

    __device__ __forceinline__ void prepare(const Params &p)
    {
        const bool some = lane_stage < n && left > 0;
        const bool copy = some && page >= 0 && page < p.pages;
        if (some && !copy)
            atomicOr(p.flags, SDA_FLAG_BOUNDS);
        page = copy ? page : -1;
        scales = p.scales + page * p.s_s0 + group * p.s_s1 + quotient(off, p.span_inv) * p.s_s2;
        const uint64_t own = copy ? low_bits(min(p.piece, left)) << (lane_piece * p.piece) : 0;
        bits = own;
        int pieces = copy;
        for (int k = 1; k < per_stage; ++k) {                   // of use to a stage's first lane
            bits |= __shfl_down_sync(~0u, own, k);
            pieces += __shfl_down_sync(~0u, static_cast<int>(copy), k);
        }
        bytes = static_cast<uint32_t>(pieces * p.piece) * S::kRowBytes;
    }

    // Stages at .. at + count - 1 of the batch into places slot, slot + 1, ...:
    // a stage's first lane announces its bytes and the tokens that it will hold.
    __device__ __forceinline__ void send(const Params &p, const CUtensorMap *tmap, const Ring &r, int slot, int count,
                                         int lane)
    {
        const uint32_t piece_bytes = static_cast<uint32_t>(p.piece) * S::kRowBytes;
        const int mine = lane_stage - at;
        const int place = slot + mine;
        const uint32_t full = r.full + 8 * place;
        const bool leads = mine >= 0 && mine < count && lane_piece == 0;
        bool copy;
        if constexpr (S::kScaled) {
            copy = mine >= 0 && mine < count && page >= 0;
            if (leads) {
                r.hdr[place] = bits;
                r.issued[place] += 1;
                if (bytes > 0)
                    mbar_expect_tx(full, bytes);
            }
        } else {
            const bool wanted = mine >= 0 && mine < count && left > 0;
            copy = wanted && page >= 0 && page < p.pages;
            if (wanted && !copy)
                atomicOr(p.flags, SDA_FLAG_BOUNDS);
            const unsigned copies = __ballot_sync(~0u, copy);
            if (leads) {
                uint64_t bits = 0;
                const unsigned of_stage = copies >> lane;       // this lane is the stage's first
                int pieces = 0;
                for (int k = 0; k < per_stage; ++k)
                    if ((of_stage >> k) & 1u) {
                        ++pieces;
                        bits |= low_bits(min(p.piece, left - k * p.piece)) << (k * p.piece);
                    }
                r.hdr[place] = bits;
                r.issued[place] += 1;
                if (pieces > 0)
                    mbar_expect_tx(full, pieces * piece_bytes);
            }
        }
        __syncwarp();
        if (copy)
            tma_load_5d(r.stages + place * S::kStageBytes + lane_piece * piece_bytes, tmap, 0, off, 0, group, page, full);
        if constexpr (S::kScaled) {             // the scales of the piece's eight-token tiles
            if (copy) {
                const uint32_t dst = r.scales + place * S::kStageScales + lane_piece * p.piece;
                copy8(dst, scales);
                if (!S::kFull || !p.one_scale) {
                    const int first = static_cast<int>(quotient(off, p.span_inv));
                    for (int k = 8; k < p.piece; k += 8)
                        copy8(dst + k, scales + (p.one_scale ? 0 : (static_cast<int>(quotient(off + k, p.span_inv)) - first) * p.s_s2));
                }
                copies_arrive(full);
            }
            __syncwarp();                       // before the stage's own arrival
        }
        if (leads)
            mbar_arrive(full);
        at += count;
    }
};

// All threads of the cluster's CTAs: what they wrote before is seen by all after.
__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return static_cast<int>(r);
}

// The address of `addr` of this CTA's shared memory in that of CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer(uint32_t addr, int rank)
{
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
    return a;
}

__device__ __forceinline__ float peer_f32(uint32_t at)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float4 peer_f32x4(uint32_t at)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

template <int KIND, int D, int MT, bool FULL, int TAKERS, int WALKED>
__global__ void __launch_bounds__(kThreads, Shape<KIND, D, MT, FULL, TAKERS, WALKED>::kPerSm)
    sda_paged_kernel(const __grid_constant__ CUtensorMap tmap, const __grid_constant__ Params p)
{
    using S = Shape<KIND, D, MT, FULL, TAKERS, WALKED>;
    constexpr bool ALONE = S::kAlone, CLUSTER = TAKERS == kCluster;     // CLUSTER: together with others
    constexpr int kUnitCost = S::kUnitCost;
    constexpr bool REGIONS = S::kRegions;
    using Line = Walk<WALKED, kUnitCost>;
    constexpr bool FP8 = S::FP8, SCALED = S::kScaled, INT8 = KIND == kScaledInt8;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int worker = warp / MT, mt = warp % MT;               // of the CTA; the warp's tile of query rows
    const uint32_t sbase = smem_u32(smem) + worker * S::kRing * S::kStageBytes;
    const uint32_t bars = smem_u32(smem) + S::kBarOff;
    const uint32_t full_bar = bars + 8 * worker * S::kRing, empty_bar = full_bar + 8 * S::kStages;
    uint64_t *hdr = reinterpret_cast<uint64_t *>(smem + S::kHdrOff) + worker * S::kRing;
    int *issued = reinterpret_cast<int *>(smem + S::kIssuedOff) + worker * S::kRing;
    int *timed_out = reinterpret_cast<int *>(smem + S::kCtlOff);
    long long *sums = reinterpret_cast<long long *>(smem + S::kCtlOff + 16);

    if (threadIdx.x < S::kStages) {
        mbar_init(bars + 8 * threadIdx.x, 1);
        mbar_init(bars + 8 * (S::kStages + threadIdx.x), MT > 1 ? MT - 1 : 1);   // the worker's other warps
        (reinterpret_cast<int *>(smem + S::kIssuedOff))[threadIdx.x] = 0;
        mbar_init_fence();
    }
    if (threadIdx.x == 0) {
        *timed_out = 0;
        asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&tmap)) : "memory");
    }
    pdl_launch_dependents();
    __syncthreads();
    pdl_wait();

    // What is needed between units only: this warp's place, its feed's, the line.
    WarpState<Line> *state = reinterpret_cast<WarpState<Line> *>(smem + S::kStateOff) + warp;
    if constexpr (ALONE) {
        Segment &seg = state->here.seg;
        const unsigned of_cluster = CLUSTER ? p.cluster : 1;
        const unsigned unit = blockIdx.x / of_cluster;
        const int mine = static_cast<int>(blockIdx.x - unit * of_cluster) * S::kWorkers + worker;
        const int all = static_cast<int>(of_cluster) * S::kWorkers;
        seg.request = static_cast<int>(unit / static_cast<unsigned>(p.groups));
        seg.group = static_cast<int>(unit) - seg.request * p.groups;
        seg.len = Line::length(p, seg.request);
        seg.tiles = Line::tiles_of(p, seg.len);
        seg.first = seg.tiles * mine / all;
        seg.last = seg.tiles * (mine + 1) / all;
    } else {
        long long total;
        int used, v;
        const Part part = find_part<S::kWorkers, Line, kUnitCost>(p, sums, worker, total, used, v);
        state->here.walk = state->ahead.walk = {part.left, part.request, part.group, part.tile};
        state->part_end = part.start + part.left;
        state->total = total;
        state->used = used;
        state->number = v;
    }
    __syncwarp();
    Feed<S> feed;
    const uint32_t scale_base = smem_u32(smem) + S::kScaleOff + worker * S::kRing * S::kStageScales;
    const Ring place = {sbase, full_bar, scale_base, hdr, issued};
    if (mt == 0)
        feed.start(p, ALONE ? &state->here : &state->ahead, lane);

    const int g = lane >> 2, t = lane & 3;      // fragment row and column pair
    const int H = p.heads, R = p.rows;
    const float ks = KIND == kE4m3 ? load_now(p.k_scale) : 1.0f, vs = KIND == kE4m3 ? load_now(p.v_scale) : 1.0f;
    auto token_of = [&](int r) { return (r * p.head_inv) >> 16; };      // of a query row

    const int r0 = 16 * mt + g, r1 = r0 + 8;    // this thread's query rows
    // query token of each row; rows past R repeat the last token's limits
    const int j0 = min(token_of(r0), p.query_len - 1), j1 = min(token_of(r1), p.query_len - 1);

    // Shared-memory offsets of this lane's K rows and V rows in a stage.  A
    // stage holds its pieces one after another, each [band][token][128 bytes].
    const uint32_t bstride = static_cast<uint32_t>(FULL ? S::kSlots : p.piece) * 128u;
    const int mi = lane >> 3;
    const int ksw = slot_of(g), vsw = slot_of(lane & 7);
    constexpr int NT = S::kSlots / 8, KS = S::kSlots / 16, NC = D * S::kElt / 64;
    constexpr uint64_t kAll = S::kSlots >= 64 ? ~0ull : (1ull << S::kSlots) - 1ull;
    uint32_t tile_off[NT];                      // of the 8-slot tiles
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int k = 8 * i / p.piece;
        tile_off[i] = FULL             ? 1024u * i
                      : 8 * i < p.tile ? k * bstride * S::kBands + (8 * i - k * p.piece) * 128u : 0u;
    }

    const int tile_scale_step = FULL && p.one_scale ? 0 : 8;

    int ring = 0;                               // the worker's next stage: its place and parity
    uint32_t parity = 0;
    bool dead = false, started = false;

    for (bool more = true; more; more = !ALONE) {
        int common, left;                       // tokens that every row sees, from the segment's first on; its stages
        const uint16_t *q_rows;                 // the unit's first query row
        {
            Segment seg;
            if constexpr (ALONE) {
                seg = state->here.seg;
                // A cluster's CTAs all come to its barriers, whatever each has read (lengths that
                // change meanwhile must not leave some of them waiting).
                if (!CLUSTER && seg.tiles == 0)
                    break;
            } else {
                if (!state->here.next(p, state->part_end, seg))
                    break;
            }
            common = seg.len - p.query_len + 1 - seg.first * p.tile;
            left = seg.last - seg.first;
            q_rows = p.query + (static_cast<int64_t>(seg.request) * p.query_len * p.groups + seg.group) * p.q_s0;
        }

        // ---- Q fragments: thread t of k-step kk holds the four dims that its
        // K words hold.  FP8: the fp16 product takes q scaled by a power of two
        // that puts the row's largest |q| in [2^14, 2^15), undone in the logit
        // scale: any bf16 row is exact down to 2^-31 of its largest value.
        uint32_t qf[S::kSteps][4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = k ? r1 : r0, rq = r < R ? r : 0;      // rows past R read row 0: zeros in the end
            const int jq = token_of(rq);
            const uint16_t *q = q_rows + static_cast<int64_t>(jq) * p.groups * p.q_s0 + (rq - jq * H) * p.q_s1 +
                                (FP8 ? 16 : 8) * t;
            auto dim = [](int kk) { return FP8 ? 64 * (kk >> 2) + 4 * (kk & 3) : 32 * (kk >> 1) + 4 * (kk & 1); };
            if (p.q_vec) {
#pragma unroll
                for (int kk = 0; kk < S::kSteps; ++kk) {
                    const uint2 w = *reinterpret_cast<const uint2 *>(q + dim(kk));
                    qf[kk][k] = w.x;
                    qf[kk][2 + k] = w.y;
                }
            } else {
#pragma unroll
                for (int kk = 0; kk < S::kSteps; ++kk) {
                    const uint16_t *w = q + dim(kk);
                    qf[kk][k] = w[0] | (static_cast<uint32_t>(w[1]) << 16);
                    qf[kk][2 + k] = w[2] | (static_cast<uint32_t>(w[3]) << 16);
                }
            }
        }
        if (!started) {
            started = true;
            if (mt == 0)                        // behind the first Q, which would wait behind the stages
                feed.fill(p, &tmap, place, lane);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {           // not before the loads have had that time
            const uint32_t keep = (k ? r1 : r0) < R ? ~0u : 0u;
#pragma unroll
            for (int kk = 0; kk < S::kSteps; ++kk) {
                qf[kk][k] &= keep;
                qf[kk][2 + k] &= keep;
            }
        }
        float sl[2] = {p.scale * kLog2e * ks, p.scale * kLog2e * ks};   // logit scales in log2 units
        float from[2] = {0.0f, 0.0f};           // what the rows' scores begin at
        if constexpr (FP8) {
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t mx = 0;
#pragma unroll
                for (int kk = 0; kk < S::kSteps; ++kk)
                    mx = max(max(mx, max(qf[kk][k] & 0x7FFFu, (qf[kk][k] >> 16) & 0x7FFFu)),
                             max(qf[kk][2 + k] & 0x7FFFu, (qf[kk][2 + k] >> 16) & 0x7FFFu));
                mx = max(mx, __shfl_xor_sync(~0u, mx, 1));
                mx = max(mx, __shfl_xor_sync(~0u, mx, 2));
                const int e = mx ? min(126, max(-126, 141 - max(1, static_cast<int>(mx >> 7)))) : 0;
                const float up = __int_as_float((127 + e) << 23);
                sl[k] *= __int_as_float((127 - e) << 23);       // exact
#pragma unroll
                for (int kk = 0; kk < S::kSteps; ++kk)
#pragma unroll
                    for (int i = k; i < 4; i += 2) {
                        qf[kk][i] = pack_f16(__uint_as_float(qf[kk][i] << 16) * up,
                                             __uint_as_float(qf[kk][i] & 0xFFFF0000u) * up);
                        if constexpr (INT8) {   // as the products take it
                            const float2 x = __half22float2(*reinterpret_cast<const __half2 *>(&qf[kk][i]));
                            from[k] += x.x + x.y;
                        }
                    }
                if constexpr (INT8) {
                    from[k] += __shfl_xor_sync(~0u, from[k], 1);
                    from[k] += __shfl_xor_sync(~0u, from[k], 2);
                    from[k] *= -kKeyBias * kKeyUnit;
                }
            }
        }

        const uint32_t qshared = smem_u32(smem) + S::kQOff + warp * S::kQBytes + lane * 16;
        if constexpr (S::kQShared) {
#pragma unroll
            for (int kk = 0; kk < S::kSteps; ++kk)
                asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(qshared + kk * 512), "r"(qf[kk][0]),
                             "r"(qf[kk][1]), "r"(qf[kk][2]), "r"(qf[kk][3])
                             : "memory");
        }

        float o[D / 8][4];
#pragma unroll
        for (int n = 0; n < D / 8; ++n)
            o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.0f;
        float m_run[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.0f, 0.0f};
        // Outputs of a quantised cache are in units of a power of two that is at least the
        // largest value scale so far of tokens that all rows see, so that weights times
        // scales fit fp16.
        float unit = kSmallestScale;

        for (; left > 0; --left, common -= FULL ? S::kSlots : p.tile) {
            if (!dead) {
                const bool ok = mbar_wait(full_bar + 8 * ring, parity, p.wait_ns);
                if (!__all_sync(~0u, ok)) {
                    if (lane == 0) {
                        atomicOr(p.flags, SDA_FLAG_TIMEOUT);
                        *timed_out = 1;
                    }
                    dead = true;
                }
            }
            const uint64_t loaded = dead ? 0ull : hdr[ring];
            auto work = [&](auto plain) {
                constexpr bool kPlain = decltype(plain)::value;
                const uint32_t sb = sbase + ring * S::kStageBytes;

                // ---- S = Q K^T: tile i, column g is slot 8i + slot_of(g).
                float sc[NT][4];
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    sc[i][0] = sc[i][1] = INT8 ? from[0] : 0.0f;
                    sc[i][2] = sc[i][3] = INT8 ? from[1] : 0.0f;
                }
                const uint32_t krow = sb + ksw * 128u;
                constexpr int kGroup = NT < 4 ? NT : 4;         // tiles, independent chains, at a time
#pragma unroll
                for (int i0 = 0; i0 < NT; i0 += kGroup) {
#pragma unroll
                    for (int c = 0; c < NC; ++c) {
                        // a chunk of 16 bytes: four k-steps of E4M3 or two of bf16
                        const uint32_t off = (c >> 1) * bstride + ((((c & 1) * 4 + t) ^ ksw) << 4);
                        uint32_t w[kGroup][4];
#pragma unroll
                        for (int i = 0; i < kGroup; ++i) {
                            const uint4 x = lds128(krow + tile_off[i0 + i] + off);
                            w[i][0] = x.x;
                            w[i][1] = x.y;
                            w[i][2] = x.z;
                            w[i][3] = x.w;
                        }
                        constexpr int kChunkSteps = FP8 ? 4 : 2;
#pragma unroll
                        for (int k = 0; k < kChunkSteps; ++k) {
                            uint32_t q[4];
                            if constexpr (S::kQShared) {
                                const uint4 x = lds128(qshared + (kChunkSteps * c + k) * 512);
                                q[0] = x.x;
                                q[1] = x.y;
                                q[2] = x.z;
                                q[3] = x.w;
                            } else {
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    q[i] = qf[kChunkSteps * c + k][i];
                            }
#pragma unroll
                            for (int i = 0; i < kGroup; ++i) {
                                if constexpr (FP8) {
                                    const uint2 x = key_pairs<KIND>(w[i][k]);
                                    mma16816<true>(sc[i0 + i], q, x.x, x.y);
                                } else {
                                    mma16816<false>(sc[i0 + i], q, w[i][2 * k], w[i][2 * k + 1]);
                                }
                            }
                        }
                    }
                }

                // ---- Mask; c0/c2 of tile i are slot 8i + t, c1/c3 slot 8i + t + 4.
                float mx0 = -INFINITY, mx1 = -INFINITY;
                const uint64_t s0 = kPlain ? kAll : loaded & low_bits(common + j0);
                const uint64_t s1 = kPlain ? kAll : loaded & low_bits(common + j1);
                const uint64_t seen = kPlain ? kAll : loaded & low_bits(common);       // by all rows
                // The value scales of the tiles that all rows see, then what their weights are
                // multiplied by.
                float of_value[SCALED ? NT : 1], top_scale = 0.0f;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    float sl0 = sl[0], sl1 = sl[1];
                    if constexpr (SCALED) {
                        const float2 tile_scales = lds64(scale_base + ring * S::kStageScales + i * tile_scale_step);
                        sl0 *= tile_scales.x;
                        sl1 *= tile_scales.x;
                        if constexpr (INT8) {   // not before the key scale: next to a large query it would overflow
                            sl0 *= 1.0f / kKeyUnit;
                            sl1 *= 1.0f / kKeyUnit;
                        }
                        // where nothing was loaded it may be anything
                        of_value[i] = kPlain || ((seen >> (8 * i)) & 0xFFull) ? tile_scales.y : 0.0f;
                        top_scale = fmaxf(top_scale, of_value[i]);
                    }
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        const int slot = 8 * i + t + 4 * h;
                        sc[i][h] = kPlain || ((s0 >> slot) & 1ull) ? sc[i][h] * sl0 : -INFINITY;
                        sc[i][2 + h] = kPlain || ((s1 >> slot) & 1ull) ? sc[i][2 + h] * sl1 : -INFINITY;
                    }
                    mx0 = fmaxf(mx0, fmaxf(sc[i][0], sc[i][1]));
                    mx1 = fmaxf(mx1, fmaxf(sc[i][2], sc[i][3]));
                }

                // ---- Running maximum and sum.  The maximum may lag by
                // kRescaleSlack, so that outputs are seldom rescaled.
                mx0 = fmaxf(mx0, __shfl_xor_sync(~0u, mx0, 1));
                mx0 = fmaxf(mx0, __shfl_xor_sync(~0u, mx0, 2));
                mx1 = fmaxf(mx1, __shfl_xor_sync(~0u, mx1, 1));
                mx1 = fmaxf(mx1, __shfl_xor_sync(~0u, mx1, 2));
                if (__any_sync(~0u, mx0 > m_run[0] + S::kRescaleSlack || mx1 > m_run[1] + S::kRescaleSlack) ||
                    (SCALED && top_scale > unit)) {
                    const float n0 = fmaxf(m_run[0], mx0), n1 = fmaxf(m_run[1], mx1);
                    float a0 = n0 == -INFINITY ? 1.0f : fast_exp2(m_run[0] - n0);
                    float a1 = n1 == -INFINITY ? 1.0f : fast_exp2(m_run[1] - n1);
                    m_run[0] = n0;
                    m_run[1] = n1;
                    l_run[0] *= a0;
                    l_run[1] *= a1;
                    if (SCALED && top_scale > unit) {
                        const float more = power_from(top_scale);
                        const float less = unit * reciprocal_of_power(more);
                        unit = more;
                        a0 *= less;
                        a1 *= less;
                    }
#pragma unroll
                    for (int n = 0; n < D / 8; ++n) {
                        o[n][0] *= a0;
                        o[n][1] *= a0;
                        o[n][2] *= a1;
                        o[n][3] *= a1;
                    }
                }
                if constexpr (SCALED) {
                    const float per_unit = reciprocal_of_power(unit);
#pragma unroll
                    for (int i = 0; i < NT; ++i)
                        of_value[i] *= per_unit;
                }
                const float ref0 = m_run[0] == -INFINITY ? 0.0f : m_run[0] - S::kLift;
                const float ref1 = m_run[1] == -INFINITY ? 0.0f : m_run[1] - S::kLift;
#pragma unroll
                for (int i = 0; i < NT; ++i) {
                    sc[i][0] = fast_exp2(sc[i][0] - ref0);      // -inf gives 0
                    sc[i][1] = fast_exp2(sc[i][1] - ref0);
                    sc[i][2] = fast_exp2(sc[i][2] - ref1);
                    sc[i][3] = fast_exp2(sc[i][3] - ref1);
                    l_run[0] += sc[i][0] + sc[i][1];
                    l_run[1] += sc[i][2] + sc[i][3];
                }

                // ---- O += P V.  P in 11 bits (fp16, next to E4M3 values' 4), or in
                // two bf16 parts.  Tokens that only some rows see come below.
                auto both = [&](uint32_t km, int s) {           // V words of slots s, s + 4
                    return (((km >> s) & 1u) ? 0x0000FFFFu : 0u) | (((km >> (s + 4)) & 1u) ? 0xFFFF0000u : 0u);
                };
                auto weight = [&](int i, int k, uint32_t km, int s) {   // of slot s + t + 4 (k & 1) in mask km
                    return kPlain || ((km >> (s + t + 4 * (k & 1))) & 1u) ? sc[i][k] : 0.0f;
                };
                if constexpr (S::kSlots == 8) {
                    const uint32_t km = static_cast<uint32_t>(seen) & 0xFFu;
                    if (kPlain || km) {
                        uint32_t pa[2], pb[2];
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            const float lo = weight(0, 2 * k, km, 0), hi = weight(0, 2 * k + 1, km, 0);
                            split_bf16(lo, hi, pa[k], pb[k]);
                        }
                        pv_accumulate8<D, !kPlain>(o, pa, pb, sb + vsw * 128u, bstride, mi, vsw, both(km, t));
                    }
                }
#pragma unroll
                for (int k2 = 0; k2 < KS; ++k2) {
                    const uint32_t km = static_cast<uint32_t>(seen >> (16 * k2)) & 0xFFFFu;
                    if (!kPlain && km == 0)
                        continue;
                    uint32_t pa[4], pb[4] = {0, 0, 0, 0};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int i = 2 * k2 + (k >> 1), c = 2 * (k & 1);
                        const float lo = weight(i, c, km, 8 * (k >> 1)), hi = weight(i, c + 1, km, 8 * (k >> 1));
                        if constexpr (SCALED)
                            pa[k] = pack_f16(lo * of_value[i], hi * of_value[i]);
                        else if constexpr (FP8)
                            pa[k] = pack_f16(lo, hi);
                        else
                            split_bf16(lo, hi, pa[k], pb[k]);
                    }
                    const uint32_t vrow = sb + ((mi & 1) ? tile_off[2 * k2 + 1] : tile_off[2 * k2]) + vsw * 128u;
                    pv_accumulate<KIND, D, !kPlain>(o, pa, pb, vrow, bstride, mi, vsw, both(km, t), both(km, t + 8));
                }
                // ---- The newest query_len - 1 tokens, which only some rows see:
                // one at a time in fp32, so that a value that is not a number
                // reaches the rows that see it alone, and a larger value scale
                // costs no row that does not see it bits of its weights.
                if constexpr (!kPlain && !REGIONS) {
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
                        if constexpr (SCALED) {
                            const float of = lds64(scale_base + ring * S::kStageScales + (s >> 3) * tile_scale_step).y;
                            if (of * kFarBelow > unit) {        // the outputs so far keep their bits, down to fp32's least
                                const float more = power_from(of), less = unit * reciprocal_of_power(more);
                                unit = more;
#pragma unroll
                                for (int n = 0; n < D / 8; ++n) {
                                    o[n][0] *= less;
                                    o[n][1] *= less;
                                    o[n][2] *= less;
                                    o[n][3] *= less;
                                }
                            }
                            p0 *= of * reciprocal_of_power(unit);
                            p1 *= of * reciprocal_of_power(unit);
                        }
                        const bool see0 = s < common + j0, see1 = s < common + j1;
                        const uint32_t vrow = sb + off + (s & 7) * 128u + 4 * t;
                        constexpr int kFirst = D * S::kElt / 16;
#pragma unroll
                        for (int c = 0; c < kFirst; ++c) {
                            const int idx = kFirst + c;
                            const uint32_t w = lds32(vrow + (idx >> 3) * bstride + (((idx & 7) ^ (s & 7)) << 4));
                            if constexpr (FP8) {
                                const float4 x = word_values<KIND>(w);
                                if (see0) {
                                    o[2 * c][0] += p0 * x.x;
                                    o[2 * c + 1][0] += p0 * x.y;
                                    o[2 * c][1] += p0 * x.z;
                                    o[2 * c + 1][1] += p0 * x.w;
                                }
                                if (see1) {
                                    o[2 * c][2] += p1 * x.x;
                                    o[2 * c + 1][2] += p1 * x.y;
                                    o[2 * c][3] += p1 * x.z;
                                    o[2 * c + 1][3] += p1 * x.w;
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
            if (mt > 0) {
                if (lane == 0)
                    mbar_arrive(empty_bar + 8 * ring);
            } else if (!dead) {
                if (MT > 1 && !__all_sync(~0u, mbar_wait(empty_bar + 8 * ring, parity, p.wait_ns))) {
                    if (lane == 0) {
                        atomicOr(p.flags, SDA_FLAG_TIMEOUT);
                        *timed_out = 1;
                    }
                    dead = true;
                } else {
                    feed.issue(p, &tmap, place, ring, lane);
                }
            }
            if (++ring == S::kRing) {
                ring = 0;
                parity ^= 1u;
            }
        }

        // ---- The unit's result, or its piece's.
        const volatile Segment &at = state->here.seg;
        const Segment seg = {at.request, at.group, at.first, at.last, at.tiles, at.len};
        const int v = static_cast<const volatile WarpState<Line> *>(state)->number;
        const int64_t out_row0 = static_cast<int64_t>(seg.request) * p.query_len * p.groups + seg.group;
        auto row_of = [&](int r) { return out_row0 + static_cast<int64_t>(token_of(r)) * p.groups; };
        auto gate_of = [&](int r, int h) {      // of query row r, head h
            const unsigned row = static_cast<unsigned>(seg.request);
            const unsigned token = REGIONS ? quotient(row, p.region_groups_inv) : 0u;
            const int group = REGIONS ? static_cast<int>(row - token * p.region_groups) : seg.group;
            return gate_factor(p.gate[(REGIONS ? static_cast<int64_t>(token)
                                               : static_cast<int64_t>(seg.request) * p.query_len + token_of(r)) * p.g_s0 +
                                      static_cast<int64_t>(group * H + h) * p.g_s1]);
        };
        const bool begins = seg.first == 0, ends = seg.last == seg.tiles;
        const bool whole = begins && ends;
        const int64_t piece = static_cast<int64_t>(v) * 2 + (begins ? 1 : 0);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            l_run[k] += __shfl_xor_sync(~0u, l_run[k], 1);
            l_run[k] += __shfl_xor_sync(~0u, l_run[k], 2);
            m_run[k] -= S::kLift;               // what sums and outputs are relative to
        }
        // A long unit's pieces of neighbouring workers are merged by the CTA where
        // they are all that its workers have: one piece for the join, not four.
        // The CTA's part of the line lies in the unit, and its first worker has a
        // tile (so every worker comes here once, with this segment).
        constexpr bool kShares = ALONE && S::kWorkers > 1;
        bool merged = kShares, from_start = false;
        if (S::kWorkers > 1 && !ALONE && !whole && state->used == p.workers) {
            const long long n = state->total, u0 = state->here.unit;
            const int w0 = static_cast<int>(blockIdx.x) * S::kWorkers;
            const long long x0 = boundary(p, n, w0);
            merged = x0 >= u0 && boundary(p, n, w0 + 1) > u0 + kUnitCost &&
                     boundary(p, n, w0 + S::kWorkers) <= u0 + seg.tiles + kUnitCost;
            from_start = x0 <= u0 + kUnitCost;                  // the first worker's piece begins the unit
        }
        if (merged) {
            // A worker's stages are used up, so its part of the ring can hold its output.
            constexpr int kRows = 16 * MT, kOut = S::kRing * S::kStageBytes / 4;       // of a worker
            constexpr int kStride = kRows * (D + 4) <= kOut ? D + 4 : D;
            static_assert(kRows * kStride <= kOut, "merge buffer");
            float *outs = reinterpret_cast<float *>(smem), *stats = reinterpret_cast<float *>(smem + S::kStatsOff);
            float *units = reinterpret_cast<float *>(smem + S::kUnitsOff);
            if (SCALED && mt == 0 && lane == 0)
                units[worker] = unit;
            if constexpr (MT > 1)
                __syncthreads();                // all of the worker's warps are through its last stage
            else
                __syncwarp();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 16 * mt + g + 8 * k;              // of the worker
                // one piece of the CTA's for the join: the first worker's
                if (!ALONE && worker > 0 && t == 0 && r < R)
                    p.part_lse[piece * R + r] = -INFINITY;
                if (t == 0)
                    *reinterpret_cast<float2 *>(stats + (worker * kRows + r) * 2) = make_float2(m_run[k], l_run[k]);
                float *dst = outs + worker * kOut + r * kStride;
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    if constexpr (FP8) {
                        *reinterpret_cast<float4 *>(dst + 16 * c + 4 * t) =
                            make_float4(o[2 * c][2 * k], o[2 * c + 1][2 * k], o[2 * c][2 * k + 1], o[2 * c + 1][2 * k + 1]);
                    } else {
                        *reinterpret_cast<float2 *>(dst + 16 * c + 2 * t) = make_float2(o[2 * c][2 * k], o[2 * c][2 * k + 1]);
                        *reinterpret_cast<float2 *>(dst + 16 * c + 8 + 2 * t) =
                            make_float2(o[2 * c + 1][2 * k], o[2 * c + 1][2 * k + 1]);
                    }
                }
            }
            if constexpr (CLUSTER) {
                // ---- A CTA's share of the rows, from the pieces of all workers of the cluster:
                // a lane looks at a piece's maximum, sum and unit, then all lanes add the outputs up.
                cluster_sync();
                const int lg_c = __ffs(p.cluster) - 1, pieces = p.cluster * S::kWorkers;
                const int lg = (MT == 1 ? 3 : 2) + (R <= 8 * MT ? 1 : 0) + lg_c;       // threads of a row
                const int r = static_cast<int>(threadIdx.x >> lg) * p.cluster + cluster_rank();
                const int rr = r < R ? r : 0, c0 = static_cast<int>(threadIdx.x) & ((1 << lg) - 1);
                const int among = min(32, 1 << lg), k = lane & (among - 1), lane0 = lane - k;   // pieces <= among
                const uint32_t stats_at = smem_u32(stats), outs_at = smem_u32(outs), units_at = smem_u32(units);
                float m = -INFINITY, l = 0.0f, u = 1.0f;
                if (k < pieces) {
                    const int cta = k / S::kWorkers, w = k - cta * S::kWorkers;
                    m = peer_f32(peer(stats_at + (w * kRows + rr) * 8, cta));
                    l = peer_f32(peer(stats_at + (w * kRows + rr) * 8 + 4, cta));
                    if constexpr (SCALED)
                        u = peer_f32(peer(units_at + w * 4, cta));
                }
                float M = m;
                for (int i = among / 2; i; i >>= 1)
                    M = fmaxf(M, __shfl_xor_sync(~0u, M, i));
                float of = m == -INFINITY ? 1.0f : fast_exp2(m - M);    // all of a worker that saw nothing is 0 (or not a number)
                float L = l * of;
                for (int i = among / 2; i; i >>= 1)
                    L += __shfl_xor_sync(~0u, L, i);
                const bool empty = M == -INFINITY && L == 0.0f;
                of *= (empty ? 0.0f : 1.0f / L) * u;
                const int h = rr - token_of(rr) * H;
                float f = 1.0f;
                if (p.gate)
                    f = gate_of(rr, h);
                uint16_t *out = p.output + row_of(rr) * p.o_s0 + h * p.o_s1;
                for (int d0 = 0; d0 < D; d0 += 4 << lg) {       // as many turns for every lane
                    const int d = d0 + 4 * c0;
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    // sixteen loads from other SMs on their way at a time (four: 2 us more)
#pragma unroll 16
                    for (int i = 0; i < pieces; ++i) {
                        const float g = __shfl_sync(~0u, of, lane0 + i);
                        if (d < D) {
                            const int cta = i / S::kWorkers, w = i - cta * S::kWorkers;
                            const float4 y = peer_f32x4(peer(outs_at + (w * kOut + rr * kStride + d) * 4, cta));
                            x.x += g * y.x;
                            x.y += g * y.y;
                            x.z += g * y.z;
                            x.w += g * y.w;
                        }
                    }
                    if (d < D && r < R && seg.len >= 0) {       // below 0: left as it was
                        const uint2 w = make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
                        if (p.o_vec) {
                            *reinterpret_cast<uint2 *>(out + d) = w;
                        } else {
                            out[d] = static_cast<uint16_t>(w.x);
                            out[d + 1] = static_cast<uint16_t>(w.x >> 16);
                            out[d + 2] = static_cast<uint16_t>(w.y);
                            out[d + 3] = static_cast<uint16_t>(w.y >> 16);
                        }
                    }
                }
                if (c0 == 0 && r < R && seg.len >= 0 && p.lse)
                    p.lse[row_of(r) * p.l_s0 + h * p.l_s1] = (empty ? -INFINITY : M + log2f(L)) * kLn2;
                cluster_sync();                 // the others have read this CTA's pieces
                break;                          // the unit is done
            }
            __syncthreads();
            const int64_t first = static_cast<int64_t>(v - worker) * 2 + (from_start ? 1 : 0);
            // As many threads for a row as there are for 16, or 8, of each tile.
            const int lg = (MT == 1 ? 3 : 2) + (R <= 8 * MT ? 1 : 0);
            const int r = static_cast<int>(threadIdx.x) >> lg, c0 = static_cast<int>(threadIdx.x) & ((1 << lg) - 1);
            if (r < R) {
                float2 st[S::kWorkers];
                float M = -INFINITY, L = 0.0f;
#pragma unroll
                for (int w = 0; w < S::kWorkers; ++w) {
                    st[w] = *reinterpret_cast<const float2 *>(stats + (w * kRows + r) * 2);
                    M = fmaxf(M, st[w].x);
                }
#pragma unroll
                for (int w = 0; w < S::kWorkers; ++w) {         // all of a worker that saw nothing is 0 (or not a number)
                    st[w].x = st[w].x == -INFINITY ? 1.0f : fast_exp2(st[w].x - M);
                    L += st[w].y * st[w].x;
                }
                const bool empty = M == -INFINITY && L == 0.0f;
                const float inv = empty ? 0.0f : 1.0f / L;
                const int h = r - token_of(r) * H;
                uint16_t *out = nullptr;
                float f = 1.0f;
                if constexpr (SCALED) {
#pragma unroll
                    for (int w = 0; w < S::kWorkers; ++w)
                        st[w].x *= units[w];
                }
                if constexpr (ALONE) {
                    f = vs;
                    if (p.gate)
                        f *= gate_of(r, h);
                    out = p.output + row_of(r) * p.o_s0 + h * p.o_s1;
                }
                float *part = p.partial + (first * R + r) * D;
#pragma unroll 2
                for (int d = 4 * c0; d < D; d += 4 << lg) {
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                    for (int w = 0; w < S::kWorkers; ++w) {
                        const float4 y = *reinterpret_cast<const float4 *>(outs + w * kOut + r * kStride + d);
                        const float of = st[w].x * inv;
                        x.x += of * y.x;
                        x.y += of * y.y;
                        x.z += of * y.z;
                        x.w += of * y.w;
                    }
                    if constexpr (!ALONE) {
                        *reinterpret_cast<float4 *>(part + d) = x;
                    } else {
                        const uint2 w = make_uint2(pack_bf16(x.x * f, x.y * f), pack_bf16(x.z * f, x.w * f));
                        if (p.o_vec) {
                            *reinterpret_cast<uint2 *>(out + d) = w;
                        } else {
                            out[d] = static_cast<uint16_t>(w.x);
                            out[d + 1] = static_cast<uint16_t>(w.x >> 16);
                            out[d + 2] = static_cast<uint16_t>(w.y);
                            out[d + 3] = static_cast<uint16_t>(w.y >> 16);
                        }
                    }
                }
                if (c0 == 0) {
                    const float lse2 = empty ? -INFINITY : M + log2f(L);
                    if (!ALONE)
                        p.part_lse[first * R + r] = lse2;
                    else if (p.lse)
                        p.lse[row_of(r) * p.l_s0 + h * p.l_s1] = lse2 * kLn2;
                }
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int r = k ? r1 : r0;
            const float L = l_run[k];
            if (kShares || merged || r >= R)
                continue;
            // only a row that saw nothing is empty: a sum that is not a number goes on
            const bool empty = m_run[k] == -INFINITY && L == 0.0f;
            const float lse2 = empty ? -INFINITY : m_run[k] + log2f(L);
            const int h = r - token_of(r) * H;
            const int64_t row = row_of(r);
            float f = empty ? 0.0f : 1.0f / L;
            if constexpr (SCALED)
                f *= unit;
            if (whole) {
                f *= vs;
                if (p.gate)
                    f *= gate_of(r, h);
                if (t == 0 && p.lse)
                    p.lse[row * p.l_s0 + h * p.l_s1] = lse2 * kLn2;
            } else if (t == 0) {
                p.part_lse[piece * R + r] = lse2;
            }
            uint16_t *out = p.output + row * p.o_s0 + h * p.o_s1;
            float *part = p.partial + (piece * R + r) * D;
            // E4M3: thread t has four dims of each 16; bf16: two of each 8
            constexpr int kRun = FP8 ? 4 : 2, kRuns = D / (4 * kRun);
            out += kRun * t;
            part += kRun * t;
            auto value = [&](int c, int i) { return (FP8 ? o[2 * c + (i & 1)][2 * k + (i >> 1)] : o[c][2 * k + i]) * f; };
            if (!whole) {
#pragma unroll
                for (int c = 0; c < kRuns; ++c) {
                    if constexpr (FP8)
                        *reinterpret_cast<float4 *>(part + 16 * c) =
                            make_float4(value(c, 0), value(c, 1), value(c, 2), value(c, 3));
                    else
                        *reinterpret_cast<float2 *>(part + 8 * c) = make_float2(value(c, 0), value(c, 1));
                }
            } else if (p.o_vec) {
#pragma unroll
                for (int c = 0; c < kRuns; ++c) {
                    const uint32_t w = pack_bf16(value(c, 0), value(c, 1));
                    if constexpr (FP8)
                        *reinterpret_cast<uint2 *>(out + 16 * c) = make_uint2(w, pack_bf16(value(c, 2), value(c, 3)));
                    else
                        *reinterpret_cast<uint32_t *>(out + 8 * c) = w;
                }
            } else {
#pragma unroll
                for (int c = 0; c < kRuns; ++c)
#pragma unroll
                    for (int i = 0; i < kRun; ++i)
                        out[4 * kRun * c + i] = __bfloat16_as_ushort(__float2bfloat16_rn(value(c, i)));
            }
        }
        // ---- The worker that has a cut unit's first tile lists it for the join.
        if (!ALONE && begins && !ends && mt == 0 && lane == 0) {
            const long long end = state->here.unit + kUnitCost + seg.tiles;     // past the unit's last tile
            const int n = static_cast<int>((end * state->used - 1) / state->total) - v + 1;
            const int rows = n > kManyPieces ? 1 : kJoinWarps, items = (R + rows - 1) / rows;
            const unsigned at = atomicAdd(p.flags + kItemWord, static_cast<unsigned>(items));
            for (int i = 0; i < items; ++i) {
                if (at + i >= kMaxItems) {                              // never, by what kMaxItems counts
                    atomicOr(p.flags, SDA_FLAG_BOUNDS);
                    break;
                }
                p.items[at + i] = {n, seg.request, seg.group, v, i * rows, min(rows, R - i * rows), {0, 0}};
            }
        }
    }

    // Requests without tokens: zeros.  A CTA alone with a unit knows its own.
    for (int q = blockIdx.x; q < (CLUSTER ? gridDim.x : ALONE ? p.requests * p.groups : p.requests); q += gridDim.x) {
        if (CLUSTER && cluster_rank() > 0)
            break;
        const int request = ALONE ? state->here.seg.request : q, g0 = ALONE ? state->here.seg.group : 0;
        const int len = ALONE ? state->here.seg.len : Line::length(p, q);
        if (!REGIONS && threadIdx.x == 0 && (!ALONE || len == p.cap) && p.seq_lens[request * p.len_s] > p.cap)
            atomicOr(p.flags, SDA_FLAG_BOUNDS);
        if (len != 0 || CLUSTER)                // a cluster has merged nothing to zeros
            continue;
        for (int gr = warp + g0 * H; gr < (ALONE ? (g0 + 1) * H : p.groups * H); gr += kWarps)          // [group][head]
            for (int j = 0; j < p.query_len; ++j) {
                const int h = gr % H;
                const int64_t row = (static_cast<int64_t>(request) * p.query_len + j) * p.groups + gr / H;
                uint16_t *out = p.output + row * p.o_s0 + h * p.o_s1;
                for (int d = lane; d < D; d += 32)
                    out[d] = 0;
                if (lane == 0 && p.lse)
                    p.lse[row * p.l_s0 + h * p.l_s1] = -INFINITY;
            }
    }

    // After a wait that ran out, copies may be in flight: they land before the
    // block's memory can go to another.
    __syncthreads();
    if (*timed_out && threadIdx.x < S::kStages) {
        const int n = reinterpret_cast<int *>(smem + S::kIssuedOff)[threadIdx.x];
        if (n > 0 && !mbar_wait(bars + 8 * threadIdx.x, static_cast<uint32_t>(n - 1) & 1u, kDrainLimitNs))
            atomicOr(p.flags, SDA_FLAG_TIMEOUT);
    }
}

template <int KIND, int D, int MT, bool FULL, int TAKERS, int WALKED>
sda_status launch_shape(const CUtensorMap &tmap, const Params &p, void *stream)
{
    using S = Shape<KIND, D, MT, FULL, TAKERS, WALKED>;
    static size_t raised[64] = {};
    if (!raise_smem(sda_paged_kernel<KIND, D, MT, FULL, TAKERS, WALKED>, S::kBytes, raised))
        return SDA_ERR_CUDA;
    return launch_pdl_clusters(sda_paged_kernel<KIND, D, MT, FULL, TAKERS, WALKED>, dim3(static_cast<unsigned>(p.ctas)),
                               dim3(kThreads), S::kBytes, TAKERS == kCluster ? p.cluster : 1, stream, tmap, p);
}

template <int KIND, int D, int MT, int TAKERS, int WALKED>
sda_status launch_pieces(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return p.piece == Shape<KIND, D, MT, true, TAKERS>::kSlots ? launch_shape<KIND, D, MT, true, TAKERS, WALKED>(tmap, p, stream)
                                                               : launch_shape<KIND, D, MT, false, TAKERS, WALKED>(tmap, p, stream);
}

template <int KIND, int D, int MT, int WALKED>
sda_status launch_tiles(const CUtensorMap &tmap, const Params &p, void *stream)
{
    // clusters: where the host chooses them
    if constexpr (Shape<KIND, D, MT, true>::kScaled && MT <= 2)
        if (p.cluster > 1)
            return launch_pieces<KIND, D, MT, kCluster, WALKED>(tmap, p, stream);
    return p.cta_units ? launch_pieces<KIND, D, MT, kCta, WALKED>(tmap, p, stream)
                       : launch_pieces<KIND, D, MT, kOnLine, WALKED>(tmap, p, stream);
}

template <int KIND, int D>
sda_status launch_dim(const CUtensorMap &tmap, const Params &p, void *stream)
{
    const int tiles = tiles_of_rows(p.rows);
    return tiles == 1   ? launch_tiles<KIND, D, 1, kTokens>(tmap, p, stream)
           : tiles == 2 ? launch_tiles<KIND, D, 2, kTokens>(tmap, p, stream)
                        : launch_tiles<KIND, D, 4, kTokens>(tmap, p, stream);
}

// Regions: a row of at most 16 heads is one tile.
template <int KIND, int D>
sda_status launch_regions(const CUtensorMap &tmap, const Params &p, void *stream)
{
    return p.extents ? launch_pieces<KIND, D, 1, kOnLine, kExtents>(tmap, p, stream)
                     : launch_tiles<KIND, D, 1, kRegions>(tmap, p, stream);
}

// One translation unit per head size and cache type.
using Launch = sda_status(const CUtensorMap &tmap, const Params &p, void *stream);
Launch launch_bf16_64, launch_bf16_128, launch_bf16_192, launch_bf16_256;
Launch launch_fp8_64, launch_fp8_128, launch_fp8_192, launch_fp8_256;
Launch launch_qe4m3_64, launch_qe4m3_128, launch_qe4m3_192, launch_qe4m3_256;
Launch launch_qint8_64, launch_qint8_128, launch_qint8_192, launch_qint8_256;
Launch regions_qe4m3_64, regions_qe4m3_128, regions_qe4m3_192, regions_qe4m3_256;
Launch regions_qint8_64, regions_qint8_128, regions_qint8_192, regions_qint8_256;

}  // namespace paged
}  // namespace sda
