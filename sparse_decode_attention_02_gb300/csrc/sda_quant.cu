// Keys and values into a quantised cache, and back out of it.
//
// Append.  A block of `span` places of a head has one scale for its keys and one
// for its values.  With a = the largest finite |x| of the rows that a step writes
// into the block, the least scale that holds them is
//     E4M3      the smallest power of two s with a <= 448 s
//     integers  a / 127
// (at least 2^-126).  Where the rows begin the block that is its scale; else the
// larger of it and the scale that is there, and if that grew by a factor 1 / f the
// places before the rows are rounded again: e4m3(f e), or rint(f e).  A power of two
// costs an E4M3 block nothing (its elements have an exponent of their own) and makes f
// exact, so that elements but the smallest keep their value however often a scale
// grows.  Integers lose half a step of the new scale each time.
//
// Neighbouring rows with consecutive slots in one block are a run, and a run of one
// head's keys or values is the unit of work: its largest element must be known before the
// first is written.  A CTA lists the runs that begin in some rows, once for all of its
// warps, and a team of them takes each: all eight where there is one (a prompt's block), a
// warp where there are many (a decode batch).  A run's first loads stay in registers for
// the second pass.  16,363 tokens of 4 heads of 192 dims: 18 to 19 us in E4M3, 24 in integers
// (75.5 MB, floor 11; 15.7 from L2: bound by the start and by the chain slots, run, rows,
// maximum, stores of 3.4 waves of CTAs); a decode batch of 256 3.7 to 4.2 us, one token 2.3.
// Those batches are steps in which no scale grows.  One in which every block's does, with 15
// places before the row to round again on average, takes 14.5 us, integers 16.3 (4.9 and 5.1
// without, from as many caches in turn): a warp does a head's keys or values alone.
// The first CTAs write nothing: they look for a block whose rows stand in two places, which
// would be two runs that race for its scale and its places.
//
// Read.  One pass, bound by memory: a byte in and two out an element.  A thread keeps
// to 16 elements of a head's row and walks over tokens, whose places are looked up
// once for a CTA.  131,003 tokens of the same heads 92 us, 6.5 TB/s; twelve contexts of 2K to
// 8K (integers, 2 heads of 128 dims) 17 us (13 where the reads' 25 MB lie in L2), where the
// look-ups before the first store are a third.
#include "sda_quant.cuh"

#include <algorithm>
#include <type_traits>

namespace {

using namespace sda;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
// Rows that a CTA lists runs of: a prompt's blocks of 64 tokens one each (20 us; with 32 rows 25, with 128 27).
constexpr int kMaxChunk = 64;
// A CTA that looks for blocks in two places takes those that begin in one part of kLookRows rows and
// compares them with another part behind it, every two parts once.  Beside four requests' tokens or a
// prompt's they end before the others do (0.0 to 0.3 us more; 4000 requests' tokens of one head of 64 dims
// 6.0 -> 6.9, 16,001 of a prompt's 4.4 -> 5.1; with parts of 1024 rows 7.1 and 5.6, of 512 6.2 and 6.3).  Of more
// rows than kMaxLooked they would be the call: 32,001 rows 7.1 -> 8.3.
constexpr int kLookBits = 11, kLookRows = 1 << kLookBits, kMaxLooked = 1 << 14;
// 8-element pieces that a thread keeps between the passes, the rest is loaded again: what
// four CTAs an SM have registers for, and 64 tokens of 192 dims need (six 22.6 us, three CTAs with eight 22.4).
constexpr int kKept = 7;

struct AppendParams {
    const uint16_t *key, *value;
    int64_t k_s0, k_s1, v_s0, v_s1;
    const int64_t *slots;
    uint8_t *cache;
    int64_t c_s0, c_s1, c_s2;
    float *scales;
    int64_t s_s0, s_s1, s_s2;
    unsigned int *flags;
    uint32_t cache_slots;                       // pages * block
    unsigned long long block_inv, span_inv, vecs_inv;       // inverse_of a page's places, a block's, 8-element pieces of a row
    int tokens, groups, dim, block, span, chunk;
    int lookers, look_parts;                    // CTAs ahead of the others that look for blocks in two places; parts
};

// A run of rows in one block, of one head's keys or values.
struct Run {
    uint8_t *cache;                             // the block's first place
    float *scale;
    int row, place, length;                     // first row and place; (within the CTA's window of rows)
};

// Four fp32 values to E4M3 bytes, rounded to nearest even, saturated at 448.
__device__ __forceinline__ uint32_t to_e4m3(float a, float b, float c, float d)
{
    uint16_t lo, hi;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
    return lo | (static_cast<uint32_t>(hi) << 16);
}

// Four fp32 values to integers, rounded to nearest even, at most 127 in size; not a number: 0.
__device__ __forceinline__ uint32_t to_int8(float a, float b, float c, float d)
{
    auto one = [](float x) { return static_cast<uint32_t>(max(-127, min(127, __float2int_rn(x)))) & 0xFFu; };
    return one(a) | (one(b) << 8) | (one(c) << 16) | (one(d) << 24);
}

template <bool INT8>
__device__ __forceinline__ uint32_t to_elements(float a, float b, float c, float d)
{
    return INT8 ? to_int8(a, b, c, d) : to_e4m3(a, b, c, d);
}

// A word's four elements.
template <bool INT8>
__device__ __forceinline__ float4 from_elements(uint32_t w)
{
    uint32_t lo, hi;
    if constexpr (INT8) {
        const uint32_t x = w ^ 0x80808080u;
        lo = int8x2_to_f16x2<0, 1>(x);
        hi = int8x2_to_f16x2<2, 3>(x);
    } else {
        lo = e4m3x2_to_f16x2(w);
        hi = e4m3x2_to_f16x2(w >> 16);
    }
    const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&lo));
    const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
    return make_float4(a.x, a.y, b.x, b.y);
}

// The least scale that holds values of up to `largest`, finite and >= 0.
template <bool INT8>
__device__ __forceinline__ float least_scale(float largest)
{
    if constexpr (INT8) {
        return fmaxf(__fdiv_rn(largest, 127.0f), kSmallestScale);
    } else {
        // largest = m 2^k with 1 <= m < 2, 448 = 1.75 * 2^8: 2^(k - 8), or twice that where m > 1.75
        const uint32_t bits = __float_as_uint(largest);
        const int e = static_cast<int>(bits >> 23) - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
        return __uint_as_float(static_cast<uint32_t>(max(e, 1)) << 23);
    }
}

// The larger |x| of the bf16 pairs in a and b, half by half and with any sign; not a
// number if one is not.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The same over finite values only, as bits.
__device__ __forceinline__ uint32_t larger_finite(uint32_t a, uint32_t b)
{
    b &= 0x7FFF7FFFu;
    b &= ((b & 0xFFFFu) >= 0x7F80u ? 0u : 0xFFFFu) | (b >= 0x7F800000u ? 0u : 0xFFFF0000u);
    return __vmaxu2(a, b);
}

// Eight values over the scale, as elements.  `inverse`: the scale's reciprocal, in fp32.
template <bool INT8, bool POWER_OF_TWO>
__device__ __forceinline__ uint2 quantise(const uint4 &v, float scale, float inverse)
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
        x[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
    if constexpr (INT8) {
        // The product by the reciprocal is off by 2^-23 of itself at most, the quotient in
        // fp32 by 2^-24: away from a border by more than 2^-15 (of values up to 127) both
        // round to the same integer.  1.5 * 2^23 added to it leaves it in the low bits.
        constexpr float kInteger = 12582912.0f;
        uint32_t bits[8];
        bool clear = true;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float y = x[i] * inverse, z = y + kInteger;
            clear = clear && fabsf(y - (z - kInteger)) < 0.5f - 0x1p-15f;       // not so if y is not finite
            bits[i] = __float_as_uint(z);
        }
        if (clear)
            return make_uint2(bytes_of<0x5410u>(bytes_of<0x0040u>(bits[0], bits[1]), bytes_of<0x0040u>(bits[2], bits[3])),
                              bytes_of<0x5410u>(bytes_of<0x0040u>(bits[4], bits[5]), bytes_of<0x0040u>(bits[6], bits[7])));
    }
    if constexpr (!INT8 && POWER_OF_TWO) {             // the quotient, exactly (or next to 0, and less than E4M3 has)
        const __nv_bfloat162 f = __bfloat162bfloat162(__float2bfloat16_rn(inverse));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat162 y = __hmul2(*reinterpret_cast<const __nv_bfloat162 *>(&w[i]), f);
            const uint32_t z = *reinterpret_cast<const uint32_t *>(&y);
            x[2 * i] = __uint_as_float(z << 16);
            x[2 * i + 1] = __uint_as_float(z & 0xFFFF0000u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            x[i] = __fdiv_rn(x[i], scale);
    }
    return make_uint2(to_elements<INT8>(x[0], x[1], x[2], x[3]), to_elements<INT8>(x[4], x[5], x[6], x[7]));
}

// A thread's 8-element pieces of a run.  WIDE, threads for a row or more: each keeps to
// a place in the row, and those beyond whole rows have none.  Else a row's pieces by turns.
template <class T, bool WIDE>
struct Pieces {
    T *at;
    int row, vec;
    int64_t step;                               // in elements: to the next piece
    int rows, threads, vecs;                    // rows of all threads at a time; pieces of a row
    int64_t wrap;                               // (not WIDE) more, where the next is the first of its row

    __device__ __forceinline__ Pieces(T *base, int64_t stride, int tid, int threads, const AppendParams &p)
        : threads(threads), vecs(p.dim / 8)
    {
        rows = static_cast<int>(quotient(threads, p.vecs_inv));
        row = WIDE ? static_cast<int>(quotient(tid, p.vecs_inv)) : 0;
        vec = tid - row * vecs;
        at = base + row * stride + 8 * vec;
        if (WIDE && row >= rows)
            row = INT32_MAX / 2;
        step = WIDE ? rows * stride : 8 * threads;
        wrap = WIDE ? 0 : stride - 8 * ((vecs - vec + threads - 1) / threads) * threads;
    }

    __device__ __forceinline__ void next()
    {
        at += step;
        if constexpr (WIDE) {
            row += rows;
        } else {
            vec += threads;
            if (vec >= vecs) {
                vec %= threads;
                at += wrap;
                ++row;
            }
        }
    }
};

constexpr uint32_t kNone = ~0u;                 // not a slot, nor a block: there are fewer

// Row r's slot; kNone for padding, with `outside` where it is not in the cache, and past the rows.
__device__ __forceinline__ uint32_t slot_of(const AppendParams &p, int r, bool &outside)
{
    const int64_t slot = r >= 0 && r < p.tokens ? p.slots[r] : -1;
    if (static_cast<uint64_t>(slot) < p.cache_slots)
        return static_cast<uint32_t>(slot);
    outside = outside || slot != -1;
    return kNone;
}

// Whether a block of which rows begin (behind a row of another, or of none) in this looker's part of
// the rows has others that begin there too, or in the part behind that it looks at.  `blocks`: a
// hash table with room for twice a part.
__device__ __forceinline__ bool block_in_two_places(const AppendParams &p, uint32_t (&blocks)[2 * kLookRows], int looker)
{
    const int part = looker % p.look_parts, behind = part + 1 + looker / p.look_parts;
    const int tid = static_cast<int>(threadIdx.x);
    if (behind > part + 1 && behind >= p.look_parts)
        return false;
    auto home = [](uint32_t b) { return (b * 2654435769u) >> (31 - kLookBits); };        // 2^32 / golden ratio
    auto after = [](uint32_t at) { return (at + 1) % (2 * kLookRows); };
    bool outside = false, twice = false;
    // the block that row r begins, or kNone
    auto begun = [&](int r) {
        const uint32_t slot = slot_of(p, r, outside), before = slot_of(p, r - 1, outside);
        const uint32_t block = quotient(slot, p.span_inv);
        return slot != kNone && (before == kNone || quotient(before, p.span_inv) != block) ? block : kNone;
    };
    constexpr int kEach = kLookRows / kThreads;
    uint32_t b[kEach];
    auto load = [&](int from) {
#pragma unroll
        for (int k = 0; k < kEach; ++k)
            b[k] = begun(from + k * kThreads + tid);
    };
    for (int i = tid; i < 2 * kLookRows; i += kThreads)
        blocks[i] = kNone;
    load(part * kLookRows);
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (b[k] != kNone)
            for (uint32_t at = home(b[k]), was;; at = after(at)) {
                was = atomicCAS(&blocks[at], kNone, b[k]);
                if (was == kNone || was == b[k]) {
                    twice = twice || was == b[k];
                    break;
                }
            }
    __syncthreads();
    load(behind * kLookRows);
#pragma unroll
    for (int k = 0; k < kEach; ++k)
        if (b[k] != kNone)
            for (uint32_t at = home(b[k]); blocks[at] != kNone; at = after(at))
                twice = twice || blocks[at] == b[k];
    return twice;
}

template <bool INT8>
__global__ void __launch_bounds__(kThreads, 4) sda_quantised_append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ Run runs[kMaxChunk];             // that begin in this chunk
    __shared__ uint32_t goes_on[kWarps];        // rows of the window that continue the one before, a bit each
    __shared__ int count;
    __shared__ uint32_t tops[2][kWarps];        // largest element of each warp, by turns
    __shared__ uint32_t looked[2 * kLookRows];
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (static_cast<int>(blockIdx.x) < p.lookers) {
        if (block_in_two_places(p, looked, static_cast<int>(blockIdx.x)))
            atomicOr(p.flags, SDA_FLAG_BOUNDS);
        return;
    }
    const unsigned units = 2 * p.groups, cta = blockIdx.x - p.lookers;
    const int unit = static_cast<int>(cta % units);
    const int row0 = static_cast<int>(cta / units) * p.chunk;
    const bool value = unit & 1;
    const int group = unit >> 1;

    // ---- Runs.  The window is a row a thread; a run begins where the row before lies in
    // another block (or nowhere).
    if (threadIdx.x == 0)
        count = 0;
    const int r = row0 + static_cast<int>(threadIdx.x);         // < 2^29
    bool outside = false;
    const uint32_t slot = slot_of(p, r, outside), before = slot_of(p, r - 1, outside);
    if (outside && p.flags)
        atomicOr(p.flags, SDA_FLAG_BOUNDS);
    const bool joins = slot != kNone && before != kNone && quotient(slot, p.span_inv) == quotient(before, p.span_inv);
    const unsigned on = __ballot_sync(~0u, joins && slot == before + 1);
    if (lane == 0)
        goes_on[warp] = on;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.chunk && slot != kNone) {
        if (!joins) {
            const uint32_t page = quotient(slot, p.block_inv), off = slot - page * p.block;
            const uint32_t part = quotient(off, p.span_inv), place = off - part * p.span;
            int length = 1, i = static_cast<int>(threadIdx.x) + 1;              // rows of the window from here that go on
            while (i < kThreads) {
                const uint32_t stops = ~goes_on[i >> 5] >> (i & 31);
                const int some = stops ? __ffs(stops) - 1 : 32;
                length += min(some, 32 - (i & 31));
                if (stops && some < 32 - (i & 31))
                    break;
                i = (i | 31) + 1;
            }
            runs[atomicAdd(&count, 1)] = {p.cache + page * p.c_s0 + group * p.c_s1 + (value ? p.dim : 0) + (off - place) * p.c_s2,
                                          p.scales + page * p.s_s0 + group * p.s_s1 + part * p.s_s2 + (value ? 1 : 0), r,
                                          static_cast<int>(place), length};
        } else if (slot != before + 1 && p.flags) {             // the block's rows are not in order: left out
            atomicOr(p.flags, SDA_FLAG_BOUNDS);
        }
    }
    __syncthreads();
    const int n = count;
    const int team = n <= 1 ? kWarps : n <= 2 ? kWarps / 2 : n <= 4 ? kWarps / 4 : 1;       // warps of one
    const int mine = warp / team, teams = kWarps / team;
    const int tid = (warp % team) * 32 + lane, threads = team * 32;
    auto together = [&] {
        if (team == 1)
            __syncwarp();
        else
            asm volatile("bar.sync %0, %1;" ::"r"(1 + mine), "r"(threads) : "memory");
    };

    const uint16_t *src = value ? p.value + group * p.v_s1 : p.key + group * p.k_s1;
    const int64_t src_row = value ? p.v_s0 : p.k_s0;
    int turn = 0;
    auto run = [&](int i, auto wide) {
        using In = Pieces<const uint16_t, decltype(wide)::value>;
        using Out = Pieces<uint8_t, decltype(wide)::value>;
        const Run &its = runs[i];
        const int r0 = its.row, place = its.place;
        float *at = its.scale;
        const float had = place > 0 ? *at : 0.0f;
        int length = its.length;
        if (r0 - row0 + length >= kThreads) {   // it goes on behind the window, up to the block's end
            const int64_t first = p.slots[r0];
            for (int most = min(p.span - place, p.tokens - r0); length < most;) {
                const bool one = length + lane < most && p.slots[r0 + length + lane] == first + length + lane;
                const unsigned m = __ballot_sync(~0u, one);
                length += m == ~0u ? 32 : __ffs(~m) - 1;
                if (m != ~0u)
                    break;
            }
        }

        // ---- The largest element; the first pieces stay in registers.
        const uint16_t *rows = src + r0 * src_row;
        uint4 kept[kKept];
        uint32_t top = 0;
        auto top_of = [](uint32_t top, const uint4 &v) { return larger(larger(larger(larger(top, v.x), v.y), v.z), v.w); };
        {
            In in(rows, src_row, tid, threads, p);
#pragma unroll
            for (int k = 0; k < kKept; ++k) {
                kept[k] = in.row < length ? *reinterpret_cast<const uint4 *>(in.at) : make_uint4(0, 0, 0, 0);
                in.next();
            }
            const bool rest = in.row < length;
#pragma unroll
            for (int k = 0; k < kKept; ++k)
                top = top_of(top, kept[k]);
            if (rest)
                for (; in.row < length; in.next())
                    top = top_of(top, *reinterpret_cast<const uint4 *>(in.at));
        }
        auto over_team = [&](uint32_t x, int which) {
            x = __reduce_max_sync(~0u, max(x & 0x7FFFu, (x >> 16) & 0x7FFFu));
            if (team > 1) {
                if (lane == 0)
                    tops[which][warp] = x;
                together();
                x = __reduce_max_sync(~0u, lane < team ? tops[which][mine * team + lane] : 0u);
            }
            return x;
        };
        top = over_team(top, turn);
        if (top >= 0x7F80u) {                   // something is not finite: the rest decides
            if (tid == 0 && p.flags)
                atomicOr(p.flags, SDA_FLAG_NONFINITE);
            together();                         // `tops` has been read
            top = 0;
            for (In in(rows, src_row, tid, threads, p); in.row < length; in.next()) {
                const uint4 v = *reinterpret_cast<const uint4 *>(in.at);
                top = larger_finite(larger_finite(larger_finite(larger_finite(top, v.x), v.y), v.z), v.w);
            }
            top = over_team(top, turn);
            together();
        }
        const float need = least_scale<INT8>(__uint_as_float(top << 16));
        const float scale = fmaxf(had, need);
        if (team == 1)
            __syncwarp();                       // every thread has read the scale that was there (else before the team's maximum)
        if (tid == 0 && (place == 0 || scale != had))
            *at = scale;

        // ---- Places before the rows, where the scale grew.
        if (place > 0 && scale > had) {
            const float factor = __fdiv_rn(had, scale);
            const int pieces = p.dim / 16;
            for (int k = tid; k < place * pieces; k += threads) {
                const int row = k / pieces;
                uint4 *v = reinterpret_cast<uint4 *>(its.cache + row * p.c_s2 + 16 * (k - row * pieces));
                const uint4 x = *v;
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
                uint32_t z[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float4 y = from_elements<INT8>(w[j]);
                    z[j] = to_elements<INT8>(y.x * factor, y.y * factor, y.z * factor, y.w * factor);
                }
                *v = make_uint4(z[0], z[1], z[2], z[3]);
            }
        }

        // ---- The rows.
        auto write = [&](auto power_of_two) {
            constexpr bool kPower = decltype(power_of_two)::value;
            const float inverse = __frcp_rn(scale);
            Out out(its.cache + place * p.c_s2, p.c_s2, tid, threads, p);
#pragma unroll
            for (int k = 0; k < kKept; ++k) {
                if (out.row < length)
                    *reinterpret_cast<uint2 *>(out.at) = quantise<INT8, kPower>(kept[k], scale, inverse);
                out.next();
            }
            if (out.row < length) {
                In in(rows, src_row, tid, threads, p);
                for (int k = 0; k < kKept; ++k)
                    in.next();
                for (; out.row < length; in.next(), out.next())
                    *reinterpret_cast<uint2 *>(out.at) =
                        quantise<INT8, kPower>(*reinterpret_cast<const uint4 *>(in.at), scale, inverse);
            }
        };
        if (!INT8 && (__float_as_uint(scale) & 0x7FFFFFu) == 0 && scale < 0x1p126f)
            write(std::true_type{});
        else
            write(std::false_type{});
    };
    for (int i = mine; i < n; i += teams, turn ^= 1) {
        if (threads >= p.dim / 8)
            run(i, std::true_type{});
        else
            run(i, std::false_type{});
    }
}

// ---------------------------------------------------------------------------
// Read
// ---------------------------------------------------------------------------

// Rows of a thread, at most: six CTAs an SM with four loads each in flight (twelve contexts
// 17.3 us; eight rows at four CTAs 22.6, at three 21.3), which leave a thread 40 registers and
// spill 12 bytes of it beside E4M3, 4 beside integers.
constexpr int kReadTurns = 4;
constexpr int kMaxReadRows = kThreads / 2 * kReadTurns;         // of a CTA (16 dims: two threads a row)

struct ReadParams {
    const uint8_t *cache;
    int64_t c_s0, c_s1, c_s2;
    const float *scales;
    int64_t s_s0, s_s1, s_s2;
    const int32_t *table;
    int64_t t_s0;
    const int32_t *starts, *first;              // first: NULL or where each request is read from
    int64_t first_s;
    uint16_t *key, *value;
    int64_t k_s0, k_s1, v_s0, v_s1;
    unsigned int *flags;
    long long pages;
    unsigned long long block_inv, span_inv;
    int rows, groups, dim, block, requests, width;
    int lanes, turns;                           // rows of a CTA at a time, and how often
    int wide;                                   // rows on 32-byte boundaries
};

template <bool INT8>
__global__ void __launch_bounds__(kThreads, 6) sda_quantised_read_kernel(const __grid_constant__ ReadParams p)
{
    extern __shared__ int64_t where[];          // [rows of the CTA] x (place in the cache, -1: none; its scales')
    __shared__ int32_t starts_here[kThreads], first_here[kThreads];
    pdl_launch_dependents();
    pdl_wait();
    const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.groups));
    const int per = p.lanes * p.turns;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(p.groups)) * per;
    const int rows = static_cast<int>(min(static_cast<int64_t>(per), p.rows - row0));

    // ---- The rows' requests: the last start at or before the row.  Few requests' starts
    // (and where they are read from) are looked at here once, at the same time; of many
    // a sample by all threads at a time, for the first and for the last row.
    const bool few = p.requests < kThreads;
    int q0, q1;
    if (few) {
        for (int i = threadIdx.x; i <= p.requests; i += blockDim.x) {
            starts_here[i] = p.starts[i];
            first_here[i] = p.first && i < p.requests ? p.first[i * p.first_s] : 0;
        }
        q0 = 0;
        q1 = p.requests - 1;
    } else {
#pragma unroll 1
        for (int which = 0; which < 2; ++which) {
            const int64_t r = row0 + (which ? rows - 1 : 0);
            int lo = 0, size = p.requests + 1;
            while (size > 1) {
                const int step = (size + blockDim.x - 1) / blockDim.x, at = static_cast<int>(threadIdx.x) * step;
                const int before = __syncthreads_count(at < size && p.starts[lo + at] <= r);
                if (before == 0) {
                    lo = -1;
                    break;
                }
                lo += (before - 1) * step;
                size = min(step, size - (before - 1) * step);
            }
            if (which)
                q1 = min(lo, p.requests - 1);
            else
                q0 = max(lo, 0);
        }
    }
    __syncthreads();
    const int32_t *starts = few ? starts_here : p.starts;
    for (int i = threadIdx.x; i < rows; i += blockDim.x) {
        const int r = static_cast<int>(row0) + i;
        int lo = q0, hi = q1;
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (starts[mid] <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        int64_t place = -1, scale = 0;
        if (lo <= hi && r >= starts[lo] && r < starts[lo + 1]) {
            const int first = few ? first_here[lo] : p.first ? p.first[lo * p.first_s] : 0;
            const int64_t token = static_cast<int64_t>(r) - starts[lo] + first;
            const bool inside = token >= 0 && token <= INT32_MAX;
            const int col = inside ? static_cast<int>(quotient(static_cast<uint32_t>(token), p.block_inv)) : p.width;
            const int page = col < p.width ? p.table[lo * p.t_s0 + col] : -1;
            if (page >= 0 && page < p.pages) {
                const int off = static_cast<int>(token - static_cast<int64_t>(col) * p.block);
                place = page * p.c_s0 + off * p.c_s2;
                scale = page * p.s_s0 + static_cast<int64_t>(quotient(static_cast<uint32_t>(off), p.span_inv)) * p.s_s2;
            } else if (p.flags) {
                atomicOr(p.flags, SDA_FLAG_BOUNDS);
            }
        }
        where[2 * i] = place;
        where[2 * i + 1] = scale;
    }
    __syncthreads();

    // ---- A thread's 16 elements of a row, keys or values, row after row.
    const int pieces = p.dim / 16, cols = 2 * pieces;
    const int y = static_cast<int>(threadIdx.x) / cols, col = static_cast<int>(threadIdx.x) - y * cols;
    const bool value = col >= pieces;
    uint16_t *out = value ? p.value : p.key;
    if (y >= p.lanes || !out)
        return;
    const int dims = 16 * (value ? col - pieces : col);
    out += group * (value ? p.v_s1 : p.k_s1) + dims;
    const int64_t out_row = value ? p.v_s0 : p.k_s0;
    const uint8_t *src = p.cache + group * p.c_s1 + 16 * col;
    const float *scales = p.scales + group * p.s_s1 + (value ? 1 : 0);
    uint4 x[kReadTurns];
    float s[kReadTurns];
#pragma unroll
    for (int k = 0; k < kReadTurns; ++k) {
        const int i = y + k * p.lanes;
        const bool some = k < p.turns && i < rows && where[2 * i] >= 0;
        x[k] = make_uint4(0, 0, 0, 0);
        s[k] = -1.0f;
        if (some) {
            x[k] = *reinterpret_cast<const uint4 *>(src + where[2 * i]);
            s[k] = scales[where[2 * i + 1]];
        }
    }
#pragma unroll
    for (int k = 0; k < kReadTurns; ++k) {
        const int i = y + k * p.lanes;
        if (k >= p.turns || i >= rows || where[2 * i] < 0)
            continue;
        const uint32_t w[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
        uint32_t z[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const float4 v = from_elements<INT8>(w[j]);
            z[2 * j] = pack_bf16(v.x * s[k], v.y * s[k]);
            z[2 * j + 1] = pack_bf16(v.z * s[k], v.w * s[k]);
        }
        uint16_t *dst = out + (row0 + i) * out_row;
        if (p.wide) {
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(z[0]), "r"(z[1]), "r"(z[2]),
                         "r"(z[3]), "r"(z[4]), "r"(z[5]), "r"(z[6]), "r"(z[7])
                         : "memory");
        } else {
            reinterpret_cast<uint4 *>(dst)[0] = make_uint4(z[0], z[1], z[2], z[3]);
            reinterpret_cast<uint4 *>(dst)[1] = make_uint4(z[4], z[5], z[6], z[7]);
        }
    }
}

// [T, G, D] bf16 rows on 16-byte boundaries: SDA_OK, or what is wrong.
sda_status check_rows(const sda_tensor *t, int64_t tokens, int64_t groups, int64_t dim)
{
    if (!dims_ok(t, 3) || t->dtype != SDA_DTYPE_BF16 || t->shape[0] != tokens || t->shape[1] != groups ||
        t->shape[2] != dim || t->stride[2] != 1)
        return SDA_ERR_INVALID;
    const bool rows_ok = t->shape[0] <= 1 || (t->stride[0] * 2) % 16 == 0;
    const bool heads_ok = t->shape[1] <= 1 || (t->stride[1] * 2) % 16 == 0;
    return rows_ok && heads_ok && aligned(t->data, 16) ? SDA_OK : SDA_ERR_UNSUPPORTED;
}

sda_status check_workspace(const void *workspace, size_t bytes)
{
    return workspace ? (aligned(workspace, 256) && bytes >= kHeaderBytes ? SDA_OK : SDA_ERR_WORKSPACE)
           : bytes   ? SDA_ERR_WORKSPACE
                     : SDA_OK;
}

}  // namespace

extern "C" sda_status sparse_decode_quantised_append(const sda_tensor *key, const sda_tensor *value, const sda_tensor *slots,
                                                     const sda_tensor *cache, const sda_tensor *scales, void *workspace,
                                                     size_t workspace_bytes, void *stream)
{
    if (!dims_ok(key, 3) || !dims_ok(slots, 1) || slots->dtype != SDA_DTYPE_INT64)
        return SDA_ERR_INVALID;
    const int64_t tokens = key->shape[0], groups = key->shape[1], dim = key->shape[2];
    for (const sda_tensor *t : {key, value}) {
        const sda_status st = check_rows(t, tokens, groups, dim);
        if (st != SDA_OK)
            return st;
    }
    if (slots->shape[0] != tokens || (tokens > 1 && slots->stride[0] != 1))
        return SDA_ERR_INVALID;
    if (dim < 16 || dim % 16 != 0 || dim > 512 || tokens > (1 << 28))
        return SDA_ERR_UNSUPPORTED;
    QuantisedCache q;
    sda_status st = check_quantised(cache, scales, dim, q);
    if (st != SDA_OK)
        return st;
    if (q.groups != groups)
        return SDA_ERR_INVALID;
    if (q.pages * q.block >= UINT32_MAX)
        return SDA_ERR_UNSUPPORTED;
    st = check_workspace(workspace, workspace_bytes);
    if (st != SDA_OK || tokens == 0)
        return st;
    for (const sda_tensor *t : {key, value, slots, cache, scales})
        if (!t->data)
            return SDA_ERR_INVALID;

    AppendParams p = {};
    p.key = static_cast<const uint16_t *>(key->data);
    p.value = static_cast<const uint16_t *>(value->data);
    p.k_s0 = key->stride[0], p.k_s1 = key->stride[1];
    p.v_s0 = value->stride[0], p.v_s1 = value->stride[1];
    p.slots = static_cast<const int64_t *>(slots->data);
    p.cache = static_cast<uint8_t *>(const_cast<void *>(cache->data));
    p.c_s0 = cache->stride[0], p.c_s1 = cache->stride[1], p.c_s2 = cache->stride[2];
    p.scales = static_cast<float *>(const_cast<void *>(scales->data));
    p.s_s0 = scales->stride[0], p.s_s1 = scales->stride[1], p.s_s2 = scales->stride[2];
    p.flags = static_cast<unsigned int *>(workspace);
    p.cache_slots = static_cast<uint32_t>(q.pages * q.block);
    p.block_inv = inverse_of(static_cast<unsigned>(q.block));
    p.span_inv = inverse_of(static_cast<unsigned>(q.span));
    p.vecs_inv = inverse_of(static_cast<unsigned>(dim / 8));
    p.tokens = static_cast<int>(tokens);
    p.groups = static_cast<int>(groups);
    p.dim = static_cast<int>(dim);
    p.block = static_cast<int>(q.block);
    p.span = static_cast<int>(q.span);
    const int sms = sm_count();
    if (sms < 1)
        return SDA_ERR_CUDA;
    // As many rows to a CTA as leave each SM two of them, at least one a warp.
    p.chunk = kMaxChunk;
    while (p.chunk > kWarps && (tokens + p.chunk - 1) / p.chunk * 2 * groups < 2 * sms)
        p.chunk /= 2;
    if (p.flags && tokens > 1 && tokens <= kMaxLooked) {
        p.look_parts = static_cast<int>((tokens + kLookRows - 1) / kLookRows);
        p.lookers = p.look_parts * std::max(1, p.look_parts - 1);
    }
    const int64_t ctas = (tokens + p.chunk - 1) / p.chunk * 2 * groups + p.lookers;
    if (ctas > INT32_MAX)
        return SDA_ERR_UNSUPPORTED;
    auto kernel = q.int8 ? sda_quantised_append_kernel<true> : sda_quantised_append_kernel<false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), 0, stream, p);
}

extern "C" sda_status sparse_decode_quantised_read(const sda_tensor *cache, const sda_tensor *scales,
                                                   const sda_tensor *block_table, const sda_tensor *token_starts,
                                                   const sda_tensor *first_tokens, const sda_tensor *key,
                                                   const sda_tensor *value, void *workspace, size_t workspace_bytes,
                                                   void *stream)
{
    const sda_tensor *lead = key ? key : value;
    if (!lead || !dims_ok(lead, 3) || !dims_ok(block_table, 2) || block_table->dtype != SDA_DTYPE_INT32 ||
        !dims_ok(token_starts, 1) || token_starts->dtype != SDA_DTYPE_INT32)
        return SDA_ERR_INVALID;
    const int64_t rows = lead->shape[0], groups = lead->shape[1], dim = lead->shape[2];
    for (const sda_tensor *t : {key, value})
        if (t) {
            const sda_status st = check_rows(t, rows, groups, dim);
            if (st != SDA_OK)
                return st;
            if ((rows > 1 && t->stride[0] == 0) || (groups > 1 && t->stride[1] == 0))
                return SDA_ERR_INVALID;         // rows that are written must be apart
        }
    const int64_t requests = token_starts->shape[0] - 1;
    if (requests < 0 || (requests > 0 && token_starts->stride[0] != 1) || block_table->shape[0] < requests ||
        (block_table->shape[1] > 1 && block_table->stride[1] != 1))
        return SDA_ERR_INVALID;
    if (first_tokens && (!dims_ok(first_tokens, 1) || first_tokens->dtype != SDA_DTYPE_INT32 ||
                         first_tokens->shape[0] != requests))
        return SDA_ERR_INVALID;
    if (dim < 16 || dim % 16 != 0 || dim > 512 || rows > (1 << 30) || requests > (1 << 30) ||
        block_table->shape[1] > INT32_MAX)
        return SDA_ERR_UNSUPPORTED;
    QuantisedCache q;
    sda_status st = check_quantised(cache, scales, dim, q);
    if (st != SDA_OK)
        return st;
    if (q.groups != groups)
        return SDA_ERR_INVALID;
    st = check_workspace(workspace, workspace_bytes);
    if (st != SDA_OK || rows == 0 || requests == 0)
        return st;
    for (const sda_tensor *t : {cache, scales, token_starts, lead, key && value ? value : lead})
        if (!t->data)
            return SDA_ERR_INVALID;
    if ((first_tokens && !first_tokens->data) || (block_table->shape[1] > 0 && !block_table->data))
        return SDA_ERR_INVALID;

    ReadParams p = {};
    p.cache = static_cast<const uint8_t *>(cache->data);
    p.c_s0 = cache->stride[0], p.c_s1 = cache->stride[1], p.c_s2 = cache->stride[2];
    p.scales = static_cast<const float *>(scales->data);
    p.s_s0 = scales->stride[0], p.s_s1 = scales->stride[1], p.s_s2 = scales->stride[2];
    p.table = static_cast<const int32_t *>(block_table->data);
    p.t_s0 = block_table->stride[0];
    p.starts = static_cast<const int32_t *>(token_starts->data);
    if (first_tokens) {
        p.first = static_cast<const int32_t *>(first_tokens->data);
        p.first_s = first_tokens->stride[0];
    }
    auto out16 = [](const sda_tensor *t) { return t ? static_cast<uint16_t *>(const_cast<void *>(t->data)) : nullptr; };
    p.key = out16(key);
    p.value = out16(value);
    if (key)
        p.k_s0 = key->stride[0], p.k_s1 = key->stride[1];
    if (value)
        p.v_s0 = value->stride[0], p.v_s1 = value->stride[1];
    p.flags = static_cast<unsigned int *>(workspace);
    p.pages = q.pages;
    p.block_inv = inverse_of(static_cast<unsigned>(q.block));
    p.span_inv = inverse_of(static_cast<unsigned>(q.span));
    p.rows = static_cast<int>(rows);
    p.groups = static_cast<int>(groups);
    p.dim = static_cast<int>(dim);
    p.block = static_cast<int>(q.block);
    p.requests = static_cast<int>(requests);
    p.width = static_cast<int>(block_table->shape[1]);
    const int sms = sm_count();
    if (sms < 1)
        return SDA_ERR_CUDA;
    p.wide = 1;
    for (const sda_tensor *t : {key, value})
        if (t && (!aligned(t->data, 32) || (rows > 1 && t->stride[0] % 16 != 0) || (groups > 1 && t->stride[1] % 16 != 0)))
            p.wide = 0;
    const int cols = static_cast<int>(dim) / 8;
    p.lanes = kThreads / cols;
    // As many rows to a thread as leave each SM two CTAs.
    p.turns = kReadTurns;
    while (p.turns > 1 && (rows + p.lanes * p.turns - 1) / (p.lanes * p.turns) * groups < 2 * sms)
        p.turns /= 2;
    const int per = p.lanes * p.turns;
    const int64_t ctas = (rows + per - 1) / per * groups;
    if (ctas > INT32_MAX)
        return SDA_ERR_UNSUPPORTED;
    const size_t smem = 2 * sizeof(int64_t) * static_cast<size_t>(per);
    static_assert(2 * sizeof(int64_t) * kMaxReadRows <= 48 * 1024, "shared memory");
    auto kernel = q.int8 ? sda_quantised_read_kernel<true> : sda_quantised_read_kernel<false>;
    return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(static_cast<unsigned>(p.lanes * cols)), smem, stream, p);
}
