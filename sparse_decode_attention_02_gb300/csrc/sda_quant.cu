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
// first is written.  A CTA looks at some rows for runs that begin there, and a team of
// its warps takes each: all eight where there is one (a prompt's block), a warp
// where there are many (a decode batch).  The rows' first loads are kept in registers
// for the second pass.
//
// Read.  One pass, bound by memory: a byte in and two out an element.  A thread keeps
// to 16 elements of a head's row and walks over tokens, whose places are looked up
// once for a CTA.
#include "sda_quant.cuh"

#include <algorithm>

namespace {

using namespace sda;

constexpr int kWarps = 8;
constexpr int kThreads = kWarps * 32;
constexpr int kMaxChunk = 64;                   // rows that a CTA looks at for runs
constexpr int kKept = 8;                        // 8-element pieces that a thread keeps between the passes

struct AppendParams {
    const uint16_t *key, *value;
    int64_t k_s0, k_s1, v_s0, v_s1;
    const int64_t *slots;
    uint8_t *cache;
    int64_t c_s0, c_s1, c_s2;
    float *scales;
    int64_t s_s0, s_s1, s_s2;
    unsigned int *flags;
    int64_t cache_slots;                        // pages * block
    int tokens, groups, dim, block, span, chunk;
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

// The larger |x| of the bf16 pairs in a and b, half by half, as bits.
__device__ __forceinline__ uint32_t larger(uint32_t a, uint32_t b)
{
    return __vmaxu2(a, b & 0x7FFF7FFFu);
}

// The same over finite values only.
__device__ __forceinline__ uint32_t larger_finite(uint32_t a, uint32_t b)
{
    b &= 0x7FFF7FFFu;
    b &= ((b & 0xFFFFu) >= 0x7F80u ? 0u : 0xFFFFu) | (b >= 0x7F800000u ? 0u : 0xFFFF0000u);
    return __vmaxu2(a, b);
}

template <bool INT8>
__device__ __forceinline__ uint2 quantise(const uint4 &v, float scale, float inverse)
{
    // x / scale; where the scale is a power of two the product by its reciprocal is the same
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        x[i] = __uint_as_float(i & 1 ? w[i >> 1] & 0xFFFF0000u : w[i >> 1] << 16);
        x[i] = inverse != 0.0f ? x[i] * inverse : __fdiv_rn(x[i], scale);
    }
    return make_uint2(to_elements<INT8>(x[0], x[1], x[2], x[3]), to_elements<INT8>(x[4], x[5], x[6], x[7]));
}

template <bool INT8>
__global__ void __launch_bounds__(kThreads) sda_quantised_append_kernel(const __grid_constant__ AppendParams p)
{
    __shared__ int runs[kMaxChunk];             // first rows of the runs that begin in this chunk
    __shared__ int count;
    __shared__ uint32_t tops[2][kWarps];        // largest element of each warp, by turns
    pdl_launch_dependents();
    pdl_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int units = 2 * p.groups;
    const int unit = static_cast<int>(blockIdx.x % static_cast<unsigned>(units));
    const int row0 = static_cast<int>(blockIdx.x / static_cast<unsigned>(units)) * p.chunk;
    const bool value = unit & 1;
    const int group = unit >> 1;
    auto valid = [&](int64_t slot) { return slot >= 0 && slot < p.cache_slots; };

    // ---- Runs: rows whose neighbour before them lies in another block.
    if (threadIdx.x == 0)
        count = 0;
    __syncthreads();
    if (static_cast<int>(threadIdx.x) < p.chunk && row0 + static_cast<int>(threadIdx.x) < p.tokens) {
        const int r = row0 + threadIdx.x;
        const int64_t slot = p.slots[r], before = r > 0 ? p.slots[r - 1] : -1;
        if (valid(slot)) {
            const bool joins = valid(before) && before / p.span == slot / p.span;
            if (!joins)
                runs[atomicAdd(&count, 1)] = r;
            else if (slot != before + 1 && p.flags)             // the block's rows are not in order: left out
                atomicOr(p.flags, SDA_FLAG_BOUNDS);
        } else if (slot != -1 && p.flags) {
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

    const int vecs = p.dim / 8;                 // 8-element pieces of a row
    const int row_step = threads / vecs, vec_step = threads - row_step * vecs;
    const uint16_t *src = value ? p.value + group * p.v_s1 : p.key + group * p.k_s1;
    const int64_t src_row = value ? p.v_s0 : p.k_s0;
    int turn = 0;
    for (int i = mine; i < n; i += teams, turn ^= 1) {
        const int r0 = runs[i];
        const int64_t slot = p.slots[r0];
        const int64_t page = slot / p.block;
        const int off = static_cast<int>(slot - page * p.block), part = off / p.span, place = off - part * p.span;
        float *at = p.scales + page * p.s_s0 + group * p.s_s1 + part * p.s_s2 + (value ? 1 : 0);
        const float had = place > 0 ? *at : 0.0f;
        // its length: rows with consecutive slots, up to the block's end
        int length = min(p.span - place, p.tokens - r0);
        for (int k = 0; k < length; k += 32) {
            const bool goes_on = k + lane < length && p.slots[r0 + k + lane] == slot + k + lane;
            const unsigned m = __ballot_sync(~0u, goes_on);
            if (m != ~0u) {
                length = min(length, k + __ffs(~m) - 1);
                break;
            }
        }

        // ---- The largest element; the first pieces stay in registers.
        const uint16_t *rows = src + r0 * src_row;
        uint4 kept[kKept];
        uint32_t top = 0;
        int row = tid / vecs, vec = tid - row * vecs;
        auto step = [&](int &row, int &vec) {
            row += row_step;
            vec += vec_step;
            if (vec >= vecs) {
                vec -= vecs;
                ++row;
            }
        };
        const int row_first = row, vec_first = vec;
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            kept[k] = make_uint4(0, 0, 0, 0);
            if (row < length)
                kept[k] = *reinterpret_cast<const uint4 *>(rows + row * src_row + 8 * vec);
            step(row, vec);
        }
        const int row_rest = row, vec_rest = vec;
#pragma unroll
        for (int k = 0; k < kKept; ++k)
            top = larger(larger(larger(larger(top, kept[k].x), kept[k].y), kept[k].z), kept[k].w);
        for (; row < length; step(row, vec)) {
            const uint4 v = *reinterpret_cast<const uint4 *>(rows + row * src_row + 8 * vec);
            top = larger(larger(larger(larger(top, v.x), v.y), v.z), v.w);
        }
        auto over_team = [&](uint32_t x, int which) {
            x = __reduce_max_sync(~0u, max(x & 0xFFFFu, x >> 16));
            if (team > 1) {
                if (lane == 0)
                    tops[which][warp] = x;
                together();
                x = 0;
                for (int w = 0; w < team; ++w)
                    x = max(x, tops[which][mine * team + w]);
            }
            return x;
        };
        top = over_team(top, turn);
        if (top >= 0x7F80u) {                   // something is not finite: the rest decides
            if (tid == 0 && p.flags)
                atomicOr(p.flags, SDA_FLAG_NONFINITE);
            together();                         // `tops` has been read
            top = 0;
            row = row_first;
            vec = vec_first;
            for (; row < length; step(row, vec)) {
                const uint4 v = *reinterpret_cast<const uint4 *>(rows + row * src_row + 8 * vec);
                top = larger_finite(larger_finite(larger_finite(larger_finite(top, v.x), v.y), v.z), v.w);
            }
            top = over_team(top, turn);
            together();
        }
        const float need = least_scale<INT8>(__uint_as_float(top << 16));
        const float scale = fmaxf(had, need);
        together();                             // every thread has read the scale that was there
        if (tid == 0 && (place == 0 || scale != had))
            *at = scale;

        // ---- Places before the rows, where the scale grew.
        uint8_t *base = p.cache + page * p.c_s0 + group * p.c_s1 + (value ? p.dim : 0);
        if (place > 0 && scale > had) {
            const float factor = __fdiv_rn(had, scale);
            const int pieces = p.dim / 16;
            uint8_t *first = base + static_cast<int64_t>(off - place) * p.c_s2;
            for (int k = tid; k < place * pieces; k += threads) {
                const int row = k / pieces;
                uint4 *v = reinterpret_cast<uint4 *>(first + row * p.c_s2 + 16 * (k - row * pieces));
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
        const uint32_t bits = __float_as_uint(scale);
        // 2^-k for 2^k; its exponent is in 1..252, so that the reciprocal is normal
        const float inverse = (bits & 0x7FFFFFu) == 0 && (bits >> 23) < 253u ? __uint_as_float((254u << 23) - bits) : 0.0f;
        uint8_t *out = base + off * p.c_s2;
        row = row_first;
        vec = vec_first;
#pragma unroll
        for (int k = 0; k < kKept; ++k) {
            if (row < length)
                *reinterpret_cast<uint2 *>(out + row * p.c_s2 + 8 * vec) = quantise<INT8>(kept[k], scale, inverse);
            step(row, vec);
        }
        row = row_rest;
        vec = vec_rest;
        for (; row < length; step(row, vec)) {
            const uint4 v = *reinterpret_cast<const uint4 *>(rows + row * src_row + 8 * vec);
            *reinterpret_cast<uint2 *>(out + row * p.c_s2 + 8 * vec) = quantise<INT8>(v, scale, inverse);
        }
    }
}

// ---------------------------------------------------------------------------
// Read
// ---------------------------------------------------------------------------

constexpr int kReadTurns = 8;                   // rows of a thread, at most
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
};

template <bool INT8>
__global__ void __launch_bounds__(kThreads) sda_quantised_read_kernel(const __grid_constant__ ReadParams p)
{
    extern __shared__ int64_t where[];          // [rows of the CTA] x (place in the cache, -1: none; its scales')
    __shared__ int owners[2];                   // requests of the CTA's first and last row
    pdl_launch_dependents();
    pdl_wait();
    const int group = static_cast<int>(blockIdx.x % static_cast<unsigned>(p.groups));
    const int per = p.lanes * p.turns;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x / static_cast<unsigned>(p.groups)) * per;
    const int rows = static_cast<int>(min(static_cast<int64_t>(per), p.rows - row0));

    // ---- The requests of the first and the last row, all threads' samples of the
    // starts at a time: the last start at or before the row.
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
        if (threadIdx.x == 0)
            owners[which] = lo;
    }
    __syncthreads();
    const int q0 = max(owners[0], 0), q1 = min(owners[1], p.requests - 1);
    for (int i = threadIdx.x; i < rows; i += blockDim.x) {
        const int r = static_cast<int>(row0) + i;
        int lo = q0, hi = q1;
        while (lo < hi) {                       // the last request that begins at or before the row
            const int mid = (lo + hi + 1) >> 1;
            if (p.starts[mid] <= r)
                lo = mid;
            else
                hi = mid - 1;
        }
        int64_t place = -1, scale = 0;
        if (lo <= hi && r >= p.starts[lo] && r < p.starts[lo + 1]) {
            const int64_t token = static_cast<int64_t>(r) - p.starts[lo] + (p.first ? p.first[lo * p.first_s] : 0);
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
        uint4 *dst = reinterpret_cast<uint4 *>(out + (row0 + i) * out_row);
        dst[0] = make_uint4(z[0], z[1], z[2], z[3]);
        dst[1] = make_uint4(z[4], z[5], z[6], z[7]);
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
    p.cache_slots = q.pages * q.block;
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
    const int64_t ctas = (tokens + p.chunk - 1) / p.chunk * 2 * groups;
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
