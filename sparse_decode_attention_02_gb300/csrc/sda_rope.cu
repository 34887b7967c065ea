// Rotary positions with several axes, and keys and values into the paged cache.
//
// A pair (a, b) turned by the angle t becomes (a cos t - b sin t, b cos t + a
// sin t), t = position * inv_freq.  In turns, t / 2 pi = position * f with f held
// as a 64-bit fraction of a turn: the low 64 bits of the integer product are the
// fractional turn, so an angle of any position is reduced with no loss beyond
// f's own last bit (2^-33 of a turn at position 2^31), where an fp32 angle near
// 2^18 is off by 2^-6.
//
// The work is one pass over q, k and v, bound by memory.  A CTA takes one or
// more tokens: its threads fill a table of the tokens' (cos, sin) pairs in
// shared memory, once for all heads, while their first loads are in flight;
// then each thread keeps to one 16-dim chunk and walks over its rows, the next
// one loaded while one is turned, neighbouring lanes on neighbouring bytes.
// 16,363 tokens of 16 heads of 192 dims and 4 groups into an E4M3 cache: 147 us,
// 880 MB at 6.0 TB/s, reads and writes in equal parts; a decode batch of 256, 5.9
// us, and one token, 3.0 to 3.6 us, are latency: slot, angle, row and store once through.
// Five CTAs an SM and a row ahead: six 151 us, four 153; four rows ahead at two
// CTAs 227; query and key rows in the same CTAs 166.
#include "sda_common.cuh"

#include <algorithm>
#include <cmath>

namespace {

using namespace sda;

constexpr int kMaxThreads = 256;
constexpr int kMaxAxes = 4;
constexpr int kPairs = 8;                       // pairs of a chunk: 16 dims
constexpr int kMaxTokens = 16;                  // of a CTA
constexpr int kQueryTokens = 8;                 // of a CTA with queries, where there are many

struct RopeParams {
    const uint16_t *query, *key, *value;
    uint16_t *query_out;
    void *cache;
    int64_t q_s0, q_s1, o_s0, o_s1, k_s0, k_s1, v_s0, v_s1;
    int64_t c_s0, c_s1, c_s2;
    const int32_t *positions;
    int64_t p_s0, p_s1;
    const float *inv_freq;
    const int64_t *slots;
    const float *k_scale, *v_scale;
    unsigned int *flags;
    int64_t cache_slots;                        // pages * block
    float amplitude;
    int tokens, heads, groups, dim, half, block;   // half: pairs a head turns
    int axes, interleaved, sections[kMaxAxes];
    int query_ctas, query_tokens, kv_tokens;    // CTAs for the query; tokens of a CTA, of either kind
    int parts;                                  // CTAs that share the heads of the same tokens
};

__device__ __forceinline__ uint2 quantise(const float (&x)[8], float scale)
{
    // e4m3(x / scale): the quotient in fp32, then one rounding to E4M3.
    uint32_t w[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        uint16_t h[2];
#pragma unroll
        for (int j = 0; j < 2; ++j)
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(h[j])
                : "f"(__fdiv_rn(x[4 * k + 2 * j + 1], scale)), "f"(__fdiv_rn(x[4 * k + 2 * j], scale)));
        w[k] = h[0] | (static_cast<uint32_t>(h[1]) << 16);
    }
    return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint4 round_bf16(const float (&x)[8])
{
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ void widen(const uint4 &v, float (&x)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(w[i] << 16);
        x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// 2^64 / (2 pi) * |f|, modulo 2^64: a frequency in radians as a fraction of a
// turn, from f's 24-bit significand times the 64-bit constant.
__device__ __forceinline__ unsigned long long turns_of(float f)
{
    constexpr unsigned long long kPerRadian = 0x28BE60DB9391054Aull;    // floor(2^64 / (2 pi))
    const uint32_t bits = __float_as_uint(f);
    const int exponent = (bits >> 23) & 0xFF;
    const unsigned long long m = (bits & 0x7FFFFFu) | (exponent ? 0x800000u : 0u);
    const unsigned long long lo = m * kPerRadian, hi = __umul64hi(m, kPerRadian);
    const int down = 150 - max(exponent, 1);                            // f = m * 2^-down
    const unsigned long long t = down <= 0    ? (down > -64 ? lo << -down : 0ull)
                                 : down < 64  ? (lo >> down) | (hi << (64 - down))
                                 : down < 128 ? hi >> (down - 64)
                                              : 0ull;
    return bits >> 31 ? 0ull - t : t;
}

// One CTA's rows: the query heads, or the key and value heads, of its tokens.  A
// thread owns chunk j of its rows: 16 dims as two runs of eight.  Turned chunks
// hold eight pairs: dims (8j.., half + 8j..) or, adjacent, 16j..16j+15; the
// chunks behind them pass through.
template <bool KV, bool FP8, bool ADJACENT>
__device__ __forceinline__ void rope_rows(const RopeParams &p, float4 *turn, int64_t *cache_at, int t0, int tokens,
                                          int part)
{
    const int chunks = p.dim / 16, lanes = blockDim.x / chunks;
    const int j = threadIdx.x % chunks, y = threadIdx.x / chunks;
    const bool turned = j < p.half / kPairs;
    const int lo = turned && !ADJACENT ? kPairs * j : 16 * j;
    const int hi = turned && !ADJACENT ? p.half + kPairs * j : 16 * j + 8;
    const int heads = KV ? 2 * p.groups : p.heads;              // of a token: keys, then values

    // This thread's rows: number part * lanes + y of the CTA's, and every
    // `step`-th after it; the next is loaded while one is turned.
    const int step = lanes * p.parts;
    int tok = 0, head = part * lanes + y;       // of the next row; token >= tokens: none
    uint4 a, b;                                 // its two runs
    auto load = [&] {
        while (head >= heads && tok < tokens) {
            head -= heads;
            ++tok;
        }
        if (tok < tokens) {
            const bool v = KV && head >= p.groups;
            const uint16_t *src = !KV  ? p.query + (t0 + tok) * p.q_s0 + head * p.q_s1
                                  : !v ? p.key + (t0 + tok) * p.k_s0 + head * p.k_s1
                                       : p.value + (t0 + tok) * p.v_s0 + (head - p.groups) * p.v_s1;
            a = *reinterpret_cast<const uint4 *>(src + (v ? 16 * j : lo));
            b = *reinterpret_cast<const uint4 *>(src + (v ? 16 * j + 8 : hi));
        }
    };
    load();

    // ---- The tokens' places and (cos, sin) of their angles.
    for (int i = threadIdx.x; i < tokens; i += blockDim.x) {
        int64_t place = 0;
        if (p.slots) {
            const int64_t slot = p.slots[t0 + i];
            const bool bad = slot < 0 || (p.key && slot >= p.cache_slots);
            if (bad && slot != -1 && p.flags)
                atomicOr(p.flags, SDA_FLAG_BOUNDS);
            if (!bad && KV) {
                const int64_t page = slot / p.block;
                place = page * p.c_s0 + (slot - page * p.block) * p.c_s2;
            }
            place = bad ? -1 : place;
        }
        cache_at[i] = place;
    }
    for (int i = threadIdx.x; i < p.half * tokens; i += blockDim.x) {
        const int tk = i / p.half, pair = i - tk * p.half;
        int axis = 0;
        if (p.interleaved) {
            const int ax = pair % p.axes;
            axis = ax > 0 && pair / p.axes < p.sections[ax] ? ax : 0;
        } else {
            int end = p.sections[0];
            while (axis + 1 < p.axes && pair >= end)
                end += p.sections[++axis];
        }
        const long long pos = p.positions[axis * p.p_s0 + static_cast<int64_t>(t0 + tk) * p.p_s1];
        const long long turns = static_cast<long long>(static_cast<unsigned long long>(pos) * turns_of(p.inv_freq[pair]));
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f, &s, &c);   // * 2^-31
        reinterpret_cast<float2 *>(turn)[i] = make_float2(c * p.amplitude, s * p.amplitude);
    }
    __syncthreads();

    const float ks = FP8 && KV ? *p.k_scale : 1.0f, vs = FP8 && KV ? *p.v_scale : 1.0f;
    while (tok < tokens) {
        const int t = tok, h = head;
        float x[8], z[8];
        widen(a, x);
        widen(b, z);
        head += step;
        load();
        const int64_t token_at = cache_at[t];
        if (token_at < 0)
            continue;
        const bool v = KV && h >= p.groups;
        if (turned && !v) {
            const float4 *cs = turn + (t * p.half + kPairs * j) / 2;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float4 w = cs[i];                     // pairs 2i, 2i + 1 of the chunk
                float *r = ADJACENT ? (i < 2 ? x : z) + 4 * (i & 1) : nullptr;
                float &a0 = ADJACENT ? r[0] : x[2 * i], &b0 = ADJACENT ? r[1] : z[2 * i];
                float &a1 = ADJACENT ? r[2] : x[2 * i + 1], &b1 = ADJACENT ? r[3] : z[2 * i + 1];
                const float u0 = a0, u1 = a1;
                a0 = u0 * w.x - b0 * w.y;
                b0 = b0 * w.x + u0 * w.y;
                a1 = u1 * w.z - b1 * w.w;
                b1 = b1 * w.z + u1 * w.w;
            }
        }
        if constexpr (!KV) {
            uint16_t *dst = p.query_out + (t0 + t) * p.o_s0 + h * p.o_s1;
            *reinterpret_cast<uint4 *>(dst + lo) = round_bf16(x);
            *reinterpret_cast<uint4 *>(dst + hi) = round_bf16(z);
        } else {
            const int64_t place = token_at + (v ? h - p.groups : h) * p.c_s1;
            const int d0 = v ? p.dim + 16 * j : lo, d1 = v ? p.dim + 16 * j + 8 : hi;
            if constexpr (FP8) {
                uint8_t *dst = static_cast<uint8_t *>(p.cache) + place;
                *reinterpret_cast<uint2 *>(dst + d0) = quantise(x, v ? vs : ks);
                *reinterpret_cast<uint2 *>(dst + d1) = quantise(z, v ? vs : ks);
            } else {
                uint16_t *dst = static_cast<uint16_t *>(p.cache) + place;
                *reinterpret_cast<uint4 *>(dst + d0) = round_bf16(x);
                *reinterpret_cast<uint4 *>(dst + d1) = round_bf16(z);
            }
        }
    }
}

template <bool FP8, bool ADJACENT>
__global__ void __launch_bounds__(kMaxThreads, 5) sda_rope_kernel(const __grid_constant__ RopeParams p)
{
    extern __shared__ float4 turn[];            // [tokens][half / 2]: (cos, sin, cos, sin) of two pairs
    __shared__ int64_t cache_at[kMaxTokens];    // each token's place in the cache, -1: a row to leave out
    pdl_launch_dependents();
    pdl_wait();
    const int cta = static_cast<int>(blockIdx.x);
    if (cta < p.query_ctas) {
        const int t0 = cta / p.parts * p.query_tokens;
        rope_rows<false, FP8, ADJACENT>(p, turn, cache_at, t0, min(p.tokens - t0, p.query_tokens), cta % p.parts);
    } else {
        const int t0 = (cta - p.query_ctas) / p.parts * p.kv_tokens;
        rope_rows<true, FP8, ADJACENT>(p, turn, cache_at, t0, min(p.tokens - t0, p.kv_tokens),
                                       (cta - p.query_ctas) % p.parts);
    }
}

// [T, heads, D] bf16 with 16-byte aligned rows: SDA_OK, or what is wrong.
sda_status check_rows(const sda_tensor *t, int64_t tokens, int64_t dim)
{
    if (!dims_ok(t, 3) || t->dtype != SDA_DTYPE_BF16 || t->shape[0] != tokens || t->shape[2] != dim ||
        t->stride[2] != 1)
        return SDA_ERR_INVALID;
    if (t->shape[1] > (1 << 20))
        return SDA_ERR_UNSUPPORTED;
    const bool rows_ok = t->shape[0] <= 1 || (t->stride[0] * 2) % 16 == 0;
    const bool heads_ok = t->shape[1] <= 1 || (t->stride[1] * 2) % 16 == 0;
    return rows_ok && heads_ok && aligned(t->data, 16) ? SDA_OK : SDA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" sda_status sparse_decode_rope_append(const sda_tensor *query, const sda_tensor *query_out,
                                                const sda_tensor *key, const sda_tensor *value,
                                                const sda_tensor *positions, const sda_tensor *inv_freq,
                                                const int32_t *sections, int interleaved_axes,
                                                int adjacent_pairs, float amplitude, const sda_tensor *slots,
                                                const sda_tensor *cache, const float *k_scale,
                                                const float *v_scale, void *workspace, size_t workspace_bytes,
                                                void *stream)
{
    // ---- Contract.
    const sda_tensor *lead = query ? query : key;
    if (!lead || !dims_ok(lead, 3) || !query != !query_out || !key != !value || (key && (!cache || !slots)))
        return SDA_ERR_INVALID;
    const int64_t tokens = lead->shape[0], dim = lead->shape[2];
    for (const sda_tensor *t : {query, query_out, key, value})
        if (t) {
            const sda_status st = check_rows(t, tokens, dim);
            if (st != SDA_OK)
                return st;
        }
    if ((query && query->shape[1] != query_out->shape[1]) || (key && key->shape[1] != value->shape[1]))
        return SDA_ERR_INVALID;
    // Rows that are written must be apart.
    if (query_out && ((tokens > 1 && query_out->stride[0] == 0) ||
                      (query_out->shape[1] > 1 && query_out->stride[1] == 0)))
        return SDA_ERR_INVALID;
    if (query && query->data == query_out->data &&
        ((tokens > 1 && query->stride[0] != query_out->stride[0]) ||
         (query->shape[1] > 1 && query->stride[1] != query_out->stride[1])))
        return SDA_ERR_INVALID;
    if (dim < 16 || dim % 16 != 0 || dim > 512 || tokens > (1 << 28))
        return SDA_ERR_UNSUPPORTED;
    if (!std::isfinite(amplitude))
        return SDA_ERR_INVALID;
    int64_t half = 0, axes = 1;
    int32_t parts[kMaxAxes] = {};
    if (positions) {
        if (!dims_ok(positions, 2) || positions->dtype != SDA_DTYPE_INT32 || positions->shape[1] != tokens ||
            !dims_ok(inv_freq, 1) || inv_freq->dtype != SDA_DTYPE_FP32)
            return SDA_ERR_INVALID;
        axes = positions->shape[0];
        half = inv_freq->shape[0];
        if (axes < 1 || axes > kMaxAxes || 2 * half > dim || (half > 1 && inv_freq->stride[0] != 1) ||
            (!sections && axes != 1))
            return SDA_ERR_INVALID;
        if (half < 8 || half % 8 != 0)
            return SDA_ERR_UNSUPPORTED;
        int64_t sum = 0;
        for (int a = 0; a < axes; ++a) {
            parts[a] = sections ? sections[a] : static_cast<int32_t>(half);
            if (parts[a] < 0)
                return SDA_ERR_INVALID;
            sum += parts[a];
            if (interleaved_axes && a > 0 && parts[a] > (half - a + axes - 1) / axes)
                return SDA_ERR_INVALID;
        }
        if (sum != half)
            return SDA_ERR_INVALID;
    }
    if (slots && (!dims_ok(slots, 1) || slots->dtype != SDA_DTYPE_INT64 || slots->shape[0] != tokens ||
                  (tokens > 1 && slots->stride[0] != 1)))
        return SDA_ERR_INVALID;
    bool fp8 = false;
    if (key) {
        fp8 = is_fp8(cache);
        if (!dims_ok(cache, 4) || (!fp8 && cache->dtype != SDA_DTYPE_BF16) || cache->shape[3] != 2 * dim ||
            cache->shape[1] != key->shape[1] || cache->stride[3] != 1 || cache->shape[0] < 1 ||
            cache->shape[2] < 1)
            return SDA_ERR_INVALID;
        if (fp8 && (!k_scale || !v_scale))
            return SDA_ERR_INVALID;
        const int elt = fp8 ? 1 : 2;
        if (cache->shape[2] > INT32_MAX || !aligned(cache->data, 16))
            return SDA_ERR_UNSUPPORTED;
        for (int i = 0; i < 3; ++i)
            if (cache->stride[i] <= 0 || (cache->stride[i] * elt) % 16 != 0)
                return SDA_ERR_UNSUPPORTED;
    }
    if (workspace ? (!aligned(workspace, 256) || workspace_bytes < kHeaderBytes) : workspace_bytes != 0)
        return SDA_ERR_WORKSPACE;
    const int64_t heads = query ? query->shape[1] : 0, groups = key ? key->shape[1] : 0;
    if (tokens == 0 || heads + groups == 0)
        return SDA_OK;
    for (const sda_tensor *t : {query, query_out, key, value, positions, slots, key ? cache : nullptr})
        if (t && !t->data && !(t == query && heads == 0) && !(t == query_out && heads == 0) && groups + heads > 0)
            return SDA_ERR_INVALID;
    if (positions && !inv_freq->data)
        return SDA_ERR_INVALID;

    RopeParams p = {};
    auto in16 = [](const sda_tensor *t) { return static_cast<const uint16_t *>(t->data); };
    if (query && heads > 0) {
        p.query = in16(query);
        p.query_out = static_cast<uint16_t *>(const_cast<void *>(query_out->data));
        p.q_s0 = query->stride[0], p.q_s1 = query->stride[1];
        p.o_s0 = query_out->stride[0], p.o_s1 = query_out->stride[1];
    }
    if (key && groups > 0) {
        p.key = in16(key);
        p.value = in16(value);
        p.k_s0 = key->stride[0], p.k_s1 = key->stride[1];
        p.v_s0 = value->stride[0], p.v_s1 = value->stride[1];
        p.cache = const_cast<void *>(cache->data);
        p.c_s0 = cache->stride[0], p.c_s1 = cache->stride[1], p.c_s2 = cache->stride[2];
        p.cache_slots = cache->shape[0] * cache->shape[2];
        p.block = static_cast<int>(cache->shape[2]);
        p.k_scale = k_scale;
        p.v_scale = v_scale;
    }
    if (positions) {
        p.positions = static_cast<const int32_t *>(positions->data);
        p.p_s0 = positions->stride[0], p.p_s1 = positions->stride[1];
        p.inv_freq = static_cast<const float *>(inv_freq->data);
    }
    p.slots = slots ? static_cast<const int64_t *>(slots->data) : nullptr;
    p.flags = static_cast<unsigned int *>(workspace);
    p.amplitude = amplitude;
    p.tokens = static_cast<int>(tokens);
    p.heads = static_cast<int>(heads);
    p.groups = static_cast<int>(groups);
    p.dim = static_cast<int>(dim);
    p.half = static_cast<int>(half);
    p.axes = static_cast<int>(axes);
    p.interleaved = interleaved_axes ? 1 : 0;
    for (int a = 0; a < kMaxAxes; ++a)
        p.sections[a] = parts[a];

    const int sms = sm_count();
    if (sms < 1)
        return SDA_ERR_CUDA;
    const int chunks = static_cast<int>(dim) / 16, most = kMaxThreads / chunks;
    // Many tokens (sixteen an SM): a few to a CTA, so that the table of angles keeps
    // all threads busy (64 heads of 192 dims and 4 groups, E4M3, against one each:
    // 16,000 tokens 151 us, 179; 1,000 tokens 18.5, 16.1; four and sixteen to a CTA
    // 154, 156).  Few: a token to a CTA, its heads shared by CTAs until each SM has
    // one (the same heads: one token 3.7 us, unshared 4.3; 64 tokens 4.2, with two
    // CTAs an SM 4.9).  Keys and values have CTAs of their own, with more tokens for
    // their fewer rows.
    const int rows = static_cast<int>(std::max(heads, 2 * groups));
    const bool many = tokens >= 16 * static_cast<int64_t>(sms);
    p.query_tokens = many ? kQueryTokens : 1;
    p.kv_tokens = many ? static_cast<int>(std::clamp<int64_t>(kQueryTokens * heads / std::max<int64_t>(1, 2 * groups),
                                                              kQueryTokens, kMaxTokens))
                       : 1;
    auto blocks = [&](int64_t h, int per) { return h > 0 ? (tokens + per - 1) / per : 0; };
    const int64_t ctas = blocks(heads, p.query_tokens) + blocks(groups, p.kv_tokens);
    p.parts = 1;
    while (ctas * p.parts < sms && p.parts * most < rows)
        p.parts *= 2;
    p.query_ctas = static_cast<int>(blocks(heads, p.query_tokens) * p.parts);
    // Threads for as many rows at a time as take the fewest turns, none of them short.
    const int longest = rows * (heads > 0 ? p.query_tokens : p.kv_tokens);
    const int turns = (longest + most * p.parts - 1) / (most * p.parts);
    const int lanes = (longest + turns * p.parts - 1) / (turns * p.parts);
    const dim3 grid(static_cast<unsigned>(ctas * p.parts)), block(static_cast<unsigned>(chunks * lanes));
    const size_t smem = sizeof(float2) * static_cast<size_t>(std::max(p.query_tokens, p.kv_tokens)) *
                        static_cast<size_t>(half);
    auto kernel = fp8 ? (adjacent_pairs ? sda_rope_kernel<true, true> : sda_rope_kernel<true, false>)
                      : (adjacent_pairs ? sda_rope_kernel<false, true> : sda_rope_kernel<false, false>);
    return launch_pdl(kernel, grid, block, smem, stream, p);
}
