// Rotary positions with several axes, and keys and values into the paged cache.
//
// A pair (a, b) turned by the angle t becomes (a cos t - b sin t, b cos t + a
// sin t), t = position * inv_freq.  In turns, t / 2 pi = position * f with f in
// [0, 1) held as a 64-bit fraction: the low 64 bits of the integer product are
// the fractional turn, so an angle of any position is reduced with no loss
// beyond f's own 2^-53, where an fp32 angle near 2^18 is off by 2^-6.
//
// The work is one pass over q, k and v: bound by memory.  A CTA takes one or
// more tokens: its threads first fill a table of the tokens' (cos, sin) pairs
// in shared memory, once for all heads; then each thread keeps the eight pairs
// of its chunk of a head in registers and walks over the heads, 32 bytes in and
// 32 out at a time, neighbouring lanes on neighbouring bytes.
#include "sda_common.cuh"

#include <cmath>

namespace {

using namespace sda;

constexpr int kMaxThreads = 256;
constexpr int kMaxAxes = 4;
constexpr int kPairs = 8;                       // pairs of a chunk: 16 dims
constexpr int kAhead = 2;                       // heads a thread loads before it turns them

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
    int per_cta, parts;                         // tokens a CTA takes; CTAs that share a token's heads
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

// A thread owns chunk j of the heads: 16 dims as two runs of eight.  Turned
// chunks hold eight pairs: dims (8j.., half + 8j..) or, adjacent, 16j..16j+15;
// the chunks behind them pass through.
template <bool FP8, bool ADJACENT>
__global__ void __launch_bounds__(kMaxThreads) sda_rope_kernel(const __grid_constant__ RopeParams p)
{
    extern __shared__ float2 turn[];            // [per_cta][half] (cos, sin)
    pdl_launch_dependents();
    pdl_wait();

    const int chunks = p.dim / 16, lanes = blockDim.x / chunks;
    const int j = threadIdx.x % chunks, y = threadIdx.x / chunks;
    const int part = blockIdx.x % p.parts;
    const int t0 = static_cast<int>(blockIdx.x / p.parts) * p.per_cta, t1 = min(p.tokens, t0 + p.per_cta);
    const bool turned = j < p.half / kPairs;
    const int lo = turned && !ADJACENT ? kPairs * j : 16 * j;
    const int hi = turned && !ADJACENT ? p.half + kPairs * j : 16 * j + 8;

    // ---- (cos, sin) of the tokens' angles.
    for (int i = threadIdx.x; i < p.half * (t1 - t0); i += blockDim.x) {
        const int tok = i / p.half, pair = i - tok * p.half;
        int axis = 0;
        if (p.interleaved) {
            const int a = pair % p.axes;
            axis = a > 0 && pair / p.axes < p.sections[a] ? a : 0;
        } else {
            int end = p.sections[0];
            while (axis + 1 < p.axes && pair >= end)
                end += p.sections[++axis];
        }
        const double f = static_cast<double>(p.inv_freq[pair]) * 0.15915494309189533577;   // / 2 pi
        const unsigned long long frac = __double2ull_rn((f - floor(f)) * 18446744073709551616.0);
        const long long pos = p.positions[axis * p.p_s0 + static_cast<int64_t>(t0 + tok) * p.p_s1];
        const long long turns = static_cast<long long>(static_cast<unsigned long long>(pos) * frac);
        float s, c;
        sincospif(static_cast<float>(static_cast<int>(turns >> 32)) * 4.656612873077393e-10f, &s, &c);   // * 2^-31
        turn[i] = make_float2(c * p.amplitude, s * p.amplitude);
    }
    __syncthreads();

    const float ks = FP8 && p.key ? *p.k_scale : 1.0f, vs = FP8 && p.key ? *p.v_scale : 1.0f;
    const int total = p.heads + (p.key ? 2 * p.groups : 0);      // q heads, then k, then v
    const int stride = lanes * p.parts;
    if (y >= lanes)
        return;
    for (int t = t0; t < t1; ++t) {
        int64_t slot = -1;
        if (p.slots) {
            slot = p.slots[t];
            if (slot < 0 || (p.key && slot >= p.cache_slots)) {
                if (slot != -1 && p.flags && threadIdx.x == 0)
                    atomicOr(p.flags, SDA_FLAG_BOUNDS);
                continue;
            }
        }
        int64_t page = 0, off = 0;
        if (p.key) {
            page = slot / p.block;
            off = slot - page * p.block;
        }
        float2 cs[kPairs];
        if (turned) {
#pragma unroll
            for (int i = 0; i < kPairs; ++i)
                cs[i] = turn[(t - t0) * p.half + kPairs * j + i];
        }
        for (int h0 = part * lanes + y; h0 < total; h0 += stride * kAhead) {
            uint4 a[kAhead], b[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int h = h0 + k * stride;
                if (h < total) {
                    const int kh = h - p.heads;                  // >= 0: k head, then v head
                    const uint16_t *src = kh < 0 ? p.query + t * p.q_s0 + h * p.q_s1
                                          : kh < p.groups ? p.key + t * p.k_s0 + kh * p.k_s1
                                                          : p.value + t * p.v_s0 + (kh - p.groups) * p.v_s1;
                    const bool v = kh >= p.groups;
                    a[k] = *reinterpret_cast<const uint4 *>(src + (v ? 16 * j : lo));
                    b[k] = *reinterpret_cast<const uint4 *>(src + (v ? 16 * j + 8 : hi));
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const int h = h0 + k * stride;
                if (h >= total)
                    break;
                const int kh = h - p.heads;
                const bool v = kh >= p.groups;
                float x[8], z[8];
                widen(a[k], x);
                widen(b[k], z);
                if (turned && !v) {
                    if constexpr (ADJACENT) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float x0 = x[2 * i], x1 = x[2 * i + 1], z0 = z[2 * i], z1 = z[2 * i + 1];
                            x[2 * i] = x0 * cs[i].x - x1 * cs[i].y;
                            x[2 * i + 1] = x1 * cs[i].x + x0 * cs[i].y;
                            z[2 * i] = z0 * cs[4 + i].x - z1 * cs[4 + i].y;
                            z[2 * i + 1] = z1 * cs[4 + i].x + z0 * cs[4 + i].y;
                        }
                    } else {
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            const float x0 = x[i], z0 = z[i];
                            x[i] = x0 * cs[i].x - z0 * cs[i].y;
                            z[i] = z0 * cs[i].x + x0 * cs[i].y;
                        }
                    }
                }
                const int d0 = v ? 16 * j : lo, d1 = v ? 16 * j + 8 : hi;
                if (kh < 0) {
                    uint16_t *dst = p.query_out + t * p.o_s0 + h * p.o_s1;
                    *reinterpret_cast<uint4 *>(dst + d0) = round_bf16(x);
                    *reinterpret_cast<uint4 *>(dst + d1) = round_bf16(z);
                } else {
                    const int64_t at = page * p.c_s0 + (v ? kh - p.groups : kh) * p.c_s1 + off * p.c_s2 +
                                       (v ? p.dim : 0);
                    if constexpr (FP8) {
                        uint8_t *dst = static_cast<uint8_t *>(p.cache) + at;
                        *reinterpret_cast<uint2 *>(dst + d0) = quantise(x, v ? vs : ks);
                        *reinterpret_cast<uint2 *>(dst + d1) = quantise(z, v ? vs : ks);
                    } else {
                        uint16_t *dst = static_cast<uint16_t *>(p.cache) + at;
                        *reinterpret_cast<uint4 *>(dst + d0) = round_bf16(x);
                        *reinterpret_cast<uint4 *>(dst + d1) = round_bf16(z);
                    }
                }
            }
        }
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
    const int chunks = static_cast<int>(dim) / 16, lanes = kMaxThreads / chunks;
    const int total = static_cast<int>(heads + 2 * groups);
    // Many tokens: four to a CTA, so that the table of angles keeps all threads
    // busy.  Few: a token's heads are shared by CTAs until each SM has two.
    p.per_cta = tokens >= 16 * static_cast<int64_t>(sms) ? 4 : 1;
    const int64_t ctas = (tokens + p.per_cta - 1) / p.per_cta;
    p.parts = 1;
    while (ctas * p.parts < 2 * sms && p.parts * lanes < total)
        p.parts *= 2;
    const dim3 grid(static_cast<unsigned>(ctas * p.parts)), block(static_cast<unsigned>(chunks * lanes));
    const size_t smem = sizeof(float2) * static_cast<size_t>(p.per_cta) * static_cast<size_t>(half);
    auto kernel = fp8 ? (adjacent_pairs ? sda_rope_kernel<true, true> : sda_rope_kernel<true, false>)
                      : (adjacent_pairs ? sda_rope_kernel<false, true> : sda_rope_kernel<false, false>);
    return launch_pdl(kernel, grid, block, smem, stream, p);
}
