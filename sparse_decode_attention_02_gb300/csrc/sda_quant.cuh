// The quantised cache: elements of one byte (E4M3, or integers -127..127) and a
// scale for each block of `span` tokens of a head, for its keys and for its values.
// What the kernels and entry points that deal with it share.
#pragma once

#include "sda_common.cuh"

namespace sda {

// The smallest scale: quotients by it and its reciprocal are normal numbers.
constexpr float kSmallestScale = 1.17549435e-38f;               // 2^-126

// Two E4M3 bytes (low byte -> low half) to two fp16 values, exactly.
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t two)
{
    uint32_t r;
    const uint16_t v = static_cast<uint16_t>(two);
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(v));
    return r;
}

template <uint32_t SEL>
__device__ __forceinline__ uint32_t bytes_of(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "n"(SEL));
    return r;
}

// 8-bit integers to fp16, exactly: byte + 128 in the low bits of 1024 is 1152 more
// than the integer (a conversion by byte permutes as in Kim et al., "Who Says Elephants
// Can't Run: Bringing Large Scale MoE Models into Cloud Scale Production", 2022).
// `biased`: the word with each byte's top bit flipped; A, B: which of its bytes go to
// the low and the high half.
template <int A, int B>
__device__ __forceinline__ uint32_t int8x2_to_f16x2(uint32_t biased)
{
    const uint32_t x = bytes_of<(0x4000u | (B << 8) | 0x40u | A)>(biased, 0x64646464u);
    const uint32_t bias = 0x64806480u;                          // 1152, twice
    const __half2 h = __hsub2(*reinterpret_cast<const __half2 *>(&x), *reinterpret_cast<const __half2 *>(&bias));
    return *reinterpret_cast<const uint32_t *>(&h);
}

// Host: what an entry point has to know of a quantised cache, or what is wrong.
struct QuantisedCache {
    bool int8;
    int64_t pages, groups, block, span;
};

inline sda_status check_quantised(const sda_tensor *cache, const sda_tensor *scales, int64_t dim, QuantisedCache &q)
{
    if (!dims_ok(cache, 4) || !dims_ok(scales, 4) || scales->dtype != SDA_DTYPE_FP32)
        return SDA_ERR_INVALID;
    q.int8 = cache->dtype == SDA_DTYPE_INT8;
    if (!q.int8 && !is_fp8(cache))
        return SDA_ERR_INVALID;
    q.pages = cache->shape[0];
    q.groups = cache->shape[1];
    q.block = cache->shape[2];
    if (cache->shape[3] != 2 * dim || cache->stride[3] != 1 || q.pages < 1 || q.groups < 1 || q.block < 1)
        return SDA_ERR_INVALID;
    const int64_t parts = scales->shape[2];
    if (scales->shape[0] != q.pages || scales->shape[1] != q.groups || parts < 1 || q.block % parts != 0 ||
        scales->shape[3] != 2 || scales->stride[3] != 1)
        return SDA_ERR_INVALID;
    q.span = q.block / parts;
    if (q.span % 8 != 0 || q.pages > INT32_MAX || q.block > (1 << 24) || q.groups > (1 << 16))
        return SDA_ERR_UNSUPPORTED;
    if (!aligned(cache->data, 16) || !aligned(scales->data, 8))
        return SDA_ERR_UNSUPPORTED;
    for (int i = 0; i < 3; ++i)
        if (cache->stride[i] <= 0 || cache->stride[i] % 16 != 0 || scales->stride[i] <= 0 || scales->stride[i] % 2 != 0)
            return SDA_ERR_UNSUPPORTED;
    return SDA_OK;
}

// x / d as a product: floor(x * inverse_of(d) / 2^64) is exact for x, d < 2^32
// (d == 1 has no 64-bit inverse: 0 stands for it).
constexpr unsigned long long inverse_of(unsigned d)
{
    return d > 1 ? ~0ull / d + 1 : 0;
}

__device__ __forceinline__ uint32_t quotient(uint32_t x, unsigned long long inverse)
{
    return inverse ? static_cast<uint32_t>(__umul64hi(x, inverse)) : x;
}

}  // namespace sda
