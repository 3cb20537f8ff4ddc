// cache_q4.cuh -- reading a paged cache of Q4_0 blocks in the attention
// kernels: places of tokens, copies to shared memory and codes as binary16.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "attention_plan.cuh"
#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

// log2 of the unit in which a row's p, l and O are held.  p is at most 2^8 (what
// a reference lets it grow to), so 2^7 of it are 2^15 in binary16, and p is normal
// there down to 2^-21.  Without it what is below 2^-14 loses 2^-25, and below
// 2^-25 all of itself: a prompt's rows after 262144 tokens of 2^-25.6 of the
// first one's weight each, 0.5 % together, then had no weight but the first's.
constexpr float kLift = 7.f;

// A row's c with what undoes its scaling in it, within fp32's normal range: an
// infinite one, or one that underflowed to 0, would make NaN of a score that is
// 0 or masked (0 times infinity).  At the lower end every exponent is 0 either
// way: scores are below 2^40.
__device__ __forceinline__ float in_range(float c) { return fmaxf(fminf(c, 3e38f), 0x1p-126f); }

// The cache as the attention kernels take it.
struct CacheQ4 {
    KvQ4View c;
    uint32_t bias;  // kNibbleBias
};
inline CacheQ4 cache_q4(const KvQ4View &c) { return CacheQ4{c, kNibbleBias}; }

// Codes as {byte, token of the page, key head, page}, rows swizzled over their
// own length.
bool make_codes_map(EncodeTiledFn enc, CUtensorMap *map, const uint8_t *base, const int64_t (&stride)[3],
                    const KvQ4View &c, int box1) {
    const int row = c.head_dim / 2;
    const cuuint64_t dims[4] = {(cuuint64_t)row, (cuuint64_t)c.page_size, (cuuint64_t)c.kv_heads, (cuuint64_t)c.pages};
    const cuuint64_t strides[3] = {(cuuint64_t)stride[2], (cuuint64_t)stride[1], (cuuint64_t)stride[0]};
    const cuuint32_t box[4] = {(cuuint32_t)row, (cuuint32_t)box1, 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, row == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B,
               CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Asynchronous copies of 16, 8 or 4 bytes; where `skip`, nothing is read and
// zeros are written.  (A predicate, not a size of 0: the compiler makes one
// instruction of it.)
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool skip) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %2, 0;\n\t"
        "cp.async.cg.shared.global [%0], [%1], 16, p;\n\t}" ::"r"(dst),
        "l"(src), "r"((uint32_t)skip)
        : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src, bool skip) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.u32 p, %3, 0;\n\t"
        "cp.async.ca.shared.global [%0], [%1], %2, p;\n\t}" ::"r"(dst),
        "l"(src), "n"(kBytes), "r"((uint32_t)skip)
        : "memory");
}
// An arrival on `bar` once the thread's copies so far have landed (one of the
// arrivals that the barrier counts).
__device__ __forceinline__ void copy_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
// The thread's copies have landed.
__device__ __forceinline__ void copy_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

__device__ __forceinline__ uint32_t lds32(uint32_t a) {
    uint32_t v;
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
    uint2 v;
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint32_t lds16(uint32_t a) {
    uint16_t v;
    asm volatile("ld.shared.b16 %0, [%1];" : "=h"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "r"(a)
                 : "memory");
    return v;
}
__device__ __forceinline__ void sts128(uint32_t a, const uint32_t (&v)[4]) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3])
                 : "memory");
}

__device__ __forceinline__ __half2 as_half2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }
__device__ __forceinline__ uint32_t as_bits(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }

// The codes less 8 of the low nibbles of a word's bytes 0 and 2, and of their
// high nibbles, as binary16 pairs: a nibble in the mantissa of 1024 makes 1024
// + code, or 1024 + 16 code four bits higher; both steps are exact.  `bias`
// holds kNibbleBias.
__device__ __forceinline__ uint32_t low_codes(uint32_t w, uint32_t bias) {
    return as_bits(__hsub2(as_half2(and_or<0x000F000Fu>(w, bias)), __half2half2(__ushort_as_half(0x6408))));
}
__device__ __forceinline__ uint32_t high_codes(uint32_t w, uint32_t bias) {
    return as_bits(__hfma2(as_half2(and_or<0x00F000F0u>(w, bias)), __half2half2(__ushort_as_half(0x2C00)),
                           __half2half2(__ushort_as_half(0xD480))));
}
__device__ __forceinline__ uint32_t times(uint32_t a, __half2 b) { return as_bits(__hmul2(as_half2(a), b)); }

}  // namespace

}  // namespace q4_0
