// cache_q4.cuh -- reading a paged cache of Q4_0 blocks in the attention
// kernels: places of tokens, copies to shared memory and codes as binary16.
#pragma once

#include <cuda_fp16.h>
#include <stdint.h>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

// The cache with what divides a token's number by the page size: t /
// page_size = umulhi(t, magic) >> shift for t < 2^31.
struct CacheQ4 {
    KvQ4View c;
    uint32_t page_magic, page_shift;
    uint32_t bias;  // kNibbleBias
};

inline CacheQ4 cache_q4(const KvQ4View &c) {
    CacheQ4 r{c, 0, 0, kNibbleBias};
    // with 2^s < page_size <= 2^(s + 1), floor(t m / 2^(32 + s)) for m the next
    // whole number from 2^(32 + s) / page_size; page_size is at least 8
    while ((2 << r.page_shift) < c.page_size) ++r.page_shift;
    r.page_magic = (uint32_t)(((1ull << (32 + r.page_shift)) + c.page_size - 1) / c.page_size);
    return r;
}

// Page and slot of a token of a sequence; a page out of range is reported and
// `ok` is cleared.
struct Slot {
    int page, off;
};
__device__ __forceinline__ Slot slot_of(const CacheQ4 &c, const int32_t *table, int token, bool &ok, unsigned int *err) {
    Slot s{0, 0};
    if (!ok) return s;
    const int index = __umulhi((uint32_t)token, c.page_magic) >> c.page_shift;
    s.page = table[index], s.off = token - index * c.c.page_size;
    if (s.page < 0 || s.page >= c.c.pages) {
        report_index(err);
        ok = false;
        s = Slot{0, 0};
    }
    return s;
}

// Asynchronous copies of 16, 8 or 4 bytes; nothing is read and zeros are
// written where `bytes` is 0.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
template <int kBytes>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(kBytes), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// An arrival on `bar` once the thread's copies so far have landed (one of the
// arrivals that the barrier counts).
__device__ __forceinline__ void copy_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}
template <int kLeft>
__device__ __forceinline__ void copy_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(kLeft) : "memory");
}


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
