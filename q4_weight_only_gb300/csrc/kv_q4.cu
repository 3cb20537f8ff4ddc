// kv_q4.cu -- a paged key and value cache in Q4_0 blocks: queries and keys of
// fused QKV rows rotated by position, keys and values quantised as they are
// appended, and tokens read back (declared in include/q4_0.h).
//
// Mathematics: a key's pair (a, b) at position t becomes
//   (a cos - b sin, b cos + a sin),  cos, sin = table[t][p],
// every product and sum rounded to fp32 by itself: the codes are discontinuous
// in their inputs, so an fma in the place of a product and a sum would give
// others here and there than any other fp32 implementation does.  A block of
// 32 elements w of a head is then
//   d = (w of the largest |w|, the first of equals) / -8,
//   code = clamp(round(w / d) + 8, 0, 15), halves away from zero,
// and 8 where d is 0 (elements of 2^-147 and less in size), with d in fp32 for
// the codes and rounded to binary16 for the cache: the
// rules of the weights' quantizer (quantize.cu), element j of a block in the
// low half of byte j, j + 16 in its high half.  A block reads back as
// d (code - 8), exactly in fp32.
//
// Bounds and measurements (40 query heads on 8 key heads of 128, device time):
// * append: 8191 fp32 rows, 330 MB read and written, take 60 us (a copy's rate:
//   50).  Every byte moves once; a row is a chain of its copy, its place, the
//   rotation and the blocks, of which six CTAs an SM hide one another's waits
//   (five, without spills: 64 us; seven: 71).  A reciprocal and a rounding
//   constant make a code in four instructions; a floor and its distance to a
//   half in each code took 69 us, a division in each 72.
// * read: the writes, at 0.94 of a copy's rate.  82 thousand rows to bfloat16,
//   430 MB read and written, take 68 us; 94 with one row's reads at a time.
// * Few rows take what two small launches do: 7 us an append with its read.
//
// This translation unit must not be built with fast-math: the codes depend on
// correctly rounded division and on roundf's tie rule.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr int kVec = 8;  // elements of one work item
constexpr int kThreads = 256;
constexpr int kPieceBytes = 32 * 1024;  // most of a row that one CTA holds
constexpr float kLargest = 65504.f;     // of an element: what binary16 holds, and what attention reads

// Division of whole numbers below 2^24 by one below 2^8: floor(a / b) =
// umulhi(a, ceil(2^32 / b)), since a b < 2^32; b = 1 has no such factor.
struct Divisor {
    uint32_t by, magic;
    explicit Divisor(int b) : by(b), magic(b == 1 ? 0 : (uint32_t)(((1ull << 32) + b - 1) / b)) {}
    __device__ __forceinline__ int operator()(int a) const { return by == 1 ? a : (int)__umulhi((uint32_t)a, magic); }
};

// Four consecutive elements as fp32.
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u), __uint_as_float(a.y << 16),
                       __uint_as_float(a.y & 0xFFFF0000u));
}

// (a, b) -> (a cos - b sin, b cos + a sin), without an fma.
__device__ __forceinline__ void turn(float &a, float &b, float cosv, float sinv) {
    const float a0 = a;
    a = __fsub_rn(__fmul_rn(a0, cosv), __fmul_rn(b, sinv));
    b = __fadd_rn(__fmul_rn(b, cosv), __fmul_rn(a0, sinv));
}

// clamp(round(w / d), -8, 7) + 8, halves away from zero; d is not 0.
__device__ __forceinline__ uint32_t code_of(float w, float d) {
    return (uint32_t)(int)(fminf(fmaxf(roundf(__fdiv_rn(w, d)), -8.f), 7.f) + 8.f);
}

// The codes of eight elements, w[0] in the lowest four bits.  q = w / d rounded
// twice, by the reciprocal and the product, is within 3 2^-24 |w / d| < 2^-19
// of the quotient that code_of rounds: they round to the same whole number
// unless q is next to a half, and then the quotients decide.
__device__ __forceinline__ uint32_t codes_of(const float (&w)[8], float d) {
    const float inv = __frcp_rn(d), base = 12582920.f;  // 1.5 2^23 + 8: whole numbers are its last bits
    uint32_t codes = 0;
    bool sure = true;
#pragma unroll
    for (int i = 7; i >= 0; --i) {
        const float q = w[i] * inv, t = __fadd_rn(q, base);
        sure &= fabsf(q - __fsub_rn(t, base)) < 0.5f - 0x1p-19f;  // (false for NaN)
        codes = codes * 16 + min(__float_as_uint(t) & 31u, 15u);
    }
    if (!sure) {
        codes = 0;
        for (int i = 7; i >= 0; --i) codes = codes * 16 + code_of(w[i], d);
    }
    return codes;
}

// The largest of three, NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// A quad of lanes (`mask`) quantises a block, lane j of it elements 4j .. 4j +
// 3 (u) and 16 + 4j .. (v), to bytes 4j .. 4j + 3 of `codes`.
__device__ __forceinline__ void quantise_quad(float4 u, float4 v, int j, uint32_t mask, uint8_t *codes,
                                              uint16_t *scale) {
    // the largest element, and the largest of their opposites
    float up = max3_nan(max3_nan(max3_nan(u.x, u.y, u.z), u.w, v.x), v.y, max3_nan(v.z, v.z, v.w));
    float down = max3_nan(max3_nan(max3_nan(-u.x, -u.y, -u.z), -u.w, -v.x), -v.y, max3_nan(-v.z, -v.z, -v.w));
#pragma unroll
    for (int d = 1; d <= 2; d <<= 1) {
        const float a = __shfl_xor_sync(mask, up, d), z = __shfl_xor_sync(mask, down, d);
        up = max3_nan(up, a, a), down = max3_nan(down, z, z);
    }
    uint32_t w = 0x88888888u;
    uint16_t s = 0;
    if (!(up <= kLargest && down <= kLargest)) {
        s = 0x7FFF;  // the block reads back as NaN
    } else if (up > 0.f || down > 0.f) {
        float value = up > down ? up : -down;
        if (up == down) {
            // elements of both signs: the first of them
            const float e[8] = {u.x, u.y, u.z, u.w, v.x, v.y, v.z, v.w};
            int first = 64;  // twice its index, and one more if it is negative
#pragma unroll
            for (int i = 7; i >= 0; --i)
                if (fabsf(e[i]) == up) first = 2 * (4 * j + (i & 3) + (i & 4) * 4) + (e[i] < 0.f);
#pragma unroll
            for (int d = 1; d <= 2; d <<= 1) first = min(first, __shfl_xor_sync(mask, first, d));
            value = first & 1 ? -up : up;
        }
        const float d = __fmul_rn(value, -0.125f);
        s = __half_as_ushort(__float2half_rn(d));
        const float e[8] = {u.x, v.x, u.y, v.y, u.z, v.z, u.w, v.w};
        if (d != 0.f) w = codes_of(e, d);
    }
    *reinterpret_cast<uint32_t *>(codes + 4 * j) = w;
    if (j == 0) *scale = s;
}

// The place of a row of the batch: its sequence's page and the token in it.
struct Place {
    int pos, page, off;
    bool in_sequence, ok;
};

__device__ __forceinline__ Place place_of(const KvQ4View &c, int row, int ended) {
    Place p{0, -1, 0, false, false};
    p.in_sequence = ended < c.sequences && row >= c.q_start[0];
    if (!p.in_sequence) return p;
    p.pos = c.kv_len[ended] - c.q_start[ended + 1] + row;
    const int index = p.pos >= 0 ? p.pos / c.page_size : -1;
    p.page = index >= 0 && index < c.table_width ? c.page_table[(int64_t)ended * c.table_stride + index] : -1;
    p.off = p.pos - index * c.page_size;
    p.ok = p.page >= 0 && p.page < c.pages;
    return p;
}

// blockIdx.x: row of qkv, blockIdx.y: piece of `heads` heads of the row.  One
// bulk copy brings the piece to shared memory while the CTA finds the row's
// place in the cache.  Queries are rotated to q_out, keys in shared memory
// (in the piece itself for fp32, beside it for bfloat16), and four lanes then
// quantise a block.
template <typename T>
__global__ void __launch_bounds__(kThreads, 6)
    kv_append_q4_kernel(const KvAppendArgs a, const KvQ4View c, int heads, Divisor per_head, Divisor blocks,
                        unsigned int *err) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full;
    __shared__ int abort_flag;
    constexpr bool kInPlace = sizeof(T) == 4;
    T *piece = reinterpret_cast<T *>(smem);
    const int row = blockIdx.x, head0 = blockIdx.y * heads;
    const int n_heads = min(heads, a.q_heads + 2 * c.kv_heads - head0);
    // keys [key0, value0) and values [value0, n_heads) of the piece
    const int key0 = min(max(a.q_heads - head0, 0), n_heads);
    const int value0 = min(max(a.q_heads + c.kv_heads - head0, 0), n_heads);
    // keys in fp32, by the head's number in the piece
    float *keys = kInPlace ? reinterpret_cast<float *>(smem)
                           : reinterpret_cast<float *>(smem + heads * c.head_dim * sizeof(T)) - key0 * c.head_dim;
    if (threadIdx.x == 0) {
        mbar_init(&full, 1);
        abort_flag = 0;
        mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    if (threadIdx.x == 0) {
        const uint32_t bytes = (uint32_t)(n_heads * c.head_dim * sizeof(T));
        mbar_arrive_expect_tx(&full, bytes);
        bulk_g2s(smem, static_cast<const T *>(a.qkv) + (int64_t)row * a.qkv_stride + (int64_t)head0 * c.head_dim, bytes,
                 &full);
    }
    // the sequence the row belongs to: how many end at or before it
    int ended = 0;
    for (int base = 0; base < c.sequences; base += kThreads) {
        const int b = base + threadIdx.x;
        ended += __syncthreads_count(b < c.sequences && c.q_start[b + 1] <= row);
    }
    const Place place = place_of(c, row, ended);
    bool ok = place.ok;
    int turn_row = 0;
    if (place.in_sequence) {
        if (a.rot) turn_row = a.row_positions ? a.row_positions[row] : place.pos;
        if (a.rot && (turn_row < 0 || turn_row >= a.positions)) ok = false;
        if (!ok && threadIdx.x == 0) report_index(err);
    }
    const bool landed = mbar_wait(&full, 0, &abort_flag, err);
    // (every thread waits for the same barrier, but gives up by itself)
    if (!__syncthreads_and(ok && landed)) {
        // a wait that was given up has been reported; the copy lands first
        if (!landed) mbar_drain(&full, 0);
        return;
    }
    const float *cs = a.cos_sin + (int64_t)turn_row * a.rot;
    __nv_bfloat16 *q_row = a.q_out + (int64_t)row * a.q_heads * c.head_dim;
    const int items = c.head_dim / kVec, half = a.rot / 2;  // of a head
    for (int it = threadIdx.x; it < value0 * items; it += kThreads) {
        const int in_piece = per_head(it), i = it - in_piece * items;
        const bool turned = i * kVec < a.rot, query = in_piece < key0;
        if (kInPlace && !turned && !query) continue;
        // first elements of the item's two halves
        int e0 = i * kVec, e1 = e0 + 4;
        if (turned && !a.interleaved) e0 = i * 4, e1 = half + i * 4;
        const T *s = piece + in_piece * c.head_dim;
        float4 u = load4(s + e0), v = load4(s + e1);
        if (turned) {
            const float4 cosv = load4(cs + i * 4), sinv = load4(cs + half + i * 4);
            if (a.interleaved) {
                turn(u.x, u.y, cosv.x, sinv.x), turn(u.z, u.w, cosv.y, sinv.y);
                turn(v.x, v.y, cosv.z, sinv.z), turn(v.z, v.w, cosv.w, sinv.w);
            } else {
                turn(u.x, v.x, cosv.x, sinv.x), turn(u.y, v.y, cosv.y, sinv.y);
                turn(u.z, v.z, cosv.z, sinv.z), turn(u.w, v.w, cosv.w, sinv.w);
            }
        }
        if (query) {
            __nv_bfloat16 *dst = q_row + (int64_t)(head0 + in_piece) * c.head_dim;
            *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w));
            *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
        } else {
            float *dst = keys + in_piece * c.head_dim;
            *reinterpret_cast<float4 *>(dst + e0) = u;
            *reinterpret_cast<float4 *>(dst + e1) = v;
        }
    }
    if (key0 == n_heads) return;
    __syncthreads();
    const int j = threadIdx.x & 3, per_token = c.head_dim / 32;
    const uint32_t quad = 15u << (threadIdx.x & 28);
    for (int it = threadIdx.x >> 2; it < (n_heads - key0) * per_token; it += kThreads / 4) {
        const int of = blocks(it), in_piece = key0 + of, block = it - of * per_token, e = block * 32 + 4 * j;
        const bool key = in_piece < value0;
        float4 u, v;
        if (key) {
            u = load4(keys + in_piece * c.head_dim + e), v = load4(keys + in_piece * c.head_dim + e + 16);
        } else {
            u = load4(piece + in_piece * c.head_dim + e), v = load4(piece + in_piece * c.head_dim + e + 16);
        }
        const int head = head0 + in_piece - a.q_heads - (key ? 0 : c.kv_heads);
        const int64_t *st = key ? c.k_stride : c.v_stride, *ss = key ? c.k_scale_stride : c.v_scale_stride;
        uint8_t *codes = (key ? c.k : c.v) + place.page * st[0] + head * st[1] + place.off * st[2] + block * 16;
        uint16_t *scale = (key ? c.k_scale : c.v_scale) + place.page * ss[0] + head * ss[1] + place.off * ss[2] + block;
        quantise_quad(u, v, j, quad, codes, scale);
    }
}

template <typename T>
cudaError_t launch_append(const KvAppendArgs &a, const KvQ4View &c, int64_t rows, cudaStream_t s, unsigned int *err) {
    // a head is at most 4 KB (head_dim <= 1024)
    const int all = a.q_heads + 2 * c.kv_heads, fit = kPieceBytes / (c.head_dim * (int)sizeof(T));
    const int pieces = (all + fit - 1) / fit, heads = (all + pieces - 1) / pieces;
    int smem = heads * c.head_dim * (int)sizeof(T);
    if (sizeof(T) == 2) smem += (heads < c.kv_heads ? heads : c.kv_heads) * c.head_dim * 4;
    // past 48 KB, the kernel's own variables among them, a launch has to ask
    if (smem > 47 * 1024) {
        const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(kv_append_q4_kernel<T>), smem);
        if (e != cudaSuccess) return e;
    }
    return launch_pdl(kv_append_q4_kernel<T>, dim3((unsigned)rows, pieces), dim3(kThreads), smem, s, a, c, heads,
                      Divisor(c.head_dim / kVec), Divisor(c.head_dim / 32), err);
}

// What the four bytes of `w`, codes, stand for: a byte in the upper mantissa of
// 2^23 is 2^16 (128 + code), and (128 + code) d - 136 d is exact.
__device__ __forceinline__ float4 values4(uint32_t w, float d) {
    const float unit = d * 0x1p-16f, less = -136.f * d;
    auto value = [&](uint32_t sel) { return fmaf(__uint_as_float(__byte_perm(w, 0x4B000000u, sel)), unit, less); };
    return make_float4(value(0x7044), value(0x7144), value(0x7244), value(0x7344));
}

__device__ __forceinline__ void store8(float *p, float4 a, float4 b) {
    *reinterpret_cast<float4 *>(p) = a;
    *reinterpret_cast<float4 *>(p + 4) = b;
}
__device__ __forceinline__ void store8(__nv_bfloat16 *p, float4 a, float4 b) {
    *reinterpret_cast<uint4 *>(p) =
        make_uint4(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w), pack_bf16(b.x, b.y), pack_bf16(b.z, b.w));
}

// Rows of a CTA, of whose places each warp finds one or two: 16 where there are
// enough of them to fill the SMs.  With 8 and with 16 rows, to bfloat16, us:
//   rows           515         4096        16384        32768        65536
//   8 x 128     3.7, 5.2     6.5, 7.3   17.0, 18.4   30.3, 30.5   56.9, 55.3
//   4 x 64      2.9, 3.6     4.2, 4.4    9.5, 8.0    18.3, 14.5   34.1, 26.1
//   32 x 128    7.0, 11.8   18.6, 21.7  55.3, 61.3  104.9, 107.9
// The two cross between 5 thousand rows (small ones) and 50 thousand.
constexpr int kReadRows = 8, kMostReadRows = 16, kManyRows = 16384;

// blockIdx.x: `per_cta` rows of the batch.  A thread reads half a block (8
// bytes of codes) of every few rows and writes its 16 values: `width` threads
// have a row at once (a row's half blocks, kThreads at most).  Bound by the
// writes.
template <typename T>
__global__ void __launch_bounds__(kThreads) kv_read_q4_kernel(const KvQ4View c, int rows, int per_cta, int width,
                                                              T *k_out, T *v_out, unsigned int *err) {
    __shared__ int2 at[kMostReadRows];  // page (-1: none) and token of each row
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = blockIdx.x * per_cta;
    for (int r = warp; r < per_cta; r += kThreads / 32) {
        const int row = row0 + r;
        int ended = 0;
        for (int base = 0; base < c.sequences; base += 32) {
            const int b = base + lane;
            ended += __popc(__ballot_sync(0xffffffffu, b < c.sequences && c.q_start[b + 1] <= row));
        }
        if (lane == 0) {
            const Place p = row < rows ? place_of(c, row, ended) : Place{};
            if (p.in_sequence && !p.ok) report_index(err);
            at[r] = make_int2(p.ok ? p.page : -1, p.off);
        }
    }
    __syncthreads();
    const int halves = c.head_dim / 16, per_side = c.kv_heads * halves;
    const int at_once = kThreads / width, first = threadIdx.x / width;
    if (first >= at_once) return;
    for (int i = threadIdx.x - first * width; i < 2 * per_side; i += width) {
        const bool key = i < per_side;
        const int in_side = key ? i : i - per_side, head = in_side / halves, h = in_side - head * halves;
        const int64_t *st = key ? c.k_stride : c.v_stride, *ss = key ? c.k_scale_stride : c.v_scale_stride;
        const uint8_t *codes = (key ? c.k : c.v) + head * st[1] + h * 8;
        const uint16_t *scales = (key ? c.k_scale : c.v_scale) + head * ss[1] + (h >> 1);
        T *out = (key ? k_out : v_out) + ((int64_t)row0 * c.kv_heads + head) * c.head_dim + (h >> 1) * 32 + (h & 1) * 8;
        const int row_step = c.kv_heads * c.head_dim;
        // several rows' reads are under way at once
        constexpr int kAtOnce = 4;
        for (int r0 = first; r0 < per_cta; r0 += kAtOnce * at_once) {
            uint2 w[kAtOnce];
            uint16_t d[kAtOnce];
            bool ok[kAtOnce];
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                const int r = r0 + x * at_once;
                const int2 place = r < per_cta ? at[r] : make_int2(-1, 0);
                ok[x] = place.x >= 0;
                if (!ok[x]) continue;
                // (32 by 64 bits: two instructions a product)
                const uint64_t page = (uint32_t)place.x, off = (uint32_t)place.y;
                w[x] = *reinterpret_cast<const uint2 *>(codes + page * st[0] + off * st[2]);
                d[x] = scales[page * ss[0] + off * ss[2]];
            }
#pragma unroll
            for (int x = 0; x < kAtOnce; ++x) {
                if (!ok[x]) continue;
                const float f = __half2float(__ushort_as_half(d[x]));
                T *dst = out + (int64_t)(r0 + x * at_once) * row_step;
                const uint32_t low = 0x0F0F0F0Fu;
                store8(dst, values4(w[x].x & low, f), values4(w[x].y & low, f));
                store8(dst + 16, values4(w[x].x >> 4 & low, f), values4(w[x].y >> 4 & low, f));
            }
        }
    }
}

}  // namespace

cudaError_t launch_kv_append_q4(const KvAppendArgs &a, const KvQ4View &c, int64_t rows, bool bf16, cudaStream_t s,
                                unsigned int *err) {
    return bf16 ? launch_append<__nv_bfloat16>(a, c, rows, s, err) : launch_append<float>(a, c, rows, s, err);
}

cudaError_t launch_kv_read_q4(const KvQ4View &c, int64_t rows, void *k_out, void *v_out, bool bf16, cudaStream_t s,
                              unsigned int *err) {
    const int per_cta = rows < kManyRows ? kReadRows : kMostReadRows;
    const dim3 grid((unsigned)((rows + per_cta - 1) / per_cta));
    const int halves = 2 * c.kv_heads * (c.head_dim / 16), width = halves < kThreads ? halves : kThreads;
    if (bf16)
        return launch_pdl(kv_read_q4_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, s, c, (int)rows, per_cta, width,
                          static_cast<__nv_bfloat16 *>(k_out), static_cast<__nv_bfloat16 *>(v_out), err);
    return launch_pdl(kv_read_q4_kernel<float>, grid, dim3(kThreads), 0, s, c, (int)rows, per_cta, width,
                      static_cast<float *>(k_out), static_cast<float *>(v_out), err);
}

}  // namespace q4_0
