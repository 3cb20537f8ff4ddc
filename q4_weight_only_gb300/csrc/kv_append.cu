// kv_append.cu -- queries and keys of fused QKV rows rotated by position,
// keys and values appended to a paged cache (declared in include/q4_0.h).
//
// Mathematics: for pair p of a head and the row's position t,
//   (a, b) -> (a cos - b sin, b cos + a sin),  cos, sin = table[t][p],
// where the pair is elements (p, p + rot/2), or (2p, 2p + 1) when
// interleaved; elements past rot and the values are copied.  One rounding,
// to bfloat16 at the store: the rotation is fp32 and the cache and the
// attention kernel hold bfloat16.
#include <cuda_bf16.h>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr int kVec = 8;  // elements of one work item: four pairs
constexpr int kThreads = 256;
constexpr int kPieceBytes = 32 * 1024;  // most of a row that one CTA holds

// Four consecutive elements as fp32.
__device__ __forceinline__ float4 load4(const float *p) { return *reinterpret_cast<const float4 *>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16 *p) {
    const uint2 a = *reinterpret_cast<const uint2 *>(p);
    return make_float4(__uint_as_float(a.x << 16), __uint_as_float(a.x & 0xFFFF0000u), __uint_as_float(a.y << 16),
                       __uint_as_float(a.y & 0xFFFF0000u));
}

// (a, b) -> (a cos - b sin, b cos + a sin)
__device__ __forceinline__ void turn(float &a, float &b, float cosv, float sinv) {
    const float a0 = a;
    a = a0 * cosv - b * sinv;
    b = b * cosv + a0 * sinv;
}

// blockIdx.x: row of qkv, blockIdx.y: piece of `heads` heads of the row.
// Bound by the read of qkv and the writes: 8191 fp32 rows of 7168 (352 MB)
// take 57 us, 6.2 TB/s, 0.91 of what a copy reaches; 8191 bf16 rows (239 MB)
// 45 us, 5.3 TB/s, half the bytes behind the same look-ups.  One bulk copy
// brings the piece to shared memory while the CTA finds the row's place in the
// cache (sequence, length, page); several CTAs an SM keep their pieces in
// flight (loads into registers, 64 bytes a thread, took 76 us).  Few rows are
// bound by latency: 16 or 272 rows take 6.3 us, 4.3 of it a launch that does
// nothing, the rest the reads for the row's place and its cosines.
template <typename T>
__global__ void __launch_bounds__(kThreads, 6) kv_append_kernel(const KvAppendArgs a, const KvCacheView c, int heads,
                                                                unsigned int *err) {
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ uint64_t full;
    __shared__ int abort_flag;
    const T *piece = reinterpret_cast<const T *>(smem);
    const int row = blockIdx.x, head0 = blockIdx.y * heads;
    const int n_heads = min(heads, a.q_heads + 2 * c.kv_heads - head0);
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
    bool ok = ended < c.sequences && row >= c.q_start[0];  // else: a row of no sequence
    int pos = 0, turn_row = 0, page = 0, off = 0;
    if (ok) {
        pos = c.kv_len[ended] - c.q_start[ended + 1] + row;
        if (a.rot) turn_row = a.row_positions ? a.row_positions[row] : pos;
        const int index = pos >= 0 ? pos / c.page_size : -1;
        page = index >= 0 && index < c.table_width ? c.page_table[(int64_t)ended * c.table_stride + index] : -1;
        off = pos - index * c.page_size;
        const bool turns = !a.rot || (turn_row >= 0 && turn_row < a.positions);
        if (!turns || page < 0 || page >= c.pages) {
            if (threadIdx.x == 0) report_index(err);
            ok = false;
        }
    }
    const bool landed = mbar_wait(&full, 0, &abort_flag, err);
    if (!ok || !landed) {
        // a wait that was given up has been reported; the copy lands first
        if (!landed) mbar_drain(&full, 0);
        return;
    }
    const float *cs = a.cos_sin + (int64_t)turn_row * a.rot;
    __nv_bfloat16 *q_row = a.q_out + (int64_t)row * a.q_heads * c.head_dim;
    __nv_bfloat16 *k_row = c.k + page * c.k_stride[0] + off * c.k_stride[2];
    __nv_bfloat16 *v_row = c.v + page * c.v_stride[0] + off * c.v_stride[2];
    const int per_head = c.head_dim / kVec, half = a.rot / 2;
    for (int it = threadIdx.x; it < n_heads * per_head; it += kThreads) {
        const int in_piece = it / per_head, i = it - in_piece * per_head, head = head0 + in_piece;
        const bool turned = head < a.q_heads + c.kv_heads && i * kVec < a.rot;
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
        __nv_bfloat16 *dst;
        const int kv_head = head - a.q_heads;
        if (kv_head < 0)
            dst = q_row + (int64_t)head * c.head_dim;
        else if (kv_head < c.kv_heads)
            dst = k_row + kv_head * c.k_stride[1];
        else
            dst = v_row + (kv_head - c.kv_heads) * c.v_stride[1];
        *reinterpret_cast<uint2 *>(dst + e0) = make_uint2(pack_bf16(u.x, u.y), pack_bf16(u.z, u.w));
        *reinterpret_cast<uint2 *>(dst + e1) = make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
    }
}

template <typename T>
cudaError_t launch_typed(const KvAppendArgs &a, const KvCacheView &c, int64_t rows, cudaStream_t s, unsigned int *err) {
    // a head is at most 4 KB (head_dim <= 1024)
    const int all = a.q_heads + 2 * c.kv_heads, fit = kPieceBytes / (c.head_dim * (int)sizeof(T));
    const int pieces = (all + fit - 1) / fit, heads = (all + pieces - 1) / pieces;
    const int smem = heads * c.head_dim * (int)sizeof(T);
    return launch_pdl(kv_append_kernel<T>, dim3((unsigned)rows, pieces), dim3(kThreads), smem, s, a, c, heads, err);
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, const KvCacheView &c, int64_t rows, bool bf16, cudaStream_t s,
                             unsigned int *err) {
    return bf16 ? launch_typed<__nv_bfloat16>(a, c, rows, s, err) : launch_typed<float>(a, c, rows, s, err);
}

}  // namespace q4_0
