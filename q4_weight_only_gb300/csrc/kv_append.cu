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

constexpr int kVec = 16;  // elements of one work item: eight pairs
constexpr int kMaxThreads = 512;

// Eight consecutive elements as fp32.
__device__ __forceinline__ void load8(const float *p, float (&v)[8]) {
    const float4 a = __ldg(reinterpret_cast<const float4 *>(p)), b = __ldg(reinterpret_cast<const float4 *>(p) + 1);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w;
    v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}

__device__ __forceinline__ void load8(const __nv_bfloat16 *p, float (&v)[8]) {
    const uint4 a = __ldg(reinterpret_cast<const uint4 *>(p));
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ void store8(__nv_bfloat16 *p, const float (&v)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// One CTA per row of qkv.
template <typename T>
__global__ void __launch_bounds__(kMaxThreads) kv_append_kernel(const KvAppendArgs a, const KvCacheView c,
                                                                unsigned int *err) {
    pdl_launch_dependents();
    pdl_wait();
    const int row = blockIdx.x;
    // the sequence the row belongs to: how many end at or before it
    int ended = 0;
    for (int base = 0; base < c.sequences; base += blockDim.x) {
        const int b = base + threadIdx.x;
        ended += __syncthreads_count(b < c.sequences && c.q_start[b + 1] <= row);
    }
    if (ended >= c.sequences || row < c.q_start[0]) return;  // a row of no sequence
    const int pos = c.kv_len[ended] - c.q_start[ended + 1] + row;
    const int turn = a.row_positions ? a.row_positions[row] : pos;
    const int page_index = pos >= 0 ? pos / c.page_size : -1;
    const int page = page_index >= 0 && page_index < c.table_width
                         ? c.page_table[(int64_t)ended * c.table_stride + page_index]
                         : -1;
    const bool bad_turn = turn < 0 || turn >= a.positions;
    if (bad_turn || page < 0 || page >= c.pages) {
        if (threadIdx.x == 0) atomicExch(err, kErrBadIndex);
        return;
    }
    const int off = pos - page_index * c.page_size;
    const int per_head = c.head_dim / kVec;
    const int items = (a.q_heads + 2 * c.kv_heads) * per_head;
    const int half = a.rot / 2;
    const T *src = static_cast<const T *>(a.qkv) + (int64_t)row * a.qkv_stride;
    const float *cs = a.cos_sin + (int64_t)turn * a.rot;
    for (int it = threadIdx.x; it < items; it += blockDim.x) {
        const int head = it / per_head, piece = it - head * per_head;
        const bool turned = head < a.q_heads + c.kv_heads && piece * kVec < a.rot;
        // first element of each half of the item
        int e0 = piece * kVec, e1 = e0 + 8;
        if (turned && !a.interleaved) e0 = piece * 8, e1 = half + piece * 8;
        const T *s = src + (int64_t)head * c.head_dim;
        float u[8], v[8];
        load8(s + e0, u);
        load8(s + e1, v);
        if (turned) {
            float cosv[8], sinv[8];
            load8(cs + piece * 8, cosv);
            load8(cs + half + piece * 8, sinv);
            if (a.interleaved) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float &x = i < 4 ? u[2 * i] : v[2 * i - 8], &y = i < 4 ? u[2 * i + 1] : v[2 * i - 7];
                    const float x0 = x;
                    x = x0 * cosv[i] - y * sinv[i];
                    y = y * cosv[i] + x0 * sinv[i];
                }
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float x0 = u[i];
                    u[i] = x0 * cosv[i] - v[i] * sinv[i];
                    v[i] = v[i] * cosv[i] + x0 * sinv[i];
                }
            }
        }
        __nv_bfloat16 *dst;
        if (head < a.q_heads)
            dst = a.q_out + ((int64_t)row * a.q_heads + head) * c.head_dim;
        else if (head < a.q_heads + c.kv_heads)
            dst = c.k + page * c.k_stride[0] + (head - a.q_heads) * c.k_stride[1] + off * c.k_stride[2];
        else
            dst = c.v + page * c.v_stride[0] + (head - a.q_heads - c.kv_heads) * c.v_stride[1] + off * c.v_stride[2];
        store8(dst + e0, u);
        store8(dst + e1, v);
    }
}

}  // namespace

cudaError_t launch_kv_append(const KvAppendArgs &a, const KvCacheView &c, int64_t rows, bool bf16, cudaStream_t s,
                             unsigned int *err) {
    const int items = (a.q_heads + 2 * c.kv_heads) * (c.head_dim / kVec);
    const int threads = items >= kMaxThreads ? kMaxThreads : (items + 31) / 32 * 32;
    auto *kernel = bf16 ? kv_append_kernel<__nv_bfloat16> : kv_append_kernel<float>;
    return launch_pdl(kernel, dim3((unsigned)rows), dim3(threads), 0, s, a, c, err);
}

}  // namespace q4_0
