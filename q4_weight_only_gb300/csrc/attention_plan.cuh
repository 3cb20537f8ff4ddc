// attention_plan.cuh -- how the attention kernels share the work of a ragged
// batch, and what their host sides have in common.
//
// An item is some rows of one sequence and key head; its cost is the number of
// key tiles it sees, weighted.  Every CTA takes an equal share of all cost, in
// item order; an item that a share's boundary cuts leaves pieces that a join
// kernel adds in share order.  A kernel's parameters P hold the batch (sequence()
// below) and come with
//   items_of(p, sequence)           its items for one key head,
//   item_range(p, sequence, item)   the key tiles an item sees,
//   tile_cost(p, range)             the cost of one of them,
//   item_cost(p, sequence, item)    that of all, and
//   largest_cost(p)                 the largest tile_cost.
#pragma once

#include <cuda.h>
#include <stdint.h>

#include <mutex>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

// Flags of a CTA's record.
constexpr int kHeadPiece = 1;     // its first piece continues an item of an earlier CTA
constexpr int kHeadGoesOn = 2;    // ... which also goes on in the next CTA
constexpr int kTailPiece = 4;     // its last piece starts an item that goes on in the next CTA

// Bits 0 .. n - 1.
__device__ __forceinline__ uint32_t below(int n) {
    return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1;
}

// One sequence of the batch, clamped to what the arrays can hold.
struct Sequence {
    int row0, len, kv;  // first row of q, rows, tokens in the cache
};

template <typename P>
__device__ __forceinline__ Sequence sequence(const P &p, int b) {
    Sequence s;
    const int r0 = min(max(p.q_start[b], 0), p.rows);
    const int r1 = min(max(p.q_start[b + 1], r0), min(p.rows, r0 + p.max_q_len));
    s.row0 = r0;
    s.len = r1 - r0;
    s.kv = (int)min((int64_t)max(p.kv_len[b], 0), (int64_t)p.table_width * p.page_size);
    return s;
}

// Whether the arrays hold what the call promised of sequence b.
template <typename P>
__device__ __forceinline__ bool sequence_fits(const P &p, const Sequence &s, int b) {
    return p.q_start[b] == s.row0 && p.q_start[b + 1] == s.row0 + s.len && p.kv_len[b] == s.kv;
}

// Where a CTA's share begins.
template <int kThreads>
struct Start {
    int64_t left;  // cost from the start of the first item to the end of the share
    int head, b, item, t0;
    Sequence s;
    int64_t warp_sum[kThreads / 32];
};

__device__ __forceinline__ Sequence shuffle(const Sequence &s, int lane) {
    return Sequence{__shfl_sync(0xffffffffu, s.row0, lane), __shfl_sync(0xffffffffu, s.len, lane),
                    __shfl_sync(0xffffffffu, s.kv, lane)};
}

// Cost (for one key head) of each lane's sequence; the warp takes the items
// of a long one together.
template <typename P>
__device__ __forceinline__ int64_t sequence_cost(const P &p, const Sequence &s, int lane) {
    const int n = items_of(p, s);
    int64_t mine = n == 1 ? item_cost(p, s, 0) : 0;
    for (uint32_t many = __ballot_sync(0xffffffffu, n > 1); many; many &= many - 1) {
        const int src = __ffs(many) - 1;
        const Sequence t = shuffle(s, src);
        const int nt = items_of(p, t);
        int64_t sum = 0;
        for (int i = lane; i < nt; i += 32) sum += item_cost(p, t, i);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, d);
        if (lane == src) mine = sum;
    }
    return mine;
}

template <typename T>
__device__ __forceinline__ T warp_inclusive(T v, int lane) {
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
        const T o = __shfl_up_sync(0xffffffffu, v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// floor(all * i / n) without a product past 64 bits.
template <typename T>
__device__ __forceinline__ T share_start(T all, T n, T i) {
    const T each = all / n;
    return each * i + (all - each * n) * i / n;
}

// Where this CTA's share begins.  Called by all threads; the result is in
// `st` after the call.
template <int kThreads, typename P>
__device__ __forceinline__ void locate(const P &p, Start<kThreads> &st, int cta, int ctas) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    Sequence s;
    int64_t mine, first;  // cost of this thread's sequence, and of the ones before it
    int64_t before = 0;   // cost of earlier rounds' sequences
    // a round: one sequence a thread
    auto round = [&](int b0) {
        const int b = b0 + tid;
        s = Sequence{0, 0, 0};
        if (b < p.sequences) s = sequence(p, b);
        mine = sequence_cost(p, s, lane);
        const int64_t incl = warp_inclusive(mine, lane);
        if (lane == 31) st.warp_sum[warp] = incl;
        __syncthreads();
        int64_t sum = 0, ahead = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            const int64_t v = st.warp_sum[w];
            if (w < warp) ahead += v;
            sum += v;
        }
        __syncthreads();
        first = before + ahead + incl - mine;
        before += sum;
        return b;
    };
    for (int b0 = 0; b0 < p.sequences; b0 += kThreads) {
        const int b = round(b0);
        if (cta == 0 && b < p.sequences && !sequence_fits(p, s, b)) report_index(p.err);
    }
    const int64_t each = before, all = each * p.kv_heads;
    // A key tile belongs to the share in which it ends.  Every share but the
    // empty ones at the end has a tile (it is at least one tile's cost long):
    // an item's pieces are in consecutive CTAs.
    const int64_t n = min(max(all / largest_cost(p), (int64_t)(all > 0)), (int64_t)ctas);
    if (cta >= n) {
        if (tid == 0) st.left = 0;
        __syncthreads();
        return;
    }
    int64_t u0, u1;
    int head;
    if (all < (1ll << 31)) {
        u0 = share_start<uint32_t>((uint32_t)all, (uint32_t)n, cta);
        u1 = share_start<uint32_t>((uint32_t)all, (uint32_t)n, cta + 1);
        head = (int)((uint32_t)u0 / (uint32_t)each);
    } else {
        u0 = share_start<int64_t>(all, n, cta);
        u1 = share_start<int64_t>(all, n, cta + 1);
        head = (int)(u0 / each);
    }
    const int64_t goal = u0 - head * each;  // where the share begins within its key head
    const bool again = p.sequences > kThreads;
    before = 0;
    for (int b0 = 0; b0 < p.sequences; b0 += kThreads) {
        if (again) round(b0);
        const uint32_t hit = __ballot_sync(0xffffffffu, goal >= first && goal < first + mine);
        if (!hit) continue;
        // the warp that has the sequence looks through its items
        const int src = __ffs(hit) - 1;
        const Sequence t = shuffle(s, src);
        const int nt = items_of(p, t);
        int64_t rest = goal - __shfl_sync(0xffffffffu, first, src);
        for (int i0 = 0; i0 < nt; i0 += 32) {
            const int64_t k = i0 + lane < nt ? item_cost(p, t, i0 + lane) : 0;
            const int64_t incl = warp_inclusive(k, lane);
            if (rest >= incl - k && rest < incl) {
                const int64_t in = rest - (incl - k);
                st.head = head, st.b = b0 + warp * 32 + src, st.item = i0 + lane, st.s = t;
                st.t0 = (int)(in / tile_cost(p, item_range(p, t, i0 + lane)));
                st.left = u1 - u0 + in;
            }
            const int64_t sum = __shfl_sync(0xffffffffu, incl, 31);
            if (rest < sum) break;
            rest -= sum;
        }
    }
    __syncthreads();
}

using EncodeTiledFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *, const cuuint64_t *,
                                   const cuuint64_t *, const cuuint32_t *, const cuuint32_t *, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void *f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

int current_sms() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? device_sm_count(dev) : 0;
}

}  // namespace

}  // namespace q4_0
