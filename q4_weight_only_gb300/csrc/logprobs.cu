// logprobs.cu -- log probability of a given token per row of logits, with
// the row's entropy and its top alternatives (declared in include/q4_0.h).
//
// Mathematics, over one read of a row x: with a running maximum m,
//   s = sum e^(x - m),   t = sum (x - m) e^(x - m),
// both rescaled when m grows (t also shifts: t + (m_old - m_new) s), so
//   lse = m + ln s,   logprob = x[token] - lse,   entropy = ln s - t / s.
// All statistics are fp32.  Ranking uses 64-bit keys (order-preserving bits
// of x, then the complement of the index), so equal logits rank by lowest
// index whatever order threads meet them in.
//
// Top alternatives in the same read: a block keeps a threshold key, known to
// be at most the row's k-th largest, and appends only larger keys to a
// buffer.  The threshold starts as the k-th largest of the per-thread best
// keys of the first chunk (k keys at or above it exist), and is raised the
// same way, with the buffer cut to its k largest, when the buffer could
// overflow: at most k threads of a chunk then hold candidates, 16 each, so
// the buffer never overflows, for any order of the logits.
#include <cuda_bf16.h>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 16;                     // logits of one thread in a chunk
constexpr int kChunk = kThreads * kPerThread;
constexpr int kBuffer = 1024;                      // candidate keys a block holds
constexpr int kMaxTop = 32;                        // one list of alternatives per warp
constexpr float kLog2e = 1.4426950408889634f;
static_assert(kMaxTop * kPerThread + kMaxTop <= kBuffer, "a raised threshold must leave room for a chunk");

using Key = unsigned long long;  // 0: none

__device__ __forceinline__ Key make_key(float x, uint32_t index) {
    x += 0.f;  // -0 ranks as +0
    uint32_t b = __float_as_uint(x);
    b = x != x ? 0xFFFFFFFFu : b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);  // NaN ranks first
    return (Key)b << 32 | (0xFFFFFFFFu - index);
}

__device__ __forceinline__ float key_value(Key k) {
    const uint32_t b = (uint32_t)(k >> 32);
    return b == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u)
                            : __uint_as_float(b ^ ((b >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

__device__ __forceinline__ uint32_t key_index(Key k) { return 0xFFFFFFFFu - (uint32_t)k; }

// Largest of a and b; NaN if either is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// ----------------------------------------------------------- sorted lists

// A bitonic sequence over the warp, one key per lane, into descending order.
__device__ __forceinline__ Key warp_merge_desc(Key k, int lane) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        const Key o = __shfl_xor_sync(0xffffffffu, k, d);
        const bool keep_max = (lane & d) == 0;
        k = (k > o) == keep_max ? k : o;
    }
    return k;
}

// Any 32 keys into descending order.
__device__ __forceinline__ Key warp_sort_desc(Key k, int lane) {
#pragma unroll
    for (int n = 2; n <= 32; n <<= 1) {
#pragma unroll
        for (int d = n >> 1; d >= 1; d >>= 1) {
            const Key o = __shfl_xor_sync(0xffffffffu, k, d);
            const bool keep_max = ((lane & d) == 0) == ((lane & n) == 0);
            k = (k > o) == keep_max ? k : o;
        }
    }
    return k;
}

// The 32 largest of two descending lists, descending.  `reversed` holds the
// second list with lane l carrying its element 31 - l.
__device__ __forceinline__ Key warp_top_of_two(Key a, Key reversed, int lane) {
    return warp_merge_desc(a > reversed ? a : reversed, lane);
}

struct Shared {
    Key buffer[kBuffer];
    Key lists[kWarps][kMaxTop];
    float m[kWarps], s[kWarps], t[kWarps];
    int count;
};

// The block's 32 largest keys from one descending list per warp; the result
// is in sh.lists[0] after the call (which starts and ends with a barrier).
__device__ __forceinline__ void block_top(Shared &sh, Key mine, int warp, int lane) {
    __syncthreads();
    sh.lists[warp][lane] = mine;
#pragma unroll
    for (int step = kWarps / 2; step >= 1; step >>= 1) {
        __syncthreads();
        if (warp < step) {
            mine = warp_top_of_two(mine, sh.lists[warp + step][31 - lane], lane);
            sh.lists[warp][lane] = mine;
        }
    }
    __syncthreads();
}

// One descending list per warp of n buffered keys (n <= kBuffer).
__device__ __forceinline__ Key warp_list(const Key *buffer, int n, int warp, int lane) {
    constexpr int kOwn = kBuffer / kWarps;
    static_assert(kOwn % 32 == 0, "");
    Key mine = 0;
    // entries are dealt to the warps 32 at a time
#pragma unroll
    for (int j = 0; j < kOwn / 32; ++j) {
        const int i = (j * kWarps + warp) * 32;
        if (i >= n) break;
        const Key k = warp_sort_desc(i + lane < n ? buffer[i + lane] : 0, lane);
        mine = j == 0 ? k : warp_top_of_two(mine, __shfl_xor_sync(0xffffffffu, k, 31), lane);
    }
    return mine;
}

// ------------------------------------------------------------- statistics

struct Stats {
    float m, s, t;
};

__device__ __forceinline__ Stats join(const Stats &a, const Stats &b) {
    Stats r;
    r.m = fmaxf(a.m, b.m);
    const float base = r.m == -INFINITY ? 0.f : r.m;
    // a side without any finite logit has s = t = 0, and its shift is cut off
    const float da = fmaxf(a.m - base, -1e30f), db = fmaxf(b.m - base, -1e30f);
    const float fa = ex2(da * kLog2e), fb = ex2(db * kLog2e);
    r.s = a.s * fa + b.s * fb;
    r.t = (a.t + da * a.s) * fa + (b.t + db * b.s) * fb;
    return r;
}

// The block's statistics from each thread's, in every thread of warp 0.
__device__ __forceinline__ Stats block_join(Shared &sh, Stats v, int warp, int lane) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1)
        v = join(v, Stats{__shfl_xor_sync(0xffffffffu, v.m, d), __shfl_xor_sync(0xffffffffu, v.s, d),
                          __shfl_xor_sync(0xffffffffu, v.t, d)});
    if (lane == 0) sh.m[warp] = v.m, sh.s[warp] = v.s, sh.t[warp] = v.t;
    __syncthreads();
    if (warp == 0) {
        const int w = lane < kWarps ? lane : 0;
        v = Stats{lane < kWarps ? sh.m[w] : -INFINITY, lane < kWarps ? sh.s[w] : 0.f, lane < kWarps ? sh.t[w] : 0.f};
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1)
            v = join(v, Stats{__shfl_xor_sync(0xffffffffu, v.m, d), __shfl_xor_sync(0xffffffffu, v.s, d),
                              __shfl_xor_sync(0xffffffffu, v.t, d)});
    }
    return v;
}

template <typename T>
__device__ __forceinline__ float to_float(T v) {
    return static_cast<float>(v);
}
template <>
__device__ __forceinline__ float to_float(__nv_bfloat16 v) {
    return __bfloat162float(v);
}

// Results of one row, written by warp 0 (lane l has the l-th largest key).
template <typename T>
__device__ __forceinline__ void finish_row(const LogprobArgs &a, int row, Stats v, Key best, int lane,
                                           unsigned int *err) {
    const bool empty = v.m == -INFINITY && v.s == 0.f;  // every logit is -inf
    const float ln_s = logf(v.s);
    const float lse = empty ? -INFINITY : v.m + ln_s;
    if (lane == 0) {
        float lp = 0.f;
        if (a.tokens) {
            const int64_t token = a.tokens[row];
            if (token >= a.vocab) {
                atomicExch(err, kErrBadIndex);
                lp = __uint_as_float(0x7FC00000u);
            } else if (token >= 0) {
                const float x = to_float(static_cast<const T *>(a.logits)[(int64_t)row * a.row_stride + token]);
                lp = empty ? -INFINITY : x - lse;
            }
            a.logprob[row] = lp;
        }
        const float h = ln_s - v.t / v.s;
        a.entropy[row] = empty ? 0.f : (h < 0.f ? 0.f : h);
    }
    if (lane < a.top) {
        const int64_t o = (int64_t)row * a.top + lane;
        a.top_logprob[o] = empty ? -INFINITY : key_value(best) - lse;
        a.top_ids[o] = key_index(best);
    }
}

// ------------------------------------------------------------------ loads

// kPerThread logits of one thread: 16-byte vectors, kThreads vectors apart.
// `p` is 16-byte aligned and element 0 of it has index `first`; elements
// outside [lo, hi) read as -inf.
template <typename T>
__device__ __forceinline__ void load_chunk(const T *p, int first, int lo, int hi, int tid, float (&x)[kPerThread]) {
    constexpr int kV = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < kPerThread / kV; ++j) {
        const int o = (j * kThreads + tid) * kV, i = first + o;
        float *d = x + j * kV;
        if (i >= lo && i + kV <= hi) {
            const uint4 w = __ldcs(reinterpret_cast<const uint4 *>(p + o));
            const uint32_t r[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                if constexpr (sizeof(T) == 4) {
                    d[e] = __uint_as_float(r[e]);
                } else {
                    d[2 * e] = __uint_as_float(r[e] << 16);
                    d[2 * e + 1] = __uint_as_float(r[e] & 0xFFFF0000u);
                }
            }
        } else {
#pragma unroll
            for (int e = 0; e < kV; ++e) d[e] = i + e >= lo && i + e < hi ? to_float(p[o + e]) : -INFINITY;
        }
    }
}

// Index (within the chunk) of a thread's e-th logit.
template <typename T>
__device__ __forceinline__ int chunk_index(int e, int tid) {
    constexpr int kV = 16 / sizeof(T);
    return (e / kV * kThreads + tid) * kV + e % kV;
}

// Partial results of a row's split: statistics, then the keys.
struct Partial {
    float m, s, t, unused;
    Key keys[kMaxTop];
};

// blockIdx.y: row, blockIdx.x: split of the row.
template <typename T>
__global__ void __launch_bounds__(kThreads, 2) token_logprobs_kernel(const LogprobArgs a, Partial *part, int span,
                                                                     unsigned int *err) {
    __shared__ Shared sh;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int row = blockIdx.y;
    const T *x0 = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride;
    const int lo = blockIdx.x * span, hi = min(a.vocab, lo + span);
    // start the vectors on a 16-byte boundary at or before the first logit
    const int skew = (int)((reinterpret_cast<uintptr_t>(x0 + lo) & 15u) / sizeof(T));
    if (tid == 0) sh.count = 0;

    Stats st{-INFINITY, 0.f, 0.f};
    Key limit = 0;                // candidates are keys above it
    float limit_x = -INFINITY;    // its value
    bool seeded = false;          // false: everything is a candidate
    int bound = 0;                // at least sh.count, the same in every thread

    float x[kPerThread], next[kPerThread];
    load_chunk<T>(x0 + lo - skew, lo - skew, lo, hi, tid, x);
    for (int first = lo - skew; first < hi; first += kChunk) {
        if (first + kChunk < hi) load_chunk<T>(x0 + first + kChunk, first + kChunk, lo, hi, tid, next);
        float top = x[0], top_n = x[0];
#pragma unroll
        for (int e = 1; e < kPerThread; ++e) top = fmaxf(top, x[e]), top_n = max_nan(top_n, x[e]);
        if (top > st.m) {
            const float d = fmaxf(st.m - top, -1e30f), f = ex2(d * kLog2e);
            st.t = (st.t + d * st.s) * f;
            st.s *= f;
            st.m = top;
        }
        const float base = st.m == -INFINITY ? 0.f : st.m;
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) {
            const float d = max_nan(x[e] - base, -1e30f);  // -inf: cut off, so that d * 0 is 0
            const float p = ex2(d * kLog2e);
            st.s += p;
            st.t = fmaf(d, p, st.t);
        }
        if (a.top > 0) {
            const bool any = !seeded || !(top_n <= limit_x);
            int hits = __syncthreads_count(any);
            if (hits && bound + hits * kPerThread > kBuffer) {
                bound = sh.count;
                __syncthreads();
                if (bound + hits * kPerThread > kBuffer) {
                    // cut the buffer to its 32 largest, then raise the
                    // threshold to the top-th largest of the threads' best keys
                    if (bound > kMaxTop) {
                        block_top(sh, warp_list(sh.buffer, bound, warp, lane), warp, lane);
                        if (tid < kMaxTop) sh.buffer[tid] = sh.lists[0][tid];
                        bound = kMaxTop;
                        if (tid == 0) sh.count = kMaxTop;
                        const Key k = sh.lists[0][a.top - 1];
                        if (k > limit) limit = k;
                    }
                    Key mine = 0;
#pragma unroll
                    for (int e = 0; e < kPerThread; ++e) {
                        const int i = first + chunk_index<T>(e, tid);
                        const Key k = make_key(x[e], i);
                        if (i >= lo && i < hi && k > mine) mine = k;
                    }
                    block_top(sh, warp_sort_desc(mine, lane), warp, lane);
                    const Key k = sh.lists[0][a.top - 1];
                    // keys equal to the new threshold stay candidates
                    if (k > 0 && k - 1 > limit) limit = k - 1;
                    limit_x = limit ? key_value(limit) : -INFINITY;
                    if (limit && limit_x != limit_x) limit_x = INFINITY;
                    seeded = limit != 0;
                    hits = kMaxTop;
                    __syncthreads();
                }
            }
            if (any) {
#pragma unroll
                for (int e = 0; e < kPerThread; ++e) {
                    const int i = first + chunk_index<T>(e, tid);
                    if (seeded && x[e] < limit_x) continue;
                    const Key k = make_key(x[e], i);
                    if (i >= lo && i < hi && k > limit) sh.buffer[atomicAdd(&sh.count, 1)] = k;
                }
            }
            bound += hits * kPerThread;
        }
#pragma unroll
        for (int e = 0; e < kPerThread; ++e) x[e] = next[e];
    }
    Key best = 0;
    if (a.top > 0) {
        __syncthreads();
        block_top(sh, warp_list(sh.buffer, sh.count, warp, lane), warp, lane);
        if (warp == 0) best = sh.lists[0][lane];
    }
    st = block_join(sh, st, warp, lane);
    if (warp != 0) return;
    if (gridDim.x == 1) {
        finish_row<T>(a, row, st, best, lane, err);
    } else {
        Partial &o = part[(int64_t)row * gridDim.x + blockIdx.x];
        if (lane == 0) o.m = st.m, o.s = st.s, o.t = st.t;
        o.keys[lane] = best;
    }
}

// Joins the splits of a row, in split order.  One CTA per row.
template <typename T>
__global__ void __launch_bounds__(kThreads) logprobs_join_kernel(const LogprobArgs a, const Partial *part, int splits,
                                                                 unsigned int *err) {
    __shared__ Shared sh;
    pdl_launch_dependents();
    pdl_wait();
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, row = blockIdx.x;
    const Partial *p = part + (int64_t)row * splits;
    Key best = 0;
    if (a.top > 0) {
        for (int i = warp; i < splits; i += kWarps)  // descending lists already
            best = warp_top_of_two(best, p[i].keys[31 - lane], lane);
        block_top(sh, best, warp, lane);
        best = sh.lists[0][lane];
    }
    Stats st{-INFINITY, 0.f, 0.f};
    for (int i = tid; i < splits; i += kThreads) st = join(st, Stats{p[i].m, p[i].s, p[i].t});
    st = block_join(sh, st, warp, lane);
    if (warp == 0) finish_row<T>(a, row, st, best, lane, err);
}

// Splits of a row: enough CTAs for two per SM, none with less than
// kMinSpan logits.
constexpr int kMinSpan = 2048;

int logprob_splits(int rows, int vocab, int sms) {
    const int64_t want = (2 * (int64_t)sms + rows - 1) / rows;
    const int64_t most = (vocab + kMinSpan - 1) / kMinSpan;
    const int64_t s = want < most ? want : most;
    return rows >= sms || s < 2 ? 1 : (int)s;
}

int current_sms() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? device_sm_count(dev) : 0;
}

template <typename T>
cudaError_t launch_typed(const LogprobArgs &a, void *workspace, cudaStream_t s, unsigned int *err) {
    int splits = logprob_splits(a.rows, a.vocab, current_sms());
    // a span of whole 128-byte lines
    const int span = ((a.vocab + splits - 1) / splits + 63) / 64 * 64;
    splits = (a.vocab + span - 1) / span;
    Partial *part = static_cast<Partial *>(workspace);
    for (int r0 = 0; r0 < a.rows; r0 += 65535) {  // the rows are a grid dimension
        LogprobArgs b = a;
        b.rows = a.rows - r0 < 65535 ? a.rows - r0 : 65535;
        b.logits = static_cast<const T *>(a.logits) + (int64_t)r0 * a.row_stride;
        if (a.tokens) b.tokens = a.tokens + r0, b.logprob = a.logprob + r0;
        b.entropy = a.entropy + r0;
        if (a.top) b.top_logprob = a.top_logprob + (int64_t)r0 * a.top, b.top_ids = a.top_ids + (int64_t)r0 * a.top;
        cudaError_t e = launch_pdl(token_logprobs_kernel<T>, dim3(splits, b.rows), dim3(kThreads), 0, s, b, part, span,
                                   err);
        if (e != cudaSuccess) return e;
        if (splits > 1) {
            e = launch_pdl(logprobs_join_kernel<T>, dim3(b.rows), dim3(kThreads), 0, s, b, (const Partial *)part,
                           splits, err);
            if (e != cudaSuccess) return e;
        }
    }
    return cudaSuccess;
}

}  // namespace

size_t token_logprobs_workspace_bytes(int rows, int vocab, int /*top*/) {
    const int splits = logprob_splits(rows, vocab, current_sms());
    return splits > 1 ? ((size_t)rows * splits * sizeof(Partial) + 255) / 256 * 256 : 0;
}

cudaError_t launch_token_logprobs(const LogprobArgs &a, bool bf16, void *workspace, cudaStream_t s,
                                  unsigned int *err) {
    return bf16 ? launch_typed<__nv_bfloat16>(a, workspace, s, err) : launch_typed<float>(a, workspace, s, err);
}

}  // namespace q4_0
