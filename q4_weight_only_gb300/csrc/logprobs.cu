// logprobs.cu -- log probability of a given token per row of logits, with
// the row's entropy and its top alternatives (declared in include/q4_0.h).
//
// Mathematics, over one read of a row x: with a running maximum m and, in
// base 2, y = (x - m) log2 e,
//   s = sum 2^y,   t = sum y 2^y,
// both rescaled when m grows (t also shifts by (m_old - m_new) log2 e s),
//   logprob = (x[token] - m) - ln s,  entropy = (log2 s - t / s) ln 2.
// m is subtracted before the product with log2 e: the largest logit has y = 0
// exactly, s >= 1, no log probability is above 0, and an error does not grow
// with an offset of the row.  (x log2 e - (m log2 e) as one fma has the
// rounding of m's product in every y, whole exponents from 1e9 on; it took 2
// of the 201 us below less.)  All statistics are fp32.  Ranking uses 64-bit
// keys (order-preserving bits of x, then the complement of the index), so
// equal logits rank by lowest index whatever order threads meet them in.
//
// Top alternatives in the same read: every warp keeps a threshold key, below
// the row's k-th largest, and appends only larger keys to a buffer of its
// own.  The threshold starts below the k-th largest of the block's per-thread
// best keys of the first chunk (k keys at or above that one exist); a warp
// whose buffer is full cuts it to its 32 largest and raises its threshold to
// the k-th of them, so any order of the logits is handled.  Warps meet only
// at the first chunk and the end of a row: with a barrier a chunk, each
// waited for the one warp that had found candidates.  Code that runs for the
// few candidates is kept short (unrolled over a thread's 16 logits, each of
// its rare runs waited a microsecond for instructions) and takes the logits
// of two such threads at a time, a lane each (one at a time: 217 us below).
//
// Bound by the one read of the logits: chunks of 8192 logits stream through
// a ring of bulk copies (96 KB in flight a block, two blocks an SM) that
// runs on over the ends of rows.  Where there are few rows a cluster of up to
// eight blocks shares one, and the first of them joins what the others leave
// in its shared memory: a second kernel for that, with its workspace, made
// one row of 32000 take 12.5 us, for 10.4.  Measured: 2048 fp32 rows of
// 131072 take 201 us with 20 alternatives (5.3 TB/s) and 154 us with none
// (7.0 TB/s, what a copy reaches).  bf16 rows of the same length are bound by
// their instructions, 20 a logit with 20 alternatives and 12 with none: 201
// and 124 us, where their bytes would take 79.  16 bf16 rows of
// 128257 take 14.6 us, most of it launch, first chunks and the end of the row.
#include <cuda_bf16.h>

#include <type_traits>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr int kThreads = 512;                       // that take logits; one more warp copies
constexpr int kWarps = kThreads / 32;
constexpr int kPerThread = 16;                     // logits of one thread in a chunk
constexpr int kChunk = kThreads * kPerThread;
constexpr int kMaxTop = 32;                        // one key a lane
constexpr int kBuffer = 2 * kMaxTop;               // candidate keys a warp holds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kFloor = -1000.f;                  // 2^kFloor is 0, and kFloor * 0 is too
constexpr float kFar = 1e37f;                      // beyond it (x - m) log2 e may overflow
constexpr int kRingBytes = 96 * 1024;
constexpr int kMaxCluster = 8;                     // blocks that share a row

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

// Largest; NaN if one is.
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b, float c) {
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}
__device__ __forceinline__ float min3(float a, float b, float c) {
    float r;
    asm("min.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// The float at or below which a logit is no candidate: the value of the
// threshold key, above every number when that is a NaN.
__device__ __forceinline__ float limit_value(Key limit) {
    const float x = key_value(limit);
    return x != x ? INFINITY : x;
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

constexpr int kMaxStages = 6;

// What a block of a cluster leaves with the first one.
struct Partial {
    float m, s, t, unused;
    Key keys[kMaxTop];
};

struct Shared {
    uint64_t full[kMaxStages], empty[kMaxStages];
    int abort;
    Key buffer[kWarps][kBuffer];
    Key lists[kWarps][kMaxTop];
    float m[kWarps], s[kWarps], t[kWarps];
    Partial part[kMaxCluster];
};

// The block's 32 largest keys from one descending list in each of the first
// `lists` warps; the result is in sh.lists[0] after the call (which starts
// and ends with a barrier).
__device__ __forceinline__ void block_top(Shared &sh, Key mine, int lists, int warp, int lane) {
    named_bar_sync(1, kThreads);
    sh.lists[warp][lane] = warp < lists ? mine : 0;
    for (int step = kWarps / 2; step >= 1; step >>= 1) {
        if (step >= lists) continue;
        named_bar_sync(1, kThreads);
        if (warp < step) {
            mine = warp_top_of_two(mine, sh.lists[warp + step][31 - lane], lane);
            sh.lists[warp][lane] = mine;
        }
    }
    named_bar_sync(1, kThreads);
}

// The 32 largest of a warp's n buffered keys, descending.
__device__ __forceinline__ Key warp_list(const Key *buffer, int n, int lane) {
    Key k = warp_sort_desc(lane < n ? buffer[lane] : 0, lane);
    if (n > 32) {
        const Key o = warp_sort_desc(lane + 32 < n ? buffer[lane + 32] : 0, lane);
        k = warp_top_of_two(k, __shfl_xor_sync(0xffffffffu, o, 31), lane);
    }
    return k;
}

// ------------------------------------------------------------- statistics

struct Stats {
    float m, s, t;
};

// The exponent that takes sums with reference m to reference `to`; cut off
// further apart than any sum reaches.
__device__ __forceinline__ float shift(float m, float to) {
    return m == to ? 0.f : fmaxf((m - to) * kLog2e, -1e30f);
}

// The warp's statistics from its lanes'.
__device__ __forceinline__ Stats warp_join(Stats v) {
    float m = v.m;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    // a lane without any finite logit has s = t = 0, and its shift is cut off
    const float base = m == -INFINITY ? 0.f : m, d0 = shift(v.m, base), f = ex2(d0);
    v.t = (v.t + d0 * v.s) * f;
    v.s *= f;
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
        v.s += __shfl_xor_sync(0xffffffffu, v.s, d);
        v.t += __shfl_xor_sync(0xffffffffu, v.t, d);
    }
    v.m = m;
    return v;
}

// The block's statistics from each thread's, in warp 0.
__device__ __forceinline__ Stats block_join(Shared &sh, Stats v, int warp, int lane) {
    v = warp_join(v);
    if (lane == 0) sh.m[warp] = v.m, sh.s[warp] = v.s, sh.t[warp] = v.t;
    named_bar_sync(1, kThreads);
    if (warp == 0) {
        const int w = lane < kWarps ? lane : 0;
        v = warp_join(Stats{lane < kWarps ? sh.m[w] : -INFINITY, lane < kWarps ? sh.s[w] : 0.f,
                            lane < kWarps ? sh.t[w] : 0.f});
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

// The given token of a row, and its logit where there is one.
struct Given {
    int64_t token;
    float x;
};

template <typename T>
__device__ __forceinline__ float given_logit(const LogprobArgs &a, int row, int64_t token) {
    if (token < 0 || token >= a.vocab) return 0.f;
    return to_float(static_cast<const T *>(a.logits)[(int64_t)row * a.row_stride + token]);
}

// Results of one row, written by warp 0 (lane l has the l-th largest key,
// lane 0 the given token).
__device__ __forceinline__ void finish_row(const LogprobArgs &a, int row, const Given &g, Stats v, Key best, int lane,
                                           unsigned int *err) {
    const bool empty = v.m == -INFINITY && v.s == 0.f;  // every logit is -inf
    const float log_s = log2f(v.s), ln_s = log_s * kLn2;
    if (lane == 0) {
        if (a.tokens) {
            float lp = empty ? -INFINITY : (g.x - v.m) - ln_s;
            if (g.token < 0) lp = 0.f;
            if (g.token >= a.vocab) {
                report_index(err);
                lp = __uint_as_float(0x7FC00000u);
            }
            a.logprob[row] = lp;
        }
        const float h = (log_s - v.t / v.s) * kLn2;
        a.entropy[row] = empty ? 0.f : (h < 0.f ? 0.f : h);
    }
    if (lane < a.top) {
        const int64_t o = (int64_t)row * a.top + lane;
        a.top_logprob[o] = empty ? -INFINITY : (key_value(best) - v.m) - ln_s;
        a.top_ids[o] = key_index(best);
    }
}

// ------------------------------------------------------------------ loads

// kPerThread logits of one thread from a chunk in shared memory: 16-byte
// vectors, kThreads vectors apart.  Element 0 of the chunk has index `first`;
// outside [lo, hi) (`edge`: the chunk has such elements) logits read as -inf.
template <typename T>
__device__ __forceinline__ void load_chunk(const T *chunk, bool edge, int first, int lo, int hi, int tid,
                                           float (&x)[kPerThread]) {
    constexpr int kV = 16 / sizeof(T);
#pragma unroll
    for (int j = 0; j < kPerThread / kV; ++j) {
        const int o = (j * kThreads + tid) * kV;
        float *d = x + j * kV;
        const uint4 w = *reinterpret_cast<const uint4 *>(chunk + o);
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
        if (edge) {
#pragma unroll
            for (int e = 0; e < kV; ++e)
                if (first + o + e < lo || first + o + e >= hi) d[e] = -INFINITY;
        }
    }
}

// Index (within the chunk) of a thread's e-th logit.
template <typename T>
__device__ __forceinline__ int chunk_index(int e, int tid) {
    constexpr int kV = 16 / sizeof(T);
    return (e / kV * kThreads + tid) * kV + e % kV;
}

// A split of a row, and the 16-byte granules that hold it: the copies start
// at the boundary at or before the first logit and end at the one at or
// after the last; no other memory is touched.
template <typename T>
struct Span {
    const T *src;
    int begin, lo, hi, chunks;
    __device__ __forceinline__ Span(const LogprobArgs &a, int unit, int splits, int span) {
        const int row = unit / splits;
        lo = (unit - row * splits) * span, hi = min(a.vocab, lo + span);
        const T *x = static_cast<const T *>(a.logits) + (int64_t)row * a.row_stride + lo;
        const int skew = (int)((reinterpret_cast<uintptr_t>(x) & 15u) / sizeof(T));
        src = x - skew, begin = lo - skew;
        chunks = (hi - begin + kChunk - 1) / kChunk;
    }
    __device__ __forceinline__ uint32_t bytes(int c) const {
        const int64_t left = ((int64_t)(hi - begin) * sizeof(T) + 15) / 16 * 16 - (int64_t)c * kChunk * sizeof(T);
        return (uint32_t)min(left, (int64_t)(kChunk * sizeof(T)));
    }
};

// Each CTA takes the units (rows, or one split of one row) blockIdx.x,
// + gridDim.x, ...; its ring runs on over their ends, so the next unit's
// first chunks arrive while the last one is finished.  The splits of a row
// are the CTAs of a cluster, with one unit each.
template <typename T>
__global__ void __launch_bounds__(kThreads + 32, 2) token_logprobs_kernel(const LogprobArgs a, int splits, int span,
                                                                          int units, unsigned int *err) {
    constexpr int kChunkBytes = kChunk * sizeof(T), kStages = kRingBytes / kChunkBytes;
    extern __shared__ __align__(128) uint8_t ring[];
    __shared__ Shared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], kWarps);
        }
        sh.abort = 0;
        mbar_fence_init();
    }
    __syncthreads();
    if (splits > 1) cluster_arrive();  // this block's shared memory is there
    pdl_launch_dependents();
    pdl_wait();
    if (warp == kWarps) {
        // copies of all chunks, in order; a warp of its own, because every
        // delay of it starves the others
        uint32_t copies = 0, phase = 1;
        int slot = 0;
        bool ok = lane == 0;
        for (int unit = blockIdx.x; unit < units && ok; unit += gridDim.x) {
            const Span<T> w(a, unit, splits, span);
            for (int c = 0; c < w.chunks && ok; ++c) {
                ok = mbar_wait(&sh.empty[slot], phase, &sh.abort, err);
                if (!ok) break;
                const uint32_t bytes = w.bytes(c);
                mbar_arrive_expect_tx(&sh.full[slot], bytes);
                bulk_g2s(ring + slot * kChunkBytes, w.src + (int64_t)c * kChunk, bytes, &sh.full[slot]);
                ++copies;
                if (++slot == kStages) slot = 0, phase ^= 1;
            }
        }
        // the last copies land before the CTA may exit
        for (uint32_t c = copies > kStages ? copies - kStages : 0; c < copies; ++c)
            mbar_drain(&sh.full[c % kStages], c / kStages & 1);
        __syncwarp();
        if (splits > 1) {
            cluster_wait();
            cluster_arrive();
            cluster_wait();
        }
        return;
    }
    bool ok = true;
    int slot = 0;
    uint32_t phase = 0;

    for (int unit = blockIdx.x; unit < units; unit += gridDim.x) {
        const Span<T> w(a, unit, splits, span);
        const int lo = w.lo, hi = w.hi;
        // the token is read at the start of the row and its logit at the last
        // chunk: waited for where it is used, each would show
        Given given{-1, 0.f};
        const bool mine_to_give = tid == 0 && blockIdx.x % splits == 0 && a.tokens;
        if (mine_to_give) given.token = a.tokens[unit / splits];
        Stats st{-INFINITY, 0.f, 0.f};
        Key limit = 0;                // candidates are keys above it; the same across the warp
        float limit_x = -INFINITY;    // its value
        int count = 0;                // keys in the warp's buffer
        Key *buffer = sh.buffer[warp];
        for (int c = 0; c < w.chunks; ++c) {
            const int first = w.begin + c * kChunk;
            ok = mbar_wait(&sh.full[slot], phase, &sh.abort, err) && ok;
            float x[kPerThread];
            load_chunk<T>(reinterpret_cast<const T *>(ring + slot * kChunkBytes), first < lo || first + kChunk > hi,
                          first, lo, hi, tid, x);
            float top = max_nan(x[0], x[1]);  // NaN if one is
            float low = fminf(x[0], x[1]);
#pragma unroll
            for (int e = 2; e < kPerThread; e += 2) {
                top = max_nan(top, x[e], x[e + 1]);
                low = min3(low, x[e], x[e + 1]);
            }
            // a NaN leaves m as it is and reaches s and t below
            if (top > st.m) {
                const float d = shift(st.m, top), f = ex2(d);
                st.t = (st.t + d * st.s) * f;
                st.s *= f;
                st.m = top;
            }
            const float base = st.m == -INFINITY ? 0.f : st.m;
            const uint64_t c2 = pack2(kLog2e, kLog2e), m2 = pack2(-base, -base);
            uint64_t s2 = pack2(st.s, 0.f), t2 = pack2(st.t, 0.f);
            auto add = [&](auto far) {
#pragma unroll
                for (int e = 0; e < kPerThread; e += 2) {
                    float y0, y1;
                    unpack2(mul2(add2(pack2(x[e], x[e + 1]), m2), c2), y0, y1);
                    // -inf, or a product that overflowed: 2^y is 0, and y 2^y
                    // must be
                    if (decltype(far)::value) y0 = max_nan(y0, kFloor), y1 = max_nan(y1, kFloor);
                    const uint64_t p = pack2(ex2(y0), ex2(y1));
                    s2 = add2(s2, p);
                    t2 = fma2(pack2(y0, y1), p, t2);
                }
            };
            if (__any_sync(0xffffffffu, low < -kFar || st.m > kFar))
                add(std::true_type{});
            else
                add(std::false_type{});
            float u, v;
            unpack2(s2, u, v);
            st.s = u + v;
            unpack2(t2, u, v);
            st.t = u + v;
            if (mine_to_give && c + 1 == w.chunks) given.x = given_logit<T>(a, unit / splits, given.token);
            const T *chunk = reinterpret_cast<const T *>(ring + slot * kChunkBytes);
            if (a.top > 0) {
                if (c == 0) {
                    // this thread's best key
                    Key mine = 0;
                    if (top == top) {
                        int at = 0;
#pragma unroll
                        for (int e = kPerThread - 1; e >= 0; --e) at = x[e] == top ? chunk_index<T>(e, tid) : at;
                        if (first + at >= lo && first + at < hi) mine = make_key(top, first + at);
                    }
                    if (!mine) {  // a NaN, or only logits outside the row and -inf
#pragma unroll 1
                        for (int e = 0; e < kPerThread; ++e) {
                            const int o = chunk_index<T>(e, tid), i = first + o;
                            if (i < lo || i >= hi) continue;
                            const Key k = make_key(to_float(chunk[o]), i);
                            if (k > mine) mine = k;
                        }
                    }
                    block_top(sh, warp_sort_desc(mine, lane), kWarps, warp, lane);
                    const Key best = sh.lists[0][a.top - 1];
                    if (best > 0) limit = best - 1;  // equal keys are candidates
                    limit_x = limit ? limit_value(limit) : -INFINITY;
                }
                // Threads that may hold a candidate, two of them a step and
                // 16 lanes to each.  In a
                // later chunk a logit that equals the threshold's ranks
                // below it.
                const bool hit = !limit || !(c == 0 ? top < limit_x : top <= limit_x);
                for (uint32_t m = __ballot_sync(0xffffffffu, hit); m;) {
                    const int l0 = __ffs(m) - 1;
                    m &= m - 1;
                    const int of = lane < kPerThread ? l0 : m ? __ffs(m) - 1 : -1;
                    m &= m - 1;
                    const int o = chunk_index<T>(lane & 15, warp * 32 + max(of, 0)), i = first + o;
                    Key k = 0;
                    if (of >= 0 && i >= lo && i < hi) k = make_key(to_float(chunk[o]), i);
                    const bool mine = k > limit;
                    const uint32_t all = __ballot_sync(0xffffffffu, mine);
                    if (count + __popc(all) > kBuffer) {
                        const Key kept = warp_list(buffer, count, lane);
                        __syncwarp();
                        buffer[lane] = kept;
                        count = kMaxTop;
                        const Key least = __shfl_sync(0xffffffffu, kept, a.top - 1);
                        if (least > limit) limit = least, limit_x = limit_value(limit);
                    }
                    if (mine) buffer[count + __popc(all & ((1u << lane) - 1))] = k;
                    count += __popc(all);
                    __syncwarp();
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.empty[slot]);
            if (++slot == kStages) slot = 0, phase ^= 1;
        }
        if (named_bar_or(1, kThreads, !ok)) break;  // a wait was abandoned, and reported
        Key ranked = 0;
        if (a.top > 0) {
            block_top(sh, warp_list(buffer, count, lane), kWarps, warp, lane);
            if (warp == 0) ranked = sh.lists[0][lane];
        }
        st = block_join(sh, st, warp, lane);
        if (splits == 1) {
            if (warp == 0) finish_row(a, unit, given, st, ranked, lane, err);
            // the other warps go on: they meet warp 0 before they write what
            // it still reads
            continue;
        }
        // the cluster's one unit: every block's results to the first
        const int rank = blockIdx.x % splits;
        cluster_wait();
        if (warp == 0) {
            const uint32_t to = first_block(&sh.part[rank]);
            if (lane == 0) store_cluster(to, __float_as_uint(st.m), __float_as_uint(st.s));
            if (lane == 0) store_cluster(to + 8, __float_as_uint(st.t), 0);
            store_cluster(to + 16 + 8 * lane, (uint32_t)ranked, (uint32_t)(ranked >> 32));
            __syncwarp();
        }
        cluster_arrive();
        cluster_wait();
        if (rank == 0) {
            const Partial &mine = sh.part[lane < splits ? lane : 0];
            if (warp == 0)
                st = warp_join(Stats{lane < splits ? mine.m : -INFINITY, lane < splits ? mine.s : 0.f,
                                     lane < splits ? mine.t : 0.f});
            if (a.top > 0) {
                block_top(sh, warp < splits ? sh.part[warp].keys[lane] : 0, splits, warp, lane);
                ranked = sh.lists[0][lane];
            }
            if (warp == 0) finish_row(a, unit / splits, given, st, ranked, lane, err);
        }
        return;
    }
    // a wait was abandoned (blocks that share a row still meet)
    if (splits > 1) {
        cluster_wait();
        cluster_arrive();
        cluster_wait();
    }
}

// Blocks that share a row: as many as leave no SM with more than two, none
// with fewer than kMinSpan logits.
constexpr int kMinSpan = 1024;

int logprob_splits(int rows, int vocab, int sms) {
    int n = 1;
    while (n < kMaxCluster && (int64_t)rows * n * 2 <= 2 * sms && vocab / (n * 2) >= kMinSpan) n *= 2;
    return n;
}

int current_sms() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? device_sm_count(dev) : 0;
}

template <typename T>
cudaError_t launch_typed(const LogprobArgs &a, cudaStream_t s, unsigned int *err) {
    const int sms = current_sms();
    if (sms < 1) return cudaErrorInvalidDevice;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(token_logprobs_kernel<T>), kRingBytes);
    if (e != cudaSuccess) return e;
    const int splits = logprob_splits(a.rows, a.vocab, sms);
    // spans of whole 128-byte lines; the last is shorter
    const int span = ((a.vocab + splits - 1) / splits + 63) / 64 * 64;
    const int units = a.rows * splits, ctas = units < 2 * sms ? units : 2 * sms;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kThreads + 32);
    cfg.dynamicSmemBytes = kRingBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = splits, attr[1].val.clusterDim.y = 1, attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, token_logprobs_kernel<T>, a, splits, span, units, err);
}

}  // namespace

cudaError_t launch_token_logprobs(const LogprobArgs &a, bool bf16, cudaStream_t s, unsigned int *err) {
    return bf16 ? launch_typed<__nv_bfloat16>(a, s, err) : launch_typed<float>(a, s, err);
}

}  // namespace q4_0
