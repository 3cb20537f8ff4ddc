// attention.cu -- causal attention over a paged bfloat16 cache (declared in
// include/q4_0.h): single tokens, drafts, chunks and whole prompts of a
// ragged batch, optionally with a sliding window and first tokens that stay
// visible.
//
// Mathematics, for a query row at position t and the keys j it sees
// (j <= t, and j > t - window or j < sinks): with a running reference m,
//   p_j = 2^(c (s_j - m)),  l = sum p_j,  O = sum p_j v_j,  out = O / l,
// s_j = q . k_j, c = scale * log2 e, all of s, l, O and m in fp32.  m follows
// the running maximum only when a row's maximum grew by more than 2^8 in p:
// the result does not depend on m, p <= 2^8 keeps every sum far inside
// fp32, and most tiles then skip the correction of O.  p is rounded to
// bfloat16 for the second product: the MMA takes one operand type, and V is
// bfloat16; l sums p before the rounding.
//
// Layout of work.  The rows of a tile are (token, head of the group) pairs:
// all query heads that share a key head read each key tile once, and a tile
// of 128 rows spans few tokens, so little of a causal or windowed tile is
// masked.  An item is two tiles (A and B) of one sequence and key head; its
// cost is the number of 128-token key tiles it sees.  One CTA per SM takes
// an equal share of all key tiles, in item order, whatever the batch looks
// like; an item that a share's boundary cuts leaves partial results that
// attention_join_kernel adds in share order, so results are deterministic.
//
// Warps: 0 copies Q and the ring of K and V tiles (TMA; page boxes that no
// query sees are not read: an out-of-range page coordinate fills zeros),
// 1 issues the MMAs, 2-5 and 6-9 do the softmax of tile A and of tile B, one
// thread per row, S and P in tensor memory.  While one tile is in softmax
// the tensor cores work on the other.
#include <cuda.h>
#include <cuda_bf16.h>

#include <mutex>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr int kTile = 128;      // rows of a tile, and tokens of a key tile
constexpr int kThreads = 320;
constexpr int kStages = 5;      // K or V tiles in the ring
constexpr int kStatBytes = 2048;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;    // log2 of the growth of a row's maximum that moves its reference

struct Params {
    const int32_t *page_table, *q_start, *kv_len;
    int64_t table_stride;
    int sequences, table_width, pages, page_size;
    int rows, q_heads, kv_heads, group, window, sinks;
    int tokens;  // per tile: 128 / group
    int box;     // token rows of one K or V copy
    int max_q_len;
    int piece_rows;  // rows a piece can have: one tile's when max_q_len fits it
    float scale_log2;
    void *out;
    float *lse;
    int out_bf16;
    float *part;      // [CTA][head piece, tail piece][piece_rows][D], unnormalised
    float2 *part_ml;  // the rows' (m * scale_log2, l)
    int4 *record;     // per CTA: flags, then sequence, first token and key head of the tail piece
    unsigned int *err;
};

// Flags of a CTA's record.
constexpr int kHeadPiece = 1;     // its first piece continues an item of an earlier CTA
constexpr int kHeadGoesOn = 2;    // ... which also goes on in the next CTA
constexpr int kTailPiece = 4;     // its last piece starts an item that goes on in the next CTA

// One sequence of the batch, clamped to what the arrays can hold.
struct Sequence {
    int row0, len, kv;  // first row of q, rows, tokens in the cache
};

__device__ __forceinline__ Sequence sequence(const Params &p, int b) {
    Sequence s;
    const int r0 = min(max(p.q_start[b], 0), p.rows);
    const int r1 = min(max(p.q_start[b + 1], r0), min(p.rows, r0 + p.max_q_len));
    s.row0 = r0;
    s.len = r1 - r0;
    s.kv = (int)min((int64_t)max(p.kv_len[b], 0), (int64_t)p.table_width * p.page_size);
    return s;
}

// Whether the arrays hold what the call promised of sequence b.
__device__ __forceinline__ bool sequence_fits(const Params &p, const Sequence &s, int b) {
    return p.q_start[b] == s.row0 && p.q_start[b + 1] == s.row0 + s.len && p.kv_len[b] == s.kv;
}

__device__ __forceinline__ int items_of(const Params &p, const Sequence &s) {
    return (s.len + 2 * p.tokens - 1) / (2 * p.tokens);
}

// The tokens the queries of an item see: [0, sink_end) and [lo, hi), and the
// key tiles that hold them: `sink_tiles` from token 0, then from tile `wtile`.
struct Range {
    int pos0;  // position of the item's first query
    int tokens;
    int lo, hi, sink_end;
    int sink_tiles, wtile, n;
};

__device__ __forceinline__ Range item_range(const Params &p, const Sequence &s, int item) {
    Range r;
    const int i0 = item * 2 * p.tokens;
    r.tokens = min(2 * p.tokens, s.len - i0);
    r.pos0 = s.kv - s.len + i0;
    r.hi = max(r.pos0 + r.tokens, 0);
    r.lo = p.window ? min(max(r.pos0 - p.window + 1, 0), r.hi) : 0;
    r.sink_end = min(p.sinks, r.lo);
    r.wtile = r.lo / kTile;
    r.sink_tiles = min((r.sink_end + kTile - 1) / kTile, r.wtile);
    // a row that sees nothing still needs its output: one empty tile
    r.n = max(r.sink_tiles + (r.hi + kTile - 1) / kTile - r.wtile, 1);
    return r;
}

__device__ __forceinline__ int key_tile(const Range &r, int t) { return t < r.sink_tiles ? t : r.wtile + t - r.sink_tiles; }

// A CTA's share of the key tiles, item by item; every warp walks it alike.
struct Cursor {
    int head, b, item;   // the current item
    int t0, t1;          // its key tiles in this share
    int64_t left;        // key tiles of the share from t0 on
    Sequence s;
    Range r;

    __device__ __forceinline__ void enter(const Params &p) {
        r = item_range(p, s, item);
        t1 = (int)min((int64_t)r.n, t0 + left);
    }
    // Next item with work; false at the end of the share.
    __device__ __forceinline__ bool next(const Params &p) {
        left -= t1 - t0;
        if (left <= 0) return false;
        t0 = 0;
        if (++item >= items_of(p, s)) {
            item = 0;
            int scanned = 0;
            do {
                if (++b >= p.sequences) {
                    b = 0;
                    ++head;
                }
                s = sequence(p, b);
            } while (s.len == 0 && ++scanned <= p.sequences);
            if (s.len == 0) return false;
        }
        enter(p);
        return true;
    }
};

struct Start {
    int64_t left;
    int head, b, item, t0;
    int64_t warp_sum[kThreads / 32];
};

// Key tiles of a sequence (one key head).
__device__ __forceinline__ int64_t sequence_tiles(const Params &p, const Sequence &s) {
    const int n = items_of(p, s);
    int64_t sum = 0;
    for (int i = 0; i < n; ++i) sum += item_range(p, s, i).n;
    return sum;
}

// Where this CTA's share begins.  Called by all threads; the result is in
// `st` after the call.
__device__ __forceinline__ void locate(const Params &p, Start &st, int cta, int ctas) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int64_t goal = -1;  // the share's first tile within its key head, from the second pass on
    int64_t left = 0;
    int head = 0;
    for (int pass = 0; pass < 2; ++pass) {
        int64_t before = 0;  // tiles of the sequences ahead of this round's
        for (int b0 = 0; b0 < p.sequences; b0 += kThreads) {
            const int b = b0 + tid;
            Sequence s{0, 0, 0};
            if (b < p.sequences) {
                s = sequence(p, b);
                if (pass == 0 && cta == 0 && !sequence_fits(p, s, b)) atomicExch(p.err, kErrBadIndex);
            }
            const int64_t mine = sequence_tiles(p, s);
            int64_t incl = mine;
#pragma unroll
            for (int d = 1; d < 32; d <<= 1) {
                const int64_t o = __shfl_up_sync(0xffffffffu, incl, d);
                if (lane >= d) incl += o;
            }
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
            const int64_t first = before + ahead + incl - mine;
            if (pass == 1 && goal >= first && goal < first + mine) {
                int64_t rest = goal - first;
                int it = 0;
                for (;; ++it) {
                    const int n = item_range(p, s, it).n;
                    if (rest < n) break;
                    rest -= n;
                }
                st.head = head, st.b = b, st.item = it, st.t0 = (int)rest, st.left = left;
            }
            before += sum;
        }
        if (pass == 0) {
            const int64_t all = before * p.kv_heads;
            // no share is empty before the last one that is not: an item's
            // pieces are in consecutive CTAs
            const int64_t n = min(all, (int64_t)ctas);
            if (cta >= n) {
                if (tid == 0) st.left = 0;
                break;
            }
            const int64_t u0 = all / n * cta + all % n * cta / n;
            left = all / n * (cta + 1) + all % n * (cta + 1) / n - u0;
            head = (int)(u0 / before);
            goal = u0 - head * before;
        }
    }
    __syncthreads();
}

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;                 // 64-element column blocks
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kBlock = kTile * 128;             // bytes of one column block
    static constexpr int kQ = 0;
    static constexpr int kRing = 2 * kTileBytes;
    static constexpr int kBars = kRing + kStages * kTileBytes;
    static constexpr int kSmem = kBars + kStatBytes + 1024;  // + alignment
};

struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full, q_empty;
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t drain;
    uint32_t tmem;
    int abort;
    Start start;
};
static_assert(sizeof(Bars) <= kStatBytes, "");

// Tensor memory columns.
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int g) { return g * 128; }
__device__ __forceinline__ uint32_t col_o(int g) { return 256 + g * 128; }

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p) {
    using L = Layout<D>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *ring = smem + L::kRing;
    Bars &bar = *reinterpret_cast<Bars *>(smem + L::kBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = &bar.abort;

    if (warp == 1) tmem_alloc(&bar.tmem, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        mbar_init(&bar.q_full, 1);
        mbar_init(&bar.q_empty, 1);
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar.s_full[g], 1);
            mbar_init(&bar.p_full[g], 4);
            mbar_init(&bar.o_full[g], 1);
        }
        mbar_init(&bar.drain, 1);
        bar.abort = 0;
        mbar_fence_init();
        tma_prefetch_desc(&qmap);
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
    }
    pdl_launch_dependents();
    pdl_wait();
    locate(p, bar.start, blockIdx.x, gridDim.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    Cursor cur;
    cur.left = bar.start.left;
    bool work = cur.left > 0;
    if (work) {
        cur.head = bar.start.head, cur.b = bar.start.b, cur.item = bar.start.item, cur.t0 = bar.start.t0;
        cur.s = sequence(p, cur.b);
        cur.enter(p);
    }

    if (warp == 0) {
        // ---------------------------------------------------- copies
        uint32_t fills = 0;  // K and V tiles copied so far
        uint32_t items = 0;
        bool ok = true;
        const int boxes = kTile / p.box;
        for (; work && ok; work = cur.next(p), ++items) {
            // Q: one copy per 64-element block and tile
            if (!__all_sync(0xffffffffu, mbar_wait(&bar.q_empty, (items & 1) ^ 1, abort_flag, p.err))) break;
            const int tiles = cur.r.tokens > p.tokens ? 2 : 1;
            const uint32_t qbytes = (uint32_t)(p.tokens * p.group * 128);
            if (lane == 0) {
                mbar_arrive_expect_tx(&bar.q_full, tiles * L::kHalves * qbytes);
                for (int g = 0; g < tiles; ++g)
                    for (int h = 0; h < L::kHalves; ++h)
                        tma_load_4d(smem + L::kQ + g * L::kTileBytes + h * L::kBlock, &qmap, h * 64, 0, cur.head,
                                    cur.s.row0 + cur.item * 2 * p.tokens + g * p.tokens, &bar.q_full);
            }
            for (int t = cur.t0; t < cur.t1 && ok; ++t) {
                // lane i: box i of the tile; a box no query sees (or of a bad
                // page) takes the page coordinate past the end, which reads zeros
                const int tok = key_tile(cur.r, t) * kTile + lane * p.box;
                int page = p.pages, off = 0;
                if (lane < boxes &&
                    (tok < cur.r.sink_end || (tok < cur.r.hi && tok + p.box > cur.r.lo))) {
                    const int index = tok / p.page_size;
                    page = p.page_table[(int64_t)cur.b * p.table_stride + index];
                    off = tok - index * p.page_size;
                    if (page < 0 || page >= p.pages) {
                        atomicExch(p.err, kErrBadIndex);
                        page = p.pages;
                    }
                }
#pragma unroll
                for (int kv = 0; kv < 2 && ok; ++kv, ++fills) {
                    const int slot = fills % kStages;
                    ok = __all_sync(0xffffffffu,
                                    mbar_wait(&bar.empty[slot], (fills / kStages & 1) ^ 1, abort_flag, p.err));
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bar.full[slot], L::kTileBytes);
                    __syncwarp();
                    if (lane < boxes) {
                        uint8_t *dst = ring + slot * L::kTileBytes + lane * p.box * 128;
#pragma unroll
                        for (int h = 0; h < L::kHalves; ++h)
                            tma_load_4d(dst + h * L::kBlock, kv ? &vmap : &kmap, h * 64, off, cur.head, page,
                                        &bar.full[slot]);
                    }
                    __syncwarp();
                }
            }
        }
        // every copy has landed before the CTA may exit (at once unless a
        // wait was abandoned)
        for (uint32_t i = 0; i < kStages; ++i) {
            if (i >= fills) break;
            const uint32_t last = (fills - 1 - i) / kStages * kStages + i;  // last fill of slot i
            mbar_drain(&bar.full[i], last / kStages & 1);
        }
        if (items && *abort_flag) mbar_drain(&bar.q_full, (items - 1) & 1);
    } else if (warp == 1) {
        // ------------------------------------------------------ MMAs
        constexpr uint32_t idesc_qk = idesc_bf16_f32(kTile, kTile, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(kTile, D, true);
        uint32_t fills = 0;  // ring position of the next K tile
        uint32_t items = 0;
        uint32_t p_phase[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t *b, uint32_t parity) {
            ok = __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err));
            return ok;
        };
        // S_g = Q_g K^T
        auto scores = [&](int g, int slot) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint64_t a = smem_desc_k128(smem + L::kQ + g * L::kTileBytes + (k >> 2) * L::kBlock);
                    const uint64_t b = smem_desc_k128(ring + slot * L::kTileBytes + (k >> 2) * L::kBlock);
                    mma_f16_ss(tmem + col_s(g), a + 2 * (k & 3), b + 2 * (k & 3), idesc_qk, k != 0);
                }
                mma_commit(&bar.s_full[g]);
            }
            __syncwarp();
        };
        // O_g (+)= P_g V
        auto values = [&](int g, int slot, bool first) {
            tc_fence_after();
            if (elect_one()) {
#pragma unroll
                for (int k = 0; k < kTile / 16; ++k)
                    mma_f16_ts(tmem + col_o(g), tmem + col_s(g) + 8 * k,
                               smem_desc_mn128(ring + slot * L::kTileBytes + k * 16 * 128, L::kBlock), idesc_pv,
                               !first || k != 0);
                mma_commit(&bar.o_full[g]);
            }
            __syncwarp();
        };
        auto release = [&](uint64_t *b) {
            if (elect_one()) mma_commit(b);
            __syncwarp();
        };
        for (; work && ok; work = cur.next(p), ++items) {
            const int tiles = cur.r.tokens > p.tokens ? 2 : 1;
            if (!wait(&bar.q_full, items & 1)) break;
            if (!wait(&bar.full[fills % kStages], fills / kStages & 1)) break;
            for (int g = 0; g < tiles; ++g) scores(g, fills % kStages);
            release(&bar.empty[fills % kStages]);
            for (int t = cur.t0; t < cur.t1; ++t, fills += 2) {
                const uint32_t v = fills + 1, k = fills + 2;
                const bool more = t + 1 < cur.t1;
                if (!more) release(&bar.q_empty);
                if (!wait(&bar.full[v % kStages], v / kStages & 1)) break;
                // values of tokens that no query of the item sees may be
                // anything (0 * NaN): clear those rows of the tile
                const int tok0 = key_tile(cur.r, t) * kTile;
                if (tok0 + kTile > cur.r.hi || (tok0 < cur.r.lo && tok0 + kTile > cur.r.sink_end)) {
                    for (int i = lane; i < kTile * 8; i += 32) {
                        const int tok = tok0 + (i >> 3);
                        if (tok < cur.r.sink_end || (tok >= cur.r.lo && tok < cur.r.hi)) continue;
#pragma unroll
                        for (int h = 0; h < L::kHalves; ++h)
                            *reinterpret_cast<uint4 *>(ring + v % kStages * L::kTileBytes + h * L::kBlock + i * 16) =
                                make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                }
                if (more && !wait(&bar.full[k % kStages], k / kStages & 1)) break;
                for (int g = 0; g < tiles; ++g) {
                    if (!wait(&bar.p_full[g], p_phase[g])) break;
                    p_phase[g] ^= 1;
                    values(g, v % kStages, t == cur.t0);
                    if (more) scores(g, k % kStages);
                }
                if (!ok) break;
                release(&bar.empty[v % kStages]);
                if (more) release(&bar.empty[k % kStages]);
            }
        }
        // every MMA has finished before tensor memory is released
        if (elect_one()) mma_commit(&bar.drain);
        __syncwarp();
        mbar_drain(&bar.drain, 0);
    } else {
        // --------------------------------------------------- softmax
        const int g = (warp - 2) >> 2;                 // tile
        const int quad = warp & 3;                     // its tensor-memory lanes
        const int row = quad * 32 + lane;              // row of the tile
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t ts = tmem + lanes + col_s(g), to = tmem + lanes + col_o(g);
        const int my_token = row / p.group, my_head = row - my_token * p.group;
        const float c = p.scale_log2;
        uint32_t s_phase = 0, o_phase = 0;
        bool ok = true;
        auto wait = [&](uint64_t *b, uint32_t parity) {
            ok = __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err));
            return ok;
        };
        int flags = 0;
        for (; work && ok; work = cur.next(p)) {
            if (g == 1 && cur.r.tokens <= p.tokens) {
                // no tile B; only the record needs the piece
            } else {
                const int i = g * p.tokens + my_token;  // token within the item
                const bool valid = my_token < p.tokens && i < cur.r.tokens;
                const bool busy = __any_sync(0xffffffffu, valid);
                const int pos = cur.r.pos0 + i;
                // positions of the tile's first and last query
                const int pos_a = cur.r.pos0 + g * p.tokens;
                const int pos_z = cur.r.pos0 + min((g + 1) * p.tokens, cur.r.tokens) - 1;
                float m = -INFINITY, l = 0.f;
                for (int t = cur.t0; t < cur.t1; ++t) {
                    if (!wait(&bar.s_full[g], s_phase)) break;
                    s_phase ^= 1;
                    tc_fence_after();
                    if (busy) {
                        uint32_t s[4][32];
#pragma unroll
                        for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s[q]);
                        tmem_wait_ld();
                        const int tok0 = key_tile(cur.r, t) * kTile;
                        if (tok0 + kTile - 1 > pos_a ||
                            (p.window && tok0 <= pos_z - p.window && tok0 + kTile > p.sinks)) {
                            const int last = pos - tok0;
                            const int first = p.window ? pos - p.window + 1 - tok0 : -1;
                            const int sink = p.sinks - tok0;
#pragma unroll
                            for (int q = 0; q < 4; ++q)
#pragma unroll
                                for (int e = 0; e < 32; ++e) {
                                    const int j = q * 32 + e;
                                    if (j > last || (j < first && j >= sink)) s[q][e] = 0xFF800000u;
                                }
                        }
                        float top = -INFINITY;
#pragma unroll
                        for (int q = 0; q < 4; ++q)
#pragma unroll
                            for (int e = 0; e < 32; e += 2)
                                top = fmaxf(fmaxf(top, __uint_as_float(s[q][e])), __uint_as_float(s[q][e + 1]));
                        const bool grew = top > m && (m == -INFINITY || (top - m) * c > kGrow);
                        if (__any_sync(0xffffffffu, grew)) {
                            const float m_new = fmaxf(m, top);
                            const float f = m == -INFINITY ? 0.f : ex2((m - m_new) * c);
                            l *= f;
                            m = m_new;
                            if (t > cur.t0) {
                                // O of the earlier tiles is complete: scale it
                                if (!wait(&bar.o_full[g], o_phase ^ 1)) break;
                                tc_fence_after();
#pragma unroll
                                for (int d = 0; d < D; d += 32) {
                                    uint32_t o[32];
                                    tmem_ld32(to + d, o);
                                    tmem_wait_ld();
#pragma unroll
                                    for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                                    tmem_st32(to + d, o);
                                }
                            }
                        }
                        const float mc = m == -INFINITY ? 0.f : m * c;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            uint32_t w[16];
#pragma unroll
                            for (int e = 0; e < 16; ++e) {
                                const float a = ex2(fmaf(__uint_as_float(s[q][2 * e]), c, -mc));
                                const float b = ex2(fmaf(__uint_as_float(s[q][2 * e + 1]), c, -mc));
                                l += a + b;
                                w[e] = pack_bf16(a, b);
                            }
                            tmem_st16(ts + q * 16, w);
                        }
                        tmem_wait_st();
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.p_full[g]);
                    o_phase ^= 1;
                }
                if (!ok) break;
                // o_phase counts the tiles' second products: wait for the last
                if (!wait(&bar.o_full[g], o_phase ^ 1)) break;
                tc_fence_after();
                if (busy) {
                    const bool whole = cur.t0 == 0 && cur.t1 == cur.r.n;
                    const float mc = m == -INFINITY ? -INFINITY : m * c;
                    const int64_t at =
                        ((int64_t)cur.s.row0 + cur.item * 2 * p.tokens + i) * p.q_heads + cur.head * p.group + my_head;
                    const int piece = blockIdx.x * 2 + (cur.t0 == 0 ? 1 : 0);
                    const int prow = piece * p.piece_rows + g * kTile + row;
                    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
#pragma unroll
                    for (int d = 0; d < D; d += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + d, o);
                        tmem_wait_ld();
                        if (!valid) {
                        } else if (!whole) {
                            float4 *dst = reinterpret_cast<float4 *>(p.part + (int64_t)prow * D + d);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]),
                                                     __uint_as_float(o[4 * e + 2]), __uint_as_float(o[4 * e + 3]));
                        } else if (p.out_bf16) {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.out) + at * D + d);
#pragma unroll
                            for (int e = 0; e < 4; ++e) {
                                uint32_t w[4];
#pragma unroll
                                for (int f = 0; f < 4; ++f)
                                    w[f] = pack_bf16(__uint_as_float(o[8 * e + 2 * f]) * inv,
                                                     __uint_as_float(o[8 * e + 2 * f + 1]) * inv);
                                dst[e] = make_uint4(w[0], w[1], w[2], w[3]);
                            }
                        } else {
                            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at * D + d);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                dst[e] = make_float4(__uint_as_float(o[4 * e]) * inv, __uint_as_float(o[4 * e + 1]) * inv,
                                                     __uint_as_float(o[4 * e + 2]) * inv,
                                                     __uint_as_float(o[4 * e + 3]) * inv);
                        }
                        __syncwarp();
                    }
                    if (valid) {
                        if (!whole)
                            p.part_ml[prow] = make_float2(mc, l);
                        else if (p.lse)
                            p.lse[at] = (mc + __log2f(l)) * kLn2;
                    }
                }
                tc_fence_before();
            }
            if (cur.t0 > 0) flags |= kHeadPiece | (cur.t1 < cur.r.n ? kHeadGoesOn : 0);
            if (cur.t0 == 0 && cur.t1 < cur.r.n) {
                flags |= kTailPiece;
                if (warp == 2 && lane == 0) p.record[blockIdx.x] = make_int4(flags, cur.b, cur.item, cur.head);
            }
        }
        if (warp == 2 && lane == 0 && !(flags & kTailPiece)) p.record[blockIdx.x] = make_int4(flags, 0, 0, 0);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// Adds the pieces of the items that a share's boundary cut.  blockIdx.x: the
// CTA whose tail piece starts the item; one warp per row of it.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ Params p, int ctas) {
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 rec = p.record[blockIdx.x];
    if (!(rec.x & kTailPiece)) return;
    const int row = blockIdx.y * 8 + warp;
    const int g = row / kTile, in_tile = row - g * kTile;
    const int token = g * p.tokens + in_tile / p.group, head = in_tile % p.group;
    const Sequence s = sequence(p, rec.y);
    const Range r = item_range(p, s, rec.z);
    if (row >= p.piece_rows || in_tile >= p.tokens * p.group || token >= r.tokens) return;
    // pieces: this CTA's tail, then the heads of the next ones
    int n = 1;
    for (int e = blockIdx.x + 1; e < ctas; ++e) {
        const int f = p.record[e].x;
        if (!(f & kHeadPiece)) break;
        ++n;
        if (!(f & kHeadGoesOn)) break;
    }
    auto place = [&](int i) { return ((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * p.piece_rows + row; };
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, p.part_ml[place(i)].x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    const float base = m == -INFINITY ? 0.f : m;
    constexpr int kOwn = D / 32;
    float acc[kOwn] = {}, l = 0.f;
    for (int i = 0; i < n; ++i) {
        const float2 ml = p.part_ml[place(i)];
        const float f = ex2(ml.x - base);
        l += ml.y * f;
        const float *o = p.part + (int64_t)place(i) * D + lane * kOwn;
#pragma unroll
        for (int e = 0; e < kOwn; ++e) acc[e] += o[e] * f;
    }
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int64_t at = ((int64_t)s.row0 + rec.z * 2 * p.tokens + token) * p.q_heads + rec.w * p.group + head;
#pragma unroll
    for (int e = 0; e < kOwn; e += 2) {
        const int64_t o = at * D + lane * kOwn + e;
        if (p.out_bf16)
            *reinterpret_cast<uint32_t *>(static_cast<__nv_bfloat16 *>(p.out) + o) =
                pack_bf16(acc[e] * inv, acc[e + 1] * inv);
        else
            *reinterpret_cast<float2 *>(static_cast<float *>(p.out) + o) =
                make_float2(acc[e] * inv, acc[e + 1] * inv);
    }
    if (p.lse && lane == 0) p.lse[at] = (m + __log2f(l)) * kLn2;
}

// -------------------------------------------------------------------- host

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

// A 4-D bfloat16 tensor with 64-element rows of its copies swizzled over 128
// bytes; strides in elements.
bool make_map(EncodeTiledFn enc, CUtensorMap *map, const void *base, const int64_t (&dim)[4],
              const int64_t (&stride)[3], int box1, int box3) {
    const cuuint64_t dims[4] = {(cuuint64_t)dim[0], (cuuint64_t)dim[1], (cuuint64_t)dim[2], (cuuint64_t)dim[3]};
    const cuuint64_t strides[3] = {(cuuint64_t)stride[0] * 2, (cuuint64_t)stride[1] * 2, (cuuint64_t)stride[2] * 2};
    const cuuint32_t box[4] = {64, (cuuint32_t)box1, 1, (cuuint32_t)box3};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int gcd(int a, int b) { return b ? gcd(b, a % b) : a; }

// Rows of an item that has at most max_q_len tokens.
int item_rows(int group, int max_q_len) {
    const int tokens = kTile / group;
    return max_q_len <= tokens ? max_q_len * group : 2 * kTile;
}

struct WorkspaceLayout {
    size_t ml_off, rec_off, bytes;
    WorkspaceLayout(int ctas, int D, int piece_rows) {
        const size_t rows = (size_t)ctas * 2 * piece_rows;
        ml_off = rows * D * 4;
        rec_off = ml_off + rows * 8;
        bytes = (rec_off + (size_t)ctas * 16 + 255) / 256 * 256;
    }
};

template <int D>
cudaError_t launch_d(const AttentionArgs &a, const KvCacheView &c, void *workspace, int ctas, cudaStream_t s,
                     unsigned int *err) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    Params p{};
    p.page_table = c.page_table, p.q_start = c.q_start, p.kv_len = c.kv_len, p.table_stride = c.table_stride;
    p.sequences = c.sequences, p.table_width = c.table_width, p.pages = c.pages, p.page_size = c.page_size;
    p.rows = a.rows, p.q_heads = a.q_heads, p.kv_heads = c.kv_heads, p.group = a.q_heads / c.kv_heads;
    p.window = a.window, p.sinks = a.sinks;
    p.tokens = kTile / p.group;
    p.box = gcd(c.page_size, kTile);
    p.scale_log2 = a.scale * kLog2e;
    p.out = a.out, p.lse = a.lse, p.out_bf16 = a.out_bf16;
    p.max_q_len = a.max_q_len;
    p.piece_rows = item_rows(p.group, a.max_q_len);
    const WorkspaceLayout w(ctas, D, p.piece_rows);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.part = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + w.ml_off);
    p.record = reinterpret_cast<int4 *>(ws + w.rec_off);
    p.err = err;
    CUtensorMap qmap, kmap, vmap;
    // q as {element, head of the group, key head, row}
    if (!make_map(enc, &qmap, a.q, {D, p.group, p.kv_heads, a.rows},
                  {a.q_head_stride, a.q_head_stride * p.group, a.q_row_stride}, p.group, p.tokens))
        return cudaErrorInvalidValue;
    // k and v as {element, token of the page, key head, page}
    if (!make_map(enc, &kmap, c.k, {D, c.page_size, c.kv_heads, c.pages},
                  {c.k_stride[2], c.k_stride[1], c.k_stride[0]}, p.box, 1) ||
        !make_map(enc, &vmap, c.v, {D, c.page_size, c.kv_heads, c.pages},
                  {c.v_stride[2], c.v_stride[1], c.v_stride[0]}, p.box, 1))
        return cudaErrorInvalidValue;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(attention_kernel<D>), Layout<D>::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attention_kernel<D>, dim3(ctas), dim3(kThreads), Layout<D>::kSmem, s, qmap, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    return launch_pdl(attention_join_kernel<D>, dim3(ctas, (p.piece_rows + 7) / 8), dim3(256), 0, s, p, ctas);
}

int current_sms() {
    int dev = 0;
    return cudaGetDevice(&dev) == cudaSuccess ? device_sm_count(dev) : 0;
}

}  // namespace

size_t attention_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q_len) {
    return WorkspaceLayout(current_sms(), head_dim, item_rows(q_heads / kv_heads, max_q_len)).bytes;
}

cudaError_t launch_attention(const AttentionArgs &a, const KvCacheView &c, void *workspace, cudaStream_t s,
                             unsigned int *err) {
    const int sms = current_sms();
    if (sms < 1) return cudaErrorInvalidDevice;
    return c.head_dim == 128 ? launch_d<128>(a, c, workspace, sms, s, err)
                             : launch_d<64>(a, c, workspace, sms, s, err);
}

}  // namespace q4_0
