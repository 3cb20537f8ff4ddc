// attention.cu -- causal attention over a paged bfloat16 cache (declared in
// include/q4_0.h): single tokens, drafts, chunks and whole prompts of a
// ragged batch, optionally with a sliding window and first tokens that stay
// visible.
//
// Mathematics, for a query row at position t and the keys j it sees
// (j <= t, and j > t - window or j < sinks): with a running reference m,
//   p_j = 2^(c s_j - c m),  l = sum p_j,  O = sum p_j v_j,  out = O / l,
// s_j = q . k_j, c = scale * log2 e, all of s, l, O and c m in fp32.  c m is
// kept rounded, and its rounding is the same in all of a row.  It follows
// the running maximum only when a row's maximum grew by more than 2^8 in p:
// the result does not depend on m, p <= 2^8 (2^72 where c m is near 2^30)
// keeps every sum inside fp32, and most tiles then skip the correction of O.
// p is rounded to bfloat16 for the second product: the MMA takes one operand
// type, and V is bfloat16; l sums p before the rounding.
//
// Layout of work.  The rows of a tile are (token, head of the group) pairs:
// all query heads that share a key head read each key tile once, and a tile
// of 128 rows spans few tokens, so little of a causal or windowed tile is
// masked.  An item is two tiles (A and B) of one sequence and key head; its
// cost is the number of 128-token key tiles it sees, each weighted by whether
// one tile or two share it.  One CTA per SM takes an equal share of all cost,
// in item order, whatever the batch looks like; an item that a share's
// boundary cuts leaves partial results that attention_join_kernel adds in
// share order, so results are deterministic.
//
// Warps: 0 copies Q and K tiles and 2 V tiles into rings (TMA; boxes of a
// page that no query sees are not read: an out-of-range page coordinate fills
// zeros), 1 issues the MMAs, 3 hands out the items, 4-7 and 8-11 do the
// softmax of group A and of group B, one thread per row, S and P in tensor
// memory.  While one group is in softmax the tensor cores work on the other.
// In an item of two tiles a group has one tile each; in a narrow item (one
// tile: single tokens, drafts, a chunk's end) the groups take the key tiles
// in turn, and group A adds B's O to its own at the end.
//
// Bounds and measurements (bfloat16, 40 query heads on 8 key heads of 128
// unless stated; device time):
// * A new token of each of many long sequences reads its cache once and is
//   bound by that: 64 sequences under a window of 4096, 1.08 GB, 175 us (6.2
//   TB/s, 0.91 of a copy's rate); 16 of 1 to 8 thousand tokens, 347 MB, 67 us
//   (5.2 TB/s), of which 16 us are launch, the search for a share's start,
//   the first reads and the join.
// * A prompt is bound by the chain softmax -> P V and the next Q K of a group
//   (1500 + 1800 cycles a pair of tiles at D = 128, of which the tensor cores
//   are busy 2048): 8192 tokens after 8192 others take 1.34 to 1.38 ms, 1.49
//   to 1.54 PFLOP/s (1.43 ms in a long run, at the board's power limit).
//   TMEM is full (two S, two O), so a group's next scores cannot start
//   earlier.  A shorter softmax would show; the exponential units are not
//   what bounds it (a polynomial on the multiply-add units for 1/8 to 1/2 of
//   the elements made it 3 to 18 % slower).
// * Prompts of 2500 to 3500 tokens under a window of 1000 (24 heads on 4, D =
//   64) take 142 us: 2750 cycles a pair of tiles, and 10000 more an item of
//   ten, for masks at both ends of the window, both groups' start at once,
//   the last product and the rows' stores.  With 40 heads on 8, D = 128, they
//   take 265 us.
// * One token after 2047 takes 16.7 us against a floor of 1.2: 4.3 launch, 4
//   join, the rest reads that wait for one another.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>
#include <mutex>
#include <type_traits>

#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr int kTile = 128;      // rows of a tile, and tokens of a key tile
constexpr int kThreads = 384;
// registers a thread: the launch gives 168 each; the copy and MMA warps give
// theirs up to the softmax warps (128 * 56 + 256 * 224 = 384 * 168)
constexpr int kRoleRegs = 56, kSoftmaxRegs = 224;
constexpr int kStatBytes = 2048;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;    // log2 of the growth of a row's maximum that moves its reference
// Every p of a row has 2^(the rounding of c m) as a factor.  Where c m is
// beyond this, that would leave fp32, and fp32 scores that differ are 64
// apart at least: the next power of two in the place of c gives the same
// p, 1 or nothing, without a rounding.
constexpr float kHuge = 1 << 30;

struct Params {
    const int32_t *page_table, *q_start, *kv_len;
    int64_t table_stride;
    int sequences, table_width, pages, page_size;
    int rows, q_heads, kv_heads, group, window, sinks;
    int tokens;  // per tile: 128 / group
    int box;     // token rows of one K or V copy
    int cost[2];  // of a key tile of a narrow item and of one of two tiles
    int max_q_len;
    int piece_rows;  // rows a piece can have: one tile's when max_q_len fits it
    float scale_log2, scale_pow2, scale_back;  // scale * log2 e, the next power of two, and their ratio
    void *out;
    float *lse;
    int out_bf16;
    float *part;      // [CTA][head piece, tail piece][piece_rows][D], unnormalised
    float2 *part_ml;  // the rows' (m * scale_log2, l)
    int4 *record;     // per CTA: flags, then first row of q, tokens and key head of the tail piece's item
    unsigned int *err;
};

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

// A CTA's part of an item, as warp 3 hands it to the others.
struct Item {
    int t0, t1, n;       // its key tiles [t0, t1) of the item's n; t0 == t1: the share has ended
    int head, b;         // key head and sequence
    int row0, tokens;    // first row of q, and tokens
    int pos0;            // position of the first
    int lo, hi, sink_end, sink_tiles, wtile;  // as in Range
    __device__ __forceinline__ int key_tile(int t) const { return t < sink_tiles ? t : wtile + t - sink_tiles; }
};

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

__device__ __forceinline__ int tile_cost(const Params &p, const Range &r) { return p.cost[r.tokens > p.tokens]; }

__device__ __forceinline__ int64_t item_cost(const Params &p, const Sequence &s, int item) {
    const Range r = item_range(p, s, item);
    return (int64_t)r.n * tile_cost(p, r);
}

// Cost (for one key head) of each lane's sequence; the warp takes the items
// of a long one together.
__device__ __forceinline__ int64_t sequence_cost(const Params &p, const Sequence &s, int lane) {
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
__device__ __forceinline__ void locate(const Params &p, Start &st, int cta, int ctas) {
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
    const int64_t n = min(max(all / p.cost[1], (int64_t)(all > 0)), (int64_t)ctas);
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

// f(0), f(1), ... f(N - 1) with constants as arguments.
template <int N, typename F>
__device__ __forceinline__ void each_step(F &&f) {
    if constexpr (N > 0) {
        each_step<N - 1>(f);
        f(std::integral_constant<uint32_t, N - 1>{});
    }
}

template <int D>
struct Layout {
    static constexpr int kHalves = D / 64;                 // 64-element column blocks
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kBlock = kTile * 128;             // bytes of one column block
    static constexpr int kStages = D == 128 ? 5 : 10;      // K or V tiles in the ring
    static constexpr int kQTiles = D == 128 ? 2 : 4;       // Q tiles held
    static constexpr int kQ = 0;
    static constexpr int kRing = kQTiles * kTileBytes;
    static constexpr int kBars = kRing + kStages * kTileBytes;
    static constexpr int kSmem = kBars + kStatBytes + 1024;  // + alignment
};

constexpr int kItems = 4;     // items handed out ahead
constexpr int kReaders = 11;  // warps that read them

constexpr int kMaxQTiles = 4;

template <int kStages>
struct Bars {
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full[kMaxQTiles], q_empty[kMaxQTiles];
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t b_done, merged;  // narrow items: B's O and (m, l) are ready; A has read them
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t drain;
    Item item[kItems];
    float2 ml[kTile];
    uint32_t tmem;
    uint32_t fills[2], q_fills;  // copies made: past the last K and V tile's ring position, and of Q
    int abort;
    Start start;
};
static_assert(sizeof(Bars<10>) <= kStatBytes, "");

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
    constexpr int kStages = L::kStages;
    Bars<kStages> &bar = *reinterpret_cast<Bars<kStages> *>(smem + L::kBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = &bar.abort;

    if (warp == 1) tmem_alloc(&bar.tmem, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; i < L::kQTiles; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
        }
        for (int g = 0; g < 2; ++g) {
            mbar_init(&bar.s_full[g], 1);
            mbar_init(&bar.p_full[g], 4);
            mbar_init(&bar.o_full[g], 1);
        }
        mbar_init(&bar.b_done, 4);
        mbar_init(&bar.merged, 4);
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&bar.item_full[i], 1);
            mbar_init(&bar.item_empty[i], kReaders);
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

    // The next item of the share, or false at its end or when a wait was
    // abandoned; done_item() hands its record back.
    uint32_t items = 0;
    Item cur;
    auto next_item = [&]() {
        const int i = items % kItems;
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.item_full[i], items / kItems & 1, abort_flag, p.err))) return false;
        cur = bar.item[i];
        return cur.t0 < cur.t1;
    };
    auto done_item = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.item_empty[items % kItems]);
        ++items;
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegs));
        if (warp == 0 || warp == 2) {
            // ------------------------------------------------ copies
            // K and V tiles alternate in one ring; each warp fills its own.
            // A warp may not be two uses of a slot ahead (its wait would take
            // the older phase for the newer): the MMA warp frees tiles in an
            // order in which the slot of fill f - 7, waited for at fill
            // f - 2, is freed after that of f - 10.
            const int kv = warp >> 1;  // warp 0: Q and K, warp 2: V
            const CUtensorMap *map = kv ? &vmap : &kmap;
            uint32_t fill = kv;        // ring position of the next tile
            uint32_t slot = kv, phase = 1;
            bool ok = true;
            const int boxes = kTile / p.box, per_load = 32 / boxes;
            // Page numbers are loaded for 32 boxes at a time (lane i: box
            // i % boxes of tile i / boxes) and one load ahead of the copies,
            // across items: a load a tile, waited for, bound the stream.
            struct Group {
                int tiles;                 // 0: the share has ended
                int page, off;             // off < 0: a box that no query sees
                int head, row0, tokens;    // tokens 0: not the item's first group
            };
            int t = 0;
            uint32_t q = 0;  // Q tiles copied
            bool open = false;  // `cur` holds an item with tiles from t on
            auto fetch = [&]() {
                Group o{};
                if (!open) {
                    if (!next_item()) return o;
                    open = true;
                    t = cur.t0;
                    o.row0 = cur.row0, o.tokens = cur.tokens;
                }
                o.head = cur.head;
                o.tiles = min(per_load, cur.t1 - t);
                o.off = -1;
                const int mine = lane / boxes;
                if (mine < o.tiles) {
                    const int tok = cur.key_tile(t + mine) * kTile + (lane - mine * boxes) * p.box;
                    // only boxes that hold a token some query sees
                    if (tok < cur.sink_end || (tok < cur.hi && tok + p.box > cur.lo)) {
                        const int index = tok / p.page_size;
                        o.page = p.page_table[(int64_t)cur.b * p.table_stride + index];
                        o.off = tok - index * p.page_size;
                    }
                }
                t += o.tiles;
                if (t == cur.t1) {
                    open = false;
                    done_item();
                }
                return o;
            };
            Group now = fetch();
            while (ok && now.tiles) {
                const Group then = fetch();
                if (now.off < 0 || now.page < 0 || now.page >= p.pages) {
                    // a page coordinate past the end reads zeros
                    if (now.off >= 0) report_index(p.err);
                    now.page = p.pages, now.off = 0;
                }
                for (int j = 0; j < now.tiles; ++j) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar.empty[slot], phase, abort_flag, p.err));
                    if (!ok) break;
                    const bool issue = elect_one();
                    uint8_t *dst = ring + slot * L::kTileBytes;
                    if (issue) mbar_arrive_expect_tx(&bar.full[slot], L::kTileBytes);
                    for (int i = 0; i < boxes; ++i, dst += p.box * 128) {
                        const int page = __shfl_sync(0xffffffffu, now.page, j * boxes + i);
                        const int off = __shfl_sync(0xffffffffu, now.off, j * boxes + i);
                        if (issue) {
#pragma unroll
                            for (int h = 0; h < L::kHalves; ++h)
                                tma_load_4d(dst + h * L::kBlock, map, h * 64, off, now.head, page, &bar.full[slot]);
                        }
                    }
                    __syncwarp();
                    fill += 2;
                    slot += 2;
                    if (slot >= kStages) slot -= kStages, phase ^= 1;
                    // an item's Q after its first K tile: Q waits for room
                    for (; kv == 0 && now.tokens > 0; now.tokens -= p.tokens, now.row0 += p.tokens) {
                        const int at = q % L::kQTiles;
                        ok = __all_sync(0xffffffffu, mbar_wait(&bar.q_empty[at], (q / L::kQTiles & 1) ^ 1, abort_flag,
                                                               p.err));
                        if (!ok) break;
                        if (elect_one()) {
                            mbar_arrive_expect_tx(&bar.q_full[at], L::kHalves * p.tokens * p.group * 128);
                            for (int h = 0; h < L::kHalves; ++h)
                                tma_load_4d(smem + L::kQ + at * L::kTileBytes + h * L::kBlock, &qmap, h * 64, 0,
                                            now.head, now.row0, &bar.q_full[at]);
                        }
                        __syncwarp();
                        ++q;
                    }
                    if (!ok) break;
                }
                now = then;
            }
            if (lane == 0) {
                bar.fills[kv] = fill;
                if (kv == 0) bar.q_fills = q;
            }
        } else if (warp == 3) {
            // ------------------------------------------------- items
            int flags = 0;
            int4 tail = make_int4(0, 0, 0, 0);
            int64_t left = bar.start.left;
            int head = bar.start.head, b = bar.start.b, it = bar.start.item, t0 = bar.start.t0;
            Sequence s = bar.start.s;
            int n_items = items_of(p, s);
            for (;; ++items) {
                Item o{};
                int64_t cost = 0;
                if (left > 0) {
                    const Range r = item_range(p, s, it);
                    const int each = tile_cost(p, r);
                    cost = (int64_t)r.n * each;
                    o.t0 = t0, o.t1 = left >= cost ? r.n : (int)(left / each), o.n = r.n;
                    o.head = head, o.b = b, o.row0 = s.row0 + it * 2 * p.tokens, o.tokens = r.tokens, o.pos0 = r.pos0;
                    o.lo = r.lo, o.hi = r.hi, o.sink_end = r.sink_end, o.sink_tiles = r.sink_tiles, o.wtile = r.wtile;
                    if (o.t0 > 0) flags |= kHeadPiece | (o.t1 < o.n ? kHeadGoesOn : 0);
                    if (o.t0 == 0 && o.t1 > 0 && o.t1 < o.n)
                        flags |= kTailPiece, tail = make_int4(0, o.row0, o.tokens, head);
                }
                const int i = items % kItems;
                if (!__all_sync(0xffffffffu,
                                mbar_wait(&bar.item_empty[i], (items / kItems & 1) ^ 1, abort_flag, p.err)))
                    break;
                if (lane == 0) {
                    bar.item[i] = o;
                    mbar_arrive(&bar.item_full[i]);
                }
                __syncwarp();
                left -= cost;
                if (o.t0 == o.t1) break;
                t0 = 0;
                if (left > 0 && ++it >= n_items) {
                    it = 0;
                    int scanned = 0;
                    do {
                        if (++b >= p.sequences) {
                            b = 0;
                            ++head;
                        }
                        s = sequence(p, b);
                    } while (s.len == 0 && ++scanned <= p.sequences);
                    n_items = items_of(p, s);
                }
            }
            tail.x = flags;
            if (lane == 0) p.record[blockIdx.x] = tail;
        } else if (warp == 1) {
        // ------------------------------------------------------ MMAs
        constexpr uint32_t idesc_qk = idesc_bf16_f32(kTile, kTile, false);
        constexpr uint32_t idesc_pv = idesc_bf16_f32(kTile, D, true);
        uint32_t fills = 0;  // ring position of the next K tile
        uint32_t q = 0;      // Q tiles of earlier items
        uint32_t p_phase[2] = {0, 0};
        bool ok = true;
        auto wait = [&](uint64_t *b, uint32_t parity) {
            ok = __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err));
            return ok;
        };
        // The instruction rate of this warp bounds the loop: each descriptor
        // is one addition to the low word (the start address), which no
        // offset carries out of.
        const uint64_t q_desc = smem_desc_k128(smem + L::kQ), v_desc = smem_desc_mn128(ring, L::kBlock);
        const uint32_t hi = (uint32_t)(q_desc >> 32);  // the same for all three
        const uint32_t q_lo = (uint32_t)q_desc, k_lo = (uint32_t)smem_desc_k128(ring), v_lo = (uint32_t)v_desc;
        constexpr uint32_t kTileStep = L::kTileBytes >> 4, kBlockStep = L::kBlock >> 4;
        // S_g = Q K^T with Q tile `qt`, for the `last` time (one elected
        // thread)
        auto scores = [&](int g, uint32_t qt, uint32_t slot, bool last) {
            qt %= L::kQTiles;
            const uint32_t a = q_lo + qt * kTileStep, b = k_lo + slot * kTileStep, d = tmem + col_s(g);
            each_step<D / 16>([&](auto step) {
                constexpr uint32_t k = decltype(step)::value, off = (k >> 2) * kBlockStep + 2 * (k & 3);
                mma_f16_ss_at<off, off>(d, a, b, hi, idesc_qk, k != 0);
            });
            mma_commit(&bar.s_full[g]);
            if (last) mma_commit(&bar.q_empty[qt]);
        };
        auto q_full = [&](uint32_t qt) { return wait(&bar.q_full[qt % L::kQTiles], qt / L::kQTiles & 1); };
        // O_g (+)= P_g V (one elected thread)
        auto values = [&](int g, uint32_t slot, bool first) {
            const uint32_t a = tmem + col_s(g), b = v_lo + slot * kTileStep, d = tmem + col_o(g);
            each_step<kTile / 16>([&](auto step) {
                constexpr uint32_t k = decltype(step)::value;
                mma_f16_ts_at<8 * k, k * (16 * 128 >> 4)>(d, a, b, hi, idesc_pv, !first || k != 0);
            });
            mma_commit(&bar.o_full[g]);
        };
        auto full = [&](uint32_t fill) { return wait(&bar.full[fill % kStages], fill / kStages & 1); };
        // Values of tokens that no query of the item sees may be anything
        // (0 * NaN): clear the rows of the tile in [from, to).
        auto clear_rows = [&](int slot, int from, int to) {
            uint8_t *tile = ring + slot * L::kTileBytes;
            for (int i = from * 8 + lane; i < to * 8; i += 32)
#pragma unroll
                for (int h = 0; h < L::kHalves; ++h)
                    *reinterpret_cast<uint4 *>(tile + h * L::kBlock + i * 16) = make_uint4(0, 0, 0, 0);
        };
        // Boxes that no query sees were filled with zeros; what remains are
        // the unseen ends of the boxes that hold the ends of the seen ranges.
        auto clear_unseen = [&](int t, int slot) {
            const int tok0 = cur.key_tile(t) * kTile;
            const int sink = cur.sink_end - tok0, lo = cur.lo - tok0, hi = cur.hi - tok0;
            if (hi >= kTile && (lo <= 0 || sink >= kTile)) return;
            const int mask = ~(p.box - 1);  // a power of two
            if (sink > 0 && sink < kTile) clear_rows(slot, sink, min((sink - 1 & mask) + p.box, max(lo, sink)));
            if (lo > 0 && lo < kTile) clear_rows(slot, max(lo & mask, max(sink, 0)), lo);
            if (hi > 0 && hi < kTile) clear_rows(slot, hi, (hi - 1 & mask) + p.box);
            fence_proxy_async_smem();
            __syncwarp();
        };
        for (; ok && next_item(); done_item()) {
            const bool wide = cur.tokens > p.tokens;
            const int n = cur.t1 - cur.t0;
            if (!q_full(q)) break;
            if (wide) {
                uint32_t slot_k = fills % kStages, slot_v = (fills + 1) % kStages;
                if (!full(fills) || !q_full(q + 1)) break;
                tc_fence_after();
                if (elect_one()) {
                    scores(0, q, slot_k, n == 1);
                    scores(1, q + 1, slot_k, n == 1);
                    mma_commit(&bar.empty[slot_k]);
                }
                __syncwarp();
                for (int t = 0; t < n; ++t) {
                    const uint32_t v = fills + 2 * t + 1;
                    const bool more = t + 1 < n;
                    slot_v = v % kStages, slot_k = (v + 1) % kStages;
                    if (!full(v)) break;
                    clear_unseen(cur.t0 + t, slot_v);
                    if (more && !full(v + 1)) break;
                    if (!wait(&bar.p_full[0], p_phase[0])) break;
                    p_phase[0] ^= 1;
                    tc_fence_after();
                    if (elect_one()) {
                        values(0, slot_v, t == 0);
                        if (more) scores(0, q, slot_k, t + 2 == n);
                    }
                    __syncwarp();
                    if (!wait(&bar.p_full[1], p_phase[1])) break;
                    p_phase[1] ^= 1;
                    tc_fence_after();
                    if (elect_one()) {
                        values(1, slot_v, t == 0);
                        mma_commit(&bar.empty[slot_v]);
                        if (more) {
                            scores(1, q + 1, slot_k, t + 2 == n);
                            mma_commit(&bar.empty[slot_k]);
                        }
                    }
                    __syncwarp();
                }
            } else {
                // the first scores of both groups, then tile t's values and
                // the scores of tile t + 2
                for (int t = 0; ok && t < min(n, 2); ++t) {
                    const uint32_t k = fills + 2 * t;
                    if (!full(k)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        scores(t, q, k % kStages, t + 1 == n);
                        mma_commit(&bar.empty[k % kStages]);
                    }
                    __syncwarp();
                }
                for (int t = 0; ok && t < n; ++t) {
                    const uint32_t v = fills + 2 * t + 1, k = v + 3;
                    const int g = t & 1;
                    if (!full(v)) break;
                    clear_unseen(cur.t0 + t, v % kStages);
                    if (!wait(&bar.p_full[g], p_phase[g])) break;
                    p_phase[g] ^= 1;
                    tc_fence_after();
                    if (elect_one()) {
                        values(g, v % kStages, t < 2);
                        mma_commit(&bar.empty[v % kStages]);
                    }
                    __syncwarp();
                    if (t + 2 >= n) continue;
                    if (!full(k)) break;
                    tc_fence_after();
                    if (elect_one()) {
                        scores(g, q, k % kStages, t + 3 == n);
                        mma_commit(&bar.empty[k % kStages]);
                    }
                    __syncwarp();
                }
            }
            if (!ok) break;
            fills += 2 * n;
            q += wide ? 2 : 1;
        }
        // every MMA has finished before tensor memory is released
        if (elect_one()) mma_commit(&bar.drain);
        __syncwarp();
        mbar_drain(&bar.drain, 0);
        }
    } else {
        // --------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kSoftmaxRegs));
        const int g = (warp - 4) >> 2;                 // group
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
        uint32_t merge_phase = 0;
        bool unmerged = false;  // group B: A may not have read O of the last item yet
        for (; ok && next_item(); done_item()) {
            const bool wide = cur.tokens > p.tokens;
            const int half = wide ? g : 0;                  // the tile of the item
            const int i = half * p.tokens + my_token;       // token within the item
            const bool valid = my_token < p.tokens && i < cur.tokens;
            const bool busy = __any_sync(0xffffffffu, valid);
            const int pos = cur.pos0 + i;
            // positions of the tile's first and last query
            const int pos_a = cur.pos0 + half * p.tokens;
            const int pos_z = cur.pos0 + min((half + 1) * p.tokens, cur.tokens) - 1;
            const int step = wide ? 1 : 2;
            // A row whose maximum grew moves the references of its warp's
            // rows (each its own, one by one, took prompts 1 to 4 % longer).
            // Lanes that are no row of the item must not: they hold other
            // sequences' rows, or what an earlier kernel left in shared
            // memory.  Nothing is above their reference.
            float mc = valid ? -INFINITY : INFINITY, c_row = c, l = 0.f;
            bool started = false;
            for (int t = cur.t0 + (wide ? 0 : g); t < cur.t1; t += step) {
                if (!wait(&bar.s_full[g], s_phase)) break;
                s_phase ^= 1;
                tc_fence_after();
                if (busy) {
                    uint32_t s[4][32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s[q]);
                    tmem_wait_ld();
                    const int tok0 = cur.key_tile(t) * kTile;
                    if (tok0 + kTile - 1 > pos_a || (p.window && tok0 <= pos_z - p.window && tok0 + kTile > p.sinks)) {
                        const int end = pos + 1 - tok0;
                        const int first = p.window ? end - p.window : 0;
                        const int sink = p.sinks - tok0;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const uint32_t seen = below(end - q * 32) & (~below(first - q * 32) | below(sink - q * 32));
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                if (!(seen >> e & 1)) s[q][e] = 0xFF800000u;
                        }
                    }
                    // four chains each for the maximum and the sum: one
                    // would bind the loop by its latency
                    float top4[4];
#pragma unroll
                    for (int q = 0; q < 4; ++q) top4[q] = fmaxf(__uint_as_float(s[q][0]), __uint_as_float(s[q][1]));
#pragma unroll
                    for (int e = 2; e < 32; e += 2)
#pragma unroll
                        for (int q = 0; q < 4; ++q)
                            top4[q] = max3(top4[q], __uint_as_float(s[q][e]), __uint_as_float(s[q][e + 1]));
                    const float top = fmaxf(max3(top4[0], top4[1], top4[2]), top4[3]);
                    // (nothing is above an infinite reference)
                    if (__any_sync(0xffffffffu, fmaf(top, c_row, -mc) > kGrow)) {
                        const float c_top = fabsf(top * c) > kHuge ? p.scale_pow2 : c;
                        const float mc_new = __fmul_rn(top, c_top);
                        const bool above = mc_new > mc;
                        const float f = mc == -INFINITY ? 0.f : above ? ex2(mc - mc_new) : 1.f;
                        l *= f;
                        if (above) mc = mc_new, c_row = c_top;
                        if (started) {
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
                    const float base = mc == -INFINITY ? 0.f : mc;
                    const uint64_t c2 = pack2(c_row, c_row), mc2 = pack2(-base, -base);
                    uint64_t sum[4] = {pack2(l, 0.f), 0, 0, 0};
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) {
                            float a, b;
                            const uint64_t s2 = pack2(__uint_as_float(s[q][2 * e]), __uint_as_float(s[q][2 * e + 1]));
                            unpack2(fma2(s2, c2, mc2), a, b);
                            a = ex2(a), b = ex2(b);
                            sum[e & 3] = add2(sum[e & 3], pack2(a, b));
                            w[e] = pack_bf16(a, b);
                        }
                        tmem_st16(ts + q * 16, w);
                    }
                    float la, lb;
                    unpack2(add2(add2(sum[0], sum[1]), add2(sum[2], sum[3])), la, lb);
                    l = la + lb;
                    tmem_wait_st();
                }
                if (unmerged) {
                    if (!wait(&bar.merged, merge_phase ^ 1)) break;
                    unmerged = false;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.p_full[g]);
                o_phase ^= 1;
                started = true;
            }
            if (!ok) break;
            // o_phase counts the group's second products: wait for the last
            if (started && !wait(&bar.o_full[g], o_phase ^ 1)) break;
            tc_fence_after();
            mc *= c_row == c ? 1.f : p.scale_back;
            if (!wide && g == 1) {
                if (unmerged && !wait(&bar.merged, merge_phase ^ 1)) break;
                bar.ml[row] = make_float2(mc, l);
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bar.b_done);
                unmerged = true;
                merge_phase ^= 1;
            } else {
                float fa = 1.f, fb = 0.f, top = mc;
                if (!wide) {
                    if (!wait(&bar.b_done, merge_phase)) break;
                    merge_phase ^= 1;
                    tc_fence_after();
                    const float2 other = bar.ml[row];
                    top = fmaxf(mc, other.x);
                    const float base = top == -INFINITY ? 0.f : top;
                    fa = ex2(mc - base), fb = ex2(other.x - base);
                    l = l * fa + other.y * fb;
                }
                const bool both = !wide && cur.t1 - cur.t0 > 1;
                if (busy) {
                    const bool whole = cur.t0 == 0 && cur.t1 == cur.n;
                    const int64_t at = ((int64_t)cur.row0 + i) * p.q_heads + cur.head * p.group + my_head;
                    const int piece = blockIdx.x * 2 + (cur.t0 == 0 ? 1 : 0);
                    const int prow = piece * p.piece_rows + half * kTile + row;
                    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
                    if (whole) fa *= inv, fb *= inv;
#pragma unroll
                    for (int d = 0; d < D; d += 32) {
                        uint32_t o[32];
                        tmem_ld32(to + d, o);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * fa);
                        if (both) {
                            uint32_t ob[32];
                            tmem_ld32(to + (col_o(1) - col_o(0)) + d, ob);
                            tmem_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e)
                                o[e] = __float_as_uint(fmaf(__uint_as_float(ob[e]), fb, __uint_as_float(o[e])));
                        }
                        if (valid) {
                            // 32 bytes a store: a thread's row is its own
                            // lines, so a warp's store is one line per lane
                            if (whole && p.out_bf16) {
                                __nv_bfloat16 *dst = static_cast<__nv_bfloat16 *>(p.out) + at * D + d;
                                uint32_t w[16];
#pragma unroll
                                for (int e = 0; e < 16; ++e)
                                    w[e] = pack_bf16(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
                                store32(dst, w);
                                store32(dst + 16, w + 8);
                            } else {
                                float *dst = whole ? static_cast<float *>(p.out) + at * D + d
                                                   : p.part + (int64_t)prow * D + d;
#pragma unroll
                                for (int e = 0; e < 4; ++e) store32(dst + 8 * e, o + 8 * e);
                            }
                        }
                        __syncwarp();
                    }
                    if (valid) {
                        if (!whole)
                            p.part_ml[prow] = make_float2(top, l);
                        else if (p.lse)
                            p.lse[at] = (top + __log2f(l)) * kLn2;
                    }
                }
                tc_fence_before();
                if (!wide) {
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.merged);
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (bar.abort && tid == 0) {
        // a wait was abandoned: copies in flight land before the CTA exits
        // (otherwise every copy was waited for by its reader)
        for (uint32_t i = 0; i < kStages; ++i) {
            int last = -1;
            for (uint32_t f = i; f < max(bar.fills[0], bar.fills[1]); f += kStages)
                if (f < bar.fills[f & 1]) last = f;
            if (last >= 0) mbar_drain(&bar.full[i], last / kStages & 1);
        }
        for (uint32_t f = max(bar.q_fills, (uint32_t)L::kQTiles) - L::kQTiles; f < bar.q_fills; ++f)
            mbar_drain(&bar.q_full[f % L::kQTiles], f / L::kQTiles & 1);
    }
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

// Adds the pieces of the items that a share's boundary cut.  blockIdx.x: the
// CTA whose tail piece starts the item; a warp takes every (gridDim.y * 8)-th
// of its rows.  Latency bounds it: two reads that wait for one another (the
// records; a row's (m, l) and first two pieces of O), with the next row's
// ahead.  It takes 4 us of a call for one token, 10 of one for prompts.
template <int D>
__global__ void __launch_bounds__(256) attention_join_kernel(const __grid_constant__ Params p, int ctas) {
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4 rec = p.record[blockIdx.x];
    // pieces: this CTA's tail, then the heads of the next ones
    int n = 1;
    for (bool more = true; more; n += 32) {
        const int e = blockIdx.x + n + lane;
        const int f = e < ctas ? p.record[e].x : 0;
        // the first CTA whose piece is not of the item, or is its last
        const uint32_t none = __ballot_sync(0xffffffffu, !(f & kHeadPiece));
        const uint32_t last = __ballot_sync(0xffffffffu, (f & kHeadPiece) && !(f & kHeadGoesOn));
        const int end_none = none ? __ffs(none) - 1 : 32, end_last = last ? __ffs(last) : 33;
        const int end = min(end_none, end_last);
        if (end <= 32 && (none | last)) {
            n += end - 32;
            more = false;
        }
    }
    if (!(rec.x & kTailPiece)) return;
    constexpr int kOwn = D / 32;
    using Own = typename std::conditional<kOwn == 4, float4, float2>::type;
    const int rows = rec.z <= p.tokens ? min(p.piece_rows, rec.z * p.group) : p.piece_rows, step = gridDim.y * 8;
    int row = blockIdx.y * 8 + warp;
    auto place = [&](int i, int r) { return ((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * p.piece_rows + r; };
    auto piece = [&](int i, int r) {
        return *reinterpret_cast<const Own *>(p.part + (int64_t)place(i, r) * D + lane * kOwn);
    };
    // an item that was cut has two pieces at least; the next row's are read
    // ahead
    Own v0{}, v1{};
    float2 ml0{};
    auto read = [&](int r) {
        if (r >= rows) return;
        v0 = piece(0, r), v1 = piece(1, r), ml0 = p.part_ml[place(min(lane, n - 1), r)];
    };
    read(row);
    for (; row < rows; row += step) {
        const int g = row / kTile, in_tile = row - g * kTile;
        const int in_token = in_tile / p.group, head = in_tile - in_token * p.group, token = g * p.tokens + in_token;
        const Own w0 = v0, w1 = v1;
        const float2 ml = ml0;
        read(row + step);
        if (in_token >= p.tokens || token >= rec.z) continue;
        float m = ml.x;
        for (int i = lane + 32; i < n; i += 32) m = fmaxf(m, p.part_ml[place(i, row)].x);
#pragma unroll
        for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
        const float base = m == -INFINITY ? 0.f : m;
        float acc[kOwn] = {}, l = 0.f;
        auto add = [&](const Own &v, float pm, float pl) {
            const float *o = reinterpret_cast<const float *>(&v);
            const float f = ex2(pm - base);
            l += pl * f;
#pragma unroll
            for (int e = 0; e < kOwn; ++e) acc[e] += o[e] * f;
        };
        add(w0, __shfl_sync(0xffffffffu, ml.x, 0), __shfl_sync(0xffffffffu, ml.y, 0));
        add(w1, __shfl_sync(0xffffffffu, ml.x, 1), __shfl_sync(0xffffffffu, ml.y, 1));
#pragma unroll 4
        for (int i = 2; i < n; ++i) {
            const float2 more_ml = p.part_ml[place(i, row)];
            add(piece(i, row), more_ml.x, more_ml.y);
        }
        const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
        const int64_t at = ((int64_t)rec.y + token) * p.q_heads + rec.w * p.group + head;
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
    // whole pages, or their largest power of two; at most 64 rows, so that
    // little of a tile is left to clear by hand
    p.box = gcd(c.page_size, 64);
    p.scale_log2 = a.scale * kLog2e;
    int exponent;
    const float mantissa = frexpf(p.scale_log2, &exponent);
    p.scale_pow2 = mantissa == 0.5f ? p.scale_log2 : ldexpf(1.f, exponent);
    p.scale_back = p.scale_log2 / p.scale_pow2;
    p.out = a.out, p.lse = a.lse, p.out_bf16 = a.out_bf16;
    p.max_q_len = a.max_q_len;
    // Where both kinds of item can meet, a key tile of two tiles takes about
    // 1.7 us and one of a narrow item 1.2.
    const bool mixed = a.max_q_len > p.tokens;
    p.cost[0] = mixed ? 2 : 1, p.cost[1] = mixed ? 3 : 1;
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
    const int blocks = (p.piece_rows + 7) / 8;  // a row a warp; past 8 blocks an item is slower (32: by 3 us)
    return launch_pdl(attention_join_kernel<D>, dim3(ctas, blocks < 8 ? blocks : 8), dim3(256), 0, s, p, ctas);
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
