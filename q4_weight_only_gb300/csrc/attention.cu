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
//   join, the rest reads that wait for one another.  (Of a row of such calls,
//   whose launches overlap, each takes 14.6.)
//
// A cache in Q4_0 blocks (attention_q4_wide_kernel; sequences of few rows are
// attention_q4.cu's).  The same warps, and four more: codes and scales come
// through a ring of their own, warps 12 to 15 unpack tiles of binary16 from it
// into the ring that the MMAs read, and the softmax warps turn their rows of Q
// to binary16.  p is binary16 too, held times 2^7 (kLift) as l and O are.  The
// copies are a quarter of the bytes; what bounds a tile is the unpacking and
// what it costs the others:
// * 8192 tokens after 8192 others take 1.56 ms, 1.32 PFLOP/s (of a row of
//   replayed calls; one call among others 1.59); 1.43 with the
//   unpacking left out, 1.36 without the copies too (timing only).  Its warps
//   work 2240 of a pair of tiles' 3600 cycles, their stores of 64 KB compete
//   with the MMAs' reads for shared memory, and their code with the softmax's
//   for the instruction caches: waits for instructions are 2.1 an issue under a
//   window, where they are 0.7 with the bfloat16 cache.  Three unpacking warps
//   in the copy warps' places took 3.28 ms; four that copied for themselves
//   1.94.
// * The windowed prompts at D = 64 take 187 us; 176 without unpacking and
//   copies.  Turning a Q to binary16, and its scores waiting for that, take 5000
//   cycles an item.
// * 5 drafted tokens of 16 sequences under a window of 4096: 61 us (bfloat16:
//   58), 39 without unpacking and copies.
// * Not faster: rings of 3 unpacked tiles and 6 of codes instead of 4 and 3 (D
//   = 64: 6 and 12 instead of 8 and 6; prompts 3 % slower, the others level); Q
//   turned by the unpacking warps (windowed prompts 193 -> 206 us, a prompt of
//   8192 1.56 -> 1.62 ms) or before the last item's output is written (197,
//   1.57); more registers for the copy warps (56 + 40 + 2 * 208; level).
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>
#include <type_traits>

#include "attention_plan.cuh"
#include "cache_q4.cuh"
#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr int kTile = 128;      // rows of a tile, and tokens of a key tile
// Threads and their registers.  The launch gives 168 each; the copy and MMA
// warps give theirs up to the softmax warps (128 * 56 + 256 * 224 = 384 *
// 168).  4 bits: warps 12 to 15 unpack a tile's four parts of 32 tokens (128 *
// (48 + 48) + 256 * 208 = 512 * 128).
template <bool kQ4>
struct Roles {
    static constexpr int kThreads = kQ4 ? 512 : 384;
    static constexpr int kRoleRegs = kQ4 ? 48 : 56, kUnpackRegs = 48, kSoftmaxRegs = kQ4 ? 208 : 224;
    static constexpr int kReaders = kQ4 ? 15 : 11;  // warps that read items
};
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;    // log2 of the growth of a row's maximum that moves its reference
// Every p of a row has 2^(the rounding of c m) as a factor.  Where c m is
// beyond this, that would leave fp32, and fp32 scores that differ are 64
// apart at least: the next power of two in the place of c gives the same
// p, 1 or nothing, without a rounding.
constexpr float kHuge = 1 << 30;
// binary16 holds less: below 2^26 the reference is off by at most 4, twice
// (rounded, and lifted), so p at most 2^15 where it is set, as by growth; a
// score's own rounding to fp32 is up to 4 in the exponent there.
constexpr float kHugeQ4 = 1 << 26;

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

// The same over a cache in Q4_0 blocks.
struct ParamsQ4 : Params {
    CacheQ4 cache;
    int least;  // sequences of fewer (token, head of the group) rows are another kernel's
};

__device__ __forceinline__ int items_of(const Params &p, const Sequence &s) {
    return (s.len + 2 * p.tokens - 1) / (2 * p.tokens);
}
__device__ __forceinline__ int items_of(const ParamsQ4 &p, const Sequence &s) {
    return s.len * p.group < p.least ? 0 : items_of(static_cast<const Params &>(p), s);
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

__device__ __forceinline__ int tile_cost(const Params &p, const Range &r) { return p.cost[r.tokens > p.tokens]; }

__device__ __forceinline__ int largest_cost(const Params &p) { return p.cost[1]; }

__device__ __forceinline__ int64_t item_cost(const Params &p, const Sequence &s, int item) {
    const Range r = item_range(p, s, item);
    return (int64_t)r.n * tile_cost(p, r);
}

// f(0), f(1), ... f(N - 1) with constants as arguments.
template <int N, typename F>
__device__ __forceinline__ void each_step(F &&f) {
    if constexpr (N > 0) {
        each_step<N - 1>(f);
        f(std::integral_constant<uint32_t, N - 1>{});
    }
}

template <int D, bool kQ4>
struct Layout {
    static constexpr int kHalves = D / 64;                 // 64-element column blocks
    static constexpr int kTileBytes = kTile * D * 2;
    static constexpr int kBlock = kTile * 128;             // bytes of one column block
    static constexpr int kStages = kQ4 ? (D == 128 ? 4 : 8) : (D == 128 ? 5 : 10);  // K or V tiles in the ring
    static constexpr int kCodeStages = D == 128 ? 3 : 6;                            // 4 bits: tiles' codes
    static constexpr int kQTiles = D == 128 ? 2 : 4;       // Q tiles held
    static constexpr int kQ = 0;
    static constexpr int kRing = kQTiles * kTileBytes;
    // 4 bits: the unpacking warps' code and the softmax's keep each other
    // waiting for instructions, so what can be is rolled.  At D = 128 masks are
    // a pass over S of their own (windowed prompts 300 -> 283 us; D = 64: 193 ->
    // 196), and only the unpacking, which bounds it, is straight-line code
    // (rolled: a prompt of 8192 1556 -> 1640; D = 64: 193 against 196).
    static constexpr bool kMaskPass = kQ4 && D == 128;
    static constexpr int kColumnsAtOnce = kQ4 ? 1 : 4;  // 32 columns of O
    // 4 bits: a ring of tiles' codes and scales
    static constexpr int kCodes = kRing + kStages * kTileBytes;
    static constexpr int kCodeRow = D / 2, kScaleRow = D / 16, kCodeBytes = kTile * (kCodeRow + kScaleRow);
    static constexpr int kBars = kCodes + (kQ4 ? kCodeStages * kCodeBytes : 0);
    static constexpr int kStatBytes = kQ4 ? 4096 : 2048;
    static constexpr int kSmem = kBars + kStatBytes + 1024;  // + alignment
};

// Items handed out ahead.  A warp that copies looks for the next item's tiles
// while it holds tiles of this one: the item that the next one takes the place
// of must not need them.
constexpr int kItems = 4;
static_assert(kItems >= 2, "");

constexpr int kMaxQTiles = 4;

template <int kStages, bool kQ4>
struct Bars {
    static constexpr int kMaxCodes = 6;
    uint64_t full[kStages], empty[kStages];
    uint64_t q_full[kMaxQTiles], q_empty[kMaxQTiles];
    uint64_t s_full[2], p_full[2], o_full[2];
    uint64_t b_done, merged;  // narrow items: B's O and (m, l) are ready; A has read them
    uint64_t item_full[kItems], item_empty[kItems];
    uint64_t drain;
    Item item[kItems];
    float2 ml[kTile];
    // 4 bits: the ring of codes, Q tiles turned to binary16 and what undoes
    // their rows' scaling
    uint64_t q_ready[kQ4 ? kMaxQTiles : 1];
    uint64_t codes_full[kQ4 ? kMaxCodes : 1], codes_empty[kQ4 ? kMaxCodes : 1];
    float q_down[kQ4 ? 2 : 1][kQ4 ? kTile : 1];
    uint32_t tmem;
    uint32_t fills[2], q_fills;  // copies made: past the last K and V tile's ring position, and of Q
    int abort;
    Start<Roles<kQ4>::kThreads> start;
};
static_assert(sizeof(Bars<10, false>) <= Layout<64, false>::kStatBytes, "");
static_assert(sizeof(Bars<8, true>) <= Layout<64, true>::kStatBytes, "");

// Tensor memory columns.
constexpr uint32_t kTmemCols = 512;
__device__ __forceinline__ uint32_t col_s(int g) { return g * 128; }
__device__ __forceinline__ uint32_t col_o(int g) { return 256 + g * 128; }

// A row of a Q tile to binary16 in place, times a power of two that brings its
// largest element to [2^14, 2^15): exact for every element within 2^29 of the
// largest, off by at most 2^-39 of that below.  Returns the power's inverse; a
// row of zeros or with an infinity or NaN is not scaled.
template <int D>
__device__ __forceinline__ float q_to_f16(uint8_t *tile, int block, int row) {
    uint32_t top2 = 0;  // as whole numbers, sizes of bfloat16 pairs are ordered
    auto at = [&](int i) {
        return reinterpret_cast<uint4 *>(tile + (i >> 3) * block + row * 128 + (((i & 7) ^ (row & 7)) << 4));
    };
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = *at(i);
        top2 = __vmaxu2(top2, __vmaxu2(__vmaxu2(v.x & 0x7FFF7FFFu, v.y & 0x7FFF7FFFu),
                                       __vmaxu2(v.z & 0x7FFF7FFFu, v.w & 0x7FFF7FFFu)));
    }
    const uint32_t top = max(top2 & 0xFFFFu, top2 >> 16);
    const int exponent = (int)(top >> 7);
    const int up = top && exponent < 255 ? min(14 + 127 - exponent, 100) : 0;
    const float f = __uint_as_float((uint32_t)(127 + up) << 23);
    auto turn = [&](uint32_t w) {
        return pack_f16(__uint_as_float(w << 16) * f, __uint_as_float(w & 0xFFFF0000u) * f);
    };
#pragma unroll 4
    for (int i = 0; i < D / 8; ++i) {
        const uint4 v = *at(i);
        *at(i) = make_uint4(turn(v.x), turn(v.y), turn(v.z), turn(v.w));
    }
    return __uint_as_float((uint32_t)(127 - up) << 23);
}

// P: Params, or ParamsQ4 for a cache in 4 bits: kmap and vmap are then of its
// codes, which warps 12 to 15 unpack into the ring of tiles.
template <int D, typename P>
__device__ __forceinline__ void attend(const CUtensorMap &qmap, const CUtensorMap &kmap, const CUtensorMap &vmap,
                                       const P &p) {
    constexpr bool kQ4 = std::is_same<P, ParamsQ4>::value;
    using L = Layout<D, kQ4>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    uint8_t *ring = smem + L::kRing;
    constexpr int kStages = L::kStages, kCodeStages = L::kCodeStages;
    Bars<kStages, kQ4> &bar = *reinterpret_cast<Bars<kStages, kQ4> *>(smem + L::kBars);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = &bar.abort;

    if (warp == 1) tmem_alloc(&bar.tmem, kTmemCols);
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[i], kQ4 ? kTile / 32 : 1);
            mbar_init(&bar.empty[i], 1);
        }
        for (int i = 0; kQ4 && i < kCodeStages; ++i) {
            mbar_init(&bar.codes_full[i], 1 + 32);  // the codes' bytes, and each lane's scales
            mbar_init(&bar.codes_empty[i], kTile / 32);
        }
        for (int i = 0; i < L::kQTiles; ++i) {
            mbar_init(&bar.q_full[i], 1);
            mbar_init(&bar.q_empty[i], 1);
            if (kQ4) mbar_init(&bar.q_ready[i], 4);
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
            mbar_init(&bar.item_empty[i], Roles<kQ4>::kReaders);
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
    locate<Roles<kQ4>::kThreads>(p, bar.start, blockIdx.x, gridDim.x);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = bar.tmem;

    // The next item of the share, or false at its end or when a wait was
    // abandoned; done_item() hands its record back.  4 bits: the record is
    // read where it lies, a copy of it would spill other registers.
    uint32_t items = 0;
    Item copy;
    auto item = [&]() -> const Item & {
        if constexpr (kQ4) return bar.item[items % kItems];
        return copy;
    };
    auto next_item = [&]() {
        const int i = items % kItems;
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.item_full[i], items / kItems & 1, abort_flag, p.err))) return false;
        if constexpr (!kQ4) copy = bar.item[i];
        return item().t0 < item().t1;
    };
    auto done_item = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.item_empty[items % kItems]);
        ++items;
    };

    // Warp 3 hands out the items.
    struct Publisher {
        int64_t left;
        int flags, head, b, it, t0, n_items;
        uint32_t count;
        int4 tail;
        Sequence s;
    };
    auto publisher = [&]() {
        return Publisher{bar.start.left, 0, bar.start.head, bar.start.b, bar.start.item, bar.start.t0,
                         items_of(p, bar.start.s), 0, make_int4(0, 0, 0, 0), bar.start.s};
    };
    // The next one, or one without tiles at the share's end; false after that
    // and when a wait was abandoned.
    auto publish = [&](Publisher &w) {
        Item o{};
        int64_t cost = 0;
        if (w.left > 0) {
            const Range r = item_range(p, w.s, w.it);
            const int each = tile_cost(p, r);
            cost = (int64_t)r.n * each;
            o.t0 = w.t0, o.t1 = w.left >= cost ? r.n : (int)(w.left / each), o.n = r.n;
            o.head = w.head, o.b = w.b, o.row0 = w.s.row0 + w.it * 2 * p.tokens, o.tokens = r.tokens, o.pos0 = r.pos0;
            o.lo = r.lo, o.hi = r.hi, o.sink_end = r.sink_end, o.sink_tiles = r.sink_tiles, o.wtile = r.wtile;
            if (o.t0 > 0) w.flags |= kHeadPiece | (o.t1 < o.n ? kHeadGoesOn : 0);
            if (o.t0 == 0 && o.t1 > 0 && o.t1 < o.n)
                w.flags |= kTailPiece, w.tail = make_int4(0, o.row0, o.tokens, w.head);
        }
        const int i = w.count % kItems;
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.item_empty[i], (w.count / kItems & 1) ^ 1, abort_flag, p.err)))
            return false;
        if (lane == 0) {
            bar.item[i] = o;
            mbar_arrive(&bar.item_full[i]);
        }
        __syncwarp();
        ++w.count;
        w.left -= cost;
        if (o.t0 == o.t1) return false;
        w.t0 = 0;
        if (w.left > 0 && ++w.it >= w.n_items) {
            w.it = 0;
            int scanned = 0;
            do {
                if (++w.b >= p.sequences) {
                    w.b = 0;
                    ++w.head;
                }
                w.s = sequence(p, w.b);
                w.n_items = items_of(p, w.s);
            } while (w.n_items == 0 && ++scanned <= p.sequences);
        }
        return true;
    };
    auto publish_end = [&](Publisher &w) {
        w.tail.x = w.flags;
        if (lane == 0) p.record[blockIdx.x] = w.tail;
    };
    // A tile of Q into its slot, when there is room.
    auto load_q = [&](uint32_t q, int head, int row0) {
        const int at = q % L::kQTiles;
        if (!__all_sync(0xffffffffu, mbar_wait(&bar.q_empty[at], (q / L::kQTiles & 1) ^ 1, abort_flag, p.err)))
            return false;
        if (elect_one()) {
            mbar_arrive_expect_tx(&bar.q_full[at], L::kHalves * p.tokens * p.group * 128);
            for (int h = 0; h < L::kHalves; ++h)
                tma_load_4d(smem + L::kQ + at * L::kTileBytes + h * L::kBlock, &qmap, h * 64, 0, head, row0,
                            &bar.q_full[at]);
        }
        __syncwarp();
        return true;
    };

    // 4 bits.  Warp 12 + i unpacks part i, tokens 32 i to 32 i + 31, of every
    // tile from the ring of codes to the ring of tiles.  A lane has a token: a
    // store is then 16 bytes of 32 rows, which the tiles' swizzle spreads over
    // the banks.
    auto unpack = [&]() {
        if constexpr (kQ4) {
            const int row = (warp - 12) * 32 + lane;
            const uint32_t bias = p.cache.bias, codes = smem_u32(smem + L::kCodes), tiles = smem_u32(ring) + row * 128;
            const int turn = D == 128 ? row >> 1 & 3 : row >> 2 & 1;  // the swizzle of a row of codes
            constexpr int kBlocksAtOnce = D == 128 ? 4 : 1;  // of a token
            uint32_t from = 0, from_phase = 0, slot = 0, phase = 1;
            bool ok = true;
            for (; ok && next_item(); done_item()) {
                for (int n = 2 * (item().t1 - item().t0); n > 0; --n) {
                    ok = __all_sync(0xffffffffu, mbar_wait(&bar.codes_full[from], from_phase, abort_flag, p.err) &&
                                                     mbar_wait(&bar.empty[slot], phase, abort_flag, p.err));
                    if (!ok) break;
                    const uint32_t src = codes + from * L::kCodeBytes;
                    uint2 d;
                    if (D == 128)
                        d = lds64(src + kTile * L::kCodeRow + row * 8);
                    else
                        d.x = d.y = lds32(src + kTile * L::kCodeRow + row * 4);
                    const uint32_t dst = tiles + slot * L::kTileBytes, blocks = src + row * L::kCodeRow;
                    uint4 next = lds128(blocks + turn * 16);
#pragma unroll kBlocksAtOnce
                    for (int j = 0; j < D / 32; ++j) {
                        const uint4 x = next;
                        // (no load passes the stores below)
                        if (j + 1 < D / 32) next = lds128(blocks + ((j + 1) ^ turn) * 16);
                        const __half2 scale = as_half2(__byte_perm(j & 2 ? d.y : d.x, 0, j & 1 ? 0x3232 : 0x1010));
                        const uint32_t at = dst + (j >> 1) * L::kBlock, chunk = (j & 1) * 4;
                        const uint32_t words[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            // eight bytes: elements 8h .. 8h + 7 of the block and 16 further
                            uint32_t lo[4], hi[4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const uint32_t w = __byte_perm(words[2 * h + i / 2], 0, i & 1 ? 0x4342 : 0x4140);
                                lo[i] = times(low_codes(w, bias), scale), hi[i] = times(high_codes(w, bias), scale);
                            }
                            sts128(at + (((chunk + h) ^ (row & 7)) * 16), lo);
                            sts128(at + (((chunk + h + 2) ^ (row & 7)) * 16), hi);
                        }
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        mbar_arrive(&bar.full[slot]);
                        mbar_arrive(&bar.codes_empty[from]);
                    }
                    if (++from == kCodeStages) from = 0, from_phase ^= 1;
                    if (++slot == kStages) slot = 0, phase ^= 1;
                }
                if (!ok) break;
            }
        }
    };

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Roles<kQ4>::kRoleRegs));
        if (warp == 0 || warp == 2) {
            // ------------------------------------------------ copies
            // K and V tiles (4 bits: their codes and scales) alternate in one
            // ring; each warp fills its own.
            // A warp may not be two uses of a slot ahead (its wait would take
            // the older phase for the newer): the MMA warp frees tiles in an
            // order in which the slot of fill f - 7, waited for at fill
            // f - 2, is freed after that of f - 10.
            const int kv = warp >> 1;  // warp 0: Q and K, warp 2: V
            constexpr int kRingStages = kQ4 ? kCodeStages : kStages;
            uint64_t *const full = kQ4 ? bar.codes_full : bar.full, *const empty = kQ4 ? bar.codes_empty : bar.empty;
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
                int clip;                  // 4 bits: tokens [0, a) and [b, e) of the box are seen, 7 bits each
            };
            int t = 0;
            uint32_t q = 0;  // Q tiles copied
            bool open = false;  // an item is held with tiles from t on
            auto fetch = [&]() {
                Group o{};
                if (!open) {
                    if (!next_item()) return o;
                    open = true;
                    t = item().t0;
                    if (!kQ4) o.row0 = item().row0, o.tokens = item().tokens;
                }
                o.head = item().head;
                o.tiles = min(per_load, item().t1 - t);
                o.off = -1;
                const int mine = lane / boxes;
                if (mine < o.tiles) {
                    const int tok = item().key_tile(t + mine) * kTile + (lane - mine * boxes) * p.box;
                    // only boxes that hold a token some query sees
                    if (tok < item().sink_end || (tok < item().hi && tok + p.box > item().lo)) {
                        const int index = tok / p.page_size;
                        o.page = p.page_table[(int64_t)item().b * p.table_stride + index];
                        o.off = tok - index * p.page_size;
                        if (kQ4) {
                            const int a = min(max(item().sink_end - tok, 0), p.box);
                            const int b = max(item().lo - tok, 0), e = min(item().hi - tok, p.box);
                            o.clip = a | min(b, p.box) << 7 | e << 14;
                        }
                    }
                }
                t += o.tiles;
                if (t == item().t1) {
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
                    ok = __all_sync(0xffffffffu, mbar_wait(&empty[slot], phase, abort_flag, p.err));
                    if (!ok) break;
                    const bool issue = elect_one();
                    uint8_t *dst = kQ4 ? smem + L::kCodes + slot * L::kCodeBytes : ring + slot * L::kTileBytes;
                    if (issue) mbar_arrive_expect_tx(&full[slot], kQ4 ? kTile * L::kCodeRow : L::kTileBytes);
                    if constexpr (kQ4) {
                        // Scales of the tokens that some query sees.  Others'
                        // become zeros: their values may be anything (0 *
                        // NaN).
                        const KvQ4View &c = p.cache.c;
                        const int64_t *st = kv ? c.v_scale_stride : c.k_scale_stride;
                        const uint16_t *base = (kv ? c.v_scale : c.k_scale) + now.head * st[1];
                        const uint32_t to = smem_u32(dst) + kTile * L::kCodeRow;
                        const int shift = __ffs(p.box) - 1;
#pragma unroll 1
                        for (int t = lane; t < kTile; t += 32) {
                            const int box = t >> shift, in_box = t & (p.box - 1);
                            const int page = __shfl_sync(0xffffffffu, now.page, j * boxes + box);
                            const int off = __shfl_sync(0xffffffffu, now.off, j * boxes + box) + in_box;
                            const int clip = __shfl_sync(0xffffffffu, now.clip, j * boxes + box);
                            const bool in_window = in_box >= (clip >> 7 & 127) && in_box < clip >> 14;
                            const bool seen = page < p.pages && (in_box < (clip & 127) || in_window);
                            copy_small<L::kScaleRow>(to + t * L::kScaleRow,
                                                     base + (seen ? page * st[0] + off * st[2] : 0), !seen);
                        }
                        copy_arrive(&full[slot]);
                    }
                    for (int i = 0; i < boxes; ++i, dst += p.box * (kQ4 ? L::kCodeRow : 128)) {
                        const int page = __shfl_sync(0xffffffffu, now.page, j * boxes + i);
                        const int off = __shfl_sync(0xffffffffu, now.off, j * boxes + i);
                        if (issue) {
#pragma unroll
                            for (int h = 0; h < (kQ4 ? 1 : L::kHalves); ++h)
                                tma_load_4d(dst + h * L::kBlock, map, h * 64, off, now.head, page, &full[slot]);
                        }
                    }
                    __syncwarp();
                    fill += 2;
                    slot += 2;
                    if (slot >= kRingStages) slot -= kRingStages, phase ^= 1;
                    // an item's Q after its first K tile: Q waits for room
                    for (; !kQ4 && kv == 0 && now.tokens > 0; now.tokens -= p.tokens, now.row0 += p.tokens) {
                        ok = load_q(q, now.head, now.row0);
                        if (!ok) break;
                        ++q;
                    }
                    if (!ok) break;
                }
                now = then;
            }
            if (lane == 0) {
                bar.fills[kv] = fill;
                if (!kQ4 && kv == 0) bar.q_fills = q;
            }
        } else if (warp == 3) {
            // ------------------------------------------------- items
            Publisher w = publisher();
            if constexpr (kQ4) {
                // and copies each item's Q, with the next item handed out:
                // the copying warps have no registers for it
                uint32_t q = 0;
                bool ok = true, more = publish(w);
                for (uint32_t i = 0; ok && bar.item[i % kItems].t0 < bar.item[i % kItems].t1; ++i) {
                    if (more) more = publish(w);
                    const Item &o = bar.item[i % kItems];
                    for (int done = 0; ok && done < o.tokens; done += p.tokens) {
                        ok = load_q(q, o.head, o.row0 + done);
                        q += ok;
                    }
                }
                if (lane == 0) bar.q_fills = q;
            } else {
                while (publish(w)) {}
            }
            publish_end(w);
        } else if (warp == 1) {
        // ------------------------------------------------------ MMAs
        constexpr uint32_t idesc_qk = kQ4 ? idesc_f16_f32(kTile, kTile) : idesc_bf16_f32(kTile, kTile, false);
        constexpr uint32_t idesc_pv = kQ4 ? idesc_f16_f32(kTile, D, true) : idesc_bf16_f32(kTile, D, true);
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
        auto q_full = [&](uint32_t qt) {
            return wait(kQ4 ? &bar.q_ready[qt % L::kQTiles] : &bar.q_full[qt % L::kQTiles], qt / L::kQTiles & 1);
        };
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
        // (4 bits: their scales were copied as zeros.)
        auto clear_unseen = [&](int t, int slot) {
            if (kQ4) return;
            const int tok0 = item().key_tile(t) * kTile;
            const int sink = item().sink_end - tok0, lo = item().lo - tok0, hi = item().hi - tok0;
            if (hi >= kTile && (lo <= 0 || sink >= kTile)) return;
            const int mask = ~(p.box - 1);  // a power of two
            if (sink > 0 && sink < kTile) clear_rows(slot, sink, min((sink - 1 & mask) + p.box, max(lo, sink)));
            if (lo > 0 && lo < kTile) clear_rows(slot, max(lo & mask, max(sink, 0)), lo);
            if (hi > 0 && hi < kTile) clear_rows(slot, hi, (hi - 1 & mask) + p.box);
            fence_proxy_async_smem();
            __syncwarp();
        };
        for (; ok && next_item(); done_item()) {
            const bool wide = item().tokens > p.tokens;
            const int n = item().t1 - item().t0;
            if (!q_full(q)) break;
            if (wide) {
                uint32_t slot_k = fills % kStages, slot_v = (fills + 1) % kStages;
                if (!full(fills) || (!kQ4 && !q_full(q + 1))) break;
                tc_fence_after();
                if constexpr (kQ4) {
                    // group B turns its Q to binary16 when it is done with the
                    // last item: A does not wait for that
                    if (elect_one()) scores(0, q, slot_k, n == 1);
                    __syncwarp();
                    if (!q_full(q + 1)) break;
                    tc_fence_after();
                }
                if (elect_one()) {
                    if (!kQ4) scores(0, q, slot_k, n == 1);
                    scores(1, q + 1, slot_k, n == 1);
                    mma_commit(&bar.empty[slot_k]);
                }
                __syncwarp();
                for (int t = 0; t < n; ++t) {
                    const uint32_t v = fills + 2 * t + 1;
                    const bool more = t + 1 < n;
                    slot_v = v % kStages, slot_k = (v + 1) % kStages;
                    if (!full(v)) break;
                    clear_unseen(item().t0 + t, slot_v);
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
                    clear_unseen(item().t0 + t, v % kStages);
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
    } else if (kQ4 && warp >= 12) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Roles<kQ4>::kUnpackRegs));
        unpack();
    } else {
        // --------------------------------------------------- softmax
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Roles<kQ4>::kSoftmaxRegs));
        const int g = (warp - 4) >> 2;                 // group
        const int quad = warp & 3;                     // its tensor-memory lanes
        const int row = quad * 32 + lane;              // row of the tile
        const uint32_t lanes = (uint32_t)(quad * 32) << 16;
        const uint32_t ts = tmem + lanes + col_s(g), to = tmem + lanes + col_o(g);
        const int my_token = row / p.group;
        uint32_t s_phase = 0, o_phase = 0, q_tiles = 0;
        bool ok = true;
        auto wait = [&](uint64_t *b, uint32_t parity) {
            ok = __all_sync(0xffffffffu, mbar_wait(b, parity, abort_flag, p.err));
            return ok;
        };
        uint32_t merge_phase = 0;
        bool unmerged = false;  // group B: A may not have read O of the last item yet
        for (; ok && next_item(); done_item()) {
            const bool wide = item().tokens > p.tokens;
            const int half = wide ? g : 0;                  // the tile of the item
            const int i = half * p.tokens + my_token;       // token within the item
            const bool valid = my_token < p.tokens && i < item().tokens;
            const bool busy = __any_sync(0xffffffffu, valid);
            const int pos = item().pos0 + i;
            const int step = wide ? 1 : 2;
            if constexpr (kQ4) {
                // the group's tile of Q to binary16; a narrow item's is group A's
                const uint32_t qt = q_tiles + half, at = qt % L::kQTiles, parity = qt / L::kQTiles & 1;
                q_tiles += wide ? 2 : 1;
                if (wide || g == 0) {
                    if (!wait(&bar.q_full[at], parity)) break;
                    uint8_t *tile = smem + L::kQ + at * L::kTileBytes;
                    bar.q_down[half][row] = valid ? q_to_f16<D>(tile, L::kBlock, row) : 1.f;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bar.q_ready[at]);
                } else if (!wait(&bar.q_ready[at], parity)) {
                    break;
                }
            }
            // scale * log2 e, and the next power of two, for the row as it is
            auto c_of = [&](float scale) { return kQ4 ? in_range(scale * bar.q_down[half][row]) : scale; };
            // A row whose maximum grew moves the references of its warp's
            // rows (each its own, one by one, took prompts 1 to 4 % longer).
            // Lanes that are no row of the item must not: they hold other
            // sequences' rows, or what an earlier kernel left in shared
            // memory.  Nothing is above their reference.
            float mc = valid ? -INFINITY : INFINITY, c_row = c_of(p.scale_log2), l = 0.f;
            bool started = false;
            for (int t = item().t0 + (wide ? 0 : g); t < item().t1; t += step) {
                if (!wait(&bar.s_full[g], s_phase)) break;
                s_phase ^= 1;
                tc_fence_after();
                if (busy) {
                    // whether some query of the tile does not see some key,
                    // and which of keys 32 q to 32 q + 31 this row sees
                    auto cut = [&](int tok0) {
                        // positions of the tile's first and last query
                        const int pos_a = item().pos0 + half * p.tokens;
                        const int pos_z = item().pos0 + min((half + 1) * p.tokens, item().tokens) - 1;
                        return tok0 + kTile - 1 > pos_a ||
                               (p.window && tok0 <= pos_z - p.window && tok0 + kTile > p.sinks);
                    };
                    auto seen_of = [&](int tok0, int q) {
                        const int end = pos + 1 - tok0;
                        const int first = p.window ? end - p.window : 0;
                        const int sink = p.sinks - tok0;
                        return below(end - q * 32) & (~below(first - q * 32) | below(sink - q * 32));
                    };
                    if constexpr (L::kMaskPass) {
                        const int tok0 = item().key_tile(t) * kTile;
                        if (cut(tok0)) {
#pragma unroll 1
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t seen = seen_of(tok0, q);
                                if (__all_sync(0xffffffffu, seen == ~0u)) continue;
                                uint32_t v[32];
                                tmem_ld32(ts + q * 32, v);
                                tmem_wait_ld();
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(seen >> e & 1)) v[e] = 0xFF800000u;
                                tmem_st32(ts + q * 32, v);
                            }
                            tmem_wait_st();
                        }
                    }
                    uint32_t s[4][32];
#pragma unroll
                    for (int q = 0; q < 4; ++q) tmem_ld32(ts + q * 32, s[q]);
                    tmem_wait_ld();
                    if constexpr (!L::kMaskPass) {
                        const int tok0 = item().key_tile(t) * kTile;
                        if (cut(tok0)) {
#pragma unroll
                            for (int q = 0; q < 4; ++q) {
                                const uint32_t seen = seen_of(tok0, q);
#pragma unroll
                                for (int e = 0; e < 32; ++e)
                                    if (!(seen >> e & 1)) s[q][e] = 0xFF800000u;
                            }
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
                    // 4 bits: references are kLift below the maximum, p that
                    // much larger
                    constexpr float lift = kQ4 ? kLift : 0.f;
                    // (nothing is above an infinite reference)
                    if (__any_sync(0xffffffffu, fmaf(top, c_row, -mc) > kGrow + lift)) {
                        const float c = c_of(p.scale_log2);
                        const float c_top = fabsf(top * c) > (kQ4 ? kHugeQ4 : kHuge) ? c_of(p.scale_pow2) : c;
                        float mc_new = __fmul_rn(top, c_top);
                        if (kQ4) mc_new = __fsub_rn(mc_new, lift);
                        const bool above = mc_new > mc;
                        const float f = mc == -INFINITY ? 0.f : above ? ex2(mc - mc_new) : 1.f;
                        l *= f;
                        if (above) mc = mc_new, c_row = c_top;
                        if (started) {
                            // O of the earlier tiles is complete: scale it
                            if (!wait(&bar.o_full[g], o_phase ^ 1)) break;
                            tc_fence_after();
#pragma unroll L::kColumnsAtOnce
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
                            w[e] = kQ4 ? pack_f16(a, b) : pack_bf16(a, b);
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
            mc *= c_row == c_of(p.scale_log2) ? 1.f : p.scale_back;
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
                const bool both = !wide && item().t1 - item().t0 > 1;
                if (busy) {
                    const bool whole = item().t0 == 0 && item().t1 == item().n;
                    const int my_head = row - my_token * p.group;
                    const int64_t at = ((int64_t)item().row0 + i) * p.q_heads + item().head * p.group + my_head;
                    const int piece = blockIdx.x * 2 + (item().t0 == 0 ? 1 : 0);
                    const int prow = piece * p.piece_rows + half * kTile + row;
                    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
                    if (whole) fa *= inv, fb *= inv;
#pragma unroll L::kColumnsAtOnce
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
        constexpr uint32_t kRingStages = kQ4 ? kCodeStages : kStages;
        for (uint32_t i = 0; i < kRingStages; ++i) {
            int last = -1;
            for (uint32_t f = i; f < max(bar.fills[0], bar.fills[1]); f += kRingStages)
                if (f < bar.fills[f & 1]) last = f;
            if (last >= 0) mbar_drain(kQ4 ? &bar.codes_full[i] : &bar.full[i], last / kRingStages & 1);
        }
        for (uint32_t f = max(bar.q_fills, (uint32_t)L::kQTiles) - L::kQTiles; f < bar.q_fills; ++f)
            mbar_drain(&bar.q_full[f % L::kQTiles], f / L::kQTiles & 1);
    }
    if (warp == 1) tmem_dealloc(tmem, kTmemCols);
}

template <int D>
__global__ void __launch_bounds__(Roles<false>::kThreads, 1)
    attention_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                     const __grid_constant__ CUtensorMap vmap, const __grid_constant__ Params p) {
    attend<D>(qmap, kmap, vmap, p);
}

template <int D>
__global__ void __launch_bounds__(Roles<true>::kThreads, 1)
    attention_q4_wide_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                             const __grid_constant__ CUtensorMap vmap, const __grid_constant__ ParamsQ4 p) {
    attend<D>(qmap, kmap, vmap, p);
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

// What the kernels of both caches take; View: KvCacheView or KvQ4View.
template <int D, typename View>
void fill_params(Params &p, const AttentionArgs &a, const View &c, void *workspace, int ctas, unsigned int *err) {
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
    // 1.7 us and one of a narrow item 1.2.  (Read from L2, 1.57 and 1.00, at D =
    // 64 1.27 and 0.81.  In 4 bits, where both are unpacked whole, the two are
    // nearer to one another: 1.79 and 1.40, 1.59 and 1.16.)
    const bool mixed = a.max_q_len > p.tokens;
    p.cost[0] = mixed ? 2 : 1, p.cost[1] = mixed ? 3 : 1;
    p.piece_rows = item_rows(p.group, a.max_q_len);
    const WorkspaceLayout w(ctas, D, p.piece_rows);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.part = reinterpret_cast<float *>(ws);
    p.part_ml = reinterpret_cast<float2 *>(ws + w.ml_off);
    p.record = reinterpret_cast<int4 *>(ws + w.rec_off);
    p.err = err;
}

// q as {element, head of the group, key head, row}
template <int D>
bool make_q_map(EncodeTiledFn enc, CUtensorMap *map, const AttentionArgs &a, const Params &p) {
    return make_map(enc, map, a.q, {D, p.group, p.kv_heads, a.rows},
                    {a.q_head_stride, a.q_head_stride * p.group, a.q_row_stride}, p.group, p.tokens);
}

template <int D>
cudaError_t launch_join(const Params &p, int ctas, cudaStream_t s) {
    const int blocks = (p.piece_rows + 7) / 8;  // a row a warp; past 8 blocks an item is slower (32: by 3 us)
    return launch_pdl(attention_join_kernel<D>, dim3(ctas, blocks < 8 ? blocks : 8), dim3(256), 0, s, p, ctas);
}

template <int D>
cudaError_t launch_d(const AttentionArgs &a, const KvCacheView &c, void *workspace, int ctas, cudaStream_t s,
                     unsigned int *err) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    Params p{};
    fill_params<D>(p, a, c, workspace, ctas, err);
    CUtensorMap qmap, kmap, vmap;
    if (!make_q_map<D>(enc, &qmap, a, p)) return cudaErrorInvalidValue;
    // k and v as {element, token of the page, key head, page}
    if (!make_map(enc, &kmap, c.k, {D, c.page_size, c.kv_heads, c.pages},
                  {c.k_stride[2], c.k_stride[1], c.k_stride[0]}, p.box, 1) ||
        !make_map(enc, &vmap, c.v, {D, c.page_size, c.kv_heads, c.pages},
                  {c.v_stride[2], c.v_stride[1], c.v_stride[0]}, p.box, 1))
        return cudaErrorInvalidValue;
    constexpr int kSmem = Layout<D, false>::kSmem;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(attention_kernel<D>), kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attention_kernel<D>, dim3(ctas), dim3(Roles<false>::kThreads), kSmem, s, qmap, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    return launch_join<D>(p, ctas, s);
}

template <int D>
cudaError_t launch_q4_d(const AttentionArgs &a, const KvQ4View &c, int least, void *workspace, int ctas, cudaStream_t s,
                        unsigned int *err) {
    EncodeTiledFn enc = encode_fn();
    if (!enc) return cudaErrorNotSupported;
    ParamsQ4 p{};
    fill_params<D>(p, a, c, workspace, ctas, err);
    p.cache = cache_q4(c);
    p.least = least;
    CUtensorMap qmap, kmap, vmap;
    if (!make_q_map<D>(enc, &qmap, a, p) || !make_codes_map(enc, &kmap, c.k, c.k_stride, c, p.box) ||
        !make_codes_map(enc, &vmap, c.v, c.v_stride, c, p.box))
        return cudaErrorInvalidValue;
    constexpr int kSmem = Layout<D, true>::kSmem;
    cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(attention_q4_wide_kernel<D>), kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(attention_q4_wide_kernel<D>, dim3(ctas), dim3(Roles<true>::kThreads), kSmem, s, qmap, kmap, vmap, p);
    if (e != cudaSuccess) return e;
    return launch_join<D>(p, ctas, s);
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

cudaError_t launch_attention_q4_wide(const AttentionArgs &a, const KvQ4View &c, int least, void *workspace,
                                     cudaStream_t s, unsigned int *err) {
    const int sms = current_sms();
    if (sms < 1) return cudaErrorInvalidDevice;
    return c.head_dim == 128 ? launch_q4_d<128>(a, c, least, workspace, sms, s, err)
                             : launch_q4_d<64>(a, c, least, workspace, sms, s, err);
}

}  // namespace q4_0
