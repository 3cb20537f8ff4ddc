// attention_q4.cu -- causal attention over a paged cache in Q4_0 blocks
// (declared in include/q4_0.h).
//
// Mathematics, for a query row at position t and the keys j it sees
// (j <= t, and j > t - window or j < sinks): with a running reference m,
//   p_j = 2^(c (s_j - m)),  l = sum p_j,  O = sum p_j v_j,  out = O / l,
// s_j = q . k_j, c = scale * log2 e, all of s, m, l and O in fp32.  The
// reference follows the running maximum only when a row's maximum grew by more
// than 2^8 in p: the result does not depend on it, and most steps then skip the
// correction of O.  The difference s - m is made before the product with c: a
// certain key has p = 1 exactly.  p, l and O are held times 2^7 (kLift).
//
// Operands of the tensor cores are binary16:
// * a key's codes, exactly, as the numbers below binary16's normal range that
//   their bits are where they lie; its blocks' scales multiply the blocks' dot
//   products in fp32, and one more product takes the codes' 8 too many off (as
//   two binary16 parts, 2^-23 of what they hold);
// * a value d (code - 8), rounded (2^-11): the format holds elements up to
//   65504;
// * a query row times a power of two that brings its largest element to
//   [2^14, 2^15), undone in c: exact for every element within 2^31 of the
//   largest, off by at most 2^-39 of that below; elements that meet high
//   nibbles, read as 16 codes, a sixteenth of that: exact within 2^27, off by at
//   most 2^-35 below;
// * p, at most 2^8, times 2^7, rounded (2^-11 of p, and 2^-32 where p is below
//   2^-21); l sums it before the rounding.
//
// Two kernels.  Sequences of few rows, (token, head of the group) pairs, are this
// file's: at most 8 in a call whose bound is above 16 and whose groups have at
// most 8 heads, else at most 16 (item_rows).  Their rows are the narrow operand
// of m16n8k16 products with the keys and values as the wide one, which warps
// unpack straight from the codes into their registers.  Nothing unpacked is
// written anywhere, and a tcgen05 operand in shared memory is not worth it for
// codes that so few rows use: 64 sequences' next tokens take twice as long there
// (353 and 700 us).  Longer sequences fill tcgen05's tiles of 128 rows and are
// attention.cu's 4-bit variant: 16 sequences' 5 drafted tokens by 5 heads, 25
// rows each, take 61 us there, and 85 as two items of 16 here.
//
// Layout of work: an item is 8 or 16 rows of one sequence and key head, its
// cost the key tiles it sees; CTAs, one an SM, take equal shares of all cost,
// and attention_q4_join_kernel adds what a share's boundary cut, in share
// order.
//
// Bounds and measurements (40 query heads on 8 key heads of 128, device time):
// * 64 sequences' next tokens, 4 to 32 thousand tokens each, 1.29 GB: 353 us,
//   3.6 TB/s, 0.55 of a copy's rate, where the bfloat16 cache takes 662.  Copies
//   alone take 241 us and the arithmetic alone 258: 400 warp instructions for
//   16 keys and values fill 60 % of the issue slots (logic and integers 49 %
//   of their pipe, multiply-adds 36 %, tensor 20 %, HBM 50 %).
// * 16 sequences of 1 to 8 thousand, 98 MB: 41 us (bfloat16: 68), of which 12
//   are the launches, the first reads and the join.
// * One token after 2047: 11.7 us (bfloat16: 14.8).
// * Pages that hold a head's tokens in a row are 12 % faster than pages that
//   hold a token's heads in a row: a token's scales of one head are 8 bytes,
//   and a sector of 32 holds four tokens' of the head then (605 against 807 MB
//   into the SMs for 32 sequences of 16384; 155 against 177 us).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cmath>
#include <type_traits>

#include "attention_plan.cuh"
#include "cache_q4.cuh"
#include "q4_0_internal.h"
#include "q4_0_ptx.cuh"

namespace q4_0 {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kGrow = 8.f;  // log2 of the growth of a row's maximum that moves its reference
constexpr int kTile = 128;    // tokens of a key tile
constexpr int kStep = 32;     // keys of a warp's part of one
// A nibble that is left where it is, in the low bits of a binary16, is a
// number below its normal range: code / kCodeUnit, exactly.
constexpr float kCodeUnit = 16777216.f;
// What the codes' 8 too many come to in a block, -8 sum q, is held as two
// binary16 parts in a unit of its own: at most 2^15, and what the two leave out
// is 2^-23 of it.  In the unit of the codes the second part would mostly be
// below binary16's normal range, where 2^-25 is lost of it whatever the block
// holds: beside an element a thousand times the rest, 2^-12 of the other
// blocks' sum |q k|.  Undoing it costs 8 multiplications a tile of 8 rows in
// 400 instructions (32 single tokens of 16384: 151.6 -> 153.0 us; sums that
// start from -8 sum q in fp32 instead of zeros are as good and need no such
// product, but four registers a block: 154.6, and 69 -> 90 with 16 heads of 128
// on one).
constexpr float kLessUnit = 65536.f;

struct Params {
    CacheQ4 cache;
    // the batch, as sequence() reads it
    const int32_t *page_table, *q_start, *kv_len;
    int64_t table_stride;
    int sequences, table_width, pages, page_size, rows, max_q_len;
    int q_heads, kv_heads, group, window, sinks;
    int most_rows;              // of a sequence; longer ones are another kernel's
    int step_pages, step_rest;  // kCopyTurns tiles by page_size
    int item_rows;              // rows of an item: (token, head of the group) pairs of a sequence, in order
    const __nv_bfloat16 *q;
    int64_t q_row_stride, q_head_stride;
    float scale_log2;
    void *out;
    float *lse;
    int out_bf16;
    float *part;       // [CTA][head piece, tail piece][item_rows][D], unnormalised
    float4 *part_mlc;  // the rows' m, l and c
    // per CTA: flags, then first row (token * group + head), rows and key head
    // of the tail piece's item
    int4 *record;
    unsigned int *err;
};

__device__ __forceinline__ int items_of(const Params &p, const Sequence &s) {
    return s.len * p.group > p.most_rows ? 0 : (s.len * p.group + p.item_rows - 1) / p.item_rows;
}

// The tokens the rows of an item see, [0, sink_end) and [lo, hi), and the key
// tiles that hold them: `sink_tiles` from token 0, then from tile `wtile`.
struct Range {
    int row0, rows;   // the item's first row within the sequence, and its rows
    int first, last;  // positions of its first and last row
    int lo, hi, sink_end;
    int sink_tiles, wtile, n;
};

__device__ __forceinline__ Range item_range(const Params &p, const Sequence &s, int item) {
    Range r;
    r.row0 = item * p.item_rows;
    r.rows = min(p.item_rows, s.len * p.group - r.row0);
    r.first = s.kv - s.len + r.row0 / p.group;
    r.last = s.kv - s.len + (r.row0 + r.rows - 1) / p.group;
    r.hi = max(r.last + 1, 0);
    r.lo = p.window ? min(max(r.first - p.window + 1, 0), r.hi) : 0;
    r.sink_end = min(p.sinks, r.lo);
    r.wtile = r.lo / kTile;
    r.sink_tiles = min((r.sink_end + kTile - 1) / kTile, r.wtile);
    // rows that see nothing still need their output: one empty tile
    r.n = max(r.sink_tiles + (r.hi + kTile - 1) / kTile - r.wtile, 1);
    return r;
}

__device__ __forceinline__ int tile_cost(const Params &, const Range &) { return 1; }
__device__ __forceinline__ int largest_cost(const Params &) { return 1; }
__device__ __forceinline__ int64_t item_cost(const Params &p, const Sequence &s, int item) {
    return item_range(p, s, item).n;
}

// A CTA's part of an item.
struct Item {
    int t0, t1, n;    // its key tiles [t0, t1) of the item's n; t0 == t1: the share has ended
    int head, b;      // key head and sequence
    int q_row, before;  // first row of q of the sequence, and the position of its first new token
    Range r;
    __device__ __forceinline__ int key_tile(int t) const { return t < r.sink_tiles ? t : r.wtile + t - r.sink_tiles; }
};

// ------------------------------------------------------------- instructions

__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// An 8 x 8 matrix of 16-bit elements, transposed within the warp.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// --------------------------------------------------------------- the kernel

// Threads and their registers: the launch gives 128 each, the eight warps that
// copy give theirs up to the eight that compute (256 * 88 + 256 * 168 = 512 *
// 128).
constexpr int kThreads = 512, kCopyWarps = 8, kComputeWarps = 8;
constexpr int kCopyRegs = 88, kComputeRegs = 168;
constexpr int kTurns = kComputeWarps / (kTile / kStep);  // tiles computed at once
constexpr int kCopyTurns = kCopyWarps / 2;               // and copied at once
// Items handed out ahead.  Warp 0 looks for its next tile, kCopyTurns on and so
// up to as many items on, before it copies the one it has: the item that the
// one it then hands out takes the place of must not need that copy.
constexpr int kItems = 8;
static_assert(kItems >= kCopyTurns + 2, "");

template <int D, int NT>
struct Layout {
    static constexpr int kRows = NT * 8, kBlocks = D / 32, kTiles = D / 16;
    static constexpr int kRow = D / 2, kScales = D / 16;  // bytes of a token's codes, and of its scales
    // a tile's codes of keys and values, then the scales of both
    static constexpr int kV = kTile * kRow, kKScale = 2 * kV, kVScale = kKScale + kTile * kScales;
    static constexpr int kStageBytes = kVScale + kTile * kScales;
    // each warp's O, element by element as its lanes hold it, and the merged rows
    static constexpr int kOne = NT * kTiles * 4 * 32 * 4;
    static constexpr int kStages = D == 128 ? (NT == 1 ? 10 : 8) : (NT == 1 ? 20 : 16);
    static constexpr int kO = kStages * kStageBytes, kOut = kO + kComputeWarps * kOne;
    static constexpr int kBars = kOut + kRows * D * 4, kStatBytes = 4096;
    static constexpr int kSmem = kBars + kStatBytes + 1024;  // + alignment
    // Where 16-byte chunk `c` of a token's row is: the swizzle of a copy whose
    // rows are 64 (32) bytes.
    static __device__ __forceinline__ int chunk(int token, int c) {
        return c ^ (D == 128 ? token >> 1 & 3 : token >> 2 & 1);
    }
    // Token number `i` of a tile of 16 keys, by its place in the MMAs' rows: the
    // four lanes that read two neighbouring values' words at once then read
    // different banks, whatever the swizzle.
    static __device__ __forceinline__ int token(int i) {
        return D == 128 ? (i & 8) | (i & 4) | (i & 1) << 1 | (i >> 1 & 1) : (i & 8) | (i & 1) << 2 | (i >> 1 & 3);
    }
};

template <int D, int NT>
struct Bars {
    using L = Layout<D, NT>;
    uint64_t full[2][L::kStages], empty[L::kStages];  // keys and values; both have been used
    uint64_t item_full[kItems], item_empty[kItems];
    Item item[kItems];
    float2 warp_ml[kComputeWarps][L::kRows];  // a warp's m and l, then its factor in the merge
    float4 row_mlc[L::kRows];
    int abort;
    Start<kThreads> start;
};

// Warps: 0 to 7 copy key tiles into one ring, even ones keys and odd ones
// values, each pair every fourth tile; warp 0 hands out the items too.  8 to 15
// compute: four share a tile, 32 tokens each, and the two fours take the tiles
// in turn.  Each has a reference, a sum and an O of its own, which are merged
// at the end of an item's piece.
//
// The copies are asynchronous ones of 16 bytes a lane: a row of codes is 64
// (32) bytes, and tensor copies took 4.6 cycles a row whatever its length (64
// requests of up to 32768 tokens: copies alone 300 us against 234).
template <int D, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    attention_q4_kernel(const __grid_constant__ Params p) {
    using L = Layout<D, NT>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~static_cast<uintptr_t>(1023));
    Bars<D, NT> &bar = *reinterpret_cast<Bars<D, NT> *>(smem + L::kBars);
    static_assert(sizeof(Bars<D, NT>) <= L::kStatBytes, "");
    constexpr int NB = L::kBlocks, MT = L::kTiles, kStages = L::kStages;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int *abort_flag = &bar.abort;
    if (tid == 0) {
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bar.full[0][i], 32);  // each lane's copies
            mbar_init(&bar.full[1][i], 32);
            mbar_init(&bar.empty[i], kTile / kStep);
        }
        for (int i = 0; i < kItems; ++i) {
            mbar_init(&bar.item_full[i], 1);
            mbar_init(&bar.item_empty[i], kCopyWarps + kComputeWarps);
        }
        bar.abort = 0;
        mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    locate<kThreads>(p, bar.start, blockIdx.x, gridDim.x);
    __syncthreads();

    uint32_t items = 0;
    auto item = [&]() -> const Item & { return bar.item[items % kItems]; };
    // Whether the item's record is there (false: a wait was abandoned).
    auto item_there = [&]() {
        uint64_t *const full = &bar.item_full[items % kItems];
        return __all_sync(0xffffffffu, mbar_wait(full, items / kItems & 1, abort_flag, p.err));
    };
    auto done_item = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.item_empty[items % kItems]);
        ++items;
    };

    if (warp < kCopyWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kCopyRegs));
        // ------------------------------------------------------ items
        int flags = 0;
        int4 tail = make_int4(0, 0, 0, 0);
        int64_t left = bar.start.left;
        int head = bar.start.head, b = bar.start.b, it = bar.start.item, t0 = bar.start.t0;
        Sequence s = bar.start.s;
        int n_items = items_of(p, s);
        uint32_t handed = 0;
        // Hands out the next item, or one without tiles at the share's end;
        // false after that and when a wait was abandoned.
        auto publish = [&]() {
            Item o{};
            if (left > 0) {
                o.r = item_range(p, s, it);
                o.t0 = t0, o.t1 = left >= o.r.n ? o.r.n : (int)left, o.n = o.r.n;
                o.head = head, o.b = b, o.q_row = s.row0, o.before = s.kv - s.len;
                if (o.t0 > 0) flags |= kHeadPiece | (o.t1 < o.n ? kHeadGoesOn : 0);
                if (o.t0 == 0 && o.t1 < o.n)
                    flags |= kTailPiece, tail = make_int4(0, s.row0 * p.group + o.r.row0, o.r.rows, head);
            }
            const int i = handed % kItems;
            if (!__all_sync(0xffffffffu, mbar_wait(&bar.item_empty[i], (handed / kItems & 1) ^ 1, abort_flag, p.err)))
                return false;
            if (lane == 0) {
                bar.item[i] = o;
                mbar_arrive(&bar.item_full[i]);
            }
            __syncwarp();
            ++handed;
            if (o.t0 == o.t1) return false;
            left -= o.n;
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
                    n_items = items_of(p, s);
                } while (n_items == 0 && ++scanned <= p.sequences);
            }
            return true;
        };
        bool more = warp == 0 && publish();
        // ----------------------------------------------------- copies
        const int kv = warp & 1, turn = warp >> 1;  // keys or values, and which of four tiles
        const KvQ4View &c = p.cache.c;
        // Lane i < 16 has group i of a tile, 8 tokens, which are in one page.
        // Page numbers are loaded a tile ahead of the copies, across items;
        // within a run of tiles the page table's index moves by the same
        // step, without a division.
        struct Tile {
            int page, off;  // of the lane's group; off < 0: no row sees any of it
            int head;       // < 0: the share has ended
            uint32_t seen;  // whether some row sees the lane's tokens 32 i + lane, bit i
        };
        int t = 0, t1 = 0, index = 0, off = 0;
        uint32_t fill = turn;  // of the ring: tile t is fill number `fill`, tile t1 of the item `end`
        uint32_t end = 0;
        auto look = [&]() {
            Tile k{0, -1, -1, 0};
            int last = t;
            t += kCopyTurns;
            while (t >= t1) {
                if (t1) done_item();
                if (!item_there() || item().t0 >= item().t1) return k;
                // the item's first tile is fill number `end`
                t = item().t0 + (int)(fill - end), t1 = item().t1, last = -1;
                end += t1 - item().t0;
                // warp 0 hands out an item when it comes to the one before
                if (more) more = publish();
            }
            fill += kCopyTurns;
            const Item &i = item();
            const int tile = i.key_tile(t), first = tile * kTile, token = first + (lane & 15) * 8;
            if (last < 0 || tile != i.key_tile(last) + kCopyTurns) {
                index = token / p.page_size, off = token - index * p.page_size;
            } else {
                index += p.step_pages, off += p.step_rest;
                if (off >= p.page_size) off -= p.page_size, ++index;
            }
            k.head = i.head;
            const int sink_end = i.r.sink_end, lo = i.r.lo, hi = i.r.hi;
            k.seen = 15;
            if (first < lo || first + kTile > hi) {
                k.seen = 0;
#pragma unroll
                for (int x = 0; x < kTile / 32; ++x) {
                    const int tok = first + x * 32 + lane;
                    if (tok < sink_end || (tok >= lo && tok < hi)) k.seen |= 1u << x;
                }
            }
            if (lane < 16 && (token < sink_end || (token + 8 > lo && token < hi))) {
                k.page = p.page_table[(int64_t)i.b * p.table_stride + index];
                k.off = off;
            }
            return k;
        };
        const uint8_t *base = kv ? c.v : c.k;
        const uint16_t *scale_base = kv ? c.v_scale : c.k_scale;
        const int64_t *cs = kv ? c.v_stride : c.k_stride, *ss = kv ? c.v_scale_stride : c.k_scale_stride;
        // the lane's place within the tokens of one copy: a row's chunk, and a
        // scale's token of eight
        constexpr int kChunks = L::kRow / 16, kAtOnce = 32 / kChunks;
        const int row = lane / kChunks, chunk = lane % kChunks;
        const int64_t lane_bytes = (row & 7) * cs[2] + chunk * 16, lane_scale = (lane & 7) * ss[2];
        const uint32_t lane_to = smem_u32(smem) + (kv ? L::kV : 0) + row * L::kRow + L::chunk(row, chunk) * 16;
        const uint32_t lane_scale_to = smem_u32(smem) + (kv ? L::kVScale : L::kKScale) + lane * L::kScales;
        Tile now = look();
        for (uint32_t slot = turn, phase = 1; now.head >= 0;) {
            const Tile then = look();
            bool some = now.off >= 0;
            if (some && (now.page < 0 || now.page >= p.pages)) {
                if (kv == 0) report_index(p.err);
                some = false;
            }
            // tokens that no row sees, or without a page, become zeros
            const uint32_t groups = __ballot_sync(0xffffffffu, some);
            const int64_t page = some ? now.page : 0, at = some ? now.off : 0;
            const uint64_t codes = reinterpret_cast<uint64_t>(base + page * cs[0] + now.head * cs[1] + at * cs[2]);
            const uint64_t scales =
                reinterpret_cast<uint64_t>(scale_base + page * ss[0] + now.head * ss[1] + at * ss[2]);
            if (!__all_sync(0xffffffffu, mbar_wait(&bar.empty[slot], phase, abort_flag, p.err))) break;
            const uint32_t to = lane_to + slot * L::kStageBytes;
#pragma unroll
            for (int j = 0; j < kTile / kAtOnce; ++j) {
                const int group = D == 128 ? j : 2 * j + (lane >> 4);
                const uint64_t from = __shfl_sync(0xffffffffu, codes, group) + lane_bytes;
                copy16(to + j * kAtOnce * L::kRow, reinterpret_cast<const void *>(from), !(groups >> group & 1));
            }
            const uint32_t scale_to = lane_scale_to + slot * L::kStageBytes;
#pragma unroll
            for (int x = 0; x < kTile / 32; ++x) {
                const int group = 4 * x + (lane >> 3);
                const uint64_t from = __shfl_sync(0xffffffffu, scales, group) + 2 * lane_scale;
                const bool seen = (groups >> group & 1) && (now.seen >> x & 1);
                copy_small<L::kScales>(scale_to + x * 32 * L::kScales, reinterpret_cast<const void *>(from), !seen);
            }
            copy_arrive(&bar.full[kv][slot]);
            slot += kCopyTurns;
            if (slot >= kStages) slot -= kStages, phase ^= 1;
            now = then;
        }
        copy_wait_all();
        if (warp == 0) {
            tail.x = flags;
            if (lane == 0) p.record[blockIdx.x] = tail;
        }
    } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kComputeRegs));
    const int g = lane >> 2, t = lane & 3, ctid = tid - kCopyWarps * 32, cwarp = warp - kCopyWarps;
    const int part = cwarp & 3, turn = cwarp >> 2;  // of a tile, and which of two tiles
    const uint32_t bias = p.cache.bias, ring = smem_u32(smem);
    float *merged = reinterpret_cast<float *>(smem + L::kOut);
    uint32_t fill = 0;       // tiles of earlier items
    uint32_t slot = turn, phase = 0;  // of the warp's next tile
    // Every warp takes part in an item's barriers, also one whose wait was
    // given up: it only leaves its sums as they are.
    for (;; done_item()) {
        if (named_bar_or(1, kComputeWarps * 32, !item_there())) break;
        const Item &i = item();
        const int t0 = i.t0, t1 = i.t1, tiles = t1 - t0, head = i.head;
        if (tiles <= 0) break;
        const Range r = i.r;
        const int q_row = i.q_row, before = i.before;

        // ---------------------------------------------------- queries
        // q as the second operand: column g of tile n, for block j and half x
        // of it elements 4t + x, 4t + x + 2 and 16 further
        uint32_t qf[NT][NB][2][2];
        uint32_t less[NT];
        float cs[NT][2];  // c of columns 2t and 2t + 1
        int pos[NT][2];  // their positions
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int row = n * 8 + g;
            uint2 lo[NB], hi[NB];
            float top = 0.f;
#pragma unroll
            for (int j = 0; j < NB; ++j) lo[j] = hi[j] = make_uint2(0, 0);
            if (row < r.rows) {
                const int token = (r.row0 + row) / p.group, in_group = r.row0 + row - token * p.group;
                const __nv_bfloat16 *src =
                    p.q + (q_row + token) * p.q_row_stride + (head * p.group + in_group) * p.q_head_stride;
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    lo[j] = *reinterpret_cast<const uint2 *>(src + 32 * j + 4 * t);
                    hi[j] = *reinterpret_cast<const uint2 *>(src + 32 * j + 16 + 4 * t);
                }
            }
            auto low = [](uint32_t w) { return __uint_as_float(w << 16); };
            auto high = [](uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); };
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                top = fmaxf(top, fmaxf(fmaxf(fabsf(low(lo[j].x)), fabsf(high(lo[j].x))),
                                       fmaxf(fabsf(low(lo[j].y)), fabsf(high(lo[j].y)))));
                top = fmaxf(top, fmaxf(fmaxf(fabsf(low(hi[j].x)), fabsf(high(hi[j].x))),
                                       fmaxf(fabsf(low(hi[j].y)), fabsf(high(hi[j].y)))));
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // 2^up brings the largest element to [2^14, 2^15); a row of
            // zeros or with an infinity is left alone
            const int exponent = (int)(__float_as_uint(top) >> 23) - 127;
            const int up = top > 0.f && top < INFINITY ? min(14 - exponent, 100) : 0;
            const float f = __uint_as_float((uint32_t)(127 + up) << 23);
            const float down = __uint_as_float((uint32_t)(127 - up) << 23);
            const float row_c = in_range(p.scale_log2 * (down * kCodeUnit));
#pragma unroll
            for (int x = 0; x < 2; ++x) cs[n][x] = __shfl_sync(0xffffffffu, row_c, (2 * t + x) * 4);
            auto pair = [&](float a, float z, float f) { return pack_f16(a * f, z * f); };
            uint32_t less_hi[NB / 2], less_lo[NB / 2];
#pragma unroll
            for (int j = 0; j < NB; ++j) {
                // a high nibble is read as 16 codes
                const float f16 = f * 0.0625f;
                qf[n][j][0][0] = pair(low(lo[j].x), low(lo[j].y), f);
                qf[n][j][1][0] = pair(high(lo[j].x), high(lo[j].y), f);
                qf[n][j][0][1] = pair(low(hi[j].x), low(hi[j].y), f16);
                qf[n][j][1][1] = pair(high(hi[j].x), high(hi[j].y), f16);
                // what the codes' 8 too many come to, in two binary16 parts
                float sum = 0.f;
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float2 u = __half22float2(as_half2(qf[n][j][x][0]));
                    const float2 v = __half22float2(as_half2(qf[n][j][x][1]));
                    sum += (u.x + u.y) + 16.f * (v.x + v.y);
                }
                sum += __shfl_xor_sync(0xffffffffu, sum, 1);
                sum += __shfl_xor_sync(0xffffffffu, sum, 2);
                sum *= -8.f * kLessUnit / kCodeUnit;
                const __half top_part = __float2half_rn(sum), rest = __float2half_rn(sum - __half2float(top_part));
                const uint32_t at = j & 1 ? 16 : 0;
                if (at == 0) less_hi[j / 2] = less_lo[j / 2] = 0;
                less_hi[j / 2] |= (uint32_t)__half_as_ushort(top_part) << at;
                less_lo[j / 2] |= (uint32_t)__half_as_ushort(rest) << at;
            }
            // lanes t: blocks 0 and 1, then 2 and 3 (none at D = 64), of both parts
            less[n] = t < 2 ? less_hi[t & (NB / 2 - 1)] : less_lo[t & (NB / 2 - 1)];
            if (D == 64 && (t & 1)) less[n] = 0;
#pragma unroll
            for (int x = 0; x < 2; ++x) pos[n][x] = before + (r.row0 + n * 8 + 2 * t + x) / p.group;
        }

        // -------------------------------------------------------- keys
        float m[NT][2], l[NT][2], o[NT][MT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            m[n][0] = m[n][1] = -INFINITY, l[n][0] = l[n][1] = 0.f;
#pragma unroll
            for (int i = 0; i < MT; ++i) o[n][i][0] = o[n][i][1] = o[n][i][2] = o[n][i][3] = 0.f;
        }
        for (int tile = (fill & 1) == (uint32_t)turn ? 0 : 1; tile < tiles; tile += kTurns) {
            if (!__all_sync(0xffffffffu, mbar_wait(&bar.full[0][slot], phase, abort_flag, p.err))) break;
            const uint32_t st = ring + slot * L::kStageBytes;
            const uint32_t k_codes = st + part * kStep * L::kRow, v_codes = k_codes + L::kV;
            const uint32_t k_scales = st + L::kKScale + part * kStep * L::kScales;
            const uint32_t v_scales = st + L::kVScale + part * kStep * L::kScales;
            // scores: keys by queries, two tiles of 16 keys
            float sc[2][NT][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int r0 = h * 16 + L::token(g), r1 = r0 + 8;
                uint32_t d0[NB / 2], d1[NB / 2];
                if (D == 128) {
                    const uint2 x = lds64(k_scales + r0 * 8), y = lds64(k_scales + r1 * 8);
                    d0[0] = x.x, d0[NB / 2 - 1] = x.y, d1[0] = y.x, d1[NB / 2 - 1] = y.y;
                } else {
                    d0[0] = lds32(k_scales + r0 * 4), d1[0] = lds32(k_scales + r1 * 4);
                }
                // the scales times what the codes' 8 come to
                const uint32_t e0 = t & 1 ? d0[NB / 2 - 1] : d0[0], e1 = t & 1 ? d1[NB / 2 - 1] : d1[0];
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    sc[h][n][0] = sc[h][n][1] = sc[h][n][2] = sc[h][n][3] = 0.f;
                    mma16816(sc[h][n], e0, e1, 0u, 0u, less[n], 0u);
#pragma unroll
                    for (int x = 0; x < 4; ++x) sc[h][n][x] *= 1.f / kLessUnit;
                }
#pragma unroll
                for (int j = 0; j < NB; ++j) {
                    const uint32_t w0 = lds32(k_codes + r0 * L::kRow + L::chunk(r0, j) * 16 + t * 4);
                    const uint32_t w1 = lds32(k_codes + r1 * L::kRow + L::chunk(r1, j) * 16 + t * 4);
                    float acc[NT][4] = {};
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t u0 = w0 >> 8 * x, u1 = w1 >> 8 * x;
                        const uint32_t a0 = u0 & 0x000F000Fu, a1 = u1 & 0x000F000Fu;
                        const uint32_t a2 = u0 & 0x00F000F0u, a3 = u1 & 0x00F000F0u;
#pragma unroll
                        for (int n = 0; n < NT; ++n) mma16816(acc[n], a0, a1, a2, a3, qf[n][j][x][0], qf[n][j][x][1]);
                    }
                    const __half2 e0 = as_half2(d0[j / 2]), e1 = as_half2(d1[j / 2]);
                    const float f0 = j & 1 ? __high2float(e0) : __low2float(e0);
                    const float f1 = j & 1 ? __high2float(e1) : __low2float(e1);
#pragma unroll
                    for (int n = 0; n < NT; ++n) {
                        sc[h][n][0] = fmaf(f0, acc[n][0], sc[h][n][0]), sc[h][n][1] = fmaf(f0, acc[n][1], sc[h][n][1]);
                        sc[h][n][2] = fmaf(f1, acc[n][2], sc[h][n][2]), sc[h][n][3] = fmaf(f1, acc[n][3], sc[h][n][3]);
                    }
                }
            }
            const int tok0 = i.key_tile(t0 + tile) * kTile + part * kStep;
            if (tok0 + kStep - 1 > r.first || (p.window && tok0 <= r.last - p.window && tok0 + kStep > p.sinks)) {
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int n = 0; n < NT; ++n)
#pragma unroll
                        for (int x = 0; x < 4; ++x) {
                            const int tok = tok0 + h * 16 + L::token(g) + (x >> 1) * 8, at = pos[n][x & 1];
                            if (tok > at || (p.window && tok <= at - p.window && tok >= p.sinks))
                                sc[h][n][x] = -INFINITY;
                        }
            }
            // references that a score outgrew move, in all lanes of a column
            bool grew = false;
            float top[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    top[n][x] = fmaxf(fmaxf(sc[0][n][x], sc[0][n][x + 2]), fmaxf(sc[1][n][x], sc[1][n][x + 2]));
                    grew |= (top[n][x] - m[n][x]) * cs[n][x] > kGrow;
                }
            if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    float f[2];
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        float v = fmaxf(top[n][x], m[n][x]);
#pragma unroll
                        for (int d = 4; d <= 16; d <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, d));
                        f[x] = m[n][x] == v ? 1.f : ex2((m[n][x] - v) * cs[n][x]);
                        m[n][x] = v;
                        l[n][x] *= f[x];
                    }
#pragma unroll
                    for (int j = 0; j < MT; ++j) {
                        o[n][j][0] *= f[0], o[n][j][1] *= f[1];
                        o[n][j][2] *= f[0], o[n][j][3] *= f[1];
                    }
                }
            }
            // p as the second operand of values by queries
            uint32_t pf[2][NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                const float base[2] = {m[n][0] == -INFINITY ? 0.f : m[n][0], m[n][1] == -INFINITY ? 0.f : m[n][1]};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    float e[4];
#pragma unroll
                    for (int x = 0; x < 4; ++x) {
                        e[x] = ex2(fmaf(sc[h][n][x] - base[x & 1], cs[n][x & 1], kLift));
                        l[n][x & 1] += e[x];
                    }
                    pf[h][n][0] = transpose8x8(as_bits(__floats2half2_rn(e[0], e[1])));
                    pf[h][n][1] = transpose8x8(as_bits(__floats2half2_rn(e[2], e[3])));
                }
            }
            // values: a lane's 16 (D = 64: 8) elements of a token are 8 (4)
            // bytes, all of one block
            if (!__all_sync(0xffffffffu, mbar_wait(&bar.full[1][slot], phase, abort_flag, p.err))) break;
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                uint32_t w[4][D / 64], d[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int tok = h * 16 + L::token(2 * t + (k & 1)) + (k >> 1) * 8;
                    if (D == 128) {
                        const uint2 x = lds64(v_codes + tok * L::kRow + L::chunk(tok, g >> 1) * 16 + (g & 1) * 8);
                        w[k][0] = x.x, w[k][D / 64 - 1] = x.y;
                        d[k] = lds16(v_scales + tok * 8 + (g >> 1) * 2);
                    } else {
                        w[k][0] = lds32(v_codes + tok * L::kRow + L::chunk(tok, g >> 2) * 16 + (g & 3) * 4);
                        d[k] = lds16(v_scales + tok * 4 + (g >> 2) * 2);
                    }
                }
                const __half2 d01 = as_half2(__byte_perm(d[0], d[1], 0x5410));
                const __half2 d23 = as_half2(__byte_perm(d[2], d[3], 0x5410));
#pragma unroll
                for (int j = 0; j < D / 64; ++j)
#pragma unroll
                    for (int half = 0; half < 2; ++half) {
                        const uint32_t sel = half ? 0x7632 : 0x5410;
                        const uint32_t a = __byte_perm(w[0][j], w[1][j], sel), z = __byte_perm(w[2][j], w[3][j], sel);
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const uint32_t u = a >> 8 * x, y = z >> 8 * x;
                            const uint32_t a0 = times(low_codes(u, bias), d01), a1 = times(high_codes(u, bias), d01);
                            const uint32_t a2 = times(low_codes(y, bias), d23), a3 = times(high_codes(y, bias), d23);
#pragma unroll
                            for (int n = 0; n < NT; ++n)
                                mma16816(o[n][(j * 2 + half) * 2 + x], a0, a1, a2, a3, pf[h][n][0], pf[h][n][1]);
                        }
                    }
            }
            // (the stage's words have all been used)
            __syncwarp();
            if (lane == 0) mbar_arrive(&bar.empty[slot]);
            slot += kTurns;
            if (slot >= kStages) slot -= kStages, phase ^= 1;
        }
        fill += tiles;

        // ------------------------------------------------------- merge
        float *mine = reinterpret_cast<float *>(smem + L::kO + cwarp * L::kOne);
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int j = 0; j < MT; ++j)
#pragma unroll
                for (int x = 0; x < 4; ++x) mine[((n * MT + j) * 4 + x) * 32 + lane] = o[n][j][x];
#pragma unroll
            for (int x = 0; x < 2; ++x) {
#pragma unroll
                for (int d = 4; d <= 16; d <<= 1) l[n][x] += __shfl_xor_sync(0xffffffffu, l[n][x], d);
                if (g == 0) {
                    bar.warp_ml[cwarp][n * 8 + 2 * t + x] = make_float2(m[n][x], l[n][x]);
                    if (cwarp == 0) bar.row_mlc[n * 8 + 2 * t + x].z = cs[n][x];
                }
            }
        }
        named_bar_sync(1, kComputeWarps * 32);
        const bool whole = t0 == 0 && t1 == i.n;
        if (ctid < L::kRows) {
            const float row_c = bar.row_mlc[ctid].z;
            float top = -INFINITY, sum = 0.f;
#pragma unroll
            for (int w = 0; w < kComputeWarps; ++w) top = fmaxf(top, bar.warp_ml[w][ctid].x);
#pragma unroll
            for (int w = 0; w < kComputeWarps; ++w) {
                const float2 ml = bar.warp_ml[w][ctid];
                // a warp without a tile has no reference, and a sum of 0
                const float f = ml.x == top ? 1.f : ex2((ml.x - top) * row_c);
                sum += ml.y * f;
                bar.warp_ml[w][ctid].x = f;
            }
            const float inv = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
            if (whole)
                for (int w = 0; w < kComputeWarps; ++w) bar.warp_ml[w][ctid].x *= inv;
            bar.row_mlc[ctid].x = top, bar.row_mlc[ctid].y = sum;
        }
        named_bar_sync(1, kComputeWarps * 32);
        const float *parts = reinterpret_cast<const float *>(smem + L::kO);
        for (int e = ctid; e < L::kRows * D; e += kComputeWarps * 32) {
            const int le = e & 31, x = e >> 5 & 3, j = (e >> 7) % MT, n = (e >> 7) / MT, gg = le >> 2;
            const int row = n * 8 + 2 * (le & 3) + (x & 1);
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kComputeWarps; ++w) v = fmaf(bar.warp_ml[w][row].x, parts[w * (L::kOne / 4) + e], v);
            // the lane's byte of its block, and the element it holds
            const int byte = (D == 128 ? 8 * (gg & 1) : 4 * (gg & 3)) + j;
            const int d = (D == 128 ? 32 * (gg >> 1) : 32 * (gg >> 2)) + byte + (x >> 1) * 16;
            merged[row * D + d] = v;
        }
        named_bar_sync(1, kComputeWarps * 32);
        const int f0 = q_row * p.group + r.row0;
        const int piece = (blockIdx.x * 2 + (t0 == 0 ? 1 : 0)) * p.item_rows;
        // place of a row of the item in [rows][q_heads]
        auto place = [&](int row) {
            const int token = (f0 + row) / p.group;
            return (int64_t)token * p.q_heads + head * p.group + (f0 + row - token * p.group);
        };
        for (int e = ctid * 4; e < r.rows * D; e += kComputeWarps * 32 * 4) {
            const int row = e / D, d = e - row * D;
            const float4 v = *reinterpret_cast<const float4 *>(merged + e);
            const int64_t at = place(row) * D + d;
            if (!whole)
                *reinterpret_cast<float4 *>(p.part + (int64_t)(piece + row) * D + d) = v;
            else if (p.out_bf16)
                *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(p.out) + at) =
                    make_uint2(pack_bf16(v.x, v.y), pack_bf16(v.z, v.w));
            else
                *reinterpret_cast<float4 *>(static_cast<float *>(p.out) + at) = v;
        }
        if (ctid < r.rows) {
            const float4 mlc = bar.row_mlc[ctid];
            if (!whole)
                p.part_mlc[piece + ctid] = mlc;
            else if (p.lse)
                p.lse[place(ctid)] = (mlc.x * mlc.z + (__log2f(mlc.y) - kLift)) * kLn2;
        }
    }
    }
}

// Adds the pieces of the items that a share's boundary cut.  blockIdx.x: the
// CTA whose tail piece starts the item, blockIdx.y: a row of it; its warps take
// the pieces in turn.  Latency bounds it: the records, then a row's (m, l, c)
// and pieces of O at once.
template <int D>
__global__ void __launch_bounds__(256) attention_q4_join_kernel(const __grid_constant__ Params p, int ctas) {
    __shared__ float sums[8][D];
    pdl_launch_dependents();
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row = blockIdx.y;
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
    if (!(rec.x & kTailPiece) || row >= rec.z) return;
    constexpr int kOwn = D / 32;
    using Own = typename std::conditional<kOwn == 4, float4, float2>::type;
    auto place = [&](int i) { return (int64_t)((blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * p.item_rows + row; };
    auto piece = [&](int i) { return *reinterpret_cast<const Own *>(p.part + place(i) * D + lane * kOwn); };
    // the warp's first pieces are read with the statistics
    Own first[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) first[k] = piece(min(warp + 8 * k, n - 1));
    float m = -INFINITY;
    for (int i = lane; i < n; i += 32) m = fmaxf(m, p.part_mlc[place(i)].x);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, d));
    float l = 0.f;
    const float c = p.part_mlc[place(0)].z;
    auto factor = [&](float x) { return x == m ? 1.f : ex2((x - m) * c); };
    for (int i = lane; i < n; i += 32) {
        const float4 mlc = p.part_mlc[place(i)];
        l += mlc.y * factor(mlc.x);
    }
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) l += __shfl_xor_sync(0xffffffffu, l, d);
    float acc[kOwn] = {};
    auto add = [&](const Own &v, int i) {
        const float *o = reinterpret_cast<const float *>(&v), f = factor(p.part_mlc[place(i)].x);
#pragma unroll
        for (int e = 0; e < kOwn; ++e) acc[e] = fmaf(o[e], f, acc[e]);
    };
#pragma unroll
    for (int k = 0; k < 4; ++k)
        if (warp + 8 * k < n) add(first[k], warp + 8 * k);
    for (int i = warp + 32; i < n; i += 8) add(piece(i), i);
#pragma unroll
    for (int e = 0; e < kOwn; ++e) sums[warp][lane * kOwn + e] = acc[e];
    __syncthreads();
    const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
    const int token = (rec.y + row) / p.group;
    const int64_t at = (int64_t)token * p.q_heads + rec.w * p.group + (rec.y + row - token * p.group);
    const int d = threadIdx.x;
    if (d < D) {
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += sums[w][d];
        store_y(static_cast<float *>(p.out), at * D + d, v * inv, p.out_bf16);
    }
    if (p.lse && d == 0) p.lse[at] = (m * c + (__log2f(l) - kLift)) * kLn2;
}

// -------------------------------------------------------------------- host

// The most rows (tokens times heads of the group) of a sequence that this kernel
// takes; those of longer ones fill tcgen05's tiles (attention.cu).
constexpr int kMostRows = 16;

// Rows of an item, and the most of a sequence that this kernel takes: 16 where
// no sequence can bring more, or one token's heads need it; else one tile of 8,
// for the single tokens of a mixed batch.  That sends sequences of 9 to 16 rows
// beside longer ones to tcgen05, whose launch such a call makes anyway.  Two
// items of 8 for each of them instead: 16 drafts of 2 or 3 tokens by 5 heads
// after 8192 beside a chunk of 256 156 -> 165 us, without the chunk level (107
// and 105 to 108), 64 of them after 16384 669 -> 593.
int item_rows(int group, int max_q_len) {
    const int64_t most = (int64_t)group * max_q_len;
    return most <= 8 || (most > kMostRows && group <= 8) ? 8 : kMostRows;
}

struct WorkspaceLayout {
    size_t mlc_off, rec_off, bytes;
    WorkspaceLayout(int ctas, int D, int rows_each) {
        const size_t rows = (size_t)ctas * 2 * rows_each;
        mlc_off = rows * D * 4;
        rec_off = mlc_off + rows * 16;
        bytes = (rec_off + (size_t)ctas * 16 + 255) / 256 * 256;
    }
};

template <int D, int NT>
cudaError_t launch_narrow(const Params &p, int ctas, cudaStream_t s) {
    constexpr int kSmem = Layout<D, NT>::kSmem;
    const cudaError_t e = ensure_smem_attr(reinterpret_cast<const void *>(attention_q4_kernel<D, NT>), kSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(attention_q4_kernel<D, NT>, dim3(ctas), dim3(kThreads), kSmem, s, p);
}

template <int D>
cudaError_t launch_d(const AttentionArgs &a, const KvQ4View &c, void *workspace, int ctas, cudaStream_t s,
                     unsigned int *err) {
    Params p{};
    p.cache = cache_q4(c);
    p.page_table = c.page_table, p.q_start = c.q_start, p.kv_len = c.kv_len, p.table_stride = c.table_stride;
    p.sequences = c.sequences, p.table_width = c.table_width, p.pages = c.pages, p.page_size = c.page_size;
    p.rows = a.rows, p.max_q_len = a.max_q_len;
    p.step_pages = kCopyTurns * kTile / c.page_size, p.step_rest = kCopyTurns * kTile % c.page_size;
    p.q_heads = a.q_heads, p.kv_heads = c.kv_heads, p.group = a.q_heads / c.kv_heads;
    p.window = a.window, p.sinks = a.sinks;
    p.item_rows = p.most_rows = item_rows(p.group, a.max_q_len);
    p.q = a.q, p.q_row_stride = a.q_row_stride, p.q_head_stride = a.q_head_stride;
    p.scale_log2 = a.scale * kLog2e;
    p.out = a.out, p.lse = a.lse, p.out_bf16 = a.out_bf16;
    const WorkspaceLayout w(ctas, D, p.item_rows);
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    p.part = reinterpret_cast<float *>(ws);
    p.part_mlc = reinterpret_cast<float4 *>(ws + w.mlc_off);
    p.record = reinterpret_cast<int4 *>(ws + w.rec_off);
    p.err = err;
    const cudaError_t e = p.item_rows == 8 ? launch_narrow<D, 1>(p, ctas, s) : launch_narrow<D, 2>(p, ctas, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(attention_q4_join_kernel<D>, dim3(ctas, p.item_rows), dim3(256), 0, s, p, ctas);
}

}  // namespace

size_t attention_q4_workspace_bytes(int q_heads, int kv_heads, int head_dim, int max_q_len) {
    const int group = q_heads / kv_heads;
    const size_t narrow = WorkspaceLayout(current_sms(), head_dim, item_rows(group, max_q_len)).bytes;
    return narrow + ((int64_t)group * max_q_len > kMostRows
                         ? attention_workspace_bytes(q_heads, kv_heads, head_dim, max_q_len)
                         : 0);
}

cudaError_t launch_attention_q4(const AttentionArgs &a, const KvQ4View &c, void *workspace, cudaStream_t s,
                                unsigned int *err) {
    const int sms = current_sms(), group = a.q_heads / c.kv_heads;
    if (sms < 1) return cudaErrorInvalidDevice;
    const bool both = (int64_t)group * a.max_q_len > kMostRows;
    // Where all but one sequence can have max_q_len tokens and the last one more
    // than this kernel's, none has few unless there are rows of no sequence (and
    // then it is the other kernel's too).  A kernel that finds nothing to do
    // takes 6 us of a call.
    const int64_t least = a.rows - (c.sequences - 1ll) * a.max_q_len;
    const bool all_long = both && least * group > item_rows(group, a.max_q_len);
    cudaError_t e = cudaSuccess;
    if (group <= kMostRows && !all_long)
        e = (c.head_dim == 128 ? launch_d<128> : launch_d<64>)(a, c, workspace, sms, s, err);
    if (e != cudaSuccess || !both) return e;
    const int rows = item_rows(group, a.max_q_len);
    uint8_t *rest = static_cast<uint8_t *>(workspace) + WorkspaceLayout(sms, c.head_dim, rows).bytes;
    return launch_attention_q4_wide(a, c, all_long ? 1 : rows + 1, rest, s, err);
}

}  // namespace q4_0
