// kv_attention.cu -- attention of new tokens over the paged K/V cache that kv_matmul_paged fills.
//
// kv_matmul_ragged_paged (Modular MAX, nn/kv_cache_ragged): Args kv_collection (the K and V
// cache), layer_idx, input_row_offsets.  Heads in groups of G share keys and values, so the
// queries of a group's heads are rows of one product:
//     S = Q K^T  [rows x keys],   O = softmax(scale S) V  [rows x D]
// with row = token * G + head, and 128 rows of whole tokens make a tile of queries.
//
// An item is up to two tiles of one request and one head of keys.  Two tiles (a chunk) take each
// tile of 128 keys in turn; one tile (few tokens, a single one above all) takes even and odd tiles
// of keys in turn, with sums of their own that are joined at the item's end.  Either way a step is
// one product of 128 x 128 scores, steps alternate between two stages, and a stage has four softmax
// warps and, in tensor memory, its O and its weights (the second product's A operand).  Scores
// leave tensor memory as soon as they are there, so that the next step's are computed while these
// go through the softmax: with D = 128 one place serves both stages, since the values' product of
// the step two before runs between two steps' scores.
//
// The key axis of all items is one line of 128-key tiles, cut into equal parts, one for each CTA:
// a CTA starts at most one item that it does not finish and finishes at most one that it did not
// start.  Such parts leave unnormalised fp32 sums, maxima and totals in the workspace and a second
// kernel joins them; whole items are written directly.  A window's items leave out the tiles
// between the first tokens and the window.
//
// Roles of a CTA: warps 0-3 and 4-7 the softmax of a stage, 8 and 9 the MMAs of a stage's scores,
// 10 those of both stages' values, 11 the schedule and all loads, 12-15 the epilogue; these also
// ready values where not every row attends every key, since a zero weight must not meet infinities
// and NaN: rows that no token attends are cleared, others looked through.  Scores are kept in base 2;
// the running maximum moves only when a row's new maximum exceeds it by 2^8, since any reference
// works as long as nothing overflows, so O is hardly ever rescaled (by every new maximum, prompts
// and windows take 11 to 12 % longer).
//
// Bytes: every key and value of the cache once a request and head of keys and per 256 rows of
// queries, these and the output once.  Measured on a GB300 (6 781 GB/s of a copy, 1 888 TFLOP/s of a
// matrix product, both measured), whole calls:
//   4 requests x 1 token, 32 heads on 8 of keys, D = 128, 65 536 keys: 164 us, 6.55 TB/s, bound by HBM;
//   64 x 1 token, 512 to 4096 keys: 105 us, 5.7 TB/s, HBM and the calls' start and join;
//   1 x 2048 tokens behind 16 384: 365 us, 1.60 PFLOP/s, alone, 393 us and 1.49 PFLOP/s one call after
//     another, when the power limit lowers the clock (a matrix product then runs at 1.69).  A step
//     (128 x 128 scores of a stage) takes 1 450 cycles, of which its 16 MMAs take 1 024 and without
//     the softmax 1 205: one place for the scores of both stages, the chain from scores to weights,
//     and shared memory's bandwidth, which products with both operands there use up;
//   2 x 2048 to 4096 tokens, 64 heads on 8, D = 64, the last 1024 keys and the first 4: 195 us.  A
//     step takes 1 090 cycles, the exponentials 512 of them, an item's three tiles with masks
//     about a fifth of its time and its start and end a sixth.
#include <atomic>

#include "kv_device.cuh"
#include "kv_internal.h"

namespace pkm {
namespace {

constexpr int kScoreWarp = 8, kOutWarp = 10, kLoadWarp = 11, kEndWarp = 12;
constexpr int kThreads = 16 * 32;
// Registers of the two softmax groups, of the issuing and loading warps and of the epilogue, of the
// 4 x 128 that the block starts with.  (An epilogue of 104, which spills, and a softmax of 176: 1 %
// longer; a softmax of 160, which spills, prompts and windows 7 to 8 %; an epilogue of 88: prompts 7 %.)
constexpr int kStartRegs = 128, kSoftRegs = 168, kIssueRegs = 64, kEndRegs = 112;
static_assert(2 * kSoftRegs + kIssueRegs + kEndRegs <= 4 * kStartRegs, "registers of the block");
constexpr int kTile = 128;          // keys of a tile, rows of a tile of queries
constexpr int kMaxStages = 6;       // tiles of queries, keys or values in shared memory
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kWeightCol = 384;    // TMEM column of the weights, 64 a stage
// An item's start and end, in tiles (with 1 prompts of many lengths take 5 % longer and small ragged
// chunks 18 %, with 3 1.5 and 3 %).
constexpr int kItemCost = 2;
constexpr uint64_t kDrainNs = 1000000;  // a role that gave up leaves its loads time to land
constexpr float kLazy = 8.0f;       // base-2 growth of a maximum that is let pass
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// a / b; the 64-bit division is a long routine, which is there once, and the operands are hardly
// ever that large.
static __device__ __noinline__ int64_t long_quotient(int64_t a, int64_t b) { return a / b; }

__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return long_quotient(a, b);
}

// Sum of floor((a * i + b) / m) over i < n, for a, b >= 0: Euclid's steps on a and m.
static __device__ __noinline__ int64_t floor_sum(int64_t n, int64_t m, int64_t a, int64_t b) {
    int64_t sum = 0;
    while (n > 0) {
        if (a >= m) {
            const int64_t k = quotient(a, m);
            sum += (n & 1 ? n * ((n - 1) / 2) : (n / 2) * (n - 1)) * k;
            a -= k * m;
        }
        if (b >= m) {
            const int64_t k = quotient(b, m);
            sum += n * k;
            b -= k * m;
        }
        const int64_t y = a * n + b;
        if (y < m) break;
        n = quotient(y, m);
        b = y - n * m;
        const int64_t t = m;
        m = a;
        a = t;
    }
    return sum;
}

// One request as the schedule sees it.  Item j has its tokens from j * T on.
struct Request {
    int64_t first;   // its first row
    int64_t len;     // cached tokens before its new ones
    int32_t n;       // its new tokens (0 too where the page table does not hold them all)
    int32_t items;   // of one head of keys

    __device__ __forceinline__ bool load(const KvAttentionArgs& a, int b) {
        const int64_t rows = a.total_rows;
        const int64_t lo = min(static_cast<int64_t>(__ldg(a.row_offsets + b)), rows);
        const int64_t hi = min(static_cast<int64_t>(__ldg(a.row_offsets + b + 1)), rows);
        first = lo;
        n = hi > lo ? static_cast<int32_t>(hi - lo) : 0;
        len = __ldg(a.cache_lengths + b);
        const bool held = n == 0 || len + n <= static_cast<int64_t>(a.max_pages) * a.page_size;
        if (!held) n = 0;
        items = (n + 2 * a.tile_tokens - 1) / (2 * a.tile_tokens);
        return held;
    }
    // Tiles that hold the first tokens, and those between them and the window of the token at
    // position p.
    __device__ __forceinline__ int32_t gap(const KvAttentionArgs& a, int64_t p) const {
        if (a.window == 0) return 0;
        const int64_t from = p - a.window + 1;
        return from <= 0 ? 0 : max(static_cast<int32_t>(from >> 7) - a.sink_tiles, 0);
    }
    __device__ __forceinline__ int32_t tokens(const KvAttentionArgs& a, int32_t j) const {
        return min(2 * a.tile_tokens, n - j * 2 * a.tile_tokens);
    }
    __device__ __forceinline__ int32_t tiles(const KvAttentionArgs& a, int32_t j) const {
        const int64_t at = len + static_cast<int64_t>(j) * 2 * a.tile_tokens;
        return static_cast<int32_t>((at + tokens(a, j) + kTile - 1) >> 7) - gap(a, at);
    }
    // Units of the items before j < items; an item has kItemCost besides its tiles.
    __device__ __forceinline__ int64_t units_before(const KvAttentionArgs& a, int64_t j) const {
        if (j == 0) return 0;
        const int64_t t = 2 * a.tile_tokens;
        int64_t sum = kItemCost * j + floor_sum(j, kTile, t, len + t + kTile - 1);
        if (a.window > 0) {
            // the first item whose gap is not below 0
            const int64_t from = len - a.window + 1 - static_cast<int64_t>(a.sink_tiles) * kTile;
            const int64_t j0 = from >= 0 ? 0 : quotient(t - 1 - from, t);
            if (j > j0) sum -= floor_sum(j - j0, kTile, t, from + j0 * t);
        }
        return sum;
    }
    __device__ __forceinline__ int64_t head_units(const KvAttentionArgs& a) const {
        return n == 0 ? 0 : units_before(a, items - 1) + tiles(a, items - 1) + kItemCost;
    }
};

// The part of an item that a CTA has, as its warps see it: tiles [x0, x1) of the item's list, which
// all take from the last to the first.  Tile x of the list is x, or x + gap from `lead` on.
struct Part {
    int64_t pos;         // position of the first token
    int32_t row, b;      // its row, and the request
    int32_t tokens, head;
    int32_t x0, x1, lead, gap;
    int32_t wide;        // two tiles of queries
    int32_t whole;       // all tiles of the item
    int32_t left;        // CTAs that share the item, if it starts here (0: it does not)
    int32_t diagonal[2], edge[2];  // tiles that a tile of queries' tokens do not all attend (Masked)

    __device__ __forceinline__ int32_t tile(int32_t x) const { return x >= lead ? x + gap : x; }
};
constexpr int kParts = 4;  // that the schedule is ahead at most
constexpr int kFound = 8;  // parts whose finds are kept
// Tiles of a part that are looked through: three at the diagonal of 256 tokens, three at the window's
// edge, and the last of the first tokens.
constexpr int kFoundBits = 8;

struct Bars {
    uint64_t k_full[kMaxStages];   // a tile of keys is there
    uint64_t k_empty[kMaxStages];  // its MMAs are done
    uint64_t v_full[kMaxStages];   // of values
    uint64_t v_empty[kMaxStages];
    uint64_t v_own[kMaxStages];    // values that are looked through first are there
    uint64_t q_full[kMaxStages], q_empty[kMaxStages];
    uint64_t s_full[2];          // a step's scores are complete
    uint64_t s_empty[2];         // they have been read
    uint64_t p_full[2];          // its weights are written
    uint64_t p_empty[2];         // they are used up, and O holds them
    uint64_t stats_full[2];      // a part's maxima and sums on the stage
    uint64_t o_full[2];          // and its O
    uint64_t o_empty[2];         // both have been read
    uint64_t part_full[kParts], part_empty[kParts];
    uint64_t mma_done[3];
    Part part[kParts];
    union {
        float2 stats[2][kTile];            // of the stages
        int64_t scratch[kThreads / 32];  // of the plan
    };
    int64_t units;               // units of all items
    int64_t first_unit;          // this CTA's share begins here
    int64_t share;               // and has so many units
    int64_t into, each;          // units of its first request before it, and of one of its heads
    Request first;
    int32_t request, head, item, unit;  // its first unit
    int32_t ctas;                // that have a share
    // What the epilogue's warps found, by a part's number and the warp: the number's last byte, and a
    // bit for each tile looked through, counted from the part's last, of whose quarter some rows that
    // not all tokens attend had infinities or NaN.  A warp is less than eight parts ahead of another:
    // the schedule keeps four, and a warp has taken the one behind that of its epilogue.
    uint16_t nonfinite[kFound][4];
    uint32_t tmem_base;
    int abort_flag;
};

template <int DB>  // 64-column blocks of a head
struct Shape {
    static constexpr int kCols = DB * 64;
    static constexpr int kBytes = DB * 128 * 128;   // of a tile
    // Keys of the step at hand and the next; values of the two steps before it, whose weights are
    // not ready, and the next.
    static constexpr int kKeyStages = DB == 2 ? 2 : 4, kValueStages = DB == 2 ? 3 : 6;
    // Tiles of queries: of the item at hand and, with D = 64, the next.  With D = 128 these come when
    // the item's last scores are done, behind the next item's first keys and values.
    static constexpr int kQueryStages = DB == 2 ? 2 : 4;
    static constexpr int kBeforeQueries = DB == 2 ? 1 : 0;
    // TMEM columns of a stage's O and scores; the first kScores of them are places of their own
    static constexpr int kScores = DB == 2 ? 1 : 2;
    __device__ static constexpr uint32_t out_col(int stage) { return stage * kCols; }
    __device__ static constexpr uint32_t score_col(int stage) { return 2 * kCols + (kScores > 1 ? stage * 128 : 0); }
    static_assert(2 * kCols + kScores * 128 <= kWeightCol, "tensor memory");
    static constexpr size_t kOffKeys = size_t(kQueryStages) * kBytes;
    static constexpr size_t kOffValues = kOffKeys + size_t(kKeyStages) * kBytes;
    static constexpr size_t kOffBars = kOffValues + size_t(kValueStages) * kBytes;
    static constexpr size_t kSmem = kOffBars + sizeof(Bars);
    static_assert(kSmem <= 232448, "shared memory budget of one sm_103a CTA");
};

// A CTA's share of the units of all items, walked item by item.  After next() returned true the
// part is tiles [x0, x1) of the item's list.
struct Walk {
    int64_t u;       // first unit behind the part
    int64_t left;    // units of the share behind the part
    int32_t at;      // unit of the item behind the part
    int32_t b, head, item;
    Request r;
    int32_t units_each;         // units of the item
    int32_t token0, tokens;     // of the request
    int32_t tiles, gap, x0, x1;

    __device__ __forceinline__ Walk(const KvAttentionArgs& a, const Bars* bars) {
        left = bars->share;
        u = bars->first_unit;
        b = bars->request;
        head = bars->head;
        item = bars->item;
        at = bars->unit;
        tokens = x0 = x1 = 0;
        if (left > 0) {
            r = bars->first;
            set_item(a);
        }
    }
    __device__ __forceinline__ void set_item(const KvAttentionArgs& a) {
        token0 = item * 2 * a.tile_tokens;
        tokens = r.tokens(a, item);
        tiles = r.tiles(a, item);
        gap = r.gap(a, r.len + token0);
        units_each = tiles + kItemCost;
    }
    __device__ __forceinline__ bool next(const KvAttentionArgs& a) {
        do {
            if (left <= 0) return false;
            if (at == units_each) {
                at = 0;
                if (++item == r.items) {
                    item = 0;
                    if (++head == a.num_kv_heads) {
                        head = 0;
                        do r.load(a, ++b);  // units are left: a request further on has them
                        while (r.n == 0);
                    }
                }
                set_item(a);
            }
            const int32_t take = static_cast<int32_t>(min(static_cast<int64_t>(units_each - at), left));
            x0 = max(at - kItemCost, 0);
            at += take;
            x1 = max(at - kItemCost, 0);
            u += take;
            left -= take;
        } while (x1 == x0);  // a share can end within an item's first units
        return true;
    }
    // Whether the item reads any of the positions pos .. pos + count - 1 of one page: those past its
    // last token may have no page yet, and the pages between the first tokens and the window none
    // any more.
    __device__ __forceinline__ bool reads(const KvAttentionArgs& a, int64_t pos, int32_t count) const {
        if (pos >= r.len + token0 + tokens) return false;
        return a.window == 0 || pos < a.sinks || pos + count > r.len + token0 - a.window + 1;
    }
};

// Counts the units of all requests and cuts out the CTA's share; every thread sums a run of
// requests, and a warp finds the item within the request.  (Loops that are not unrolled and calls:
// the code runs once, and is fetched for that.)
__device__ __forceinline__ void plan(const KvAttentionArgs& a, Bars* bars) {
    const int64_t per = (static_cast<int64_t>(a.batch) + kThreads - 1) / kThreads, all = a.batch;
    const int b0 = static_cast<int>(min(threadIdx.x * per, all));
    const int b1 = static_cast<int>(min(b0 + per, all));
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t sum = 0, at = 0, u = -1, ctas = 0, total = 0;
    if (threadIdx.x == 0) bars->share = 0;
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {
#pragma unroll 1
        for (int b = b0; b < b1; ++b) {
            Request r;
            if (!r.load(a, b) && pass == 0) report(a.status, PKM_ERR_OUT_OF_RANGE);
            const int64_t each = r.head_units(a), units = each * a.num_kv_heads;
            if (pass == 0) {
                sum += units;
            } else if (u < at + units) {
                bars->first_unit = u;
                bars->share = quotient(total * (blockIdx.x + 1), ctas) - u;
                bars->request = b;
                bars->first = r;
                bars->each = each;
                bars->into = u - at;
                break;
            }
            at += units;
        }
        if (pass == 1) break;
        int64_t incl = sum;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int64_t o = __shfl_up_sync(0xffffffffu, incl, sh);
            if (lane >= sh) incl += o;
        }
        if (lane == 31) bars->scratch[warp] = incl;
        __syncthreads();
        int64_t before = 0;
#pragma unroll 1
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) before += bars->scratch[w];
            total += bars->scratch[w];
        }
        ctas = min(static_cast<int64_t>(gridDim.x), total);
        if (threadIdx.x == 0) {
            bars->units = total;
            bars->ctas = static_cast<int32_t>(ctas);
        }
        if (blockIdx.x < ctas) u = quotient(total * blockIdx.x, ctas);
        at = before + incl - sum;
        if (u < at || u >= at + sum) break;
    }
    __syncthreads();
    if (warp != 0 || bars->share == 0) return;
    const Request r = bars->first;
    const int64_t head = quotient(bars->into, bars->each), into = bars->into - head * bars->each;
    int64_t lo = 0, n = r.items, passed = 0;  // the last item with no more units before it
#pragma unroll 1
    while (n > 1) {
        const int64_t step = (n + 31) / 32, j = lane * step;
        const int64_t units = j < n ? r.units_before(a, lo + j) : INT64_MAX;
        const uint32_t below = __ballot_sync(0xffffffffu, units <= into);
        const int k = 31 - __clz(static_cast<int>(below));
        passed = __shfl_sync(0xffffffffu, units, k);
        lo += k * step;
        n = min(step, n - k * step);
    }
    if (lane == 0) {
        bars->head = static_cast<int32_t>(head);
        bars->item = static_cast<int32_t>(lo);
        bars->unit = static_cast<int32_t>(into - passed);
    }
}

// Asks for the arrays that the first loads depend on one after the other (offsets, lengths, page
// table) to be brought into L2, all at once and before they may be read.
__device__ __forceinline__ void prefetch_tables(const KvAttentionArgs& a) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t line = t * 32;  // 32-bit entries
    if (line <= a.batch) prefetch_l2(a.row_offsets + line);
    if (line < a.batch) prefetch_l2(a.cache_lengths + line);
    if (line < static_cast<int64_t>(a.batch) * a.max_pages) prefetch_l2(a.page_table + line);
}

// Page and slot of position pos of request b if it is read.  The page's number is on its way until
// it is asked for: -1 (loads as zeros) if nothing is read and for ids that the cache does not have,
// which are reported.
struct Place {
    uint32_t id;
    int32_t slot;
    bool read;
    __device__ __forceinline__ Place(const KvAttentionArgs& a, int b, int64_t pos, bool read_)
        : id(0), slot(0), read(read_) {
        if (!read) return;
        // pos / page_size for positions below 2^33: off by less than 2^-31 before rounding down
        const int64_t lp = a.page_inverse == 0 ? pos : __umul64hi(pos, a.page_inverse);
        slot = static_cast<int32_t>(pos - lp * a.page_size);
        id = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + lp);
    }
    __device__ __forceinline__ int32_t page(const KvAttentionArgs& a) const {
        if (!read) return -1;
        if (id < static_cast<uint32_t>(a.num_pages)) return static_cast<int32_t>(id);
        report(a.status, PKM_ERR_OUT_OF_RANGE);
        return -1;
    }
    // Offset of the slot in the layer, or -1.
    __device__ __forceinline__ int64_t offset(const KvAttentionArgs& a) const {
        const int32_t p = page(a);
        return p < 0 ? -1 : p * a.page_stride + slot * a.slot_stride;
    }
};

// Infinities and NaN of a packed pair of bf16 become zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

// Whether there are any: an exponent of ones carries into the sign's place.
__device__ __forceinline__ bool any_nonfinite(const uint4& v) {
    const auto top = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
    return ((top(v.x) | top(v.y) | top(v.z) | top(v.w)) & 0x80008000u) != 0;
}

// Readies a quarter of a tile of values, 32 rows, for tokens that attend some of them: rows that no
// token attends become zero, infinities and NaN of rows that some tokens attend become zero too, and
// rows that all attend stay.  Returns whether there were any such.  `none` and `all` have a bit a row.
template <int DB>
__device__ __forceinline__ bool look_through(uint32_t tile, int quarter, uint32_t none, uint32_t all) {
    const int lane = threadIdx.x & 31;
    const bool some = (none | all) != ~0u;
    bool found = false;
    // 32 lanes take 512 bytes, four rows of a block; the place in the block does not matter
#pragma unroll 1
    for (int i = 0; i < DB * 8; i += 8) {
        const uint32_t from = tile + (quarter * DB * 8 + i) * 512 + lane * 16;
        const auto row = [&](int k) -> int {
            const int at = (i + k) * 4 + (lane >> 3);  // among all blocks' rows
            return at / (8 * DB) * 8 + (at & 7);
        };
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (none >> row(k) & 1u) st_shared_v4(from + k * 512, 0u, 0u, 0u, 0u);
        if (!some) continue;
        uint4 v[8];
        bool bad = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = ld_shared_v4(from + k * 512);
#pragma unroll
        for (int k = 0; k < 8; ++k) bad = bad || any_nonfinite(v[k]);
        if (!bad) continue;
#pragma unroll 1
        for (int k = 0; k < 8; ++k) {
            const uint4 w = ld_shared_v4(from + k * 512);
            if (!any_nonfinite(w) || (all >> row(k) & 1u)) continue;
            found = true;
            st_shared_v4(from + k * 512, finite2(w.x), finite2(w.y), finite2(w.z), finite2(w.w));
        }
    }
    return __any_sync(0xffffffffu, found);
}

// The tiles that not all tokens of a tile of queries attend, the first of them at position p: from
// `diagonal` on, and those with keys behind the first tokens (from tile `sinks` on) up to the
// window's `edge`.
struct Masked {
    int32_t diagonal, sinks, edge;
    __device__ __forceinline__ Masked(const KvAttentionArgs& a, int64_t p, int32_t count)
        : diagonal(static_cast<int32_t>((p + 1) >> 7)), sinks(a.sinks >> 7), edge(-1) {
        const int64_t out = p + count - 1 - a.window;  // the last position outside a window
        if (a.window > 0 && out >= 0) edge = static_cast<int32_t>(out >> 7);
    }
    __device__ __forceinline__ Masked(const KvAttentionArgs& a, int32_t d, int32_t e)
        : diagonal(d), sinks(a.sinks >> 7), edge(e) {}
    __device__ __forceinline__ bool any(int32_t kt) const {
        return kt >= diagonal || (kt <= edge && kt >= sinks);
    }
};

// Place in a part's list from which to look for masked tiles behind place x, whose tile is not: over
// those between the diagonal and the window's edge (which has another place in a list with a gap).
__device__ __forceinline__ int32_t past_whole(const Part& p, const Masked& masks, int32_t x) {
    return min(x - 1, masks.edge >= p.lead ? max(masks.edge - p.gap, p.lead - 1) : masks.edge);
}

// Which keys of a tile a token at position p attends: those before `end`, from `lo` on or before
// `sinks`.
struct Attended {
    int32_t end, lo, sinks;
    __device__ __forceinline__ Attended(const KvAttentionArgs& a, int64_t p, int32_t kt) {
        const int64_t c0 = static_cast<int64_t>(kt) * kTile;
        const auto inside = [](int64_t v) -> int32_t {
            return static_cast<int32_t>(min(max(v, static_cast<int64_t>(0)), static_cast<int64_t>(kTile)));
        };
        end = inside(p + 1 - c0);
        lo = a.window > 0 ? inside(p - a.window + 1 - c0) : 0;
        sinks = inside(a.sinks - c0);
    }
    // of the 32 keys from c on
    __device__ __forceinline__ uint32_t bits(int32_t c) const {
        const auto below = [](int32_t n) -> uint32_t {
            return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
        };
        return below(end - c) & (~below(lo - c) | below(sinks - c));
    }
};

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// A value that is the same in every lane of the warp, through a shuffle, from which the compiler
// sees that it is: addresses made of it then use uniform registers, where MMAs take their operands.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __shfl_sync(0xffffffffu, v, 0); }

// Waits with all lanes of a warp; the verdict is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& wc) {
    return __all_sync(0xffffffffu, mbar_wait_inl(bar, parity, wc));
}

template <int DB, bool TMA>
__global__ void __launch_bounds__(kThreads, 1)
    kv_attention_kernel(const __grid_constant__ KvMaps maps, const KvAttentionArgs a,
                        const KvWorkspace ws) {
    using S = Shape<DB>;
    constexpr int D = S::kCols;
    extern __shared__ __align__(1024) uint8_t smem[];  // swizzle atoms of 1024 bytes
    uint8_t *sQ = smem, *sK = smem + S::kOffKeys, *sV = smem + S::kOffValues;
    Bars* bars = reinterpret_cast<Bars*>(smem + S::kOffBars);
    // the same in every lane, seen by the compiler through the shuffle
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kMaxStages; ++i) {
            mbar_init(&bars->k_full[i], 1);
            mbar_init(&bars->k_empty[i], 2);  // both stages
            mbar_init(&bars->v_full[i], 4);   // lanes of the loader, or the warps that look through
            mbar_init(&bars->v_empty[i], 1);
            mbar_init(&bars->v_own[i], 1);
            mbar_init(&bars->q_full[i], 1);
            mbar_init(&bars->q_empty[i], 2);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&bars->s_full[i], 1);
            mbar_init(&bars->s_empty[i], 4);
            mbar_init(&bars->p_full[i], 4);
            mbar_init(&bars->p_empty[i], 1);
            mbar_init(&bars->stats_full[i], 4);
            mbar_init(&bars->o_full[i], 1);
            mbar_init(&bars->o_empty[i], 4);
        }
        for (int i = 0; i < kFound * 4; ++i) bars->nonfinite[i / 4][i % 4] = 0;
        for (int i = 0; i < kParts; ++i) {
            mbar_init(&bars->part_full[i], 1);
            mbar_init(&bars->part_empty[i], 15);  // all warps but the loader
        }
        for (int i = 0; i < 3; ++i) mbar_init(&bars->mma_done[i], 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kLoadWarp && lane == 0) {
        tma_prefetch_map(&maps.q);
        tma_prefetch_map(&maps.q_one);
        if (TMA) {
            tma_prefetch_map(&maps.k);
            tma_prefetch_map(&maps.v);
        }
    }
    if (warp == kScoreWarp) {
        tmem_alloc(&bars->tmem_base, kTmemCols);
        tmem_relinquish();
    }
    prefetch_tables(a);
    griddep_wait();  // launched while the work before may still run: nothing is read before
    plan(a, bars);
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    const WaitCtl wc{&bars->abort_flag, a.status, a.timeout_ns};
    // The softmax warps keep the time limit: whatever stalls stalls them.  The issuing and loading
    // warps' waits end with their abort flag, or after tries that take longer.
    const uint32_t tries = static_cast<uint32_t>(min(a.timeout_ns / 8, uint64_t{UINT32_MAX}));
    const auto issue_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_flag(bar, parity, wc.abort_flag, tries));
    };
    uint32_t parts = 0;  // that the warp has seen
    Part part;
    // Takes the next part; false behind the last one, or when a wait ran out.
    const auto next_part = [&](const auto& wait_part) -> bool {
        const uint32_t at = parts % kParts, phase = (parts / kParts) & 1;
        ++parts;
        if (!wait_part(&bars->part_full[at], phase)) return false;
        part = bars->part[at];
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars->part_empty[at]);
        return __all_sync(0xffffffffu, part.x1 > part.x0);
    };
    uint32_t n = 0;  // steps of the parts before

    if (warp < kScoreWarp) {
        // ---------------- softmax: row = lane of tensor memory ----------------
        warpgroup_reg_alloc<kSoftRegs>();
        const int stage = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const int group = a.num_heads / a.num_kv_heads;
        const int row_token = row / group;
        const float scale2 = a.scale * kLog2e, mul = scale2 > 0.0f ? scale2 : 1.0f;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const uint32_t scores = lanes + S::score_col(stage), weights = lanes + kWeightCol + stage * 64;
        const uint32_t out = lanes + S::out_col(stage);
        uint32_t uses = 0;
        bool next = false;  // the next step's scores are there
        // A wait that runs out is looked at where the next scores have to be waited for, as they have
        // behind it: their issuer leaves too.  What is computed until then is not used.
        bool ok = true;
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            ok = mbar_wait_inl(bar, parity, wc) && ok;
            __syncwarp();
        };
        const auto part_wait = [&](uint64_t* bar, uint32_t parity) -> bool { return warp_wait(bar, parity, wc); };
        while (__all_sync(0xffffffffu, ok) && next_part(part_wait)) {
            const int tiles = part.x1 - part.x0, steps = part.wide ? 2 * tiles : tiles;
            const int mine = stage ^ (n & 1);       // the stage's first step
            const int sub = part.wide ? mine : 0;   // its tile of queries
            const int count = min(a.tile_tokens, part.tokens - sub * a.tile_tokens);
            const bool busy = (warp & 3) * 32 < count * group;  // the warp has rows
            const int64_t pos = part.pos + sub * a.tile_tokens + row_token;
            const Masked masks(a, sub ? part.diagonal[1] : part.diagonal[0], sub ? part.edge[1] : part.edge[0]);
            float m = -INFINITY, l = 0.0f, ref = 0.0f;  // ref: m, or 0 before there is one
            for (int x = mine; x < steps; x += 2) {
                const uint32_t turn = (n + x) >> 1;  // of the stage
                if (!__all_sync(0xffffffffu, next)) {
                    wait(&bars->s_full[stage], turn & 1);
                    if (!__all_sync(0xffffffffu, ok)) break;
                }
                tc_fence_after();
                if (!busy) {
                    next = false;
                    if (lane == 0) mbar_arrive(&bars->s_empty[stage]);
                    if (turn > 0) wait(&bars->p_empty[stage], (turn - 1) & 1);
                    if (lane == 0) mbar_arrive(&bars->p_full[stage]);
                    continue;
                }
                // Masks are put into the scores where they lie, and so is a scale that is not positive,
                // which the maximum would have to know: a short loop, since long straight code that runs
                // once in a while is fetched for hundreds of cycles.
                const int32_t kt = part.tile(part.x1 - 1 - (part.wide ? x >> 1 : x));
                if (masks.any(kt) || !(scale2 > 0.0f)) {
                    const Attended may(a, pos, kt);
                    const float factor = scale2 > 0.0f ? 1.0f : scale2;
#pragma unroll 1
                    for (int c = 0; c < kTile; c += 32) {
                        const uint32_t bits = may.bits(c);
                        if (__all_sync(0xffffffffu, bits == ~0u) && factor == 1.0f) continue;
                        uint32_t v[32];
                        if (__all_sync(0xffffffffu, bits == 0)) {
#pragma unroll
                            for (int k = 0; k < 32; ++k) v[k] = __float_as_uint(-INFINITY);
                        } else {
                            tmem_ld_x32(scores + c, v);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 32; ++k)
                                v[k] = __float_as_uint((bits >> k) & 1u ? __uint_as_float(v[k]) * factor : -INFINITY);
                        }
                        tmem_st_x32(scores + c, v);
                    }
                    tmem_st_wait();
                }
                // The second half is on its way while the first half's maximum is taken.
                uint32_t s[4][32];
                tmem_ld_x32(scores, s[0]);
                tmem_ld_x32(scores + 32, s[1]);
                tmem_ld_wait();
#pragma unroll
                for (int c = 0; c < 64; ++c) asm volatile("" : "+r"(s[c >> 5][c & 31]));  // not before
                tmem_ld_x32(scores + 64, s[2]);
                tmem_ld_x32(scores + 96, s[3]);
                const auto f = [&](int c) -> float { return __uint_as_float(s[c >> 5][c & 31]); };
                float t0 = f(0), t1 = f(1), t2 = f(2), t3 = f(3);
#pragma unroll
                for (int c = 4; c < 60; c += 8) {
                    t0 = fmax3(t0, f(c), f(c + 1));
                    t1 = fmax3(t1, f(c + 2), f(c + 3));
                    t2 = fmax3(t2, f(c + 4), f(c + 5));
                    t3 = fmax3(t3, f(c + 6), f(c + 7));
                }
                t0 = fmax3(t0, f(60), f(61));
                t1 = fmax3(t1, f(62), f(63));
                tmem_ld_wait();
#pragma unroll
                for (int c = 64; c < 128; ++c) asm volatile("" : "+r"(s[c >> 5][c & 31]));
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->s_empty[stage]);
                // the stage's step before is done: O holds still, and its weights' place is free
                const bool ready = turn == 0 || mbar_test(&bars->p_empty[stage], (turn - 1) & 1);
#pragma unroll
                for (int c = 64; c < 128; c += 8) {
                    t0 = fmax3(t0, f(c), f(c + 1));
                    t1 = fmax3(t1, f(c + 2), f(c + 3));
                    t2 = fmax3(t2, f(c + 4), f(c + 5));
                    t3 = fmax3(t3, f(c + 6), f(c + 7));
                }
                const float top = fmaxf(fmax3(t0, t1, t2), t3) * mul;
                const bool move = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
                if (__any_sync(0xffffffffu, move || !ready)) {
                    if (turn > 0) wait(&bars->p_empty[stage], (turn - 1) & 1);
                    tc_fence_after();
                    const float back = move && m > -INFINITY ? exp2_approx(m - top) : 1.0f;
                    if (x > mine && __any_sync(0xffffffffu, back != 1.0f)) {
#pragma unroll 1
                        for (int c = 0; c < D; c += 16) {
                            uint32_t o[16];
                            tmem_ld_x16(out + c, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * back);
                            tmem_st_x16(out + c, o);
                        }
                    }
                    l *= back;
                    if (move) m = ref = top;
                }
                tc_fence_after();
                // The weights are rounded to bf16, by up to 2^-8 of each: the second product's
                // operands have one type, and the values are bf16.  Their sum stays in fp32, unrounded.
                // Sixteen at a time go through the same operation: written value by value, the order
                // that comes out waits for every exponential, 1550 cycles a step instead of 930.
                float sum[4] = {};
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t p[32];
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        float e[16];
#pragma unroll
                        for (int k = 0; k < 16; k += 2)
                            fma2x(e[k], e[k + 1], f(h * 64 + g * 16 + k), f(h * 64 + g * 16 + k + 1), mul, mul,
                                  -ref, -ref);
#pragma unroll
                        for (int k = 0; k < 16; ++k) e[k] = exp2_approx(e[k]);
#pragma unroll
                        for (int k = 0; k < 8; ++k) {
                            add2(sum[2 * (k & 1)], sum[2 * (k & 1) + 1], e[2 * k], e[2 * k + 1]);
                            p[g * 8 + k] = pack_bf16x2(e[2 * k], e[2 * k + 1]);
                        }
                    }
                    tmem_st_x32(weights + h * 32, p);
                }
                l += ((sum[0] + sum[2]) + (sum[1] + sum[3]));
                next = mbar_test(&bars->s_full[stage], (turn + 1) & 1);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->p_full[stage]);
            }
            n += steps;
            if (mine >= steps || !__all_sync(0xffffffffu, ok)) continue;
            if (uses > 0) wait(&bars->o_empty[stage], (uses - 1) & 1);  // read with its O
            bars->stats[stage][row] = make_float2(m, l);
            ++uses;
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->stats_full[stage]);
        }
    } else if (warp < kEndWarp) {
        warpgroup_reg_dealloc<kIssueRegs>();
      if (warp < kLoadWarp) {
        // ---------------- MMA issuers, all lanes together ----------------
        // The tensor cores queue little work ahead, so what a warp needs for its waits and
        // descriptors has to go by during the others' MMAs.
        // A wait that runs out is looked at once a step; what is issued until then is not used.
        bool failed = false;
        const auto wait = [&](uint64_t* bar, uint32_t parity) {
            failed |= !mbar_wait_flag(bar, parity, wc.abort_flag, tries);
        };
        const auto go_on = [&] { return !__any_sync(0xffffffffu, failed); };
        RingPos at;
        if (warp < kOutWarp) {
            // The scores of a stage.  Both stages wait for all keys and queries and release them, the
            // other stage's too: a wait cannot tell a phase from the one two before or behind, so
            // that neither may miss one.
            const uint32_t stage = warp & 1;
            const uint32_t id = idesc_bf16(128, kTile, false, false);
            const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, DB * 1024);
            const uint32_t d = tmem + S::score_col(stage);
            uint32_t queries = 0;
            const auto pass = [&] {  // over a tile of the other stage
                wait(&bars->k_full[at.stage], at.phase);
                if (lane == 0) mbar_arrive(&bars->k_empty[at.stage]);
                __syncwarp();
                at.next(S::kKeyStages);
            };
            while (go_on() && next_part(issue_wait)) {
                const bool wide = __any_sync(0xffffffffu, part.wide != 0);
                const int tiles = __shfl_sync(0xffffffffu, part.x1 - part.x0, 0), steps = wide ? 2 * tiles : tiles;
                const int mine = (n & 1) ^ stage;  // the stage's first step
                const uint32_t query = queries + (wide ? mine : 0);
                for (uint32_t q = queries; q < queries + (wide ? 2 : 1); ++q) {
                    wait(&bars->q_full[q % S::kQueryStages], (q / S::kQueryStages) & 1);
                    if ((wide ? q != query : mine >= steps) && lane == 0)
                        mbar_arrive(&bars->q_empty[q % S::kQueryStages]);
                    __syncwarp();
                }
                if (!wide && mine == 1) pass();
#pragma unroll 1
                for (int x = mine; x < steps; x += 2) {
                    const uint64_t qd = desc_add_bytes(q_desc, uniform(query % S::kQueryStages) * S::kBytes);
                    const uint64_t kd = desc_add_bytes(k_desc, uniform(at.stage) * S::kBytes);
                    wait(&bars->k_full[at.stage], at.phase);
                    // the scores that were in the place before have been read
                    const uint32_t before = n + x - S::kScores;
                    if (n + x >= S::kScores) wait(&bars->s_empty[before & 1], (before >> 1) & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int kb = 0; kb < DB; ++kb)
                        mma4_bf16_elect<2, 2>(d, desc_add_bytes(qd, kb * 16384), desc_add_bytes(kd, kb * 1024), id, kb);
                    mma_commit_elect(&bars->s_full[stage]);
                    if (x + 2 >= steps) mma_commit_elect(&bars->q_empty[query % S::kQueryStages]);
                    mma_commit_elect(&bars->k_empty[at.stage]);
                    at.next(S::kKeyStages);
                    if (!wide && x + 1 < steps) pass();
                    if (!go_on()) break;
                }
                n += steps;
                queries += wide ? 2 : 1;
            }
        } else {
            const uint32_t id = idesc_bf16(128, D, false, true);
            const uint64_t v_desc = sdesc_sw128(smem_u32(sV), 1024, DB * 1024);
            uint32_t empty_phase = 3;  // a bit for each stage; the first wait passes
            while (go_on() && next_part(issue_wait)) {
                const bool wide = __any_sync(0xffffffffu, part.wide != 0);
                const int tiles = __shfl_sync(0xffffffffu, part.x1 - part.x0, 0), steps = wide ? 2 * tiles : tiles;
#pragma unroll 1
                for (int x = 0; x < steps; ++x, ++n) {
                    const uint32_t stage = uniform(n & 1);
                    const bool odd = wide && (x & 1);
                    const uint64_t vd = desc_add_bytes(v_desc, uniform(at.stage) * S::kBytes);
                    const uint32_t d = tmem + S::out_col(stage), p = tmem + kWeightCol + stage * 64;
                    if (!odd) wait(&bars->v_full[at.stage], at.phase);
                    if (x < 2) {
                        wait(&bars->o_empty[stage], empty_phase >> stage & 1);
                        empty_phase ^= 1u << stage;
                    }
                    wait(&bars->p_full[stage], (n >> 1) & 1);
                    tc_fence_after();
#pragma unroll 1
                    for (int h = 0; h < 2; ++h)  // 16 keys: two atoms of each block
                        mma4_bf16_ts_elect<DB * 128>(d, p + 32 * h, desc_add_bytes(vd, h * 8 * DB * 1024), id,
                                                     (x >> 1) | h);
                    mma_commit_elect(&bars->p_empty[stage]);
                    if (x + 2 >= steps) mma_commit_elect(&bars->o_full[stage]);
                    if (!wide || odd) {
                        mma_commit_elect(&bars->v_empty[at.stage]);
                        at.next(S::kValueStages);
                    }
                    if (!go_on()) break;
                }
            }
        }
        uint64_t* mma_done = &bars->mma_done[warp - kScoreWarp];
        mma_commit_elect(mma_done);
        mbar_wait_inl(mma_done, 0, wc, false);
      } else {
        // ---------------- schedule, queries, keys, values ----------------
        Walk w(a, bars);
        const int group = a.num_heads / a.num_kv_heads;
        const int64_t sharing = bars->ctas;
        RingPos kpos, vpos;
        uint32_t queries = 0;
        bool ok = true, more = true;
        const auto publish = [&]() -> bool {
            const uint32_t at = parts % kParts;
            if (!issue_wait(&bars->part_empty[at], ((parts / kParts) & 1) ^ 1)) return false;
            ++parts;
            more = __any_sync(0xffffffffu, w.next(a));
            int left = 0;
            if (more && w.x0 == 0 && w.x1 < w.tiles) {
                // those behind this CTA whose shares begin before the item's end: floor(units c / sharing) < end
                const int64_t end = (w.u + (w.units_each - w.at)) * sharing, units = bars->units;
                uint32_t begin = ~0u;
                left = 1;
                for (int64_t c = blockIdx.x + 1 + lane; begin == ~0u; c += 32) {
                    begin = __ballot_sync(0xffffffffu, c < sharing && units * c < end);
                    left += __popc(begin);
                }
            }
            if (lane == 0) {
                Part* p = &bars->part[at];
                p->x0 = p->x1 = 0;
                if (more) {
                    const bool wide = w.tokens > a.tile_tokens;
                    p->pos = w.r.len + w.token0;
                    p->row = static_cast<int32_t>(w.r.first) + w.token0;
                    p->b = w.b;
                    p->tokens = w.tokens;
                    p->head = w.head;
                    p->x0 = w.x0;
                    p->x1 = w.x1;
                    p->lead = w.gap > 0 ? a.sink_tiles : INT32_MAX;
                    p->gap = w.gap;
                    p->wide = wide;
                    p->whole = w.x0 == 0 && w.x1 == w.tiles;
                    p->left = left;
                    for (int i = 0; i < 2; ++i) {
                        const Masked m(a, p->pos + i * a.tile_tokens,
                                       min(a.tile_tokens, w.tokens - i * a.tile_tokens));
                        p->diagonal[i] = m.diagonal;
                        p->edge[i] = m.edge;
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&bars->part_full[at]);
            return more;
        };
        const auto load_queries = [&]() -> bool {
            const int subs = w.tokens > a.tile_tokens ? 2 : 1;
            for (int sub = 0; sub < subs; ++sub, ++queries) {
                const uint32_t q = queries % S::kQueryStages;
                if (!issue_wait(&bars->q_empty[q], ((queries / S::kQueryStages) & 1) ^ 1)) return false;
                const int32_t token0 = w.token0 + sub * a.tile_tokens;
                const bool one = w.tokens - sub * a.tile_tokens == 1;
                if (lane == 0)
                    mbar_arrive_expect_tx(&bars->q_full[q], DB * 128 * group * (one ? 1 : a.tile_tokens));
                __syncwarp();
                if (lane < DB)
                    tma_load_3d(sQ + q * S::kBytes + lane * 16384, one ? &maps.q_one : &maps.q,
                                &bars->q_full[q], lane * 64, w.head * group,
                                static_cast<int32_t>(w.r.first + token0));
            }
            return true;
        };
        if constexpr (TMA) {
            const int slots = maps.slots, boxes = kTile / slots;
            while (ok && publish()) {
                const Masked masks(a, w.r.len + w.token0, w.tokens);
                const int32_t lead = w.gap > 0 ? a.sink_tiles : INT32_MAX;
                const int before = max(w.x1 - S::kBeforeQueries, w.x0);  // the last tile before the queries
                if (S::kBeforeQueries == 0) ok = load_queries();
                for (int x = w.x1 - 1; ok && x >= w.x0; --x) {
                    const int32_t kt = x >= lead ? x + w.gap : x;
                    const int64_t pos = static_cast<int64_t>(kt) * kTile + lane * slots;
                    const Place place(a, w.b, pos, lane < boxes && w.reads(a, pos, slots));
                    const int32_t page = place.page(a);
                    ok = issue_wait(&bars->k_empty[kpos.stage], kpos.phase ^ 1);
                    if (!ok) break;
                    if (lane == 0) mbar_arrive_expect_tx(&bars->k_full[kpos.stage], S::kBytes);
                    __syncwarp();
                    const uint32_t box = lane * slots * DB * 128;
                    if (lane < boxes)
                        tma_load_5d(sK + kpos.stage * S::kBytes + box, &maps.k, &bars->k_full[kpos.stage], 0, 0,
                                    w.head * DB, place.slot >> 3, page);
                    kpos.next(S::kKeyStages);
                    ok = issue_wait(&bars->v_empty[vpos.stage], vpos.phase ^ 1);
                    if (!ok) break;
                    const bool masked = masks.any(kt);
                    uint64_t* bar = masked ? &bars->v_own[vpos.stage] : &bars->v_full[vpos.stage];
                    if (lane == 0) mbar_arrive_expect_tx(bar, S::kBytes);
                    else if (!masked && lane < 4) mbar_arrive(bar);
                    __syncwarp();
                    if (lane < boxes)
                        tma_load_5d(sV + vpos.stage * S::kBytes + box, &maps.v, bar, 0, 0, w.head * DB,
                                    place.slot >> 3, page);
                    vpos.next(S::kValueStages);
                    if (S::kBeforeQueries > 0 && x == before) ok = load_queries();
                }
            }
        } else {
            // Row by row: a row's 16-byte chunks to their places in the swizzled atoms, keys and values
            // of a tile together, since a row's place is found once for both.  A tile is handed over
            // when the next one is on its way, or before any longer wait.  Bound by the warp's
            // instructions, 6 500 cycles a tile with D = 128: a chunk behind 16 384 keys takes 2.3 times
            // as long as by TMA, single tokens 1.8 times (keys and values each by themselves, every
            // row's page asked for when it is due: 3.1 to 3.6 times).
            bool pending = false, pending_masked = false;
            uint32_t pending_keys = 0, pending_values = 0;
            const auto hand_over = [&] {
                __syncwarp();
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&bars->k_full[pending_keys]);
                if (pending_masked) {
                    if (lane == 0) mbar_arrive(&bars->v_own[pending_values]);
                } else if (lane < 4) {
                    mbar_arrive(&bars->v_full[pending_values]);
                }
                pending = false;
            };
            const auto flush = [&] {
                cp_async_wait<0>();
                if (pending) hand_over();
            };
            constexpr int kChunks = DB * 8, kRows = 32 / kChunks;  // of a row; rows at once
            const int chunk = lane % kChunks, first = lane / kChunks;
            while (ok) {
                flush();
                if (!publish()) break;
                const Masked masks(a, w.r.len + w.token0, w.tokens);
                const int32_t lead = w.gap > 0 ? a.sink_tiles : INT32_MAX;
                const uint16_t* columns = a.cache_layer + w.head * D + chunk * 8;
                const auto place_of = [&](int x, int k) -> Place {  // of the lane's row of 32
                    const int64_t pos = static_cast<int64_t>(x >= lead ? x + w.gap : x) * kTile + k * 32 + lane;
                    return Place(a, w.b, pos, x >= w.x0 && w.reads(a, pos, 1));
                };
                Place place = place_of(w.x1 - 1, 0);
                ok = load_queries();
                for (int x = w.x1 - 1; ok && x >= w.x0; --x) {
                    const int32_t kt = x >= lead ? x + w.gap : x;
                    uint64_t *k_empty = &bars->k_empty[kpos.stage], *v_empty = &bars->v_empty[vpos.stage];
                    if (!__all_sync(0xffffffffu,
                                    mbar_try_wait(k_empty, kpos.phase ^ 1) && mbar_try_wait(v_empty, vpos.phase ^ 1))) {
                        flush();
                        ok = issue_wait(k_empty, kpos.phase ^ 1) && issue_wait(v_empty, vpos.phase ^ 1);
                        if (!ok) break;
                    }
                    uint32_t keys = smem_u32(sK) + kpos.stage * S::kBytes + (chunk >> 3) * 1024;
                    uint32_t values = smem_u32(sV) + vpos.stage * S::kBytes + (chunk >> 3) * 1024;
#pragma unroll 1
                    for (int k = 0; k < 4; ++k) {
                        int64_t offset = place.offset(a);
                        place = place_of(k < 3 ? x : x - 1, (k + 1) & 3);  // comes during these rows
                        const uint32_t there = __ballot_sync(0xffffffffu, offset >= 0) >> first;
                        if (offset < 0) offset = 0;
#pragma unroll 1
                        for (int i = 0; i < 32; i += 8) {
#pragma unroll
                            for (int j = 0; j < 8; j += kRows) {
                                const int r = j + first;  // of the atom
                                const uint16_t* from = columns + __shfl_sync(0xffffffffu, offset, i + r);
                                const uint32_t to = r * 128 + (((chunk & 7) ^ r) << 4), bytes = (there >> (i + j) & 1u) * 16;
                                cp_async_16(keys + to, from, bytes);
                                cp_async_16(values + to, from + a.kv_stride, bytes);
                            }
                            keys += DB * 1024;
                            values += DB * 1024;
                        }
                    }
                    cp_async_commit();
                    if (pending) {
                        cp_async_wait<1>();
                        hand_over();
                    }
                    pending = true;
                    pending_masked = masks.any(kt);
                    pending_keys = kpos.stage;
                    pending_values = vpos.stage;
                    kpos.next(S::kKeyStages);
                    vpos.next(S::kValueStages);
                }
            }
            flush();
        }
        if (*wc.abort_flag) spin_ns(kDrainNs);
      }
    } else {
        // ---------------- values looked through, and the epilogue ----------------
        warpgroup_reg_dealloc<kEndRegs>();
        const int row = (warp & 3) * 32 + lane;
        const int group = a.num_heads / a.num_kv_heads;
        const int row_token = row / group, row_head = row - row_token * group;
        const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        // A part can take longer than the time limit, which the softmax warps keep step by step: the
        // epilogue's waits end with the abort flag, or after many times the limit.
        const auto end_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
            bool done = false;
#pragma unroll 1
            for (int i = 0; i < 64 && !done && !*wc.abort_flag; ++i)
                done = mbar_wait_flag(bar, parity, wc.abort_flag, tries);
            return __all_sync(0xffffffffu, done);
        };
        uint32_t tiles_before = 0, own_phase = 0;
        uint32_t use = 0;  // phases of the stages' uses, a bit each
        KvItem left{0, 0, 0, 0};
        bool ok = true;
        Part now;
        uint32_t number = 0;  // of the part `now`; 0 before the first
        int x = 0;
        uint32_t looked = 0, found = 0;  // tiles of the part looked through, and what the warp found there
        const auto note = [&](uint32_t part, uint32_t tiles) {
            *const_cast<volatile uint16_t*>(&bars->nonfinite[part % kFound][warp & 3]) =
                static_cast<uint16_t>(part << kFoundBits | tiles);
        };
        while (true) {
            // Values of tiles with keys that not every token attends are looked through, from a part's
            // last tile: those at the diagonal, then those at the window's edge and between it and the
            // first tokens.  The next part's diagonal comes before this part's epilogue, for which it
            // need not wait.
            bool more = true;
            const uint32_t following = number + 1;
            Part p = now;
#pragma unroll 1
            for (int turn = number > 0 ? 0 : 1; ok && turn < 2; ++turn) {
                if (turn == 1) {
                    if (number > 0) tiles_before += now.x1 - now.x0;
                    more = next_part(end_wait);
                    if (!more) break;
                    p = part;
                    x = p.x1 - 1;
                    looked = found = 0;
                    if (lane == 0) note(following, 0);
                }
                const Masked masks(a, p.diagonal[0], p.wide ? p.edge[1] : p.edge[0]);
#pragma unroll 1
                while (x >= p.x0) {
                    const int32_t kt = p.tile(x);
                    if (kt < (turn == 1 ? masks.diagonal : masks.sinks)) break;
                    if (!masks.any(kt)) {
                        x = past_whole(p, masks, x);
                        continue;
                    }
                    const uint32_t tile = tiles_before + (p.x1 - 1 - x), at = tile % S::kValueStages;
                    ok = end_wait(&bars->v_own[at], (own_phase >> at) & 1);
                    if (!ok) break;
                    own_phase ^= 1u << at;
                    // the key of the lane's row, and whether any token attends it, and all
                    const int64_t key = static_cast<int64_t>(kt) * kTile + row, last = p.pos + p.tokens - 1;
                    const bool sink = a.window == 0 || key < a.sinks;
                    const uint32_t none =
                        __ballot_sync(0xffffffffu, key > last || !(sink || key > p.pos - a.window));
                    const uint32_t all = __ballot_sync(0xffffffffu, key <= p.pos && (sink || key > last - a.window));
                    const uint32_t of = turn == 1 ? following : number;
                    if (look_through<DB>(smem_u32(sV) + at * S::kBytes, warp & 3, none, all)) {
                        found |= 1u << looked;
                        if (lane == 0) note(of, found);
                    }
                    ++looked;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&bars->v_full[at]);
                    --x;
                }
            }
            if (!ok || (number == 0 && !more)) break;
            if (number == 0) {
                now = p;
                number = 1;
                continue;
            }
            const int tiles = now.x1 - now.x0, steps = now.wide ? 2 * tiles : tiles;
            const int first = n & 1;             // the first step's stage
            const bool join = !now.wide && steps > 1;
            n += steps;
            for (int sub = 0; ok && sub < (now.wide ? 2 : 1); ++sub) {
                const int stage = first ^ sub;
                // maxima and sums of a stage's use, and its O complete
                const auto take = [&](int stage, float2& st) -> bool {
                    const uint32_t phase = use >> stage & 1;
                    use ^= 1u << stage;
                    if (!end_wait(&bars->stats_full[stage], phase) || !end_wait(&bars->o_full[stage], phase)) return false;
                    st = bars->stats[stage][row];
                    return true;
                };
                float2 st, so;
                float f0 = 1.0f, f1 = 0.0f;  // factors of this stage's sums and of the other's
                ok = take(stage, st) && (!join || take(stage ^ 1, so));
                if (!ok) break;
                if (join) {
                    const float top = fmaxf(st.x, so.x);
                    f0 = st.x == -INFINITY ? 0.0f : exp2_approx(st.x - top);
                    f1 = so.x == -INFINITY ? 0.0f : exp2_approx(so.x - top);
                    st = make_float2(top, st.y * f0 + so.y * f1);
                }
                tc_fence_after();
                const int count = min(a.tile_tokens, now.tokens - sub * a.tile_tokens);
                const bool valid = row_token < count, whole = now.whole != 0;
                const float inv = whole ? rcp_approx(st.y) : 1.0f;  // a sum of 0, all scores -inf: NaN
                // tiles whose quarter had infinities or NaN
                const auto had = [&](int quarter) -> uint32_t {
                    const uint32_t w = *const_cast<volatile uint16_t*>(&bars->nonfinite[number % kFound][quarter]);
                    return w >> kFoundBits == (number & 255u) ? w & ((1u << kFoundBits) - 1u) : 0u;
                };
                const uint32_t mend = had(0) | had(1) | had(2) | had(3);
                const int64_t out_row =
                    (static_cast<int64_t>(now.row) + sub * a.tile_tokens + row_token) * a.num_heads +
                    now.head * group + row_head;
                const int64_t slot = 2 * static_cast<int64_t>(blockIdx.x) + (now.x0 > 0 ? 0 : 1);
                const int slot_row = sub * kTile + row;
                if ((warp & 3) * 32 < count * group) {
#pragma unroll 1
                    for (int c = 0; c < D; c += 16) {
                        uint32_t o[16];
                        tmem_ld_x16(lanes + S::out_col(stage) + c, o);
                        if (join) {
                            uint32_t o1[16];
                            tmem_ld_x16(lanes + S::out_col(stage ^ 1) + c, o1);
                            tmem_ld_wait();
#pragma unroll
                            for (int k = 0; k < 16; ++k)
                                o[k] = __float_as_uint(__uint_as_float(o[k]) * f0 + __uint_as_float(o1[k]) * f1);
                        } else {
                            tmem_ld_wait();
                        }
                        if (valid && whole) {
                            uint32_t h[8];
#pragma unroll
                            for (int k = 0; k < 8; ++k)
                                h[k] = pack_bf16x2(__uint_as_float(o[2 * k]) * inv, __uint_as_float(o[2 * k + 1]) * inv);
                            uint16_t* to = a.out + out_row * D + c;
                            if (sectors) {
                                st_v8(to, h);
                            } else {
                                st_v4(to, make_uint4(h[0], h[1], h[2], h[3]));
                                st_v4(to + 8, make_uint4(h[4], h[5], h[6], h[7]));
                            }
                        } else if (valid) {
                            float* to = reinterpret_cast<float*>(a.workspace) + (slot * ws.rows + slot_row) * D + c;
                            st_v8(to, o);
                            st_v8(to + 8, o + 8);
                        }
                        __syncwarp();
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&bars->o_empty[stage]);
                    if (join) mbar_arrive(&bars->o_empty[stage ^ 1]);
                }
                if (mend != 0 && (warp & 3) * 32 < count * group) {
                    // Infinities and NaN that were made zero for the rows that do not attend them.  The
                    // warp reads the values again, only in the quarters of tiles that had any; each lane
                    // gathers which columns of its row meet +inf and -inf (NaN: both), and a column gets
                    // its sum once.  (2048 tokens behind 16 384 with NaN for all new values: 414 us instead
                    // of 369; a chunk of 4096 in a window of 1024: 517 instead of 197.)
                    constexpr int kChunks = DB * 8, kRows = 32 / kChunks;  // of a row; rows of a load
                    constexpr int kAhead = 4;  // loads at once (2 and 8: calls full of NaN 2 to 10 % longer)
                    const Masked masks(a, now.diagonal[0], now.wide ? now.edge[1] : now.edge[0]);
                    const int64_t pos = now.pos + sub * a.tile_tokens + row_token, last = now.pos + now.tokens - 1;
                    uint32_t up[2 * DB], down[2 * DB];  // a bit a column
#pragma unroll
                    for (int w = 0; w < 2 * DB; ++w) up[w] = down[w] = 0;
                    uint32_t bit = 1;  // of the tile
#pragma unroll 1
                    for (int y = now.x1 - 1; y >= now.x0 && bit <= mend;) {
                        const int32_t kt = now.tile(y);
                        if (!masks.any(kt)) {
                            y = past_whole(now, masks, y);
                            continue;
                        }
#pragma unroll 1
                        for (int quarter = 0; quarter < 4; ++quarter) {
                            if ((had(quarter) & bit) == 0) continue;
                            const int64_t key0 = static_cast<int64_t>(kt) * kTile + quarter * 32, key = key0 + lane;
                            // of the keys that some token of the item attends
                            const bool read =
                                key <= last && (a.window == 0 || key < a.sinks || key > now.pos - a.window);
                            const int64_t at = Place(a, now.b, key, read).offset(a);
#pragma unroll 1
                            for (int i = 0; i < 32; i += kAhead * kRows) {
                                uint4 v[kAhead];
#pragma unroll
                                for (int j = 0; j < kAhead; ++j) {
                                    const int64_t from = __shfl_sync(0xffffffffu, at, i + j * kRows + lane / kChunks);
                                    v[j] = make_uint4(0u, 0u, 0u, 0u);
                                    if (from >= 0)
                                        v[j] = ld_nc_v4(a.cache_layer + a.kv_stride + from + now.head * D +
                                                        lane % kChunks * 8);
                                }
#pragma unroll
                                for (int j = 0; j < kAhead; ++j) {
                                    if (!__any_sync(0xffffffffu, any_nonfinite(v[j]))) continue;
                                    // the lane's eight columns in their place among 32
                                    uint32_t plus = 0, minus = 0;
#pragma unroll
                                    for (int k = 0; k < 8; ++k) {
                                        const uint32_t w = k < 2 ? v[j].x : k < 4 ? v[j].y : k < 6 ? v[j].z : v[j].w;
                                        const uint32_t h = k & 1 ? w >> 16 : w & 0xffffu;
                                        const uint32_t column = 1u << ((lane & 3) * 8 + k);
                                        if ((h & 0x7f80u) != 0x7f80u) continue;
                                        if (h != 0xff80u) plus |= column;
                                        if (h != 0x7f80u) minus |= column;
                                    }
#pragma unroll
                                    for (int sh = 1; sh < 4; sh <<= 1) {
                                        plus |= __shfl_xor_sync(0xffffffffu, plus, sh);
                                        minus |= __shfl_xor_sync(0xffffffffu, minus, sh);
                                    }
#pragma unroll
                                    for (int r = 0; r < kRows; ++r) {
                                        const int64_t k = key0 + i + j * kRows + r;
                                        const bool attends =
                                            k <= pos && (a.window == 0 || k < a.sinks || k > pos - a.window);
#pragma unroll
                                        for (int w = 0; w < 2 * DB; ++w) {
                                            const uint32_t u = __shfl_sync(0xffffffffu, plus, r * kChunks + w * 4);
                                            const uint32_t d = __shfl_sync(0xffffffffu, minus, r * kChunks + w * 4);
                                            if (attends) up[w] |= u, down[w] |= d;
                                        }
                                    }
                                }
                            }
                        }
                        bit <<= 1;
                        --y;
                    }
                    // The stores before are the lane's own.
#pragma unroll
                    for (int w = 0; w < 2 * DB; ++w) {
                        if (!valid) up[w] = down[w] = 0;
#pragma unroll 1
                        for (uint32_t u = up[w], d = down[w], c = w * 32; (u | d) != 0; u >>= 8, d >>= 8, c += 8) {
                            if (((u | d) & 0xffu) == 0) continue;
                            const auto sum = [&](float o, int k) -> float {  // column c + k
                                if ((d >> k & 1u) != 0) o -= INFINITY;
                                return (u >> k & 1u) != 0 ? o + INFINITY : o;
                            };
                            if (whole) {
                                uint4* to = reinterpret_cast<uint4*>(a.out + out_row * D + c);
                                uint4 o = *to;
                                const auto pair = [&](uint32_t h, int k) -> uint32_t {
                                    return pack_bf16x2(sum(__uint_as_float(h << 16), k),
                                                       sum(__uint_as_float(h & 0xffff0000u), k + 1));
                                };
                                o = make_uint4(pair(o.x, 0), pair(o.y, 2), pair(o.z, 4), pair(o.w, 6));
                                *to = o;
                            } else {
                                float4* to = reinterpret_cast<float4*>(reinterpret_cast<float*>(a.workspace) +
                                                                       (slot * ws.rows + slot_row) * D + c);
                                const float4 o0 = to[0], o1 = to[1];
                                to[0] = make_float4(sum(o0.x, 0), sum(o0.y, 1), sum(o0.z, 2), sum(o0.w, 3));
                                to[1] = make_float4(sum(o1.x, 4), sum(o1.y, 5), sum(o1.z, 6), sum(o1.w, 7));
                            }
                        }
                    }
                    __syncwarp();
                }
                if (valid && whole && a.lse != nullptr)
                    a.lse[out_row] = st.y != 0.0f ? (st.x + __log2f(st.y)) * kLn2 : -INFINITY;
                if (valid && !whole)
                    reinterpret_cast<float2*>(a.workspace + ws.stats)[slot * ws.rows + slot_row] = st;
            }
            if (now.left > 0) left = KvItem{now.row, now.head * group, now.tokens, now.left};
            if (!ok || !more) break;
            now = p;
            number = following;
        }
        if (warp == kEndWarp && lane == 0) {
            if (!ok) left.tokens = 0;
            reinterpret_cast<KvItem*>(a.workspace + ws.items)[blockIdx.x] = left;
        }
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == kScoreWarp) tmem_dealloc(tmem, kTmemCols);
}

constexpr int kJoinWarps = 8, kJoinThreads = kJoinWarps * 32;
constexpr int kJoinBlocks = 4;  // of an SM (3: small ragged chunks 3 % longer; 5, which spill: 4, and windows 2 %)
// Rows that a lane joins at a time (with 4, which spill, small ragged chunks take 10 % longer, prompts
// and single tokens in a window 3 to 5 %).
constexpr int kJoinRows = 2;
// Parts that a warp joins alone, and of items of few rows, whose blocks have nothing else to do.
constexpr int kFewParts = 8, kFewRows = 8, kFewPartsOfFewRows = 2;

// Joins the parts of the items that several CTAs share: with M the largest of the parts' maxima,
// out = sum 2^(m_k - M) O_k / sum 2^(m_k - M) l_k, the parts always in the same order.  A lane takes
// four columns of two rows, a warp two or, with D = 64, four rows (of items of few rows two); rows of
// many parts are taken one by one by the warps of a block, which share the parts.  The sums are still
// in L2.  Bound by latency with few rows (7 us by itself, most of it before the launch's end) and by
// its instructions where every CTA leaves 256 rows of an item (39 000 rows of two parts: 14 us).
template <int DB>
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks)
    kv_join_kernel(const KvAttentionArgs a, const KvWorkspace ws, const int ctas) {
    constexpr int D = DB * 64;
    constexpr int kLanes = D / 4, kAtOnce = 32 / kLanes;  // lanes of a row, rows of a load
    const auto task_rows = [](int rows) -> int { return rows > kFewRows ? kJoinRows * kAtOnce : 2; };
    __shared__ KvItem items[kKvMaxCtas];
    __shared__ int begins[2][kKvMaxCtas + 1];  // tasks of items of few parts, and of many
    __shared__ float4 sums[kJoinWarps][32];
    __shared__ float2 totals[kJoinWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = a.num_heads / a.num_kv_heads;
    griddep_launch_dependents();
    griddep_wait();
    const KvItem* left = reinterpret_cast<const KvItem*>(a.workspace + ws.items);
    if (warp < 2) {
        constexpr int kItems = (kKvMaxCtas + 31) / 32;
        int n[kItems], sum = 0;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int p = lane * kItems + k;
            n[k] = 0;
            if (p < ctas) {
                const KvItem it = left[p];
                if (warp == 0) items[p] = it;
                const int rows = it.tokens * group;
                const bool many = it.parts > (rows > kFewRows ? kFewParts : kFewPartsOfFewRows);
                if (many == (warp == 1)) n[k] = many ? rows : (rows + task_rows(rows) - 1) / task_rows(rows);
            }
            sum += n[k];
        }
        int incl = sum;
#pragma unroll
        for (int sh = 1; sh < 32; sh <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, incl, sh);
            if (lane >= sh) incl += o;
        }
        int at = incl - sum;
#pragma unroll
        for (int k = 0; k < kItems; ++k) {
            const int p = lane * kItems + k;
            if (p <= ctas) begins[warp][p] = at;
            at += n[k];
        }
        if (lane == 31) begins[warp][ctas] = incl;
    }
    __syncthreads();
    const float* parts = reinterpret_cast<const float*>(a.workspace);
    const float2* stats = reinterpret_cast<const float2*>(a.workspace + ws.stats);
    const auto find = [&](const int* begin, int f) -> int {  // the item of a task
        int p = 0, behind = ctas;
        while (behind - p > 1) {
            const int mid = (p + behind) / 2;
            if (begin[mid] <= f) p = mid;
            else behind = mid;
        }
        return p;
    };
    struct Row {
        int64_t out;    // its row of the output
        int32_t slot;   // and of a part
    };
    const auto place = [&](const KvItem& it, int row) -> Row {
        const int token = row / group, head = row - token * group, sub = token >= a.tile_tokens ? 1 : 0;
        return Row{(it.row + token) * a.num_heads + it.head + head,
                   sub * kTile + (token - sub * a.tile_tokens) * group + head};
    };
    // part k of the item that CTA p starts: the CTA's second slot, then the first slots of those behind
    const auto slot = [&](int p, int k) -> int64_t {
        return (2 * static_cast<int64_t>(p + k) + (k == 0 ? 1 : 0)) * ws.rows;
    };
    struct Sum {
        float top = -INFINITY, total = 0.0f;
        float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        __device__ __forceinline__ void add(float2 s, float4 v) {
            const float m = fmaxf(top, s.x);
            const float f0 = top == -INFINITY ? 0.0f : exp2_approx(top - m);
            const float f1 = s.x == -INFINITY ? 0.0f : exp2_approx(s.x - m);
            top = m;
            total = total * f0 + s.y * f1;
            o = make_float4(o.x * f0 + v.x * f1, o.y * f0 + v.y * f1, o.z * f0 + v.z * f1, o.w * f0 + v.w * f1);
        }
    };
    const int col = (lane % kLanes) * 4;
    const auto finish = [&](const Sum& x, int64_t out) {
        const float inv = 1.0f / x.total;  // a sum of 0, all scores -inf: NaN
        *reinterpret_cast<uint2*>(a.out + out * D + col) =
            make_uint2(pack_bf16x2(x.o.x * inv, x.o.y * inv), pack_bf16x2(x.o.z * inv, x.o.w * inv));
        if (a.lse != nullptr && col == 0)
            a.lse[out] = x.total != 0.0f ? (x.top + __log2f(x.total)) * kLn2 : -INFINITY;
    };
    for (int f = blockIdx.x * kJoinWarps + warp; f < begins[0][ctas]; f += gridDim.x * kJoinWarps) {
        const int p = find(begins[0], f);
        const KvItem it = items[p];
        const int rows = it.tokens * group, each = task_rows(rows);
        const int row0 = (f - begins[0][p]) * each + lane / kLanes;
        Sum x[kJoinRows];
        Row r[kJoinRows];
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i) r[i] = place(it, min(row0 + i * kAtOnce, rows - 1));
        for (int k = 0; k < it.parts; ++k) {
            float2 s[kJoinRows];
            float4 v[kJoinRows];
#pragma unroll
            for (int i = 0; i < kJoinRows; ++i) {
                if (i * kAtOnce >= each) break;
                const int64_t at = slot(p, k) + r[i].slot;
                s[i] = __ldcg(stats + at);
                v[i] = __ldcg(reinterpret_cast<const float4*>(parts + at * D + col));
            }
#pragma unroll
            for (int i = 0; i < kJoinRows; ++i)
                if (i * kAtOnce < each) x[i].add(s[i], v[i]);
        }
#pragma unroll
        for (int i = 0; i < kJoinRows; ++i)
            if (i * kAtOnce < each && row0 + i * kAtOnce < rows) finish(x[i], r[i].out);
    }
    for (int f = blockIdx.x; f < begins[1][ctas]; f += gridDim.x) {
        const int p = find(begins[1], f);
        const KvItem it = items[p];
        const Row r = place(it, f - begins[1][p]);
        Sum x;
#pragma unroll 4
        for (int k = warp * kAtOnce + lane / kLanes; k < it.parts; k += kJoinWarps * kAtOnce) {
            const int64_t at = slot(p, k) + r.slot;
            x.add(__ldcg(stats + at), __ldcg(reinterpret_cast<const float4*>(parts + at * D + col)));
        }
        if constexpr (kAtOnce == 2) {  // the other half of the lanes had other parts
            const float2 s = make_float2(__shfl_xor_sync(0xffffffffu, x.top, 16), __shfl_xor_sync(0xffffffffu, x.total, 16));
            const float4 v = make_float4(__shfl_xor_sync(0xffffffffu, x.o.x, 16), __shfl_xor_sync(0xffffffffu, x.o.y, 16),
                                         __shfl_xor_sync(0xffffffffu, x.o.z, 16), __shfl_xor_sync(0xffffffffu, x.o.w, 16));
            x.add(s, v);
        }
        if (lane == 0) totals[warp] = make_float2(x.top, x.total);
        sums[warp][lane] = x.o;
        __syncthreads();
        if (warp == 0) {
            Sum y;
            for (int k = 0; k < kJoinWarps; ++k) y.add(totals[k], sums[k][lane]);
            if (lane < kLanes) finish(y, r.out);
        }
        __syncthreads();
    }
}

template <int DB, bool TMA>
cudaError_t launch_shape(const KvMaps& maps, const KvAttentionArgs& args, const KvWorkspace& ws,
                         int ctas, int num_sms, cudaStream_t stream) {
    constexpr size_t smem = Shape<DB>::kSmem;
    // once a device: the attribute stays (every thread sets the same value)
    static std::atomic<uint64_t> set[2] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 128;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!known || !(set[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        // the register split takes what the block starts with
        cudaFuncAttributes attr;
        e = cudaFuncGetAttributes(&attr, kv_attention_kernel<DB, TMA>);
        if (e != cudaSuccess) return e;
        if (attr.numRegs != kStartRegs) return cudaErrorInvalidKernelImage;
        e = cudaFuncSetAttribute(kv_attention_kernel<DB, TMA>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(smem));
        if (e != cudaSuccess) return e;
        if (known) set[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    e = launch_dependent(kv_attention_kernel<DB, TMA>, static_cast<unsigned>(ctas), kThreads, smem,
                         stream, maps, args, ws);
    if (e != cudaSuccess) return e;
    return launch_dependent(kv_join_kernel<DB>, static_cast<unsigned>(num_sms) * kJoinBlocks, kJoinThreads, 0,
                            stream, args, ws, ctas);
}

}  // namespace

cudaError_t launch_kv_attention(const KvMaps& maps, KvAttentionArgs args, int num_sms,
                                cudaStream_t stream) {
    const KvWorkspace ws =
        kv_workspace(args.total_rows, args.num_heads, args.num_kv_heads, args.head_size);
    const int ctas = num_sms < kKvMaxCtas ? num_sms : kKvMaxCtas;
    const bool tma = maps.slots > 0;
    const auto launch = args.head_size == 64 ? (tma ? launch_shape<1, true> : launch_shape<1, false>)
                                             : (tma ? launch_shape<2, true> : launch_shape<2, false>);
    return launch(maps, args, ws, ctas, num_sms, stream);
}

}  // namespace pkm
