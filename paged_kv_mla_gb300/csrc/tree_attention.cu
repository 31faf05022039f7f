// tree_attention.cu -- absorbed MLA attention of new tokens (one, a chain, a drafted tree)
// over the paged latent cache, on CTA pairs.
//
// mla_prefill_decode_graph_fp8 (Modular MAX, attention/gpu/mla_graph), its decode path: Args
// q, input_row_offsets, kv_collection, layer_idx, Parameters scale, mask_str.  Every head of
// a request reads the same latent row L_t (C = R + P columns), so the new tokens' heads are
// the rows of one matrix product, and the same tile of L serves twice:
//     S = Q L^T                  [rows x keys], all C columns
//     O = softmax(scale S) L     [rows x R],    the first R columns of L
//
// An item is 128 query rows (token, head) of one request.  The fp32 accumulator of 128 rows
// x 512 columns would fill the whole tensor memory of an SM, so a pair of CTAs shares an
// item: with tcgen05.mma.cta_group::2, M = 128, each CTA holds 64 rows, spread over all 128
// lanes (lanes 0-63 hold the first half of the columns, lanes 64-127 the second), and 512
// columns of O take 256 TMEM columns, next to two 128-key score tiles of 64.  For S the pair
// splits the keys (each CTA loads 64 keys, all columns), for O the columns (each CTA loads
// all 128 keys, half the columns): a latent value comes from L2 once as key and once as
// value.  What the values cost in loads, the full-rate MMA gives back: the 64-row form of a
// single CTA runs at half the rate.
//
// The key axis of all items is one line of 128-key tiles, cut into equal parts, one for each
// pair: a pair starts at most one item that it does not finish and finishes at most one that
// it did not start.  Such parts leave unnormalised fp32 sums, maxima and totals in the
// workspace and a second kernel joins them; whole items are written directly.
//
// Roles of a CTA: warps 0-7 softmax and epilogue, 8 MMA issue (even CTA), 9 queries, 10 asks for
// keys to be brought into L2 ahead of their loads, 12-15 keys, 16-19 values (by loads 12-19 both).
// Scores are kept in base 2; the running maximum moves only when a row's new maximum exceeds
// it by 2^8, since any reference works as long as nothing overflows, so the accumulator is
// hardly ever rescaled.
//
// What threads write for the MMAs (weights, rows brought by loads, values looked through) each
// CTA's tensor core reads from its own shared memory, on behalf of the even CTA's issuing warp.
// A writer's fence.proxy.async comes first; its arrival at the even CTA's barrier then publishes
// shared memory at cluster scope, and the issuer's waits for such arrivals acquire it.  Both are
// fences for shared memory alone: a cluster-scope release of all memory took 1430 cycles of
// every tile.
//
// Measured (R = 512, P = 64, 128 heads, L2 cold; floor = bytes or operations at the rates of a
// plain copy and a large library product):
//   16 trees of 16-64 tokens, histories of 512-4096: 319 to 324 us, 1.32 PFLOP/s (0.69).  The tensor
//     cores are at work for 65 % of the attention's 291 us: a tile takes 2600 cycles, of which its
//     MMAs 2176, and an item's start and end 5 us more, eight times a pair.  L2 gives 13 TB/s, 52 %
//     of what its counters allow.  The join takes 14 us when nothing overlaps it.
//   64 users x 1 token, histories of 512-4096, pages of 128: 55.5 us, floor 28 us (3.3 TB/s).  1.5
//     items a pair: 10 us to start, 15 us of items' starts and ends, 8 us to join.
//   4 users x 1 token, histories of 32768: 44.8 us, floor 23 us (3.4 TB/s), likewise.
//   32 chains of 1-4 tokens over the quantised cache: 106 us, floor 26 us.  Rows brought by loads
//     are bound by the instructions that convert them: 3 us a tile.  A request's rows are converted
//     for each of its items, 2.6 times here, and half of the values once more for the other CTA.
// The comments at single choices below say what the other side cost when the choice was made.
#include <cuda_fp16.h>

#include <atomic>

#include "pkm_device.cuh"
#include "pkm_internal.h"

namespace pkm {
namespace {

// Pages by TMA, bf16 rows by loads, quantised rows whose codes fill both sets of blocks (a rank of
// 512) and others, whose rope columns lie among them.
enum Source { kTma, kRows, kCodes, kCodesNarrow };

constexpr int kSoftWarps = 8, kMmaWarp = 8, kQueryWarp = 9, kFetchWarp = 10, kKeyWarp = 12, kValueWarp = 16;
constexpr int kThreads = 20 * 32;
// Registers of the four-warp groups (two of softmax warps, the issuing warps, two of loaders), of
// the 5 x 96 that the block starts with: by loads the rows on their way need more.
constexpr int kIssueRegs = 64, kMoreRegs = 112;
// An item's start and end, in tiles: 5 us against 1.4 us of a tile by TMA and 3 us of one by loads
// (large drafted trees with 2: 3 % longer, ragged ones with 6: 6 %; chains over the quantised cache
// with 2: 3 %, with 3: 4 %).
constexpr int item_cost(Source src) { return src == kTma ? 4 : 1; }
constexpr int kKeys = 128;          // keys of a tile (64 loaded by each CTA as keys)
constexpr int kBlocks = 9;          // 64-column blocks of a latent row
constexpr int kBlockBytes = 64 * 128;
constexpr int kKeyGroups = 2;       // key blocks waited for and released together: 0-3, 4-8
constexpr int kQueryBlocks = kTreeKeyBlocks;  // query blocks kept in tensor memory, the others in shared
constexpr int kValueBytes = kKeys * 128;  // one of a CTA's up to four 64-column value blocks
constexpr int kValueRing = 3;       // groups of two value blocks in flight
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kScoreCol = 256; // TMEM column of the first score tile
constexpr uint32_t kQueryCol = 384; // TMEM column of the queries, 32 a block
constexpr uint64_t kDrainNs = 1000000;  // a role that gave up leaves its loads time to land
constexpr float kLazy = 8.0f;       // base-2 growth of a maximum that is let pass
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

// a / b; the 64-bit division is a long routine, and the operands are hardly ever that large.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// One request as the schedule sees it.
struct Request {
    int64_t first;   // its first row
    int32_t n;       // its new tokens
    int64_t len;     // cached tokens before them
    int64_t kv;      // positions that exist: len + n, cut at the page-table row
    int32_t tiles;   // 128-key tiles
    int32_t items;   // 128-row items
    int32_t units_each;  // units of an item

    __device__ __forceinline__ void load(const TreeAttentionArgs& a, int b) {
        const int64_t rows = a.total_rows;
        const int64_t lo = min(static_cast<int64_t>(__ldg(a.row_offsets + b)), rows);
        const int64_t hi = min(static_cast<int64_t>(__ldg(a.row_offsets + b + 1)), rows);
        first = lo;
        n = hi > lo ? static_cast<int32_t>(hi - lo) : 0;
        len = __ldg(a.cache_lengths + b);
        kv = min(len + n, static_cast<int64_t>(a.max_pages) * a.page_size);
        tiles = static_cast<int32_t>((kv + kKeys - 1) / kKeys);
        units_each = tiles + a.item_cost;
        items = static_cast<int32_t>((static_cast<int64_t>(n) * a.num_heads + 127) / 128);
    }
    __device__ __forceinline__ int64_t units() const {
        return n > 0 ? static_cast<int64_t>(units_each) * items : 0;
    }
};

struct Bars {
    uint64_t k_full[kKeyGroups];   // even CTA: a group of blocks of both CTAs' keys is there
    uint64_t k_empty[kKeyGroups];  // both: its MMAs are done
    uint64_t v_full[kValueRing];   // even CTA: a group of both CTAs' value blocks is there
    uint64_t v_empty[kValueRing];  // both: its MMAs are done
    uint64_t v_own[kValueRing];    // both: values that the CTA looks through first are there
    uint64_t q_full, q_empty;   // the item's query rows
    uint64_t s_full[2];         // both: a score tile is complete
    uint64_t p_full;            // even CTA: both CTAs' weights are written
    uint64_t o_full;            // both: the tile's weights are used up and O is current
    uint64_t o_empty;           // even CTA: both CTAs' epilogues have read O
    uint64_t mma_done;
    int64_t units;              // units of all items
    int64_t first_unit;         // this pair's share begins here
    int32_t share;              // and has so many units
    int32_t request, item, unit;  // its first unit
    Request first;              // the request of that
    int32_t progress;           // tiles whose keys have been asked for
    uint32_t tmem_base;
    int abort_flag;
};

constexpr size_t kOffQ = 0;
constexpr size_t kOffK = kOffQ + size_t(kBlocks - kQueryBlocks) * kBlockBytes;
constexpr size_t kOffV = kOffK + size_t(kBlocks) * kBlockBytes;
constexpr size_t kOffP = kOffV + size_t(kValueRing) * 2 * kValueBytes;
constexpr size_t kOffMax = kOffP + 2 * size_t(kBlockBytes);
constexpr size_t kOffBars = kOffMax + 2 * 256 * sizeof(float);
constexpr size_t kSmemBytes = kOffBars + sizeof(Bars);
static_assert(kSmemBytes <= 232448, "shared memory budget of one sm_103a CTA");

// A pair's share of the units of all items, walked item by item.  An item has a unit for each
// of its tiles, behind item_cost units that stand for its start and end.  After next()
// returned true, the part is tiles [kt0, kt1) of item `item` of request r, which all roles take
// from the last to the first: the drafts' tiles, whose masks have to be fetched and whose values
// looked through, come while the item's start has to be waited for anyhow (taken last they
// delayed the item's end by 2 to 3 us).
struct Walk {
    int64_t u;       // first unit behind the part
    int32_t left;    // units of the share behind the part
    int32_t at;      // unit of the item behind the part
    int b;
    Request r;
    int32_t item, kt0, kt1;

    __device__ __forceinline__ explicit Walk(const Bars* bars) {
        left = bars->share;
        b = bars->request;
        item = bars->item;
        at = bars->unit;
        u = bars->first_unit;
        r = bars->first;
    }
    __device__ __forceinline__ bool next(const TreeAttentionArgs& a) {
        do {
            if (left <= 0) return false;
            if (at == r.units_each) {
                at = 0;
                if (++item == r.items) {
                    item = 0;
                    do r.load(a, ++b);  // units are left: a request further on has them
                    while (r.units() == 0);
                }
            }
            const int32_t take = min(r.units_each - at, left);
            kt0 = max(at - a.item_cost, 0);
            at += take;
            kt1 = max(at - a.item_cost, 0);
            u += take;
            left -= take;
        } while (kt1 == kt0);  // a share can end within an item's first units
        return true;
    }
    // The first tiles of an item hold cached tokens alone, which every row attends.
    __device__ __forceinline__ int32_t cached_tiles() const {
        return static_cast<int32_t>(min(r.len, r.kv) / kKeys);
    }
};

// Counts the units of all requests and cuts out the pair's share; every thread sums a run of
// requests.  `scratch`: an int64 of shared memory for every warp.
__device__ __forceinline__ void plan(const TreeAttentionArgs& a, Bars* bars, int64_t* scratch,
                                     int64_t pair, int64_t pairs) {
    const int64_t per = (static_cast<int64_t>(a.batch) + kThreads - 1) / kThreads, all = a.batch;
    const int b0 = static_cast<int>(min(threadIdx.x * per, all));
    const int b1 = static_cast<int>(min(b0 + per, all));
    int64_t sum = 0;
    Request r;
    for (int b = b0; b < b1; ++b) {
        r.load(a, b);
        sum += r.units();
        if (r.n > 0 && r.kv < r.len + r.n) report(a.status, PKM_ERR_OUT_OF_RANGE);
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int64_t incl = sum;
#pragma unroll
    for (int sh = 1; sh < 32; sh <<= 1) {
        const int64_t o = __shfl_up_sync(0xffffffffu, incl, sh);
        if (lane >= sh) incl += o;
    }
    if (lane == 31) scratch[warp] = incl;
    if (threadIdx.x == 0) bars->share = bars->progress = 0;
    __syncthreads();
    int64_t before = 0, total = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        if (w < warp) before += scratch[w];
        total += scratch[w];
    }
    if (threadIdx.x == 0) bars->units = total;
    pairs = min(pairs, total);  // no pair without a unit lies between two that share an item
    if (pair >= pairs) return;
    const int64_t u = quotient(total * pair, pairs);
    int64_t at = before + incl - sum;
    if (at <= u && u < at + sum)
        for (int b = b0; b < b1; ++b) {
            if (per > 1) r.load(a, b);
            if (u < at + r.units()) {
                bars->first_unit = u;
                bars->share = static_cast<int32_t>(quotient(total * (pair + 1), pairs) - u);
                bars->request = b;
                bars->first = r;
                const int32_t item = static_cast<int32_t>(quotient(u - at, r.units_each));
                bars->item = item;
                bars->unit = static_cast<int32_t>((u - at) - static_cast<int64_t>(item) * r.units_each);
                break;
            }
            at += r.units();
        }
}

// Asks for the arrays that the first loads depend on one after the other (offsets, lengths, page
// table) to be brought into L2, all at once and before they may be read: with the queries' later
// blocks (see fetch) 0.5 to 2 us of a call with cold inputs.
__device__ __forceinline__ void prefetch_tables(const TreeAttentionArgs& a) {
    const int64_t t = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int64_t line = t * 32;  // 32-bit entries
    if (line <= a.batch) prefetch_l2(a.row_offsets + line);
    if (line < a.batch) prefetch_l2(a.cache_lengths + line);
    if (line < static_cast<int64_t>(a.batch) * a.max_pages) prefetch_l2(a.page_table + line);
}

// Page and slot of position pos of request b; page -1 (loads as zeros) at or past kv and for
// ids that the cache does not have, which are reported.
struct Place {
    int32_t page, slot;
    __device__ __forceinline__ Place(const TreeAttentionArgs& a, int b, int64_t pos, int64_t kv)
        : page(-1), slot(0) {
        if (pos >= kv) return;
        const int64_t lp = quotient(pos, a.page_size);
        slot = static_cast<int32_t>(pos - lp * a.page_size);
        const uint32_t id = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + lp);
        if (id < static_cast<uint32_t>(a.num_pages)) page = static_cast<int32_t>(id);
        else report(a.status, PKM_ERR_OUT_OF_RANGE);
    }
    // Offset of the slot in the layer, or -1.
    __device__ __forceinline__ int64_t offset(const TreeAttentionArgs& a) const {
        return page < 0 ? -1 : page * a.page_stride + slot * a.slot_stride;
    }
};

// Infinities and NaN of a packed pair of bf16 become zero.
__device__ __forceinline__ uint32_t finite2(uint32_t w) {
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0x0000ffffu;
    return w;
}

__device__ __forceinline__ uint4 finite8(uint4 v) {
    return make_uint4(finite2(v.x), finite2(v.y), finite2(v.z), finite2(v.w));
}

// Whether there are any: an exponent of ones carries into the sign's place.
__device__ __forceinline__ bool any_nonfinite(const uint4& v) {
    const auto top = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
    return ((top(v.x) | top(v.y) | top(v.z) | top(v.w)) & 0x80008000u) != 0;
}

// Four e4m3 codes times a scale, each product rounded to fp32 and then to bf16.  The halves that
// the codes unpack to are widened by the mixed-precision add of -0, which keeps a zero's sign
// and leaves the conversion unit to the unpacking.
__device__ __forceinline__ uint2 dequant4(uint32_t codes, float scale) {
    float f0, f1, f2, f3;
    asm("{\n\t.reg .b16 l, h, a, b, c, d;\n\t.reg .b32 lo, hi;\n\t"
        "mov.b32 {l, h}, %4;\n\t"
        "cvt.rn.f16x2.e4m3x2 lo, l;\n\t"
        "cvt.rn.f16x2.e4m3x2 hi, h;\n\t"
        "mov.b32 {a, b}, lo;\n\t"
        "mov.b32 {c, d}, hi;\n\t"
        "add.rn.f32.f16 %0, a, 0f80000000;\n\t"
        "add.rn.f32.f16 %1, b, 0f80000000;\n\t"
        "add.rn.f32.f16 %2, c, 0f80000000;\n\t"
        "add.rn.f32.f16 %3, d, 0f80000000;\n\t}"
        : "=f"(f0), "=f"(f1), "=f"(f2), "=f"(f3)
        : "r"(codes));
    float a, b, c, d;
    mul2(a, b, f0, f1, scale, scale);
    mul2(c, d, f2, f3, scale, scale);
    return make_uint2(pack_bf16x2(a, b), pack_bf16x2(c, d));
}

// A row of each tile (a lane's own), moved back a tile at a time: its page id first, on its way
// while other work is done, then its place in 16-byte units of the layer (kNoRow past the last
// row, before the first tile and for ids that the cache does not have, which are reported).
constexpr uint32_t kNoRow = 0xffffffffu;
struct Row {
    int32_t left;  // rows from it to the last
    int32_t page, slot;
    uint32_t id, unit;

    __device__ __forceinline__ void start(const TreeAttentionArgs& a, int64_t pos, int64_t end) {
        left = static_cast<int32_t>(end - pos);
        const int64_t lp = quotient(pos, a.page_size);
        page = static_cast<int32_t>(lp);
        slot = static_cast<int32_t>(pos - lp * a.page_size);
    }
    __device__ __forceinline__ void fetch(const uint32_t* table, bool tile) {
        id = ld_nc_u32_if(table + page, tile && left > 0);
    }
};

// How rows lie in the layer: all in 16-byte units, whose number fits 32 bits.
struct Layout {
    uint32_t pages, page_units, slot_units;
    int32_t page_size, tile_pages, tile_slots;  // a tile is so many pages and slots

    __device__ __forceinline__ Layout(const TreeAttentionArgs& a, int unit_shift)
        : pages(static_cast<uint32_t>(a.num_pages)),
          page_units(static_cast<uint32_t>(a.page_stride >> unit_shift)),
          slot_units(static_cast<uint32_t>(a.slot_stride >> unit_shift)),
          page_size(a.page_size),
          tile_pages(kKeys / a.page_size),
          tile_slots(kKeys % a.page_size) {}
    // The place of the row whose id was fetched, then back to the tile before.  `tile`: the part
    // has the tile.
    __device__ __forceinline__ void resolve(const TreeAttentionArgs& a, Row& r, bool tile) const {
        const bool exists = tile && r.left > 0, have = exists && r.id < pages;
        r.unit = have ? r.id * page_units + r.slot * slot_units : kNoRow;
        if (exists && !have) report(a.status, PKM_ERR_OUT_OF_RANGE);
        r.left += kKeys;
        r.page -= tile_pages;
        r.slot -= tile_slots;
        const bool under = r.slot < 0;
        r.page -= under ? 1 : 0;
        r.slot += under ? page_size : 0;
    }
};

// 16 columns of a latent row on their way from the cache to shared memory: bf16, or (in lo) e4m3
// codes.
struct Piece {
    uint4 lo, hi;

    // `upper`: the upper 8 columns exist
    __device__ __forceinline__ void load_bf16(const uint8_t* from, uint32_t unit, bool upper) {
        const uint8_t* p = from + static_cast<uint64_t>(unit) * 16;
        lo = ld_nc_v4_if(p, unit != kNoRow);
        hi = ld_nc_v4_if(p + 16, unit != kNoRow && upper);
    }
    __device__ __forceinline__ void load_codes(const uint8_t* from, uint32_t unit) {
        lo = ld_nc_v4_if(from + static_cast<uint64_t>(unit) * 16, unit != kNoRow);
    }
    __device__ __forceinline__ void dequant(float scale, uint4& l, uint4& h) const {
        const uint2 d0 = dequant4(lo.x, scale), d1 = dequant4(lo.y, scale);
        const uint2 d2 = dequant4(lo.z, scale), d3 = dequant4(lo.w, scale);
        l = make_uint4(d0.x, d0.y, d1.x, d1.y);
        h = make_uint4(d2.x, d2.y, d3.x, d3.y);
    }
};

// Which of the 32 keys c0 .. c0+31 a token may attend; the words of its mask that they need are
// asked for a tile ahead.
struct Attended {
    uint32_t word[2];

    __device__ __forceinline__ void fetch(const TreeAttentionArgs& a, const Request& r, int32_t token, int64_t c0) {
        const int64_t w0 = max(c0 - r.len, static_cast<int64_t>(0)) >> 5;  // of the first draft
        const uint32_t* row = a.mask + (r.first + token) * a.mask_words + w0;
#pragma unroll
        for (int k = 0; k < 2; ++k) word[k] = ld_nc_u32_if(row + k, a.mask != nullptr && w0 + k < a.mask_words);
    }
    __device__ __forceinline__ uint32_t bits(const TreeAttentionArgs& a, const Request& r, int32_t token, int64_t c0) const {
        const auto low = [](int64_t n) -> uint32_t {
            return n <= 0 ? 0u : n >= 32 ? ~0u : (1u << n) - 1u;
        };
        const uint32_t exist = low(r.kv - c0);
        if (a.mask == nullptr) return exist & low(r.len + token + 1 - c0);
        const int64_t j0 = c0 - r.len;  // draft of the first key
        if (j0 <= 0) return exist & (low(-j0) | (j0 > -32 ? word[0] << -j0 : 0u));
        return exist & __funnelshift_r(word[0], word[1], static_cast<uint32_t>(j0 & 31));
    }
};

// Block n of a CTA's value blocks: of every four blocks the even CTA has the first two.
__device__ __forceinline__ int value_block(int rank, int n) { return 4 * (n >> 1) + 2 * rank + (n & 1); }

__device__ __forceinline__ float exp2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Waits with all lanes of a warp; the verdict is the same in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const WaitCtl& wc) {
    return __all_sync(0xffffffffu, mbar_wait_inl(bar, parity, wc));
}

// Warp i of the eight that bring the rows of a CTA by loads, as keys and as values in one go: the
// tile's columns come in two sets of four blocks (the ninth block with the second), and of each
// set a warp brings
//   - of one of its two pairs of blocks 16 of the CTA's own 64 keys; the pair that the CTA has as
//     values is stored a second time as those;
//   - of that pair 8 of the other CTA's 64 keys, as values;
//   - of the ninth block 8 of its 16 keys.
// Eight lanes take a row's 128 columns; lane l keeps row l of its own 16 or of the other 8, that
// is, finds its page and loads its scale.  When a set is stored the next one is asked for.
//
// One copy of the code serves all warps and both sets, with few branches: the warps wait for
// instructions more than for loads.  For 32 chains over the quantised cache a form in which four
// warps brought all keys and four all values, which converts 1.9 times as much, took half as long
// again; a scale of its own for every piece and 64 columns of a row at a time 13 % more; sixteen
// warps, or a second set of registers for the rows on their way, changed nothing.
template <Source SRC, typename Queries>
__device__ __forceinline__ void by_loads(const TreeAttentionArgs& a, Bars* bars, uint8_t* smem,
                                         uint32_t rank, int i, int kblocks, int vgroups,
                                         uint32_t k_full, uint32_t tries, const WaitCtl& wc,
                                         const Queries& queries) {
    constexpr bool kQuant = SRC == kCodes || SRC == kCodesNarrow;
    const int lane = threadIdx.x & 31;
    // a lane's row of each four and its 16 columns of the pair: lanes that store together have
    // two rows' same columns, whose 16-byte chunks lie in different banks
    const int sub = (lane >> 2 & 1) | (lane >> 4 << 1), part = (lane & 3) | (lane >> 3 & 1) << 2;
    const int R = a.kv_lora_rank, pair = i & 1;
    const int sets = kblocks > kQueryBlocks ? 2 : 1;
    const int own0 = rank * 64 + (i >> 1) * 16;  // the tile's rows that it brings as keys
    const int other0 = (rank ^ 1) * 64 + i * 8;  // and as values alone
    const int ninth = pair * 8 + (lane >> 3);    // of its 16 rows, and 4 further on
    const int ninth_c = 8 * 64 + (lane & 7) * 8;
    // Chunk c of row r lies at chunk c ^ (r & 7), and the rows here are sub + 4 n.
    const uint32_t at = (part >> 2) * kBlockBytes + sub * 128 + ((((part & 3) * 2) ^ sub) << 4);
    const uint32_t at2 = (part >> 2) * kValueBytes + at - (part >> 2) * kBlockBytes;
    const uint32_t keys_at = smem_u32(smem) + kOffK + (i >> 1) * 16 * 128;
    const uint32_t values_at = smem_u32(smem) + kOffV;
    const Layout layout(a, kQuant ? 4 : 3);
    const uint8_t* layer = kQuant ? a.qcache_layer : reinterpret_cast<const uint8_t*>(a.cache_layer);
    // bytes of a row before column c, which `codes` says are codes
    const auto before = [&](int c, bool codes) { return codes ? c : 2 * c - (kQuant ? R : 0); };
    const auto are_codes = [&](int set, int pair) {
        return SRC == kCodes || (SRC == kCodesNarrow && set * 256 + pair * 128 < R);
    };
    Piece own[4], other[2];
    uint4 last[2];
    uint32_t scale = 0;
    Row row{};
    RingPos ring;
    uint32_t g = 0;
    bool ok = true;
    Walk w(bars);
    const auto load = [&](int set) {
        uint32_t u[6], u9[2];
#pragma unroll
        for (int n = 0; n < 6; ++n) u[n] = __shfl_sync(0xffffffffu, row.unit, n * 4 + sub);
#pragma unroll
        for (int n = 0; n < 2; ++n) u9[n] = __shfl_sync(0xffffffffu, row.unit, ninth + 4 * n);
        const int col0 = set * 256 + pair * 128 + part * 16;
        const int col1 = set * 256 + static_cast<int>(rank) * 128 + part * 16;
        if (kQuant) {  // the lane's row's
            const int scaled = set * 2 + (lane < 16 ? pair : static_cast<int>(rank));
            scale = ld_nc_u32_if(layer + 2 * a.cols - R + scaled * 4 + static_cast<uint64_t>(row.unit) * 16,
                                 row.unit != kNoRow && scaled * 128 < R);
        }
        const bool codes0 = are_codes(set, pair), codes1 = are_codes(set, rank);
        const uint8_t *from0 = layer + before(col0, codes0), *from1 = layer + before(col1, codes1);
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (codes0) own[n].load_codes(from0, u[n]);
            else own[n].load_bf16(from0, col0 < a.cols ? u[n] : kNoRow, col0 + 8 < a.cols);
        }
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            if (codes1) other[n].load_codes(from1, u[4 + n]);
            else other[n].load_bf16(from1, col1 < a.cols ? u[4 + n] : kNoRow, col1 + 8 < a.cols);
        }
        if (set == 0 || kblocks < kBlocks) return;
#pragma unroll
        for (int n = 0; n < 2; ++n)
            last[n] = ld_nc_v4_if(layer + before(ninth_c, false) + static_cast<uint64_t>(u9[n]) * 16,
                                  u9[n] != kNoRow && ninth_c < a.cols);
    };
    while (ok && __any_sync(0xffffffffu, w.next(a))) {
        const int tiles = __shfl_sync(0xffffffffu, w.kt1 - w.kt0, 0);
        const int64_t pos0 = static_cast<int64_t>(w.kt1 - 1) * kKeys;
        const int64_t end = min(w.r.kv, static_cast<int64_t>(w.kt1) * kKeys);
        const uint32_t* table = a.page_table + static_cast<int64_t>(w.b) * a.max_pages;
        // rows of the tile at hand that are cached ones, if not all (and behind the first draft's
        // tile less than none)
        int cached = __shfl_sync(
            0xffffffffu, static_cast<int>(min(w.r.len - pos0, static_cast<int64_t>(kKeys))), 0);
        row.start(a, pos0 + (lane < 16 ? own0 + lane : lane < 24 ? other0 + lane - 16 : 0), end);
        const auto rows = [&](int t) {  // of tile t of the part, and the id of the next
            layout.resolve(a, row, t < tiles);
            row.fetch(table, t + 1 < tiles);
        };
        row.fetch(table, true);
        rows(0);
        load(0);
        int t = 0;
        int set = 0;
#pragma unroll 1
        while (t < tiles) {
            ok = mbar_wait_flag(&bars->k_empty[set], (g & 1) ^ 1, wc.abort_flag, tries);
            if (set < vgroups)
                ok = ok && mbar_wait_flag(&bars->v_empty[ring.stage], ring.phase ^ 1, wc.abort_flag, tries);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const int next = set + 1 == sets ? 0 : set + 1;
            if (next == 0) rows(t + 1);
            float f[6];
#pragma unroll
            for (int n = 0; n < 6; ++n)
                f[n] = kQuant ? __uint_as_float(__shfl_sync(0xffffffffu, scale, n * 4 + sub)) : 0.0f;
            const uint32_t k0 = keys_at + (set * 4 + pair * 2) * kBlockBytes + at;
            const uint32_t values = values_at + ring.stage * 2 * kValueBytes + at2;
            const auto put = [&](uint32_t to, int n, const uint4& lo, const uint4& hi) {
                const uint32_t p = (to + n * 512) ^ ((n & 1) << 6);
                st_shared_v4(p, lo.x, lo.y, lo.z, lo.w);
                st_shared_v4(p ^ 16, hi.x, hi.y, hi.z, hi.w);
            };
            // drafts' infinities and NaN are no values, as in the loads by TMA
            const auto put_value = [&](uint32_t to, int n, uint4 lo, uint4 hi, int r) {
                if (cached < kKeys && r >= cached) {
                    lo = finite8(lo);
                    hi = finite8(hi);
                }
                put(to, n, lo, hi);
            };
            const bool codes0 = are_codes(set, pair), codes1 = are_codes(set, rank);
            const bool both = set < vgroups && pair == static_cast<int>(rank);
#pragma unroll
            for (int n = 0; n < 4; ++n) {
                uint4 lo = own[n].lo, hi = own[n].hi;
                if (codes0) own[n].dequant(f[n], lo, hi);
                put(k0, n, lo, hi);
                if (both) put_value(values + own0 * 128, n, lo, hi, own0 + n * 4 + sub);
            }
            if (set < vgroups) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    uint4 lo = other[n].lo, hi = other[n].hi;
                    if (codes1) other[n].dequant(f[4 + n], lo, hi);
                    put_value(values + other0 * 128, n, lo, hi, other0 + n * 4 + sub);
                }
            }
            if (set == 1 && kblocks == kBlocks) {
#pragma unroll
                for (int n = 0; n < 2; ++n) {
                    const int r = ninth + 4 * n;
                    st_shared_v4(keys_at + 8 * kBlockBytes + r * 128 + (((lane & 7) ^ (r & 7)) << 4),
                                 last[n].x, last[n].y, last[n].z, last[n].w);
                }
            }
            load(next);
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive_publish(k_full + set * 8);
            if (set < vgroups) ring.next(kValueRing);
            if (t + set == 0) ok = queries(w);
            if (!ok) break;
            set = next;
            if (set > 0) continue;
            ++t;
            cached = min(cached + kKeys, kKeys);
            ++g;
            if (i == 0 && lane == 0) bars->progress = static_cast<int32_t>(g);
        }
    }
    if (!ok && lane == 0) bars->progress = INT32_MAX;
}

template <Source SRC>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    tree_attention_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_k0,
                          const __grid_constant__ CUtensorMap tm_k1,
                          const __grid_constant__ CUtensorMap tm_v, const TreeAttentionArgs a,
                          const TreeWorkspace ws, const TreeBoxes tb) {
    extern __shared__ __align__(1024) uint8_t smem[];  // swizzle atoms of 1024 bytes
    uint8_t* sQ = smem + kOffQ;
    uint8_t* sK = smem + kOffK;
    uint8_t* sV = smem + kOffV;
    uint8_t* sP = smem + kOffP;
    float* s_max = reinterpret_cast<float*>(smem + kOffMax);
    Bars* bars = reinterpret_cast<Bars*>(smem + kOffBars);

    // Values that are the same in every lane pass through a shuffle, from which the compiler
    // sees that they are: branches and addresses made of them then use uniform registers,
    // where MMAs and TMA loads take their operands.  With operands that have to be moved there
    // one by one, an MMA took 75 to 165 cycles to issue instead of 32 to execute.
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x >> 5), 0);
    const int lane = threadIdx.x & 31;
    const uint32_t rank = __shfl_sync(0xffffffffu, cluster_ctarank(), 0);
    const bool leader = rank == 0;
    const int64_t pairs = gridDim.x / 2, pair = blockIdx.x / 2;
    const int R = a.kv_lora_rank;
    const int kblocks = (a.cols + 63) / 64;
    const int vgroups = (R + 255) / 256;        // groups of two value blocks of each CTA
    const int vblocks = 2 * vgroups;

    if (threadIdx.x == 0) {
        for (int i = 0; i < kKeyGroups; ++i) {
            // one box: one arrival, with the bytes; boxes of a block: one each; by loads: eight
            // warps of each CTA
            const int from = i == 0 ? 0 : kQueryBlocks, to = i == 0 ? min(kblocks, kQueryBlocks) : kblocks;
            const int blocks = max(to - from, 1);
            mbar_init(&bars->k_full[i], SRC != kTma ? 16 : tb.key_blocks > 1 ? 1 : blocks);
            mbar_init(&bars->k_empty[i], 1);
        }
        for (int i = 0; i < kValueRing; ++i) {
            mbar_init(&bars->v_full[i], 4);  // two blocks, two CTAs
            mbar_init(&bars->v_empty[i], 1);
            mbar_init(&bars->v_own[i], tb.value_blocks > 1 ? 1 : 2);  // warps that load
        }
        for (int i = 0; i < 2; ++i) mbar_init(&bars->s_full[i], 1);
        mbar_init(&bars->q_full, 1 + 2 * 8);  // the TMA bytes, and warps of each CTA
        mbar_init(&bars->q_empty, 1);
        mbar_init(&bars->p_full, 2 * kSoftWarps);
        mbar_init(&bars->o_full, 1);
        mbar_init(&bars->o_empty, 2 * kSoftWarps);
        mbar_init(&bars->mma_done, 1);
        bars->abort_flag = 0;
        fence_mbar_init();
    }
    if (warp == kQueryWarp && lane == 0) {
        tma_prefetch_map(&tm_q);
        tma_prefetch_map(&tm_k0);
        tma_prefetch_map(&tm_k1);
        tma_prefetch_map(&tm_v);
    }
    if (warp == kMmaWarp) {
        tmem_alloc_pair(&bars->tmem_base, kTmemCols);
        tmem_relinquish_pair();
    }
    __syncwarp();
    cluster_arrive();  // the barriers are set up; the peer may signal them behind cluster_wait
    prefetch_tables(a);
    griddep_wait();  // launched while the work before may still run: nothing is read before
    plan(a, bars, reinterpret_cast<int64_t*>(s_max), pair, pairs);
    griddep_launch_dependents();
    tc_fence_before();
    __syncthreads();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, bars->tmem_base, 0);
    const WaitCtl wc{&bars->abort_flag, a.status, a.timeout_ns};
    // The softmax warps keep the time limit: whatever stalls stalls them.  The issuing and
    // loading warps' waits end with their abort flag, or after tries that take longer.  (With
    // mbar_wait's exits in the loop the scores' MMAs took 50 cycles each instead of 30.)
    const uint32_t tries =
        static_cast<uint32_t>(min(a.timeout_ns / 8, uint64_t{UINT32_MAX}));
    const auto issue_wait = [&](uint64_t* bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait_flag(bar, parity, wc.abort_flag, tries));
    };
    const int64_t sharing = min(pairs, bars->units);  // pairs with a share

    if (warp < kSoftWarps) {
        // ---------------- softmax and epilogue: row = lane of the CTA's 64 ----------------
        // Warps w and w + 4 share 32 lanes; lanes 0-63 have the first 64 keys (and half of O's
        // columns), and each of the two warps takes 32 of the keys (half of the lanes' columns).
        // With one warp for both large drafted trees took 4 % longer.
        if constexpr (SRC == kTma) warpgroup_reg_alloc<kMoreRegs>();
        Walk w(bars);
        const int half = warp >> 1 & 1, part = warp >> 2;
        const int row = (warp & 1) * 32 + lane;       // of this CTA's 64
        const int quarter = (half * 2 + part) * 64 + row;  // place of a row's maximum and sum
        const float scale2 = a.scale * kLog2e;
        const uint32_t tlane = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t p_row = smem_u32(sP) + half * kBlockBytes + row * 128;
        const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
        const uint32_t p_full = mapa_shared(smem_u32(&bars->p_full), 0);
        const uint32_t o_empty = mapa_shared(smem_u32(&bars->o_empty), 0);
        // the four warps that share rows
        const auto meet = [&] { named_bar_sync(3 + (warp & 1), 128); };
        uint32_t g = 0;
        int32_t left_rows = 0, left_parts = 0;
        int64_t left_first = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            const int64_t rows_all = static_cast<int64_t>(w.r.n) * a.num_heads;
            const int64_t rr = static_cast<int64_t>(w.item) * 128 + rank * 64 + row;
            const int32_t token =
                min(static_cast<int32_t>(quotient(rr, a.num_heads)), w.r.n - 1);
            float m = -INFINITY, l = 0.0f;
            Attended mask;
            const int32_t cached = w.cached_tiles();
            const auto key0 = [&](int32_t kt) { return static_cast<int64_t>(kt) * kKeys + half * 64 + part * 32; };
            if (w.kt1 > cached) mask.fetch(a, w.r, token, key0(w.kt1 - 1));
            for (int32_t kt = w.kt1 - 1; kt >= w.kt0; --kt, ++g) {
                const bool partial = kt >= cached;
                uint32_t may = ~0u;
                if (partial) may = mask.bits(a, w.r, token, key0(kt));
                if (kt > cached && kt > w.kt0) mask.fetch(a, w.r, token, key0(kt - 1));
                if (!warp_wait(&bars->s_full[g & 1], (g >> 1) & 1, wc)) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                uint32_t x[32];
                tmem_ld_x32(tmem + tlane + kScoreCol + (g & 1) * 64 + part * 32, x);
                tmem_ld_wait();
                float s[32];
#pragma unroll
                for (int k = 0; k < 16; ++k)
                    mul2(s[2 * k], s[2 * k + 1], __uint_as_float(x[2 * k]),
                         __uint_as_float(x[2 * k + 1]), scale2, scale2);
                if (partial) {
#pragma unroll
                    for (int k = 0; k < 32; ++k) s[k] = (may >> k) & 1u ? s[k] : -INFINITY;
                }
                float t0 = s[0], t1 = s[1], t2 = s[2], t3 = s[3];
#pragma unroll
                for (int k = 4; k < 32; k += 4) {
                    t0 = fmaxf(t0, s[k]);
                    t1 = fmaxf(t1, s[k + 1]);
                    t2 = fmaxf(t2, s[k + 2]);
                    t3 = fmaxf(t3, s[k + 3]);
                }
                float* mx = s_max + (g & 1) * 256;
                mx[quarter] = fmaxf(fmaxf(t0, t1), fmaxf(t2, t3));
                meet();
                if (*wc.abort_flag) {
                    ok = false;
                    break;
                }
                const float top = fmaxf(fmaxf(mx[row], mx[64 + row]), fmaxf(mx[128 + row], mx[192 + row]));
                const bool move = top > m + kLazy || (m == -INFINITY && top > -INFINITY);
                const float m_new = move ? top : m;
                const float back = move && m > -INFINITY ? exp2_approx(m - m_new) : move ? 0.0f : 1.0f;
                m = m_new;
                const float ref = m == -INFINITY ? 0.0f : m;
                // The weights are rounded to bf16, by up to 2^-8 of each: the second product's
                // operands have one type, and the values are bf16.  Their sum stays in fp32, unrounded.
                // (Outputs are 2.1e-3 of their size from 64 bits; with weights in fp32 1.7e-3, which
                // is the rounding of the outputs themselves.)
                float sum0 = 0.0f, sum1 = 0.0f;
                uint32_t p[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    const float e0 = exp2_approx(s[2 * k] - ref);
                    const float e1 = exp2_approx(s[2 * k + 1] - ref);
                    sum0 += e0;
                    sum1 += e1;
                    p[k] = pack_bf16x2(e0, e1);
                }
                l = l * back + (sum0 + sum1);
                // the weights are finished before the wait, not after it
#pragma unroll
                for (int k = 0; k < 16; ++k) asm volatile("" : "+r"(p[k]));
                // the previous tile's weights are used up, and O holds it
                if (g > 0 &&
                    !warp_wait(&bars->o_full, (g - 1) & 1, wc)) {
                    ok = false;
                    break;
                }
                if (kt + 1 < w.kt1 && __any_sync(0xffffffffu, move)) {
                    tc_fence_after();
                    for (int v = part * vblocks; v < (part + 1) * vblocks; ++v) {
                        uint32_t o[32];
                        tmem_ld_x32(tmem + tlane + v * 32, o);
                        tmem_ld_wait();
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            o[k] = __float_as_uint(__uint_as_float(o[k]) * back);
                        tmem_st_x32(tmem + tlane + v * 32, o);
                    }
                    tmem_st_wait();
                }
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    st_shared_v4(p_row + (((part * 4 + j) ^ (row & 7)) << 4), p[4 * j], p[4 * j + 1],
                                 p[4 * j + 2], p[4 * j + 3]);
                fence_proxy_async_smem();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_publish(p_full);
            }
            if (!ok) break;
            if (!warp_wait(&bars->o_full, (g - 1) & 1, wc)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // in the place of the last tile's maxima, which all have read when O is complete
            float* sums = s_max + ((g - 1) & 1) * 256;
            sums[quarter] = l;
            meet();
            if (*wc.abort_flag) {
                ok = false;
                break;
            }
            // the same order in all four warps
            l = (sums[row] + sums[64 + row]) + (sums[128 + row] + sums[192 + row]);
            const int v0 = part * vgroups, v1 = v0 + vgroups;  // this warp's blocks of O
            const bool whole = w.kt0 == 0 && w.kt1 == w.r.tiles;
            const int64_t row0 = w.r.first * a.num_heads + rr - lane;  // of this warp's 32
            if (whole) {
                const float inv = l != 0.0f ? 1.0f / l : 0.0f;
                // A lane stores whole sectors of its row where the output allows: as fast as
                // through shared memory by TMA, and 2 % less for large drafted trees than whole
                // lines from there by the lanes.
                for (int c = 2 * v0; c < 2 * v1; ++c) {  // 32 columns
                    const int col = value_block(half, c >> 1) * 64 + (c & 1) * 32;
                    if (col >= R) break;
                    uint32_t x[32], p[16];
                    tmem_ld_x32(tmem + tlane + c * 32, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 16; ++k)
                        p[k] = pack_bf16x2(__uint_as_float(x[2 * k]) * inv, __uint_as_float(x[2 * k + 1]) * inv);
                    if (rr >= rows_all) continue;
                    uint16_t* out = a.out + (row0 + lane) * R + col;
                    if (sectors) {
#pragma unroll
                        for (int k = 0; k < 2; ++k) st_v8(out + 16 * k, p + 8 * k);
                    } else {
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            st_v4(out + 8 * k, make_uint4(p[4 * k], p[4 * k + 1], p[4 * k + 2], p[4 * k + 3]));
                    }
                }
                if (half + part == 0 && rr < rows_all && a.lse != nullptr)
                    a.lse[row0 + lane] = l != 0.0f ? m * kLn2 + logf(l) : -INFINITY;
            } else {
                const int64_t slot = 2 * pair + (w.kt0 > 0 ? 0 : 1);
                // four columns of consecutive rows side by side: whole lines, without staging
                const int at = rank * 64 + row;
                float4* to = reinterpret_cast<float4*>(a.workspace + ws.parts) +
                               slot * (R / 4) * ws.rows + at;
                const auto put = [&](int quads, const uint32_t(&x)[32]) {
                    if (rr >= rows_all) return;
#pragma unroll
                    for (int k = 0; k < 8; ++k)
                        st_v4(to + static_cast<int64_t>(quads + k) * ws.rows,
                              make_uint4(x[4 * k], x[4 * k + 1], x[4 * k + 2], x[4 * k + 3]));
                };
                for (int c = 2 * v0; c < 2 * v1; ++c) {  // 32 columns
                    const int col = value_block(half, c >> 1) * 64 + (c & 1) * 32;
                    if (col >= R) break;
                    uint32_t x[32];
                    tmem_ld_x32(tmem + tlane + c * 32, x);
                    tmem_ld_wait();
                    put(col / 4, x);
                }
                if (half + part == 0 && rr < rows_all)
                    reinterpret_cast<float2*>(a.workspace + ws.stats)[slot * ws.rows + at] =
                        make_float2(m, l);
                if (w.kt0 == 0) {
                    const int64_t end = w.u + (w.r.tiles - w.kt1);
                    left_first = row0 - rank * 64 - (warp & 1) * 32;
                    left_rows = static_cast<int32_t>(
                        min(rows_all - static_cast<int64_t>(w.item) * 128, static_cast<int64_t>(128)));
                    left_parts = static_cast<int32_t>((end * sharing - 1) / bars->units - pair) + 1;
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(o_empty);
        }
        if (!ok) named_bar_arrive(3 + (warp & 1), 128);  // releases the warps that share its rows
        if (leader && threadIdx.x == 0) {
            TreeItem* items = reinterpret_cast<TreeItem*>(a.workspace + ws.items);
            items[pair] = TreeItem{left_first, ok ? left_rows : 0, left_parts};
        }
    } else if (warp < kKeyWarp) {
      warpgroup_reg_dealloc<kIssueRegs>();
      if (warp == kMmaWarp) {
        // ---------------- MMA issuer (even CTA), all lanes together ----------------
        if (leader) {
            Walk w(bars);
            // A wait that runs out is looked at once a tile; what is issued until then is not used.
            bool failed = false;
            const auto wait = [&](uint64_t* bar, uint32_t parity) {
                failed |= !mbar_wait_flag(bar, parity, wc.abort_flag, tries);
            };
            const auto wait_cluster = [&](uint64_t* bar, uint32_t parity) {
                failed |= !mbar_wait_flag<true>(bar, parity, wc.abort_flag, tries);
            };
            const auto keys_wait = [&](uint64_t* bar, uint32_t parity) {
                if constexpr (SRC == kTma) wait(bar, parity);
                else wait_cluster(bar, parity);
            };
            const uint32_t id_s = idesc_bf16(128, kKeys, false, false);
            const uint32_t id_o = idesc_bf16(128, 256, false, true);
            const uint64_t q_desc = sdesc_sw128(smem_u32(sQ), 16, 1024);
            const uint64_t k_desc = sdesc_sw128(smem_u32(sK), 16, 1024);
            const uint64_t p_desc = sdesc_sw128(smem_u32(sP), 16, 1024);
            const uint64_t v_desc = sdesc_sw128(smem_u32(sV), kValueBytes, 1024);
            uint32_t g = 0, item = 0;
            bool first = false;   // the tile whose values come next starts its item
            RingPos vring;
            // O (+)= P V of a tile; `first`: of its item
            const auto values = [&](uint32_t tile, bool first) {
                const uint32_t ph = tile & 1;
                wait_cluster(&bars->p_full, ph);
                if (first && item > 1) wait(&bars->o_empty, item & 1);
                tc_fence_after();
                const uint32_t keep = first ? 0u : 1u;
#pragma unroll 1
                for (int vg = 0; vg < vgroups; ++vg) {
                    const uint32_t v = vring.stage;
                    if (SRC == kTma) {  // by loads they are there with the tile's keys
                        wait_cluster(&bars->v_full[v], vring.phase);
                        tc_fence_after();
                    }
                    const uint64_t vd = desc_add_bytes(v_desc, v * 2 * kValueBytes);
#pragma unroll 1
                    for (int h = 0; h < 2; ++h) {  // 64 keys: one block of P
                        const uint64_t pd = desc_add_bytes(p_desc, h * kBlockBytes);
                        const uint64_t vh = desc_add_bytes(vd, h * 64 * 128);
#pragma unroll
                        for (int k = 0; k < 4; ++k)  // 16 keys: 32 bytes of P, 2048 of V
                            mma_bf16_pair_elect(tmem + vg * 128, pd + 2 * k, vh + 128 * k, id_o,
                                                (h | k) != 0 ? 1u : keep);
                    }
                    mma_commit_pair_elect(&bars->v_empty[v], 3);
                    vring.next(kValueRing);
                }
                mma_commit_pair_elect(&bars->o_full, 3);
            };
            int tiles = 0, t = 0;
            while (true) {
                const bool next_item = t == tiles;
                if (!next_item) {
                    const uint32_t d = tmem + kScoreCol + (g & 1) * 64;
                    // Rolled loops without branches: unrolled or with the choice of the A operand
                    // inside, the same MMAs took 10 to 65 % longer to issue.
                    if (SRC != kTma && t > 0) {
                        values(g - 1, first);
                        first = false;
                    }
                    keys_wait(&bars->k_full[0], g & 1);
                    tc_fence_after();
                    const int first_blocks = min(kblocks, kQueryBlocks);
#pragma unroll 1
                    for (int kb = 0; kb < first_blocks; ++kb) {
                        const uint64_t kd = desc_add_bytes(k_desc, kb * kBlockBytes);
                        const uint32_t qt = tmem + kQueryCol + kb * 32;
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            mma_bf16_pair_ts_elect(d, qt + k * 8, kd + 2 * k, id_s,
                                                   (kb | k) != 0 ? 1u : 0u);
                    }
                    mma_commit_pair_elect(&bars->k_empty[0], 3);
                    if (kblocks > kQueryBlocks) {
                        keys_wait(&bars->k_full[1], g & 1);
                        tc_fence_after();
#pragma unroll 1
                        for (int kb = kQueryBlocks; kb < kblocks; ++kb) {
                            const uint64_t kd = desc_add_bytes(k_desc, kb * kBlockBytes);
                            const uint64_t qd = desc_add_bytes(q_desc, (kb - kQueryBlocks) * kBlockBytes);
#pragma unroll
                            for (int k = 0; k < 4; ++k)
                                mma_bf16_pair_elect(d, qd + 2 * k, kd + 2 * k, id_s, 1u);
                        }
                        mma_commit_pair_elect(&bars->k_empty[1], 3);
                    }
                    mma_commit_pair_elect(&bars->s_full[g & 1], 3);
                    if (t + 1 == tiles) mma_commit_pair_elect(&bars->q_empty, 3);
                    ++g;
                    ++t;
                }
                // The values of the tile before, behind this tile's scores (by loads before them:
                // those loads take longer than the weights, and need the values' place); those
                // of an item's last tile before the next item's queries are waited for.
                if (next_item ? g > 0 : SRC == kTma && t > 1) {
                    values(next_item ? g - 1 : g - 2, first);
                    first = false;
                }
                if (!next_item && t == 1) first = true;
                if (__any_sync(0xffffffffu, failed)) break;
                if (next_item) {
                    if (!__any_sync(0xffffffffu, w.next(a))) break;
                    tiles = __shfl_sync(0xffffffffu, w.kt1 - w.kt0, 0);
                    t = 0;
                    ++item;
                    wait(&bars->q_full, (item - 1) & 1);
                }
            }
            mma_commit_pair_elect(&bars->mma_done, 1);
            mbar_wait_inl(&bars->mma_done, 0, wc, false);
        }
      } else if (warp == kFetchWarp) {
        // Asks for keys to be brought into L2 ahead of their loads, which are issued when their
        // shared memory is free, too late to wait for DRAM: for wide boxes as soon as the keys of
        // the tile before are asked for, for other loads, which take longer, two tiles earlier.
        // (64 users x 1 token, wide boxes: two tiles earlier 8 % longer, never 6 %; ragged trees in
        // small pages: one tile ahead 3 % longer, never 8 %; chains over the quantised cache: one
        // tile ahead 7 %.)  With wide boxes a request's first item alone asks: with all of them
        // large drafted trees took 2 % longer.
        const int ahead = SRC == kTma && tb.key_blocks > 1 ? 0 : 2;
        Walk w(bars);
        volatile int32_t* progress = &bars->progress;
        const int bytes = SRC >= kCodes ? R + 2 * (a.cols - R) + 4 * (R / 128) : 2 * a.cols;
        int g = 0;
        bool ok = true;
        while (ok && w.next(a))
            for (int32_t kt = w.kt1 - 1; kt >= w.kt0; --kt, ++g) {
                // naps of 100 ns on average, as many as make the limit
                for (uint64_t n = 0; ok && g - ahead > *progress; ++n) {
                    ok = n < a.timeout_ns / 100 && !*wc.abort_flag;
                    __nanosleep(100);
                }
                if (!ok) break;
                if (ahead == 0 && w.item > 0) continue;
                for (int x = 0; x < 2; ++x) {
                    const int64_t pos = static_cast<int64_t>(kt) * kKeys + rank * 64 + x * 32 + lane;
                    const int64_t row = Place(a, w.b, pos, w.r.kv).offset(a);
                    if (row < 0) continue;
                    const uint8_t* from = SRC >= kCodes
                                              ? a.qcache_layer + row
                                              : reinterpret_cast<const uint8_t*>(a.cache_layer + row);
                    for (int c = 0; c < bytes; c += 128) prefetch_l2(from + c);
                    prefetch_l2(from + bytes - 1);
                }
            }
      } else if (warp == kQueryWarp) {
        // ---------------- queries: this CTA's 64 rows of each item, the later blocks --------
        Walk w(bars);
        const uint32_t q_full = mapa_shared(smem_u32(&bars->q_full), 0);
        uint32_t item = 0;
        bool ok = true;
        while (ok && w.next(a)) {
            ok = issue_wait(&bars->q_empty, (item & 1) ^ 1);
            if (!ok) break;
            const int64_t row = w.r.first * a.num_heads + static_cast<int64_t>(w.item) * 128 + rank * 64;
            const int blocks = max(kblocks - kQueryBlocks, 0);
            if (leader && lane == 0)
                mbar_arrive_expect_tx(&bars->q_full, 2 * blocks * kBlockBytes);
            if (lane < blocks)
                tma_load_2d_pair(sQ + lane * kBlockBytes, &tm_q, q_full,
                                 (kQueryBlocks + lane) * 64, static_cast<int32_t>(row));
            ++item;
        }
        if (!ok) spin_ns(kDrainNs);
      }
    } else {
        // ---------------- keys and values ----------------
        if constexpr (SRC != kTma) warpgroup_reg_alloc<kMoreRegs>();
        // Keys: this CTA's 64 of each tile, all columns, warp i bringing blocks i, i + 4 and
        // i + 8, or by boxes of whole groups group i.  Values: all 128 keys, this CTA's
        // columns, warp i bringing block i of its group i / 2 (past the CTA's last block it
        // only signals), or by boxes of both blocks the even warp.
        const bool keys = warp < kValueWarp;
        const int i = warp & 3;
        const uint32_t k_full = mapa_shared(smem_u32(bars->k_full), 0);
        const uint32_t v_full = mapa_shared(smem_u32(bars->v_full), 0);
        const uint32_t q_full = mapa_shared(smem_u32(&bars->q_full), 0);
        uint32_t g = 0, item = 0;
        bool ok = true;
        // The first query blocks of an item go to tensor memory: lanes 32 i .. 32 i + 31 by the key
        // and the value warp i, two blocks each.  The key warp asks for them to be brought into L2
        // and loads them behind its first tile: loads before would make the keys' page ids wait
        // for them (they share the few scoreboards).  The value warp loads its own before the
        // values (ragged trees: behind the first tile's, or all by the key warp, 5 % longer).
        constexpr int kAtOnce = SRC == kTma ? 2 : 1;  // blocks in flight
        const int first_kb = keys ? 0 : kQueryBlocks / 2, last_kb = first_kb + kQueryBlocks / 2;
        const auto fetch = [&](const Walk& w, int kb, uint32_t(&x)[kAtOnce][32]) {
            const int64_t row = w.r.first * a.num_heads + static_cast<int64_t>(w.item) * 128 +
                                rank * 64 + (i & 1) * 32 + lane;
            const uint16_t* q = a.q + row * a.cols;
            const bool have = row < static_cast<int64_t>(a.total_rows) * a.num_heads;
#pragma unroll
            for (int k = 0; k < 8 * kAtOnce; ++k) {
                const int c = kb * 64 + k * 8;
                const uint4 v = ld_nc_v4_if(q + c, have && c < a.cols);
                x[k >> 3][4 * (k & 7)] = v.x;
                x[k >> 3][4 * (k & 7) + 1] = v.y;
                x[k >> 3][4 * (k & 7) + 2] = v.z;
                x[k >> 3][4 * (k & 7) + 3] = v.w;
            }
        };
        const auto ask = [&](const Walk& w) {  // into L2, a line a block
            const int64_t row = w.r.first * a.num_heads + static_cast<int64_t>(w.item) * 128 +
                                rank * 64 + (i & 1) * 32 + lane;
            const uint16_t* q = a.q + row * a.cols;
            if (row < static_cast<int64_t>(a.total_rows) * a.num_heads)
                for (int kb = first_kb; kb < last_kb && kb < kblocks; ++kb) prefetch_l2(q + kb * 64);
        };
        const auto queries = [&](const Walk& w) -> bool {
            uint32_t x[kAtOnce][32];
            fetch(w, first_kb, x);
            if (SRC != kTma) ask(w);
            if (!issue_wait(&bars->q_empty, (item & 1) ^ 1)) return false;
            tc_fence_after();
#pragma unroll 1
            for (int kb = first_kb; kb < last_kb; kb += kAtOnce) {
                if (kb > first_kb) fetch(w, kb, x);
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k)
                    tmem_st_x32(tmem + (static_cast<uint32_t>(i * 32) << 16) + kQueryCol + (kb + k) * 32,
                                x[k]);
            }
            tmem_st_wait();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(q_full);
            ++item;
            return true;
        };
        Walk w(bars);
        if constexpr (SRC == kTma) {
            // A box brings a whole group, or one block: a load takes the TMA unit about 130
            // cycles and 0.8 for each of its 128-byte rows, so few wide ones are better.
            const bool wide = keys ? tb.key_blocks > 1 : tb.value_blocks > 1;
            const int slots = keys ? tb.key_slots : tb.value_slots;
            const int boxes = (keys ? 64 : kKeys) / slots;
            const uint32_t block = keys ? kBlockBytes : kValueBytes;
            if (keys) {
                const bool idle = wide && (i > 1 || (i == 1 && kblocks <= kQueryBlocks));
                const CUtensorMap* map = wide && i == 1 ? &tm_k1 : &tm_k0;
                const int step = wide ? kBlocks : 4;  // blocks between those of this warp
                const int brings = !wide ? 1 : i == 0 ? kTreeKeyBlocks : kTreeLastKeyBlocks;
                while (ok && __any_sync(0xffffffffu, w.next(a))) {
                    const int tiles = __shfl_sync(0xffffffffu, w.kt1 - w.kt0, 0);
                    ask(w);
                    for (int t = 0; t < tiles; ++t) {
                        if (!idle) {
                            const int64_t pos0 = static_cast<int64_t>(w.kt1 - 1 - t) * kKeys + rank * 64;
                            const Place at(a, w.b, lane < boxes ? pos0 + lane * slots : w.r.kv, w.r.kv);
                            for (int blk = wide ? i * kTreeKeyBlocks : i; blk < kblocks; blk += step) {
                                const uint32_t group = blk < kQueryBlocks ? 0 : 1;
                                ok = issue_wait(&bars->k_empty[group], (g & 1) ^ 1);
                                if (!ok) break;
                                if (leader && lane == 0)
                                    mbar_arrive_expect_tx(&bars->k_full[group], 2 * brings * block);
                                for (int x = 0; x < boxes; ++x)
                                    tma_load_4d_pair_elect(
                                        sK + blk * block + x * slots * 128, map, k_full + group * 8,
                                        wide ? 0 : blk * 64, __shfl_sync(0xffffffffu, at.slot, x),
                                        __shfl_sync(0xffffffffu, at.page, x), wide ? blk : 0);
                            }
                            if (!ok) break;
                            ++g;
                            if (i == 0 && lane == 0) bars->progress = static_cast<int32_t>(g);
                        }
                        if (t == 0) ok = queries(w);
                        if (!ok || idle) break;
                    }
                }
                if (!ok && lane == 0) bars->progress = INT32_MAX;
            } else {
                RingPos ring;            // place of the tile's first group
                uint32_t own_phase = 0;  // bit s: phase of v_own[s], which both groups use in turn
                const int first_block = value_block(rank, i);
                const int brings = wide ? ((i & 1) ? 0 : kTreeValueBlocks) : 1;
                while (ok && __any_sync(0xffffffffu, w.next(a))) {
                    ok = queries(w);
                    if (i >= 2 * vgroups) continue;
                    const int tiles = ok ? __shfl_sync(0xffffffffu, w.kt1 - w.kt0, 0) : 0;
                    const int behind = __shfl_sync(0xffffffffu, w.kt1 - w.cached_tiles(), 0);
                    for (int t = 0; t < tiles; ++t) {
                        const int64_t pos0 = static_cast<int64_t>(w.kt1 - 1 - t) * kKeys;
                        const Place at(a, w.b, lane < boxes ? pos0 + lane * slots : w.r.kv, w.r.kv);
                        RingPos mine = ring;
                        if (i >= 2) mine.next(kValueRing);
                        const uint32_t s = mine.stage;
                        uint8_t* dst = sV + s * 2 * kValueBytes + (i & 1) * kValueBytes;
                        ok = issue_wait(&bars->v_empty[s], mine.phase ^ 1);
                        if (!ok) break;
                        if (t >= behind) {
                            if (lane == 0) {
                                if (leader) mbar_arrive_expect_tx(&bars->v_full[s], 2 * brings * block);
                                else mbar_arrive_remote(v_full + s * 8);
                            }
                            for (int x = 0; brings > 0 && x < boxes; ++x)
                                tma_load_4d_pair_elect(
                                    dst + x * slots * 128, &tm_v, v_full + s * 8,
                                    wide ? 0 : first_block * 64, __shfl_sync(0xffffffffu, at.slot, x),
                                    __shfl_sync(0xffffffffu, at.page, x), wide ? first_block : 0);
                        } else {
                            // Drafts, which not every query attends, and rows past the last: a
                            // zero weight must not meet an infinity or NaN.  The CTA loads them
                            // for itself and makes those zero before it passes the block on.
                            // (A query that attends such a draft has it in its scores.)
                            if (lane == 0 && (brings > 0 || !wide))
                                mbar_arrive_expect_tx(&bars->v_own[s], brings * block);
                            for (int x = 0; brings > 0 && x < boxes; ++x)
                                tma_load_4d_elect(
                                    dst + x * slots * 128, &tm_v, &bars->v_own[s],
                                    wide ? 0 : first_block * 64, __shfl_sync(0xffffffffu, at.slot, x),
                                    __shfl_sync(0xffffffffu, at.page, x), wide ? first_block : 0);
                            ok = issue_wait(&bars->v_own[s], (own_phase >> s) & 1);
                            if (!ok) break;
                            const int drafts = static_cast<int>(
                                max(min(w.r.len, w.r.kv) - pos0, static_cast<int64_t>(0)));
                            const uint32_t from = smem_u32(dst) + (lane & 7) * 16;
                            // eight rows' chunks at a time, hardly ever one to be mended
#pragma unroll 1
                            for (int r = drafts & ~31; r < kKeys; r += 32) {
                                uint4 v[8];
#pragma unroll
                                for (int k = 0; k < 8; ++k)
                                    v[k] = ld_shared_v4(from + (r + k * 4 + (lane >> 3)) * 128);
#pragma unroll
                                for (int k = 0; k < 8; ++k) {
                                    const int x = r + k * 4 + (lane >> 3);
                                    if (x < drafts || !any_nonfinite(v[k])) continue;
                                    v[k] = finite8(v[k]);
                                    st_shared_v4(from + x * 128, v[k].x, v[k].y, v[k].z, v[k].w);
                                }
                            }
                            fence_proxy_async_smem();
                            __syncwarp();
                            if (lane == 0) mbar_arrive_publish(v_full + s * 8);
                        }
                        for (int v = 0; v < vgroups; ++v) {
                            if (t < behind) own_phase ^= 1u << ring.stage;
                            ring.next(kValueRing);
                        }
                    }
                }
            }
            if (!ok) spin_ns(kDrainNs);
        } else {
            by_loads<SRC>(a, bars, smem, rank, warp - kKeyWarp, kblocks, vgroups, k_full, tries, wc,
                          queries);
        }
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync_all();
    tc_fence_after();
    if (warp == kMmaWarp) tmem_dealloc_pair(tmem, kTmemCols);
}

constexpr int kJoinWarps = 8, kJoinThreads = kJoinWarps * 32;
// Blocks of an SM, all of them resident when the attention ends: with three the registers for a
// row's columns spilled (one user 1 us longer), with four more had to wait for the first.
constexpr int kJoinBlocks = 2;
constexpr int kFewParts = 8;  // that a warp joins alone (4 and 16: the same)

// Where the items of the pairs begin among the tasks of one kind, and the item of a task.
struct JoinTasks {
    int begins[kTreeMaxPairs + 1];

    // The last pair whose first task is at or before f.
    __device__ __forceinline__ int pair_of(int f, int pairs) const {
        int p = 0, behind = pairs;
        while (behind - p > 1) {
            const int mid = (p + behind) / 2;
            if (begins[mid] <= f) p = mid;
            else behind = mid;
        }
        return p;
    }
};

// Joins the parts of the items that several pairs share: with M the largest of the parts'
// maxima, out = sum 2^(m_k - M) O_k / sum 2^(m_k - M) l_k, the parts always in the same order.
// A lane has a row and 16 (few parts) or 32 of its columns.  Few parts, as of a batch whose
// items are cut a few times, are one warp's task each; many parts, as of few long histories,
// are dealt to the warps of a block, which meet in shared memory and then each finish a share
// of the columns.  Bound by latency: 5 to 9 us behind the attention's end for 10 to 40 MB of sums
// out of L2, 1 of them to start and 1 to find the tasks.
__global__ void __launch_bounds__(kJoinThreads, kJoinBlocks)
    tree_join_kernel(const TreeAttentionArgs a, const TreeWorkspace ws, const int pairs) {
    __shared__ TreeItem items[kTreeMaxPairs];
    __shared__ JoinTasks few, many;
    __shared__ float sums[kJoinWarps][32][32], tops[kJoinWarps][32], totals[kJoinWarps][32];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int R = a.kv_lora_rank;
    const bool sectors = (reinterpret_cast<uintptr_t>(a.out) & 31u) == 0;
    griddep_launch_dependents();
    griddep_wait();
    const TreeItem* left = reinterpret_cast<const TreeItem*>(a.workspace + ws.items);
    if (warp < 2) {  // the first for the items of few parts, the second for the others
        constexpr int kEach = (kTreeMaxPairs + 31) / 32;
        const int columns = warp == 0 ? R / 16 : R / 32;
        int* begins = warp == 0 ? few.begins : many.begins;
        int n[kEach], sum = 0;
#pragma unroll
        for (int k = 0; k < kEach; ++k) {
            const int p = lane * kEach + k;
            n[k] = 0;
            if (p < pairs) {
                const TreeItem it = left[p];
                if (warp == 0) items[p] = it;
                if ((it.parts <= kFewParts) == (warp == 0)) n[k] = (max(it.rows, 0) + 31) / 32 * columns;
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
        for (int k = 0; k < kEach; ++k) {
            const int p = lane * kEach + k;
            if (p <= pairs) begins[p] = at;
            at += n[k];
        }
    }
    __syncthreads();
    const float2* stats = reinterpret_cast<const float2*>(a.workspace + ws.stats);
    const float4* parts = reinterpret_cast<const float4*>(a.workspace + ws.parts);
    // part k of pair p's item: the pair's second slot, then the first slots of the pairs behind
    const auto slot = [](int p, int k) -> int64_t {
        return 2 * static_cast<int64_t>(p + k) + (k == 0 ? 1 : 0);
    };
    const int warp_tasks = few.begins[pairs], block_tasks = many.begins[pairs];
    for (int f = blockIdx.x * kJoinWarps + warp; f < warp_tasks; f += gridDim.x * kJoinWarps) {
        const int p = few.pair_of(f, pairs);
        const TreeItem it = items[p];
        const int task = f - few.begins[p], cg = task % (R / 16), row = task / (R / 16) * 32 + lane;
        if (row >= it.rows) continue;
        float top = -INFINITY, total = 0.0f;
        float o[16] = {};
        for (int k = 0; k < it.parts; ++k) {
            const float2 s = __ldcg(stats + slot(p, k) * ws.rows + row);
            const float4* from = parts + (slot(p, k) * (R / 4) + cg * 4) * ws.rows + row;
            float4 v[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) v[i] = __ldcg(from + static_cast<int64_t>(i) * ws.rows);
            const float m = fmaxf(top, s.x);
            const float f0 = top == -INFINITY ? 0.0f : exp2f(top - m);
            const float f1 = s.x == -INFINITY ? 0.0f : exp2f(s.x - m);
            top = m;
            total = total * f0 + s.y * f1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                o[4 * i] = o[4 * i] * f0 + v[i].x * f1;
                o[4 * i + 1] = o[4 * i + 1] * f0 + v[i].y * f1;
                o[4 * i + 2] = o[4 * i + 2] * f0 + v[i].z * f1;
                o[4 * i + 3] = o[4 * i + 3] * f0 + v[i].w * f1;
            }
        }
        const float inv = total != 0.0f ? 1.0f / total : 0.0f;
        uint16_t* out = a.out + (it.first + row) * R + cg * 16;
        uint32_t x[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) x[i] = pack_bf16x2(o[2 * i] * inv, o[2 * i + 1] * inv);
        if (sectors) {
            st_v8(out, x);
        } else {
            st_v4(out, make_uint4(x[0], x[1], x[2], x[3]));
            st_v4(out + 8, make_uint4(x[4], x[5], x[6], x[7]));
        }
        if (a.lse != nullptr && cg == 0)
            a.lse[it.first + row] = total != 0.0f ? top * kLn2 + logf(total) : -INFINITY;
    }
    for (int f = blockIdx.x; f < block_tasks; f += gridDim.x) {
        const int p = many.pair_of(f, pairs);
        const TreeItem it = items[p];
        const int task = f - many.begins[p];
        const int row_groups = (it.rows + 31) / 32;
        const int row = task % row_groups * 32 + lane, cg = task / row_groups;
        const bool live = row < it.rows;
        float top = -INFINITY, total = 0.0f;
        float o[32] = {};
        if (live)
#pragma unroll 2
            for (int k = warp; k < it.parts; k += kJoinWarps) {
                const float4* from = parts + (slot(p, k) * (R / 4) + cg * 8) * ws.rows + row;
                const float2 s = __ldcg(stats + slot(p, k) * ws.rows + row);
                float4 v[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = __ldcg(from + static_cast<int64_t>(i) * ws.rows);
                const float m = fmaxf(top, s.x);
                const float f0 = top == -INFINITY ? 0.0f : exp2f(top - m);
                const float f1 = s.x == -INFINITY ? 0.0f : exp2f(s.x - m);
                top = m;
                total = total * f0 + s.y * f1;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    o[4 * i] = o[4 * i] * f0 + v[i].x * f1;
                    o[4 * i + 1] = o[4 * i + 1] * f0 + v[i].y * f1;
                    o[4 * i + 2] = o[4 * i + 2] * f0 + v[i].z * f1;
                    o[4 * i + 3] = o[4 * i + 3] * f0 + v[i].w * f1;
                }
            }
        tops[warp][lane] = top;
        totals[warp][lane] = total;
#pragma unroll
        for (int i = 0; i < 32; ++i) sums[warp][i][lane] = o[i];
        __syncthreads();
        if (live) {
            float m = -INFINITY;
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k) m = fmaxf(m, tops[k][lane]);
            float x[4] = {}, sum = 0.0f;  // four columns a warp
#pragma unroll
            for (int k = 0; k < kJoinWarps; ++k) {
                const float t = tops[k][lane];
                const float w = t == -INFINITY ? 0.0f : exp2f(t - m);
                sum = fmaf(totals[k][lane], w, sum);
#pragma unroll
                for (int e = 0; e < 4; ++e) x[e] = fmaf(sums[k][warp * 4 + e][lane], w, x[e]);
            }
            const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;
            *reinterpret_cast<uint2*>(a.out + (it.first + row) * R + cg * 32 + warp * 4) =
                make_uint2(pack_bf16x2(x[0] * inv, x[1] * inv), pack_bf16x2(x[2] * inv, x[3] * inv));
            if (a.lse != nullptr && cg == 0 && warp == 0)
                a.lse[it.first + row] = sum != 0.0f ? m * kLn2 + logf(sum) : -INFINITY;
        }
        __syncthreads();
    }
}

template <Source SRC>
cudaError_t launch_source(const CUtensorMap& tm_q, const CUtensorMap& tm_k0, const CUtensorMap& tm_k1,
                          const CUtensorMap& tm_v, TreeAttentionArgs args,
                          const TreeWorkspace& ws, const TreeBoxes& boxes, int pairs,
                          cudaStream_t stream) {
    // once a device: the attribute stays (every thread sets the same value)
    static std::atomic<uint64_t> set[2] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const bool known = dev >= 0 && dev < 128;
    const uint64_t bit = uint64_t{1} << (dev & 63);
    if (!known || !(set[dev >> 6].load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(tree_attention_kernel<SRC>,
                                 cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(kSmemBytes));
        if (e != cudaSuccess) return e;
        if (known) set[dev >> 6].fetch_or(bit, std::memory_order_relaxed);
    }
    args.item_cost = item_cost(SRC);
    return launch_dependent(tree_attention_kernel<SRC>, static_cast<unsigned>(2 * pairs), kThreads,
                            kSmemBytes, stream, tm_q, tm_k0, tm_k1, tm_v, args, ws, boxes);
}

}  // namespace

cudaError_t launch_tree_attention(const CUtensorMap& tm_q, const CUtensorMap& tm_k0, const CUtensorMap& tm_k1,
                                  const CUtensorMap& tm_v, TreeAttentionArgs args, TreeBoxes boxes,
                                  int num_sms, cudaStream_t stream) {
    const TreeWorkspace ws = tree_workspace(args.total_rows, args.num_heads, args.kv_lora_rank);
    const int pairs = num_sms / 2 < kTreeMaxPairs ? num_sms / 2 : kTreeMaxPairs;
    // Boxes of at least 8 slots are whole swizzle atoms; smaller ones come by loads (pages of 128 that
    // way: 64 users x 1 token 1.6 times as long, large drafted trees 2.3 times).  With a rank of 512
    // no rope columns lie in the sets of four blocks, whose code then has no branches (with them
    // chains over the quantised cache take 1.3 times as long).
    const cudaError_t e =
        args.qcache_layer != nullptr
            ? (args.kv_lora_rank == 512 ? launch_source<kCodes> : launch_source<kCodesNarrow>)(
                  tm_q, tm_k0, tm_k1, tm_v, args, ws, boxes, pairs, stream)
        : boxes.key_slots >= 8 ? launch_source<kTma>(tm_q, tm_k0, tm_k1, tm_v, args, ws, boxes, pairs, stream)
                   : launch_source<kRows>(tm_q, tm_k0, tm_k1, tm_v, args, ws, boxes, pairs, stream);
    if (e != cudaSuccess) return e;
    return launch_dependent(tree_join_kernel, static_cast<unsigned>(num_sms) * kJoinBlocks, kJoinThreads, 0,
                            stream, args, ws, pairs);
}

}  // namespace pkm
