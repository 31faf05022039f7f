// kv_rope.cu -- positions of new queries and keys, and the keys' and values' way into the
// paged K/V cache.
//
// kv_matmul_ragged_paged (Modular MAX, nn/kv_cache_ragged) writes keys and values; freqs_cis
// of mla_prefill_decode_graph_fp8 (attention/gpu/mla_graph) gives the rotary factors.  Here a
// token has a position on each of up to four axes (time, height, width), and pair j of a
// head's columns turns by the factor j of the position on the axis that the pair belongs to:
//     (x0, x1) -> (x0 c - x1 s, x0 s + x1 c)     in fp32, rounded once to bf16,
// pair j being columns (2j, 2j + 1) or (j, j + P/2).  Columns past the first P are copied.
//
// A streaming kernel: every value once in and once out.  An item is one row and a group of its
// heads, in the line of queries, keys and values; a thread has a unit of eight columns, which
// holds four whole pairs, keeps their factors in registers and walks over heads, four loads in
// flight.  The columns are asked for before the row's position and slot, which hang on a chain
// of loads (offsets, length, page id).
//
// Bound by the latency of those chains and by how many blocks an SM holds: 5 000 rows of 32 heads of
// queries and 8 of keys and values, D = 128, three axes (126 MB) take 27 us, 4.7 TB/s.  Blocks that
// stay and walk over items (39 us with one item a block), all positions of a row loaded at once and
// divisions by multiplication make it so.  Blocks an SM: 8 take 30.5 us, 9 28.7, 11 and 12, which
// spill, 32; heads in flight: three 27.3 us, two 31, six (7 blocks) 28.9.  37 rows take what a call
// takes from the host, 12 us.
#include "pkm_device.cuh"
#include "kv_internal.h"

namespace pkm {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // heads of an item a thread has
constexpr int kBlocks = 10;  // of an SM, all resident

// Columns of a turned unit: 16 bytes in the interleaved layout, twice 8 bytes (four columns of
// each half) in the half layout; copied units are 16 bytes in both.
__device__ __forceinline__ uint4 load_unit(const uint16_t* p, int second) {
    if (second == 0) return *reinterpret_cast<const uint4*>(p);
    const uint2 a = *reinterpret_cast<const uint2*>(p);
    const uint2 b = *reinterpret_cast<const uint2*>(p + second);
    return make_uint4(a.x, a.y, b.x, b.y);
}

__device__ __forceinline__ void store_unit(uint16_t* p, int second, uint4 w) {
    if (second == 0) {
        *reinterpret_cast<uint4*>(p) = w;
    } else {
        *reinterpret_cast<uint2*>(p) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2*>(p + second) = make_uint2(w.z, w.w);
    }
}

template <bool HALF>
__device__ __forceinline__ uint4 turned(uint4 v, const float (&cs)[8]) {
    float f[8], o[8];
    bf16x2_to_f32(v.x, f[0], f[1]);
    bf16x2_to_f32(v.y, f[2], f[3]);
    bf16x2_to_f32(v.z, f[4], f[5]);
    bf16x2_to_f32(v.w, f[6], f[7]);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = HALF ? k : 2 * k, j = HALF ? k + 4 : 2 * k + 1;
        const float c = cs[2 * k], s = cs[2 * k + 1];
        o[i] = fmaf(f[i], c, -f[j] * s);
        o[j] = fmaf(f[i], s, f[j] * c);
    }
    return make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                      pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
}

// Request of row r, or -1 when none covers it, found by all lanes of a warp: each step looks at
// 32 entries that divide what is left.
__device__ __forceinline__ int request_of(const uint32_t* offsets, int batch, uint32_t r) {
    const int lane = threadIdx.x & 31;
    int lo = 0, n = batch + 1;  // the last entry at or below r is among lo .. lo + n - 1
    while (n > 1) {
        const int step = (n + 31) / 32;
        const int at = lane * step;
        const bool below = at < n && __ldg(offsets + lo + at) <= r;
        const uint32_t m = __ballot_sync(0xffffffffu, below);
        if ((m & 1u) == 0) return -1;
        const int k = 31 - __clz(static_cast<int>(m));
        lo += k * step;
        n = min(step, n - k * step);
    }
    return lo < batch && __ldg(offsets + lo) <= r ? lo : -1;
}

template <bool HALF>
__global__ void __launch_bounds__(kThreads, kBlocks) kv_rope_kernel(const KvRopeArgs a) {
    const int units = a.head_size / 8;
    const int heads_per_pass = kThreads / units;
    const int u = threadIdx.x % units, h_in = threadIdx.x / units;
    const int group = heads_per_pass * kUnroll;
    // the line of a row's heads: queries, keys, values
    const int first_value = a.num_heads + a.num_kv_heads;
    const int heads = first_value + (a.v != nullptr ? a.num_kv_heads : 0);
    const int groups = (heads + group - 1) / group;
    const bool turns = u * 8 < a.rope_dim;
    const int col = HALF && turns ? u * 4 : u * 8;
    const int second = HALF && turns ? a.rope_dim / 2 : 0;
    const bool in_use = h_in < heads_per_pass;
    const uint32_t axes = turns ? a.unit_axes[u] : 0;
    const uint32_t rows = static_cast<uint32_t>(a.total_rows);
    const uint32_t covered = __ldg(a.row_offsets), behind = __ldg(a.row_offsets + a.batch);

    // a block's items are gridDim.x apart in the line of all rows' groups of heads
    const int step = static_cast<int>(gridDim.x % groups);
    int g = static_cast<int>(blockIdx.x % groups) - step;
    uint32_t it = blockIdx.x / groups - gridDim.x / groups;
    while (true) {
        it += gridDim.x / groups;
        g += step;
        if (g >= groups) {
            g -= groups;
            ++it;
        }
        if (it >= rows) break;
        const int64_t r = it;
        const int h0 = g * group + h_in;
        uint4 v[kUnroll];
        const uint16_t* q = a.q + r * a.q_row_stride + col;
        const uint16_t* k = a.k + r * a.k_row_stride + col;
        const uint16_t* values = a.v + r * a.v_row_stride + u * 8;  // copied in whole units
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = h0 + i * heads_per_pass;
            if (!in_use || h >= heads) continue;
            if (h < a.num_heads) v[i] = load_unit(q + h * a.q_head_stride, second);
            else if (h >= first_value) v[i] = load_unit(values + (h - first_value) * a.v_head_stride, 0);
            else if (a.k != nullptr) v[i] = load_unit(k + (h - a.num_heads) * a.k_head_stride, second);
        }
        // all positions at once; the factors do not wait for the row's request
        uint32_t pos[4];
#pragma unroll
        for (int n = 0; n < 4; ++n)
            pos[n] = n < a.num_axes ? __ldg(a.positions + static_cast<int64_t>(n) * a.total_rows + r) : 0;
        const bool inside = max(max(pos[0], pos[1]), max(pos[2], pos[3])) < static_cast<uint32_t>(a.max_seq_len);
        float cs[8] = {};
        if (inside && turns) {
            const auto factors = [&](uint32_t axis) -> const float* {
                const uint32_t lo = axis & 1u ? pos[1] : pos[0], hi = axis & 1u ? pos[3] : pos[2];
                return a.freqs + static_cast<int64_t>(axis & 2u ? hi : lo) * a.rope_dim + u * 8;
            };
            if (axes == (axes & 3u) * 0x55u) {  // the four pairs are of one axis
                const float4* f = reinterpret_cast<const float4*>(factors(axes & 3u));
                const float4 f0 = __ldg(f), f1 = __ldg(f + 1);
                cs[0] = f0.x, cs[1] = f0.y, cs[2] = f0.z, cs[3] = f0.w;
                cs[4] = f1.x, cs[5] = f1.y, cs[6] = f1.z, cs[7] = f1.w;
            } else {
#pragma unroll
                for (int n = 0; n < 4; ++n) {
                    const float2 f = __ldg(reinterpret_cast<const float2*>(factors(axes >> (2 * n) & 3u)) + n);
                    cs[2 * n] = f.x;
                    cs[2 * n + 1] = f.y;
                }
            }
        }
        if (it < covered || it >= behind) continue;  // of no request
        if (!inside) {
            if (threadIdx.x == 0) report(a.status, PKM_ERR_OUT_OF_RANGE);
            continue;
        }
        uint16_t* cell = nullptr;  // the row's slot
        if (g * group + group > a.num_heads) {
            const int b = request_of(a.row_offsets, a.batch, it);
            if (b >= 0) {
                const uint64_t at = static_cast<uint64_t>(__ldg(a.cache_lengths + b)) + (it - __ldg(a.row_offsets + b));
                // at / page_size for positions below 2^33: off by less than 2^-31 before rounding down
                const uint64_t lp = a.page_inverse == 0 ? at : __umul64hi(at, a.page_inverse);
                uint32_t page = UINT32_MAX;
                if (lp < static_cast<uint64_t>(a.max_pages))
                    page = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + lp);
                if (page < static_cast<uint32_t>(a.num_pages))
                    cell = a.cache_layer + static_cast<int64_t>(page) * a.page_stride +
                           static_cast<int64_t>(at - lp * a.page_size) * a.slot_stride;
                else if (threadIdx.x == 0)
                    report(a.status, PKM_ERR_OUT_OF_RANGE);
            }
        }
        if (!in_use) continue;
        uint16_t* q_out = a.q_out + r * a.q_out_row_stride + col;
        if (a.k == nullptr && cell != nullptr && turns) {  // keys, turned in place
#pragma unroll
            for (int i = 0; i < kUnroll; ++i) {
                const int h = h0 + i * heads_per_pass;
                if (h >= a.num_heads && h < first_value)
                    v[i] = load_unit(cell + (h - a.num_heads) * a.head_size + col, second);
            }
        }
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = h0 + i * heads_per_pass;
            if (h >= heads) continue;
            if (h >= first_value) {
                if (cell != nullptr)
                    store_unit(cell + a.kv_stride + (h - first_value) * a.head_size + u * 8, 0, v[i]);
                continue;
            }
            const bool query = h < a.num_heads;
            if (!query && cell == nullptr) continue;
            uint16_t* to = query ? q_out + h * a.q_out_head_stride : cell + (h - a.num_heads) * a.head_size + col;
            if (turns) store_unit(to, second, turned<HALF>(v[i], cs));
            else if (query ? a.q != a.q_out : a.k != nullptr) store_unit(to, 0, v[i]);
        }
    }
}

}  // namespace

cudaError_t launch_kv_rope(KvRopeArgs args, int num_sms, cudaStream_t stream) {
    const int group = kThreads / (args.head_size / 8) * kUnroll;
    const int64_t heads = args.num_heads + static_cast<int64_t>(args.num_kv_heads) * (args.v != nullptr ? 2 : 1);
    const int64_t groups = (heads + group - 1) / group;
    const int64_t items = args.total_rows * groups, most = static_cast<int64_t>(num_sms) * kBlocks;
    unsigned blocks = static_cast<unsigned>(items < most ? items : most);
    if (items > most && most % groups == 0) --blocks;  // all blocks meet all groups of heads
    if (args.half)
        kv_rope_kernel<true><<<blocks, kThreads, 0, stream>>>(args);
    else
        kv_rope_kernel<false><<<blocks, kThreads, 0, stream>>>(args);
    return cudaGetLastError();
}

}  // namespace pkm
