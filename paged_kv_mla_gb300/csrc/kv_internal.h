// kv_internal.h -- argument blocks passed from the C entry points (api.cu) to the kernels on heads
// of the paged K/V cache (kv_rope.cu, kv_attention.cu).  Not part of the ABI.
#pragma once

#include "pkm_internal.h"

namespace pkm {

// One turn of new queries and keys and the write of keys and values, already validated
// (strides in elements).
struct KvRopeArgs {
    const uint16_t* q;             // [total_rows, num_heads, D] by strides
    uint16_t* q_out;
    int64_t q_row_stride, q_head_stride, q_out_row_stride, q_out_head_stride;
    const uint16_t* k;             // [total_rows, num_kv_heads, D], or null: in the cache already
    const uint16_t* v;             // likewise, or null: the V plane stays
    int64_t k_row_stride, k_head_stride, v_row_stride, v_head_stride;
    int32_t num_heads, num_kv_heads, head_size, rope_dim;
    const uint32_t* row_offsets;   // [batch + 1]
    int32_t batch, total_rows;
    const uint32_t* positions;     // [num_axes, total_rows]
    int32_t num_axes;
    uint8_t unit_axes[32];         // of the four pairs of every eight columns, two bits each
    const float* freqs;            // [max_seq_len, P]
    int32_t max_seq_len;
    int32_t half;                  // pairs (j, j + P/2) instead of (2j, 2j + 1)
    uint64_t page_inverse;         // floor(2^64 / page_size) + 1, or 0 for pages of one slot
    uint16_t* cache_layer;         // cache data + layer_idx * layer_stride
    int64_t page_stride, slot_stride, kv_stride;
    int32_t num_pages, page_size, max_pages;
    const uint32_t* page_table;
    const uint32_t* cache_lengths;
    int32_t* status;
};

// One attention over the paged K/V cache, already validated (strides in elements); the queries come
// by tensor maps.
struct KvAttentionArgs {
    const uint32_t* row_offsets;   // [batch + 1]
    int32_t batch, total_rows, num_heads, num_kv_heads, head_size;
    float scale;
    int32_t window;                // last positions that a token attends, or 0: all
    int32_t sinks;                 // first positions that it attends besides
    int32_t sink_tiles;            // 128-key tiles that hold them
    int32_t tile_tokens;           // tokens of a 128-row tile of queries
    uint64_t page_inverse;         // floor(2^64 / page_size) + 1, or 0 for pages of one slot
    const uint16_t* cache_layer;   // cache data + layer_idx * layer_stride
    int64_t page_stride, slot_stride, kv_stride;
    int32_t num_pages, page_size, max_pages;
    const uint32_t* page_table;
    const uint32_t* cache_lengths;
    uint16_t* out;                 // [total_rows, num_heads, D]
    float* lse;                    // [total_rows, num_heads], or null
    uint8_t* workspace;
    int32_t* status;
    uint64_t timeout_ns;
};

// Workspace of the attention: what CTAs that share an item (the query rows of one request, of one
// head of keys, up to 256 of them) leave for the kernel that joins their parts.  A CTA starts at
// most one item that it does not finish and finishes at most one that it did not start, so it has
// two slots.
constexpr int kKvMaxCtas = 160;
struct KvItem {         // an item that a CTA starts and leaves unfinished (tokens = 0: none)
    int64_t row;        // its first token's row
    int32_t head;       // its first head
    int32_t tokens, parts;
};
struct KvWorkspace {
    int32_t rows;       // query rows (token, head) that a slot holds
    size_t stats;       // float2 [2 * kKvMaxCtas, rows]: maximum (base 2) and sum, behind
                        // fp32 [2 * kKvMaxCtas, rows, D], unnormalised
    size_t items;       // KvItem [kKvMaxCtas]
    size_t bytes;
};

// Tokens of a 128-row tile of queries, the heads of a group side by side.
inline int32_t kv_tile_tokens(int32_t num_heads, int32_t num_kv_heads) {
    return 128 / (num_heads / num_kv_heads);
}

inline KvWorkspace kv_workspace(int32_t total_rows, int32_t num_heads, int32_t num_kv_heads,
                                int32_t head_size) {
    const auto up = [](size_t v) { return (v + 255) & ~static_cast<size_t>(255); };
    const int32_t group = num_heads / num_kv_heads;
    KvWorkspace w{};
    w.rows = total_rows <= kv_tile_tokens(num_heads, num_kv_heads) ? total_rows * group : 256;
    const size_t slots = 2 * kKvMaxCtas;
    w.stats = up(slots * w.rows * head_size * sizeof(float));
    w.items = w.stats + up(slots * w.rows * 2 * sizeof(float));
    w.bytes = w.items + up(kKvMaxCtas * sizeof(KvItem));
    return w;
}

// Tensor maps of the attention: the queries in boxes of a tile's tokens and of one token, and the
// two planes of the cache in boxes of `slots` slots of one page (0: loaded row by row).
struct KvMaps {
    CUtensorMap q, q_one, k, v;
    int32_t slots;
};

cudaError_t launch_kv_rope(KvRopeArgs args, int num_sms, cudaStream_t stream);
cudaError_t launch_kv_attention(const KvMaps& maps, KvAttentionArgs args, int num_sms,
                                cudaStream_t stream);

}  // namespace pkm
