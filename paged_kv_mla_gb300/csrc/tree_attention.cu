// tree_attention.cu -- absorbed MLA attention of new (drafted) tokens over the paged latent
// cache: one warp per (token, head), online softmax, fp32 throughout.
#include "pkm_device.cuh"
#include "pkm_internal.h"

namespace pkm {
namespace {

constexpr int kThreads = 128;
constexpr int kPieces = 3;  // 8-column pieces a lane holds of a row of up to 768 columns

__device__ __forceinline__ void unpack8(const uint4 v, float (&f)[8]) {
    bf16x2_to_f32(v.x, f[0], f[1]);
    bf16x2_to_f32(v.y, f[2], f[3]);
    bf16x2_to_f32(v.z, f[4], f[5]);
    bf16x2_to_f32(v.w, f[6], f[7]);
}

__device__ __forceinline__ float e4m3_value(uint8_t c) {
    const uint32_t e = (c >> 3) & 15u, m = c & 7u;
    float v = e == 0 ? static_cast<float>(m) * 0x1p-9f
                     : (1.0f + static_cast<float>(m) * 0.125f) * exp2f(static_cast<float>(e) - 7.0f);
    if (e == 15 && m == 7) v = __int_as_float(0x7fffffff);
    return (c & 128u) ? -v : v;
}

__global__ void __launch_bounds__(kThreads) tree_attention_kernel(const TreeAttentionArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    if (row >= static_cast<int64_t>(a.total_rows) * a.num_heads) return;
    const int64_t r = row / a.num_heads;
    const uint32_t* iro = a.row_offsets;
    const int64_t end = min(static_cast<int64_t>(__ldg(iro + a.batch)), static_cast<int64_t>(a.total_rows));
    if (r >= end || r < static_cast<int64_t>(__ldg(iro))) return;
    int lo = 0, hi = a.batch;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (static_cast<int64_t>(__ldg(iro + mid)) <= r) lo = mid;
        else hi = mid;
    }
    const int b = lo;
    const int64_t first = __ldg(iro + b);
    const int64_t n = min(static_cast<int64_t>(__ldg(iro + b + 1)), end) - first;
    const int64_t i = r - first;
    const int64_t len = __ldg(a.cache_lengths + b);
    int64_t kv = len + n;
    const int64_t held = static_cast<int64_t>(a.max_pages) * a.page_size;
    if (kv > held) {
        kv = held;
        if (lane == 0) report(a.status, PKM_ERR_OUT_OF_RANGE);
    }
    const int cols = a.cols, rank = a.kv_lora_rank;
    float q[kPieces][8], o[kPieces][8] = {};
    for (int p = 0; p < kPieces; ++p) {
        const int c = (lane + 32 * p) * 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < cols) v = *reinterpret_cast<const uint4*>(a.q + row * cols + c);
        unpack8(v, q[p]);
    }
    float m = -INFINITY, l = 0.0f;
    for (int64_t t = 0; t < kv; ++t) {
        if (t >= len) {
            const int64_t j = t - len;
            bool seen = j <= i;
            if (a.mask != nullptr)
                seen = j < 32 * static_cast<int64_t>(a.mask_words) &&
                       ((__ldg(a.mask + r * a.mask_words + j / 32) >> (j % 32)) & 1u);
            if (!seen) continue;
        }
        const uint32_t page = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + t / a.page_size);
        if (page >= static_cast<uint32_t>(a.num_pages)) {
            if (lane == 0) report(a.status, PKM_ERR_OUT_OF_RANGE);
            continue;
        }
        const int64_t off = page * a.page_stride + (t % a.page_size) * a.slot_stride;
        float k[kPieces][8], s = 0.0f;
        for (int p = 0; p < kPieces; ++p) {
            const int c = (lane + 32 * p) * 8;
            for (int e = 0; e < 8; ++e) k[p][e] = 0.0f;
            if (c < cols) {
                if (a.qcache_layer == nullptr) {
                    unpack8(*reinterpret_cast<const uint4*>(a.cache_layer + off + c), k[p]);
                } else if (c >= rank) {
                    unpack8(*reinterpret_cast<const uint4*>(a.qcache_layer + off + rank + 2 * (c - rank)), k[p]);
                } else {
                    const float scale = *reinterpret_cast<const float*>(
                        a.qcache_layer + off + rank + 2 * (cols - rank) + 4 * (c / 128));
                    for (int e = 0; e < 8; ++e)
                        k[p][e] = __bfloat162float(__float2bfloat16_rn(
                            e4m3_value(a.qcache_layer[off + c + e]) * scale));
                }
            }
            for (int e = 0; e < 8; ++e) s = fmaf(q[p][e], k[p][e], s);
        }
        for (int sh = 16; sh >= 1; sh >>= 1) s += __shfl_xor_sync(0xffffffffu, s, sh);
        s *= a.scale;
        const float m_new = fmaxf(m, s);
        const float f = m == -INFINITY ? 0.0f : expf(m - m_new), w = expf(s - m_new);
        l = l * f + w;
        m = m_new;
        for (int p = 0; p < kPieces; ++p)
            for (int e = 0; e < 8; ++e) o[p][e] = o[p][e] * f + w * k[p][e];
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    for (int p = 0; p < kPieces; ++p) {
        const int c = (lane + 32 * p) * 8;
        if (c >= rank) continue;
        st_v4(a.out + row * rank + c,
              make_uint4(pack_bf16x2(o[p][0] * inv, o[p][1] * inv), pack_bf16x2(o[p][2] * inv, o[p][3] * inv),
                         pack_bf16x2(o[p][4] * inv, o[p][5] * inv), pack_bf16x2(o[p][6] * inv, o[p][7] * inv)));
    }
    if (lane == 0 && a.lse != nullptr) a.lse[row] = l > 0.0f ? m + logf(l) : -INFINITY;
}

}  // namespace

cudaError_t launch_tree_attention(TreeAttentionArgs args, int num_sms, cudaStream_t stream) {
    (void)num_sms;
    const int64_t rows = static_cast<int64_t>(args.total_rows) * args.num_heads;
    tree_attention_kernel<<<static_cast<unsigned>((rows + 3) / 4), kThreads, 0, stream>>>(args);
    return cudaGetLastError();
}

}  // namespace pkm
