// kv_attention.cu -- attention of new tokens over the paged K/V cache that kv_matmul_paged fills.
//
// kv_matmul_ragged_paged (Modular MAX, nn/kv_cache_ragged): Args kv_collection (the K and V
// cache), layer_idx, input_row_offsets.  Heads in groups of num_heads / num_kv_heads share keys
// and values.  A warp takes one (token, head), its lanes the columns, and walks over the keys
// with a running maximum and sum.
#include "pkm_device.cuh"
#include "pkm_internal.h"

namespace pkm {
namespace {

constexpr int kWarps = 8;
constexpr float kLn2 = 0.6931471805599453f, kLog2e = 1.4426950408889634f;

template <int E>  // columns of a lane
__global__ void __launch_bounds__(kWarps * 32) kv_attention_kernel(const KvAttentionArgs a) {
    const int lane = threadIdx.x & 31;
    const int64_t all = static_cast<int64_t>(a.total_rows) * a.num_heads;
    const int64_t task = static_cast<int64_t>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    if (task >= all) return;
    const int64_t r = task / a.num_heads;
    const int h = static_cast<int>(task % a.num_heads);
    const int kvh = h / (a.num_heads / a.num_kv_heads);
    int b = -1;
    for (int lo = 0, hi = a.batch; b < 0;) {
        if (hi - lo <= 1) b = lo;
        else if (__ldg(a.row_offsets + (lo + hi) / 2) <= r) lo = (lo + hi) / 2;
        else hi = (lo + hi) / 2;
    }
    if (r < __ldg(a.row_offsets + b) || r >= __ldg(a.row_offsets + b + 1)) return;
    const int64_t p = static_cast<int64_t>(__ldg(a.cache_lengths + b)) + r - __ldg(a.row_offsets + b);
    const uint16_t* q = a.q + r * a.q_row_stride + h * a.q_head_stride + lane * E;
    float qv[E], o[E] = {};
    for (int e = 0; e < E; e += 2) bf16x2_to_f32(*reinterpret_cast<const uint32_t*>(q + e), qv[e], qv[e + 1]);
    float m = -INFINITY, l = 0.0f;
    int64_t first = 0;
    if (a.window > 0 && p >= a.window) first = p + 1 - a.window;
    const int64_t sinks = min(first, static_cast<int64_t>(a.sinks));
    for (int64_t n = 0; n < sinks + p + 1 - first; ++n) {
        const int64_t t = n < sinks ? n : first + n - sinks;
        const int64_t lp = t / a.page_size;
        uint32_t page = UINT32_MAX;
        if (lp < a.max_pages) page = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + lp);
        if (page >= static_cast<uint32_t>(a.num_pages)) {
            if (lane == 0) report(a.status, PKM_ERR_OUT_OF_RANGE);
            continue;
        }
        const uint16_t* k = a.cache_layer + page * a.page_stride + (t % a.page_size) * a.slot_stride +
                            kvh * a.head_size + lane * E;
        float s = 0.0f, x[E];
        for (int e = 0; e < E; e += 2) {
            bf16x2_to_f32(*reinterpret_cast<const uint32_t*>(k + e), x[e], x[e + 1]);
            s += qv[e] * x[e] + qv[e + 1] * x[e + 1];
        }
        for (int d = 16; d > 0; d /= 2) s += __shfl_xor_sync(0xffffffffu, s, d);
        s *= a.scale * kLog2e;
        const float top = fmaxf(m, s);
        const float back = m == -INFINITY ? 0.0f : exp2f(m - top);
        const float w = exp2f(s - top);
        m = top;
        l = l * back + w;
        for (int e = 0; e < E; e += 2) {
            bf16x2_to_f32(*reinterpret_cast<const uint32_t*>(k + a.kv_stride + e), x[e], x[e + 1]);
            o[e] = o[e] * back + w * x[e];
            o[e + 1] = o[e + 1] * back + w * x[e + 1];
        }
    }
    const float inv = l > 0.0f ? 1.0f / l : 0.0f;
    for (int e = 0; e < E; e += 2)
        *reinterpret_cast<uint32_t*>(a.out + task * a.head_size + lane * E + e) =
            pack_bf16x2(o[e] * inv, o[e + 1] * inv);
    if (lane == 0 && a.lse != nullptr) a.lse[task] = m * kLn2 + logf(l);
}

}  // namespace

cudaError_t launch_kv_attention(KvAttentionArgs args, int, cudaStream_t stream) {
    const int64_t all = static_cast<int64_t>(args.total_rows) * args.num_heads;
    const unsigned blocks = static_cast<unsigned>((all + kWarps - 1) / kWarps);
    if (args.head_size == 64)
        kv_attention_kernel<2><<<blocks, kWarps * 32, 0, stream>>>(args);
    else
        kv_attention_kernel<4><<<blocks, kWarps * 32, 0, stream>>>(args);
    return cudaGetLastError();
}

}  // namespace pkm
