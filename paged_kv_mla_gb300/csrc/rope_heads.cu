// rope_heads.cu -- position rotation of the rope columns of every head of the queries.
//
// mla_prefill_decode_graph_fp8 (Modular MAX, attention/gpu/mla_graph), Args q (the query
// rows [tot_seq_len, num_heads, nope + rope]) and freqs_cis (rotary factors per position,
// [max_seq_len, qk_rope_head_dim]).  Row r turns by the P/2 (cos, sin) pairs of
// freqs_cis[positions[r]]: pair j is columns (2j, 2j + 1) in the interleaved layout and
// (j, j + P/2) in the half layout, and
//     (x0, x1) -> (x0 c - x1 s, x0 s + x1 c)     in fp32, rounded once to bf16.
//
// A streaming kernel: 2P bytes in and out per head, and the row's 4P bytes of factors once.
// A thread owns four pairs (eight columns) of a row and keeps their factors in registers
// while it walks over the heads, so the factors cost one read per row instead of one per
// head; its kUnroll heads are loaded before the first is stored, so that their latencies
// overlap, and before the row's position, on which only the factors wait.
//
// Measured (4096 rows x 128 heads x 64 columns out of 192): 25.4 us with the launch, 5.3 TB/s
// (0.80 of a plain copy), 21 us under the profiler; position first 28.7 us, then blocks of 256
// threads 26.7, of 64 25.7; 2 heads in flight 28.4, 8 (blocks of 256) 32.8 us.  A few rows, as
// of a drafted tree, are a launch (7 us).
#include "pkm_device.cuh"
#include "pkm_internal.h"

namespace pkm {
namespace {

constexpr int kThreads = 128;
constexpr int kUnroll = 4;  // heads in flight per thread

// Columns a thread loads: 16 bytes in the interleaved layout, twice 8 bytes (four columns of
// each half) in the half layout.
template <bool HALF>
__device__ __forceinline__ uint4 load_unit(const uint16_t* p, int half_cols) {
    if constexpr (HALF) {
        const uint2 a = *reinterpret_cast<const uint2*>(p);
        const uint2 b = *reinterpret_cast<const uint2*>(p + half_cols);
        return make_uint4(a.x, a.y, b.x, b.y);
    } else {
        return *reinterpret_cast<const uint4*>(p);
    }
}

template <bool HALF>
__device__ __forceinline__ void turn_and_store(uint16_t* p, int half_cols, uint4 v,
                                               const float (&cs)[8]) {
    float f[8];
    bf16x2_to_f32(v.x, f[0], f[1]);
    bf16x2_to_f32(v.y, f[2], f[3]);
    bf16x2_to_f32(v.z, f[4], f[5]);
    bf16x2_to_f32(v.w, f[6], f[7]);
    float o[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int i = HALF ? k : 2 * k, j = HALF ? k + 4 : 2 * k + 1;
        const float c = cs[2 * k], s = cs[2 * k + 1];
        o[i] = fmaf(f[i], c, -f[j] * s);
        o[j] = fmaf(f[i], s, f[j] * c);
    }
    const uint4 w = make_uint4(pack_bf16x2(o[0], o[1]), pack_bf16x2(o[2], o[3]),
                               pack_bf16x2(o[4], o[5]), pack_bf16x2(o[6], o[7]));
    if constexpr (HALF) {
        *reinterpret_cast<uint2*>(p) = make_uint2(w.x, w.y);
        *reinterpret_cast<uint2*>(p + half_cols) = make_uint2(w.z, w.w);
    } else {
        *reinterpret_cast<uint4*>(p) = w;
    }
}

// One block takes items (a row, a group of heads); unit u of a row is its pairs 4u .. 4u+3.
template <bool HALF>
__global__ void __launch_bounds__(kThreads) rope_heads_kernel(const RopeHeadsArgs a) {
    const int units = a.rope_dim / 8;
    const int heads_per_pass = kThreads / units;
    const int u = threadIdx.x % units, h_in = threadIdx.x / units;
    if (h_in >= heads_per_pass) return;
    const int group = heads_per_pass * kUnroll;
    const int groups = (a.num_heads + group - 1) / group;
    const int64_t items = static_cast<int64_t>(a.total_rows) * groups;
    const int half_cols = a.rope_dim / 2;
    for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
        const int64_t r = it / groups;
        const int h0 = static_cast<int>(it % groups) * group + h_in;
        const int col = HALF ? u * 4 : u * 8;
        const uint16_t* x = a.x + r * a.x_row_stride + col;
        uint16_t* y = a.y + r * a.y_row_stride + col;
        // the columns first: they need not wait for the position, as the factors do
        uint4 v[kUnroll];
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = h0 + i * heads_per_pass;
            if (h < a.num_heads) v[i] = load_unit<HALF>(x + h * a.x_head_stride, half_cols);
        }
        const uint32_t pos = __ldg(a.positions + r);
        if (pos >= static_cast<uint32_t>(a.max_seq_len)) {
            if (threadIdx.x == 0) report(a.status, PKM_ERR_OUT_OF_RANGE);
            continue;
        }
        const float4* fr = reinterpret_cast<const float4*>(
            a.freqs + static_cast<int64_t>(pos) * a.rope_dim + u * 8);
        const float4 c0 = __ldg(fr), c1 = __ldg(fr + 1);
        const float cs[8] = {c0.x, c0.y, c0.z, c0.w, c1.x, c1.y, c1.z, c1.w};
#pragma unroll
        for (int i = 0; i < kUnroll; ++i) {
            const int h = h0 + i * heads_per_pass;
            if (h < a.num_heads)
                turn_and_store<HALF>(y + h * a.y_head_stride, half_cols, v[i], cs);
        }
    }
}

}  // namespace

cudaError_t launch_rope_heads(RopeHeadsArgs args, int num_sms, cudaStream_t stream) {
    const int units = args.rope_dim / 8;
    const int group = kThreads / units * kUnroll;
    const int64_t items = static_cast<int64_t>(args.total_rows) *
                          ((args.num_heads + group - 1) / group);
    // at most eight blocks an SM are resident; beyond that blocks walk over the items
    const int64_t most = static_cast<int64_t>(num_sms) * 64;
    const unsigned blocks = static_cast<unsigned>(items < most ? items : most);
    if (args.half)
        rope_heads_kernel<true><<<blocks, kThreads, 0, stream>>>(args);
    else
        rope_heads_kernel<false><<<blocks, kThreads, 0, stream>>>(args);
    return cudaGetLastError();
}

}  // namespace pkm
