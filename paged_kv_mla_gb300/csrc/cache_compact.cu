// cache_compact.cu -- the accepted rows of a request's drafted tokens move to the front of
// its drafted region, in every layer of a paged cache.
//
// The cache is the PagedKVCacheCollection of kv_matmul_ragged_paged and
// mla_prefill_decode_graph_fp8 (Modular MAX; Args kv_collection); the pages describe writing
// behind each request's existing length, not what follows a rejected draft.  With the
// accepted drafts a[0] < a[1] < ... of request b, slot(len_b + j) = slot(len_b + a[j]).
//
// The moves of one request overlap (a destination can be a later move's source), so their
// order matters.  Since a increases strictly, a[j] >= j, and a source is never a destination
// of an earlier move: taking the moves in order is safe.  A thread owns 16 bytes of the row
// in one layer and makes all of the request's moves for them, so no two threads depend on
// each other and no barrier is needed; it loads kGroup rows before it stores the first,
// which the same argument allows, so that their latencies overlap.
//
// Bound by latency: a launch, then lengths and list, page ids, rows, one after the other.
// Measured: 128 requests x 8 rows of 1152 bytes x 16 layers 8.2 us (17 MB: 2.1 TB/s), 10.2 us
// while the offsets were found twice; one request is the call on the host, 7 to 8 us.
#include "pkm_device.cuh"
#include "pkm_internal.h"

namespace pkm {
namespace {

constexpr int kThreads = 256;
constexpr int kTable = 64;  // moves whose offsets are held in shared memory at a time
constexpr int kGroup = 8;   // rows in flight per thread

// Byte offset of a position's slot inside a layer, or -1 outside the page table or cache.
__device__ __forceinline__ int64_t slot_offset(const CompactArgs& a, int b, uint64_t pos) {
    const uint64_t lp = pos / static_cast<uint64_t>(a.page_size);
    if (lp >= static_cast<uint64_t>(a.max_pages)) return -1;
    const uint32_t page = __ldg(a.page_table + static_cast<int64_t>(b) * a.max_pages + lp);
    if (page >= static_cast<uint32_t>(a.num_pages)) return -1;
    return static_cast<int64_t>(page) * a.page_stride +
           static_cast<int64_t>(pos % static_cast<uint64_t>(a.page_size)) * a.slot_stride;
}

template <typename T>
__device__ __forceinline__ void move_rows(uint8_t* base, const int64_t* src, const int64_t* dst,
                                          int n) {
    for (int j = 0; j < n; j += kGroup) {
        T v[kGroup];
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
            if (j + k < n) v[k] = *reinterpret_cast<const T*>(base + src[j + k]);
#pragma unroll
        for (int k = 0; k < kGroup; ++k)
            if (j + k < n && src[j + k] != dst[j + k])
                *reinterpret_cast<T*>(base + dst[j + k]) = v[k];
    }
}

__global__ void __launch_bounds__(kThreads) cache_compact_kernel(const CompactArgs a) {
    __shared__ int64_t src[kTable], dst[kTable];
    const int b = blockIdx.x;
    const uint32_t len = __ldg(a.cache_lengths + b);
    const uint32_t count = __ldg(a.counts + b);
    const uint32_t* acc = a.accepted + static_cast<int64_t>(b) * a.max_accepted;
    // The request as a whole is checked first: it moves completely or not at all.  The list is
    // read along with its count, and the first table of offsets is filled in passing.
    int bad = 0;
    for (int j = threadIdx.x; j < a.max_accepted; j += kThreads) {
        const uint32_t t = __ldg(acc + j), before = j > 0 ? __ldg(acc + j - 1) : 0u;
        if (static_cast<uint32_t>(j) >= count) break;
        if (j > 0 && t <= before) bad = max(bad, int(PKM_ERR_INVALID_ARG));
        const int64_t from = slot_offset(a, b, static_cast<uint64_t>(len) + t);
        const int64_t to = slot_offset(a, b, static_cast<uint64_t>(len) + j);
        if (from < 0 || to < 0) bad = max(bad, int(PKM_ERR_OUT_OF_RANGE));
        if (j < kTable) {
            src[j] = from;
            dst[j] = to;
        }
    }
    if (count > static_cast<uint32_t>(a.max_accepted)) bad = PKM_ERR_INVALID_ARG;
    const bool any = __syncthreads_or(bad) != 0;
    if (bad != 0 && blockIdx.y == 0) report(a.status, bad);
    if (blockIdx.y == 0 && threadIdx.x == 0 && a.new_lengths != nullptr)
        a.new_lengths[b] = any ? len : len + count;
    if (any) return;
    const int wide = a.payload / 16, words = (a.payload % 16) / 4;
    const int per_row = wide + words;
    const int64_t units = static_cast<int64_t>(a.layer_count) * a.planes * per_row;
    for (uint32_t j0 = 0; j0 < count; j0 += kTable) {
        const int n = static_cast<int>(min(count - j0, static_cast<uint32_t>(kTable)));
        if (j0 > 0) {
            __syncthreads();  // the table's readers of the previous round are done
            for (int j = threadIdx.x; j < n; j += kThreads) {
                src[j] = slot_offset(a, b, static_cast<uint64_t>(len) + __ldg(acc + j0 + j));
                dst[j] = slot_offset(a, b, static_cast<uint64_t>(len) + j0 + j);
            }
            __syncthreads();
        }
        for (int64_t u = static_cast<int64_t>(blockIdx.y) * kThreads + threadIdx.x; u < units;
             u += static_cast<int64_t>(gridDim.y) * kThreads) {
            const int piece = static_cast<int>(u % per_row);
            const int64_t plane = u / per_row;
            uint8_t* base = a.data + (plane / a.planes) * a.layer_stride +
                            (plane % a.planes) * a.kv_stride;
            if (piece < wide)
                move_rows<uint4>(base + piece * 16, src, dst, n);
            else
                move_rows<uint32_t>(base + wide * 16 + (piece - wide) * 4, src, dst, n);
        }
    }
}

}  // namespace

cudaError_t launch_cache_compact(CompactArgs args, cudaStream_t stream) {
    const int per_row = args.payload / 16 + (args.payload % 16) / 4;
    const int64_t units = static_cast<int64_t>(args.layer_count) * args.planes * per_row;
    int64_t y = (units + kThreads - 1) / kThreads;
    if (y > 65535) y = 65535;
    const dim3 grid(static_cast<unsigned>(args.batch), static_cast<unsigned>(y));
    cache_compact_kernel<<<grid, kThreads, 0, stream>>>(args);
    return cudaGetLastError();
}

}  // namespace pkm
