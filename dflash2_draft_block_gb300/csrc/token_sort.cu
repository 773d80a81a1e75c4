// Token ids sorted for a gradient fold: (id, position) pairs in order of id, equal ids in
// order of position, so that every sum over a token's positions has one fixed order.
//
// A stable radix sort from the low digit up, by one thread-block cluster in one launch.
// CTA c of the cluster owns the c-th contiguous range of positions and warp w of it the
// w-th part of that, so (CTA, warp, step, lane) is the order of positions.  A pass over a
// digit of up to 9 bits:
//   1. every warp counts its digits in a histogram of its own (shared memory);
//   2. a digit's counts are scanned over the CTA's warps; the CTAs' totals are read
//      through distributed shared memory, which gives each CTA where its share of every
//      digit starts;
//   3. every warp walks its part again and scatters: a lane's place is its digit's start
//      plus the number of lower lanes of the warp with the same digit.
// The cluster barrier between passes also orders the passes' pairs, which go through L2.
//
// Bound: latency.  151,936 tokens are 18 bits, two passes; 16 CTAs (the largest cluster)
// hold 16,384 positions in one step of every warp.  A grid-wide sort would read the same
// few megabytes faster but needs a launch or a software barrier a step.
#include <cooperative_groups.h>

#include <mutex>
#include <unordered_map>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace df2 {
namespace {

constexpr int kSortThreads = 1024;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;

// hist [bins][kSortWarps + 1], total [bins], start [bins], carry [kSortWarps]
constexpr int kHistLd = kSortWarps + 1;  // odd: a digit's counts and a warp's both spread over the banks
size_t sort_smem(int bins) { return size_t(bins) * (kHistLd + 2) * 4 + kSortWarps * 4; }

__device__ __forceinline__ uint32_t key_of(const SortJob& j, int64_t n) {
    const int32_t id = __ldg(j.ids + n);
    if (id < 0) return uint32_t(j.V);
    if (id >= j.V) {
        if (j.status) atomicOr(j.status, DF2_STATUS_ID_OUT_OF_RANGE);
        return uint32_t(j.V);
    }
    if (j.label && __ldg(j.label + uint32_t(n) / j.per_label) < 0) return uint32_t(j.V);
    return uint32_t(id);
}

__global__ void __launch_bounds__(kSortThreads) token_sort_kernel(const SortJob job, int passes, int digit_bits) {
    extern __shared__ uint32_t smem[];
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), c = int(cluster.block_rank());
    const int bins = 1 << digit_bits;
    uint32_t* hist = smem;
    uint32_t* total = hist + bins * kHistLd;
    uint32_t* start = total + bins;
    uint32_t* carry = start + bins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    const int64_t per_cta = ((job.N + C - 1) / C + 31) / 32 * 32;
    const int64_t per_warp = ((per_cta + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t cta_end = dmin<int64_t>(job.N, (c + 1) * per_cta);
    const int64_t lo = c * per_cta + warp * per_warp;
    const int64_t hi = dmin<int64_t>(cta_end, lo + per_warp);

    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * digit_bits;
        const bool first = pass == 0;
        // the last pass ends in job.pairs
        const uint64_t* src = ((passes - pass) & 1) ? job.spare : job.pairs;
        uint64_t* dst = ((passes - pass) & 1) ? job.pairs : job.spare;

        for (int i = tid; i < bins * kHistLd; i += kSortThreads) hist[i] = 0;
        __syncthreads();
        for (int64_t n = lo + lane; n - lane < hi; n += 32) {
            const bool on = n < hi;
            const uint32_t key = !on ? 0u : first ? key_of(job, n) : uint32_t(__ldcg(src + n));
            const uint32_t d = on ? (key >> shift) & (bins - 1) : uint32_t(bins);
            const unsigned same = __match_any_sync(kFull, d);
            if (on && lane == __ffs(same) - 1) hist[d * kHistLd + warp] += __popc(same);
            __syncwarp();
        }
        __syncthreads();
        for (int d = tid; d < bins; d += kSortThreads) {
            uint32_t sum = 0;
#pragma unroll 8
            for (int w = 0; w < kSortWarps; ++w) {
                const uint32_t k = hist[d * kHistLd + w];
                hist[d * kHistLd + w] = sum;
                sum += k;
            }
            total[d] = sum;
        }
        cluster.sync();
        // bins <= 512 < threads: thread d owns digit d
        uint32_t all = 0, before = 0;
        if (tid < bins)
            for (int o = 0; o < C; ++o) {
                const uint32_t k = cluster.map_shared_rank(total, o)[tid];
                if (o < c) before += k;
                all += k;
            }
        uint32_t run = all;  // inclusive scan over the warp's digits
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t k = __shfl_up_sync(kFull, run, o);
            if (lane >= o) run += k;
        }
        if (lane == 31) carry[warp] = run;
        __syncthreads();
        if (warp == 0) {
            uint32_t k = carry[lane];
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t up = __shfl_up_sync(kFull, k, o);
                if (lane >= o) k += up;
            }
            carry[lane] = k;
        }
        __syncthreads();
        if (tid < bins) start[tid] = (warp ? carry[warp - 1] : 0u) + run - all + before;
        __syncthreads();
        for (int64_t n = lo + lane; n - lane < hi; n += 32) {
            const bool on = n < hi;
            uint64_t pair = 0;
            if (on) pair = first ? (uint64_t(uint32_t(n)) << 32) | key_of(job, n) : __ldcg(src + n);
            const uint32_t d = on ? (uint32_t(pair) >> shift) & (bins - 1) : uint32_t(bins);
            const unsigned same = __match_any_sync(kFull, d);
            const int leader = __ffs(same) - 1;
            uint32_t at = 0;
            if (on && lane == leader) {
                at = hist[d * kHistLd + warp];
                hist[d * kHistLd + warp] = at + __popc(same);
            }
            at = __shfl_sync(kFull, at, leader);
            if (on) __stcg(dst + start[d] + at + __popc(same & ((1u << lane) - 1)), pair);
            __syncwarp();
        }
        cluster.sync();  // this pass's pairs are written, and nobody reads `total` any more
    }
}

// 16 CTAs where the device can place such a cluster, else 8 (every device can); asked once
// a device.
cudaError_t largest_cluster(cudaLaunchConfig_t* cfg, int* most) {
    static std::mutex mu;
    static std::unordered_map<int, int> known;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    const auto it = known.find(dev);
    if (it != known.end()) {
        *most = it->second;
        return cudaSuccess;
    }
    const size_t smem = cfg->dynamicSmemBytes;
    cfg->dynamicSmemBytes = sort_smem(kMaxBins);
    cfg->gridDim = dim3(kMaxCluster);
    cfg->attrs[0].val.clusterDim.x = kMaxCluster;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, token_sort_kernel, cfg);
    cfg->dynamicSmemBytes = smem;
    if (e != cudaSuccess) return e;
    *most = known[dev] = n > 0 ? kMaxCluster : 8;
    return cudaSuccess;
}

}  // namespace

size_t token_sort_bytes(int64_t N) { return size_t(N) * 8; }

cudaError_t token_sort_launch(const SortJob& job, cudaStream_t stream) {
    // keys 0 .. V (V: no token); equal digits a pass
    int bits = 0;
    while ((int64_t(job.V) >> bits) != 0) ++bits;
    const int passes = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
    const int digit_bits = (bits + passes - 1) / passes;
    const size_t smem = sort_smem(1 << digit_bits);
    cudaError_t e = cudaFuncSetAttribute(token_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         int(sort_smem(kMaxBins)));
    if (e == cudaSuccess) e = cudaFuncSetAttribute(token_sort_kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // one step of every warp a CTA, up to the largest cluster this device can place
    int most = 0;
    e = largest_cluster(&cfg, &most);
    if (e != cudaSuccess) return e;
    int C = 1;
    while (C < most && int64_t(C) * kSortThreads < job.N) C *= 2;
    cfg.gridDim = dim3(unsigned(C));
    attr[0].val.clusterDim.x = unsigned(C);
    e = cudaLaunchKernelEx(&cfg, token_sort_kernel, job, passes, digit_bits);
    note_launch();
    return e;
}

}  // namespace df2
