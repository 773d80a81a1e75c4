// Token ids sorted for a gradient fold: (id, position) pairs in order of id, equal ids in
// order of position, so that every sum over a token's positions has one fixed order.
//
// A stable radix sort from the low digit up, by one thread-block cluster a list, every list
// of a call in one launch.  CTA c of a cluster owns the c-th contiguous range of positions
// and warp w of it the w-th part of that, so (CTA, warp, step, lane) is the order of
// positions.  A pass over a digit of up to 9 bits:
//   1. every warp ranks its positions among those of equal digit: the lanes of a step find
//      their equals with a vote a bit (a match instruction took five times as long: its
//      time grows with the number of different digits), and a histogram of the warp's own
//      (shared memory) holds the counts of the steps before;
//   2. a digit's counts are scanned over the CTA's warps; the CTAs' totals are read
//      through distributed shared memory, which gives each CTA where its share of every
//      digit starts;
//   3. every lane scatters its pairs, from the registers that have held them since step 1
//      (lists over 16 positions a thread are read and ranked a second time).
// The cluster barrier between passes also orders the passes' pairs, which go through L2.
//
// Bound: latency.  151,936 tokens are 18 bits, two passes; 16 CTAs (the largest cluster)
// hold 16,384 positions a step of every warp.  A grid-wide sort would have more lanes but
// needs a launch or a software barrier a step.
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
    if (id < 0) return j.V;
    if (uint32_t(id) >= j.V) {
        if (j.status) atomicOr(j.status, DF2_STATUS_ID_OUT_OF_RANGE);
        return j.V;
    }
    return uint32_t(id);
}

struct SortArgs {
    SortJob job[kMaxJobs];
    int passes[kMaxJobs];
    int digit_bits[kMaxJobs];
};

// ITEMS: positions a lane holds at a time.
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) token_sort_kernel(const __grid_constant__ SortArgs args) {
    extern __shared__ uint32_t smem[];
    // let the next kernel start beside this one (one that was launched to allow it)
    asm volatile("griddepcontrol.launch_dependents;");
    cg::cluster_group cluster = cg::this_cluster();
    const int C = int(cluster.num_blocks()), c = int(cluster.block_rank());
    const SortJob& job = args.job[blockIdx.x / C];
    const int passes = args.passes[blockIdx.x / C], digit_bits = args.digit_bits[blockIdx.x / C];
    const int bins = 1 << digit_bits;
    uint32_t* hist = smem;
    uint32_t* total = hist + bins * kHistLd;
    uint32_t* start = total + bins;
    uint32_t* carry = start + bins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const unsigned below = (1u << lane) - 1;

    const int64_t per_cta = ((job.N + C - 1) / C + 31) / 32 * 32;
    const int64_t per_warp = ((per_cta + kSortWarps - 1) / kSortWarps + 31) / 32 * 32;
    const int64_t cta_end = dmin<int64_t>(job.N, (c + 1) * per_cta);
    const int64_t lo = c * per_cta + warp * per_warp;
    const int64_t hi = dmin<int64_t>(cta_end, lo + per_warp);
    const int rounds = int((per_warp + 32 * ITEMS - 1) / (32 * ITEMS));

    uint64_t pair[ITEMS];
    uint32_t rank[ITEMS];
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * digit_bits;
        // the last pass ends in job.pairs
        const uint64_t* src = ((passes - pass) & 1) ? job.spare : job.pairs;
        uint64_t* dst = ((passes - pass) & 1) ? job.pairs : job.spare;
        auto digit = [&](uint64_t x) { return (uint32_t(x) >> shift) & (bins - 1); };
        auto load = [&](int64_t from) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const int64_t n = from + i * 32 + lane;
                pair[i] = 0;
                if (n < hi) pair[i] = pass == 0 ? (uint64_t(uint32_t(n)) << 32) | key_of(job, n) : __ldcg(src + n);
            }
        };
        // each lane's rank among the warp's equal digits so far; hist holds the counts
        auto rank_all = [&](int64_t from) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if (from + i * 32 >= hi) break;
                const bool on = from + i * 32 + lane < hi;
                const uint32_t d = digit(pair[i]);
                unsigned same = __ballot_sync(kFull, on);
#pragma unroll
                for (int b = 0; b < kMaxDigitBits; ++b) {
                    const bool one = d >> b & 1;
                    const unsigned ones = __ballot_sync(kFull, one);
                    same &= one ? ones : ~ones;
                }
                const int leader = on ? __ffs(same) - 1 : lane;
                uint32_t at = 0;
                if (on && lane == leader) {
                    at = hist[d * kHistLd + warp];
                    hist[d * kHistLd + warp] = at + __popc(same);
                }
                rank[i] = __shfl_sync(kFull, at, leader) + __popc(same & below);
                __syncwarp();
            }
        };

        for (int i = tid; i < bins * kHistLd; i += kSortThreads) hist[i] = 0;
        __syncthreads();
        for (int k = 0; k < rounds; ++k) {
            load(lo + int64_t(k) * 32 * ITEMS);
            rank_all(lo + int64_t(k) * 32 * ITEMS);
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
        if (tid < bins) {
#pragma unroll 8
            for (int o = 0; o < C; ++o) {
                const uint32_t k = cluster.map_shared_rank(total, o)[tid];
                if (o < c) before += k;
                all += k;
            }
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
        for (int k = 0; k < rounds; ++k) {
            const int64_t from = lo + int64_t(k) * 32 * ITEMS;
            if (rounds > 1) {  // again, this time from the warp's share of each digit on
                load(from);
                rank_all(from);
            }
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if (from + i * 32 + lane >= hi) break;
                const uint32_t d = digit(pair[i]);
                __stcg(dst + start[d] + rank[i] + (rounds > 1 ? 0u : hist[d * kHistLd + warp]), pair[i]);
            }
        }
        cluster.sync();  // this pass's pairs are written, and nobody reads `total` any more
    }
}

// 16 CTAs where the device can place such a cluster, else 8 (every device can); asked once
// a device.
template <int ITEMS>
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
    e = cudaFuncSetAttribute(token_sort_kernel<ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sort_smem(kMaxBins)));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(token_sort_kernel<ITEMS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t probe = *cfg;
    probe.dynamicSmemBytes = sort_smem(kMaxBins);
    probe.gridDim = dim3(kMaxCluster);
    probe.attrs[0].val.clusterDim.x = kMaxCluster;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, token_sort_kernel<ITEMS>, &probe);
    if (e != cudaSuccess) return e;
    *most = known[dev] = n > 0 ? kMaxCluster : 8;
    return cudaSuccess;
}

template <int ITEMS>
cudaError_t launch(const SortArgs& args, int jobs, int64_t longest, int bins, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_smem(bins);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // one step of every warp a CTA, up to the largest cluster this device can place
    int most = 0;
    cudaError_t e = largest_cluster<ITEMS>(&cfg, &most);
    if (e != cudaSuccess) return e;
    int C = 1;
    while (C < most && int64_t(C) * kSortThreads < longest) C *= 2;
    cfg.gridDim = dim3(unsigned(C * jobs));
    attr[0].val.clusterDim.x = unsigned(C);
    e = cudaLaunchKernelEx(&cfg, token_sort_kernel<ITEMS>, args);
    note_launch();
    return e;
}

}  // namespace

size_t token_sort_bytes(int64_t N) { return size_t(N) * 8; }

cudaError_t token_sort_launch(const SortJob* jobs, int count, cudaStream_t stream) {
    SortArgs args{};
    int64_t longest = 0;
    int bins = 1;
    for (int i = 0; i < count; ++i) {
        // keys 0 .. V (V: no token); equal digits a pass
        int bits = 0;
        while ((int64_t(jobs[i].V) >> bits) != 0) ++bits;
        args.job[i] = jobs[i];
        args.passes[i] = (bits + kMaxDigitBits - 1) / kMaxDigitBits;
        args.digit_bits[i] = (bits + args.passes[i] - 1) / args.passes[i];
        longest = dmax(longest, jobs[i].N);
        bins = dmax(bins, 1 << args.digit_bits[i]);
    }
    // positions a lane at the largest cluster; longer lists are read twice a pass
    const int64_t lanes = int64_t(kMaxCluster) * kSortThreads;
    if (longest <= lanes) return launch<1>(args, count, longest, bins, stream);
    if (longest <= 4 * lanes) return launch<4>(args, count, longest, bins, stream);
    return launch<16>(args, count, longest, bins, stream);
}

}  // namespace df2
