// Token ids sorted for a gradient fold: (id, position) pairs in order of id, equal ids in
// order of position, so that every sum over a token's positions has one fixed order.
//
// A stable radix sort from the low digit up, by one thread-block cluster a list, every list
// of a call in one launch.  CTA c of a cluster owns the c-th contiguous range of positions,
// tile by tile; warp w owns the w-th part of a tile, so (CTA, tile, warp, step, lane) is the
// order of positions.  A pass over a digit of up to 9 bits:
//   1. every warp ranks its positions among those of equal digit.  A cell of shared memory
//      a (digit, warp) holds the step's lanes of that digit as a mask, and the count of the
//      steps before;
//   2. a digit's counts are scanned over the CTA's warps; the CTAs push their totals into
//      one another's shared memory, which gives each where its share of every digit starts;
//   3. the tile's pairs, kept in registers since step 1, are put in digit order in shared
//      memory and leave in runs of equal digit.
// A range of more than one tile is counted before, and ranked tile by tile.  The cluster
// barrier between passes also orders the passes' pairs, which go through L2.
//
// Bound: latency for short lists; for long ones the shared memory of the cluster's SMs.
// 151,936 tokens are 18 bits, two passes; 16 CTAs (the largest cluster) hold 262,144
// positions.  Finding a step's equals by a match instruction took 64 cycles of an SM a
// step, by nine votes 36: both queue in one unit; the masks go through shared memory.
#include <cooperative_groups.h>

#include <atomic>

#include "common.cuh"
#include "kernels.h"

namespace cg = cooperative_groups;

namespace df2 {
namespace {

constexpr int kSortThreads = 512;
constexpr int kSortWarps = kSortThreads / 32;
constexpr int kMaxCluster = 16;
constexpr int kMaxDigitBits = 9;
constexpr int kMaxBins = 1 << kMaxDigitBits;
static_assert(kMaxBins <= kSortThreads, "thread d owns digit d");
constexpr int kCellLd = kSortWarps + 1;  // odd: a digit's cells and a warp's both spread over the banks

// Words of shared memory: the cells [bins][kCellLd] (mask, count) and, once the ranks are in
// registers, the staged pairs in their place; then totals [clusters][bins], start [bins],
// local [bins], carry [kSortWarps].
template <int ITEMS>
__host__ __device__ constexpr int cell_words(int bins) {
    return bins * kCellLd > ITEMS * kSortThreads ? (bins * kCellLd * 2 + 3) / 4 * 4 : ITEMS * kSortThreads * 2;
}
template <int ITEMS>
size_t sort_smem(int bins) {
    return (size_t(cell_words<ITEMS>(bins)) + size_t(bins) * (kMaxCluster + 2) + kSortWarps) * 4;
}

struct SortArgs {
    SortJob job[kMaxJobs];
    int passes[kMaxJobs];
    int digit_bits[kMaxJobs];
};

// The exclusive sum of v over the CTA's threads.
__device__ __forceinline__ uint32_t block_exclusive(uint32_t v, uint32_t* carry, int lane, int warp) {
    uint32_t run = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t k = __shfl_up_sync(kFull, run, o);
        if (lane >= o) run += k;
    }
    if (lane == 31) carry[warp] = run;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int w = 0; w < kSortWarps; ++w) before += w < warp ? carry[w] : 0u;
    __syncthreads();
    return before + run - v;
}

// ITEMS: positions a lane holds, 512 ITEMS a tile.
template <int ITEMS>
__global__ void __launch_bounds__(kSortThreads) token_sort_kernel(const __grid_constant__ SortArgs args) {
    extern __shared__ uint32_t smem[];
    // let the next kernel start beside this one (one that was launched to allow it)
    asm volatile("griddepcontrol.launch_dependents;");
    cg::cluster_group cluster = cg::this_cluster();
    // (waited for before the first store into another CTA's shared memory: it must have begun)
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
    const int C = int(cluster.num_blocks()), c = int(cluster.block_rank());
    const bool second = int(blockIdx.x) >= C;  // (a parameter indexed by a register is slow to read)
    const SortJob job = second ? args.job[1] : args.job[0];
    const int passes = second ? args.passes[1] : args.passes[0];
    const int digit_bits = second ? args.digit_bits[1] : args.digit_bits[0];
    const int bins = 1 << digit_bits;
    uint2* cell = reinterpret_cast<uint2*>(smem);
    uint64_t* stage = reinterpret_cast<uint64_t*>(smem);
    uint32_t* totals = smem + cell_words<ITEMS>(bins);
    uint32_t* start = totals + C * bins;
    uint32_t* local = start + bins;
    uint32_t* carry = local + bins;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kTile = kSortThreads * ITEMS;

    const int64_t per_cta = (job.N + C - 1) / C;
    const int64_t lo = c * per_cta;
    const int64_t hi = dmin<int64_t>(job.N, lo + per_cta);
    const int tiles = int(dmax<int64_t>(1, (hi - lo + kTile - 1) / kTile));

    if (c == 0 && tid < 2) job.zero[tid] = 0;

    uint64_t pair[ITEMS];
    uint32_t rank[ITEMS];
    for (int pass = 0; pass < passes; ++pass) {
        const int shift = pass * digit_bits;
        // the last pass ends in job.pairs
        const uint64_t* src = ((passes - pass) & 1) ? job.spare : job.pairs;
        uint64_t* dst = ((passes - pass) & 1) ? job.pairs : job.spare;
        auto digit = [&](uint64_t x) { return (uint32_t(x) >> shift) & (bins - 1); };
        // a lane's positions of a tile: from + i * 32, those below hi
        auto first_of = [&](int tile) { return lo + int64_t(tile) * kTile + warp * (32 * ITEMS) + lane; };
        auto load = [&](int64_t from) {
            const int n = int(dmax<int64_t>(0, dmin<int64_t>(ITEMS, (hi - from + 31) / 32)));
            if (pass == 0) {
                bool bad = false;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) pair[i] = i < n ? uint32_t(__ldg(job.ids + from + i * 32)) : 0u;
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) {
                    uint32_t key = uint32_t(pair[i]);
                    if (key >= job.V) {
                        bad |= int32_t(key) >= 0;
                        key = job.V;
                    }
                    pair[i] = (uint64_t(uint32_t(from) + i * 32) << 32) | key;
                }
                if (bad && job.status) atomicOr(job.status, DF2_STATUS_ID_OUT_OF_RANGE);
            } else {
#pragma unroll
                for (int i = 0; i < ITEMS; ++i) pair[i] = i < n ? __ldcg(src + from + i * 32) : 0;
            }
            return n;
        };
        auto clear_cells = [&]() {
            for (int i = tid; i < bins * kCellLd; i += kSortThreads) cell[i] = make_uint2(0, 0);
            __syncthreads();
        };
        // each lane's rank among the warp's equal digits of the tile; then the digits' counts
        // become their sums over the warps before, and thread d gets digit d's total
        auto rank_tile = [&](int n) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                if (!__any_sync(kFull, i < n)) break;
                uint2* at = cell + digit(pair[i]) * kCellLd + warp;
                if (i < n) atomicOr(&at->x, 1u << lane);
                __syncwarp();
                const uint2 v = *at;
                const unsigned below = v.x & ((1u << lane) - 1);
                rank[i] = v.y + __popc(below);
                __syncwarp();
                if (i < n && below == 0) *at = make_uint2(0, v.y + __popc(v.x));
                __syncwarp();
            }
            __syncthreads();
            uint32_t sum = 0;
            if (tid < bins) {
#pragma unroll
                for (int w = 0; w < kSortWarps; ++w) {
                    const uint32_t k = cell[tid * kCellLd + w].y;
                    cell[tid * kCellLd + w].y = sum;
                    sum += k;
                }
            }
            return sum;
        };

        clear_cells();
        int n = 0;
        uint32_t own = 0;
        if (tiles == 1) {
            n = load(first_of(0));
            own = rank_tile(n);
        } else {
            for (int k = 0; k < tiles; ++k) {
                n = load(first_of(k));
#pragma unroll
                for (int i = 0; i < ITEMS; ++i)
                    if (i < n) atomicAdd(&cell[digit(pair[i]) * kCellLd].y, 1u);
            }
            __syncthreads();
            own = tid < bins ? cell[tid * kCellLd].y : 0u;
        }
        if (pass == 0) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
        if (tid < bins)
            for (int o = 0; o < C; ++o) cluster.map_shared_rank(totals, o)[c * bins + tid] = own;
        cluster.sync();
        uint32_t all = 0, before = 0;
        if (tid < bins) {
            for (int o = 0; o < C; ++o) {
                const uint32_t k = totals[o * bins + tid];
                before += o < c ? k : 0u;
                all += k;
            }
        }
        const uint32_t first = block_exclusive(all, carry, lane, warp) + before;
        if (tid < bins) start[tid] = first;
        for (int k = 0; k < tiles; ++k) {
            if (tiles > 1) {
                __syncthreads();
                clear_cells();
                n = load(first_of(k));
                own = rank_tile(n);
            }
            const uint32_t at = block_exclusive(own, carry, lane, warp);
            // a pair's place in the tile, and what leads from there to its place in the list
            uint32_t next = 0;
            if (tid < bins) {
                local[tid] = at;
                next = start[tid] + own;
                start[tid] -= at;
            }
            __syncthreads();
#pragma unroll
            for (int i = 0; i < ITEMS; ++i) {
                const uint32_t d = digit(pair[i]);
                rank[i] += cell[d * kCellLd + warp].y + local[d];
            }
            __syncthreads();  // the cells give way
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (i < n) stage[rank[i]] = pair[i];
            __syncthreads();
            const int held = int(dmin<int64_t>(kTile, hi - lo - int64_t(k) * kTile));
#pragma unroll 8
            for (int i = tid; i < held; i += kSortThreads) {
                const uint64_t x = stage[i];
                __stcg(dst + (start[digit(x)] + uint32_t(i)), x);
            }
            if (tiles > 1) {
                __syncthreads();
                if (tid < bins) start[tid] = next;
            }
        }
        cluster.sync();  // this pass's pairs are written, and the totals have been read
    }
}

constexpr int kMaxDevices = 64;  // whose answers are kept

// 16 CTAs where the device can place such a cluster, else 8 (every device can); asked once
// a device.  (Threads that ask at the same time set and store the same.)
template <int ITEMS>
cudaError_t largest_cluster(cudaLaunchConfig_t* cfg, int* most) {
    static std::atomic<int> known[kMaxDevices];  // 0: not asked yet
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < kMaxDevices && (*most = known[dev].load(std::memory_order_acquire)) != 0) return cudaSuccess;
    e = cudaFuncSetAttribute(token_sort_kernel<ITEMS>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             int(sort_smem<ITEMS>(kMaxBins)));
    if (e == cudaSuccess)
        e = cudaFuncSetAttribute(token_sort_kernel<ITEMS>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t probe = *cfg;
    probe.dynamicSmemBytes = sort_smem<ITEMS>(kMaxBins);
    probe.gridDim = dim3(kMaxCluster);
    probe.attrs[0].val.clusterDim.x = kMaxCluster;
    int n = 0;
    e = cudaOccupancyMaxActiveClusters(&n, token_sort_kernel<ITEMS>, &probe);
    if (e != cudaSuccess) return e;
    *most = n > 0 ? kMaxCluster : 8;
    if (dev < kMaxDevices) known[dev].store(*most, std::memory_order_release);
    return cudaSuccess;
}

template <int ITEMS>
cudaError_t launch(const SortArgs& args, int jobs, int64_t longest, int bins, cudaStream_t stream) {
    cudaLaunchConfig_t cfg{};
    cfg.blockDim = dim3(kSortThreads);
    cfg.dynamicSmemBytes = sort_smem<ITEMS>(bins);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    // one tile a CTA, up to the largest cluster this device can place
    int most = 0;
    cudaError_t e = largest_cluster<ITEMS>(&cfg, &most);
    if (e != cudaSuccess) return e;
    int C = 1;
    while (C < most && int64_t(C) * kSortThreads * ITEMS < longest) C *= 2;
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
    // the fewest positions a lane that the largest cluster covers in one tile
    const int64_t lanes = int64_t(kMaxCluster) * kSortThreads;
    if (longest <= 2 * lanes) return launch<2>(args, count, longest, bins, stream);
    if (longest <= 8 * lanes) return launch<8>(args, count, longest, bins, stream);
    return launch<32>(args, count, longest, bins, stream);
}

}  // namespace df2
