// The row-wise steps of the unary loss around its matrix products (loss_gemm.cu).
//
// With x the mapped logits of a row, t its target and M its largest logit, the loss is kept
// free of cancellation by summing the others apart from the target:
//   s = sum over v != t of exp(x_v - M),   loss = (M - x_t) + log1p(s + (exp(x_t - M) - 1))
//   dloss/dx_t = -s / (s + exp(x_t - M)),  dloss/dx_v = exp(x_v - M) / (s + exp(x_t - M))
// so a row that is all but certain keeps its small loss and gradient to fp32's precision.
//
//   live_rows_kernel   the rows that have a target, in order, copied next to each other: the
//                      products neither compute the others nor meet a NaN in them.  Bound by
//                      the copy (4096 rows of 4096: 18 us; 16,384: 46 us, 5.8 TB/s), or for few rows by
//                      two dependent loads (4 us)
//   row_loss_kernel    a row's loss from its tiles' statistics, and its e to g in place.  Bound
//                      by HBM: 4096 rows of 151,936 in 390 us, 6.4 TB/s with four loads a thread in flight
//                      (415 with one)
//   sum_parts_kernel   the rows of dh whose sums were cut, from their parts in order (13 us for
//                      20 tiles in 9 to 13 parts)
#include <cuda_fp16.h>

#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ void unpack8_f16(const uint4& w, float f[8]) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(u + k));
        f[2 * k] = v.x;
        f[2 * k + 1] = v.y;
    }
}

template <class T, class Op>
__device__ __forceinline__ T block_reduce(T v, T* shared, Op op) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = op(v, __shfl_xor_sync(kFull, v, o));
    __syncthreads();  // shared may still be read from the last time
    if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
    __syncthreads();
    v = shared[0];
#pragma unroll
    for (int k = 1; k < kThreads / 32; ++k) v = op(v, shared[k]);
    return v;
}

// A block looks after `each` rows; it counts the live ones before them by itself, so the
// rows are put in order in one launch.
__global__ void __launch_bounds__(kThreads)
live_rows_kernel(const LossRowsArgs a, const int each) {
    __shared__ int shared[kThreads / 32];
    __shared__ int place[kThreads];  // of the block's rows: its place among the live, -1: none
    __shared__ int so_far;
    asm volatile("griddepcontrol.launch_dependents;");
    const int64_t first = int64_t(blockIdx.x) * each, last = dmin<int64_t>(first + each, a.P);
    auto alive = [&](int64_t p) { const int t = a.targets[p]; return t >= 0 && t < a.V; };
    int before = 0;
    for (int64_t p = threadIdx.x; p < first; p += kThreads) before += alive(p);
    before = block_reduce(before, shared, [](int x, int y) { return x + y; });
    if (threadIdx.x < 32) {
        for (int64_t p0 = first; p0 < last; p0 += 32) {
            const int64_t p = p0 + threadIdx.x;
            const bool in = p < last, is = in && alive(p);
            const unsigned live = __ballot_sync(kFull, is);
            const int at = before + __popc(live & ((1u << threadIdx.x) - 1));
            if (in) place[p - first] = is ? at : -1;
            if (is) {
                a.map[at] = int(p);
                a.live_targets[at] = a.targets[p];
            } else if (in) {
                a.loss[p] = __int_as_float(0x7fc00000);
                if (a.lse) a.lse[p] = __int_as_float(0x7fc00000);
                if (a.status && a.targets[p] >= 0) atomicOr(a.status, DF2_STATUS_ID_OUT_OF_RANGE);
            }
            before += __popc(live);
        }
        if (threadIdx.x == 0) {
            so_far = before;
            if (last == a.P) *a.count = before;
        }
    }
    __syncthreads();
    // 16 bytes of bf16 a unit; the block's rows are one run of units
    const int units = int(a.D / 8), rows = int(last - first);
    for (int u = threadIdx.x; u < rows * units; u += kThreads) {
        const int r = u / units, at = place[r];
        if (at >= 0)
            reinterpret_cast<uint4*>(a.live_h + int64_t(at) * a.D)[u - r * units] =
                __ldcs(reinterpret_cast<const uint4*>(a.h + first * a.D) + u);
    }
    const int dh_units = a.dh ? units * (a.dh_bf16 ? 1 : 2) : 0;
    for (int u = threadIdx.x; u < rows * dh_units; u += kThreads)
        if (place[u / dh_units] < 0)
            reinterpret_cast<uint4*>(static_cast<char*>(a.dh) + first * dh_units * 16)[u] = make_uint4(0u, 0u, 0u, 0u);
    if (last == a.P) {  // rows of the last K step of dW's product
        const int64_t total = so_far, end = (total + 63) / 64 * 64;
        uint4* to = reinterpret_cast<uint4*>(a.live_h + total * a.D);
        for (int64_t u = threadIdx.x; u < (end - total) * units; u += kThreads) to[u] = make_uint4(0u, 0u, 0u, 0u);
    }
}

// grid (rows of the piece, column shares).  G: e becomes the gradient of the logits.
template <bool G>
__global__ void __launch_bounds__(kThreads) row_loss_kernel(const LossRowArgs a) {
    __shared__ float shared[kThreads / 32];
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t left = int64_t(*a.count) - a.row0;
    const int64_t live = left < 0 ? 0 : left > a.rows ? a.rows : left;
    const int64_t row = blockIdx.x;
    const int64_t share = (a.V + 2047) / 2048, c0 = 2048 * (share * blockIdx.y / gridDim.y);
    const int64_t c1 = dmin<int64_t>(2048 * (share * (blockIdx.y + 1) / gridDim.y), a.V);
    if (row >= live) {
        if (G && row < (live + 63) / 64 * 64) {  // rows of the last K step of dW's product
            uint16_t* e = a.e + row * a.e_ld;
            for (int64_t c = c0 + threadIdx.x * 8; c < c1; c += kThreads * 8)
                *reinterpret_cast<uint4*>(e + c) = make_uint4(0u, 0u, 0u, 0u);
        }
        return;
    }
    const float2* stats = a.stats + row * a.n_stats;
    const float xt = a.target_logit[a.row0 + row];
    float top = xt;
    for (int i = threadIdx.x; i < a.n_stats; i += kThreads) top = fmaxf(top, stats[i].x);
    top = block_reduce(top, shared, [](float x, float y) { return fmaxf(x, y); });
    float sum = 0.f;
    for (int i = threadIdx.x; i < a.n_stats; i += kThreads) {
        const float2 s = stats[i];
        if (s.y != 0.f) sum += s.y * exp2f((s.x - top) * kLog2e);  // no column: 0 at -inf
    }
    sum = block_reduce(sum, shared, [](float x, float y) { return x + y; });
    const int64_t p = a.map[a.row0 + row];
    const float all = sum + expf(xt - top);
    if (threadIdx.x == 0 && blockIdx.y == 0) {
        a.loss[p] = (top - xt) + log1pf(sum + expm1f(xt - top));
        if (a.lse) a.lse[p] = top + logf(all);
    }
    if (!G) return;
    const float w = (a.weights ? a.weights[p] : 1.f) * a.lm.mul / all;
    const float w_e = w / kExpScale;
    const float gt = -sum * w * (a.lm.cap > 0.f ? a.target_slope[a.row0 + row] : 1.f);
    const int64_t t = a.live_targets[a.row0 + row];
    uint16_t* e = a.e + row * a.e_ld;
    constexpr int kAhead = 4;  // units of a thread that are loaded together
    for (int64_t c = c0 + threadIdx.x * 8; c < c1; c += kAhead * kThreads * 8) {
        uint4 in[kAhead];
        float m[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = c + k * kThreads * 8;
            if (at < c1) {
                in[k] = __ldcs(reinterpret_cast<const uint4*>(e + at));
                m[k] = stats[at / kLossStats].x;  // written while this kernel may have begun: no read-only load
            }
        }
#pragma unroll
        for (int k = 0; k < kAhead; ++k) {
            const int64_t at = c + k * kThreads * 8;
            if (at >= c1) break;
            float f[8];
            unpack8_f16(in[k], f);
            const float by = m[k] == -INFINITY ? w_e : w_e * exp2f((m[k] - top) * kLog2e);
            const int64_t hit = t - at;
#pragma unroll
            for (int j = 0; j < 8; ++j) f[j] = j == hit ? gt : f[j] * by;
            *reinterpret_cast<uint4*>(e + at) =
                make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        }
    }
}

// grid (tiles that can be cut, pairs' tiles of each, 8 rows of a tile): the sums of a tile's parts,
// in order.
template <bool QUAD>
__global__ void __launch_bounds__(kThreads)
sum_parts_kernel(const int32_t* count, int64_t row0, int rows, const int32_t* map, const float* part, int64_t V,
                 int64_t D, LossDhGrid grid, void* dh, bool bf16) {
    __shared__ LossSplit shared;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t left = int64_t(*count) - row0;
    const int live = int(left < 0 ? 0 : left > rows ? rows : left);
    const int n_mu = (live + 255) / 256, steps = int((V + 63) / 64);
    if (threadIdx.x < 32) {
        const LossSplit work = loss_split(loss_cluster_tiles(n_mu, grid.n_nt, QUAD), steps, grid.units, QUAD, threadIdx.x);
        if (threadIdx.x == 0) shared = work;
    }
    __syncthreads();
    const LossSplit work = shared;
    const int tile = blockIdx.x, which = blockIdx.y;
    if (work.ways == 1 || tile >= work.rest) return;  // the product wrote dh itself
    const LossTile t = loss_tile<false, QUAD>(work.whole + tile, n_mu, grid.n_nt, work, steps, which);
    constexpr int kPairs = QUAD ? 2 : 1;
    const int64_t d = int64_t(t.nt) * 256 + (threadIdx.x & 31) * 8;
    if (d >= D) return;
    const int r = blockIdx.z * 8 + threadIdx.x / 32, m = t.mu * 256 + r;
    if (m >= live) return;
    float f[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const float* from = part + ((int64_t(tile) * kPairs + which) * 256 + r) * 256 + (threadIdx.x & 31) * 8;
#pragma unroll 4
    for (int k = 0; k < work.ways; ++k, from += int64_t(work.rest) * kPairs * 65536) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(from)), w = __ldcs(reinterpret_cast<const float4*>(from) + 1);
        f[0] += v.x;
        f[1] += v.y;
        f[2] += v.z;
        f[3] += v.w;
        f[4] += w.x;
        f[5] += w.y;
        f[6] += w.z;
        f[7] += w.w;
    }
    const int64_t o = int64_t(map[row0 + m]) * D + d;
    if (bf16) {
        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(dh) + o) =
            make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else {
        float4* to = reinterpret_cast<float4*>(static_cast<float*>(dh) + o);
        to[0] = make_float4(f[0], f[1], f[2], f[3]);
        to[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// A launch whose start may overlap the end of the kernel before it in the stream: every thread
// of these kernels waits for that one to be done before it reads or writes anything, so each is
// also done with what came before.
template <class... Params, class... Given>
cudaError_t launch_after(void (*kernel)(Params...), dim3 grid, cudaStream_t stream, Given... given) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    note_launch();
    return cudaLaunchKernelEx(&cfg, kernel, Params(given)...);
}

}  // namespace

cudaError_t loss_rows_launch(const LossRowsArgs& a, cudaStream_t stream) {
    // a row a block, or more of them where they are short or the blocks' own counting would be
    // the longer part
    int64_t each = (a.P + 4095) / 4096, full = 4096 / a.D;
    if (full > 32) full = 32;
    if (each < full) each = full;
    if (each > kThreads) each = kThreads;
    const int64_t grid = (a.P + each - 1) / each;
    live_rows_kernel<<<unsigned(grid), kThreads, 0, stream>>>(a, int(each));
    note_launch();
    return cudaGetLastError();
}

cudaError_t loss_row_launch(const LossRowArgs& a, int64_t e_rows, int num_sms, cudaStream_t stream) {
    if (!a.e) {
        return launch_after(row_loss_kernel<false>, dim3(unsigned(a.rows)), stream, a);
    } else {
        // columns shared out where the rows alone leave SMs idle
        const int64_t rows = (a.rows + 63) / 64 * 64 < e_rows ? (a.rows + 63) / 64 * 64 : e_rows;
        int64_t shares = (8 * num_sms + a.rows - 1) / a.rows;
        const int64_t most = (a.V + 2047) / 2048;
        shares = shares > most ? most : shares;
        return launch_after(row_loss_kernel<true>, dim3(unsigned(rows), unsigned(shares)), stream, a);
    }
}

cudaError_t loss_sum_parts_launch(const LossGemmArgs& a, const LossDhGrid& grid, cudaStream_t stream) {
    // at most as many tiles are left over as there are clusters, less one, or tiles at all
    const int tiles = loss_cluster_tiles(int((a.rows + 255) / 256), grid.n_nt, grid.quad);
    const dim3 blocks(unsigned(tiles < grid.units ? tiles : grid.units), grid.quad ? 2 : 1, 32);
    const float* part = a.part;
    return grid.quad ? launch_after(sum_parts_kernel<true>, blocks, stream, a.count, a.row0, a.rows, a.map, part, a.V, a.D,
                                    grid, a.out, a.out_bf16)
                     : launch_after(sum_parts_kernel<false>, blocks, stream, a.count, a.row0, a.rows, a.map, part, a.V, a.D,
                                    grid, a.out, a.out_bf16);
}

}  // namespace df2
