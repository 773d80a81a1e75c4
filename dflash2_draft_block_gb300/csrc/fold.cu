// The gradient of a table gathered by token id: out[v, :] (+)= scale * the sum over the
// positions n of token v, in order of n, of w[n] * src[n / per_row, :].
//
// The positions are sorted by token (token_sort.cu).  The sorted list is cut into chunks of
// E positions and D into slices of 8 L columns; a group of L lanes owns a (chunk, slice): a
// lane holds 8 columns' sums in fp32, loads kAhead rows before it adds the first, and
// writes a token's row when the list moves on to the next.  A token that runs over a
// chunk's end is finished by the group it began in when less than E / 2 positions are left
// of it; a longer one (a mask token can hold most of a batch) is split there, every chunk
// leaves its part in fp32, and fold_join_kernel adds the parts, one CTA a (token, slice).
// Where the cuts fall depends on the sorted list alone, so results repeat bit for bit.
//
// Without accumulate the rows of absent tokens become zeros: further CTAs of the same launch
// each take a range of rows, mark those that the sorted list holds, and clear the others,
// so every row is written once, and the writes run beside the gathers.
//
// Lists of up to kSmall positions are not sorted at all: every position looks for its equals
// in the list itself, the first of them owns the token (fold_small_kernel).
//
// Bound: HBM for the rows written (all of a large table's), L2 for the gathers.
#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kAhead = 8;
constexpr int kJoinWarps = 4;
constexpr int kSmall = 512;
constexpr int kFillRows = 4096;       // rows a fill CTA takes at most
constexpr int64_t kFillBytes = 512 * 1024;  // and the bytes, while the CTAs fill the SMs eight times

struct Plan {
    FoldArgs a[kMaxJobs];
    int count;
    int E[kMaxJobs];
    int64_t chunks[kMaxJobs];
    int slices[kMaxJobs];
    int fold_blocks[kMaxJobs];
    int fill_blocks[kMaxJobs];
    int fill_rows[kMaxJobs];
    int fill_unit[kMaxJobs];  // bytes a store
};

__device__ __forceinline__ uint32_t key_at(const uint64_t* pairs, int64_t i) {
    return uint32_t(__ldg(pairs + i));
}

// Whether the token that ends chunk [.., b) goes on for at least half positions from b.
__device__ __forceinline__ bool split_at(const uint64_t* pairs, int64_t N, int64_t b, int half) {
    return b + half <= N && key_at(pairs, b - 1) == key_at(pairs, b + half - 1);
}

template <int L>
__device__ __forceinline__ unsigned group_mask(int lane) {
    return L == 32 ? kFull : ((1u << L) - 1) << (lane & ~(L - 1));
}

// The first i >= b whose key differs from the key before b; known to lie before b + half.
template <int L>
__device__ __forceinline__ int64_t run_end(const uint64_t* pairs, int64_t N, int64_t b, int half, int lane) {
    const uint32_t k = key_at(pairs, b - 1);
    for (int o = 0; o < half; o += L) {
        const int64_t i = b + o + (lane & (L - 1));
        const unsigned other = __ballot_sync(group_mask<L>(lane), i >= N || key_at(pairs, i) != k);
        if (other) return b + o + (__ffs(other) - 1 - (lane & ~(L - 1)));
    }
    return dmin<int64_t>(N, b + half);
}

// The first position whose key is at least v, by a whole warp: 32 probes a step.
__device__ __forceinline__ int64_t lower_bound(const uint64_t* pairs, int64_t N, uint32_t v, int lane) {
    int64_t lo = 0, hi = N;
    while (hi - lo > 32) {
        const int64_t step = (hi - lo + 31) / 32, i = lo + lane * step;
        const int c = __popc(__ballot_sync(kFull, i < hi && key_at(pairs, i) < v));
        if (c == 0) return lo;
        hi = dmin<int64_t>(hi, lo + c * step);
        lo += (c - 1) * step + 1;
    }
    return lo + __popc(__ballot_sync(kFull, lo + lane < hi && key_at(pairs, lo + lane) < v));
}

// A lane's 8 columns: consecutive with vectors, else L apart.
template <int W, int L>
__device__ __forceinline__ int64_t column(int64_t slice, int gl, int i) {
    return slice * (8 * L) + (W == 8 ? gl * 8 + i : i * L + gl);
}

template <bool SRC16, int W, int L>
struct Row {
    uint4 a, b;  // as loaded: bf16 in a; fp32 in a, b (vectors), or one element a word

    // p: the row's element at the lane's first column; left: columns from there on
    __device__ __forceinline__ void load(const char* p, int64_t left) {
        constexpr int SZ = SRC16 ? 2 : 4;
        if (W == 8) {
            if (left <= 0) return;
            a = __ldg(reinterpret_cast<const uint4*>(p));
            if (!SRC16) b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
        } else {
            uint32_t w[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                w[i] = 0;
                if (i * L < left)
                    w[i] = SRC16 ? uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p + i * L * SZ))) << 16
                                 : __ldg(reinterpret_cast<const uint32_t*>(p + i * L * SZ));
            }
            a = make_uint4(w[0], w[1], w[2], w[3]);
            b = make_uint4(w[4], w[5], w[6], w[7]);
        }
    }
    __device__ __forceinline__ void get(float f[8]) const {
        if (SRC16 && W == 8) {
            unpack8(a, f);
        } else {
            f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
            f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
            f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
            f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
        }
    }
};

// out[row, lane's columns] = scale * f (+ itself).  Added in fp32 by the memory's own add:
// a row has one writer, so the result is the one rounded sum, and nobody waits for the old
// row (the add flushes subnormal operands).
template <bool OUT16, int W, int L>
__device__ __forceinline__ void put_row(const FoldArgs& a, int64_t row, int64_t slice, int gl, const float f[8]) {
    constexpr int SZ = OUT16 ? 2 : 4;
    char* p = static_cast<char*>(a.out) + (row * a.out_ld + column<W, L>(slice, gl, 0)) * SZ;
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(f[i], a.scale);
    if (W == 8) {
        if (column<W, L>(slice, gl, 0) >= a.D) return;
        if (OUT16) {
            uint4* q = reinterpret_cast<uint4*>(p);
            if (a.accumulate) {
                float o[8];
                unpack8(*q, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = __fadd_rn(o[i], g[i]);
            }
            *q = make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]), pack_bf16(g[6], g[7]));
        } else {
            float4* q = reinterpret_cast<float4*>(p);
            const float4 x = make_float4(g[0], g[1], g[2], g[3]), y = make_float4(g[4], g[5], g[6], g[7]);
            if (a.accumulate) {
                atomicAdd(q, x);
                atomicAdd(q + 1, y);
            } else {
                q[0] = x;
                q[1] = y;
            }
        }
    } else if (OUT16) {
        uint16_t* q = reinterpret_cast<uint16_t*>(p);
        if (a.accumulate) {
            uint16_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = column<W, L>(slice, gl, i) < a.D ? q[i * L] : uint16_t(0);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = __fadd_rn(bf16_to_f32(o[i]), g[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (column<W, L>(slice, gl, i) < a.D) q[i * L] = f32_to_bf16_rn(g[i]);
    } else {
        float* q = reinterpret_cast<float*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (column<W, L>(slice, gl, i) >= a.D) continue;
            if (a.accumulate) atomicAdd(q + i * L, g[i]);
            else q[i * L] = g[i];
        }
    }
}

// (a weight of one adds f as it is)
__device__ __forceinline__ void add_row(float acc[8], const float f[8], float w) {
#pragma unroll
    for (int q = 0; q < 8; ++q) acc[q] = fmaf(w, f[q], acc[q]);
}

// Whether position n has a part, and its weight.
__device__ __forceinline__ bool counts(const FoldArgs& a, uint32_t n, float* w) {
    *w = a.w ? __ldg(a.w + n) : 1.f;
    return *w != 0.f && (!a.label || __ldg(a.label + n / a.per_row) >= 0);
}

// A lane's 8 sums in the parts buffer: part s of chunk c, slice.
template <int L>
__device__ __forceinline__ float4* part_at(const FoldArgs& a, int64_t slices, int64_t c, int s, int64_t slice, int gl) {
    return reinterpret_cast<float4*>(a.parts + ((c * 2 + s) * slices + slice) * (8 * L) + gl * 8);
}

// Zeros to the rows [block * fill_rows, ..) of absent tokens.
template <bool SMALL>
__device__ void fill(const Plan& p, int job, int64_t block) {
    __shared__ uint32_t held[kFillRows / 32];
    __shared__ int64_t range[2];
    const FoldArgs& a = p.a[job];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t v0 = block * p.fill_rows[job];
    const int rows = int(dmin<int64_t>(p.fill_rows[job], a.V - v0));
    for (int i = tid; i < (rows + 31) / 32; i += kThreads) held[i] = 0;
    auto mark = [&](uint32_t r) {
        if (!(held[r >> 5] >> (r & 31) & 1)) atomicOr(&held[r >> 5], 1u << (r & 31));
    };
    if (SMALL) {
        __syncthreads();
        for (int64_t n = tid; n < a.N; n += kThreads) {
            const int64_t r = int64_t(__ldg(a.ids + n)) - v0;
            if (r >= 0 && r < rows) mark(uint32_t(r));
        }
    } else {
        if (warp < 2) {
            const int64_t at = lower_bound(a.pairs, a.N, uint32_t(v0 + (warp ? rows : 0)), lane);
            if (lane == 0) range[warp] = at;
        }
        __syncthreads();
        const int64_t lo = range[0], hi = range[1];
        if (hi - lo <= int64_t(rows) * 16 + 1024) {
            for (int64_t i = lo + tid; i < hi; i += kThreads) mark(key_at(a.pairs, i) - uint32_t(v0));
        } else {  // a token of very many positions: each row is looked up instead
            for (int r = tid; r < rows; r += kThreads) {
                int64_t x = lo, y = hi;
                while (x < y) {
                    const int64_t mid = (x + y) >> 1;
                    if (key_at(a.pairs, mid) < uint32_t(v0 + r)) x = mid + 1;
                    else y = mid;
                }
                if (x < hi && key_at(a.pairs, x) == uint32_t(v0 + r)) mark(uint32_t(r));
            }
        }
    }
    __syncthreads();
    const int sz = a.out_bf16 ? 2 : 4, unit = p.fill_unit[job];
    const int64_t ld = a.out_ld * sz, per = a.D * sz / unit;
    char* out = static_cast<char*>(a.out) + v0 * ld;
    // lanes across a row; several rows a warp where a row has few units
    int across = 32;
    while (across > 1 && across / 2 >= per) across /= 2;
    const int sub = lane & (across - 1), stride = kThreads / across;
    for (int r = tid / across; r < rows; r += stride) {
        if (held[r >> 5] >> (r & 31) & 1) continue;
        char* q = out + r * ld;
        if (unit == 16)
            for (int64_t i = sub; i < per; i += across) reinterpret_cast<uint4*>(q)[i] = make_uint4(0, 0, 0, 0);
        else if (unit == 4)
            for (int64_t i = sub; i < per; i += across) reinterpret_cast<uint32_t*>(q)[i] = 0;
        else
            for (int64_t i = sub; i < per; i += across) reinterpret_cast<uint16_t*>(q)[i] = 0;
    }
}

// A block's part in a launch of all jobs' folds and fills, the two kinds spread evenly: the
// job and the block's number there; fill: which kind.
__device__ __forceinline__ int64_t part_of(const Plan& p, int* job, bool* fill) {
    int64_t folds = 0, fills = 0;
    for (int j = 0; j < p.count; ++j) {
        folds += p.fold_blocks[j];
        fills += p.fill_blocks[j];
    }
    const int64_t b = blockIdx.x, before = b * fills / (folds + fills);
    *fill = (b + 1) * fills / (folds + fills) > before;
    int64_t n = *fill ? before : b - before;
    const int* blocks = *fill ? p.fill_blocks : p.fold_blocks;
    *job = 0;
    if (p.count > 1 && n >= blocks[0]) {
        n -= blocks[0];
        *job = 1;
    }
    return n;
}

template <bool SRC16, bool OUT16, int W, int L>
__global__ void __launch_bounds__(kThreads) fold_kernel(const __grid_constant__ Plan p) {
    // the join may take its place now: it waits for this kernel where it reads parts
    asm volatile("griddepcontrol.launch_dependents;");
    int job;
    bool is_fill;
    const int64_t block = part_of(p, &job, &is_fill);
    if (is_fill) {
        fill<false>(p, job, block);
        return;
    }
    const FoldArgs& a = p.a[job];
    const int lane = threadIdx.x & 31, gl = lane & (L - 1);
    const unsigned gmask = group_mask<L>(lane);
    const int64_t unit = (block * kThreads + threadIdx.x) / L;
    const int slices = p.slices[job], E = p.E[job], half = E / 2;
    const int64_t c = unit / slices, slice = unit - c * slices;
    if (c >= p.chunks[job]) return;
    const uint64_t* pairs = a.pairs;
    const int64_t e0 = c * E, e1 = dmin<int64_t>(e0 + E, a.N);
    int64_t i = e0, end = e1;
    bool head = false, tail = false;
    if (c > 0 && key_at(pairs, e0 - 1) == key_at(pairs, e0)) {
        head = split_at(pairs, a.N, e0, half);
        if (!head) i = run_end<L>(pairs, a.N, e0, half, lane);
    }
    if (i >= e1) return;  // a short last chunk the one before it finishes
    if (e1 < a.N && key_at(pairs, e1 - 1) == key_at(pairs, e1)) {
        tail = split_at(pairs, a.N, e1, half);
        if (!tail) end = run_end<L>(pairs, a.N, e1, half, lane);
    }

    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const uint32_t none = uint32_t(a.V);
    uint32_t cur = key_at(pairs, i);
    if (cur == none) return;
    auto leave = [&](bool is_tail) {  // the current token's sums, to its row or to its part
        if (head || is_tail) {
            float4* q = part_at<L>(a, slices, c, head ? 0 : 1, slice, gl);
            q[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            q[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        } else {
            put_row<OUT16, W, L>(a, cur, slice, gl, acc);
        }
        head = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    };
    const int64_t left = a.D - column<W, L>(slice, gl, 0);
    const char* src = static_cast<const char*>(a.src) + column<W, L>(slice, gl, 0) * (SRC16 ? 2 : 4);
    const uint64_t stride = uint64_t(a.src_ld) * (SRC16 ? 2 : 4);
    for (bool more = true; more && i < end; i += L) {
        const int n = int(dmin<int64_t>(L, end - i));
        const uint64_t pair = gl < n ? __ldg(pairs + i + gl) : uint64_t(none);
        const uint32_t key = uint32_t(pair);
        float w = 0.f;
        const bool on = key != none && counts(a, uint32_t(pair >> 32), &w);
        const uint32_t row = uint32_t(pair >> 32) / a.per_row;
        // bit k: position k has a part; a token begins at k (`none` ends the list)
        const uint32_t before = __shfl_up_sync(gmask, key, 1, L);
        unsigned live = __ballot_sync(gmask, on) >> (lane & ~(L - 1));
        unsigned begins = __ballot_sync(gmask, gl < n && key != (gl ? before : cur)) >> (lane & ~(L - 1));
        more = __shfl_sync(gmask, key, n - 1, L) != none;
        for (int j = 0; j < n; j += kAhead, live >>= kAhead, begins >>= kAhead) {
            Row<SRC16, W, L> r[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t rr = __shfl_sync(gmask, row, j + k, L);
                if (live >> k & 1) r[k].load(src + rr * stride, left);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float ww = __shfl_sync(gmask, w, j + k, L);
                if (begins >> k & 1) {
                    if (cur != none) leave(false);
                    cur = __shfl_sync(gmask, key, j + k, L);
                }
                if (live >> k & 1) {
                    float f[8];
                    r[k].get(f);
                    add_row(acc, f, ww);
                }
            }
        }
    }
    if (cur != none) leave(tail);
}

template <bool OUT16, int W, int L>
__global__ void __launch_bounds__(kJoinWarps * 32) fold_join_kernel(const __grid_constant__ Plan p) {
    __shared__ float4 sums[kJoinWarps * 32 / L][2][L];
    // Who owns a split token shows in the sorted list, which was complete before the fold
    // began; only the parts have to be waited for.  Block 0 always waits, so that this
    // kernel does not end before the fold.
    const int64_t units0 = p.chunks[0] * p.slices[0];
    const int job = blockIdx.x >= units0;
    const int64_t unit = blockIdx.x - (job ? units0 : 0);
    const FoldArgs& a = p.a[job];
    const int slices = p.slices[job], E = p.E[job], half = E / 2;
    const int64_t c = unit / slices, slice = unit - c * slices;
    const int64_t e0 = c * E, e1 = e0 + E;
    uint32_t k = 0;
    bool owner = e1 < a.N;
    if (owner) {
        k = key_at(a.pairs, e1 - 1);
        // the chunk the token begins in owns the sum
        owner = k != uint32_t(a.V) && split_at(a.pairs, a.N, e1, half) &&
                !(c > 0 && key_at(a.pairs, e0 - 1) == k);
    }
    if (owner || blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!owner) return;
    constexpr int kGroups = kJoinWarps * 32 / L;
    const int gl = threadIdx.x & (L - 1), group = threadIdx.x / L;
    int more = 0;  // the chunks after c that left a part
    for (int got = kJoinWarps * 32; got == kJoinWarps * 32;) {
        const int64_t b = (c + 1 + more + threadIdx.x) * E;
        got = __syncthreads_count(b < a.N && key_at(a.pairs, b - 1) == k && split_at(a.pairs, a.N, b, half));
        more += got;
    }
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
    for (int m = group; m <= more; m += kGroups) {
        const float4* q = part_at<L>(a, slices, c + m, m == 0 ? 1 : 0, slice, gl);
        const float4 x = __ldcg(q), y = __ldcg(q + 1);
        acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
        acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
    }
    sums[group][0][gl] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    sums[group][1][gl] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    __syncthreads();
    if (group) return;
    for (int g = 1; g < dmin(kGroups, more + 1); ++g) {
        const float4 x = sums[g][0][gl], y = sums[g][1][gl];
        acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
        acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
    }
    put_row<OUT16, W, L>(a, k, slice, gl, acc);
}

// A block a (position, slice).  The block of a token's first position sums the token: the
// list is cut in four, a warp each, and the warps' sums are added in order.
template <bool SRC16, bool OUT16, int W>
__global__ void __launch_bounds__(kThreads) fold_small_kernel(const __grid_constant__ Plan p) {
    __shared__ float4 sums[kWarps][2][32];
    int job;
    bool is_fill;
    const int64_t block = part_of(p, &job, &is_fill);
    if (is_fill) {
        fill<true>(p, job, block);
        return;
    }
    const FoldArgs& a = p.a[job];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int n = int(block / p.slices[job]);
    const int64_t slice = block - int64_t(n) * p.slices[job];
    const int32_t id = __ldg(a.ids + n);
    if (id < 0) return;
    if (id >= a.V) {
        if (threadIdx.x == 0 && a.status) atomicOr(a.status, DF2_STATUS_ID_OUT_OF_RANGE);
        return;
    }
    constexpr int kSteps = kSmall / kThreads;  // of 32 positions a warp
    const int part = (int(a.N) + kThreads - 1) / kThreads * 32;  // a warp's positions
    unsigned mine[kSteps];
    bool earlier = false;
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        const int m = warp * part + s * 32 + lane;
        const bool same = s * 32 < part && m < a.N && __ldg(a.ids + m) == id;
        earlier |= same && m < n;
        float w;
        mine[s] = __ballot_sync(kFull, same && counts(a, uint32_t(m), &w));
    }
    if (__syncthreads_or(earlier)) return;
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const int64_t left_cols = a.D - column<W, 32>(slice, lane, 0);
    const char* src = static_cast<const char*>(a.src) + column<W, 32>(slice, lane, 0) * (SRC16 ? 2 : 4);
    const uint64_t stride = uint64_t(a.src_ld) * (SRC16 ? 2 : 4);
#pragma unroll
    for (int s = 0; s < kSteps; ++s) {
        while (mine[s]) {
            Row<SRC16, W, 32> r[kAhead];
            float w[kAhead];
            unsigned left = mine[s];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (left) {
                    const uint32_t m = uint32_t(warp * part + s * 32 + __ffs(left) - 1);
                    w[k] = a.w ? __ldg(a.w + m) : 1.f;
                    r[k].load(src + m / a.per_row * stride, left_cols);
                    left &= left - 1;
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (mine[s]) {
                    float f[8];
                    r[k].get(f);
                    add_row(acc, f, w[k]);
                    mine[s] &= mine[s] - 1;
                }
            }
        }
    }
    sums[warp][0][lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    sums[warp][1][lane] = make_float4(acc[4], acc[5], acc[6], acc[7]);
    __syncthreads();
    if (warp) return;
    for (int g = 1; g < kWarps; ++g) {
        const float4 x = sums[g][0][lane], y = sums[g][1][lane];
        acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
        acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
    }
    put_row<OUT16, W, 32>(a, id, slice, lane, acc);
}

// Lanes a group: D up to 64 columns fits eight.
int lanes_of(int64_t D) { return D <= 64 ? 8 : 32; }
int64_t slices_of(int64_t D, int L) { return (D + 8 * L - 1) / (8 * L); }

// Positions a chunk: a power of two that leaves each of 152 SMs 32 warps, within 16 .. 512
// (shorter chunks leave more parts, longer ones fewer warps).
int chunk_of(int64_t N, int64_t D, int L) {
    int E = 16;
    while (E < 512 && N * slices_of(D, L) * L > int64_t(E) * 152 * 32 * 32) E *= 2;
    return E;
}

bool vectors(const void* p, int64_t ld, int64_t D, bool bf16) {
    return D % 8 == 0 && (ld * (bf16 ? 2 : 4)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

bool all_small(const FoldArgs* jobs, int count) {
    for (int i = 0; i < count; ++i)
        if (jobs[i].N > kSmall) return false;
    return true;
}

template <bool SRC16, bool OUT16, int W, int L>
cudaError_t launch(Plan& p, bool small, int64_t blocks, cudaStream_t stream) {
    if (small) {
        fold_small_kernel<SRC16, OUT16, W><<<unsigned(blocks), kThreads, 0, stream>>>(p);
        note_launch();
        return cudaGetLastError();
    }
    fold_kernel<SRC16, OUT16, W, L><<<unsigned(blocks), kThreads, 0, stream>>>(p);
    note_launch();
    cudaError_t e = cudaGetLastError();
    const int64_t units = p.chunks[0] * p.slices[0] + (p.count > 1 ? p.chunks[1] * p.slices[1] : 0);
    if (e != cudaSuccess || units == 0) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(units));
    cfg.blockDim = dim3(kJoinWarps * 32);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, fold_join_kernel<OUT16, W, L>, p);
    note_launch();
    return e;
}

}  // namespace

size_t fold_parts_bytes(int64_t N, int64_t D) {
    const int L = lanes_of(D), E = chunk_of(N, D, L);
    return size_t((N + E - 1) / E) * 2 * slices_of(D, L) * 8 * L * sizeof(float);
}

bool fold_sorts(const FoldArgs* jobs, int count) { return !all_small(jobs, count); }

cudaError_t fold_sort_launch(const FoldArgs* jobs, int count, cudaStream_t stream) {
    if (!fold_sorts(jobs, count)) return cudaSuccess;
    SortJob s[kMaxJobs];
    for (int i = 0; i < count; ++i)
        s[i] = SortJob{jobs[i].ids, jobs[i].N, uint32_t(jobs[i].V), jobs[i].pairs, jobs[i].spare, jobs[i].status};
    return token_sort_launch(s, count, stream);
}

cudaError_t fold_launch(const FoldArgs* jobs, int count, cudaStream_t stream) {
    Plan p{};
    p.count = count;
    const bool small = all_small(jobs, count);
    const int L = small ? 32 : lanes_of(jobs[0].D);
    bool vec = true;
    int64_t blocks = 0;
    for (int i = 0; i < count; ++i) {
        const FoldArgs& a = p.a[i] = jobs[i];
        vec = vec && vectors(a.src, a.src_ld, a.D, a.src_bf16) && vectors(a.out, a.out_ld, a.D, a.out_bf16);
        p.slices[i] = int(slices_of(a.D, L));
        p.E[i] = chunk_of(a.N, a.D, L);
        p.chunks[i] = (a.N + p.E[i] - 1) / p.E[i];
        const int64_t fold = small ? a.N * p.slices[i] : (p.chunks[i] * p.slices[i] * L + kThreads - 1) / kThreads;
        int64_t fill = 0;
        if (!a.accumulate) {
            const int64_t sz = a.out_bf16 ? 2 : 4, row = a.D * sz;
            const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && row % 16 == 0 && (a.out_ld * sz) % 16 == 0;
            p.fill_unit[i] = wide ? 16 : int(sz);
            int64_t rows = dmax<int64_t>(1, dmin<int64_t>(kFillRows, kFillBytes / row));
            rows = dmin(rows, dmax<int64_t>(1, a.V / (152 * 8)));
            p.fill_rows[i] = int(rows);
            fill = (a.V + p.fill_rows[i] - 1) / p.fill_rows[i];
        }
        if (fold > INT32_MAX || fill > INT32_MAX || p.chunks[i] * p.slices[i] > INT32_MAX / 2) return cudaErrorInvalidConfiguration;
        p.fold_blocks[i] = int(fold);
        p.fill_blocks[i] = int(fill);
        blocks += fold + fill;
    }
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const bool s16 = jobs[0].src_bf16, o16 = jobs[0].out_bf16;
#define DF2_FOLD(S, O)                                                                                          (vec ? (L == 8 ? launch<S, O, 8, 8>(p, small, blocks, stream) : launch<S, O, 8, 32>(p, small, blocks, stream))          : (L == 8 ? launch<S, O, 1, 8>(p, small, blocks, stream) : launch<S, O, 1, 32>(p, small, blocks, stream)))
    if (s16) return o16 ? DF2_FOLD(true, true) : DF2_FOLD(true, false);
    return o16 ? DF2_FOLD(false, true) : DF2_FOLD(false, false);
#undef DF2_FOLD
}

}  // namespace df2
