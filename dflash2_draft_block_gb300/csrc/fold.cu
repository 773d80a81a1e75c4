// The gradient of a table gathered by token id: out[v, :] (+)= scale * the sum over the
// positions n of token v, in order of n, of w[n] * src[n / per_row, :].
//
// The positions are sorted by token (token_sort.cu).  The sorted list is cut into chunks of
// E positions and D into slices of 8 L columns; a group of L lanes owns a (chunk, slice): a
// lane holds 8 columns' sums in fp32, loads kAhead rows before it adds the first, and
// writes a token's row when the list moves on to the next.  A token that runs over a
// chunk's end is finished by the group it began in when less than E / 2 positions are left
// of it; a longer one (a mask token can hold most of a batch) is split there, every chunk
// leaves its part in fp32, the group the token began in notes it down, and
// fold_join_kernel adds the parts, one CTA a (token, slice) at a time.  Where the cuts fall
// depends on the sorted list alone, so results repeat bit for bit.  Four rows in flight and
// 96 registers leave five CTAs an SM (eight rows take 122 and leave four).
//
// Where asked (fill), the rows of absent tokens become zeros in the same launch: some CTAs
// from the start, and the others when their chunks are done, take ranges of rows off a
// counter, mark those that the sorted list holds, and clear the others, so every row is
// written once, and the writes run beside the gathers.  16,384 rows of 5,120 into 248,320
// bf16 rows take 390 us (2.5 GB written, 6.95 TB/s); with a fixed share of the clearing a
// CTA 514 us at best; with 152 to 608 CTAs that only clear 418 to 409, and the gathers of
// other lists lose room to them (141 us with 608, 123 with 114, 16,384 rows of 16 at rank 256).
// Bulk copies clear what lies between a row's 16-byte boundaries, whatever its width: 37 us
// against 48 with stores an element (6,338 rows of 303 fp32 into 65,371).
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
constexpr int kAhead = 4;  // rows in flight a lane
constexpr int kJoinWarps = 8;
constexpr int kJoinBlocks = 152 * 4;  // at most: each takes split tokens in turn
constexpr int kSmall = 512;
constexpr int kFillRows = 4096;             // rows a fill takes at a time, at most
constexpr int64_t kFillBytes = 128 * 1024;  // and their bytes
constexpr int kFillBlocks = 114;            // CTAs that only fill, the first of a launch: at least,
constexpr int kAllBlocks = 152 * 5;         // and as many as make so many in all
constexpr int kZeros = 4096;                // bytes of zeros a filling CTA copies from

struct Plan {
    FoldArgs a[kMaxJobs];
    int count;
    int E[kMaxJobs];
    int64_t chunks[kMaxJobs];
    int slices[kMaxJobs];
    int fold_blocks[kMaxJobs];
    int fills[kMaxJobs];      // ranges of fill_rows rows
    int fill_blocks;          // CTAs that do nothing else
    int fill_rows[kMaxJobs];
};

__device__ __forceinline__ uint32_t key_at(const uint64_t* pairs, int64_t i) {
    return uint32_t(__ldg(pairs + i));
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

// Where a lane writes its columns of a row, and how.
struct Out {
    char* p;         // row 0 at the lane's first column
    uint64_t stride;  // bytes a row
    int64_t left;    // columns from there on
    float scale;
    bool accumulate;
};

template <int W, int L>
__device__ __forceinline__ Out out_of(const FoldArgs& a, int64_t slice, int gl) {
    const int sz = a.out_bf16 ? 2 : 4;
    const int64_t c = column<W, L>(slice, gl, 0);
    return Out{static_cast<char*>(a.out) + c * sz, uint64_t(a.out_ld) * sz, a.D - c, a.scale, a.accumulate};
}

// Adds to global memory that return nothing (of an atomicAdd on a generic pointer the old
// value comes back, wanted or not).
__device__ __forceinline__ void add1(float* p, float x) {
    asm volatile("red.relaxed.gpu.global.add.f32 [%0], %1;" ::"l"(__cvta_generic_to_global(p)), "f"(x) : "memory");
}
__device__ __forceinline__ void add4(float4* p, float4 x) {
    asm volatile("red.relaxed.gpu.global.add.v4.f32 [%0], {%1, %2, %3, %4};" ::"l"(__cvta_generic_to_global(p)),
                 "f"(x.x), "f"(x.y), "f"(x.z), "f"(x.w)
                 : "memory");
}

// A row's columns = scale * f (+ themselves).  Added in fp32 by the memory's own add: a row
// has one writer, so the result is the one rounded sum, and nobody waits for the old row.
// The add takes subnormal operands, the row's own among them, for zero: at most 1.2e-38 is
// lost a value.  Read, added and stored, which keeps them, 5,003 rows of 251 take 28.7 us
// instead of 26.6, a selector's 512 rows of 16 at rank 256 40 to 43 instead of 38.
template <bool OUT16, int W, int L>
__device__ __forceinline__ void put_columns(char* p, int64_t left, float scale, bool accumulate, float4 x, float4 y) {
    float g[8] = {x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(g[i], scale);
    if (W == 8) {
        if (left <= 0) return;
        if (OUT16) {
            uint4* q = reinterpret_cast<uint4*>(p);
            if (accumulate) {
                float o[8];
                unpack8(*q, o);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = __fadd_rn(o[i], g[i]);
            }
            *q = make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]), pack_bf16(g[6], g[7]));
        } else {
            float4* q = reinterpret_cast<float4*>(p);
            x = make_float4(g[0], g[1], g[2], g[3]);
            y = make_float4(g[4], g[5], g[6], g[7]);
            if (accumulate) {
                add4(q, x);
                add4(q + 1, y);
            } else {
                q[0] = x;
                q[1] = y;
            }
        }
    } else if (OUT16) {
        uint16_t* q = reinterpret_cast<uint16_t*>(p);
        if (accumulate) {
            uint16_t o[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = i * L < left ? q[i * L] : uint16_t(0);
#pragma unroll
            for (int i = 0; i < 8; ++i) g[i] = __fadd_rn(bf16_to_f32(o[i]), g[i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i * L < left) q[i * L] = f32_to_bf16_rn(g[i]);
    } else {
        float* q = reinterpret_cast<float*>(p);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (i * L >= left) continue;
            if (accumulate) add1(q + i * L, g[i]);
            else q[i * L] = g[i];
        }
    }
}

template <bool OUT16, int W, int L>
__device__ __noinline__ void put_columns_call(char* p, int64_t left, float scale, bool accumulate, float4 x, float4 y) {
    put_columns<OUT16, W, L>(p, left, scale, accumulate, x, y);
}

// Column by column a row takes so much code that the copies of it in the fold's loop cost
// more in instruction fetches than a call does (52 against 31 us for 5003 rows of 251);
// with vectors the call costs more (95 against 76 us for 262,144 rows of 256).
template <bool OUT16, int W, int L>
__device__ __forceinline__ void put_row(const Out& o, uint32_t row, const float f[8]) {
    const float4 x = make_float4(f[0], f[1], f[2], f[3]), y = make_float4(f[4], f[5], f[6], f[7]);
    if constexpr (W == 8) put_columns<OUT16, W, L>(o.p + row * o.stride, o.left, o.scale, o.accumulate, x, y);
    else put_columns_call<OUT16, W, L>(o.p + row * o.stride, o.left, o.scale, o.accumulate, x, y);
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

// Zeros to the rows [block * fill_rows, ..) of a job's absent tokens.
template <bool SMALL>
__device__ void fill(const Plan& p, int job, int64_t block, uint32_t* held, int64_t* range, const uint4* zeros) {
    const FoldArgs a = job ? p.a[1] : p.a[0];  // (a parameter indexed by a register is slow to read)
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
    // a row a thread: elements up to a 16-byte boundary, a bulk copy of zeros, the rest
    const int sz = a.out_bf16 ? 2 : 4;
    const int64_t ld = a.out_ld * sz, bytes = a.D * sz;
    char* out = static_cast<char*>(a.out) + v0 * ld;
    auto clear = [&](char* q, int64_t n) {
        for (int64_t o = 0; o < n; o += sz)
            if (sz == 2) *reinterpret_cast<uint16_t*>(q + o) = 0;
            else *reinterpret_cast<uint32_t*>(q + o) = 0;
    };
    for (int r = tid; r < rows; r += kThreads) {
        if (held[r >> 5] >> (r & 31) & 1) continue;
        char* q = out + r * ld;
        const int64_t head = dmin<int64_t>(-reinterpret_cast<intptr_t>(q) & 15, bytes), mid = (bytes - head) & ~int64_t(15);
        clear(q, head);
        for (int64_t o = 0; o < mid; o += kZeros)
            bulk_store(q + head + o, zeros, uint32_t(dmin<int64_t>(kZeros, mid - o)));
        clear(q + head + mid, bytes - head - mid);
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The CTA's share of all jobs' fills: ranges off the counter while there are any, or the
// range of its number.
template <bool SMALL>
__device__ void fill_all(const Plan& p) {
    __shared__ uint32_t held[kFillRows / 32];
    __shared__ int64_t range[2];
    __shared__ __align__(16) uint4 zeros[kZeros / 16];
    __shared__ int taken;
    const int total = p.fills[0] + p.fills[1];
    if (total == 0) return;
    for (int i = threadIdx.x; i < kZeros / 16; i += kThreads) zeros[i] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");  // for the copies that read them
    for (;;) {
        int u = blockIdx.x;
        if (!SMALL) {
            if (threadIdx.x == 0) taken = int(dmin(atomicAdd(p.a[0].split + 1, 1u), uint32_t(total)));
            __syncthreads();
            u = taken;
            if (u >= total) break;
        }
        const int job = u >= p.fills[0];
        fill<SMALL>(p, job, u - (job ? p.fills[0] : 0), held, range, zeros);
        if (SMALL) break;
        __syncthreads();
    }
    asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// A fold CTA's job and its number there.
__device__ __forceinline__ int64_t fold_block(const Plan& p, int* job) {
    const int64_t n = int64_t(blockIdx.x) - p.fill_blocks;
    *job = n >= p.fold_blocks[0];
    return *job ? n - p.fold_blocks[0] : n;
}

// A group's chunk and slice.
template <bool SRC16, bool OUT16, int W, int L>
__device__ __forceinline__ void fold_chunk(const Plan& p) {
    int job;
    const int64_t block = fold_block(p, &job);
    const FoldArgs& a = p.a[job];
    const int lane = threadIdx.x & 31, gl = lane & (L - 1);
    const unsigned gmask = group_mask<L>(lane);
    const int64_t unit = (block * kThreads + threadIdx.x) / L;
    const int slices = p.slices[job], E = p.E[job], half = E / 2;
    const int64_t c = unit / slices, slice = unit - c * slices;
    if (c >= p.chunks[job]) return;
    const uint64_t* pairs = a.pairs;
    const int64_t e0 = c * E, e1 = dmin<int64_t>(e0 + E, a.N);
    // the keys that decide where this group's tokens begin and end, in one round of loads:
    // before and at each end of the chunk, and half a chunk from it
    const int64_t probe = gl < 3 ? (gl == 0 ? e0 - 1 : gl == 1 ? e0 : e0 + half - 1)
                                 : (gl == 3 ? e1 - 1 : gl == 4 ? e1 : e1 + half - 1);
    const bool held = gl < 6 && probe >= 0 && probe < a.N;
    const uint64_t probed = held ? __ldg(pairs + probe) : ~uint64_t(0);
    const uint32_t pk = held ? uint32_t(probed) : 0xFFFFFFFFu;  // (no token is that)
    auto probed_key = [&](int k) { return __shfl_sync(gmask, pk, k, L); };
    const uint32_t k_before = probed_key(0), k_first = probed_key(1), k_last = probed_key(3);
    const bool crosses0 = k_before == k_first, crosses1 = k_last == probed_key(4);
    bool head = crosses0 && probed_key(2) == k_before;
    const bool tail = crosses1 && probed_key(5) == k_last;
    int64_t i = e0, end = e1;
    if (crosses0 && !head) i = run_end<L>(pairs, a.N, e0, half, lane);
    if (i >= e1) return;  // a short last chunk the one before it finishes
    if (crosses1 && !tail) end = run_end<L>(pairs, a.N, e1, half, lane);

    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    const uint32_t none = uint32_t(a.V);
    uint32_t cur = key_at(pairs, i);
    if (cur == none) return;
    const Out o = out_of<W, L>(a, slice, gl);
    auto leave = [&](bool is_tail) {  // the current token's sums, to its row or to its part
        if (head || is_tail) {
            float4* q = part_at<L>(a, slices, c, head ? 0 : 1, slice, gl);
            q[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            q[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        } else {
            put_row<OUT16, W, L>(o, cur, acc);
        }
        head = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    };
    const int64_t left = a.D - column<W, L>(slice, gl, 0);
    const char* src = static_cast<const char*>(a.src) + column<W, L>(slice, gl, 0) * (SRC16 ? 2 : 4);
    const uint64_t stride = uint64_t(a.src_ld) * (SRC16 ? 2 : 4);
    auto pairs_from = [&](int64_t at) { return at + gl < end ? __ldg(pairs + at + gl) : uint64_t(none); };
    uint64_t pair = pairs_from(i);
    for (bool more = true; more && i < end; i += L) {
        const int n = int(dmin<int64_t>(L, end - i));
        const uint64_t next = pairs_from(i + L);
        const uint32_t key = uint32_t(pair);
        float w = 0.f;
        const bool on = key != none && counts(a, uint32_t(pair >> 32), &w);
        const uint32_t row = uint32_t(pair >> 32) / a.per_row;
        // bit k: position k has a part; a token begins at k (`none` ends the list)
        const uint32_t before = __shfl_up_sync(gmask, key, 1, L);
        unsigned live = __ballot_sync(gmask, on) >> (lane & ~(L - 1));
        unsigned begins = __ballot_sync(gmask, gl < n && key != (gl ? before : cur)) >> (lane & ~(L - 1));
        more = __shfl_sync(gmask, key, n - 1, L) != none;
#pragma unroll 1
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
        pair = next;
    }
    if (cur == none) return;
    // a token that began here and goes on: the join adds its parts
    if (tail && !head && gl == 0) a.split[2 + atomicAdd(a.split, 1u)] = uint32_t(unit);
    leave(tail);
}

template <bool SRC16, bool OUT16, int W, int L>
__global__ void __launch_bounds__(kThreads, 5) fold_kernel(const __grid_constant__ Plan p) {
    // the join may take its place now: it waits for this kernel where it reads parts
    asm volatile("griddepcontrol.launch_dependents;");
    if (blockIdx.x >= p.fill_blocks) fold_chunk<SRC16, OUT16, W, L>(p);
    __syncthreads();
    fill_all<false>(p);
}

template <bool OUT16, int W, int L>
__global__ void __launch_bounds__(kJoinWarps * 32) fold_join_kernel(const __grid_constant__ Plan p) {
    constexpr int kGroups = kJoinWarps * 32 / L;
    __shared__ float4 sums[kGroups][2][L];
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int gl = threadIdx.x & (L - 1), group = threadIdx.x / L;
    const uint32_t count0 = __ldcg(p.a[0].split), count1 = p.count > 1 ? __ldcg(p.a[1].split) : 0u;
    for (uint32_t s = blockIdx.x; s < count0 + count1; s += gridDim.x) {
        const int job = s >= count0;
        const FoldArgs& a = p.a[job];
        const uint32_t unit = __ldcg(a.split + 2 + s - (job ? count0 : 0u));
        const int slices = p.slices[job], E = p.E[job], half = E / 2;
        const int64_t c = unit / slices, slice = unit - c * slices;
        const uint32_t k = key_at(a.pairs, (c + 1) * E - 1);
        int more = 0;  // the chunks after c that left a part
        for (int got = kJoinWarps * 32; got == kJoinWarps * 32;) {
            const int64_t b = (c + 1 + more + threadIdx.x) * E;
            // (a token that reaches half a chunk past b was split at b)
            got = __syncthreads_count(b + half <= a.N && key_at(a.pairs, b + half - 1) == k);
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
        if (group == 0) {
            for (int g = 1; g < dmin(kGroups, more + 1); ++g) {
                const float4 x = sums[g][0][gl], y = sums[g][1][gl];
                acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
                acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
            }
            put_row<OUT16, W, L>(out_of<W, L>(a, slice, gl), k, acc);
        }
        __syncthreads();
    }
}

// A block a (position, slice).  The block of a token's first position sums the token: the
// list is cut in four, a warp each, and the warps' sums are added in order.
template <bool SRC16, bool OUT16, int W>
__global__ void __launch_bounds__(kThreads) fold_small_kernel(const __grid_constant__ Plan p) {
    __shared__ float4 sums[kWarps][2][32];
    if (blockIdx.x < p.fill_blocks) {
        fill_all<true>(p);
        return;
    }
    int job;
    const int64_t block = fold_block(p, &job);
    const FoldArgs a = job ? p.a[1] : p.a[0];  // (a parameter indexed by a register is slow to read)
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
    put_row<OUT16, W, 32>(out_of<W, 32>(a, slice, lane), uint32_t(id), acc);
}

// Lanes a group: D up to 64 columns fits eight.
int lanes_of(int64_t D) { return D <= 64 ? 8 : 32; }
int64_t slices_of(int64_t D, int L) { return (D + 8 * L - 1) / (8 * L); }

// Positions a chunk: a power of two that leaves each of 152 SMs 32 warps, within 8 .. 512
// (shorter chunks leave more parts, longer ones fewer warps).
int chunk_of(int64_t N, int64_t D, int L) {
    int E = 8;
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
    cfg.gridDim = dim3(unsigned(dmin<int64_t>(units, kJoinBlocks)));
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

size_t fold_split_bytes(int64_t N, int64_t D) {
    const int L = lanes_of(D), E = chunk_of(N, D, L);
    return (2 + size_t((N + E - 1) / E) * slices_of(D, L)) * sizeof(uint32_t);
}

bool fold_sorts(const FoldArgs* jobs, int count) { return !all_small(jobs, count); }

cudaError_t fold_sort_launch(const FoldArgs* jobs, int count, cudaStream_t stream) {
    if (!fold_sorts(jobs, count)) return cudaSuccess;
    SortJob s[kMaxJobs];
    for (int i = 0; i < count; ++i)
        s[i] = SortJob{jobs[i].ids, jobs[i].N, uint32_t(jobs[i].V), jobs[i].pairs, jobs[i].spare, jobs[i].split,
                       jobs[i].status};
    return token_sort_launch(s, count, stream);
}

cudaError_t fold_launch(const FoldArgs* jobs, int count, cudaStream_t stream) {
    Plan p{};
    p.count = count;
    const bool small = all_small(jobs, count);
    const int L = small ? 32 : lanes_of(jobs[0].D);
    bool vec = true;
    int64_t blocks = 0, fills = 0;
    for (int i = 0; i < count; ++i) {
        const FoldArgs& a = p.a[i] = jobs[i];
        vec = vec && vectors(a.src, a.src_ld, a.D, a.src_bf16) && vectors(a.out, a.out_ld, a.D, a.out_bf16);
        p.slices[i] = int(slices_of(a.D, L));
        p.E[i] = chunk_of(a.N, a.D, L);
        p.chunks[i] = (a.N + p.E[i] - 1) / p.E[i];
        const int64_t fold = small ? a.N * p.slices[i] : (p.chunks[i] * p.slices[i] * L + kThreads - 1) / kThreads;
        int64_t fill = 0;
        if (a.fill) {
            const int64_t sz = a.out_bf16 ? 2 : 4, row = a.D * sz;
            const int64_t rows = dmin<int64_t>(dmin<int64_t>(kFillRows, kFillBytes / row), a.V / (152 * 8));
            p.fill_rows[i] = int(dmax<int64_t>(1, rows));
            fill = (a.V + p.fill_rows[i] - 1) / p.fill_rows[i];
        }
        if (fold > INT32_MAX || fill > INT32_MAX || p.chunks[i] * p.slices[i] > INT32_MAX / 2)
            return cudaErrorInvalidConfiguration;
        p.fold_blocks[i] = int(fold);
        p.fills[i] = int(fill);
        blocks += fold;
        fills += fill;
    }
    if (fills > INT32_MAX) return cudaErrorInvalidConfiguration;
    p.fill_blocks = int(small ? fills : dmin(fills, dmax<int64_t>(kFillBlocks, kAllBlocks - blocks)));
    blocks += p.fill_blocks;
    if (blocks == 0) return cudaSuccess;
    if (blocks > INT32_MAX) return cudaErrorInvalidConfiguration;
    const bool s16 = jobs[0].src_bf16, o16 = jobs[0].out_bf16;
#define DF2_FOLD(S, O)                                                                                   \
    (vec ? (L == 8 ? launch<S, O, 8, 8>(p, small, blocks, stream) : launch<S, O, 8, 32>(p, small, blocks, stream)) \
         : (L == 8 ? launch<S, O, 1, 8>(p, small, blocks, stream) : launch<S, O, 1, 32>(p, small, blocks, stream)))
    if (s16) return o16 ? DF2_FOLD(true, true) : DF2_FOLD(true, false);
    return o16 ? DF2_FOLD(false, true) : DF2_FOLD(false, false);
#undef DF2_FOLD
}

}  // namespace df2
