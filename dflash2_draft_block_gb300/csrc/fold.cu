// The gradient of a table gathered by token id: out[v, :] (+)= scale * the sum over the
// positions n of token v, in order of n, of w[n] * src[n / per_row, :].
//
// The positions arrive sorted by token (token_sort.cu).  The sorted list is cut into
// chunks of E positions and D into slices of 256 columns; a warp owns a (chunk, slice): a
// lane holds 8 columns' sums in fp32, loads kAhead rows before it adds the first, and
// writes a token's row when the list moves on to the next.  A token that runs over a
// chunk's end is finished by the warp it began in when less than E / 2 positions are left
// of it; a longer one (a mask token can hold most of a batch) is split there, every chunk
// leaves its part in fp32, and fold_join_kernel adds the parts, one CTA a (token, slice).
// Where the cuts fall depends on the sorted list alone, so results repeat bit for bit.
//
// Bound: HBM or L2.  Every row of src is read once a slice, every touched row of out is
// written once; with accumulate false a fill writes the others' zeros first.
#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kWarps = 4;
constexpr int kSlice = 256;
constexpr int kAhead = 8;
constexpr int kJoinWarps = 8;

__device__ __forceinline__ uint32_t key_at(const uint64_t* pairs, int64_t i) {
    return uint32_t(__ldg(pairs + i));
}

// Whether the token that ends chunk [.., b) goes on for at least half positions from b.
__device__ __forceinline__ bool split_at(const uint64_t* pairs, int64_t N, int64_t b, int half) {
    return b + half <= N && key_at(pairs, b - 1) == key_at(pairs, b + half - 1);
}

// The first i >= b whose key differs from the key before b; known to lie before b + half.
__device__ __forceinline__ int64_t run_end(const uint64_t* pairs, int64_t N, int64_t b, int half, int lane) {
    const uint32_t k = key_at(pairs, b - 1);
    for (int o = 0; o < half; o += 32) {
        const int64_t i = b + o + lane;
        const unsigned other = __ballot_sync(kFull, i >= N || key_at(pairs, i) != k);
        if (other) return b + o + __ffs(other) - 1;
    }
    return dmin<int64_t>(N, b + half);
}

// A lane's 8 columns: consecutive with vectors, else 32 apart.
template <int W>
__device__ __forceinline__ int64_t column(int64_t slice, int lane, int i) {
    return slice * kSlice + (W == 8 ? lane * 8 + i : i * 32 + lane);
}

template <bool SRC16, int W>
struct Row {
    uint4 a, b;  // as loaded: bf16 in a; fp32 in a, b (vectors), or one element a word

    __device__ __forceinline__ void load(const void* src, int64_t ld, int64_t row, int64_t slice, int lane, int64_t D) {
        constexpr int SZ = SRC16 ? 2 : 4;
        const char* p = static_cast<const char*>(src) + (row * ld + column<W>(slice, lane, 0)) * SZ;
        if (W == 8) {
            if (column<W>(slice, lane, 0) >= D) return;
            a = __ldg(reinterpret_cast<const uint4*>(p));
            if (!SRC16) b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
        } else {
            uint32_t* r = &a.x;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint32_t& w = i < 4 ? r[i] : (&b.x)[i - 4];
                if (column<W>(slice, lane, i) >= D) w = 0;
                else if (SRC16) w = uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p + i * 32 * SZ))) << 16;
                else w = __ldg(reinterpret_cast<const uint32_t*>(p + i * 32 * SZ));
            }
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

// out[row, lane's columns] = scale * f (+ itself)
template <bool OUT16, int W>
__device__ __forceinline__ void put_row(const FoldArgs& a, int64_t row, int64_t slice, int lane, const float f[8]) {
    constexpr int SZ = OUT16 ? 2 : 4;
    char* p = static_cast<char*>(a.out) + (row * a.out_ld + column<W>(slice, lane, 0)) * SZ;
    float g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = __fmul_rn(f[i], a.scale);
    if (W == 8) {
        if (column<W>(slice, lane, 0) >= a.D) return;
        uint4* q = reinterpret_cast<uint4*>(p);
        if (OUT16) {
            if (a.accumulate) {
                float o[8];
                unpack8(q[0], o);
#pragma unroll
                for (int i = 0; i < 8; ++i) g[i] = __fadd_rn(o[i], g[i]);
            }
            q[0] = make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]),
                              pack_bf16(g[6], g[7]));
        } else {
            float4* o = reinterpret_cast<float4*>(p);
            if (a.accumulate) {
                const float4 x = o[0], y = o[1];
                g[0] = __fadd_rn(x.x, g[0]); g[1] = __fadd_rn(x.y, g[1]);
                g[2] = __fadd_rn(x.z, g[2]); g[3] = __fadd_rn(x.w, g[3]);
                g[4] = __fadd_rn(y.x, g[4]); g[5] = __fadd_rn(y.y, g[5]);
                g[6] = __fadd_rn(y.z, g[6]); g[7] = __fadd_rn(y.w, g[7]);
            }
            o[0] = make_float4(g[0], g[1], g[2], g[3]);
            o[1] = make_float4(g[4], g[5], g[6], g[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (column<W>(slice, lane, i) >= a.D) continue;
            if (OUT16) {
                uint16_t* q = reinterpret_cast<uint16_t*>(p + i * 32 * SZ);
                *q = f32_to_bf16_rn(a.accumulate ? __fadd_rn(bf16_to_f32(*q), g[i]) : g[i]);
            } else {
                float* q = reinterpret_cast<float*>(p + i * 32 * SZ);
                *q = a.accumulate ? __fadd_rn(*q, g[i]) : g[i];
            }
        }
    }
}

// A lane's 8 sums in the parts buffer: part s of chunk c, slice.
__device__ __forceinline__ float4* part_at(const FoldArgs& a, int64_t slices, int64_t c, int s, int64_t slice, int lane) {
    return reinterpret_cast<float4*>(a.parts + (((c * 2 + s) * slices + slice) * kSlice) + lane * 8);
}

template <bool SRC16, bool OUT16, int W>
__global__ void __launch_bounds__(kWarps * 32) fold_kernel(const FoldArgs a, int E, int64_t chunks, int slices) {
    const int lane = threadIdx.x & 31;
    const int64_t unit = int64_t(blockIdx.x) * kWarps + (threadIdx.x >> 5);
    const int64_t c = unit / slices, slice = unit - c * slices;
    if (c >= chunks) return;
    const int half = E / 2;
    const int64_t e0 = c * E, e1 = dmin<int64_t>(e0 + E, a.N);
    int64_t i = e0, end = e1;
    bool head = false, tail = false;
    if (c > 0 && key_at(a.pairs, e0 - 1) == key_at(a.pairs, e0)) {
        head = split_at(a.pairs, a.N, e0, half);
        if (!head) i = run_end(a.pairs, a.N, e0, half, lane);
    }
    if (i >= e1) return;  // a short last chunk the one before it finishes
    if (e1 < a.N && key_at(a.pairs, e1 - 1) == key_at(a.pairs, e1)) {
        tail = split_at(a.pairs, a.N, e1, half);
        if (!tail) end = run_end(a.pairs, a.N, e1, half, lane);
    }

    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    uint32_t cur = key_at(a.pairs, i);
    auto leave = [&](bool is_tail) {  // the current token's sums, to its row or to its part
        if (head || is_tail) {
            float4* p = part_at(a, slices, c, head ? 0 : 1, slice, lane);
            p[0] = make_float4(acc[0], acc[1], acc[2], acc[3]);
            p[1] = make_float4(acc[4], acc[5], acc[6], acc[7]);
        } else {
            put_row<OUT16, W>(a, cur, slice, lane, acc);
        }
        head = false;
#pragma unroll
        for (int k = 0; k < 8; ++k) acc[k] = 0.f;
    };
    const uint32_t none = uint32_t(a.V);
    for (; i < end && cur != none; i += 32) {
        const int n = int(dmin<int64_t>(32, end - i));
        uint64_t pair = lane < n ? __ldg(a.pairs + i + lane) : uint64_t(none);
        float w = 0.f;
        if (a.w && uint32_t(pair) != none) w = __ldg(a.w + uint32_t(pair >> 32));
        const uint32_t key = uint32_t(pair);
        const uint32_t row = uint32_t(pair >> 32) / a.per_row;
        for (int j = 0; j < n; j += kAhead) {
            Row<SRC16, W> r[kAhead];
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t kk = __shfl_sync(kFull, key, j + k);
                const uint32_t rr = __shfl_sync(kFull, row, j + k);
                if (kk != none) r[k].load(a.src, a.src_ld, rr, slice, lane, a.D);
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t kk = __shfl_sync(kFull, key, j + k);
                const float ww = __shfl_sync(kFull, w, j + k);
                if (kk != cur && cur != none && j + k < n) {
                    leave(false);
                    cur = kk;
                }
                if (kk == cur && cur != none) {
                    float f[8];
                    r[k].get(f);
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[q] = a.w ? fmaf(ww, f[q], acc[q]) : __fadd_rn(acc[q], f[q]);
                }
            }
        }
    }
    if (cur != none) leave(tail);
}

template <bool OUT16, int W>
__global__ void __launch_bounds__(kJoinWarps * 32) fold_join_kernel(const FoldArgs a, int E, int64_t chunks, int slices) {
    __shared__ float sums[kJoinWarps][kSlice];
    const int64_t c = blockIdx.x / slices, slice = blockIdx.x - c * slices;
    const int half = E / 2;
    const int64_t e0 = c * E, e1 = e0 + E;
    if (e1 >= a.N) return;
    const uint32_t k = key_at(a.pairs, e1 - 1);
    // the chunk the token begins in owns the sum
    if (k == uint32_t(a.V) || !split_at(a.pairs, a.N, e1, half)) return;
    if (c > 0 && key_at(a.pairs, e0 - 1) == k) return;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int more = 0;  // the chunks after c that left a part
    for (int got = kJoinWarps * 32; got == kJoinWarps * 32;) {
        const int64_t b = (c + 1 + more + threadIdx.x) * E;
        got = __syncthreads_count(b < a.N && key_at(a.pairs, b - 1) == k && split_at(a.pairs, a.N, b, half));
        more += got;
    }
    float acc[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int m = warp; m <= more; m += kJoinWarps) {
        const float4* p = part_at(a, slices, c + m, m == 0 ? 1 : 0, slice, lane);
        const float4 x = __ldg(p), y = __ldg(p + 1);
        acc[0] += x.x; acc[1] += x.y; acc[2] += x.z; acc[3] += x.w;
        acc[4] += y.x; acc[5] += y.y; acc[6] += y.z; acc[7] += y.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) sums[warp][lane * 8 + i] = acc[i];
    __syncthreads();
    if (warp) return;
    for (int w = 1; w < dmin(kJoinWarps, more + 1); ++w)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[i] += sums[w][lane * 8 + i];
    put_row<OUT16, W>(a, k, slice, lane, acc);
}

// zeros in [rows, D elements of size SZ] of stride ld
__global__ void __launch_bounds__(256) fill_kernel(char* out, int64_t rows, int64_t row_bytes, int64_t ld_bytes, int unit) {
    const int64_t per = row_bytes / unit;
    const int64_t n = rows * per, step = int64_t(gridDim.x) * blockDim.x;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += step) {
        const int64_t r = ld_bytes == row_bytes ? 0 : i / per;
        char* p = out + r * ld_bytes + (i - r * per) * unit;
        if (unit == 16) *reinterpret_cast<uint4*>(p) = make_uint4(0, 0, 0, 0);
        else if (unit == 4) *reinterpret_cast<uint32_t*>(p) = 0;
        else *reinterpret_cast<uint16_t*>(p) = 0;
    }
}

int64_t slices_of(int64_t D) { return (D + kSlice - 1) / kSlice; }

// Positions a chunk: a power of two that leaves each of 152 SMs 32 warps, within 16 .. 512
// (shorter chunks leave more parts, longer ones fewer warps).
int chunk_of(int64_t N, int64_t D) {
    int E = 16;
    while (E < 512 && N * slices_of(D) > int64_t(E) * 152 * 32) E *= 2;
    return E;
}

bool vectors(const void* p, int64_t ld, int64_t D, bool bf16) {
    return D % 8 == 0 && (ld * (bf16 ? 2 : 4)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <bool SRC16, bool OUT16, int W>
cudaError_t launch(const FoldArgs& a, cudaStream_t stream) {
    const int E = chunk_of(a.N, a.D);
    const int64_t chunks = (a.N + E - 1) / E, slices = slices_of(a.D);
    const int64_t grid = (chunks * slices + kWarps - 1) / kWarps;
    if (chunks * slices > INT32_MAX) return cudaErrorInvalidConfiguration;
    fold_kernel<SRC16, OUT16, W><<<unsigned(grid), kWarps * 32, 0, stream>>>(a, E, chunks, int(slices));
    note_launch();
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess || chunks == 1) return e;
    fold_join_kernel<OUT16, W><<<unsigned(chunks * slices), kJoinWarps * 32, 0, stream>>>(a, E, chunks, int(slices));
    note_launch();
    return cudaGetLastError();
}

}  // namespace

size_t fold_parts_bytes(int64_t N, int64_t D) {
    const int64_t chunks = (N + chunk_of(N, D) - 1) / chunk_of(N, D);
    return size_t(chunks) * 2 * slices_of(D) * kSlice * sizeof(float);
}

cudaError_t fold_launch(const FoldArgs& a, cudaStream_t stream) {
    if (!a.accumulate) {
        const int64_t sz = a.out_bf16 ? 2 : 4, row = a.D * sz, ld = a.out_ld * sz;
        const bool dense = ld == row;  // one long row then
        const int64_t rows = dense ? 1 : a.V, bytes = dense ? a.V * row : row;
        const bool wide = (reinterpret_cast<uintptr_t>(a.out) & 15) == 0 && bytes % 16 == 0 && (dense || ld % 16 == 0);
        const int unit = wide ? 16 : int(sz);
        const int64_t grid = dmin<int64_t>((rows * (bytes / unit) + 255) / 256, 152 * 8);
        fill_kernel<<<unsigned(grid), 256, 0, stream>>>(static_cast<char*>(a.out), rows, bytes, dense ? bytes : ld, unit);
        note_launch();
        const cudaError_t e = cudaGetLastError();
        if (e != cudaSuccess) return e;
    }
    if (a.N == 0) return cudaSuccess;
    const bool vec = vectors(a.src, a.src_ld, a.D, a.src_bf16) && vectors(a.out, a.out_ld, a.D, a.out_bf16);
#define DF2_FOLD(S, O) (vec ? launch<S, O, 8>(a, stream) : launch<S, O, 1>(a, stream))
    if (a.src_bf16) return a.out_bf16 ? DF2_FOLD(true, true) : DF2_FOLD(true, false);
    return a.out_bf16 ? DF2_FOLD(false, true) : DF2_FOLD(false, false);
#undef DF2_FOLD
}

}  // namespace df2
