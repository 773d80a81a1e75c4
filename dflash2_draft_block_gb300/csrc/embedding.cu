// dflash2_embedding: out[n, :] = scale * table[ids[n], :], rounded once.
//
// Bound: HBM (a row in, a row out), or for a draft block's few rows the latency of one
// dependent load (id, then row).  Rows are cut into steps of 32 units of 8 elements (16
// bytes of bf16), several rows a step where rows are shorter; a warp takes kSteps
// consecutive steps, issues all of their loads before the first store, and divides once.
// Rows off 16-byte boundaries (odd D or strides) go element by element the same way.
// Stores are marked as streaming: what is worth keeping in L2 is the table's rows.  16,384 x
// 5,120 bf16 from 248,320 rows take 43 us (243 MB, 5.6 TB/s); with the units converted to
// fp32 before the branches on the id it issued 112 instructions a step (47 us).
#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kThreads = 128;
constexpr int kSteps = 4;  // a warp, where there is enough to do

// A unit as it lies in memory: 8 bf16 in a, 8 fp32 in a and b, or one element in a.x.
struct Unit {
    uint4 a, b;
};

template <bool BF16, int W>
__device__ __forceinline__ Unit read_unit(const char* p) {
    Unit u{};
    if (W == 8) {
        u.a = __ldg(reinterpret_cast<const uint4*>(p));
        if (!BF16) u.b = __ldg(reinterpret_cast<const uint4*>(p) + 1);
    } else {
        u.a.x = BF16 ? uint32_t(__ldg(reinterpret_cast<const uint16_t*>(p))) << 16
                     : __ldg(reinterpret_cast<const uint32_t*>(p));
    }
    return u;
}

template <bool IN16, bool OUT16, int W>
__device__ __forceinline__ void write_scaled(char* p, const Unit& u, float scale) {
    if (W == 1) {
        const float f = __fmul_rn(__uint_as_float(u.a.x), scale);
        if (OUT16) *reinterpret_cast<uint16_t*>(p) = f32_to_bf16_rn(f);
        else *reinterpret_cast<float*>(p) = f;
        return;
    }
    float f[8];
    if (IN16) {
        unpack8(u.a, f);
    } else {
        f[0] = __uint_as_float(u.a.x); f[1] = __uint_as_float(u.a.y);
        f[2] = __uint_as_float(u.a.z); f[3] = __uint_as_float(u.a.w);
        f[4] = __uint_as_float(u.b.x); f[5] = __uint_as_float(u.b.y);
        f[6] = __uint_as_float(u.b.z); f[7] = __uint_as_float(u.b.w);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __fmul_rn(f[i], scale);
    if (OUT16) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                       pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
    } else {
        float4* q = reinterpret_cast<float4*>(p);
        __stcs(q, make_float4(f[0], f[1], f[2], f[3]));
        __stcs(q + 1, make_float4(f[4], f[5], f[6], f[7]));
    }
}

// W: elements of a unit (8: vectors, 1: any D, stride and alignment).  S: steps a warp.
// across: lanes across a row (a power of two); chunks: steps to a row.
template <bool IN16, bool OUT16, int W, int S>
__global__ void __launch_bounds__(kThreads)
embedding_kernel(const void* __restrict__ table, int64_t ld, const int32_t* __restrict__ ids, int64_t N, int64_t V,
                 uint32_t units, int across, uint32_t chunks, float scale, void* __restrict__ out, int64_t out_ld,
                 int32_t* __restrict__ status) {
    constexpr int IN = IN16 ? 2 : 4, OUT = OUT16 ? 2 : 4;
    const int lane = threadIdx.x & 31;
    const int64_t step = (int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * S;
    int64_t group = step / chunks;  // of rows
    uint32_t chunk = uint32_t(step - group * chunks);
    const int rows = 32 / across;
    int64_t row[S];
    uint32_t unit[S];
    int32_t id[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        row[s] = group * rows + lane / across;
        unit[s] = chunk * 32 + (lane & (across - 1));
        if (unit[s] >= units || row[s] >= N) row[s] = -1;
        id[s] = row[s] >= 0 ? __ldg(ids + row[s]) : -1;
        if (++chunk == chunks) {
            chunk = 0;
            ++group;
        }
    }
    Unit u[S];
#pragma unroll
    for (int s = 0; s < S; ++s) {
        u[s] = Unit{};
        if (id[s] >= 0 && id[s] < V)
            u[s] = read_unit<IN16, W>(static_cast<const char*>(table) + id[s] * (ld * IN) + unit[s] * (W * IN));
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (row[s] < 0) continue;
        // no row was read for an id that is no token: zeros times 0, or times NaN
        float by = id[s] < 0 ? 0.f : scale;
        if (id[s] >= V) {
            by = __int_as_float(0x7fc00000);
            if (status && unit[s] == 0) atomicOr(status, DF2_STATUS_ID_OUT_OF_RANGE);
        }
        write_scaled<IN16, OUT16, W>(static_cast<char*>(out) + row[s] * (out_ld * OUT) + unit[s] * (W * OUT), u[s], by);
    }
}

bool vectors(const void* p, int64_t ld, int64_t D, bool bf16) {
    return D % 8 == 0 && (ld * (bf16 ? 2 : 4)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <bool IN16, bool OUT16>
cudaError_t launch(const EmbeddingArgs& a, cudaStream_t stream) {
    const bool vec = vectors(a.table, a.ld, a.D, IN16) && vectors(a.out, a.out_ld, a.D, OUT16);
    const uint32_t units = uint32_t(vec ? a.D / 8 : a.D);
    int across = 32;
    while (across > 1 && uint32_t(across) / 2 >= units) across /= 2;
    const uint32_t chunks = (units + 31) / 32;
    const int64_t steps = (a.N + 32 / across - 1) / (32 / across) * chunks;
    // four steps a warp once that still leaves every SM 16 warps; one each for a few rows
    const bool many = steps >= int64_t(kSteps) * 16 * 152;
    const int64_t per_cta = (many ? kSteps : 1) * (kThreads / 32);
    const int64_t grid = (steps + per_cta - 1) / per_cta;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
#define DF2_EMB(W, S)                                                                                       \
    embedding_kernel<IN16, OUT16, W, S><<<unsigned(grid), kThreads, 0, stream>>>(                           \
        a.table, a.ld, a.ids, a.N, a.V, units, across, chunks, a.scale, a.out, a.out_ld, a.status)
    if (vec && many) DF2_EMB(8, kSteps);
    else if (vec) DF2_EMB(8, 1);
    else if (many) DF2_EMB(1, kSteps);
    else DF2_EMB(1, 1);
#undef DF2_EMB
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t embedding_launch(const EmbeddingArgs& a, cudaStream_t stream) {
    if (a.table_bf16) return a.out_bf16 ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
    return a.out_bf16 ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
}

}  // namespace df2
