// dflash2_embedding: out[n, :] = scale * table[ids[n], :], rounded once.
//
// Bound: HBM (a row in, a row out), or for a draft block's few rows the latency of one
// dependent load (id, then row).  Rows are cut into steps of 32 units of 8 elements (16
// bytes of bf16), several rows a step where rows are shorter; a warp takes kSteps
// consecutive steps, issues all of their loads before the first store, and divides once.
// Rows off 16-byte boundaries (odd D or strides) go element by element the same way.
// Stores are marked as streaming: what is worth keeping in L2 is the table's rows.
#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kThreads = 128;
constexpr int kSteps = 4;  // a warp, where there is enough to do

template <bool BF16>
__device__ __forceinline__ void get8(const void* p, float f[8]) {
    if (BF16) {
        unpack8(__ldg(static_cast<const uint4*>(p)), f);
    } else {
        const float4* q = static_cast<const float4*>(p);
        const float4 a = __ldg(q), b = __ldg(q + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}

template <bool BF16>
__device__ __forceinline__ void put8(void* p, const float f[8]) {
    if (BF16) {
        __stcs(static_cast<uint4*>(p), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                                  pack_bf16(f[6], f[7])));
    } else {
        float4* q = static_cast<float4*>(p);
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
        id[s] = -1;
        if (row[s] < N && unit[s] < units) id[s] = __ldg(ids + row[s]);
        else row[s] = -1;
        if (++chunk == chunks) {
            chunk = 0;
            ++group;
        }
    }
    float f[S][W];
#pragma unroll
    for (int s = 0; s < S; ++s) {
#pragma unroll
        for (int i = 0; i < W; ++i) f[s][i] = 0.f;
        if (id[s] >= 0 && id[s] < V) {
            const char* src = static_cast<const char*>(table) + (id[s] * ld + unit[s] * W) * IN;
            if (W == 8) get8<IN16>(src, f[s]);
            else f[s][0] = IN16 ? bf16_to_f32(__ldg(reinterpret_cast<const uint16_t*>(src)))
                                : __ldg(reinterpret_cast<const float*>(src));
        }
    }
#pragma unroll
    for (int s = 0; s < S; ++s) {
        if (row[s] < 0) continue;
        if (id[s] >= V) {
#pragma unroll
            for (int i = 0; i < W; ++i) f[s][i] = __int_as_float(0x7fc00000);
            if (status && unit[s] == 0) atomicOr(status, DF2_STATUS_ID_OUT_OF_RANGE);
        }
        char* dst = static_cast<char*>(out) + (row[s] * out_ld + unit[s] * W) * OUT;
#pragma unroll
        for (int i = 0; i < W; ++i) f[s][i] = id[s] < 0 ? 0.f : __fmul_rn(f[s][i], scale);
        if (W == 8) put8<OUT16>(dst, f[s]);
        else if (OUT16) *reinterpret_cast<uint16_t*>(dst) = f32_to_bf16_rn(f[s][0]);
        else *reinterpret_cast<float*>(dst) = f[s][0];
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
