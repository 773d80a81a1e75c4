// dflash2_embedding: out[n, :] = scale * table[ids[n], :], rounded once.
//
// Bound: HBM (a row in, a row out), or for a draft block's few rows the latency of one
// dependent load (id, then row).  Rows are cut into units of 8 elements (16 bytes of
// bf16) numbered in output order; a CTA takes a contiguous run of units, so its stores
// are one contiguous piece whatever D is, and a thread issues kUnits rows' loads before
// it converts the first.  Rows off 16-byte boundaries (odd D or strides) go element by
// element through the same numbering.
#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kThreads = 256;

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
        *static_cast<uint4*>(p) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                                             pack_bf16(f[6], f[7]));
    } else {
        float4* q = static_cast<float4*>(p);
        q[0] = make_float4(f[0], f[1], f[2], f[3]);
        q[1] = make_float4(f[4], f[5], f[6], f[7]);
    }
}

// W: elements of a unit (8: vectors, 1: any D, stride and alignment).  U: units a thread.
template <bool IN16, bool OUT16, int W, int U>
__global__ void __launch_bounds__(kThreads)
embedding_kernel(const void* __restrict__ table, int64_t ld, const int32_t* __restrict__ ids, int64_t N, int64_t V,
                 uint32_t per_row, float scale, void* __restrict__ out, int64_t out_ld, int32_t* __restrict__ status) {
    constexpr int IN = IN16 ? 2 : 4, OUT = OUT16 ? 2 : 4;
    const int64_t first = int64_t(blockIdx.x) * (kThreads * U);
    const int64_t row0 = first / per_row;
    const uint32_t rem = uint32_t(first - row0 * per_row);
    int64_t row[U];
    uint32_t col[U];
    int32_t id[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t k = rem + threadIdx.x + u * kThreads;
        const uint32_t dr = k / per_row;
        row[u] = row0 + dr;
        col[u] = (k - dr * per_row) * W;
        id[u] = row[u] < N ? __ldg(ids + row[u]) : -1;
    }
    float f[U][W];
#pragma unroll
    for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < W; ++i) f[u][i] = 0.f;
        if (id[u] >= 0 && id[u] < V) {
            const char* src = static_cast<const char*>(table) + (int64_t(id[u]) * ld + col[u]) * IN;
            if (W == 8) get8<IN16>(src, f[u]);
            else f[u][0] = IN16 ? bf16_to_f32(__ldg(reinterpret_cast<const uint16_t*>(src)))
                                : __ldg(reinterpret_cast<const float*>(src));
        } else if (id[u] >= V) {
#pragma unroll
            for (int i = 0; i < W; ++i) f[u][i] = __int_as_float(0x7fc00000);
            if (status && col[u] == 0) atomicOr(status, DF2_STATUS_ID_OUT_OF_RANGE);
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        if (row[u] >= N) continue;
        char* dst = static_cast<char*>(out) + (row[u] * out_ld + col[u]) * OUT;
#pragma unroll
        for (int i = 0; i < W; ++i) f[u][i] = id[u] < 0 ? 0.f : __fmul_rn(f[u][i], scale);
        if (W == 8) put8<OUT16>(dst, f[u]);
        else if (OUT16) *reinterpret_cast<uint16_t*>(dst) = f32_to_bf16_rn(f[u][0]);
        else *reinterpret_cast<float*>(dst) = f[u][0];
    }
}

bool vectors(const void* p, int64_t ld, int64_t D, bool bf16) {
    return D % 8 == 0 && (ld * (bf16 ? 2 : 4)) % 16 == 0 && (reinterpret_cast<uintptr_t>(p) & 15) == 0;
}

template <bool IN16, bool OUT16>
cudaError_t launch(const EmbeddingArgs& a, cudaStream_t stream) {
    const bool vec = vectors(a.table, a.ld, a.D, IN16) && vectors(a.out, a.out_ld, a.D, OUT16);
    const uint32_t per_row = uint32_t(vec ? a.D / 8 : a.D);
    const int64_t units = a.N * per_row;
    // four units a thread once that still leaves every SM a CTA; one each for a few rows
    const bool many = units >= int64_t(kThreads) * 4 * 152;
    const int64_t grid = (units + kThreads * (many ? 4 : 1) - 1) / (kThreads * (many ? 4 : 1));
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
#define DF2_EMB(W, U)                                                                                       \
    embedding_kernel<IN16, OUT16, W, U><<<unsigned(grid), kThreads, 0, stream>>>(                           \
        a.table, a.ld, a.ids, a.N, a.V, per_row, a.scale, a.out, a.out_ld, a.status)
    if (vec && many) DF2_EMB(8, 4);
    else if (vec) DF2_EMB(8, 1);
    else if (many) DF2_EMB(1, 4);
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
