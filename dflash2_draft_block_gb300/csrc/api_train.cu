// The C-ABI of the training calls: argument validation, workspace layout and dispatch.
// Every rule checked here is stated beside the call in include/dflash2.h.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace {

bool dtype_ok(int d) { return d == DF2_DTYPE_BF16 || d == DF2_DTYPE_F32; }

bool element_aligned(const void* p, int dtype) {
    return (reinterpret_cast<uintptr_t>(p) & (dtype == DF2_DTYPE_BF16 ? 1u : 3u)) == 0;
}

bool finite(float x) { return x >= -FLT_MAX && x <= FLT_MAX; }

size_t round_up(size_t n) { return (n + 255) / 256 * 256; }

constexpr int64_t kMaxPositions = INT32_MAX;
constexpr int64_t kMaxColumns = int64_t(1) << 24;
constexpr int64_t kMaxElements = int64_t(1) << 40;

int check_rows(int64_t N, int64_t V, int64_t D) {
    if (N < 0 || V < 1 || D < 1) return DF2_ERR_INVALID_ARGUMENT;
    if (V > DF2_MAX_VOCAB || N > kMaxPositions || D > kMaxColumns || N * D > kMaxElements) return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

// One fold's scratch: the sorted pairs, their other half, the parts.
struct FoldSpace {
    size_t pairs, spare, parts, bytes;
};

FoldSpace fold_space(int64_t N, int64_t D) {
    FoldSpace s;
    s.pairs = 0;
    s.spare = round_up(df2::token_sort_bytes(N));
    s.parts = 2 * s.spare;
    s.bytes = s.parts + round_up(df2::fold_parts_bytes(N, D));
    return s;
}

// Sorts the ids into the scratch at base and folds (a's tensors and sizes are set).
cudaError_t sort_and_fold(df2::FoldArgs a, const int32_t* ids, const int32_t* label, uint32_t per_label, char* base,
                          int32_t* status, cudaStream_t stream) {
    const FoldSpace s = fold_space(a.N, a.D);
    if (a.N > 0) {
        df2::SortJob j{ids, a.N, uint32_t(a.V), label, per_label, reinterpret_cast<uint64_t*>(base + s.pairs),
                       reinterpret_cast<uint64_t*>(base + s.spare), status};
        const cudaError_t e = df2::token_sort_launch(j, stream);
        if (e != cudaSuccess) return e;
    }
    a.pairs = reinterpret_cast<const uint64_t*>(base + s.pairs);
    a.parts = reinterpret_cast<float*>(base + s.parts);
    return df2::fold_launch(a, stream);
}

}  // namespace

// -------------------------------------------------------------- embedding --

DF2_API int dflash2_embedding(const void* table, int table_dtype, int64_t V, int64_t D, int64_t table_ld,
                              const int32_t* ids, int64_t N, float scale, void* out, int out_dtype, int64_t out_ld,
                              int32_t* dev_status, void* stream) {
    if (!dtype_ok(table_dtype) || !dtype_ok(out_dtype) || !finite(scale)) return DF2_ERR_INVALID_ARGUMENT;
    const int rc = check_rows(N, V, D);
    if (rc != DF2_OK) return rc;
    if (table_ld < D || out_ld < D) return DF2_ERR_INVALID_ARGUMENT;
    if (N == 0) return DF2_OK;
    if (!table || !ids || !out) return DF2_ERR_INVALID_ARGUMENT;
    if (!element_aligned(table, table_dtype) || !element_aligned(out, out_dtype) || !element_aligned(ids, DF2_DTYPE_F32))
        return DF2_ERR_UNSUPPORTED;
    const df2::EmbeddingArgs a{table, table_dtype == DF2_DTYPE_BF16, table_ld, V, D, ids, N, scale, out,
                               out_dtype == DF2_DTYPE_BF16, out_ld, dev_status};
    return df2::embedding_launch(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DF2_OK : DF2_ERR_CUDA;
}

DF2_API size_t dflash2_embedding_grad_workspace_size(int64_t N, int64_t V, int64_t D) {
    if (check_rows(N, V, D) != DF2_OK || N == 0) return 0;
    return fold_space(N, D).bytes;
}

DF2_API int dflash2_embedding_grad(const void* dout, int dout_dtype, int64_t dout_ld, const int32_t* ids, int64_t N,
                                   int64_t V, int64_t D, float scale, int accumulate, void* dtable, int dtable_dtype,
                                   int64_t dtable_ld, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                   void* stream) {
    if (!dtype_ok(dout_dtype) || !dtype_ok(dtable_dtype) || !finite(scale)) return DF2_ERR_INVALID_ARGUMENT;
    const int rc = check_rows(N, V, D);
    if (rc != DF2_OK) return rc;
    if (dout_ld < D || dtable_ld < D) return DF2_ERR_INVALID_ARGUMENT;
    if (N == 0 && accumulate) return DF2_OK;
    if (!dtable || (N > 0 && (!dout || !ids))) return DF2_ERR_INVALID_ARGUMENT;
    if (!element_aligned(dout, dout_dtype) || !element_aligned(dtable, dtable_dtype) ||
        !element_aligned(ids, DF2_DTYPE_F32) || (reinterpret_cast<uintptr_t>(workspace) & 15u))
        return DF2_ERR_UNSUPPORTED;
    const size_t need = dflash2_embedding_grad_workspace_size(N, V, D);
    if (workspace_bytes < need || (need > 0 && !workspace)) return DF2_ERR_WORKSPACE_TOO_SMALL;
    df2::FoldArgs a{};
    a.N = N;
    a.V = V;
    a.D = D;
    a.src = dout;
    a.src_bf16 = dout_dtype == DF2_DTYPE_BF16;
    a.src_ld = dout_ld;
    a.per_row = 1;
    a.scale = scale;
    a.out = dtable;
    a.out_bf16 = dtable_dtype == DF2_DTYPE_BF16;
    a.out_ld = dtable_ld;
    a.accumulate = accumulate != 0;
    return sort_and_fold(a, ids, nullptr, 1, static_cast<char*>(workspace), dev_status,
                         static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? DF2_OK
               : DF2_ERR_CUDA;
}
