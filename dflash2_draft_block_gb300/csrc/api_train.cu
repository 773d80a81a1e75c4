// The C-ABI of the training calls: argument validation, workspace layout and dispatch.
// Every rule checked here is stated beside the call in include/dflash2.h.
#include <cfloat>
#include <cmath>

#include "common.cuh"
#include "kernels.h"
#include "row_spans.h"

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

// One fold's scratch: the sorted pairs, their other half, the parts, the split tokens.
struct FoldSpace {
    size_t pairs, spare, parts, split, bytes;
};

FoldSpace fold_space(int64_t N, int64_t D) {
    FoldSpace s;
    s.pairs = 0;
    s.spare = round_up(df2::token_sort_bytes(N));
    s.parts = 2 * s.spare;
    s.split = s.parts + round_up(df2::fold_parts_bytes(N, D));
    s.bytes = s.split + round_up(df2::fold_split_bytes(N, D));
    return s;
}

void set_space(df2::FoldArgs* a, char* base) {
    const FoldSpace s = fold_space(a->N, a->D);
    a->pairs = reinterpret_cast<uint64_t*>(base + s.pairs);
    a->spare = reinterpret_cast<uint64_t*>(base + s.spare);
    a->parts = reinterpret_cast<float*>(base + s.parts);
    a->split = reinterpret_cast<uint32_t*>(base + s.split);
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
    a.ids = ids;
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
    a.fill = !a.accumulate;
    a.status = dev_status;
    set_space(&a, static_cast<char*>(workspace));
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (df2::fold_sort_launch(&a, 1, st) != cudaSuccess) return DF2_ERR_CUDA;
    return df2::fold_launch(&a, 1, st) == cudaSuccess ? DF2_OK : DF2_ERR_CUDA;
}

// ---------------------------------------------------------- selector loss --

namespace {

int check_loss(int64_t P, int64_t V, int K, int r) {
    if (P < 0 || V < 1 || K < 1 || r < 1 || K > V) return DF2_ERR_INVALID_ARGUMENT;
    if (K > DF2_MAX_TOPK || r > DF2_MAX_RANK || r % 8 != 0 || V > DF2_MAX_VOCAB) return DF2_ERR_UNSUPPORTED;
    if (P > kMaxPositions / K) return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

// The rows' u and G * t, then each fold's scratch.
struct LossSpace {
    size_t u, gt, fold_b, fold_a, bytes;
};

LossSpace loss_space(int64_t P, int K, int r) {
    LossSpace s;
    const size_t rows = round_up(size_t(P) * r * sizeof(float));
    s.u = 0;
    s.gt = rows;
    s.fold_b = 2 * rows;
    s.fold_a = s.fold_b + fold_space(P * K, r).bytes;
    s.bytes = s.fold_a + fold_space(P, r).bytes;
    return s;
}

}  // namespace

DF2_API size_t dflash2_selector_loss_grad_workspace_size(int64_t P, int64_t V, int K, int r) {
    if (check_loss(P, V, K, r) != DF2_OK || P == 0) return 0;
    return loss_space(P, K, r).bytes;
}

DF2_API int dflash2_selector_loss_grad(const int32_t* pred, const int32_t* targets, int64_t P, const int32_t* topk_ids,
                                       const float* topk_vals, const float* G, const uint16_t* A, const uint16_t* Bc,
                                       int64_t V, int K, int r, const float* row_weights, int accumulate, float* loss,
                                       int32_t* label_idx, float* dscores, float* dG, void* dA, void* dBc,
                                       int table_dtype, void* workspace, size_t workspace_bytes, int32_t* dev_status,
                                       void* stream) {
    const int rc = check_loss(P, V, K, r);
    if (rc != DF2_OK) return rc;
    if (!dtype_ok(table_dtype) || (dA && dA == dBc)) return DF2_ERR_INVALID_ARGUMENT;
    if (P > 0 && (!pred || !targets || !topk_ids || !topk_vals || !G || !A || !Bc || !loss || !label_idx || !dscores || !dG))
        return DF2_ERR_INVALID_ARGUMENT;
    const void* wide[] = {G, A, Bc, dG, dA, dBc, workspace};
    for (const void* p : wide)
        if (reinterpret_cast<uintptr_t>(p) & 15u) return DF2_ERR_UNSUPPORTED;
    const void* words[] = {pred, targets, topk_ids, topk_vals, row_weights, loss, label_idx, dscores};
    for (const void* p : words)
        if (!element_aligned(p, DF2_DTYPE_F32)) return DF2_ERR_UNSUPPORTED;
    const size_t need = dflash2_selector_loss_grad_workspace_size(P, V, K, r);
    if (workspace_bytes < need || (need > 0 && !workspace)) return DF2_ERR_WORKSPACE_TOO_SMALL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    char* base = static_cast<char*>(workspace);
    const LossSpace s = loss_space(P, K, r);
    float* u = reinterpret_cast<float*>(base + s.u);
    float* gt = reinterpret_cast<float*>(base + s.gt);
    df2::FoldArgs jobs[2];
    df2::ZeroArgs zero{};
    int count = 0;
    auto add = [&](void* out, const int32_t* ids, int64_t N, const float* src, size_t space) {
        if (!out) return static_cast<df2::FoldArgs*>(nullptr);
        df2::FoldArgs& f = jobs[count++] = df2::FoldArgs{};
        f.ids = ids;
        f.N = N;
        f.V = V;
        f.D = f.src_ld = f.out_ld = r;
        f.src = src;
        f.per_row = 1;
        f.scale = 1.f;
        f.out = out;
        f.out_bf16 = table_dtype == DF2_DTYPE_BF16;
        f.accumulate = accumulate != 0;
        // The rows' kernel leaves the memory bus idle and can clear a table meanwhile, but
        // does not know which rows the fold will write again: it clears a table of which
        // few rows can be written, the folds clear the others.  (16384 x 16 at rank 256: 123
        // us, 129 with both left to the folds, 125 with both cleared here; 4096 x 64 at rank
        // 512: 156, 161, 166.  Around the threshold, by this rule against both left to the
        // folds, V = 1, 3, 4 and 8 N: 4096 x 16 at rank 256, fp32 tables: 55 92 121 204, 61 97
        // 117 187; 2048 x 32, bf16: 49 60 75 116, 52 68 78 112; 1024 x 64 at rank 512, fp32: 83
        // 158 220 386, 77 148 185 325.  So where the clearing is most of the work, past the
        // threshold in fp32, the folds would be up to a fifth faster.)
        const bool beside_rows = P > 0 && 4 * N <= V;
        f.fill = !f.accumulate && !beside_rows;
        if (!f.accumulate && beside_rows) {
            zero.p[count - 1] = static_cast<char*>(out);
            zero.bytes[count - 1] = V * r * (f.out_bf16 ? 2 : 4);
        }
        set_space(&f, base + space);
        return &f;
    };
    if (df2::FoldArgs* f = add(dBc, topk_ids, P * K, u, s.fold_b)) {
        f->w = dscores;  // zero where a row was dropped
        f->per_row = uint32_t(K);
    }
    if (df2::FoldArgs* f = add(dA, pred, P, gt, s.fold_a)) f->label = label_idx;
    // the ids alone decide the sort: the rows run beside it
    if (count && P > 0 && df2::fold_sort_launch(jobs, count, st) != cudaSuccess) return DF2_ERR_CUDA;
    if (P > 0 && df2::selector_loss_launch(pred, targets, P, topk_ids, topk_vals, G, A, Bc, V, K, r, row_weights, loss,
                                           label_idx, dscores, dG, dBc ? u : nullptr, dA ? gt : nullptr, zero, dev_status,
                                           count && df2::fold_sorts(jobs, count), st) != cudaSuccess)
        return DF2_ERR_CUDA;
    if (count && df2::fold_launch(jobs, count, st) != cudaSuccess) return DF2_ERR_CUDA;
    return DF2_OK;
}

// ---------------------------------------------------------------- dropout --

namespace {

df2::RowSpan span(const void* p, int dtype, int64_t D, int64_t ld) {
    const int64_t size = dtype == DF2_DTYPE_BF16 ? 2 : 4;
    return {reinterpret_cast<uintptr_t>(p), D * size, ld * size};
}

}  // namespace

DF2_API int dflash2_dropout(const void* x, int x_dtype, int64_t N, int64_t D, int64_t x_ld, double rate, uint64_t seed,
                            uint64_t draw, const int64_t* draw_at, const void* residual, int64_t residual_ld, void* out,
                            int out_dtype, int64_t out_ld, void* stream) {
    if (!dtype_ok(x_dtype) || !dtype_ok(out_dtype) || !(rate >= 0.0 && rate <= 1.0)) return DF2_ERR_INVALID_ARGUMENT;
    if (N < 0 || D < 1) return DF2_ERR_INVALID_ARGUMENT;
    if (N > kMaxElements / D) return DF2_ERR_UNSUPPORTED;
    if (x_ld < D || out_ld < D || (residual && residual_ld < D)) return DF2_ERR_INVALID_ARGUMENT;
    if (N == 0) return DF2_OK;
    if (!x || !out) return DF2_ERR_INVALID_ARGUMENT;
    if (!element_aligned(x, x_dtype) || !element_aligned(out, out_dtype) || !element_aligned(residual, out_dtype) ||
        (reinterpret_cast<uintptr_t>(draw_at) & 7u))
        return DF2_ERR_UNSUPPORTED;
    // in place is fine (an element is read before it is written), a shifted overlap is not
    const df2::RowSpan out_span = span(out, out_dtype, D, out_ld);
    if (df2::rows_share_bytes(span(x, x_dtype, D, x_ld), out_span, N) &&
        !(x == out && x_dtype == out_dtype && (x_ld == out_ld || N == 1)))
        return DF2_ERR_INVALID_ARGUMENT;
    if (residual && df2::rows_share_bytes(span(residual, out_dtype, D, residual_ld), out_span, N) &&
        !(residual == out && (residual_ld == out_ld || N == 1)))
        return DF2_ERR_INVALID_ARGUMENT;
    const df2::DropoutArgs a{x, x_dtype == DF2_DTYPE_BF16, x_ld, N, D, uint32_t(std::floor(rate * 65536.0 + 0.5)), seed,
                             draw, draw_at, residual, residual_ld, out, out_dtype == DF2_DTYPE_BF16, out_ld};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // a draw that is an argument would be the same in every replay of a graph
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (!draw_at && cudaStreamIsCapturing(st, &capture) != cudaSuccess) return DF2_ERR_CUDA;
    if (capture != cudaStreamCaptureStatusNone) return DF2_ERR_UNSUPPORTED;
    return df2::dropout_launch(a, st) == cudaSuccess ? DF2_OK : DF2_ERR_CUDA;
}
