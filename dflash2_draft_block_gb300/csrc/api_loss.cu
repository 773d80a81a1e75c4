// The C-ABI of the unary loss: argument validation, workspace layout and dispatch.
// Every rule checked here is stated beside the calls in include/dflash2.h.
#include <cfloat>

#include "common.cuh"
#include "kernels.h"

namespace {

// Positions a call: the blocks that put the rows with a target in order, 4,096 of them at most, each
// count the ones before them, P / 2 on average: 2,048 P reads (8 GB of L2, some ms, at 2^20).
constexpr int64_t kMaxRows = int64_t(1) << 20;
constexpr int64_t kMaxVocab = int64_t(1) << 24;
constexpr int64_t kMaxHidden = int64_t(1) << 20;
// what a piece of rows may take: factors of 16 bits (the gradients), or statistics (the loss
// alone).  Larger pieces read W fewer times; at 151,936 columns this is 14,080 rows.
constexpr int64_t kPieceBytes = int64_t(4) << 30;
constexpr int64_t kPieceStats = int64_t(1) << 30;

int64_t up(int64_t n, int64_t by) { return (n + by - 1) / by * by; }

int num_sms_current() {
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return 0;
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 0;
    return n;
}

int check_shape(int64_t P, int64_t D, int64_t V) {
    if (P < 0 || D < 1 || V < 1) return DF2_ERR_INVALID_ARGUMENT;
    if (D % 8 != 0 || P > kMaxRows || D > kMaxHidden || V > kMaxVocab) return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

// How a call is cut, and where its workspace holds what (byte offsets).
struct Plan {
    int64_t h_rows;      // live rows' copy, a multiple of 64
    int64_t rows;        // of a piece
    int64_t pieces;
    int64_t e_rows, e_ld;
    int n_stats;
    size_t count, map, targets, target_logit, target_slope, h, stats, e, part, sums, bytes;
};

Plan make_plan(int64_t P, int64_t D, int64_t V, bool dh, bool dw, int num_sms) {
    Plan p{};
    const bool grads = dh || dw;
    p.h_rows = up(P, 64);
    p.n_stats = int(up(V, 256) / df2::kLossStats);
    p.e_ld = up(V, 256);
    const int64_t row_bytes = grads ? p.e_ld * 2 : int64_t(p.n_stats) * 8;
    int64_t most = (grads ? kPieceBytes : kPieceStats) / row_bytes / 256 * 256;
    if (most < 256) most = 256;
    p.pieces = (P + most - 1) / most;
    p.rows = up((P + p.pieces - 1) / p.pieces, 256);
    if (p.rows > P) p.rows = P;
    p.e_rows = up(p.rows, 64);
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t here = at;
        at += size_t(up(int64_t(bytes), 256));
        return here;
    };
    p.count = take(4);
    p.map = take(size_t(P) * 4);
    p.targets = take(size_t(P) * 4);
    p.target_logit = take(size_t(P) * 4);
    p.target_slope = take(grads ? size_t(P) * 4 : 0);
    p.h = take(size_t(p.h_rows) * D * 2);
    p.stats = take(size_t(p.rows) * p.n_stats * 8);
    p.e = take(grads ? size_t(p.e_rows) * p.e_ld * 2 : 0);
    // parts of 256 x 256 sums: a cluster's share of them, or all that there can be
    const int64_t ways = dh ? df2::loss_way_limit((V + 63) / 64) : 1;
    const int64_t some = df2::kLossPartTiles * (num_sms / 2), all = up(p.rows, 256) / 256 * (up(D, 512) / 256) * ways;
    p.part = take(ways > 1 ? size_t(some < all ? some : all) * 65536 * 4 : 0);
    p.sums = take(dw && p.pieces > 1 ? size_t(V) * D * 4 : 0);
    p.bytes = at;
    return p;
}

bool dtype_ok(int d) { return d == DF2_DTYPE_BF16 || d == DF2_DTYPE_F32; }
size_t size_of(int dtype) { return dtype == DF2_DTYPE_BF16 ? 2 : 4; }

struct Span {
    const void* p;
    size_t bytes;
};

bool overlap(const Span& a, const Span& b) {
    if (!a.p || !b.p) return false;
    const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
    return x < y + b.bytes && y < x + a.bytes;
}

struct Call {
    const uint16_t* h;
    int64_t P, D;
    const uint16_t* W;
    int64_t V;
    df2::LogitMap lm;
    const int32_t* targets;
    const float* weights;
    float* loss;
    float* lse;
    void* dh;
    int dh_dtype;
    void* dw;
    int dw_dtype;
    bool accumulate;
    char* ws;
    int32_t* status;
    cudaStream_t stream;
};

cudaError_t run(const Call& c, const Plan& p, int num_sms) {
    const bool grads = c.dh || c.dw;
    df2::LossRowsArgs rows{};
    rows.targets = c.targets;
    rows.P = c.P;
    rows.V = c.V;
    rows.D = c.D;
    rows.h = c.h;
    rows.live_h = reinterpret_cast<uint16_t*>(c.ws + p.h);
    rows.live_targets = reinterpret_cast<int32_t*>(c.ws + p.targets);
    rows.map = reinterpret_cast<int32_t*>(c.ws + p.map);
    rows.count = reinterpret_cast<int32_t*>(c.ws + p.count);
    rows.loss = c.loss;
    rows.lse = c.lse;
    rows.dh = c.dh;
    rows.dh_bf16 = c.dh_dtype == DF2_DTYPE_BF16;
    rows.status = c.status;
    cudaError_t e = df2::loss_rows_launch(rows, c.stream);
    for (int64_t i = 0; i < p.pieces && e == cudaSuccess; ++i) {
        df2::LossGemmArgs g{};
        g.count = rows.count;
        g.row0 = i * p.rows;
        g.rows = int(c.P - g.row0 < p.rows ? c.P - g.row0 : p.rows);
        g.V = c.V;
        g.D = c.D;
        g.map = rows.map;
        g.status = c.status;
        g.targets = rows.live_targets;
        g.target_logit = reinterpret_cast<float*>(c.ws + p.target_logit);
        g.target_slope = reinterpret_cast<float*>(c.ws + p.target_slope);
        g.stats = reinterpret_cast<float2*>(c.ws + p.stats);
        g.n_stats = p.n_stats;
        g.lm = c.lm;
        g.e = grads ? reinterpret_cast<uint16_t*>(c.ws + p.e) : nullptr;
        g.e_ld = p.e_ld;
        e = df2::loss_logits_launch(g, rows.live_h, p.h_rows, c.W, num_sms, c.stream);
        if (e != cudaSuccess) break;
        const df2::LossRowArgs r{g.count, g.row0, g.rows, c.V, g.stats, g.n_stats, g.target_logit, g.target_slope, g.targets, g.map,
                                 c.weights, c.lm, c.loss, c.lse, g.e, g.e_ld};
        e = df2::loss_row_launch(r, p.e_rows, num_sms, c.stream);
        if (e != cudaSuccess) break;
        if (c.dh) {
            g.out = c.dh;
            g.out_bf16 = rows.dh_bf16;
            g.part = reinterpret_cast<float*>(c.ws + p.part);
            df2::LossDhGrid grid{};
            e = df2::loss_dh_launch(g, p.e_rows, c.W, num_sms, &grid, c.stream);
            if (e == cudaSuccess && df2::loss_way_limit((c.V + 63) / 64) > 1)
                e = df2::loss_sum_parts_launch(g, grid, c.stream);
            if (e != cudaSuccess) break;
        }
        if (c.dw) {
            g.out = c.dw;
            g.out_bf16 = c.dw_dtype == DF2_DTYPE_BF16;
            g.sums = p.pieces > 1 ? reinterpret_cast<float*>(c.ws + p.sums) : nullptr;
            g.first = i == 0;
            g.last = i + 1 == p.pieces;
            g.accumulate = c.accumulate;
            e = df2::loss_dw_launch(g, p.e_rows, rows.live_h, p.h_rows, num_sms, c.stream);
        }
    }
    return e;
}

int call(Call c, float multiplier, float cap, void* workspace, size_t workspace_bytes) {
    const int rc = check_shape(c.P, c.D, c.V);
    if (rc != DF2_OK) return rc;
    if (!(multiplier > 0.f) || !(multiplier <= FLT_MAX) || !(cap >= 0.f) || !(cap <= FLT_MAX)) return DF2_ERR_INVALID_ARGUMENT;
    // m / c is a factor of its own: neither infinite nor short of bits
    if (cap > 0.f && !(1.f / cap <= FLT_MAX && multiplier / cap <= FLT_MAX && multiplier / cap >= FLT_MIN))
        return DF2_ERR_UNSUPPORTED;
    // exp's argument is taken from the raw difference times log2(e) m (loss_gemm.cu)
    if (cap == 0.f && !(1.4426950408889634f * multiplier <= FLT_MAX)) return DF2_ERR_UNSUPPORTED;
    c.lm.mul = multiplier;
    c.lm.cap = cap;
    if (c.P > 0 && (!c.h || !c.W || !c.targets || !c.loss)) return DF2_ERR_INVALID_ARGUMENT;
    for (const void* p : {static_cast<const void*>(c.h), static_cast<const void*>(c.W), static_cast<const void*>(c.dh),
                          static_cast<const void*>(c.dw)})
        if (reinterpret_cast<uintptr_t>(p) & 15u) return DF2_ERR_UNSUPPORTED;
    for (const void* p : {static_cast<const void*>(c.targets), static_cast<const void*>(c.weights),
                          static_cast<const void*>(c.loss), static_cast<const void*>(c.lse)})
        if (reinterpret_cast<uintptr_t>(p) & 3u) return DF2_ERR_UNSUPPORTED;
    if (c.P == 0) {
        if (c.dw && !c.accumulate &&
            cudaMemsetAsync(c.dw, 0, size_t(c.V) * c.D * size_of(c.dw_dtype), c.stream) != cudaSuccess)
            return DF2_ERR_CUDA;
        return DF2_OK;
    }
    const size_t words = size_t(c.P) * 4;
    const Span in[] = {{c.h, size_t(c.P) * c.D * 2}, {c.W, size_t(c.V) * c.D * 2}, {c.targets, words}, {c.weights, words}};
    const Span out[] = {{c.dh, size_t(c.P) * c.D * size_of(c.dh_dtype)}, {c.dw, size_t(c.V) * c.D * size_of(c.dw_dtype)},
                        {c.loss, words}, {c.lse, words}};
    for (int i = 0; i < 4; ++i) {
        for (const Span& s : in)
            if (overlap(out[i], s)) return DF2_ERR_INVALID_ARGUMENT;
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return DF2_ERR_INVALID_ARGUMENT;
    }
    const int sms = num_sms_current();
    if (sms < 2) return DF2_ERR_CUDA;
    const Plan p = make_plan(c.P, c.D, c.V, c.dh, c.dw, sms);
    if (workspace_bytes < p.bytes || !workspace) return DF2_ERR_WORKSPACE_TOO_SMALL;
    if (reinterpret_cast<uintptr_t>(workspace) & 255u) return DF2_ERR_UNSUPPORTED;
    c.ws = static_cast<char*>(workspace);
    return run(c, p, sms) == cudaSuccess ? DF2_OK : DF2_ERR_CUDA;
}

size_t workspace_size(int64_t P, int64_t D, int64_t V, bool dh, bool dw) {
    if (check_shape(P, D, V) != DF2_OK || P == 0) return 0;
    const int sms = num_sms_current();
    return make_plan(P, D, V, dh, dw, sms < 2 ? 152 : sms).bytes;
}

}  // namespace

DF2_API size_t dflash2_unary_ce_workspace_size(int64_t P, int64_t D, int64_t V) {
    return workspace_size(P, D, V, false, false);
}

DF2_API int dflash2_unary_ce(const uint16_t* h, int64_t P, int64_t D, const uint16_t* W_lm, int64_t V,
                             float output_multiplier, float final_logit_softcapping, const int32_t* targets, float* loss,
                             float* lse, void* workspace, size_t workspace_bytes, int32_t* dev_status, void* stream) {
    Call c{h, P, D, W_lm, V, {}, targets, nullptr, loss, lse, nullptr, DF2_DTYPE_F32, nullptr, DF2_DTYPE_F32, false,
           nullptr, dev_status, static_cast<cudaStream_t>(stream)};
    return call(c, output_multiplier, final_logit_softcapping, workspace, workspace_bytes);
}

DF2_API size_t dflash2_unary_loss_grad_workspace_size(int64_t P, int64_t D, int64_t V, int dh, int dW) {
    return workspace_size(P, D, V, dh != 0, dW != 0);
}

DF2_API int dflash2_unary_loss_grad(const uint16_t* h, int64_t P, int64_t D, const uint16_t* W_lm, int64_t V,
                                    float output_multiplier, float final_logit_softcapping, const int32_t* targets,
                                    const float* row_weights, int accumulate, float* loss, float* lse, void* dh,
                                    int dh_dtype, void* dW, int dW_dtype, void* workspace, size_t workspace_bytes,
                                    int32_t* dev_status, void* stream) {
    if ((dh && !dtype_ok(dh_dtype)) || (dW && !dtype_ok(dW_dtype))) return DF2_ERR_INVALID_ARGUMENT;
    Call c{h, P, D, W_lm, V, {}, targets, row_weights, loss, lse, dh, dh_dtype, dW, dW_dtype, accumulate != 0,
           nullptr, dev_status, static_cast<cudaStream_t>(stream)};
    return call(c, output_multiplier, final_logit_softcapping, workspace, workspace_bytes);
}
