// dflash2_selector_loss_grad, the rows: teacher-forced scores, their K-way cross-entropy
// and every gradient of one row in one pass over its candidates' Bc rows.
//
// With a = A[pred], u = a * G and the row weight w:
//   s_j = val_j + <u, Bc[id_j]>,  loss = log sum exp(s) - s_label
//   ds_j = w * (softmax(s)_j - [j = label]),  t = sum_j ds_j Bc[id_j]
//   dG = a * t,  and for the folds into the codebooks' gradients: u (weighted by ds_j, for
//   dBc[id_j]) and G * t (for dA[pred])
//
// One CTA a row.  A group of L lanes covers r (8 columns a lane and chunk, CH chunks), and a
// lane keeps KW = 16 / CH candidates in 64 registers.  Where the CTA's warps hold the whole
// row, its values are loaded once, used for the scores and, after the softmax, again for t;
// larger rows are walked in rounds and loaded a second time for t.  Scores are summed over
// a group's lanes by halving: at every step a lane hands half of its candidates to its
// partner, so KW candidates cost about KW shuffles instead of KW * log2(L).  Products are
// packed two to an instruction.
//
// Bound: gathers from L2 and HBM (K rows of 2 r bytes each), all of a round's loads in
// flight at once, and the issue of about a thousand instructions a warp.  16,384 rows of 16
// at rank 256 take 35 us (134 MB gathered, 3.8 TB/s).  Staging the rows in shared memory
// ahead of the warps, with both contractions on mma.sync (the vectors in three bf16 parts),
// took 89 us: its loops issue more than they save and leave eight warps an SM.
//
// Gradient tables that are to be written whole may be cleared here: every CTA sends its
// share as bulk copies of zeros before its row, and the folds then write the rows of tokens
// only.  (The copies are marked to leave L2 first: as ordinary writes they drove out the
// rows that the folds read next.)
#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kMaxWarps = 8;
constexpr float kNan = __builtin_nanf("");

struct LossArgs {
    const int32_t* pred;
    const int32_t* targets;
    const int32_t* ids;
    const float* vals;
    const float* G;
    const uint16_t* A;
    const uint16_t* Bc;
    int64_t V;
    int K, r;
    const float* weights;
    float* loss;
    int32_t* label;
    float* ds;
    float* dG;
    float* u;
    float* gt;
    ZeroArgs zero;
    int64_t P;
    int32_t* status;
    bool beside;  // launched to run beside the kernel before it
};

// Two fp32 in a register pair, and two fused multiply-adds in one instruction.
__device__ __forceinline__ uint64_t pair2(float lo, float hi) {
    uint64_t d;
    asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "f"(lo), "f"(hi));
    return d;
}
__device__ __forceinline__ void split2(uint64_t d, float* lo, float* hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(*lo), "=f"(*hi) : "l"(d));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
__device__ __forceinline__ uint64_t bf16_pair(uint32_t w) { return pair2(bf16_lo(w), bf16_hi(w)); }

__device__ __forceinline__ void read8(const float* p, float f[8]) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
}

__device__ __forceinline__ void write8(float* p, const float f[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(f[4], f[5], f[6], f[7]);
}

constexpr int kZeroBytes = 4096;  // of one copy
constexpr int kZeroBlocks = 152 * 4;  // CTAs that clear, at least (where there is enough to do)

__host__ __device__ __forceinline__ int64_t zero_units(const ZeroArgs& z, int i) {
    return (z.bytes[i] + kZeroBytes - 1) / kZeroBytes;
}

// The CTA's share of the clearing, sent off by one thread; zeros: kZeroBytes of shared memory.
__device__ __forceinline__ void send_zeros(const ZeroArgs& z, float* zeros) {
    const int64_t n0 = zero_units(z, 0), n = n0 + zero_units(z, 1);
    if (n == 0) return;
    for (int i = threadIdx.x * 4; i < kZeroBytes / 4; i += blockDim.x * 4)
        *reinterpret_cast<float4*>(zeros + i) = make_float4(0.f, 0.f, 0.f, 0.f);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncthreads();
    if (threadIdx.x) return;
    const int64_t b = blockIdx.x;
    int64_t u = b * z.each + dmin<int64_t>(b, z.extra);
    for (int64_t end = u + z.each + (b < z.extra); u < end; ++u) {
        const int i = u >= n0;
        const int64_t at = (u - (i ? n0 : 0)) * kZeroBytes;
        bulk_store(z.p[i] + at, zeros, uint32_t(dmin<int64_t>(kZeroBytes, z.bytes[i] - at)));
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The end of a CTA: its copies have read their zeros; and a kernel that ran beside the one before it ends
// after it (its block 0 does), so that what follows in the stream finds both complete.
__device__ __forceinline__ void finish(const LossArgs& a) {
    if (threadIdx.x == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
    if (a.beside && blockIdx.x == 0) asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Shared memory: zeros (where there is something to clear), u [r], scores [K], t parts [warps][r], one word a warp.
constexpr size_t loss_smem(int warps, int K, int r) { return (size_t(warps + 1) * r + K + kMaxWarps) * 4; }

// L lanes a group, CH chunks of 8 columns a lane (CH > 1 only with L = 32).
template <int L, int CH>
__global__ void __launch_bounds__(kMaxWarps * 32, 2) selector_loss_kernel(const LossArgs a, int rounds) {
    constexpr int KW = 16 / CH, GROUPS = 32 / L;
    extern __shared__ float smem[];
    const int warps = blockDim.x >> 5, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int group = lane / L, gl = lane & (L - 1);
    const int64_t p = blockIdx.x;
    const bool clears = a.zero.bytes[0] + a.zero.bytes[1] > 0;
    float* su = smem + (clears ? kZeroBytes / 4 : 0);
    send_zeros(a.zero, smem);
    if (p >= a.P) {
        finish(a);
        return;
    }
    float* sc = su + a.r + (size_t(warps) * a.r);  // after the t parts
    float* st = su + a.r;
    int* sw = reinterpret_cast<int*>(sc + a.K);

    // the label's column, or none; a bad id anywhere drops the row
    const int32_t* ids = a.ids + p * a.K;
    const int32_t y = __ldg(a.targets + p), pr = __ldg(a.pred + p);
    int col = INT_MAX;
    bool bad = pr < 0 || pr >= a.V || y >= a.V;
    for (int j = threadIdx.x; j < a.K; j += blockDim.x) {
        const int32_t id = __ldg(ids + j);
        bad |= id < 0 || id >= a.V;
        if (id == y) col = min(col, j);
    }
    if (__any_sync(kFull, bad)) col = -1;
    else col = __reduce_min_sync(kFull, col);
    if (warps > 1) {
        if (lane == 0) sw[warp] = col;
        __syncthreads();
        for (int w = 0; w < warps; ++w) col = min(col, sw[w]);
    }
    if (col == -1 && threadIdx.x == 0 && a.status) atomicOr(a.status, DF2_STATUS_ID_OUT_OF_RANGE);
    bool live = col >= 0 && col < a.K;

    const float* g = a.G + p * a.r;
    const uint16_t* arow = a.A + int64_t(live ? pr : 0) * a.r;
    uint4 b[KW][CH];
    const int per_round = warps * GROUPS * KW;
    auto first_of = [&](int round) { return round * per_round + (warp * GROUPS + group) * KW; };
    // (past the last candidate or column some other value is read, and not used)
    auto gather = [&](int round) {
        const int j0 = first_of(round);
        int32_t id[KW];
#pragma unroll
        for (int k = 0; k < KW; ++k) id[k] = __ldg(ids + min(j0 + k, a.K - 1));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const int x = (c * L + gl) * 8;
            const uint16_t* col8 = a.Bc + (x < a.r ? x : 0);
#pragma unroll
            for (int k = 0; k < KW; ++k) b[k][c] = __ldg(reinterpret_cast<const uint4*>(col8 + int64_t(id[k]) * a.r));
        }
    };
    if (live) {
        gather(0);
        for (int x = threadIdx.x * 8; x < a.r; x += blockDim.x * 8) {
            float f[8], v[8];
            unpack8(__ldg(reinterpret_cast<const uint4*>(arow + x)), f);
            read8(g + x, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= f[i];
            write8(su + x, v);
            if (a.u) write8(a.u + p * a.r + x, v);
        }
        __syncthreads();
        for (int round = 0; round < rounds; ++round) {
            if (round) gather(round);
            float s[KW];
            uint64_t s2[KW];
#pragma unroll
            for (int k = 0; k < KW; ++k) s2[k] = 0;
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                const int x = (c * L + gl) * 8;
                if (x < a.r) {
                    const ulonglong2 u01 = *reinterpret_cast<const ulonglong2*>(su + x);
                    const ulonglong2 u23 = *reinterpret_cast<const ulonglong2*>(su + x + 4);
#pragma unroll
                    for (int k = 0; k < KW; ++k) {
                        s2[k] = fma2(bf16_pair(b[k][c].x), u01.x, s2[k]);
                        s2[k] = fma2(bf16_pair(b[k][c].y), u01.y, s2[k]);
                        s2[k] = fma2(bf16_pair(b[k][c].z), u23.x, s2[k]);
                        s2[k] = fma2(bf16_pair(b[k][c].w), u23.y, s2[k]);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                float lo, hi;
                split2(s2[k], &lo, &hi);
                s[k] = lo + hi;
            }
            int at = first_of(round);
            int n = KW;
#pragma unroll
            for (int o = L / 2; o; o >>= 1) {
                const bool up = lane & o;
                if (n > 1) {
                    n >>= 1;
#pragma unroll
                    for (int k = 0; k < KW / 2; ++k) {
                        if (k >= n) break;
                        const float send = up ? s[k] : s[k + n], keep = up ? s[k + n] : s[k];
                        s[k] = keep + __shfl_xor_sync(kFull, send, o);
                    }
                    at += up ? n : 0;
                } else {
                    s[0] += __shfl_xor_sync(kFull, s[0], o);
                }
            }
#pragma unroll
            for (int k = 0; k < KW; ++k)
                if (k < n && at + k < a.K) sc[at + k] = __ldg(a.vals + p * a.K + at + k) + s[k];
        }
        __syncthreads();
    }

    // softmax over the row's scores, every warp for itself
    float m = -INFINITY, sum = 0.f;
    if (live) {
        for (int j = lane; j < a.K; j += 32) m = fmaxf(m, sc[j]);
#pragma unroll
        for (int o = 16; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(kFull, m, o));
        live = m != -INFINITY;
        if (!live) {  // every candidate masked, nothing to learn; or NaN, which the maximum leaves out
            bool nan = false;
            for (int j = lane; j < a.K; j += 32) nan |= isnan(sc[j]);
            live = __any_sync(kFull, nan);
        }
        if (live) {
            for (int j = lane; j < a.K; j += 32) sum += expf(sc[j] - m);
            sum = warp_sum(sum);
        }
    }
    if (threadIdx.x == 0) {  // (before the scores give way below)
        // (the scores' difference first: next to a large m the logarithm would be rounded away)
        a.loss[p] = live ? logf(sum) + (m - sc[col]) : kNan;
        a.label[p] = live ? col : -1;
    }
    if (!live) {
        for (int j = threadIdx.x; j < a.K; j += blockDim.x) a.ds[p * a.K + j] = 0.f;
        for (int x = threadIdx.x; x < a.r; x += blockDim.x) a.dG[p * a.r + x] = 0.f;
        finish(a);
        return;
    }
    const float w = a.weights ? __ldg(a.weights + p) : 1.f, inv = 1.f / sum;
    __syncthreads();  // every warp has its maximum and sum: the scores give way to dscores
    for (int j = threadIdx.x; j < a.K; j += blockDim.x) {
        const float d = w * (expf(sc[j] - m) * inv - (j == col ? 1.f : 0.f));
        sc[j] = d;
        a.ds[p * a.K + j] = d;
    }
    __syncthreads();

    // t: a lane's columns over its candidates, then over groups, rounds and warps
    for (int round = 0; round < rounds; ++round) {
        if (rounds > 1) gather(round);
        const int j0 = first_of(round);
        float d[KW];
#pragma unroll
        for (int k = 0; k < KW; ++k) d[k] = j0 + k < a.K ? sc[j0 + k] : 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            uint64_t t2[4] = {0, 0, 0, 0};
#pragma unroll
            for (int k = 0; k < KW; ++k) {
                const uint64_t dd = pair2(d[k], d[k]);
                t2[0] = fma2(bf16_pair(b[k][c].x), dd, t2[0]);
                t2[1] = fma2(bf16_pair(b[k][c].y), dd, t2[1]);
                t2[2] = fma2(bf16_pair(b[k][c].z), dd, t2[2]);
                t2[3] = fma2(bf16_pair(b[k][c].w), dd, t2[3]);
            }
            float t[8];
#pragma unroll
            for (int i = 0; i < 4; ++i) split2(t2[i], &t[2 * i], &t[2 * i + 1]);
#pragma unroll
            for (int o = L; o < 32; o <<= 1)
#pragma unroll
                for (int i = 0; i < 8; ++i) t[i] += __shfl_xor_sync(kFull, t[i], o);
            const int x = (c * L + gl) * 8;
            if (group == 0 && x < a.r) {
                float* q = st + warp * a.r + x;
                if (round) {
                    float f[8];
                    read8(q, f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) t[i] += f[i];
                }
                write8(q, t);
            }
        }
    }
    __syncthreads();
    for (int x = threadIdx.x * 8; x < a.r; x += blockDim.x * 8) {
        float t[8], f[8], v[8];
        read8(st + x, t);
        for (int q = 1; q < warps; ++q) {
            read8(st + q * a.r + x, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) t[i] += f[i];
        }
        unpack8(__ldg(reinterpret_cast<const uint4*>(arow + x)), f);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = f[i] * t[i];
        write8(a.dG + p * a.r + x, v);
        if (a.gt) {
            read8(g + x, v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= t[i];
            write8(a.gt + p * a.r + x, v);
        }
    }
    finish(a);
}

template <int L, int CH>
cudaError_t launch(LossArgs a, int64_t P, cudaStream_t stream) {
    constexpr int per_warp = 32 / L * (16 / CH);
    // Many rows: two warps a row at most, so that rows in different phases share an SM, and
    // the second reads come from L2 (4096 rows of 64 at rank 512: 51 us, with up to four
    // warps 57, with eight 70).  Few rows: up to eight.
    const int most = P >= 152 * 4 ? 2 : kMaxWarps;
    int warps = 1;
    while (warps < most && warps * per_warp < a.K) warps *= 2;
    const int rounds = (a.K + warps * per_warp - 1) / (warps * per_warp);
    const int64_t zeros = zero_units(a.zero, 0) + zero_units(a.zero, 1);
    const size_t smem = loss_smem(warps, a.K, a.r) + (zeros ? kZeroBytes : 0);
    const int64_t blocks = dmax(P, dmin<int64_t>(zeros, kZeroBlocks));
    a.zero.each = zeros / blocks;
    a.zero.extra = zeros % blocks;
    if (smem > 48 * 1024) {
        // what the largest call of this kernel needs, whichever call asks: the allowance is the
        // kernel's, and another host thread may launch it with more meanwhile
        constexpr size_t most = loss_smem(kMaxWarps, DF2_MAX_TOPK, 8 * L * CH) + kZeroBytes;
        const cudaError_t e = cudaFuncSetAttribute(selector_loss_kernel<L, CH>,
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, int(most));
        if (e != cudaSuccess) return e;
    }
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(unsigned(blocks));
    cfg.blockDim = dim3(unsigned(warps * 32));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = a.beside ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, selector_loss_kernel<L, CH>, a, rounds);
    note_launch();
    return e;
}

}  // namespace

cudaError_t selector_loss_launch(const int32_t* pred, const int32_t* targets, int64_t P, const int32_t* ids,
                                 const float* vals, const float* G, const uint16_t* A, const uint16_t* Bc, int64_t V,
                                 int K, int r, const float* weights, float* loss, int32_t* label, float* ds, float* dG,
                                 float* u, float* gt, const ZeroArgs& zero, int32_t* status, bool beside,
                                 cudaStream_t stream) {
    const LossArgs a{pred, targets, ids, vals, G, A, Bc, V, K, r, weights, loss, label, ds, dG, u, gt, zero, P, status, beside};
    if (r <= 32) return launch<4, 1>(a, P, stream);
    if (r <= 64) return launch<8, 1>(a, P, stream);
    if (r <= 128) return launch<16, 1>(a, P, stream);
    if (r <= 256) return launch<32, 1>(a, P, stream);
    if (r <= 512) return launch<32, 2>(a, P, stream);
    if (r <= 1024) return launch<32, 4>(a, P, stream);
    if (r <= 2048) return launch<32, 8>(a, P, stream);
    return launch<32, 16>(a, P, stream);
}

}  // namespace df2
