// The matrix products of the unary loss on the tensor cores, CTA pairs on 256 x 256 tiles
// (tcgen05.mma.cta_group::2, bf16 in, fp32 sums), with three epilogues:
//   LOGITS  u = h W^T, never stored: of each row's 64 columns the largest logit M and the sum
//           of exp(u - M) over the columns other than the target's, and the target's logit.
//           With `e`, also exp(u - M) itself (times the softcap's slope) as fp16.
//   DH      dh = g W:    A = g (K-major: its rows run along K = V), B = W, MN-major
//   DW      dW = g^T h:  A = g, B = h, both MN-major (K = rows)
// An MN-major operand is staged as panels of 64 M (or N) elements by 64 K rows, as TMA's
// 128-byte swizzle writes a 64-element wide box: within a panel 8 K rows are 1024 bytes (the
// descriptor's stride offset), panels follow each other (its leading offset), and 16 K
// elements on are 2048 bytes.
//
// Sums in pieces.  The tensor core cuts each partial sum off below its last bit instead of
// rounding it, so a sum of n steps drifts towards zero by about n / 4 ulp: a logit of 4096
// products came out 4e-6 of itself too small, which a loss would show.  The MMAs
// therefore sum 1024 K elements at a time (dh and dW, whose factors have 8 bits: 4096) into one of
// two TMEM accumulators while the epilogue warps add the other to running sums in fp32 registers (64
// columns a thread, sixteen warps), rounded to nearest.  dW of up to 4096 rows is one such sum and
// goes out as it lies in TMEM; of more rows it is added up like the others (DW_LONG: one sum of 2^20
// rows came out 6e-3 too small).
//
// Roles (640 threads): warp 0 lane 0 issues the TMA loads, warp 1 lane 0 the MMAs, warps 4-19
// are the epilogue (TMEM lane = row; four warps a quarter, 64 columns each).  Tiles are
// dealt round-robin to the clusters.  Rows without a target were left out beforehand, so the
// number of rows is read from the device.  All waits are bounded.
//
// Bound: the tensor cores with many rows (4096 x 151,936 x 4096: logits with e 2.74 ms, dh 2.78,
// dW 2.57, 1.84 to 1.98 PFLOP/s by themselves; under the power limit 1.6 together); HBM with few
// (8 rows: 192 us, 6.5 TB/s); the epilogues where K is short (4096 x 32,000 x 128: logits 100 us).
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>

#include "common.cuh"
#include "kernels.h"
#include "tc_pair.cuh"
#include "tc_ptx.cuh"

namespace df2 {
namespace {

constexpr int kThreads = 640;
// Registers: launched with 96 a thread; the first four warps keep 32 and the epilogue's sixteen
// take 112 (128 * 32 + 512 * 112 = 640 * 96): what they spill goes to L2, the ring has the rest.
constexpr int kRoleRegisters = 32, kEpilogueRegisters = 112;
constexpr int kCols = kLossStats;              // columns of an epilogue thread
constexpr int kTile = 256;
constexpr int kStep = 64;                      // K elements a stage
constexpr uint32_t kOperand = 128 * kStep * 2;  // bytes a stage and CTA of one operand
constexpr int kSegment = 16;                   // stages to a partial sum of the logits (1024 K elements)
constexpr int kLongSegment = 64;               // of dh (1%: 16) and of dW
constexpr int kStagedSteps = 32;               // dW's sums of up to 64 times this many rows go out staged
constexpr uint32_t kStaging = 4096;            // bytes of an epilogue warp: 128 of each of its 32 rows
__host__ __device__ constexpr int stages(bool staged) { return staged ? 5 : 7; }
__host__ __device__ constexpr uint32_t smem_bytes(bool staged) {
    return stages(staged) * 2 * kOperand + (staged ? 16 * kStaging : 0) + (2 * stages(staged) + 5 + 16) * 8 + 16 + 1024;
}

enum { LOGITS, DH, DW, DW_LONG };

struct Work {
    LossGemmArgs a;
    int n_nt;
};

// K-major as tc::sw128_kmajor_desc; MN-major: panels kStep * 128 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool mn) {
    uint64_t d = tc::sw128_kmajor_desc(addr);
    if (mn) d = (d & ~(uint64_t(0x3FFF) << 16)) | (uint64_t(kStep * 128 >> 4) << 16);
    return d;
}

// This warp has read its part of an accumulator (its loads are complete): an arrive that orders
// nothing else.  One with release would wait until the rows stored before are in memory.
__device__ __forceinline__ void accumulator_read(uint64_t* bar, uint32_t lead) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(
                     tc::mapa_shared(tc::smem_u32(bar), lead))
                 : "memory");
}

// 32 lanes x 32 consecutive columns, ready on return.
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, float v[32]) {
    uint32_t r[32];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
        "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];\n\t"
        "tcgen05.wait::ld.sync.aligned;"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(r[i]);
}

constexpr float kLog2e = 1.4426950408889634f;

// Two fp32 to a word of two fp16 (lo in the low half), to nearest even.
__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(hi), "f"(lo));
    return w;
}

// The two halves of the x held by a thread change places: a loop over 32 columns at a time that
// keeps x in registers.  (All of a row's columns unrolled were thousands of instructions, read
// anew for every tile.)
__device__ __forceinline__ void turn(float (&x)[kCols]) {
#pragma unroll
    for (int j = 0; j < 32; ++j) {
        const float first = x[j];
        x[j] = x[j + 32];
        x[j + 32] = first;
    }
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// r = 1 / (exp(2 |y|) + 1), of which both tanh and its slope are made: |tanh y| = 1 - 2 r, and
// 1 - tanh^2 y = 4 r (1 - r), which keeps its bits where tanh is all but 1 (1 - tanh^2 itself is off
// by 3% at y = 7, and by 20% at 8).
__device__ __forceinline__ float tanh_gap(float y) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(exp2_fast(fabsf(y) * (2.f * kLog2e)) + 1.f));
    return r;
}
// `scale` times the slope.
__device__ __forceinline__ float tanh_slope(float r, float scale) {
    const float s = 4.f * scale * r;
    return fmaf(-s, r, s);
}

// cap * tanh(y), to about 2^-21 of it: 1 - 2 r, and where that would cancel the series
// y - y^3/3 + 2 y^5/15 - 17 y^7/315 + 62 y^9/2835.
__device__ __forceinline__ float bend(float y, float r, float cap) {
    const float wide = copysignf(fmaf(-2.f, r, 1.f), y);
    const float q = y * y;
    float s = fmaf(q, 0.021869488536155203f, -0.053968253968253970f);
    s = fmaf(q, s, 0.13333333333333333f);
    s = fmaf(q, s, -0.33333333333333333f);
    const float near = fmaf(y * q, s, y);
    return __fmul_rn(cap, fabsf(y) < 0.25f ? near : wide);
}

// 16 elements of bf16 or fp16, or 8 of fp32; `wide` (uniform): p is 32-byte aligned.
__device__ __forceinline__ void store8(void* p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(w[0]), "r"(w[1]),
                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        uint4* q = static_cast<uint4*>(p);
        q[0] = make_uint4(w[0], w[1], w[2], w[3]);
        q[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// One row's 64 logits of a tile (x, raw): the statistics, and e where asked, with a cap times its
// slope, in fp16 in units of 2^-15 (11 bits down to 2^-29, that is exp(x - M) at M - 20, then fewer
// until 2^-40; bf16 here and again as g would double the factors' rounding error).
template <bool E, bool CAP>
__device__ __forceinline__ void logits_epilogue(const LossGemmArgs& a, float (&x)[kCols], int row, int target, int nt,
                                                int part) {
    const int64_t c0 = int64_t(nt) * kTile + part * kCols;
    const int64_t t = target - c0;
    const float cap = a.lm.cap, mul = CAP ? a.lm.mul / cap : a.lm.mul;
    // Non-decreasing.  Rounded as written, so that the loss is the same with e and without.
    auto map = [&](float u) {
        const float y = __fmul_rn(u, mul);
        return CAP ? bend(y, tanh_gap(y), cap) : y;
    };
    // The columns left out, the target and what is no column: as bits, and in x below any logit.  (Not
    // by that value afterwards: a logit may be -infinity itself, which a cap makes -cap.)
    uint32_t out_lo = 0u, out_hi = 0u;
    if ((t >= 0 && t < kCols) || c0 + kCols > a.V) {
        const int end = c0 >= a.V ? 0 : c0 + kCols > a.V ? int(a.V - c0) : kCols;
        if (CAP) {
            uint64_t out = end < kCols ? ~uint64_t(0) << end : 0u;
            if (t >= 0 && t < kCols) out |= uint64_t(1) << t;
            out_lo = uint32_t(out);
            out_hi = uint32_t(out >> 32);
        }
        float xt = 0.f;
#pragma unroll 1
        for (int c = 0; c < kCols; c += 32) {
#pragma unroll
            for (int j = 0; j < 32; ++j) {
                if (c + j == t) xt = x[j];
                if (c + j == t || c + j >= end) x[j] = -INFINITY;
            }
            turn(x);
        }
        if (t >= 0 && t < kCols) {
            a.target_logit[a.row0 + row] = map(xt);
            if (E && CAP) a.target_slope[a.row0 + row] = tanh_slope(tanh_gap(__fmul_rn(xt, mul)), 1.f);
        }
    }
    float top = -INFINITY;
#pragma unroll
    for (int j = 0; j < kCols; ++j) top = fmaxf(top, x[j]);
    const bool none = CAP ? (out_lo & out_hi) == 0xFFFFFFFFu : top == -INFINITY;
    // x - M in the units of the logits as they are mapped: without a cap the multiplier waits
    const float base = none ? 0.f : CAP ? map(top) : top;
    const float by = CAP ? kLog2e : __fmul_rn(kLog2e, mul);
    float sum[4] = {0.f, 0.f, 0.f, 0.f};
    uint16_t* out = E ? a.e + int64_t(row) * a.e_ld + c0 : nullptr;
    auto columns = [&](int at, int c) {  // x[at .. at + 32), the row's columns from c on
        const uint32_t left_out = c == 0 ? out_lo : out_hi;
#pragma unroll
        for (int j0 = 0; j0 < 32; j0 += 16) {
            uint32_t word[8];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                float e[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float u = x[at + j0 + j + k], y = __fmul_rn(u, mul), r = CAP ? tanh_gap(y) : 0.f;
                    const float v = CAP ? bend(y, r, cap) : u;
                    e[k] = exp2_fast(__fmul_rn(__fsub_rn(v, base), by));
                    if (CAP && (left_out >> (j0 + j + k) & 1u)) e[k] = 0.f;
                    sum[(j + k) & 3] = __fadd_rn(sum[(j + k) & 3], e[k]);
                    e[k] *= CAP ? tanh_slope(r, kExpScale) : kExpScale;
                }
                if (E) word[j / 2] = pack_f16(e[0], e[1]);
            }
            if (E) store8(out + c + j0, word, true);
        }
    };
    if (CAP) {
#pragma unroll 1
        for (int c = 0; c < kCols; c += 32) {
            columns(0, c);
            turn(x);
        }
    } else {
#pragma unroll
        for (int c = 0; c < kCols; c += 32) columns(c, c);
    }
    a.stats[int64_t(row) * a.n_stats + nt * (kTile / kCols) + part] =
        make_float2(none ? top : CAP ? base : __fmul_rn(top, mul), (sum[0] + sum[1]) + (sum[2] + sum[3]));
}

// The first 32 of x += the columns [0, n) (n a multiple of 8) at p: their loads are waited for once.
template <int N>
__device__ __forceinline__ void add_row(float (&x)[N], int n, const float* p) {
    float4 f[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        f[j] = 4 * j < n ? reinterpret_cast<const float4*>(p)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        x[4 * j] += f[j].x;
        x[4 * j + 1] += f[j].y;
        x[4 * j + 2] += f[j].z;
        x[4 * j + 3] += f[j].w;
    }
}

template <int N>
__device__ __forceinline__ void add_row(float (&x)[N], int n, const uint16_t* p) {
    uint4 w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = 8 * j < n ? reinterpret_cast<const uint4*>(p)[j] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        float f[8];
        unpack8(w[j], f);
#pragma unroll
        for (int k = 0; k < 8; ++k) x[8 * j + k] += f[k];
    }
}

// The first 32 of x, of which n (a multiple of 8) exist, to `to`.
template <bool B16, int N>
__device__ __forceinline__ void write32(const float (&x)[N], int n, void* to, bool wide) {
    char* p = static_cast<char*>(to);
    if (B16) {
#pragma unroll
        for (int s = 0; s < 32; s += 16) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = pack_bf16(x[s + 2 * j], x[s + 2 * j + 1]);
            if (s + 16 <= n) store8(p + 2 * s, w, wide);
            else if (s < n) *reinterpret_cast<uint4*>(p + 2 * s) = make_uint4(w[0], w[1], w[2], w[3]);
        }
    } else {
#pragma unroll
        for (int s = 0; s < 32; s += 8) {
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) w[j] = __float_as_uint(x[s + j]);
            if (s < n) store8(p + 4 * s, w, wide);
        }
    }
}

// One row's columns [0, n) (n a multiple of 8) to `out`.
template <bool B16>
__device__ __forceinline__ void write_row(float (&x)[kCols], int n, void* out) {
    const bool wide = (reinterpret_cast<uintptr_t>(out) & 31) == 0;
#pragma unroll 1
    for (int c = 0; c < kCols; c += 32) {
        write32<B16>(x, n - c, static_cast<char*>(out) + c * (B16 ? 2 : 4), wide);
        turn(x);
    }
}

// A warp's 32 rows and 64 columns of dW from (m0, n0), through its staging: 128 bytes a row at a
// time, as TMA swizzles them.  there: the tile is in dW; any: there is a sum in TMEM, whose
// barrier is waited for.  False where a wait gave up.
template <bool B16>
__device__ __forceinline__ bool staged_tile(const CUtensorMap& map, bool plus, bool there, bool any, int n0, int m0, int D,
                                            uint32_t taddr, uint8_t* staging, uint64_t* loaded, uint32_t* loaded_phase,
                                            uint64_t* tfull, uint32_t tphase, int lane, volatile int* abort_flag) {
    constexpr int kWide = B16 ? 64 : 32;  // columns of 128 bytes
    auto begin = [&](int c) {  // the staging is free again; what is added to comes in
        if (lane == 0) {
            asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
            if (plus) {
                tc::mbar_arrive_expect_tx(loaded, kStaging);
                tc::tma_load_2d(staging, &map, loaded, n0 + c, m0, tc::l2_policy_evict_first());
            }
        }
        __syncwarp();
    };
    if (there) begin(0);
    bool ok = true;
    if (any) {
        ok = __all_sync(kFull, tc::mbar_wait(tfull, tphase, abort_flag));
        tc::fence_after_sync();
    }
    if (there && plus && !ok) {  // the copy in flight ends before the block does
        volatile int never = 0;
        tc::mbar_wait(loaded, *loaded_phase, &never);
    }
    if (!ok || !there) return ok;
    uint4* own = reinterpret_cast<uint4*>(staging + lane * 128);
#pragma unroll 1
    for (int c = 0; c < kCols; c += kWide) {
        if (n0 + c >= D) break;
        if (c > 0) begin(c);
        if (plus) {
            ok = __all_sync(kFull, tc::mbar_wait(loaded, *loaded_phase, abort_flag));
            if (!ok) {
                volatile int never = 0;
                tc::mbar_wait(loaded, *loaded_phase, &never);
                return false;
            }
            *loaded_phase ^= 1;
        }
#pragma unroll
        for (int s = 0; s < kWide; s += 32) {
            float v[32];
            if (any) {
                tmem_ld32(taddr + c + s, v);
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.f;
            }
            constexpr int kEach = B16 ? 8 : 4;  // columns of 16 bytes
#pragma unroll
            for (int j = 0; j < 32; j += kEach) {
                uint4* at = own + (((s + j) / kEach) ^ (lane & 7));
                if (plus) {
                    const uint4 o = *at;
                    if (B16) {
                        float f[8];
                        unpack8(o, f);
#pragma unroll
                        for (int k = 0; k < 8; ++k) v[j + (k % kEach)] += f[k];
                    } else {
                        v[j] += __uint_as_float(o.x);
                        v[j + 1] += __uint_as_float(o.y);
                        v[j + 2] += __uint_as_float(o.z);
                        v[j + 3] += __uint_as_float(o.w);
                    }
                }
                if constexpr (B16)
                    *at = make_uint4(pack_bf16(v[j], v[j + 1]), pack_bf16(v[j + 2], v[j + 3]), pack_bf16(v[j + 4], v[j + 5]),
                                     pack_bf16(v[j + 6], v[j + 7]));
                else
                    *at = make_uint4(__float_as_uint(v[j]), __float_as_uint(v[j + 1]), __float_as_uint(v[j + 2]),
                                     __float_as_uint(v[j + 3]));
            }
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
            asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                             reinterpret_cast<uint64_t>(&map)),
                         "r"(n0 + c), "r"(m0), "r"(tc::smem_u32(staging))
                         : "memory");
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
        }
    }
    return true;
}

// QUAD: a cluster of two pairs on neighbouring tiles that share an operand (LOGITS: two M units
// and W's rows; the gradients: two N tiles and g's): the first pair's CTAs load it for the CTA
// of the same rank in the other pair too, and a stage is free when both pairs' MMAs have read
// it.  A tile past the end is computed on zeros and not written.
// STAGED (dW, one piece): rows go out, and what they are added to comes in, by TMA through a
// staging of each epilogue warp, for short products, whose time is the tile's way out: a row a
// lane costs the memory pipeline a cycle for each 16 bytes.  64 rows x 151,936 x 4096 in bf16: 225
// us (5.5 TB/s) instead of 290, added to old values 420 (5.9 TB/s) instead of 660; 1,024 rows 4%
// of the whole call, 2,048 2%, and none added.  It takes two stages of the ring.
template <int MODE, bool E, bool CAP, bool QUAD, bool STAGED>
__global__ void __launch_bounds__(kThreads, 1)
loss_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                 const __grid_constant__ CUtensorMap tm_out, const __grid_constant__ Work w) {
    constexpr int kStages = stages(STAGED);
    constexpr bool DW_ANY = MODE == DW || MODE == DW_LONG;
    constexpr bool A_MN = DW_ANY, B_MN = MODE != LOGITS;
    const LossGemmArgs& a = w.a;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
    uint8_t* staging = smem + size_t(kStages) * 2 * kOperand;
    uint64_t* full = reinterpret_cast<uint64_t*>(staging + (STAGED ? 16 * kStaging : 0));
    uint64_t* empty = full + kStages;
    uint64_t* tfull = empty + kStages;
    uint64_t* tempty = tfull + 2;
    uint64_t* mma_done = tempty + 2;
    uint64_t* loaded = mma_done + 1;  // of the epilogue warps
    uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(loaded + 16);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t crank = tc::cluster_ctarank(), lead = crank & ~1u;  // in the cluster; its pair's leader
    const int rank = int(crank & 1), which = int(crank >> 1);          // in the pair; which pair
    const bool leader = rank == 0;
    constexpr int kPairs = QUAD ? 2 : 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kStages; ++s) {
            tc::mbar_init(&full[s], 1);
            tc::mbar_init(&empty[s], kPairs);
        }
        for (int b = 0; b < 2; ++b) {
            tc::mbar_init(&tfull[b], 1);
            tc::mbar_init(&tempty[b], 32);  // the epilogue warps of both CTAs
        }
        tc::mbar_init(mma_done, 1);
        for (int i = 0; i < 16; ++i) tc::mbar_init(&loaded[i], 1);
        *abort_flag = 0;
        tc::fence_mbar_init();
    }
    if (warp == 1) {
        tc::tmem_alloc_pair(tmem_holder, 512);
        tc::tmem_relinquish_pair();
    }
    if (warp == 0 && lane == 0) {
        tc::prefetch_tmap(&tm_a);
        tc::prefetch_tmap(&tm_b);
        if (STAGED) tc::prefetch_tmap(&tm_out);
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::cluster_sync_all();
    tc::fence_after_sync();
    const uint32_t tmem_base = *tmem_holder;
    asm volatile("griddepcontrol.launch_dependents;");
    asm volatile("griddepcontrol.wait;" ::: "memory");  // what is above may overlap the kernel before

    // the rows of this piece that have a target
    const int64_t left = int64_t(*a.count) - a.row0;
    const int live = left < 0 ? 0 : left > a.rows ? a.rows : int(left);
    const int n_mu = (int(DW_ANY ? a.V : live) + kTile - 1) / kTile;
    const int k_total = (int(MODE == LOGITS ? a.D : MODE == DH ? a.V : live) + kStep - 1) / kStep;
    const int units = int(gridDim.x) / (2 * kPairs), unit = int(blockIdx.x) / (2 * kPairs);
    const int n_nt = w.n_nt;
    const int tiles = MODE == LOGITS ? loss_cluster_tiles(n_nt, n_mu, QUAD) : loss_cluster_tiles(n_mu, n_nt, QUAD);
    const LossSplit work = MODE == DH ? loss_split(tiles, k_total, units, QUAD, lane) : LossSplit{tiles, 0, 1};
    const int total = work.items();

    auto tile = [&](int i) { return loss_tile<MODE == LOGITS, QUAD>(i, n_mu, n_nt, work, k_total, which); };

    const int segment = MODE == DW ? max(k_total, 1) : MODE == LOGITS ? kSegment : kLongSegment;
    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRoleRegisters));
        if (warp == 0 && lane == 0) {
            // ------------------------------------------------------ TMA producer
            // h stays in L2; W leaves it first where it is read once (one M unit: 2%), and as it comes
            // where other clusters read it, too (first: it was read twice, 2%)
            const uint64_t keep = tc::l2_policy_evict_last(), normal = tc::l2_policy_evict_normal();
            const uint64_t weights = n_mu == 1 ? tc::l2_policy_evict_first() : normal;
            const uint64_t pol_a = MODE == LOGITS ? keep : normal, pol_b = DW_ANY ? keep : weights;
            int stage = 0;
            uint32_t phase = 0;
            int8_t armed[kStages];
            for (int s = 0; s < kStages; ++s) armed[s] = -1;
            bool ok = true;
            for (int i = unit; i < total && ok; i += units) {
                const LossTile t = tile(i);
                for (int k = t.k0; k < t.k1; ++k) {
                    if (!tc::mbar_wait(&empty[stage], phase ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    if (leader) tc::mbar_arrive_expect_tx(&full[stage], 4 * kOperand);
                    uint8_t* da = smem + size_t(stage) * 2 * kOperand;
                    uint8_t* db = da + kOperand;
                    const uint32_t fb = tc::mapa_shared(tc::smem_u32(&full[stage]), lead);
                    const int ma = t.mu * kTile + rank * 128, nb = t.nt * kTile + rank * 128;
                    // the operand that a cluster shares is loaded once, by its first pair
                    const uint16_t both = uint16_t((1u << crank) | (1u << (crank + 2)));
                    auto own = [&](uint8_t* to, const CUtensorMap* map, int x, int y, uint64_t policy) {
                        tc::tma_load_2d_pair(to, map, fb, x, y, policy);
                    };
                    auto shared = [&](uint8_t* to, const CUtensorMap* map, int x, int y, uint64_t policy) {
                        if (!QUAD || t.alone) tc::tma_load_2d_pair(to, map, fb, x, y, policy);
                        else if (which == 0) tc::tma_load_2d_pair_mc(to, map, fb, both, x, y, policy);
                    };
                    if (MODE == LOGITS) {
                        own(da, &tm_a, k * kStep, int(a.row0) + ma, pol_a);
                        shared(db, &tm_b, k * kStep, nb, pol_b);
                    } else {
                        if (A_MN) {
                            shared(da, &tm_a, ma, k * kStep, pol_a);
                            shared(da + kOperand / 2, &tm_a, ma + 64, k * kStep, pol_a);
                        } else {
                            shared(da, &tm_a, k * kStep, ma, pol_a);
                        }
                        const int kb = k * kStep + (DW_ANY ? int(a.row0) : 0);
                        own(db, &tm_b, nb, kb, pol_b);
                        own(db + kOperand / 2, &tm_b, nb + 64, kb, pol_b);
                    }
                    armed[stage] = int8_t(phase);
                    if (++stage == kStages) {
                        stage = 0;
                        phase ^= 1;
                    }
                }
            }
            if (!ok && leader) {
                // wait (bounded) for the copies in flight; the pair's other CTA's complete on these
                // barriers too, and it leaves only after the closing cluster barrier
                volatile int never = 0;
                for (int s = 0; s < kStages; ++s)
                    if (armed[s] >= 0) tc::mbar_wait(&full[s], uint32_t(armed[s]), &never);
            }
        }
        if (warp == 1 && lane == 0 && leader) {
            // -------------------------------------------------------- MMA issuer
            constexpr uint32_t idesc =
                tc::idesc_bf16_f32(256, 256) | (A_MN ? 1u << 15 : 0u) | (B_MN ? 1u << 16 : 0u);
            int stage = 0, buf = 0;
            uint32_t phase = 0, tphase = 0;
            bool ok = true;
            for (int i = unit; i < total && ok; i += units) {
                int k0, k1;
                loss_steps(i, work, k_total, &k0, &k1);
                for (int k = k0; k < k1 && ok; k += segment) {
                    if (!tc::mbar_wait_cluster(&tempty[buf], tphase ^ 1, abort_flag)) {
                        ok = false;
                        break;
                    }
                    tc::fence_after_sync();
                    const uint32_t d = tmem_base + uint32_t(buf * kTile);
                    const int end = min(k + segment, k1);
                    for (int kk = k; kk < end; ++kk) {
                        if (!tc::mbar_wait(&full[stage], phase, abort_flag)) {
                            ok = false;
                            break;
                        }
                        tc::fence_after_sync();
                        const uint32_t sa = tc::smem_u32(smem + size_t(stage) * 2 * kOperand), sb = sa + kOperand;
#pragma unroll
                        for (int q = 0; q < kStep / 16; ++q)
                            tc::mma_bf16_pair(d, operand_desc(sa + q * (A_MN ? 2048 : 32), A_MN),
                                              operand_desc(sb + q * (B_MN ? 2048 : 32), B_MN), idesc,
                                              (kk != k || q != 0) ? 1u : 0u);
                        tc::mma_commit_pair(&empty[stage], QUAD ? 0xF : 0x3);
                        if (++stage == kStages) {
                            stage = 0;
                            phase ^= 1;
                        }
                    }
                    if (ok) tc::mma_commit_pair(&tfull[buf], uint16_t(0x3u << lead));
                    buf ^= 1;
                    if (buf == 0) tphase ^= 1;
                }
            }
            tc::mma_commit_pair(mma_done, uint16_t(0x3u << lead));
            volatile int never = 0;
            tc::mbar_wait(mma_done, 0, &never);
        }
    } else {
        // ---------------------------------------------------------- epilogue
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kEpilogueRegisters));
        const int quarter = warp & 3, part = (warp >> 2) - 1;
        int buf = 0;
        uint32_t tphase = 0, loaded_phase = 0;
        bool ok = true;
        for (int i = unit; i < total && ok; i += units) {
            const LossTile t = tile(i);
            const int m = t.mu * kTile + rank * 128 + quarter * 32 + lane;
            if constexpr (STAGED) {
                const int m0 = m - lane, n0 = t.nt * kTile + part * kCols;
                const bool there = m0 < a.V && n0 < a.D, any = t.k1 > t.k0;
                const uint32_t taddr =
                    tmem_base + (uint32_t(quarter * 32) << 16) + uint32_t(buf * kTile + part * kCols);
                if (a.out_bf16)
                    ok = staged_tile<true>(tm_out, a.accumulate, there, any, n0, m0, int(a.D), taddr, staging + (warp - 4) * kStaging,
                                           &loaded[warp - 4], &loaded_phase, &tfull[buf], tphase, lane, abort_flag);
                else
                    ok = staged_tile<false>(tm_out, a.accumulate, there, any, n0, m0, int(a.D), taddr, staging + (warp - 4) * kStaging,
                                            &loaded[warp - 4], &loaded_phase, &tfull[buf], tphase, lane, abort_flag);
                if (!ok) break;
                if (any) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) accumulator_read(&tempty[buf], lead);
                    buf ^= 1;
                    if (buf == 0) tphase ^= 1;
                }
            } else if constexpr (MODE == DW) {
                // straight from TMEM, 32 columns at a time: a sum of rows is one partial sum.  What a
                // bf16 dW holds is on its way while the product is summed; an fp32 one's, to L2.
                const bool any = t.k1 > t.k0;
                const int n0 = t.nt * kTile + part * kCols, n = min(kCols, int(a.D) - n0);
                const int64_t o = int64_t(m) * a.D + n0;
                uint4 old[kCols / 8];
                const bool plus16 = a.last && a.accumulate && a.out_bf16;
#pragma unroll
                for (int j = 0; j < kCols / 8; ++j)
                    old[j] = plus16 && m < a.V && 8 * j < n
                                 ? reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(a.out) + o)[j]
                                 : make_uint4(0u, 0u, 0u, 0u);
                if (a.last && a.accumulate && !a.out_bf16 && m < a.V && n > 0) {
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<float*>(a.out) + o));
                    if (n > 32) asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<float*>(a.out) + o + 32));
                }
                if (any) {
                    ok = __all_sync(kFull, tc::mbar_wait(&tfull[buf], tphase, abort_flag));
                    if (!ok) break;
                    tc::fence_after_sync();
                }
                const uint32_t taddr =
                    tmem_base + (uint32_t(quarter * 32) << 16) + uint32_t(buf * kTile + part * kCols);
#pragma unroll
                for (int c = 0; c < kCols; c += 32) {
                    if (c >= n) break;
                    float v[32];
                    if (any) {
                        tmem_ld32(taddr + c, v);
                    } else {
#pragma unroll
                        for (int j = 0; j < 32; ++j) v[j] = 0.f;
                    }
                    if (m < a.V) {
                        if (a.sums && !a.first) add_row(v, n - c, a.sums + o + c);
                        void* to = a.sums + o + c;
                        if (a.last && a.out_bf16) to = static_cast<uint16_t*>(a.out) + o + c;
                        else if (a.last) to = static_cast<float*>(a.out) + o + c;
                        const bool wide = (reinterpret_cast<uintptr_t>(to) & 31) == 0;
                        if (a.last && a.out_bf16) {
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                float f[8];
                                unpack8(old[c / 8 + j], f);
#pragma unroll
                                for (int k = 0; k < 8; ++k) v[8 * j + k] += f[k];
                            }
                            write32<true>(v, n - c, to, wide);
                        } else {
                            if (a.last && a.accumulate) add_row(v, n - c, static_cast<const float*>(to));
                            write32<false>(v, n - c, to, wide);
                        }
                    }
                    __syncwarp();  // whole again for the next load from TMEM
                }
                if (any) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) accumulator_read(&tempty[buf], lead);
                    buf ^= 1;
                    if (buf == 0) tphase ^= 1;
                }
            } else {
                // the row's target, or its place in dh: read before the product is waited for
                const int place = !DW_ANY && m < live ? (MODE == LOGITS ? a.targets : a.map)[a.row0 + m] : 0;
                float x[kCols];
#pragma unroll
                for (int j = 0; j < kCols; ++j) x[j] = 0.f;
                for (int k = t.k0; k < t.k1; k += segment) {
                    ok = __all_sync(kFull, tc::mbar_wait(&tfull[buf], tphase, abort_flag));
                    if (!ok) break;
                    tc::fence_after_sync();
                    const uint32_t taddr =
                        tmem_base + (uint32_t(quarter * 32) << 16) + uint32_t(buf * kTile + part * kCols);
#pragma unroll
                    for (int c = 0; c < kCols; c += 32) {
                        float v[32];
                        tmem_ld32(taddr + c, v);
#pragma unroll
                        for (int j = 0; j < 32; ++j) x[c + j] += v[j];
                    }
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) accumulator_read(&tempty[buf], lead);
                    buf ^= 1;
                    if (buf == 0) tphase ^= 1;
                }
                if (!ok) break;
                if (MODE == LOGITS) {
                    if (m < live && t.nt < n_nt) logits_epilogue<E, CAP>(a, x, m, place, t.nt, part);
                    __syncwarp();
                } else if (MODE == DW_LONG) {
                    const int n0 = t.nt * kTile + part * kCols, n = min(kCols, int(a.D) - n0);
#pragma unroll 1
                    for (int c = 0; c < kCols; c += 32) {
                        const int64_t o = int64_t(m) * a.D + n0 + c;
                        if (m < a.V && c < n) {
                            if (a.sums && !a.first) add_row(x, n - c, a.sums + o);
                            void* to = a.sums + o;
                            if (a.last) to = static_cast<char*>(a.out) + o * (a.out_bf16 ? 2 : 4);
                            const bool wide = (reinterpret_cast<uintptr_t>(to) & 31) == 0;
                            if (a.last && a.out_bf16) {
                                if (a.accumulate) add_row(x, n - c, static_cast<const uint16_t*>(to));
                                write32<true>(x, n - c, to, wide);
                            } else {
                                if (a.last && a.accumulate) add_row(x, n - c, static_cast<const float*>(to));
                                write32<false>(x, n - c, to, wide);
                            }
                        }
                        turn(x);
                    }
                    __syncwarp();
                } else {
                    const int n0 = t.nt * kTile + part * kCols, n = min(kCols, int(a.D) - n0);
                    if (m < live && n > 0) {
                        const int64_t o = t.part < 0 ? int64_t(place) * a.D + n0
                                                     : (int64_t(t.part * kPairs + which) * kTile + (m - t.mu * kTile)) * kTile +
                                                           part * kCols;
                        if (t.part < 0 && a.out_bf16) write_row<true>(x, n, static_cast<uint16_t*>(a.out) + o);
                        else write_row<false>(x, n, (t.part < 0 ? static_cast<float*>(a.out) : a.part) + o);
                    }
                    __syncwarp();
                }
            }
        }
        if (STAGED && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }

    tc::fence_before_sync();
    __syncthreads();
    // a pair's MMAs read both CTAs' shared memory and write their TMEM, and copies go to every
    // CTA of a cluster: none frees TMEM or exits before all are done
    tc::cluster_sync_all();
    if (threadIdx.x == 0 && *abort_flag && a.status) atomicOr(a.status, DF2_STATUS_WAIT_TIMEOUT);
    if (warp == 1) {
        tc::fence_after_sync();
        tc::tmem_dealloc_pair(tmem_base, 512);
    }
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* p = nullptr;
        cudaDriverEntryPointQueryResult q{};
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            p = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
    }();
    return fn;
}

// Boxes of 128 bytes of a row by box_rows rows.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols, int64_t ld, int box_rows, bool f32 = false) {
    auto fn = encode_fn();
    if (!fn) return false;
    const cuuint64_t dims[2] = {cuuint64_t(cols), cuuint64_t(rows)}, strides[1] = {cuuint64_t(ld) * (f32 ? 4 : 2)};
    const cuuint32_t box[2] = {f32 ? 32u : 64u, cuuint32_t(box_rows)}, estr[2] = {1, 1};
    return fn(m, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The kernels' shared memory is the same for every call: allowed once on each device.
template <int MODE, bool E, bool CAP, bool QUAD, bool STAGED>
cudaError_t smem_once() {
    static std::atomic<uint64_t> done{0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
    e = allow_smem<loss_gemm_kernel<MODE, E, CAP, QUAD, STAGED>>(smem_bytes(STAGED));
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
    return e;
}

template <int MODE, bool E, bool CAP, bool QUAD, bool STAGED>
cudaError_t launch_clusters(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to, const Work& w, int64_t clusters,
                            cudaStream_t stream) {
    const cudaError_t e = smem_once<MODE, E, CAP, QUAD, STAGED>();
    if (e != cudaSuccess) return e;
    constexpr unsigned kCtas = QUAD ? 4 : 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kCtas * unsigned(clusters));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem_bytes(STAGED);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    note_launch();
    return cudaLaunchKernelEx(&cfg, loss_gemm_kernel<MODE, E, CAP, QUAD, STAGED>, ta, tb, to, w);
}

// Clusters of two pairs (four SMs of one GPC) that run at once on the current device, asked
// once; 0 where the question fails.
template <int MODE, bool E, bool CAP, bool STAGED>
int quad_slots() {
    constexpr int kDevices = 64;
    static std::mutex mu;
    static int known[kDevices];  // plus one
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= kDevices) return 0;
    std::lock_guard<std::mutex> lock(mu);
    if (known[dev] == 0) {
        if (smem_once<MODE, E, CAP, true, STAGED>() != cudaSuccess) return 0;
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(4);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = smem_bytes(STAGED);
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = 4;
        attr[0].val.clusterDim.y = 1;
        attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if (cudaOccupancyMaxActiveClusters(&n, loss_gemm_kernel<MODE, E, CAP, true, STAGED>, &cfg) != cudaSuccess) n = 0;
        known[dev] = n + 1;
    }
    return known[dev] - 1;
}

// `across` tiles by `shared` ones that neighbours share an operand along.
template <int MODE, bool E = false, bool CAP = false, bool STAGED = false>
cudaError_t launch(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& to, const Work& w, int64_t across,
                   int64_t shared, int num_sms, cudaStream_t stream) {
    const int slots = shared > 1 ? quad_slots<MODE, E, CAP, STAGED>() : 0;
    const int64_t tiles = loss_cluster_tiles(int(across), int(shared), slots > 0), pairs = num_sms / 2;
    if (slots > 0) return launch_clusters<MODE, E, CAP, true, STAGED>(ta, tb, to, w, tiles < slots ? tiles : slots, stream);
    return launch_clusters<MODE, E, CAP, false, STAGED>(ta, tb, to, w, tiles < pairs ? tiles : pairs, stream);
}

int64_t up(int64_t n, int64_t by) { return (n + by - 1) / by; }

}  // namespace

cudaError_t loss_logits_launch(const LossGemmArgs& a, const uint16_t* h, int64_t h_rows, const uint16_t* W, int num_sms,
                               cudaStream_t stream) {
    CUtensorMap ta, tb;
    if (!make_map(&ta, h, h_rows, a.D, a.D, 128) || !make_map(&tb, W, a.V, a.D, a.D, 128)) return cudaErrorInvalidValue;
    const Work w{a, int(up(a.V, kTile))};
    const int64_t rows = up(a.rows, kTile);
    if (a.lm.cap > 0.f)
        return a.e ? launch<LOGITS, true, true>(ta, tb, tb, w, w.n_nt, rows, num_sms, stream)
                   : launch<LOGITS, false, true>(ta, tb, tb, w, w.n_nt, rows, num_sms, stream);
    return a.e ? launch<LOGITS, true, false>(ta, tb, tb, w, w.n_nt, rows, num_sms, stream)
               : launch<LOGITS, false, false>(ta, tb, tb, w, w.n_nt, rows, num_sms, stream);
}

cudaError_t loss_dh_launch(const LossGemmArgs& a, int64_t e_rows, const uint16_t* W, int num_sms, LossDhGrid* grid,
                           cudaStream_t stream) {
    CUtensorMap ta, tb;
    if (!make_map(&ta, a.e, e_rows, a.V, a.e_ld, 128) || !make_map(&tb, W, a.V, a.D, a.D, 64)) return cudaErrorInvalidValue;
    const Work w{a, int(up(a.D, kTile))};
    bool quad = w.n_nt > 1;
    int slots = quad ? quad_slots<DH, false, false, false>() : 0;
    quad = slots > 0;
    if (!quad) slots = num_sms / 2;
    // a cluster for each part there can be: how many there are follows from the live rows
    const int64_t most = int64_t(loss_cluster_tiles(int(up(a.rows, kTile)), w.n_nt, quad)) * loss_way_limit(up(a.V, kStep));
    *grid = {w.n_nt, int(most < slots ? most : slots), quad};
    return quad ? launch_clusters<DH, false, false, true, false>(ta, tb, tb, w, grid->units, stream)
                : launch_clusters<DH, false, false, false, false>(ta, tb, tb, w, grid->units, stream);
}

cudaError_t loss_dw_launch(const LossGemmArgs& a, int64_t e_rows, const uint16_t* h, int64_t h_rows, int num_sms,
                           cudaStream_t stream) {
    CUtensorMap ta, tb;
    if (!make_map(&ta, a.e, e_rows, a.V, a.e_ld, 64) || !make_map(&tb, h, h_rows, a.D, a.D, 64)) return cudaErrorInvalidValue;
    const Work w{a, int(up(a.D, kTile))};
    const int64_t across = up(a.V, kTile);
    if (a.first && a.last && up(a.rows, kStep) <= kStagedSteps) {
        CUtensorMap to;
        if (!make_map(&to, a.out, a.V, a.D, a.D, 32, !a.out_bf16)) return cudaErrorInvalidValue;
        return launch<DW, false, false, true>(ta, tb, to, w, across, w.n_nt, num_sms, stream);
    }
    if (up(a.rows, kStep) > kLongSegment) return launch<DW_LONG>(ta, tb, tb, w, across, w.n_nt, num_sms, stream);
    return launch<DW>(ta, tb, tb, w, across, w.n_nt, num_sms, stream);
}

}  // namespace df2
