// dflash2_adamw: one AdamW step over many tensors.
//
// Per element, in fp32 operations that are rounded one by one (no fused multiply-add, so
// the moments depend on the formula alone and not on how a compiler contracts it; the
// division of the update is the fast one, within 2 ulp of an lr-sized term):
//   g = grad * grad_scale
//   m = m * beta1 + g * (1 - beta1)
//   v = v * beta2 + (g * (1 - beta2)) * g
//   s = sqrt(v)
//   w = w * (1 - lr * wd) - (m / (s * (1 / sqrt(1 - beta2^t)) + eps)) * (lr / (1 - beta1^t))
//
// States in 8 bits hold m and s (the root, not v: its range in powers of two is half
// of v's) as e4m3 values in units of absmax / 448 of each block of 256 elements.
// The root keeps one more rule: above zero it is at least e4m3's smallest value
// above zero, 2^-9.  Rounded to zero it would leave eps alone under a nonzero m, and
// one step of m / eps; rounded up it only makes that element's step smaller.  The
// block's largest value is held exactly (to an ulp), so a block whose gradients fade
// fades with its scale although e4m3's steps are wider than one step's decay.
//
// Bound: HBM.  A step reads w, g, m, v and writes w, m, v (and the bf16 copy of a master
// weight) once: 28 bytes an element with everything in fp32.  One warp owns a block of 256
// elements, 8 a lane: the block's maxima are warp shuffles, every load is 16 bytes a lane,
// and all of a lane's loads are issued before the first use, the gradient scale's among
// them.  Four warps a CTA: its warps end together, and a smaller CTA gives way sooner (213
// against 222 us with eight, 8-bit states of 78.8 M bf16 weights with masters: 6.7 TB/s;
// the exact division in the update, all else as it is, takes 238 us).  Two blocks a warp with
// the next one's loads in flight need 126 registers and took 303 us.  States in fp32 with
// bf16 weights, gradients and masters: 42.9 M weights in 175 us, 6.9 TB/s.
// One launch covers up to kManyTensors tensors: their descriptors travel as the
// kernel's parameters, so nothing is uploaded and no table of addresses outlives the
// call; a warp finds its tensor by bisection over the block counts.
#include <cuda_fp8.h>

#include <cmath>

#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kBlock = DF2_ADAMW_BLOCK;  // elements a warp owns, and that share a scale
constexpr int kWarps = 4;
constexpr int kFewTensors = 16;
constexpr int kManyTensors = 320;
constexpr float kE4m3Max = 448.f;
constexpr float kE4m3Min = 0.001953125f;       // 2^-9
constexpr float kTiny = 7.888609052210118e-31f;  // 2^-100: a block below it holds zeros

struct Entry {
    void* p;
    float* master;
    const void* g;
    void* m;
    void* v;
    float* ms;
    float* vs;
    int64_t n;
    float keep;      // 1 - lr * weight_decay
    float step;      // lr / (1 - beta1^t)
    int64_t flags;   // kP16 | kG16 | kVec
};
enum : int64_t { kP16 = 1, kG16 = 2, kVec = 4 };

template <int CAP>
struct Args {
    Entry e[CAP];
    int first[CAP + 1];  // the tensor's first block
    int count;
    float b1, c1, b2, c2, inv_bc2, eps;
    const float* grad_scale;
};
static_assert(sizeof(Args<kManyTensors>) <= 32764, "kernel parameters");

__device__ __forceinline__ float load1(const void* p, int64_t i, bool bf16) {
    return bf16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// 8 consecutive elements from i (a multiple of 8 past a 16-byte boundary).
__device__ __forceinline__ void load8(const void* p, int64_t i, bool bf16, float f[8]) {
    if (bf16) {
        unpack8(__ldcs(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i)), f);
    } else {
        const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        const float4 a = __ldcs(q), b = __ldcs(q + 1);
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
}

__device__ __forceinline__ void store8(void* p, int64_t i, bool bf16, const float f[8]) {
    if (bf16) {
        uint4 w;
        uint32_t* o = &w.x;
#pragma unroll
        for (int k = 0; k < 4; ++k) o[k] = pack_bf16(f[2 * k], f[2 * k + 1]);
        __stcs(reinterpret_cast<uint4*>(static_cast<uint16_t*>(p) + i), w);
    } else {
        float4* q = reinterpret_cast<float4*>(static_cast<float*>(p) + i);
        __stcs(q, make_float4(f[0], f[1], f[2], f[3]));
        __stcs(q + 1, make_float4(f[4], f[5], f[6], f[7]));
    }
}

__device__ __forceinline__ float e4m3_to_f32(uint8_t c) {
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(__nv_fp8_storage_t(c), __NV_E4M3)));
}

// Two codes of a word (byte 2*k and the next), exactly.
__device__ __forceinline__ float2 e4m3x2_to_f32(uint32_t w, int k) {
    return __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(w >> (16 * k)), __NV_E4M3)));
}

__device__ __forceinline__ uint32_t f32_to_e4m3x2(float lo, float hi) {
    return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3));
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
    for (int o = 16; o; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
    return v;
}

// One state's 8 values of a lane, to codes in units of the block's scale.
template <bool ROOT>
__device__ __forceinline__ uint2 quantise(const float x[8], float top, float* scale) {
    const bool held = top >= kTiny;
    const float inv = held ? __fmul_rn(__frcp_rn(top), kE4m3Max) : 0.f;
    *scale = held ? __fmul_rn(top, 1.f / kE4m3Max) : 0.f;
    float q[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        q[k] = __fmul_rn(x[k], inv);
        if (ROOT && x[k] > 0.f) q[k] = fmaxf(q[k], held ? kE4m3Min : 0.f);
    }
    return make_uint2(f32_to_e4m3x2(q[0], q[1]) | (f32_to_e4m3x2(q[2], q[3]) << 16),
                      f32_to_e4m3x2(q[4], q[5]) | (f32_to_e4m3x2(q[6], q[7]) << 16));
}

template <int BITS, int CAP>
__global__ void __launch_bounds__(kWarps * 32) adamw_kernel(const __grid_constant__ Args<CAP> a) {
    const int blk = blockIdx.x * kWarps + (threadIdx.x >> 5);
    const int lane = threadIdx.x & 31;
    if (blk >= a.first[a.count]) return;
    const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f;
    int lo = 0, hi = a.count;  // first[lo] <= blk < first[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a.first[mid] <= blk) lo = mid;
        else hi = mid;
    }
    const Entry& t = a.e[lo];
    const int64_t b = blk - a.first[lo];
    const int64_t i0 = b * kBlock + lane * 8;
    const int left = int(dmax<int64_t>(0, dmin<int64_t>(8, t.n - i0)));  // this lane's live elements
    const bool p16 = t.flags & kP16, g16 = t.flags & kG16;
    const bool vec = (t.flags & kVec) && left == 8;
    void* wp = t.master ? static_cast<void*>(t.master) : t.p;
    const bool w16 = p16 && !t.master;

    float w[8], g[8], m[8], v[8];
    float sm = 0.f, sv = 0.f;
    if (BITS == 8) {
        sm = t.ms[b];
        sv = t.vs[b];
    }
    if (vec) {
        load8(wp, i0, w16, w);
        load8(t.g, i0, g16, g);
        if (BITS == 8) {
            const uint2 cm = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.m) + i0));
            const uint2 cv = __ldcs(reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(t.v) + i0));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 fm = e4m3x2_to_f32(k < 2 ? cm.x : cm.y, k & 1);
                const float2 fv = e4m3x2_to_f32(k < 2 ? cv.x : cv.y, k & 1);
                m[2 * k] = fm.x;
                m[2 * k + 1] = fm.y;
                v[2 * k] = fv.x;
                v[2 * k + 1] = fv.y;
            }
        } else {
            load8(t.m, i0, false, m);
            load8(t.v, i0, false, v);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            const bool on = k < left;
            w[k] = on ? load1(wp, i0 + k, w16) : 0.f;
            g[k] = on ? load1(t.g, i0 + k, g16) : 0.f;
            if (BITS == 8) {
                m[k] = on ? e4m3_to_f32(static_cast<const uint8_t*>(t.m)[i0 + k]) : 0.f;
                v[k] = on ? e4m3_to_f32(static_cast<const uint8_t*>(t.v)[i0 + k]) : 0.f;
            } else {
                m[k] = on ? static_cast<const float*>(t.m)[i0 + k] : 0.f;
                v[k] = on ? static_cast<const float*>(t.v)[i0 + k] : 0.f;
            }
        }
    }

    if (!isfinite(gs)) return;  // no usable gradient: the step is left out
    float top_m = 0.f, top_s = 0.f;  // (elements past the end are zeros all through)
    float root[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        const float gk = __fmul_rn(g[k], gs);
        if (BITS == 8) {
            m[k] = __fmul_rn(m[k], sm);
            const float s = __fmul_rn(v[k], sv);
            v[k] = __fmul_rn(s, s);
        }
        m[k] = __fadd_rn(__fmul_rn(m[k], a.b1), __fmul_rn(gk, a.c1));
        v[k] = __fadd_rn(__fmul_rn(v[k], a.b2), __fmul_rn(__fmul_rn(gk, a.c2), gk));
        root[k] = __fsqrt_rn(v[k]);
        const float den = __fadd_rn(__fmul_rn(root[k], a.inv_bc2), a.eps);
        w[k] = __fsub_rn(__fmul_rn(w[k], t.keep), __fmul_rn(__fdividef(m[k], den), t.step));
        if (BITS == 8) {
            top_m = fmaxf(top_m, fabsf(m[k]));
            top_s = fmaxf(top_s, root[k]);
        }
    }

    uint2 cm = make_uint2(0, 0), cv = make_uint2(0, 0);
    if (BITS == 8) {
        cm = quantise<false>(m, warp_max(top_m), &sm);
        cv = quantise<true>(root, warp_max(top_s), &sv);
        if (lane == 0) {
            t.ms[b] = sm;
            t.vs[b] = sv;
        }
    }
    if (vec) {
        store8(wp, i0, w16, w);
        if (t.master) store8(t.p, i0, p16, w);
        if (BITS == 8) {
            __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.m) + i0), cm);
            __stcs(reinterpret_cast<uint2*>(static_cast<uint8_t*>(t.v) + i0), cv);
        } else {
            store8(t.m, i0, false, m);
            store8(t.v, i0, false, v);
        }
    } else {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            if (k >= left) break;
            if (w16) static_cast<uint16_t*>(wp)[i0 + k] = f32_to_bf16_rn(w[k]);
            else static_cast<float*>(wp)[i0 + k] = w[k];
            if (t.master) {
                if (p16) static_cast<uint16_t*>(t.p)[i0 + k] = f32_to_bf16_rn(w[k]);
                else static_cast<float*>(t.p)[i0 + k] = w[k];
            }
            if (BITS == 8) {
                static_cast<uint8_t*>(t.m)[i0 + k] = uint8_t((k < 4 ? cm.x : cm.y) >> (8 * (k & 3)));
                static_cast<uint8_t*>(t.v)[i0 + k] = uint8_t((k < 4 ? cv.x : cv.y) >> (8 * (k & 3)));
            } else {
                static_cast<float*>(t.m)[i0 + k] = m[k];
                static_cast<float*>(t.v)[i0 + k] = v[k];
            }
        }
    }
}

struct Hyper {
    double beta1, beta2, eps;
    int64_t step;
    const float* grad_scale;
};

bool aligned(const void* p, size_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

// The next launch's tensors from `at` on: as many as fit CAP descriptors and a grid.
template <int BITS, int CAP>
int launch_some(const dflash2_adamw_tensor* ts, int count, int* at, const Hyper& h, cudaStream_t stream) {
    Args<CAP> a;
    a.count = 0;
    a.first[0] = 0;
    const double t = double(h.step);
    a.b1 = float(h.beta1);
    a.c1 = float(1.0 - h.beta1);
    a.b2 = float(h.beta2);
    a.c2 = float(1.0 - h.beta2);
    a.inv_bc2 = float(1.0 / std::sqrt(1.0 - std::pow(h.beta2, t)));
    a.eps = float(h.eps);
    a.grad_scale = h.grad_scale;
    const double bc1 = 1.0 - std::pow(h.beta1, t);
    int64_t blocks = 0;
    for (; *at < count && a.count < CAP; ++*at) {
        const dflash2_adamw_tensor& s = ts[*at];
        if (s.n == 0) continue;
        const int64_t nb = (s.n + kBlock - 1) / kBlock;
        if (blocks + nb > INT32_MAX - kWarps) break;
        Entry& e = a.e[a.count];
        e.p = s.param;
        e.master = s.master;
        e.g = s.grad;
        e.m = s.exp_avg;
        e.v = s.exp_avg_2;
        e.ms = s.exp_avg_scale;
        e.vs = s.exp_avg_2_scale;
        e.n = s.n;
        e.keep = float(1.0 - s.lr * s.weight_decay);
        e.step = float(s.lr / bc1);
        e.flags = (s.param_dtype == DF2_DTYPE_BF16 ? kP16 : 0) | (s.grad_dtype == DF2_DTYPE_BF16 ? kG16 : 0);
        const size_t state_align = BITS == 8 ? 8 : 16;
        if (aligned(s.param, 16) && aligned(s.master, 16) && aligned(s.grad, 16) &&
            aligned(s.exp_avg, state_align) && aligned(s.exp_avg_2, state_align))
            e.flags |= kVec;
        blocks += nb;
        a.first[++a.count] = int(blocks);
    }
    if (a.count == 0) return DF2_OK;
    adamw_kernel<BITS, CAP><<<unsigned((blocks + kWarps - 1) / kWarps), kWarps * 32, 0, stream>>>(a);
    note_launch();
    return cudaGetLastError() == cudaSuccess ? DF2_OK : DF2_ERR_CUDA;
}

template <int BITS>
int launch_all(const dflash2_adamw_tensor* ts, int count, const Hyper& h, cudaStream_t stream) {
    for (int at = 0; at < count;) {
        // the parameters are copied at launch: few tensors take the small struct
        const int rc = count - at <= kFewTensors ? launch_some<BITS, kFewTensors>(ts, count, &at, h, stream)
                                                 : launch_some<BITS, kManyTensors>(ts, count, &at, h, stream);
        if (rc != DF2_OK) return rc;
    }
    return DF2_OK;
}

bool fraction(double x) { return x >= 0.0 && x < 1.0; }
bool finite_nonneg(double x) { return x >= 0.0 && x <= 1e300; }

int check_tensor(const dflash2_adamw_tensor& s, int bits) {
    if (s.n < 0 || !finite_nonneg(s.lr) || !finite_nonneg(s.weight_decay)) return DF2_ERR_INVALID_ARGUMENT;
    for (int d : {s.param_dtype, s.grad_dtype})
        if (d != DF2_DTYPE_BF16 && d != DF2_DTYPE_F32) return DF2_ERR_INVALID_ARGUMENT;
    if (s.n == 0) return DF2_OK;
    if (!s.param || !s.grad || !s.exp_avg || !s.exp_avg_2) return DF2_ERR_INVALID_ARGUMENT;
    if (bits == 8 && (!s.exp_avg_scale || !s.exp_avg_2_scale)) return DF2_ERR_INVALID_ARGUMENT;
    const size_t state = bits == 8 ? 1 : 4;
    if (!aligned(s.param, s.param_dtype == DF2_DTYPE_BF16 ? 2 : 4) || !aligned(s.master, 4) ||
        !aligned(s.grad, s.grad_dtype == DF2_DTYPE_BF16 ? 2 : 4) || !aligned(s.exp_avg, state) ||
        !aligned(s.exp_avg_2, state) || !aligned(s.exp_avg_scale, 4) || !aligned(s.exp_avg_2_scale, 4))
        return DF2_ERR_UNSUPPORTED;
    if ((s.n + kBlock - 1) / kBlock > INT32_MAX - kWarps) return DF2_ERR_UNSUPPORTED;
    return DF2_OK;
}

}  // namespace
}  // namespace df2

DF2_API int dflash2_adamw(const dflash2_adamw_tensor* tensors, int count, int state_bits, double beta1, double beta2,
                          double eps, int64_t step, const float* grad_scale, void* stream) {
    if (count < 0 || (state_bits != 32 && state_bits != 8) || step < 1) return DF2_ERR_INVALID_ARGUMENT;
    if (!df2::fraction(beta1) || !df2::fraction(beta2) || !df2::finite_nonneg(eps)) return DF2_ERR_INVALID_ARGUMENT;
    if (count > 0 && !tensors) return DF2_ERR_INVALID_ARGUMENT;
    if (!df2::aligned(grad_scale, 4)) return DF2_ERR_UNSUPPORTED;
    bool any = false;
    for (int i = 0; i < count; ++i) {
        const int rc = df2::check_tensor(tensors[i], state_bits);
        if (rc != DF2_OK) return rc;
        any |= tensors[i].n > 0;
    }
    if (!any) return DF2_OK;
    const df2::Hyper h{beta1, beta2, eps, step, grad_scale};
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    // the step's number and rates are arguments: a graph would repeat this one step
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    if (cudaStreamIsCapturing(st, &capture) != cudaSuccess) return DF2_ERR_CUDA;
    if (capture != cudaStreamCaptureStatusNone) return DF2_ERR_UNSUPPORTED;
    return state_bits == 8 ? df2::launch_all<8>(tensors, count, h, st) : df2::launch_all<32>(tensors, count, h, st);
}
