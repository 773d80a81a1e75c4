// dflash2_dropout: out = keep ? x * scale : 0 (+ residual), the mask made from a counter.
//
// Element i of the tensor (its index in [N, D], whatever the strides) is kept where the
// 16-bit word i % 8 of Philox4x32-10(key = seed, counter = (i / 8, draw)) is at least
// `drop` = round(rate * 65536): the mask is a function of the seed, the draw and i, so the
// gradient makes it again and nothing is stored.  (Philox: Salmon, Moraes, Dror, Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011; constants and rounds from there.)
// One call gives 128 bits, so 16-bit words serve 8 elements; 32-bit words would double
// the integer work of each element for a rate finer than 2^-16.
//
// Bound: HBM, closely followed by the integer unit (20 wide products a counter).  A thread owns
// the 8 elements of one counter, two counters where there are many: 16 bytes of bf16 a load.  The
// rounds' keys are parameters and the words are compared in place, in the upper half of a
// word.  16,384 x 5,120 bf16 with a residual: 76 us (6.6 TB/s; 80 with the keys stepped and a
// mask of bits made, 80 with one counter a thread, 76 with four); without a residual 59 us (5.6
// TB/s, the integer unit); 16,384 x 4,096 bf16 added to fp32: 98 us (6.8 TB/s).
// Tensors off 16-byte boundaries (odd D or strides) go element by element: a warp makes
// the masks of 32 counters, one a lane, as 8 bits each, and then walks the 256 elements
// with its lanes side by side, each taking its bit from the lane that made it.
#include "common.cuh"
#include "kernels.h"

namespace df2 {
namespace {

constexpr int kThreads = 256;

struct Args {
    const void* x;
    const void* res;
    void* out;
    int64_t x_ld, res_ld, out_ld;
    int64_t total, D;         // elements; a row's (flat: all of them)
    uint32_t last_dropped;    // drop - 1 in the upper half, ones below: the largest word that is dropped
    bool none;                // drop = 0
    float scale;
    uint64_t draw;
    const int64_t* draw_at;
    uint32_t key[20];         // of the rounds
};

// The 128 bits of counter q.  The rounds' keys come from the kernel's parameters, ready to use.
__device__ __forceinline__ void words(const Args& a, uint64_t q, uint64_t draw, uint32_t (&c)[4]) {
    c[0] = uint32_t(q);
    c[1] = uint32_t(q >> 32);
    c[2] = uint32_t(draw);
    c[3] = uint32_t(draw >> 32);
#pragma unroll
    for (int r = 0; r < 10; ++r) {
        const uint64_t m = uint64_t(c[0]) * 0xD2511F53u, n = uint64_t(c[2]) * 0xCD9E8D57u;
        c[0] = uint32_t(n >> 32) ^ c[1] ^ a.key[2 * r];
        c[1] = uint32_t(n);
        c[2] = uint32_t(m >> 32) ^ c[3] ^ a.key[2 * r + 1];
        c[3] = uint32_t(m);
    }
}

// Whether element e of the counter's 8 is kept: its 16 bits are compared in the upper half of a word.
__device__ __forceinline__ bool kept(const Args& a, const uint32_t (&c)[4], int e) {
    return a.none || (e & 1 ? c[e / 2] : c[e / 2] << 16) > a.last_dropped;
}

template <bool B16>
__device__ __forceinline__ float read1(const void* p, int64_t i) {
    return B16 ? bf16_to_f32(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// One element at a time, any stride and alignment.
template <bool IN16, bool OUT16, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ Args a) {
    const int lane = threadIdx.x & 31;
    const int64_t warp = int64_t(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
    const int64_t base = warp * 256;
    if (base >= a.total) return;
    const uint64_t draw = a.draw_at ? uint64_t(*a.draw_at) : a.draw;
    uint32_t c[4], mine = 0;
    words(a, uint64_t(warp) * 32 + lane, draw, c);
#pragma unroll
    for (int e = 0; e < 8; ++e) mine |= uint32_t(kept(a, c, e)) << e;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const int64_t i = base + j * 32 + lane;
        const uint32_t m = __shfl_sync(kFull, mine, j * 4 + (lane >> 3));
        if (i >= a.total) continue;
        const int64_t row = i / a.D, col = i - row * a.D;
        float y = 0.f;
        if ((m >> (lane & 7)) & 1u) y = __fmul_rn(read1<IN16>(a.x, row * a.x_ld + col), a.scale);
        if (RES) y = __fadd_rn(y, read1<OUT16>(a.res, row * a.res_ld + col));
        const int64_t o = row * a.out_ld + col;
        if (OUT16) static_cast<uint16_t*>(a.out)[o] = f32_to_bf16_rn(y);
        else static_cast<float*>(a.out)[o] = y;
    }
}

// 8 consecutive elements as they lie in memory (16 bytes of bf16, 32 of fp32).
template <bool B16>
struct Eight {
    uint4 a, b;
    __device__ __forceinline__ void read(const void* p, int64_t i) {
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const char*>(p) + i * (B16 ? 2 : 4));
        a = *q;
        if (!B16) b = q[1];
    }
    __device__ __forceinline__ void to(float f[8]) const {
        if (B16) {
            unpack8(a, f);
        } else {
            f[0] = __uint_as_float(a.x); f[1] = __uint_as_float(a.y);
            f[2] = __uint_as_float(a.z); f[3] = __uint_as_float(a.w);
            f[4] = __uint_as_float(b.x); f[5] = __uint_as_float(b.y);
            f[6] = __uint_as_float(b.z); f[7] = __uint_as_float(b.w);
        }
    }
};

// 8 elements a thread, `U` of them: FLAT tensors are one row (the last unit may be short),
// others have rows of whole units.
template <bool IN16, bool OUT16, bool RES, bool FLAT, int U>
__global__ void __launch_bounds__(kThreads) dropout_units_kernel(const __grid_constant__ Args a, const int64_t units,
                                                                 const uint32_t per_row) {
    const int64_t first = int64_t(blockIdx.x) * (kThreads * U) + threadIdx.x;
    const uint64_t draw = a.draw_at ? uint64_t(*a.draw_at) : a.draw;
    Eight<IN16> x[U];
    Eight<OUT16> r[U];
    int64_t row[U];
    uint32_t unit[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t q = first + k * kThreads;
        row[k] = -1;
        if (q >= units) continue;
        if (FLAT) {
            if (q * 8 + 8 > a.total) continue;  // the last, short unit
            row[k] = 0;
            x[k].read(a.x, q * 8);
            if (RES) r[k].read(a.res, q * 8);
        } else {
            row[k] = units <= UINT32_MAX ? int64_t(uint32_t(q) / per_row) : q / per_row;
            unit[k] = uint32_t(q - row[k] * per_row);
            x[k].read(a.x, row[k] * a.x_ld + int64_t(unit[k]) * 8);
            if (RES) r[k].read(a.res, row[k] * a.res_ld + int64_t(unit[k]) * 8);
        }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
        const int64_t q = first + k * kThreads;
        if (q >= units) continue;
        uint32_t c[4];
        words(a, uint64_t(q), draw, c);
        if (FLAT && row[k] < 0) {
            uint32_t m = 0;
#pragma unroll
            for (int e = 0; e < 8; ++e) m |= uint32_t(kept(a, c, e)) << e;
            for (int64_t i = q * 8; i < a.total; ++i) {
                float y = (m >> (i & 7)) & 1u ? __fmul_rn(read1<IN16>(a.x, i), a.scale) : 0.f;
                if (RES) y = __fadd_rn(y, read1<OUT16>(a.res, i));
                if (OUT16) static_cast<uint16_t*>(a.out)[i] = f32_to_bf16_rn(y);
                else static_cast<float*>(a.out)[i] = y;
            }
            continue;
        }
        float f[8], g[8];
        x[k].to(f);
        if (RES) r[k].to(g);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            f[e] = kept(a, c, e) ? __fmul_rn(f[e], a.scale) : 0.f;
            if (RES) f[e] = __fadd_rn(f[e], g[e]);
        }
        const int64_t o = FLAT ? q * 8 : row[k] * a.out_ld + int64_t(unit[k]) * 8;
        if (OUT16) {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + o) = make_uint4(
                pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        } else {
            float4* d = reinterpret_cast<float4*>(static_cast<float*>(a.out) + o);
            d[0] = make_float4(f[0], f[1], f[2], f[3]);
            d[1] = make_float4(f[4], f[5], f[6], f[7]);
        }
    }
}

bool lined_up(const void* p, int64_t ld, int64_t D, bool flat, bool b16) {
    return (reinterpret_cast<uintptr_t>(p) & 15) == 0 && (flat || (D % 8 == 0 && ld * (b16 ? 2 : 4) % 16 == 0));
}

template <bool IN16, bool OUT16, bool RES>
cudaError_t launch(Args a, int64_t N, cudaStream_t stream) {
    const bool flat = N == 1 || (a.x_ld == a.D && a.out_ld == a.D && (!RES || a.res_ld == a.D));
    const bool units = lined_up(a.x, a.x_ld, a.D, flat, IN16) && lined_up(a.out, a.out_ld, a.D, flat, OUT16) &&
                       (!RES || lined_up(a.res, a.res_ld, a.D, flat, OUT16)) && (flat || a.D / 8 <= UINT32_MAX);
    if (flat) a.D = a.x_ld = a.out_ld = a.res_ld = a.total;
    const int64_t n = units ? (a.total + 7) / 8 : (a.total + 255) / 256 * 32;  // threads' worth
    // two units a thread once that still leaves every SM eight CTAs
    const bool many = units && n >= int64_t(2) * kThreads * 8 * 152;
    const int64_t per_cta = kThreads * (many ? 2 : 1), grid = (n + per_cta - 1) / per_cta;
    if (grid > INT32_MAX) return cudaErrorInvalidConfiguration;
    const unsigned g = unsigned(grid);
    const uint32_t row = uint32_t(flat ? 1 : a.D / 8);
    if (!units) dropout_kernel<IN16, OUT16, RES><<<g, kThreads, 0, stream>>>(a);
    else if (flat && many) dropout_units_kernel<IN16, OUT16, RES, true, 2><<<g, kThreads, 0, stream>>>(a, n, row);
    else if (flat) dropout_units_kernel<IN16, OUT16, RES, true, 1><<<g, kThreads, 0, stream>>>(a, n, row);
    else if (many) dropout_units_kernel<IN16, OUT16, RES, false, 2><<<g, kThreads, 0, stream>>>(a, n, row);
    else dropout_units_kernel<IN16, OUT16, RES, false, 1><<<g, kThreads, 0, stream>>>(a, n, row);
    note_launch();
    return cudaGetLastError();
}

}  // namespace

cudaError_t dropout_launch(const DropoutArgs& d, cudaStream_t stream) {
    Args a{};
    a.x = d.x;
    a.res = d.res;
    a.out = d.out;
    a.x_ld = d.x_ld;
    a.res_ld = d.res_ld;
    a.out_ld = d.out_ld;
    a.total = d.N * d.D;
    a.D = d.D;
    a.last_dropped = uint32_t((uint64_t(d.drop) << 16) - 1);
    a.none = d.drop == 0;
    a.scale = d.drop < 65536 ? 65536.f / float(65536 - d.drop) : 0.f;
    a.draw = d.draw;
    a.draw_at = d.draw_at;
    uint32_t k0 = uint32_t(d.seed), k1 = uint32_t(d.seed >> 32);
    for (int r = 0; r < 10; ++r, k0 += 0x9E3779B9u, k1 += 0xBB67AE85u) {
        a.key[2 * r] = k0;
        a.key[2 * r + 1] = k1;
    }
    const int kind = (d.x_bf16 ? 4 : 0) | (d.out_bf16 ? 2 : 0) | (d.res ? 1 : 0);
    switch (kind) {
        case 0: return launch<false, false, false>(a, d.N, stream);
        case 1: return launch<false, false, true>(a, d.N, stream);
        case 2: return launch<false, true, false>(a, d.N, stream);
        case 3: return launch<false, true, true>(a, d.N, stream);
        case 4: return launch<true, false, false>(a, d.N, stream);
        case 5: return launch<true, false, true>(a, d.N, stream);
        case 6: return launch<true, true, false>(a, d.N, stream);
        default: return launch<true, true, true>(a, d.N, stream);
    }
}

}  // namespace df2
