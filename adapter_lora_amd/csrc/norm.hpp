// Root-mean-square norm of rows with the residual's addition before it and
// an output in 8 bits (OCP e4m3 or integers, one fp32 scale per row) beside or
// instead of the output in the storage type.  With h = x + residual in fp32:
//     residual_out = round(h)
//     v            = h * rsqrt(mean(h^2) + eps) * weight
//     out          = round(v)
//     scale        = max|v| / 448,   out8 = e4m3(v / scale)
//     scale        = max|v| / 127,   out8 = the integer nearest to v / scale
// and, without the norm, v = x (weights at load time, activations).
//
// One pass: a row's values stay in registers between the two uses, so x and
// the residual are read once and every output is written once; the row's sum
// of squares and its largest |h * weight| are reduced together (the norm's
// factor is common to the row, so max|v| = rsqrt(..) * max|h * weight|).
// Statistics and products are fp32; each output is rounded once, from the
// unrounded v or h.
//
// What bounds it: every operand crosses HBM once.  2048 rows of 4096 in bf16
// with the residual and all outputs 16.3 us (75.5 MB, 4.6 TB/s; a large copy
// reaches 5.1), 4099 rows of 5128 in fp32 to fp32 37.4 (168 MB, 4.5), a weight of
// 28672 x 4096 to 8 bits 72.9 (352 MB, 4.8; 84 with the norm's branches in the same
// kernel and clamps before the conversion: the arithmetic of a value counts), to
// integers 72 to 78.  32 rows 3.3 to 4.6 us, a launch and two round trips; few long rows
// to integers 5.2 (64 of 14336, to e4m3 3.9: the correction of ties).
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace mlora {

constexpr float kE4M3Max = 448.f;

// 8 fp32 values to 8 storage elements
__device__ __forceinline__ void st8(float* p, const float* v) {
    *reinterpret_cast<float4*>(p) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(v[4], v[5], v[6], v[7]);
}
__device__ __forceinline__ void st8(uint16_t* p, const float* v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16(v[2 * i]) | (f32_to_bf16(v[2 * i + 1]) << 16);
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}

// Four fp32 values of at most 448 (1 + 2^-22) to four e4m3 bytes, round to nearest
// even: the largest finite value, 448, takes everything below 464, so a last-bit
// excess of v / scale needs no clamp.  NaN stays NaN.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float d) {
    int r = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    r = __builtin_amdgcn_cvt_pk_fp8_f32(c, d, r, true);
    return (uint32_t)r;
}

// The integer nearest to v / s, ties to the even one, in the low byte, for
// |v| <= 127 s (1 + 2^-23) and inv = 1 / s.  The sum v inv + 1.5 2^23 rounds the
// product to an integer at once and leaves it in its low bits; r = v - q s is
// exact (q has 7 bits, and next to s the values lie as close as v's own), so |r|
// against s / 2 tells whether the reciprocal's last bit took the wrong side.
constexpr float kIntMagic = 12582912.f;
__device__ __forceinline__ uint32_t int8_of(float v, float inv, float s, float& r) {
    const float m = fmaf(v, inv, kIntMagic);
    r = fmaf(kIntMagic - m, s, v);
    return __float_as_uint(m);
}

// Eight values to bytes.  A quotient's last bit matters next to a tie only: one
// branch over all eight (bf16 rows have many values of half the largest one,
// 63.5 scales, so the side is the scale's own rounding and cannot be left open).
__device__ __forceinline__ uint2 pack_int8(const float (&v)[8], float inv, float s) {
    uint32_t q[8];
    float r[8], far = 0.f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        q[e] = int8_of(v[e], inv, s, r[e]);
        far = fmaxf(far, fabsf(r[e]));
    }
    const float h = 0.5f * s;
    if (far >= h) {                      // infinite and NaN scales: no |r| reaches them
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const bool up = r[e] > h || (r[e] == h && (q[e] & 1u));
            const bool down = r[e] < -h || (r[e] == -h && (q[e] & 1u));
            q[e] += up ? 1u : down ? 0xffffffffu : 0u;
        }
    }
    const uint32_t a = __builtin_amdgcn_perm(q[1], q[0], 0x0c0c0400u), b = __builtin_amdgcn_perm(q[3], q[2], 0x04000c0cu);
    const uint32_t c = __builtin_amdgcn_perm(q[5], q[4], 0x0c0c0400u), d = __builtin_amdgcn_perm(q[7], q[6], 0x04000c0cu);
    return make_uint2(a | b, c | d);
}

// Largest of the wavefront's values, as unsigned integers (wave-uniform).
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) {
        const uint32_t t = (uint32_t)__shfl_xor((int)v, o, kWave);
        v = v > t ? v : t;
    }
    return v;
}

// WPR wavefronts per row, CPL chunks of 8 values per lane: a row of up to
// 512 * WPR * CPL values.  Without NORM: v = x, out8 and scale alone.
template <typename T, int WPR, int CPL, bool NORM, bool INT8>
__global__ __launch_bounds__(WPR * kWave < 256 ? 256 : WPR * kWave) void k_rms_norm(NormParams p) {
    constexpr int kRows = WPR < 4 ? 4 / WPR : 1;          // rows per workgroup
    __shared__ float s_sum[kRows * WPR];
    __shared__ uint32_t s_max[kRows * WPR];
    const int wave = (int)threadIdx.x / kWave;
    const int lane = lane_id();
    const int wr = wave % WPR;
    const int64_t row = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * kRows + wave / WPR;
    const bool live = row < p.M;
    const int64_t m = live ? row : p.M - 1;
    const T* x = static_cast<const T*>(p.x) + m * p.ldx;
    const T* res = static_cast<const T*>(p.res) + m * p.ldr;
    const T* w = static_cast<const T*>(p.w);

    float h[CPL][8], g[CPL][8];
    float sum = 0.f;
    uint32_t top = 0;
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int k = ((c * WPR + wr) * kWave + lane) * 8;
#pragma unroll
        for (int e = 0; e < 8; ++e) h[c][e] = 0.f, g[c][e] = 0.f;
        if (k < p.K) {
            Io<T>::ld8(x + k, h[c]);
            if constexpr (NORM) Io<T>::ld8(w + k, g[c]);
            if (NORM && p.res) {
                float r[8];
                Io<T>::ld8(res + k, r);
#pragma unroll
                for (int e = 0; e < 8; ++e) h[c][e] += r[e];
            }
        }
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            if constexpr (NORM) sum += h[c][e] * h[c][e];
            // |v| as an integer: ordered like the value, with NaN above
            // infinity, so a NaN of the row reaches its scale
            const float v = NORM ? h[c][e] * g[c][e] : h[c][e];
            const uint32_t u = __float_as_uint(v) & 0x7fffffffu;
            top = top > u ? top : u;
        }
    if constexpr (NORM) sum = wave_total(sum);
    top = wave_umax(top);
    if constexpr (WPR > 1) {
        if (lane == 0) s_sum[wave] = sum, s_max[wave] = top;
        __syncthreads();
        sum = 0.f;
        top = 0;
        const int w0 = wave / WPR * WPR;
#pragma unroll
        for (int i = 0; i < WPR; ++i) {
            sum += s_sum[w0 + i];
            const uint32_t t = s_max[w0 + i];
            top = top > t ? top : t;
        }
    }
    if (!live) return;
    const float rstd = NORM ? 1.f / sqrtf(sum / (float)p.K + p.eps) : 1.f;
    float inv = 0.f, den = 0.f, s8 = 0.f;
    if (p.out8) {
        const float amax = __uint_as_float(top) * rstd;
        // the smallest normal number bounds the scale, so 1 / scale is finite
        float s = amax / (INT8 ? 127.f : kE4M3Max);
        s = s < 1.17549435e-38f ? (amax == 0.f ? 1.f : 1.17549435e-38f) : s;
        inv = 1.f / s;
        s8 = s;
        den = s < INFINITY ? s : 0.f;
        if (wr == 0 && lane == 0) p.scale[m] = s;
    }
#pragma unroll
    for (int c = 0; c < CPL; ++c) {
        const int k = ((c * WPR + wr) * kWave + lane) * 8;
        if (k >= p.K) continue;
        if (NORM && p.res_out) st8(static_cast<T*>(p.res_out) + m * p.ldro + k, h[c]);
        float v[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = NORM ? h[c][e] * rstd * g[c][e] : h[c][e];
        if (NORM && p.out) st8(static_cast<T*>(p.out) + m * p.ldo + k, v);
        if constexpr (INT8) {
            uint2 q = pack_int8(v, inv, s8);
            if (s8 == INFINITY) {        // the row's infinities take the largest integer
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t b = fabsf(v[e]) < INFINITY ? 0u : v[e] > 0.f ? 0x7fu : 0x81u;
                    uint32_t& w = e < 4 ? q.x : q.y;
                    w = (w & ~(0xffu << 8 * (e % 4))) | b << 8 * (e % 4);
                }
            }
            *reinterpret_cast<uint2*>(p.out8 + m * p.ldo8 + k) = q;
        } else if (p.out8) {
            // v / scale, the reciprocal's product corrected by its residue:
            // bf16 values over a bf16 maximum are often ties of e4m3, and a
            // last-bit error of the quotient would round them the wrong way
            // (an infinite scale: den = 0 leaves finite values at 0)
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float t = v[e] * inv;
                v[e] = fmaf(fmaf(-t, den, v[e]), inv, t);
            }
            const uint2 q = make_uint2(pack_e4m3(v[0], v[1], v[2], v[3]),
                                       pack_e4m3(v[4], v[5], v[6], v[7]));
            *reinterpret_cast<uint2*>(p.out8 + m * p.ldo8 + k) = q;
        }
    }
}

template <typename T, int WPR, int CPL>
hipError_t launch_norm_as(const NormParams& p, hipStream_t st) {
    constexpr int kRows = WPR < 4 ? 4 / WPR : 1;
    constexpr int kThreads = WPR * kWave < 256 ? 256 : WPR * kWave;
    // a grid has fewer than 2^32 threads along x: more rows continue along y
    const unsigned wgs = (unsigned)(((int64_t)p.M + kRows - 1) / kRows);
    const unsigned gx = wgs < (1u << 21) ? wgs : 1u << 21;
    const dim3 grid(gx, (wgs + gx - 1) / gx);
    if (p.int8) {                    // out8 is there (checked by the caller)
        if (p.w) hipLaunchKernelGGL((k_rms_norm<T, WPR, CPL, true, true>), grid, dim3(kThreads), 0, st, p);
        else hipLaunchKernelGGL((k_rms_norm<T, WPR, CPL, false, true>), grid, dim3(kThreads), 0, st, p);
    } else {
        if (p.w) hipLaunchKernelGGL((k_rms_norm<T, WPR, CPL, true, false>), grid, dim3(kThreads), 0, st, p);
        else hipLaunchKernelGGL((k_rms_norm<T, WPR, CPL, false, false>), grid, dim3(kThreads), 0, st, p);
    }
    return hipGetLastError();
}

// A row is spread over as many wavefronts as have work: its loads are all in
// flight at once, in few registers.  Measured against one wavefront (four past K =
// 4096) and against half the wavefronts, in a graph over twelve inputs in turn, each
// with all outputs (colder than the trace's 16.3 us for the second): 32 x 4096 4.2 / 10.4
// / 4.9 us, 2048 x 4096 19.7 / 24.3 / 19.8, 64 x 14336 7.3 / 12.4 / 8.6, 2048 x 14336 58.0 /
// 64.8 / 59.1; to 8 bits alone 3.3 / 4.6 / 3.4, 8.8 / 10.1 / 8.3, 3.8 / 4.7 / 3.9, 20.1 / 21.7 /
// 20.5.
template <typename T>
hipError_t launch_norm_t(const NormParams& p, hipStream_t st) {
    const int chunks = (p.K + 511) / 512;        // 512 values per wavefront and chunk
    if (chunks <= 1) return launch_norm_as<T, 1, 1>(p, st);
    if (chunks <= 2) return launch_norm_as<T, 2, 1>(p, st);
    if (chunks <= 4) return launch_norm_as<T, 4, 1>(p, st);
    if (chunks <= 8) return launch_norm_as<T, 8, 1>(p, st);
    if (chunks <= 16) return launch_norm_as<T, 16, 1>(p, st);
    if (chunks <= 32) return launch_norm_as<T, 16, 2>(p, st);
    return launch_norm_as<T, 16, 4>(p, st);      // K <= 32768 (checked by the caller)
}

hipError_t launch_rms_norm(int dtype, const NormParams& p, hipStream_t st) {
    return dtype == LORA_BF16 ? launch_norm_t<uint16_t>(p, st) : launch_norm_t<float>(p, st);
}

}  // namespace mlora
