// A shared projection in 8 bits (OCP e4m3, one fp32 scale per token and per
// output column) beside the adapters of the batch, for up to 64 tokens in one
// launch:
//     y[m, n] = xs[m] ws[n] sum_k x8[m, k] W8[n, k]
//             + sum_{j < rp} S[p, sl, j] B_i[n, j],   S = x A_i^T
// (sorted position p, adapter i, slice sl holding n; the second term is absent
// for tokens without an adapter and for rank-0 slots).  y is written once.
//
// What bounds it: W8 is read once, N K bytes, and everything else is small, so
// the launch is a stream of W8 with the rest hidden behind it.
//   producers (first in the grid): unit = (segment, 16 S columns), the whole
//     of K over eight waves, bf16 MFMA 16 x 16 x 32, joined through LDS.  S
//     goes to tagged exchange slots already split into the bf16 hi / lo pair
//     that the second product takes: one 32-bit word per value.
//   consumers: unit = 16 NR output columns of one slice for every token, K over
//     eight waves (v_mfma_f32_16x16x128_f8f6f4, W rows as the first operand so
//     that a lane ends with four consecutive columns of one token).  Only after
//     its share of W8 is read and multiplied does a workgroup look at the
//     slots, which are full by then; each wave then adds the deltas of every
//     eighth segment to its own partial sums, and the eight partial sums are
//     joined through LDS in a fixed order.
// A consumer waits for producers only, which wait for nothing and come first
// in the grid; the waits are bounded and report LORA_DEVERR_WAIT.
//
// Sums are fp32; S enters its product as the sum of two bf16 values (an error
// of 2^-17 of S at most); y is rounded once.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace mlora {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

// 16 x 16 x 128 on e4m3 operands (format code 0 for both), without block
// scales.  Lane l supplies row / column l % 16 and 32 values of K; which 32
// does not matter as long as both operands agree.
__device__ __forceinline__ f32x4_t mfma_e4m3(const uint4& a0, const uint4& a1, const uint4& b0,
                                             const uint4& b1, f32x4_t c) {
    const i32x8_t a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
    const i32x8_t b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

constexpr int kFpThreads = 512;
constexpr int kFpWaves = kFpThreads / kWave;
constexpr int kFpSLD = LORA_MAX_RANK + 8;      // bf16 row stride of the staged S

struct Fp8Params {
    LinearArgs a;
    const uint8_t* W;
    int64_t ldw;
    const float* w_scale;
    const uint8_t* x8;
    int64_t ldx8;
    const float* x_scale;
    const uint16_t* x;
    int64_t ldx;
    uint16_t* y;
    int64_t ldy;
    slot_t* slots;               // [64][cols]: sorted position, S column (hi / lo pair, tag)
    int jb;                      // 16-column blocks of an S row
    int n_prod;                  // producer workgroups
    int tile_start[LORA_MAX_SLICES + 1];
    WaitCtl wc;
};

// fp32 as the sum of two bf16 values, in one word
__device__ __forceinline__ uint32_t hi_lo(float f) {
    const uint32_t h = f32_to_bf16(f);
    const uint32_t l = f32_to_bf16(f - bf16_to_f32(h));
    return (h << 16) | l;
}

__device__ __forceinline__ uint4 and4(const uint4& v, uint32_t m) {
    return make_uint4(v.x & m, v.y & m, v.z & m, v.w & m);
}

// S of one segment's tokens for 16 S columns: red[wave] holds the wave's
// partial sums over its K share, joined and published by the first waves.
template <int TB>
__device__ __forceinline__ void fp8_producer(const Fp8Params& p, uint32_t tag, float4* red) {
    const LinearArgs& a = p.a;
    const int u = (int)blockIdx.x;
    const int s = u / p.jb, jb = u % p.jb;
    if (s >= a.num_segments[0]) return;
    const int id = a.req_to_lora[s];
    if (id < 0 || id >= a.L) {
        table_fault(a.err, true);
        return;
    }
    const int rp = a.rank[id];
    const int per = a.r_max / 16;
    const int sl = jb / per, j0 = (jb % per) * 16;
    if (j0 >= rp) return;
    const int p0 = a.seg_indptr[s], p1 = a.seg_indptr[s + 1];
    if (table_fault(a.err, p0 < 0 || p1 > a.M || p1 < p0)) return;
    const int ms = p1 - p0;
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const int lr = lane % 16, lq = lane / 16;
    const uint16_t* A = static_cast<const uint16_t*>(a.A) + a.a_off[id] + (int64_t)(sl * rp + j0 + lr) * a.K;
    const uint16_t* xr[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        int m = a.sorted_idx[min(p0 + min(t * 16 + lr, ms - 1), a.M - 1)];
        if (table_fault(a.err, m < 0 || m >= a.M)) m = min(max(m, 0), a.M - 1);
        xr[t] = p.x + (int64_t)m * p.ldx;
    }
    f32x4_t acc[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int steps = (a.K + 31) / 32;
    for (int i0 = wave; i0 < steps; i0 += 4 * kFpWaves) {
        uint4 va[4], vx[4][TB];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int k = (i0 + q * kFpWaves) * 32 + lq * 8;
            const int kc = min(k, a.K - 8);
            va[q] = ld16(A + kc);
            const uint32_t mk = opaque_mask(k < a.K);
#pragma unroll
            for (int t = 0; t < TB; ++t) vx[q][t] = and4(ld16(xr[t] + kc), mk);
        }
#pragma unroll
        for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int t = 0; t < TB; ++t)
                if (t * 16 < ms) acc[t] = mfma_bf16(va[q], vx[q][t], acc[t]);
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
        red[(wave * TB + t) * kWave + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    if (wave >= TB || wave * 16 >= ms) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kFpWaves; ++w) {
        const float4 t = red[(w * TB + wave) * kWave + lane];
        v.x += t.x; v.y += t.y; v.z += t.z; v.w += t.w;
    }
    const int pos = wave * 16 + lr;
    if (pos >= ms) return;
    slot_t* d = p.slots + (int64_t)(p0 + pos) * a.cols + sl * a.r_max + j0 + lq * 4;
    const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int q = 0; q < 4; ++q) slot_put(d + q, __uint_as_float(hi_lo(f[q])), tag);
}

template <int TB, int NR>
__global__ __launch_bounds__(kFpThreads) void k_linear_fp8(Fp8Params p) {
    __shared__ float4 red[kFpWaves * TB * NR * kWave];
    __shared__ uint16_t sHi[TB * 16 * kFpSLD], sLo[TB * 16 * kFpSLD];
    __shared__ int s_rp[TB * 16];
    const LinearArgs& a = p.a;
    const uint32_t tag = launch_tag();
    if ((int)blockIdx.x < p.n_prod) {
        fp8_producer<TB>(p, tag, red);
        return;
    }
    const int ct = (int)blockIdx.x - p.n_prod;
    const int tid = threadIdx.x;
    const int lane = lane_id(), wave = tid / kWave;
    const int lr = lane % 16, lq = lane / 16;
    int sl = 0;
    while (sl + 1 < a.n_sl && ct >= p.tile_start[sl + 1]) ++sl;
    const int n0 = (int)(a.slice_off[sl] + (int64_t)(ct - p.tile_start[sl]) * (16 * NR));
    const int n1 = (int)min((int64_t)n0 + 16 * NR, a.slice_off[sl + 1]);

    // ---- base product
    const uint8_t* Wr[NR];
#pragma unroll
    for (int r = 0; r < NR; ++r) Wr[r] = p.W + (int64_t)min(n0 + r * 16 + lr, n1 - 1) * p.ldw;
    const uint8_t* xr[TB];
    float xs[TB];
    int tok[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        int m = a.sorted_idx[min(t * 16 + lr, a.M - 1)];
        if (table_fault(a.err, m < 0 || m >= a.M)) m = (m < 0 || m >= a.M) ? -1 : m;
        tok[t] = t * 16 + lr < a.M ? m : -1;
        m = max(m, 0);
        xr[t] = p.x8 + (int64_t)m * p.ldx8;
        xs[t] = p.x_scale[m];
    }
    f32x4_t acc[NR][TB];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int U = TB * NR >= 8 ? 1 : TB >= 2 || NR >= 2 ? 2 : 4;   // K steps whose loads are in flight together
    const int steps = (a.K + 127) / 128;
    for (int i0 = wave; i0 < steps; i0 += U * kFpWaves) {
        uint4 vw[U][NR][2], vx[U][TB][2];
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const int k = (i0 + q * kFpWaves) * 128 + h * 64 + lq * 16;
                const int kc = min(k, a.K - 16);
                const uint32_t mk = opaque_mask(k < a.K);
#pragma unroll
                for (int r = 0; r < NR; ++r) vw[q][r][h] = ld16(Wr[r] + kc);
#pragma unroll
                for (int t = 0; t < TB; ++t) vx[q][t][h] = and4(ld16(xr[t] + kc), mk);
            }
#pragma unroll
        for (int q = 0; q < U; ++q)
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int t = 0; t < TB; ++t)
                    acc[r][t] = mfma_e4m3(vw[q][r][0], vw[q][r][1], vx[q][t][0], vx[q][t][1], acc[r][t]);
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
        float ws[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) ws[q] = p.w_scale[min(n0 + r * 16 + lq * 4 + q, n1 - 1)];
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[r][t][q] *= xs[t] * ws[q];
    }

    // ---- deltas: lane s holds segment s (at most 64 of them)
    const int nseg = a.num_segments[0];
    const int seg = min(lane, a.s_max - 1);
    int q_id = a.req_to_lora[seg];
    const int q_p0 = a.seg_indptr[seg], q_p1 = a.seg_indptr[seg + 1];
    const bool seg_ok = lane < nseg && q_id >= 0 && q_id < a.L;
    const bool range_ok = q_p0 >= 0 && q_p1 >= q_p0 && q_p1 <= a.M;
    table_fault(a.err, lane < nseg && !(seg_ok && range_ok));
    q_id = seg_ok ? q_id : 0;
    const int q_rp = seg_ok && (!kTableChecks || range_ok) ? a.rank[q_id] : 0;
    const int64_t q_bo = a.b_off[q_id];
    if (__ballot(q_rp > 0) != 0ull) {
        if (tid < TB * 16) s_rp[tid] = 0;
        __syncthreads();
        if (wave == 0 && q_rp > 0)
            for (int i = max(q_p0, 0); i < min(q_p1, a.M); ++i) s_rp[i] = q_rp;
        __syncthreads();
        // the slots of every position's own rank; the others stay zero
        bool lost = false;
        for (int e = tid; e < TB * 16 * a.r_max; e += kFpThreads) {
            const int pos = e / a.r_max, j = e % a.r_max;
            uint32_t w = 0;
            if (j < s_rp[pos]) {
                const slot_t* src = p.slots + (int64_t)pos * a.cols + sl * a.r_max + j;
                const uint32_t want = tag ^ p.wc.poll_xor;
                slot_t v = slot_load(src);
                int spin = 0;
                while (!slot_full(v, want) && spin < p.wc.max_spin) {
                    __builtin_amdgcn_s_sleep(1);
                    v = slot_load(src);
                    ++spin;
                }
                lost |= !slot_full(v, want);
                w = (uint32_t)v;
            }
            sHi[pos * kFpSLD + j] = (uint16_t)(w >> 16);
            sLo[pos * kFpSLD + j] = (uint16_t)w;
        }
        if (lost) atomicOr(a.err, LORA_DEVERR_WAIT);
        __syncthreads();
        for (int s = wave; s < nseg; s += kFpWaves) {
            const int rp = __builtin_amdgcn_readlane(q_rp, s);
            if (rp == 0) continue;
            const int p0 = __builtin_amdgcn_readlane(q_p0, s), p1 = __builtin_amdgcn_readlane(q_p1, s);
            const uint16_t* B = static_cast<const uint16_t*>(a.B) + readlane64(q_bo, s);
#pragma unroll
            for (int j = 0; j < LORA_MAX_RANK / 32; ++j) {
                const int jj = j * 32 + lq * 8;
                if (j * 32 >= rp) continue;
                const uint32_t mj = opaque_mask(jj < rp);
                uint4 b[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r)
                    b[r] = and4(ld16(B + (int64_t)min(n0 + r * 16 + lr, n1 - 1) * rp + min(jj, rp - 8)), mj);
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    if (t * 16 >= p1 || t * 16 + 16 <= p0) continue;
                    const int pos = t * 16 + lr;
                    const uint32_t mp = opaque_mask(pos >= p0 && pos < p1 && jj < rp);
                    const uint4 h = and4(*reinterpret_cast<const uint4*>(sHi + pos * kFpSLD + jj), mp);
                    const uint4 l = and4(*reinterpret_cast<const uint4*>(sLo + pos * kFpSLD + jj), mp);
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        acc[r][t] = mfma_bf16(b[r], h, acc[r][t]);
                        acc[r][t] = mfma_bf16(b[r], l, acc[r][t]);
                    }
                }
            }
        }
    }

    // ---- join the eight partial sums; four columns of one token per thread
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t)
            red[(wave * NR * TB + r * TB + t) * kWave + lane] =
                make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
    __syncthreads();
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            if ((r * TB + t) % kFpWaves != wave) continue;
            float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int w = 0; w < kFpWaves; ++w) {
                const float4 f = red[(w * NR * TB + r * TB + t) * kWave + lane];
                v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
            }
            const int n = n0 + r * 16 + lq * 4;          // slices are multiples of 8 wide
            if (tok[t] >= 0 && n < n1)
                *reinterpret_cast<uint2*>(p.y + (int64_t)tok[t] * p.ldy + n) =
                    make_uint2(f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16),
                               f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16));
        }
}

template <int TB, int NR>
hipError_t launch_linear_fp8_as(Fp8Params& p, hipStream_t st) {
    int t = 0;
    for (int s = 0; s < p.a.n_sl; ++s) {
        p.tile_start[s] = t;
        t += (int)((p.a.slice_off[s + 1] - p.a.slice_off[s] + 16 * NR - 1) / (16 * NR));
    }
    p.tile_start[p.a.n_sl] = t;
    p.jb = p.a.cols / 16;
    p.n_prod = p.a.s_max * p.jb;
    hipLaunchKernelGGL((k_linear_fp8<TB, NR>), dim3((unsigned)(p.n_prod + t)), dim3(kFpThreads), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_linear_fp8(const LinearArgs& a, const void* W8, int64_t ldw, const float* w_scale,
                             const void* x8, int64_t ldx8, const float* x_scale, const void* x,
                             int64_t ldx, void* y, int64_t ldy, void* ws, hipStream_t st) {
    Fp8Params p{};
    p.a = a;
    p.W = static_cast<const uint8_t*>(W8);
    p.ldw = ldw;
    p.w_scale = w_scale;
    p.x8 = static_cast<const uint8_t*>(x8);
    p.ldx8 = ldx8;
    p.x_scale = x_scale;
    p.x = static_cast<const uint16_t*>(x);
    p.ldx = ldx;
    p.y = static_cast<uint16_t*>(y);
    p.ldy = ldy;
    p.slots = reinterpret_cast<slot_t*>(static_cast<char*>(ws) + linear_ws_layout(0, a.K, a.cols).slots);
    p.wc = wait_ctl();
    if (a.M <= 16) return launch_linear_fp8_as<1, 1>(p, st);
    if (a.M <= 32) return launch_linear_fp8_as<2, 1>(p, st);
    return launch_linear_fp8_as<4, 2>(p, st);
}

}  // namespace mlora
