// A whole Mixture-of-Experts layer for up to 64 tokens, adapters included, in
// two launches:
//     logits = x Wr^T,  p = softmax(logits),  the topk largest (ties to the
//     lowest expert), their weights p or p / sum(p)
//     (g, u) = W_gu[e] x + B_gu[l, e] (A_gu[l, e] x)      per (token, expert)
//     h      = weight * silu(g) * u                       rounded to bf16
//     out    = sum over the token's experts of W_d[e] h + B_d[l, e] (A_d[l, e] h)
//
// What bounds it: each expert that some token chose is read once, 3 H I
// values; tokens, adapters and the router are small beside that.  Both
// launches are streams of expert rows through bf16 MFMA (16 x 16 x 32, the
// expert's rows as the first operand, tokens as columns), with the rest done
// by workgroups that come first in the grid and overlap the stream:
//   first launch   router (one workgroup per token), then one per (token,
//                  expert) pair that computes its adapter's A_gu x, then the
//                  consumers, which walk (expert, 16 gate and 16 up rows);
//   second launch  one per pair for A_d h, then the consumers of 16 output
//                  rows, all chosen experts in one sum: the routing weight is
//                  already in h, so a token's experts simply add up.
// Results cross workgroups of a launch through tagged exchange slots
// (common.hpp); whoever waits comes later in the grid than whom it waits for,
// and every wait is bounded.
//
// The weight is folded into h before h is rounded, so there is one rounding
// where a separate weighting of the down product would have a second sum.
// Experts in 8 bits (e4m3, one fp32 scale per row) are widened to bf16, which
// is exact, and their scale is applied to the fp32 sums.  Router sums, softmax,
// gate / up sums and the output's sum are fp32; S = A x enters its product as
// a bf16 hi / lo pair.
#pragma once

#include "common.hpp"
#include "kernels.hpp"

namespace mlora {

constexpr int kMdThreads = 512;
constexpr int kMdWaves = kMdThreads / kWave;
constexpr int kMdMaxE = 256;
constexpr int kMdMaxPairs = LORA_DECODE_MAX_M * 16;

__device__ __forceinline__ uint32_t md_hi_lo(float f) {
    const uint32_t h = f32_to_bf16(f);
    const uint32_t l = f32_to_bf16(f - bf16_to_f32(h));
    return (h << 16) | l;
}

__device__ __forceinline__ uint32_t slot_wait(const slot_t* s, uint32_t want, int max_spin, bool* lost) {
    slot_t v = slot_load(s);
    int spin = 0;
    while (!slot_full(v, want) && spin < max_spin) {
        __builtin_amdgcn_s_sleep(1);
        v = slot_load(s);
        ++spin;
    }
    *lost |= !slot_full(v, want);
    return (uint32_t)v;
}

typedef __bf16 md_bf16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ float md_dot8(const uint4& a, const uint4& b, float c) {
    const uint32_t aw[4] = {a.x, a.y, a.z, a.w}, bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(md_bf16x2_t, aw[i]),
                                            __builtin_bit_cast(md_bf16x2_t, bw[i]), c, false);
    return c;
}

// 16 e4m3 bytes to 16 bf16 values (exact), as two MFMA operands
__device__ __forceinline__ void widen16(const uint4& q, uint4& a, uint4& b) {
    typedef __bf16 v2 __attribute__((ext_vector_type(2)));
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        o[2 * i] = __builtin_bit_cast(uint32_t, (v2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, false));
        o[2 * i + 1] = __builtin_bit_cast(uint32_t, (v2)__builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w[i], 1.0f, true));
    }
    a = make_uint4(o[0], o[1], o[2], o[3]);
    b = make_uint4(o[4], o[5], o[6], o[7]);
}

// Adapter of token m, or -1 (none, disabled, or outside the table).
__device__ __forceinline__ int md_adapter(const MoeDecodeParams& p, int m) {
    if (p.L == 0) return -1;
    const int l = p.ids[m];
    if (l < 0 || l >= p.L) return -1;
    return p.enabled[l] != 0 ? l : -1;
}

// ---------------------------------------------------------------- router
__device__ __forceinline__ void md_router(const MoeDecodeParams& p, uint32_t tag, int m, float* s_logit) {
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const uint16_t* x = p.x + (int64_t)m * p.ldx;
    for (int e = wave; e < p.E; e += kMdWaves) {
        const uint16_t* w = p.router + (int64_t)e * p.H;
        float c = 0.f;
#pragma unroll 4
        for (int k = lane * 8; k < p.H; k += kWave * 8) c = md_dot8(ld16(x + k), ld16(w + k), c);
        c = wave_total(c);
        if (lane == 0) s_logit[e] = c;
    }
    __syncthreads();
    if (wave != 0) return;
    // four experts a lane; a logit as an ordered integer, so that the largest
    // (logit, lowest expert) is one 64-bit maximum
    float v[4];
    unsigned long long key[4];
    float mx = -INFINITY;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const int e = q * kWave + lane;
        const bool in = e < p.E;
        v[q] = in ? s_logit[e] : -INFINITY;
        mx = fmaxf(mx, v[q]);
        const uint32_t b = __float_as_uint(v[q]);
        const uint32_t o = (b & 0x80000000u) ? ~b : (b | 0x80000000u);
        key[q] = in ? ((unsigned long long)o << 32) | (uint32_t)(kMdMaxE - 1 - e) : 0ull;
    }
#pragma unroll
    for (int o = kWave / 2; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor(mx, o, kWave));
    float sum = 0.f;
#pragma unroll
    for (int q = 0; q < 4; ++q) sum += q * kWave + lane < p.E ? expf(v[q] - mx) : 0.f;
    sum = wave_total(sum);
    // lane j keeps the j-th choice
    int mine = 0;
    float pw = 0.f, chosen = 0.f;
    for (int j = 0; j < p.topk; ++j) {
        unsigned long long best = 0ull;
#pragma unroll
        for (int q = 0; q < 4; ++q) best = key[q] > best ? key[q] : best;
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) {
            const unsigned long long t = __shfl_xor(best, o, kWave);
            best = t > best ? t : best;
        }
        const int e = kMdMaxE - 1 - (int)(uint32_t)best;
#pragma unroll
        for (int q = 0; q < 4; ++q)
            if (q * kWave + lane == e) key[q] = 0ull;
        const float w = expf(s_logit[e] - mx) / sum;
        chosen += w;
        if (lane == j) mine = e, pw = w;
    }
    if (lane < p.topk) {
        if (p.renorm) pw /= chosen;
        const int f = m * p.topk + lane, P = p.M * p.topk;
        slot_put(p.route + f, __int_as_float(mine), tag);
        slot_put(p.route + P + f, pw, tag);
        p.route_ids[f] = mine;
        if (p.out_ids) p.out_ids[f] = mine;
        if (p.out_w) p.out_w[f] = pw;
    }
}

// ---------------------------------------------------------------- shrink of one pair
// S[j] = A[j, :] . v over K for the rank's r rows: wave w takes rows w, w + 8, ...
__device__ __forceinline__ void md_shrink(const uint16_t* A, const uint16_t* v, int K, int r, slot_t* S,
                                          uint32_t tag) {
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    for (int j = wave * 2; j < r; j += 2 * kMdWaves) {         // r is a multiple of 16
        const uint16_t* a0 = A + (int64_t)j * K;
        const uint16_t* a1 = a0 + K;
        float c0 = 0.f, c1 = 0.f;
#pragma unroll 4
        for (int k = lane * 8; k < K; k += kWave * 8) {
            const uint4 t = ld16(v + k);
            c0 = md_dot8(ld16(a0 + k), t, c0);
            c1 = md_dot8(ld16(a1 + k), t, c1);
        }
        c0 = wave_total(c0);
        c1 = wave_total(c1);
        if (lane == 0) {
            slot_put(S + j, __uint_as_float(md_hi_lo(c0)), tag);
            slot_put(S + j + 1, __uint_as_float(md_hi_lo(c1)), tag);
        }
    }
}

// ---------------------------------------------------------------- routing tables in LDS
struct MdRoute {
    unsigned long long mask[kMdMaxE];      // tokens of each expert
    int16_t active[kMdMaxE];               // experts with tokens, ascending
    int16_t exp_[kMdMaxPairs];             // expert of a pair, -1: none
    int n_active;
};

// After exp_ is filled: masks and the list of active experts.  Ends with a barrier.
__device__ __forceinline__ void md_tables(const MoeDecodeParams& p, MdRoute& r) {
    const int tid = threadIdx.x, lane = lane_id();
    const int P = p.M * p.topk;
    for (int e = tid; e < kMdMaxE; e += kMdThreads) r.mask[e] = 0ull;
    __syncthreads();
    for (int f = tid; f < P; f += kMdThreads)
        if (r.exp_[f] >= 0) atomicOr(&r.mask[r.exp_[f]], 1ull << (f / p.topk));
    __syncthreads();
    if (tid < kWave) {
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += kWave) {
            const bool on = e0 + lane < p.E && r.mask[e0 + lane] != 0ull;
            const unsigned long long b = __ballot(on);
            if (on) r.active[n + __popcll(b & ((1ull << lane) - 1ull))] = (int16_t)(e0 + lane);
            n += __popcll(b);
        }
        if (lane == 0) r.n_active = n;
    }
    __syncthreads();
}

// 16 rows of an expert's weight, one 64-value block of K: two operands a lane
// (values 16 lq .. 16 lq + 15 of the block).
template <bool W8> struct MdRow;
template <> struct MdRow<false> {
    uint4 q[2];
    __device__ __forceinline__ void load(const void* row, int k) {
        q[0] = ld16(static_cast<const uint16_t*>(row) + k);
        q[1] = ld16(static_cast<const uint16_t*>(row) + k + 8);
    }
    __device__ __forceinline__ void operands(uint4& a, uint4& b) const { a = q[0]; b = q[1]; }
};
template <> struct MdRow<true> {
    uint4 q;
    __device__ __forceinline__ void load(const void* row, int k) { q = ld16(static_cast<const uint8_t*>(row) + k); }
    __device__ __forceinline__ void operands(uint4& a, uint4& b) const { widen16(q, a, b); }
};

__device__ __forceinline__ uint4 md_and(const uint4& v, uint32_t m) {
    return make_uint4(v.x & m, v.y & m, v.z & m, v.w & m);
}

// Deltas of one expert added to acc: for every adapter among the expert's
// tokens (lane t of `ad`: adapter of column t, -1 none; `pair`: its pair
// index), B rows times the S columns of its tokens.  Groups are dealt to the
// waves in turn, `deal` counting them across calls.
template <int NT, int TB>
__device__ __forceinline__ void md_delta(const MoeDecodeParams& p, const uint16_t* B, int64_t per_l,
                                         const int64_t* row, const slot_t* S, int ad, int pair, int wave,
                                         int& deal, uint32_t want, bool* lost, f32x4_t (&acc)[NT][TB]) {
    const int lane = lane_id(), lr = lane % 16, lq = lane / 16;
    unsigned long long rem = __ballot(ad >= 0);
    while (rem) {
        const int l = __builtin_amdgcn_readlane(ad, __ffsll((long long)rem) - 1);
        const unsigned long long same = __ballot(ad == l);
        rem &= ~same;
        if (deal++ % kMdWaves != wave) continue;
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            if (((same >> (16 * t)) & 0xffffull) == 0ull) continue;
            const bool on = (same >> (16 * t + lr)) & 1ull;
            const int f = __shfl(pair, 16 * t + lr, kWave);
            for (int j = lq * 8; j - lq * 8 < p.r; j += 32) {
                uint32_t w[8];
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    w[q] = on && j < p.r ? slot_wait(S + (int64_t)f * p.r + j + q, want, p.wc.max_spin, lost) : 0u;
                uint4 h, lo;
                h.x = (w[0] >> 16) | (w[1] & 0xffff0000u); lo.x = (w[0] & 0xffffu) | (w[1] << 16);
                h.y = (w[2] >> 16) | (w[3] & 0xffff0000u); lo.y = (w[2] & 0xffffu) | (w[3] << 16);
                h.z = (w[4] >> 16) | (w[5] & 0xffff0000u); lo.z = (w[4] & 0xffffu) | (w[5] << 16);
                h.w = (w[6] >> 16) | (w[7] & 0xffff0000u); lo.w = (w[6] & 0xffffu) | (w[7] << 16);
                const uint32_t mj = opaque_mask(j < p.r);
#pragma unroll
                for (int n = 0; n < NT; ++n) {
                    const uint4 b = md_and(ld16(B + l * per_l + row[n] * p.r + min(j, p.r - 8)), mj);
                    acc[n][t] = mfma_bf16(b, h, acc[n][t]);
                    acc[n][t] = mfma_bf16(b, lo, acc[n][t]);
                }
            }
        }
    }
}

// ---------------------------------------------------------------- first launch
struct MdUnit {              // one (expert, 16 gate + 16 up rows) unit
    int e, n0, ne;
};

template <bool W8, int TB>
__device__ __forceinline__ void md_gate_up(const MoeDecodeParams& p, const MdUnit& u, const int16_t* s_tok,
                                           const int16_t* s_pair, const int16_t* s_ad, const float* s_w,
                                           float4* red, uint32_t want, bool* lost) {
    constexpr int kBytes = W8 ? 1 : 2;
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    const int lr = lane % 16, lq = lane / 16;
    const int gi = min(u.n0 + lr, p.I - 1);
    const int64_t row_g = (int64_t)u.e * 2 * p.I + gi, row_u = row_g + p.I;
    const char* W = static_cast<const char*>(p.W_gu);
    const void* rg = W + row_g * p.H * kBytes;
    const void* ru = W + row_u * p.H * kBytes;
    const uint16_t* xr[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) xr[t] = p.x + (int64_t)s_tok[min(t * 16 + lr, u.ne - 1)] * p.ldx;
    f32x4_t acc[2][TB];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[n][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    constexpr int U = TB == 1 ? 4 : TB == 2 ? 3 : 2;
    const int blocks = (p.H + 63) / 64;
    for (int b0 = wave; b0 < blocks; b0 += U * kMdWaves) {
        MdRow<W8> g[U], v[U];
        uint4 xv[U][TB][2];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int k = (b0 + q * kMdWaves) * 64 + lq * 16;
            // H is a multiple of 8: a lane's second half may lie past the end
            const int kc = min(k, p.H - (W8 ? 16 : 8)), kd = min(k + 8, p.H - 8);
            if constexpr (W8) {
                g[q].load(rg, kc);
                v[q].load(ru, kc);
            } else {
                g[q].q[0] = ld16(static_cast<const uint16_t*>(rg) + kc);
                g[q].q[1] = ld16(static_cast<const uint16_t*>(rg) + kd);
                v[q].q[0] = ld16(static_cast<const uint16_t*>(ru) + kc);
                v[q].q[1] = ld16(static_cast<const uint16_t*>(ru) + kd);
            }
            const uint32_t m0 = opaque_mask(k < p.H), m1 = opaque_mask(k + 8 < p.H);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                xv[q][t][0] = md_and(ld16(xr[t] + min(k, p.H - 8)), m0);
                xv[q][t][1] = md_and(ld16(xr[t] + kd), m1);
            }
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            uint4 a, b, c, d;
            g[q].operands(a, b);
            v[q].operands(c, d);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                acc[0][t] = mfma_bf16(a, xv[q][t][0], acc[0][t]);
                acc[1][t] = mfma_bf16(c, xv[q][t][0], acc[1][t]);
                acc[0][t] = mfma_bf16(b, xv[q][t][1], acc[0][t]);
                acc[1][t] = mfma_bf16(d, xv[q][t][1], acc[1][t]);
            }
        }
    }
    if constexpr (W8) {
        const float* sg = p.s_gu + (int64_t)u.e * 2 * p.I;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const int n = min(u.n0 + lq * 4 + q, p.I - 1);
            const float a = sg[n], b = sg[n + p.I];
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[0][t][q] *= a, acc[1][t][q] *= b;
        }
    }
    if (p.L > 0) {
        const int c = min(lane, u.ne - 1);
        const int ad = lane < u.ne ? s_ad[c] : -1;
        int deal = 0;
        const int64_t row[2] = {row_g, row_u};
        md_delta<2, TB>(p, p.B_gu, (int64_t)p.E * 2 * p.I * p.r, row, p.S_gu, ad, s_pair[c], wave, deal, want,
                        lost, acc);
    }
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int t = 0; t < TB; ++t)
            red[((wave * 2 + n) * TB + t) * kWave + lane] =
                make_float4(acc[n][t][0], acc[n][t][1], acc[n][t][2], acc[n][t][3]);
    __syncthreads();
    const int pos = wave * 16 + lr, n = u.n0 + lq * 4;       // wave t < TB finishes token block t
    if (wave < TB && pos < u.ne && n < p.I) {
        float g[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kMdWaves; ++w) {
            const float4 a = red[((w * 2) * TB + wave) * kWave + lane];
            const float4 b = red[((w * 2 + 1) * TB + wave) * kWave + lane];
            g[0] += a.x; g[1] += a.y; g[2] += a.z; g[3] += a.w;
            v[0] += b.x; v[1] += b.y; v[2] += b.z; v[3] += b.w;
        }
        const int f = s_pair[pos];
        uint32_t o[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = f32_to_bf16(s_w[f] * (g[q] / (1.f + expf(-g[q]))) * v[q]);
        *reinterpret_cast<uint2*>(p.h + (int64_t)f * p.I + n) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
    }
    __syncthreads();
}

template <bool W8>
__global__ __launch_bounds__(kMdThreads) void k_moe_gate_up(MoeDecodeParams p, int shrinks) {
    __shared__ float4 red[kMdWaves * 2 * 4 * kWave];
    __shared__ MdRoute rt;
    __shared__ float s_w[kMdMaxPairs];
    __shared__ int16_t s_tok[LORA_DECODE_MAX_M], s_pair[LORA_DECODE_MAX_M], s_ad[LORA_DECODE_MAX_M];
    const int tid = threadIdx.x;
    const uint32_t tag = launch_tag(), want = tag ^ p.wc.poll_xor;
    const int P = p.M * p.topk;
    bool lost = false;
    int blk = (int)blockIdx.x;
    if (blk < p.M) {
        md_router(p, tag, blk, s_w);
        return;
    }
    blk -= p.M;
    if (blk < shrinks) {
        const int m = blk / p.topk, l = md_adapter(p, m);
        if (l < 0) return;
        const int e = (int)slot_wait(p.route + blk, want, p.wc.max_spin, &lost);
        if (lost) {
            if (tid == 0) atomicOr(p.err, LORA_DEVERR_WAIT);
            return;
        }
        const int64_t slot = p.shared_outer ? l : (int64_t)l * p.E + e;
        md_shrink(p.A_gu + slot * p.r * p.H, p.x + (int64_t)m * p.ldx, p.H, p.r, p.S_gu + (int64_t)blk * p.r, tag);
        return;
    }
    blk -= shrinks;
    for (int f = tid; f < P; f += kMdThreads) {
        bool gone = false;
        const int e = (int)slot_wait(p.route + f, want, p.wc.max_spin, &gone);
        s_w[f] = __uint_as_float(slot_wait(p.route + P + f, want, p.wc.max_spin, &gone));
        rt.exp_[f] = (int16_t)(gone ? -1 : e);
        lost |= gone;
    }
    md_tables(p, rt);
    const int tiles = (p.I + 15) / 16;
    const int units = rt.n_active * tiles;
    const int G = (int)gridDim.x - p.M - shrinks;
    for (int u = blk; u < units; u += G) {
        const int e = rt.active[u / tiles];
        const unsigned long long mask = rt.mask[e];
        if (tid < kWave && ((mask >> tid) & 1ull)) {
            const int at = __popcll(mask & ((1ull << tid) - 1ull));
            int f = tid * p.topk;
            while (rt.exp_[f] != e) ++f;
            s_tok[at] = (int16_t)tid;
            s_pair[at] = (int16_t)f;
            s_ad[at] = (int16_t)md_adapter(p, tid);
        }
        __syncthreads();
        const MdUnit un{e, (u % tiles) * 16, (int)__popcll(mask)};
        switch ((un.ne + 15) / 16) {
            case 1: md_gate_up<W8, 1>(p, un, s_tok, s_pair, s_ad, s_w, red, want, &lost); break;
            case 2: md_gate_up<W8, 2>(p, un, s_tok, s_pair, s_ad, s_w, red, want, &lost); break;
            case 3: md_gate_up<W8, 3>(p, un, s_tok, s_pair, s_ad, s_w, red, want, &lost); break;
            default: md_gate_up<W8, 4>(p, un, s_tok, s_pair, s_ad, s_w, red, want, &lost); break;
        }
    }
    if (lost) atomicOr(p.err, LORA_DEVERR_WAIT);
}

// ---------------------------------------------------------------- second launch
template <bool W8, int TB>
__global__ __launch_bounds__(kMdThreads) void k_moe_down(MoeDecodeParams p, int shrinks) {
    constexpr int kBytes = W8 ? 1 : 2;
    __shared__ float4 red[kMdWaves * TB * kWave];
    __shared__ MdRoute rt;
    __shared__ int16_t fmap[kMdMaxE][TB * 16];      // pair of (active expert, token), -1: none
    const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
    const int lr = lane % 16, lq = lane / 16;
    const uint32_t tag = launch_tag(), want = tag ^ p.wc.poll_xor;
    const int P = p.M * p.topk;
    bool lost = false;
    int blk = (int)blockIdx.x;
    if (blk < shrinks) {
        const int m = blk / p.topk, l = md_adapter(p, m);
        if (l < 0) return;
        const int e = p.route_ids[blk];
        md_shrink(p.A_d + ((int64_t)l * p.E + e) * p.r * p.I, p.h + (int64_t)blk * p.I, p.I, p.r,
                  p.S_d + (int64_t)blk * p.r, tag);
        return;
    }
    blk -= shrinks;
    const int tiles = (p.H + 15) / 16;
    const int split = blk / tiles, n0 = (blk % tiles) * 16;
    for (int f = tid; f < P; f += kMdThreads) rt.exp_[f] = (int16_t)p.route_ids[f];
    md_tables(p, rt);
    const int na = rt.n_active;
    for (int i = tid; i < na * TB * 16; i += kMdThreads) {
        const int e = rt.active[i / (TB * 16)], m = i % (TB * 16);
        int f = -1;
        if ((rt.mask[e] >> m) & 1ull) {
            f = m * p.topk;
            while (rt.exp_[f] != e) ++f;
        }
        fmap[i / (TB * 16)][m] = (int16_t)f;
    }
    __syncthreads();

    const int nr = min(n0 + lr, p.H - 1);
    const char* W = static_cast<const char*>(p.W_d);
    f32x4_t acc[1][TB], part[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[0][t] = f32x4_t{0.f, 0.f, 0.f, 0.f}, part[t] = acc[0][t];
    const int KB = (p.I + 63) / 64;                 // 64-value blocks of one expert
    const int total = na * KB;
    const int t0 = (int)((int64_t)total * split / p.splits), t1 = (int)((int64_t)total * (split + 1) / p.splits);
    constexpr int U = TB == 1 ? 4 : TB == 2 ? 3 : 2;
    int cur = -1;
    auto fold = [&](int ea) {                       // the scale of the expert just left
        const float* s = p.s_d + (int64_t)rt.active[ea] * p.H;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const float v = s[min(n0 + lq * 4 + q, p.H - 1)];
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[0][t][q] += part[t][q] * v, part[t][q] = 0.f;
        }
    };
    for (int b0 = t0 + wave; b0 < t1; b0 += U * kMdWaves) {
        MdRow<W8> w[U];
        uint4 hv[U][TB][2];
        int ea[U];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int b = b0 + q * kMdWaves;
            const bool in = b < t1;
            ea[q] = min(b, total - 1) / KB;
            const int k = (min(b, total - 1) - ea[q] * KB) * 64 + lq * 16;
            const char* row = W + ((int64_t)rt.active[ea[q]] * p.H + nr) * p.I * kBytes;
            const int kc = min(k, p.I - (W8 ? 16 : 8)), kd = min(k + 8, p.I - 8);
            if constexpr (W8) {
                w[q].load(row, kc);
            } else {
                w[q].q[0] = ld16(reinterpret_cast<const uint16_t*>(row) + kc);
                w[q].q[1] = ld16(reinterpret_cast<const uint16_t*>(row) + kd);
            }
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                const int f = fmap[ea[q]][t * 16 + lr];
                const uint16_t* hr = p.h + (int64_t)max(f, 0) * p.I;
                hv[q][t][0] = ld16_if(hr + min(k, p.I - 8), in && f >= 0 && k < p.I, p.h);
                hv[q][t][1] = ld16_if(hr + kd, in && f >= 0 && k + 8 < p.I, p.h);
            }
        }
#pragma unroll
        for (int q = 0; q < U; ++q) {
            if (W8 && ea[q] != cur) {
                if (cur >= 0) fold(cur);
                cur = ea[q];
            }
            uint4 a, b;
            w[q].operands(a, b);
#pragma unroll
            for (int t = 0; t < TB; ++t) {
                f32x4_t& c = W8 ? part[t] : acc[0][t];
                c = mfma_bf16(a, hv[q][t][0], c);
                c = mfma_bf16(b, hv[q][t][1], c);
            }
        }
    }
    if (W8 && cur >= 0) fold(cur);
    if (p.L > 0) {
        const int ad0 = lane < p.M ? md_adapter(p, lane) : -1;
        int deal = 0;
        for (int i = split; i < na; i += p.splits) {
            const int e = rt.active[i];
            const int f = lane < TB * 16 ? fmap[i][lane] : -1;
            const int64_t row[1] = {p.shared_outer ? (int64_t)nr : (int64_t)e * p.H + nr};
            md_delta<1, TB>(p, p.B_d, (int64_t)(p.shared_outer ? 1 : p.E) * p.H * p.r, row, p.S_d,
                            f >= 0 ? ad0 : -1, f, wave, deal, want, &lost, acc);
        }
    }
#pragma unroll
    for (int t = 0; t < TB; ++t)
        red[(wave * TB + t) * kWave + lane] = make_float4(acc[0][t][0], acc[0][t][1], acc[0][t][2], acc[0][t][3]);
    __syncthreads();
    const int m = wave * 16 + lr, n = n0 + lq * 4;
    if (wave < TB && m < p.M && n < p.H) {
        float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int w = 0; w < kMdWaves; ++w) {
            const float4 a = red[(w * TB + wave) * kWave + lane];
            v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
        }
        if (split < p.splits - 1) {
            slot_t* d = p.join + ((int64_t)split * p.M + m) * p.H + n;
#pragma unroll
            for (int q = 0; q < 4; ++q) slot_put(d + q, v[q], tag);
        } else {
            // the last split of a tile adds the others, in split order
            for (int s = 0; s < p.splits - 1; ++s) {
                const slot_t* d = p.join + ((int64_t)s * p.M + m) * p.H + n;
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += __uint_as_float(slot_wait(d + q, want, p.wc.max_spin, &lost));
            }
            *reinterpret_cast<uint2*>(p.out + (int64_t)m * p.ldo + n) =
                make_uint2(f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16), f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16));
        }
    }
    if (lost) atomicOr(p.err, LORA_DEVERR_WAIT);
}

int moe_decode_splits(int H, int I) {
    const int tiles = (H + 15) / 16, blocks = (I + 63) / 64;
    const int want = (512 + tiles - 1) / tiles;
    return max(1, min(min(want, 16), blocks / kMdWaves));
}

template <bool W8>
hipError_t launch_moe_decode_t(const MoeDecodeParams& p, hipStream_t st) {
    const int P = p.M * p.topk;
    const int shrinks = p.L > 0 ? P : 0;
    const int units = min(p.E, P) * ((p.I + 15) / 16);
    hipLaunchKernelGGL(k_moe_gate_up<W8>, dim3((unsigned)(p.M + shrinks + min(units, 512))), dim3(kMdThreads), 0, st,
                       p, shrinks);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const unsigned grid = (unsigned)(shrinks + (p.H + 15) / 16 * p.splits);
    if (p.M <= 16) hipLaunchKernelGGL((k_moe_down<W8, 1>), dim3(grid), dim3(kMdThreads), 0, st, p, shrinks);
    else if (p.M <= 32) hipLaunchKernelGGL((k_moe_down<W8, 2>), dim3(grid), dim3(kMdThreads), 0, st, p, shrinks);
    else hipLaunchKernelGGL((k_moe_down<W8, 4>), dim3(grid), dim3(kMdThreads), 0, st, p, shrinks);
    return hipGetLastError();
}

hipError_t launch_moe_decode(const MoeDecodeParams& p, hipStream_t st) {
    return p.s_gu ? launch_moe_decode_t<true>(p, st) : launch_moe_decode_t<false>(p, st);
}

}  // namespace mlora
