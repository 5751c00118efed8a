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
//   producers (first in the grid): unit = (segment, 16 S columns, half of K or
//     all of it) over eight wavefronts, bf16 MFMA 16 x 16 x 32, joined through
//     LDS.  S goes to tagged exchange slots in fp32, one a value and half; the
//     consumers add the halves and split the sum into the bf16 hi / lo pair of
//     their product.
//   consumers: unit = 16 NR output columns of one slice for every token, K over
//     eight wavefronts (v_mfma_f32_16x16x128_f8f6f4, W rows as the first
//     operand so that a lane ends with four consecutive columns of one token).
//     Only after its share of W8 is read and multiplied does a workgroup look
//     at the slots, which are full by then; each wavefront then adds the
//     deltas of every eighth segment to its own partial sums, and the eight
//     partial sums join through LDS in a fixed order.
// Both read rows as whole 128-byte segments and change lanes through LDS
// (row_stage.hpp).  A consumer waits for producers only, which wait for
// nothing and come first in the grid; the waits are bounded and report
// LORA_DEVERR_WAIT.
//
// The matrix unit's sums of e4m3 products: it lines the products of eight
// neighbouring values of K up to the largest exponent among them and drops what
// lies below 2^-13 of it (seen with single products; every e4m3 form does), then
// adds the eights in fp32.  That is some 2^-14 of a sum's magnitudes, far below
// the 2^-4 to which the operands were rounded; widening both to bf16 would avoid
// it at half the matrix rate.  Everything else is fp32; S enters its product as
// the sum of two bf16 values (an error of 2^-17 of S at most); y is rounded once.
//
// Measured: one token to 4096 + 1024 + 1024 columns, K = 4096, 9.9 us; 32 tokens of
// 32 mixed adapters to 4096 columns 12.8, without adapters 8.3.  W8's 25 and 17 MB
// would take 4.9 and 3.3 at the rate of a large copy: what is left is the launch,
// the first loads' round trips (index, rows, S, join) and the producers' chain.
#pragma once

#include "common.hpp"
#include "kernels.hpp"
#include "row_stage.hpp"

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
    slot_t* slots;               // [chunks][64][cols]: half of K, sorted position, S column
    const float* S;              // without slots: fp32 [M][cols], sorted rows
    int chunks, chunk_kb;        // halves of K (one for short K), their blocks of 64 values
    int jb;                      // 16-column blocks of an S row
    int n_prod;                  // producer workgroups
    int tile_start[LORA_MAX_SLICES + 1];
    WaitCtl wc;
};

// uint4 of a wavefront's stage: 16 NR rows of W (or A) and 16 token rows,
// later its partial sums
constexpr int fp8_stage(int TB, int NR) {
    return (NR + 1) * 128 > NR * TB * kWave ? (NR + 1) * 128 : NR * TB * kWave;
}

// S of one segment's tokens for 16 S columns and half of K.  What names the
// unit's rows (segment, tokens and, for tables of up to 64 slots, every slot's
// rank and offset) is loaded in one round; then come four blocks of A a
// wavefront at once, the whole half of K = 4096.
template <int TB>
__device__ __forceinline__ void fp8_producer(const Fp8Params& p, uint32_t tag, uint4* smem, int words) {
    const LinearArgs& a = p.a;
    const int c = (int)blockIdx.x % p.chunks, u = (int)blockIdx.x / p.chunks;
    const int s = u / p.jb, jb = u % p.jb;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int lr = lane % 16, lq = lane / 16;
    const int slot = min(lane, a.L - 1);
    const int rank_l = a.rank[slot];
    const int64_t off_l = a.a_off[slot];
    const int tok_l = a.sorted_idx[min(lane, a.M - 1)];
    const int nseg = a.num_segments[0];
    const int id = __builtin_amdgcn_readfirstlane(a.req_to_lora[s]);
    const int p0 = __builtin_amdgcn_readfirstlane(a.seg_indptr[s]);
    const int p1 = __builtin_amdgcn_readfirstlane(a.seg_indptr[s + 1]);
    if (s >= nseg) return;
    if (id < 0 || id >= a.L) {
        table_fault(a.err, true);
        return;
    }
    const int rp = a.L <= kWave ? __builtin_amdgcn_readlane(rank_l, id) : __builtin_amdgcn_readfirstlane(a.rank[id]);
    const int64_t off = a.L <= kWave ? readlane64(off_l, id) : a.a_off[id];
    const int per = a.r_max / 16;
    const int sl = jb / per, j0 = (jb % per) * 16;
    if (j0 >= rp) return;
    if (table_fault(a.err, p0 < 0 || p1 > a.M || p1 < p0)) return;

    const uint16_t* A = static_cast<const uint16_t*>(a.A) + off + (int64_t)(sl * rp + j0) * a.K;
    const __amdgpu_buffer_rsrc_t ra = uniform_rsrc(A, (uint32_t)(16 * a.K * 2));
    const __amdgpu_buffer_rsrc_t rx = uniform_rsrc(p.x, (uint32_t)(((int64_t)(a.M - 1) * p.ldx + a.K) * 2));
    uint32_t off_a[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) off_a[i] = (uint32_t)((8 * i + lane / 8) * a.K * 2 + (lane % 8) * 16);
    uint4* st = smem + wave * words;
    uint4* sx = st + 16 * 8;
    const StageAt at;
    constexpr int U = 4;
    const int ms = min(p1 - p0, TB * 16);
    const int KB = min((a.K + 63) / 64, (c + 1) * p.chunk_kb);
    f32x4_t acc[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) acc[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int b0 = c * p.chunk_kb + wave; b0 < KB; b0 += U * kFpWaves) {
        uint4 va[U][2], vx[U][2];
#pragma unroll
        for (int q = 0; q < U; ++q) {
            const int kb = b0 + q * kFpWaves;
            const bool in = kb < KB && kb * 64 + lane % 8 * 8 < a.K;
#pragma unroll
            for (int i = 0; i < 2; ++i) va[q][i] = buf_ld16_at<true>(ra, in ? off_a[i] : kBufOff, (uint32_t)kb * 128u);
        }
#pragma unroll
        for (int t = 0; t < TB; ++t) {               // 16 of the segment's tokens
            if (t * 16 >= ms) break;
            uint32_t off_x[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int k = t * 16 + 8 * i + lane / 8;
                int m = __shfl(tok_l, min(p0 + k, a.M - 1), kWave);
                if (table_fault(a.err, m < 0 || m >= a.M)) m = min(max(m, 0), a.M - 1);
                off_x[i] = k < ms ? (uint32_t)m * (uint32_t)p.ldx * 2u + (lane % 8) * 16 : kBufOff;
            }
#pragma unroll
            for (int q = 0; q < U; ++q) {
                const int kb = b0 + q * kFpWaves;
                const bool in = kb < KB && kb * 64 + lane % 8 * 8 < a.K;
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    vx[q][i] = buf_ld16_at<false>(rx, in ? off_x[i] : kBufOff, (uint32_t)kb * 128u);
            }
#pragma unroll
            for (int q = 0; q < U; ++q) {
#pragma unroll
                for (int i = 0; i < 2; ++i) st[at.piece(i)] = va[q][i], sx[at.piece(i)] = vx[q][i];
                stage_order();
#pragma unroll
                for (int j = 0; j < 2; ++j) acc[t] = mfma_bf16(st[at.half(0, j)], sx[at.half(0, j)], acc[t]);
                stage_order();
            }
        }
    }
    float4* red = reinterpret_cast<float4*>(st);
#pragma unroll
    for (int t = 0; t < TB; ++t) red[t * kWave + lane] = make_float4(acc[t][0], acc[t][1], acc[t][2], acc[t][3]);
    __syncthreads();
    const int pos = wave * 16 + lr;
    if (wave >= TB || pos >= ms) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kFpWaves; ++w) {
        const float4 f = reinterpret_cast<const float4*>(smem + w * words)[wave * kWave + lane];
        v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
    }
    slot_t* d = p.slots + ((int64_t)c * LORA_DECODE_MAX_M + p0 + pos) * a.cols + sl * a.r_max + j0 + lq * 4;
    slot_put(d, v.x, tag);
    slot_put(d + 1, v.y, tag);
    slot_put(d + 2, v.z, tag);
    slot_put(d + 3, v.w, tag);
}

// SLOTS: up to 64 tokens, producers in the same launch.  Otherwise S is read
// from memory (p.S, an earlier launch's), and a consumer takes the columns'
// product for one group of 64 sorted positions; the groups of a column tile
// follow each other on one L2 (every eighth workgroup).  With TB = 4 and NR = 1 the
// 128 registers are full: one value (SLOTS) or six are spilled across the loop over K,
// none within it.
template <int TB, int NR, bool SLOTS>
__global__ __launch_bounds__(kFpThreads, TB * NR == 8 ? 2 : 4) void k_linear_fp8(Fp8Params p) {
    constexpr int kStage = fp8_stage(TB, NR);
    __shared__ uint4 smem[kFpWaves * kStage];
    __shared__ __attribute__((aligned(16))) uint16_t sHi[TB * 16 * kFpSLD], sLo[TB * 16 * kFpSLD];
    __shared__ int s_rp[TB * 16];
    const LinearArgs& a = p.a;
    const uint32_t tag = launch_tag();
    if (SLOTS && (int)blockIdx.x < p.n_prod) {
        fp8_producer<TB>(p, tag, smem, kStage);
        return;
    }
    int ct = (int)blockIdx.x - p.n_prod, base = 0, M = a.M;
    if constexpr (!SLOTS) {
        const int groups = (a.M + 63) / 64, v = (int)blockIdx.x / 8;
        ct = v / groups * 8 + (int)blockIdx.x % 8;
        base = v % groups * 64;
        M = min(64, a.M - base);
        if (ct >= p.tile_start[a.n_sl]) return;
    }
    const int32_t* sorted = a.sorted_idx + base;
    const int tid = threadIdx.x;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane % 16, lq = lane / 16;
    int sl = 0;
    while (sl + 1 < a.n_sl && ct >= p.tile_start[sl + 1]) ++sl;
    const int n0 = (int)(a.slice_off[sl] + (int64_t)(ct - p.tile_start[sl]) * (16 * NR));
    const int n1 = (int)min((int64_t)n0 + 16 * NR, a.slice_off[sl + 1]);

    // small loads ahead of the stream (loads return in order): the tokens of
    // the rows that this lane loads and of its column, the segments (lane s:
    // the group's segment s, at most 64 of them)
    int m_row[2 * TB], tok[TB];
#pragma unroll
    for (int i = 0; i < 2 * TB; ++i) m_row[i] = sorted[min(8 * i + lane / 8, M - 1)];
#pragma unroll
    for (int t = 0; t < TB; ++t) tok[t] = sorted[min(t * 16 + lr, M - 1)];
    int nseg = __builtin_amdgcn_readfirstlane(a.num_segments[0]);
    int seg0 = 0;
    if constexpr (!SLOTS) {
        // the last segment that starts at or before `base`
        const int stride = (a.L + kWave) / kWave;        // ceil((L + 1) / 64)
        const int v1 = a.seg_indptr[min(lane * stride, a.L)];
        seg0 = (63 - __clzll((long long)__ballot(lane * stride <= a.L && v1 <= base))) * stride;
        if (stride > 1) {
            const int v2 = a.seg_indptr[min(seg0 + lane, a.L)];
            seg0 += 63 - __clzll((long long)__ballot(lane < stride && seg0 + lane <= a.L && v2 <= base));
        }
    }
    const int seg = min(seg0 + lane, a.L - 1);
    int q_id = a.req_to_lora[seg];
    int q_p0 = a.seg_indptr[seg], q_p1 = a.seg_indptr[seg + 1];
    nseg = min(nseg - seg0, kWave);

    // ---- base product
    const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(p.W + (int64_t)n0 * p.ldw, (uint32_t)((n1 - n0 - 1) * p.ldw + a.K));
    const __amdgpu_buffer_rsrc_t rx = uniform_rsrc(p.x8, (uint32_t)((int64_t)(a.M - 1) * p.ldx8 + a.K));
    uint32_t off_w[2 * NR], off_x[2 * TB];
#pragma unroll
    for (int i = 0; i < 2 * NR; ++i)
        off_w[i] = (uint32_t)(min(8 * i + lane / 8, n1 - n0 - 1) * p.ldw) + (lane % 8) * 16;
    // blocks of 128 values in flight: W rows come from HBM, token rows from L2
    constexpr int U = TB * NR == 8 ? 4 : 4 / NR, UX = TB * NR == 8 ? 2 : TB == 1 ? U : 4 / TB;
    const int KB = (a.K + 127) / 128;
    uint4 vw[U][2 * NR], vx[UX][2 * TB];
    auto load_w = [&](int q, int kb) {
        const bool in = kb * 128 + lane % 8 * 16 < a.K;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) vw[q][i] = buf_ld16_at<true>(rw, in ? off_w[i] : kBufOff, (uint32_t)kb * 128u);
    };
    auto load_x = [&](int q, int kb) {
        const bool in = kb * 128 + lane % 8 * 16 < a.K;
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i) vx[q][i] = buf_ld16_at<false>(rx, in ? off_x[i] : kBufOff, (uint32_t)kb * 128u);
    };
    load_w(0, wave);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        if (table_fault(a.err, tok[t] < 0 || tok[t] >= a.M) && (tok[t] < 0 || tok[t] >= a.M)) tok[t] = -1;
        if (t * 16 + lr >= M) tok[t] = -1;
    }
#pragma unroll
    for (int i = 0; i < 2 * TB; ++i) {
        const int m = m_row[i];
        const bool ok = 8 * i + lane / 8 < M && (!kTableChecks || (m >= 0 && m < a.M));
        off_x[i] = ok ? (uint32_t)m * (uint32_t)p.ldx8 + (lane % 8) * 16 : kBufOff;
    }
#pragma unroll
    for (int q = 0; q < UX; ++q) load_x(q, wave + q * kFpWaves);
    // the rest of W only now, a round trip later: with all of it queued at once
    // the producers' rows of A come behind 16 MB of W
#pragma unroll
    for (int q = 1; q < U; ++q) load_w(q, wave + q * kFpWaves);
    // what the first loads name
    const bool seg_ok = lane < nseg && q_id >= 0 && q_id < a.L;
    const bool range_ok = q_p0 >= 0 && q_p1 >= q_p0 && q_p1 <= a.M;
    table_fault(a.err, lane < nseg && !(seg_ok && range_ok));
    q_p0 = max(q_p0 - base, 0);
    q_p1 = min(q_p1 - base, M);
    q_id = seg_ok ? q_id : 0;
    const int rank_l = a.rank[q_id];
    const int64_t q_bo = a.b_off[q_id];
    float xs[TB], ws[NR][4];
#pragma unroll
    for (int t = 0; t < TB; ++t) xs[t] = p.x_scale[max(tok[t], 0)];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int q = 0; q < 4; ++q) ws[r][q] = p.w_scale[min(n0 + r * 16 + lq * 4 + q, n1 - 1)];
    if (tid < TB * 16) s_rp[tid] = 0;

    uint4* st = smem + wave * kStage;
    uint4* sx = st + NR * 16 * 8;
    const StageAt at;
    f32x4_t acc[NR][TB];
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) acc[r][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int b0 = wave; b0 < KB; b0 += U * kFpWaves) {
#pragma unroll
        for (int q = 0; q < U; ++q) {
            // blocks past K read zeros (no memory is touched), and add none
#pragma unroll
            for (int i = 0; i < 2 * NR; ++i) st[at.piece(i)] = vw[q][i];
            uint4 w[NR][2];
#pragma unroll
            for (int t = 0; t < TB; ++t) {
#pragma unroll
                for (int i = 0; i < 2; ++i) sx[at.piece(i)] = vx[q % UX][2 * t + i];
                stage_order();
                if (t == 0)
#pragma unroll
                    for (int r = 0; r < NR; ++r) w[r][0] = st[at.half(r, 0)], w[r][1] = st[at.half(r, 1)];
                const uint4 x0 = sx[at.half(0, 0)], x1 = sx[at.half(0, 1)];
#pragma unroll
                for (int r = 0; r < NR; ++r) acc[r][t] = mfma_e4m3(w[r][0], w[r][1], x0, x1, acc[r][t]);
                stage_order();
            }
            load_w(q, b0 + (q + U) * kFpWaves);
            load_x(q % UX, b0 + (q + UX) * kFpWaves);
        }
    }
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t)
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[r][t][q] *= xs[t] * ws[r][q];

    // ---- deltas
    const int q_rp = seg_ok && q_p0 < q_p1 && (!kTableChecks || range_ok) ? rank_l : 0;
    if (__ballot(q_rp > 0) != 0ull) {
        // B rows of the wavefront's first segments, in flight while S is read
        constexpr int PB = TB * NR >= 4 ? 2 : 3;
        uint4 pb[PB][NR][2];
        auto load_b = [&](uint4 (&b)[NR][2], int s, int rp) {
            const uint16_t* B = static_cast<const uint16_t*>(a.B) + readlane64(q_bo, s);
#pragma unroll
            for (int r = 0; r < NR; ++r)
#pragma unroll
                for (int j = 0; j < 2; ++j)
                    b[r][j] = ld16(B + (int64_t)min(n0 + r * 16 + lr, n1 - 1) * rp + min(j * 32 + lq * 8, rp - 8));
        };
#pragma unroll
        for (int i = 0; i < PB; ++i) {
            const int s = wave + i * kFpWaves, rp = __builtin_amdgcn_readlane(q_rp, s);
            if (rp > 0) load_b(pb[i], s, rp);
        }
        __syncthreads();
        if (wave == 0 && q_rp > 0)
            for (int i = q_p0; i < q_p1; ++i) s_rp[i] = q_rp;
        __syncthreads();
        // S: the slots of every position's own rank, four a thread in flight
        // together; positions and columns without one become zeros
        const uint32_t want = tag ^ p.wc.poll_xor;
        const int total = TB * 16 * a.r_max;             // a multiple of 4
        bool lost = false;
        for (int e = tid * 4; e < total; e += kFpThreads * 4) {
            const int pos = e / a.r_max, j = e % a.r_max;
            const bool on = j < s_rp[pos];               // ranks are multiples of 16
            float f[4] = {0.f, 0.f, 0.f, 0.f};
            if constexpr (SLOTS) {
                const slot_t* src = p.slots + (int64_t)(on ? pos : 0) * a.cols + sl * a.r_max + (on ? j : 0);
                const int64_t second = p.chunks > 1 ? (int64_t)LORA_DECODE_MAX_M * a.cols : 0;
                int spin = 0;
                // one slot is polled until it is full, then all are read: polls of
                // all of them by every consumer slowed the producers down
                while (on && spin < p.wc.max_spin && !slot_full(slot_load(src), want)) {
                    __builtin_amdgcn_s_sleep(2);
                    ++spin;
                }
                for (; on; ++spin) {
                    slot_t v[8];
                    bool full = true;
#pragma unroll
                    for (int q = 0; q < 4; ++q) v[q] = slot_load(src + q), v[4 + q] = slot_load(src + second + q);
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        full &= slot_full(v[q], want) && slot_full(v[4 + q], want);
                        f[q] = __uint_as_float((uint32_t)v[q]);
                        if (second) f[q] += __uint_as_float((uint32_t)v[4 + q]);
                    }
                    if (full) break;
                    if (spin >= p.wc.max_spin) {
                        lost = true;
                        break;
                    }
                    __builtin_amdgcn_s_sleep(1);
                }
            } else if (on) {
                const float4 v = *reinterpret_cast<const float4*>(p.S + (int64_t)(base + pos) * a.cols + sl * a.r_max + j);
                f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
            }
            const uint32_t w[4] = {hi_lo(f[0]), hi_lo(f[1]), hi_lo(f[2]), hi_lo(f[3])};
            *reinterpret_cast<uint2*>(sHi + pos * kFpSLD + j) =
                make_uint2((w[0] >> 16) | (w[1] & 0xffff0000u), (w[2] >> 16) | (w[3] & 0xffff0000u));
            *reinterpret_cast<uint2*>(sLo + pos * kFpSLD + j) =
                make_uint2((w[0] & 0xffffu) | (w[1] << 16), (w[2] & 0xffffu) | (w[3] << 16));
        }
        if (lost) atomicOr(a.err, LORA_DEVERR_WAIT);
        __syncthreads();
        auto add = [&](int s, const uint4 (&pbs)[NR][2]) {
            const int rp = __builtin_amdgcn_readlane(q_rp, s);
            const int p0 = __builtin_amdgcn_readlane(q_p0, s), p1 = __builtin_amdgcn_readlane(q_p1, s);
#pragma unroll
            for (int j = 0; j < LORA_MAX_RANK / 32; ++j) {
                const int jj = j * 32 + lq * 8;
                if (j * 32 >= rp) continue;
                uint4 b[NR];
#pragma unroll
                for (int r = 0; r < NR; ++r) b[r] = and4(pbs[r][j], opaque_mask(jj < rp));
#pragma unroll
                for (int t = 0; t < TB; ++t) {
                    if (t * 16 >= p1 || t * 16 + 16 <= p0) continue;
                    const int pos = t * 16 + lr;
                    const bool mine = pos >= p0 && pos < p1;
                    const uint32_t mp = opaque_mask(mine && jj < rp);
                    const uint4 h = and4(*reinterpret_cast<const uint4*>(sHi + pos * kFpSLD + jj), mp);
                    const uint4 l = and4(*reinterpret_cast<const uint4*>(sLo + pos * kFpSLD + jj), mp);
#pragma unroll
                    for (int r = 0; r < NR; ++r) {
                        // other tokens keep their sums: their zeros times an
                        // adapter's infinities would not be zero
                        const f32x4_t v = mfma_bf16(b[r], l, mfma_bf16(b[r], h, acc[r][t]));
#pragma unroll
                        for (int q = 0; q < 4; ++q) acc[r][t][q] = mine ? v[q] : acc[r][t][q];
                    }
                }
            }
        };
#pragma unroll
        for (int i = 0; i < PB; ++i)
            if (__builtin_amdgcn_readlane(q_rp, wave + i * kFpWaves) > 0) add(wave + i * kFpWaves, pb[i]);
        for (int s = wave + PB * kFpWaves; s < nseg; s += kFpWaves) {
            const int rp = __builtin_amdgcn_readlane(q_rp, s);
            if (rp == 0) continue;
            load_b(pb[0], s, rp);
            add(s, pb[0]);
        }
    }

    // ---- join the eight partial sums; four columns of one token per lane
    float4* red = reinterpret_cast<float4*>(st);
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t)
            red[(r * TB + t) * kWave + lane] =
                make_float4(acc[r][t][0], acc[r][t][1], acc[r][t][2], acc[r][t][3]);
    __syncthreads();
    if (wave >= NR * TB) return;
    float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int w = 0; w < kFpWaves; ++w) {
        const float4 f = reinterpret_cast<const float4*>(smem + w * kStage)[wave * kWave + lane];
        v[0] += f.x; v[1] += f.y; v[2] += f.z; v[3] += f.w;
    }
    int m = tok[0];
#pragma unroll
    for (int t = 1; t < TB; ++t) m = wave % TB == t ? tok[t] : m;
    const int n = n0 + wave / TB * 16 + lq * 4;          // slices are multiples of 8 wide
    if (m >= 0 && n < n1)
        *reinterpret_cast<uint2*>(p.y + (int64_t)m * p.ldy + n) =
            make_uint2(f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16), f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16));
}

// ---------------------------------------------------------------- shrink for the larger product
// S (fp32 [M][cols], sorted rows) of up to 16 rows of one tile of the schedule
// for 16 S columns: the producers' product over all of K, four blocks of both
// operands in flight a wavefront, with plain stores (the product that reads S
// is the next launch).  One launch instead of lora_shrink's two, and no partial
// sums in memory; every 16 columns of rank read the rows of x again (from L2).
__global__ __launch_bounds__(kFpThreads, 4) void k_shrink_rows(LinearArgs a, const uint16_t* x, int64_t ldx,
                                                               float* S) {
    __shared__ uint4 smem[kFpWaves * 32 * 8];
    const int jbs = a.cols / 16;
    int u = (int)blockIdx.x;
    const int jb = u % jbs;
    u /= jbs;
    const int t0 = u % 4 * 16, tile = u / 4;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int lr = lane % 16, lq = lane / 16;
    // one round of loads: the tile, its rows, every slot's rank and offset
    const int slot = min(lane, a.L - 1);
    const int rank_l = a.rank[slot];
    const int64_t off_l = a.a_off[slot];
    int m_row[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) m_row[i] = a.tile_rows[(int64_t)tile * LORA_TILE_ROWS + t0 + 8 * i + lane / 8];
    const int id = __builtin_amdgcn_readfirstlane(a.tile_info[tile * 4 + 1]);
    const int p0 = __builtin_amdgcn_readfirstlane(a.tile_info[tile * 4 + 2]) + t0;
    const int ms = min(__builtin_amdgcn_readfirstlane(a.tile_info[tile * 4 + 3]) - t0, 16);
    if (tile >= a.num_tiles[0] || ms <= 0) return;
    if (id < 0 || id >= a.L) {
        table_fault(a.err, true);
        return;
    }
    const int rp = a.L <= kWave ? __builtin_amdgcn_readlane(rank_l, id) : __builtin_amdgcn_readfirstlane(a.rank[id]);
    const int64_t off = a.L <= kWave ? readlane64(off_l, id) : a.a_off[id];
    const int per = a.r_max / 16;
    const int sl = jb / per, j0 = (jb % per) * 16;
    if (j0 >= rp) return;
    if (table_fault(a.err, p0 < 0 || p0 + ms > a.M)) return;

    const uint16_t* A = static_cast<const uint16_t*>(a.A) + off + (int64_t)(sl * rp + j0) * a.K;
    const __amdgpu_buffer_rsrc_t ra = uniform_rsrc(A, (uint32_t)(16 * a.K * 2));
    uint32_t off_a[2];
    const uint16_t* xr[2];
    const int first = __builtin_amdgcn_readfirstlane(m_row[0]);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        off_a[i] = (uint32_t)((8 * i + lane / 8) * a.K * 2 + (lane % 8) * 16);
        // rows past the tile's repeat its first one and are not stored
        int m = 8 * i + lane / 8 < ms ? m_row[i] : first;
        if (table_fault(a.err, m < 0 || m >= a.M)) m = min(max(m, 0), a.M - 1);
        xr[i] = x + (int64_t)m * ldx + (lane % 8) * 8;
    }
    uint4* st = smem + wave * 32 * 8;
    uint4* sx = st + 16 * 8;
    const StageAt at;
    constexpr int U = 4;
    const int KB = (a.K + 63) / 64;
    uint4 va[U][2], vx[U][2];
    auto load = [&](int q, int kb) {
        // A past K reads zeros; the x values they meet are some of the row's own
        const bool in = kb * 64 + lane % 8 * 8 < a.K;
        const int k = min(kb * 64, a.K - 8 - lane % 8 * 8);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            va[q][i] = buf_ld16_at<false>(ra, in ? off_a[i] : kBufOff, (uint32_t)kb * 128u);
            vx[q][i] = ld16(xr[i] + k);
        }
    };
#pragma unroll
    for (int q = 0; q < U; ++q) load(q, wave + q * kFpWaves);
    f32x4_t acc = f32x4_t{0.f, 0.f, 0.f, 0.f};
    for (int b0 = wave; b0 < KB; b0 += U * kFpWaves)
#pragma unroll
        for (int q = 0; q < U; ++q) {
#pragma unroll
            for (int i = 0; i < 2; ++i) st[at.piece(i)] = va[q][i], sx[at.piece(i)] = vx[q][i];
            stage_order();
            load(q, b0 + (q + U) * kFpWaves);
#pragma unroll
            for (int j = 0; j < 2; ++j) acc = mfma_bf16(st[at.half(0, j)], sx[at.half(0, j)], acc);
            stage_order();
        }
    float4* red = reinterpret_cast<float4*>(st);
    red[lane] = make_float4(acc[0], acc[1], acc[2], acc[3]);
    __syncthreads();
    if (wave != 0 || lr >= ms) return;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kFpWaves; ++w) {
        const float4 f = reinterpret_cast<const float4*>(smem + w * 32 * 8)[lane];
        v.x += f.x; v.y += f.y; v.z += f.z; v.w += f.w;
    }
    *reinterpret_cast<float4*>(S + (int64_t)(p0 + lr) * a.cols + sl * a.r_max + j0 + lq * 4) = v;
}

hipError_t launch_shrink_rows(const LinearArgs& a, const void* x, int64_t ldx, float* S, hipStream_t st) {
    const int tiles = a.M / LORA_TILE_ROWS + a.s_max;
    hipLaunchKernelGGL(k_shrink_rows, dim3((unsigned)(tiles * 4 * (a.cols / 16))), dim3(kFpThreads), 0, st, a,
                       static_cast<const uint16_t*>(x), ldx, S);
    return hipGetLastError();
}

template <int TB, int NR, bool SLOTS = true>
hipError_t launch_linear_fp8_as(Fp8Params& p, hipStream_t st) {
    int t = 0;
    for (int s = 0; s < p.a.n_sl; ++s) {
        p.tile_start[s] = t;
        t += (int)((p.a.slice_off[s + 1] - p.a.slice_off[s] + 16 * NR - 1) / (16 * NR));
    }
    p.tile_start[p.a.n_sl] = t;
    unsigned grid;
    if (SLOTS) {
        p.jb = p.a.cols / 16;
        // K in halves shortens the chain that the consumers wait for, as long
        // as both halves' workgroups fit the chip in one round (in one and in
        // two, 32 adapters: 4096 x 4096 with 32 tokens 14.3 / 12.9 us, 64 tokens
        // 18.1 / 16.9; three slices, 768 halves, 64 tokens 26.6 / 28.5)
        p.chunks = p.a.K > 1024 && 2 * p.a.s_max * p.jb <= 256 ? 2 : 1;
        p.chunk_kb = ((p.a.K + 63) / 64 + p.chunks - 1) / p.chunks;
        p.n_prod = p.a.s_max * p.jb * p.chunks;
        grid = (unsigned)(p.n_prod + t);
    } else {
        grid = (unsigned)((p.a.M + 63) / 64 * ((t + 7) / 8 * 8));
    }
    hipLaunchKernelGGL((k_linear_fp8<TB, NR, SLOTS>), dim3(grid), dim3(kFpThreads), 0, st, p);
    return hipGetLastError();
}

static Fp8Params fp8_params(const LinearArgs& a, const void* W8, int64_t ldw, const float* w_scale, const void* x8,
                            int64_t ldx8, const float* x_scale, const void* x, int64_t ldx, void* y, int64_t ldy) {
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
    return p;
}

hipError_t launch_linear_fp8(const LinearArgs& a, const void* W8, int64_t ldw, const float* w_scale,
                             const void* x8, int64_t ldx8, const float* x_scale, const void* x,
                             int64_t ldx, void* y, int64_t ldy, void* ws, hipStream_t st) {
    Fp8Params p = fp8_params(a, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, y, ldy);
    p.slots = reinterpret_cast<slot_t*>(static_cast<char*>(ws) + linear_ws_layout(0, a.K, a.cols).slots);
    p.wc = wait_ctl();
    // A unit reads every token row once: twice the columns halve that and the
    // units, which pays from the width where units of 32 keep enough compute units
    // busy: for up to 16 tokens the later the longer K.  Measured, 16 against 32
    // columns, one slice with 32 adapters, 1 / 16 tokens: K = 512, N = 2048 6.1 / 6.2 and
    // 7.2 / 7.2 us, 4096 7.2 / 6.4 and 8.3 / 7.5; K = 2048, N = 4096 8.2 / 7.0 and 9.5 / 8.5,
    // 14336 17.3 / 10.9 and 21.1 / 15.0; K = 4096, N = 4096 8.9 / 9.5 and 10.8 / 11.5, 6144
    // 10.9 / 9.7 and 13.2 / 12.8, 28672 34.8 / 28.7 and 42.7 / 34.5; K = 8192, N = 6144 14.7 /
    // 14.8 and 18.1 / 19.5, 8192 18.2 / 19.5 and 21.8 / 22.8, 14336 26.6 / 27.0 and 33.9 / 33.2.
    // For more tokens the deltas count: 32 and 64 tokens, N = 6144, K = 4096, one slice 18.9
    // / 16.7 and 24.0 / 23.0, three slices 21.4 / 25.4 and 26.9 / 29.4, without adapters 12.2 /
    // 10.2 and 16.2 / 14.0; N = 8192 20.0 / 17.6 and 25.7 / 24.1, 25.6 / 26.6 and 31.3 / 39.0,
    // 12.9 / 11.2 and 16.9 / 15.2 (K = 512 to 8192 alike); one slice, N = 4096 13.5 / 16.0 and
    // 17.0 / 22.3, 28672 52.3 / 45.2 and 70.6 / 73.5.
    const int64_t units = a.slice_off[a.n_sl] / 32;
    const int64_t few = a.K <= 2048 ? 128 : a.K < 8192 ? 192 : 448;
    const bool wide = units >= (a.M <= 16 ? few : 256);
    if (a.M <= 16) return wide ? launch_linear_fp8_as<1, 2>(p, st) : launch_linear_fp8_as<1, 1>(p, st);
    if (a.M <= 32) return wide ? launch_linear_fp8_as<2, 2>(p, st) : launch_linear_fp8_as<2, 1>(p, st);
    return wide ? launch_linear_fp8_as<4, 2>(p, st) : launch_linear_fp8_as<4, 1>(p, st);
}

hipError_t launch_linear_fp8_groups(const LinearArgs& a, const void* W8, int64_t ldw, const float* w_scale,
                                    const void* x8, int64_t ldx8, const float* x_scale, const float* S,
                                    void* y, int64_t ldy, hipStream_t st) {
    Fp8Params p = fp8_params(a, W8, ldw, w_scale, x8, ldx8, x_scale, nullptr, 0, y, ldy);
    p.S = S;
    // 32 columns a unit halve the reads of x; 16 where that leaves most of the
    // compute units without one (16 against 32 columns, K = 4096: 65 tokens to 2048
    // columns 18.6 / 20.3 us, to 4096 25.4 / 21.8; 512 tokens to 512 20.4 / 22.5, to
    // 1024 27.4 / 22.7)
    const int64_t units = (a.M + 63) / 64 * (a.slice_off[a.n_sl] / 32);
    return units >= 192 ? launch_linear_fp8_as<4, 2, false>(p, st) : launch_linear_fp8_as<4, 1, false>(p, st);
}

}  // namespace mlora
