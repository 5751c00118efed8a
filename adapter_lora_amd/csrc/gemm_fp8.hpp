// The shared projection in 8 bits beside the adapters for more tokens than one
// decode launch takes (see linear_fp8.hpp for the formula): lora_shrink writes
// S, then one product on e4m3 operands whose epilogue scales the sums by xs
// ws, adds S B_i^T and rounds y once.
//
// The unit, the LDS ring, the swizzle and the epilogue are those of the bf16
// product (gemm.hip): 128 sorted positions x 256 output columns, four waves,
// stages of 128 bytes per row.  A stage holds 128 values of K instead of 64
// and takes 16 v_mfma_f32_32x32x64_f8f6f4 of 64 cycles instead of 32 of 32, so
// the same bytes through LDS carry twice the operations.
#pragma once

#include "common.hpp"
#include "kernels.hpp"
#include "linear_fp8.hpp"

namespace mlora {

constexpr int kG8K = 128;                // K per stage

// 32 x 32 x 64 on e4m3 operands, without block scales: lane l supplies row /
// column l % 32 and 32 values of K (any 32, the same for both operands).
__device__ __forceinline__ f32x16_t mfma32_e4m3(const uint4& a0, const uint4& a1, const uint4& b0,
                                                const uint4& b1, f32x16_t c) {
    const i32x8_t a = {(int)a0.x, (int)a0.y, (int)a0.z, (int)a0.w, (int)a1.x, (int)a1.y, (int)a1.z, (int)a1.w};
    const i32x8_t b = {(int)b0.x, (int)b0.y, (int)b0.z, (int)b0.w, (int)b1.x, (int)b1.y, (int)b1.z, (int)b1.w};
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, c, 0, 0, 0, 0, 0, 0);
}

struct GemmFp8Params {
    LinearArgs a;
    const uint8_t* x;
    int64_t ldx;
    const float* x_scale;
    const uint8_t* W;
    int64_t ldw;
    const float* w_scale;
    uint16_t* y;
    int64_t ldy;
    const float* S;              // fp32 [M][cols], sorted rows
    int col_tiles;               // 256-column tiles over all slices
    int tile_start[LORA_MAX_SLICES + 1];
    int nk2;                     // stages, rounded up to even
    int seg_stride;              // ceil((L + 1) / 64): first-round search stride
};

__global__ __launch_bounds__(kGThreads, 1) void k_gemm_fp8(GemmFp8Params p) {
    __shared__ uint4 smem[kGRing * kGStage];
    __shared__ int s_tok[kGM];
    __shared__ float s_xs[kGM];
    const LinearArgs& a = p.a;
    const int u = (int)blockIdx.x;
    const int rt = u / p.col_tiles;
    const int ct = u % p.col_tiles;
    const int tid = threadIdx.x;
    const int lane = lane_id();
    const int wave = tid / kWave;
    const int lr = lane % 32, lh = lane / 32;
    const int p0 = rt * kGM;
    const int rows = min(kGM, a.M - p0);
    const int K = a.K;      // one byte per value: a stage is 128 of them

    // first round of the segment search, needed only by the epilogue:
    // lane j holds seg_indptr[j * stride] (entries past the segments hold
    // the number of tokens with an adapter)
    const int L = a.L;
    const int srch1 = a.seg_indptr[min(lane * p.seg_stride, L)];
    const int m_valid = a.seg_indptr[L];
    const int nseg = a.num_segments[0];
    // with fewer than 64 adapter slots the stride is 1 and lane j holds
    // segment start j; with it, lane j also loads segment j's adapter and
    // slot j's rank and B offset, so the unit's segments need no further
    // round of loads
    const bool quick = L < kWave;
    const int lq = min(lane, max(L - 1, 0));
    const int q_id = a.req_to_lora[lq];
    const int q_rk = a.rank[lq];
    const int64_t q_bo = a.b_off[lq];

    if (tid < kGM) {
        int m = tid < rows ? a.sorted_idx[p0 + tid] : -1;
        // (checked builds) a token index outside the batch is never stored
        if (table_fault(a.err, tid < rows && (m < 0 || m >= a.M))) {
            if (tid < rows && (m < 0 || m >= a.M)) m = -1;
        }
        s_tok[tid] = m;
        s_xs[tid] = m >= 0 ? p.x_scale[m] : 0.f;
    }

    // ---- columns of the unit (one slice)
    int sl = 0;
    while (sl + 1 < a.n_sl && ct >= p.tile_start[sl + 1]) ++sl;
    const int n0 = (int)(a.slice_off[sl] + (int64_t)(ct - p.tile_start[sl]) * kGN);
    const int n1 = (int)min((int64_t)n0 + kGN, a.slice_off[sl + 1]);

    // ---- staging: thread t loads 16-byte chunk t % 8 of rows t / 8 + 32 i
    const int tr = tid / 8, tc = tid % 8;
    const uint8_t* xrow[kGXL];
#pragma unroll
    for (int i = 0; i < kGXL; ++i) {
        const int m = a.sorted_idx[p0 + min(tr + 32 * i, rows - 1)];
        xrow[i] = p.x + (int64_t)((kTableChecks && (m < 0 || m >= a.M)) ? 0 : m) * p.ldx;
    }
    const uint8_t* wrow[kGWL];
#pragma unroll
    for (int i = 0; i < kGWL; ++i)
        wrow[i] = p.W + (int64_t)min(n0 + tr + 32 * i, n1 - 1) * p.ldw;

    uint4 rs[2][kGXL + kGWL];   // stages in flight (stage s in slot s % 2)
    auto kx = [&](int s) { return min(s * kG8K + tc * 16, K - 16); };
    auto gload = [&](int s, int slot) {
        const int k = kx(s);
#pragma unroll
        for (int i = 0; i < kGXL; ++i) rs[slot][i] = ld16(xrow[i] + k);
#pragma unroll
        for (int i = 0; i < kGWL; ++i) rs[slot][kGXL + i] = ld16(wrow[i] + k);
    };
    auto lstore = [&](int s, int slot) {
        // x values past K are cleared; W there meets only those zeros
        const uint32_t m = opaque_mask(s * kG8K + tc * 16 < K);
        uint4* st = smem + (s % kGRing) * kGStage;
#pragma unroll
        for (int i = 0; i < kGXL; ++i) {
            const uint4 v = rs[slot][i];
            st[gsw(tr + 32 * i, tc)] = make_uint4(v.x & m, v.y & m, v.z & m, v.w & m);
        }
#pragma unroll
        for (int i = 0; i < kGWL; ++i) st[kGM * 8 + gsw(tr + 32 * i, tc)] = rs[slot][kGXL + i];
    };
    // one load or one LDS write of the twelve per thread and stage
    // (i < 4: x rows, else W rows); `i` is a literal at every call
    auto gload1 = [&](int s, int slot, int i) {
        rs[slot][i] = ld16((i < kGXL ? xrow[i] : wrow[i - kGXL]) + kx(s));
    };
    auto lstore1 = [&](int s, int slot, int i) {
        uint4* st = smem + (s % kGRing) * kGStage;
        if (i < kGXL) {
            const uint32_t m = opaque_mask(s * kG8K + tc * 16 < K);
            const uint4 v = rs[slot][i];
            st[gsw(tr + 32 * i, tc)] = make_uint4(v.x & m, v.y & m, v.z & m, v.w & m);
        } else {
            st[kGM * 8 + gsw(tr + 32 * (i - kGXL), tc)] = rs[slot][i];
        }
    };
    // MFMA operands of K step t (64 values) of stage s: two 16-byte chunks a lane
    struct Ops {
        uint4 a[kGRB][2];
        uint4 b[kGCB][2];
    };
    // one of the twelve operand reads of K step t (j < 8: x rows, else W rows)
    auto oread1 = [&](Ops& o, int s, int t, int j) {
        const uint4* st = smem + (s % kGRing) * kGStage;
        const int blk = j / 2, h = j % 2;
        const int c = 4 * t + 2 * h + lh;
        if (blk < kGRB) o.a[blk][h] = st[gsw(blk * 32 + lr, c)];
        else o.b[blk - kGRB][h] = st[kGM * 8 + gsw(wave * 64 + (blk - kGRB) * 32 + lr, c)];
    };

    f32x16_t acc[kGRB][kGCB];
#pragma unroll
    for (int rb = 0; rb < kGRB; ++rb)
#pragma unroll
        for (int cb = 0; cb < kGCB; ++cb)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[rb][cb][q] = 0.f;
    auto mfma1 = [&](const Ops& o, int i) {
        const int rb = i / kGCB, cb = i % kGCB;
        acc[rb][cb] = mfma32_e4m3(o.a[rb][0], o.a[rb][1], o.b[cb][0], o.b[cb][1], acc[rb][cb]);
    };

    // prologue: stages 0 and 1 in LDS, stages 2 and 3 in flight, the first
    // operands of stage 0 read
    gload(0, 0);
    gload(1, 1);
    lstore(0, 0);
    gload(2, 0);
    lstore(1, 1);
    gload(3, 1);
    __syncthreads();
    Ops o0;
#pragma unroll
    for (int j = 0; j < 12; ++j) oread1(o0, 0, 0, j);

    // the unit's first two segments (start, end, rank, B offset; rank 0:
    // none), for the B operands loaded during the last two stages
    int sfirst = 0;
    int pk_beg[2] = {0, 0}, pk_end[2] = {0, 0}, pk_rp[2] = {0, 0};
    int64_t pk_bo[2] = {0, 0};
    if (quick && p0 < m_valid) {
        sfirst = 63 - __clzll((long long)__ballot(lane <= L && srch1 <= p0));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int sj = sfirst + j;
            if (sj >= nseg) break;
            pk_beg[j] = __builtin_amdgcn_readlane(srch1, sj);
            pk_end[j] = __builtin_amdgcn_readlane(srch1, sj + 1);
            const int id = __builtin_amdgcn_readlane(q_id, sj);
            if (pk_beg[j] < p0 + rows && id >= 0 && id < L) {
                pk_rp[j] = __builtin_amdgcn_readlane(q_rk, id);
                pk_bo[j] = readlane64(q_bo, id);
            }
        }
    }

    // stage ks; `slot` (ks & 1) is a literal at every call.  The ring slot of
    // stage ks + 2 was last read (stage ks - 1) before the previous barrier;
    // stage ks + 1 was written a stage ago, before that barrier.  Each MFMA (64
    // cycles) is followed by its share of the stage's other work in a fixed
    // order: operand reads for the next K step throughout, the writes of
    // stage ks + 2 during the first K step, the loads of stage ks + 4 (into the
    // registers just written out) during the second.
    //
    // `mode` (a literal at every call): 0 = as above; 1 = no global loads
    // (stages ks + 4 do not exist); 2 = MFMAs and operand reads only (the
    // last two stages: nothing left to write, no barrier); 3 = the same
    // without the reads for a next stage.
    auto step = [&](int ks, int slot, int mode) {
        Ops o1;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mfma1(o0, i);
            if (i < 6) oread1(o1, ks, 1, 2 * i), oread1(o1, ks, 1, 2 * i + 1);
            if (mode < 2) {
                lstore1(ks + 2, slot, i);
                if (i >= 4) lstore1(ks + 2, slot, 4 + i);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            mfma1(o1, i);
            if (i < 6 && mode < 3) oread1(o0, ks + 1, 0, 2 * i), oread1(o0, ks + 1, 0, 2 * i + 1);
            if (mode == 0) {
                gload1(ks + 4, slot, i);
                if (i >= 4) gload1(ks + 4, slot, 4 + i);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (mode < 2) __syncthreads();
    };
    int ks = 0;
    for (; ks + 4 < p.nk2; ks += 2) {
        step(ks, 0, 0);
        step(ks + 1, 1, 0);
    }
    if (p.nk2 >= 4) {
        step(ks, 0, 1);
        step(ks + 1, 1, 1);
        ks += 2;
    }

    // ---- LoRA operands, loaded during the last two stages: the unit's S
    // values for this slice, the same for every segment (thread t: row t / 2,
    // rank positions 32 (t % 2) + 4 e, clamped into the row; positions past a
    // segment's rank are never multiplied), and the B operands of the first
    // two segments (rank steps t < rp / 16, as below)
    const bool lora = p0 < m_valid && a.r_max > 0;
    float4 sv[8];
    uint4 pb[2][kGCB][4];
    if (lora) {
        const int srow = min(p0 + tid / 2, a.M - 1);
        const float* sp = p.S + (int64_t)srow * a.cols + sl * a.r_max;
#pragma unroll
        for (int e = 0; e < 8; ++e)
            sv[e] = *reinterpret_cast<const float4*>(sp + min((tid % 2) * 32 + 4 * e, a.r_max - 4));
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (pk_rp[j] == 0) continue;
            const int rp = pk_rp[j];
            const uint16_t* Bt = reinterpret_cast<const uint16_t*>(a.B) + pk_bo[j];
#pragma unroll
            for (int cb = 0; cb < kGCB; ++cb) {
                const int n = min(n0 + wave * 64 + cb * 32 + lr, n1 - 1);
#pragma unroll
                for (int t = 0; t < 4; ++t)
                    pb[j][cb][t] = ld16(Bt + (int64_t)n * rp + min(t * 16, rp - 16) + lh * 8);
            }
        }
    }
    step(ks, 0, 2);
    step(ks + 1, 1, 3);
    // ---- dequantization: row 8 (q / 4) + 4 lh + q % 4 of block rb, column lr of block cb
#pragma unroll
    for (int cb = 0; cb < kGCB; ++cb) {
        const float ws = p.w_scale[min(n0 + wave * 64 + cb * 32 + lr, n1 - 1)];
#pragma unroll
        for (int rb = 0; rb < kGRB; ++rb)
#pragma unroll
            for (int q = 0; q < 16; ++q)
                acc[rb][cb][q] *= s_xs[rb * 32 + (q / 4) * 8 + lh * 4 + q % 4] * ws;
    }
    __syncthreads();     // every wave is done with the ring

    // ---- LoRA epilogue: the unit's S values as a bf16 hi / lo pair in LDS,
    // then one pass per segment that meets the unit's rows, its S rows picked
    // by a row mask on the operand
    if (lora) {
        uint16_t* sHi = reinterpret_cast<uint16_t*>(smem);   // the ring is free now
        uint16_t* sLo = sHi + kGM * kSLD;
        {
            const int row = tid / 2, j0 = (tid % 2) * 32;
#pragma unroll
            for (int e = 0; e < 8; ++e) {
                const float f[4] = {sv[e].x, sv[e].y, sv[e].z, sv[e].w};
                uint32_t h[4], l[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    h[q] = f32_to_bf16(f[q]);
                    l[q] = f32_to_bf16(f[q] - bf16_to_f32(h[q]));
                }
                *reinterpret_cast<uint2*>(sHi + row * kSLD + j0 + 4 * e) =
                    make_uint2(h[0] | (h[1] << 16), h[2] | (h[3] << 16));
                *reinterpret_cast<uint2*>(sLo + row * kSLD + j0 + 4 * e) =
                    make_uint2(l[0] | (l[1] << 16), l[2] | (l[3] << 16));
            }
        }
        __syncthreads();
        // segment of sorted position p0: the last s with seg_indptr[s] <= p0
        int s0 = sfirst;
        if (!quick) {
            const uint64_t b1 = __ballot(lane * p.seg_stride <= L && srch1 <= p0);
            const int lo = (63 - __clzll((long long)b1)) * p.seg_stride;
            const int v2 = a.seg_indptr[min(lo + lane, L)];
            const uint64_t b2 = __ballot(lane < p.seg_stride && lo + lane <= L && v2 <= p0);
            s0 = lo + 63 - __clzll((long long)b2);
        }
        for (int s = s0; s < nseg; ++s) {
            const int k = quick ? s - s0 : 2;       // 0, 1: the prefetched segments
            int beg, end, rp;
            int64_t bo = 0;
            uint4 bop[kGCB][4];
            if (k == 0) {
                beg = pk_beg[0]; end = pk_end[0]; rp = pk_rp[0];
            } else if (k == 1) {
                beg = pk_beg[1]; end = pk_end[1]; rp = pk_rp[1];
            } else {
                beg = a.seg_indptr[s];
                end = a.seg_indptr[s + 1];
                const int id = a.req_to_lora[s];
                const bool id_ok = id >= 0 && id < L;   // never index past the table
                table_fault(a.err, beg < p0 + rows && !id_ok);
                rp = (beg < p0 + rows && id_ok) ? a.rank[id] : 0;
                bo = id_ok ? a.b_off[id] : 0;
            }
            if (beg >= p0 + rows) break;
            if (rp == 0) continue;
            if (k == 0) {
#pragma unroll
                for (int cb = 0; cb < kGCB; ++cb)
#pragma unroll
                    for (int t = 0; t < 4; ++t) bop[cb][t] = pb[0][cb][t];
            } else if (k == 1) {
#pragma unroll
                for (int cb = 0; cb < kGCB; ++cb)
#pragma unroll
                    for (int t = 0; t < 4; ++t) bop[cb][t] = pb[1][cb][t];
            } else {
                const uint16_t* Bt = reinterpret_cast<const uint16_t*>(a.B) + bo;
#pragma unroll
                for (int cb = 0; cb < kGCB; ++cb) {
                    const int n = min(n0 + wave * 64 + cb * 32 + lr, n1 - 1);
#pragma unroll
                    for (int t = 0; t < 4; ++t)
                        bop[cb][t] = ld16(Bt + (int64_t)n * rp + min(t * 16, rp - 16) + lh * 8);
                }
            }
            const int r0 = max(beg - p0, 0), r1 = min(end - p0, rows);
#pragma unroll
            for (int rb = 0; rb < kGRB; ++rb) {
                if (rb * 32 + 32 <= r0 || rb * 32 >= r1) continue;
                const int row = rb * 32 + lr;
                const uint32_t m = opaque_mask(row >= r0 && row < r1);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t * 16 >= rp) continue;
                    const int o = row * kSLD + t * 16 + lh * 8;
                    const uint4 h0 = *reinterpret_cast<const uint4*>(sHi + o);
                    const uint4 l0 = *reinterpret_cast<const uint4*>(sLo + o);
                    const uint4 h = make_uint4(h0.x & m, h0.y & m, h0.z & m, h0.w & m);
                    const uint4 l = make_uint4(l0.x & m, l0.y & m, l0.z & m, l0.w & m);
#pragma unroll
                    for (int cb = 0; cb < kGCB; ++cb) {
                        acc[rb][cb] = mfma32_bf16(h, bop[cb][t], acc[rb][cb]);
                        acc[rb][cb] = mfma32_bf16(l, bop[cb][t], acc[rb][cb]);
                    }
                }
            }
        }
        __syncthreads();     // the output staging below reuses the S rows' LDS
    }

    // ---- store through LDS (the ring is free: every wave has passed the last
    // barrier): each wave stages its 128 x 64 block as bf16, rows of 72
    // values, then writes whole 16-byte row pieces.  acc[rb][cb][q] is row
    // 32 rb + 8 (q / 4) + 4 lh + q % 4, column 64 w + 32 cb + lr.  A wave reads
    // back only what it wrote itself, so no barrier is needed.
    {
        constexpr int OLD = 72;
        uint16_t* so = reinterpret_cast<uint16_t*>(smem) + wave * kGM * OLD;
#pragma unroll
        for (int rb = 0; rb < kGRB; ++rb)
#pragma unroll
            for (int cb = 0; cb < kGCB; ++cb)
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    so[(rb * 32 + (q / 4) * 8 + lh * 4 + q % 4) * OLD + cb * 32 + lr] =
                        (uint16_t)f32_to_bf16(acc[rb][cb][q]);
        const int c = lane % 8;
        const int n = n0 + wave * 64 + c * 8;       // slices are multiples of 8 wide
#pragma unroll
        for (int j = 0; j < kGM / 8; ++j) {
            const int row = j * 8 + lane / 8;
            const int m = s_tok[row];
            const uint4 v = *reinterpret_cast<const uint4*>(so + row * OLD + c * 8);
            if (m >= 0 && n < n1) *reinterpret_cast<uint4*>(p.y + (int64_t)m * p.ldy + n) = v;
        }
    }
}

hipError_t launch_gemm_fp8(const LinearArgs& a, const void* x8, int64_t ldx8, const float* x_scale,
                           const void* W8, int64_t ldw, const float* w_scale, const float* S, void* y,
                           int64_t ldy, hipStream_t st) {
    GemmFp8Params p{};
    p.a = a;
    p.x = static_cast<const uint8_t*>(x8);
    p.ldx = ldx8;
    p.x_scale = x_scale;
    p.W = static_cast<const uint8_t*>(W8);
    p.ldw = ldw;
    p.w_scale = w_scale;
    p.y = static_cast<uint16_t*>(y);
    p.ldy = ldy;
    p.S = S;
    int t = 0;
    for (int s = 0; s < a.n_sl; ++s) {
        p.tile_start[s] = t;
        t += (int)((a.slice_off[s + 1] - a.slice_off[s] + kGN - 1) / kGN);
    }
    p.tile_start[a.n_sl] = t;
    p.col_tiles = t;
    const int nk = (a.K + kG8K - 1) / kG8K;
    p.nk2 = (nk + 1) / 2 * 2;
    p.seg_stride = (a.L + 1 + kWave - 1) / kWave;
    const int row_units = (a.M + kGM - 1) / kGM;
    const unsigned grid = (unsigned)(row_units * p.col_tiles);
    hipLaunchKernelGGL(k_gemm_fp8, dim3(grid), dim3(kGThreads), 0, st, p);
    return hipGetLastError();
}

}  // namespace mlora
