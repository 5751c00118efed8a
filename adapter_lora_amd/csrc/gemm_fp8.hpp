// The shared projection in 8 bits beside the adapters for more tokens than one
// decode launch takes (see linear_fp8.hpp for the formula): lora_shrink writes
// S, then one product on e4m3 or integer operands whose epilogue scales the sums by
// xs ws, adds S B_i^T and rounds y once.  Batches that fill the chip with them take
// tiles of 256 x 256 (gemm_ring.hpp); the units here are for the others.
//
// Work unit = (32 RB consecutive sorted positions, 128 CB output columns of one
// slice); the rows of a unit may belong to several segments and to tokens
// without an adapter.  Four waves, one per SIMD, side by side; each owns all
// rows of 32 CB columns: RB x CB blocks of v_mfma_f32_32x32x64_f8f6f4 (64 cycles
// each), W rows as the first operand, so that a lane holds four consecutive
// columns of one token, K in stages of 128.
//   128 x 256 (RB 4, CB 2): a stage takes 0.85 us on every compute unit, 2.5
//     PFLOP/s; a large library product of this type reaches 2.6 on the same
//     card.  With the LDS writes left out a stage took 0.62 us, with the loads
//     left out 0.74; a third stage of loads in flight changed nothing, and
//     256 x 256 units (fewer LDS accesses per MFMA, all 512 registers) ran at
//     the same rate.
//   64 x 128 (RB 2, CB 1): two to a compute unit, for batches with too few large
//     units to fill the chip.
//
// Both operands go through an LDS ring of three stages (rows of 128 bytes, 48 KB
// or 24 KB a stage).  Global loads read whole row segments (eight
// lanes each), two stages ahead in registers; a stage is written to the ring
// two stages before its use, so the next one is always readable and each wave
// fetches its first operands while it multiplies the last of the current one.
// One barrier per stage.  Chunk c of row r stands at c ^ (r / 2) % 8: operand
// reads (32 rows, one chunk) and writes (8 rows, 8 chunks) meet distinct banks,
// and rows 32 apart are a constant apart.  With one wave per SIMD every other
// instruction is issued between two MFMAs, so the addresses are kept to one
// addition per operand and stage: the ring slots are scalar offsets, W is read
// through a buffer resource whose scalar offset is the stage, and only x rows
// (tokens, any distance apart) have 64-bit addresses.
//
// The unit order gives workgroups that share an L2 (every eighth one) the same
// columns of W for consecutive row tiles.
#pragma once

#include "common.hpp"
#include "kernels.hpp"
#include "linear_fp8.hpp"

namespace mlora {

constexpr int kG8K = 128;                          // K per stage

// Shape of a unit: 32 RB rows, 128 CB columns; four waves side by side.
template <int RB_, int CB_> struct G8Shape {
    static constexpr int RB = RB_, CB = CB_;
    static constexpr int M = 32 * RB, N = 128 * CB;
    static constexpr int Stage = (M + N) * kG8K;         // bytes of a ring slot
    static constexpr int XL = M / 32, WL = N / 32;       // rows loaded per thread and stage
    static constexpr int Waves = RB * CB >= 8 ? 1 : 2;   // per SIMD
};

// Running maximum of bf16 values without their signs, two by two: an infinity or
// NaN is 0x7f80 or more.
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
__device__ __forceinline__ u16x2_t max_magnitude(const uint4& v, u16x2_t m) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2_t, w[i] & 0x7fff7fffu));
    return m;
}

// bf16 values, infinities and NaN as zeros
__device__ __forceinline__ uint32_t finite_or_zero(uint32_t w) {
    return ((w & 0x7f80u) == 0x7f80u ? 0u : w & 0xffffu) | ((w & 0x7f800000u) == 0x7f800000u ? 0u : w & 0xffff0000u);
}
__device__ __forceinline__ uint4 finite_or_zero(const uint4& v) {
    return make_uint4(finite_or_zero(v.x), finite_or_zero(v.y), finite_or_zero(v.z), finite_or_zero(v.w));
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
    int row_tiles;
    int col_tiles;               // 256-column tiles over all slices
    int tile_start[LORA_MAX_SLICES + 1];
    int nk2;                     // stages, rounded up to even
    int seg_stride;              // ceil((L + 1) / 64): first-round search stride
};

}  // namespace mlora

#include "gemm_ring.hpp"

namespace mlora {

template <typename F, typename G>
__global__ __launch_bounds__(kGThreads, G::Waves) void k_gemm_8bit(GemmFp8Params p) {
    constexpr int kGM = G::M, kGN = G::N, kGXL = G::XL, kGWL = G::WL, kGRB = G::RB, kGCB = G::CB;
    constexpr int kG8Stage = G::Stage, kWN = 32 * kGCB;          // columns of a wave
    __shared__ uint4 smem[kGRing * kG8Stage / 16];
    __shared__ int s_tok[kGM];
    __shared__ float s_xs[kGM];
    __shared__ __attribute__((aligned(16))) float s_ws[kGN];
    const LinearArgs& a = p.a;
    // columns ct = 8 j + u % 8, bands of up to eight row tiles
    const int u = (int)blockIdx.x / 8;
    const int cts = (p.col_tiles + 7) / 8;
    const int band = u / (8 * cts), v8 = u % (8 * cts);
    const int in_band = min(8, p.row_tiles - band * 8);
    const int rt = band * 8 + v8 % in_band;
    const int ct = v8 / in_band * 8 + (int)blockIdx.x % 8;
    if (ct >= p.col_tiles) return;
    const int tid = threadIdx.x;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane % 32, lh = lane / 32;
    const int p0 = rt * kGM;
    const int rows = min(kGM, a.M - p0);
    const int K = a.K;

    // ---- columns of the unit (one slice)
    int sl = 0;
    while (sl + 1 < a.n_sl && ct >= p.tile_start[sl + 1]) ++sl;
    const int n0 = (int)(a.slice_off[sl] + (int64_t)(ct - p.tile_start[sl]) * kGN);
    const int n1 = (int)min((int64_t)n0 + kGN, a.slice_off[sl + 1]);

    // ---- staging: thread t loads 16-byte chunk t % 8 of rows t / 8 + 32 i.
    // The token indices are asked for first, the W rows need none of them.
    const int tr = tid / 8, tc = tid % 8;
    int xm[kGXL];
#pragma unroll
    for (int i = 0; i < kGXL; ++i) xm[i] = a.sorted_idx[p0 + min(tr + 32 * i, rows - 1)];
    int my_tok = tid < rows ? a.sorted_idx[p0 + tid] : -1;
    const __amdgpu_buffer_rsrc_t rw =
        uniform_rsrc(p.W + (int64_t)n0 * p.ldw, (uint32_t)((n1 - n0 - 1) * p.ldw + K));
    uint32_t woff[kGWL];
#pragma unroll
    for (int i = 0; i < kGWL; ++i)
        woff[i] = (uint32_t)(min(tr + 32 * i, n1 - n0 - 1) * p.ldw) + tc * 16;
    const uint8_t* xrow[kGXL];
    uint4 rs[2][kGXL + kGWL];   // stages in flight (stage s in slot s % 2)
    // W past K reads zeros; the x values it meets there are some of the row's own
    auto gload_w = [&](int s, int slot, int i) {
        rs[slot][kGXL + i] = buf_ld16_at<false>(rw, s * kG8K + tc * 16 < K ? woff[i] : kBufOff, (uint32_t)s * kG8K);
    };
    auto gload_x = [&](int s, int slot, int i) {
        rs[slot][i] = ld16(xrow[i] + min(s * kG8K + tc * 16, K - 16));
    };
    char* const lds = reinterpret_cast<char*>(smem);
    const int put = tr * 128 + (tc ^ (tr / 2 % 8)) * 16;
    auto lstore = [&](int ring, int slot, int i) {
        *reinterpret_cast<uint4*>(lds + put + ring + i * 4096) = rs[slot][i];
    };
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < kGWL; ++i) gload_w(s, s, i);
#pragma unroll
    for (int i = 0; i < kGXL; ++i) {
        const int m = (kTableChecks && (xm[i] < 0 || xm[i] >= a.M)) ? 0 : xm[i];
        xrow[i] = p.x + (int64_t)m * p.ldx;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < kGXL; ++i) gload_x(s, s, i);

    // (checked builds) a token index outside the batch is never stored
    if (table_fault(a.err, tid < rows && (my_tok < 0 || my_tok >= a.M))) {
        if (tid < rows && (my_tok < 0 || my_tok >= a.M)) my_tok = -1;
    }
    const float my_xs = p.x_scale[max(my_tok, 0)];
    const float my_ws = p.w_scale[min(n0 + tid, n1 - 1)];
    static_assert(kGThreads >= kGN && kGThreads >= kGM, "one row, one column scale per thread");
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

    // ---- operands: K step t of a stage is chunks 4 t + 2 h + lh, h = 0, 1
    int get[2][2];               // [t][h]: row lr
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int h = 0; h < 2; ++h) get[t][h] = lr * 128 + ((4 * t + 2 * h + lh) ^ (lr / 2 % 8)) * 16;
    const int wpart = (kGM + wave * kWN) * 128;
    struct Ops {
        uint4 x[kGRB][2];
        uint4 w[kGCB][2];
    };
    // one of the operand reads of K step t (x rows first)
    auto oread1 = [&](Ops& o, int ring, int t, int j) {
        const int blk = j / 2, h = j % 2;
        if (blk < kGRB) o.x[blk][h] = *reinterpret_cast<const uint4*>(lds + (get[t][h] + ring) + blk * 4096);
        else o.w[blk - kGRB][h] = *reinterpret_cast<const uint4*>(lds + (get[t][h] + ring + wpart) + (blk - kGRB) * 4096);
    };

    typename F::Acc32 sum[kGRB][kGCB];
#pragma unroll
    for (int rb = 0; rb < kGRB; ++rb)
#pragma unroll
        for (int cb = 0; cb < kGCB; ++cb)
#pragma unroll
            for (int q = 0; q < 16; ++q) sum[rb][cb][q] = 0;
    auto mfma1 = [&](const Ops& o, int i) {
        const int rb = i / kGCB, cb = i % kGCB;
        sum[rb][cb] = F::mma32(o.w[cb][0], o.w[cb][1], o.x[rb][0], o.x[rb][1], sum[rb][cb]);
    };

    // prologue: stages 0 and 1 in LDS, stages 2 and 3 in flight, the first
    // operands of stage 0 read
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
        for (int i = 0; i < kGXL + kGWL; ++i) lstore(s * kG8Stage, s, i);
#pragma unroll
        for (int i = 0; i < kGWL; ++i) gload_w(s + 2, s, i);
#pragma unroll
        for (int i = 0; i < kGXL; ++i) gload_x(s + 2, s, i);
    }
    if (tid < kGM) {
        s_tok[tid] = my_tok;
        s_xs[tid] = my_xs;
    }
    if (tid < kGN) s_ws[tid] = my_ws;
    __syncthreads();
    Ops o0;
    constexpr int kReads = 2 * (kGRB + kGCB), kMf = kGRB * kGCB, kLd = kGXL + kGWL;
#pragma unroll
    for (int j = 0; j < kReads; ++j) oread1(o0, 0, 0, j);

    // segment s of the unit: rows [beg, end) of the sorted order, the adapter's
    // rank (0: none) and B offset; beg past the unit: no more segments
    struct Seg {
        int beg, end, rp;
        int64_t bo;
    };
    auto segment = [&](int s) {
        Seg g{INT32_MAX, 0, 0, 0};
        if (s >= nseg) return g;
        int id;
        if (quick) {
            g.beg = __builtin_amdgcn_readlane(srch1, s);
            g.end = __builtin_amdgcn_readlane(srch1, s + 1);
            id = __builtin_amdgcn_readlane(q_id, s);
        } else {
            g.beg = __builtin_amdgcn_readfirstlane(a.seg_indptr[s]);
            g.end = __builtin_amdgcn_readfirstlane(a.seg_indptr[s + 1]);
            id = __builtin_amdgcn_readfirstlane(a.req_to_lora[s]);
        }
        if (g.beg >= p0 + rows) return g;
        const bool id_ok = id >= 0 && id < L;   // never index past the table
        table_fault(a.err, !id_ok);
        if (!id_ok) return g;
        g.rp = quick ? __builtin_amdgcn_readlane(q_rk, id) : __builtin_amdgcn_readfirstlane(a.rank[id]);
        g.bo = quick ? readlane64(q_bo, id) : readlane64(a.b_off[id], 0);
        return g;
    };
    auto load_b = [&](uint4 (&b)[kGCB][4], const Seg& g) {
        if (g.rp == 0) return;
        const uint16_t* Bt = reinterpret_cast<const uint16_t*>(a.B) + g.bo;
#pragma unroll
        for (int cb = 0; cb < kGCB; ++cb) {
            const int n = min(n0 + wave * kWN + cb * 32 + lr, n1 - 1);
#pragma unroll
            for (int t = 0; t < 4; ++t)
                b[cb][t] = ld16(Bt + (int64_t)n * g.rp + min(t * 16, g.rp - 16) + lh * 8);
        }
    };
    // the segment that holds sorted position p0: the last s with seg_indptr[s] <= p0
    const bool lora = p0 < m_valid && a.r_max > 0;
    int s0 = 0;
    if (lora) {
        const uint64_t b1 = __ballot(lane * p.seg_stride <= L && srch1 <= p0);
        s0 = (63 - __clzll((long long)b1)) * p.seg_stride;
        if (!quick) {
            const int v2 = a.seg_indptr[min(s0 + lane, L)];
            const uint64_t b2 = __ballot(lane < p.seg_stride && s0 + lane <= L && v2 <= p0);
            s0 += 63 - __clzll((long long)b2);
        }
    }

    // stage ks; `slot` (ks & 1) is a literal at every call; r0, r1, r2 are the
    // ring offsets of stages ks, ks + 1 and ks + 2.  The ring slot of stage
    // ks + 2 was last read (stage ks - 1) before the previous barrier; stage
    // ks + 1 was written a stage ago, before that barrier.  Each MFMA (64
    // cycles) is followed by its share of the stage's other work in a fixed
    // order: operand reads for the next K step throughout, the writes of
    // stage ks + 2 during the first K step, the loads of stage ks + 4 (into the
    // registers just written out) during the second.
    //
    // `mode` (a literal at every call): 0 = as above; 1 = no global loads
    // (stages ks + 4 do not exist); 2 = MFMAs and operand reads only (the
    // last two stages: nothing left to write, no barrier); 3 = the same
    // without the reads for a next stage.
    int r0 = 0, r1 = kG8Stage, r2 = 2 * kG8Stage;
    auto step = [&](int ks, int slot, int mode) {
        Ops o1;
#pragma unroll
        for (int i = 0; i < kMf; ++i) {
            mfma1(o0, i);
#pragma unroll
            for (int j = i * kReads / kMf; j < (i + 1) * kReads / kMf; ++j) oread1(o1, r0, 1, j);
            if (mode < 2)
#pragma unroll
                for (int j = i * kLd / kMf; j < (i + 1) * kLd / kMf; ++j) lstore(r2, slot, j);
            __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < kMf; ++i) {
            mfma1(o1, i);
            if (mode < 3)
#pragma unroll
                for (int j = i * kReads / kMf; j < (i + 1) * kReads / kMf; ++j) oread1(o0, r1, 0, j);
            if (mode == 0)
#pragma unroll
                for (int j = i * kLd / kMf; j < (i + 1) * kLd / kMf; ++j) {
                    if (j < kGWL) gload_w(ks + 4, slot, j);
                    else gload_x(ks + 4, slot, j - kGWL);
                }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (mode < 2) __syncthreads();
        const int t = r0;
        r0 = r1; r1 = r2; r2 = t;
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
    // values for this slice, the same for every segment (kSV of a row per
    // thread, clamped into the row; positions past a segment's rank are never
    // multiplied), and the B operands of the first segment (rank steps
    // t < rp / 16, as below)
    constexpr int kSV = kGM * LORA_MAX_RANK / kGThreads, kSVT = LORA_MAX_RANK / kSV;
    float4 sv[kSV / 4];
    uint4 pb[2][kGCB][4];
    Seg sg[2] = {{INT32_MAX, 0, 0, 0}, {INT32_MAX, 0, 0, 0}};
    if (lora) {
        const int srow = min(p0 + tid / kSVT, a.M - 1);
        const float* sp = p.S + (int64_t)srow * a.cols + sl * a.r_max;
#pragma unroll
        for (int e = 0; e < kSV / 4; ++e)
            sv[e] = *reinterpret_cast<const float4*>(sp + min((tid % kSVT) * kSV + 4 * e, a.r_max - 4));
        sg[0] = segment(s0);
        load_b(pb[0], sg[0]);
    }
    step(ks, 0, 2);
    step(ks + 1, 1, 3);
    // ---- dequantization: row lr of block rb, columns 8 (q / 4) + 4 lh + q % 4 of block cb
    f32x16_t acc[kGRB][kGCB];
    float xs[kGRB];
#pragma unroll
    for (int rb = 0; rb < kGRB; ++rb) xs[rb] = s_xs[rb * 32 + lr];
#pragma unroll
    for (int cb = 0; cb < kGCB; ++cb)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
            const float4 ws = *reinterpret_cast<const float4*>(s_ws + wave * kWN + cb * 32 + 8 * g + 4 * lh);
#pragma unroll
            for (int rb = 0; rb < kGRB; ++rb) {
                acc[rb][cb][4 * g] = (float)sum[rb][cb][4 * g] * (xs[rb] * ws.x);
                acc[rb][cb][4 * g + 1] = (float)sum[rb][cb][4 * g + 1] * (xs[rb] * ws.y);
                acc[rb][cb][4 * g + 2] = (float)sum[rb][cb][4 * g + 2] * (xs[rb] * ws.z);
                acc[rb][cb][4 * g + 3] = (float)sum[rb][cb][4 * g + 3] * (xs[rb] * ws.w);
            }
        }
    __syncthreads();     // every wave is done with the ring

    // ---- LoRA epilogue: the unit's S values as a bf16 hi / lo pair in LDS,
    // then one pass per segment that meets the unit's rows, its S rows picked
    // by a row mask on the operand
    bool special = false;        // B rows of this wave's columns with an infinity or NaN
    if (lora) {
        uint16_t* sHi = reinterpret_cast<uint16_t*>(smem);   // the ring is free now
        uint16_t* sLo = sHi + kGM * kSLD;
        {
            const int row = tid / kSVT, j0 = (tid % kSVT) * kSV;
#pragma unroll
            for (int e = 0; e < kSV / 4; ++e) {
                const uint32_t h0 = pack_bf16(sv[e].x, sv[e].y), h1 = pack_bf16(sv[e].z, sv[e].w);
                const uint32_t l0 = pack_bf16(sv[e].x - __uint_as_float(h0 << 16), sv[e].y - __uint_as_float(h0 & 0xffff0000u));
                const uint32_t l1 = pack_bf16(sv[e].z - __uint_as_float(h1 << 16), sv[e].w - __uint_as_float(h1 & 0xffff0000u));
                *reinterpret_cast<uint2*>(sHi + row * kSLD + j0 + 4 * e) = make_uint2(h0, h1);
                *reinterpret_cast<uint2*>(sLo + row * kSLD + j0 + 4 * e) = make_uint2(l0, l1);
            }
        }
        __syncthreads();
        // A block of 32 rows that a segment covers in part has zeros for its
        // other tokens, and zeros times an infinity are not zero: infinities and
        // NaN of B stay out of this product and join the segment's own tokens
        // at the end.  (A select for every partly covered sum, which the AGPRs
        // that hold them cannot take, cost 93 -> 105 us at 512 x 28672.)
        auto add = [&](int beg, int end, int rp, uint4 (&bop)[kGCB][4]) {
            const int b0 = max(beg - p0, 0), b1 = min(end - p0, rows);
            u16x2_t top = {0, 0};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t * 16 >= rp) continue;
#pragma unroll
                for (int cb = 0; cb < kGCB; ++cb) top = max_magnitude(bop[cb][t], top);
            }
            if (__ballot(top[0] >= 0x7f80 || top[1] >= 0x7f80) != 0ull) {
                special = true;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int cb = 0; cb < kGCB; ++cb) bop[cb][t] = finite_or_zero(bop[cb][t]);
            }
#pragma unroll
            for (int rb = 0; rb < kGRB; ++rb) {
                if (rb * 32 + 32 <= b0 || rb * 32 >= b1) continue;
                const int row = rb * 32 + lr;
                const uint32_t m = opaque_mask(row >= b0 && row < b1);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t * 16 >= rp) continue;
                    const int o = row * kSLD + t * 16 + lh * 8;
                    const uint4 h = and4(*reinterpret_cast<const uint4*>(sHi + o), m);
                    const uint4 l = and4(*reinterpret_cast<const uint4*>(sLo + o), m);
#pragma unroll
                    for (int cb = 0; cb < kGCB; ++cb) {
                        acc[rb][cb] = mfma32_bf16(bop[cb][t], h, acc[rb][cb]);
                        acc[rb][cb] = mfma32_bf16(bop[cb][t], l, acc[rb][cb]);
                    }
                }
            }
        };
        // the next segment's B rows are in flight while one is added
        for (int s = s0; sg[0].beg < p0 + rows; s += 2) {
            sg[1] = segment(s + 1);
            load_b(pb[1], sg[1]);
            if (sg[0].rp > 0) add(sg[0].beg, sg[0].end, sg[0].rp, pb[0]);
            sg[0] = segment(s + 2);
            load_b(pb[0], sg[0]);
            if (sg[1].beg < p0 + rows && sg[1].rp > 0) add(sg[1].beg, sg[1].end, sg[1].rp, pb[1]);
        }
        __syncthreads();     // the output staging below reuses the S rows' LDS
    }

    // ---- store through LDS (the ring is free: every wave has passed the last
    // barrier): each wave stages its part as bf16, rows of 8 values more than
    // its columns, then writes whole row pieces.  A wave reads back only what
    // it wrote itself, so no barrier is needed.
    constexpr int OLD = kWN + 8, kCh = kWN / 8;     // 16-byte chunks of a row
    uint16_t* so = reinterpret_cast<uint16_t*>(smem) + wave * kGM * OLD;
    static_assert(4 * kGM * OLD * 2 <= kGRing * kG8Stage && 2 * kGM * kSLD * 2 <= kGRing * kG8Stage,
                  "staged output and S must fit the ring");
#pragma unroll
    for (int rb = 0; rb < kGRB; ++rb)
#pragma unroll
        for (int cb = 0; cb < kGCB; ++cb)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<uint2*>(so + (rb * 32 + lr) * OLD + cb * 32 + 8 * g + 4 * lh) =
                    make_uint2(pack_bf16(acc[rb][cb][4 * g], acc[rb][cb][4 * g + 1]),
                               pack_bf16(acc[rb][cb][4 * g + 2], acc[rb][cb][4 * g + 3]));
    stage_order();
    if (special) {
        // what the product left out, one column a lane: an infinity or NaN
        // whatever the finite terms are, so it may be added to the rounded sum.
        // The whole wavefront walks the segments, whose entries any lane may
        // hold; only the columns are fewer than the lanes.
        const int col = min(n0 + wave * kWN + lane, n1 - 1);
        for (int s = s0;; ++s) {
            const Seg g = segment(s);
            if (g.beg >= p0 + rows) break;
            const uint16_t* B = reinterpret_cast<const uint16_t*>(a.B) + g.bo + (int64_t)col * g.rp;
            for (int j = 0; lane < kWN && j < g.rp; ++j) {
                if ((B[j] & 0x7f80u) != 0x7f80u) continue;
                const float b = bf16_to_f32(B[j]);
                for (int row = max(g.beg - p0, 0); row < min(g.end - p0, rows); ++row) {
                    uint16_t& o = so[row * OLD + lane];
                    o = (uint16_t)f32_to_bf16(bf16_to_f32(o) + b * p.S[(int64_t)(p0 + row) * a.cols + sl * a.r_max + j]);
                }
            }
        }
        stage_order();
    }
    const int c = lane % kCh;
    const int n = n0 + wave * kWN + c * 8;          // slices are multiples of 8 wide
#pragma unroll
    for (int j = 0; j < kGM * kCh / kWave; ++j) {
        const int row = j * (kWave / kCh) + lane / kCh;
        const int m = s_tok[row];
        const uint4 v = *reinterpret_cast<const uint4*>(so + row * OLD + c * 8);
        if (m >= 0 && n < n1) *reinterpret_cast<uint4*>(p.y + (int64_t)m * p.ldy + n) = v;
    }
}

template <typename F, typename G>
hipError_t launch_gemm_8bit_as(GemmFp8Params& p, hipStream_t st) {
    const LinearArgs& a = p.a;
    int t = 0;
    for (int s = 0; s < a.n_sl; ++s) {
        p.tile_start[s] = t;
        t += (int)((a.slice_off[s + 1] - a.slice_off[s] + G::N - 1) / G::N);
    }
    p.tile_start[a.n_sl] = t;
    p.col_tiles = t;
    p.row_tiles = (a.M + G::M - 1) / G::M;
    const unsigned grid = (unsigned)(p.row_tiles * ((p.col_tiles + 7) / 8 * 8));
    hipLaunchKernelGGL((k_gemm_8bit<F, G>), dim3(grid), dim3(kGThreads), 0, st, p);
    return hipGetLastError();
}

template <typename F>
hipError_t launch_gemm_8bit(const LinearArgs& a, const void* x8, int64_t ldx8, const float* x_scale,
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
    auto columns = [&](int width) {              // column tiles of that width
        int64_t t = 0;
        for (int i = 0; i < a.n_sl; ++i) t += (a.slice_off[i + 1] - a.slice_off[i] + width - 1) / width;
        return t;
    };
    const int nk = (a.K + kG8K - 1) / kG8K;
    p.nk2 = (nk + 1) / 2 * 2;
    p.seg_stride = (a.L + 1 + kWave - 1) / kWave;
    // Small units finish sooner while they fit the chip in few rounds.  A round of
    // 256 small ones (two share a compute unit) takes 1.4 us and 8.5 for every 4096
    // of K, a round of 256 large ones 8 and 20 (the first loads, deltas and store do
    // not grow with K, so short K favours the small ones).  Measured calls, small
    // against large (8 adapters): K = 512, 256 x 4096 12.6 / 21.6 us, 768 x 8192 20.4
    // / 22.4, 512 x 28672 32.2 / 38.1; K = 1024, 512 x 14336 25.9 / 26.4, 512 x 28672
    // 43.4 / 46.9; K = 2048, 768 x 4096 22.8 / 30.3, 512 x 14336 37.9 / 34.1; K = 4096,
    // 256 x 4096 25.3 / 43.2, 768 x 8192 49.8 / 47.0, 2048 x 4096 61.0 / 52.4, 512 x 28672
    // 103 / 87; K = 8192, 768 x 4096 61.2 / 73.0, 768 x 8192 85.5 / 74.6; K = 16384, 768 x
    // 4096 107 / 124, 2048 x 4096 202 / 146.  (Past 4096 rounds, 2^20 units, large ones
    // keep the grid below 2^32 threads.)
    const int64_t ns = columns(128), nl = columns(256), K = a.K;
    const int64_t small = ((a.M + 63) / 64 * ns + 255) / 256, large = ((a.M + 127) / 128 * nl + 255) / 256;
    const int64_t cost_s = small <= 4096 ? small * (14 * 4096 + 85 * K) : INT64_MAX;
    const int64_t cost_l = large * (80 * 4096 + 200 * K);
    // Tiles of 256 x 256 (gemm_ring.hpp) run at 2.7 PFLOP/s and more and lose most where
    // they do not fill the chip: a round takes 1.2 (K = 512) to 1.6 (K = 4096) times one
    // of the large units.  Measured calls in int8, the units' better choice against tiles
    // (8 adapters): K = 512, 512 x 28672 33.9 / 33.7 us; K = 1024, 1024 x 14336 40.0 / 37.8;
    // K = 2048, 768 x 8192 34.7 / 52.4; K = 4096, 300 x 28672 82.5 / 75.6, 512 x 28672 (12
    // adapters, 36 runs) 107 / 90, 2048 x 4096 59.8 / 85.5, 4096 x 4096 105 / 88, 8192 x 4096
    // 200 / 165, 2048 x 28672 312 / 286; K = 8192, 1024 x 8192 92 / 135.  In e4m3 4096 x 4096
    // 98 / 86, 8192 x 4096 170 / 144, 512 x 28672 101 / 87, 2048 x 4096 55 / 79.  The sums
    // are the same bits either way.
    //
    // A tile walks the segments of its 256 rows one after the other, which small units
    // hide behind each other and large ones have half as many of.  The host knows the
    // slots, not the segments: it counts every slot as used evenly.  Measured in e4m3,
    // units against tiles: 394 x 608 to 28800 with 8 / 16 / 48 / 256 slots 39.9 / 43.4 / 64.2
    // / 177 us against 38.7 / 45.4 / 77.0 / 246; 975 x 1344 to 11496 with 32 / 60 / 128 53.7 / 63.0
    // / 97.3 and 52.6 / 65.5 / 112; 512 x 4096 to 28672 with 60 / 128 / 256 145 / 207 / 283 and 134
    // / 198 / 288; 2079 x 4480 to 7096 with 256 192 and 154.
    const int64_t tiles = (int64_t)((a.M + kRingRows - 1) / kRingRows) * nl;
    const int64_t slots = a.L < a.M ? a.L : a.M;
    auto met = [&](int64_t rows) { return std::min(slots, slots * rows / a.M + 1); };
    const int64_t cost_r = tiles <= (1 << 22) ? (tiles + 255) / 256 * (115 * 4096 + 330 * K + 10240 * met(256)) : INT64_MAX;
    if (cost_r < (cost_s < cost_l ? cost_s : cost_l + large * 6144 * met(128))) return launch_gemm_ring<F>(p, st);
    if (cost_s < cost_l) return launch_gemm_8bit_as<F, G8Shape<2, 1>>(p, st);
    return launch_gemm_8bit_as<F, G8Shape<4, 2>>(p, st);
}

// Any number of tokens, S by way of memory: shrink, then one of the products.
template <typename F>
hipError_t launch_linear_8bit_many(const LinearArgs& a, const void* W8, int64_t ldw, const float* w_scale,
                                  const void* x8, int64_t ldx8, const float* x_scale, const void* x,
                                  int64_t ldx, float* S, void* y, int64_t ldy, void* ws, hipStream_t st) {
    // One launch over all of K reads the rows of x again for every 16 columns of
    // S; partial sums over K (two launches) read them once.  Measured, the call
    // with one and the other, 4096 wide: 512 tokens of 64 columns 41.5 / 45.8 us,
    // 1024 44.3 / 45.4, 2048 57.1 / 55.5; 1024 tokens of 192 columns 55.0 / 52.6;
    // 16384 tokens of 16 columns 195 / 203.
    const bool rows = a.cols == 16 || (int64_t)a.M * a.cols <= 65536;
    const hipError_t e = rows ? launch_shrink_rows(a, static_cast<const uint16_t*>(x), ldx, S, st)
                              : launch_shrink(a, x, ldx, S, ws, st);
    if (e != hipSuccess) return e;
    // The decode kernel over groups of 64 tokens while one round of its units
    // (32 columns a group) is enough and K is long enough for eight wavefronts
    // to share.  Measured, small units of the product against groups, with 24
    // adapters (segments follow each other in a unit of the product, in a group the
    // eight wavefronts share them), 8, and none: 65 tokens, 2048 columns, K = 2048 31.6 /
    // 19.0 us, -, 11.4 / 11.9, K = 4096 41.5 / 22.6, -, 16.3 / 12.0; 128 tokens, 4096
    // columns, K = 1024 -, 14.9 / 18.2, -, K = 2048 25.7 / 21.0, 17.5 / 18.8, 11.5 / 13.6, K
    // = 4096 36.0 / 25.7, 26.0 / 22.6, 17.6 / 15.6; 512 tokens, 1024 columns, 8 adapters, K =
    // 2048 16.0 / 20.3, 4096 23.4 / 23.4, 8192 36.6 / 31.6.
    const int64_t units = (a.M + 63) / 64 * ((a.slice_off[a.n_sl] + 31) / 32);
    if (units <= 256 && a.K >= 2048 && ldx8 < INT32_MAX / (int64_t)a.M)
        return launch_linear_8bit_groups<F>(a, W8, ldw, w_scale, x8, ldx8, x_scale, S, y, ldy, st);
    return launch_gemm_8bit<F>(a, x8, ldx8, x_scale, W8, ldw, w_scale, S, y, ldy, st);
}

hipError_t launch_linear_8bit(bool int8, const LinearArgs& a, const void* W8, int64_t ldw, const float* w_scale,
                              const void* x8, int64_t ldx8, const float* x_scale, const void* x, int64_t ldx,
                              void* y, int64_t ldy, void* ws, hipStream_t st) {
    return int8 ? launch_linear_8bit<FmtInt8>(a, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, y, ldy, ws, st)
                : launch_linear_8bit<FmtE4m3>(a, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, y, ldy, ws, st);
}

hipError_t launch_linear_8bit_many(bool int8, const LinearArgs& a, const void* W8, int64_t ldw, const float* w_scale,
                                   const void* x8, int64_t ldx8, const float* x_scale, const void* x, int64_t ldx,
                                   float* S, void* y, int64_t ldy, void* ws, hipStream_t st) {
    return int8 ? launch_linear_8bit_many<FmtInt8>(a, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, S, y, ldy, ws, st)
                : launch_linear_8bit_many<FmtE4m3>(a, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, S, y, ldy, ws, st);
}

}  // namespace mlora
