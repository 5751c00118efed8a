// The shared projection in 8 bits beside the adapters in tiles of 256 sorted
// positions by 256 output columns of one slice (see linear_fp8.hpp for the formula
// and gemm_fp8.hpp for the call): the main loop of ring_product.hpp, then the
// scales, the deltas of the tile's segments and one rounding.
//
// What bounds it: the matrix unit and the clock that its power leaves.  512 tokens to
// 28672 columns, K = 4096, and 8192 tokens to 4096, the calls with their shrink: int8 90
// and 166 us (in units of 128 x 256 103 and 189), e4m3 87 and 144 (101 and 170); the
// kernel's share in int8 82 and 150.
//
// Segments: the tile's rows may belong to several and to tokens without an adapter.
// S goes to LDS once as a bf16 hi / lo pair; each segment multiplies its rows of it,
// picked by a mask on the operand, with its adapter's B rows on the same 32 x 32
// blocks of sums.
#pragma once

#include "common.hpp"
#include "formats.hpp"
#include "kernels.hpp"
#include "ring_product.hpp"

namespace mlora {

// A wave-uniform entry of a table that the launch only reads, by way of the scalar
// cache.  (Behind the loads to LDS the compiler takes the tables as changed and reads
// them as vectors, whose waits then include the B rows in flight.)
template <typename T> __device__ __forceinline__ T table_entry(const T* table, int i) {
    typedef const __attribute__((address_space(4))) T entry_t;
    return reinterpret_cast<entry_t*>(reinterpret_cast<uintptr_t>(table))[i];
}

// Keeps a block of sums together in accumulation registers: split into its elements
// across the branches below, the sums are spilled.  (11 other values in int8 and 12 in
// e4m3 still are, before and behind the main loop, none within it.)
template <typename A> __device__ __forceinline__ void keep_block(A& v) { asm volatile("" : "+a"(v)); }

template <typename R>
__device__ __forceinline__ void ring_tile(const GemmFp8Params& p, uint4* smem, int sl, int p0, int rows, int n0, int cols) {
    constexpr int RB = R::RB, CB = R::CB, NX = R::NX, kM = R::kRows;
    const LinearArgs& a = p.a;
    const int tid = threadIdx.x;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane % 32, lh = lane / 32;
    const int r0 = R::row0(wave), c0 = R::col0(wave), L = a.L;

    int m_in[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) m_in[i] = a.sorted_idx[p0 + min(R::load_row(wave, i), rows - 1)];
    int my_tok = tid < rows ? a.sorted_idx[p0 + tid] : -1;
    // what the epilogue needs of the segments: lane j holds seg_indptr[j seg_stride], and
    // with fewer than 64 slots (stride 1) segment j's adapter, slot j's rank and B offset
    const int srch1 = a.seg_indptr[min(lane * p.seg_stride, L)];
    const int m_valid = a.seg_indptr[L];
    const int nseg = a.num_segments[0];
    const bool quick = L < kWave;
    const int lq = min(lane, max(L - 1, 0));
    const int q_id = a.req_to_lora[lq];
    const int q_rk = a.rank[lq];
    const int64_t q_bo = a.b_off[lq];
    float my_xs, my_ws;
    // the tile's S values for this slice: thread t four of row t / 16 + 16 e, clamped into
    // the row (positions past a segment's rank are never multiplied)
    const bool lora = p0 < m_valid && a.r_max > 0;
    constexpr int kSV = kM / 16;
    const int srow = tid / 16, sj = tid % 16 * 4;
    float4 sv[kSV];
    auto load_s = [&]() {
        const float* sp = p.S + sl * a.r_max + min(sj, a.r_max - 4);
#pragma unroll
        for (int e = 0; e < kSV; ++e)
            sv[e] = *reinterpret_cast<const float4*>(sp + (int64_t)min(p0 + srow + 16 * e, a.M - 1) * a.cols);
    };
    // segment s of the tile: rows [beg, end) of the sorted order, the adapter's
    // rank (0: none) and B offset; beg past the tile: no more segments
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
            g.beg = __builtin_amdgcn_readfirstlane(table_entry(a.seg_indptr, s));
            g.end = __builtin_amdgcn_readfirstlane(table_entry(a.seg_indptr, s + 1));
            id = __builtin_amdgcn_readfirstlane(table_entry(a.req_to_lora, s));
        }
        if (g.beg >= p0 + rows) return g;
        const bool id_ok = id >= 0 && id < L;   // never index past the table
        table_fault(a.err, !id_ok);
        if (!id_ok) return g;
        g.rp = quick ? __builtin_amdgcn_readlane(q_rk, id) : __builtin_amdgcn_readfirstlane(table_entry(a.rank, id));
        g.bo = quick ? readlane64(q_bo, id) : readlane64(table_entry(a.b_off, id), 0);
        return g;
    };
    auto load_b = [&](uint4 (&b)[CB][4], const Seg& g) {
        if (g.rp == 0) return;
        const uint16_t* Bt = reinterpret_cast<const uint16_t*>(a.B) + g.bo;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
            const int n = n0 + min(c0 + cb * 32 + lr, cols - 1);
#pragma unroll
            for (int t = 0; t < 4; ++t) b[cb][t] = ld16(Bt + (int64_t)n * g.rp + min(t * 16, g.rp - 16) + lh * 8);
        }
    };
    // the segment that holds sorted position p0: the last s with seg_indptr[s] <= p0
    int s0 = 0;
    uint4 pb[2][CB][4];
    Seg sg[2] = {{INT32_MAX, 0, 0, 0}, {INT32_MAX, 0, 0, 0}};
    auto first_segment = [&]() {
        const uint64_t b1 = __ballot(lane * p.seg_stride <= L && srch1 <= p0);
        s0 = (63 - __clzll((long long)b1)) * p.seg_stride;
        if (!quick) {
            const int v2 = a.seg_indptr[min(s0 + lane, L)];
            const uint64_t b2 = __ballot(lane < p.seg_stride && s0 + lane <= L && v2 <= p0);
            s0 += 63 - __clzll((long long)b2);
        }
        sg[0] = segment(s0);
        load_b(pb[0], sg[0]);
    };
    auto x_rows = [&](const char* (&xp)[NX]) {
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int m = (kTableChecks && (m_in[i] < 0 || m_in[i] >= a.M)) ? 0 : m_in[i];
            xp[i] = reinterpret_cast<const char*>(p.x) + (int64_t)m * p.ldx + R::load_byte(wave);
        }
        // (checked builds) a token index outside the batch is never stored
        if (table_fault(a.err, tid < rows && (my_tok < 0 || my_tok >= a.M))) {
            if (tid < rows && (my_tok < 0 || my_tok >= a.M)) my_tok = -1;
        }
        my_xs = p.x_scale[max(my_tok, 0)];
        my_ws = p.w_scale[n0 + min(tid, cols - 1)];
    };
    typename R::Acc sum[RB][CB];
    ring_product<R>(smem, reinterpret_cast<const char*>(p.W) + (int64_t)n0 * p.ldw, p.ldw, cols, a.K, 0, x_rows, sum);

    // ---- scales: row 32 rb + lr, columns 32 cb + 8 (q / 4) + 4 lh + q % 4 of the wave's part
    constexpr int kScalesAt = 2 * kM * kSLD * 2;     // behind S's two halves
    static_assert(kScalesAt % 16 == 0 && kScalesAt + 3 * kRingRows * 4 <= kRingLds, "S and the scales fit the LDS");
    int* const s_tok = reinterpret_cast<int*>(reinterpret_cast<char*>(smem) + kScalesAt);
    float* const s_xs = reinterpret_cast<float*>(s_tok + kRingRows);
    float* const s_ws = s_xs + kRingRows;
    s_tok[tid] = my_tok;
    s_xs[tid] = my_xs;
    s_ws[tid] = my_ws;
    __syncthreads();
    // in place, a block at a time: both types of sums at once would not fit the registers
    float xs[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) xs[rb] = s_xs[r0 + rb * 32 + lr];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        float4 ws[4];
#pragma unroll
        for (int g = 0; g < 4; ++g) ws[g] = *reinterpret_cast<const float4*>(s_ws + c0 + cb * 32 + 8 * g + 4 * lh);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            f32x16_t f;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                f[4 * g] = (float)sum[rb][cb][4 * g] * (xs[rb] * ws[g].x);
                f[4 * g + 1] = (float)sum[rb][cb][4 * g + 1] * (xs[rb] * ws[g].y);
                f[4 * g + 2] = (float)sum[rb][cb][4 * g + 2] * (xs[rb] * ws[g].z);
                f[4 * g + 3] = (float)sum[rb][cb][4 * g + 3] * (xs[rb] * ws[g].w);
            }
            sum[rb][cb] = __builtin_bit_cast(typename R::Acc, f);
            keep_block(sum[rb][cb]);
            __builtin_amdgcn_sched_barrier(0);
        }
    }

    uint16_t* const sHi = reinterpret_cast<uint16_t*>(smem);
    uint16_t* const sLo = sHi + kM * kSLD;
    if (lora) {
        first_segment();
        load_s();
#pragma unroll
        for (int e = 0; e < kSV; ++e) {
            const uint32_t h0 = pack_bf16(sv[e].x, sv[e].y), h1 = pack_bf16(sv[e].z, sv[e].w);
            const uint32_t l0 = pack_bf16(sv[e].x - __uint_as_float(h0 << 16), sv[e].y - __uint_as_float(h0 & 0xffff0000u));
            const uint32_t l1 = pack_bf16(sv[e].z - __uint_as_float(h1 << 16), sv[e].w - __uint_as_float(h1 & 0xffff0000u));
            *reinterpret_cast<uint2*>(sHi + (srow + 16 * e) * kSLD + sj) = make_uint2(h0, h1);
            *reinterpret_cast<uint2*>(sLo + (srow + 16 * e) * kSLD + sj) = make_uint2(l0, l1);
        }
    }
    __syncthreads();
    // ---- deltas.  A block of 32 rows that a segment covers in part has zeros for its
    // other tokens, and zeros times an infinity are not zero: infinities and NaN of B
    // stay out of this product and join the segment's own tokens at the end.
    bool special = false;        // B rows of this wave's columns with an infinity or NaN
    if (lora) {
        auto add = [&](int beg, int end, int rp, uint4 (&bop)[CB][4]) {
            const int b0 = max(beg - p0, 0), b1 = min(end - p0, rows);
            u16x2_t top = {0, 0};
#pragma unroll
            for (int t = 0; t < 4; ++t) {
                if (t * 16 >= rp) continue;
#pragma unroll
                for (int cb = 0; cb < CB; ++cb) top = max_magnitude(bop[cb][t], top);
            }
            if (__ballot(top[0] >= 0x7f80 || top[1] >= 0x7f80) != 0ull) {
                special = true;
#pragma unroll
                for (int t = 0; t < 4; ++t)
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) bop[cb][t] = finite_or_zero(bop[cb][t]);
            }
#pragma unroll
            for (int rb = 0; rb < RB; ++rb) {
                if (r0 + rb * 32 + 32 <= b0 || r0 + rb * 32 >= b1) continue;
                const int row = r0 + rb * 32 + lr;
                const uint32_t m = opaque_mask(row >= b0 && row < b1);
#pragma unroll
                for (int t = 0; t < 4; ++t) {
                    if (t * 16 >= rp) continue;
                    const int o = row * kSLD + t * 16 + lh * 8;
                    const uint4 h = and4(*reinterpret_cast<const uint4*>(sHi + o), m);
                    const uint4 l = and4(*reinterpret_cast<const uint4*>(sLo + o), m);
#pragma unroll
                    for (int cb = 0; cb < CB; ++cb) {
                        const f32x16_t v = mfma32_bf16(bop[cb][t], h, __builtin_bit_cast(f32x16_t, sum[rb][cb]));
                        sum[rb][cb] = __builtin_bit_cast(typename R::Acc, mfma32_bf16(bop[cb][t], l, v));
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
    }

    // ---- one rounding
    uint16_t* dst[RB][2];
    bool ok[RB][2];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int m = s_tok[r0 + rb * 32 + 16 * h + lane % 16];
            ok[rb][h] = m >= 0;
            dst[rb][h] = p.y + (int64_t)max(m, 0) * p.ldy + n0 + c0 + 8 * store_chunk();
        }
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const bool in = c0 + cb * 32 + 8 * store_chunk() < cols;       // slices are multiples of 8 wide
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            keep_block(sum[rb][cb]);
            store_block(__builtin_bit_cast(f32x16_t, sum[rb][cb]), {dst[rb][0] + cb * 32, dst[rb][1] + cb * 32},
                        {ok[rb][0] && in, ok[rb][1] && in});
            __builtin_amdgcn_sched_barrier(0);
        }
    }
    if (special) {
        // what the product left out, one column a lane: an infinity or NaN whatever
        // the finite terms are, so it may be added to the rounded sum.  The whole
        // wavefront walks the segments, whose entries any lane may hold, over its own
        // outputs, once they have arrived.
        __threadfence();
        for (int s = s0;; ++s) {
            const Seg g = segment(s);
            if (g.beg >= p0 + rows) break;
            for (int c = c0 + lane; c < min(c0 + CB * 32, cols); c += kWave) {
                const uint16_t* B = reinterpret_cast<const uint16_t*>(a.B) + g.bo + (int64_t)(n0 + c) * g.rp;
                for (int j = 0; j < g.rp; ++j) {
                    if ((B[j] & 0x7f80u) != 0x7f80u) continue;
                    const float b = bf16_to_f32(B[j]);
                    for (int row = max(g.beg - p0, r0); row < min(min(g.end - p0, rows), r0 + RB * 32); ++row) {
                        if (s_tok[row] < 0) continue;
                        uint16_t& o = p.y[(int64_t)s_tok[row] * p.ldy + n0 + c];
                        o = (uint16_t)f32_to_bf16(bf16_to_f32(o) + b * p.S[(int64_t)(p0 + row) * a.cols + sl * a.r_max + j]);
                    }
                }
            }
        }
    }
}

template <typename F>
__global__ __launch_bounds__(kRingThreads, 1) void k_gemm_ring(GemmFp8Params p) {
    __shared__ uint4 smem[kRingLds / 16];
    const LinearArgs& a = p.a;
    // four row tiles by eight column tiles to each of the eight L2s at a time
    const int v = (int)blockIdx.x / 8;
    const int id = v / 32 * 256 + (int)blockIdx.x % 8 * 32 + v % 32;
    if (id >= p.row_tiles * p.col_tiles) return;
    const int band = id / (4 * p.col_tiles), in = id % (4 * p.col_tiles);
    const int deep = min(4, p.row_tiles - band * 4);
    const int p0 = (band * 4 + in % deep) * kRingRows, ct = in / deep;
    int sl = 0;
    while (sl + 1 < a.n_sl && ct >= p.tile_start[sl + 1]) ++sl;
    const int n0 = (int)(a.slice_off[sl] + (int64_t)(ct - p.tile_start[sl]) * kRingCols);
    const int cols = (int)min((int64_t)kRingCols, a.slice_off[sl + 1] - n0);
    const int rows = min(kRingRows, a.M - p0);
    if (rows > 128) ring_tile<Ring256<F>>(p, smem, sl, p0, rows, n0, cols);
    else ring_tile<Ring128<F>>(p, smem, sl, p0, rows, n0, cols);
}

template <typename F> hipError_t launch_gemm_ring(GemmFp8Params& p, hipStream_t st) {
    const LinearArgs& a = p.a;
    int t = 0;
    for (int s = 0; s < a.n_sl; ++s) {
        p.tile_start[s] = t;
        t += (int)((a.slice_off[s + 1] - a.slice_off[s] + kRingCols - 1) / kRingCols);
    }
    p.tile_start[a.n_sl] = t;
    p.col_tiles = t;
    p.row_tiles = (a.M + kRingRows - 1) / kRingRows;
    const unsigned grid = (unsigned)(((int64_t)p.row_tiles * p.col_tiles + 255) / 256 * 256);
    hipLaunchKernelGGL((k_gemm_ring<F>), dim3(grid), dim3(kRingThreads), 0, st, p);
    return hipGetLastError();
}

}  // namespace mlora
