// The base products of the experts for any number of tokens (SGLang "LoRA + MoE"
// page, the expert GEMMs that the deltas of stage 1.5 and 3.5 are added to):
// the batch's (token, chosen expert) pairs in the experts' order, and one matrix
// product with each expert's weights over its own share of the rows.
#pragma once

#include "common.hpp"
#include "formats.hpp"
#include "kernels.hpp"
#include "row_stage.hpp"

namespace mlora {

// ---------------------------------------------------------------- grouping
// pairs: the pair indices f = m topk + k by ascending expert, equal experts in
// ascending f, pairs of experts outside [0, E) last; offsets [E + 1]: the first
// position of each expert and the end of the last.
//
// A stable counting sort.  A workgroup of 16 wavefronts places kGroupChunk pairs,
// and counts all the others itself: how many of each expert stand before its own
// and how many there are in all.  So one launch does without a word between
// workgroups; reading the ids again costs each workgroup 4 P bytes from the L2
// (65536 pairs, four workgroups: 256 KB each), and one workgroup is all there is
// up to 16384 pairs.
constexpr int kGroupThreads = 1024;
constexpr int kGroupWaves = kGroupThreads / kWave;
constexpr int kGroupChunk = 16 * kGroupThreads;
constexpr int kGroupMaxE = 256;
constexpr int kGroupCached = 4;                    // ids of a wavefront's first passes, kept in registers

__global__ __launch_bounds__(kGroupThreads) void k_moe_group(const int32_t* __restrict__ ids, int P, int E,
                                                             int32_t* __restrict__ pairs,
                                                             int32_t* __restrict__ offsets) {
    __shared__ int s_row[kGroupWaves][kGroupMaxE + 1];   // counts, then next positions, of each wavefront
    __shared__ int s_before[kGroupMaxE + 1], s_after[kGroupMaxE + 1];
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int NB = E + 1;
    const int b0 = (int)blockIdx.x * kGroupChunk, b1 = min(P, b0 + kGroupChunk);
    // a wavefront's part: passes of 64 pairs
    const int passes = (b1 - b0 + kGroupThreads - 1) / kGroupThreads;
    const int c0 = min(b1, b0 + wave * passes * kWave), c1 = min(b1, c0 + passes * kWave);
    int kept[kGroupCached];
#pragma unroll
    for (int i = 0; i < kGroupCached; ++i) kept[i] = ids[min(c0 + i * kWave + lane, P - 1)];
    for (int i = tid; i < kGroupWaves * NB; i += kGroupThreads) s_row[i / NB][i % NB] = 0;
    for (int i = tid; i < NB; i += kGroupThreads) s_before[i] = s_after[i] = 0;
    __syncthreads();
    auto bucket = [&](int v) { return (uint32_t)v < (uint32_t)E ? v : E; };
    for (int i = tid; i < b0; i += kGroupThreads) atomicAdd(&s_before[bucket(ids[i])], 1);
    for (int i = b1 + tid; i < P; i += kGroupThreads) atomicAdd(&s_after[bucket(ids[i])], 1);

    // lanes of the pass whose expert is the same, one ballot per bit
    const int nbits = 32 - __clz(E);
    auto peers = [&](int b, bool act) {
        unsigned long long same = __ballot(act);
        for (int i = 0; i < nbits; ++i) {
            const bool bit = (b >> i) & 1;
            const unsigned long long bb = __ballot(bit);
            same &= bit ? bb : ~bb;
        }
        return same;
    };
    const unsigned long long below = (1ull << lane) - 1ull;
    int* my = s_row[wave];
    auto count = [&](int i, int v) {
        if (c0 + i * kWave + lane < c1) atomicAdd(&my[bucket(v)], 1);
    };
#pragma unroll
    for (int i = 0; i < kGroupCached; ++i) count(i, kept[i]);
    for (int i = kGroupCached; c0 + i * kWave < c1; ++i) count(i, ids[min(c0 + i * kWave + lane, P - 1)]);
    __syncthreads();

    // one thread per expert: its positions in this workgroup's part by wavefront,
    // and its total; then one wavefront turns the totals into first positions
    if (tid < NB) {
        int c[kGroupWaves], run = 0;
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) c[w] = s_row[w][tid];
        const int before = s_before[tid];
#pragma unroll
        for (int w = 0; w < kGroupWaves; ++w) {
            s_row[w][tid] = before + run;
            run += c[w];
        }
        s_after[tid] += before + run;
    }
    __syncthreads();
    if (wave == 0) {
        int run = 0;
        for (int e0 = 0; e0 < NB; e0 += kWave) {
            const int e = e0 + lane;
            const int n = e < NB ? s_after[e] : 0;
            const int inc = wave_incl_scan(n);
            if (e < NB) {
                s_before[e] = run + inc - n;
                if (blockIdx.x == 0) offsets[e] = run + inc - n;
            }
            run += __builtin_amdgcn_readlane(inc, kWave - 1);
        }
    }
    __syncthreads();
    auto place = [&](int i, int v) {
        const int f = c0 + i * kWave + lane;
        const bool act = f < c1;
        const int b = bucket(v);
        const unsigned long long same = peers(b, act);
        const int rank = __popcll(same & below);
        if (act) pairs[s_before[b] + my[b] + rank] = f;
        // every lane has read its position before the first of its equals moves it
        __builtin_amdgcn_wave_barrier();
        if (act && rank == 0) my[b] += __popcll(same);
        __builtin_amdgcn_wave_barrier();
    };
#pragma unroll
    for (int i = 0; i < kGroupCached; ++i)
        if (c0 + i * kWave < c1) place(i, kept[i]);
    for (int i = kGroupCached; c0 + i * kWave < c1; ++i) place(i, ids[min(c0 + i * kWave + lane, P - 1)]);
}

// No pairs: every share is empty.
__global__ void k_moe_group_none(int n, int32_t* offsets) {
    for (int i = threadIdx.x; i < n; i += blockDim.x) offsets[i] = 0;
}

hipError_t launch_moe_group(const int32_t* topk_ids, int P, int E, int32_t* pairs, int32_t* offsets,
                            hipStream_t st) {
    if (P == 0) {
        hipLaunchKernelGGL(k_moe_group_none, dim3(1), dim3(kWave), 0, st, E + 1, offsets);
        return hipGetLastError();
    }
    hipLaunchKernelGGL(k_moe_group, dim3((unsigned)((P + kGroupChunk - 1) / kGroupChunk)), dim3(kGroupThreads), 0,
                       st, topk_ids, P, E, pairs, offsets);
    return hipGetLastError();
}

// ---------------------------------------------------------------- shares and tiles
// 16 zero bytes: what rows of x read past K
__device__ const uint4 k_zeros = {0, 0, 0, 0};

struct Tile {
    int e;              // expert; -1: no such tile
    int pos, rows;      // its sorted positions [pos, pos + rows)
    int rt, rts;        // row tile of the expert, and how many it has
    int64_t in;         // the tile's number among the expert's
    int64_t total;      // all tiles
};

// Tile `id` of the experts' shares cut into row tiles of `height` positions, each
// `cols` column tiles wide (64-bit: a share may have many).  Offsets are clamped
// into the list, so whatever they hold, no position lies outside it.
__device__ __forceinline__ Tile find_tile(const int32_t* offsets, int E, int P, int height, int cols, int64_t id) {
    const int lane = lane_id();
    int o0[4], o1[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int e = c * kWave + lane;
        o0[c] = c * kWave < E ? offsets[min(e, E)] : 0;
        o1[c] = c * kWave < E ? offsets[min(e + 1, E)] : 0;
    }
    Tile t{-1, 0, 0, 0, 0, 0, 0};
    int64_t run = 0;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        if (c * kWave >= E) break;
        const int a = min(max(o0[c], 0), P), n = max(min(o1[c], P) - a, 0);
        const int tiles = (n + height - 1) / height;
        const int inc = wave_incl_scan(tiles);
        const int all = __builtin_amdgcn_readlane(inc, kWave - 1);
        if (t.e < 0 && id < (run + all) * cols) {
            const uint64_t hit = __ballot(id < (run + inc) * cols);
            const int l = __builtin_ctzll(hit);
            const int first = __builtin_amdgcn_readlane(inc - tiles, l);
            t.e = c * kWave + l;
            t.rts = __builtin_amdgcn_readlane(tiles, l);
            t.in = id - (run + first) * cols;
            t.pos = __builtin_amdgcn_readlane(a, l);
            t.rows = __builtin_amdgcn_readlane(n, l);
        }
        run += all;
    }
    t.total = run * cols;
    return t;
}

// ---------------------------------------------------------------- few rows a share
// Work unit = (expert with at least one pair, 16 NR output columns) for all of the
// expert's rows, 16 TB at a time; K over eight wavefronts in blocks of 128 bytes,
// whose partial sums join through LDS.  What bounds it: the touched experts' rows
// of W, read once; they stream past the few rows of x.  Both are read as whole
// 128-byte segments and change lanes through LDS (row_stage.hpp).
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / kWave;

constexpr int few_stage(int TB, int NR) {
    return (NR + 1) * 128 > NR * TB * kWave ? (NR + 1) * 128 : NR * TB * kWave;
}

template <typename F, int TB, int NR>
__global__ __launch_bounds__(kFewThreads, TB * NR == 8 ? 2 : 4) void k_experts_few(ExpertsParams p) {
    constexpr int kStage = few_stage(TB, NR);
    __shared__ uint4 smem[kFewWaves * kStage];
    const int tid = threadIdx.x;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane % 16, lq = lane / 16;
    const Tile tile = find_tile(p.offsets, p.E, p.P, 1 << 24, p.col_tiles, blockIdx.x);
    if (tile.e < 0) return;
    const int n0 = (int)tile.in * 16 * NR, n1 = min(n0 + 16 * NR, p.N);
    const int Kb = p.Kb, KB = (Kb + 127) / 128;
    const int64_t row0 = (int64_t)tile.e * p.N + n0;
    const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(p.W + row0 * Kb, (uint32_t)((n1 - n0) * Kb));
    const __amdgpu_buffer_rsrc_t rx =
        uniform_rsrc(p.x, (uint32_t)((int64_t)(p.x_rows - 1) * p.ldx + Kb));      // below 2 GiB (the launcher's rule)
    uint32_t off_w[2 * NR];
#pragma unroll
    for (int i = 0; i < 2 * NR; ++i)
        off_w[i] = (uint32_t)(min(8 * i + lane / 8, n1 - n0 - 1) * Kb) + (lane % 8) * 16;
    constexpr int U = TB * NR == 8 ? 4 : 4 / NR, UX = TB * NR == 8 ? 2 : TB == 1 ? U : 4 / TB;
    uint4 vw[U][2 * NR], vx[UX][2 * TB];
    uint32_t off_x[2 * TB];
    auto load_w = [&](int q, int kb) {
        const bool in = kb * 128 + lane % 8 * 16 < Kb;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) vw[q][i] = buf_ld16_at<true>(rw, in ? off_w[i] : kBufOff, (uint32_t)kb * 128u);
    };
    auto load_x = [&](int q, int kb) {
        const bool in = kb * 128 + lane % 8 * 16 < Kb;
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i) vx[q][i] = buf_ld16_at<false>(rx, in ? off_x[i] : kBufOff, (uint32_t)kb * 128u);
    };
    uint4* st = smem + wave * kStage;
    uint4* sx = st + NR * 16 * 8;
    const StageAt at;
    // the block of outputs that this wavefront joins and stores: rows 16 jt + lr,
    // columns 16 jr + 4 lq + q
    const int jr = wave / TB, jt = wave % TB;
    const int n = n0 + jr * 16 + lq * 4;                 // N is a multiple of 8
    for (int r0 = 0; r0 < tile.rows; r0 += 16 * TB) {
        const int rows = min(16 * TB, tile.rows - r0);
        const int32_t* list = p.pairs + tile.pos + r0;
        uint32_t f_row[2 * TB];
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i) f_row[i] = (uint32_t)list[min(8 * i + lane / 8, rows - 1)];
        uint32_t f_out = (uint32_t)list[min(jt * 16 + lr, rows - 1)];
#pragma unroll
        for (int q = 0; q < U; ++q) load_w(q, wave + q * kFewWaves);
        // whatever the list holds, no row outside the batch is read or written
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i) {
            const uint32_t f = min(f_row[i], (uint32_t)p.P - 1);
            const uint32_t row = p.x_div > 1 ? f / (uint32_t)p.x_div : f;
            off_x[i] = 8 * i + lane / 8 < rows ? row * (uint32_t)p.ldx + (lane % 8) * 16 : kBufOff;
        }
        f_out = min(f_out, (uint32_t)p.P - 1);
#pragma unroll
        for (int q = 0; q < UX; ++q) load_x(q, wave + q * kFewWaves);
        float xs = 1.f, ws[4] = {1.f, 1.f, 1.f, 1.f};
        if (F::kScaled && wave < NR * TB) {
            xs = p.x_scale[p.x_div > 1 ? f_out / (uint32_t)p.x_div : f_out];
#pragma unroll
            for (int q = 0; q < 4; ++q) ws[q] = p.w_scale[(int64_t)tile.e * p.N + min(n + q, p.N - 1)];
        }
        typename F::Acc16 sum[NR][TB];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[r][t][q] = 0;
        for (int b0 = wave; b0 < KB; b0 += U * kFewWaves) {
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
                    for (int r = 0; r < NR; ++r) sum[r][t] = F::mma16(w[r][0], w[r][1], x0, x1, sum[r][t]);
                    stage_order();
                }
                load_w(q, b0 + (q + U) * kFewWaves);
                load_x(q % UX, b0 + (q + UX) * kFewWaves);
            }
        }
        // join the eight partial sums in a fixed order; four columns of a row a lane
        typedef typename F::Acc16 acc_t;
        acc_t* red = reinterpret_cast<acc_t*>(st);
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int t = 0; t < TB; ++t) red[(r * TB + t) * kWave + lane] = sum[r][t];
        __syncthreads();
        if (wave < NR * TB) {
            acc_t v = reinterpret_cast<const acc_t*>(smem)[wave * kWave + lane];
#pragma unroll
            for (int w = 1; w < kFewWaves; ++w) v += reinterpret_cast<const acc_t*>(smem + w * kStage)[wave * kWave + lane];
            float o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = F::kScaled ? (float)v[q] * (xs * ws[q]) : (float)v[q];
            if (jt * 16 + lr < rows && n < n1)
                *reinterpret_cast<uint2*>(p.y + (int64_t)f_out * p.ldy + n) = make_uint2(pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3]));
        }
        __syncthreads();                 // the next rows use the same LDS
    }
}

// ---------------------------------------------------------------- many rows a share
// Work unit = (up to 256 consecutive positions of one expert's share, 256 output
// columns), four waves, one per SIMD, K in stages of 128 bytes a row.
//
// Both operands go from global memory straight to LDS (no registers, no LDS write
// instructions), whole 128-byte row segments: eight lanes a row, the chunk that a
// lane reads permuted so that chunk c of row r comes to stand at c ^ (r / 2) % 8,
// where operand reads (32 rows, one chunk) meet distinct banks.  Rings of XD
// stages of x and WD of W fill the 160 KB; the loads of a stage are spread evenly
// between the MFMAs of the one before, x first.  The operands of the last K step of
// a stage are in registers one step early, so the one barrier of a stage stands in
// front of that step: behind it the stage's slots are free for the next loads and
// the following stage can be read, and no MFMA waits for either.
//
// A share's last tile has fewer rows: the waves of a unit with up to 192, 128 or 64
// rows take 96 x 128, 128 x 64 and 64 x 64 outputs each instead of 128 x 128, with
// as many fewer MFMAs, and rings as deep as 160 KB allow.
//
// The loads to LDS are written in assembly because the compiler waits for all of
// them at every LDS read; they have no output registers, and the waits that their
// data needs stand in turn().
typedef __attribute__((address_space(3))) char lds_char_t;

__device__ __forceinline__ void dma_global(const char* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
__device__ __forceinline__ void dma_buffer(u32x4_vt r, uint32_t voff, uint32_t soff, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff), "s"(r),
                 "s"(soff)
                 : "memory");
}

constexpr int kShareThreads = 256;
constexpr int kShareRows = 256, kShareCols = 256;
constexpr int kShareLds = 160 * 1024;

template <typename F, int WM, int RB, int CB, int XD, int WD>
__device__ __forceinline__ void tile_product(const ExpertsParams& p, uint4* smem, int e, int pos, int rows, int n0) {
    constexpr int kRows = 32 * RB * WM, WN = 4 / WM;
    static_assert(32 * CB * WN == kShareCols, "four waves share the columns");
    constexpr int kX = kRows * 128, kW = kShareCols * 128;          // bytes of a ring slot
    static_assert(XD >= 2 && WD >= XD && XD * kX + WD * kW <= kShareLds, "rings fit the LDS");
    constexpr int NX = kRows / 32, NW = kShareCols / 32;            // loads of a wave and stage
    constexpr int kLoads = NX + NW;
    constexpr int kWords = F::kWords, MF = RB * CB;
    constexpr int kTotal = MF * (kWords == 1 ? 4 : 2);             // MFMAs of a stage
    constexpr int kPost = kWords == 1 ? MF : kTotal - MF / 2;      // of them behind the barrier
    constexpr int kReads = (RB + CB) * kWords;                     // operand reads of a step
    constexpr int kEarly = (kPost * kLoads + kTotal - 1) / kTotal; // loads issued behind the barrier
    // what may still be on its way when a stage is read: the stages after it
    constexpr int kAhead = (XD - 2) * NX + (WD - 2) * NW;

    const int tid = threadIdx.x;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane % 32, lh = lane / 32;
    const int cols = min(kShareCols, p.N - n0);
    const int Kb = p.Kb, nk = (Kb + 127) / 128;

    // ---- loads: wave w takes the 8-row blocks w + 4 i, lane l row l / 8 of a block
    const int ch = ((lane % 8) ^ (lane / 16 + 4 * (wave & 1))) * 16;   // the lane's bytes of a 128-byte segment
    const int lrow = 8 * wave + lane / 8;
    uint32_t f_in[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) f_in[i] = (uint32_t)p.pairs[pos + min(lrow + 32 * i, rows - 1)];
    uint32_t f_out = (uint32_t)p.pairs[pos + min(tid, rows - 1)];
    const uint64_t wa = (uint64_t)(uintptr_t)(p.W + ((int64_t)e * p.N + n0) * Kb);
    const u32x4_vt rw = {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)wa),
                         (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(wa >> 32)),
                         (uint32_t)__builtin_amdgcn_readfirstlane(cols * Kb), 0x00020000u};
    uint32_t woff[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) woff[i] = (uint32_t)(min(lrow + 32 * i, cols - 1) * Kb + ch);
    const char* xp[NX];
    const char* const zeros = reinterpret_cast<const char*>(&k_zeros);
    const uint32_t dst = (uint32_t)(uintptr_t)(lds_char_t*)smem + wave * 1024;

    // the loads under way: stage sx of x into ring slot lx, stage sw of W into lw
    int lx = 0, lw = 0, inc = 0;
    uint32_t so = 0;
    bool win = true;
    auto begin_x = [&](int st, int slot) {
        lx = slot;
        inc = st + 1 < nk ? 128 : 0;                 // stages past the last read it again
        if (st == nk - 1 && Kb % 128 != 0) {
#pragma unroll
            for (int i = 0; i < NX; ++i) xp[i] = st * 128 + ch < Kb ? xp[i] : zeros;
        }
    };
    auto begin_w = [&](int st, int slot) {
        lw = slot;
        so = (uint32_t)st * 128u;
        win = st * 128 + ch < Kb;                    // past K: zeros, and no memory is touched
    };
    auto load_x = [&](int i) {
        dma_global(xp[i], dst + lx + i * 4096);
        xp[i] += inc;
    };
    auto load_w = [&](int i) { dma_buffer(rw, win ? woff[i] : kBufOff, so, dst + lw + i * 4096); };
    auto load_at = [&](int at) {                     // the loads due after MFMA `at` behind the barrier
#pragma unroll
        for (int j = 0; j < kLoads; ++j) {
            if (j * kTotal / kLoads != at) continue;
            if (j < NX) load_x(j);
            else load_w(j - NX);
        }
    };
    int xs[XD], wsl[WD];                             // ring slots of stages s, s + 1, ..
#pragma unroll
    for (int i = 0; i < XD; ++i) xs[i] = i * kX;
#pragma unroll
    for (int i = 0; i < WD; ++i) wsl[i] = XD * kX + i * kW;

    // prologue: W first, whose addresses need no pair
    begin_w(0, wsl[0]);
#pragma unroll
    for (int i = 0; i < NW; ++i) load_w(i);
#pragma unroll
    for (int i = 0; i < NX; ++i) {
        const uint32_t f = min(f_in[i], (uint32_t)p.P - 1);     // whatever the list holds, a row of the batch
        xp[i] = p.x + (int64_t)(p.x_div > 1 ? f / (uint32_t)p.x_div : f) * p.ldx + ch;
    }
    f_out = min(f_out, (uint32_t)p.P - 1);
    float my_xs = 1.f, my_ws = 1.f;
    if constexpr (F::kScaled) {
        my_xs = p.x_scale[p.x_div > 1 ? f_out / (uint32_t)p.x_div : f_out];
        my_ws = p.w_scale[(int64_t)e * p.N + n0 + min(tid, cols - 1)];
    }
#pragma unroll
    for (int st = 0; st < WD - 1; ++st) {
        if (st < XD - 1) {
            begin_x(st, xs[st]);
#pragma unroll
            for (int i = 0; i < NX; ++i) load_x(i);
        }
        if (st > 0) {
            begin_w(st, wsl[st]);
#pragma unroll
            for (int i = 0; i < NW; ++i) load_w(i);
        }
    }
    begin_x(XD - 1, xs[XD - 1]);
    begin_w(WD - 1, wsl[WD - 1]);
#pragma unroll
    for (int i = 0; i < kPost; ++i) load_at(i);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kAhead + kEarly) : "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");

    // ---- operands: 16-byte chunks of rows lr of the wave's blocks
    const char* const lds = reinterpret_cast<const char*>(smem);
    int get[4];                                      // [step, word]
#pragma unroll
    for (int c = 0; c < 4; ++c) {
        const int chunk = kWords == 1 ? 2 * c + lh : 4 * (c / 2) + 2 * (c % 2) + lh;
        get[c] = lr * 128 + (chunk ^ (lr / 2 % 8)) * 16;
    }
    const int xpart = wave / WN * RB * 4096, wpart = wave % WN * CB * 4096;
    struct Ops {
        uint4 x[RB][kWords], w[CB][kWords];
    };
    auto read1 = [&](Ops& o, int x0, int w0, int t, int j) {
        const int b = j / kWords, h = j % kWords, c = t * kWords + h;
        if (b < CB) o.w[b][h] = *reinterpret_cast<const uint4*>(lds + (w0 + wpart + get[c]) + b * 4096);
        else o.x[b - CB][h] = *reinterpret_cast<const uint4*>(lds + (x0 + xpart + get[c]) + (b - CB) * 4096);
    };
    typename F::Acc32 acc[RB][CB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int q = 0; q < 16; ++q) acc[rb][cb][q] = 0;
    auto mfma1 = [&](const Ops& o, int i) {
        const int rb = i / CB, cb = i % CB;
        acc[rb][cb] = F::mma32_step(o.w[cb], o.x[rb], acc[rb][cb]);
    };
    Ops oa, ob;
#pragma unroll
    for (int j = 0; j < kReads; ++j) read1(oa, xs[0], wsl[0], 0, j);

    // The one barrier of stage s: the operands of its last step are in registers
    // (lgkmcnt), so its ring slots are free behind it; the stages up to s + 1 have
    // arrived, in every wave.
    auto turn = [&](int s) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        begin_x(s + XD, xs[0]);
        begin_w(s + WD, wsl[0]);
        __builtin_amdgcn_sched_barrier(0);
    };
    // MFMAs [i0, i1) of a step, number `at` and on behind the barrier, with `reads`
    // (a step's operands into o, spread evenly) and the loads that are due
    auto run = [&](const Ops& cur, int i0, int i1, int at, Ops* next, int x0, int w0, int t) {
#pragma unroll
        for (int i = i0; i < i1; ++i) {
            mfma1(cur, i);
            if (next)
#pragma unroll
                for (int j = 0; j < kReads; ++j)
                    if (i0 + j * (i1 - i0) / kReads == i) read1(*next, x0, w0, t, j);
            load_at(at + i - i0);
            __builtin_amdgcn_sched_barrier(0);
        }
    };
    for (int s = 0; s < nk; ++s) {
        if constexpr (kWords == 1) {
            run(oa, 0, MF, kPost, &ob, xs[0], wsl[0], 1);
            run(ob, 0, MF, kPost + MF, &oa, xs[0], wsl[0], 2);
            run(oa, 0, MF, kPost + 2 * MF, &ob, xs[0], wsl[0], 3);
            turn(s);
            run(ob, 0, MF, 0, &oa, xs[1], wsl[1], 0);
        } else {
            run(oa, 0, MF / 2, kPost, &ob, xs[0], wsl[0], 1);
            turn(s);
            run(oa, MF / 2, MF, 0, nullptr, 0, 0, 0);
            run(ob, 0, MF, MF - MF / 2, &oa, xs[1], wsl[1], 0);
        }
        const int x0 = xs[0], w0 = wsl[0];
#pragma unroll
        for (int i = 0; i + 1 < XD; ++i) xs[i] = xs[i + 1];
        xs[XD - 1] = x0;
#pragma unroll
        for (int i = 0; i + 1 < WD; ++i) wsl[i] = wsl[i + 1];
        wsl[WD - 1] = w0;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();                                 // the rings are free

    // ---- scales, one rounding, whole row pieces through LDS
    constexpr int kStaged = kShareRows * kShareCols * 2;
    int* const s_f = reinterpret_cast<int*>(reinterpret_cast<char*>(smem) + kStaged);
    float* const s_xs = reinterpret_cast<float*>(s_f + kShareRows);
    float* const s_ws = s_xs + kShareRows;
    s_f[tid] = tid < rows ? (int)f_out : -1;
    s_xs[tid] = my_xs;
    s_ws[tid] = my_ws;
    __syncthreads();
    const int r0 = wave / WN * RB * 32, c0 = wave % WN * CB * 32;
    constexpr int kCh = CB * 4;                      // 16-byte chunks of a wave's row
    auto swz = [](int row) { return kCh == 16 ? row % 16 : row / 2 % 8; };
    uint16_t* const so16 = reinterpret_cast<uint16_t*>(smem) + wave * RB * 32 * CB * 32;
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
        const int row = rb * 32 + lr;
        const float rs = F::kScaled ? s_xs[r0 + row] : 1.f;
#pragma unroll
        for (int cb = 0; cb < CB; ++cb)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                float v[4];
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] = (float)acc[rb][cb][4 * g + q];
                if constexpr (F::kScaled) {
                    const float4 ws = *reinterpret_cast<const float4*>(s_ws + c0 + cb * 32 + 8 * g + 4 * lh);
                    v[0] *= rs * ws.x;
                    v[1] *= rs * ws.y;
                    v[2] *= rs * ws.z;
                    v[3] *= rs * ws.w;
                }
                *reinterpret_cast<uint2*>(so16 + row * CB * 32 + ((cb * 4 + g) ^ swz(row)) * 8 + lh * 4) =
                    make_uint2(pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3]));
            }
    }
    stage_order();                                   // a wave reads back what it wrote itself
#pragma unroll
    for (int j = 0; j < RB * 32 * kCh / kWave; ++j) {
        const int row = j * (kWave / kCh) + lane / kCh, c = lane % kCh;
        const uint4 v = *reinterpret_cast<const uint4*>(so16 + row * CB * 32 + (c ^ swz(row)) * 8);
        const int f = s_f[r0 + row], n = c0 + c * 8;
        if (f >= 0 && n < cols) *reinterpret_cast<uint4*>(p.y + (int64_t)f * p.ldy + n0 + n) = v;
    }
}

template <typename F>
__global__ __launch_bounds__(kShareThreads, 1) void k_experts_tile(ExpertsParams p) {
    __shared__ uint4 smem[kShareLds / 16];
    // 32 tiles in a row (four row tiles by eight column tiles of an expert) to each
    // of the eight L2s, every eighth workgroup on one of them
    const int v = (int)blockIdx.x / 8;
    const int64_t id = (int64_t)(v / 32) * 256 + (int)blockIdx.x % 8 * 32 + v % 32;
    const Tile t = find_tile(p.offsets, p.E, p.P, kShareRows, p.col_tiles, id);
    if (t.e < 0) return;
    const int band = (int)(t.in / (4 * p.col_tiles)), in = (int)(t.in % (4 * p.col_tiles));
    const int deep = min(4, t.rts - band * 4);
    const int rt = band * 4 + in % deep, n0 = in / deep * kShareCols;
    const int pos = t.pos + rt * kShareRows, rows = min(kShareRows, t.rows - rt * kShareRows);
    if (rows > 192) tile_product<F, 2, 4, 4, 2, 3>(p, smem, t.e, pos, rows, n0);
    else if (rows > 128) tile_product<F, 2, 3, 4, 2, 3>(p, smem, t.e, pos, rows, n0);
    else if (rows > 64) tile_product<F, 1, 4, 2, 3, 3>(p, smem, t.e, pos, rows, n0);
    else tile_product<F, 1, 2, 2, 4, 4>(p, smem, t.e, pos, rows, n0);
}

// ---------------------------------------------------------------- launch
template <typename F, int TB, int NR> hipError_t launch_few(ExpertsParams& p, hipStream_t st) {
    p.col_tiles = (p.N + 16 * NR - 1) / (16 * NR);
    const int shares = p.E < p.P ? p.E : p.P;
    hipLaunchKernelGGL((k_experts_few<F, TB, NR>), dim3((unsigned)((int64_t)shares * p.col_tiles)), dim3(kFewThreads), 0,
                       st, p);
    return hipGetLastError();
}

template <typename F> hipError_t launch_experts_as(ExpertsParams& p, hipStream_t st) {
    const int shares = p.E < p.P ? p.E : p.P;
    const int64_t extent = (int64_t)(p.x_rows - 1) * p.ldx + p.Kb;
    if (p.P <= 16 * shares && extent < INT32_MAX) {
        if (p.P <= 8 * shares) return launch_few<F, 1, 1>(p, st);
        return launch_few<F, 2, 1>(p, st);
    }
    p.col_tiles = (p.N + kShareCols - 1) / kShareCols;
    const int64_t tiles = ((int64_t)p.P / kShareRows + shares) * p.col_tiles;
    hipLaunchKernelGGL((k_experts_tile<F>), dim3((unsigned)((tiles + 255) / 256 * 256)), dim3(kShareThreads), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_experts(int wdtype, ExpertsParams& p, hipStream_t st) {
    if (wdtype == LORA_BF16) return launch_experts_as<FmtBf16>(p, st);
    if (wdtype == LORA_E4M3) return launch_experts_as<FmtE4m3>(p, st);
    return launch_experts_as<FmtInt8>(p, st);
}

}  // namespace mlora
