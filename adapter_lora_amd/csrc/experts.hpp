// The base products of the experts for any number of tokens (SGLang "LoRA + MoE"
// page, the expert GEMMs that the deltas of stage 1.5 and 3.5 are added to):
// the batch's (token, chosen expert) pairs in the experts' order, and one matrix
// product with each expert's weights over its own share of the rows.
#pragma once

#include "common.hpp"
#include "formats.hpp"
#include "kernels.hpp"
#include "ring_product.hpp"
#include "row_stage.hpp"

namespace mlora {

// ---------------------------------------------------------------- grouping
// pairs: the pair indices f = m topk + k by ascending expert, equal experts in
// ascending f, pairs of experts outside [0, E) last; offsets [E + 1]: the first
// position of each expert and the end of the last.
//
// A stable counting sort.  A workgroup of 16 wavefronts places `chunk` pairs, and
// counts all the others itself: how many of each expert stand before its own and how
// many there are in all.  So one launch does without a word between workgroups;
// reading the ids again costs each workgroup 4 P bytes from the L2.
constexpr int kGroupThreads = 1024;
constexpr int kGroupWaves = kGroupThreads / kWave;
constexpr int kGroupMaxE = 256;
constexpr int kGroupCached = 4;                    // ids of a wavefront's first passes, kept in registers

__global__ __launch_bounds__(kGroupThreads) void k_moe_group(const int32_t* __restrict__ ids, int P, int E, int chunk,
                                                             int32_t* __restrict__ pairs,
                                                             int32_t* __restrict__ offsets) {
    __shared__ int s_row[kGroupWaves][kGroupMaxE + 1];   // counts, then next positions, of each wavefront
    __shared__ int s_before[kGroupMaxE + 1], s_after[kGroupMaxE + 1];
    const int tid = threadIdx.x, lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int NB = E + 1;
    const int b0 = (int)blockIdx.x * chunk, b1 = min(P, b0 + chunk);
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
    auto count_others = [&](int* sums, int lo, int hi) {       // P < 2^24 + 1
        for (int i = lo + tid; i < hi; i += 4 * kGroupThreads) {
            int v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = ids[min(i + j * kGroupThreads, P - 1)];
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (i + j * kGroupThreads < hi) atomicAdd(&sums[bucket(v[j])], 1);
        }
    };
    count_others(s_before, 0, b0);
    count_others(s_after, b1, P);

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
        stage_order();
        if (act && rank == 0) my[b] += __popcll(same);
        stage_order();
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
    // As many workgroups as place their pairs in one pass, until the others' ids are what
    // takes the time (1 / 4 / 16 passes: 9186 pairs of 64 experts 4.4 / 5.6 / 9.1 us, 32768 of
    // 128 6.9 / 8.1 / 17.8, 65536 of 256 10.6 / 11.8 / 22.2, 524288 of 64 99 / 88 / 97, 2^23
    // 23800 / 6290 / 1760; one token 2.6).
    const int chunk = (P <= 65536 ? 1 : 16) * kGroupThreads;
    hipLaunchKernelGGL(k_moe_group, dim3((unsigned)((P + chunk - 1) / chunk)), dim3(kGroupThreads), 0, st, topk_ids, P, E,
                       chunk, pairs, offsets);
    return hipGetLastError();
}

// ---------------------------------------------------------------- shares and tiles
// The x row of pair f < 2^24: f, or f / topk by its reciprocal (2^32 / topk rounded
// up, exact for these f).
__device__ __forceinline__ uint32_t pair_row(const ExpertsParams& p, uint32_t f) {
    return p.x_inv ? __umulhi(f, p.x_inv) : f;
}

// The experts' shares, expert 64 c + l in lane l: first position and pairs.  Offsets
// are clamped into the list, so whatever they hold, no position lies outside it.
template <int NC> struct Shares {
    int pos[NC], n[NC];
    __device__ __forceinline__ Shares(const int32_t* offsets, int E, int P) {
        const int lane = lane_id();
        int o0[NC], o1[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            o0[c] = offsets[min(c * kWave + lane, E)];
            o1[c] = offsets[min(c * kWave + lane + 1, E)];
        }
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            pos[c] = min(max(o0[c], 0), P);
            n[c] = max(min(o1[c], P) - pos[c], 0);
        }
    }
};

// Rows [pos, pos + rows) of expert e's share, column tile ct; e = -1: none.  alone: they
// are the whole share.
struct Tile {
    int e = -1, pos = 0, rows = 0, ct = 0;
    bool alone = false;
};

// n / cols by the reciprocal 2^32 / cols rounded up, which is one too many at most.
__device__ __forceinline__ int div_cols(const ExpertsParams& p, int n) {
    const int q = (int)__umulhi((uint32_t)n, p.cols_inv);
    return p.col_tiles == 1 ? n : q - (n < q * p.col_tiles);
}

// Position of set bit `nth` of a mask (wave-uniform; nth below its bits).
__device__ __forceinline__ int nth_bit(uint64_t mask, int nth) {
    const int lane = lane_id();
    const bool hit = (mask >> lane & 1) && __popcll(mask & ((1ull << lane) - 1ull)) == nth;
    return __builtin_ctzll(__ballot(hit));
}

// Part `nth` of the shares cut into parts of up to ROWS positions.
template <int NC, int ROWS> __device__ __forceinline__ Tile find_part(const ExpertsParams& p, int nth) {
    const Shares<NC> sh(p.offsets, p.E, p.P);
    Tile t;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int parts = (sh.n[c] + ROWS - 1) / ROWS, inc = wave_incl_scan(parts);
        const uint64_t past = __ballot(nth < inc);
        if (t.e < 0 && past != 0ull) {
            const int l = __builtin_ctzll(past);
            const int before = (nth - __builtin_amdgcn_readlane(inc - parts, l)) * ROWS;
            t.e = c * kWave + l;
            t.pos = __builtin_amdgcn_readlane(sh.pos[c], l) + before;
            t.rows = min(ROWS, __builtin_amdgcn_readlane(sh.n[c], l) - before);
        }
        nth -= __builtin_amdgcn_readlane(inc, kWave - 1);
    }
    return t;
}

// Tile `id` of the shares cut into tiles of 256 rows.  Order: expert by expert, whose
// tiles of W come back while they are near, the tiles of more than 192 rows before
// the share's last, in bands of four row tiles.  The experts of the last kTailTiles
// tiles together by size, so that the long ones do not begin last.
constexpr int kTailTiles = 512;

template <int NC> __device__ __forceinline__ Tile find_tile(const ExpertsParams& p, int id) {
    const Shares<NC> sh(p.offsets, p.E, p.P);
    const int lane = lane_id(), cols = p.col_tiles;
    int size[NC], full[NC], before[NC];      // class of the last tile (0: none), tiles above 192, earlier experts' tiles
    int total = 0;
    Tile t;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const int left = sh.n[c] % kRingRows;
        size[c] = left == 0 || left > 192 ? 0 : (left + 63) / 64;
        full[c] = sh.n[c] / kRingRows + (left > 192);
        const int tiles = full[c] + (size[c] > 0), inc = wave_incl_scan(tiles);
        before[c] = total + inc - tiles;
        total += __builtin_amdgcn_readlane(inc, kWave - 1);
    }
    if (id >= total * cols) return t;
    // the expert that holds the tile; the first whose tiles all belong to the tail
    const int at = div_cols(p, id), tail = total - div_cols(p, kTailTiles);
    int w0 = 0, w1 = NC * kWave, skip = 0, t0 = NC * kWave, tskip = 0;
    bool found = false;
#pragma unroll
    for (int c = NC - 1; c >= 0; --c) {
        const uint64_t late = __ballot(before[c] >= tail), here = __ballot(before[c] <= at);
        if (late != 0ull) {
            const int l = __builtin_ctzll(late);
            t0 = c * kWave + l;
            tskip = __builtin_amdgcn_readlane(before[c], l);
        }
        if (!found && here != 0ull) {
            const int l = 63 - __builtin_clzll(here);
            found = true;
            w0 = c * kWave + l;
            w1 = w0 + 1;
            skip = __builtin_amdgcn_readlane(before[c], l);
        }
    }
    if (w0 >= t0) w0 = t0, w1 = NC * kWave, skip = tskip;
    id -= skip * cols;
    // among experts w0 .. w1: the large tiles, then the others by size
    int run = 0, rt = 0;
#pragma unroll
    for (int c = 0; c < NC; ++c) {
        const bool in = c * kWave + lane >= w0 && c * kWave + lane < w1;
        const int tiles = in ? full[c] : 0, inc = wave_incl_scan(tiles);
        const uint64_t hit = __ballot(id < (run + inc) * cols);
        if (t.e < 0 && hit != 0ull) {
            const int l = __builtin_ctzll(hit);
            const int rts = __builtin_amdgcn_readlane(tiles, l);
            const int in_e = id - (run + __builtin_amdgcn_readlane(inc - tiles, l)) * cols;
            const int band = div_cols(p, in_e) / 4, k = in_e - band * 4 * cols, deep = min(4, rts - band * 4);
            t.e = c * kWave + l;
            t.ct = deep == 4 ? k / 4 : deep == 3 ? (int)__umulhi((uint32_t)k, 0x55555556u) : deep == 2 ? k / 2 : k;
            rt = band * 4 + k - t.ct * deep;
            t.pos = __builtin_amdgcn_readlane(sh.pos[c], l);
            t.rows = __builtin_amdgcn_readlane(sh.n[c], l);
        }
        run += __builtin_amdgcn_readlane(inc, kWave - 1);
    }
    id -= run * cols;
    if (t.e < 0) {
        int nth = div_cols(p, id);
        t.ct = id - nth * cols;
#pragma unroll
        for (int k = 3; k > 0; --k) {
#pragma unroll
            for (int c = 0; c < NC; ++c) {
                const bool in = c * kWave + lane >= w0 && c * kWave + lane < w1;
                const uint64_t some = __ballot(in && size[c] == k);
                const int all = __popcll(some);
                if (t.e < 0 && nth < all) {
                    const int l = nth_bit(some, nth);
                    t.e = c * kWave + l;
                    t.pos = __builtin_amdgcn_readlane(sh.pos[c], l);
                    t.rows = __builtin_amdgcn_readlane(sh.n[c], l);
                    rt = t.rows / kRingRows;
                }
                nth -= all;
            }
        }
    }
    t.alone = t.rows <= kRingRows;
    t.pos += rt * kRingRows;
    t.rows = min(kRingRows, t.rows - rt * kRingRows);
    return t;
}

// ---------------------------------------------------------------- few rows a share
// Work unit = (up to 64 positions of an expert's share, 32 output columns), 16 TB of them
// at a time; K over eight wavefronts in blocks of 128 bytes, whose partial sums join
// through LDS.  What bounds it: the touched experts' rows
// of W, read once; they stream past the few rows of x.  Both are read as whole
// 128-byte segments and change lanes through LDS (row_stage.hpp).
//
// Measured: 8 rows each of 8 experts of 28672 x 4096 in bf16 273 us, 1.88 GB at 6.9 TB/s (a
// large copy, read and written, 5.1); one token to 4 of 40 experts of 2848 x 2064 in int8
// 9.7 us, 23.5 MB: with W in the caches 5.6, of which the share is found in 0.5, the
// loads are issued in 1.5, multiplied in 1.4, joined and stored in 0.3.  64 positions a
// unit, for routing that is far from even: 512 rows over 64 x (2816, 2048) in bf16 118 us
// evenly, with half of them on one expert 135 (141 in one unit), with all 50 (144); in
// units of 32 134 and 49.
constexpr int kFewThreads = 512;
constexpr int kFewWaves = kFewThreads / kWave;
constexpr int kFewCols = 32, kFewRows = 64;

template <typename F, int TB, bool NT>
__global__ __launch_bounds__(kFewThreads, 4) void k_experts_few(ExpertsParams p) {
    constexpr int NR = kFewCols / 16;
    constexpr int kStage = (NR + 1) * 128;           // uint4 of a wavefront: rows of W and of x, later its sums
    static_assert(NR * TB * kWave <= kStage, "sums fit the stage");
    __shared__ uint4 smem[kFewWaves * kStage];
    const int tid = threadIdx.x;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane % 16, lq = lane / 16;
    const int nth = div_cols(p, (int)blockIdx.x);
    const Tile tile = p.E <= kWave ? find_part<1, kFewRows>(p, nth) : find_part<kGroupMaxE / kWave, kFewRows>(p, nth);
    if (tile.e < 0) return;
    const int n0 = ((int)blockIdx.x - nth * p.col_tiles) * 16 * NR, n1 = min(n0 + 16 * NR, p.N);
    const int Kb = p.Kb, KB = (Kb + 127) / 128;
    const int64_t row0 = (int64_t)tile.e * p.N + n0;
    const __amdgpu_buffer_rsrc_t rw = uniform_rsrc(p.W + row0 * Kb, (uint32_t)((n1 - n0) * Kb));
    const __amdgpu_buffer_rsrc_t rx =
        uniform_rsrc(p.x, (uint32_t)((int64_t)(p.x_rows - 1) * p.ldx + Kb));      // below 2 GiB (the launcher's rule)
    uint32_t off_w[2 * NR];
#pragma unroll
    for (int i = 0; i < 2 * NR; ++i)
        off_w[i] = (uint32_t)(min(8 * i + lane / 8, n1 - n0 - 1) * Kb) + (lane % 8) * 16;
    // blocks in flight: W comes from HBM, x from L2.  A second block of x where 128
    // registers hold it (spilled, 8 x (4096, 14336) in e4m3 took 93 and 102 us, with one
    // block 75 and 77).
    constexpr int U = 2, UX = TB == 1 && F::kWords == 1 ? 2 : 1;
    uint4 vw[U][2 * NR], vx[UX][2 * TB];
    uint32_t off_x[2 * TB];
    const int steps = (KB + kFewWaves - 1) / kFewWaves;
    const int first = k_phase(n0 / 512, steps);
    auto block = [&](int s) {
        const int at = s + first;
        return s < steps ? (at < steps ? at : at - steps) * kFewWaves + wave : KB;
    };
    auto load_w = [&](int q, int s) {
        const int kb = block(s);
        const bool in = kb * 128 + lane % 8 * 16 < Kb;
#pragma unroll
        for (int i = 0; i < 2 * NR; ++i) vw[q][i] = buf_ld16_at<NT>(rw, in ? off_w[i] : kBufOff, (uint32_t)kb * 128u);
    };
    auto load_x = [&](int q, int s) {
        const int kb = block(s);
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
        for (int q = 0; q < U; ++q) load_w(q, q);
        // whatever the list holds, no row outside the batch is read or written
#pragma unroll
        for (int i = 0; i < 2 * TB; ++i) {
            const uint32_t f = min(f_row[i], (uint32_t)p.P - 1);
            off_x[i] = 8 * i + lane / 8 < rows ? pair_row(p, f) * (uint32_t)p.ldx + (lane % 8) * 16 : kBufOff;
        }
        f_out = min(f_out, (uint32_t)p.P - 1);
#pragma unroll
        for (int q = 0; q < UX; ++q) load_x(q, q);
        // the scales come with the first blocks where the registers hold them (with 32 rows
        // int8 spilled)
        float xs = 1.f, ws[4] = {1.f, 1.f, 1.f, 1.f};
        auto scales = [&]() {
            xs = p.x_scale[pair_row(p, f_out)];
#pragma unroll
            for (int q = 0; q < 4; ++q) ws[q] = p.w_scale[(int64_t)tile.e * p.N + min(n + q, p.N - 1)];
        };
        if constexpr (F::kScaled && TB == 1) scales();
        typename F::Acc16 sum[NR][TB];
#pragma unroll
        for (int r = 0; r < NR; ++r)
#pragma unroll
            for (int t = 0; t < TB; ++t)
#pragma unroll
                for (int q = 0; q < 4; ++q) sum[r][t][q] = 0;
        for (int b0 = 0; b0 < steps; b0 += U) {
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
                load_w(q, b0 + q + U);
                load_x(q % UX, b0 + q + UX);
            }
        }
        if constexpr (F::kScaled && TB > 1)
            if (wave < NR * TB) scales();
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
// Work unit = (up to 256 consecutive positions of one expert's share, 256 or 128 output
// columns), four waves, one per SIMD, K in stages of 128 bytes a row.
//
// The main loop and the forms for tiles with fewer rows (a share's last ones) stand
// in ring_product.hpp.
//
// What bounds it: with up to about 100 rows a share the stream of W (64 rows each of 8
// experts of 28672 x 4096 in bf16 333 us, 1.88 GB at 5.6 TB/s), past that the matrix
// unit (1024 rows each of 8 experts of 4096 x 14336 in bf16 751 us, 1.28 PFLOP/s) and the
// rounds: 240 to 1148 rows, the same number in all, leave 640 tiles of all sizes
// for two and a half rounds, 928 us.  Not faster: tiles of two workgroups a compute
// unit (3 % below 64 rows, 13 to 34 % slower at 100), the last rows of shares in tiles
// of half the columns (6 % at best, mostly slower), all tiles in the order of their size
// (4096 rows to 8 experts of 28672 x 4096 in e4m3 555 us against 471: W comes twice from
// memory).

template <typename R, bool NT = false>
__device__ __forceinline__ void share_tile(const ExpertsParams& p, uint4* smem, const Tile& t) {
    const int e = t.e, pos = t.pos, rows = t.rows, n0 = t.ct * R::kCols;
    typedef typename R::F F;
    constexpr int RB = R::RB, CB = R::CB, NX = R::NX;
    const int tid = threadIdx.x;
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int lr = lane % 32, lh = lane / 32;
    const int cols = min(R::kCols, p.N - n0);
    uint32_t f_in[NX];
#pragma unroll
    for (int i = 0; i < NX; ++i) f_in[i] = (uint32_t)p.pairs[pos + min(R::load_row(wave, i), rows - 1)];
    uint32_t f_out = (uint32_t)p.pairs[pos + min(tid, rows - 1)];
    float my_xs = 1.f, my_ws = 1.f;
    auto x_rows = [&](const char* (&xp)[NX]) {
        // whatever the list holds, a row of the batch
#pragma unroll
        for (int i = 0; i < NX; ++i)
            xp[i] = p.x + (int64_t)pair_row(p, min(f_in[i], (uint32_t)p.P - 1)) * p.ldx + R::load_byte(wave);
        f_out = min(f_out, (uint32_t)p.P - 1);
        if constexpr (F::kScaled) {
            my_xs = p.x_scale[pair_row(p, f_out)];
            my_ws = p.w_scale[(int64_t)e * p.N + n0 + min(tid, cols - 1)];
        }
    };
    typename R::Acc acc[RB][CB];
    ring_product<R, NT>(smem, p.W + ((int64_t)e * p.N + n0) * p.Kb, p.Kb, cols, p.Kb, k_phase(n0 / 1024, (p.Kb + 127) / 128),
                    x_rows, acc);

    // ---- scales, one rounding
    int* const s_f = reinterpret_cast<int*>(smem);
    float* const s_xs = reinterpret_cast<float*>(s_f + kRingRows);
    float* const s_ws = s_xs + kRingRows;
    s_f[tid] = tid < rows ? (int)f_out : -1;
    s_xs[tid] = my_xs;
    s_ws[tid] = my_ws;
    __syncthreads();
    const int r0 = R::row0(wave), c0 = R::col0(wave);
    uint16_t* dst[RB][2];
    bool ok[RB][2];
    float rs[RB];
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int f = s_f[r0 + rb * 32 + 16 * h + lane % 16];
            ok[rb][h] = f >= 0;
            dst[rb][h] = p.y + (int64_t)max(f, 0) * p.ldy + n0 + c0 + 8 * store_chunk();
        }
        rs[rb] = s_xs[r0 + rb * 32 + lr];
    }
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
        const bool in = c0 + cb * 32 + 8 * store_chunk() < cols;       // N is a multiple of 8
        float4 ws[4];
        if constexpr (F::kScaled)
#pragma unroll
            for (int g = 0; g < 4; ++g) ws[g] = *reinterpret_cast<const float4*>(s_ws + c0 + cb * 32 + 8 * g + 4 * lh);
#pragma unroll
        for (int rb = 0; rb < RB; ++rb) {
            f32x16_t v;
#pragma unroll
            for (int q = 0; q < 16; ++q) v[q] = (float)acc[rb][cb][q];
            if constexpr (F::kScaled)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    v[4 * g] *= rs[rb] * ws[g].x;
                    v[4 * g + 1] *= rs[rb] * ws[g].y;
                    v[4 * g + 2] *= rs[rb] * ws[g].z;
                    v[4 * g + 3] *= rs[rb] * ws[g].w;
                }
            store_block(v, {dst[rb][0] + cb * 32, dst[rb][1] + cb * 32}, {ok[rb][0] && in, ok[rb][1] && in});
        }
    }
}

template <typename F, bool HALF>
__global__ __launch_bounds__(kRingThreads, 1) void k_experts_tile(ExpertsParams p) {
    __shared__ uint4 smem[kRingLds / 16];
    // 32 tiles in a row (four row tiles by eight column tiles of an expert) to each
    // of the eight L2s, every eighth workgroup on one of them
    const int v = (int)blockIdx.x / 8;
    const int id = v / 32 * 256 + (int)blockIdx.x % 8 * 32 + v % 32;
    const Tile t = p.E <= kWave ? find_tile<1>(p, id) : find_tile<kGroupMaxE / kWave>(p, id);
    if (t.e < 0) return;
    // With up to 192 rows W bounds the tile, and is not kept if no other reads it.
    const bool once = p.whole_lines && t.alone;
    if constexpr (HALF) {
        if (t.rows > 192) share_tile<Half256<F>>(p, smem, t);
        else if (t.rows > 128) once ? share_tile<Half192<F>, true>(p, smem, t) : share_tile<Half192<F>>(p, smem, t);
        else if (t.rows > 64) once ? share_tile<Half128<F>, true>(p, smem, t) : share_tile<Half128<F>>(p, smem, t);
        else once ? share_tile<Half64<F>, true>(p, smem, t) : share_tile<Half64<F>>(p, smem, t);
    } else {
        if (t.rows > 192) share_tile<Ring256<F>>(p, smem, t);
        else if (t.rows > 128) once ? share_tile<Ring192<F>, true>(p, smem, t) : share_tile<Ring192<F>>(p, smem, t);
        else if (t.rows > 64) once ? share_tile<Ring128<F>, true>(p, smem, t) : share_tile<Ring128<F>>(p, smem, t);
        else once ? share_tile<Ring64<F>, true>(p, smem, t) : share_tile<Ring64<F>>(p, smem, t);
    }
}

// ---------------------------------------------------------------- launch
static void set_cols(ExpertsParams& p, int width) {
    p.col_tiles = (p.N + width - 1) / width;
    p.cols_inv = (uint32_t)(((1ull << 32) + p.col_tiles - 1) / p.col_tiles);   // (unused for one)
}

template <typename F, int TB> hipError_t launch_few(ExpertsParams& p, hipStream_t st) {
    set_cols(p, kFewCols);
    const int parts = (p.E < p.P ? p.E : p.P) + p.P / kFewRows;
    const dim3 grid((unsigned)(parts * p.col_tiles)), block(kFewThreads);
    if (p.whole_lines) hipLaunchKernelGGL((k_experts_few<F, TB, true>), grid, block, 0, st, p);
    else hipLaunchKernelGGL((k_experts_few<F, TB, false>), grid, block, 0, st, p);
    return hipGetLastError();
}

template <typename F> hipError_t launch_experts_as(ExpertsParams& p, hipStream_t st) {
    const int shares = p.E < p.P ? p.E : p.P;
    // W is read past the caches where its rows are whole lines: 8 x (28672, 4096) in bf16,
    // 8 rows 299 -> 273 us here, 64 rows 353 -> 333 in tiles.  Of lines that two rows
    // share the second read then comes from afar too: 40 x (2848, 2064), 8 rows in tiles
    // 98 -> 127 us.
    p.whole_lines = p.Kb % 128 == 0 && (uintptr_t)p.W % 128 == 0;
    const int64_t extent = (int64_t)(p.x_rows - 1) * p.ldx + p.Kb;
    const int64_t cols = (p.N + kRingCols - 1) / kRingCols, units = shares * cols;
    // The streaming form as long as 16 rows at a time take in most shares (it reads a
    // share's W again for every further 16).  With short rows of W its many workgroups
    // wait more than they read, and the tiles are ahead once most experts have rows.
    // Up to twice the rows in its form of 32 where the tiles would leave compute units
    // without one, or come in one short round.  Measured in graphs over several weights,
    // shares of 0.5 to 1.5 times the rows named, 16 rows at a time / 32 / tiles; us:
    //   8 x (28672, 4096), 8 rows: bf16 273 / 280 / 304, int8 146 / 155 / 156; 16 rows: - / 300 /
    //     310, - / 172 / 162
    //   8 x (4096, 14336), 8 rows: 143 / 145 / 138, 72 / 74 / 72; 16 rows: - / 153 / 140, - / 78 / 73
    //   8 x (4096, 4096), 8 rows: 42 / 44 / 58, 24 / 26 / 30; 16 rows: - / 45 / 57, - / 26 / 31
    //   64 x (2816, 2048), 8 rows: 117 / 123 / 122, 72 / 78 / 66
    //   64 x (2048, 1408), 8 rows: 71 / 77 / 60, 46 / 50 / 35
    //   40 x (2848, 2064), 8 rows: 96 / 103 / 98, 62 / 68 / 56; 6 of the 40 with 2 rows: 22 / 23 / 24,
    //     15 / 17 / 15; 2 of them: 10 / 10 / 21, 8 / 9 / 13
    // (e4m3 within 4 % of int8.)
    const bool fits = extent < INT32_MAX && (shares + p.P / kFewRows) * (int64_t)((p.N + kFewCols - 1) / kFewCols) < (1 << 23);
    if (fits && p.P <= 8 * shares && (p.Kb >= 4096 || p.P < 2 * p.E || units < 256)) return launch_few<F, 1>(p, st);
    if (fits && p.P <= 16 * shares && (units < 128 || (units < 256 && p.Kb <= 8192))) return launch_few<F, 2>(p, st);
    // Tiles of half the columns while a round of whole ones would leave compute units
    // without one.  Whole / half: 8 x (4096, 14336), 64 rows bf16 258 / 175 us, int8 132 / 89;
    // 160 rows 326 / 226, 174 / 116; 256 rows (256 tiles) 349 / 383, 188 / 196; 64 x (2816,
    // 2048), 64 rows 169 / 172, 84 / 93.
    const bool half = ((int64_t)p.P / kRingRows + shares) * cols < 256;
    set_cols(p, half ? kRingCols / 2 : kRingCols);
    const int64_t tiles = ((int64_t)p.P / kRingRows + shares) * p.col_tiles;
    const dim3 grid((unsigned)((tiles + 255) / 256 * 256));
    if (half) hipLaunchKernelGGL((k_experts_tile<F, true>), grid, dim3(kRingThreads), 0, st, p);
    else hipLaunchKernelGGL((k_experts_tile<F, false>), grid, dim3(kRingThreads), 0, st, p);
    return hipGetLastError();
}

hipError_t launch_experts(int wdtype, ExpertsParams& p, hipStream_t st) {
    if (wdtype == LORA_BF16) return launch_experts_as<FmtBf16>(p, st);
    if (wdtype == LORA_E4M3) return launch_experts_as<FmtE4m3>(p, st);
    return launch_experts_as<FmtInt8>(p, st);
}

}  // namespace mlora
