// A tile of a product x W^T of 128-byte K stages on the matrix unit, both operands
// by way of rings in LDS: the main loop of the products with many rows (the
// experts' shares, the 8-bit projections).
//
// Tile = up to 256 rows of x by 256 rows of W (output columns), four waves, one per
// SIMD.  Both operands go from global memory straight to LDS (no registers, no LDS
// write instructions), whole 128-byte row segments: eight lanes a row, the chunk
// that a lane reads permuted so that chunk c of row r comes to stand at
// c ^ (r / 2) % 8, where operand reads (32 rows, one chunk) meet distinct banks.
// Rings of XD stages of x and WD of W fill the 160 KB; the loads of a stage are
// spread evenly between the MFMAs of the one before, x first.  The operands of the
// last K step of a stage are in registers one step early, so the one barrier of a
// stage stands in front of that step: behind it the stage's slots are free for the
// next loads and the following stage can be read, and no MFMA waits for either.
//
// What bounds it: 256 x 256 because a stage then asks LDS for 128 KB of operand
// reads and 64 KB of arriving loads in the 2048 cycles of its MFMAs, three quarters
// of what it gives (128 x 256: 1.1 times).  The last stages of W are the ones that
// come from far; a third one in flight took 8192^3 in e4m3 from 429 to 389 us, and
// spreading the loads instead of issuing them together bf16 from 940 to 795.
// Measured there 1.38 to 1.41 PFLOP/s in bf16, 2.9 in e4m3, 2.6 in int8; a large
// library product on the same card 1.37, 2.9 and 2.1.  With the loads taken out
// 1.62, 3.4 and 3.0 on the same values (zeros: 2.1, 4.0, 3.9: the rest is the
// clock, which falls with the power that real values take).
//
// Tiles with fewer rows: the waves of one with up to 192, 128 or 64 rows take
// 96 x 128, 128 x 64 and 64 x 64 outputs each instead of 128 x 128, with as many
// fewer MFMAs, and rings as deep as 160 KB allow.  Tiles of 128 columns likewise, for
// grids that would not fill the chip.
//
// The loads to LDS are written in assembly because the compiler waits for all of
// them at every LDS read; they have no output registers, and the waits that their
// data needs stand in turn().
#pragma once

#include "common.hpp"
#include "formats.hpp"
#include "row_stage.hpp"

namespace mlora {

constexpr int kRingThreads = 256;
constexpr int kRingRows = 256, kRingCols = 256;
constexpr int kRingLds = 160 * 1024;

// 16 zero bytes: what rows of x read past K
static __device__ const uint4 k_zeros = {0, 0, 0, 0};

typedef __attribute__((address_space(3))) char lds_char_t;

__device__ __forceinline__ void dma_global(const char* p, uint32_t lds) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(lds), "v"(p) : "memory");
}
// NT: read once, not kept in the caches
template <bool NT> __device__ __forceinline__ void dma_buffer(u32x4_vt r, uint32_t voff, uint32_t soff, uint32_t lds) {
    if constexpr (NT)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen nt lds" ::"s"(lds), "v"(voff),
                     "s"(r), "s"(soff)
                     : "memory");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, %3 offen lds" ::"s"(lds), "v"(voff),
                     "s"(r), "s"(soff)
                     : "memory");
}

// WM waves share the rows, 4 / WM the columns; a wave takes RB x CB blocks of 32 x 32.
template <typename F_, int WM_, int RB_, int CB_, int XD_, int WD_> struct Ring {
    typedef F_ F;
    static constexpr int WM = WM_, RB = RB_, CB = CB_, XD = XD_, WD = WD_;
    static constexpr int WN = 4 / WM, kRows = 32 * RB * WM, kCols = 32 * CB * WN;
    static constexpr int kX = kRows * 128, kW = kCols * 128;          // bytes of a ring slot
    static_assert(XD >= 2 && WD >= XD && WD <= XD + 1 && XD * kX + WD * kW <= kRingLds, "rings fit the LDS");
    static constexpr int NX = kRows / 32, NW = kCols / 32;            // loads of a wave and stage
    typedef typename F::Acc32 Acc;
    // the first row and column of a wave's part
    __device__ static int row0(int wave) { return wave / WN * RB * 32; }
    __device__ static int col0(int wave) { return wave % WN * CB * 32; }
    // row of the tile that lane l of wave w loads with its load i, the lane's bytes
    // of a 128-byte segment
    __device__ static int load_row(int wave, int i) { return 8 * wave + lane_id() / 8 + 32 * i; }
    __device__ static int load_byte(int wave) { return ((lane_id() % 8) ^ (lane_id() / 16 + 4 * (wave & 1))) * 16; }
};
template <typename F> using Ring256 = Ring<F, 2, 4, 4, 2, 3>;
template <typename F> using Ring192 = Ring<F, 2, 3, 4, 2, 3>;
template <typename F> using Ring128 = Ring<F, 1, 4, 2, 3, 3>;
template <typename F> using Ring64 = Ring<F, 1, 2, 2, 4, 4>;
// half the columns
template <typename F> using Half256 = Ring<F, 2, 4, 2, 3, 4>;
template <typename F> using Half192 = Ring<F, 2, 3, 2, 4, 4>;
template <typename F> using Half128 = Ring<F, 2, 2, 2, 5, 5>;
template <typename F> using Half64 = Ring<F, 2, 1, 2, 6, 6>;

// acc[rb][cb]: columns 32 cb + 8 (q / 4) + 4 (l / 32) + q % 4 of row 32 rb + l % 32 of
// the wave's part.  W: the tile's rows, `cols` of them, Kb bytes of K each, ldw apart
// (256 ldw below 2 GiB); x_rows(xp) gives the addresses of the rows that this lane
// loads (load_row(wave, i), any row that may be read past the tile's), load_byte
// added.  On return every wave is done with the LDS.
//
// The stages of K begin at k0 and go round.  NT: no other tile reads these rows of W.
template <typename R, bool NT = false, typename XRows>
__device__ __forceinline__ void ring_product(uint4* smem, const char* W, int64_t ldw, int cols, int Kb, int k0, XRows x_rows,
                                             typename R::Acc (&acc)[R::RB][R::CB]) {
    typedef typename R::F F;
    constexpr int RB = R::RB, CB = R::CB, XD = R::XD, WD = R::WD, NX = R::NX, NW = R::NW;
    constexpr int kX = R::kX, kW = R::kW;
    constexpr int kLoads = NX + NW;
    constexpr int kWords = F::kWords, MF = RB * CB;
    constexpr int kTotal = MF * (kWords == 1 ? 4 : 2);             // MFMAs of a stage
    constexpr int kPost = kWords == 1 ? MF : kTotal - MF / 2;      // of them behind the barrier
    constexpr int kReads = (RB + CB) * kWords;                     // operand reads of a step
    constexpr int kEarly = (kPost * kLoads + kTotal - 1) / kTotal; // loads issued behind the barrier
    // what may still be on its way when a stage is read: the stages after it (W of the
    // stage WD on is issued behind x of the one XD on)
    constexpr int kAhead = (XD - 2) * NX + (WD - 2) * NW;

    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int lr = lane % 32, lh = lane / 32;
    const int nk = (Kb + 127) / 128;

    // ---- loads: wave w takes the 8-row blocks w + 4 i, lane l row l / 8 of a block
    const int ch = R::load_byte(wave);
    const uint64_t wa = (uint64_t)(uintptr_t)W;
    const u32x4_vt rw = {(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)wa),
                         (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(wa >> 32)),
                         (uint32_t)__builtin_amdgcn_readfirstlane((int)((cols - 1) * ldw + Kb)), 0x00020000u};
    uint32_t woff[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) woff[i] = (uint32_t)(min(R::load_row(wave, i), cols - 1) * ldw) + ch;
    const char* xp[NX];
    const char* const zeros = reinterpret_cast<const char*>(&k_zeros);
    const uint32_t dst = (uint32_t)(uintptr_t)(lds_char_t*)smem + wave * 1024;

    // the loads under way: stage kx of x into ring slot lx, stage kw of W into lw, with
    // x_left and w_left to come.  The stages begin at k0 and go round.  Past K and past
    // the last one: zeros, and no memory of theirs is touched.
    int lx = 0, lw = 0, inc = 0, kx = k0, kw = k0, x_left = nk, w_left = nk;
    uint32_t so = 0;
    bool win = true, xin = true;
    auto begin_x = [&](int slot) {
        lx = slot;
        xin = x_left > 0 && kx * 128 + ch < Kb;
        inc = kx + 1 < nk ? 128 : 128 - nk * 128;
        kx = kx + 1 < nk ? kx + 1 : 0;
        --x_left;
    };
    auto begin_w = [&](int slot) {
        lw = slot;
        so = (uint32_t)kw * 128u;
        win = w_left > 0 && kw * 128 + ch < Kb;
        kw = kw + 1 < nk ? kw + 1 : 0;
        --w_left;
    };
    auto load_x = [&](int i) {
        dma_global(xin ? xp[i] : zeros, dst + lx + i * 4096);
        xp[i] += inc;
    };
    auto load_w = [&](int i) { dma_buffer<NT>(rw, win ? woff[i] : kBufOff, so, dst + lw + i * 4096); };
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

    // prologue.  The compiler waits for the loads behind x_rows with every load in
    // flight, so none of the ring's is issued before them.
    x_rows(xp);
#pragma unroll
    for (int i = 0; i < NX; ++i) xp[i] += k0 * 128;
#pragma unroll
    for (int st = 0; st < WD - 1; ++st) {
        begin_w(wsl[st]);
#pragma unroll
        for (int i = 0; i < NW; ++i) load_w(i);
        if (st >= XD - 1) continue;
        begin_x(xs[st]);
#pragma unroll
        for (int i = 0; i < NX; ++i) load_x(i);
    }
    begin_x(xs[XD - 1]);
    begin_w(wsl[WD - 1]);
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
    const int xpart = R::row0(wave) * 128, wpart = R::col0(wave) * 128;
    struct Ops {
        uint4 x[RB][kWords], w[CB][kWords];
    };
    auto read1 = [&](Ops& o, int x0, int w0, int t, int j) {
        const int b = j / kWords, h = j % kWords, c = t * kWords + h;
        if (b < CB) o.w[b][h] = *reinterpret_cast<const uint4*>(lds + (w0 + wpart + get[c]) + b * 4096);
        else o.x[b - CB][h] = *reinterpret_cast<const uint4*>(lds + (x0 + xpart + get[c]) + (b - CB) * 4096);
    };
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
    auto turn = [&]() {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(kAhead) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
        begin_x(xs[0]);
        begin_w(wsl[0]);
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
            turn();
            run(ob, 0, MF, 0, &oa, xs[1], wsl[1], 0);
        } else {
            run(oa, 0, MF / 2, kPost, &ob, xs[0], wsl[0], 1);
            turn();
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
}

// The rows of a block of 32 x 32 sums as its stores take them: lane l stores row
// l % 16 and row 16 + l % 16, 16 bytes from column 8 store_chunk().
__device__ __forceinline__ int store_chunk() { return (lane_id() / 16 % 2) * 2 + lane_id() / 32; }

// Rounds a block of sums (row l % 32, columns as in ring_product) and stores it:
// `dst` the lane's two rows at its column, 64 consecutive bytes of 16 rows an
// instruction.  Straight from the registers: two exchanges of half the lanes bring a
// row's eight columns together and its four pieces side by side.  By way of LDS
// in whole row pieces a tile's epilogue took 7.3 us, with the first exchange alone (32
// bytes of 32 rows) 4.7.
__device__ __forceinline__ void store_block(const f32x16_t& v, uint16_t* const (&dst)[2], const bool (&ok)[2]) {
    uint32_t w[2][4];                    // columns 8 (2 i + l / 32) of row l % 32
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float* const f = reinterpret_cast<const float*>(&v) + 8 * i;
        const auto lo = __builtin_amdgcn_permlane32_swap(pack_bf16(f[0], f[1]), pack_bf16(f[4], f[5]), false, false);
        const auto hi = __builtin_amdgcn_permlane32_swap(pack_bf16(f[2], f[3]), pack_bf16(f[6], f[7]), false, false);
        w[i][0] = lo[0], w[i][1] = hi[0], w[i][2] = lo[1], w[i][3] = hi[1];
    }
    uint32_t o[2][4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        const auto s = __builtin_amdgcn_permlane16_swap(w[0][q], w[1][q], false, false);
        o[0][q] = s[0], o[1][q] = s[1];
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
        if (ok[h]) *reinterpret_cast<uint4*>(dst[h]) = make_uint4(o[h][0], o[h][1], o[h][2], o[h][3]);
}

}  // namespace mlora
