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
// expert's rows as the first operand, the expert's own tokens as columns), with
// the rest done by workgroups that come first in the grid and overlap the
// stream:
//   first launch   router (one workgroup per token), then 16 rows of A_gu x per
//                  workgroup and (token, expert) pair, then the consumers, which
//                  walk (up to 32 tokens of an expert, 16 gate and 16 up rows);
//   second launch  16 rows of A_d h per workgroup and pair, then the consumers of
//                  32 output rows and a share of all chosen experts: the routing
//                  weight is already in h, so a token's experts simply add up.
// Measured, first and second launch: 1 token, 2 of 8 experts of 4096 x 14336 in
// bf16 80 and 41 us (5.9 and 5.7 TB/s of expert rows; a large copy reaches 5.1
// with its writes); 64 tokens, all 8 of them 331 and 171 (5.7, 5.5); 27 tokens, 4
// of 40 experts of 2064 x 1424 in 8 bits 72 and 44 (3.0, 2.5): there the stream
// runs at 6 TB/s as well, between 12 us in which the router works (9 as a launch of its
// own) and every workgroup makes its tables, 6 until the first loads, and a ragged end.
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
#include "row_stage.hpp"

namespace mlora {

constexpr int kMdThreads = 256;
constexpr int kMdWaves = kMdThreads / kWave;
// Consumers of the first launch: three per compute unit, as many as its LDS holds
// (five, with the same units in shorter turns: 27 tokens, top 4 of 40 experts 127 us
// a layer against 117, 32 tokens of 8 experts in 8 bits 160 / 149; as many fewer as
// there are producers: 92 / 76 the launch).
constexpr int kMdResident = 3 * 256;
constexpr int kMdMaxSplits = 32;
constexpr int kMdMaxE = 256;
constexpr int kMdMaxPairs = LORA_DECODE_MAX_M * 16;
constexpr int kMdMaxGroups = kMdMaxE + kMdMaxPairs / 33 + 1;   // a second group takes 33 tokens

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

// Eight consecutive slots, their loads in flight together; zeros unless `on`.
__device__ __forceinline__ void slot_wait8(const slot_t* s, bool on, uint32_t want, int max_spin, bool* lost,
                                           uint32_t* w) {
    for (int spin = 0;; ++spin) {
        slot_t v[8];
        bool full = true;
#pragma unroll
        for (int q = 0; q < 8; ++q) v[q] = on ? slot_load(s + q) : 0ull;
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            full &= slot_full(v[q], want);
            w[q] = (uint32_t)v[q];
        }
        if (__ballot(on && !full) == 0ull) break;
        if (spin >= max_spin) {
            *lost |= on && !full;
            break;
        }
        __builtin_amdgcn_s_sleep(1);
    }
}

// v += four consecutive slots of each of n (at most four) places `step` apart, in
// order, their loads in flight together.
__device__ __forceinline__ void slot_add4x4(const slot_t* s, int64_t step, int n, uint32_t want, int max_spin,
                                            bool* lost, float (&v)[4]) {
    for (int spin = 0;; ++spin) {
        slot_t f[4][4];
        bool full = true;
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) f[j][q] = slot_load(s + min(j, n - 1) * step + q);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
            for (int q = 0; q < 4; ++q) full &= slot_full(f[j][q], want);
        if (full || spin >= max_spin) {
            *lost |= !full;
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int q = 0; q < 4; ++q) v[q] += j < n ? __uint_as_float((uint32_t)f[j][q]) : 0.f;
            return;
        }
        __builtin_amdgcn_s_sleep(1);
    }
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

// S values of the gate / up products that a workgroup keeps in LDS; a call with
// more (pairs times rank) reads the slots again for every unit.  Measured with and
// without: top 8 of 128 experts, rank 16, 4 tokens 78 / 104 us a layer, 16 tokens
// 104 / 136; top 4 of 40, rank 32, 27 tokens 116 / 111.
constexpr int kMdMaxS = 4096;

// Token of pair f < 1024: f / topk by the reciprocal, rounded up to 16 bits (off by
// less than f / 65536 < 1 / 16, and topk <= 16).
__device__ __forceinline__ int md_token(const MoeDecodeParams& p, int f) { return f * p.topk_inv >> 16; }

// Adapter of token m, or -1 (none, disabled, or outside the table).
__device__ __forceinline__ int md_adapter(const MoeDecodeParams& p, int m) {
    if (p.L == 0) return -1;
    const int l = p.ids[m];
    if (l < 0 || l >= p.L) return -1;
    return p.enabled[l] != 0 ? l : -1;
}

// ---------------------------------------------------------------- router
// Logits of one token: AT experts of a wavefront together, UN chunks of 512
// values of each in flight.
template <int AT, int UN>
__device__ __forceinline__ void md_logits(const MoeDecodeParams& p, const uint16_t* x, float* s_logit) {
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    for (int e0 = wave; e0 < p.E; e0 += AT * kMdWaves) {
        const uint16_t* w[AT];
        float c[AT];
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            w[i] = p.router + (int64_t)min(e0 + i * kMdWaves, p.E - 1) * p.H;
            c[i] = 0.f;
        }
#pragma unroll UN
        for (int k = lane * 8; k < p.H; k += kWave * 8) {
            const uint4 v = ld16(x + k);
#pragma unroll
            for (int i = 0; i < AT; ++i) c[i] = md_dot8(ld16(w[i] + k), v, c[i]);
        }
#pragma unroll
        for (int i = 0; i < AT; ++i) {
            c[i] = wave_total(c[i]);
            if (lane == 0 && e0 + i * kMdWaves < p.E) s_logit[e0 + i * kMdWaves] = c[i];
        }
    }
}

__device__ __forceinline__ void md_router(const MoeDecodeParams& p, uint32_t tag, int m, float* s_logit) {
    const int lane = lane_id(), wave = (int)threadIdx.x / kWave;
    const uint16_t* x = p.x + (int64_t)m * p.ldx;
    // an expert's row is a chain of loads: eight experts at a time (one expert, in
    // chunks of eight, made 4 tokens of 128 experts 93 us a layer against 78)
    md_logits<8, 2>(p, x, s_logit);
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
// S[j] = A[j, :] . v over K for 16 of the rank's rows, four a wavefront.
__device__ __forceinline__ void md_shrink(const uint16_t* A, const uint16_t* v, int K, slot_t* S, uint32_t tag) {
    const int lane = lane_id(), j = (int)threadIdx.x / kWave * 4;
    const uint16_t* a = A + (int64_t)j * K;
    float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
    for (int k = lane * 8; k < K; k += kWave * 8) {
        const uint4 t = ld16(v + k);
#pragma unroll
        for (int q = 0; q < 4; ++q) c[q] = md_dot8(ld16(a + (int64_t)q * K + k), t, c[q]);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        c[q] = wave_total(c[q]);
        if (lane == 0) slot_put(S + j + q, __uint_as_float(hi_lo(c[q])), tag);
    }
}
static_assert(kMdWaves * 4 == 16, "a shrink workgroup takes 16 rows");

// ---------------------------------------------------------------- routing tables in LDS
struct MdRoute {
    unsigned long long mask[kMdMaxE];      // tokens of each expert
    int16_t group[kMdMaxGroups];           // groups of up to 32 of an expert's tokens: expert, and
                                           // 256 times the group's number within it
    int16_t base[kMdMaxE];                 // an expert's first place in `list`
    int16_t exp_[kMdMaxPairs];             // expert of a pair, -1: none
    int16_t list[kMdMaxPairs];             // pairs by expert, then token
    int n_groups, n_max;                   // groups; most tokens of one expert
};

// After exp_ is filled: the rest.  Ends with a barrier.
__device__ __forceinline__ void md_tables(const MoeDecodeParams& p, MdRoute& r) {
    const int tid = threadIdx.x, lane = lane_id();
    const int P = p.M * p.topk;
    for (int e = tid; e < kMdMaxE; e += kMdThreads) r.mask[e] = 0ull;
    __syncthreads();
    for (int f = tid; f < P; f += kMdThreads)
        if (r.exp_[f] >= 0) atomicOr(&r.mask[r.exp_[f]], 1ull << md_token(p, f));
    __syncthreads();
    if (tid < kWave) {
        int pairs = 0, most = 0, groups = 0;
        for (int e0 = 0; e0 < p.E; e0 += kWave) {
            const int c = e0 + lane < p.E ? __popcll(r.mask[e0 + lane]) : 0;
            const unsigned long long b = __ballot(c > 0);
            const int incl = wave_incl_scan(c);
            if (c > 0) r.base[e0 + lane] = (int16_t)(pairs + incl - c);
            // at most 64 tokens: one or two groups
            const unsigned long long two = __ballot(c > 32);
            const unsigned long long lt = (1ull << lane) - 1ull;
            const int g = groups + __popcll(b & lt) + __popcll(two & lt);
            if (c > 0) r.group[g] = (int16_t)(e0 + lane);
            if (c > 32) r.group[g + 1] = (int16_t)(e0 + lane + kMdMaxE);
            groups += __popcll(b) + __popcll(two);
            pairs += __builtin_amdgcn_readlane(incl, kWave - 1);
            most = max(most, c);
        }
#pragma unroll
        for (int o = kWave / 2; o > 0; o >>= 1) most = max(most, __shfl_xor(most, o, kWave));
        if (lane == 0) r.n_groups = groups, r.n_max = most;
    }
    __syncthreads();
    for (int f = tid; f < P; f += kMdThreads) {
        const int e = r.exp_[f];
        if (e >= 0) r.list[r.base[e] + __popcll(r.mask[e] & ((1ull << md_token(p, f)) - 1ull))] = (int16_t)f;
    }
    __syncthreads();
}

// LDS values that are the same in every lane, as scalars.
__device__ __forceinline__ int md_uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ unsigned long long md_uni(unsigned long long v) {
    return ((unsigned long long)(uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32)) << 32) |
           (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
}

// ---------------------------------------------------------------- the stream
// One block: 128 bytes of each of 32 expert rows (64 values of K in bf16, 128 in
// 8 bits) and the same values of 8 XP token rows, in registers from their load
// to their turn.  A wavefront keeps U = md_flight blocks in flight and works in
// rounds of U.  Twelve wavefronts of a compute unit have 50 KB or more of expert
// rows on their way with one each, which is what latency times bandwidth asks
// for; more of them pays where the next block's address waits for nothing (one
// token of two bf16 experts: 1 block 127 us a call, 2 124, 4 122) and costs where
// rounds end ragged (12 tokens of H = 4096 in rounds of 3: 234, of 2 222; 27
// tokens of 40 experts in 8 bits, rounds of 2: 123, of 1 114).
constexpr int md_flight(bool w8) { return w8 ? 1 : 2; }

constexpr int md_blocks_of(int XP) { return (XP + 1) / 2; }      // 16-column token blocks

template <bool W8, int XP> struct MdBlock {
    static constexpr int XH = W8 ? 2 : 1;          // 64-value parts of a block
    static constexpr int KV = 64 * XH;
    uint4 w[4];
    uint4 x[XH][XP];
};

// Where a wavefront's loads go: lane l takes row l / 8 of each group of eight
// and chunk l % 8 of its 128 bytes.
template <int XP> struct MdRows {
    uint32_t w[4];                                 // byte offsets in the expert's matrix
    uint32_t x[XP];                                // in the token matrix; kBufOff: no such row
};

template <bool W8, int XP>
__device__ __forceinline__ void md_issue(MdBlock<W8, XP>& b, __amdgpu_buffer_rsrc_t rw, __amdgpu_buffer_rsrc_t rx,
                                         const MdRows<XP>& r, int kb, int K) {
    using B = MdBlock<W8, XP>;
    const int c = lane_id() % 8;
    // chunks past the end of the row read zeros, in both operands
    const bool w_in = kb * B::KV + c * (W8 ? 16 : 8) < K;
#pragma unroll
    for (int i = 0; i < 4; ++i) b.w[i] = buf_ld16_at<true>(rw, w_in ? r.w[i] : kBufOff, (uint32_t)kb * 128u);
#pragma unroll
    for (int h = 0; h < B::XH; ++h) {
        const bool x_in = kb * B::KV + h * 64 + c * 8 < K;
#pragma unroll
        for (int i = 0; i < XP; ++i)
            b.x[h][i] = buf_ld16_at<false>(rx, x_in ? r.x[i] : kBufOff, (uint32_t)(kb * B::XH + h) * 128u);
    }
}

// uint4 of LDS per wavefront: 32 expert rows and 16 token rows
constexpr int kMdStage = (32 + 16) * 8;

// acc[n][t] += rows 16 n .. 16 n + 15 times token block t over the block's
// values.  `refill` issues the block's next loads once its registers are free.
// With XP = 1 the operand's columns 8 to 15 are whatever LDS holds: they only
// reach sums that nobody reads.
template <bool W8, int XP, typename F>
__device__ __forceinline__ void md_consume(MdBlock<W8, XP>& b, uint4* st, const StageAt& at,
                                           f32x4_t (&acc)[2][md_blocks_of(XP)], F refill) {
    using B = MdBlock<W8, XP>;
    constexpr int TB = md_blocks_of(XP);
    constexpr int PT = XP == 1 ? 1 : 2;            // pieces of a token block
    uint4* sx = st + 32 * 8;
#pragma unroll
    for (int i = 0; i < 4; ++i) st[at.piece(i)] = b.w[i];
#pragma unroll
    for (int h = 0; h < B::XH; ++h)
#pragma unroll
        for (int t = 0; t < TB; ++t) {
#pragma unroll
            for (int i = 0; i < PT; ++i) sx[at.piece(i)] = b.x[h][2 * t + i];
            stage_order();
            if (h == B::XH - 1 && t == TB - 1) refill();
            uint4 a[2][2];
            if constexpr (W8) {
#pragma unroll
                for (int n = 0; n < 2; ++n) widen16(st[at.half(n, h)], a[n][0], a[n][1]);
            } else {
#pragma unroll
                for (int n = 0; n < 2; ++n)
#pragma unroll
                    for (int j = 0; j < 2; ++j) a[n][j] = st[at.half(n, j)];
            }
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                // in 8 bits a lane's chunk is 16 values: their two halves
                const uint4 v = sx[W8 ? at.two(0, j) : at.half(0, j)];
#pragma unroll
                for (int n = 0; n < 2; ++n) acc[n][t] = mfma_bf16(a[n][j], v, acc[n][t]);
            }
            stage_order();
        }
}

// Deltas of one expert, dealt to the wavefronts: step d is one 32-wide part j
// of the rank for one adapter among the expert's tokens (`ad`: lane t holds
// the adapter of column t, -1 for none), and wavefront d % kMdWaves takes it.
struct MdStep {
    int l, j;                     // adapter (-1: no such step), first rank position
    unsigned long long cols;      // its columns
};
__device__ __forceinline__ MdStep md_step(int ad, int r, int d) {
    const int per = (r + 31) / 32;
    unsigned long long rem = __ballot(ad >= 0);
    MdStep s{-1, 0, 0ull};
    for (int g = d / per; rem; --g) {
        const int l = __builtin_amdgcn_readlane(ad, __ffsll((long long)rem) - 1);
        const unsigned long long same = __ballot(ad == l);
        if (g == 0) {
            s.l = l;
            s.j = d % per * 32;
            s.cols = same;
            break;
        }
        rem &= ~same;
    }
    return s;
}

// A step's two operands of B rows: rows row[n] of the adapter's matrix.
__device__ __forceinline__ void md_step_load(const MoeDecodeParams& p, const uint16_t* B, int64_t per_l,
                                             const int64_t (&row)[2], const MdStep& s, uint4 (&b)[2]) {
    const int j = s.j + lane_id() / 16 * 8;
    const uint32_t mj = opaque_mask(j < p.r);
#pragma unroll
    for (int n = 0; n < 2; ++n)
        b[n] = and4(ld16(B + max(s.l, 0) * per_l + row[n] * p.r + min(j, p.r - 8)), mj);
}

// acc += B S for the step's columns.  S rows by pair: from `sS` when the
// workgroup holds them in LDS, else from their exchange slots.
template <int TB>
__device__ __forceinline__ void md_step_add(const MoeDecodeParams& p, const uint32_t* sS, const slot_t* S,
                                            const MdStep& s, int pair, const uint4 (&b)[2], uint32_t want,
                                            bool* lost, f32x4_t (&acc)[2][TB]) {
    const int lane = lane_id(), lr = lane % 16;
    const int j = s.j + lane / 16 * 8;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
        if (((s.cols >> (16 * t)) & 0xffffull) == 0ull) continue;
        const bool col = (s.cols >> (16 * t + lr)) & 1ull, on = col && j < p.r;
        const int at = __shfl(pair, 16 * t + lr, kWave) * p.r + min(j, p.r - 8);
        uint32_t w[8];
        if (sS) {
            const uint32_t m = opaque_mask(on);
            const uint4 a = and4(*reinterpret_cast<const uint4*>(sS + at), m);
            const uint4 c = and4(*reinterpret_cast<const uint4*>(sS + at + 4), m);
            w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
            w[4] = c.x; w[5] = c.y; w[6] = c.z; w[7] = c.w;
        } else {
            slot_wait8(S + at, on, want, p.wc.max_spin, lost, w);
        }
        uint4 h, lo;
        h.x = (w[0] >> 16) | (w[1] & 0xffff0000u); lo.x = (w[0] & 0xffffu) | (w[1] << 16);
        h.y = (w[2] >> 16) | (w[3] & 0xffff0000u); lo.y = (w[2] & 0xffffu) | (w[3] << 16);
        h.z = (w[4] >> 16) | (w[5] & 0xffff0000u); lo.z = (w[4] & 0xffffu) | (w[5] << 16);
        h.w = (w[6] >> 16) | (w[7] & 0xffff0000u); lo.w = (w[6] & 0xffffu) | (w[7] << 16);
        // other columns keep their sums: their zeros times an adapter's
        // infinities would not be zero
#pragma unroll
        for (int n = 0; n < 2; ++n) {
            const f32x4_t v = mfma_bf16(b[n], lo, mfma_bf16(b[n], h, acc[n][t]));
#pragma unroll
            for (int q = 0; q < 4; ++q) acc[n][t][q] = col ? v[q] : acc[n][t][q];
        }
    }
}

// ---------------------------------------------------------------- first launch
// The consumers: units u = first, first + stride, ... of (up to 32 tokens of an
// expert, 16 gate and 16 up rows).  The wavefronts share a unit's K, block by
// block in turn; the loads of the next unit are issued from the last round of the
// one before, so the stream does not stop at its end.
template <bool W8, int XP>
__device__ __forceinline__ void md_gate_up(const MoeDecodeParams& p, const MdRoute& rt, const float* s_w,
                                           const int16_t* s_ad, uint32_t* s_S, uint4* smem, int first, int stride,
                                           uint32_t want, bool* lost) {
    using B = MdBlock<W8, XP>;
    constexpr int TB = md_blocks_of(XP);
    constexpr int kBytes = W8 ? 1 : 2, U = md_flight(W8);
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int lr = lane % 16, lq = lane / 16;
    uint4* st = smem + wave * kMdStage;
    const StageAt at;
    const int tiles = (p.I + 15) / 16;
    const int units = md_uni(rt.n_groups) * tiles;
    const int KB = (p.H + B::KV - 1) / B::KV;
    const int nb = ((KB + kMdWaves - 1) / kMdWaves + U - 1) / U * U;    // blocks per wavefront and unit
    const uint32_t ebytes = (uint32_t)(2 * p.I) * (uint32_t)p.H * kBytes;
    const __amdgpu_buffer_rsrc_t rx = uniform_rsrc(p.x, (uint32_t)(((int64_t)(p.M - 1) * p.ldx + p.H) * 2));

    MdRows<XP> rows;
    const char* wbase = nullptr;
    int u_load = first, b_load = 0;
    auto set_rows = [&]() {                        // the unit that loads are issued for
        if (u_load >= units) return;
        const int g = md_uni((int)rt.group[u_load / tiles]);
        const int e = g % kMdMaxE, skip = g / kMdMaxE * 32;
        const int n0 = (u_load % tiles) * 16;
        wbase = static_cast<const char*>(p.W_gu) + (int64_t)e * 2 * p.I * p.H * kBytes;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int n = min(n0 + (i % 2) * 8 + lane / 8, p.I - 1) + (i / 2) * p.I;
            rows.w[i] = (uint32_t)n * (uint32_t)p.H * kBytes + (lane % 8) * 16;
        }
        const int ne = __popcll(md_uni(rt.mask[e])) - skip, base = md_uni((int)rt.base[e]) + skip;
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            const int t = 8 * i + lane / 8;
            rows.x[i] = t < ne ? (uint32_t)(md_token(p, rt.list[base + t])) * (uint32_t)p.ldx * 2u + (lane % 8) * 16
                               : kBufOff;
        }
    };
    // U blocks are issued at a time, one after the other
    auto issue = [&](B& b, int q) {
        const int kb = (b_load + q) * kMdWaves + wave;
        const bool on = u_load < units && kb < KB;
        md_issue<W8, XP>(b, uniform_rsrc(wbase, on ? ebytes : 0u), rx, rows, on ? kb : KB, p.H);
    };
    auto issued = [&]() {
        b_load += U;
        if (b_load < nb) return;
        b_load = 0;
        u_load += stride;
        set_rows();
    };
    set_rows();
    B blk[U];
#pragma unroll
    for (int q = 0; q < U; ++q) issue(blk[q], q);
    issued();

    for (int u = first; u < units; u += stride) {
        const int g = md_uni((int)rt.group[u / tiles]);
        const int e = g % kMdMaxE, skip = g / kMdMaxE * 32;
        const int n0 = (u % tiles) * 16;
        const int ne = min(__popcll(md_uni(rt.mask[e])) - skip, 32), base = md_uni((int)rt.base[e]) + skip;
        f32x4_t acc[2][TB];
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int t = 0; t < TB; ++t) acc[n][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
        // what the unit's end needs, loaded ahead of its stream: the scales and
        // the B rows of the wavefront's first delta step
        float sg[W8 ? 8 : 1];
        if constexpr (W8) {
            const float* sc = p.s_gu + (int64_t)e * 2 * p.I + min(n0 + lq * 4, p.I - 4);
#pragma unroll
            for (int q = 0; q < 4; ++q) sg[q] = sc[q], sg[4 + q] = sc[p.I + q];
        }
        const int f = rt.list[base + min(lane, ne - 1)];
        const int ad = p.L > 0 && lane < ne ? s_ad[md_token(p, f)] : -1;
        const int64_t row_g = (int64_t)e * 2 * p.I + min(n0 + lr, p.I - 1);
        const int64_t row[2] = {row_g, row_g + p.I};
        MdStep step = md_step(ad, p.r, wave);
        uint4 bop[2];
        if (step.l >= 0) md_step_load(p, p.B_gu, (int64_t)p.E * 2 * p.I * p.r, row, step, bop);
        for (int b = 0; b < nb; b += U) {
#pragma unroll
            for (int q = 0; q < U; ++q) md_consume<W8, XP>(blk[q], st, at, acc, [&]() { issue(blk[q], q); });
            issued();
        }
        if constexpr (W8) {
            // columns past I (a ragged last tile) are never stored
#pragma unroll
            for (int q = 0; q < 4; ++q)
#pragma unroll
                for (int t = 0; t < TB; ++t) acc[0][t][q] *= sg[q], acc[1][t][q] *= sg[4 + q];
        }
        if (p.L > 0) {
            if (u == first && s_S) {               // every unit reads S: once from the slots into LDS
                for (int i = (int)threadIdx.x * 8; i < p.M * p.topk * p.r; i += kMdThreads * 8) {
                    uint32_t w[8];
                    slot_wait8(p.S_gu + i, s_ad[i / (p.topk * p.r)] >= 0, want, p.wc.max_spin, lost, w);
                    *reinterpret_cast<uint4*>(s_S + i) = make_uint4(w[0], w[1], w[2], w[3]);
                    *reinterpret_cast<uint4*>(s_S + i + 4) = make_uint4(w[4], w[5], w[6], w[7]);
                }
                __syncthreads();
            }
            for (int d = wave; step.l >= 0;) {
                md_step_add<TB>(p, s_S, p.S_gu, step, f, bop, want, lost, acc);
                d += kMdWaves;
                step = md_step(ad, p.r, d);
                if (step.l >= 0) md_step_load(p, p.B_gu, (int64_t)p.E * 2 * p.I * p.r, row, step, bop);
            }
        }
        // the wavefronts' partial sums join in a fixed order through the stages
        float4* red = reinterpret_cast<float4*>(st);
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int t = 0; t < TB; ++t)
                red[(n * TB + t) * kWave + lane] = make_float4(acc[n][t][0], acc[n][t][1], acc[n][t][2], acc[n][t][3]);
        __syncthreads();
        const int pos = wave * 16 + lr, n = n0 + lq * 4;     // wave t < TB finishes token block t
        if (wave < TB && pos < ne && n < p.I) {
            float g[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 2
            for (int w = 0; w < kMdWaves; ++w) {
                const float4* src = reinterpret_cast<const float4*>(smem + w * kMdStage);
                const float4 a = src[wave * kWave + lane], c = src[(TB + wave) * kWave + lane];
                g[0] += a.x; g[1] += a.y; g[2] += a.z; g[3] += a.w;
                v[0] += c.x; v[1] += c.y; v[2] += c.z; v[3] += c.w;
            }
            const int f = rt.list[base + pos];
            uint32_t o[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) o[q] = f32_to_bf16(s_w[f] * (g[q] / (1.f + expf(-g[q]))) * v[q]);
            *reinterpret_cast<uint2*>(p.h + (int64_t)f * p.I + n) = make_uint2(o[0] | (o[1] << 16), o[2] | (o[3] << 16));
        }
        __syncthreads();
    }
}

// XPM: most pieces of eight tokens of one group, by M: 1, 2 or 4.  The variant
// taken is the one of the batch's busiest expert, as fewer pieces are less to
// load, stage and multiply (four pieces always, against this: 16 tokens, top 8 of
// 128 experts in 8 bits 127 / 104 us a layer, 27 tokens, top 4 of 40 130 / 116, 1
// token, 2 of 8 experts in bf16 128 / 125).  Kernels of their own for few tokens
// spare those the registers of the widest (12 tokens of 8 experts 227 to 238 us,
// from one kernel for all 239).  The widest, XPM = 4, fills its 168 registers: five or
// six values are spilled before the units and read back after them (one or two once a
// unit), 70 to 80 scalar ones go to lanes of vector registers.
template <bool W8, int XPM>
__global__ __launch_bounds__(kMdThreads, 3) void k_moe_gate_up(MoeDecodeParams p, int shrinks) {
    __shared__ uint4 smem[kMdWaves * kMdStage];
    __shared__ MdRoute rt;
    __shared__ float s_w[kMdMaxPairs];
    __shared__ __attribute__((aligned(16))) uint32_t s_S[kMdMaxS];
    __shared__ int16_t s_ad[LORA_DECODE_MAX_M];
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
        const int parts = p.r / 16, f = blk / parts, j0 = blk % parts * 16;
        const int m = md_token(p, f), l = md_adapter(p, m);
        if (l < 0) return;
        const int e = (int)slot_wait(p.route + f, want, p.wc.max_spin, &lost);
        if (lost) {
            if (tid == 0) atomicOr(p.err, LORA_DEVERR_WAIT);
            return;
        }
        const int64_t slot = p.shared_outer ? l : (int64_t)l * p.E + e;
        md_shrink(p.A_gu + (slot * p.r + j0) * p.H, p.x + (int64_t)m * p.ldx, p.H, p.S_gu + (int64_t)f * p.r + j0, tag);
        return;
    }
    blk -= shrinks;
    if (tid < p.M) s_ad[tid] = (int16_t)md_adapter(p, tid);
    for (int f = tid; f < P; f += kMdThreads) {
        bool gone = false;
        const int e = (int)slot_wait(p.route + f, want, p.wc.max_spin, &gone);
        s_w[f] = __uint_as_float(slot_wait(p.route + P + f, want, p.wc.max_spin, &gone));
        rt.exp_[f] = (int16_t)(gone ? -1 : e);
        lost |= gone;
    }
    md_tables(p, rt);
    const int stride = (int)gridDim.x - p.M - shrinks;
    uint32_t* S = P * p.r <= kMdMaxS ? s_S : nullptr;
    const int most = md_uni(rt.n_max);
    if (XPM == 1 || most <= 8)
        md_gate_up<W8, 1>(p, rt, s_w, s_ad, S, smem, blk, stride, want, &lost);
    else if (XPM == 2 || most <= 16)
        md_gate_up<W8, 2>(p, rt, s_w, s_ad, S, smem, blk, stride, want, &lost);
    else
        md_gate_up<W8, XPM>(p, rt, s_w, s_ad, S, smem, blk, stride, want, &lost);
    if (lost) atomicOr(p.err, LORA_DEVERR_WAIT);
}

// ---------------------------------------------------------------- second launch
// The consumers of the second launch: 32 output rows and one share of the blocks
// of all groups (up to 32 tokens of an expert).  A group's sums have its own
// tokens as columns; they are added to the workgroup's output, one fp32 value a
// row and token, which each wavefront holds for itself in LDS (`out`).  So an
// expert's values, infinities among them, reach the tokens that chose it and no
// others, and columns do not grow with the batch.
constexpr int kMdOut = 36;                         // floats of a token's 32 rows, spread over banks

template <bool W8, int XP>
__device__ __forceinline__ void md_down(const MoeDecodeParams& p, const MdRoute& rt, const int16_t* s_ad, float* out,
                                        uint4* st, int n0, int split, uint32_t want, bool* lost) {
    using B = MdBlock<W8, XP>;
    constexpr int TB = md_blocks_of(XP);
    constexpr int kBytes = W8 ? 1 : 2, U = md_flight(W8);
    const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x / kWave);
    const int lr = lane % 16, lq = lane / 16;
    const StageAt at;
    const int ng = md_uni(rt.n_groups);
    const int KB = (p.I + B::KV - 1) / B::KV;               // blocks of one group
    const int total = ng * KB;
    const int t0 = (int)((int64_t)total * split / p.splits), t1 = (int)((int64_t)total * (split + 1) / p.splits);
    const uint32_t ebytes = (uint32_t)p.H * (uint32_t)p.I * kBytes;
    const __amdgpu_buffer_rsrc_t rh = uniform_rsrc(p.h, (uint32_t)(p.M * p.topk) * (uint32_t)p.I * 2u);
    struct Group {
        int e, base, ne;
    };
    auto group = [&](int g) {
        const int v = md_uni((int)rt.group[g]), e = v % kMdMaxE, skip = v / kMdMaxE * 32;
        return Group{e, md_uni((int)rt.base[e]) + skip, min((int)__popcll(md_uni(rt.mask[e])) - skip, 32)};
    };

    MdRows<XP> rows;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        rows.w[i] = (uint32_t)min(n0 + 8 * i + lane / 8, p.H - 1) * (uint32_t)p.I * kBytes + (lane % 8) * 16;
    const char* wbase = nullptr;
    int g_load = t0 / KB, kb_load = 0;                      // group and block of the next load
    // a part: one group's blocks of this share, [beg, end), every kMdWaves-th of
    // them this wavefront's, their number rounded up to U
    auto part_end = [&](int g) { return min(KB, t1 - g * KB); };
    auto part_beg = [&](int g) { return max(0, t0 - g * KB); };
    auto part_blocks = [&](int g) {
        return ((part_end(g) - part_beg(g) + kMdWaves - 1) / kMdWaves + U - 1) / U * U;
    };
    int left = 0, end_load = 0;
    auto set_rows = [&]() {
        if (g_load * KB >= t1) return;
        const Group g = group(g_load);
        wbase = static_cast<const char*>(p.W_d) + (int64_t)g.e * p.H * p.I * kBytes;
        left = part_blocks(g_load);
        end_load = part_end(g_load);
        kb_load = part_beg(g_load) + wave;
#pragma unroll
        for (int i = 0; i < XP; ++i) {
            const int t = 8 * i + lane / 8;
            rows.x[i] = t < g.ne ? (uint32_t)rt.list[g.base + t] * (uint32_t)p.I * 2u + (lane % 8) * 16 : kBufOff;
        }
    };
    auto issue = [&](B& b, int q) {
        const int kb = kb_load + q * kMdWaves;
        const bool on = g_load * KB < t1 && kb < end_load;
        md_issue<W8, XP>(b, uniform_rsrc(wbase, on ? ebytes : 0u), rh, rows, on ? kb : KB, p.I);
    };
    auto issued = [&]() {
        kb_load += U * kMdWaves;
        left -= U;
        if (left > 0) return;
        ++g_load;
        set_rows();
    };
    set_rows();
    B blk[U];
#pragma unroll
    for (int q = 0; q < U; ++q) issue(blk[q], q);
    issued();

    f32x4_t part[2][TB];
    auto clear = [&]() {
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int t = 0; t < TB; ++t) part[n][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    };
    // the group's sums, times the rows' scales, to its tokens' rows
    auto add = [&](const Group& g, const float (&s)[2][4]) {
        stage_order();
#pragma unroll
        for (int t = 0; t < TB; ++t) {
            if (16 * t + lr >= g.ne) continue;
            float* d = out + md_token(p, rt.list[g.base + 16 * t + lr]) * kMdOut + lq * 4;
#pragma unroll
            for (int n = 0; n < 2; ++n) {
                float4* o = reinterpret_cast<float4*>(d + 16 * n);
                float4 v = *o;
                v.x += part[n][t][0] * s[n][0];
                v.y += part[n][t][1] * s[n][1];
                v.z += part[n][t][2] * s[n][2];
                v.w += part[n][t][3] * s[n][3];
                *o = v;
            }
        }
    };
    float one[2][4];
#pragma unroll
    for (int n = 0; n < 2; ++n)
#pragma unroll
        for (int q = 0; q < 4; ++q) one[n][q] = 1.f;
    for (int a = t0 / KB; a * KB < t1; ++a) {
        const Group g = group(a);
        const int nb = part_blocks(a);
        float s[2][4];
        if constexpr (W8) {                                 // loaded ahead of the part's stream
            const float* sc = p.s_d + (int64_t)g.e * p.H;
#pragma unroll
            for (int n = 0; n < 2; ++n)
#pragma unroll
                for (int q = 0; q < 4; ++q) s[n][q] = sc[min(n0 + 16 * n + lq * 4 + q, p.H - 1)];
        }
        clear();
        for (int b = 0; b < nb; b += U) {
#pragma unroll
            for (int q = 0; q < U; ++q) md_consume<W8, XP>(blk[q], st, at, part, [&]() { issue(blk[q], q); });
            issued();
        }
        add(g, W8 ? s : one);
    }
    if (p.L > 0) {
        const int64_t per_l = (int64_t)(p.shared_outer ? 1 : p.E) * p.H * p.r;
        const int64_t r0 = min(n0 + lr, p.H - 1), r1 = min(n0 + 16 + lr, p.H - 1);
        // the wavefront's steps over the split's groups, dealt in turn; the B
        // rows of one are in flight while the one before is added
        struct Task {
            MdStep s;
            int pair;
            Group g;
        };
        int deal = 0, i = split, d = -1;
        auto next = [&](uint4 (&b)[2]) {
            for (; i < ng; i += p.splits, d = -1) {
                const Group g = group(i);
                const int f = lane < g.ne ? rt.list[g.base + lane] : 0;
                const int ad = lane < g.ne ? s_ad[md_token(p, f)] : -1;
                for (++d;; ++d) {
                    const MdStep s = md_step(ad, p.r, d);
                    if (s.l < 0) break;
                    if (deal++ % kMdWaves != wave) continue;
                    const int64_t eb = p.shared_outer ? 0 : (int64_t)g.e * p.H;
                    const int64_t row[2] = {eb + r0, eb + r1};
                    md_step_load(p, p.B_d, per_l, row, s, b);
                    return Task{s, f, g};
                }
            }
            return Task{MdStep{-1, 0, 0ull}, 0, Group{0, 0, 0}};
        };
        auto delta = [&](const Task& k, const uint4 (&b)[2]) {
            clear();
            md_step_add<TB>(p, nullptr, p.S_d, k.s, k.pair, b, want, lost, part);
            add(k.g, one);
        };
        uint4 b0[2], b1[2];
        Task k0 = next(b0);
        while (k0.s.l >= 0) {
            const Task k1 = next(b1);
            delta(k0, b0);
            if (k1.s.l < 0) break;
            k0 = next(b0);
            delta(k1, b1);
        }
    }
}

// MT: most tokens, 32 or 64.  The outputs of 64 leave LDS for two workgroups a
// compute unit, those of 32 for three (two always: 16 tokens, top 8 of 128 experts
// 113 us a layer in place of 108, 27 tokens, top 4 of 40 122 / 117, the others within
// 2%).
template <bool W8, int MT>
__global__ __launch_bounds__(kMdThreads, MT > 32 ? 2 : 3) void k_moe_down(MoeDecodeParams p, int shrinks) {
    __shared__ uint4 smem[kMdWaves * kMdStage];
    __shared__ __attribute__((aligned(16))) float s_out[kMdWaves][MT * kMdOut];
    __shared__ MdRoute rt;
    __shared__ int16_t s_ad[LORA_DECODE_MAX_M];
    const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t tag = launch_tag(), want = tag ^ p.wc.poll_xor;
    const int P = p.M * p.topk;
    bool lost = false;
    int id = (int)blockIdx.x;
    if (id < shrinks) {
        const int parts = p.r / 16, f = id / parts, j0 = id % parts * 16;
        const int l = md_adapter(p, md_token(p, f));
        if (l < 0) return;
        md_shrink(p.A_d + (((int64_t)l * p.E + p.route_ids[f]) * p.r + j0) * p.I, p.h + (int64_t)f * p.I, p.I,
                  p.S_d + (int64_t)f * p.r + j0, tag);
        return;
    }
    id -= shrinks;
    const int tiles = (p.H + 31) / 32;
    const int split = id / tiles, n0 = (id % tiles) * 32;
    for (int f = tid; f < P; f += kMdThreads) rt.exp_[f] = (int16_t)p.route_ids[f];
    if (tid < p.M) s_ad[tid] = (int16_t)md_adapter(p, tid);
    for (int i = tid % kWave; i < p.M * kMdOut / 4; i += kWave)
        reinterpret_cast<float4*>(s_out[wave])[i] = make_float4(0.f, 0.f, 0.f, 0.f);
    md_tables(p, rt);
    const int most = md_uni(rt.n_max);
    uint4* st = smem + wave * kMdStage;
    if (most <= 8)
        md_down<W8, 1>(p, rt, s_ad, s_out[wave], st, n0, split, want, &lost);
    else if (most <= 16)
        md_down<W8, 2>(p, rt, s_ad, s_out[wave], st, n0, split, want, &lost);
    else
        md_down<W8, 4>(p, rt, s_ad, s_out[wave], st, n0, split, want, &lost);
    __syncthreads();
    // the wavefronts' sums in a fixed order, then the splits', four at a time and,
    // for few tokens, by several threads a place (a power of two, side by side)
    int subs = 1;
    while (subs < 8 && p.M * 8 * subs * 2 <= kMdThreads) subs *= 2;
    for (int i = tid; i < p.M * 8 * subs; i += kMdThreads) {
        const int sub = i % subs, m = i / subs / 8, c = i / subs % 8 * 4, n = n0 + c;
        if (n >= p.H) continue;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        if (sub == 0)
#pragma unroll
            for (int w = 0; w < kMdWaves; ++w) {
                const float4 a = *reinterpret_cast<const float4*>(s_out[w] + m * kMdOut + c);
                v[0] += a.x; v[1] += a.y; v[2] += a.z; v[3] += a.w;
            }
        const int64_t per = (int64_t)p.M * p.H;
        slot_t* d = p.join + (int64_t)m * p.H + n;
        if (split < p.splits - 1) {
            if (sub == 0)
#pragma unroll
                for (int q = 0; q < 4; ++q) slot_put(d + split * per + q, v[q], tag);
            continue;
        }
        // the last split of a tile adds the others
        for (int s = sub; s < p.splits - 1; s += 4 * subs)
            slot_add4x4(d + s * per, subs * per, min((p.splits - 2 - s) / subs + 1, 4), want, p.wc.max_spin, &lost, v);
        for (int o = 1; o < subs; o *= 2)
#pragma unroll
            for (int q = 0; q < 4; ++q) v[q] += __shfl_xor(v[q], o, kWave);
        if (sub == 0)
            *reinterpret_cast<uint2*>(p.out + (int64_t)m * p.ldo + n) =
                make_uint2(f32_to_bf16(v[0]) | (f32_to_bf16(v[1]) << 16), f32_to_bf16(v[2]) | (f32_to_bf16(v[3]) << 16));
    }
    if (lost) atomicOr(p.err, LORA_DEVERR_WAIT);
}

int moe_decode_max_splits(int H, int M) {
    // as many as keep every consumer resident at once, without the producers; half
    // of that: 64 tokens, top 8 of 128 experts 314 against 255 us a layer, 1 token, 2
    // of 8 experts 128 / 125, 8 tokens of 16 small experts 28 / 28; half again as
    // many: 281 / 258, 128 / 127, 31 / 30, and 27 tokens, top 4 of 40 125 / 117
    const int tiles = (H + 31) / 32;
    const int most = 256 * (M > 32 ? 2 : 3) / tiles;
    return most < 1 ? 1 : most > kMdMaxSplits ? kMdMaxSplits : most;
}

int moe_decode_splits(int H, int M, int64_t blocks) {
    const int most = moe_decode_max_splits(H, M);
    // two blocks a wavefront in each (with at most 16 splits whatever the blocks,
    // against this: 49 tokens of 10 experts of 1120 x 144 35.4 / 33.5 us a layer, 8
    // tokens, top 8 of 57 experts of 304 x 1648 67.7 / 62.6)
    const int64_t n = blocks / (2 * kMdWaves);
    return n < 1 ? 1 : n < most ? (int)n : most;
}

template <bool W8>
hipError_t launch_moe_decode_t(const MoeDecodeParams& p, hipStream_t st) {
    const int P = p.M * p.topk;
    const int shrinks = p.L > 0 ? P * (p.r / 16) : 0;
    const int units = min(min(p.E, P) + P / 33, kMdMaxGroups) * ((p.I + 15) / 16);
    const dim3 g1((unsigned)(p.M + shrinks + min(units, kMdResident))), g2((unsigned)(shrinks + (p.H + 31) / 32 * p.splits));
    const dim3 t(kMdThreads);
    if (p.M <= 8) hipLaunchKernelGGL((k_moe_gate_up<W8, 1>), g1, t, 0, st, p, shrinks);
    else if (p.M <= 16) hipLaunchKernelGGL((k_moe_gate_up<W8, 2>), g1, t, 0, st, p, shrinks);
    else hipLaunchKernelGGL((k_moe_gate_up<W8, 4>), g1, t, 0, st, p, shrinks);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    if (p.M <= 32) hipLaunchKernelGGL((k_moe_down<W8, 32>), g2, t, 0, st, p, shrinks);
    else hipLaunchKernelGGL((k_moe_down<W8, LORA_DECODE_MAX_M>), g2, t, 0, st, p, shrinks);
    return hipGetLastError();
}

hipError_t launch_moe_decode(const MoeDecodeParams& p, hipStream_t st) {
    return p.s_gu ? launch_moe_decode_t<true>(p, st) : launch_moe_decode_t<false>(p, st);
}

}  // namespace mlora
