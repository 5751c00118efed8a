// Rows of a weight or activation matrix from global memory to MFMA operands.
//
// The 16 x 16 MFMA forms take row l % 16 in lane l, so a load straight into
// operand registers gives neighbouring lanes different rows: each 16-byte
// piece is a cache line of its own, and the vector memory unit handles one
// line per cycle, 64 cycles for the kilobyte of one load.  Measured on the
// MoE layer, the streams ran at that unit's pace (experts in 8 bits 2.2 TB/s,
// in bf16 3.4 to 5.0; as here 6 and 5.5 to 5.9).  Here a load takes eight whole 128-byte row segments
// (eight lanes each, 16 cycles), and the rows change lanes through a region of
// LDS that belongs to the wavefront alone: no barrier, and the loads of later
// blocks stay in flight in registers meanwhile.
//
// A region holds rows of 128 bytes; 16-byte chunk c of row r stands at
// 8 r + (c ^ (r / 2) % 8), so the writes (8 rows, 8 chunks) and the operand
// reads (16 rows, one chunk) both meet distinct banks.  Rows 16 apart keep the
// permutation, rows 8 apart flip its bit 2: StageAt holds the few lane
// addresses from which every access of a region is a constant away.
#pragma once

#include "common.hpp"

namespace mlora {

// Where the products that stream W begin their `steps` steps of K, which then go round:
// by groups of neighbouring tiles, spread evenly (the golden ratio's multiples).  Where
// all that stream at a time read the same bytes of rows a power of two apart, few of
// the memory's channels serve them: the experts of few rows, 8 x (28672, 4096) in bf16,
// 335 us from step 0, 265 so, and (4096, 4096) 57 and 41.  Neighbours that all differ
// lose what two of their row tiles share in the L2 (8192 rows of 8 x (4096, 14336) in
// tiles 965 us, in groups of four tiles 921), and eight starts in turn, tile by tile,
// fall in step with the channels again (40 rows of 8 x (28672, 4096) 441 us, 339).
__device__ __forceinline__ int k_phase(int group, int steps) {
    return (int)__umulhi((uint32_t)group * 0x9E3779B1u, (uint32_t)steps);
}

struct StageAt {
    int put[2];       // row l / 8 (+ 8), chunk l % 8
    int get[2];       // row l % 16, chunk l / 16 (+ 4)
    int pair[2];      // row l % 16, chunk 2 (l / 16) (+ 1)
    __device__ __forceinline__ StageAt() {
        const int l = lane_id(), r = l / 8, lr = l % 16, lq = l / 16, s = (lr / 2) % 8;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            put[i] = r * 8 + ((l % 8) ^ (r / 2 + 4 * i));
            get[i] = lr * 8 + ((lq + 4 * i) ^ s);
            pair[i] = lr * 8 + ((2 * lq + i) ^ s);
        }
    }
    // piece i: rows 8 i .. 8 i + 7
    __device__ __forceinline__ int piece(int i) const { return put[i % 2] + 64 * i; }
    // rows 16 n .. 16 n + 15
    __device__ __forceinline__ int half(int n, int i) const { return get[i] + 128 * n; }
    __device__ __forceinline__ int two(int n, int i) const { return pair[i] + 128 * n; }
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

// Orders a wavefront's LDS writes before its later reads of other lanes'
// data: LDS serves a wavefront in order, the compiler only has to keep it.
__device__ __forceinline__ void stage_order() {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
}

// 16 bytes at voff + soff (soff wave-uniform); reads zeros when voff lies past
// the resource.  NT: non-temporal, for rows that are read once.
template <bool NT>
__device__ __forceinline__ uint4 buf_ld16_at(__amdgpu_buffer_rsrc_t r, uint32_t voff, uint32_t soff) {
    const u32x4_vt v = __builtin_amdgcn_raw_buffer_load_b128(r, voff, soff, NT ? 2 : 0);
    return make_uint4(v[0], v[1], v[2], v[3]);
}

// The resource of a wave-uniform address.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t uniform_rsrc(const void* base, uint32_t bytes) {
    const uint64_t a = (uint64_t)(uintptr_t)base;
    const uint32_t lo = __builtin_amdgcn_readfirstlane((uint32_t)a);
    const uint32_t hi = __builtin_amdgcn_readfirstlane((uint32_t)(a >> 32));
    return buf_rsrc(reinterpret_cast<const void*>((uintptr_t)(((uint64_t)hi << 32) | lo)),
                    __builtin_amdgcn_readfirstlane(bytes));
}

}  // namespace mlora
