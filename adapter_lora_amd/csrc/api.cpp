// C ABI entry points: argument checks, workspace layout, launches.
// Nothing here allocates device memory or synchronises (except
// lora_read_device_error, which is documented to synchronise).
#include <dlfcn.h>
#include <hip/hip_runtime.h>
#include <stdint.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <vector>

#include "../../include/mlora.h"
#include "common.hpp"
#include "kernels.hpp"

using namespace mlora;

namespace {

constexpr size_t kAlign = 256;
inline size_t up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

lora_status from_hip(hipError_t e) { return e == hipSuccess ? LORA_OK : LORA_HIP_ERROR; }

// The sticky error word of a linear workspace (its first word).
int* ws_error(void* workspace) { return &reinterpret_cast<WsHeader*>(workspace)->error; }

// roctx ranges around the entry points that launch work, for profiler
// timelines (rocprofv3 --marker-trace).  Off unless MLORA_ROCTX=1 when the
// first call is made; the roctx library is then looked up at run time, so
// the library has no link dependency on it and a call pays one branch when
// ranges are off.
struct Roctx {
    int (*push)(const char*) = nullptr;
    int (*pop)() = nullptr;
    Roctx() {
        const char* on = getenv("MLORA_ROCTX");
        if (!on || strcmp(on, "1") != 0) return;
        void* h = dlopen("librocprofiler-sdk-roctx.so.1", RTLD_NOW | RTLD_LOCAL);
        if (!h) h = dlopen("libroctx64.so.4", RTLD_NOW | RTLD_LOCAL);
        if (!h) return;
        push = reinterpret_cast<int (*)(const char*)>(dlsym(h, "roctxRangePushA"));
        pop = reinterpret_cast<int (*)()>(dlsym(h, "roctxRangePop"));
        if (!push || !pop) push = nullptr, pop = nullptr;
    }
};

const Roctx& roctx() {
    static const Roctx r;
    return r;
}

class Range {
  public:
    explicit Range(const char* name) : on_(roctx().push != nullptr) {
        if (on_) roctx().push(name);
    }
    ~Range() {
        if (on_) roctx().pop();
    }
    Range(const Range&) = delete;
    Range& operator=(const Range&) = delete;

  private:
    bool on_;
};

int64_t n_total(const lora_weights_t* w) { return w->slice_offsets[w->n_slices]; }

lora_status check_weights(const lora_weights_t* w) {
    if (!w) return LORA_INVALID_ARG;
    if (w->dtype != LORA_F32 && w->dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (w->K <= 0 || w->K % 8 != 0) return LORA_INVALID_ARG;
    if (w->n_slices < 1 || w->n_slices > LORA_MAX_SLICES) return LORA_INVALID_ARG;
    if (w->L < 1 || w->L > LORA_MAX_ADAPTERS) return LORA_INVALID_ARG;
    if (w->r_max < LORA_RANK_ALIGN || w->r_max > LORA_MAX_RANK || w->r_max % LORA_RANK_ALIGN)
        return LORA_INVALID_ARG;
    if (w->slice_offsets[0] != 0) return LORA_INVALID_ARG;
    for (int s = 0; s < w->n_slices; ++s) {
        const int64_t n = w->slice_offsets[s + 1] - w->slice_offsets[s];
        if (n <= 0 || n % 8 != 0) return LORA_INVALID_ARG;
    }
    if (n_total(w) > INT32_MAX) return LORA_UNSUPPORTED;
    if (!w->A || !w->B || !w->a_off || !w->b_off || !w->rank) return LORA_INVALID_ARG;
    if (!aligned16(w->A) || !aligned16(w->B)) return LORA_INVALID_ARG;
    return LORA_OK;
}

lora_status check_segments(const lora_segments_t* seg, const lora_weights_t* w, int M) {
    if (!seg || !seg->sorted_idx || !seg->seg_indptr || !seg->req_to_lora || !seg->num_segments ||
        !seg->tile_info || !seg->tile_rows || !seg->num_tiles)
        return LORA_INVALID_ARG;
    if (seg->L != w->L) return LORA_INVALID_ARG;
    if (seg->max_tiles < lora_tile_capacity(M, w->L)) return LORA_INVALID_ARG;
    return LORA_OK;
}

lora_status check_rows(const void* p, int64_t ld, int64_t width) {
    if (!p || !aligned16(p)) return LORA_INVALID_ARG;
    if (ld < width || ld % 8 != 0) return LORA_INVALID_ARG;
    return LORA_OK;
}

LinearArgs make_args(const lora_weights_t* w, const lora_segments_t* seg, int M) {
    LinearArgs a{};
    a.dtype = w->dtype;
    a.K = w->K;
    a.n_sl = w->n_slices;
    a.L = w->L;
    a.r_max = w->r_max;
    a.M = M;
    a.s_max = std::min(w->L, M);
    a.cols = w->n_slices * w->r_max;
    for (int s = 0; s <= w->n_slices; ++s) a.slice_off[s] = w->slice_offsets[s];
    a.A = w->A;
    a.B = w->B;
    a.a_off = w->a_off;
    a.b_off = w->b_off;
    a.rank = w->rank;
    a.sorted_idx = seg->sorted_idx;
    a.seg_indptr = seg->seg_indptr;
    a.req_to_lora = seg->req_to_lora;
    a.num_segments = seg->num_segments;
    a.tile_info = seg->tile_info;
    a.tile_rows = seg->tile_rows;
    a.num_tiles = seg->num_tiles;
    a.max_tiles = seg->max_tiles;
    return a;
}

LinearWs layout_for(const lora_weights_t* w, int M) {
    return linear_ws_layout(M, w->K, w->n_slices * w->r_max);
}

}  // namespace

namespace mlora {

// header | decode slots [Cd][64][cols] | shrink partials [C][M][cols] |
// S [M][cols], with Cd = ceil(K / kDecKChunk) and C = ceil(K / kKChunk).
// The header and decode region do not depend on M, so calls of any M may
// share one workspace.
LinearWs linear_ws_layout(int M, int K, int cols) {
    LinearWs ws{};
    const size_t C = (size_t)kchunks(K);
    const size_t Cd = (size_t)((K + kDecKChunk - 1) / kDecKChunk);
    size_t off = 0;
    ws.header = off;
    off += up(sizeof(WsHeader));
    ws.slots = off;
    off += up(Cd * LORA_DECODE_MAX_M * (size_t)cols * sizeof(slot_t));
    ws.partial = off;
    off += up(C * (size_t)M * cols * sizeof(float));
    ws.S = off;
    off += up((size_t)M * cols * sizeof(float));
    ws.total = off;
    return ws;
}

MoeWs moe_ws_layout(int L, int mtp, int r, int Kmax) {
    MoeWs ws{};
    // partials: fp32 values per K chunk of kKChunk (fp32 path), or 8-byte
    // tagged exchange slots per K chunk of 1024 (bf16 path)
    const size_t C = (size_t)kchunks(Kmax);
    const size_t C8 = (size_t)(Kmax + 1023) / 1024;
    const size_t rows = (size_t)L * mtp;
    size_t off = 0;
    ws.header = off;
    off += up(sizeof(WsHeader));
    ws.partial = off;
    off += up(std::max(C * sizeof(float), C8 * sizeof(uint64_t)) * rows * r);
    ws.S = off;
    off += up(rows * r * sizeof(float));
    ws.total = off;
    return ws;
}

// Host-side checks of the single-launch decode's arguments other than the
// workspace (w already checked, 0 <= M <= LORA_DECODE_MAX_M).
lora_status fused_decode_check(const lora_weights_t* w, const int32_t* ids, const void* x,
                               int64_t ldx, int32_t M, void* y, int64_t ldy, int32_t* sorted_idx,
                               int32_t* seg_indptr, int32_t* req_to_lora, int32_t* num_segments,
                               int32_t* tile_info, int32_t* tile_rows, int32_t* num_tiles,
                               int32_t max_tiles) {
    lora_status st;
    if (sorted_idx) {
        if (!seg_indptr || !req_to_lora || !num_segments || !tile_info || !tile_rows || !num_tiles)
            return LORA_INVALID_ARG;
        if (max_tiles < lora_tile_capacity(M, w->L)) return LORA_INVALID_ARG;
    }
    if (M == 0) return LORA_OK;
    if (!ids) return LORA_INVALID_ARG;
    if ((st = check_rows(x, ldx, w->K)) != LORA_OK) return st;
    return check_rows(y, ldy, n_total(w));
}

// Launch of the single-launch decode (arguments checked by
// fused_decode_check), shared by lora_fused_decode and its allocation-free
// form; `ws` is an exchange workspace already known to be large enough and
// errors go to `err` (null: the workspace's own error word).
lora_status fused_decode(const lora_weights_t* w, const int32_t* ids,
                         const int32_t* adapter_enabled, const void* x, int64_t ldx, int32_t M,
                         void* y, int64_t ldy, int32_t* sorted_idx, int32_t* seg_indptr,
                         int32_t* req_to_lora, int32_t* num_segments, int32_t* tile_info,
                         int32_t* tile_rows, int32_t* num_tiles, int32_t max_tiles, void* ws,
                         int32_t* err, hipStream_t stream) {
    const bool table = sorted_idx != nullptr;
    if (M == 0) {
        if (!table) return LORA_OK;
        return from_hip(launch_build_segments(nullptr, nullptr, 0, w->L, sorted_idx, seg_indptr,
                                              req_to_lora, num_segments, tile_info, tile_rows,
                                              num_tiles, max_tiles, stream));
    }
    // segment-table fields of the args are unused in ids mode
    lora_segments_t none{};
    LinearArgs a = make_args(w, &none, M);
    const SegOut out{sorted_idx, seg_indptr, req_to_lora, num_segments, tile_info, tile_rows,
                     num_tiles};
    return from_hip(launch_decode_fused(a, ids, adapter_enabled, out, x, ldx, y, ldy, ws, err,
                                        stream));
}

}  // namespace mlora

extern "C" {

int32_t lora_abi_version(void) { return MLORA_ABI_VERSION; }

const char* lora_status_string(lora_status s) {
    switch (s) {
        case LORA_OK: return "ok";
        case LORA_INVALID_ARG: return "invalid argument";
        case LORA_UNSUPPORTED: return "unsupported shape or option";
        case LORA_HIP_ERROR: return "HIP launch error";
    }
    return "unknown status";
}

size_t lora_workspace_size(const lora_weights_t* w, int32_t M) {
    if (check_weights(w) != LORA_OK || M < 0) return 0;
    return layout_for(w, M).total;
}

lora_status lora_workspace_init(void* workspace, size_t bytes, hipStream_t stream) {
    const Range range("lora_workspace_init");
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1))) return LORA_INVALID_ARG;
    return from_hip(launch_fill_zero(workspace, bytes, stream));
}

lora_status lora_read_device_error(void* workspace, int32_t* out, hipStream_t stream) {
    const Range range("lora_read_device_error");
    if (!workspace || !out) return LORA_INVALID_ARG;
    int v = 0;
    hipError_t e = hipMemcpyAsync(&v, workspace, sizeof(int), hipMemcpyDeviceToHost, stream);
    if (e == hipSuccess) e = hipStreamSynchronize(stream);
    if (e != hipSuccess) return LORA_HIP_ERROR;
    *out = v;
    if (v != 0) {
        e = launch_fill_zero(workspace, sizeof(int), stream);
        if (e == hipSuccess) e = hipStreamSynchronize(stream);
        if (e != hipSuccess) return LORA_HIP_ERROR;
    }
    return LORA_OK;
}

lora_status lora_table_plan(int32_t L, const int32_t* ranks, int32_t n_slices, int32_t K,
                            int64_t N_total, int32_t* rank_pad, int64_t* a_off, int64_t* b_off,
                            int64_t* a_elems, int64_t* b_elems) {
    if (L < 1 || L > LORA_MAX_ADAPTERS || !ranks || !rank_pad || !a_off || !b_off || !a_elems ||
        !b_elems)
        return LORA_INVALID_ARG;
    if (n_slices < 1 || n_slices > LORA_MAX_SLICES || K <= 0 || K % 8 || N_total <= 0 ||
        N_total % 8)
        return LORA_INVALID_ARG;
    for (int i = 0; i < L; ++i)
        if (ranks[i] < 0 || ranks[i] > LORA_MAX_RANK) return LORA_INVALID_ARG;
    for (int i = 0; i < L; ++i)
        rank_pad[i] = (ranks[i] + LORA_RANK_ALIGN - 1) / LORA_RANK_ALIGN * LORA_RANK_ALIGN;
    // rank-group major: every slot of padded rank 16, then 32, 48, 64; slots
    // in index order inside a group
    int64_t ao = 0, bo = 0;
    for (int rp = LORA_RANK_ALIGN; rp <= LORA_MAX_RANK; rp += LORA_RANK_ALIGN) {
        for (int i = 0; i < L; ++i) {
            if (rank_pad[i] != rp) continue;
            a_off[i] = ao;
            b_off[i] = bo;
            ao += (int64_t)n_slices * rp * K;
            bo += N_total * rp;
        }
    }
    for (int i = 0; i < L; ++i)
        if (rank_pad[i] == 0) a_off[i] = b_off[i] = 0;
    *a_elems = ao;
    *b_elems = bo;
    return LORA_OK;
}

lora_status lora_pack_adapter(int32_t dtype, int32_t K, int64_t N_total, int32_t n_slices,
                              int32_t rank, int32_t rank_pad, const void* A_src,
                              const void* B_src, void* A_dst, void* B_dst, hipStream_t stream) {
    const Range range("lora_pack_adapter");
    if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (K <= 0 || N_total <= 0 || n_slices < 1 || n_slices > LORA_MAX_SLICES) return LORA_INVALID_ARG;
    if (rank < 0 || rank > LORA_MAX_RANK) return LORA_INVALID_ARG;
    if (rank_pad != (rank + LORA_RANK_ALIGN - 1) / LORA_RANK_ALIGN * LORA_RANK_ALIGN)
        return LORA_INVALID_ARG;
    if (rank == 0) return LORA_OK;
    if (!A_src || !B_src || !A_dst || !B_dst) return LORA_INVALID_ARG;
    return from_hip(launch_pack_adapter(dtype, K, N_total, n_slices, rank, rank_pad, A_src, B_src,
                                        A_dst, B_dst, stream));
}

int32_t lora_tile_capacity(int32_t M, int32_t L) {
    if (M < 0 || L < 1) return 0;
    return M / LORA_TILE_ROWS + std::min(L, M);
}

lora_status lora_build_segments(const int32_t* ids, const int32_t* adapter_enabled, int32_t M,
                                int32_t L, int32_t* sorted_idx, int32_t* seg_indptr,
                                int32_t* req_to_lora, int32_t* num_segments, int32_t* tile_info,
                                int32_t* tile_rows, int32_t* num_tiles, int32_t max_tiles,
                                hipStream_t stream) {
    const Range range("lora_build_segments");
    if (M < 0 || M > (1 << 24) || L < 1 || L > LORA_MAX_ADAPTERS) return LORA_INVALID_ARG;
    if (!seg_indptr || !req_to_lora || !num_segments || !num_tiles) return LORA_INVALID_ARG;
    if (max_tiles < lora_tile_capacity(M, L)) return LORA_INVALID_ARG;
    if (M > 0 && (!ids || !sorted_idx || !tile_info || !tile_rows)) return LORA_INVALID_ARG;
    return from_hip(launch_build_segments(ids, adapter_enabled, M, L, sorted_idx, seg_indptr,
                                          req_to_lora, num_segments, tile_info, tile_rows,
                                          num_tiles, max_tiles, stream));
}

lora_status lora_shrink(const lora_weights_t* w, const void* x, int64_t ldx, int32_t M,
                        const lora_segments_t* seg, float* S, void* workspace,
                        size_t workspace_bytes, hipStream_t stream) {
    const Range range("lora_shrink");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (M < 0 || M > (1 << 24)) return LORA_INVALID_ARG;
    if ((st = check_segments(seg, w, M)) != LORA_OK) return st;
    if (M == 0) return LORA_OK;
    if ((st = check_rows(x, ldx, w->K)) != LORA_OK) return st;
    if (!S || !aligned16(S)) return LORA_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)))
        return LORA_INVALID_ARG;
    if (workspace_bytes < layout_for(w, M).total) return LORA_INVALID_ARG;
    LinearArgs a = make_args(w, seg, M);
    a.err = ws_error(workspace);
    return from_hip(launch_shrink(a, x, ldx, S, workspace, stream));
}

lora_status lora_expand_add(const lora_weights_t* w, const float* S, int32_t M,
                            const lora_segments_t* seg, void* y, int64_t ldy,
                            hipStream_t stream) {
    const Range range("lora_expand_add");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (M < 0 || M > (1 << 24)) return LORA_INVALID_ARG;
    if ((st = check_segments(seg, w, M)) != LORA_OK) return st;
    if (M == 0) return LORA_OK;
    if (!S || !aligned16(S)) return LORA_INVALID_ARG;
    if ((st = check_rows(y, ldy, n_total(w))) != LORA_OK) return st;
    const LinearArgs a = make_args(w, seg, M);
    return from_hip(launch_expand(a, S, y, ldy, stream));
}

lora_status lora_shrink_expand_add(const lora_weights_t* w, const void* x, int64_t ldx,
                                   int32_t M, const lora_segments_t* seg, void* y, int64_t ldy,
                                   void* workspace, size_t workspace_bytes, hipStream_t stream) {
    const Range range("lora_shrink_expand_add");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (M < 0 || M > (1 << 24)) return LORA_INVALID_ARG;
    if ((st = check_segments(seg, w, M)) != LORA_OK) return st;
    if (M == 0) return LORA_OK;
    if ((st = check_rows(x, ldx, w->K)) != LORA_OK) return st;
    if ((st = check_rows(y, ldy, n_total(w))) != LORA_OK) return st;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)))
        return LORA_INVALID_ARG;
    const LinearWs L = layout_for(w, M);
    if (workspace_bytes < L.total) return LORA_INVALID_ARG;
    LinearArgs a = make_args(w, seg, M);
    a.err = ws_error(workspace);
    if (M <= LORA_DECODE_MAX_M)
        return from_hip(launch_decode_fused(a, nullptr, nullptr, SegOut{}, x, ldx, y, ldy,
                                            workspace, nullptr, stream));
    float* S = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + L.S);
    hipError_t e = launch_shrink(a, x, ldx, S, workspace, stream);
    if (e != hipSuccess) return LORA_HIP_ERROR;
    return from_hip(launch_expand(a, S, y, ldy, stream));
}

lora_status lora_linear_fused(const lora_weights_t* w, const void* W, int64_t ldw,
                              const void* x, int64_t ldx, int32_t M, const lora_segments_t* seg,
                              void* y, int64_t ldy, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    const Range range("lora_linear_fused");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (w->dtype != LORA_BF16) return LORA_UNSUPPORTED;
    if (M < 0 || M > (1 << 24)) return LORA_INVALID_ARG;
    if ((st = check_segments(seg, w, M)) != LORA_OK) return st;
    if (M == 0) return LORA_OK;
    if ((st = check_rows(W, ldw, w->K)) != LORA_OK) return st;
    if ((st = check_rows(x, ldx, w->K)) != LORA_OK) return st;
    if ((st = check_rows(y, ldy, n_total(w))) != LORA_OK) return st;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)))
        return LORA_INVALID_ARG;
    const LinearWs L = layout_for(w, M);
    if (workspace_bytes < L.total) return LORA_INVALID_ARG;
    LinearArgs a = make_args(w, seg, M);
    a.err = ws_error(workspace);
    float* S = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + L.S);
    hipError_t e = launch_shrink(a, x, ldx, S, workspace, stream);
    if (e != hipSuccess) return LORA_HIP_ERROR;
    return from_hip(launch_gemm_lora(a, x, ldx, W, ldw, S, y, ldy, stream));
}

lora_status lora_fused_decode(const lora_weights_t* w, const int32_t* ids,
                              const int32_t* adapter_enabled, const void* x, int64_t ldx,
                              int32_t M, void* y, int64_t ldy, int32_t* sorted_idx,
                              int32_t* seg_indptr, int32_t* req_to_lora, int32_t* num_segments,
                              int32_t* tile_info, int32_t* tile_rows, int32_t* num_tiles,
                              int32_t max_tiles, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    const Range range("lora_fused_decode");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (M < 0) return LORA_INVALID_ARG;
    if (M > LORA_DECODE_MAX_M) return LORA_UNSUPPORTED;
    if ((st = fused_decode_check(w, ids, x, ldx, M, y, ldy, sorted_idx, seg_indptr, req_to_lora,
                                 num_segments, tile_info, tile_rows, num_tiles, max_tiles)) !=
        LORA_OK)
        return st;
    if (M > 0 && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)) ||
                  workspace_bytes < layout_for(w, M).total))
        return LORA_INVALID_ARG;
    return fused_decode(w, ids, adapter_enabled, x, ldx, M, y, ldy, sorted_idx, seg_indptr,
                        req_to_lora, num_segments, tile_info, tile_rows, num_tiles, max_tiles,
                        workspace, nullptr, stream);
}

lora_status lora_fused_decode_noalloc(const lora_weights_t* w, const int32_t* ids,
                                      const int32_t* adapter_enabled, const void* x, int64_t ldx,
                                      int32_t M, void* y, int64_t ldy, int32_t* sorted_idx,
                                      int32_t* seg_indptr, int32_t* req_to_lora,
                                      int32_t* num_segments, int32_t* tile_info,
                                      int32_t* tile_rows, int32_t* num_tiles, int32_t max_tiles,
                                      int32_t* error_word, hipStream_t stream) {
    const Range range("lora_fused_decode_noalloc");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (M < 0) return LORA_INVALID_ARG;
    if (M > LORA_DECODE_MAX_M) return LORA_UNSUPPORTED;
    // header and exchange slots (M plays no part) must fit the fixed array
    if (layout_for(w, 0).total > (size_t)LORA_NOALLOC_SCRATCH_BYTES) return LORA_UNSUPPORTED;
    if ((st = fused_decode_check(w, ids, x, ldx, M, y, ldy, sorted_idx, seg_indptr, req_to_lora,
                                 num_segments, tile_info, tile_rows, num_tiles, max_tiles)) !=
        LORA_OK)
        return st;
    void* scratch = nullptr;
    if (M > 0 && noalloc_scratch(&scratch) != hipSuccess) return LORA_HIP_ERROR;
    return fused_decode(w, ids, adapter_enabled, x, ldx, M, y, ldy, sorted_idx, seg_indptr,
                        req_to_lora, num_segments, tile_info, tile_rows, num_tiles, max_tiles,
                        scratch, error_word, stream);
}

lora_status lora_pack_embedding_adapter(int32_t dtype, int32_t vocab, int64_t emb, int32_t rank,
                                        int32_t rank_pad, const void* A_src, const void* B_src,
                                        void* A_dst, void* B_dst, hipStream_t stream) {
    const Range range("lora_pack_embedding_adapter");
    if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (vocab <= 0 || vocab % 8 || emb <= 0 || emb % 8) return LORA_INVALID_ARG;
    if (rank < 0 || rank > LORA_MAX_RANK) return LORA_INVALID_ARG;
    if (rank_pad != (rank + LORA_RANK_ALIGN - 1) / LORA_RANK_ALIGN * LORA_RANK_ALIGN)
        return LORA_INVALID_ARG;
    if (rank == 0) return LORA_OK;
    if (!A_src || !B_src || !A_dst || !B_dst) return LORA_INVALID_ARG;
    return from_hip(launch_pack_embedding_adapter(dtype, vocab, emb, rank, rank_pad, A_src, B_src,
                                                  A_dst, B_dst, stream));
}

lora_status lora_embedding_shrink(const lora_weights_t* w, const int32_t* tokens, int32_t M,
                                  const lora_segments_t* seg, float* S, hipStream_t stream) {
    const Range range("lora_embedding_shrink");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (w->n_slices != 1) return LORA_INVALID_ARG;
    if (M < 0 || M > (1 << 24)) return LORA_INVALID_ARG;
    if ((st = check_segments(seg, w, M)) != LORA_OK) return st;
    if (M == 0) return LORA_OK;
    if (!tokens || !S || !aligned16(S)) return LORA_INVALID_ARG;
    const LinearArgs a = make_args(w, seg, M);
    return from_hip(launch_embedding_shrink(a, tokens, S, stream));
}

lora_status lora_embedding_decode(const lora_weights_t* w, const int32_t* ids,
                                  const int32_t* adapter_enabled, const int32_t* tokens,
                                  int32_t M, void* y, int64_t ldy, int32_t* sorted_idx,
                                  int32_t* seg_indptr, int32_t* req_to_lora,
                                  int32_t* num_segments, int32_t* tile_info, int32_t* tile_rows,
                                  int32_t* num_tiles, int32_t max_tiles, hipStream_t stream) {
    const Range range("lora_embedding_decode");
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (w->n_slices != 1) return LORA_INVALID_ARG;
    if (M < 0) return LORA_INVALID_ARG;
    if (M > LORA_DECODE_MAX_M) return LORA_UNSUPPORTED;
    const bool table = sorted_idx != nullptr;
    if (table) {
        if (!seg_indptr || !req_to_lora || !num_segments || !tile_info || !tile_rows || !num_tiles)
            return LORA_INVALID_ARG;
        if (max_tiles < lora_tile_capacity(M, w->L)) return LORA_INVALID_ARG;
    }
    if (M == 0) {
        if (!table) return LORA_OK;
        return from_hip(launch_build_segments(nullptr, nullptr, 0, w->L, sorted_idx, seg_indptr,
                                              req_to_lora, num_segments, tile_info, tile_rows,
                                              num_tiles, max_tiles, stream));
    }
    if (!ids || !tokens) return LORA_INVALID_ARG;
    if ((st = check_rows(y, ldy, n_total(w))) != LORA_OK) return st;
    lora_segments_t none{};
    const LinearArgs a = make_args(w, &none, M);
    const SegOut out{sorted_idx, seg_indptr, req_to_lora, num_segments, tile_info, tile_rows,
                     num_tiles};
    return from_hip(launch_embedding_decode(a, ids, adapter_enabled, tokens, out, y, ldy, stream));
}

// ------------------------------------------------------------------ MoE
int32_t lora_moe_align_capacity(int32_t M, int32_t topk, int32_t E, int32_t block_size_m) {
    if (M < 0 || topk < 1 || E < 1 || block_size_m < 1) return 0;
    const int64_t cap = (int64_t)M * topk + (int64_t)E * (block_size_m - 1);
    const int64_t r = (cap + block_size_m - 1) / block_size_m * block_size_m;
    return r > INT32_MAX ? 0 : (int32_t)r;
}

static lora_status check_align(const lora_moe_align_t* al, int M, int topk, int E) {
    if (!al || !al->sorted_token_ids || !al->expert_ids || !al->ntpp) return LORA_INVALID_ARG;
    const int bs = al->block_size_m;
    if (bs < 16 || bs > 256 || bs % 16) return LORA_INVALID_ARG;
    if (al->max_tokens_padded % bs) return LORA_INVALID_ARG;
    if (al->max_tokens_padded < lora_moe_align_capacity(M, topk, E, bs)) return LORA_INVALID_ARG;
    return LORA_OK;
}

static lora_status check_moe_weights(const lora_moe_weights_t* w) {
    if (!w) return LORA_INVALID_ARG;
    if (w->dtype != LORA_F32 && w->dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (w->L < 1 || w->L > LORA_MAX_ADAPTERS || w->E < 1 || w->E > 256) return LORA_INVALID_ARG;
    if (w->H <= 0 || w->H % 8 || w->I <= 0 || w->I % 8) return LORA_INVALID_ARG;
    if (w->r < LORA_RANK_ALIGN || w->r > LORA_MAX_RANK || w->r % LORA_RANK_ALIGN) return LORA_INVALID_ARG;
    if (!w->A_gu || !w->B_gu || !w->A_d || !w->B_d || !w->adapter_enabled) return LORA_INVALID_ARG;
    if (!aligned16(w->A_gu) || !aligned16(w->B_gu) || !aligned16(w->A_d) || !aligned16(w->B_d))
        return LORA_INVALID_ARG;
    return LORA_OK;
}

lora_status lora_moe_align(const int32_t* topk_ids, const int32_t* ids,
                           const int32_t* adapter_enabled, int32_t M, int32_t topk, int32_t E,
                           int32_t L, int32_t block_size_m, int32_t max_tokens_padded,
                           int32_t* sorted_token_ids, int32_t* expert_ids, int32_t* ntpp,
                           hipStream_t stream) {
    const Range range("lora_moe_align");
    if (M < 0 || topk < 1 || topk > 16 || E < 1 || E > 256 || L < 1 || L > LORA_MAX_ADAPTERS)
        return LORA_INVALID_ARG;
    if ((int64_t)M * topk > (1 << 24)) return LORA_INVALID_ARG;
    if (!adapter_enabled) return LORA_INVALID_ARG;
    if (M > 0 && (!topk_ids || !ids)) return LORA_INVALID_ARG;
    const lora_moe_align_t out{sorted_token_ids, expert_ids, ntpp, max_tokens_padded,
                               block_size_m};
    lora_status st = check_align(&out, M, topk, E);
    if (st != LORA_OK) return st;
    return from_hip(launch_moe_align(topk_ids, ids, adapter_enabled, M, topk, E, L,
                                     sorted_token_ids, expert_ids, ntpp, max_tokens_padded,
                                     block_size_m, stream));
}

size_t lora_moe_workspace_size(const lora_moe_weights_t* w, int32_t max_tokens_padded) {
    if (check_moe_weights(w) != LORA_OK || max_tokens_padded < 0) return 0;
    return moe_ws_layout(w->L, max_tokens_padded, w->r, std::max(w->H, w->I)).total;
}

static MoeArgs make_moe(const lora_moe_weights_t* w, int M, int topk, const lora_moe_align_t* al) {
    MoeArgs a{};
    a.dtype = w->dtype;
    a.L = w->L; a.E = w->E; a.H = w->H; a.I = w->I; a.r = w->r;
    a.shared_outer = w->shared_outer != 0;
    a.M = M; a.topk = topk;
    a.max_tokens_padded = al->max_tokens_padded;
    a.block_size_m = al->block_size_m;
    a.A_gu = w->A_gu; a.B_gu = w->B_gu; a.A_d = w->A_d; a.B_d = w->B_d;
    a.adapter_enabled = w->adapter_enabled;
    a.sorted_token_ids = al->sorted_token_ids;
    a.expert_ids = al->expert_ids;
    a.ntpp = al->ntpp;
    return a;
}

static lora_status moe_delta(const lora_moe_weights_t* w, int which, const void* in, int64_t ld_in,
                             int32_t M, int32_t topk, const lora_moe_align_t* al, void* out,
                             int64_t ld_out, void* ws, size_t ws_bytes, hipStream_t stream) {
    lora_status st = check_moe_weights(w);
    if (st != LORA_OK) return st;
    if (M < 0 || topk < 1 || topk > 16 || (int64_t)M * topk > (1 << 24)) return LORA_INVALID_ARG;
    if ((st = check_align(al, M, topk, w->E)) != LORA_OK) return st;
    if (M == 0) return LORA_OK;
    const int K = which == 0 ? w->H : w->I;
    const int N = which == 0 ? 2 * w->I : w->H;
    if ((st = check_rows(in, ld_in, K)) != LORA_OK) return st;
    if ((st = check_rows(out, ld_out, N)) != LORA_OK) return st;
    if (!ws || (reinterpret_cast<uintptr_t>(ws) & (kAlign - 1))) return LORA_INVALID_ARG;
    if (ws_bytes < lora_moe_workspace_size(w, al->max_tokens_padded)) return LORA_INVALID_ARG;
    const MoeArgs a = make_moe(w, M, topk, al);
    return from_hip(launch_moe_delta(a, which, in, ld_in, out, ld_out, ws, stream));
}

lora_status lora_moe_gate_up_add(const lora_moe_weights_t* w, const void* x, int64_t ldx,
                                 int32_t M, int32_t topk, const lora_moe_align_t* align,
                                 void* cache1, int64_t ld1, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream) {
    const Range range("lora_moe_gate_up_add");
    return moe_delta(w, 0, x, ldx, M, topk, align, cache1, ld1, workspace, workspace_bytes, stream);
}

lora_status lora_moe_down_add(const lora_moe_weights_t* w, const void* cache2, int64_t ld2,
                              int32_t M, int32_t topk, const lora_moe_align_t* align,
                              void* cache3, int64_t ld3, void* workspace, size_t workspace_bytes,
                              hipStream_t stream) {
    const Range range("lora_moe_down_add");
    return moe_delta(w, 1, cache2, ld2, M, topk, align, cache3, ld3, workspace, workspace_bytes,
                     stream);
}

lora_status lora_moe_silu_and_mul(int32_t dtype, const void* cache1, int64_t ld1, void* cache2,
                                  int64_t ld2, int32_t P, int32_t I, hipStream_t stream) {
    const Range range("lora_moe_silu_and_mul");
    if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (P < 0 || I <= 0 || I % 8) return LORA_INVALID_ARG;
    if (P == 0) return LORA_OK;
    lora_status st = check_rows(cache1, ld1, 2 * (int64_t)I);
    if (st != LORA_OK) return st;
    if ((st = check_rows(cache2, ld2, I)) != LORA_OK) return st;
    return from_hip(launch_silu_and_mul(dtype, cache1, ld1, cache2, ld2, P, I, stream));
}

lora_status lora_moe_topk_reduce(int32_t dtype, const void* cache3, int64_t ld3,
                                 const float* topk_weights, void* out, int64_t ldo, int32_t M,
                                 int32_t topk, int32_t H, hipStream_t stream) {
    const Range range("lora_moe_topk_reduce");
    if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (M < 0 || topk < 1 || topk > 16 || H <= 0 || H % 8) return LORA_INVALID_ARG;
    if (M == 0) return LORA_OK;
    if (!topk_weights) return LORA_INVALID_ARG;
    lora_status st = check_rows(cache3, ld3, H);
    if (st != LORA_OK) return st;
    if ((st = check_rows(out, ldo, H)) != LORA_OK) return st;
    return from_hip(launch_topk_reduce(dtype, cache3, ld3, topk_weights, out, ldo, M, topk, H,
                                       stream));
}

// ------------------------------------------------------------------ 8-bit decoder layer
static lora_status rms_norm(int int8, int32_t dtype, const void* x, int64_t ldx, const void* residual, int64_t ldr,
                            const void* weight, float eps, int32_t M, int32_t K, void* residual_out, int64_t ldro,
                            void* out, int64_t ldo, void* out8, int64_t ldo8, float* scale, hipStream_t stream) {
    if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (M < 0 || K <= 0 || K % 8) return LORA_INVALID_ARG;
    if (K > kNormMaxK) return LORA_UNSUPPORTED;
    if (M == 0) return LORA_OK;
    if ((!out && !out8) || !scale != !out8 || (residual_out && !residual)) return LORA_INVALID_ARG;
    if (int8 && !out8) return LORA_INVALID_ARG;
    if (!(eps >= 0.f)) return LORA_INVALID_ARG;
    lora_status st = check_rows(x, ldx, K);
    if (st == LORA_OK) st = check_rows(weight, K, K);
    if (st == LORA_OK && residual) st = check_rows(residual, ldr, K);
    if (st == LORA_OK && residual_out) st = check_rows(residual_out, ldro, K);
    if (st == LORA_OK && out) st = check_rows(out, ldo, K);
    if (st == LORA_OK && out8) st = check_rows(out8, ldo8, K);
    if (st != LORA_OK) return st;
    const NormParams p{x, ldx, residual, ldr, residual_out, ldro, weight, eps, out, ldo,
                       static_cast<uint8_t*>(out8), ldo8, scale, M, K, int8};
    return from_hip(launch_rms_norm(dtype, p, stream));
}

static lora_status quantize_rows(int int8, int32_t dtype, const void* x, int64_t ldx, int32_t M, int32_t K, void* out8,
                                 int64_t ldo8, float* scale, hipStream_t stream) {
    if (dtype != LORA_F32 && dtype != LORA_BF16) return LORA_INVALID_ARG;
    if (M < 0 || K <= 0 || K % 8) return LORA_INVALID_ARG;
    if (K > kNormMaxK) return LORA_UNSUPPORTED;
    if (M == 0) return LORA_OK;
    lora_status st = check_rows(x, ldx, K);
    if (st == LORA_OK) st = check_rows(out8, ldo8, K);
    if (st != LORA_OK) return st;
    if (!scale) return LORA_INVALID_ARG;
    const NormParams p{x, ldx, nullptr, 0, nullptr, 0, nullptr, 0.f, nullptr, 0,
                       static_cast<uint8_t*>(out8), ldo8, scale, M, K, int8};
    return from_hip(launch_rms_norm(dtype, p, stream));
}

lora_status lora_rms_norm(int32_t dtype, const void* x, int64_t ldx, const void* residual,
                          int64_t ldr, const void* weight, float eps, int32_t M, int32_t K,
                          void* residual_out, int64_t ldro, void* out, int64_t ldo, void* out8,
                          int64_t ldo8, float* scale, hipStream_t stream) {
    const Range range("lora_rms_norm");
    return rms_norm(0, dtype, x, ldx, residual, ldr, weight, eps, M, K, residual_out, ldro, out, ldo, out8,
                    ldo8, scale, stream);
}

lora_status lora_quantize_rows(int32_t dtype, const void* x, int64_t ldx, int32_t M, int32_t K,
                               void* out8, int64_t ldo8, float* scale, hipStream_t stream) {
    const Range range("lora_quantize_rows");
    return quantize_rows(0, dtype, x, ldx, M, K, out8, ldo8, scale, stream);
}

lora_status lora_rms_norm_int8(int32_t dtype, const void* x, int64_t ldx, const void* residual,
                               int64_t ldr, const void* weight, float eps, int32_t M, int32_t K,
                               void* residual_out, int64_t ldro, void* out, int64_t ldo, void* out8,
                               int64_t ldo8, float* scale, hipStream_t stream) {
    const Range range("lora_rms_norm_int8");
    return rms_norm(1, dtype, x, ldx, residual, ldr, weight, eps, M, K, residual_out, ldro, out, ldo, out8,
                    ldo8, scale, stream);
}

lora_status lora_quantize_rows_int8(int32_t dtype, const void* x, int64_t ldx, int32_t M, int32_t K,
                                    void* out8, int64_t ldo8, float* scale, hipStream_t stream) {
    const Range range("lora_quantize_rows_int8");
    return quantize_rows(1, dtype, x, ldx, M, K, out8, ldo8, scale, stream);
}

// rows that are addressed with 32-bit byte offsets
static bool below_2gib(int64_t rows, int64_t ld, int bytes) { return ld < (int64_t)INT32_MAX / bytes / rows; }

// rows of 8-bit values read 16 bytes at a time
static lora_status check_rows8(const void* p, int64_t ld, int64_t width) {
    if (!p || !aligned16(p) || ld < width || ld % 16 != 0) return LORA_INVALID_ARG;
    return LORA_OK;
}

// sums of products of two 8-bit integers (-128 among them) stay within 32 bits
constexpr int kInt8MaxK = 131056;

static lora_status linear_8bit(bool int8, const lora_weights_t* w, const void* W8, int64_t ldw, const float* w_scale,
                               const void* x8, int64_t ldx8, const float* x_scale, const void* x, int64_t ldx,
                               int32_t M, const lora_segments_t* seg, void* y, int64_t ldy, void* workspace,
                               size_t workspace_bytes, hipStream_t stream) {
    lora_status st = check_weights(w);
    if (st != LORA_OK) return st;
    if (w->dtype != LORA_BF16 || w->K % 16) return LORA_UNSUPPORTED;
    if (int8 && w->K > kInt8MaxK) return LORA_UNSUPPORTED;
    if (M < 0 || M > (1 << 24)) return LORA_INVALID_ARG;
    if ((st = check_segments(seg, w, M)) != LORA_OK) return st;
    if (M == 0) return LORA_OK;
    if ((st = check_rows8(W8, ldw, w->K)) != LORA_OK) return st;
    if ((st = check_rows8(x8, ldx8, w->K)) != LORA_OK) return st;
    if ((st = check_rows(x, ldx, w->K)) != LORA_OK) return st;
    if ((st = check_rows(y, ldy, n_total(w))) != LORA_OK) return st;
    if (!w_scale || !x_scale) return LORA_INVALID_ARG;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)))
        return LORA_INVALID_ARG;
    const LinearWs L = layout_for(w, M);
    if (workspace_bytes < L.total) return LORA_INVALID_ARG;
    LinearArgs a = make_args(w, seg, M);
    a.err = ws_error(workspace);
    if (M <= LORA_DECODE_MAX_M) {
        // 32-bit offsets over the token rows, 32 rows of W8 and 16 (bf16) of A
        if (!below_2gib(M, ldx, 2) || !below_2gib(M, ldx8, 1) || !below_2gib(32, ldw, 1))
            return LORA_UNSUPPORTED;
        return from_hip(launch_linear_8bit(int8, a, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, y, ldy,
                                           workspace, stream));
    }
    float* S = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + L.S);
    if (!below_2gib(256, ldw, 1)) return LORA_UNSUPPORTED;     // 256 rows of W8
    return from_hip(launch_linear_8bit_many(int8, a, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, S, y, ldy,
                                            workspace, stream));
}

lora_status lora_linear_fp8(const lora_weights_t* w, const void* W8, int64_t ldw,
                            const float* w_scale, const void* x8, int64_t ldx8,
                            const float* x_scale, const void* x, int64_t ldx, int32_t M,
                            const lora_segments_t* seg, void* y, int64_t ldy, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    const Range range("lora_linear_fp8");
    return linear_8bit(false, w, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, M, seg, y, ldy, workspace,
                       workspace_bytes, stream);
}

lora_status lora_linear_int8(const lora_weights_t* w, const void* W8, int64_t ldw,
                             const float* w_scale, const void* x8, int64_t ldx8,
                             const float* x_scale, const void* x, int64_t ldx, int32_t M,
                             const lora_segments_t* seg, void* y, int64_t ldy, void* workspace,
                             size_t workspace_bytes, hipStream_t stream) {
    const Range range("lora_linear_int8");
    return linear_8bit(true, w, W8, ldw, w_scale, x8, ldx8, x_scale, x, ldx, M, seg, y, ldy, workspace,
                       workspace_bytes, stream);
}

// ------------------------------------------------------------------ experts' products
static bool pairs_ok(int32_t M, int32_t topk, int32_t E) {
    return M >= 0 && topk >= 1 && topk <= 16 && E >= 1 && E <= 256 && (int64_t)M * topk <= (1 << 24);
}

lora_status lora_moe_group(const int32_t* topk_ids, int32_t M, int32_t topk, int32_t E, int32_t* pairs,
                           int32_t* offsets, hipStream_t stream) {
    const Range range("lora_moe_group");
    if (!pairs_ok(M, topk, E) || !offsets) return LORA_INVALID_ARG;
    if (M > 0 && (!topk_ids || !pairs)) return LORA_INVALID_ARG;
    return from_hip(launch_moe_group(topk_ids, M * topk, E, pairs, offsets, stream));
}

lora_status lora_moe_linear(int32_t wdtype, const void* W, const float* w_scale, int32_t E, int32_t N, int32_t K,
                            const int32_t* pairs, const int32_t* offsets, const void* x, int64_t ldx,
                            const float* x_scale, int32_t M, int32_t topk, int32_t pair_rows, void* y, int64_t ldy,
                            hipStream_t stream) {
    const Range range("lora_moe_linear");
    if (wdtype != LORA_BF16 && wdtype != LORA_E4M3 && wdtype != LORA_INT8) return LORA_INVALID_ARG;
    const bool eight = wdtype != LORA_BF16;
    if (!pairs_ok(M, topk, E)) return LORA_INVALID_ARG;
    if (N <= 0 || N % 8 || K <= 0 || K % (eight ? 16 : 8)) return LORA_INVALID_ARG;
    if (eight != (w_scale != nullptr) || eight != (x_scale != nullptr)) return LORA_INVALID_ARG;
    if (K > kInt8MaxK) return LORA_UNSUPPORTED;      // and 32-bit offsets within 256 rows of W
    if (M == 0) return LORA_OK;
    if (!pairs || !offsets || !W || !aligned16(W)) return LORA_INVALID_ARG;
    lora_status st = eight ? check_rows8(x, ldx, K) : check_rows(x, ldx, K);
    if (st == LORA_OK) st = check_rows(y, ldy, N);
    if (st != LORA_OK) return st;
    const int P = M * topk, wide = eight ? 1 : 2;
    // a grid has fewer than 2^32 threads
    if (((int64_t)P / 256 + std::min(E, P) + 1) * (((int64_t)N + 255) / 256) > (1 << 23)) return LORA_UNSUPPORTED;
    ExpertsParams p{};
    p.W = static_cast<const char*>(W);
    p.w_scale = w_scale;
    p.pairs = pairs;
    p.offsets = offsets;
    p.x = static_cast<const char*>(x);
    p.ldx = ldx * wide;
    p.x_scale = x_scale;
    p.y = static_cast<uint16_t*>(y);
    p.ldy = ldy;
    p.E = E; p.N = N; p.Kb = K * wide; p.P = P;
    p.x_inv = pair_rows || topk == 1 ? 0 : (uint32_t)(((1ull << 32) + topk - 1) / topk);
    p.x_rows = pair_rows ? P : M;
    return from_hip(launch_experts(wdtype, p, stream));
}

static lora_status check_experts(const lora_moe_experts_t* ex, const lora_moe_weights_t* w) {
    if (!ex) return LORA_INVALID_ARG;
    if (ex->wdtype != LORA_BF16 && ex->wdtype != LORA_E4M3) return LORA_INVALID_ARG;
    const int q = ex->wdtype == LORA_E4M3 ? 16 : 8;
    if (ex->E < 1 || ex->E > 256 || ex->topk < 1 || ex->topk > 16 || ex->topk > ex->E)
        return LORA_INVALID_ARG;
    if (ex->H <= 0 || ex->H % q || ex->I <= 0 || ex->I % q) return LORA_INVALID_ARG;
    if (!ex->router || !ex->W_gu || !ex->W_d || !aligned16(ex->router) || !aligned16(ex->W_gu) ||
        !aligned16(ex->W_d))
        return LORA_INVALID_ARG;
    if ((ex->wdtype == LORA_E4M3) != (ex->s_gu != nullptr) || !ex->s_gu != !ex->s_d)
        return LORA_INVALID_ARG;
    // 32-bit offsets within one expert's matrix and over the rows of h
    if (!below_2gib(2 * (int64_t)ex->I, ex->H, 2) ||
        !below_2gib((int64_t)LORA_DECODE_MAX_M * ex->topk, ex->I, 2))
        return LORA_UNSUPPORTED;
    if (!w) return LORA_OK;
    const lora_status st = check_moe_weights(w);
    if (st != LORA_OK) return st;
    if (w->dtype != LORA_BF16) return LORA_UNSUPPORTED;
    return w->E == ex->E && w->H == ex->H && w->I == ex->I ? LORA_OK : LORA_INVALID_ARG;
}

namespace {
// header | routing slots [2][P] | S of gate/up [P][r] | S of down [P][r] | joined
// partial sums [splits - 1][M][H] of the M with most | chosen experts [P] | h [M
// topk][I], with P = 64 topk.  The slot regions do not depend on M, so calls of any M may share a
// workspace: no plain value ever stands where another call looks for a tag.
struct MoeDecodeWs {
    size_t route, s_gu, s_d, join, ids, h, total;
};

MoeDecodeWs moe_decode_ws(const lora_moe_experts_t* ex, int r, int M) {
    MoeDecodeWs l{};
    const size_t P = (size_t)LORA_DECODE_MAX_M * ex->topk;
    size_t off = up(sizeof(WsHeader));
    auto take = [&off](size_t bytes) {
        const size_t at = off;
        off += up(bytes);
        return at;
    };
    l.route = take(2 * P * sizeof(slot_t));
    l.s_gu = take(P * r * sizeof(slot_t));
    l.s_d = take(P * r * sizeof(slot_t));
    const size_t few = (size_t)(moe_decode_max_splits(ex->H, 32) - 1) * 32;
    const size_t many = (size_t)(moe_decode_max_splits(ex->H, LORA_DECODE_MAX_M) - 1) * LORA_DECODE_MAX_M;
    l.join = take(std::max(few, many) * ex->H * sizeof(slot_t));
    l.ids = take(P * sizeof(int32_t));
    l.h = take((size_t)M * ex->topk * ex->I * sizeof(uint16_t));
    l.total = off;
    return l;
}
}  // namespace

size_t lora_moe_decode_workspace_size(const lora_moe_weights_t* w, const lora_moe_experts_t* ex,
                                      int32_t M) {
    if (check_experts(ex, w) != LORA_OK || M < 0 || M > LORA_DECODE_MAX_M) return 0;
    return moe_decode_ws(ex, w ? w->r : 0, M).total;
}

lora_status lora_moe_decode(const lora_moe_weights_t* w, const lora_moe_experts_t* ex,
                            const int32_t* ids, const void* x, int64_t ldx, int32_t M, void* out,
                            int64_t ldo, int32_t* topk_ids, float* topk_weights, void* workspace,
                            size_t workspace_bytes, hipStream_t stream) {
    const Range range("lora_moe_decode");
    lora_status st = check_experts(ex, w);
    if (st != LORA_OK) return st;
    if (M < 0) return LORA_INVALID_ARG;
    if (M > LORA_DECODE_MAX_M) return LORA_UNSUPPORTED;
    if (M == 0) return LORA_OK;
    if (w && !ids) return LORA_INVALID_ARG;
    if ((st = check_rows(x, ldx, ex->H)) != LORA_OK) return st;
    if ((st = check_rows(out, ldo, ex->H)) != LORA_OK) return st;
    if (!below_2gib(M, ldx, 2)) return LORA_UNSUPPORTED;
    if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & (kAlign - 1)))
        return LORA_INVALID_ARG;
    const MoeDecodeWs l = moe_decode_ws(ex, w ? w->r : 0, M);
    if (workspace_bytes < l.total) return LORA_INVALID_ARG;
    char* ws = static_cast<char*>(workspace);
    auto u16 = [](const void* q) { return static_cast<const uint16_t*>(q); };
    MoeDecodeParams p{};
    p.M = M; p.topk = ex->topk; p.E = ex->E; p.H = ex->H; p.I = ex->I;
    p.renorm = ex->renormalize != 0;
    p.topk_inv = (65536 + ex->topk - 1) / ex->topk;
    p.x = u16(x); p.ldx = ldx;
    p.router = u16(ex->router);
    p.W_gu = ex->W_gu; p.W_d = ex->W_d; p.s_gu = ex->s_gu; p.s_d = ex->s_d;
    if (w) {
        p.L = w->L; p.r = w->r; p.shared_outer = w->shared_outer != 0;
        p.A_gu = u16(w->A_gu); p.B_gu = u16(w->B_gu); p.A_d = u16(w->A_d); p.B_d = u16(w->B_d);
        p.enabled = w->adapter_enabled;
    }
    p.ids = ids;
    p.out = static_cast<uint16_t*>(out); p.ldo = ldo;
    p.out_ids = topk_ids; p.out_w = topk_weights;
    p.err = ws_error(workspace);
    p.route = reinterpret_cast<slot_t*>(ws + l.route);
    p.route_ids = reinterpret_cast<int32_t*>(ws + l.ids);
    p.S_gu = reinterpret_cast<slot_t*>(ws + l.s_gu);
    p.S_d = reinterpret_cast<slot_t*>(ws + l.s_d);
    p.join = reinterpret_cast<slot_t*>(ws + l.join);
    p.h = reinterpret_cast<uint16_t*>(ws + l.h);
    const int64_t row = (int64_t)ex->I * (ex->wdtype == LORA_E4M3 ? 1 : 2);
    p.splits = moe_decode_splits(ex->H, M, (int64_t)std::min(ex->E, M * ex->topk) * ((row + 127) / 128));
    p.wc = wait_ctl();
    return from_hip(launch_moe_decode(p, stream));
}

}  // extern "C"
