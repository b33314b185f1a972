// Host side of the attention operators' C ABI (include/gdn.h): argument
// validation, workspace layout and kernel launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>

#include "gdn.h"
#include "gdn_checks.h"
#include "gdn_kernels.h"

namespace {

using namespace gdn::checks;

gdn_status check_rope(int B, int T, int H, int Hk, int d, int pairs, int dtype, bool varlen) {
    if (H < 1 || Hk < 1 || pairs < 0) return GDN_ERR_INVALID_ARG;
    if (H > 1024 || Hk > 1024 || (d != 32 && d != 64 && d != 128 && d != 256) || pairs % 4 != 0) return GDN_ERR_UNSUPPORTED;
    if (2 * pairs > d) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_sizes(B, T, 1, dtype, varlen));
    if (token_count(B, T, varlen) > INT32_MAX) return GDN_ERR_UNSUPPORTED;  // a grid's blocks
    return GDN_OK;
}

gdn_status rope_args(gdn::RopeArgs& a, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     const float* q_weight, const float* k_weight, const float* inv_freq, const int32_t* positions,
                     const int32_t* cu_seqlens, int B, int T, int H, int Hk, int d, int pairs, int interleaved,
                     float eps, int dtype) {
    GDN_TRY(check_rope(B, T, H, Hk, d, pairs, dtype, cu_seqlens != nullptr));
    if (pairs > 0 && !inv_freq) return GDN_ERR_INVALID_ARG;
    a.tokens = token_count(B, T, cu_seqlens != nullptr);
    if (a.tokens > 0) {
        GDN_TRY(check_rows(q, q_stride, static_cast<int64_t>(H) * d, dtype));
        GDN_TRY(check_rows(k, k_stride, static_cast<int64_t>(Hk) * d, dtype));
    }
    GDN_TRY(check_dense({q_weight, k_weight, inv_freq}));
    GDN_TRY(check_cu(cu_seqlens));
    GDN_TRY(check_cu(positions));
    a.q = q; a.k = k; a.q_stride = q_stride; a.k_stride = k_stride; a.q_weight = q_weight; a.k_weight = k_weight;
    a.inv_freq = inv_freq; a.positions = positions; a.cu_seqlens = cu_seqlens;
    a.nseq = B; a.T = T; a.H = H; a.Hk = Hk; a.d = d; a.pairs = pairs; a.interleaved = interleaved != 0;
    a.dtype = dtype; a.eps = eps;
    a.share = gdn::rope_share(a.tokens, std::max(H, Hk), d);
    a.blocks = static_cast<unsigned>(gdn::rope_blocks(a.tokens, std::max(H, Hk), d));
    return GDN_OK;
}

gdn_status check_window(int B, int T, int H, int Hk, int d, int window, int sinks, float scale, bool varlen) {
    if (H < 1 || Hk < 1 || H % Hk != 0 || window < 1 || sinks < 0) return GDN_ERR_INVALID_ARG;
    if (!(scale > 0.f) || scale > 3e38f) return GDN_ERR_INVALID_ARG;
    if ((d != 64 && d != 128) || H > 1024 || sinks > gdn::kWindowMaxSinks) return GDN_ERR_UNSUPPORTED;
    GDN_TRY(check_sizes(B, T, H * d, GDN_BF16, varlen));
    // blocks of a grid, and the copies' row coordinates
    const long long tokens = token_count(B, T, varlen);
    if (tokens >= (1LL << 31) - 256 || (tokens / 32 + B) * H * (d / 8) >= (1LL << 31) * 8) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

// An input that the kernels copy in 16-byte pieces: present, rows at least `row` apart.
gdn_status check_pieces(const void* p, int64_t stride, int64_t row) {
    if (!p || stride < row || stride >= (1LL << 38)) return GDN_ERR_INVALID_ARG;
    return off16(p) || stride % 8 != 0 ? GDN_ERR_MISALIGNED : GDN_OK;
}

long long tile_slots(int B, int T, int rows, bool varlen) {
    if (varlen) return static_cast<long long>(T / rows) + B;
    return static_cast<long long>(B) * (T > rows ? (T + rows - 1) / rows : 1);
}

// What the backward keeps beside its outputs: delta, the first tokens' partial
// sums, and those of heads in pieces.
struct WindowLayout {
    int window, sinks;  // no longer than the row; no first tokens where the window leaves none out
    int far_tokens;
    long long far_slots;
    int pieces;
    size_t far, heads, total;
};
WindowLayout window_layout(int B, int T, int H, int Hk, int d, int window, int sinks, bool varlen) {
    WindowLayout L{};
    L.window = std::min(window, std::max(T, 1));
    L.sinks = window >= T ? 0 : sinks;
    const long long reach = (gdn::kWindowTile - 1 + static_cast<long long>(L.window) - 1) / gdn::kWindowTile + 1;
    L.far_tokens = static_cast<int>(std::min<long long>(reach * gdn::kWindowTile, 1 << 30));
    L.far_slots = L.sinks > 0 ? tile_slots(B, T, L.far_tokens, varlen) : 0;
    L.far = round_up(sizeof(float) * (varlen ? 1 : B) * static_cast<size_t>(H) * T);
    L.pieces = gdn::window_pieces(tile_slots(B, T, gdn::kWindowTile, varlen) + L.far_slots, H, Hk);
    L.heads = L.far + round_up(sizeof(float) * L.far_slots * L.pieces * Hk * 2 * L.sinks * d);
    const long long tokens = token_count(B, T, varlen);
    L.total = L.heads + (L.pieces > 1 ? round_up(sizeof(float) * L.pieces * tokens * Hk * 2 * d) : 0);
    return L;
}

gdn_status window_args(gdn::WindowArgs& a, const WindowLayout& L, const gdn_bf16* q, int64_t q_stride, const gdn_bf16* k,
                       int64_t k_stride, const gdn_bf16* v, int64_t v_stride, const int32_t* cu_seqlens, int B, int T,
                       int H, int Hk, int d, float scale) {
    const bool varlen = cu_seqlens != nullptr;
    GDN_TRY(check_cu(cu_seqlens));
    if (T > 0) {
        GDN_TRY(check_pieces(q, q_stride, static_cast<int64_t>(H) * d));
        GDN_TRY(check_pieces(k, k_stride, static_cast<int64_t>(Hk) * d));
        GDN_TRY(check_pieces(v, v_stride, static_cast<int64_t>(Hk) * d));
    }
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.cu_seqlens = cu_seqlens; a.tokens = token_count(B, T, varlen);
    a.nseq = B; a.T = T; a.H = H; a.Hk = Hk; a.d = d; a.window = L.window; a.sinks = L.sinks; a.scale = scale;
    a.far_tokens = L.far_tokens; a.far_slots = L.far_slots; a.pieces = L.pieces;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_rope_fwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* q_weight,
                        const float* k_weight, const float* inv_freq, const int32_t* positions,
                        const int32_t* cu_seqlens, void* q_out, void* k_out, int B, int T, int H, int Hk, int d,
                        int pairs, int interleaved, float eps, int dtype, cudaStream_t stream) {
    gdn::RopeArgs a{};
    GDN_TRY(rope_args(a, q, q_stride, k, k_stride, q_weight, k_weight, inv_freq, positions, cu_seqlens, B, T, H, Hk, d,
                      pairs, interleaved, eps, dtype));
    GDN_TRY(check_dense({q_out, k_out}));
    if (a.tokens == 0) return GDN_OK;
    if (!q_out || !k_out) return GDN_ERR_INVALID_ARG;
    if (!(a.err = gdn::device_error_word())) return GDN_ERR_CUDA;
    a.q_out = q_out; a.k_out = k_out;
    return gdn::count_launch(gdn::launch_rope_fwd(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_rope_bwd_workspace_size(int B, int T, int H, int Hk, int d, int varlen) {
    if (check_rope(B, T, H, Hk, d, 0, 0, varlen != 0) != GDN_OK) return 0;
    const long long tokens = token_count(B, T, varlen != 0);
    return round_up(sizeof(float) * 2 * gdn::rope_blocks(tokens, std::max(H, Hk), d) * d);
}

gdn_status gdn_rope_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* q_weight,
                        const float* k_weight, const float* inv_freq, const int32_t* positions,
                        const int32_t* cu_seqlens, const void* dq_out, const void* dk_out, void* dq, void* dk,
                        float* dq_weight, float* dk_weight, int B, int T, int H, int Hk, int d, int pairs,
                        int interleaved, float eps, int dtype, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
    gdn::RopeArgs a{};
    GDN_TRY(rope_args(a, q, q_stride, k, k_stride, q_weight, k_weight, inv_freq, positions, cu_seqlens, B, T, H, Hk, d,
                      pairs, interleaved, eps, dtype));
    if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr))
        return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_dense({dq_out, dk_out, dq, dk, dq_weight, dk_weight}));
    const bool par = dq_weight || dk_weight;
    if (par) GDN_TRY(check_ws(workspace, workspace_bytes, gdn_rope_bwd_workspace_size(B, T, H, Hk, d, cu_seqlens != nullptr)));
    if (a.tokens > 0) {
        if (!dq_out || !dk_out || !dq || !dk) return GDN_ERR_INVALID_ARG;
        if (!(a.err = gdn::device_error_word())) return GDN_ERR_CUDA;
        a.dq_out = dq_out; a.dk_out = dk_out; a.dq = dq; a.dk = dk;
        a.partial = par ? static_cast<float*>(workspace) : nullptr;
        if (!gdn::count_launch(gdn::launch_rope_bwd(a, stream))) return GDN_ERR_CUDA;
    }
    if (!par) return GDN_OK;
    gdn::ColumnSumArgs c{};
    c.partial = static_cast<float*>(workspace); c.c0 = c.c1 = d; c.cols = c.stride = 2LL * d;
    c.rows = static_cast<int>(a.blocks);
    c.out[0] = dq_weight; c.out[1] = dk_weight;
    return gdn::count_launch(gdn::launch_column_sum(c, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_window_fwd(const gdn_bf16* q, int64_t q_stride, const gdn_bf16* k, int64_t k_stride, const gdn_bf16* v,
                          int64_t v_stride, const int32_t* cu_seqlens, gdn_bf16* out, float* lse, int B, int T, int H,
                          int Hk, int d, int window, int sinks, float scale, cudaStream_t stream) {
    GDN_TRY(check_window(B, T, H, Hk, d, window, sinks, scale, cu_seqlens != nullptr));
    gdn::WindowArgs a{};
    const bool varlen = cu_seqlens != nullptr;
    GDN_TRY(window_args(a, window_layout(B, T, H, Hk, d, window, sinks, varlen), q, q_stride, k, k_stride, v, v_stride,
                        cu_seqlens, B, T, H, Hk, d, scale));
    GDN_TRY(check_dense({out, lse}));
    if (T == 0) return GDN_OK;
    if (!out) return GDN_ERR_INVALID_ARG;
    if (!(a.err = gdn::device_error_word())) return GDN_ERR_CUDA;
    a.out = out; a.lse = lse;
    a.slots = tile_slots(B, T, gdn::window_fwd_rows(H, Hk), varlen);
    return gdn::count_launch(gdn::launch_window_fwd(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_window_bwd_workspace_size(int B, int T, int H, int Hk, int d, int window, int sinks, int varlen) {
    if (check_window(B, T, H, Hk, d, window, sinks, 1.f, varlen != 0) != GDN_OK) return 0;
    return window_layout(B, T, H, Hk, d, window, sinks, varlen != 0).total;
}

gdn_status gdn_window_bwd(const gdn_bf16* q, int64_t q_stride, const gdn_bf16* k, int64_t k_stride, const gdn_bf16* v,
                          int64_t v_stride, const int32_t* cu_seqlens, const gdn_bf16* out, const float* lse,
                          const gdn_bf16* d_out, gdn_bf16* dq, gdn_bf16* dk, gdn_bf16* dv, int B, int T, int H, int Hk,
                          int d, int window, int sinks, float scale, void* workspace, size_t workspace_bytes,
                          cudaStream_t stream) {
    GDN_TRY(check_window(B, T, H, Hk, d, window, sinks, scale, cu_seqlens != nullptr));
    gdn::WindowArgs a{};
    const bool varlen = cu_seqlens != nullptr;
    const WindowLayout L = window_layout(B, T, H, Hk, d, window, sinks, varlen);
    GDN_TRY(window_args(a, L, q, q_stride, k, k_stride, v, v_stride, cu_seqlens, B, T, H, Hk, d, scale));
    GDN_TRY(check_dense({out, lse, d_out, dq, dk, dv}));
    if (T == 0) return GDN_OK;
    if (!out || !lse || !d_out || !dq || !dk || !dv) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_ws(workspace, workspace_bytes, L.total));
    if (!(a.err = gdn::device_error_word())) return GDN_ERR_CUDA;
    a.out = const_cast<gdn_bf16*>(out); a.lse = const_cast<float*>(lse); a.d_out = d_out;
    a.dq = dq; a.dk = dk; a.dv = dv;
    a.delta = static_cast<float*>(workspace);
    a.far_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.far);
    a.head_part = reinterpret_cast<float*>(static_cast<char*>(workspace) + L.heads);
    a.slots = tile_slots(B, T, gdn::kWindowTile, varlen);
    return gdn::count_launch(gdn::launch_window_bwd(a, stream), L.sinks > 0 || L.pieces > 1 ? 4 : 3) ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_window_step(const gdn_bf16* q, int64_t q_stride, const gdn_bf16* k, int64_t k_stride, const gdn_bf16* v,
                           int64_t v_stride, gdn_bf16* k_cache, gdn_bf16* v_cache, const int32_t* lengths,
                           const int32_t* slots, gdn_bf16* out, int B, int S, int H, int Hk, int d, int window,
                           int sinks, float scale, cudaStream_t stream) {
    GDN_TRY(check_window(B, 1, H, Hk, d, window, sinks, scale, false));
    if (window > gdn::checks::kMaxT) return GDN_ERR_UNSUPPORTED;
    if (!k_cache || !v_cache || !lengths || !out || S < 1 || (!slots && S < B)) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_pieces(q, q_stride, static_cast<int64_t>(H) * d));
    GDN_TRY(check_pieces(k, k_stride, static_cast<int64_t>(Hk) * d));
    GDN_TRY(check_pieces(v, v_stride, static_cast<int64_t>(Hk) * d));
    GDN_TRY(check_dense({k_cache, v_cache, out}));
    GDN_TRY(check_cu(lengths));
    GDN_TRY(check_cu(slots));
    gdn::WindowStepArgs a{};
    if (!(a.err = gdn::device_error_word())) return GDN_ERR_CUDA;
    a.q = q; a.k = k; a.v = v; a.q_stride = q_stride; a.k_stride = k_stride; a.v_stride = v_stride;
    a.k_cache = k_cache; a.v_cache = v_cache; a.lengths = lengths; a.slots = slots; a.out = out;
    a.B = B; a.S = S; a.H = H; a.Hk = Hk; a.d = d; a.rows = sinks + window; a.window = window; a.sinks = sinks;
    a.scale = scale;
    gdn::window_step_shape(a);
    return gdn::count_launch(gdn::launch_window_step(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_window_fill(const gdn_bf16* k, int64_t k_stride, const gdn_bf16* v, int64_t v_stride,
                           const int32_t* cu_seqlens, const int32_t* slots, gdn_bf16* k_cache, gdn_bf16* v_cache, int B,
                           int T, int S, int Hk, int d, int window, int sinks, cudaStream_t stream) {
    GDN_TRY(check_window(B, T, Hk, Hk, d, window, sinks, 1.f, cu_seqlens != nullptr));
    if (window > gdn::checks::kMaxT) return GDN_ERR_UNSUPPORTED;
    if (!k_cache || !v_cache || S < 1 || (!slots && S < B)) return GDN_ERR_INVALID_ARG;
    if (T > 0) {
        GDN_TRY(check_pieces(k, k_stride, static_cast<int64_t>(Hk) * d));
        GDN_TRY(check_pieces(v, v_stride, static_cast<int64_t>(Hk) * d));
    }
    GDN_TRY(check_dense({k_cache, v_cache}));
    GDN_TRY(check_cu(cu_seqlens));
    GDN_TRY(check_cu(slots));
    if (T == 0) return GDN_OK;
    gdn::WindowFillArgs a{};
    if (!(a.err = gdn::device_error_word())) return GDN_ERR_CUDA;
    a.k = k; a.v = v; a.k_stride = k_stride; a.v_stride = v_stride; a.k_cache = k_cache; a.v_cache = v_cache;
    a.cu_seqlens = cu_seqlens; a.slots = slots; a.nseq = B; a.T = T; a.S = S; a.Hk = Hk; a.d = d; a.window = window;
    a.sinks = sinks;
    return gdn::count_launch(gdn::launch_window_fill(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
