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

gdn_status check_rope(int B, int T, int H, int Hk, int d, int pairs, int dtype) {
    if (H < 1 || Hk < 1 || pairs < 0) return GDN_ERR_INVALID_ARG;
    if (H > 1024 || Hk > 1024 || (d != 32 && d != 64 && d != 128 && d != 256) || pairs % 4 != 0) return GDN_ERR_UNSUPPORTED;
    if (2 * pairs > d) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_sizes(B, T, 1, dtype));
    if (static_cast<long long>(B) * T > INT32_MAX) return GDN_ERR_UNSUPPORTED;  // a grid's blocks
    return GDN_OK;
}

gdn_status rope_args(gdn::RopeArgs& a, const void* q, int64_t q_stride, const void* k, int64_t k_stride,
                     const float* q_weight, const float* k_weight, const float* inv_freq, const int32_t* positions,
                     const int32_t* cu_seqlens, int B, int T, int H, int Hk, int d, int pairs, int interleaved,
                     float eps, int dtype, bool backward) {
    GDN_TRY(check_rope(B, T, H, Hk, d, pairs, dtype));
    if (pairs > 0 && !inv_freq) return GDN_ERR_INVALID_ARG;
    a.tokens = cu_seqlens ? T : static_cast<long long>(B) * T;
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
    a.tile = gdn::rope_tile(a.tokens, H + Hk);
    a.blocks = static_cast<unsigned>(gdn::rope_blocks(a.tokens, H + Hk, backward));
    if (a.tokens > 0 && !(a.err = gdn::device_error_word())) return GDN_ERR_CUDA;
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
                      pairs, interleaved, eps, dtype, false));
    GDN_TRY(check_dense({q_out, k_out}));
    if (a.tokens == 0) return GDN_OK;
    if (!q_out || !k_out) return GDN_ERR_INVALID_ARG;
    a.q_out = q_out; a.k_out = k_out;
    return gdn::count_launch(gdn::launch_rope_fwd(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_rope_bwd_workspace_size(int B, int T, int H, int Hk, int d, int varlen) {
    if (check_rope(B, T, H, Hk, d, 0, 0) != GDN_OK) return 0;
    const long long tokens = varlen ? T : static_cast<long long>(B) * T;
    return round_up(sizeof(float) * 2 * gdn::rope_blocks(tokens, H + Hk, true) * d);
}

gdn_status gdn_rope_bwd(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const float* q_weight,
                        const float* k_weight, const float* inv_freq, const int32_t* positions,
                        const int32_t* cu_seqlens, const void* dq_out, const void* dk_out, void* dq, void* dk,
                        float* dq_weight, float* dk_weight, int B, int T, int H, int Hk, int d, int pairs,
                        int interleaved, float eps, int dtype, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
    gdn::RopeArgs a{};
    GDN_TRY(rope_args(a, q, q_stride, k, k_stride, q_weight, k_weight, inv_freq, positions, cu_seqlens, B, T, H, Hk, d,
                      pairs, interleaved, eps, dtype, true));
    if ((q_weight != nullptr) != (dq_weight != nullptr) || (k_weight != nullptr) != (dk_weight != nullptr))
        return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_dense({dq_out, dk_out, dq, dk, dq_weight, dk_weight}));
    const bool par = dq_weight || dk_weight;
    if (par) GDN_TRY(check_ws(workspace, workspace_bytes, gdn_rope_bwd_workspace_size(B, T, H, Hk, d, cu_seqlens != nullptr)));
    if (a.tokens > 0) {
        if (!dq_out || !dk_out || !dq || !dk) return GDN_ERR_INVALID_ARG;
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

}  // extern "C"
