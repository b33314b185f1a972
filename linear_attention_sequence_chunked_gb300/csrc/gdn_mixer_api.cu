// Host side of the mixer operators' C ABI (include/gdn.h): argument
// validation, workspace layout and kernel launches.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <initializer_list>

#include "gdn.h"
#include "gdn_kernels.h"

namespace {

constexpr size_t kAlign = 256;
constexpr int kMaxT = 1 << 30;

size_t round_up(size_t x) { return (x + kAlign - 1) / kAlign * kAlign; }
bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off_elem(const void* p, int dtype) { return reinterpret_cast<uintptr_t>(p) % (dtype == GDN_F32 ? 4 : 2) != 0; }

gdn_status check_dense(std::initializer_list<const void*> ptrs) {
    for (const void* p : ptrs)
        if (p && off16(p)) return GDN_ERR_MISALIGNED;
    return GDN_OK;
}
gdn_status check_cu(const int32_t* cu) { return reinterpret_cast<uintptr_t>(cu) & 3u ? GDN_ERR_MISALIGNED : GDN_OK; }

// A strided input: present, aligned to its element, rows at least `row` apart.
gdn_status check_rows(const void* p, int64_t stride, int64_t row, int dtype) {
    if (!p || stride < row || stride >= (1LL << 40)) return GDN_ERR_INVALID_ARG;
    return off_elem(p, dtype) ? GDN_ERR_MISALIGNED : GDN_OK;
}

gdn_status check_ws(const void* p, size_t bytes, size_t need) {
    if (need == 0) return GDN_OK;
    if (!p || bytes < need) return GDN_ERR_INVALID_ARG;
    return reinterpret_cast<uintptr_t>(p) & (kAlign - 1) ? GDN_ERR_MISALIGNED : GDN_OK;
}

gdn_status check_sizes(int B, int T, int D, int dtype) {
    if (B < 1 || T < 0 || D < 1) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (B > 65535 || T > kMaxT || D > 65536) return GDN_ERR_UNSUPPORTED;
    if (static_cast<long long>(B) * T >= (1LL << 40) / D) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

gdn_status check_conv(int B, int T, int D, int W, int activation, int dtype) {
    const gdn_status st = check_sizes(B, T, D, dtype);
    if (st != GDN_OK) return st;
    if (W < 2 || W > 4) return GDN_ERR_UNSUPPORTED;
    if (activation != GDN_ACT_NONE && activation != GDN_ACT_SILU) return GDN_ERR_INVALID_ARG;
    return GDN_OK;
}

gdn_status check_ssm(int B, int T, int D, int G, int N, int dtype) {
    const gdn_status st = check_sizes(B, T, D, dtype);
    if (st != GDN_OK) return st;
    if (G < 1 || D % G != 0) return GDN_ERR_INVALID_ARG;
    if (N != 8 && N != 16 && N != 32 && N != 64 && N != 128) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

#define GDN_TRY(expr)                          \
    do {                                       \
        const gdn_status st_ = (expr);         \
        if (st_ != GDN_OK) return st_;         \
    } while (0)

// Time blocks (or chunks) of `tb` tokens, as find_block counts them.
long long block_slots(int B, int T, int tb, bool varlen) {
    if (varlen) return static_cast<long long>(T / tb) + B;
    return static_cast<long long>(B) * (T > tb ? (T + tb - 1) / tb : 1);
}

size_t conv_ws(int B, int T, int D, int W, bool varlen) {
    // packed: T tokens in all
    const long long slots = block_slots(B, T, gdn::conv_block_tokens(varlen ? 1 : B, T, D, 1, 0), varlen);
    return round_up(sizeof(float) * gdn::conv_partial_rows(slots) * (W + 1) * D);
}

size_t ssm_saved(int B, int T, int D, int N, bool varlen) {
    const long long slots = varlen ? static_cast<long long>(T / gdn::kSsmChunk) + B
                                   : static_cast<long long>(B) * ((T + gdn::kSsmChunk - 1) / gdn::kSsmChunk);
    return round_up(sizeof(float) * slots * D * N);
}

// Segments of a scan, and the workspace that joins them.
struct SsmSplit {
    int seg;
    long long slots;
    int kernels;       // launched by the scan itself
    bool joined;       // by a kernel of its own
    size_t dt, total;  // carry_dt's offset (carry is at 0); 0 bytes: not split
};
SsmSplit ssm_split(int B, int T, int D, int G, int N, bool varlen, bool backward) {
    SsmSplit s{};
    s.seg = gdn::ssm_segment(B, T, D, G, N, varlen, backward);
    s.slots = block_slots(B, T, s.seg, varlen);
    s.kernels = 1;
    if (s.seg < T) {
        // a sequence's segments are joined where they start up to 32 of them
        // (a few hundred instructions per warp and one kernel less: 4 x 4096 x 2048
        // in seven 269 us, 273 by the kernel), beyond that by a kernel that walks
        // them once.  The forward takes packed sequences to be at most four times
        // their mean (1 x 4000 x 512, N = 32, 62 segments: nine equal sequences 43
        // us instead of 46, one long one 52 instead of 48; the reverse mode gains 2
        // of 140 and loses 24)
        const long long longest = varlen && !backward ? std::min<long long>(T, 4LL * T / std::max(B, 1)) : T;
        s.joined = (longest - 1) / s.seg >= 32 || (T - 1) / s.seg >= 64;
        s.kernels = s.joined ? 3 : 2;
        s.dt = round_up(sizeof(float) * s.slots * D * N);
        s.total = s.dt + round_up(sizeof(float) * s.slots * D);
    }
    return s;
}
void set_split(gdn::SsmArgs& a, const SsmSplit& s, void* workspace) {
    a.seg = s.seg;
    a.slots = s.slots;
    a.joined = s.joined;
    if (s.total) {
        a.carry = static_cast<float*>(workspace);
        a.carry_dt = reinterpret_cast<float*>(static_cast<char*>(workspace) + s.dt);
    }
}

struct SsmBwdLayout {
    size_t bc, par, carry, total;
};
SsmBwdLayout ssm_bwd_layout(int B, int T, int D, int G, int N, bool varlen) {
    SsmBwdLayout L{};
    const long long rows = varlen ? T : static_cast<long long>(B) * T;
    L.bc = 0;
    L.par = round_up(sizeof(float) * gdn::ssm_group_blocks(D, G, N) * static_cast<long long>(G) * rows * 2 * N);
    const SsmSplit split = ssm_split(B, T, D, G, N, varlen, true);
    L.carry = L.par + round_up(sizeof(float) * split.slots * gdn::ssm_par_stride(D, N));
    L.total = L.carry + split.total;
    return L;
}

gdn_status check_norm(int64_t rows, int C, int groups, int activation, int dtype) {
    if (rows < 0 || C < 1 || groups < 1 || C % groups != 0) return GDN_ERR_INVALID_ARG;
    if (activation < GDN_ACT_NONE || activation > GDN_ACT_SIGMOID) return GDN_ERR_INVALID_ARG;
    if (dtype != GDN_BF16 && dtype != GDN_F32) return GDN_ERR_INVALID_ARG;
    if (C / groups > gdn::kNormMaxGroup || rows >= (1LL << 40) / C) return GDN_ERR_UNSUPPORTED;
    if (rows > gdn::norm_max_groups(C / groups) / groups) return GDN_ERR_UNSUPPORTED;
    return GDN_OK;
}

}  // namespace

extern "C" {

gdn_status gdn_conv_fwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                        const void* initial_state, const int32_t* cu_seqlens, void* y, void* final_state, int B, int T,
                        int D, int W, int activation, int dtype, cudaStream_t stream) {
    GDN_TRY(check_conv(B, T, D, W, activation, dtype));
    if (!weight || (T > 0 && !y)) return GDN_ERR_INVALID_ARG;
    if (T > 0) GDN_TRY(check_rows(x, x_stride, D, dtype));
    GDN_TRY(check_dense({weight, bias, initial_state, y, final_state}));
    GDN_TRY(check_cu(cu_seqlens));
    if (final_state && final_state == initial_state) return GDN_ERR_INVALID_ARG;
    if (T == 0 && !final_state) return GDN_OK;
    int* err = gdn::device_error_word();
    if (!err) return GDN_ERR_CUDA;
    gdn::ConvArgs a{};
    a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias; a.initial_state = initial_state;
    a.cu_seqlens = cu_seqlens; a.y = y; a.final_state = final_state;
    a.N = B; a.T = T; a.D = D; a.W = W; a.activation = activation; a.dtype = dtype; a.err = err;
    a.tb = gdn::conv_block_tokens(cu_seqlens ? 1 : B, T, D, 0, dtype);
    a.slots = block_slots(B, T, a.tb, cu_seqlens != nullptr);
    return gdn::count_launch(gdn::launch_conv_fwd(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_conv_bwd_workspace_size(int B, int T, int D, int W, int varlen) {
    if (check_conv(B, T, D, W, 0, 0) != GDN_OK) return 0;
    return conv_ws(B, T, D, W, varlen != 0);
}

gdn_status gdn_conv_bwd(const void* x, int64_t x_stride, const float* weight, const float* bias,
                        const void* initial_state, const int32_t* cu_seqlens, const void* d_out,
                        const void* d_final_state, void* dx, float* dweight, float* dbias, void* d_initial_state,
                        int B, int T, int D, int W, int activation, int dtype, void* workspace, size_t workspace_bytes,
                        cudaStream_t stream) {
    GDN_TRY(check_conv(B, T, D, W, activation, dtype));
    if (!weight || !dweight || (T > 0 && (!d_out || !dx))) return GDN_ERR_INVALID_ARG;
    if (T > 0) GDN_TRY(check_rows(x, x_stride, D, dtype));
    GDN_TRY(check_dense({weight, bias, initial_state, d_out, d_final_state, dx, dweight, dbias, d_initial_state}));
    GDN_TRY(check_cu(cu_seqlens));
    GDN_TRY(check_ws(workspace, workspace_bytes, conv_ws(B, T, D, W, cu_seqlens != nullptr)));
    int* err = gdn::device_error_word();
    if (!err) return GDN_ERR_CUDA;
    gdn::ConvArgs a{};
    a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias; a.initial_state = initial_state;
    a.cu_seqlens = cu_seqlens; a.d_out = d_out; a.d_final_state = d_final_state; a.dx = dx;
    a.d_initial_state = d_initial_state; a.partial = static_cast<float*>(workspace);
    a.N = B; a.T = T; a.D = D; a.W = W; a.activation = activation; a.dtype = dtype; a.err = err;
    a.tb = gdn::conv_block_tokens(cu_seqlens ? 1 : B, T, D, 1, 0);
    a.slots = block_slots(B, T, a.tb, cu_seqlens != nullptr);
    if (!gdn::count_launch(gdn::launch_conv_bwd(a, stream))) return GDN_ERR_CUDA;
    gdn::ColumnSumArgs c{};
    c.partial = a.partial; c.cols = c.stride = static_cast<long long>(W + 1) * D; c.c1 = D; c.W = W;
    c.rows = static_cast<int>(gdn::conv_partial_rows(a.slots));
    c.out[0] = dweight; c.out[1] = dbias;
    return gdn::count_launch(gdn::launch_column_sum(c, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_conv_step(const void* x, int64_t x_stride, const float* weight, const float* bias, const void* state,
                         void* out_state, const int32_t* slots, void* y, int B, int S, int D, int W, int activation,
                         int dtype, cudaStream_t stream) {
    GDN_TRY(check_conv(B, 1, D, W, activation, dtype));
    if (!weight || !state || !out_state || !y || S < 1 || (!slots && S < B)) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_rows(x, x_stride, D, dtype));
    GDN_TRY(check_dense({weight, bias, state, out_state, y}));
    GDN_TRY(check_cu(slots));
    int* err = gdn::device_error_word();
    if (!err) return GDN_ERR_CUDA;
    gdn::ConvStepArgs a{};
    a.x = x; a.x_stride = x_stride; a.weight = weight; a.bias = bias; a.state = state; a.out_state = out_state;
    a.slots = slots; a.y = y; a.B = B; a.S = S; a.D = D; a.W = W; a.activation = activation; a.dtype = dtype;
    a.err = err;
    return gdn::count_launch(gdn::launch_conv_step(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_ssm_saved_size(int B, int T, int D, int N, int varlen) {
    if (check_ssm(B, T, D, 1, N, 0) != GDN_OK) return 0;
    return ssm_saved(B, T, D, N, varlen != 0);
}

size_t gdn_ssm_fwd_workspace_size(int B, int T, int D, int G, int N, int varlen) {
    if (check_ssm(B, T, D, G, N, 0) != GDN_OK) return 0;
    return ssm_split(B, T, D, G, N, varlen != 0, false).total;
}

gdn_status gdn_ssm_fwd(const void* u, int64_t u_stride, const void* dt, int64_t dt_stride, const float* A,
                       const void* Bm, int64_t B_stride, const void* Cm, int64_t C_stride, const float* D_skip,
                       const void* z, int64_t z_stride, const float* dt_bias, int dt_softplus,
                       const float* initial_state, const int32_t* cu_seqlens, void* out, float* final_state,
                       void* saved, size_t saved_bytes, int B, int T, int D, int G, int N, int dtype, void* workspace,
                       size_t workspace_bytes, cudaStream_t stream) {
    GDN_TRY(check_ssm(B, T, D, G, N, dtype));
    if (!A || (T > 0 && !out)) return GDN_ERR_INVALID_ARG;
    if (T > 0) {
        GDN_TRY(check_rows(u, u_stride, D, dtype));
        GDN_TRY(check_rows(dt, dt_stride, D, dtype));
        if (z) GDN_TRY(check_rows(z, z_stride, D, dtype));
        GDN_TRY(check_rows(Bm, B_stride, static_cast<int64_t>(G) * N, dtype));
        GDN_TRY(check_rows(Cm, C_stride, static_cast<int64_t>(G) * N, dtype));
    }
    GDN_TRY(check_dense({A, D_skip, dt_bias, initial_state, out, final_state}));
    GDN_TRY(check_cu(cu_seqlens));
    const bool varlen = cu_seqlens != nullptr;
    if (saved) GDN_TRY(check_ws(saved, saved_bytes, ssm_saved(B, T, D, N, varlen)));
    const SsmSplit split = ssm_split(B, T, D, G, N, varlen, false);
    GDN_TRY(check_ws(workspace, workspace_bytes, split.total));
    if (T == 0 && !final_state) return GDN_OK;
    int* err = gdn::device_error_word();
    if (!err) return GDN_ERR_CUDA;
    gdn::SsmArgs a{};
    a.u = u; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm;
    a.u_stride = u_stride; a.dt_stride = dt_stride; a.z_stride = z_stride; a.B_stride = B_stride; a.C_stride = C_stride;
    a.A = A; a.D_skip = D_skip; a.dt_bias = dt_bias; a.softplus = dt_softplus != 0;
    a.initial_state = initial_state; a.cu_seqlens = cu_seqlens; a.out = out; a.final_state = final_state;
    a.saved = static_cast<float*>(saved);
    a.nseq = B; a.T = T; a.D = D; a.G = G; a.N = N; a.dtype = dtype; a.err = err;
    set_split(a, split, workspace);
    return gdn::count_launch(gdn::launch_ssm_fwd(a, stream), split.kernels) ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_ssm_bwd_workspace_size(int B, int T, int D, int G, int N, int varlen) {
    if (check_ssm(B, T, D, G, N, 0) != GDN_OK) return 0;
    return ssm_bwd_layout(B, T, D, G, N, varlen != 0).total;
}

gdn_status gdn_ssm_bwd(const void* u, int64_t u_stride, const void* dt, int64_t dt_stride, const float* A,
                       const void* Bm, int64_t B_stride, const void* Cm, int64_t C_stride, const float* D_skip,
                       const void* z, int64_t z_stride, const float* dt_bias, int dt_softplus,
                       const int32_t* cu_seqlens, const void* d_out, const float* d_final_state, const void* saved,
                       size_t saved_bytes, void* du, void* ddt, void* dz, void* dB, void* dC, float* dA, float* dD,
                       float* ddt_bias, float* d_initial_state, int B, int T, int D, int G, int N, int dtype,
                       void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    GDN_TRY(check_ssm(B, T, D, G, N, dtype));
    if (!A || !dA) return GDN_ERR_INVALID_ARG;
    if (T > 0) {
        if (!d_out || !du || !ddt || !dB || !dC || (z != nullptr) != (dz != nullptr)) return GDN_ERR_INVALID_ARG;
        GDN_TRY(check_rows(u, u_stride, D, dtype));
        GDN_TRY(check_rows(dt, dt_stride, D, dtype));
        if (z) GDN_TRY(check_rows(z, z_stride, D, dtype));
        GDN_TRY(check_rows(Bm, B_stride, static_cast<int64_t>(G) * N, dtype));
        GDN_TRY(check_rows(Cm, C_stride, static_cast<int64_t>(G) * N, dtype));
    }
    GDN_TRY(check_dense({A, D_skip, dt_bias, d_out, d_final_state, du, ddt, dz, dB, dC, dA, dD, ddt_bias, d_initial_state}));
    GDN_TRY(check_cu(cu_seqlens));
    const bool varlen = cu_seqlens != nullptr;
    GDN_TRY(check_ws(saved, saved_bytes, ssm_saved(B, T, D, N, varlen)));
    const SsmBwdLayout L = ssm_bwd_layout(B, T, D, G, N, varlen);
    GDN_TRY(check_ws(workspace, workspace_bytes, L.total));
    int* err = gdn::device_error_word();
    if (!err) return GDN_ERR_CUDA;
    char* ws = static_cast<char*>(workspace);
    gdn::SsmArgs a{};
    a.u = u; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm;
    a.u_stride = u_stride; a.dt_stride = dt_stride; a.z_stride = z_stride; a.B_stride = B_stride; a.C_stride = C_stride;
    a.A = A; a.D_skip = D_skip; a.dt_bias = dt_bias; a.softplus = dt_softplus != 0; a.cu_seqlens = cu_seqlens;
    a.saved = static_cast<float*>(const_cast<void*>(saved));
    a.d_out = d_out; a.d_final_state = d_final_state; a.du = du; a.ddt = ddt; a.dz = dz;
    a.d_initial_state = d_initial_state;
    a.bc_part = reinterpret_cast<float*>(ws + L.bc); a.par_part = reinterpret_cast<float*>(ws + L.par);
    a.nseq = B; a.T = T; a.D = D; a.G = G; a.N = N; a.dtype = dtype; a.err = err;
    const SsmSplit split = ssm_split(B, T, D, G, N, varlen, true);
    set_split(a, split, ws + L.carry);
    if (!gdn::count_launch(gdn::launch_ssm_bwd(a, stream), split.kernels)) return GDN_ERR_CUDA;
    gdn::SsmBcArgs bc{};
    bc.bc_part = a.bc_part; bc.dB = dB; bc.dC = dC; bc.rows = varlen ? T : static_cast<long long>(B) * T;
    bc.G = G; bc.N = N; bc.blocks = gdn::ssm_group_blocks(D, G, N); bc.dtype = dtype;
    if (!gdn::count_launch(gdn::launch_ssm_bc(bc, stream), bc.rows > 0)) return GDN_ERR_CUDA;
    gdn::ColumnSumArgs c{};
    c.partial = a.par_part; c.c0 = static_cast<long long>(D) * N; c.c1 = D; c.cols = c.c0 + 2LL * D;
    c.stride = gdn::ssm_par_stride(D, N);
    c.rows = static_cast<int>(split.slots); c.out[0] = dA; c.out[1] = dD; c.out[2] = ddt_bias;
    return gdn::count_launch(gdn::launch_column_sum(c, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_ssm_step(const void* u, int64_t u_stride, const void* dt, int64_t dt_stride, const float* A,
                        const void* Bm, int64_t B_stride, const void* Cm, int64_t C_stride, const float* D_skip,
                        const void* z, int64_t z_stride, const float* dt_bias, int dt_softplus, const float* state,
                        float* out_state, const int32_t* slots, void* out, int B, int S, int D, int G, int N, int dtype,
                        cudaStream_t stream) {
    GDN_TRY(check_ssm(B, 1, D, G, N, dtype));
    if (!A || !state || !out_state || !out || S < 1 || (!slots && S < B)) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_rows(u, u_stride, D, dtype));
    GDN_TRY(check_rows(dt, dt_stride, D, dtype));
    if (z) GDN_TRY(check_rows(z, z_stride, D, dtype));
    GDN_TRY(check_rows(Bm, B_stride, static_cast<int64_t>(G) * N, dtype));
    GDN_TRY(check_rows(Cm, C_stride, static_cast<int64_t>(G) * N, dtype));
    GDN_TRY(check_dense({A, D_skip, dt_bias, state, out_state, out}));
    GDN_TRY(check_cu(slots));
    int* err = gdn::device_error_word();
    if (!err) return GDN_ERR_CUDA;
    gdn::SsmStepArgs a{};
    a.u = u; a.dt = dt; a.z = z; a.Bm = Bm; a.Cm = Cm;
    a.u_stride = u_stride; a.dt_stride = dt_stride; a.z_stride = z_stride; a.B_stride = B_stride; a.C_stride = C_stride;
    a.A = A; a.D_skip = D_skip; a.dt_bias = dt_bias; a.softplus = dt_softplus != 0;
    a.state = state; a.out_state = out_state; a.slots = slots; a.out = out;
    a.B = B; a.S = S; a.D = D; a.G = G; a.N = N; a.dtype = dtype; a.err = err;
    return gdn::count_launch(gdn::launch_ssm_step(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

gdn_status gdn_norm_fwd(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, const float* weight,
                        const float* bias, void* y, int64_t rows, int C, int groups, float eps, int activation,
                        int center, int gate_first, int dtype, cudaStream_t stream) {
    GDN_TRY(check_norm(rows, C, groups, activation, dtype));
    if (rows == 0) return GDN_OK;
    if (!y) return GDN_ERR_INVALID_ARG;
    GDN_TRY(check_rows(x, x_stride, C, dtype));
    if (gate) GDN_TRY(check_rows(gate, gate_stride, C, dtype));
    GDN_TRY(check_dense({weight, bias, y}));
    gdn::NormArgs a{};
    a.x = x; a.gate = gate; a.x_stride = x_stride; a.gate_stride = gate_stride; a.weight = weight; a.bias = bias;
    a.y = y; a.rows = rows; a.C = C; a.groups = groups; a.eps = eps; a.activation = activation;
    a.center = center != 0; a.gate_first = gate_first != 0; a.dtype = dtype;
    return gdn::count_launch(gdn::launch_norm_fwd(a, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

size_t gdn_norm_bwd_workspace_size(int64_t rows, int C, int groups, int dtype) {
    if (check_norm(rows, C, groups, 0, dtype) != GDN_OK) return 0;
    return round_up(sizeof(float) * 2 * static_cast<size_t>(gdn::norm_partial_rows(rows, C, groups, dtype)) * C);
}

gdn_status gdn_norm_bwd(const void* x, int64_t x_stride, const void* gate, int64_t gate_stride, const float* weight,
                        const float* bias, const void* d_out, void* dx, void* dgate, float* dweight, float* dbias,
                        int64_t rows, int C, int groups, float eps, int activation, int center, int gate_first,
                        int dtype, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
    GDN_TRY(check_norm(rows, C, groups, activation, dtype));
    if ((weight != nullptr) != (dweight != nullptr) || (bias != nullptr) != (dbias != nullptr)) return GDN_ERR_INVALID_ARG;
    if (rows > 0) {
        if (!d_out || !dx || (gate != nullptr) != (dgate != nullptr)) return GDN_ERR_INVALID_ARG;
        GDN_TRY(check_rows(x, x_stride, C, dtype));
        if (gate) GDN_TRY(check_rows(gate, gate_stride, C, dtype));
    }
    GDN_TRY(check_dense({weight, bias, d_out, dx, dgate, dweight, dbias}));
    const bool par = dweight || dbias;
    if (par) GDN_TRY(check_ws(workspace, workspace_bytes, gdn_norm_bwd_workspace_size(rows, C, groups, dtype)));
    gdn::NormArgs a{};
    a.x = x; a.gate = gate; a.x_stride = x_stride; a.gate_stride = gate_stride; a.weight = weight; a.bias = bias;
    a.d_out = d_out; a.dx = dx; a.dgate = dgate; a.partial = par ? static_cast<float*>(workspace) : nullptr;
    a.rows = rows; a.C = C; a.groups = groups; a.eps = eps; a.activation = activation;
    a.center = center != 0; a.gate_first = gate_first != 0; a.dtype = dtype;
    if (rows > 0 && !gdn::count_launch(gdn::launch_norm_bwd(a, stream))) return GDN_ERR_CUDA;
    if (!par) return GDN_OK;
    gdn::ColumnSumArgs c{};
    c.partial = a.partial; c.c0 = C; c.c1 = C; c.cols = c.stride = bias ? 2LL * C : C;
    c.rows = gdn::norm_partial_rows(rows, C, groups, dtype);
    c.out[0] = dweight; c.out[1] = dbias;
    return gdn::count_launch(gdn::launch_column_sum(c, stream)) ? GDN_OK : GDN_ERR_CUDA;
}

}  // extern "C"
