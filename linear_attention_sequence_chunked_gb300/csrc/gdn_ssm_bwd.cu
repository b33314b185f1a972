// Reverse mode of the selective state space scan (gdn_ssm_common.cuh has the
// forward's formulas and the layout).  With dy = d_out silu(z) and e_t the
// gradient of h_t,
//   e_t  = C_t dy_t + a_{t+1} e_{t+1},   a_t = exp(dt_t A)   (from d_final_state)
//   dC_t = sum_d dy_t h_t,   dB_t = sum_d e_t x_t,   dx_t = sum_n e_t B_t
//   q_t  = a_t e_t h_{t-1}:  ddt_t = u_t dx_t + sum_n A q_t,   dA = sum_t dt_t q_t
//   du_t = dt_t dx_t + D dy_t,   dD = sum_t dy_t u_t,   dz_t = d_out_t y_t silu'(z_t)
//   ddt_raw = ddt sigmoid(dt_raw + bias),   ddt_bias = sum_t ddt_raw.
// A warp walks its tokens from the last tile to the first.  It reads the tile's
// start state that the forward kept, runs the tile forward once more with the
// 16 decays and states in registers, then back.  Sums over a channel's lanes
// and over the warp's channels halve the values with each shuffle.  dB and dC
// of a warp's CH channels go out as partial rows, dA, dD and ddt_bias as one
// partial row per sequence; two small kernels add those up in a fixed order.
#include "gdn_ssm_common.cuh"

namespace gdn {

namespace {

using namespace ssm;

template <int N>
constexpr int kWarps = N >= 64 ? 2 : 4;

// Sums of v[0..7] over the CH channels of a warp (lanes LPC apart): value i of
// channel lane ch is then the sum of v[i * min(CH, 8) + ch mod 8].
template <int LPC, int CH>
__device__ __forceinline__ void across_channels(float (&v)[8], int ch) {
#pragma unroll
    for (int m = 1; m < CH; m *= 2) {
        if (m < 8) {
            const bool hi = (ch & m) != 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (i < 4 / m) {
                    const float send = hi ? v[2 * i] : v[2 * i + 1];
                    const float keep = hi ? v[2 * i + 1] : v[2 * i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, m * LPC);
                }
            }
        } else {
            v[0] += __shfl_xor_sync(0xffffffffu, v[0], m * LPC);
        }
    }
}

template <typename T, int N, bool VEC>
__global__ void __launch_bounds__(32 * kWarps<N>) ssm_bwd_kernel(const SsmArgs p, int seg, long long slots, int blocks) {
    using G = Geo<N, 4>;
    constexpr int CH = G::CH, EPL = G::EPL, LPC = G::LPC;
    constexpr int M8 = CH < 8 ? CH : 8;
    struct alignas(16) Tile {
        float2 dtx[K][CH];
        float dy[K][CH];
        float B[K][N];
        float C[K][N];
        float y[K][CH];
        float dx[K][CH];
        float da[K][CH];
    };
    __shared__ __align__(16) Tile tiles[kWarps<N>];
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * kWarps<N> + (threadIdx.x >> 5);
    const int nblk = blocks * p.G;
    if (unit >= slots * nblk) return;
    const long long slot = unit / nblk;
    const int block = static_cast<int>(unit % nblk);
    float* par = p.par_part + slot * ssm_par_stride(p.D, N);
    Place w;
    if (!find_place<CH>(p, slot, block, seg, blocks, w)) return;
    Tile& tile = tiles[threadIdx.x >> 5];

    const int ch = lane / LPC, q = lane % LPC;
    const bool mine = ch < w.nd;
    const long long so = (static_cast<long long>(w.n) * p.D + w.d0 + ch) * N + 4 * q;
    const long long ao = static_cast<long long>(w.d0 + ch) * N + 4 * q;
    float A2[4], g[4], dA[4] = {0.f, 0.f, 0.f, 0.f};
    {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), s = a;
        if (mine) {
            a = *reinterpret_cast<const float4*>(p.A + ao);
            if (w.last && p.d_final_state) s = *reinterpret_cast<const float4*>(p.d_final_state + so);
        }
        A2[0] = a.x * kLog2e; A2[1] = a.y * kLog2e; A2[2] = a.z * kLog2e; A2[3] = a.w * kLog2e;
        g[0] = s.x; g[1] = s.y; g[2] = s.z; g[3] = s.w;
    }
    const int tok = lane / G::PARTS, c0 = lane % G::PARTS * EPL;
    const int ne = tok < K ? max(0, min(EPL, w.nd - c0)) : 0;
    float dskip[EPL], bias[EPL], s_dD[EPL], s_db[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        dskip[e] = (p.D_skip && e < ne) ? p.D_skip[w.d0 + c0 + e] : 0.f;
        bias[e] = (p.dt_bias && e < ne) ? p.dt_bias[w.d0 + c0 + e] : 0.f;
        s_dD[e] = s_db[e] = 0.f;
    }
    const long long row0 = static_cast<long long>(w.b) * p.T;
    const T* u = static_cast<const T*>(p.u) + row0 * p.u_stride + w.d0 + c0;
    const T* dt = static_cast<const T*>(p.dt) + row0 * p.dt_stride + w.d0 + c0;
    const T* z = p.z ? static_cast<const T*>(p.z) + row0 * p.z_stride + w.d0 + c0 : nullptr;
    const long long dense = row0 * p.D + w.d0 + c0;
    const T* d_out = static_cast<const T*>(p.d_out) + dense;
    T* du = static_cast<T*>(p.du) + dense;
    T* ddt = static_cast<T*>(p.ddt) + dense;
    T* dz = z ? static_cast<T*>(p.dz) + dense : nullptr;
    const T* Bm = static_cast<const T*>(p.Bm) + row0 * p.B_stride + w.g * N;
    const T* Cm = static_cast<const T*>(p.Cm) + row0 * p.C_stride + w.g * N;
    using Rows = RowTile<T, N, VEC>;
    const long long rows = p.cu_seqlens ? p.T : static_cast<long long>(p.nseq) * p.T;
    float* bc = p.bc_part + (static_cast<long long>(block) * rows + row0) * 2 * N;

    const int tiles_n = (w.s1 - w.s0 + K - 1) / K;
    for (int it = tiles_n - 1; it >= 0; --it) {
        const int t = w.s0 + it * K;
        const int nt = min(K, w.s1 - t);
        const int n_in = tok < nt ? ne : 0;
        float4 hs = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mine) hs = *reinterpret_cast<const float4*>(p.saved + ((w.chunk0 + it) * p.D + w.d0 + ch) * N + 4 * q);
        float ux[EPL], rx[EPL], zx[EPL], gx[EPL];
        unpack<T, EPL>(load_raw<T, EPL, VEC>(u + (t + tok) * p.u_stride, n_in), ux);
        unpack<T, EPL>(load_raw<T, EPL, VEC>(dt + (t + tok) * p.dt_stride, n_in), rx);
        if (z) unpack<T, EPL>(load_raw<T, EPL, VEC>(z + (t + tok) * p.z_stride, n_in), zx);
        unpack<T, EPL>(load_raw<T, EPL, VEC>(d_out + (t + tok) * static_cast<long long>(p.D), n_in), gx);
        {
            Rows r;
            r.load(Bm + t * p.B_stride, p.B_stride, nt, lane);
            r.store(&tile.B[0][0], lane);
            r.load(Cm + t * p.C_stride, p.C_stride, nt, lane);
            r.store(&tile.C[0][0], lane);
        }
        if (tok < K) {
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                float d = rx[e] + bias[e];
                if (p.softplus) d = softplus(d);
                d = e < n_in ? d : 0.f;
                tile.dtx[tok][c0 + e] = make_float2(d, d * ux[e]);
                tile.dy[tok][c0 + e] = z ? gx[e] * zx[e] * sigmoid(zx[e]) : gx[e];
            }
        }
        __syncwarp();
        // the tile forward again: decays and the state before every token
        float a[K][4], h[K + 1][4], s1[K], s2[K];
        h[0][0] = hs.x; h[0][1] = hs.y; h[0][2] = hs.z; h[0][3] = hs.w;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float2 d = tile.dtx[k][ch];
            const float4 b = *reinterpret_cast<const float4*>(&tile.B[k][4 * q]);
            const float4 c = *reinterpret_cast<const float4*>(&tile.C[k][4 * q]);
            const float bv[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                a[k][i] = ex2(d.x * A2[i]);
                h[k + 1][i] = fmaf(a[k][i], h[k][i], d.y * bv[i]);
            }
            s1[k] = fmaf(c.x, h[k + 1][0], c.y * h[k + 1][1]) + fmaf(c.z, h[k + 1][2], c.w * h[k + 1][3]);
        }
        put_channel_sums<LPC, CH>(s1, q, ch, &tile.y[0][0]);
        // and back
#pragma unroll
        for (int k = K - 1; k >= 0; --k) {
            const float2 d = tile.dtx[k][ch];
            const float dy = tile.dy[k][ch];
            const float4 b = *reinterpret_cast<const float4*>(&tile.B[k][4 * q]);
            const float4 c = *reinterpret_cast<const float4*>(&tile.C[k][4 * q]);
            const float bv[4] = {b.x, b.y, b.z, b.w}, cv[4] = {c.x, c.y, c.z, c.w};
            float v[8], sx = 0.f, sa = 0.f;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float e = fmaf(cv[i], dy, g[i]);
                v[i] = e * d.y;
                v[4 + i] = dy * h[k + 1][i];
                sx = fmaf(e, bv[i], sx);
                g[i] = a[k][i] * e;
                const float qq = g[i] * h[k][i];
                sa = fmaf(A2[i], qq, sa);
                dA[i] = fmaf(d.x, qq, dA[i]);
            }
            s1[k] = sx;
            s2[k] = sa;
            across_channels<LPC, CH>(v, ch);
            if (k < nt && ch < 8) {
#pragma unroll
                for (int i = 0; i < 8 / M8; ++i) {
                    const int idx = i * M8 + ch;
                    bc[(t + k) * static_cast<long long>(2 * N) + (idx >> 2) * N + 4 * q + (idx & 3)] = v[i];
                }
            }
        }
        put_channel_sums<LPC, CH>(s1, q, ch, &tile.dx[0][0]);
        put_channel_sums<LPC, CH>(s2, q, ch, &tile.da[0][0]);
        __syncwarp();
        if (n_in > 0) {
            float o1[EPL], o2[EPL], o3[EPL];
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                const float2 d = tile.dtx[tok][c0 + e];
                const float dy = tile.dy[tok][c0 + e], dx = tile.dx[tok][c0 + e];
                const float y = fmaf(dskip[e], ux[e], tile.y[tok][c0 + e]);
                float dr = fmaf(ux[e], dx, tile.da[tok][c0 + e] * (1.f / kLog2e));
                if (p.softplus) dr *= sigmoid(rx[e] + bias[e]);
                o1[e] = fmaf(d.x, dx, dskip[e] * dy);
                o2[e] = dr;
                o3[e] = z ? gx[e] * y * dsilu(zx[e], sigmoid(zx[e])) : 0.f;
                if (e < n_in) {
                    s_dD[e] = fmaf(dy, ux[e], s_dD[e]);
                    s_db[e] += dr;
                }
            }
            const long long at = (t + tok) * static_cast<long long>(p.D);
            store_raw<T, EPL, VEC>(du + at, pack<T, EPL>(o1), n_in);
            store_raw<T, EPL, VEC>(ddt + at, pack<T, EPL>(o2), n_in);
            if (z) store_raw<T, EPL, VEC>(dz + at, pack<T, EPL>(o3), n_in);
        }
        __syncwarp();
    }
    if (mine) {
        *reinterpret_cast<float4*>(par + ao) = make_float4(dA[0], dA[1], dA[2], dA[3]);
        if (w.first && p.d_initial_state) *reinterpret_cast<float4*>(p.d_initial_state + so) = make_float4(g[0], g[1], g[2], g[3]);
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        const float sd = over_tokens<G::PARTS>(s_dD[e]), sb = over_tokens<G::PARTS>(s_db[e]);
        if (lane < G::PARTS && e < ne) {
            par[static_cast<long long>(p.D) * N + w.d0 + c0 + e] = sd;
            par[static_cast<long long>(p.D) * N + p.D + w.d0 + c0 + e] = sb;
        }
    }
}

// dB and dC: the partial rows of a group's channel blocks, added in order.
template <typename T>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const SsmBcArgs p) {
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int w2 = 2 * p.N;
    const long long per = p.rows * w2;
    if (id >= per * p.G) return;
    const int g = static_cast<int>(id / per);
    const long long row = id % per / w2;
    const int col = static_cast<int>(id % w2);
    const float* src = p.bc_part + static_cast<long long>(g) * p.blocks * per + id % per;
    float s = 0.f;
#pragma unroll 8
    for (int i = 0; i < p.blocks; ++i) s += __ldg(src + i * per);
    T* out = static_cast<T*>(col < p.N ? p.dB : p.dC);
    out[(row * p.G + g) * p.N + (col < p.N ? col : col - p.N)] = from_f32<T>(s);
}

template <typename T, int N>
cudaError_t bwd_n(const SsmArgs& a, cudaStream_t stream) {
    const int blocks = ssm_group_blocks(a.D, a.G, N);
    const long long units = static_cast<long long>(a.nseq) * blocks * a.G;
    const unsigned grid = static_cast<unsigned>((units + kWarps<N> - 1) / kWarps<N>);
    // out is not written here; d_out, du, ddt and dz are dense rows of D as it is, 16-byte aligned all
    if (all_vec<T, N, 4>(a))
        ssm_bwd_kernel<T, N, true><<<grid, 32 * kWarps<N>, 0, stream>>>(a, 1 << 30, a.nseq, blocks);
    else
        ssm_bwd_kernel<T, N, false><<<grid, 32 * kWarps<N>, 0, stream>>>(a, 1 << 30, a.nseq, blocks);
    return cudaGetLastError();
}

}  // namespace

int ssm_group_blocks(int D, int G, int N) {
    const int ch = 128 / N;
    return (D / G + ch - 1) / ch;
}

cudaError_t launch_ssm_bwd(const SsmArgs& a, cudaStream_t stream) {
#define GDN_SSM_N(T)                                 \
    switch (a.N) {                                   \
        case 8: return bwd_n<T, 8>(a, stream);       \
        case 16: return bwd_n<T, 16>(a, stream);     \
        case 32: return bwd_n<T, 32>(a, stream);     \
        case 64: return bwd_n<T, 64>(a, stream);     \
        default: return bwd_n<T, 128>(a, stream);    \
    }
    if (a.dtype == 0) {
        GDN_SSM_N(uint16_t)
    }
    GDN_SSM_N(float)
#undef GDN_SSM_N
}

cudaError_t launch_ssm_bc(const SsmBcArgs& a, cudaStream_t stream) {
    const long long n = a.rows * 2 * a.N * a.G;
    if (n == 0) return cudaSuccess;
    const unsigned grid = static_cast<unsigned>((n + 255) / 256);
    if (a.dtype == 0)
        ssm_bc_kernel<uint16_t><<<grid, 256, 0, stream>>>(a);
    else
        ssm_bc_kernel<float><<<grid, 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace gdn
