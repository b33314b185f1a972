// Selective state space scan: forward, and the single-token step for decode.
// The layout is described in gdn_ssm_common.cuh; gdn_ssm_bwd.cu holds the
// reverse mode.
#include "gdn_ssm_common.cuh"

namespace gdn {

namespace {

using namespace ssm;

template <int N>
constexpr int kWarps = N >= 64 ? 2 : 4;

template <typename T, int N>
__global__ void __launch_bounds__(32 * kWarps<N>) ssm_fwd_kernel(const SsmArgs p, int seg, long long slots, int blocks) {
    using G = Geo<N>;
    constexpr int CH = G::CH, EPL = G::EPL;
    struct Tile {
        float2 dtx[K][CH];
        float B[K][N];
        float C[K][N];
        float y[K][CH];
    };
    __shared__ __align__(16) Tile tiles[kWarps<N>];
    if (blockIdx.x == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const int lane = threadIdx.x & 31;
    const long long unit = static_cast<long long>(blockIdx.x) * kWarps<N> + (threadIdx.x >> 5);
    const int nblk = blocks * p.G;
    if (unit >= slots * nblk) return;
    Place w;
    if (!find_place<CH>(p, unit / nblk, static_cast<int>(unit % nblk), seg, blocks, w)) return;
    Tile& tile = tiles[threadIdx.x >> 5];

    // this lane's states
    const int ch = lane / G::LPC, q = lane % G::LPC;
    const bool mine = ch < w.nd;
    const long long so = (static_cast<long long>(w.n) * p.D + w.d0 + ch) * N + 4 * q;
    float A2[4], h[4];
    {
        float4 a = make_float4(0.f, 0.f, 0.f, 0.f), s = a;
        if (mine) {
            a = *reinterpret_cast<const float4*>(p.A + static_cast<long long>(w.d0 + ch) * N + 4 * q);
            if (w.first && p.initial_state) s = *reinterpret_cast<const float4*>(p.initial_state + so);
        }
        A2[0] = a.x * kLog2e; A2[1] = a.y * kLog2e; A2[2] = a.z * kLog2e; A2[3] = a.w * kLog2e;
        h[0] = s.x; h[1] = s.y; h[2] = s.z; h[3] = s.w;
    }
    // its share of a tile's elements
    const int tok = lane / G::PARTS, c0 = lane % G::PARTS * EPL;
    const int ne = tok < K ? max(0, min(EPL, w.nd - c0)) : 0;
    float dskip[EPL], bias[EPL];
#pragma unroll
    for (int e = 0; e < EPL; ++e) {
        dskip[e] = (p.D_skip && e < ne) ? p.D_skip[w.d0 + c0 + e] : 0.f;
        bias[e] = (p.dt_bias && e < ne) ? p.dt_bias[w.d0 + c0 + e] : 0.f;
    }
    const long long row0 = static_cast<long long>(w.b) * p.T;
    const T* u = static_cast<const T*>(p.u) + row0 * p.u_stride + w.d0 + c0;
    const T* dt = static_cast<const T*>(p.dt) + row0 * p.dt_stride + w.d0 + c0;
    const T* z = p.z ? static_cast<const T*>(p.z) + row0 * p.z_stride + w.d0 + c0 : nullptr;
    const T* Bm = static_cast<const T*>(p.Bm) + row0 * p.B_stride + w.g * N;
    const T* Cm = static_cast<const T*>(p.Cm) + row0 * p.C_stride + w.g * N;
    T* out = static_cast<T*>(p.out) + row0 * p.D + w.d0 + c0;
    const bool vec_u = can_vec<T>(u, p.u_stride, EPL), vec_dt = can_vec<T>(dt, p.dt_stride, EPL);
    const bool vec_z = z && can_vec<T>(z, p.z_stride, EPL), vec_o = can_vec<T>(out, p.D, EPL);
    using Rows = RowTile<T, N>;
    const bool vec_B = can_vec<T>(Bm, p.B_stride, Rows::PE), vec_C = can_vec<T>(Cm, p.C_stride, Rows::PE);

    for (int t = w.s0; t < w.s1; t += K) {
        const int nt = min(K, w.s1 - t);
        const int n_in = tok < nt ? ne : 0;
        if (p.saved && mine)
            *reinterpret_cast<float4*>(p.saved + ((w.chunk0 + (t - w.s0) / K) * p.D + w.d0 + ch) * N + 4 * q) =
                make_float4(h[0], h[1], h[2], h[3]);
        float ux[EPL], zx[EPL];
        {
            float dx[EPL];
            unpack<T, EPL>(load_raw<T, EPL>(u + (t + tok) * p.u_stride, vec_u, n_in), ux);
            unpack<T, EPL>(load_raw<T, EPL>(dt + (t + tok) * p.dt_stride, vec_dt, n_in), dx);
            if (z) unpack<T, EPL>(load_raw<T, EPL>(z + (t + tok) * p.z_stride, vec_z, n_in), zx);
            Rows r;
            r.load(Bm + t * p.B_stride, p.B_stride, vec_B, nt, lane);
            r.store(&tile.B[0][0], lane);
            r.load(Cm + t * p.C_stride, p.C_stride, vec_C, nt, lane);
            r.store(&tile.C[0][0], lane);
            if (tok < K) {
#pragma unroll
                for (int e = 0; e < EPL; ++e) {
                    float d = dx[e] + bias[e];
                    if (p.softplus) d = softplus(d);
                    d = e < n_in ? d : 0.f;
                    tile.dtx[tok][c0 + e] = make_float2(d, d * ux[e]);
                }
            }
        }
        __syncwarp();
        float y[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const float2 d = tile.dtx[k][ch];
            const float4 b = *reinterpret_cast<const float4*>(&tile.B[k][4 * q]);
            const float4 c = *reinterpret_cast<const float4*>(&tile.C[k][4 * q]);
            h[0] = fmaf(ex2(d.x * A2[0]), h[0], d.y * b.x);
            h[1] = fmaf(ex2(d.x * A2[1]), h[1], d.y * b.y);
            h[2] = fmaf(ex2(d.x * A2[2]), h[2], d.y * b.z);
            h[3] = fmaf(ex2(d.x * A2[3]), h[3], d.y * b.w);
            y[k] = fmaf(c.x, h[0], c.y * h[1]) + fmaf(c.z, h[2], c.w * h[3]);
        }
        put_channel_sums<G::LPC, CH>(y, q, ch, &tile.y[0][0]);
        __syncwarp();
        if (n_in > 0) {
            float o[EPL];
#pragma unroll
            for (int e = 0; e < EPL; ++e) {
                o[e] = fmaf(dskip[e], ux[e], tile.y[tok][c0 + e]);
                if (z) o[e] *= zx[e] * sigmoid(zx[e]);
            }
            store_raw<T, EPL>(out + (t + tok) * static_cast<long long>(p.D), pack<T, EPL>(o), vec_o, n_in);
        }
        __syncwarp();  // the next tile overwrites this one
    }
    if (w.last && p.final_state && mine) *reinterpret_cast<float4*>(p.final_state + so) = make_float4(h[0], h[1], h[2], h[3]);
}

// One token: lane q of a channel updates four of its states where they lie.
// Bound by HBM: the state is read and written once.
template <typename T, int N>
__global__ void __launch_bounds__(256) ssm_step_kernel(const SsmStepArgs p) {
    constexpr int LPC = N / 4;
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const int q = static_cast<int>(id % LPC);
    const long long bd = id / LPC;
    const bool live = bd < static_cast<long long>(p.B) * p.D;  // whole channels: a channel's lanes agree
    const long long b = live ? bd / p.D : 0;
    const int d = live ? static_cast<int>(bd % p.D) : 0;
    long long slot = b;
    bool on = live;
    if (p.slots && live) {
        slot = p.slots[b];
        if (slot >= p.S) record_error(p.err, kErrBadSlot);
        on = slot >= 0 && slot < p.S;
    }
    float y = 0.f, uu = 0.f;
    if (on) {
        const long long so = (slot * p.D + d) * N + 4 * q;
        const float4 s = *reinterpret_cast<const float4*>(p.state + so);
        const float4 a = __ldg(reinterpret_cast<const float4*>(p.A + static_cast<long long>(d) * N + 4 * q));
        const int g = d / (p.D / p.G);
        const T* Bm = static_cast<const T*>(p.Bm) + b * p.B_stride + g * N + 4 * q;
        const T* Cm = static_cast<const T*>(p.Cm) + b * p.C_stride + g * N + 4 * q;
        float bv[4], cv[4], h[4];
        unpack<T, 4>(load_raw<T, 4>(Bm, can_vec<T>(Bm, 4, 4), 4), bv);
        unpack<T, 4>(load_raw<T, 4>(Cm, can_vec<T>(Cm, 4, 4), 4), cv);
        uu = to_f32(static_cast<const T*>(p.u)[b * p.u_stride + d]);
        float dt = to_f32(static_cast<const T*>(p.dt)[b * p.dt_stride + d]) + (p.dt_bias ? __ldg(p.dt_bias + d) : 0.f);
        if (p.softplus) dt = softplus(dt);
        const float x = dt * uu, d2 = dt * kLog2e;
        h[0] = fmaf(ex2(d2 * a.x), s.x, x * bv[0]);
        h[1] = fmaf(ex2(d2 * a.y), s.y, x * bv[1]);
        h[2] = fmaf(ex2(d2 * a.z), s.z, x * bv[2]);
        h[3] = fmaf(ex2(d2 * a.w), s.w, x * bv[3]);
        *reinterpret_cast<float4*>(p.out_state + so) = make_float4(h[0], h[1], h[2], h[3]);
        y = fmaf(cv[0], h[0], cv[1] * h[1]) + fmaf(cv[2], h[2], cv[3] * h[3]);
    }
#pragma unroll
    for (int m = LPC / 2; m > 0; m /= 2) y += __shfl_xor_sync(0xffffffffu, y, m);
    if (live && q == 0) {
        if (on && p.D_skip) y = fmaf(__ldg(p.D_skip + d), uu, y);
        if (on && p.z) {
            const float z = to_f32(static_cast<const T*>(p.z)[b * p.z_stride + d]);
            y *= z * sigmoid(z);
        }
        static_cast<T*>(p.out)[b * p.D + d] = from_f32<T>(y);
    }
}

template <typename T, int N>
cudaError_t fwd_n(const SsmArgs& a, cudaStream_t stream) {
    const int blocks = (a.D / a.G + Geo<N>::CH - 1) / Geo<N>::CH;
    const long long units = static_cast<long long>(a.nseq) * blocks * a.G;
    ssm_fwd_kernel<T, N><<<static_cast<unsigned>((units + kWarps<N> - 1) / kWarps<N>), 32 * kWarps<N>, 0, stream>>>(
        a, 1 << 30, a.nseq, blocks);
    return cudaGetLastError();
}

template <typename T, int N>
cudaError_t step_n(const SsmStepArgs& a, cudaStream_t stream) {
    const long long threads = static_cast<long long>(a.B) * a.D * (N / 4);
    ssm_step_kernel<T, N><<<static_cast<unsigned>((threads + 255) / 256), 256, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace

#define GDN_SSM_N(fn, T)                          \
    switch (a.N) {                                \
        case 8: return fn<T, 8>(a, stream);       \
        case 16: return fn<T, 16>(a, stream);     \
        case 32: return fn<T, 32>(a, stream);     \
        case 64: return fn<T, 64>(a, stream);     \
        default: return fn<T, 128>(a, stream);    \
    }
#define GDN_SSM_DISPATCH(fn)              \
    if (a.dtype == 0) {                   \
        GDN_SSM_N(fn, uint16_t)           \
    }                                     \
    GDN_SSM_N(fn, float)

cudaError_t launch_ssm_fwd(const SsmArgs& a, cudaStream_t stream) { GDN_SSM_DISPATCH(fwd_n) }
cudaError_t launch_ssm_step(const SsmStepArgs& a, cudaStream_t stream) { GDN_SSM_DISPATCH(step_n) }

}  // namespace gdn
