// Gated linear recurrence: forward, reverse mode and the single-token step.
//
//   L_t = -rate softplus(lam) sigmoid(r_t),  a_t = exp(L_t),  m_t = sqrt(1 - a_t^2)
//   h_t = a_t h_{t-1} + m_t sigmoid(i_t) x_t
//
// per channel.  A token's map h -> a h + b composes with its neighbours', so a
// row of T tokens is cut into strips of kStrip tokens.  A warp holds two strips
// side by side in time, 16 lanes each with two channels a lane; it copies its
// tokens to shared memory one round ahead, forms their (a, b) in registers and
// composes them from a zero state, the strips' products (P, H) meet in shared
// memory, and each lane then walks its tokens again from the state that they
// really start from.  Every input is read once and every output written once.  A
// block is kWarps warps on consecutive tokens; where the channels alone do not
// fill the GPU a cluster of blocks works side by side on consecutive stretches
// and exchanges one (P, H) per block and channel through distributed shared
// memory.  The cluster then takes the next stretch, with the state it ended in.
// All compositions run in a fixed order.
//
// HBM would move the bytes in 40 us; 4 x 4096 x 2048 bf16 take 66 us forward (4.1
// TB/s) and 136 reverse (3.4 TB/s), 1 x 65536 x 1024 152 and 321.  What bounds them is
// latency at few warps: 12.6 active an SM forward, with 53 % of the issue slots used
// (35 instructions per element and lane pair, 26 of them the formulas' own), 46 % of
// HBM's rate and 30 % of the exponential unit's; 13.8, 39 %, 28 % and 15 % in the
// packed reverse.  Each round ends in the block's and the cluster's barrier with
// nothing between arriving and waiting, and 256 blocks on 304 places leave 48 SMs with
// one.  Sixteen tokens a strip forward and eight in reverse are what fits 128
// registers, two blocks an SM; four warps a block took 106 us and sixteen 83 where
// eight took 71.
//
// Packed sequences are one row: a sequence's first token starts from its own
// initial state, and a strip that holds such a token ignores what comes in.  The
// whole cluster waits in a round in which a warp goes through such a strip with
// its states and offsets: 1 x 16384 x 2048 bf16 take 74 us forward and 158 in
// reverse, in 12 sequences 86 and 194, in 64 94 and 235.  (Offsets in global
// memory: 94 and 197, 110 and 245.)
#include <algorithm>
#include <type_traits>

#include "gdn_cluster.cuh"
#include "gdn_kernels.h"
#include "gdn_launch.h"
#include "gdn_mix_common.cuh"

namespace gdn {

namespace {

using namespace mix;

constexpr int kWarps = 8;
constexpr int kChannels = 32;  // of a block
// Tokens of a lane's strip: what a round costs beside its tokens' own arithmetic
// is shared by more of them, as far as the registers go.
constexpr int kStripFwd = 2 * kGatedStrip, kStripBwd = kGatedStrip;

// ---------------------------------------------------------------- the gates

__device__ __forceinline__ Two same(float c) { return two(c, c); }

// exp(L) - 1 for -1/2 <= L <= 0, by the exponential series up to L^9 / 9! (what is
// cut off is below 2^-30 of it; with the roundings the error reaches 1.6 x 2^-24)
__device__ __forceinline__ Two expm1_series(Two L) {
    Two s = fma2(L, same(1.f / 362880.f), same(1.f / 40320.f));
    s = fma2(L, s, same(1.f / 5040.f));
    s = fma2(L, s, same(1.f / 720.f));
    s = fma2(L, s, same(1.f / 120.f));
    s = fma2(L, s, same(1.f / 24.f));
    s = fma2(L, s, same(1.f / 6.f));
    s = fma2(L, s, same(0.5f));
    s = fma2(L, s, same(1.f));
    return mul2(L, s);
}
// a = exp(L) and 1 - a^2 = -u (2 + u) with u = a - 1.  Each is taken from where it
// has its digits: u from the series and a = 1 + u where the decay is weak, a from the
// exponential and u = a - 1 where it is strong, since the gradients through a decay
// are proportional to a, however small it is.  SMALL: no L of this warp's channels is
// below -1/2, whatever the gate.
template <bool SMALL>
__device__ __forceinline__ void decay(Two L, Two& a, Two& gap) {
    Two u = expm1_series(L);
    a = add2(same(1.f), u);
    if constexpr (!SMALL) {
        float l0, l1, u0, u1, a0, a1;
        split(L, l0, l1);
        split(u, u0, u1);
        split(a, a0, a1);
        if (l0 < -0.5f) {
            a0 = ex2(kLog2e * l0);
            u0 = a0 - 1.f;
        }
        if (l1 < -0.5f) {
            a1 = ex2(kLog2e * l1);
            u1 = a1 - 1.f;
        }
        u = two(u0, u1);
        a = two(a0, a1);
    }
    gap = mul2(u, fma2(same(-1.f), u, same(-2.f)));
}
// f(std::true_type) where `yes`, else f(std::false_type): one branch around a loop
template <typename F>
__device__ __forceinline__ void with_flag(bool yes, F&& f) {
    if (yes)
        f(std::true_type{});
    else
        f(std::false_type{});
}
__device__ __forceinline__ float root(float x) {
    float y;
    asm("sqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ Two root_2(Two x) {
    float a, b;
    split(x, a, b);
    return two(root(a), root(b));
}

// ---------------------------------------------------------------- sequences

// The offsets of packed sequences, from shared memory where they fit: looked up
// where a strip crosses one, while the whole cluster waits.
constexpr int kOffsets = 512;
struct Offsets {
    const int32_t* at;
    int nseq;
};
// (whole block; the copies are there after its next barrier)
__device__ __forceinline__ Offsets offsets_of(const GatedArgs& p, int32_t* held) {
    if (p.nseq >= kOffsets) return Offsets{p.cu_seqlens, p.nseq};
    for (int n = threadIdx.x; n <= p.nseq; n += 32 * kWarps) held[n] = p.cu_seqlens[n];
    return Offsets{held, p.nseq};
}

// The sequence that holds a token of the row, and its ends.
struct Seq {
    int n, s0, s1;
};
__device__ __forceinline__ Seq find_seq(const Offsets& p, int t) {
    int lo = 0, hi = p.nseq - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (p.at[mid] <= t)
            lo = mid;
        else
            hi = mid - 1;
    }
    return Seq{lo, p.at[lo], p.at[lo + 1]};
}

// The next and the previous sequence that has tokens (malformed offsets stay in bounds).
__device__ __forceinline__ int next_seq(const Offsets& p, int n) {
    do ++n;
    while (n < p.nseq - 1 && p.at[n] == p.at[n + 1]);
    return min(n, p.nseq - 1);
}
__device__ __forceinline__ int previous_seq(const Offsets& p, int n) {
    do --n;
    while (n > 0 && p.at[n] == p.at[n + 1]);
    return max(n, 0);
}
// Where sequences begin and end among a strip's nk tokens from t0 on, as bits, and
// the sequences of the first and the last beginning and of the last end.
struct Marks {
    uint32_t starts, ends;
    int first, begun, last;
};
__device__ __forceinline__ Marks marks_of(const Offsets& p, const Seq& q, int t0, int nk) {
    Marks m{q.s0 == t0 ? 1u : 0u, 0, q.n, q.n, q.n};
    int e = q.s1, n = q.n;
    for (int i = 0; i < nk && e > t0 && e <= t0 + nk; ++i) {
        m.ends |= 1u << (e - 1 - t0);
        m.last = n;
        if (e == t0 + nk) break;
        n = next_seq(p, n);
        if (m.starts == 0) m.first = n;
        m.starts |= 1u << (e - t0);
        m.begun = n;
        e = p.at[n + 1];
    }
    return m;
}

// ---------------------------------------------------------------- exchange

// A map of two channels: h -> P h + H, or h -> H where `cut`.
struct Map {
    Two P, H;
    int cut;
};
__device__ __forceinline__ Two pass(const Map& m, Two h) {
    return m.cut ? m.H : fma2(m.P, h, m.H);
}
struct Exchange {
    float4 warp[2][kWarps][kChannels / 2];  // (P, H) of a channel pair: P0, P1, H0, H1
    float4 block[2][kGatedMaxCluster][kChannels / 2];
};
// A product of decays is never negative, so P0 = -1 says that the map is cut.
template <bool CUTS>
__device__ __forceinline__ Map map_of(const float4& v) {
    return Map{two(v.x, v.y), two(v.z, v.w), CUTS && v.x == -1.f};
}
template <bool CUTS>
__device__ __forceinline__ float4 packed(Two P, Two H, int cut) {
    float4 v;
    split(P, v.x, v.y);
    split(H, v.z, v.w);
    if (CUTS && cut) v.x = -1.f;
    return v;
}

// From each lane's own map (`later`: its strip is the warp's second) to the value
// that reaches its strip; `carry`, what reaches the cluster's stretch, becomes
// what leaves it.  CUTS: some maps may ignore what comes in.
template <bool CUTS>
__device__ __forceinline__ Two exchange(Exchange& sm, int parity, int warp, int lane, uint32_t rank, int C, const Map& own,
                                        bool later, Two& carry) {
    const int pr = lane & 15;
    Map far;
    far.P.v = __shfl_xor_sync(0xffffffffu, own.P.v, 16);
    far.H.v = __shfl_xor_sync(0xffffffffu, own.H.v, 16);
    far.cut = CUTS ? __shfl_xor_sync(0xffffffffu, own.cut, 16) : 0;
    if (lane < 16)  // the pair in order
        sm.warp[parity][warp][pr] = packed<CUTS>(mul2(own.P, far.P), later ? pass(own, far.H) : pass(far, own.H), own.cut | far.cut);
    __syncthreads();
    const auto strip = [&](int w) { return map_of<CUTS>(sm.warp[parity][w][pr]); };
    Two mine = carry;
    if (C > 1) {
        if (threadIdx.x < 16) {  // the whole block's map
            Two P = same(1.f), H = same(0.f);
            int cut = 0;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const Map m = strip(w);
                H = pass(m, H);
                P = mul2(P, m.P);
                cut |= m.cut;
            }
            const float4 v = packed<CUTS>(P, H, cut);
            for (int c = 0; c < C; ++c) cluster::store(&sm.block[parity][rank][pr], c, v);
        }
        cluster::sync();
        for (int c = 0; c < C; ++c) {
            if (c == static_cast<int>(rank)) mine = carry;
            carry = pass(map_of<CUTS>(sm.block[parity][c][pr]), carry);
        }
#pragma unroll
        for (int w = 0; w < kWarps - 1; ++w)
            if (w < warp) mine = pass(strip(w), mine);
    } else {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            if (w == warp) mine = carry;
            carry = pass(strip(w), carry);
        }
    }
    return later ? pass(far, mine) : mine;
}

// ---------------------------------------------------------------- memory

// A state's two channels (nd of them: 0, 1 or 2), zeros where there is none
__device__ __forceinline__ Two load_state(const float* base, long long n, int D, int d, int nd) {
    if (!base) return same(0.f);
    const float* q = base + n * D + d;
    return two(nd > 0 ? q[0] : 0.f, nd > 1 ? q[1] : 0.f);
}
__device__ __forceinline__ void touch_state(const float* base, long long n, int D, int d) {
    if (base) asm volatile("prefetch.global.L1 [%0];" ::"l"(base + n * D + d));
}
__device__ __forceinline__ void store_state(float* base, long long n, int D, int d, int nd, Two h) {
    float a, b;
    split(h, a, b);
    float* q = base + n * D + d;
    if (nd == 2 && !(D & 1)) {
        *reinterpret_cast<float2*>(q) = make_float2(a, b);
        return;
    }
    if (nd > 0) q[0] = a;
    if (nd > 1) q[1] = b;
}
// EVEN: rows of an even number of channels, so a pair is one access
template <typename T, bool EVEN>
__device__ __forceinline__ void store_pair(T* q, int nd, Two v) {
    store_raw<T, 2, EVEN>(q, pack_2<T, 2>(&v), nd);
}
template <typename T, int PB>
constexpr bool kEven = PB == 16 || (PB == 4 && sizeof(T) == 2);
// A pair of channels of a tile in shared memory
template <typename T>
__device__ __forceinline__ Two pair_at(const T* q) {
    Raw<T, 2> r;
    if constexpr (sizeof(T) == 2)
        r.w[0] = *reinterpret_cast<const uint32_t*>(q);
    else
        *reinterpret_cast<uint2*>(r.w) = *reinterpret_cast<const uint2*>(q);
    return two(r.get(0), r.get(1));
}

// A warp's copies of its SPAN x kChannels tiles of one input to shared memory,
// zeros behind the row's end and its last channel, in pieces of PB bytes (PB = 0:
// element by element and at once, for 2-byte elements at odd places).
template <typename T, int SPAN, int PB>
struct Copier {
    static constexpr int CE = PB ? PB / static_cast<int>(sizeof(T)) : 1, PER = kChannels / CE, LINES = 32 / PER > 0 ? 32 / PER : 1;
    static constexpr int COUNT = SPAN * PER / 32;
    const T* at;       // this lane's first piece of the row's first tile
    long long stride;
    int row, col, nc;
    __device__ __forceinline__ Copier(const void* base, long long stride_, long long row0, int d0, int nc_, int lane)
        : stride(stride_), row(lane / PER), col(lane % PER * CE), nc(nc_) {
        at = static_cast<const T*>(base) + row0 * stride + d0 + row * stride + col;
    }
    // the tile of tokens [t, t + SPAN) of T
    __device__ __forceinline__ void operator()(T* dst, int t, int tokens, int lane) const {
        const T* src = at + t * stride;
        const int left = tokens - t - row;
        T* to = dst + lane * CE;
#pragma unroll
        for (int i = 0; i < COUNT; ++i) {
            // (PER > 32: a line takes several turns)
            constexpr int turns = PER > 32 ? PER / 32 : 1;
            const int line = i / turns * LINES, c = i % turns * 32 * CE;
            const bool ok = line < left && col + c < nc;
            const T* from = ok ? src + line * stride + c : static_cast<const T*>(at);
            if constexpr (PB != 0)
                copy_async<T, CE>(to + i * 32 * CE, from, ok);
            else
                to[i * 32 * CE] = ok ? *from : T(0);
        }
    }
};

template <typename T, int N, int SPAN>
struct alignas(16) Tiles {
    T v[2][N][SPAN][kChannels];
};

// What the two kernels share: the warp's place in its row.
template <typename T>
struct Place {
    int warp, lane, sub, row, D, d0, d, nd, nc, C;
    uint32_t rank;
    __device__ __forceinline__ Place(const GatedArgs& p) {
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        sub = lane >> 4;
        C = p.cluster;
        row = blockIdx.y;
        rank = C > 1 ? cluster::rank() : 0;
        D = p.D;
        d0 = blockIdx.x / C * kChannels;
        nc = min(kChannels, D - d0);
        d = d0 + (lane & 15) * 2;
        nd = max(0, min(2, D - d));
    }
};

// ---------------------------------------------------------------- forward

// SEQS: packed sequences, whose ends may lie anywhere; otherwise a row is one
// sequence, and its initial state is what reaches its first strip.
template <typename T, int PB, bool SEQS>
__global__ void __launch_bounds__(32 * kWarps, 2) gated_fwd_kernel(const GatedArgs p) {
    constexpr int KS = kStripFwd, SPAN = 2 * KS;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Exchange sm;
    __shared__ int32_t held[SEQS ? kOffsets : 1];
    const Place<T> w(p);
    Tiles<T, 3, SPAN>& tile = reinterpret_cast<Tiles<T, 3, SPAN>*>(smem)[w.warp];
    if (SEQS && blockIdx.x == 0 && w.row == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const Offsets cu = SEQS ? offsets_of(p, held) : Offsets{nullptr, 1};
    if (SEQS) __syncthreads();
    const float s0 = w.nd > 0 ? -p.rate * softplus(p.lam[w.d]) : 0.f, s1 = w.nd > 1 ? -p.rate * softplus(p.lam[w.d + 1]) : 0.f;
    const Two scale = two(s0, s1);
    const bool small = __all_sync(0xffffffffu, s0 >= -0.5f && s1 >= -0.5f);
    const long long row0 = static_cast<long long>(w.row) * p.T;
    const Copier<T, SPAN, PB> cr(p.r, p.r_stride, row0, w.d0, w.nc, w.lane), ci(p.i, p.i_stride, row0, w.d0, w.nc, w.lane),
        cx(p.x, p.x_stride, row0, w.d0, w.nc, w.lane);
    T* y = static_cast<T*>(p.y) + row0 * p.D + w.d;
    const int spans = (p.T + SPAN - 1) / SPAN, strips = (p.T + kGatedStrip - 1) / kGatedStrip;
    const auto start_of = [&](int n) { return load_state(p.initial_state, n, w.D, w.d, w.nd); };
    if (p.final_state && w.rank == 0 && w.sub == 0) {  // sequences without tokens
        const int first = SEQS ? 0 : w.row, last = SEQS ? p.nseq : w.row + 1;
        for (int n = first + w.warp; n < last; n += kWarps) {
            if (SEQS ? cu.at[n] < cu.at[n + 1] : p.T > 0) continue;
            store_state(p.final_state, n, w.D, w.d, w.nd, start_of(n));
        }
    }
    const int mine0 = static_cast<int>(w.rank) * kWarps + w.warp, step = w.C * kWarps;
    const auto fetch = [&](int s, int stage) {  // the span s, if there is one
        if (s < spans) {
            cr(&tile.v[stage][0][0][0], s * SPAN, p.T, w.lane);
            ci(&tile.v[stage][1][0][0], s * SPAN, p.T, w.lane);
            cx(&tile.v[stage][2][0][0], s * SPAN, p.T, w.lane);
        }
        commit_copies();
    };
    fetch(mine0, 0);
    if (w.C > 1) cluster::sync();  // every block of the cluster is there
    Two carry = SEQS ? same(0.f) : start_of(w.row);
    Seq q{w.row, 0, SEQS ? 0 : p.T};  // that of the strip's first token
    for (int b0 = 0, round = 0; b0 < spans; b0 += step, ++round) {
        const int s = b0 + mine0;
        const int t0 = s * SPAN + w.sub * KS;  // this lane's first token: below 2^30 + 2^13
        const int nk = max(0, min(KS, p.T - t0));
        fetch(s + step, (round + 1) & 1);
        if (SEQS && nk > 0 && t0 >= q.s1) q = find_seq(cu, t0);
        // the strip holds a sequence's end, or (packed) its beginning
        const bool ends = q.s1 <= t0 + KS || (SEQS && q.s0 == t0);
        Marks mk{0, q.s1 - 1 - t0 < KS && nk > 0 ? 1u << (q.s1 - 1 - t0) : 0u, w.row, w.row, w.row};
        Two h0 = same(0.f);  // the first's initial state, on its way with the copies
        if (SEQS && ends) {
            mk = marks_of(cu, q, t0, nk);
            if (mk.starts) h0 = start_of(mk.first);
        }
        wait_copies<1>();
        __syncwarp();
        Two a[KS], b[KS];
        Map m{same(1.f), same(0.f), 0};
        if (s < spans) {
            const T* v = &tile.v[round & 1][0][w.sub * KS][(w.lane & 15) * 2];
            with_flag(small, [&](auto size) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    Two gap;
                    decay<decltype(size)::value>(mul2(scale, sigmoid_2(pair_at(v + k * kChannels))), a[k], gap);
                    const Two si = sigmoid_2(pair_at(v + (SPAN + k) * kChannels));
                    b[k] = mul2(root_2(gap), mul2(si, pair_at(v + (2 * SPAN + k) * kChannels)));
                }
            });
            if (!ends) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    m.H = fma2(a[k], m.H, b[k]);
                    m.P = mul2(m.P, a[k]);
                }
            }
            if (ends) {
                if (SEQS) {
                    // an initial state joins its first token's input, and nothing else comes in
                    int n = mk.first;
                    for (uint32_t left = mk.starts; left; left &= left - 1) {
                        const int at = __ffs(left) - 1;
#pragma unroll
                        for (int k = 0; k < KS; ++k)
                            if (k == at) b[k] = fma2(a[k], h0, b[k]);
                        n = next_seq(cu, n);
                        if (left & (left - 1)) h0 = start_of(n);
                    }
                    m.cut = mk.starts != 0;
                }
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    if (SEQS && (mk.starts >> k) & 1) m.H = same(0.f);
                    if (k < nk) m.H = fma2(a[k], m.H, b[k]);
                    m.P = mul2(m.P, a[k]);
                }
            }
        }
        Two h = exchange<SEQS>(sm, round & 1, w.warp, w.lane, w.rank, w.C, m, w.sub != 0, carry);
        T* to = y + static_cast<long long>(t0) * p.D;
        float* keep = p.saved ? p.saved + (static_cast<long long>(w.row) * strips + t0 / kGatedStrip) * p.D : nullptr;
        if (!ends) {
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (k % kGatedStrip == 0 && keep) store_state(keep, k / kGatedStrip, w.D, w.d, w.nd, h);
                h = fma2(a[k], h, b[k]);
                store_pair<T, kEven<T, PB>>(to, w.nd, h);
                to += p.D;
            }
        } else {
            int n = SEQS ? q.n : w.row;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (k >= nk) continue;
                if (k % kGatedStrip == 0 && keep) store_state(keep, k / kGatedStrip, w.D, w.d, w.nd, h);
                if (SEQS && (mk.starts >> k) & 1) h = same(0.f);
                h = fma2(a[k], h, b[k]);
                store_pair<T, kEven<T, PB>>(to, w.nd, h);
                to += p.D;
                if ((mk.ends >> k) & 1) {
                    if (p.final_state) store_state(p.final_state, n, w.D, w.d, w.nd, h);
                    if (SEQS) n = next_seq(cu, n);
                }
            }
        }
    }
    if (w.C > 1) cluster::sync();  // the others may still write here
}

// ---------------------------------------------------------------- reverse mode

// With c_t = a_t dh_t, the gradient that reaches h_{t-1}, dh_t = dout_t + c_{t+1}:
// c composes backwards as h does forwards, from the last strip to the first.
// The states before each token come from the strip's saved start.
//   dL = dh (a h_{t-1} - a^2 / m sigmoid(i) x);  dr = dL L (1 - sigmoid(r));
//   d(sigmoid(i) x) = dh m;  dlam = -rate sigmoid(lam) sum dL sigmoid(r)
// Where m = 0 (a rounds to 1) a^2 / m L has the limit 0, and the term is left out.
template <typename T, int PB, bool SEQS>
__global__ void __launch_bounds__(32 * kWarps, sizeof(T) == 2 ? 2 : 1) gated_bwd_kernel(const GatedArgs p) {
    constexpr int KS = kStripBwd, SPAN = 2 * KS;
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ Exchange sm;
    __shared__ int32_t held[SEQS ? kOffsets : 1];
    __shared__ float2 part[kWarps][32];
    const Place<T> w(p);
    Tiles<T, 4, SPAN>& tile = reinterpret_cast<Tiles<T, 4, SPAN>*>(smem)[w.warp];
    if (SEQS && blockIdx.x == 0 && w.row == 0) check_offsets(p.cu_seqlens, p.nseq, p.T, p.err);
    const Offsets cu = SEQS ? offsets_of(p, held) : Offsets{nullptr, 1};
    if (SEQS) __syncthreads();
    const float s0 = w.nd > 0 ? -p.rate * softplus(p.lam[w.d]) : 0.f, s1 = w.nd > 1 ? -p.rate * softplus(p.lam[w.d + 1]) : 0.f;
    const Two scale = two(s0, s1);
    const bool small = __all_sync(0xffffffffu, s0 >= -0.5f && s1 >= -0.5f);
    const long long row0 = static_cast<long long>(w.row) * p.T;
    const Copier<T, SPAN, PB> cr(p.r, p.r_stride, row0, w.d0, w.nc, w.lane), ci(p.i, p.i_stride, row0, w.d0, w.nc, w.lane),
        cx(p.x, p.x_stride, row0, w.d0, w.nc, w.lane), cg(p.d_out, p.D, row0, w.d0, w.nc, w.lane);
    const long long out0 = row0 * p.D + w.d;
    const int spans = (p.T + SPAN - 1) / SPAN, strips = (p.T + KS - 1) / KS;
    const auto start_of = [&](int n) { return load_state(p.initial_state, n, w.D, w.d, w.nd); };
    const auto end_of = [&](int n) { return load_state(p.d_final_state, n, w.D, w.d, w.nd); };
    if (p.d_initial_state && w.rank == 0 && w.sub == 0) {  // sequences without tokens pass the final state's gradient on
        const int first = SEQS ? 0 : w.row, last = SEQS ? p.nseq : w.row + 1;
        for (int n = first + w.warp; n < last; n += kWarps) {
            if (SEQS ? cu.at[n] < cu.at[n + 1] : p.T > 0) continue;
            store_state(p.d_initial_state, n, w.D, w.d, w.nd, end_of(n));
        }
    }
    const int mine0 = static_cast<int>(w.rank) * kWarps + w.warp, step = w.C * kWarps;
    const auto fetch = [&](int s, int stage) {
        if (s >= 0) {
            cr(&tile.v[stage][0][0][0], s * SPAN, p.T, w.lane);
            ci(&tile.v[stage][1][0][0], s * SPAN, p.T, w.lane);
            cx(&tile.v[stage][2][0][0], s * SPAN, p.T, w.lane);
            cg(&tile.v[stage][3][0][0], s * SPAN, p.T, w.lane);
        }
        commit_copies();
    };
    fetch(spans - 1 - mine0, 0);
    if (w.C > 1) cluster::sync();  // every block of the cluster is there
    Two carry = SEQS ? same(0.f) : end_of(w.row), dlam = same(0.f);
    Seq q{w.row, SEQS ? p.T : 0, p.T};  // that of the strip's first token
    for (int b0 = 0, round = 0; b0 < spans; b0 += step, ++round) {
        const int s = spans - 1 - (b0 + mine0);  // from the last span on
        const int t0 = s * SPAN + w.sub * KS;
        const int nk = s < 0 ? 0 : max(0, min(KS, p.T - t0));
        __syncwarp();  // everyone is through with the tile that this one replaces
        fetch(s - step, (round + 1) & 1);
        Two h = same(0.f);
        if (nk > 0) h = load_state(p.saved, static_cast<long long>(w.row) * strips + 2 * s + w.sub, w.D, w.d, w.nd);
        if (SEQS && nk > 0 && t0 < q.s0) q = find_seq(cu, t0);
        // the strip holds a sequence's beginning, or (packed) its end, or is not full
        const bool ends = q.s0 == t0 || nk < KS || (SEQS && q.s1 <= t0 + KS);
        Marks mk{t0 == 0 ? 1u : 0u, 0, w.row, w.row, w.row};
        if (SEQS && ends) {
            mk = marks_of(cu, q, t0, nk);
            // (no registers to hold them: they come as far as the cache)
            if (mk.starts && w.nd > 0) touch_state(p.initial_state, mk.first, w.D, w.d);
            if (mk.ends && w.nd > 0) touch_state(p.d_final_state, mk.last, w.D, w.d);
        }
        wait_copies<1>();
        __syncwarp();
        const T* v = &tile.v[round & 1][0][w.sub * KS][(w.lane & 15) * 2];
        const auto at = [&](int which, int k) { return pair_at(v + (which * SPAN + k) * kChannels); };
        // per token: a, m, sigmoid(i) and the state before it
        Two a[KS], mt[KS], si[KS], hp[KS];
        Map m{same(1.f), same(0.f), 0};
        if (nk > 0) {
            with_flag(small, [&](auto size) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    Two gap;
                    decay<decltype(size)::value>(mul2(scale, sigmoid_2(at(0, k))), a[k], gap);
                    mt[k] = root_2(gap);
                    si[k] = sigmoid_2(at(1, k));
                }
            });
            int n = mk.first;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                if (SEQS && (mk.starts >> k) & 1) {
                    h = start_of(n);
                    n = next_seq(cu, n);
                }
                hp[k] = h;
                h = fma2(a[k], h, mul2(mt[k], mul2(si[k], at(2, k))));
            }
            if (!ends) {
#pragma unroll
                for (int k = KS - 1; k >= 0; --k) {
                    m.H = mul2(a[k], add2(at(3, k), m.H));
                    m.P = mul2(m.P, a[k]);
                }
            } else {
                n = mk.last;
                m.cut = SEQS && mk.ends != 0;
#pragma unroll
                for (int k = KS - 1; k >= 0; --k) {
                    if (k >= nk) continue;  // the row's last strip may be short: its other tokens are not there
                    if (SEQS && (mk.ends >> k) & 1) {  // nothing comes from the next sequence
                        m.H = end_of(n);
                        n = previous_seq(cu, n);
                    }
                    m.H = mul2(a[k], add2(at(3, k), m.H));
                    m.P = mul2(m.P, a[k]);
                }
            }
        }
        __syncwarp();
        Two c = exchange<SEQS>(sm, round & 1, w.warp, w.lane, w.rank, w.C, m, w.sub == 0, carry);
        if (nk > 0) {
            long long o = out0 + static_cast<long long>(t0 + KS - 1) * p.D;
            const auto token = [&](int k) {
                const Two dh = add2(at(3, k), c), sr = sigmoid_2(at(0, k)), gx = mul2(si[k], at(2, k));
                float m0, m1;
                split(mt[k], m0, m1);
                const Two inv = two(m0 > 0.f ? rcp(m0) : 0.f, m1 > 0.f ? rcp(m1) : 0.f);
                // a h_{t-1} - a^2 / m gx = a (h_{t-1} - a / m gx)
                const Two past = fma2(mul2(mul2(a[k], inv), same(-1.f)), gx, hp[k]);
                c = mul2(a[k], dh);
                const Two dL = mul2(c, past), dg = mul2(dh, mt[k]);
                dlam = fma2(dL, sr, dlam);
                store_pair<T, kEven<T, PB>>(static_cast<T*>(p.dx) + o, w.nd, mul2(dg, si[k]));
                store_pair<T, kEven<T, PB>>(static_cast<T*>(p.dr) + o, w.nd, mul2(mul2(dL, mul2(scale, sr)), fma2(same(-1.f), sr, same(1.f))));
                store_pair<T, kEven<T, PB>>(static_cast<T*>(p.di) + o, w.nd, mul2(mul2(dg, gx), fma2(same(-1.f), si[k], same(1.f))));
            };
            if (!ends) {
#pragma unroll
                for (int k = KS - 1; k >= 0; --k, o -= p.D) token(k);
            } else {
                int end = mk.last, start = mk.begun;
#pragma unroll
                for (int k = KS - 1; k >= 0; --k, o -= p.D) {
                    if (k >= nk) continue;
                    if (SEQS && (mk.ends >> k) & 1) {
                        c = end_of(end);
                        end = previous_seq(cu, end);
                    }
                    token(k);
                    if ((mk.starts >> k) & 1) {
                        if (p.d_initial_state) store_state(p.d_initial_state, start, w.D, w.d, w.nd, c);
                        if (SEQS) start = previous_seq(cu, start);
                    }
                }
            }
        }
    }
    float a0, a1;
    split(dlam, a0, a1);
    part[w.warp][w.lane] = make_float2(a0, a1);
    __syncthreads();
    if (threadIdx.x < kChannels) {  // a channel per thread
        const int pr = threadIdx.x / 2, d = w.d0 + static_cast<int>(threadIdx.x);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < kWarps; ++k) {
            const float2 u = part[k][pr], v = part[k][16 + pr];
            sum += threadIdx.x & 1 ? u.y + v.y : u.x + v.x;
        }
        if (d < p.D) p.partial[(static_cast<long long>(w.row) * w.C + w.rank) * p.D + d] = -p.rate * sigmoid(p.lam[d]) * sum;
    }
    if (w.C > 1) cluster::sync();
}

// ---------------------------------------------------------------- one token

// Four channels a thread in accesses of all four, or, where widths, strides or
// addresses do not allow it, one; each input and state once through registers.  Bound
// by the launch (64 x 2048 bf16: 2.7 us inside a graph, 0.3 of bytes).
template <typename T, int E>
__global__ void __launch_bounds__(256) gated_step_kernel(const GatedStepArgs p) {
    const int per = p.D / E;  // (E is one where it does not divide the width)
    const long long id = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long b = id / per;
    if (b >= p.B) return;
    const int d = static_cast<int>(id % per) * E;
    long long slot = b;
    if (p.slots) {
        slot = p.slots[b];
        if (slot >= p.S) record_error(p.err, kErrBadSlot);
    }
    const bool on = slot >= 0 && slot < p.S;
    const int n = on ? E : 0;
    const Raw<float, E> rl = load_raw<float, E>(p.lam + d, E);
    const Raw<T, E> rr = load_raw<T, E>(static_cast<const T*>(p.r) + b * p.r_stride + d, n);
    const Raw<T, E> ri = load_raw<T, E>(static_cast<const T*>(p.i) + b * p.i_stride + d, n);
    const Raw<T, E> rx = load_raw<T, E>(static_cast<const T*>(p.x) + b * p.x_stride + d, n);
    Raw<float, E> h;  // not load_raw: the cache may be written in place
    const long long so = (on ? slot : 0) * p.D + d;
#pragma unroll
    for (int e = 0; e < E; ++e) h.w[e] = 0;
    if (on) {
        if constexpr (E == 4) {
            const float4 v = *reinterpret_cast<const float4*>(p.state + so);
            h.w[0] = __float_as_uint(v.x); h.w[1] = __float_as_uint(v.y);
            h.w[2] = __float_as_uint(v.z); h.w[3] = __float_as_uint(v.w);
        } else {
            h.w[0] = __float_as_uint(p.state[so]);
        }
    }
    float out[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        Two a, gap;
        decay<false>(same(-p.rate * softplus(rl.get(e)) * sigmoid(rr.get(e))), a, gap);
        float a0, m0, skip;
        split(a, a0, skip);
        split(gap, m0, skip);
        out[e] = on ? fmaf(a0, h.get(e), root(m0) * (sigmoid(ri.get(e)) * rx.get(e))) : 0.f;
    }
    if (on) store_raw<float, E>(p.out_state + so, pack<float, E>(out), E);
    store_raw<T, E>(static_cast<T*>(p.y) + b * p.D + d, pack<T, E>(out), E);
}

// ---------------------------------------------------------------- launches

// Every row of these starts at a multiple of `bytes`
template <typename T>
bool fits(int bytes, int D, std::initializer_list<const void*> ptrs, std::initializer_list<long long> strides) {
    const int E = bytes / static_cast<int>(sizeof(T));
    if (D % E != 0) return false;
    for (const void* q : ptrs)
        if (q && reinterpret_cast<uintptr_t>(q) % bytes != 0) return false;
    for (long long s : strides)
        if (s % E != 0) return false;
    return true;
}

template <auto kernel>
cudaError_t launch_clusters(size_t smem, const GatedArgs& a, cudaStream_t stream) {
    static std::atomic<uint64_t> done{0};
    const cudaError_t e = allow_once(kernel, smem, false, done);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>((a.D + kChannels - 1) / kChannels * a.cluster), a.rows);
    cfg.blockDim = dim3(32 * kWarps);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = a.cluster;
    attr.val.clusterDim.y = 1;
    attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = a.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <typename T, int PB>
cudaError_t launch_pieces(const GatedArgs& a, bool backward, cudaStream_t stream) {
    constexpr size_t bwd = sizeof(Tiles<T, 4, 2 * kStripBwd>) * kWarps, fwd = sizeof(Tiles<T, 3, 2 * kStripFwd>) * kWarps;
    if (a.cu_seqlens)
        return backward ? launch_clusters<gated_bwd_kernel<T, PB, true>>(bwd, a, stream)
                        : launch_clusters<gated_fwd_kernel<T, PB, true>>(fwd, a, stream);
    return backward ? launch_clusters<gated_bwd_kernel<T, PB, false>>(bwd, a, stream)
                    : launch_clusters<gated_fwd_kernel<T, PB, false>>(fwd, a, stream);
}
// Copies to shared memory in the widest pieces that every row starts on: 4 x 4096
// x 2048 bf16 65 us forward in 16 bytes, 126 in 4, 174 one element at a time (2 x
// 2048 x 2048 fp32 29 and 58).
template <typename T>
cudaError_t launch(const GatedArgs& a, bool backward, cudaStream_t stream) {
    const auto ok = [&](int bytes) { return fits<T>(bytes, a.D, {a.x, a.r, a.i}, {a.x_stride, a.r_stride, a.i_stride}); };
    if (ok(16)) return launch_pieces<T, 16>(a, backward, stream);
    if constexpr (sizeof(T) == 2) {
        if (!ok(4)) return launch_pieces<T, 0>(a, backward, stream);
    }
    return launch_pieces<T, 4>(a, backward, stream);
}

}  // namespace

// Blocks of a row side by side: as many as are resident together, none without a
// span.  Forward and reverse in us with 1, 2, 4 and 8 of them: 1 x 65536 x 1024
// 586 / 1410, 387 / 911, 197 / 520, 152 / 321; 1 x 16384 x 2048 150 / 375, 102 / 259,
// 75 / 159, 82 / 171 (four are what is resident); 1 x 4096 x 256 39 / 78, 28 / 53,
// 16 / 30, 10 / 18; but 4 x 4096 x 2048, where the rows fill the GPU, 65 / 136,
// 74 / 157, 76 / 163, 91 / 177.
int gated_cluster(int rows, int T, int D, int dtype, bool backward) {
    const long long units = static_cast<long long>(rows) * ((D + kChannels - 1) / kChannels);
    const int slots = 152 * (dtype == 1 ? 1 : 2), span = 2 * (backward ? kStripBwd : kStripFwd);
    int c = 1;
    while (c < kGatedMaxCluster && units * c * 2 <= slots && static_cast<long long>(T) > static_cast<long long>(c) * kWarps * span) c *= 2;
    return c;
}

cudaError_t launch_gated_fwd(const GatedArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, false, stream) : launch<uint16_t>(a, false, stream);
}
cudaError_t launch_gated_bwd(const GatedArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch<float>(a, true, stream) : launch<uint16_t>(a, true, stream);
}

namespace {
template <typename T>
cudaError_t launch_step(const GatedStepArgs& a, cudaStream_t stream) {
    const bool vec = fits<T>(4 * static_cast<int>(sizeof(T)), a.D, {a.x, a.r, a.i}, {a.x_stride, a.r_stride, a.i_stride});
    const long long n = static_cast<long long>(a.B) * (vec ? a.D / 4 : a.D);
    const unsigned blocks = static_cast<unsigned>((n + 255) / 256);
    if (vec)
        gated_step_kernel<T, 4><<<blocks, 256, 0, stream>>>(a);
    else
        gated_step_kernel<T, 1><<<blocks, 256, 0, stream>>>(a);
    return cudaGetLastError();
}
}  // namespace

cudaError_t launch_gated_step(const GatedStepArgs& a, cudaStream_t stream) {
    return a.dtype == 1 ? launch_step<float>(a, stream) : launch_step<uint16_t>(a, stream);
}

}  // namespace gdn
