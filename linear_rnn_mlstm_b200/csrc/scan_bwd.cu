// Backward of the selective state-space scan.  With the gated cotangent
// e_t = dy_t z_t sigmoid(z_t), the decay a_t = exp(d_t A) and the states formed
// again from the inputs:
//
//   g_t = C_t e_t + a_{t+1} g_{t+1}            (cotangent of the state)
//   dC_t = sum_c e_t h_t,  dB_t = sum_c g_t d_t x_t
//   s1 = sum_n g_t B_t,  s2 = sum_n A g_t a_t h_{t-1},  dA = sum_t d_t g_t a_t h_{t-1}
//   dx = s1 d_t + D e_t,  ddelta = (s2 + s1 x_t) softplus',  dz = dy y' silu'(z)
//
// Three passes over segments of 64 tokens, so that every segment of every
// channel runs at once:
//   1. scan_bwd_summary: each segment's state from a zero start, also as it is at
//      every 8th token, and what the segment's outputs alone send back to the
//      state before it, sum_t (prod a) C_t e_t; all from one sweep in token order.
//   2. scan_bwd_fold: chains them, states forwards and cotangents backwards.
//   3. scan_bwd_grad: chunk by chunk from a segment's last, 8 tokens are run
//      forwards with states and decays kept in registers, and backwards.  A chunk
//      starts from pass 1's state plus the segment's true start, decayed.
//      (Forming the chunks' starts by a second sweep in this pass cost 22 of its
//      91 instructions per pair of states; the stored ones cost 16 bytes of
//      traffic per (channel, token) at N = 16.)
// Every sum over channels or tokens has a fixed order: registers over a warp's
// channel groups, shuffles, shared memory over the CTA's warps, and rows of
// partial sums over CTAs in a last pass.  No atomics.
//
// Lanes: LN share a channel, two states each (packed fp32 pairs).  The 8 tokens
// of a chunk times a warp's 32 / LN channels are 32 (channel, token) pairs at
// LN = 8, so a lane also prepares the step size and finishes the gradients of
// one pair (two at LN = 4, for up to 8 states); sums over states reach it by state_sum.
//
// What bounds it: issue slots, about 80 instructions per pair of states and warp in
// pass 3, 26 of them the recurrences' own, the others the pairs' preparation and
// finish, three sums over states and two over channels; and next to them shared memory's
// rate, which 8- and 16-byte reads take two and four cycles of.  Measured on one B200 for
// 4 x 2048 x 2048 x 16 bf16, gated: 0.60 ms (summary 151 us, fold 26, gradients 426,
// last sums 16), floor 36 us at HBM's rate; 1 x 8192 x 2048 0.60 ms with 16 states, 0.38
// with 8.  Steps: 0.99 ms as first built; registers held to
// 128 for two CTAs per SM 0.78; chunk starts stored, their copies a chunk ahead 0.73
// (read when needed 1.06); B and C read where they are used, which ends the spills, 0.67;
// one kernel for the last sums 0.66; 32 segments' loads in flight in the fold 0.65; one
// barrier a chunk and the rates in shared memory 0.62; a chunk's three state sums together,
// C read once, 0.60; growing states kept in fp32's range at no cost (by a branch on large
// exponents 0.615; the summary checks once a segment, once a chunk took 3 us more).  Slower: d, d x and e stored as pairs and read by token with the
// decays kept 0.75, B and C widened 0.61, packed additions in the sums over lanes 0.61.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "scan.cuh"

namespace xlstm {

xlstm_status check_scan(int B, int S, int C, int N, int G, xlstm_dtype dt, xlstm_delta_act act);

namespace {

constexpr int kSeg = 64;                     // tokens per segment
constexpr int kTok = 8;                      // tokens per chunk
constexpr int kWarps = 8, kThreads = kWarps * 32;
constexpr float kFar = 8.5e37f;              // 2^126
// M, a template argument below: channel groups that a warp works through one after the
// other.  Two share the sums over channels; one makes twice the CTAs of half the length
// and half the shared memory.  bf16 4 x 2048 x 2048: 600 us with two, 679 with one; where
// two would not give every SM a CTA, and in fp32, whose tiles leave room for one CTA of
// two groups per SM, one is faster (when both were last built: 2 x 333 x 272 fp32 26 us
// against 38, 1 x 2048 x 2048 fp32 205 against 262).

struct ScanBwdArgs {
    const void *x, *delta, *Bm, *Cm, *z, *dy;
    const float *A, *D, *delta_bias, *h0, *dh;
    void *dx, *ddelta, *dz, *dBm, *dCm;
    float *dA, *dD, *ddelta_bias, *dh0;
    float *hseg, *gseg, *dseg;               // [segs, B, C, N] twice, [segs, B, C]
    float *hchunk, *dchunk;                  // [segs * 8, B, C, N], [segs * 8, B, C]: a chunk's start within its segment, half the sum of d before it
    float *part_bc, *part_c;                 // [blocks, B, S, G, 2, N]; [B * segs] rows of dA [C, N], dD [C], ddelta_bias [C]
    int B, S, C, N, G, segs;
    int soft;
};

template <typename T, int LN, int M> struct Shape {
    static constexpr int CPW = 32 / LN;                       // channels of a group
    static constexpr int CB = kWarps * M * CPW;         // channels of a CTA
    static constexpr int PITCH = CB + 16 / (int)sizeof(T);    // tokens of one channel in different banks
    static constexpr int NP = 2 * LN;
    static constexpr int PAIRS = LN < kTok ? kTok / LN : 1;   // (channel, token) pairs of a lane
};

template <typename T, int LN, int M> struct Inputs {
    using P = Shape<T, LN, M>;
    T x[kSeg][P::PITCH], delta[kSeg][P::PITCH], z[kSeg][P::PITCH], dy[kSeg][P::PITCH];
    T Bm[kSeg][P::NP], Cm[kSeg][P::NP];      // as they come: widened here they cost pass 3 12 us more, for shared memory's rate
    float pair[kWarps][3][P::CPW][kTok];     // a chunk's d, d x and e
    float2 channel[P::CB];                   // delta_bias and D
};
template <typename T, int LN, int M> struct Work : Inputs<T, LN, M> {
    using P = Shape<T, LN, M>;
    float2 own[2][kWarps][M][32];                       // a chunk's start from a zero state of the segment,
    float past[2][kWarps][M][32];                       // half the sum of d before it (two chunks),
    float2 before[kWarps][M][32];                       // and the segment's true start
    float4 carry[kWarps][M][32];                        // a g of the chunk behind, dA
    float2 sums[kWarps][M][32];                         // dD and ddelta_bias of a pair's lane
    float2 rates[kWarps][M][32];                        // load_rates
    static constexpr int REDS = LN == 32 || (LN == 4 && M == 2) ? 1 : 2;   // two (one barrier a chunk) while two CTAs fit an SM
    float red[REDS][kWarps][kTok][2][P::NP];            // the warps' dB and dC of a chunk
};

// Where a CTA and its lanes stand.
template <typename T, int LN, int M> struct Place {
    using P = Shape<T, LN, M>;
    int g, blk, c0, nc, b, seg, t0, nt, warp, lane, sub;
    __device__ __forceinline__ Place(const ScanBwdArgs &a) {
        const int per_group = a.C / a.G, blocks = (per_group + P::CB - 1) / P::CB;
        g = blockIdx.x / blocks;
        blk = blockIdx.x % blocks;
        nc = min(P::CB, per_group - blk * P::CB);
        c0 = g * per_group + blk * P::CB;
        b = blockIdx.z;
        seg = blockIdx.y;
        t0 = seg * kSeg;
        nt = min(kSeg, a.S - t0);
        warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        sub = lane % LN;
    }
    // the channel (within the CTA) of a lane's states in a group, and its tokens as a pair's lane
    __device__ __forceinline__ int channel(int grp) const { return (warp * M + grp) * P::CPW + lane / LN; }
    __device__ __forceinline__ int token(int j) const { return LN < kTok ? sub * P::PAIRS + j : sub / (LN < kTok ? 1 : LN / kTok); }
    __device__ __forceinline__ bool pairs() const { return LN < kTok || sub % (LN < kTok ? 1 : LN / kTok) == 0; }
};

// A lane's two decay rates, times log2 e; next to zero where there is no such channel or
// state (of zero itself an infinite step size would make a NaN, which a lane's sums spread).
template <typename T, int LN, int M>
__device__ __forceinline__ float2 load_rates(const ScanBwdArgs &a, const Place<T, LN, M> &p, int ch) {
    float2 r = both(-1.17549435e-38f);
    const float *A = a.A + (size_t)(p.c0 + ch) * a.N + 2 * p.sub;
    if (ch < p.nc && 2 * p.sub < a.N) r.x = __ldg(A) * kLog2e;
    if (ch < p.nc && 2 * p.sub + 1 < a.N) r.y = __ldg(A + 1) * kLog2e;
    return r;
}
template <typename T, int LN, int M>
__device__ __forceinline__ void load_inputs(const ScanBwdArgs &a, const Place<T, LN, M> &p, Inputs<T, LN, M> &sm) {
    using P = Shape<T, LN, M>;
    constexpr int VN = Vec<T>::N, CH = P::CB / VN, NV = P::NP / VN;
    const size_t row0 = (size_t)p.b * a.S + p.t0;
    for (int i = threadIdx.x; i < kSeg * CH; i += kThreads) {
        const int r = i / CH, c = (i % CH) * VN;
        const bool ok = r < p.nt && c < p.nc;
        const size_t at = ok ? (row0 + r) * a.C + p.c0 + c : 0;
        copy16(&sm.x[r][c], (const T *)a.x + at, ok);
        copy16(&sm.delta[r][c], (const T *)a.delta + at, ok);
        copy16(&sm.dy[r][c], (const T *)a.dy + at, ok);
        if (a.z) copy16(&sm.z[r][c], (const T *)a.z + at, ok);
    }
    if ((a.N * sizeof(T)) % 16 == 0) {
        for (int i = threadIdx.x; i < kSeg * NV; i += kThreads) {
            const int r = i / NV, n = (i % NV) * VN;
            const bool ok = r < p.nt && n < a.N;               // zeros past the end and past N
            const size_t at = ok ? ((row0 + r) * a.G + p.g) * a.N + n : 0;
            copy16(&sm.Bm[r][n], (const T *)a.Bm + at, ok);
            copy16(&sm.Cm[r][n], (const T *)a.Cm + at, ok);
        }
    } else {
        for (int i = threadIdx.x; i < kSeg * P::NP; i += kThreads) {
            const int r = i / P::NP, n = i % P::NP;
            const bool ok = r < p.nt && n < a.N;
            const size_t at = ((row0 + r) * a.G + p.g) * a.N + n;
            sm.Bm[r][n] = ok ? ((const T *)a.Bm)[at] : from_f32<T>(0.f);
            sm.Cm[r][n] = ok ? ((const T *)a.Cm)[at] : from_f32<T>(0.f);
        }
    }
    copies_commit();
    for (int c = threadIdx.x; c < P::CB; c += kThreads) {
        const bool ok = c < p.nc;
        sm.channel[c] = make_float2(ok && a.delta_bias ? a.delta_bias[p.c0 + c] : 0.f, ok && a.D ? a.D[p.c0 + c] : 0.f);
    }
    copies_wait<0>();
    __syncthreads();
}

// What a pair's lane knows of its (channel, token).
struct PairInputs {
    float x, v, d, e, dy, z;
};

// Forms a chunk's step sizes and cotangents, one (channel, token) pair per lane,
// and leaves them for the warp in sm.pair.
template <typename T, int LN, int M>
__device__ __forceinline__ void prepare(const ScanBwdArgs &a, const Place<T, LN, M> &p, Inputs<T, LN, M> &sm, int grp, int chunk,
                                        PairInputs (&pairs)[Shape<T, LN, M>::PAIRS]) {
    const int ch = p.channel(grp);
    __syncwarp();                                              // the last chunk's readers are through
#pragma unroll
    for (int j = 0; j < Shape<T, LN, M>::PAIRS; ++j) {
        PairInputs q = {};
        const int t = chunk * kTok + p.token(j);
        if (p.pairs()) {
            if (ch < p.nc && t < p.nt) {
                q.x = to_f32(sm.x[t][ch]);
                q.v = to_f32(sm.delta[t][ch]) + sm.channel[ch].x;
                q.d = step_size(q.v, a.soft);
                q.e = q.dy = to_f32(sm.dy[t][ch]);
                if (a.z) {
                    q.z = to_f32(sm.z[t][ch]);
                    q.e *= q.z * logistic(q.z);
                }
            }
            float *to = &sm.pair[p.warp][0][p.lane / LN][p.token(j)];
            to[0] = q.d;
            to[Shape<T, LN, M>::CPW * kTok] = q.d * q.x;
            to[2 * Shape<T, LN, M>::CPW * kTok] = q.e;
        }
        pairs[j] = q;
    }
    __syncwarp();
}

// A chunk's 8 values of d (which 0), d x (1) or e (2) of this lane's channel.
template <typename T, int LN, int M>
__device__ __forceinline__ void read_pairs(const Place<T, LN, M> &p, const Inputs<T, LN, M> &sm, int which, float *f) {
    const float4 *from = reinterpret_cast<const float4 *>(&sm.pair[p.warp][which][p.lane / LN][0]);
    const float4 lo = from[0], hi = from[1];
    f[0] = lo.x; f[1] = lo.y; f[2] = lo.z; f[3] = lo.w;
    f[4] = hi.x; f[5] = hi.y; f[6] = hi.z; f[7] = hi.w;
}

// Sums of 8 values over the LN lanes of a channel: p[j] becomes that of the lane's
// token j.
template <int LN> __device__ __forceinline__ void state_sum(float *p, int sub) {
#pragma unroll
    for (int m = LN / 2, n = kTok / 2; m > 0; m >>= 1, n >>= 1) {
        if (n > 0) {
            const bool up = sub & m;
#pragma unroll
            for (int i = 0; i < n; ++i) {
                const float keep = up ? p[i + n] : p[i], give = up ? p[i] : p[i + n];
                p[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
            }
        } else {
            p[0] += __shfl_xor_sync(0xffffffffu, p[0], m);
        }
    }
}

// Sums of v[token][4] over the 32 / LN channels of a warp: each round the lanes
// share out the tokens, so that lane group j ends with 8 * LN / 32 of them.
template <int LN> __device__ __forceinline__ void channel_sum(float *v, int lane) {
#pragma unroll
    for (int m = 16, n = kTok / 2; m >= LN; m >>= 1, n >>= 1) {
        const bool up = lane & m;
#pragma unroll
        for (int i = 0; i < 4 * n; ++i) {
            const float keep = up ? v[i + 4 * n] : v[i], give = up ? v[i] : v[i + 4 * n];
            v[i] = keep + __shfl_xor_sync(0xffffffffu, give, m);
        }
    }
}

// A lane's two states in block `block` of a [.., C, N] array.
template <typename T, int LN, int M>
__device__ __forceinline__ float2 load_states(const float *from, size_t block, const ScanBwdArgs &a, const Place<T, LN, M> &p, int ch) {
    float2 r = both(0.f);
    const float *f = from + (block * a.C + p.c0 + ch) * a.N + 2 * p.sub;
    if (ch < p.nc && 2 * p.sub < a.N) r.x = f[0];
    if (ch < p.nc && 2 * p.sub + 1 < a.N) r.y = f[1];
    return r;
}
// The same into shared memory, on its way until copies_wait.
template <typename T, int LN, int M>
__device__ __forceinline__ void fetch_states(float2 *to, const float *from, size_t block, const ScanBwdArgs &a, const Place<T, LN, M> &p,
                                             int ch) {
    const bool in0 = ch < p.nc && 2 * p.sub < a.N, in1 = ch < p.nc && 2 * p.sub + 1 < a.N;
    const float *f = from + (in0 ? (block * a.C + p.c0 + ch) * a.N + 2 * p.sub : 0);
    if (a.N % 2 == 0) {
        copy8(to, f, in0);
    } else {
        copy4(&to->x, f, in0);
        copy4(&to->y, in1 ? f + 1 : f, in1);
    }
}
template <typename T, int LN, int M>
__device__ __forceinline__ void store_states(float *to, size_t block, const ScanBwdArgs &a, const Place<T, LN, M> &p, int ch, float2 v) {
    float *f = to + (block * a.C + p.c0 + ch) * a.N + 2 * p.sub;
    if (ch < p.nc && 2 * p.sub < a.N) f[0] = v.x;
    if (ch < p.nc && 2 * p.sub + 1 < a.N) f[1] = v.y;
}

template <typename T, int LN, int M>
__global__ void __launch_bounds__(kThreads) scan_bwd_summary_kernel(ScanBwdArgs a) {
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Inputs<T, LN, M> &sm = *reinterpret_cast<Inputs<T, LN, M> *>(smem_raw);
    const Place<T, LN, M> p(a);
    load_inputs<T, LN, M>(a, p, sm);
    for (int grp = 0; grp < M; ++grp) {
        const int ch = p.channel(grp);
        const float2 A2 = load_rates(a, p, ch);
        float2 h = both(0.f), back = both(0.f), prod = both(1.f);
        float total = 0.f;
        for (int k = 0; k * kTok < p.nt; ++k) {
            const size_t chunk = ((size_t)p.seg * (kSeg / kTok) + k) * a.B + p.b;
            store_states(a.hchunk, chunk, a, p, ch, h);
            if (p.sub == 0 && ch < p.nc) a.dchunk[chunk * a.C + p.c0 + ch] = 0.5f * total;
            PairInputs pairs[Shape<T, LN, M>::PAIRS];
            prepare(a, p, sm, grp, k, pairs);
            float d[kTok], u[kTok], e[kTok];
            read_pairs(p, sm, 0, d);
            read_pairs(p, sm, 1, u);
            read_pairs(p, sm, 2, e);
#pragma unroll
            for (int i = 0; i < kTok; ++i) {
                const int t = k * kTok + i;
                const float2 bv = widen(reinterpret_cast<const Pair<T> *>(&sm.Bm[t][0])[p.sub]);
                const float2 cv = widen(reinterpret_cast<const Pair<T> *>(&sm.Cm[t][0])[p.sub]);
                const float2 decay = exp2_fast2(mul2(both(d[i]), A2));
                h = fma2(decay, h, mul2(both(u[i]), bv));
                prod = mul2(prod, decay);
                back = fma2(prod, mul2(both(e[i]), cv), back);
                total += d[i];
            }
        }
        // a growing state's product that left fp32: the sum again, without it
        if (__any_sync(0xffffffffu, !(prod.x < kFar && prod.y < kFar))) {
            const float *pair = &sm.pair[p.warp][0][p.lane / LN][0];
            float sum = 0.f;
            back = both(0.f);
            for (int k = 0; k * kTok < p.nt; ++k) {
                PairInputs pairs[Shape<T, LN, M>::PAIRS];
                prepare(a, p, sm, grp, k, pairs);
#pragma unroll 1
                for (int i = 0; i < kTok; ++i) {
                    const float2 cv = widen(reinterpret_cast<const Pair<T> *>(&sm.Cm[k * kTok + i][0])[p.sub]);
                    sum += pair[i];
                    back = carried(mul2(both(0.5f * sum), A2), mul2(both(pair[2 * Shape<T, LN, M>::CPW * kTok + i]), cv), back);
                }
            }
        }
        const size_t block = (size_t)p.seg * a.B + p.b;
        store_states(a.hseg, block, a, p, ch, h);
        store_states(a.gseg, block, a, p, ch, back);
        if (p.sub == 0 && ch < p.nc) a.dseg[block * a.C + p.c0 + ch] = total;
    }
    pdl_launch_dependents();
}

// hseg becomes the state each segment starts from, gseg the cotangent that the
// later segments (and dh) send to its end; dh0 what reaches the first.  A grid row for
// each direction (2 x 333 x 272 x 8 fp32: the backward 25.6 us, with one row 26.8) from
// five segments on (one segment, 16 x 16 tokens x 4096 x 16: 70 us with one row, 77 with two).
// U segments' loads are in flight at a time, in 128 registers for 32 of them (4 x 2048 x
// 2048 x 16: the fold 27 us, with 8 of them 45); up to eight segments take 4, for the
// waves that the registers cost (one segment as above 70 us, with 8 of them 84).
constexpr int kFoldThreads = 256;
template <int U> __global__ void __launch_bounds__(kFoldThreads) scan_bwd_fold_kernel(ScanBwdArgs a) {
    const size_t n = (size_t)a.B * a.C * a.N, i = (size_t)blockIdx.x * kFoldThreads + threadIdx.x;
    pdl_wait();
    if (i >= n) return;
    const size_t bc = i / a.N, rows = (size_t)a.B * a.C;
    const float A2 = a.A[(bc % a.C) * a.N + i % a.N] * kLog2e;
    if (blockIdx.y == 0) {
        float h = a.h0 ? a.h0[i] : 0.f;
        for (int s0 = 0; s0 < a.segs; s0 += U) {
            float own[U], d[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                own[j] = s0 + j < a.segs ? a.hseg[(s0 + j) * n + i] : 0.f;
                d[j] = s0 + j < a.segs ? a.dseg[(s0 + j) * rows + bc] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (s0 + j >= a.segs) break;
                a.hseg[(s0 + j) * n + i] = h;
                h = carried(0.5f * (A2 * d[j]), h, own[j]);
            }
        }
    }
    if (blockIdx.y + 1 == gridDim.y) {
        float g = a.dh ? a.dh[i] : 0.f;
        for (int s0 = a.segs - 1; s0 >= 0; s0 -= U) {
            float own[U], d[U];
#pragma unroll
            for (int j = 0; j < U; ++j) {
                own[j] = s0 >= j ? a.gseg[(s0 - j) * n + i] : 0.f;
                d[j] = s0 >= j ? a.dseg[(s0 - j) * rows + bc] : 0.f;
            }
#pragma unroll
            for (int j = 0; j < U; ++j) {
                if (s0 < j) break;
                a.gseg[(s0 - j) * n + i] = g;
                g = carried(0.5f * (A2 * d[j]), g, own[j]);
            }
        }
        if (a.dh0) a.dh0[i] = g;
    }
    pdl_launch_dependents();
}

template <typename T, int LN, int M>
__global__ void __launch_bounds__(kThreads, 2) scan_bwd_grad_kernel(ScanBwdArgs a) {
    using P = Shape<T, LN, M>;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Work<T, LN, M> &sm = *reinterpret_cast<Work<T, LN, M> *>(smem_raw);
    static_assert(sizeof(sm) <= 228 * 1024 / 2 - 1024, "two CTAs per SM");
    const Place<T, LN, M> p(a);
    load_inputs<T, LN, M>(a, p, sm);                             // nothing that the passes before write
    pdl_wait();
    const int chunks = (p.nt + kTok - 1) / kTok;

    const size_t block = (size_t)p.seg * a.B + p.b;
    for (int grp = 0; grp < M; ++grp) {
        const float2 g = load_states(a.gseg, block, a, p, p.channel(grp));
        sm.carry[p.warp][grp][p.lane] = make_float4(g.x, g.y, 0.f, 0.f);
        sm.sums[p.warp][grp][p.lane] = both(0.f);
        sm.rates[p.warp][grp][p.lane] = load_rates(a, p, p.channel(grp));
        fetch_states(&sm.before[p.warp][grp][p.lane], a.hseg, block, a, p, p.channel(grp));
    }
    // a chunk's starts arrive while the chunk behind it is worked on; every lane fetches
    // what it reads itself
    auto fetch = [&](int k) {
        const size_t chunk = ((size_t)p.seg * (kSeg / kTok) + k) * a.B + p.b;
        for (int grp = 0; grp < M; ++grp) {
            const int ch = p.channel(grp);
            fetch_states(&sm.own[k & 1][p.warp][grp][p.lane], a.hchunk, chunk, a, p, ch);
            const bool in = ch < p.nc;
            copy4(&sm.past[k & 1][p.warp][grp][p.lane], a.dchunk + (in ? chunk * a.C + p.c0 + ch : 0), in);
        }
    };
    fetch(chunks - 1);
    copies_commit();
    // this CTA's rows of part_bc, from the segment's first token on
    float *bc_rows = a.part_bc + ((((size_t)p.blk * a.B + p.b) * a.S + p.t0) * a.G + p.g) * 2 * a.N;

    for (int k = chunks - 1; k >= 0; --k) {
        if (k > 0) fetch(k - 1);
        copies_commit();
        copies_wait<1>();
        float2 dB[kTok], dC[kTok];
#pragma unroll
        for (int i = 0; i < kTok; ++i) dB[i] = dC[i] = both(0.f);
        // a token's B and C of this lane's states, read where they are used: held over the
        // chunk they would take 16 registers more
        auto bv = [&](int i) { return widen(reinterpret_cast<const volatile Pair<T> *>(&sm.Bm[k * kTok + i][0])[p.sub]); };
        auto cv = [&](int i) { return widen(reinterpret_cast<const volatile Pair<T> *>(&sm.Cm[k * kTok + i][0])[p.sub]); };
#pragma unroll 1
        for (int grp = 0; grp < M; ++grp) {
            const int ch = p.channel(grp);
            const float2 A2 = sm.rates[p.warp][grp][p.lane];
            PairInputs pairs[P::PAIRS];
            prepare(a, p, sm, grp, k, pairs);
            const float2 h0 = carried(mul2(both(sm.past[k & 1][p.warp][grp][p.lane]), A2), sm.before[p.warp][grp][p.lane],
                                      sm.own[k & 1][p.warp][grp][p.lane]);
            float d[kTok], f[kTok];
            float2 h[kTok];
            read_pairs(p, sm, 0, d);
            read_pairs(p, sm, 1, f);
            {
                float2 at = h0;
#pragma unroll
                for (int i = 0; i < kTok; ++i) {
                    h[i] = at = fma2(exp2_fast2(mul2(both(d[i]), A2)), at, mul2(both(f[i]), bv(i)));
                }
            }
            const float4 carry = sm.carry[p.warp][grp][p.lane];
            float2 ag = make_float2(carry.x, carry.y), dA = make_float2(carry.z, carry.w);
            float s1[kTok], s2[kTok], y[kTok], e[kTok];
            read_pairs(p, sm, 2, e);
#pragma unroll
            for (int i = kTok - 1; i >= 0; --i) {
                const float2 c2 = cv(i), ch2 = mul2(c2, h[i]), g = fma2(both(e[i]), c2, ag);
                y[i] = ch2.x + ch2.y;
                dB[i] = fma2(both(f[i]), g, dB[i]);
                dC[i] = fma2(both(e[i]), h[i], dC[i]);
                const float2 gb = mul2(g, bv(i));
                s1[i] = gb.x + gb.y;
                ag = mul2(exp2_fast2(mul2(both(d[i]), A2)), g);
                const float2 w = mul2(ag, i > 0 ? h[i > 0 ? i - 1 : 0] : h0);
                const float2 wa = mul2(w, A2);
                s2[i] = wa.x + wa.y;
                dA = fma2(both(d[i]), w, dA);
            }
            sm.carry[p.warp][grp][p.lane] = make_float4(ag.x, ag.y, dA.x, dA.y);
            state_sum<LN>(s1, p.sub);
            state_sum<LN>(s2, p.sub);
            if (a.z) state_sum<LN>(y, p.sub);
            if (p.pairs()) {
                const float skip = sm.channel[ch].y;
#pragma unroll
                for (int j = 0; j < P::PAIRS; ++j) {
                    const PairInputs &q = pairs[j];
                    const int t = k * kTok + p.token(j);
                    // the rates carry a factor log2 e
                    const float ddelta = fmaf(s1[j], q.x, s2[j] * (1.f / kLog2e)) * (a.soft ? logistic(q.v) : 1.f);
                    if (a.z) {
                        const float sg = logistic(q.z);
                        sm.z[t][ch] = from_f32<T>(q.dy * fmaf(skip, q.x, y[j]) * sg * fmaf(q.z, 1.f - sg, 1.f));
                    }
                    sm.x[t][ch] = from_f32<T>(fmaf(s1[j], q.d, skip * q.e));
                    sm.delta[t][ch] = from_f32<T>(ddelta);
                    if (t < p.nt) {
                        float2 &sum = sm.sums[p.warp][grp][p.lane];
                        sum = make_float2(fmaf(q.e, q.x, sum.x), sum.y + ddelta);
                    }
                }
            }
        }
        // dB and dC over the channels: the warp's lanes, then the warps
        float v[kTok * 4];
#pragma unroll
        for (int i = 0; i < kTok; ++i) {
            v[4 * i] = dB[i].x; v[4 * i + 1] = dB[i].y;
            v[4 * i + 2] = dC[i].x; v[4 * i + 3] = dC[i].y;
        }
        channel_sum<LN>(v, p.lane);
        auto &red = sm.red[k % Work<T, LN, M>::REDS];
        {
            constexpr int H = kTok * LN / 32;                 // tokens whose sums this lane holds
            const int i0 = p.lane / LN * H;
#pragma unroll
            for (int i = 0; i < H; ++i) {
                reinterpret_cast<float2 *>(&red[p.warp][i0 + i][0][0])[p.sub] = make_float2(v[4 * i], v[4 * i + 1]);
                reinterpret_cast<float2 *>(&red[p.warp][i0 + i][1][0])[p.sub] = make_float2(v[4 * i + 2], v[4 * i + 3]);
            }
        }
        __syncthreads();
        float *part = bc_rows + (size_t)k * kTok * 2 * a.G * a.N;
        for (int i = threadIdx.x; i < kTok * 2 * P::NP; i += kThreads) {
            const int t = i / (2 * P::NP), which = i / P::NP % 2, n = i % P::NP;
            if (k * kTok + t >= p.nt || n >= a.N) continue;
            float s = 0.f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) s += (&red[w][0][0][0])[i];
            part[(size_t)(t * a.G * 2 + which) * a.N + n] = s;
        }
        if (Work<T, LN, M>::REDS == 1) __syncthreads();
    }
    __syncthreads();                                           // the gradients that the warps left in sm

    pdl_launch_dependents();
    // the segment's outputs; its rows of dA, dD and ddelta_bias
    constexpr int VN = Vec<T>::N, CH = P::CB / VN;
    const size_t row0 = (size_t)p.b * a.S + p.t0;
    for (int i = threadIdx.x; i < p.nt * CH; i += kThreads) {
        const int r = i / CH, c = (i % CH) * VN;
        if (c >= p.nc) continue;
        const size_t at = (row0 + r) * a.C + p.c0 + c;
        __stcs(reinterpret_cast<uint4 *>((T *)a.dx + at), *reinterpret_cast<const uint4 *>(&sm.x[r][c]));
        __stcs(reinterpret_cast<uint4 *>((T *)a.ddelta + at), *reinterpret_cast<const uint4 *>(&sm.delta[r][c]));
        if (a.z) __stcs(reinterpret_cast<uint4 *>((T *)a.dz + at), *reinterpret_cast<const uint4 *>(&sm.z[r][c]));
    }
    float *row = a.part_c + ((size_t)p.b * a.segs + p.seg) * a.C * (a.N + 2);
    for (int grp = 0; grp < M; ++grp) {
        const int ch = p.channel(grp);
        const float4 carry = sm.carry[p.warp][grp][p.lane];
        if (ch < p.nc) {
            float *dA = row + (size_t)(p.c0 + ch) * a.N + 2 * p.sub;
            if (2 * p.sub < a.N) dA[0] = carry.z;
            if (2 * p.sub + 1 < a.N) dA[1] = carry.w;
        }
        float2 s = sm.sums[p.warp][grp][p.lane];
#pragma unroll
        for (int m = LN / 2; m > 0; m >>= 1) {
            s.x += __shfl_xor_sync(0xffffffffu, s.x, m);
            s.y += __shfl_xor_sync(0xffffffffu, s.y, m);
        }
        if (p.sub == 0 && ch < p.nc) {
            row[(size_t)a.C * a.N + p.c0 + ch] = s.x;
            row[(size_t)a.C * (a.N + 1) + p.c0 + ch] = s.y;
        }
    }
}

// The last sums, each in a fixed order.  The first `bc_ctas` CTAs: dB and dC over the
// channel blocks, one number a thread.  The others: dA, dD and ddelta_bias over the
// rows that the segments left, kFoldCols columns a CTA.
constexpr int kFoldCols = 32, kFoldLanes = 8;
template <typename T> __global__ void __launch_bounds__(256) scan_bwd_finish_kernel(ScanBwdArgs a, int blocks, unsigned bc_ctas) {
    __shared__ float red[kFoldLanes][kFoldCols];
    pdl_wait();
    pdl_launch_dependents();
    float s = 0.f;
    if (blockIdx.x < bc_ctas) {
        const size_t n = (size_t)a.B * a.S * a.G * 2 * a.N, i = (size_t)blockIdx.x * 256 + threadIdx.x;
        if (i >= n) return;
#pragma unroll 8
        for (int k = 0; k < blocks; ++k) s += a.part_bc[k * n + i];
        const size_t row = i / (2 * a.N);
        const int m = (int)(i % (2 * a.N));
        if (m < a.N) ((T *)a.dBm)[row * a.N + m] = from_f32<T>(s);
        else ((T *)a.dCm)[row * a.N + m - a.N] = from_f32<T>(s);
        return;
    }
    const int cols = a.C * (a.N + 2), rows = a.B * a.segs;
    const int tx = threadIdx.x % kFoldCols, ty = threadIdx.x / kFoldCols;
    const int col = (blockIdx.x - bc_ctas) * kFoldCols + tx;
    if (col < cols) {
#pragma unroll 8
        for (int r = ty; r < rows; r += kFoldLanes) s += a.part_c[(size_t)r * cols + col];
    }
    red[ty][tx] = s;
    __syncthreads();
    if (ty != 0 || col >= cols) return;
#pragma unroll
    for (int l = 1; l < kFoldLanes; ++l) s += red[l][tx];
    const int nA = a.C * a.N;
    if (col < nA) a.dA[col] = s;
    else if (col < nA + a.C) { if (a.dD) a.dD[col - nA] = s; }
    else if (a.ddelta_bias) a.ddelta_bias[col - nA - a.C] = s;
}

int bwd_lanes(int N) { return N <= 8 ? 4 : N <= 16 ? 8 : N <= 32 ? 16 : 32; }

struct BwdPlan {
    int segs, blocks;
    int groups;                               // M above
    size_t hseg, gseg, dseg, hchunk, dchunk, part_bc, part_c, total;   // offsets in floats
};
BwdPlan plan_bwd(int B, int S, int C, int N, int G, xlstm_dtype dt) {
    BwdPlan p;
    p.segs = (S + kSeg - 1) / kSeg;
    const int cb = kWarps * (32 / bwd_lanes(N));
    const auto blocks_of = [&](int m) { return (C / G + m * cb - 1) / (m * cb); };
    p.groups = dt == XLSTM_F32 || (long long)B * G * blocks_of(2) * p.segs <= num_sms_current_device() ? 1 : 2;
    p.blocks = blocks_of(p.groups);
    size_t off = 0;
    auto take = [&](size_t n) {
        const size_t at = off;
        off = (off + n + 63) & ~size_t(63);
        return at;
    };
    const size_t bc = (size_t)B * C;
    p.hseg = take(p.segs * bc * N);
    p.gseg = take(p.segs * bc * N);
    p.dseg = take(p.segs * bc);
    p.hchunk = take((size_t)p.segs * (kSeg / kTok) * bc * N);
    p.dchunk = take((size_t)p.segs * (kSeg / kTok) * bc);
    p.part_bc = take((size_t)p.blocks * B * S * G * 2 * N);
    p.part_c = take(p.segs * bc * (N + 2));
    p.total = off;
    return p;
}

template <typename T> cudaError_t launch_finish(const ScanBwdArgs &a, int blocks, cudaStream_t st) {
    KernelTimer timer("scan_bwd_finish", st);
    const unsigned bc_ctas = (unsigned)(((size_t)a.B * a.S * a.G * 2 * a.N + 255) / 256);
    const unsigned col_ctas = (unsigned)((a.C * (a.N + 2) + kFoldCols - 1) / kFoldCols);
    return launch_chained(scan_bwd_finish_kernel<T>, dim3(bc_ctas + col_ctas), dim3(256), 0, st, a, blocks, bc_ctas);
}

template <typename T, int LN, int M> cudaError_t run_bwd(const ScanBwdArgs &a, int blocks, cudaStream_t st) {
    cudaError_t e;
    const dim3 grid(a.G * blocks, a.segs, a.B);
    {
        const size_t smem = sizeof(Inputs<T, LN, M>);
        e = cudaFuncSetAttribute(scan_bwd_summary_kernel<T, LN, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        KernelTimer timer("scan_bwd_summary", st);
        scan_bwd_summary_kernel<T, LN, M><<<grid, kThreads, smem, st>>>(a);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    {
        KernelTimer timer("scan_bwd_fold", st);
        const size_t n = (size_t)a.B * a.C * a.N;
        e = launch_chained(a.segs <= 8 ? scan_bwd_fold_kernel<4> : scan_bwd_fold_kernel<32>, dim3((unsigned)((n + kFoldThreads - 1) / kFoldThreads), a.segs <= 4 ? 1 : 2), dim3(kFoldThreads), 0, st, a);
        if (e != cudaSuccess) return e;
    }
    {
        const size_t smem = sizeof(Work<T, LN, M>);
        e = cudaFuncSetAttribute(scan_bwd_grad_kernel<T, LN, M>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        KernelTimer timer("scan_bwd_grad", st);
        if ((e = launch_chained(scan_bwd_grad_kernel<T, LN, M>, grid, dim3(kThreads), smem, st, a)) != cudaSuccess) return e;
    }
    return launch_finish<T>(a, blocks, st);
}
template <typename T, int M> cudaError_t run_bwd_lanes(const ScanBwdArgs &a, int blocks, cudaStream_t st) {
    switch (bwd_lanes(a.N)) {
        case 4: return run_bwd<T, 4, M>(a, blocks, st);
        case 8: return run_bwd<T, 8, M>(a, blocks, st);
        case 16: return run_bwd<T, 16, M>(a, blocks, st);
        default: return run_bwd<T, 32, M>(a, blocks, st);
    }
}
template <typename T> cudaError_t dispatch_bwd(const ScanBwdArgs &a, const BwdPlan &p, cudaStream_t st) {
    if (sizeof(T) == 2 && p.groups == 2) return run_bwd_lanes<T, sizeof(T) == 2 ? 2 : 1>(a, p.blocks, st);
    return run_bwd_lanes<T, 1>(a, p.blocks, st);
}

xlstm_status check_scan_bwd(int B, int S, int C, int N, int G, xlstm_dtype dt, xlstm_delta_act act) {
    const xlstm_status bad = check_scan(B, S, C, N, G, dt, act);
    if (bad != XLSTM_OK) return bad;
    return S > 65535 * kSeg ? XLSTM_ERR_SHAPE : XLSTM_OK;      // segments ride in a grid dimension
}

}  // namespace
}  // namespace xlstm

extern "C" xlstm_status xlstm_ssm_scan_bwd_workspace_size(int B, int S, int C, int N, int G, xlstm_dtype dt,
                                                          size_t *bytes) {
    using namespace xlstm;
    if (!bytes) return XLSTM_ERR_NULL;
    const xlstm_status bad = check_scan_bwd(B, S, C, N, G, dt, XLSTM_DELTA_PLAIN);
    if (bad != XLSTM_OK) return bad;
    *bytes = plan_bwd(B, S, C, N, G, dt).total * sizeof(float);
    return XLSTM_OK;
}

extern "C" xlstm_status xlstm_ssm_scan_bwd(const void *x, const void *delta, const float *A, const void *Bm,
                                           const void *Cm, const float *D, const void *z,
                                           const float *delta_bias, const float *h0, const void *dy,
                                           const float *dh, void *dx, void *ddelta, float *dA, void *dBm,
                                           void *dCm, float *dD, void *dz, float *ddelta_bias, float *dh0,
                                           int B, int S, int C, int N, int G, xlstm_dtype dt,
                                           xlstm_delta_act act, void *workspace, size_t workspace_bytes,
                                           void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_ssm_scan_bwd");
    const xlstm_status bad = check_scan_bwd(B, S, C, N, G, dt, act);
    if (bad != XLSTM_OK) return bad;
    if (!A || !dA) return XLSTM_ERR_NULL;
    const bool tokens = B > 0 && S > 0;
    if (tokens && (!x || !delta || !Bm || !Cm || !dy || !dx || !ddelta || !dBm || !dCm)) return XLSTM_ERR_NULL;
    if (tokens && (z == nullptr) != (dz == nullptr)) return XLSTM_ERR_NULL;
    const void *in[] = {x, delta, A, Bm, Cm, D, z, delta_bias, h0, dy, dh};
    const void *out[] = {dx, ddelta, dA, dBm, dCm, dD, dz, ddelta_bias, dh0};
    for (const void *i : in)
        if (misaligned16(i)) return XLSTM_ERR_ALIGN;
    for (const void *o : out)
        if (misaligned16(o)) return XLSTM_ERR_ALIGN;
    if (misaligned16(workspace)) return XLSTM_ERR_ALIGN;
    for (int o = 0; o < 9; ++o) {
        if (!out[o]) continue;
        for (const void *i : in)
            if (out[o] == i) return XLSTM_ERR_UNSUPPORTED;
        for (int j = 0; j < o; ++j)
            if (out[o] == out[j]) return XLSTM_ERR_UNSUPPORTED;
    }
    const BwdPlan pl = plan_bwd(B, S, C, N, G, dt);
    if (pl.total > 0 && (!workspace || workspace_bytes < pl.total * sizeof(float))) return XLSTM_ERR_WORKSPACE;
    float *ws = (float *)workspace;
    ScanBwdArgs a = {x, delta, Bm, Cm, z, dy, A, D, delta_bias, h0, dh, dx, ddelta, dz, dBm, dCm, dA, dD, ddelta_bias, dh0,
                     ws + pl.hseg, ws + pl.gseg, ws + pl.dseg, ws + pl.hchunk, ws + pl.dchunk, ws + pl.part_bc, ws + pl.part_c,
                     B, S, C, N, G, pl.segs, act == XLSTM_DELTA_SOFTPLUS};
    cudaStream_t st = (cudaStream_t)cuda_stream;
    cudaError_t e = cudaSuccess;
    if (tokens) {
        e = dt == XLSTM_BF16 ? dispatch_bwd<__nv_bfloat16>(a, pl, st) : dispatch_bwd<float>(a, pl, st);
    } else if (B > 0 && dh0) {                                 // no token: the cotangent passes through
        const size_t n = (size_t)B * C * N * sizeof(float);
        e = dh ? cudaMemcpyAsync(dh0, dh, n, cudaMemcpyDeviceToDevice, st) : cudaMemsetAsync(dh0, 0, n, st);
    }
    if (!tokens && e == cudaSuccess)                           // and every sum over tokens is zero
        e = dt == XLSTM_BF16 ? launch_finish<__nv_bfloat16>(a, pl.blocks, st) : launch_finish<float>(a, pl.blocks, st);
    return e == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}
