// Selective state-space scan, forward: prompts (one pass, or segments joined where
// there are few channels) and single tokens.
//
//   d_t = softplus(delta_t + bias),  h_t[n] = 2^(d_t A[n] log2 e) h_{t-1}[n] + d_t x_t B_t[n]
//   y_t = (sum_n C_t[n] h_t[n] + D x_t) z_t sigmoid(z_t)
//
// What bounds it: one exponential per (token, channel, state).  The special
// function units do 16 a clock and SM, so N = 16 states cost nearly three times what
// reading and writing a bf16 token at HBM's rate does, and the kernel is laid
// out to keep those units fed:
//  - LN lanes share a channel, two states each; the pair's products are packed
//    fp32 operations, half the instructions.
//  - Scan warps do nothing but the recurrence.  Helper warps of the same CTA fetch
//    tiles of TT tokens (cp.async ring), form d and d x of the next tile, and
//    finish y of the last one (sum of the lanes' parts, skip, gate, store)
//    meanwhile; one barrier per tile swaps the buffers.
//  - A CTA holds CB channels of one batch row and walks along the tokens.  Where
//    B * C gives too few CTAs, the tokens are cut into P segments: a first pass
//    leaves each segment's state from a zero start and its sum of d, a fold
//    chains them (decay over a segment: exp(A sum d)), the second pass runs
//    every segment from its true start.  That forms each exponential twice.
// Measured on one B200 (bf16, N 16, gated): 1 x 16384 x 2048 0.33 ms, 38 cycles a
// token and scan warp (29 with the helpers idle) against 20 of special functions and
// 24 of issue, 17.7 of them the scan warp's; 16 x 2048 x 2048 0.49 ms, 0.45 ps a state,
// 32 cycles, where loads from shared memory are at 0.85 of their rate.
// Steps on the way for 1 x 2048 x 2048: one helper group and copies one tile ahead
// 80 us; copies four tiles ahead and two helper groups 70; y's sums over lanes as
// partial sums through shared memory, with every load written before the stores, 53
// (by shuffles in the scan warp 65); B and C read as they come instead of widened by
// the helpers 47; registers for two CTAs per SM 46; fetching with the step sizes, y
// alone in the other group 44.  No faster: deeper or shallower blocks in the scan
// warps, pairs of tokens instead of states in a packed operation (both 46); tiles of
// 64 tokens 41, but 81 against 75 at two sequences, for the shared memory.  Two
// channels, or four states, a lane: 460 against 488 us at 16 sequences, 266 against 248
// at 8, where the halved grid ends in a half-empty wave.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "scan.cuh"

namespace xlstm {
namespace {

constexpr int kHelpers = 128;                // threads of each of the two helper groups
constexpr int kAhead = 4;                    // tiles in flight: one tile is scanned faster than HBM answers
constexpr int kRing = kAhead + 4;            // raw tiles: two behind (y's skip and gate), one at work, those in flight

struct ScanArgs {
    const void *x, *delta, *Bm, *Cm, *z;
    const float *A, *D, *delta_bias, *h0;
    const int *lengths;
    void *y;
    float *h_out;
    float *seg_state, *seg_delta;            // [P-1, B, C, N], [P-1, B, C]
    int B, S, C, N, G;
    int seg, P;                              // tokens per segment, segments
    int soft;
};

// Tile shape for LN lanes per channel.
template <int LN> struct Tile {
    static constexpr int SW = LN <= 8 ? 4 : 8;            // scan warps
    static constexpr int CPW = 32 / LN;                   // channels per scan warp
    static constexpr int CB = SW * CPW;                   // channels per CTA
    static constexpr int TT = 32;                         // tokens per tile
    static constexpr int NP = 2 * LN;                     // states, padded
    static constexpr int DS = TT + 2;                     // row pitch of du: no two channels of a warp in one bank
    static constexpr int R = LN < 8 ? LN : 8;             // partial sums of a y that the scan warps leave
    static constexpr int RP = CB + (LN == 4 ? 8 : 4);     // pitches of a partial and of a token: a scan warp's
    static constexpr int TP = R * RP + 16;                // stores and the readers' vectors meet each bank once
    static constexpr int THREADS = SW * 32 + 2 * kHelpers;
};

// Shared memory of one CTA, in this order.
template <typename T, int LN> struct Smem {
    using L = Tile<LN>;
    T x[kRing][L::TT][L::CB], delta[kRing][L::TT][L::CB], z[kRing][L::TT][L::CB];
    T Bm[kRing][L::TT][L::NP], Cm[kRing][L::TT][L::NP];
    float2 du[2][L::CB][L::DS];              // (d, d x)
    float ps[2][L::TT][L::TP];               // y's partial sums: [token][partial][channel], padded
};

// The CTA's barrier, reached by the scan warps and the helper warps in their own code.
template <int THREADS> __device__ __forceinline__ void cta_barrier() {
    asm volatile("barrier.cta.sync 1, %0;" ::"n"(THREADS) : "memory");
}

// CTAs per SM that shared memory holds (228 KB, 1 KB of it the system's per CTA): two for
// bf16 and more than 8 states, else one.
template <typename T, int LN> constexpr int scan_fit() { return 228 * 1024 / ((int)sizeof(Smem<T, LN>) + 1024); }
static_assert(scan_fit<__nv_bfloat16, 4>() == 1 && scan_fit<__nv_bfloat16, 8>() == 2 && scan_fit<__nv_bfloat16, 16>() == 2 &&
              scan_fit<__nv_bfloat16, 32>() == 2, "CTAs per SM, bf16");
static_assert(scan_fit<float, 4>() == 1 && scan_fit<float, 8>() == 1 && scan_fit<float, 16>() == 1 && scan_fit<float, 32>() == 1,
              "CTAs per SM, fp32");

// CTAs per SM that the registers are held to: two in bf16, but one where 512 threads would
// spill (rows of B and C in registers; the first pass).  Up to 8 states only one fits, and
// the bound still pays: left open the first pass takes 110 registers and no longer spills
// 4 bytes, and 1 x 16384 x 1024 x 8 takes 161 us, 159 as it is (1 x 8192 x 2048 x 8: 179, 178).
__host__ __device__ constexpr int scan_resident(int bytes, int LN, bool out, bool whole) {
    return bytes == 4 || (LN >= 16 && !(out && whole)) ? 1 : 2;
}

// WHOLE: rows of B and C are 16-byte pieces.  (1 x 16384 x 2048 x 13 takes 0.53 ms, the
// 16 states of whole pieces 0.33; with each row read when its tile was fetched 0.94.)
template <typename T, int LN, bool OUT, bool WHOLE>
__global__ void __launch_bounds__(Tile<LN>::THREADS, scan_resident(sizeof(T), LN, OUT, WHOLE)) scan_kernel(ScanArgs a) {
    using L = Tile<LN>;
    constexpr int TT = L::TT, CB = L::CB, VN = Vec<T>::N;
    extern __shared__ __align__(16) unsigned char smem_raw[];
    Smem<T, LN> &sm = *reinterpret_cast<Smem<T, LN> *>(smem_raw);
    const int per_group = a.C / a.G, blocks = (per_group + CB - 1) / CB;
    const int g = blockIdx.x / blocks, cb = (blockIdx.x % blocks) * CB;
    const int nc = min(CB, per_group - cb);                // channels of this CTA, a multiple of 8
    const int c0 = g * per_group + cb;
    const int b = blockIdx.z, seg = blockIdx.y;
    pdl_wait();
    int len = a.S;
    if (a.lengths) len = max(0, min(a.lengths[b], a.S));
    const int t_begin = min(seg * a.seg, len), t_end = min(t_begin + a.seg, len);
    const int tiles = (t_end - t_begin + TT - 1) / TT;

    const int tid = threadIdx.x;
    const size_t row0 = (size_t)b * a.S;
    if (tid >= L::SW * 32 + kHelpers) {
        // ------------------------------------------------------- helpers: finishing y
        const int hid = tid - L::SW * 32 - kHelpers;
        constexpr int Q = CB / 4;                          // channel quads; kHelpers is a multiple
        const int quad = (hid % Q) * 4;
        const bool mine = quad < nc;
        float skip[4] = {0.f, 0.f, 0.f, 0.f};
        if (OUT && mine && a.D) unpack4(a.D + c0 + quad, skip);
        auto finish = [&](int k) {                          // skip, gate, store
            const int slot = k % kRing, buf = k & 1, t0 = t_begin + k * TT;
            T *y = (T *)a.y + (row0 + t0) * a.C + c0 + quad;
            for (int r = hid / Q; r < TT; r += kHelpers / Q) {
                if (!mine || t0 + r >= t_end) break;
                float xv[4];
                unpack4(&sm.x[slot][r][quad], xv);
                float2 lo = make_float2(skip[0] * xv[0], skip[1] * xv[1]), hi = make_float2(skip[2] * xv[2], skip[3] * xv[3]);
#pragma unroll
                for (int j = 0; j < L::R; ++j) {
                    const float4 v = *reinterpret_cast<const float4 *>(&sm.ps[buf][r][j * L::RP + quad]);
                    lo = add2(lo, make_float2(v.x, v.y));
                    hi = add2(hi, make_float2(v.z, v.w));
                }
                float out[4] = {lo.x, lo.y, hi.x, hi.y};
                if (a.z) {
                    float zv[4];
                    unpack4(&sm.z[slot][r][quad], zv);
#pragma unroll
                    for (int e = 0; e < 4; ++e) out[e] *= zv[e] * logistic(zv[e]);
                }
                store4(y + (size_t)r * a.C, out);
            }
        };
        cta_barrier<L::THREADS>();
        for (int k = 0; k < tiles + 2; ++k) {
            if (OUT && k >= 2) finish(k - 2);
            cta_barrier<L::THREADS>();
        }
    } else if (tid >= L::SW * 32) {
        // ----------------------------- helpers: fetching, the recurrence's d and d x
        const int hid = tid - L::SW * 32;
        constexpr int Q = CB / 4;
        const int quad = (hid % Q) * 4;
        const bool mine = quad < nc;
        float bias[4] = {0.f, 0.f, 0.f, 0.f};
        if (mine && a.delta_bias) unpack4(a.delta_bias + c0 + quad, bias);
        // states past N are zero throughout: no copy reaches them
        if (a.N < L::NP) {
            const int pad = L::NP - a.N;
            for (int i = hid; i < kRing * TT * pad; i += kHelpers) {
                const int r = i / pad, n = a.N + i % pad;
                (&sm.Bm[0][0][0])[r * L::NP + n] = from_f32<T>(0.f);
                if (OUT) (&sm.Cm[0][0][0])[r * L::NP + n] = from_f32<T>(0.f);
            }
        }

        // Tile k: x, delta and z in 16-byte pieces by some threads, B and C by the others.
        constexpr int CH = CB / VN, NV = L::NP / VN, XS = TT * CH, BS = TT * NV;
        const T *x0 = (const T *)a.x + (row0 + t_begin) * a.C + c0, *d0 = (const T *)a.delta + (row0 + t_begin) * a.C + c0;
        const T *z0 = OUT && a.z ? (const T *)a.z + (row0 + t_begin) * a.C + c0 : nullptr;
        const size_t bc_row = (size_t)a.G * a.N, bc0 = (row0 + t_begin) * bc_row + (size_t)g * a.N;
        const T *b0 = (const T *)a.Bm + bc0, *v0 = (const T *)a.Cm + bc0;
        auto fetch = [&](int k) {
            const int slot = k % kRing, left = t_end - t_begin - k * TT;
#pragma unroll
            for (int i0 = 0; i0 < XS + BS; i0 += kHelpers) {
                const int i = i0 + hid;
                if (i < XS) {
                    const int r = i / CH, c = (i % CH) * VN;
                    const bool ok = r < left && c < nc;
                    const size_t at = ok ? (size_t)(k * TT + r) * a.C + c : 0;
                    copy16(&sm.x[slot][r][c], x0 + at, ok);
                    copy16(&sm.delta[slot][r][c], d0 + at, ok);
                    if (z0) copy16(&sm.z[slot][r][c], z0 + at, ok);
                } else if (i < XS + BS && WHOLE) {
                    const int r = (i - XS) / NV, n = ((i - XS) % NV) * VN;
                    if (n < a.N) {
                        const bool ok = r < left;
                        const size_t at = ok ? (size_t)(k * TT + r) * bc_row + n : 0;
                        copy16(&sm.Bm[slot][r][n], b0 + at, ok);
                        if (OUT) copy16(&sm.Cm[slot][r][n], v0 + at, ok);
                    }
                }
            }
        };
        // Rows of B and C that are not whole 16-byte pieces pass registers: loaded before the
        // step's own work, stored after it.
        constexpr int SCALARS = WHOLE ? 1 : (TT * L::NP + kHelpers - 1) / kHelpers;
        T held_b[SCALARS], held_c[SCALARS];
        auto load_rows = [&](int k) {
            const int left = t_end - t_begin - k * TT;
#pragma unroll
            for (int j = 0; j < SCALARS; ++j) {
                const int i = hid + j * kHelpers, r = i / L::NP, n = i % L::NP;
                held_b[j] = held_c[j] = from_f32<T>(0.f);
                if (r < left && r < TT && n < a.N) {
                    const size_t at = (size_t)(k * TT + r) * bc_row + n;
                    held_b[j] = b0[at];
                    if (OUT) held_c[j] = v0[at];
                }
            }
        };
        auto store_rows = [&](int k) {
            const int slot = k % kRing;
#pragma unroll
            for (int j = 0; j < SCALARS; ++j) {
                const int i = hid + j * kHelpers, r = i / L::NP, n = i % L::NP;
                if (r >= TT) continue;
                sm.Bm[slot][r][n] = held_b[j];               // zeros past N
                if (OUT) sm.Cm[slot][r][n] = held_c[j];
            }
        };
        // one group of copies per tile, also where there is no such tile, so that
        // "all but the last kAhead - 1 groups" is always the next tile
        for (int k = 0; k < kAhead; ++k) {
            if (k < tiles) {
                fetch(k);
                if (!WHOLE) {
                    load_rows(k);
                    store_rows(k);
                }
            }
            copies_commit();
        }
        copies_wait<kAhead - 1>();
        cta_barrier<L::THREADS>();
        for (int k = 0; k < tiles + 2; ++k) {
            const bool more = k + kAhead < tiles, rows = more && !WHOLE;
            if (more) fetch(k + kAhead);
            if (rows) load_rows(k + kAhead);
            copies_commit();
            if (k < tiles) {
                const int slot = k % kRing, buf = k & 1, left = t_end - t_begin - k * TT;
                for (int r = hid / Q; r < TT; r += kHelpers / Q) {
                    float xv[4], dv[4];
                    unpack4(&sm.x[slot][r][quad], xv);
                    unpack4(&sm.delta[slot][r][quad], dv);
                    // past the end nothing decays and nothing is added
                    const bool live = mine && r < left;
#pragma unroll
                    for (int e = 0; e < 4; e += 2) {
                        const float2 v = add2(make_float2(dv[e], dv[e + 1]), make_float2(bias[e], bias[e + 1]));
                        float2 d = a.soft ? softplus2(v) : v, u = mul2(d, make_float2(xv[e], xv[e + 1]));
                        if (!live) d = u = both(0.f);
                        sm.du[buf][quad + e][r] = make_float2(d.x, u.x);
                        sm.du[buf][quad + e + 1][r] = make_float2(d.y, u.y);
                    }
                }
            }
            if (rows) store_rows(k + kAhead);
            copies_wait<kAhead - 1>();
            cta_barrier<L::THREADS>();
        }
    } else {
        // --------------------------------------------------------- scan warps
        const int lane = tid & 31, sub = lane % LN, ch = (tid >> 5) * L::CPW + lane / LN;
        const int n0 = 2 * sub, c = c0 + ch;
        const bool in0 = ch < nc && n0 < a.N, in1 = ch < nc && n0 + 1 < a.N;
        float2 A2 = make_float2(0.f, 0.f), h = make_float2(0.f, 0.f);
        const size_t at = ((size_t)b * a.C + c) * a.N + n0;
        if (in0) A2.x = a.A[(size_t)c * a.N + n0] * kLog2e;
        if (in1) A2.y = a.A[(size_t)c * a.N + n0 + 1] * kLog2e;
        if (OUT) {
            const float *from = seg == 0 ? a.h0 : a.seg_state + (size_t)(seg - 1) * a.B * a.C * a.N;
            if (from && in0) h.x = from[at];
            if (from && in1) h.y = from[at + 1];
        }
        float total = 0.f;                                  // sum of d, the first pass's
        cta_barrier<L::THREADS>();
        for (int k = 0; k < tiles + 2; ++k) {
            if (k >= 1 && k <= tiles) {
                const int buf = (k - 1) & 1, slot = (k - 1) % kRing;
                float part = 0.f, p[LN / L::R];
                constexpr int U = LN / L::R;                // tokens that share the shuffles, where there are any
                float *ps = &sm.ps[buf][sub / L::R][(sub % L::R) * L::RP + ch];
                // Blocks of four tokens in three stages (load, exponentials, recurrence), each
                // block's loads two blocks early: a store to shared memory holds back the loads
                // written after it, and with one scan warp per scheduler nothing else hides the
                // latencies.
                float4 du[2][2];
                Pair<T> bv[2][4], cv[2][4];
                float2 decay[4], ub[4];
                auto load = [&](int t, int w) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        if (i % 2 == 0) du[w][i / 2] = *reinterpret_cast<const float4 *>(&sm.du[buf][ch][t + i]);
                        bv[w][i] = reinterpret_cast<const Pair<T> *>(&sm.Bm[slot][t + i][0])[sub];
                        if (OUT) cv[w][i] = reinterpret_cast<const Pair<T> *>(&sm.Cm[slot][t + i][0])[sub];
                    }
                };
                auto exponentials = [&](int w) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float4 v = du[w][i / 2];
                        const float d = i % 2 ? v.z : v.x, u = i % 2 ? v.w : v.y;
                        decay[i] = exp2_fast2(mul2(both(d), A2));
                        ub[i] = mul2(both(u), widen(bv[w][i]));
                        if (!OUT) part += d;
                    }
                };
                load(0, 0);
                load(4, 1);
                exponentials(0);
#pragma unroll
                for (int t = 0; t < TT; t += 4) {
                    float2 hs[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) h = hs[i] = fma2(decay[i], h, ub[i]);
                    float2 cs[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) cs[i] = OUT ? widen(cv[(t / 4) & 1][i]) : both(0.f);
                    if (t + 8 < TT) load(t + 8, (t / 4) & 1);
                    if (t + 4 < TT) exponentials((t / 4 + 1) & 1);
                    if (OUT) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            p[i % U] = fmaf(cs[i].y, hs[i].y, cs[i].x * hs[i].x);
                            if (i % U == U - 1) ps[(t + i + 1 - U) * L::TP] = partial_sum<LN, L::R>(p, sub);
                        }
                    }
                }
                total += part;
            }
            cta_barrier<L::THREADS>();
        }
        pdl_launch_dependents();
        if (OUT) {
            if (seg == a.P - 1 && a.h_out) {
                if (in0) a.h_out[at] = h.x;
                if (in1) a.h_out[at + 1] = h.y;
            }
        } else {
            float *to = a.seg_state + (size_t)seg * a.B * a.C * a.N;
            if (in0) to[at] = h.x;
            if (in1) to[at + 1] = h.y;
            if (sub == 0 && ch < nc) a.seg_delta[((size_t)seg * a.B + b) * a.C + c] = total;
        }
    }
}

// Turns each segment's own state into the state that the next one starts from.
__global__ void __launch_bounds__(256) scan_fold_kernel(ScanArgs a) {
    const size_t n = (size_t)a.B * a.C * a.N, i = (size_t)blockIdx.x * 256 + threadIdx.x;
    pdl_wait();
    pdl_launch_dependents();
    if (i >= n) return;
    const size_t bc = i / a.N;
    const float A2 = a.A[(bc % a.C) * a.N + i % a.N] * kLog2e;
    float h = a.h0 ? a.h0[i] : 0.f;
    constexpr int U = 16;                                   // segments whose loads are in flight
    for (int p0 = 0; p0 < a.P - 1; p0 += U) {
        float own[U], d[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            own[j] = p0 + j < a.P - 1 ? a.seg_state[(size_t)(p0 + j) * n + i] : 0.f;
            d[j] = p0 + j < a.P - 1 ? a.seg_delta[(size_t)(p0 + j) * a.B * a.C + bc] : 0.f;
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            if (p0 + j >= a.P - 1) break;
            h = carried(0.5f * (A2 * d[j]), h, own[j]);
            a.seg_state[(size_t)(p0 + j) * n + i] = h;
        }
    }
}

// ------------------------------------------------------------- single token
struct StepScanArgs {
    const void *x, *delta, *Bm, *Cm, *z;
    const float *A, *D, *delta_bias;
    float *h;
    void *y;
    int B, C, N, G;
    int soft;
};

// The token reads and writes the whole fp32 state and little else, so it is a
// stream through HBM.  VEC: N is 4, 8, 16, 32 or 64; N / 4 lanes share a channel,
// one 16-byte vector of its state each.  Otherwise a quarter of 2^k >= N lanes shares it,
// four numbers each.  The batch rows lie in the grid's
// second dimension.  256 x 4096 x 16 bf16 (floor 22 us): 28 us, issue at 0.77 of its
// rate; 41 with a one-dimensional grid, for its 64-bit divisions.  Fewer instructions a
// state were no gain: one thread for several rows (95 registers) 56 against the 41, two
// vectors a lane 47 against 28, for loads and stores in 32-byte pieces.
template <typename T, int LPC, bool VEC>
__global__ void __launch_bounds__(256) scan_step_kernel(StepScanArgs a) {
    const int i = blockIdx.x * 256 + threadIdx.x, sub = i % LPC;
    const bool live = i / LPC < a.C;                  // the last warp's shuffles need all lanes
    const int c = live ? i / LPC : 0;
    const size_t at = (size_t)blockIdx.y * a.C + c;
    const size_t row = ((size_t)blockIdx.y * a.G + (a.G > 1 ? c / (a.C / a.G) : 0)) * a.N;
    float *h = a.h + at * a.N;
    float p = 0.f;
    float4 hv = make_float4(0.f, 0.f, 0.f, 0.f);
    if (VEC && live) hv = __ldcs(reinterpret_cast<const float4 *>(h) + sub);   // channel 0's owner is writing it
    const float xv = to_f32(((const T *)a.x)[at]);
    const float zv = a.z ? to_f32(((const T *)a.z)[at]) : 0.f;
    const float d = step_size(to_f32(((const T *)a.delta)[at]) + (a.delta_bias ? __ldg(a.delta_bias + c) : 0.f), a.soft);
    const float u = d * xv;
    if (VEC) {
        float bv[4], cv[4];
        unpack4((const T *)a.Bm + row + 4 * sub, bv);
        unpack4((const T *)a.Cm + row + 4 * sub, cv);
        const float4 Av = __ldg(reinterpret_cast<const float4 *>(a.A + (size_t)c * a.N) + sub);
        float4 o;
        o.x = fmaf(exp2_fast(d * (Av.x * kLog2e)), hv.x, u * bv[0]);
        o.y = fmaf(exp2_fast(d * (Av.y * kLog2e)), hv.y, u * bv[1]);
        o.z = fmaf(exp2_fast(d * (Av.z * kLog2e)), hv.z, u * bv[2]);
        o.w = fmaf(exp2_fast(d * (Av.w * kLog2e)), hv.w, u * bv[3]);
        if (live) __stcs(reinterpret_cast<float4 *>(h) + sub, o);
        p = fmaf(cv[0], o.x, fmaf(cv[1], o.y, fmaf(cv[2], o.z, cv[3] * o.w)));
    } else if (live) {
        float hn[4], An[4], bn[4], cn[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = sub + j * LPC;
            hn[j] = An[j] = bn[j] = cn[j] = 0.f;
            if (n < a.N) {
                hn[j] = __ldcs(h + n);
                An[j] = __ldg(a.A + (size_t)c * a.N + n) * kLog2e;
                bn[j] = to_f32(((const T *)a.Bm)[row + n]);
                cn[j] = to_f32(((const T *)a.Cm)[row + n]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int n = sub + j * LPC;
            if (n >= a.N) continue;
            const float v = fmaf(exp2_fast(d * An[j]), hn[j], u * bn[j]);
            __stcs(h + n, v);
            p = fmaf(cn[j], v, p);
        }
    }
#pragma unroll
    for (int o = LPC / 2; o > 0; o >>= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
    if (live && sub == 0) {
        if (a.D) p = fmaf(__ldg(a.D + c), xv, p);
        if (a.z) p *= zv * logistic(zv);
        ((T *)a.y)[at] = from_f32<T>(p);
    }
}

int lanes_for(int N) {                        // lanes per channel, two states each
    int l = 4;
    while (2 * l < N) l <<= 1;
    return l;
}

// Segments: one where the channels alone give at least half of the SMs a CTA
// (two passes form every exponential twice), else enough for two CTAs an SM, of at
// least two tiles each.  Where an SM holds one CTA (`scan_fit`) the second follows the first:
// half as many segments are faster for few channels (fp32, 16384 tokens, 16 states: 64
// channels 27 us against 34) and slower for more (512 channels 163 against 149).
void plan_scan(int B, int S, int C, int N, int G, int *seg, int *P) {
    const int ln = lanes_for(N), cb = ln == 4 ? 32 : ln == 32 ? 8 : 16, tt = 32;
    const int sms = num_sms_current_device();
    const long long ctas = (long long)B * G * ((C / G + cb - 1) / cb);
    const int tiles = (S + tt - 1) / tt;
    int p = 1;
    if (ctas > 0 && 2 * ctas < sms) {
        p = (int)(2LL * sms / ctas);
        if (p > tiles / 2) p = tiles / 2;
        if (p < 1) p = 1;
    }
    const int per = tiles == 0 ? 0 : (tiles + p - 1) / p;
    *P = per == 0 ? 1 : (tiles + per - 1) / per;
    *seg = per * tt;
}

template <typename T, int LN, bool OUT, bool WHOLE> cudaError_t launch_scan(const ScanArgs &a, cudaStream_t st) {
    using L = Tile<LN>;
    const size_t smem = sizeof(Smem<T, LN>);
    cudaError_t e = cudaFuncSetAttribute(scan_kernel<T, LN, OUT, WHOLE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    const int blocks = (a.C / a.G + L::CB - 1) / L::CB;
    const dim3 grid(a.G * blocks, OUT ? a.P : a.P - 1, a.B);
    KernelTimer timer(OUT ? "scan_output" : "scan_summary", st);
    if (OUT && a.P > 1) return launch_chained(scan_kernel<T, LN, OUT, WHOLE>, grid, dim3(L::THREADS), smem, st, a);
    scan_kernel<T, LN, OUT, WHOLE><<<grid, L::THREADS, smem, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int LN, bool WHOLE> cudaError_t run_scan(const ScanArgs &a, cudaStream_t st) {
    if (a.P > 1) {
        cudaError_t e = launch_scan<T, LN, false, WHOLE>(a, st);
        if (e != cudaSuccess) return e;
        KernelTimer timer("scan_fold", st);
        const size_t n = (size_t)a.B * a.C * a.N;
        e = launch_chained(scan_fold_kernel, dim3((unsigned)((n + 255) / 256)), dim3(256), 0, st, a);
        if (e != cudaSuccess) return e;
    }
    return launch_scan<T, LN, true, WHOLE>(a, st);
}

template <typename T, bool WHOLE> cudaError_t dispatch_lanes(const ScanArgs &a, cudaStream_t st) {
    switch (lanes_for(a.N)) {
        case 4: return run_scan<T, 4, WHOLE>(a, st);
        case 8: return run_scan<T, 8, WHOLE>(a, st);
        case 16: return run_scan<T, 16, WHOLE>(a, st);
        default: return run_scan<T, 32, WHOLE>(a, st);
    }
}
template <typename T> cudaError_t dispatch_scan(const ScanArgs &a, cudaStream_t st) {
    return (a.N * sizeof(T)) % 16 == 0 ? dispatch_lanes<T, true>(a, st) : dispatch_lanes<T, false>(a, st);
}

template <typename T> cudaError_t dispatch_step(const StepScanArgs &a, cudaStream_t st) {
    KernelTimer timer("scan_step", st);
#define XLSTM_STEP(LPC, VEC)                                                                                       \
    scan_step_kernel<T, LPC, VEC><<<dim3((unsigned)(((long long)a.C * LPC + 255) / 256), a.B), 256, 0, st>>>(a);   \
    return cudaGetLastError();
    switch (a.N) {
        case 4: XLSTM_STEP(1, true)
        case 8: XLSTM_STEP(2, true)
        case 16: XLSTM_STEP(4, true)
        case 32: XLSTM_STEP(8, true)
        case 64: XLSTM_STEP(16, true)
        default: break;
    }
    if (a.N <= 8) { XLSTM_STEP(2, false) }
    if (a.N <= 16) { XLSTM_STEP(4, false) }
    if (a.N <= 32) { XLSTM_STEP(8, false) }
    XLSTM_STEP(16, false)
#undef XLSTM_STEP
}

}  // namespace

xlstm_status check_scan(int B, int S, int C, int N, int G, xlstm_dtype dt, xlstm_delta_act act) {
    if (dt != XLSTM_F32 && dt != XLSTM_BF16) return XLSTM_ERR_DTYPE;
    if (act != XLSTM_DELTA_PLAIN && act != XLSTM_DELTA_SOFTPLUS) return XLSTM_ERR_DTYPE;
    if (B < 0 || B > 65535 || S < 0 || S > (1 << 30)) return XLSTM_ERR_SHAPE;
    if (C < 8 || C > 65536 || C % 8 != 0 || N < 1 || N > 64) return XLSTM_ERR_SHAPE;
    if (G < 1 || C % G != 0 || (C / G) % 8 != 0) return XLSTM_ERR_SHAPE;
    if ((long long)B * S > (1LL << 40) / C || (long long)B * S > (1LL << 40) / (G * N)) return XLSTM_ERR_SHAPE;
    return XLSTM_OK;
}

}  // namespace xlstm

extern "C" xlstm_status xlstm_ssm_scan_fwd_workspace_size(int B, int S, int C, int N, int G, xlstm_dtype dt,
                                                          size_t *bytes) {
    using namespace xlstm;
    if (!bytes) return XLSTM_ERR_NULL;
    const xlstm_status bad = check_scan(B, S, C, N, G, dt, XLSTM_DELTA_PLAIN);
    if (bad != XLSTM_OK) return bad;
    int seg, P;
    plan_scan(B, S, C, N, G, &seg, &P);
    *bytes = (size_t)(P - 1) * B * C * (N + 1) * sizeof(float);
    return XLSTM_OK;
}

extern "C" xlstm_status xlstm_ssm_scan_fwd(const void *x, const void *delta, const float *A, const void *Bm,
                                           const void *Cm, const float *D, const void *z,
                                           const float *delta_bias, const float *h0, const int *lengths,
                                           void *y, float *h_out, int B, int S, int C, int N, int G,
                                           xlstm_dtype dt, xlstm_delta_act act, void *workspace,
                                           size_t workspace_bytes, void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_ssm_scan_fwd");
    const xlstm_status bad = check_scan(B, S, C, N, G, dt, act);
    if (bad != XLSTM_OK) return bad;
    if (B == 0) return XLSTM_OK;
    if (!A || (S > 0 && (!x || !delta || !Bm || !Cm || !y))) return XLSTM_ERR_NULL;
    const void *ptrs[] = {x, delta, A, Bm, Cm, D, z, delta_bias, h0, y, h_out, workspace};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    if (misaligned4(lengths)) return XLSTM_ERR_ALIGN;          // read one by one
    const void *in[] = {x, delta, A, Bm, Cm, D, z, delta_bias, h0, lengths}, *out[] = {y, h_out};
    for (const void *o : out)
        for (const void *i : in)
            if (o && o == i) return XLSTM_ERR_UNSUPPORTED;
    if (y && y == (const void *)h_out) return XLSTM_ERR_UNSUPPORTED;
    ScanArgs a = {x, delta, Bm, Cm, z, A, D, delta_bias, h0, lengths, y, h_out, nullptr, nullptr, B, S, C, N, G, 0, 1,
                  act == XLSTM_DELTA_SOFTPLUS};
    plan_scan(B, S, C, N, G, &a.seg, &a.P);
    const size_t states = (size_t)(a.P - 1) * B * C;
    if (a.P > 1 && (!workspace || workspace_bytes < states * (N + 1) * sizeof(float))) return XLSTM_ERR_WORKSPACE;
    a.seg_state = (float *)workspace;
    a.seg_delta = a.seg_state ? a.seg_state + states * N : nullptr;
    const cudaError_t e = dt == XLSTM_BF16 ? dispatch_scan<__nv_bfloat16>(a, (cudaStream_t)cuda_stream)
                                           : dispatch_scan<float>(a, (cudaStream_t)cuda_stream);
    return e == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}

extern "C" xlstm_status xlstm_ssm_scan_step(const void *x, const void *delta, const float *A, const void *Bm,
                                            const void *Cm, const float *D, const void *z,
                                            const float *delta_bias, float *h, void *y, int B, int C, int N,
                                            int G, xlstm_dtype dt, xlstm_delta_act act, void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_ssm_scan_step");
    const xlstm_status bad = check_scan(B, 1, C, N, G, dt, act);
    if (bad != XLSTM_OK) return bad;
    if (B == 0) return XLSTM_OK;
    if (!x || !delta || !A || !Bm || !Cm || !h || !y) return XLSTM_ERR_NULL;
    const void *ptrs[] = {x, delta, A, Bm, Cm, D, z, delta_bias, h, y};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    const void *in[] = {x, delta, A, Bm, Cm, D, z, delta_bias};
    for (const void *i : in)
        if (i && (i == (const void *)h || i == y)) return XLSTM_ERR_UNSUPPORTED;
    if (y == (const void *)h) return XLSTM_ERR_UNSUPPORTED;
    StepScanArgs a = {x, delta, Bm, Cm, z, A, D, delta_bias, h, y, B, C, N, G, act == XLSTM_DELTA_SOFTPLUS};
    const cudaError_t e = dt == XLSTM_BF16 ? dispatch_step<__nv_bfloat16>(a, (cudaStream_t)cuda_stream)
                                           : dispatch_step<float>(a, (cudaStream_t)cuda_stream);
    return e == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}
