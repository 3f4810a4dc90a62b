// The block's entry: the residual stream's addition, root-mean-square norm and
// an optional 8-bit (e4m3) output with scales, in one pass; and its backward.
//
//   s = x + residual,  rstd = 1 / sqrt(mean_c(s^2) + eps),  y = s * rstd * gamma
//   scale = max(max|y| over the group / 448, 2^-126),  q = e4m3(y / scale)
//
// Every element is read and written once and costs a handful of operations, so
// the op is bound by HBM bandwidth.  A row is held in registers between the sum
// of squares and the outputs: V 16-byte vectors per thread, a warp per row up
// to 128 vectors and one CTA per row above that.  Measured on one B200 (bf16,
// residual; floor at 6.53 TB/s): 8192 x 2048 22.6 us (20.5); 16384 x 2048 with e4m3
// and a scale per 128 channels 41 us (36); 256 x 4096 with one scale per row 3.9 us (1.1; its
// 7 MB read from HBM or from L2 alike).
//
// Backward, with n = s * rstd and g = gamma * dy:
//   dx = rstd * (g - n * mean_c(g * n)) + ds,  dgamma = sum_rows dy * n
// A CTA walks over many rows and keeps its channels' share of dgamma in
// registers; the CTAs' shares go to the workspace and a second kernel adds them
// in a fixed order, so the result does not depend on scheduling.  8192 x 2048 bf16:
// 32.5 us (floor 20.6), 27 of them the first kernel, which waits for its loads with
// 16 warps per SM; a ring of four rows in shared memory (35 us) and more, smaller
// CTAs without a row ahead (33 us) were no faster.
#include <math.h>
#include <stdint.h>

#include "common.cuh"
#include "kernels.h"
#include "profile.h"
#include "vec.cuh"

namespace xlstm {
namespace {

constexpr int kWarpRowThreads = 256;         // CTA of the warp-per-row form: 8 rows
constexpr int kMaxVectors = 4;               // 16-byte vectors a thread holds of a row
constexpr int kMaxC = 8192;                  // 512 threads of 4 fp32 vectors

// Threads of the widest CTA that a form is launched with.
__host__ __device__ constexpr int max_threads(int V, bool warp) { return warp ? kWarpRowThreads : V == 2 ? 256 : 512; }
constexpr float kE4m3Max = 448.f;
constexpr float kMinScale = 1.17549435e-38f; // 2^-126: the scale of a group of zeros

// The larger magnitude of two numbers, NaN if either is one (fmaxf would drop it);
// the sign means nothing until fabsf.
__device__ __forceinline__ float max_magnitude(float a, float b) {
    float r;
    asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// Two numbers to e4m3, nearest, ties to even, held to +-448, NaN kept; the first in the
// low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float2 v) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(v.y), "f"(v.x));
    return r;
}

// Sum over the threads of one row: a warp (WARP) or the whole CTA.  `red` holds
// one float per warp and is a different buffer in consecutive calls, so one
// barrier per call is enough.
template <bool WARP> __device__ __forceinline__ float row_sum(float x, float *red) {
    x = warp_sum(x);
    if (WARP) return x;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    return warp_sum((threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f);
}
// The largest magnitude over the same threads.
template <bool WARP> __device__ __forceinline__ float row_max(float x, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max_magnitude(x, __shfl_xor_sync(0xffffffffu, x, o));
    if (WARP) return x;
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = x;
    __syncthreads();
    const int nw = blockDim.x >> 5;
    x = (threadIdx.x & 31) < nw ? red[threadIdx.x & 31] : 0.f;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x = max_magnitude(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

template <typename T> __device__ __forceinline__ void load_gamma(const float *gamma, int c0, float *g) {
#pragma unroll
    for (int e = 0; e < Vec<T>::N; e += 4) {
        const float4 v = __ldg(reinterpret_cast<const float4 *>(gamma + c0 + e));
        g[e] = v.x; g[e + 1] = v.y; g[e + 2] = v.z; g[e + 3] = v.w;
    }
}

// x, residual, s and y carry no __restrict__: s may be residual and y may be x
// (every element is read by the thread that writes it, before it does).
struct NormArgs {
    const void *x, *residual;
    const float *gamma;
    void *s, *y;
    uint8_t *q;
    float *scales, *rstd;
    int rows, C, group;          // group 0: one scale per row
    float eps;
};

template <typename T, int V, bool WARP>
__global__ void __launch_bounds__(max_threads(V, WARP)) rmsnorm_kernel(NormArgs a) {
    constexpr int VN = Vec<T>::N;
    __shared__ float red[2][32];
    const int lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int per_row = WARP ? 32 : blockDim.x;
    const long long row = WARP ? (long long)blockIdx.x * (kWarpRowThreads / 32) + (threadIdx.x >> 5)
                               : (long long)blockIdx.x;
    if (row >= a.rows) return;                        // a whole warp (WARP) or never
    const int nvec = a.C / VN;
    const size_t base = (size_t)row * a.C;
    const uint4 *xv = reinterpret_cast<const uint4 *>((const T *)a.x + base);
    const uint4 *rv = a.residual ? reinterpret_cast<const uint4 *>((const T *)a.residual + base) : nullptr;

    uint4 xr[V], rr[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = lane + k * per_row;
        xr[k] = rr[k] = make_uint4(0, 0, 0, 0);
        if (v < nvec) {
            xr[k] = __ldcs(xv + v);
            if (rv) rr[k] = __ldcs(rv + v);
        }
    }
    constexpr int VP = VN / 2;                        // pairs of a vector
    float2 val[V][VP], sq = both(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        unpack<T>(xr[k], &val[k][0].x);
        if (rv) {
            float2 rf[VP];
            unpack<T>(rr[k], &rf[0].x);
#pragma unroll
            for (int e = 0; e < VP; ++e) val[k][e] = add2(val[k][e], rf[e]);
        }
#pragma unroll
        for (int e = 0; e < VP; ++e) sq = fma2(val[k][e], val[k][e], sq);
        const int v = lane + k * per_row;
        if (a.s && v < nvec) __stcs(reinterpret_cast<uint4 *>((T *)a.s + base) + v, pack<T>(&val[k][0].x));
    }
    // the statistics use the fp32 sum, not s as rounded to T
    const float rstd = rsqrtf(row_sum<WARP>(sq.x + sq.y, red[0]) / (float)a.C + a.eps);
    if (a.rstd && lane == 0) a.rstd[row] = rstd;

    float top[V];                                     // a vector's largest magnitude, where q wants it
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = lane + k * per_row;
        top[k] = 0.f;
        if (v < nvec) {
            float2 g[VP];
            load_gamma<T>(a.gamma, v * VN, &g[0].x);
#pragma unroll
            for (int e = 0; e < VP; ++e) val[k][e] = mul2(mul2(val[k][e], both(rstd)), g[e]);
            if (a.y) __stcs(reinterpret_cast<uint4 *>((T *)a.y + base) + v, pack<T>(&val[k][0].x));
            if (a.q) {
#pragma unroll
                for (int e = 0; e < VP; ++e) top[k] = max_magnitude(max_magnitude(val[k][e].x, val[k][e].y), top[k]);
            }
        }
    }
    if (!a.q) return;
    if (a.group == 0) {
        float all = top[0];
#pragma unroll
        for (int k = 1; k < V; ++k) all = max_magnitude(all, top[k]);
        all = row_max<WARP>(all, red[1]);
#pragma unroll
        for (int k = 0; k < V; ++k) top[k] = all;
    }
    const int lanes_per_group = a.group / VN;         // 0, or a power of two up to a warp
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int v = lane + k * per_row;
        // C is a multiple of the group, so a group's lanes all hold vectors of the row or none does
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            if (o < lanes_per_group) top[k] = max_magnitude(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
        if (v >= nvec) continue;
        // the scale and its reciprocal are within two fp32 steps of the quotients, a
        // 2^19th of the e4m3 rounding that follows (divisions, a
        // loop over the shuffles and a conversion call made instructions the limit: 55 us
        // for 16384 x 2048 bf16, 41 now)
        const float scale = max_magnitude(fabsf(top[k]) * (1.f / kE4m3Max), kMinScale), inv = reciprocal_fast(scale);
        uint32_t w[VN / 4];
#pragma unroll
        for (int e = 0; e < VP; e += 2) {
            w[e / 2] = e4m3_pair(mul2(val[k][e], both(inv))) | (e4m3_pair(mul2(val[k][e + 1], both(inv))) << 16);
        }
        uint32_t *qv = reinterpret_cast<uint32_t *>(a.q + base) + (size_t)v * (VN / 4);
        if (VN == 8) __stcs(reinterpret_cast<uint2 *>(qv), make_uint2(w[0], w[VN / 4 - 1]));
        else __stcs(qv, w[0]);
        if (a.group == 0) {
            if (v == 0) a.scales[row] = scale;
        } else if (v % lanes_per_group == 0) {
            a.scales[(size_t)row * (a.C / a.group) + v / lanes_per_group] = scale;
        }
    }
}

struct NormBwdArgs {
    const void *dy, *ds, *s;
    const float *gamma, *rstd;
    void *dx;
    float *partial;              // [gridDim.x, C]
    int rows, C;
};

template <typename T, int V, bool WARP>
__global__ void __launch_bounds__(max_threads(V, WARP)) rmsnorm_bwd_kernel(NormBwdArgs a) {
    constexpr int VN = Vec<T>::N;
    __shared__ float red[2][32];
    extern __shared__ float share[];                  // [C], WARP form only
    const int lane = WARP ? (threadIdx.x & 31) : threadIdx.x;
    const int per_row = WARP ? 32 : blockDim.x;
    const int rows_per_cta = WARP ? kWarpRowThreads / 32 : 1;
    const int slot = WARP ? (threadIdx.x >> 5) : 0;
    const int nvec = a.C / VN;
    // the scale, in registers where they suffice: read from L1 twice a row it took as
    // much of L1's rate as the rows
    constexpr bool HELD = V <= 2;
    float held[HELD ? V : 1][VN];
    if (HELD) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (lane + k * per_row < nvec) load_gamma<T>(a.gamma, (lane + k * per_row) * VN, held[k]);
    }
    float dg[V][VN];
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int e = 0; e < VN; ++e) dg[k][e] = 0.f;
    // the next row's vectors are loaded before this one's sum (where registers allow)
    constexpr bool AHEAD = V <= 2;
    const long long first = (long long)blockIdx.x * rows_per_cta + slot, stride = (long long)gridDim.x * rows_per_cta;
    uint4 yr[V], sr[V], dr[V], yn[V], sn[V], dn[V];
    auto load = [&](long long row, uint4 *y4, uint4 *s4, uint4 *d4) {
        const size_t base = (size_t)row * a.C;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * per_row;
            y4[k] = s4[k] = d4[k] = make_uint4(0, 0, 0, 0);
            if (v < nvec && row < a.rows) {
                y4[k] = __ldcs(reinterpret_cast<const uint4 *>((const T *)a.dy + base) + v);
                s4[k] = __ldcs(reinterpret_cast<const uint4 *>((const T *)a.s + base) + v);
                if (a.ds) d4[k] = __ldcs(reinterpret_cast<const uint4 *>((const T *)a.ds + base) + v);
            }
        }
    };
    if (AHEAD) load(first, yn, sn, dn);
    int turn = 0;
    float rstd_next = first < a.rows ? __ldg(a.rstd + first) : 0.f;
    for (long long row = first; row < a.rows; row += stride, turn ^= 1) {
        const size_t base = (size_t)row * a.C;
        if (AHEAD) {
#pragma unroll
            for (int k = 0; k < V; ++k) { yr[k] = yn[k]; sr[k] = sn[k]; dr[k] = dn[k]; }
            load(row + stride, yn, sn, dn);
        } else {
            load(row, yr, sr, dr);
        }
        const float rstd = rstd_next;                 // a row ahead too
        if (row + stride < a.rows) rstd_next = __ldg(a.rstd + row + stride);
        // n and g are formed twice, from the vectors as loaded: held across the
        // sum they would cost twice the registers
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * per_row;
            if (v >= nvec) continue;
            float g[VN], n[VN], gam[VN];
            unpack<T>(yr[k], g);
            unpack<T>(sr[k], n);
            if (HELD) {
#pragma unroll
                for (int e = 0; e < VN; ++e) gam[e] = held[HELD ? k : 0][e];
            } else {
                load_gamma<T>(a.gamma, v * VN, gam);
            }
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                n[e] *= rstd;
                dg[k][e] += g[e] * n[e];
                dot += g[e] * gam[e] * n[e];
            }
        }
        const float mean = row_sum<WARP>(dot, red[turn]) / (float)a.C;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * per_row;
            if (v >= nvec) continue;
            float g[VN], n[VN], gam[VN], out[VN];
            unpack<T>(yr[k], g);
            unpack<T>(sr[k], n);
            unpack<T>(dr[k], out);
            if (HELD) {
#pragma unroll
                for (int e = 0; e < VN; ++e) gam[e] = held[HELD ? k : 0][e];
            } else {
                load_gamma<T>(a.gamma, v * VN, gam);
            }
#pragma unroll
            for (int e = 0; e < VN; ++e) {
                const float dn = rstd * (g[e] * gam[e] - n[e] * rstd * mean);
                out[e] = a.ds ? out[e] + dn : dn;
            }
            __stcs(reinterpret_cast<uint4 *>((T *)a.dx + base) + v, pack<T>(out));
        }
    }
    pdl_launch_dependents();
    float *part = a.partial + (size_t)blockIdx.x * a.C;
    if (WARP) {
        // the warps add their shares one after another
        for (int w = 0; w < kWarpRowThreads / 32; ++w) {
            if (slot == w) {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int v = lane + k * per_row;
                    if (v >= nvec) continue;
#pragma unroll
                    for (int e = 0; e < VN; ++e) {
                        const int c = v * VN + e;
                        share[c] = w == 0 ? dg[k][e] : share[c] + dg[k][e];
                    }
                }
            }
            __syncthreads();
        }
        for (int c = threadIdx.x; c < a.C; c += kWarpRowThreads) part[c] = share[c];
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int v = lane + k * per_row;
            if (v >= nvec) continue;
#pragma unroll
            for (int e = 0; e < VN; e += 4)
                *reinterpret_cast<float4 *>(part + v * VN + e) =
                    make_float4(dg[k][e], dg[k][e + 1], dg[k][e + 2], dg[k][e + 3]);
        }
    }
}

// The form a row of nvec vectors takes: a warp per row up to 32 * kMaxVectors
// vectors, else one CTA with two vectors a thread, or four above 512 vectors.
struct RowForm {
    bool warp;
    int vectors, threads;
};
RowForm row_form(int nvec) {
    RowForm f;
    f.warp = nvec <= 32 * kMaxVectors;
    int v = f.warp ? (nvec + 31) / 32 : 2;
    if (v == 3) v = 4;
    if (!f.warp && nvec > 512) v = kMaxVectors;
    f.vectors = v;
    f.threads = f.warp ? kWarpRowThreads : ((nvec + v - 1) / v + 31) / 32 * 32;
    return f;
}

// CTAs of the backward: enough to fill the SMs, few enough that their shares of
// dgamma stay small next to the rows.
int bwd_ctas(int rows, int C, int vn) {
    const RowForm f = row_form(C / vn);
    const int rows_per_cta = f.warp ? kWarpRowThreads / 32 : 1;
    const long long needed = ((long long)rows + rows_per_cta - 1) / rows_per_cta;
    const int wave = num_sms_current_device() * (f.threads <= 256 ? 4 : 2);
    return needed < wave ? (int)needed : wave;
}

#define XLSTM_NORM_FORMS(LAUNCH) \
    if (f.warp) {                \
        if (f.vectors == 1) { LAUNCH(1, true) }  \
        if (f.vectors == 2) { LAUNCH(2, true) }  \
        if (f.vectors == 4) { LAUNCH(4, true) }  \
    } else {                     \
        if (f.vectors == 2) { LAUNCH(2, false) } \
        if (f.vectors == 4) { LAUNCH(4, false) } \
    }

template <typename T> cudaError_t launch_norm(const NormArgs &a, cudaStream_t st) {
    const RowForm f = row_form(a.C / Vec<T>::N);
    const unsigned grid = f.warp ? (unsigned)(((long long)a.rows + 7) / 8) : (unsigned)a.rows;
    KernelTimer timer("rmsnorm", st);
#define XLSTM_LAUNCH(V, W)                                      \
    rmsnorm_kernel<T, V, W><<<grid, f.threads, 0, st>>>(a);     \
    return cudaGetLastError();
    XLSTM_NORM_FORMS(XLSTM_LAUNCH)
#undef XLSTM_LAUNCH
    return cudaErrorInvalidValue;
}

template <typename T> cudaError_t launch_norm_bwd(const NormBwdArgs &a, int ctas, cudaStream_t st) {
    const RowForm f = row_form(a.C / Vec<T>::N);
    const size_t smem = f.warp ? (size_t)a.C * sizeof(float) : 0;
    KernelTimer timer("rmsnorm_bwd", st);
#define XLSTM_LAUNCH(V, W)                                               \
    rmsnorm_bwd_kernel<T, V, W><<<ctas, f.threads, smem, st>>>(a);       \
    return cudaGetLastError();
    XLSTM_NORM_FORMS(XLSTM_LAUNCH)
#undef XLSTM_LAUNCH
    return cudaErrorInvalidValue;
}

xlstm_status check_norm_shape(int rows, int C, xlstm_dtype dt) {
    if (dt != XLSTM_F32 && dt != XLSTM_BF16) return XLSTM_ERR_DTYPE;
    if (rows < 0 || C < 8 || C > kMaxC || C % 8 != 0) return XLSTM_ERR_SHAPE;
    return XLSTM_OK;
}

}  // namespace
}  // namespace xlstm

extern "C" xlstm_status xlstm_rmsnorm_fwd(const void *x, const void *residual, const float *gamma,
                                          void *s, void *y, void *q, float *scales, float *rstd,
                                          int rows, int C, int group, float eps, xlstm_dtype dt,
                                          void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_rmsnorm_fwd");
    const xlstm_status bad = check_norm_shape(rows, C, dt);
    if (bad != XLSTM_OK) return bad;
    if (!(eps > 0.f) || !(eps < INFINITY)) return XLSTM_ERR_UNSUPPORTED;
    if (q && group != 0 && ((group != 32 && group != 64 && group != 128) || C % group != 0))
        return XLSTM_ERR_UNSUPPORTED;
    if (rows == 0) return XLSTM_OK;
    if (!x || !gamma || (!y && !q) || (q == nullptr) != (scales == nullptr)) return XLSTM_ERR_NULL;
    if (s && !residual) return XLSTM_ERR_UNSUPPORTED;
    const void *ptrs[] = {x, residual, gamma, s, y, q, scales, rstd};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    // outputs apart from each other and from the inputs, but s on residual and y on x
    const void *in[] = {x, residual, gamma}, *out[] = {s, y, q, scales, rstd};
    for (int i = 0; i < 5; ++i) {
        if (!out[i]) continue;
        for (int j = 0; j < 3; ++j)
            if (out[i] == in[j] && !(i == 0 && j == 1) && !(i == 1 && j == 0)) return XLSTM_ERR_UNSUPPORTED;
        for (int j = 0; j < i; ++j)
            if (out[i] == out[j]) return XLSTM_ERR_UNSUPPORTED;
    }
    NormArgs a = {x, residual, gamma, s, y, (uint8_t *)q, scales, rstd, rows, C, q ? group : 0, eps};
    cudaStream_t st = (cudaStream_t)cuda_stream;
    const cudaError_t e = dt == XLSTM_BF16 ? launch_norm<__nv_bfloat16>(a, st) : launch_norm<float>(a, st);
    return e == cudaSuccess ? XLSTM_OK : XLSTM_ERR_CUDA;
}

extern "C" xlstm_status xlstm_rmsnorm_bwd_workspace_size(int rows, int C, xlstm_dtype dt, size_t *bytes) {
    using namespace xlstm;
    if (!bytes) return XLSTM_ERR_NULL;
    const xlstm_status bad = check_norm_shape(rows, C, dt);
    if (bad != XLSTM_OK) return bad;
    *bytes = (size_t)bwd_ctas(rows, C, dt == XLSTM_BF16 ? 8 : 4) * C * sizeof(float);
    return XLSTM_OK;
}

extern "C" xlstm_status xlstm_rmsnorm_bwd(const void *dy, const void *ds, const void *s,
                                          const float *gamma, const float *rstd, void *dx,
                                          float *dgamma, int rows, int C, xlstm_dtype dt,
                                          void *workspace, size_t workspace_bytes, void *cuda_stream) {
    using namespace xlstm;
    CallRange range("xlstm_rmsnorm_bwd");
    const xlstm_status bad = check_norm_shape(rows, C, dt);
    if (bad != XLSTM_OK) return bad;
    if (!dgamma || !gamma || (rows > 0 && (!dy || !s || !rstd || !dx))) return XLSTM_ERR_NULL;
    const void *ptrs[] = {dy, ds, s, gamma, rstd, dx, dgamma, workspace};
    for (const void *p : ptrs)
        if (misaligned16(p)) return XLSTM_ERR_ALIGN;
    const void *in[] = {dy, ds, s, gamma, rstd}, *out[] = {dx, dgamma};
    for (const void *o : out)
        for (const void *i : in)
            if (o && o == i) return XLSTM_ERR_UNSUPPORTED;
    if (dx == (const void *)dgamma) return XLSTM_ERR_UNSUPPORTED;
    cudaStream_t st = (cudaStream_t)cuda_stream;
    const int ctas = bwd_ctas(rows, C, dt == XLSTM_BF16 ? 8 : 4);
    const size_t need = (size_t)ctas * C * sizeof(float);
    if (need > 0 && (!workspace || workspace_bytes < need)) return XLSTM_ERR_WORKSPACE;
    NormBwdArgs a = {dy, ds, s, gamma, rstd, dx, (float *)workspace, rows, C};
    if (ctas > 0) {
        const cudaError_t e = dt == XLSTM_BF16 ? launch_norm_bwd<__nv_bfloat16>(a, ctas, st)
                                               : launch_norm_bwd<float>(a, ctas, st);
        if (e != cudaSuccess) return XLSTM_ERR_CUDA;
    }
    return launch_sum_rows((const float *)workspace, dgamma, nullptr, C, ctas, C, st) == cudaSuccess ? XLSTM_OK
                                                                                       : XLSTM_ERR_CUDA;
}
