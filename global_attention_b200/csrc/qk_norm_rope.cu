// qk_norm_rope.cu — per-head RMSNorm and partial rotation of q and k in one pass, forward and
// backward (include/zgcm_qkrope.h: the C ABI at the end of this file).
//
//   y = R(pos) (gamma x r),  r = 1/sqrt(mean x^2 + eps);   R rotates pairs (i, i + half)
//   u = R^T dy;  dgamma = sum u x r;  dx = r (gamma u - x r^2 mean(gamma u x))
//
// Bound by HBM: forward reads x and writes y, backward reads x and dy and writes dx, and no
// value is used twice except by its own row.  A row of 128 belongs to 16 lanes, 8 elements
// each (one 16-byte access of a 16-bit type), so its sums are 4 shuffles and it is read once.
// The angles depend on the token alone: a CTA forms the cosines and sines of its few tokens
// once (fp64 product and reduction: at position 262143 an fp32 product is off by 0.016 rad)
// and each half-warp keeps its 8 pairs in registers over all the heads it takes of one token.
// The partner of element d is d +- half, in another lane at an offset that depends on half: it
// goes through shared memory, the rotated elements only.
#include <math.h>

#include <initializer_list>

#include <cuda_fp16.h>

#include "common.cuh"
#include "zgcm_qkrope.h"

namespace zgcm {
namespace {

constexpr int QR_THREADS = 256;
constexpr int QR_HW = QR_THREADS / 16;   // half-warps of a CTA
constexpr int QR_MAX_TT = 4;             // tokens per CTA and step
constexpr int QR_BWD_CTAS = 592;         // most CTAs of the backward (4 per SM), one dgamma partial each

struct Rows {
    char* p;
    long long ts, hs;   // elements
};

struct QrParams {
    Rows q, k, yq, yk, dq, dk;   // forward: q, k -> yq, yk.  backward: q, k, yq = dqr, yk = dkr -> dq, dk
    const float* gamma_q;
    const float* gamma_k;
    const int* pos;
    float* part;                 // backward: [CTAs][2][128] partial dgamma
    int T, Hq, Hkv, half, tt;    // tt: tokens per CTA step (a power of two, at most QR_MAX_TT)
    float eps;
    double turns[kMaxHalf];      // rope_base^(-2i/rope_dims) / 2 pi
};

template <typename T> struct Vec8;
template <> struct Vec8<bf16> {
    uint4 w;
    __device__ __forceinline__ void load(const char* base, long long at) {
        w = *reinterpret_cast<const uint4*>(base + 2 * at);
    }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float f[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = unpack_bf16(u[i]);
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    static __device__ __forceinline__ void store(char* base, long long at, const float f[8]) {
        *reinterpret_cast<uint4*>(base + 2 * at) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                              pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    }
};
template <> struct Vec8<__half> {
    uint4 w;
    __device__ __forceinline__ void load(const char* base, long long at) {
        w = *reinterpret_cast<const uint4*>(base + 2 * at);
    }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float f[8]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
    static __device__ __forceinline__ void store(char* base, long long at, const float f[8]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(base + 2 * at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const char* base, long long at) {
        a = *reinterpret_cast<const float4*>(base + 4 * at);
        b = *reinterpret_cast<const float4*>(base + 4 * at + 16);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float f[8]) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    static __device__ __forceinline__ void store(char* base, long long at, const float f[8]) {
        *reinterpret_cast<float4*>(base + 4 * at) = make_float4(f[0], f[1], f[2], f[3]);
        *reinterpret_cast<float4*>(base + 4 * at + 16) = make_float4(f[4], f[5], f[6], f[7]);
    }
};

__device__ __forceinline__ float sum16(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x;
}

struct QrSmem {
    float2 cs[QR_MAX_TT][kMaxHalf];
    __align__(16) float swap[QR_HW][2][kD + 4];  // [half-warp][row parity]: rotated elements on their way to partners
};

// cosines and sines of the CTA's tokens t0 .. t0 + tt - 1
__device__ __forceinline__ void fill_angles(const QrParams& p, QrSmem& sm, int t0) {
    for (int i = threadIdx.x; i < p.tt * p.half; i += QR_THREADS) {
        const int t = i / p.half, j = i % p.half;
        if (t0 + t < p.T) {
            const double a = (double)p.pos[t0 + t] * p.turns[j];
            float s, c;
            sincospif(2.0f * (float)(a - rint(a)), &s, &c);
            sm.cs[t][j] = make_float2(c, s);
        }
    }
}

// this lane's 8 (cos, signed sin): y_d' = y_d c + y_partner s, s negative in the first half
__device__ __forceinline__ void lane_angles(const QrSmem& sm, int t, int l, int half, float c[8], float s[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
        const int d = 8 * l + e;
        c[e] = 1.f;
        s[e] = 0.f;
        if (d < 2 * half) {
            const float2 v = sm.cs[t][d < half ? d : d - half];
            c[e] = v.x;
            s[e] = d < half ? -v.y : v.y;
        }
    }
}

// z[e] = y[e] c[e] + sign * y[partner of e] s[e].  `buf`: this half-warp's row buffer, not in use by the
// row before (callers alternate two); every lane of the warp calls it.
__device__ __forceinline__ void rotate(float y[8], const float c[8], const float s[8], float sign, float* buf, int l,
                                       int half) {
    const bool rot = 8 * l < 2 * half;
    if (rot) {
        *reinterpret_cast<float4*>(buf + 8 * l) = make_float4(y[0], y[1], y[2], y[3]);
        *reinterpret_cast<float4*>(buf + 8 * l + 4) = make_float4(y[4], y[5], y[6], y[7]);
    }
    __syncwarp();
    if (rot) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int d = 8 * l + e;
            if (d < 2 * half) y[e] = fmaf(buf[d < half ? d + half : d - half], sign * s[e], y[e] * c[e]);
        }
    }
}

template <typename X, typename Y>
__global__ void __launch_bounds__(QR_THREADS) qk_norm_rope_fwd_kernel(const __grid_constant__ QrParams p) {
    __shared__ QrSmem sm;
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
    const int hpt = QR_HW / p.tt;                 // half-warps of a token
    const int tl = hw / hpt, part = hw % hpt;
    const int t = blockIdx.x * p.tt + tl;
    fill_angles(p, sm, blockIdx.x * p.tt);
    __syncthreads();
    float c[8], s[8];
    lane_angles(sm, tl, l, p.half, c, s);
    for (int side = 0; side < 2; ++side) {
        const Rows& x = side ? p.k : p.q;
        const Rows& y = side ? p.yk : p.yq;
        const int H = side ? p.Hkv : p.Hq;
        float g[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) g[e] = (side ? p.gamma_k : p.gamma_q)[8 * l + e];
        for (int h0 = 0, it = 0; h0 < H; h0 += hpt, ++it) {
            const int h = h0 + part;
            const bool on = t < p.T && h < H;
            Vec8<X> v;
            v.zero();
            if (on) v.load(x.p, t * x.ts + h * x.hs + 8 * l);
            float f[8], ss = 0.f;
            v.get(f);
#pragma unroll
            for (int e = 0; e < 8; ++e) ss = fmaf(f[e], f[e], ss);
            const float r = rsqrtf(sum16(ss) * (1.0f / kD) + p.eps);
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = f[e] * r * g[e];
            rotate(f, c, s, 1.f, sm.swap[hw][it & 1], l, p.half);
            if (on) Vec8<Y>::store(y.p, t * y.ts + h * y.hs + 8 * l, f);
        }
        __syncwarp();
    }
}

template <typename X, typename Y>
__global__ void __launch_bounds__(QR_THREADS) qk_norm_rope_bwd_kernel(const __grid_constant__ QrParams p) {
    __shared__ QrSmem sm;
    __shared__ float red[QR_HW][kD];
    const int l = threadIdx.x & 15, hw = threadIdx.x >> 4;
    const int hpt = QR_HW / p.tt;
    const int tl = hw / hpt, part = hw % hpt;
    float dg[2][8] = {};
    for (int t0 = blockIdx.x * p.tt; t0 < p.T; t0 += gridDim.x * p.tt) {
        const int t = t0 + tl;
        __syncthreads();   // the step before has read its angles
        fill_angles(p, sm, t0);
        __syncthreads();
        float c[8], s[8];
        lane_angles(sm, tl, l, p.half, c, s);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
            const Rows& x = side ? p.k : p.q;
            const Rows& dy = side ? p.yk : p.yq;
            const Rows& dx = side ? p.dk : p.dq;
            const int H = side ? p.Hkv : p.Hq;
            float g[8];
#pragma unroll
            for (int e = 0; e < 8; ++e) g[e] = (side ? p.gamma_k : p.gamma_q)[8 * l + e];
            for (int h0 = 0, it = 0; h0 < H; h0 += hpt, ++it) {
                const int h = h0 + part;
                const bool on = t < p.T && h < H;
                Vec8<X> v;
                Vec8<Y> w;
                v.zero();
                w.zero();
                if (on) {
                    v.load(x.p, t * x.ts + h * x.hs + 8 * l);
                    w.load(dy.p, t * dy.ts + h * dy.hs + 8 * l);
                }
                float f[8], u[8], ss = 0.f, sx = 0.f;
                v.get(f);
                w.get(u);
                rotate(u, c, s, -1.f, sm.swap[hw][it & 1], l, p.half);
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    ss = fmaf(f[e], f[e], ss);
                    sx = fmaf(f[e], u[e] * g[e], sx);
                }
                ss = sum16(ss);
                sx = sum16(sx);
                const float r = rsqrtf(ss * (1.0f / kD) + p.eps);
                const float m = r * r * sx * (1.0f / kD);     // r mean(gamma u xhat)
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    if (on) dg[side][e] = fmaf(u[e], f[e] * r, dg[side][e]);
                    u[e] = r * fmaf(-f[e], m, u[e] * g[e]);
                }
                if (on) Vec8<X>::store(dx.p, t * dx.ts + h * dx.hs + 8 * l, u);
            }
            __syncwarp();
        }
    }
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int e = 0; e < 8; ++e) red[hw][8 * l + e] = dg[side][e];
        __syncthreads();
        if (threadIdx.x < kD) {
            float a = 0.f;
            for (int i = 0; i < QR_HW; ++i) a += red[i][threadIdx.x];
            p.part[((size_t)blockIdx.x * 2 + side) * kD + threadIdx.x] = a;
        }
    }
}

// dgamma[side][d] = sum over the CTAs' partials, in a fixed order: a CTA takes 32 of the 256
// columns, each of its 8 warps every 8th partial.
__global__ void __launch_bounds__(256) qk_dgamma_kernel(const float* part, int n, float* dgamma_q, float* dgamma_k) {
    __shared__ float red[8][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    float a = 0.f;
    for (int i = w; i < n; i += 8) a += part[(size_t)i * 2 * kD + col];
    red[w][lane] = a;
    __syncthreads();
    if (w == 0) {
        for (int i = 1; i < 8; ++i) a += red[i][lane];
        (col < kD ? dgamma_q : dgamma_k)[col % kD] = a;
    }
}

// Tokens per CTA step: one while that leaves CTAs for every SM, else 4 (the angles of 4
// tokens fill half the CTA's threads and the 40 rows of each go to 4 half-warps).
int tokens_per_step(int T) { return T <= 592 ? 1 : QR_MAX_TT; }

int bwd_ctas(int T) {
    const int tt = tokens_per_step(T);
    const int n = (T + tt - 1) / tt;
    return n < QR_BWD_CTAS ? n : QR_BWD_CTAS;
}

template <typename X, typename Y>
cudaError_t launch(const QrParams& p, bool bwd, cudaStream_t stream) {
    if (bwd) {
        qk_norm_rope_bwd_kernel<X, Y><<<bwd_ctas(p.T), QR_THREADS, 0, stream>>>(p);
    } else {
        qk_norm_rope_fwd_kernel<X, Y><<<(p.T + p.tt - 1) / p.tt, QR_THREADS, 0, stream>>>(p);
    }
    return cudaGetLastError();
}

template <typename X>
cudaError_t launch_y(const QrParams& p, int y_type, bool bwd, cudaStream_t stream) {
    return y_type == ZGCM_BF16   ? launch<X, bf16>(p, bwd, stream)
           : y_type == ZGCM_FP16 ? launch<X, __half>(p, bwd, stream)
                                 : launch<X, float>(p, bwd, stream);
}

cudaError_t launch_types(const QrParams& p, int x_type, int y_type, bool bwd, cudaStream_t stream) {
    return x_type == ZGCM_BF16   ? launch_y<bf16>(p, y_type, bwd, stream)
           : x_type == ZGCM_FP16 ? launch_y<__half>(p, y_type, bwd, stream)
                                 : launch_y<float>(p, y_type, bwd, stream);
}

bool ok_type(int t) { return t == ZGCM_BF16 || t == ZGCM_FP16 || t == ZGCM_FP32; }

int check(const float* gamma_q, const float* gamma_k, const int* pos, int T, int Hq, int Hkv, int D, int x_type,
          int y_type, int rope_dims, double rope_base, float eps, std::initializer_list<zgcm_rows> rows) {
    if (T < 0 || Hq < 1 || Hkv < 1 || D < 1 || !ok_type(x_type) || !ok_type(y_type)) return ZGCM_ERR_INVALID_ARG;
    if (rope_dims < 0 || rope_dims > D || (rope_dims & 1)) return ZGCM_ERR_INVALID_ARG;
    if (rope_dims > 0 && !(rope_base > 0.0 && isfinite(rope_base))) return ZGCM_ERR_INVALID_ARG;
    if (!(eps >= 0.f) || !isfinite(eps)) return ZGCM_ERR_INVALID_ARG;
    if (D != kD) return ZGCM_ERR_UNSUPPORTED;
    if ((long double)T * (Hq > Hkv ? Hq : Hkv) * D >= (long double)(1ULL << 40)) return ZGCM_ERR_UNSUPPORTED;
    if (T == 0) return ZGCM_OK;
    if (!gamma_q || !gamma_k || !pos) return ZGCM_ERR_INVALID_ARG;
    for (const zgcm_rows& r : rows)
        if (!r.ptr) return ZGCM_ERR_INVALID_ARG;
    for (const void* p : {(const void*)gamma_q, (const void*)gamma_k, (const void*)pos})
        if (reinterpret_cast<uintptr_t>(p) & 15u) return ZGCM_ERR_ALIGNMENT;
    for (const zgcm_rows& r : rows)
        if ((reinterpret_cast<uintptr_t>(r.ptr) & 15u) || (r.t_stride & 7) || (r.h_stride & 7)) return ZGCM_ERR_ALIGNMENT;
    return ZGCM_OK;
}

Rows rows_of(const zgcm_rows& r) { return Rows{static_cast<char*>(r.ptr), r.t_stride, r.h_stride}; }

void fill(QrParams& p, zgcm_rows q, zgcm_rows k, const float* gamma_q, const float* gamma_k, const int* pos, int T,
          int Hq, int Hkv, int rope_dims, double rope_base, float eps) {
    p.q = rows_of(q);
    p.k = rows_of(k);
    p.gamma_q = gamma_q;
    p.gamma_k = gamma_k;
    p.pos = pos;
    p.part = nullptr;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.half = rope_dims / 2;
    p.tt = tokens_per_step(T);
    p.eps = eps;
    for (int i = 0; i < kMaxHalf; ++i)
        p.turns[i] = i < p.half ? pow(rope_base, -2.0 * i / rope_dims) * 0.15915494309189535 : 0.0;
}

}  // namespace
}  // namespace zgcm

using namespace zgcm;

extern "C" {

int zgcm_qk_norm_rope_fwd(zgcm_rows q, zgcm_rows k, const float* gamma_q, const float* gamma_k, const int* pos, int T,
                          int Hq, int Hkv, int D, int x_type, int y_type, int rope_dims, double rope_base, float eps,
                          zgcm_rows qr, zgcm_rows kr, void* cuda_stream) {
    const int st = check(gamma_q, gamma_k, pos, T, Hq, Hkv, D, x_type, y_type, rope_dims, rope_base, eps, {q, k, qr, kr});
    if (st != ZGCM_OK || T == 0) return st;
    QrParams p;
    fill(p, q, k, gamma_q, gamma_k, pos, T, Hq, Hkv, rope_dims, rope_base, eps);
    p.yq = rows_of(qr);
    p.yk = rows_of(kr);
    p.dq = p.dk = Rows{nullptr, 0, 0};
    return launch_types(p, x_type, y_type, false, static_cast<cudaStream_t>(cuda_stream)) == cudaSuccess ? ZGCM_OK
                                                                                                        : ZGCM_ERR_CUDA;
}

size_t zgcm_qk_norm_rope_bwd_workspace_size(int T) {
    return T < 1 ? 0 : (size_t)bwd_ctas(T) * 2 * kD * sizeof(float);
}

int zgcm_qk_norm_rope_bwd(zgcm_rows q, zgcm_rows k, const float* gamma_q, const float* gamma_k, const int* pos,
                          zgcm_rows dqr, zgcm_rows dkr, int T, int Hq, int Hkv, int D, int x_type, int y_type,
                          int rope_dims, double rope_base, float eps, zgcm_rows dq, zgcm_rows dk, float* dgamma_q,
                          float* dgamma_k, void* workspace, size_t workspace_bytes, void* cuda_stream) {
    const int st = check(gamma_q, gamma_k, pos, T, Hq, Hkv, D, x_type, y_type, rope_dims, rope_base, eps,
                         {q, k, dqr, dkr, dq, dk});
    if (st != ZGCM_OK) return st;
    if (!dgamma_q || !dgamma_k) return ZGCM_ERR_INVALID_ARG;
    if (((uintptr_t)dgamma_q | (uintptr_t)dgamma_k) & 15u) return ZGCM_ERR_ALIGNMENT;
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (T == 0) {
        if (cudaMemsetAsync(dgamma_q, 0, kD * sizeof(float), stream) != cudaSuccess) return ZGCM_ERR_CUDA;
        return cudaMemsetAsync(dgamma_k, 0, kD * sizeof(float), stream) == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
    }
    if (!workspace || workspace_bytes < zgcm_qk_norm_rope_bwd_workspace_size(T)) return ZGCM_ERR_WORKSPACE;
    if (reinterpret_cast<uintptr_t>(workspace) & 15u) return ZGCM_ERR_ALIGNMENT;
    QrParams p;
    fill(p, q, k, gamma_q, gamma_k, pos, T, Hq, Hkv, rope_dims, rope_base, eps);
    p.yq = rows_of(dqr);
    p.yk = rows_of(dkr);
    p.dq = rows_of(dq);
    p.dk = rows_of(dk);
    p.part = static_cast<float*>(workspace);
    if (launch_types(p, x_type, y_type, true, stream) != cudaSuccess) return ZGCM_ERR_CUDA;
    qk_dgamma_kernel<<<2 * kD / 32, 256, 0, stream>>>(p.part, bwd_ctas(T), dgamma_q, dgamma_k);
    return cudaGetLastError() == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}

}  // extern "C"
