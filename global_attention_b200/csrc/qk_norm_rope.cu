// qk_norm_rope.cu — per-head RMSNorm and partial rotation of q and k in one pass, forward and
// backward (include/zgcm_qkrope.h: the C ABI at the end of this file).
//
//   y = R(pos) (gamma x r),  r = 1/sqrt(mean x^2 + eps);   R rotates pairs (i, i + half)
//   u = R^T dy;  dgamma = sum u x r;  dx = r (gamma u - x r^2 mean(gamma u x))
//
// Bound by HBM: forward reads x and writes y, backward reads x and dy and writes dx, and no
// value is used twice except by its own row.  What has to stay small beside it is the number of
// instructions: at the rate of HBM an SM has 88 issue slots for a row forward.  Measured on a B200 in a graph's replays, 32 + 8
// heads, bf16: 65536 tokens forward 223 us, 6.0 TB/s (93% of a copy's rate), backward 352 us, 5.7 TB/s; 64 tokens 3.1 us, 1000
// backward 12.0 us.
// So a row of
// 128 belongs to 8 lanes, 16 elements each in two chunks (8 l .. and 64 + 8 l .., one 16-byte
// access of a 16-bit type each): a warp works on 4 rows at once, their sums are 3 shuffles, and
// the layer's rotated dims, 42 of 128, lie in the first chunks alone.  Two fp32 operations go in
// one instruction.  gamma and the angles make two factors for an element and token,
// y = (x A + x_partner B) r, kept in registers over the rows a warp takes of a token (formed from
// runs of shared memory: selecting element by element cost the forward 5%); the angles
// are formed once a warp and token (fp64 product and reduction: at position 262143 an fp32 product
// is off by 0.016 rad).  The partner of element d is d +- half, in another lane:
//   half = 21 (the layer's) and 16-bit rows: two lanes and 5 elements up, or 3 elements past
//     three lanes down: 5 words of the row as read by shuffles, shifted by an element (H21 instances: 224 us where
//     the general ones take 356, and 346 against 488 backward);
//   any other: the row's rotated elements go to shared memory as they were read, the first half
//     of them a second time behind the last (the partner is d + half modulo 2 half), and a lane
//     reads the partners of a chunk as one run of words.
#include <math.h>

#include <initializer_list>

#include <cuda_fp16.h>

#include "sm100.cuh"
#include "zgcm_qkrope.h"

namespace zgcm {
namespace {

constexpr int QR_THREADS = 256;
constexpr int QR_WARPS = QR_THREADS / 32;
constexpr int QR_MAX_WPT_LOG = 4;        // at most 16 warps share a token's rows
constexpr int QR_FWD_CTAS = 444;         // most CTAs of the forward (3 per SM)
constexpr int QR_BWD_CTAS = 296;         // most CTAs of the backward (2 per SM), one dgamma partial each
constexpr int kHalf21 = 21;              // the layer's rope_dims / 2

struct Rows {
    char* p;
    uint32_t ts, hs;   // elements
};

struct QrParams {
    Rows q, k, yq, yk, dq, dk;   // forward: q, k -> yq, yk.  backward: q, k, yq = dqr, yk = dkr -> dq, dk
    const float* gamma_q;
    const float* gamma_k;
    const int* pos;
    float* part;                 // backward: [CTAs][2][128] partial dgamma
    int T, Hq, Hkv, half, wpt_log;   // log2 of the warps of a token
    int fours_q, fours;              // fours of rows of a token's q, of both
    float eps;
    double turns[kMaxHalf];      // rope_base^(-2i/rope_dims) / 2 pi
};

// 8 elements of a row: kWords 32-bit words
template <typename T> struct Vec8;
template <> struct Vec8<bf16> {
    static constexpr int kWords = 4;
    uint4 w;
    __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
    __device__ __forceinline__ void set(const uint32_t (&u)[4]) { w = make_uint4(u[0], u[1], u[2], u[3]); }
    __device__ __forceinline__ void load(const char* base, long long at) {
        w = *reinterpret_cast<const uint4*>(base + 2 * at);
    }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 f[4]) const {
        f[0] = unpack_bf16(w.x);
        f[1] = unpack_bf16(w.y);
        f[2] = unpack_bf16(w.z);
        f[3] = unpack_bf16(w.w);
    }
    static __device__ __forceinline__ void store(char* base, long long at, const float2 f[4]) {
        *reinterpret_cast<uint4*>(base + 2 * at) = make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y),
                                                              pack_bf16(f[2].x, f[2].y), pack_bf16(f[3].x, f[3].y));
    }
};
template <> struct Vec8<__half> {
    static constexpr int kWords = 4;
    uint4 w;
    __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? w.x : i == 1 ? w.y : i == 2 ? w.z : w.w; }
    __device__ __forceinline__ void set(const uint32_t (&u)[4]) { w = make_uint4(u[0], u[1], u[2], u[3]); }
    __device__ __forceinline__ void load(const char* base, long long at) {
        w = *reinterpret_cast<const uint4*>(base + 2 * at);
    }
    __device__ __forceinline__ void zero() { w = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float2 f[4]) const {
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __half22float2(*reinterpret_cast<const __half2*>(&u[i]));
    }
    static __device__ __forceinline__ void store(char* base, long long at, const float2 f[4]) {
        uint32_t u[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __half2 h = __float22half2_rn(f[i]);
            u[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(base + 2 * at) = make_uint4(u[0], u[1], u[2], u[3]);
    }
};
template <> struct Vec8<float> {
    static constexpr int kWords = 8;
    float4 a, b;
    __device__ __forceinline__ uint32_t word(int i) const {
        const float4& q = i < 4 ? a : b;
        const int j = i & 3;
        return __float_as_uint(j == 0 ? q.x : j == 1 ? q.y : j == 2 ? q.z : q.w);
    }
    __device__ __forceinline__ void set(const uint32_t (&u)[8]) {
        a = make_float4(__uint_as_float(u[0]), __uint_as_float(u[1]), __uint_as_float(u[2]), __uint_as_float(u[3]));
        b = make_float4(__uint_as_float(u[4]), __uint_as_float(u[5]), __uint_as_float(u[6]), __uint_as_float(u[7]));
    }
    __device__ __forceinline__ void load(const char* base, long long at) {
        a = *reinterpret_cast<const float4*>(base + 4 * at);
        b = *reinterpret_cast<const float4*>(base + 4 * at + 16);
    }
    __device__ __forceinline__ void zero() { a = b = make_float4(0.f, 0.f, 0.f, 0.f); }
    __device__ __forceinline__ void get(float2 f[4]) const {
        f[0] = make_float2(a.x, a.y);
        f[1] = make_float2(a.z, a.w);
        f[2] = make_float2(b.x, b.y);
        f[3] = make_float2(b.z, b.w);
    }
    static __device__ __forceinline__ void store(char* base, long long at, const float2 f[4]) {
        *reinterpret_cast<float4*>(base + 4 * at) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
        *reinterpret_cast<float4*>(base + 4 * at + 16) = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
    }
};

__device__ __forceinline__ float sum8(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 2);
    x += __shfl_xor_sync(0xffffffffu, x, 1);
    return x;
}
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }

// Words of a row in the exchange buffer: 128 + 64 elements and the window of the last lane past them
template <typename T> constexpr int kPitch = (kD + kD / 2 + 8) * Vec8<T>::kWords / 8 + 2;

template <typename T, bool H21> struct QrSmem {
    static constexpr int kTurned = H21 ? 64 : kD;              // the first elements, all the rotated ones among them
    __align__(16) float gamma[2][kD];
    __align__(16) float partner[2][kTurned];                   // gamma of an element's partner
    __align__(16) float turn[QR_WARPS][2][kTurned];            // the warp's token: cosines (one where nothing turns), and
                                                               // sines, as the partner is to be added (zero)
    uint32_t ring[H21 ? 1 : QR_WARPS][4][H21 ? 1 : kPitch<T>]; // [warp][row]: its rotated elements
};

template <typename T, bool H21> __device__ __forceinline__ void fill_smem(const QrParams& p, QrSmem<T, H21>& sm) {
    constexpr int N = QrSmem<T, H21>::kTurned;
    const int d = threadIdx.x & 127, side = threadIdx.x >> 7;
    const float* g = side ? p.gamma_k : p.gamma_q;
    sm.gamma[side][d] = g[d];
    if (d < N) sm.partner[side][d] = d < 2 * p.half ? g[d < p.half ? d + p.half : d - p.half] : 0.f;
    for (int i = threadIdx.x; i < QR_WARPS * 2 * N; i += QR_THREADS) (&sm.turn[0][0][0])[i] = (i / N) & 1 ? 0.f : 1.f;
    if (!H21) {
        // a lane at the end of the rotated elements reads words that no row writes, against a factor of zero: not NaN
        uint32_t* w = &sm.ring[0][0][0];
        for (int i = threadIdx.x; i < (int)(sizeof(sm.ring) / 4); i += QR_THREADS) w[i] = 0u;
    }
    __syncthreads();
}

// cosines and sines of a position into turn[0] and turn[1]; SIGN: 1 forward, -1 back
template <int SIGN, int N>
__device__ __forceinline__ void angles(const QrParams& p, float (&turn)[2][N], int at) {
    const double pos = (double)at;
    __syncwarp();   // the token before has been read
    for (int j = threadIdx.x & 31; j < p.half; j += 32) {
        const double a = pos * p.turns[j];
        float sn, co;
        sincospif(2.0f * (float)(a - rint(a)), &sn, &co);
        turn[0][j] = turn[0][j + p.half] = co;
        turn[1][j] = -SIGN * sn;
        turn[1][j + p.half] = SIGN * sn;
    }
    __syncwarp();
}

__device__ __forceinline__ void read8(const float* at, float2 x[4]) {
    const float4 a = *reinterpret_cast<const float4*>(at), b = *reinterpret_cast<const float4*>(at + 4);
    x[0] = make_float2(a.x, a.y);
    x[1] = make_float2(a.z, a.w);
    x[2] = make_float2(b.x, b.y);
    x[3] = make_float2(b.z, b.w);
}

// Partners of the 8 elements of a first chunk, half = 21: five words of the row, as many shuffles.  Lanes 0 and 1 want
// elements 21 up, words 2, 3 of the lane two up and 0, 1, 2 of the one three up; lanes 3 to 5 want 21 down, words 1, 2, 3
// of the lane three down and 0, 1 of the one two down; lane 2 has both kinds, words 2, 3 of lane 4, 0 of lane 5, 0 and 1 of
// lane 0.  So a shuffle moves one word number, but for the last, where lane 0 sends word 0, lanes 1 and 2 word 1, the
// others word 2.  (Lanes 6 and 7, and elements 42 to 47, get elements of their own row, against a factor of zero.)
template <typename T> struct Partner21 {
    int l, from0, from1, from23, from4;   // lanes of the warp
    __device__ __forceinline__ Partner21() {
        const int lane = threadIdx.x & 31, row = lane & 24;
        l = lane & 7;
        from0 = row | (l < 3 ? l + 3 : l < 6 ? l - 2 : l);
        from1 = row | (l < 2 ? l + 3 : l == 2 ? 0 : l < 6 ? l - 3 : l);
        from23 = row | (l < 3 ? l + 2 : l < 6 ? l - 3 : l);
        from4 = row | (l < 2 ? l + 3 : l < 6 ? l - 2 : l);
    }
    __device__ __forceinline__ void get(const Vec8<T>& v, float2 y[4]) const {
        const uint32_t m = 0xffffffffu;
        const uint32_t s0 = __shfl_sync(m, v.word(0), from0), s1 = __shfl_sync(m, v.word(1), from1),
                       s2 = __shfl_sync(m, v.word(2), from23), s3 = __shfl_sync(m, v.word(3), from23),
                       s4 = __shfl_sync(m, l == 0 ? v.word(0) : l < 3 ? v.word(1) : v.word(2), from4);
        const bool up = l < 3;
        const uint32_t w0 = up ? s2 : s1, w1 = up ? s3 : s2, w2 = up ? s0 : s3, w3 = l == 2 ? s4 : up ? s1 : s0,
                       w4 = l == 2 ? s1 : s4;
        const uint32_t u[4] = {__funnelshift_r(w0, w1, 16), __funnelshift_r(w1, w2, 16), __funnelshift_r(w2, w3, 16),
                               __funnelshift_r(w3, w4, 16)};
        Vec8<T> o;
        o.set(u);
        o.get(y);
    }
};

// Partners of both chunks of a row by the exchange buffer; every lane of the warp calls it.
template <typename T>
__device__ __forceinline__ void partners(const Vec8<T> (&v)[2], float2 (&y)[2][4], uint32_t* ring, int l, int half) {
    constexpr int W = Vec8<T>::kWords, per = 8 / W;      // elements of a word
    const int n = 2 * half / per, behind = (half + per - 1) / per;   // words of a row; of its first half
    __syncwarp();   // the row before has been read
#pragma unroll
    for (int ch = 0; ch < 2; ++ch)
#pragma unroll
        for (int i = 0; i < W; ++i) {
            const int w = 8 * W * ch + W * l + i;
            if (w < n) ring[w] = v[ch].word(i);
            if (w < behind) ring[n + w] = v[ch].word(i);
        }
    __syncwarp();
#pragma unroll
    for (int ch = 0; ch < 2; ++ch) {
        const int w0 = 8 * W * ch + W * l;
        uint32_t u[W];
#pragma unroll
        for (int i = 0; i < W; ++i) u[i] = 0u;
        if (w0 < n) {
            const uint32_t* at = ring + w0 + half / per;
#pragma unroll
            for (int i = 0; i < W; ++i) u[i] = at[i];
            if (per == 2) {
                const int shift = (half & 1) * 16;
                const uint32_t last = at[W];
#pragma unroll
                for (int i = 0; i < W; ++i) u[i] = __funnelshift_r(u[i], i + 1 < W ? u[i + 1] : last, shift);
            }
        }
        Vec8<T> o;
        o.set(u);
        o.get(y[ch]);
    }
}

// Rows of a token are taken in fours, those of q and then those of k.
struct Four {
    bool isq, valid;
    int h;            // this lane's row
    __device__ __forceinline__ Four(const QrParams& p, int g, int row) {
        isq = g < p.fours_q;
        h = 4 * (isq ? g : g - p.fours_q) + row;
        valid = h < (isq ? p.Hq : p.Hkv);
    }
    __device__ __forceinline__ long long at(const Rows& x, int t, int l) const {
        return (long long)((unsigned long long)(uint32_t)t * x.ts + (unsigned long long)(uint32_t)h * x.hs + 8 * l);
    }
};

template <typename X>
__device__ __forceinline__ void load_row(const Rows& q, const Rows& k, const Four& f, Vec8<X> (&v)[2], int t, int l) {
    v[0].zero();
    v[1].zero();
    if (f.valid) {
        const Rows& x = f.isq ? q : k;
        const long long at = f.at(x, t, l);
        v[0].load(x.p, at);
        v[1].load(x.p, at + 64);
    }
}

// The walk of a warp over its units: a token, or one of wpt shares of its rows.
struct Walk {
    uint32_t unit;
    int t, g, pos;   // the unit's token, first four (past the last: no such unit) and position
    __device__ __forceinline__ explicit Walk(const QrParams& p) : unit(blockIdx.x * QR_WARPS + (threadIdx.x >> 5)) { look(p); }
    __device__ __forceinline__ bool more(const QrParams& p) const { return unit < (uint32_t)p.T << p.wpt_log; }
    __device__ __forceinline__ void step(const QrParams& p) {
        unit += gridDim.x * QR_WARPS;
        look(p);
    }
    __device__ __forceinline__ void look(const QrParams& p) {
        t = pos = 0;
        g = p.fours;
        if (more(p)) {
            t = unit >> p.wpt_log;
            g = unit & ((1u << p.wpt_log) - 1);
            pos = p.pos[t];
        }
    }
};

// A warp takes its units' rows, q and k counted through, 4 at a time and the next 4, the next unit's behind the last,
// already on their way.
template <typename X, typename Y, bool H21>
__global__ void __launch_bounds__(QR_THREADS, 3) qk_norm_rope_fwd_kernel(const __grid_constant__ QrParams p) {
    __shared__ QrSmem<X, H21> sm;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7, row = lane >> 3;
    fill_smem(p, sm);
    const int step = 1 << p.wpt_log;
    const Partner21<X> p21;
    Walk at(p);
    Vec8<X> next[2];
    load_row(p.q, p.k, Four(p, at.g, row), next, at.t, l);
    while (at.more(p)) {
        const int t = at.t, g0 = at.g;
        angles<1>(p, sm.turn[warp], at.pos);
        at.step(p);
        float2 a[2][4], b[2][4];   // y_d' = y_d a + y_partner b, times r
        int side = -1;   // whose factors a, b are
        for (int g = g0; g < p.fours; g += step) {
            const Four four(p, g, row);
            Vec8<X> v[2] = {next[0], next[1]};
            const bool last = g + step >= p.fours;
            load_row(p.q, p.k, Four(p, last ? at.g : g + step, row), next, last ? at.t : t, l);
            if (side != !four.isq) {
                side = !four.isq;
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
                    const int d = 64 * ch + 8 * l;
                    read8(&sm.gamma[side][d], a[ch]);
                    if (H21 && ch == 1) break;
                    float2 co[4], si[4];
                    read8(&sm.turn[warp][0][d], co);
                    read8(&sm.turn[warp][1][d], si);
                    read8(&sm.partner[side][d], b[ch]);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        a[ch][e] = sm100::fmul2(a[ch][e], co[e]);
                        b[ch][e] = sm100::fmul2(b[ch][e], si[e]);
                    }
                }
            }
            float2 f[2][4], y[2][4];
            v[0].get(f[0]);
            v[1].get(f[1]);
            if constexpr (H21)
                p21.get(v[0], y[0]);
            else
                partners(v, y, sm.ring[H21 ? 0 : warp][row], l, p.half);
            float2 ss = sm100::fmul2(f[0][0], f[0][0]);
#pragma unroll
            for (int e = 1; e < 8; ++e) ss = sm100::ffma2(f[e >> 2][e & 3], f[e >> 2][e & 3], ss);
            const float2 r = pair(rsqrtf(sum8(ss.x + ss.y) * (1.0f / kD) + p.eps));
#pragma unroll
            for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    float2 z = sm100::fmul2(f[ch][e], a[ch][e]);
                    if (!H21 || ch == 0) z = sm100::ffma2(y[ch][e], b[ch][e], z);
                    f[ch][e] = sm100::fmul2(z, r);
                }
            if (four.valid) {
                const Rows& o = four.isq ? p.yq : p.yk;
                const long long to = four.at(o, t, l);
                Vec8<Y>::store(o.p, to, f[0]);
                Vec8<Y>::store(o.p, to + 64, f[1]);
            }
        }
    }
}

// As the forward.  dgamma: this lane's 16 sums over its q rows in registers, those over its k rows, a quarter as
// many in the layer, in shared memory; the CTA's partials at the end.
template <typename Y, bool H21> struct BwdSmem {
    QrSmem<Y, H21> s;
    float4 dgk[QR_WARPS][4][32];
};

template <typename X, typename Y, bool H21>
__global__ void __launch_bounds__(QR_THREADS, 2) qk_norm_rope_bwd_kernel(const __grid_constant__ QrParams p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    QrSmem<Y, H21>& sm = reinterpret_cast<BwdSmem<Y, H21>*>(dyn)->s;
    auto& dgk = reinterpret_cast<BwdSmem<Y, H21>*>(dyn)->dgk;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the sum of the partials may take its place early
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, l = lane & 7, row = lane >> 3;
    fill_smem(p, sm);
    float2 dg[2][4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) dgk[warp][i][lane] = make_float4(0.f, 0.f, 0.f, 0.f);
    const Partner21<Y> p21;
    const int step = 1 << p.wpt_log;
    Walk at(p);
    Vec8<X> nv[2];
    Vec8<Y> nw[2];
    load_row(p.q, p.k, Four(p, at.g, row), nv, at.t, l);
    load_row(p.yq, p.yk, Four(p, at.g, row), nw, at.t, l);
    while (at.more(p)) {
        const int t = at.t, g0 = at.g;
        float2 a[2][4], b[2][4];
        angles<-1>(p, sm.turn[warp], at.pos);
        at.step(p);
#pragma unroll
        for (int ch = 0; ch < (H21 ? 1 : 2); ++ch) {
            read8(&sm.turn[warp][0][64 * ch + 8 * l], a[ch]);
            read8(&sm.turn[warp][1][64 * ch + 8 * l], b[ch]);
        }
        for (int g = g0; g < p.fours; g += step) {
            const Four four(p, g, row);
            const Vec8<X> v[2] = {nv[0], nv[1]};
            const Vec8<Y> w[2] = {nw[0], nw[1]};
            const bool last = g + step >= p.fours;
            const Four next(p, last ? at.g : g + step, row);
            load_row(p.q, p.k, next, nv, last ? at.t : t, l);
            load_row(p.yq, p.yk, next, nw, last ? at.t : t, l);
            float2 f[2][4], u[2][4], y[2][4], ug[2][4];
#pragma unroll
            for (int ch = 0; ch < 2; ++ch) {
                v[ch].get(f[ch]);
                w[ch].get(u[ch]);
            }
            if constexpr (H21)
                p21.get(w[0], y[0]);
            else
                partners(w, y, sm.ring[H21 ? 0 : warp][row], l, p.half);
            const float* gamma = sm.gamma[four.isq ? 0 : 1] + 8 * l;
            float2 ss = pair(0.f), sx = pair(0.f);
#pragma unroll
            for (int ch = 0; ch < 2; ++ch)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    if (!H21 || ch == 0) u[ch][e] = sm100::ffma2(y[ch][e], b[ch][e], sm100::fmul2(u[ch][e], a[ch][e]));
                    ug[ch][e] = sm100::fmul2(u[ch][e], *reinterpret_cast<const float2*>(gamma + 64 * ch + 2 * e));
                    ss = sm100::ffma2(f[ch][e], f[ch][e], ss);
                    sx = sm100::ffma2(f[ch][e], ug[ch][e], sx);
                }
            const float sq = sum8(ss.x + ss.y), sd = sum8(sx.x + sx.y);
            const float r = rsqrtf(sq * (1.0f / kD) + p.eps);
            const float2 m = pair(-r * r * sd * (1.0f / kD)), rr = pair(r);     // m = -r mean(gamma u xhat)
            if (four.valid) {
                const Rows& o = four.isq ? p.dq : p.dk;
                const long long to = four.at(o, t, l);
#pragma unroll
                for (int ch = 0; ch < 2; ++ch) {
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        ug[ch][e] = sm100::fmul2(rr, sm100::ffma2(f[ch][e], m, ug[ch][e]));
                        f[ch][e] = sm100::fmul2(u[ch][e], sm100::fmul2(f[ch][e], rr));       // dgamma's term
                    }
                    Vec8<X>::store(o.p, to + 64 * ch, ug[ch]);
                }
                if (four.isq) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) dg[e >> 2][e & 3] = sm100::fadd2(dg[e >> 2][e & 3], f[e >> 2][e & 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        float4& s = dgk[warp][i][lane];
                        const float2 x = f[i >> 1][2 * (i & 1)], z = f[i >> 1][2 * (i & 1) + 1];
                        s = make_float4(s.x + x.x, s.y + x.y, s.z + z.x, s.w + z.y);
                    }
                }
            }
        }
    }
    // the CTA's sums, in a fixed order; the angles' place is free then
    float(*red)[kD] = reinterpret_cast<float(*)[kD]>(sm.turn);
    static_assert(sizeof(sm.turn) >= QR_WARPS * kD * sizeof(float), "one row of 128 sums a warp");
#pragma unroll
    for (int side = 0; side < 2; ++side) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float2 v = dg[i >> 3][(i >> 1) & 3];
            float x = (i & 1) ? v.y : v.x;
            if (side) x = reinterpret_cast<const float*>(&dgk[warp][i >> 2][lane])[i & 3];
            x += __shfl_xor_sync(0xffffffffu, x, 8);
            x += __shfl_xor_sync(0xffffffffu, x, 16);
            if (lane < 8) red[warp][64 * (i >> 3) + 8 * l + (i & 7)] = x;
        }
        __syncthreads();
        if (threadIdx.x < kD) {
            float x = 0.f;
            for (int i = 0; i < QR_WARPS; ++i) x += red[i][threadIdx.x];
            p.part[((size_t)blockIdx.x * 2 + side) * kD + threadIdx.x] = x;
        }
    }
}

// dgamma[side][d] = sum over the CTAs' partials, in a fixed order: a CTA takes 32 of the 256 columns, each of its 32 warps
// every 32nd partial, all of them on their way at once (with 8 warps and 4 loads at a time the
// gradient of 1000 tokens took 16.5 us instead of 14.4).
constexpr int QR_SUM_THREADS = 1024, QR_SUM_WARPS = QR_SUM_THREADS / 32;
__global__ void __launch_bounds__(QR_SUM_THREADS) qk_dgamma_kernel(const float* part, int n, float* dgamma_q, float* dgamma_k) {
    constexpr int MOST = (QR_BWD_CTAS + QR_SUM_WARPS - 1) / QR_SUM_WARPS;
    __shared__ float red[QR_SUM_WARPS][32];
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
    asm volatile("griddepcontrol.wait;" ::: "memory");   // the partials
    float x[MOST], a = 0.f;
#pragma unroll
    for (int i = 0; i < MOST; ++i) x[i] = w + i * QR_SUM_WARPS < n ? part[(size_t)(w + i * QR_SUM_WARPS) * 2 * kD + col] : 0.f;
#pragma unroll
    for (int i = 0; i < MOST; ++i) a += x[i];
    red[w][lane] = a;
    __syncthreads();
    if (w == 0) {
#pragma unroll
        for (int i = 1; i < QR_SUM_WARPS; ++i) a += red[i][lane];
        (col < kD ? dgamma_q : dgamma_k)[col % kD] = a;
    }
}

// Warps of a token: the most that still leaves each its own warp on an SM (16 a SM, 148 SMs), so that a decode
// step's few tokens spread over the GPU; one for long batches (the angles are formed once a warp).  Measured with room for
// 8, 16 and 32 warps an SM: 1000 tokens 6.9, 6.6, 7.6 us forward and 12.0, 11.3, 12.4 backward; 256 tokens 4.2, 4.2, 5.2
// and 7.2, 7.8, 8.6.
int warps_per_token_log(int T) {
    int n = QR_MAX_WPT_LOG;
    while (n > 0 && ((long long)T << n) > 148 * 16) --n;
    return n;
}

int all_ctas(int T) { return (int)((((long long)T << warps_per_token_log(T)) + QR_WARPS - 1) / QR_WARPS); }

int bwd_ctas(int T) {
    const int n = all_ctas(T);
    return n < QR_BWD_CTAS ? n : QR_BWD_CTAS;
}

template <typename X, typename Y, bool H21> cudaError_t launch_fwd(const QrParams& p, cudaStream_t stream) {
    qk_norm_rope_fwd_kernel<X, Y, H21><<<min(all_ctas(p.T), QR_FWD_CTAS), QR_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

template <typename X, typename Y, bool H21> cudaError_t launch_bwd(const QrParams& p, cudaStream_t stream) {
    auto kernel = qk_norm_rope_bwd_kernel<X, Y, H21>;
    constexpr size_t smem = sizeof(BwdSmem<Y, H21>);
    if (smem > 48 * 1024) {
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
    }
    kernel<<<bwd_ctas(p.T), QR_THREADS, smem, stream>>>(p);
    return cudaGetLastError();
}

template <typename X, typename Y> cudaError_t launch(const QrParams& p, bool bwd, cudaStream_t stream) {
    // by the type whose rows are exchanged: x forward, dy backward
    constexpr bool fwd16 = sizeof(X) == 2, bwd16 = sizeof(Y) == 2;
    const bool h21 = p.half == kHalf21;
    if (bwd) return bwd16 && h21 ? launch_bwd<X, Y, bwd16>(p, stream) : launch_bwd<X, Y, false>(p, stream);
    return fwd16 && h21 ? launch_fwd<X, Y, fwd16>(p, stream) : launch_fwd<X, Y, false>(p, stream);
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
    for (const zgcm_rows& r : rows)
        if (r.t_stride < 0 || r.h_stride < 0 || r.t_stride > 0xffffffffLL || r.h_stride > 0xffffffffLL) return ZGCM_ERR_UNSUPPORTED;
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

Rows rows_of(const zgcm_rows& r) { return Rows{static_cast<char*>(r.ptr), (uint32_t)r.t_stride, (uint32_t)r.h_stride}; }

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
    p.wpt_log = warps_per_token_log(T);
    p.fours_q = (Hq + 3) / 4;
    p.fours = p.fours_q + (Hkv + 3) / 4;
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
    // on the SMs while the backward's last CTAs still run
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(2 * kD / 32);
    cfg.blockDim = dim3(QR_SUM_THREADS);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, qk_dgamma_kernel, (const float*)p.part, bwd_ctas(T), dgamma_q, dgamma_k) == cudaSuccess
               ? ZGCM_OK
               : ZGCM_ERR_CUDA;
}

}  // extern "C"
