// kv8_attn.cuh — what the decode kernels over the 8-bit block cache share: a block's and the tail's part
// in one warp's running softmax (kv8_decode.cu says how and why).
#pragma once
#include <math.h>

#include "kv8.cuh"
#include "sm100.cuh"
#include "tc_rows.cuh"

namespace zgcm {
using namespace sm100;

constexpr int DK_HEADS = 8;                // heads of an item
constexpr float kInvP = 1.f / 16384.f;     // p is held times 2^14: as fp16 above its subnormals

struct DecodeKv8Params {
    CUtensorMap tm_k, tm_v;                // [n_pages * Hkv * 64, 128] bytes, box 64 rows
    Kv8 c;
    const void* q;
    const bf16* g;
    const int* pos;
    const int* blocks;
    int n_list, Hq, G, HT, W;              // HT: items of a KV head (8 heads each)
    int rows;                              // heads a record has room for: min(G, 8)
    int split, stages;                     // kv8_direct_kernel: CTAs of an item, stages of its ring
    float scale_log2;
    bf16* out;
    float* lse;
    float* part;                           // kv8_decode_kernel: records [item + CTA][rows][DK_REC]
    int* err;
};

// What a position asks for: its own block, the first block and key its window reaches, and the
// units of one item: blocks to read (some of a list may turn out to be passed over) + 1 for the tail.
struct Span {
    int own, lo, jlo, units;
    bool idle, bad;
};

__device__ __forceinline__ Span span_of(const DecodeKv8Params& p, int pos) {
    Span s;
    s.idle = pos < 0;
    s.own = s.idle ? 0 : pos / kBlk;
    s.lo = s.idle ? 0 : max(0, pos - p.W + 1);
    s.jlo = s.lo / kBlk;
    s.bad = s.own - s.jlo >= p.c.NB;
    s.units = s.idle || s.bad ? 1 : (p.blocks ? p.n_list : s.own - s.jlo) + 1;
    return s;
}

struct Meta {
    float ks, vs;
    int j;        // block, or -1: passed over
    int pad;
};

// ------------------------------------------------------------------ tensor-core and code helpers

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
// d = A B + c
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1, float c0, float c1, float c2, float c3) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%10,%11,%12,%13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
                     "{%10,%11,%12,%13};"
                     : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    mma16816<BF>(d, a0, a1, a2, a3, b0, b1, d[0], d[1], d[2], d[3]);
}

__device__ __forceinline__ uint32_t less1152(uint32_t w) {
    const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&w), __half2half2(__ushort_as_half(0x6480)));
    return *reinterpret_cast<const uint32_t*>(&x);
}
__device__ __forceinline__ uint32_t e4m3_pair(uint32_t w) {   // the low two bytes
    uint32_t r;
    asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\t}" : "=r"(r) : "r"(w));
    return r;
}
// four codes -> two fp16 pairs: of bytes 0, 1 and 2, 3
template <int CODE> __device__ __forceinline__ void pairs_near(uint32_t w, uint32_t& x, uint32_t& y) {
    if (CODE == ZGCM_E4M3) {
        x = e4m3_pair(w);
        y = e4m3_pair(w >> 16);
    } else {
        w ^= 0x80808080u;
        x = less1152(__byte_perm(w, 0x64646464u, 0x4140));
        y = less1152(__byte_perm(w, 0x64646464u, 0x4342));
    }
}
// ... of bytes 0, 2 and 1, 3
template <int CODE> __device__ __forceinline__ void pairs_apart(uint32_t w, uint32_t& x, uint32_t& y) {
    if (CODE == ZGCM_E4M3) {
        w = __byte_perm(w, 0u, 0x3120);
        x = e4m3_pair(w);
        y = e4m3_pair(w >> 16);
    } else {
        w ^= 0x80808080u;
        x = less1152(__byte_perm(w, 0x64646464u, 0x4240));
        y = less1152(__byte_perm(w, 0x64646464u, 0x4341));
    }
}

template <typename TK> struct KeyType;
template <> struct KeyType<__half> {
    static constexpr bool kBf = false;
    static __device__ __forceinline__ float2 unpack(uint32_t u) {
        return __half22float2(*reinterpret_cast<const __half2*>(&u));
    }
};
template <> struct KeyType<bf16> {
    static constexpr bool kBf = true;
    static __device__ __forceinline__ float2 unpack(uint32_t u) { return unpack_bf16(u); }
};

__device__ __forceinline__ uint32_t pack_half(float a, float b) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// a pair of values as a 16-bit pair and the pair of what the rounding left
template <bool BF> __device__ __forceinline__ void split2(float a, float b, uint32_t& hi, uint32_t& lo) {
    if (BF) {
        hi = pack_bf16(a, b);
        const float2 r = unpack_bf16(hi);
        lo = pack_bf16(a - r.x, b - r.y);
    } else {
        hi = pack_half(a, b);
        const float2 r = __half22float2(*reinterpret_cast<const __half2*>(&hi));
        lo = pack_half(a - r.x, b - r.y);
    }
}

__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}
// A warp's share of an item.  Lane (r, c) = (lane / 4, lane % 4) holds head r: of O, for i = 0 .. 7, the dims
// 16 i + 4 c + {0, 2} in e[i] and + {1, 3} in o[i] (the pairs a product leaves side by side).
struct State {
    float m, l;      // running maximum (base 2), this lane's part of the sum (times 2^14)
    float2 e[8], o[8];
};

// O of one 16-dim chunk <- O a + (its two rows: of p rounded and of what the rounding left) f
__device__ __forceinline__ void join_o(State& t, int i, const float (&e)[4], const float (&o)[4], float2 a, float2 f) {
    t.e[i] = ffma2(fadd2(make_float2(e[0], e[1]), make_float2(e[2], e[3])), f, fmul2(t.e[i], a));
    t.o[i] = ffma2(fadd2(make_float2(o[0], o[1]), make_float2(o[2], o[3])), f, fmul2(t.o[i], a));
}

// Scores of a set of keys in base 2 -> p relative to the set's own maximum (times 2^14: as fp16 down to 2^-38 of
// it, whatever the sets before had), the running maximum and sum.  a: factor for O so far; b: for this set's.
template <int N> __device__ __forceinline__ void soften(State& t, float2 (&s)[N], float& a, float& b) {
    float mt = fmaxf(s[0].x, s[0].y);
#pragma unroll
    for (int i = 1; i < N; ++i) mt = fmaxf(mt, fmaxf(s[i].x, s[i].y));
    mt = fmaxf(quad_max(mt), -3e38f);     // scores of -infinity alone have p = 0, not NaN
    const float m = fmaxf(t.m, mt);
    a = fast_exp2(t.m - m);               // 0 from the empty start
    b = fast_exp2(mt - m);
    const float2 base = make_float2(14.f - mt, 14.f - mt);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = fadd2(s[i], base);
        s[i] = make_float2(fast_exp2(s[i].x), fast_exp2(s[i].y));
        sum = fadd2(sum, s[i]);
    }
    t.l = fmaf(t.l, a, (sum.x + sum.y) * b);
    t.m = m;
}

// 32 keys of a block, those from k0
template <int CODE>
__device__ __forceinline__ void block8(State& t, const uint32_t (&q)[8][2], float qscale, uint32_t k_addr, uint32_t v_addr,
                                       const Meta& meta, int lo, int k0) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    const int mi = lane >> 3, r = lane & 7;            // ldmatrix: this lane's row r of matrix mi
    float2 s[4];
    k_addr += k0 * kD;
    v_addr += k0 * kD;
    // S: 8 keys at a time; matrices are the 16-byte chunks of the keys' rows
    const float2 f = make_float2(meta.ks * qscale, meta.ks * qscale);
#pragma unroll
    for (int n = 0; n < 4; ++n) {
        float d[4];
        const uint32_t row = k_addr + (n * 8 + r) * kD;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t w[4];
            ldsm4(row + (((4 * half + mi) ^ r) << 4), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t b0, b1;
                pairs_near<CODE>(w[i], b0, b1);
                if (half + i == 0)
                    mma16816<false>(d, q[0][0], 0u, q[0][1], 0u, b0, b1, 0.f, 0.f, 0.f, 0.f);
                else
                    mma16816<false>(d, q[4 * half + i][0], 0u, q[4 * half + i][1], 0u, b0, b1);
            }
        }
        s[n] = fmul2(make_float2(d[0], d[1]), f);
    }
    if (meta.j * kBlk + k0 < lo) {
        const int first = lo - meta.j * kBlk - k0 - 2 * c;
#pragma unroll
        for (int n = 0; n < 4; ++n) {
            if (8 * n < first) s[n].x = -INFINITY;
            if (8 * n + 1 < first) s[n].y = -INFINITY;
        }
    }
    float a, b;
    soften(t, s, a, b);
    uint32_t hi[4], lo2[4];
#pragma unroll
    for (int n = 0; n < 4; ++n) split2<false>(s[n].x, s[n].y, hi[n], lo2[n]);
    // O: 16 dims at a time (their 16-byte chunk); matrices are groups of 8 keys, transposed: a lane gets keys
    // 2c, 2c+1 of the dims 2r, 2r+1 of the chunk
    const float vs = meta.vs * (b * kInvP);
    const float2 a2 = make_float2(a, a), f2 = make_float2(vs, vs);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float e[4], o[4];
        uint32_t w[4], be[4], bo[4];
        ldsm4t(v_addr + (8 * mi + r) * kD + ((i ^ r) << 4), w);
#pragma unroll
        for (int x = 0; x < 4; ++x) pairs_apart<CODE>(w[x], be[x], bo[x]);
        mma16816<false>(e, hi[0], lo2[0], hi[1], lo2[1], be[0], be[1], 0.f, 0.f, 0.f, 0.f);
        mma16816<false>(o, hi[0], lo2[0], hi[1], lo2[1], bo[0], bo[1], 0.f, 0.f, 0.f, 0.f);
        mma16816<false>(e, hi[2], lo2[2], hi[3], lo2[3], be[2], be[3]);
        mma16816<false>(o, hi[2], lo2[2], hi[3], lo2[3], bo[2], bo[3]);
        join_o(t, i, e, o, a2, f2);
    }
}

// 16 keys of the tail, k0 .. k0 + 15 of its block, valid where first <= key <= last; 16-bit products of the
// types as they are (values in bf16 span more than fp16 does)
template <typename TK>
__device__ __forceinline__ void tail16(State& t, const uint32_t (&q)[8][2], float scale, const TK* k, const bf16* v, int k0,
                                       int first, int last) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
    uint2 kw[2][8];
    uint32_t vw[8][4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const TK* row = k + (k0 + 8 * n + r) * kD + 4 * c;
#pragma unroll
        for (int i = 0; i < 8; ++i) kw[n][i] = *reinterpret_cast<const uint2*>(row + 16 * i);
    }
    bool on[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int key = k0 + 2 * c + (x & 1) + 8 * (x >> 1);
        on[x] = key >= first && key <= last;
        // a masked row may hold anything: it must not reach the product
#pragma unroll
        for (int i = 0; i < 8; ++i)
            vw[i][x] = on[x] ? *reinterpret_cast<const uint32_t*>(v + key * kD + 16 * i + 2 * r) : 0u;
    }
    float2 s[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) mma16816<KeyType<TK>::kBf>(d, q[i][0], 0u, q[i][1], 0u, kw[n][i].x, kw[n][i].y);
        s[n].x = on[2 * n] ? d[0] * scale : -INFINITY;
        s[n].y = on[2 * n + 1] ? d[1] * scale : -INFINITY;
    }
    float a, b;
    soften(t, s, a, b);
    b *= kInvP;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) split2<true>(s[n].x, s[n].y, hi[n], lo[n]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float e[4], o[4];
        mma16816<true>(e, hi[0], lo[0], hi[1], lo[1], __byte_perm(vw[i][0], vw[i][1], 0x5410),
                       __byte_perm(vw[i][2], vw[i][3], 0x5410), 0.f, 0.f, 0.f, 0.f);
        mma16816<true>(o, hi[0], lo[0], hi[1], lo[1], __byte_perm(vw[i][0], vw[i][1], 0x7632),
                       __byte_perm(vw[i][2], vw[i][3], 0x7632), 0.f, 0.f, 0.f, 0.f);
        join_o(t, i, e, o, make_float2(a, a), make_float2(b, b));
    }
}

// out and lse of four dims of one head from its maximum, sum and O
__device__ __forceinline__ void finish4(const DecodeKv8Params& p, size_t head, int d, float m, float l, const float (&o)[4]) {
    const float inv = 1.f / (l * kInvP);
    float x[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    if (p.g) {
        const uint2 w = *reinterpret_cast<const uint2*>(p.g + head * kD + d);
        const float2 a = unpack_bf16(w.x), b = unpack_bf16(w.y);
        x[0] *= sigmoidf_(a.x);
        x[1] *= sigmoidf_(a.y);
        x[2] *= sigmoidf_(b.x);
        x[3] *= sigmoidf_(b.y);
    }
    *reinterpret_cast<uint2*>(p.out + head * kD + d) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    if (d == 0) p.lse[head] = (m + log2f(l) - 14.f) * kLn2;
}


// This lane's 32 elements of its head's q (r < nh, zeros else): chunk i's pairs 16 i + 4 c, + 2
template <typename TK>
__device__ __forceinline__ void load_q(const DecodeKv8Params& p, size_t head, bool on, uint32_t (&q)[8][2]) {
    const int c = threadIdx.x & 3;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint2 u = make_uint2(0u, 0u);
        if (on) u = *reinterpret_cast<const uint2*>(static_cast<const TK*>(p.q) + head * kD + 16 * i + 4 * c);
        q[i][0] = u.x;
        q[i][1] = u.y;
    }
}

// q as the fp16 that meets codes, and the scale of its scores in base 2: fp16 as it is, bf16 times the power of
// two that brings the head's largest element to 2^14
template <typename TK>
__device__ __forceinline__ float q_as_half(const DecodeKv8Params& p, const uint32_t (&q)[8][2], uint32_t (&h)[8][2]) {
    float mx = 0.f;
    if (KeyType<TK>::kBf) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 a = unpack_bf16(q[i][0]), b = unpack_bf16(q[i][1]);
            mx = fmaxf(mx, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
        }
        mx = quad_max(mx);
    }
    const int ex = min(254, 268 - (int)(__float_as_uint(mx) >> 23));
    const float up = __uint_as_float((uint32_t)ex << 23);   // 2^14 / 2^floor(log2 mx)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        h[i][0] = q[i][0];
        h[i][1] = q[i][1];
        if (KeyType<TK>::kBf) {
            const float2 a = unpack_bf16(q[i][0]), b = unpack_bf16(q[i][1]);
            h[i][0] = pack_half(a.x * up, a.y * up);
            h[i][1] = pack_half(b.x * up, b.y * up);
        }
    }
    return KeyType<TK>::kBf ? p.scale_log2 / up : p.scale_log2;
}

// One sequence's row without an answer: zeros and -inf for an idle sequence, NaN for a window beyond the table.  By one
// warp, for the head of each lane's row.
__device__ __forceinline__ void no_answer(const DecodeKv8Params& p, size_t head, bool idle) {
    const int c = threadIdx.x & 3;
    const uint32_t u = idle ? 0u : 0x7fff7fffu;
#pragma unroll
    for (int i = 0; i < 8; ++i) *reinterpret_cast<uint2*>(p.out + head * kD + 16 * i + 4 * c) = make_uint2(u, u);
    if (c == 0) p.lse[head] = idle ? -INFINITY : NAN;
}

// Block number `i` of an item's units as the kernel reads it: block j (-1: passed over), page (-1: none), scales.
struct Tile {
    int j, page;
    float ks, vs;
};

__device__ __forceinline__ Tile tile_of(const DecodeKv8Params& p, const Span& s, int b, int kvh, int i) {
    Tile t{s.jlo + i, -1, 0.f, 0.f};
    if (p.blocks) {
        const int* list = p.blocks + ((size_t)b * p.c.Hkv + kvh) * p.n_list + i;
        t.j = *list;
        if (t.j < s.jlo || t.j >= s.own || (i > 0 && t.j <= list[-1])) t.j = -1;
    }
    if (t.j >= 0) {
        t.page = kv8_page(p.c, b, t.j);
        t.ks = t.vs = NAN;          // a bad page reads as NaN
        if (t.page >= 0) {
            t.ks = p.c.ks[(size_t)t.page * p.c.Hkv + kvh];
            t.vs = p.c.vs[(size_t)t.page * p.c.Hkv + kvh];
        }
    }
    return t;
}

}  // namespace zgcm
