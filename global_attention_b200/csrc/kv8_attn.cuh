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
    CUtensorMap tm_k, tm_v;                // [n_pages * Hkv * 64, 128] bytes, box 32 rows
    Kv8 c;
    const void* q;
    const bf16* g;
    const int* pos;
    const int* blocks;
    int n_list, Hq, G, HT, W;              // HT: items of a KV head (8 heads each)
    int rows;                              // heads a record has room for: min(G, 8)
    int split;                             // kv8_direct_kernel: CTAs of an item
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

// an 8 x 8 matrix of 16-bit values (two a lane) transposed
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// over the 8 lanes of a column: those with the same lane % 4
__device__ __forceinline__ float column_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float column_sum(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}
__device__ __forceinline__ float quad_max(float x) {
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
}

// A warp's share of an item.  Lane (r, c) = (lane / 4, lane % 4) holds the columns 2 c and 2 c + 1 (.x and .y): of O, for
// i = 0 .. 7, the dims 16 i + 2 r in o[i][0] and 16 i + 2 r + 1 in o[i][1].
//
// Columns are heads.  p enters the second product in two halves, hi = fp16(p) and lo = fp16(p - hi), 22 bits of it (one half
// alone is off by up to 2^-12 of each p: an output that cancels to 2^-12 of sum p |v| was lost).  WIDE items (more
// than 4 heads in a group) multiply twice.  Others have the columns 4 .. 7 free: they hold the four heads again, the same
// scores, maxima and sums, but take the low halves, and O's two columns of a head are added at the item's end: no
// product more than with one half.  Measured with one half / with both (us): 64 sequences of up to 16K, INT8, 8 KV heads of 4
// 273 / 280, 4 of 8 158 / 152, 2 of 16 137 / 143; 16 of up to 8K, 4 of 8 33 / 38; 32 listed blocks 24.6 / 24.6, 4 of 8
// 16.7 / 19.4.
struct State {
    float2 m, l;      // running maximum (base 2), this lane's part of the sum (times 2^14)
    float2 o[8][2];
    __device__ __forceinline__ State() : m(make_float2(-INFINITY, -INFINITY)), l(make_float2(0.f, 0.f)) {
#pragma unroll
        for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = make_float2(0.f, 0.f);
    }
};

// O of one 16-dim chunk <- O a + d f
__device__ __forceinline__ void join_o(State& t, int i, const float (&d)[4], float2 a, float2 f) {
    t.o[i][0] = ffma2(make_float2(d[0], d[1]), f, fmul2(t.o[i][0], a));
    t.o[i][1] = ffma2(make_float2(d[2], d[3]), f, fmul2(t.o[i][1], a));
}

// Scores of a set of keys in base 2 (N of this lane's two columns) -> p relative to the set's own maximum (times 2^14: as
// fp16 down to 2^-38 of it, whatever the sets before had), the running maximum and sum.  a: factor for O so far; b: for
// this set's.
template <int N> __device__ __forceinline__ void soften(State& t, float2 (&s)[N], float2& a, float2& b) {
    float2 mt = s[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mt = make_float2(fmaxf(mt.x, s[i].x), fmaxf(mt.y, s[i].y));
    mt.x = fmaxf(column_max(mt.x), -3e38f);     // scores of -infinity alone have p = 0, not NaN
    mt.y = fmaxf(column_max(mt.y), -3e38f);
    const float2 m = make_float2(fmaxf(t.m.x, mt.x), fmaxf(t.m.y, mt.y));
    a = make_float2(fast_exp2(t.m.x - m.x), fast_exp2(t.m.y - m.y));   // 0 from the empty start
    b = make_float2(fast_exp2(mt.x - m.x), fast_exp2(mt.y - m.y));
    // the difference first, which is 0 for the largest: 14 - mt is rounded at mt's magnitude, so that from |mt| = 2^25 on p
    // could come out as 2^16, past fp16
    const float2 minus = make_float2(-mt.x, -mt.y), up = make_float2(14.f, 14.f);
    float2 sum = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = fadd2(fadd2(s[i], minus), up);
        s[i] = make_float2(fast_exp2(s[i].x), fast_exp2(s[i].y));
        sum = fadd2(sum, s[i]);
    }
    t.l = ffma2(t.l, a, fmul2(sum, b));
    t.m = m;
}

// Scores in base 2 of 32 keys at k_addr, of whose block the first `masked` are before the window: s[2 i], s[2 i + 1] of
// the keys 16 i + r and 16 i + 8 + r.
template <int CODE>
__device__ __forceinline__ void scores32(float2 (&s)[4], const uint32_t (&q)[8][2], float2 f, uint32_t k_addr, int masked) {
    const int lane = threadIdx.x & 31, r = lane >> 2;
    // ldmatrix: this lane's row of matrix mi; matrices are 8 keys (mi & 1) of a 16-byte chunk (mi >> 1)
    const int mi = lane >> 3, row = (mi & 1) * 8 + (lane & 7);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
        float d[4];
#pragma unroll
        for (int i = 0; i < 8; i += 2) {
            uint32_t w[4], x[4], y[4];
            ldsm4(k_addr + (16 * t + row) * kD + (((i + (mi >> 1)) ^ (lane & 7)) << 4), w);
#pragma unroll
            for (int j = 0; j < 4; ++j) pairs_near<CODE>(w[j], x[j], y[j]);
            if (i == 0)
                mma16816<false>(d, x[0], x[1], y[0], y[1], q[0][0], q[0][1], 0.f, 0.f, 0.f, 0.f);
            else
                mma16816<false>(d, x[0], x[1], y[0], y[1], q[i][0], q[i][1]);
            mma16816<false>(d, x[2], x[3], y[2], y[3], q[i + 1][0], q[i + 1][1]);
        }
        s[2 * t] = fmul2(make_float2(d[0], d[1]), f);
        s[2 * t + 1] = fmul2(make_float2(d[2], d[3]), f);
    }
    if (masked > 0) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (8 * i + r < masked) s[i] = make_float2(-INFINITY, -INFINITY);
    }
}

// O takes in 32 keys: b fragments of their p (two of each 16 keys; WIDE: of the high halves, then of the low ones), their
// values at v_addr.
template <int CODE, bool WIDE>
__device__ __forceinline__ void values32(State& t, const uint32_t (&pb)[WIDE ? 8 : 4], float2 a, float2 f, uint32_t v_addr) {
    const int lane = threadIdx.x & 31, mi = lane >> 3, r = lane & 7;
    // 16 dims at a time (their 16-byte chunk); matrices are groups of 8 keys, transposed: a lane gets keys
    // 2 c, 2 c + 1 of the dims 2 r, 2 r + 1 of the chunk (rows r and r + 8 of the product)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float d[4];
        uint32_t w[4], x[4], y[4];
        ldsm4t(v_addr + (8 * mi + r) * kD + ((i ^ r) << 4), w);
#pragma unroll
        for (int j = 0; j < 4; ++j) pairs_apart<CODE>(w[j], x[j], y[j]);
        mma16816<false>(d, x[0], y[0], x[1], y[1], pb[0], pb[1], 0.f, 0.f, 0.f, 0.f);
        mma16816<false>(d, x[2], y[2], x[3], y[3], pb[2], pb[3]);
        if constexpr (WIDE) {
            mma16816<false>(d, x[0], y[0], x[1], y[1], pb[4], pb[5]);
            mma16816<false>(d, x[2], y[2], x[3], y[3], pb[6], pb[7]);
        }
        join_o(t, i, d, a, f);
    }
}

// 16 keys of the tail, k0 .. k0 + 15 of its block, valid where first <= key <= last; 16-bit products of the
// types as they are (values in bf16 span more than fp16 does, so p goes in as three bf16, its 24 bits)
template <typename TK, bool WIDE> struct Tail {
    uint2 kw[2][8];
    uint32_t vw[8][4];
    __device__ __forceinline__ void load(const DecodeKv8Params& p, size_t seq_head, int k0) {
        const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
        const TK* k = reinterpret_cast<const TK*>(p.c.ktail) + seq_head * kBlkBytes + 4 * c;
        const bf16* v = p.c.vtail + seq_head * kBlkBytes + 2 * r;
#pragma unroll
        for (int n = 0; n < 2; ++n)
#pragma unroll
            for (int i = 0; i < 8; ++i) kw[n][i] = *reinterpret_cast<const uint2*>(k + (k0 + 8 * n + r) * kD + 16 * i);
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                vw[i][x] = *reinterpret_cast<const uint32_t*>(v + (k0 + 2 * c + (x & 1) + 8 * (x >> 1)) * kD + 16 * i);
    }
    __device__ __forceinline__ void take(State& t, const uint32_t (&q)[8][2], float scale, int k0, int first, int last);
};

template <typename TK, bool WIDE>
__device__ __forceinline__ void Tail<TK, WIDE>::take(State& t, const uint32_t (&q)[8][2], float scale, int k0, int first, int last) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int key = k0 + 2 * c + (x & 1) + 8 * (x >> 1);
        // a masked row may hold anything: it must not reach the product
        if (key < first || key > last) {
#pragma unroll
            for (int i = 0; i < 8; ++i) vw[i][x] = 0u;
        }
    }
    float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        mma16816<KeyType<TK>::kBf>(d, kw[0][i].x, kw[1][i].x, kw[0][i].y, kw[1][i].y, q[i][0], q[i][1]);
    float2 s[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const int key = k0 + 8 * n + r;
        const bool on = key >= first && key <= last;
        s[n] = on ? make_float2(d[2 * n] * scale, d[2 * n + 1] * scale) : make_float2(-INFINITY, -INFINITY);
    }
    float2 a, b;
    soften(t, s, a, b);
    b = fmul2(b, make_float2(kInvP, kInvP));
    uint32_t part[3][2];   // first to third part of p; not WIDE: the second in the upper columns of the first
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        const uint32_t hi = pack_bf16(s[n].x, s[n].y);
        const float2 x = unpack_bf16(hi), left = make_float2(s[n].x - x.x, s[n].y - x.y);
        const uint32_t mid = pack_bf16(left.x, left.y);
        const float2 y = unpack_bf16(mid);
        const uint32_t lo = pack_bf16(left.x - y.x, left.y - y.y);
        part[0][n] = transpose8(WIDE || c < 2 ? hi : mid);
        part[1][n] = transpose8(WIDE ? mid : c < 2 ? lo : 0u);
        part[2][n] = WIDE ? transpose8(lo) : 0u;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float e[4];
        const uint32_t a0 = __byte_perm(vw[i][0], vw[i][1], 0x5410), a1 = __byte_perm(vw[i][0], vw[i][1], 0x7632);
        const uint32_t a2 = __byte_perm(vw[i][2], vw[i][3], 0x5410), a3 = __byte_perm(vw[i][2], vw[i][3], 0x7632);
        mma16816<true>(e, a0, a1, a2, a3, part[0][0], part[0][1], 0.f, 0.f, 0.f, 0.f);
        mma16816<true>(e, a0, a1, a2, a3, part[1][0], part[1][1]);
        if (WIDE) mma16816<true>(e, a0, a1, a2, a3, part[2][0], part[2][1]);
        join_o(t, i, e, a, b);
    }
}

// Where a warp's maximum and sum go, [column]; every lane of the warp calls it.
__device__ __forceinline__ void put_ml(const State& t, float (*ml)[2]) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    const float lx = column_sum(t.l.x), ly = column_sum(t.l.y);
    if (lane < 4) {
        *reinterpret_cast<float2*>(ml[2 * c]) = make_float2(t.m.x, lx);
        *reinterpret_cast<float2*>(ml[2 * c + 1]) = make_float2(t.m.y, ly);
    }
}

// The maximum and sum of four warps' parts of column h, and the factor of warp w's
__device__ __forceinline__ float join_ml(const float (*ml)[DK_HEADS][2], int h, int w, float& m, float& l) {
    float f = 0.f;
    m = -INFINITY;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = fmaxf(m, ml[i][h][0]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        // a part without keys counts nothing; one whose scores were all NaN has a NaN sum
        const float fi = ml[i][h][1] == 0.f ? 0.f : fast_exp2(ml[i][h][0] - m);
        l = fmaf(ml[i][h][1], fi, l);
        if (i == w) f = fi;
    }
    return f;
}

__device__ __forceinline__ uint2 load_gate(const DecodeKv8Params& p, size_t head, int d) {
    return p.g ? *reinterpret_cast<const uint2*>(p.g + head * kD + d) : make_uint2(0u, 0u);
}

// out and lse of four dims of one head from its maximum, sum and O
__device__ __forceinline__ void finish4(const DecodeKv8Params& p, size_t head, int d, float m, float l, const float (&o)[4],
                                        uint2 gate) {
    const float inv = 1.f / (l * kInvP);
    float x[4] = {o[0] * inv, o[1] * inv, o[2] * inv, o[3] * inv};
    if (p.g) {
        const float2 a = unpack_bf16(gate.x), b = unpack_bf16(gate.y);
        x[0] *= sigmoidf_(a.x);
        x[1] *= sigmoidf_(a.y);
        x[2] *= sigmoidf_(b.x);
        x[3] *= sigmoidf_(b.y);
    }
    *reinterpret_cast<uint2*>(p.out + head * kD + d) = make_uint2(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]));
    if (d == 0) p.lse[head] = (m + (log2f(l) - 14.f)) * kLn2;
}


// This lane's 32 elements of its column's q (zeros past the nh heads; head: the item's first): chunk i's pairs 16 i + 4 c, + 2
template <typename TK, bool WIDE>
__device__ __forceinline__ void load_q(const DecodeKv8Params& p, size_t head, int nh, uint32_t (&q)[8][2]) {
    const int c = threadIdx.x & 3, column = (threadIdx.x & 31) >> 2, h = WIDE ? column : column & 3;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint2 u = make_uint2(0u, 0u);
        if (h < nh) u = *reinterpret_cast<const uint2*>(static_cast<const TK*>(p.q) + (head + h) * kD + 16 * i + 4 * c);
        q[i][0] = u.x;
        q[i][1] = u.y;
    }
}

// q as the fp16 that meets codes, and the scales of the scores of this lane's two columns in base 2: fp16 as it is, bf16
// times the power of two that brings the head's largest element to 2^14
template <typename TK>
__device__ __forceinline__ float2 q_as_half(const DecodeKv8Params& p, const uint32_t (&q)[8][2], uint32_t (&h)[8][2]) {
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
    if (!KeyType<TK>::kBf) return make_float2(p.scale_log2, p.scale_log2);
    const float qs = p.scale_log2 / up;   // of column r; this lane needs those of 2 c and 2 c + 1
    const int c = threadIdx.x & 3;
    return make_float2(__shfl_sync(0xffffffffu, qs, 8 * c), __shfl_sync(0xffffffffu, qs, 8 * c + 4));
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

// ------------------------------------------------------------------ a warp's stream of half blocks
//
// Two warps share a block, 32 keys each, and every warp feeds itself: lane i of it looks up the warp's block 32 n + i
// (page, scales), 32 blocks ahead, and starts its copies when their turn comes, keys and values by turns into a ring
// of 3 x 4 KB.  While keys are worked on their values and the next keys are on their way.

constexpr int kHalfKeys = kBlk / 2;
constexpr uint32_t kSlot = kHalfKeys * kD;      // bytes
constexpr int kSlots = 3;

struct Block {       // as the lane that holds it knows it
    int j, row;      // block (-1: passed over); first of its rows in the codes (-1: no page)
    float ks, vs;
};

// Block number `i` of an item's 8-bit units
__device__ __forceinline__ Block block_of(const DecodeKv8Params& p, const Span& s, int b, int kvh, int i) {
    Block t{s.jlo + i, -1, 0.f, 0.f};
    int page = -1;
    if (p.blocks) {
        const int* list = p.blocks + ((size_t)b * p.c.Hkv + kvh) * p.n_list + i;
        const int before = i > 0 ? list[-1] : -1;
        t.j = *list;
        if (t.j >= 0) page = kv8_page(p.c, b, t.j);   // before s, which waits for the position, is asked
        if (t.j < s.jlo || t.j >= s.own || t.j <= before) t.j = -1;
    } else {
        page = kv8_page(p.c, b, t.j);
    }
    if (t.j >= 0) {
        t.ks = t.vs = NAN;          // a bad page reads as NaN
        if (page >= 0) {
            const int at = page * p.c.Hkv + kvh;
            t.row = at * kBlk;
            t.ks = p.c.ks[at];
            t.vs = p.c.vs[at];
        }
    }
    return t;
}

struct WarpSmem {
    uint64_t full[kSlots];
    uint64_t pad;
    Block block[4];        // of the warp's blocks n, n + 1, n + 2
};

struct Stream {
    const DecodeKv8Params& p;
    WarpSmem& sm;
    unsigned char* ring;       // this warp's kSlots slots
    volatile int* abort;
    Block mine;                // of this lane, in the current 32
    bool ok;

    __device__ __forceinline__ Stream(const DecodeKv8Params& p_, WarpSmem& sm_, unsigned char* ring_, volatile int* abort_)
        : p(p_), sm(sm_), ring(ring_), abort(abort_), mine{-1, -1, 0.f, 0.f}, ok(true) {}

    // copy number c of the warp (keys of block c / 2 if even, else its values): by the lane that holds the block
    __device__ __forceinline__ void copy(int c) {
        if ((int)(threadIdx.x & 31) == ((c >> 1) & 31)) {
            uint64_t* bar = &sm.full[c % kSlots];
            if (mine.row >= 0) {
                mbar_expect_tx(bar, kSlot);
                tma_load_2d(ring + (c % kSlots) * kSlot, (c & 1) ? &p.tm_v : &p.tm_k, bar, 0,
                            mine.row + ((threadIdx.x >> 5) & 1) * kHalfKeys);
            } else {
                mbar_arrive(bar);
            }
        }
    }
    __device__ __forceinline__ void note(int n) {   // block n's numbers for the warp
        if ((int)(threadIdx.x & 31) == (n & 31)) sm.block[n & 3] = mine;
    }
    // the first blocks are looked up: the first copies, then (they are still on their way) the scales
    __device__ __forceinline__ void start(int blocks) {
        if (blocks > 0) {
            copy(0);
            copy(1);
        }
        if (blocks > 1) copy(2);
        if (blocks > 0) note(0);
        if (blocks > 1) note(1);
        __syncwarp();
    }
    // the slot of copy c has been read: what is next in it may come
    __device__ __forceinline__ void reuse(int next, int copies) {
        fence_proxy_async_smem();
        __syncwarp();
        if (ok && next < copies) copy(next);
    }
    __device__ __forceinline__ bool wait(int c, int where) {
        if (ok) ok = mbar_wait(&sm.full[c % kSlots], (c / kSlots) & 1, abort, where);
        ok = __all_sync(0xffffffffu, ok);
        return ok;
    }
    // Block n of `blocks`; qs: the scales of this lane's two columns' scores.  fetch(i): looks the 32 blocks from 32 i up.
    template <int CODE, bool WIDE, typename Fetch>
    __device__ __forceinline__ void take(State& t, const uint32_t (&q)[8][2], float2 qs, int lo, int n, int blocks, int where,
                                         const Fetch& fetch) {
        const uint32_t base = smem_u32(ring);
        const bool here = wait(2 * n, where);
        const Block k = sm.block[n & 3];
        const bool on = here && k.j >= 0;
        float2 s[4];
        if (on)
            scores32<CODE>(s, q, fmul2(qs, make_float2(k.ks, k.ks)), base + (2 * n) % kSlots * kSlot,
                           lo - k.j * kBlk - ((threadIdx.x >> 5) & 1) * kHalfKeys);
        reuse(2 * n + 3, 2 * blocks);
        float2 a, b;
        uint32_t pb[WIDE ? 8 : 4];
        if (on) {
            soften(t, s, a, b);
            const bool upper = (threadIdx.x & 3) >= 2;   // columns 4 .. 7
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t hi = pack_half(s[i].x, s[i].y);
                const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&hi));
                const uint32_t lo_half = pack_half(s[i].x - x.x, s[i].y - x.y);
                pb[i] = transpose8(!WIDE && upper ? lo_half : hi);
                if constexpr (WIDE) pb[4 + i] = transpose8(lo_half);
            }
        }
        if (wait(2 * n + 1, where) && on)
            values32<CODE, WIDE>(t, pb, a, fmul2(b, make_float2(k.vs * kInvP, k.vs * kInvP)), base + (2 * n + 1) % kSlots * kSlot);
        if (n + 2 < blocks && ((n + 2) & 31) == 0) mine = fetch((n + 2) >> 5);
        reuse(2 * n + 4, 2 * blocks);
        if (n + 2 < blocks) note(n + 2);
        __syncwarp();
    }
    // After a wait that expired copies can be in flight: not past them.  `n`: the block the warp gave up at.
    __device__ __forceinline__ void drain(int n, int blocks) {
        if (!ok)
            for (int c = max(0, 2 * n - 2); c < min(2 * blocks, 2 * n + 5); ++c)
                mbar_wait_drain(&sm.full[c % kSlots], (c / kSlots) & 1);
    }
};

}  // namespace zgcm
