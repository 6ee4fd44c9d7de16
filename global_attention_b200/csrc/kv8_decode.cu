// kv8_decode.cu — decode attention over the 8-bit block cache (zgcm_attn_decode_kv8 of
// include/zgcm_kv8.h): one token per sequence.
//
// Bound by reading the codes: a block of one KV head is 16 KB and serves the few query heads of
// its group.  What has to keep up with 43 bytes per SM and nanosecond is the conversion of the codes
// and the two products; on CUDA cores the products alone are 8 multiply-adds per byte for 4
// heads, more than an SM has.  So both run on the tensor cores as mma.sync m16n8k16 with
// the heads as the 16 rows (a tcgen05 tile would have 4 of its 128 rows filled, and its
// operands would have to go back to shared memory after their conversion):
//   S = Q K^T: A = q of up to 8 heads (rows 0-7, zeros below), B = 8 keys x 16 dims.
//   O = P V:   A = p in two 16-bit halves, rows 0-7 the rounded p, rows 8-15 what the rounding
//              left (so the idle rows carry p to 22 bits), B = 16 keys x 8 dims.
// Codes become fp16 exactly and their scales multiply the fp32 sums, once per block: the scores by
// ks, the block's O by vs where it joins the running O.  q as bf16 is first multiplied by a
// power of two that brings the row's largest element to 2^14 (exact but for elements 2^-28 of it).
//
// Work: the blocks of every (sequence, KV head, 8 heads) — an item — and its tail are laid end to end
// and cut into equal runs, one for each of 296 CTAs (two per SM), whatever the lengths; a CTA finds its
// run from the positions on the device, so a captured graph follows them.  One warp fetches page
// numbers and scales 32 blocks ahead and streams the codes by TMA (128-byte swizzle) into a ring of
// 6 x 16 KB; each of four warps takes every 4th block with its own running maximum, sum and O.  At an
// item's end the four are joined in a fixed order; an item that lies in one CTA is finished
// there, pieces of a cut one go to the workspace and kv8_join_kernel finishes them (started early, by
// programmatic dependent launch).  Results depend on positions and shapes alone.
#include <cudaTypedefs.h>
#include <math.h>

#include "kv8.cuh"
#include "sm100.cuh"
#include "tc_rows.cuh"

namespace zgcm {
int* library_error_word();  // zgcm_attn.cu: the site of an expired bounded wait

namespace {
using namespace sm100;

constexpr int DK_CTAS = 296;               // 148 SMs x 2
constexpr int DK_WARPS = 4;                // warps that compute; one more loads
constexpr int DK_THREADS = (DK_WARPS + 1) * 32;
constexpr int DK_STAGES = 6;
constexpr int DK_POS = 64;                 // positions of the run's sequences kept in shared memory
constexpr int DK_HEADS = 8;                // heads of an item
constexpr int DK_REC = kD + 4;             // floats of a record's head: m, l, 2 pad, O
constexpr float kInvP = 1.f / 16384.f;       // p is held times 2^14: as fp16 above its subnormals
constexpr int DK_WAIT_LOAD = 0x810, DK_WAIT_RING = 0x811;

struct DecodeKv8Params {
    CUtensorMap tm_k, tm_v;                // [n_pages * Hkv * 64, 128] bytes, box 64 rows
    Kv8 c;
    const void* q;
    const bf16* g;
    const int* pos;
    const int* blocks;
    int n_list, Hq, G, HT, W;              // HT: items of a KV head (8 heads each)
    int rows;                              // heads a record has room for: min(G, 8)
    float scale_log2;
    bf16* out;
    float* lse;
    float* part;                           // records [item + CTA][rows][DK_REC]
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

struct DecodeSmem {
    alignas(1024) unsigned char k[DK_STAGES][kBlkBytes];
    alignas(1024) unsigned char v[DK_STAGES][kBlkBytes];
    float acc[2][DK_HEADS][kD];
    float ml[DK_WARPS][DK_HEADS][2];
    Meta meta[DK_STAGES];
    uint64_t full[DK_STAGES], empty[DK_STAGES];
    int pos[DK_POS];
    long long lo, hi;
    int b0, rest0, off0;
    int abort;
};
static_assert(2 * (sizeof(DecodeSmem) + 1024 + 1024) <= 228 * 1024, "two CTAs per SM");

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
template <bool BF>
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
    if (BF)
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
    else
        asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                     : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                     : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// four codes -> two pairs of fp16 (bytes 0,1 and 2,3), exact
template <int CODE> __device__ __forceinline__ void halves4(uint32_t w, uint32_t& lo, uint32_t& hi) {
    if (CODE == ZGCM_E4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\t"
            "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        // a byte u = x + 128 under the exponent byte 0x64 is the fp16 1024 + u
        const uint32_t u = w ^ 0x80808080u;
        const uint32_t a = __byte_perm(u, 0x64646464u, 0x4140), b = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 off = __half2half2(__ushort_as_half(0x6480));   // 1152
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&a), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&b), off);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
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
__device__ __forceinline__ void warps_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

// ------------------------------------------------------------------ the walk over the units

struct Walk {
    int b, rest, off;   // sequence, item of it, unit of the item
};

struct Run {
    const DecodeKv8Params& p;
    const DecodeSmem& sm;
    __device__ __forceinline__ int pos(int b) const {
        const int i = b - sm.b0;
        return i < DK_POS ? sm.pos[i] : p.pos[b];
    }
    // n units on; stays at the end when it runs past it
    __device__ __forceinline__ void step(Walk& w, int n) const {
        w.off += n;
        const int items = p.c.Hkv * p.HT;
        while (w.b < p.c.B) {
            const int u = span_of(p, pos(w.b)).units;
            if (w.off < u) return;
            const int skip = min(w.off / u, items - w.rest);
            w.off -= skip * u;
            w.rest += skip;
            if (w.rest < items) return;
            w.rest = 0;
            ++w.b;
        }
    }
};

// units before sequence b, and in all, by one warp: *total, and the sequence that holds unit x
__device__ __forceinline__ long long count_units(const DecodeKv8Params& p, int upto) {
    long long n = 0;
    for (int b = threadIdx.x & 31; b < upto; b += 32) n += span_of(p, p.pos[b]).units;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) n += __shfl_xor_sync(0xffffffffu, n, o);
    return n * (p.c.Hkv * p.HT);
}

// Runs: as many as there are CTAs, or units when those are fewer (no run between two others is empty: an
// item's records are those of all CTAs from its first to its last).
__device__ __forceinline__ int run_count(long long total) { return (int)min(total, (long long)DK_CTAS); }
__device__ __forceinline__ long long run_start(long long total, int cta) {
    const int n = run_count(total);
    return total * min(cta, n) / n;
}
// the CTA whose run holds unit x: the last whose start is not above it
__device__ __forceinline__ int run_of(long long total, long long x) {
    return (int)(((x + 1) * run_count(total) - 1) / total);
}

// ------------------------------------------------------------------ loading warp

__device__ __forceinline__ void load_run(const DecodeKv8Params& p, DecodeSmem& sm, const Run& run, long long lo, long long hi) {
    const int lane = threadIdx.x & 31;
    Walk at{sm.b0, sm.rest0, sm.off0};
    int slot = 0;
    bool ok = true;
    for (long long x = lo; x < hi && ok; x += 32) {
        Walk w = at;
        run.step(w, lane);
        int page = -1, j = -1, kvh = 0;
        bool is8 = false;
        float ks = 0.f, vs = 0.f;
        if (x + lane < hi) {
            const Span s = span_of(p, run.pos(w.b));
            is8 = w.off < s.units - 1;
            if (is8) {
                kvh = w.rest / p.HT;
                if (p.blocks) {
                    const int* list = p.blocks + ((size_t)w.b * p.c.Hkv + kvh) * p.n_list + w.off;
                    j = *list;
                    if (j < s.jlo || j >= s.own || (w.off > 0 && j <= list[-1])) j = -1;
                } else {
                    j = s.jlo + w.off;
                }
                if (j >= 0) {
                    page = kv8_page(p.c, w.b, j);
                    ks = vs = NAN;          // a bad page reads as NaN
                    if (page >= 0) {
                        ks = p.c.ks[(size_t)page * p.c.Hkv + kvh];
                        vs = p.c.vs[(size_t)page * p.c.Hkv + kvh];
                    }
                }
            }
        }
        const uint32_t all = __ballot_sync(0xffffffffu, is8);
        for (uint32_t left = all; left; left &= left - 1, ++slot) {
            const int st = slot % DK_STAGES;
            if (lane == __ffs(left) - 1) {
                if (slot >= DK_STAGES && !mbar_wait(&sm.empty[st], (slot / DK_STAGES - 1) & 1, &sm.abort, DK_WAIT_RING))
                    ok = false;
                if (ok) {
                    sm.meta[st] = Meta{ks, vs, j, 0};
                    if (page >= 0) {
                        const int row = (page * p.c.Hkv + kvh) * kBlk;
                        mbar_expect_tx(&sm.full[st], 2 * kBlkBytes);
                        tma_load_2d(sm.k[st], &p.tm_k, &sm.full[st], 0, row);
                        tma_load_2d(sm.v[st], &p.tm_v, &sm.full[st], 0, row);
                    } else {
                        mbar_arrive(&sm.full[st]);
                    }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
        }
        run.step(at, 32);
    }
    // copies in flight (after a wait that expired there can be some): not before they have landed
    if (lane == 0)
        for (int s = max(0, slot - DK_STAGES); s < slot; ++s) mbar_wait_drain(&sm.full[s % DK_STAGES], (s / DK_STAGES) & 1);
}

// ------------------------------------------------------------------ computing warps

// A warp's share of an item.  Lane (r, c) = (lane / 4, lane % 4) holds head r: of O the dims 16 i + 4 c .. + 3
// for i = 0 .. 7.
struct State {
    float m, l;      // running maximum (base 2), this lane's part of the sum (times 2^14)
    float o[8][4];
};

// Scores of a set of keys in base 2 -> p relative to the set's own maximum (times 2^14: as fp16 down to 2^-38 of
// it, whatever the sets before had), the running maximum and sum.  a: factor for O so far; b: for this set's.
template <int N> __device__ __forceinline__ void soften(State& t, float (&s)[N], float& a, float& b) {
    float mt = s[0];
#pragma unroll
    for (int i = 1; i < N; ++i) mt = fmaxf(mt, s[i]);
    mt = fmaxf(quad_max(mt), -3e38f);     // scores of -infinity alone have p = 0, not NaN
    const float m = fmaxf(t.m, mt);
    a = fast_exp2(t.m - m);               // 0 from the empty start
    b = fast_exp2(mt - m);
    const float base = mt - 14.f;
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s[i] = fast_exp2(s[i] - base);
        sum += s[i];
    }
    t.l = fmaf(t.l, a, sum * b);
    t.m = m;
}

template <int CODE>
__device__ __forceinline__ void block8(State& t, const uint32_t (&q)[8][2], float qscale, uint32_t k_addr, uint32_t v_addr,
                                       const Meta& meta, int lo) {
    const int lane = threadIdx.x & 31, c = lane & 3;
    const int mi = lane >> 3, r = lane & 7;            // ldmatrix: this lane's row r of matrix mi
    float s[16];
    // S: 8 keys at a time; matrices are the 16-byte chunks of the keys' rows
#pragma unroll
    for (int n = 0; n < 8; ++n) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
        const uint32_t row = k_addr + (n * 8 + r) * kD;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t w[4];
            ldsm4(row + (((4 * half + mi) ^ r) << 4), w);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                uint32_t b0, b1;
                halves4<CODE>(w[i], b0, b1);
                mma16816<false>(d, q[4 * half + i][0], 0u, q[4 * half + i][1], 0u, b0, b1);
            }
        }
        s[2 * n] = d[0];
        s[2 * n + 1] = d[1];
    }
    const float f = meta.ks * qscale;
#pragma unroll
    for (int i = 0; i < 16; ++i) s[i] *= f;
    if (meta.j * kBlk < lo) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            if (meta.j * kBlk + (i >> 1) * 8 + 2 * c + (i & 1) < lo) s[i] = -INFINITY;
    }
    float a, b;
    soften(t, s, a, b);
    uint32_t hi[8], lo2[8];
#pragma unroll
    for (int n = 0; n < 8; ++n) split2<false>(s[2 * n], s[2 * n + 1], hi[n], lo2[n]);
    // O: 16 dims at a time (their 16-byte chunk); matrices are groups of 8 keys, transposed: a lane gets keys
    // 2c, 2c+1 of the dims 2r, 2r+1 of the chunk
    const float vs = meta.vs * (b * kInvP);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float e[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int half = 0; half < 2; ++half) {
            uint32_t w[4], be[4], bo[4];
            ldsm4t(v_addr + (32 * half + 8 * mi + r) * kD + ((i ^ r) << 4), w);
#pragma unroll
            for (int x = 0; x < 4; ++x) halves4<CODE>(__byte_perm(w[x], 0, 0x3120), be[x], bo[x]);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
                const int n = 4 * half + 2 * kk;
                mma16816<false>(e, hi[n], lo2[n], hi[n + 1], lo2[n + 1], be[2 * kk], be[2 * kk + 1]);
                mma16816<false>(o, hi[n], lo2[n], hi[n + 1], lo2[n + 1], bo[2 * kk], bo[2 * kk + 1]);
            }
        }
        t.o[i][0] = fmaf(e[0] + e[2], vs, t.o[i][0] * a);
        t.o[i][1] = fmaf(o[0] + o[2], vs, t.o[i][1] * a);
        t.o[i][2] = fmaf(e[1] + e[3], vs, t.o[i][2] * a);
        t.o[i][3] = fmaf(o[1] + o[3], vs, t.o[i][3] * a);
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
    float s[4];
#pragma unroll
    for (int n = 0; n < 2; ++n) {
        float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 8; ++i) mma16816<KeyType<TK>::kBf>(d, q[i][0], 0u, q[i][1], 0u, kw[n][i].x, kw[n][i].y);
        s[2 * n] = on[2 * n] ? d[0] * scale : -INFINITY;
        s[2 * n + 1] = on[2 * n + 1] ? d[1] * scale : -INFINITY;
    }
    float a, b;
    soften(t, s, a, b);
    b *= kInvP;
    uint32_t hi[2], lo[2];
#pragma unroll
    for (int n = 0; n < 2; ++n) split2<true>(s[2 * n], s[2 * n + 1], hi[n], lo[n]);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float e[4] = {0.f, 0.f, 0.f, 0.f}, o[4] = {0.f, 0.f, 0.f, 0.f};
        mma16816<true>(e, hi[0], lo[0], hi[1], lo[1], __byte_perm(vw[i][0], vw[i][1], 0x5410),
                       __byte_perm(vw[i][2], vw[i][3], 0x5410));
        mma16816<true>(o, hi[0], lo[0], hi[1], lo[1], __byte_perm(vw[i][0], vw[i][1], 0x7632),
                       __byte_perm(vw[i][2], vw[i][3], 0x7632));
        t.o[i][0] = fmaf(e[0] + e[2], b, t.o[i][0] * a);
        t.o[i][1] = fmaf(o[0] + o[2], b, t.o[i][1] * a);
        t.o[i][2] = fmaf(e[1] + e[3], b, t.o[i][2] * a);
        t.o[i][3] = fmaf(o[1] + o[3], b, t.o[i][3] * a);
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

template <typename TK, int CODE>
__device__ __forceinline__ void compute_run(const DecodeKv8Params& p, DecodeSmem& sm, const Run& run, long long lo,
                                            long long hi) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = lane >> 2, c = lane & 3;
    Walk w{sm.b0, sm.rest0, sm.off0};
    int slot = 0;   // 8-bit units of the run so far: the ring's slots, slot s for warp s % 4
    for (long long x = lo; x < hi;) {
        const Span s = span_of(p, run.pos(w.b));
        const int n = (int)min((long long)(s.units - w.off), hi - x);          // units of the item here
        const int n8 = max(0, min(w.off + n, s.units - 1) - w.off);
        const bool has_tail = w.off + n == s.units;
        const int kvh = w.rest / p.HT, ht = w.rest % p.HT;
        const int nh = min(DK_HEADS, p.G - ht * DK_HEADS);
        const size_t head = (size_t)w.b * p.Hq + (size_t)kvh * p.G + ht * DK_HEADS + r;   // this lane's head (r < nh)
        const bool one = w.off == 0 && has_tail;                               // the whole item
        State t;
        t.m = -INFINITY;
        t.l = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) t.o[i][0] = t.o[i][1] = t.o[i][2] = t.o[i][3] = 0.f;
        if (s.idle || s.bad) {
            if (warp == 0 && r < nh) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const uint32_t u = s.idle ? 0u : 0x7fff7fffu;
                    *reinterpret_cast<uint2*>(p.out + head * kD + 16 * i + 4 * c) = make_uint2(u, u);
                }
                if (c == 0) p.lse[head] = s.idle ? -INFINITY : NAN;
            }
        } else {
            uint32_t q16[8][2];
            float qs = p.scale_log2;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                uint2 u = make_uint2(0u, 0u);
                if (r < nh) u = *reinterpret_cast<const uint2*>(static_cast<const TK*>(p.q) + head * kD + 16 * i + 4 * c);
                q16[i][0] = u.x;
                q16[i][1] = u.y;
            }
            uint32_t qt[8][2];   // as they are, for the tail
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                qt[i][0] = q16[i][0];
                qt[i][1] = q16[i][1];
            }
            if (KeyType<TK>::kBf) {
                float mx = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 a = unpack_bf16(q16[i][0]), b = unpack_bf16(q16[i][1]);
                    mx = fmaxf(mx, fmaxf(fmaxf(fabsf(a.x), fabsf(a.y)), fmaxf(fabsf(b.x), fabsf(b.y))));
                }
                mx = quad_max(mx);
                const int ex = min(254, 268 - (int)(__float_as_uint(mx) >> 23));
                const float up = __uint_as_float((uint32_t)ex << 23);   // 2^14 / 2^floor(log2 mx)
                qs = p.scale_log2 / up;
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float2 a = unpack_bf16(q16[i][0]), b = unpack_bf16(q16[i][1]);
                    q16[i][0] = pack_half(a.x * up, a.y * up);
                    q16[i][1] = pack_half(b.x * up, b.y * up);
                }
            }
            for (int i = (warp - slot) & 3; i < n8; i += DK_WARPS) {
                const int sl = slot + i, st = sl % DK_STAGES;
                if (mbar_wait(&sm.full[st], (sl / DK_STAGES) & 1, &sm.abort, DK_WAIT_LOAD)) {
                    const Meta meta = sm.meta[st];
                    if (meta.j >= 0)
                        block8<CODE>(t, q16, qs, smem_u32(sm.k[st]), smem_u32(sm.v[st]), meta, s.lo);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sm.empty[st]);
            }
            if (has_tail) {
                const int last = run.pos(w.b) - s.own * kBlk, first = s.lo - s.own * kBlk;
                if (warp * 16 <= last && warp * 16 + 15 >= first) {
                    const size_t at = ((size_t)w.b * p.c.Hkv + kvh) * kBlkBytes;
                    tail16<TK>(t, qt, p.scale_log2, reinterpret_cast<const TK*>(p.c.ktail) + at, p.c.vtail + at, warp * 16,
                               first, last);
                }
            }
            // the four warps' parts into warp 0's, always in the same order
            t.l += __shfl_xor_sync(0xffffffffu, t.l, 1);
            t.l += __shfl_xor_sync(0xffffffffu, t.l, 2);
            if (c == 0) {
                sm.ml[warp][r][0] = t.m;
                sm.ml[warp][r][1] = t.l;
            }
            warps_sync();
            float m = -INFINITY, l = 0.f, f = 0.f;
#pragma unroll
            for (int i = 0; i < DK_WARPS; ++i) m = fmaxf(m, sm.ml[i][r][0]);
#pragma unroll
            for (int i = 0; i < DK_WARPS; ++i) {
                // a part without keys counts nothing; one whose scores were all NaN has a NaN sum
                const float fi = sm.ml[i][r][1] == 0.f ? 0.f : fast_exp2(sm.ml[i][r][0] - m);
                l = fmaf(sm.ml[i][r][1], fi, l);
                if (i == warp) f = fi;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) t.o[i][e] *= f;
            if (warp >= 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4*>(&sm.acc[warp - 2][r][16 * i + 4 * c]) =
                        make_float4(t.o[i][0], t.o[i][1], t.o[i][2], t.o[i][3]);
            }
            warps_sync();
            if (warp < 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float4* a = reinterpret_cast<float4*>(&sm.acc[warp][r][16 * i + 4 * c]);
                    const float4 y = *a;
                    t.o[i][0] += y.x;
                    t.o[i][1] += y.y;
                    t.o[i][2] += y.z;
                    t.o[i][3] += y.w;
                    if (warp == 1) *a = make_float4(t.o[i][0], t.o[i][1], t.o[i][2], t.o[i][3]);
                }
            }
            warps_sync();
            if (warp == 0 && r < nh) {
                const size_t item = ((size_t)w.b * p.c.Hkv + kvh) * p.HT + ht;
                float* rec = p.part + ((item + blockIdx.x) * p.rows + r) * DK_REC;
                if (!one && c == 0) *reinterpret_cast<float2*>(rec) = make_float2(m, l);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float4 y = *reinterpret_cast<const float4*>(&sm.acc[1][r][16 * i + 4 * c]);
                    const float o[4] = {t.o[i][0] + y.x, t.o[i][1] + y.y, t.o[i][2] + y.z, t.o[i][3] + y.w};
                    if (one)
                        finish4(p, head, 16 * i + 4 * c, m, l, o);
                    else
                        *reinterpret_cast<float4*>(rec + 4 + 16 * i + 4 * c) = make_float4(o[0], o[1], o[2], o[3]);
                }
            }
        }
        slot += n8;
        x += n;
        run.step(w, n);
    }
}

template <typename TK, int CODE>
__global__ void __launch_bounds__(DK_THREADS, 2) kv8_decode_kernel(const __grid_constant__ DecodeKv8Params p) {
    extern __shared__ unsigned char raw[];
    DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may take its place early
    if (warp == DK_WARPS) {
        if (lane == 0) {
            for (int i = 0; i < DK_STAGES; ++i) {
                mbar_init(&sm.full[i], 1);
                mbar_init(&sm.empty[i], 1);
            }
            sm.abort = 0;
            fence_barrier_init();
            prefetch_tmap(&p.tm_k);
            prefetch_tmap(&p.tm_v);
        }
    } else if (warp == 0) {
        const int items = p.c.Hkv * p.HT;
        const long long total = count_units(p, p.c.B);
        const long long lo = run_start(total, blockIdx.x), hi = run_start(total, blockIdx.x + 1);
        // the sequence that holds unit lo, 32 sequences at a time
        long long before = 0;
        int b0 = 0;
        for (int b = 0; b < p.c.B; b += 32) {
            const long long u = b + lane < p.c.B ? (long long)span_of(p, p.pos[b + lane]).units * items : 0;
            long long s = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const long long y = __shfl_up_sync(0xffffffffu, s, o);
                if (lane >= o) s += y;
            }
            const uint32_t in = __ballot_sync(0xffffffffu, before + s > lo);
            if (in) {
                const int f = __ffs(in) - 1;
                b0 = b + f;
                before += __shfl_sync(0xffffffffu, s - u, f);
                break;
            }
            before += __shfl_sync(0xffffffffu, s, 31);
        }
        if (lane == 0) {
            const int u = span_of(p, p.pos[b0]).units;
            const long long in = lo - before;
            sm.lo = lo;
            sm.hi = hi;
            sm.b0 = b0;
            sm.rest0 = (int)(in / u);
            sm.off0 = (int)(in % u);
        }
        for (int i = lane; i < DK_POS; i += 32)
            if (b0 + i < p.c.B) sm.pos[i] = p.pos[b0 + i];
    }
    __syncthreads();
    const Run run{p, sm};
    const long long lo = sm.lo, hi = sm.hi;
    if (warp == DK_WARPS)
        load_run(p, sm, run, lo, hi);
    else
        compute_run<TK, CODE>(p, sm, run, lo, hi);
    __syncthreads();
    if (tid == 0 && sm.abort) *p.err = sm.abort;
}

// Items that more than one CTA worked on: a block per (item, head), a warp every 4th record.
__global__ void __launch_bounds__(128) kv8_join_kernel(const __grid_constant__ DecodeKv8Params p) {
    __shared__ float ml[4][2];
    __shared__ float acc[3][kD];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int item = blockIdx.x / p.rows, row = blockIdx.x % p.rows;
    const int items = p.c.Hkv * p.HT, b = item / items, rest = item % items, kvh = rest / p.HT, ht = rest % p.HT;
    const int units = span_of(p, p.pos[b]).units;
    const long long total = count_units(p, p.c.B), start = count_units(p, b) + (long long)rest * units;
    const int c0 = run_of(total, start), c1 = run_of(total, start + units - 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // every block: the grid must not end before the records' writer
    if (c0 == c1 || ht * DK_HEADS + row >= p.G) return;
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
    for (int c = c0 + warp; c <= c1; c += 4) {
        const float* rec = p.part + (((size_t)item + c) * p.rows + row) * DK_REC;
        const float2 x = *reinterpret_cast<const float2*>(rec);
        const float4 y = *reinterpret_cast<const float4*>(rec + 4 + 4 * lane);
        if (x.y == 0.f) continue;   // no key
        const float mn = fmaxf(m, x.x), a = l == 0.f ? 0.f : fast_exp2(m - mn), f = fast_exp2(x.x - mn);
        l = l * a + x.y * f;
        o[0] = o[0] * a + y.x * f;
        o[1] = o[1] * a + y.y * f;
        o[2] = o[2] * a + y.z * f;
        o[3] = o[3] * a + y.w * f;
        m = mn;
    }
    if (lane == 0) {
        ml[warp][0] = m;
        ml[warp][1] = l;
    }
    if (warp > 0) *reinterpret_cast<float4*>(&acc[warp - 1][4 * lane]) = make_float4(o[0], o[1], o[2], o[3]);
    __syncthreads();
    if (warp > 0) return;
    float mm = m;
    for (int i = 1; i < 4; ++i) mm = fmaxf(mm, ml[i][0]);
    const float f0 = l == 0.f ? 0.f : fast_exp2(m - mm);
    l *= f0;
    for (int e = 0; e < 4; ++e) o[e] *= f0;
    for (int i = 1; i < 4; ++i) {
        const float f = ml[i][1] == 0.f ? 0.f : fast_exp2(ml[i][0] - mm);
        const float4 y = *reinterpret_cast<const float4*>(&acc[i - 1][4 * lane]);
        l = fmaf(ml[i][1], f, l);
        o[0] = fmaf(y.x, f, o[0]);
        o[1] = fmaf(y.y, f, o[1]);
        o[2] = fmaf(y.z, f, o[2]);
        o[3] = fmaf(y.w, f, o[3]);
    }
    finish4(p, (size_t)b * p.Hq + (size_t)kvh * p.G + ht * DK_HEADS + row, 4 * lane, mm, l, o);
}

bool make_map(CUtensorMap* map, const void* codes, const Kv8& c) {
    static const PFN_cuTensorMapEncodeTiled_v12000 enc = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        return cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) == cudaSuccess &&
                       q == cudaDriverEntryPointSuccess
                   ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr)
                   : nullptr;
    }();
    if (!enc) return false;
    cuuint64_t dims[2] = {kD, (cuuint64_t)c.P * c.Hkv * kBlk};
    cuuint64_t strides[1] = {kD};
    cuuint32_t box[2] = {kD, kBlk}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TK, int CODE> cudaError_t launch(const DecodeKv8Params& p, cudaStream_t stream) {
    const size_t smem = sizeof(DecodeSmem) + 1024;
    cudaError_t e = cudaFuncSetAttribute(kv8_decode_kernel<TK, CODE>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kv8_decode_kernel<TK, CODE><<<DK_CTAS, DK_THREADS, smem, stream>>>(p);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.c.B * p.c.Hkv * p.HT * p.rows));
    cfg.blockDim = dim3(128);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_join_kernel, p);
}

}  // namespace
}  // namespace zgcm

using namespace zgcm;

extern "C" {

size_t zgcm_attn_decode_kv8_workspace_size(int n_seq, int Hq, int Hkv) {
    if (n_seq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
    const int G = Hq / Hkv, HT = (G + DK_HEADS - 1) / DK_HEADS, rows = G < DK_HEADS ? G : DK_HEADS;
    return ((size_t)n_seq * Hkv * HT + DK_CTAS) * rows * DK_REC * sizeof(float);
}

int zgcm_attn_decode_kv8(const zgcm_kv8_cache* cache, const void* q, const void* g, const int* pos, const int* blocks,
                         int n_list, int Hq, int window, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* cuda_stream) {
    DecodeKv8Params p;
    const int st = kv8_check(cache, &p.c);
    if (st != ZGCM_OK) return st;
    if (Hq < 1 || Hq % p.c.Hkv != 0 || window < 1 || (blocks && n_list < 0)) return ZGCM_ERR_INVALID_ARG;
    if (!(scale > 0.f) || !isfinite(scale)) return ZGCM_ERR_INVALID_ARG;
    if (p.c.B == 0) return ZGCM_OK;
    if (!q || !pos || !out || !lse) return ZGCM_ERR_INVALID_ARG;
    if (((uintptr_t)q | (uintptr_t)g | (uintptr_t)pos | (uintptr_t)blocks | (uintptr_t)out | (uintptr_t)lse) & 15u)
        return ZGCM_ERR_ALIGNMENT;
    if (!workspace || workspace_bytes < zgcm_attn_decode_kv8_workspace_size(p.c.B, Hq, p.c.Hkv)) return ZGCM_ERR_WORKSPACE;
    if ((uintptr_t)workspace & 15u) return ZGCM_ERR_ALIGNMENT;
    p.q = q;
    p.g = static_cast<const bf16*>(g);
    p.pos = pos;
    p.blocks = blocks;
    p.n_list = blocks ? n_list : 0;
    p.Hq = Hq;
    p.G = Hq / p.c.Hkv;
    p.HT = (p.G + DK_HEADS - 1) / DK_HEADS;
    p.rows = p.G < DK_HEADS ? p.G : DK_HEADS;
    p.W = window;
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<bf16*>(out);
    p.lse = lse;
    p.part = static_cast<float*>(workspace);
    p.err = library_error_word();
    // items are counted in 32 bits (grids and records)
    if (!p.err || (long long)p.c.B * p.c.Hkv * p.HT * p.rows > 0x7fffffffLL) return ZGCM_ERR_UNSUPPORTED;
    if (!make_map(&p.tm_k, p.c.kc, p.c) || !make_map(&p.tm_v, p.c.vc, p.c)) return ZGCM_ERR_CUDA;
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const bool f8 = p.c.code == ZGCM_E4M3;
    const cudaError_t e = p.c.key == ZGCM_BF16
                              ? (f8 ? launch<bf16, ZGCM_E4M3>(p, stream) : launch<bf16, ZGCM_INT8>(p, stream))
                              : (f8 ? launch<__half, ZGCM_E4M3>(p, stream) : launch<__half, ZGCM_INT8>(p, stream));
    return e == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}

}  // extern "C"
