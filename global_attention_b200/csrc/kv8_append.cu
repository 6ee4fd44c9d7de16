// kv8_append.cu — tokens into the 8-bit block cache (zgcm_kv8_append of include/zgcm_kv8.h).
//
// A CTA takes one block of one KV head: 64 rows of keys and 64 of values, 16 KB each, read once
// into registers (thread = 4 rows x 8 elements of each), their largest magnitude, the scale,
// the codes and the mean of the keys.  Rows come from the new tokens, and for the first block
// of the call from the tail.  The tail is read and written by the same CTA (the one of the
// call's first block also takes the last), so that no other can overwrite rows it still needs.
//
// Bound by HBM for prompts (2 bytes read, 1 written per value) and by latency for single
// tokens, which move one row per head and, every 64th token, a block.
// Measured on a B200 in a graph's replays: prompts of up to 16K for 4 sequences (303 MB) 54.5 to 57.5 us on different cards, 5.6
// to 5.3 TB/s, 82 to 86% of the measured copy rate, with four CTAs an SM (64 registers); as eager calls on cold inputs 54 to
// 65 us; one token each for 64 sequences 4.8 us.
#include "kv8.cuh"
#include "sm100.cuh"

namespace zgcm {

int kv8_check(const zgcm_kv8_cache* c, Kv8* out) {
    if (!c) return ZGCM_ERR_INVALID_ARG;
    if (c->n_seq < 0 || c->n_blocks < 1 || c->n_pages < 1 || c->Hkv < 1 || c->D < 1) return ZGCM_ERR_INVALID_ARG;
    if (c->code_type != ZGCM_E4M3 && c->code_type != ZGCM_INT8) return ZGCM_ERR_INVALID_ARG;
    if (c->key_type != ZGCM_BF16 && c->key_type != ZGCM_FP16) return ZGCM_ERR_INVALID_ARG;
    if (c->D != kD) return ZGCM_ERR_UNSUPPORTED;
    // pages are addressed as rows of 128 bytes with 32-bit row numbers (256 GB), blocks of
    // sequences and heads by grid dimensions
    if ((long long)c->n_pages * c->Hkv * kBlk > 0x7fffffffLL) return ZGCM_ERR_UNSUPPORTED;
    if (c->n_blocks > (1 << 25) || c->n_seq > 65535 || c->Hkv > 65535) return ZGCM_ERR_UNSUPPORTED;
    if (c->n_seq > 0) {
        const void* ptrs[] = {c->k_codes, c->v_codes, c->k_scale, c->v_scale, c->k_mean, c->k_tail, c->v_tail, c->table};
        for (const void* p : ptrs)
            if (!p) return ZGCM_ERR_INVALID_ARG;
        for (const void* p : ptrs)
            if (reinterpret_cast<uintptr_t>(p) & 15u) return ZGCM_ERR_ALIGNMENT;
    }
    out->kc = static_cast<uint8_t*>(c->k_codes);
    out->vc = static_cast<uint8_t*>(c->v_codes);
    out->ks = c->k_scale;
    out->vs = c->v_scale;
    out->kmean = static_cast<char*>(c->k_mean);
    out->ktail = static_cast<char*>(c->k_tail);
    out->vtail = static_cast<bf16*>(c->v_tail);
    out->table = c->table;
    out->B = c->n_seq;
    out->NB = c->n_blocks;
    out->P = c->n_pages;
    out->Hkv = c->Hkv;
    out->code = c->code_type;
    out->key = c->key_type;
    return ZGCM_OK;
}

namespace {

constexpr int AP_THREADS = 256;
constexpr int AP_ROWS = kBlk / (AP_THREADS / 16);   // rows of a thread (16 threads per row, 8 elements each)

struct AppendParams {
    Kv8 c;
    const char* k;
    const char* v;
    long long kb, kt, kh, vb, vt, vh;   // element strides
    const int* pos;
    const int* count;
    int N;
};

template <typename T> __device__ __forceinline__ float2 unpack2(uint32_t u);
template <> __device__ __forceinline__ float2 unpack2<bf16>(uint32_t u) { return unpack_bf16(u); }
template <> __device__ __forceinline__ float2 unpack2<__half>(uint32_t u) {
    return __half22float2(*reinterpret_cast<const __half2*>(&u));
}

// Two quotients x / s, correctly rounded: r = 1 / s rounded to nearest; x r is off by less than two units in the last
// place, one step with the exact remainder x - q s brings it within one, and from there a second one gives the
// nearest (Markstein, IBM J. Res. Dev. 34, 1990), as long as nothing underflows: a block of smallest values is first
// multiplied by 2^100 (`up`, else 1), x and s alike.  (The division operator was half of the kernel's instructions.)
__device__ __forceinline__ float2 quotient(float2 x, float2 up, float2 minus_s, float2 r) {
    x = sm100::fmul2(x, up);
    float2 q = sm100::fmul2(x, r);
    q = sm100::ffma2(sm100::ffma2(minus_s, q, x), r, q);
    return sm100::ffma2(sm100::ffma2(minus_s, q, x), r, q);
}

// four codes of four quotients
template <int CODE> __device__ __forceinline__ uint32_t code4(float2 a, float2 b) {
    if (CODE == ZGCM_E4M3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    }
    // |x / scale| <= 127 (1 + 2^-22): in the last places of 1.5 2^23 it is rounded to nearest even, and its low byte is the code
    const float2 m = make_float2(12582912.f, 12582912.f);
    a = sm100::fadd2(a, m);
    b = sm100::fadd2(b, m);
    return __byte_perm(__byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040),
                       __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040), 0x5410);
}

// largest magnitude of a thread's values, as the bits of a 16-bit type without its sign: they order like the
// magnitudes, infinities and NaN above all finite ones
__device__ __forceinline__ uint32_t max_bits(const uint4 (&w)[AP_ROWS]) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < AP_ROWS; ++i) {
        m = __vmaxu2(m, w[i].x & 0x7fff7fffu);
        m = __vmaxu2(m, w[i].y & 0x7fff7fffu);
        m = __vmaxu2(m, w[i].z & 0x7fff7fffu);
        m = __vmaxu2(m, w[i].w & 0x7fff7fffu);
    }
    return max(m & 0xffffu, m >> 16);
}

template <typename T, int CODE>
__device__ __forceinline__ void store_codes(const uint4 (&w)[AP_ROWS], uint32_t bits, uint8_t* codes, float* scale_out) {
    const float amax = from_bits<T>(bits);
    const bool finite = isfinite(amax);
    const float scale = fmaxf(amax * (CODE == ZGCM_E4M3 ? 1.f / 448.f : 1.f / 127.f), 1.17549435e-38f);
    const float up = scale < 0x1p-80f ? 0x1p100f : 1.f, s = scale * up, r = __frcp_rn(s);
    const float2 u2 = make_float2(up, up), m2 = make_float2(-s, -s), r2 = make_float2(r, r);
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
#pragma unroll
    for (int i = 0; i < AP_ROWS; ++i) {
        const float2 a = quotient(unpack2<T>(w[i].x), u2, m2, r2), b = quotient(unpack2<T>(w[i].y), u2, m2, r2);
        const float2 c = quotient(unpack2<T>(w[i].z), u2, m2, r2), d = quotient(unpack2<T>(w[i].w), u2, m2, r2);
        uint2 y = make_uint2(code4<CODE>(a, b), code4<CODE>(c, d));
        if (!finite) y = make_uint2(0u, 0u);
        *reinterpret_cast<uint2*>(codes + (row + 16 * i) * kD + 8 * col) = y;
    }
    if (threadIdx.x == 0) *scale_out = finite ? scale : NAN;
}

// block j of KV head h of sequence b: positions [lo, hi) of it are new (lo >= start), earlier
// ones are in the tail
template <typename TK, int CODE>
__device__ __forceinline__ void do_block(const AppendParams& p, int b, int h, int j, int start, int end, int last,
                                         uint2* red, float (*sum)[kD]) {
    const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
    const int base = j * kBlk;
    const bool whole = end - base >= kBlk;
    const bool newest = j == last;
    const size_t tail = ((size_t)b * p.c.Hkv + h) * kBlkBytes;   // elements
    uint4 kw[AP_ROWS], vw[AP_ROWS];
#pragma unroll
    for (int i = 0; i < AP_ROWS; ++i) {
        const int r = row + 16 * i, t = base + r - start;   // t: number of the new token
        kw[i] = vw[i] = make_uint4(0u, 0u, 0u, 0u);
        if (t >= 0 && base + r < end) {
            kw[i] = *reinterpret_cast<const uint4*>(p.k + 2 * (b * p.kb + t * p.kt + h * p.kh + 8 * col));
            vw[i] = *reinterpret_cast<const uint4*>(p.v + 2 * (b * p.vb + t * p.vt + h * p.vh + 8 * col));
        } else if (t < 0 && whole) {
            kw[i] = *reinterpret_cast<const uint4*>(p.c.ktail + 2 * (tail + r * kD + 8 * col));
            vw[i] = *reinterpret_cast<const uint4*>(p.c.vtail + tail + r * kD + 8 * col);
        }
    }
    if (newest) {
#pragma unroll
        for (int i = 0; i < AP_ROWS; ++i) {
            const int r = row + 16 * i;
            if (base + r >= start && base + r < end) {
                *reinterpret_cast<uint4*>(p.c.ktail + 2 * (tail + r * kD + 8 * col)) = kw[i];
                *reinterpret_cast<uint4*>(p.c.vtail + tail + r * kD + 8 * col) = vw[i];
            }
        }
    }
    // the last block may be the one that pushes block last - NB out of the ring
    const int page = whole && j > last - p.c.NB ? kv8_page(p.c, b, j) : -1;
    if (page < 0) return;
    const size_t at = (size_t)page * p.c.Hkv + h;
    uint32_t mk = __reduce_max_sync(0xffffffffu, max_bits(kw)), mv = __reduce_max_sync(0xffffffffu, max_bits(vw));
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_uint2(mk, mv);
    float2 m[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < AP_ROWS; ++i) {
        const uint32_t u[4] = {kw[i].x, kw[i].y, kw[i].z, kw[i].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) m[e] = sm100::fadd2(m[e], unpack2<TK>(u[e]));
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) *reinterpret_cast<float2*>(&sum[row][8 * col + 2 * e]) = m[e];
    __syncthreads();
    const uint2 all = red[threadIdx.x & 7];
    mk = __reduce_max_sync(0xffffffffu, all.x);
    mv = __reduce_max_sync(0xffffffffu, all.y);
    store_codes<TK, CODE>(kw, mk, p.c.kc + at * kBlkBytes, p.c.ks + at);
    store_codes<bf16, CODE>(vw, mv, p.c.vc + at * kBlkBytes, p.c.vs + at);
    if (threadIdx.x < kD) {
        float a = 0.f;
#pragma unroll
        for (int i = 0; i < AP_THREADS / 16; ++i) a += sum[i][threadIdx.x];
        reinterpret_cast<TK*>(p.c.kmean)[at * kD + threadIdx.x] = TK(a * (1.0f / kBlk));
    }
}

// grid (blocks of the longest possible sequence, KV heads, sequences)
template <typename TK, int CODE>
__global__ void __launch_bounds__(AP_THREADS, 4) kv8_append_kernel(const __grid_constant__ AppendParams p) {
    __shared__ uint2 red[8];
    __shared__ __align__(16) float sum[AP_THREADS / 16][kD];
    const int b = blockIdx.z, h = blockIdx.y;
    const int start = p.pos[b];
    const int n = p.count ? max(0, min(p.N, p.count[b])) : p.N;
    if (start < 0 || n == 0 || start > 0x7fffffff - n) return;
    const int end = start + n, first = start / kBlk, last = (end - 1) / kBlk;
    const int j = first + (int)blockIdx.x;
    if (j > last || (j == last && j != first)) return;
#pragma unroll 1
    for (int at = j;; at = last) {
        do_block<TK, CODE>(p, b, h, at, start, end, last, red, sum);
        if (j != first || at == last) break;
        __syncthreads();   // the tail's old rows, red and sum have been read
    }
}

template <typename TK>
cudaError_t launch(const AppendParams& p, cudaStream_t stream) {
    const dim3 grid((p.N - 1) / kBlk + 2, p.c.Hkv, p.c.B);
    if (p.c.code == ZGCM_E4M3)
        kv8_append_kernel<TK, ZGCM_E4M3><<<grid, AP_THREADS, 0, stream>>>(p);
    else
        kv8_append_kernel<TK, ZGCM_INT8><<<grid, AP_THREADS, 0, stream>>>(p);
    return cudaGetLastError();
}

}  // namespace
}  // namespace zgcm

using namespace zgcm;

extern "C" int zgcm_kv8_append(const zgcm_kv8_cache* cache, const void* k, long long k_b_stride, long long k_t_stride,
                               long long k_h_stride, const void* v, long long v_b_stride, long long v_t_stride,
                               long long v_h_stride, const int* pos, const int* count, int N, void* cuda_stream) {
    AppendParams p;
    const int st = kv8_check(cache, &p.c);
    if (st != ZGCM_OK) return st;
    if (N < 0) return ZGCM_ERR_INVALID_ARG;
    if (p.c.B == 0 || N == 0) return ZGCM_OK;
    if (!k || !v || !pos) return ZGCM_ERR_INVALID_ARG;
    if (((uintptr_t)k | (uintptr_t)v | (uintptr_t)pos) & 15u) return ZGCM_ERR_ALIGNMENT;
    if ((uintptr_t)count & 15u) return ZGCM_ERR_ALIGNMENT;
    if ((k_b_stride | k_t_stride | k_h_stride | v_b_stride | v_t_stride | v_h_stride) & 7) return ZGCM_ERR_ALIGNMENT;
    p.k = static_cast<const char*>(k);
    p.v = static_cast<const char*>(v);
    p.kb = k_b_stride;
    p.kt = k_t_stride;
    p.kh = k_h_stride;
    p.vb = v_b_stride;
    p.vt = v_t_stride;
    p.vh = v_h_stride;
    p.pos = pos;
    p.count = count;
    p.N = N;
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = p.c.key == ZGCM_BF16 ? launch<bf16>(p, stream) : launch<__half>(p, stream);
    return e == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}
