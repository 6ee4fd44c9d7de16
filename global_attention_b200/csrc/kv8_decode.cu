// kv8_decode.cu — decode attention over the 8-bit block cache (zgcm_attn_decode_kv8 of
// include/zgcm_kv8.h): one token per sequence.
//
// A CTA takes one (sequence, query head) and a run of blocks, a warp every 4th key, a lane 4
// dims; online softmax; a second kernel joins the runs.
#include <math.h>

#include "kv8.cuh"

namespace zgcm {
namespace {

constexpr int DK_REC = kD + 4;
constexpr int DK_MAX_RUNS = 32;

struct DecodeKv8Params {
    Kv8 c;
    const void* q;
    const bf16* g;
    const int* pos;
    const int* blocks;
    int n_list, Hq, W, nrun, len;   // len: blocks of a run
    float scale_log2;
    bf16* out;
    float* lse;
    float* part;
};

template <typename TK, int CODE>
__global__ void __launch_bounds__(128) kv8_decode_kernel(const __grid_constant__ DecodeKv8Params p) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int b = blockIdx.x / p.Hq, h = blockIdx.x % p.Hq, kvh = h / (p.Hq / p.c.Hkv), run = blockIdx.y;
    const int pos = p.pos[b];
    const int own = pos < 0 ? -1 : pos / kBlk, lo = max(0, pos - p.W + 1), jlo = lo / kBlk;
    const bool bad = pos >= 0 && own - jlo >= p.c.NB;
    const TK* qp = static_cast<const TK*>(p.q) + (size_t)blockIdx.x * kD + 4 * lane;
    float q[4], o[4] = {};
    for (int e = 0; e < 4; ++e) q[e] = key_to_float(qp[e]) * p.scale_log2;
    float m = bad ? NAN : -INFINITY, l = bad ? NAN : 0.f;
    const int n = pos < 0 || bad ? 0 : (p.blocks ? p.n_list : own - jlo) + 1;   // the last one is the tail
    const int i1 = min(n, (run + 1) * p.len);
    for (int i = run * p.len; i < i1; ++i) {
        const bool tail = i == n - 1;
        int j = tail ? own : jlo + i;
        if (p.blocks && !tail) {
            const int* list = p.blocks + ((size_t)b * p.c.Hkv + kvh) * p.n_list;
            j = list[i];
            if (j < 0 || j >= own || j < jlo || (i > 0 && j <= list[i - 1])) continue;
        }
        int page = 0;
        float ks = 1.f, vs = 1.f;
        if (!tail) {
            page = kv8_page(p.c, b, j);
            if (page < 0) {
                m = l = NAN;
                break;
            }
            ks = p.c.ks[(size_t)page * p.c.Hkv + kvh];
            vs = p.c.vs[(size_t)page * p.c.Hkv + kvh];
        }
        for (int r = warp; r < kBlk; r += 4) {
            const int t = j * kBlk + r;
            if (t < lo || t > pos) continue;
            float k[4], v[4];
            if (tail) {
                const size_t at = (((size_t)b * p.c.Hkv + kvh) * kBlk + r) * kD + 4 * lane;
                for (int e = 0; e < 4; ++e) {
                    k[e] = key_to_float(reinterpret_cast<const TK*>(p.c.ktail)[at + e]);
                    v[e] = bf2f(p.c.vtail[at + e]);
                }
            } else {
                const size_t at = (((size_t)page * p.c.Hkv + kvh) * kBlk + r) * kD + 4 * lane;
                for (int e = 0; e < 4; ++e) {
                    if (CODE == ZGCM_E4M3) {
                        k[e] = float(reinterpret_cast<const __nv_fp8_e4m3*>(p.c.kc)[at + e]) * ks;
                        v[e] = float(reinterpret_cast<const __nv_fp8_e4m3*>(p.c.vc)[at + e]) * vs;
                    } else {
                        k[e] = float(reinterpret_cast<const signed char*>(p.c.kc)[at + e]) * ks;
                        v[e] = float(reinterpret_cast<const signed char*>(p.c.vc)[at + e]) * vs;
                    }
                }
            }
            const float s = warp_sum(q[0] * k[0] + q[1] * k[1] + q[2] * k[2] + q[3] * k[3]);
            const float mn = fmaxf(m, s), a = exp2f(m - mn), pr = exp2f(s - mn);
            l = l * a + pr;
            for (int e = 0; e < 4; ++e) o[e] = o[e] * a + pr * v[e];
            m = mn;
        }
    }
    float* rec = p.part + (((size_t)blockIdx.x * p.nrun + run) * 4 + warp) * DK_REC;
    if (lane == 0) {
        rec[0] = m;
        rec[1] = l;
    }
    for (int e = 0; e < 4; ++e) rec[4 + 4 * lane + e] = o[e];
}

__global__ void __launch_bounds__(kD) kv8_join_kernel(const __grid_constant__ DecodeKv8Params p) {
    const int d = threadIdx.x, bh = blockIdx.x;
    const bool idle = p.pos[bh / p.Hq] < 0;
    const float* part = p.part + (size_t)bh * p.nrun * 4 * DK_REC;
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int s = 0; s < p.nrun * 4; ++s) m = fmaxf(m, part[s * DK_REC]);
    for (int s = 0; s < p.nrun * 4; ++s) {
        const float* r = part + s * DK_REC;
        if (r[1] == 0.f) continue;   // no key (a run of NaN scores keeps its NaN sum)
        const float a = exp2f(r[0] - m);
        l += r[1] * a;
        o += r[4 + d] * a;
    }
    float x = o / l;
    if (p.g) x *= sigmoidf_(bf2f(p.g[(size_t)bh * kD + d]));
    p.out[(size_t)bh * kD + d] = __float2bfloat16_rn(idle ? 0.f : x);
    if (d == 0) p.lse[bh] = idle ? -INFINITY : (m + log2f(l)) * kLn2;
}

template <typename TK> void launch(const DecodeKv8Params& p, cudaStream_t stream) {
    const dim3 grid(p.c.B * p.Hq, p.nrun);
    if (p.c.code == ZGCM_E4M3)
        kv8_decode_kernel<TK, ZGCM_E4M3><<<grid, 128, 0, stream>>>(p);
    else
        kv8_decode_kernel<TK, ZGCM_INT8><<<grid, 128, 0, stream>>>(p);
}

}  // namespace
}  // namespace zgcm

using namespace zgcm;

extern "C" {

size_t zgcm_attn_decode_kv8_workspace_size(int n_seq, int Hq, int Hkv) {
    if (n_seq < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return 0;
    return (size_t)n_seq * Hq * DK_MAX_RUNS * 4 * DK_REC * sizeof(float);
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
    p.W = window;
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<bf16*>(out);
    p.lse = lse;
    p.part = static_cast<float*>(workspace);
    const int most = (blocks ? n_list : p.c.NB) + 1;
    p.len = (most + DK_MAX_RUNS - 1) / DK_MAX_RUNS;
    p.nrun = (most + p.len - 1) / p.len;
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    if (p.c.key == ZGCM_BF16)
        launch<bf16>(p, stream);
    else
        launch<__half>(p, stream);
    if (cudaGetLastError() != cudaSuccess) return ZGCM_ERR_CUDA;
    kv8_join_kernel<<<p.c.B * Hq, kD, 0, stream>>>(p);
    return cudaGetLastError() == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}

}  // extern "C"
