// kv8_select.cu — choice of the blocks a decode step reads (zgcm_kv8_select of
// include/zgcm_kv8.h).
//
//   score_j = max over the KV head's queries of q . k_mean_j;  the n_select highest, ties to
//   the lowest block, in ascending order.
//
// One pass over the block means, 256 bytes each.  The sums run in fp64: products of 16-bit
// values are exact there and the sum of 128 of them is off by 2^-46 of its terms at most, so the
// choice is that of the exact scores for all but astronomically close ties, and does not
// depend on the order of the sum.  A block's 128 elements belong to 8 lanes (two 16-byte
// loads each); a lane takes 4 blocks at a time against 4 heads, so an element is converted once
// for 4 heads and a query element read once for 4 blocks.
//
// A cluster of CTAs takes one (sequence, KV head): each scores a slice of the blocks and writes
// its keys (fp64 scores as ordered 64-bit integers) into the first CTA's shared memory, which
// finds the n-th highest by histograms of 11-bit digits from the top, stopping when a digit's
// bin is taken whole, and writes the list in order by one scan.
#include <cooperative_groups.h>
#include <math.h>

#include "kv8.cuh"

namespace cg = cooperative_groups;

namespace zgcm {
namespace {

constexpr int SEL_THREADS = 512;
constexpr int SEL_WARPS = SEL_THREADS / 32;
constexpr int SEL_ROWS = 4;                       // blocks of a lane at a time
constexpr int SEL_HEADS = 4;                      // heads at a time
constexpr int SEL_BITS = 11, SEL_BINS = 1 << SEL_BITS;

struct SelectParams {
    Kv8 c;
    const void* q;
    const int* pos;
    int* blocks;
    int Hq, W, n_select, n_first, n_last;
};

typedef unsigned long long u64;

__device__ __forceinline__ u64 ordered(double x) {
    const long long b = __double_as_longlong(x + 0.0);   // -0 becomes +0
    return b < 0 ? ~(u64)b : (u64)b | (1ULL << 63);
}

// exclusive scan over the CTA; every thread calls it
__device__ __forceinline__ uint32_t cta_scan(uint32_t x, uint32_t* red, uint32_t* total) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    __syncthreads();
    if (lane == 31) red[w] = s;
    __syncthreads();
    uint32_t before = 0, all = 0;
    for (int i = 0; i < SEL_WARPS; ++i) {
        const uint32_t t = red[i];
        if (i < w) before += t;
        all += t;
    }
    *total = all;
    return before + s - x;
}

struct SelSmem {
    double q[SEL_HEADS][16][8];   // [head][element of a lane][lane of the 8]
    uint32_t hist[SEL_BINS];
    uint32_t red[SEL_WARPS];
    uint32_t bin, above, count;
};

template <typename TK>
__global__ void __launch_bounds__(SEL_THREADS) kv8_select_kernel(const __grid_constant__ SelectParams p) {
    extern __shared__ __align__(16) unsigned char dyn[];
    SelSmem& sm = *reinterpret_cast<SelSmem*>(dyn);
    u64* key = reinterpret_cast<u64*>(dyn + sizeof(SelSmem));   // [candidates]; as doubles until they are sent
    double* score = reinterpret_cast<double*>(key);
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    const int item = blockIdx.x / cs, b = item / p.c.Hkv, kvh = item % p.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, l8 = lane & 7;
    const int G = p.Hq / p.c.Hkv;
    const int pos = p.pos[b];
    const int own = pos < 0 ? 0 : pos / kBlk, jlo = pos < 0 ? 0 : max(0, pos - p.W + 1) / kBlk;
    const bool reach = own - jlo < p.c.NB;        // the window's blocks are all in the table
    const int n = reach ? own - jlo : 0;          // candidates jlo .. own - 1
    int* out = p.blocks + (size_t)item * p.n_select;
    if (n <= p.n_select) {                        // the same for every CTA of the cluster
        if (rank == 0)
            for (int i = tid; i < p.n_select; i += SEL_THREADS) out[i] = i < n ? jlo + i : -1;
        return;
    }
    const int per = (n + cs - 1) / cs, r0 = min(n, rank * per), r1 = min(n, r0 + per);
    for (int h0 = 0; h0 < G; h0 += SEL_HEADS) {
        const int nh = min(SEL_HEADS, G - h0);
        __syncthreads();
        for (int i = tid; i < SEL_HEADS * kD; i += SEL_THREADS) {
            // element e of lane l is dim 8 l + e (e < 8) or 64 + 8 l + e - 8
            const int h = i / kD, e = (i / 8) % 16, l = i % 8, d = (e & 8) * 8 + 8 * l + (e & 7);
            sm.q[h][e][l] = h < nh ? (double)key_to_float(static_cast<const TK*>(
                                         p.q)[((size_t)b * p.Hq + (size_t)kvh * G + h0 + h) * kD + d])
                                   : 0.0;
        }
        __syncthreads();
        for (int rb = r0 + warp * 4 * SEL_ROWS + (lane >> 3) * SEL_ROWS; rb - (lane >> 3) * SEL_ROWS < r1;
             rb += SEL_WARPS * 4 * SEL_ROWS) {
            uint4 w[SEL_ROWS][2];
            bool ok[SEL_ROWS];
#pragma unroll
            for (int i = 0; i < SEL_ROWS; ++i) {
                const int page = rb + i < r1 ? kv8_page(p.c, b, jlo + rb + i) : -1;
                ok[i] = page >= 0;
                w[i][0] = w[i][1] = make_uint4(0u, 0u, 0u, 0u);
                if (ok[i]) {
                    const char* m = p.c.kmean + 2 * (((size_t)page * p.c.Hkv + kvh) * kD + 8 * l8);
                    w[i][0] = *reinterpret_cast<const uint4*>(m);
                    w[i][1] = *reinterpret_cast<const uint4*>(m + 128);
                }
            }
            double acc[SEL_ROWS][SEL_HEADS] = {};
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                double q[SEL_HEADS];
#pragma unroll
                for (int h = 0; h < SEL_HEADS; ++h) q[h] = sm.q[h][e][l8];
#pragma unroll
                for (int i = 0; i < SEL_ROWS; ++i) {
                    const double x = (double)key_to_float(reinterpret_cast<const TK*>(&w[i][e >> 3])[e & 7]);
#pragma unroll
                    for (int h = 0; h < SEL_HEADS; ++h) acc[i][h] = fma(q[h], x, acc[i][h]);
                }
            }
#pragma unroll
            for (int i = 0; i < SEL_ROWS; ++i) {
                double best = -INFINITY;
                bool nan = false;
#pragma unroll
                for (int h = 0; h < SEL_HEADS; ++h) {
                    double a = acc[i][h];
                    a += __shfl_xor_sync(0xffffffffu, a, 4);
                    a += __shfl_xor_sync(0xffffffffu, a, 2);
                    a += __shfl_xor_sync(0xffffffffu, a, 1);
                    if (h < nh) {
                        nan |= isnan(a);
                        best = fmax(best, a);
                    }
                }
                if (l8 == 0 && rb + i < r1) {
                    if (h0 > 0) {
                        nan |= isnan(score[rb + i]);
                        best = fmax(best, score[rb + i]);
                    }
                    score[rb + i] = !ok[i] ? -INFINITY : nan ? NAN : best;
                }
            }
        }
    }
    cluster.sync();   // the slice is scored, and the first CTA runs
    u64* dst = cluster.map_shared_rank(key, 0);
    for (int i = r0 + tid; i < r1; i += SEL_THREADS) {
        const double x = score[i];
        const u64 k = ordered(isnan(x) ? -INFINITY : x);
        dst[i] = i < p.n_first || i >= n - p.n_last ? ~0ULL : k;
    }
    cluster.sync();
    if (rank != 0) return;

    // the n_select-th highest key: `thr` and how many of the keys equal to it (at the digits
    // looked at) are taken
    u64 thr = 0, mask = 0;
    int need = p.n_select;
    for (int shift = 64 - SEL_BITS;; shift -= SEL_BITS) {
        const int s = max(shift, 0);
        const u64 digit = shift >= 0 ? SEL_BINS - 1 : (1ULL << (SEL_BITS + shift)) - 1;
        for (int i = tid; i < SEL_BINS; i += SEL_THREADS) sm.hist[i] = 0;
        __syncthreads();
        for (int i = tid; i < n; i += SEL_THREADS)
            if ((key[i] & mask) == thr) atomicAdd(&sm.hist[(key[i] >> s) & digit], 1u);
        __syncthreads();
        // bins from the highest: thread i takes the 4 bins SEL_BINS - 4 i - 1 ... - 4
        constexpr int PER = SEL_BINS / SEL_THREADS;
        uint32_t c[PER], mine = 0, all;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            c[i] = sm.hist[SEL_BINS - 1 - (tid * PER + i)];
            mine += c[i];
        }
        uint32_t before = cta_scan(mine, sm.red, &all);
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            if (before < (uint32_t)need && before + c[i] >= (uint32_t)need) {
                sm.bin = SEL_BINS - 1 - (tid * PER + i);
                sm.above = before;
                sm.count = c[i];
            }
            before += c[i];
        }
        __syncthreads();
        thr |= (u64)sm.bin << s;
        mask |= digit << s;
        need -= sm.above;
        const bool done = sm.count == (uint32_t)need || s == 0;
        __syncthreads();
        if (done) break;
    }
    // in order: thread i takes a run of candidates
    const int run = (n + SEL_THREADS - 1) / SEL_THREADS, i0 = min(n, tid * run), i1 = min(n, i0 + run);
    uint32_t gt = 0, eq = 0, all;
    for (int i = i0; i < i1; ++i) {
        gt += (key[i] & mask) > thr;
        eq += (key[i] & mask) == thr;
    }
    const uint32_t before = cta_scan(gt << 16 | eq, sm.red, &all);   // at most 16384 of each
    uint32_t at = (before >> 16) + min(before & 0xffffu, (uint32_t)need), seen = before & 0xffffu;
    for (int i = i0; i < i1; ++i) {
        const u64 k = key[i] & mask;
        const bool take = k > thr || (k == thr && seen < (uint32_t)need);
        seen += k == thr;
        if (take) out[at++] = jlo + i;
    }
}

template <typename TK> cudaError_t launch(const SelectParams& p, cudaStream_t stream) {
    const long long items = (long long)p.c.B * p.c.Hkv;
    // CTAs of a cluster: one once the (sequence, head) pairs fill the SMs, else up to 8, with at
    // least one 16-row step for each warp left
    int cs = 1;
    while (cs < 8 && items * cs < 148 && p.c.NB / (2 * cs) >= SEL_WARPS * 4 * SEL_ROWS / 2) cs *= 2;
    const int most = p.c.NB < kKv8MaxBlocks ? p.c.NB : kKv8MaxBlocks;
    const size_t smem = sizeof(SelSmem) + (size_t)most * 8;
    if (items * cs > 0x7fffffffLL) return cudaErrorInvalidValue;
    cudaError_t e = cudaFuncSetAttribute(kv8_select_kernel<TK>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * cs));
    cfg.blockDim = dim3(SEL_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_select_kernel<TK>, p);
}

}  // namespace
}  // namespace zgcm

using namespace zgcm;

extern "C" int zgcm_kv8_select(const zgcm_kv8_cache* cache, const void* q, const int* pos, int Hq, int window,
                               int n_select, int n_first, int n_last, int* blocks, void* cuda_stream) {
    SelectParams p;
    const int st = kv8_check(cache, &p.c);
    if (st != ZGCM_OK) return st;
    if (Hq < 1 || Hq % p.c.Hkv != 0 || window < 1 || n_select < 1 || n_first < 0 || n_last < 0 ||
        n_first > n_select - n_last)
        return ZGCM_ERR_INVALID_ARG;
    if (p.c.NB > kKv8MaxBlocks) return ZGCM_ERR_UNSUPPORTED;
    if (p.c.B == 0) return ZGCM_OK;
    if (!q || !pos || !blocks) return ZGCM_ERR_INVALID_ARG;
    if (((uintptr_t)q | (uintptr_t)pos | (uintptr_t)blocks) & 15u) return ZGCM_ERR_ALIGNMENT;
    p.q = q;
    p.pos = pos;
    p.blocks = blocks;
    p.Hq = Hq;
    p.W = window;
    p.n_select = n_select;
    p.n_first = n_first;
    p.n_last = n_last;
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const cudaError_t e = p.c.key == ZGCM_BF16 ? launch<bf16>(p, stream) : launch<__half>(p, stream);
    return e == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}
