// kv8_select.cu — choice of the blocks a decode step reads (zgcm_kv8_select of
// include/zgcm_kv8.h).
//
//   score_j = max over the KV head's queries of q . k_mean_j;  the n_select highest, ties to
//   the lowest block, in ascending order.
//
// One pass over the block means, 256 bytes each.  The sums run in fp64: products of 16-bit
// values are exact there and the sum of 128 of them is off by 2^-46 of its terms at most, so the
// choice is that of the exact scores for all but astronomically close ties, and does not
// depend on the order of the sum.  They go to the fp64 matrix instruction, 8 blocks by 8 heads by 4 dims: a lane
// holds a quarter of a block's mean, one run of 64 bytes, and converts each element once for all heads (as sums
// by lanes and shuffles the scores took three times the instructions, and the kernel was bound by them).
//
// A cluster of CTAs takes one (sequence, KV head): each scores a slice of the blocks and writes
// its keys (fp64 scores as ordered 64-bit integers) into the first CTA's shared memory, which finds the
// n-th highest: up to 64 keys by counting, for each, those above it; more by one histogram of 1024 equal steps between
// the lowest and the highest, counting then among the few keys of the step the n-th falls in (or
// another histogram of that step, where they are many).  One scan writes the list in order.
#include <cooperative_groups.h>
#include <math.h>

#include "kv8.cuh"

namespace cg = cooperative_groups;

namespace zgcm {
namespace {

constexpr int SEL_ROWS = 8;                       // blocks of a warp at a time
constexpr int SEL_HEADS = 8;                      // heads at a time
constexpr int SEL_AHEAD = 4;                      // steps of a warp whose page numbers are looked up together
constexpr int SEL_BITS = 10, SEL_BINS = 1 << SEL_BITS;
constexpr int SEL_LIST = 256;                     // most keys of a step ranked by counting
constexpr int SEL_FEW = 64;                       // most keys ranked by counting without a histogram

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

// d += A B for 8 x 4 and 4 x 8: a of row lane / 4 and column lane % 4, b of row lane % 4 and column lane / 4, d of row
// lane / 4 and columns 2 (lane % 4), + 1
__device__ __forceinline__ void mma_f64(double (&d)[2], double a, double b) {
    asm volatile("mma.sync.aligned.m8n8k4.row.col.f64.f64.f64.f64 {%0,%1}, {%2}, {%3}, {%0,%1};"
                 : "+d"(d[0]), "+d"(d[1])
                 : "d"(a), "d"(b));
}

// exclusive scan over the CTA; every thread calls it
template <int WARPS> __device__ __forceinline__ uint32_t cta_scan(uint32_t x, uint32_t* red) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
    uint32_t s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, s, o);
        if (lane >= o) s += t;
    }
    if (lane == 31) red[w] = s;
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i)
        if (i < w) before += red[i];
    __syncthreads();
    return before + s - x;
}

struct SelSmem {
    double q[32][4][SEL_HEADS];   // [dim of a quarter][quarter][head]
    uint32_t hist[SEL_BINS];
    u64 list[SEL_LIST];
    u64 lo[16], hi[16];           // lowest and highest key of each warp's
    u64 thr;                      // keys above it are taken, and `need_eq` of those equal to it, the first ones
    uint32_t red[16];
    uint32_t bin, above, count, n_list, need_eq;
};

// Key number i of n as one of those that compete: not the first n_first nor the last n_last
__device__ __forceinline__ bool forced(const SelectParams& p, int i, int n) { return i < p.n_first || i >= n - p.n_last; }

// sm.thr and sm.need_eq of the `need` highest keys of the list (n <= SEL_LIST of them, at least `need`)
__device__ __forceinline__ void rank_list(SelSmem& sm, int n, int need) {
    if ((int)threadIdx.x < n) {
        const u64 k = sm.list[threadIdx.x];
        int gt = 0, ge = 0;
#pragma unroll 4
        for (int i = 0; i < n; ++i) {
            const u64 x = sm.list[i];
            gt += x > k;
            ge += x >= k;
        }
        if (gt < need && need <= ge) {   // all threads of that key write the same
            sm.thr = k;
            sm.need_eq = need - gt;
        }
    }
    __syncthreads();
}

template <typename TK, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv8_select_kernel(const __grid_constant__ SelectParams p) {
    constexpr int WARPS = THREADS / 32;
    extern __shared__ __align__(16) unsigned char dyn[];
    SelSmem& sm = *reinterpret_cast<SelSmem*>(dyn);
    u64* key = reinterpret_cast<u64*>(dyn + sizeof(SelSmem));   // [candidates]; as doubles until they are sent
    double* score = reinterpret_cast<double*>(key);
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    const int item = blockIdx.x / cs, b = item / p.c.Hkv, kvh = item % p.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int G = p.Hq / p.c.Hkv;
    const int pos = p.pos[b];
    // the sequence's page numbers into L2 while its position is read
    for (int i = tid; i < (p.c.NB * 4 + 127) / 128; i += THREADS)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.table + (size_t)b * p.c.NB + min(32 * i, p.c.NB - 1)));
    const int own = pos < 0 ? 0 : pos / kBlk, jlo = pos < 0 ? 0 : max(0, pos - p.W + 1) / kBlk;
    const bool reach = own - jlo < p.c.NB;        // the window's blocks are all in the table
    const int n = reach ? own - jlo : 0;          // candidates jlo .. own - 1
    int* out = p.blocks + (size_t)item * p.n_select;
    if (n <= p.n_select) {                        // the same for every CTA of the cluster
        if (rank == 0)
            for (int i = tid; i < p.n_select; i += THREADS) out[i] = i < n ? jlo + i : -1;
        return;
    }
    for (int i = tid; i < SEL_BINS; i += THREADS) sm.hist[i] = 0;
    const int per = (n + cs - 1) / cs, r0 = min(n, rank * per), r1 = min(n, r0 + per);
    for (int h0 = 0; h0 < G; h0 += SEL_HEADS) {
        const int nh = min(SEL_HEADS, G - h0);
        __syncthreads();
        for (int i = tid; i < SEL_HEADS * kD; i += THREADS) {
            const int h = i / kD, d = i % kD;
            sm.q[d & 31][d >> 5][h] = h < nh ? (double)key_to_float(static_cast<const TK*>(
                                                   p.q)[((size_t)b * p.Hq + (size_t)kvh * G + h0 + h) * kD + d])
                                             : 0.0;
        }
        __syncthreads();
        // lane (r, c): block r of the 8, quarter c of its dims
        const int r = lane >> 2, c = lane & 3;
        int pages[SEL_AHEAD];
        uint4 next[4];
        auto means = [&](int page) {
#pragma unroll
            for (int i = 0; i < 4; ++i) next[i] = make_uint4(0u, 0u, 0u, 0u);
            if (page >= 0) {
                const char* m = p.c.kmean + 2 * (((size_t)page * p.c.Hkv + kvh) * kD + 32 * c);
#pragma unroll
                for (int i = 0; i < 4; ++i) next[i] = *reinterpret_cast<const uint4*>(m + 16 * i);
            }
        };
        for (int rb0 = r0 + warp * SEL_ROWS; rb0 < r1; rb0 += SEL_AHEAD * WARPS * SEL_ROWS) {
#pragma unroll
            for (int i = 0; i < SEL_AHEAD; ++i) {
                const int row = rb0 + i * WARPS * SEL_ROWS + r;
                pages[i] = row < r1 ? kv8_page(p.c, b, jlo + row) : -1;
            }
            means(pages[0]);
#pragma unroll
            for (int it = 0; it < SEL_AHEAD; ++it) {
            const int rb = rb0 + it * WARPS * SEL_ROWS, row = rb + r, page = pages[it];
            if (rb >= r1) break;
            const uint4 w[4] = {next[0], next[1], next[2], next[3]};
            if (it + 1 < SEL_AHEAD) means(pages[it + 1]);   // on their way while these are worked on
            double acc[2][2] = {};   // two chains
#pragma unroll
            for (int e = 0; e < 32; ++e) {
                const double x = (double)key_to_float(reinterpret_cast<const TK*>(&w[e >> 3])[e & 7]);
                mma_f64(acc[e & 1], x, sm.q[e][c][r]);
            }
            // this lane: the heads 2 c and 2 c + 1 of its block
            double best = -INFINITY;
            bool nan = false;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const double a = acc[0][i] + acc[1][i];
                if (2 * c + i < nh) {
                    nan |= isnan(a);
                    best = a > best ? a : best;
                }
            }
#pragma unroll
            for (int o = 1; o < 4; o <<= 1) {
                const double x = __shfl_xor_sync(0xffffffffu, best, o);
                best = x > best ? x : best;
            }
            nan = (__ballot_sync(0xffffffffu, nan) >> (4 * r) & 15u) != 0;
            if (c == 0 && row < r1) {
                if (h0 > 0) {
                    nan |= isnan(score[row]);
                    best = score[row] > best ? score[row] : best;
                }
                score[row] = page < 0 ? -INFINITY : nan ? NAN : best;
            }
            }
        }
    }
    if (cs > 1)
        cluster.sync();   // the slice is scored, and the first CTA runs
    else
        __syncthreads();
    u64* dst = cluster.map_shared_rank(key, 0);
    for (int i = r0 + tid; i < r1; i += THREADS) {
        const double x = score[i];
        dst[i] = ordered(isnan(x) ? -INFINITY : x);
    }
    if (cs > 1)
        cluster.sync();
    else
        __syncthreads();
    if (rank != 0) return;

    // of the keys that compete, `need` are taken
    int need = p.n_select - p.n_first - p.n_last;
    const int rivals = n - p.n_first - p.n_last;
    if (tid == 0) {
        sm.thr = ~0ULL;
        sm.need_eq = 0;
        sm.n_list = 0;
    }
    __syncthreads();
    if (need > 0 && rivals <= SEL_FEW) {
        if (tid < rivals) sm.list[tid] = key[p.n_first + tid];
        __syncthreads();
        rank_list(sm, rivals, need);
    } else if (need > 0) {
        u64 lo = ~0ULL, hi = 0;
        for (int i = p.n_first + tid; i < n - p.n_last; i += THREADS) {
            lo = min(lo, key[i]);
            hi = max(hi, key[i]);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            lo = min(lo, __shfl_xor_sync(0xffffffffu, lo, o));
            hi = max(hi, __shfl_xor_sync(0xffffffffu, hi, o));
        }
        if (lane == 0) {
            sm.lo[warp] = lo;
            sm.hi[warp] = hi;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < WARPS; ++i) {
            lo = min(lo, sm.lo[i]);
            hi = max(hi, sm.hi[i]);
        }
        u64 range = hi - lo;      // of the step looked at: keys lo .. lo + range
        for (;;) {
            const int shift = max(0, 64 - SEL_BITS - __clzll((long long)range));
            for (int i = p.n_first + tid; i < n - p.n_last; i += THREADS)
                if (key[i] - lo <= range) atomicAdd(&sm.hist[(key[i] - lo) >> shift], 1u);
            __syncthreads();
            // bins from the highest: thread i takes the next PER of them
            constexpr int PER = SEL_BINS / THREADS;
            uint32_t c[PER], mine = 0;
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                c[i] = sm.hist[SEL_BINS - 1 - (tid * PER + i)];
                mine += c[i];
            }
            uint32_t before = cta_scan<WARPS>(mine, sm.red);
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
            need -= sm.above;
            lo += (u64)sm.bin << shift;
            range = (1ULL << shift) - 1;
            const int count = sm.count;
            if (count == need || shift == 0) {   // the whole step, or equal keys
                if (tid == 0) {
                    sm.thr = shift == 0 ? lo : lo - 1;
                    sm.need_eq = shift == 0 ? need : 0;
                }
                __syncthreads();
                break;
            }
            if (count <= SEL_LIST) {
                for (int i = p.n_first + tid; i < n - p.n_last; i += THREADS)
                    if (key[i] - lo <= range) sm.list[atomicAdd(&sm.n_list, 1u)] = key[i];
                __syncthreads();
                rank_list(sm, count, need);
                break;
            }
            for (int i = tid; i < SEL_BINS; i += THREADS) sm.hist[i] = 0;
            __syncthreads();
        }
    }
    // in order: a warp takes a run of candidates, 32 at a time; first how many before each warp's
    const u64 thr = sm.thr;
    const uint32_t need_eq = sm.need_eq;
    const int run = ((n + WARPS - 1) / WARPS + 31) & ~31, i0 = min(n, warp * run), i1 = min(n, i0 + run);
    uint32_t gt = 0, eq = 0;
    for (int i = i0 + lane; i - lane < i1; i += 32) {
        const bool in = i < i1, f = in && forced(p, i, n);
        gt += __popc(__ballot_sync(0xffffffffu, f || (in && key[i] > thr)));
        eq += __popc(__ballot_sync(0xffffffffu, in && !f && key[i] == thr));
    }
    if (lane == 0) sm.red[warp] = gt << 16 | eq;   // at most 16384 of each
    __syncthreads();
    uint32_t before = 0;
#pragma unroll
    for (int i = 0; i < WARPS; ++i)
        if (i < warp) before += sm.red[i];
    uint32_t at = (before >> 16) + min(before & 0xffffu, need_eq), seen = before & 0xffffu;
    const uint32_t below = (1u << lane) - 1;
    for (int i = i0 + lane; i - lane < i1; i += 32) {
        const bool in = i < i1, f = in && forced(p, i, n), same = in && !f && key[i] == thr;
        const uint32_t all_same = __ballot_sync(0xffffffffu, same);
        const bool take = f || (in && key[i] > thr) || (same && seen + __popc(all_same & below) < need_eq);
        const uint32_t all = __ballot_sync(0xffffffffu, take);
        if (take) out[at + __popc(all & below)] = jlo + i;
        at += __popc(all);
        seen += __popc(all_same);
    }
}

template <typename TK, int THREADS> cudaError_t launch(const SelectParams& p, cudaStream_t stream) {
    const long long items = (long long)p.c.B * p.c.Hkv;
    // CTAs of a cluster: one once the (sequence, head) pairs fill the SMs, else up to 8, with at least two steps of 8
    // rows for each warp left
    int cs = 1;
    while (cs < 8 && items * cs < 148 && p.c.NB / (2 * cs) >= THREADS / 4) cs *= 2;
    const int most = p.c.NB < kKv8MaxBlocks ? p.c.NB : kKv8MaxBlocks;
    const size_t smem = sizeof(SelSmem) + (size_t)most * 8;
    if (items * cs > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kernel = kv8_select_kernel<TK, THREADS>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * cs));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Threads of a CTA: 256 for contexts of up to 512 blocks (four CTAs an SM), else 512.
template <typename TK> cudaError_t launch_threads(const SelectParams& p, cudaStream_t stream) {
    return p.c.NB <= 512 ? launch<TK, 256>(p, stream) : launch<TK, 512>(p, stream);
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
    const cudaError_t e = p.c.key == ZGCM_BF16 ? launch_threads<bf16>(p, stream) : launch_threads<__half>(p, stream);
    return e == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}
