// kv8_select.cu — choice of the blocks a decode step reads (zgcm_kv8_select of
// include/zgcm_kv8.h).
//
//   score_j = max over the KV head's queries of q . k_mean_j;  the n_select highest, ties to
//   the lowest block, in ascending order.
//
// One pass over the block means, 256 bytes each.  The choice is that of fp64 sums (products of 16-bit values
// are exact there and the sum of 128 of them is off by 2^-46 of its terms at most), but only blocks at the border
// need them: the tensor cores give every score in fp32 (16 blocks by 8 heads an instruction), off by less than
//      eps = 2^-14.5 max_h |q_h|_1 max_j |k_mean_j|_max
// (8 sums of 17 terms, each off by 2^-22 of the largest of them at most: 2^-14.9 of the terms' sum; the histogram's own
// roundings are small against the rest).  One histogram of 1024 or 4096 equal steps finds the step that holds the need-th
// highest of them, whose edges are v0 and v1; what lies above v1 + 2 eps is taken, what lies below v0 - 2 eps is not, and the
// few between are scored in fp64 and ranked by counting, unless all of them are needed.  (All scores in fp64, on the fp64
// matrix instruction, took 1.5 us for 8 blocks of a warp: 29 us for 32 of up to 256 blocks of 64 x 8 items, or 64 of 4096
// of 2 x 8, against 14.5 and 18.1 here.)  Where more than 256 are between, many equal scores say, or a score is not finite,
// all are scored in fp64 and the histogram is taken of those (as ordered 64-bit integers), as often as one step of it holds
// too many.
//
// A cluster of CTAs takes one (sequence, KV head): each scores a slice of the blocks and writes the scores into
// the first CTA's shared memory, which does the rest.  On a B200 the scoring of 64 x 8 items (26 MB of means) is 6 of the
// 14.5 us, position, page and two rounds of means one after the other; histogram, border and output are 4; of the 18.1 us
// for 2 x 8 items of 4096 blocks these are 6, in one CTA each.
#include <cooperative_groups.h>
#include <math.h>

#include "kv8_attn.cuh"

namespace cg = cooperative_groups;

namespace zgcm {
namespace {

constexpr int SEL_ROWS = 16;                      // blocks of a warp at a time
constexpr int SEL_LIST = 256;                     // most keys ranked by counting

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

__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t b = __float_as_uint(x);
    return (int)b < 0 ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float from_ordered(uint32_t k) { return __uint_as_float((int)k < 0 ? k & 0x7fffffffu : ~k); }

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

// steps of the histogram: 4 or 8 for each thread
template <int THREADS> constexpr int kSelBits = THREADS == 256 ? 10 : 12;

struct SelSmem {
    u64 list[SEL_LIST];
    uint16_t index[SEL_LIST];     // of the list's keys
    u64 lo[16], hi[16];           // lowest and highest of each warp's
    u64 thr;                      // keys above it are taken, and `need_eq` of those equal to it, the first ones
    uint32_t red[16];
    uint32_t bin, above, count, n_list, need_eq, taken;
    uint32_t mean_max;            // largest |k_mean| as its bits, q's largest 1-norm as fp32 bits
    uint32_t q1;
    uint32_t lowest, highest;     // fp32 scores of those that compete, ordered (the highest of all: one is NaN)
};

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

// The step of the histogram, counted from the top, in which the need-th falls: sm.bin, its sm.count and the number
// sm.above of those in higher steps.  The histogram is left zeroed.
template <int THREADS> __device__ __forceinline__ void find_step(SelSmem& sm, uint32_t* hist, int need) {
    constexpr int SEL_BINS = 1 << kSelBits<THREADS>, PER = SEL_BINS / THREADS;
    const int tid = threadIdx.x;
    uint32_t c[PER], mine = 0;   // steps SEL_BINS - 1 - (tid * PER + i)
#pragma unroll
    for (int i = 0; i < PER; i += 4) {
        uint4* h = reinterpret_cast<uint4*>(hist + SEL_BINS - 4 - (tid * PER + i));
        const uint4 x = *h;
        *h = make_uint4(0u, 0u, 0u, 0u);
        c[i] = x.w;
        c[i + 1] = x.z;
        c[i + 2] = x.y;
        c[i + 3] = x.x;
        mine += x.x + x.y + x.z + x.w;
    }
    uint32_t before = cta_scan<THREADS / 32>(mine, sm.red);
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
}

// The fp64 score of block j as an ordered integer, by a warp (4 lanes a head): -inf for a bad page or a NaN.
template <typename TK>
__device__ __forceinline__ u64 exact_key(const SelectParams& p, int b, int kvh, int j) {
    const int lane = threadIdx.x & 31, r = lane >> 2, c = lane & 3, G = p.Hq / p.c.Hkv;
    const int page = kv8_page(p.c, b, j);
    if (page < 0) return ordered(-INFINITY);
    const uint4* m = reinterpret_cast<const uint4*>(p.c.kmean + 2 * ((size_t)page * p.c.Hkv + kvh) * kD) + c;
    u64 best = ordered(-INFINITY);
    bool nan = false;
    for (int h0 = 0; h0 < G; h0 += 8) {
        const int h = min(h0 + r, G - 1);   // the last one again where there are no more
        const uint4* q = reinterpret_cast<const uint4*>(static_cast<const TK*>(p.q) +
                                                        ((size_t)b * p.Hq + (size_t)kvh * G + h) * kD) + c;
        double a0 = 0.0, a1 = 0.0;
        auto add = [&](uint32_t u, uint32_t v) {
            const float2 f = KeyType<TK>::unpack(u), g = KeyType<TK>::unpack(v);
            a0 = fma((double)f.x, (double)g.x, a0);
            a1 = fma((double)f.y, (double)g.y, a1);
        };
#pragma unroll 2
        for (int i = 0; i < 4; ++i) {
            const uint4 x = m[4 * i], y = q[4 * i];
            add(x.x, y.x);
            add(x.y, y.y);
            add(x.z, y.z);
            add(x.w, y.w);
        }
        double a = a0 + a1;
        a += __shfl_xor_sync(0xffffffffu, a, 1);
        a += __shfl_xor_sync(0xffffffffu, a, 2);
        nan |= isnan(a);
        if (a >= -INFINITY) best = max(best, ordered(a));
    }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) best = max(best, __shfl_xor_sync(0xffffffffu, best, o));
    return __any_sync(0xffffffffu, nan) ? ordered(-INFINITY) : best;
}

template <typename TK, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) kv8_select_kernel(const __grid_constant__ SelectParams p) {
    constexpr int WARPS = THREADS / 32, SEL_BITS = kSelBits<THREADS>, SEL_BINS = 1 << SEL_BITS;
    extern __shared__ __align__(16) unsigned char dyn[];
    SelSmem& sm = *reinterpret_cast<SelSmem*>(dyn);
    static_assert(sizeof(SelSmem) % 16 == 0, "the histogram is read by 16 bytes");
    uint32_t* hist = reinterpret_cast<uint32_t*>(dyn + sizeof(SelSmem));
    float* score = reinterpret_cast<float*>(hist + SEL_BINS);   // [candidates], of the first CTA
    u64* key = reinterpret_cast<u64*>(hist + SEL_BINS);         // the same place, where fp64 scores take over
    cg::cluster_group cluster = cg::this_cluster();
    const int cs = cluster.num_blocks(), rank = cluster.block_rank();
    const int item = blockIdx.x / cs, b = item / p.c.Hkv, kvh = item % p.c.Hkv;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int G = p.Hq / p.c.Hkv;
    const int pos = p.pos[b];
    // the sequence's page numbers into L2 while its position is read
    for (int i = tid; i < (p.c.NB * 4 + 127) / 128; i += THREADS)
        asm volatile("prefetch.global.L2 [%0];" ::"l"(p.c.table + (size_t)b * p.c.NB + min(32 * i, p.c.NB - 1)));
    for (int i = tid; i < SEL_BINS; i += THREADS) hist[i] = 0;
    if (tid == 0) {
        sm.mean_max = sm.q1 = 0;
        sm.n_list = sm.taken = 0;
        sm.lowest = ~0u;
        sm.highest = 0u;
        sm.thr = ~0ULL;
        sm.need_eq = 0;
    }
    cluster.barrier_arrive();   // shared memory is as above (waited for where it is first written to)
    const int own = pos < 0 ? 0 : pos / kBlk, jlo = pos < 0 ? 0 : max(0, pos - p.W + 1) / kBlk;
    const bool reach = own - jlo < p.c.NB;        // the window's blocks are all in the table
    const int n = reach ? own - jlo : 0;          // candidates jlo .. own - 1
    int* out = p.blocks + (size_t)item * p.n_select;
    if (n <= p.n_select) {                        // the same for every CTA of the cluster
        cluster.barrier_wait();
        if (rank == 0)
            for (int i = tid; i < p.n_select; i += THREADS) out[i] = i < n ? jlo + i : -1;
        return;
    }
    float* dst = cluster.map_shared_rank(score, 0);
    SelSmem& first = *cluster.map_shared_rank(&sm, 0);
    const int per = ((n + cs - 1) / cs + SEL_ROWS - 1) / SEL_ROWS * SEL_ROWS, r0 = min(n, rank * per), r1 = min(n, r0 + per);
    const int i0 = p.n_first, i1 = n - p.n_last;   // those that compete: the first and last ones are taken anyhow
    float q1_max = 0.f;
    bool ready = false;     // the first CTA's shared memory
    uint32_t mean_max = 0, lowest = ~0u, highest = 0u;
    for (int h0 = 0; h0 < G; h0 += SEL_ROWS / 2) {
        const int nh = min(SEL_ROWS / 2, G - h0);
        // the second operand: head r, dims 32 i + 8 c .. + 7 (both operands have the dims in this order)
        uint4 q[4];
        float q1 = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            q[i] = make_uint4(0u, 0u, 0u, 0u);
            if (r < nh)
                q[i] = *reinterpret_cast<const uint4*>(static_cast<const TK*>(p.q) +
                                                       ((size_t)b * p.Hq + (size_t)kvh * G + h0 + r) * kD + 32 * i + 8 * c);
            const float2 x = KeyType<TK>::unpack(q[i].x), y = KeyType<TK>::unpack(q[i].y);
            const float2 z = KeyType<TK>::unpack(q[i].z), w = KeyType<TK>::unpack(q[i].w);
            q1 += fabsf(x.x) + fabsf(x.y) + (fabsf(y.x) + fabsf(y.y)) + (fabsf(z.x) + fabsf(z.y) + (fabsf(w.x) + fabsf(w.y)));
        }
        q1 += __shfl_xor_sync(0xffffffffu, q1, 1);
        q1 += __shfl_xor_sync(0xffffffffu, q1, 2);
        q1_max = fmaxf(q1_max, q1);
        int pages[2];
        auto look_up = [&](int rows) {
#pragma unroll
            for (int x = 0; x < 2; ++x)
                pages[x] = rows + 8 * x + r < r1 ? kv8_page(p.c, b, jlo + rows + 8 * x + r) : -1;
        };
        look_up(r0 + warp * SEL_ROWS);
        for (int rows = r0 + warp * SEL_ROWS; rows < r1; rows += WARPS * SEL_ROWS) {
            uint4 w[2][4];
            uint32_t big[2] = {0, 0};
            const bool bad[2] = {pages[0] < 0, pages[1] < 0};
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const char* m = p.c.kmean + 2 * (((size_t)max(pages[x], 0) * p.c.Hkv + kvh) * kD + 8 * c);
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    w[x][e] = bad[x] ? make_uint4(0u, 0u, 0u, 0u) : *reinterpret_cast<const uint4*>(m + 64 * e);
            }
            look_up(rows + WARPS * SEL_ROWS);   // the next step's, while the means come
            if (!ready) cluster.barrier_wait();
            ready = true;
            float d[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                mma16816<KeyType<TK>::kBf>(d, w[0][e].x, w[1][e].x, w[0][e].y, w[1][e].y, q[e].x, q[e].y);
                mma16816<KeyType<TK>::kBf>(d, w[0][e].z, w[1][e].z, w[0][e].w, w[1][e].w, q[e].z, q[e].w);
#pragma unroll
                for (int x = 0; x < 2; ++x)
                    big[x] = __vmaxu2(__vmaxu2(big[x], __vmaxu2(w[x][e].x & 0x7fff7fffu, w[x][e].y & 0x7fff7fffu)),
                                      __vmaxu2(w[x][e].z & 0x7fff7fffu, w[x][e].w & 0x7fff7fffu));
            }
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                const int row = rows + 8 * x + r;
                // of the heads 2 c and 2 c + 1; a sum that is not finite makes the block's score NaN
                float s = -INFINITY;
                bool odd = false;
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    if (2 * c + e < nh) {
                        odd |= !isfinite(d[2 * x + e]);
                        s = fmaxf(s, d[2 * x + e]);
                    }
                s = quad_max(s);
                odd = (__ballot_sync(0xffffffffu, odd) >> (4 * r) & 15u) != 0;
                if (row < r1 && !odd) mean_max = max(mean_max, max(big[x] & 0xffffu, big[x] >> 16));
                if (c == 0 && row < r1) {
                    if (h0 > 0) s = fmaxf(s, dst[row]);
                    odd = odd || (h0 > 0 && isnan(dst[row])) || bad[x];
                    dst[row] = odd ? NAN : s;
                    if (h0 + SEL_ROWS / 2 >= G && row >= i0 && row < i1) {
                        lowest = min(lowest, ordered(s));
                        highest = max(highest, odd ? ~0u : ordered(s));
                    }
                }
            }
        }
    }
    if (!ready) cluster.barrier_wait();
    mean_max = __reduce_max_sync(0xffffffffu, mean_max);
    lowest = __reduce_min_sync(0xffffffffu, lowest);
    highest = __reduce_max_sync(0xffffffffu, highest);
    if (rank == 0 && warp == 0 && c == 0) atomicMax(&sm.q1, __float_as_uint(q1_max));   // positive: bits order as values
    if (lane == 0) {
        atomicMax(&first.mean_max, mean_max);
        atomicMin(&first.lowest, lowest);
        atomicMax(&first.highest, highest);
    }
    if (cs > 1)
        cluster.sync();
    else
        __syncthreads();
    if (rank != 0) return;

    int need = p.n_select - p.n_first - p.n_last;   // of those that compete
    const bool some = need > 0;
    bool exact = false;     // keys instead of scores
    if (some) {
        const float lo = from_ordered(sm.lowest), hi = from_ordered(sm.highest);
        const float width = hi - lo, steps = width > 0.f ? (SEL_BINS - 1) / width : 0.f;
        exact = !isfinite(width) || !isfinite(steps);   // the same for all threads
        if (!exact) {
            auto step = [&](float x) { return min(SEL_BINS - 1, (int)((x - lo) * steps)); };   // grows with x
            for (int i = i0 + tid; i < i1; i += THREADS) atomicAdd(&hist[step(score[i])], 1u);
            __syncthreads();
            find_step<THREADS>(sm, hist, need);
            // The step's edges.  Four roundings of 2^-24 in a score's place among the SEL_BINS steps and four in an edge's:
            // 2^-21 SEL_BINS of a step together; adding lo is 2^-24 of a score, within the room that eps has.
            constexpr float off = SEL_BINS * 0x1p-21f;
            const float eps = 0x1.7p-15f * __uint_as_float(sm.q1) * from_bits<TK>(sm.mean_max) + 0x1p-100f;
            const float v0 = lo + ((float)sm.bin - off) * (width / (SEL_BINS - 1)) - 2.f * eps;
            const float v1 = lo + ((float)sm.bin + (1.f + off)) * (width / (SEL_BINS - 1)) + 2.f * eps;
            // taken, not taken, and the list of those between
            uint32_t above = 0;
            for (int i = i0 + tid; i < i1; i += THREADS) {
                const float x = score[i];
                if (x > v1) {
                    score[i] = INFINITY;
                    ++above;
                } else if (x < v0) {
                    score[i] = -INFINITY;
                } else {
                    const uint32_t at = atomicAdd(&sm.n_list, 1u);
                    if (at < SEL_LIST) sm.index[at] = (uint16_t)i;
                }
            }
            above = __reduce_add_sync(0xffffffffu, above);
            if (lane == 0 && above > 0) atomicAdd(&sm.taken, above);
            __syncthreads();
            const int between = sm.n_list;
            exact = between > SEL_LIST;
            if (!exact) {
                need -= sm.taken;
                if (between == need) {   // all of them: one block is alone there as a rule
                    if (tid < between) score[sm.index[tid]] = INFINITY;
                } else {
                    for (int i = warp; i < between; i += WARPS) {
                        const u64 k = exact_key<TK>(p, b, kvh, jlo + sm.index[i]);
                        if (lane == 0) sm.list[i] = k;
                    }
                    __syncthreads();
                    if (tid < between) {
                        const u64 k = sm.list[tid];
                        const int at = sm.index[tid];
                        int before = 0;
                        for (int i = 0; i < between; ++i) before += sm.list[i] > k || (sm.list[i] == k && sm.index[i] < at);
                        score[at] = before < need ? INFINITY : -INFINITY;
                    }
                }
            }
        }
        __syncthreads();
    }
    if (exact) {
        for (int i = i0 + warp; i < i1; i += WARPS) {
            const u64 k = exact_key<TK>(p, b, kvh, jlo + i);
            if (lane == 0) key[i] = k;
        }
        if (tid == 0) sm.n_list = 0;
        __syncthreads();
        u64 lo = ~0ULL, hi = 0;
        for (int i = i0 + tid; i < i1; i += THREADS) {
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
            for (int i = i0 + tid; i < i1; i += THREADS)
                if (key[i] - lo <= range) atomicAdd(&hist[(key[i] - lo) >> shift], 1u);
            __syncthreads();
            find_step<THREADS>(sm, hist, need);
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
                for (int i = i0 + tid; i < i1; i += THREADS)
                    if (key[i] - lo <= range) sm.list[atomicAdd(&sm.n_list, 1u)] = key[i];
                __syncthreads();
                rank_list(sm, count, need);
                break;
            }
            __syncthreads();   // the step has been read
        }
    }
    __syncthreads();
    // In order: a warp takes a run of candidates, at most 32 x 32, lane i the 32 from 32 i: which of them are taken, and
    // which are equal to the threshold; then where each lane's go.
    const u64 thr = sm.thr;
    const int need_eq = sm.need_eq;
    const int run = ((n + WARPS - 1) / WARPS + 31) & ~31, w0 = warp * run;
    static_assert(kKv8MaxBlocks <= 1024 * 16, "a lane for each 32 of a warp's run");
    uint32_t mine = 0, mine_eq = 0;
    for (int it = 0; it * 32 < run; ++it) {
        const int i = w0 + it * 32 + lane;
        bool t = i < n, same = false;
        if (t && i >= i0 && i < i1) {
            if (exact) {
                t = key[i] > thr;
                same = key[i] == thr;
            } else {
                t = some && score[i] == INFINITY;
            }
        }
        const uint32_t all = __ballot_sync(0xffffffffu, t), all_same = __ballot_sync(0xffffffffu, same);
        if (it == lane) {
            mine = all;
            mine_eq = all_same;
        }
    }
    const uint32_t before = cta_scan<WARPS>(__popc(mine) << 16 | __popc(mine_eq), sm.red);   // at most 16384 of each
    int seen = before & 0xffffu, at = (before >> 16) + min(seen, need_eq);
    for (uint32_t left = mine | mine_eq; left; left &= left - 1) {
        const uint32_t bit = left & -left;
        if ((mine & bit) || seen < need_eq) out[at++] = jlo + w0 + 32 * lane + __ffs(bit) - 1;
        seen += (mine_eq & bit) != 0;
    }
}

template <typename TK, int THREADS> cudaError_t launch(const SelectParams& p, cudaStream_t stream) {
    const long long items = (long long)p.c.B * p.c.Hkv;
    // CTAs of a cluster: one once the (sequence, head) pairs fill the SMs, else up to 8, with a step of 16 rows for half of
    // the warps left at least (2 sequences of 256K with 1, 2, 4, 8 CTAs: 36.5, 24.6, 18.2, 18.2 us; 64 of 16K with 1, 2:
    // 14.5, 21.2)
    int cs = 1;
    while (cs < 8 && items * cs < 148 && p.c.NB / (2 * cs) >= THREADS / 4) cs *= 2;
    constexpr size_t fixed = sizeof(SelSmem) + (4u << kSelBits<THREADS>), most = fixed + (size_t)kKv8MaxBlocks * 8;
    if (items * cs > 0x7fffffffLL) return cudaErrorInvalidValue;
    auto kernel = kv8_select_kernel<TK, THREADS>;
    // the same limit in every call, whatever this one needs: the attribute is the kernel's, and a call on another thread may
    // set it between here and the launch
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)most);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(items * cs));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = fixed + (size_t)p.c.NB * 8;   // NB <= kKv8MaxBlocks: checked
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = cs;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Threads of a CTA: 256 for contexts of up to 1024 blocks (four CTAs an SM), else 512, since one CTA goes through all of an
// item's scores.  Measured (us, 256 / 512): 64 sequences of 16K 14.5 / 23, of 64K 38 / 47, 16 of 128K 28.8 / 26.0, 8 of
// 256K 31.4 / 27.2, 2 of 512K 36.3 / 27.5.
template <typename TK> cudaError_t launch_threads(const SelectParams& p, cudaStream_t stream) {
    return p.c.NB <= 1024 ? launch<TK, 256>(p, stream) : launch<TK, 512>(p, stream);
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
