// kv8_direct.cu — decode attention over the 8-bit block cache in one launch, for items of few blocks (a sliding
// layer's window, a list of selected blocks, short contexts): see kv8_decode.cu for the arithmetic and for the
// kernel of long ones.
//
// There the whole call is a few microseconds, most of them latencies in a row: position, page number, codes.  So a
// cluster of 1 to 16 CTAs takes an item whose units are split evenly among them; nothing but its own position
// decides a CTA's work, the rows of q and of the tail load while page numbers do, the CTAs' parts meet in
// shared memory across the cluster (each is sent its share of all, and finishes it), and there is no second kernel.  Four CTAs of
// four warps fit on an SM: their latencies overlap.
// Measured on a B200 in a graph's replays, 8 KV heads of 4: one sequence of 1000 tokens 7.6 us (an empty call takes 2); a
// window of 128 for 64 sequences 10.8 us, 23 MB; 32 selected blocks for 16 sequences 23.2 us, 70 MB, 3.0 TB/s: position, table, list, page and
// codes follow each other, 0.6 to 1 us each from HBM, and 256 CTAs' copies are not many enough to fill that time.
#include <cooperative_groups.h>

#include "kv8_attn.cuh"

namespace cg = cooperative_groups;

namespace zgcm {
namespace {

constexpr int DD_THREADS = 128;
constexpr int DD_SPLIT = 16;                // most CTAs of an item (clusters above 8 have to be allowed)
constexpr int DD_WAIT = 0x820;
constexpr size_t DD_RING = 4 * kSlots * kSlot;
static_assert(DD_RING >= 4 * DK_HEADS * (kD + 4) * sizeof(float), "the warps' parts take the ring's place");

constexpr int DD_ROW = kD + 4;   // floats of a head in a warp's part: the lanes' two heads in different banks

struct DirectSmem {
    WarpSmem warp[4];
    float ml[4][DK_HEADS][2];
    float from_ml[DD_SPLIT][DK_HEADS][2];      // [CTA of the cluster]: its maximum and sum
    float4 from[2 * DD_THREADS];               // [CTA][place of this CTA's share]: its O
    int abort;
};

__device__ __forceinline__ void prefetch_l2(const void* p, int bytes) {
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(p), "r"(bytes) : "memory");
}
__device__ __forceinline__ void prefetch_line(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

template <typename TK, int CODE, bool WIDE>
__global__ void __launch_bounds__(DD_THREADS, 4) kv8_direct_kernel(const __grid_constant__ DecodeKv8Params p) {
    extern __shared__ unsigned char raw[];
    __shared__ DirectSmem sm;
    unsigned char* ring = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    cg::cluster_group cluster = cg::this_cluster();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    const int rank = blockIdx.x % p.split, item = blockIdx.x / p.split;
    const int b = item / (p.c.Hkv * p.HT), rest = item % (p.c.Hkv * p.HT), kvh = rest / p.HT, ht = rest % p.HT;
    const int nh = min(DK_HEADS, p.G - ht * DK_HEADS);
    const size_t head0 = (size_t)b * p.Hq + (size_t)kvh * p.G + ht * DK_HEADS;
    const int pos = p.pos[b];
    // What the position will ask for, into L2 while it is read: the sequence's page numbers, and for the first CTA the
    // tail.
    const size_t seq_head = (size_t)b * p.c.Hkv + kvh;
    if (rank == 0 && lane < 2)
        prefetch_l2(lane == 0 ? p.c.ktail + seq_head * kBlkBytes * 2 + warp * 16 * kD * 2
                              : reinterpret_cast<const char*>(p.c.vtail + seq_head * kBlkBytes + warp * 16 * kD),
                    16 * kD * 2);
    if (warp == 3 && p.c.NB <= 2048)
        for (int i = lane; i < (p.c.NB * 4 + 127) / 128; i += 32) prefetch_line(p.c.table + (size_t)b * p.c.NB + min(32 * i, p.c.NB - 1));
    uint32_t qt[8][2];
    load_q<TK, WIDE>(p, head0, nh, qt);
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&sm.warp[warp].full[i], 1);
        if (warp == 0) sm.abort = 0;
        fence_barrier_init();
    }
    __syncthreads();
    if (p.split > 1) cluster_arrive();   // this CTA's shared memory may be written to
    const Span s = span_of(p, pos);
    if (s.idle || s.bad) {   // the same for the whole cluster
        if (rank == 0 && warp == 0 && r < nh) no_answer(p, head0 + r, s.idle);
        if (p.split > 1) cluster_wait();
        return;
    }
    // this thread's places, of a head and 4 dims each: of all, or of the CTA's share of them
    constexpr int EACH = WIDE ? 2 : 1, PLACES = EACH * DD_THREADS;
    const int share = PLACES / p.split;
    uint2 gate[EACH];
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int at = rank * share + tid + DD_THREADS * i, h = at >> 5;
        gate[i] = tid + DD_THREADS * i < share && h < nh ? load_gate(p, head0 + h, 4 * (at & 31)) : make_uint2(0u, 0u);
    }
    // this CTA's units, the tail the first of all; its blocks; of them this warp's pair's, every second one
    const int u0 = max(0, (int)((long long)s.units * rank / p.split) - 1);
    const int u1 = (int)((long long)s.units * (rank + 1) / p.split) - 1;
    const int team = warp >> 1, nt = (u1 - u0 - team + 1) / 2;
    Stream stream(p, sm.warp[warp], ring + warp * kSlots * kSlot, &sm.abort);
    auto fetch = [&](int batch) {   // lane i: the pair's block 32 batch + i
        const int k = 32 * batch + lane;
        return k < nt ? block_of(p, s, b, kvh, u0 + team + 2 * k) : Block{-1, -1, 0.f, 0.f};
    };
    stream.mine = fetch(0);
    stream.start(nt);

    State t;
    if (rank == 0) {   // while the first codes are on their way
        const int last = pos - s.own * kBlk, first = s.lo - s.own * kBlk;
        if (warp * 16 <= last && warp * 16 + 15 >= first) {
            Tail<TK, WIDE> tail;
            tail.load(p, seq_head, warp * 16);
            tail.take(t, qt, p.scale_log2, warp * 16, first, last);
        }
    }
    uint32_t q16[8][2];
    const float2 qs = q_as_half<TK>(p, qt, q16);
    int gave_up = 0;
    for (int k = 0; k < nt; ++k) {
        if (stream.ok) gave_up = k;
        stream.take<CODE, WIDE>(t, q16, qs, s.lo, k, nt, DD_WAIT, fetch);
    }
    stream.drain(gave_up, nt);
    // the warps' parts, in a fixed order; the ring is free once all have come here
    float(*acc)[DK_HEADS][DD_ROW] = reinterpret_cast<float(*)[DK_HEADS][DD_ROW]>(ring);   // [warp]
    put_ml(t, sm.ml[warp]);
    __syncthreads();
    float m, l;
    const float fx = join_ml(sm.ml, 2 * c, warp, m, l), fy = join_ml(sm.ml, 2 * c + 1, warp, m, l);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const int d = 16 * i + 2 * r;
        *reinterpret_cast<float2*>(&acc[warp][2 * c][d]) = make_float2(t.o[i][0].x * fx, t.o[i][1].x * fx);
        *reinterpret_cast<float2*>(&acc[warp][2 * c + 1][d]) = make_float2(t.o[i][0].y * fy, t.o[i][1].y * fy);
    }
    __syncthreads();
    if (p.split > 1) cluster_wait();   // every CTA of the cluster runs
#pragma unroll
    for (int i = 0; i < EACH; ++i) {
        const int at = tid + DD_THREADS * i, h = at >> 5, d = 4 * (at & 31);
        float4 x = *reinterpret_cast<const float4*>(&acc[0][h][d]);
#pragma unroll
        for (int w = 1; w < (WIDE ? 4 : 8); ++w) {   // the warps' columns h, then what the low halves of p gave
            const float4 y = *reinterpret_cast<const float4*>(&acc[w & 3][h + (w >> 2) * (DK_HEADS / 2)][d]);
            x = make_float4(x.x + y.x, x.y + y.y, x.z + y.z, x.w + y.w);
        }
        if (p.split == 1) {
            join_ml(sm.ml, h, 0, m, l);
            const float o[4] = {x.x, x.y, x.z, x.w};
            if (h < nh) finish4(p, head0 + h, d, m, l, o, gate[i]);
        } else {   // to the CTA whose share the place is in
            cluster.map_shared_rank(sm.from, at / share)[rank * share + at % share] = x;
        }
    }
    static_assert(DK_HEADS * DD_SPLIT <= DD_THREADS, "a thread for each head and CTA");
    if (p.split > 1) {
        if (tid < DK_HEADS * p.split) {   // every CTA's copy of the maximum and sum
            const int h = tid % DK_HEADS;
            join_ml(sm.ml, h, 0, m, l);
            *reinterpret_cast<float2*>(cluster.map_shared_rank(sm.from_ml, tid / DK_HEADS)[rank][h]) = make_float2(m, l);
        }
        cluster_arrive();
        cluster_wait();
        const int at = rank * share + tid, h = at >> 5;
        if (tid < share && h < nh) {
            float o[4] = {0.f, 0.f, 0.f, 0.f};
            m = -INFINITY;
            l = 0.f;
#pragma unroll
            for (int i = 0; i < DD_SPLIT; ++i)
                if (i < p.split) m = fmaxf(m, sm.from_ml[i][h][0]);
#pragma unroll
            for (int i = 0; i < DD_SPLIT; ++i)
                if (i < p.split) {
                    const float2 ml = *reinterpret_cast<const float2*>(sm.from_ml[i][h]);
                    const float4 y = sm.from[i * share + tid];
                    const float f = ml.y == 0.f ? 0.f : fast_exp2(ml.x - m);
                    l = fmaf(ml.y, f, l);
                    o[0] = fmaf(y.x, f, o[0]);
                    o[1] = fmaf(y.y, f, o[1]);
                    o[2] = fmaf(y.z, f, o[2]);
                    o[3] = fmaf(y.w, f, o[3]);
                }
            finish4(p, head0 + h, 4 * (at & 31), m, l, o, gate[0]);
        }
    }
    if (tid == 0 && sm.abort) *p.err = sm.abort;
}

template <typename TK, int CODE, bool WIDE> cudaError_t launch_kernel(const DecodeKv8Params& p, cudaStream_t stream) {
    const size_t smem = DD_RING + 1024;
    auto kernel = kv8_direct_kernel<TK, CODE, WIDE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    if (p.split > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.c.B * p.c.Hkv * p.HT * p.split));
    cfg.blockDim = dim3(DD_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = p.split;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename TK, int CODE> cudaError_t launch(const DecodeKv8Params& p, cudaStream_t stream) {
    return p.G > DK_HEADS / 2 ? launch_kernel<TK, CODE, true>(p, stream) : launch_kernel<TK, CODE, false>(p, stream);
}

}  // namespace

// Whether this kernel takes the call, and how an item is split.  units: the most an item can have.
//
// An item is split while there are CTA places left on the 148 SMs (two CTAs an SM) and a CTA keeps more than one unit; the
// kernel takes the call while a CTA has at most 64 units (48 where groups have more than 4 heads), or 32 where the CTAs do not
// fill the SMs, which the equal runs of kv8_decode_kernel do whatever the items.  Measured (us; int8, this kernel / that one;
// "to": lengths of half that and more, where the longest item decides):
//   8 KV heads of 4, 1 sequence of 1000 7.6 / 12.8, 16K 21.3 / 30.4, 32K (31 units a CTA) 33.2 / 37.4, 64K 60 / 51
//   16 sequences of   8K (64) 61 / 70, to 8K 57 / 55, to 16K 107 / 88
//   64 to             4K (64) 82 / 88, 8K 155 / 153, 16K 315 / 291
//   4 KV heads of 8, 1 of 32K (31) 38 / 44, 64K 63 / 49;  16 to 8K (32) 38 / 39, 12K (47) 52 / 46, 16K (64) 69 / 55
//   64 of 3000 (47) 55 / 60, to 3000 53 / 50, of 4K (64) 70 / 71, to 4K 69 / 57
// and 16 CTAs an item against 8: 1 x 4K 10.8 / 12.3, 1 x 16K 20.7 / 29.4; two CTAs an SM against four: 4 x 16K 35 / 47,
// 32 listed blocks of 16 sequences 24.9 / 25.2.
bool kv8_direct_plan(DecodeKv8Params& p, int units) {
    const long long items = (long long)p.c.B * p.c.Hkv * p.HT;
    p.split = 1;
    while (p.split < DD_SPLIT && items * p.split * 2 <= 296 && units > 2 * p.split) p.split *= 2;
    return units <= (items * p.split < 148 ? 32 : p.G > DK_HEADS / 2 ? 48 : 64) * p.split;
}

cudaError_t kv8_direct_launch(const DecodeKv8Params& p, cudaStream_t stream) {
    const bool f8 = p.c.code == ZGCM_E4M3;
    return p.c.key == ZGCM_BF16 ? (f8 ? launch<bf16, ZGCM_E4M3>(p, stream) : launch<bf16, ZGCM_INT8>(p, stream))
                                : (f8 ? launch<__half, ZGCM_E4M3>(p, stream) : launch<__half, ZGCM_INT8>(p, stream));
}

}  // namespace zgcm
