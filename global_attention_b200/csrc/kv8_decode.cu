// kv8_decode.cu — decode attention over the 8-bit block cache (zgcm_attn_decode_kv8 of
// include/zgcm_kv8.h): one token per sequence.
//
// Bound by reading the codes: a block of one KV head is 16 KB and serves the few query heads of
// its group.  What has to keep up with 43 bytes per SM and nanosecond is the conversion of the codes
// and the two products; on CUDA cores the products alone are 8 multiply-adds per byte for 4
// heads, more than an SM has.  So both run on the tensor cores as mma.sync m16n8k16, the codes as the
// 16-row operand and up to 8 heads as the 8 columns (in a tcgen05 tile the converted codes would have to go back
// to shared memory, and its 128 rows would be heads, 4 of them real, or its smallest N twice these):
//   S^T = K Q^T: 16 keys x 16 dims of codes by q of the heads;
//   O^T = V^T P: 16 dims x 16 keys of codes by p, which is S^T's result transposed in registers (movmatrix).
// p enters in two fp16 halves (kv8_attn.cuh says how, at State).
// A block takes 1360 instructions of a warp as E4M3, 1560 as INT8, for up to 4 heads, 1700 as INT8 for up to 8.  (Heads as
// rows, zero-filled to 16, with p in two halves in the idle rows, took 1750: the multiplier's four-register operand was half zeros.)
// Codes become fp16 exactly and their scales multiply the fp32 sums, once per block: the scores by
// ks, the block's O by vs where it joins the running O.  E4M3 pairs are converted by one instruction;
// an INT8 code x as the byte x + 128 under the exponent of 1024, less 1152 (taking the 128 off the
// accumulators instead saves 2 of 5 instructions but not the bits that 128 sum p costs them: out was off by 2^-16
// of a block's largest value).  q as bf16 is first multiplied by a
// power of two that brings the row's largest element to 2^14 (exact but for elements 2^-28 of it).
//
// Work: the blocks of every (sequence, KV head, 8 heads) — an item — and its tail are laid end to end
// and cut into equal runs, one for each of 592 CTAs (four per SM), whatever the lengths; a CTA finds its
// run from the positions on the device, so a captured graph follows them.  Two of a CTA's four warps take a
// block, 32 keys each, every warp with its own running maximum, sum and O and its own stream of copies
// (kv8_attn.cuh).  At an item's end the four are joined in a fixed order; an item that lies in one CTA is finished
// there, pieces of a cut one go to the workspace and kv8_join_kernel finishes them (launched early, by
// programmatic dependent launch).  Results depend on positions and shapes alone.
// Calls whose items have few blocks go to kv8_direct.cu, which says at kv8_direct_plan where the border is and why.
// Measured on a B200 (6.47 TB/s as a copy): 64 sequences of 8K to 16K, 8 KV heads of 4, INT8, 1.62 GB: 282 to 285 us in a
// graph's replays, 5.7 TB/s, 88% of the copy rate, 279 to 300 as eager calls on different cards (a seventh more with two
// CTAs an SM).  One sequence of 64K: 51 us, where the bytes take 21: some 20 us are the start, the cut items' records and the
// join.
#include <cudaTypedefs.h>
#include <math.h>

#include "kv8_attn.cuh"

namespace zgcm {
int* library_error_word();  // zgcm_attn.cu: the site of an expired bounded wait
bool kv8_direct_plan(DecodeKv8Params& p, int units);   // kv8_direct.cu
cudaError_t kv8_direct_launch(const DecodeKv8Params& p, cudaStream_t stream);

namespace {

constexpr int DK_CTAS = 592;               // 148 SMs x 4
constexpr int DK_THREADS = 128;
constexpr int DK_POS = 64;                 // positions of the run's sequences kept in shared memory
constexpr int DK_REC = kD + 4;             // floats of a record's head: m, l, 2 pad, O
constexpr int DK_WAIT = 0x810;

struct Walk {
    int b, rest, off;   // sequence, item of it, unit of the item
};

struct DecodeSmem {
    alignas(1024) unsigned char ring[4][kSlots * kSlot];
    float acc[DK_HEADS][kD];
    float ml[4][DK_HEADS][2];
    WarpSmem warp[4];
    int pos[DK_POS];
    long long sum[4];
    Walk start, end;
    int abort;
};
static_assert(4 * (sizeof(DecodeSmem) + 1024 + 1024) <= 228 * 1024, "four CTAs per SM");

// ------------------------------------------------------------------ the walk over the units

struct Run {
    const DecodeKv8Params& p;
    const DecodeSmem& sm;
    __device__ __forceinline__ int pos(int b) const {
        const int i = b - sm.start.b;
        return i < DK_POS ? sm.pos[i] : p.pos[b];
    }
    // n units on (8-bit ones alone if `codes`); stays at the end when it runs past it
    template <bool codes> __device__ __forceinline__ void step(Walk& w, int n) const {
        w.off += n;
        const int items = p.c.Hkv * p.HT;
        while (w.b < p.c.B) {
            const int u = span_of(p, pos(w.b)).units - (codes ? 1 : 0);
            if (w.off < u) return;
            const int skip = u > 0 ? min(w.off / u, items - w.rest) : items - w.rest;
            w.off -= skip * u;
            w.rest += skip;
            if (w.rest < items) return;
            w.rest = 0;
            ++w.b;
        }
    }
};

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

// Sums over a block of 128 threads; `sum` [4] in shared memory.
__device__ __forceinline__ long long cta_sum(long long x, long long* sum) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sum[threadIdx.x >> 5] = x;
    __syncthreads();
    return sum[0] + sum[1] + sum[2] + sum[3];
}

// The run of this CTA, into sm.start and sm.end; returns its number of units.
__device__ __forceinline__ int find_run(const DecodeKv8Params& p, DecodeSmem& sm) {
    const int tid = threadIdx.x, lane = tid & 31, items = p.c.Hkv * p.HT;
    const int first = tid < p.c.B ? span_of(p, p.pos[tid]).units : 0;
    long long n = first;
    for (int b = tid + DK_THREADS; b < p.c.B; b += DK_THREADS) n += span_of(p, p.pos[b]).units;
    const long long total = cta_sum(n, sm.sum) * items;
    const long long lo = run_start(total, blockIdx.x), hi = run_start(total, blockIdx.x + 1);
    if (tid == 0) sm.start = sm.end = Walk{p.c.B, 0, 0};
    long long before = 0;   // units of the sequences before these 128
    for (int b0 = 0; b0 < p.c.B; b0 += DK_THREADS) {
        const int b = b0 + tid;
        const int u = b0 == 0 ? first : b < p.c.B ? span_of(p, p.pos[b]).units : 0;
        long long s = u;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, s, o);
            if (lane >= o) s += y;
        }
        __syncthreads();
        if (lane == 31) sm.sum[tid >> 5] = s;
        __syncthreads();
        long long at = before + s - u;
        for (int w = 0; w < (tid >> 5); ++w) at += sm.sum[w];
        before += sm.sum[0] + sm.sum[1] + sm.sum[2] + sm.sum[3];
        // this thread's sequence has units [at, at + u) * items
        if (u > 0) {
            const long long x = at * items, y = x + (long long)u * items;
            if (lo >= x && lo < y) sm.start = Walk{b, (int)((lo - x) / u), (int)((lo - x) % u)};
            if (hi >= x && hi < y) sm.end = Walk{b, (int)((hi - x) / u), (int)((hi - x) % u)};
        }
        if (before * items > hi) break;
    }
    __syncthreads();
    for (int i = tid; i < DK_POS; i += DK_THREADS)
        if (sm.start.b + i < p.c.B) sm.pos[i] = p.pos[sm.start.b + i];
    __syncthreads();
    return (int)(hi - lo);
}

__device__ __forceinline__ void warps_sync() { asm volatile("bar.sync 1, 128;" ::: "memory"); }

template <typename TK, int CODE, bool WIDE>
__global__ void __launch_bounds__(DK_THREADS, 4) kv8_decode_kernel(const __grid_constant__ DecodeKv8Params p) {
    extern __shared__ unsigned char raw[];
    DecodeSmem& sm = *reinterpret_cast<DecodeSmem*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~(uintptr_t)1023);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, r = lane >> 2, c = lane & 3;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");   // the join may take its place early
    if (lane == 0) {
        for (int i = 0; i < kSlots; ++i) mbar_init(&sm.warp[warp].full[i], 1);
        if (warp == 0) sm.abort = 0;
        fence_barrier_init();
    }
    const int units = find_run(p, sm);
    const Run run{p, sm};
    const int items = p.c.Hkv * p.HT, team = warp >> 1;
    // the 8-bit units of the run: all but the tails, one at the end of each item that ends in it
    const int n_codes = units - ((sm.end.b - sm.start.b) * items + sm.end.rest - sm.start.rest);
    const int blocks = (n_codes - team + 1) / 2;       // this pair's: every second one
    Walk ahead = sm.start;                             // the 8-bit unit `taken` of the run
    run.step<true>(ahead, 0);
    int taken = 0;
    auto fetch = [&](int batch) {                      // lane i: the pair's block 32 batch + i; batches in order
        run.step<true>(ahead, 64 * batch - taken);
        taken = 64 * batch;
        Walk w = ahead;
        run.step<true>(w, team + 2 * lane);
        if (32 * batch + lane >= blocks) return Block{-1, -1, 0.f, 0.f};
        return block_of(p, span_of(p, run.pos(w.b)), w.b, w.rest / p.HT, w.off);
    };
    Stream stream(p, sm.warp[warp], sm.ring[warp], &sm.abort);
    stream.mine = fetch(0);
    stream.start(blocks);

    Walk w = sm.start;
    int slot = 0, gave_up = 0;   // 8-bit units of the run so far
    for (int left = units; left > 0;) {
        const Span s = span_of(p, run.pos(w.b));
        const int n = min(s.units - w.off, left);                              // units of the item here
        const int n8 = max(0, min(w.off + n, s.units - 1) - w.off);
        const bool has_tail = w.off + n == s.units;
        const int kvh = w.rest / p.HT, ht = w.rest % p.HT;
        const int nh = min(DK_HEADS, p.G - ht * DK_HEADS);
        const size_t head = (size_t)w.b * p.Hq + (size_t)kvh * p.G + ht * DK_HEADS;       // the item's first
        const bool one = w.off == 0 && has_tail;                               // the whole item
        if (s.idle || s.bad) {
            if (warp == 0 && r < nh) no_answer(p, head + r, s.idle);
        } else {
            State t;
            uint32_t qt[8][2], q16[8][2];   // as they are, for the tail; as fp16, for codes
            load_q<TK, WIDE>(p, head, nh, qt);
            if (has_tail) {
                const int last = run.pos(w.b) - s.own * kBlk, first = s.lo - s.own * kBlk;
                if (warp * 16 <= last && warp * 16 + 15 >= first) {
                    Tail<TK, WIDE> tail;
                    tail.load(p, (size_t)w.b * p.c.Hkv + kvh, warp * 16);
                    tail.take(t, qt, p.scale_log2, warp * 16, first, last);
                }
            }
            const float2 qs = q_as_half<TK>(p, qt, q16);
            for (int i = (team - slot) & 1; i < n8; i += 2) {
                const int k = (slot + i) >> 1;
                if (stream.ok) gave_up = k;
                stream.take<CODE, WIDE>(t, q16, qs, s.lo, k, blocks, DK_WAIT, fetch);
            }
            // the four warps' parts, always added in the same order
            put_ml(t, sm.ml[warp]);
            warps_sync();
            float m, l;
            const float fx = join_ml(sm.ml, 2 * c, warp, m, l), fy = join_ml(sm.ml, 2 * c + 1, warp, m, l);
#pragma unroll
            for (int from = 3; from >= 0; --from) {
                if (warp == from) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        float2* x = reinterpret_cast<float2*>(&sm.acc[2 * c][16 * i + 2 * r]);
                        float2* y = reinterpret_cast<float2*>(&sm.acc[2 * c + 1][16 * i + 2 * r]);
                        float2 u = make_float2(t.o[i][0].x * fx, t.o[i][1].x * fx);
                        float2 v = make_float2(t.o[i][0].y * fy, t.o[i][1].y * fy);
                        if (from < 3) {
                            u = fadd2(u, *x);
                            v = fadd2(v, *y);
                        }
                        *x = u;
                        *y = v;
                    }
                }
                warps_sync();
            }
            // places of a head and 4 dims
            const size_t item = ((size_t)w.b * p.c.Hkv + kvh) * p.HT + ht;
#pragma unroll
            for (int i = 0; i < (WIDE ? 2 : 1); ++i) {
                const int h = (tid + DK_THREADS * i) >> 5, d = 4 * (tid & 31);
                if (h < nh) {
                    join_ml(sm.ml, h, 0, m, l);
                    float4 y = *reinterpret_cast<const float4*>(&sm.acc[h][d]);
                    if (!WIDE) {   // and what the low halves of p gave
                        const float4 z = *reinterpret_cast<const float4*>(&sm.acc[h + DK_HEADS / 2][d]);
                        y = make_float4(y.x + z.x, y.y + z.y, y.z + z.z, y.w + z.w);
                    }
                    const float o[4] = {y.x, y.y, y.z, y.w};
                    if (one) {
                        finish4(p, head + h, d, m, l, o, load_gate(p, head + h, d));
                    } else {
                        float* rec = p.part + ((item + blockIdx.x) * p.rows + h) * DK_REC;
                        if (d == 0) *reinterpret_cast<float2*>(rec) = make_float2(m, l);
                        *reinterpret_cast<float4*>(rec + 4 + d) = y;
                    }
                }
            }
            warps_sync();   // the next item may write what these have read
        }
        slot += n8;
        left -= n;
        run.step<false>(w, n);
    }
    stream.drain(gave_up, blocks);
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
    __shared__ long long sum[4];
    const int units = span_of(p, p.pos[b]).units;
    long long all = 0, before = 0;
    for (int i = threadIdx.x; i < p.c.B; i += 128) {
        const int u = span_of(p, p.pos[i]).units;
        all += u;
        if (i < b) before += u;
    }
    const long long total = cta_sum(all, sum) * items, start = cta_sum(before, sum) * items + (long long)rest * units;
    const int c0 = run_of(total, start), c1 = run_of(total, start + units - 1);
    asm volatile("griddepcontrol.wait;" ::: "memory");   // every block: the grid must not end before the records' writer
    if (c0 == c1 || ht * DK_HEADS + row >= p.G) return;
    const size_t head = (size_t)b * p.Hq + (size_t)kvh * p.G + ht * DK_HEADS + row;
    const uint2 gate = warp == 0 ? load_gate(p, head, 4 * lane) : make_uint2(0u, 0u);
    float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
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
    finish4(p, head, 4 * lane, mm, l, o, gate);
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
    cuuint32_t box[2] = {kD, kHalfKeys}, estr[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(codes), dims, strides, box, estr,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <typename TK, int CODE, bool WIDE> cudaError_t launch_kernels(const DecodeKv8Params& p, cudaStream_t stream) {
    const size_t smem = sizeof(DecodeSmem) + 1024;
    auto kernel = kv8_decode_kernel<TK, CODE, WIDE>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    kernel<<<DK_CTAS, DK_THREADS, smem, stream>>>(p);
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

template <typename TK, int CODE> cudaError_t launch(const DecodeKv8Params& p, cudaStream_t stream) {
    return p.G > DK_HEADS / 2 ? launch_kernels<TK, CODE, true>(p, stream) : launch_kernels<TK, CODE, false>(p, stream);
}

// Checks and the shape-dependent part of the parameters; n_list < 0: no list.
int plan(DecodeKv8Params& p, const zgcm_kv8_cache* cache, int Hq, int window, int n_list, bool* direct) {
    const int st = kv8_check(cache, &p.c);
    if (st != ZGCM_OK) return st;
    if (Hq < 1 || Hq % p.c.Hkv != 0 || window < 1) return ZGCM_ERR_INVALID_ARG;
    p.n_list = n_list < 0 ? 0 : n_list;
    p.Hq = Hq;
    p.G = Hq / p.c.Hkv;
    p.HT = (p.G + DK_HEADS - 1) / DK_HEADS;
    p.rows = p.G < DK_HEADS ? p.G : DK_HEADS;
    p.W = window;
    // items and their heads are counted in 32 bits (grids and records)
    if ((long long)p.c.B * p.c.Hkv * p.HT * DK_HEADS > 0x7fffffffLL || n_list > 0x7ffffffe) return ZGCM_ERR_UNSUPPORTED;
    // the most units of an item: a list's entries, or the blocks that a window can touch and the table hold
    const long long touched = ((long long)window - 1 + kBlk - 1) / kBlk + 1;
    *direct = kv8_direct_plan(p, n_list >= 0 ? n_list + 1 : (int)(touched < p.c.NB ? touched : p.c.NB));
    return ZGCM_OK;
}

size_t records_bytes(const DecodeKv8Params& p) {
    return ((size_t)p.c.B * p.c.Hkv * p.HT + DK_CTAS) * p.rows * DK_REC * sizeof(float);
}

}  // namespace
}  // namespace zgcm

using namespace zgcm;

extern "C" {

size_t zgcm_attn_decode_kv8_workspace_size(const zgcm_kv8_cache* cache, int Hq, int window, int n_list) {
    DecodeKv8Params p;
    bool direct;
    if (plan(p, cache, Hq, window, n_list < 0 ? -1 : n_list, &direct) != ZGCM_OK || p.c.B == 0 || direct) return 0;
    return records_bytes(p);
}

int zgcm_attn_decode_kv8(const zgcm_kv8_cache* cache, const void* q, const void* g, const int* pos, const int* blocks,
                         int n_list, int Hq, int window, float scale, void* out, float* lse, void* workspace,
                         size_t workspace_bytes, void* cuda_stream) {
    DecodeKv8Params p;
    bool direct;
    if (blocks && n_list < 0) return ZGCM_ERR_INVALID_ARG;
    const int st = plan(p, cache, Hq, window, blocks ? n_list : -1, &direct);
    if (st != ZGCM_OK) return st;
    if (!(scale > 0.f) || !isfinite(scale)) return ZGCM_ERR_INVALID_ARG;
    if (p.c.B == 0) return ZGCM_OK;
    if (!q || !pos || !out || !lse) return ZGCM_ERR_INVALID_ARG;
    if (((uintptr_t)q | (uintptr_t)g | (uintptr_t)pos | (uintptr_t)blocks | (uintptr_t)out | (uintptr_t)lse) & 15u)
        return ZGCM_ERR_ALIGNMENT;
    if (!direct) {
        if (!workspace || workspace_bytes < records_bytes(p)) return ZGCM_ERR_WORKSPACE;
        if ((uintptr_t)workspace & 15u) return ZGCM_ERR_ALIGNMENT;
    }
    p.q = q;
    p.g = static_cast<const bf16*>(g);
    p.pos = pos;
    p.blocks = blocks;
    p.scale_log2 = scale * kLog2e;
    p.out = static_cast<bf16*>(out);
    p.lse = lse;
    p.part = static_cast<float*>(workspace);
    p.err = library_error_word();
    if (!p.err) return ZGCM_ERR_CUDA;
    if (!make_map(&p.tm_k, p.c.kc, p.c) || !make_map(&p.tm_v, p.c.vc, p.c)) return ZGCM_ERR_CUDA;
    cudaStream_t stream = static_cast<cudaStream_t>(cuda_stream);
    const bool f8 = p.c.code == ZGCM_E4M3;
    if (direct) return kv8_direct_launch(p, stream) == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
    const cudaError_t e = p.c.key == ZGCM_BF16
                              ? (f8 ? launch<bf16, ZGCM_E4M3>(p, stream) : launch<bf16, ZGCM_INT8>(p, stream))
                              : (f8 ? launch<__half, ZGCM_E4M3>(p, stream) : launch<__half, ZGCM_INT8>(p, stream));
    return e == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}

}  // extern "C"
