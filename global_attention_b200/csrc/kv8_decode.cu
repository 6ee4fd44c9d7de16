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
// ks, the block's O by vs where it joins the running O.  E4M3 pairs are converted by one instruction;
// an INT8 code x as the byte x + 128 under the exponent of 1024, less 1152 (taking the 128 off the
// accumulators instead saves 2 of 5 instructions but not the bits that 128 sum p costs them: out was off by 2^-16
// of a block's largest value).  q as bf16 is first multiplied by a
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

#include "kv8_attn.cuh"

namespace zgcm {
int* library_error_word();  // zgcm_attn.cu: the site of an expired bounded wait
bool kv8_direct_plan(DecodeKv8Params& p, int units);   // kv8_direct.cu
cudaError_t kv8_direct_launch(const DecodeKv8Params& p, cudaStream_t stream);

namespace {

constexpr int DK_CTAS = 296;               // 148 SMs x 2
constexpr int DK_WARPS = 4;                // warps that compute; one more loads
constexpr int DK_THREADS = (DK_WARPS + 1) * 32;
constexpr int DK_STAGES = 6;
constexpr int DK_POS = 64;                 // positions of the run's sequences kept in shared memory
constexpr int DK_REC = kD + 4;             // floats of a record's head: m, l, 2 pad, O
constexpr int DK_WAIT_LOAD = 0x810, DK_WAIT_RING = 0x811;

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
        Tile tile{-1, -1, 0.f, 0.f};
        bool is8 = false;
        int kvh = 0;
        if (x + lane < hi) {
            const Span s = span_of(p, run.pos(w.b));
            is8 = w.off < s.units - 1;
            kvh = w.rest / p.HT;
            if (is8) tile = tile_of(p, s, w.b, kvh, w.off);
        }
        const uint32_t all = __ballot_sync(0xffffffffu, is8);
        for (uint32_t left = all; left; left &= left - 1, ++slot) {
            const int st = slot % DK_STAGES;
            if (lane == __ffs(left) - 1) {
                if (slot >= DK_STAGES && !mbar_wait(&sm.empty[st], (slot / DK_STAGES - 1) & 1, &sm.abort, DK_WAIT_RING))
                    ok = false;
                if (ok) {
                    sm.meta[st] = Meta{tile.ks, tile.vs, tile.j, 0};
                    if (tile.page >= 0) {
                        const int row = (tile.page * p.c.Hkv + kvh) * kBlk;
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
        for (int i = 0; i < 8; ++i) t.e[i] = t.o[i] = make_float2(0.f, 0.f);
        if (s.idle || s.bad) {
            if (warp == 0 && r < nh) no_answer(p, head, s.idle);
        } else {
            uint32_t qt[8][2], q16[8][2];   // as they are, for the tail; as fp16, for codes
            load_q<TK>(p, head, r < nh, qt);
            const float qs = q_as_half<TK>(p, qt, q16);
            for (int i = ((warp >> 1) - slot) & 1; i < n8; i += 2) {
                const int sl = slot + i, st = sl % DK_STAGES;
                if (mbar_wait(&sm.full[st], (sl / DK_STAGES) & 1, &sm.abort, DK_WAIT_LOAD)) {
                    const Meta meta = sm.meta[st];
                    if (meta.j >= 0)
                        block8<CODE>(t, q16, qs, smem_u32(sm.k[st]), smem_u32(sm.v[st]), meta, s.lo, (warp & 1) * 32);
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
            const float2 ff = make_float2(f, f);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                t.e[i] = fmul2(t.e[i], ff);
                t.o[i] = fmul2(t.o[i], ff);
            }
            if (warp >= 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    *reinterpret_cast<float4*>(&sm.acc[warp - 2][r][16 * i + 4 * c]) =
                        make_float4(t.e[i].x, t.o[i].x, t.e[i].y, t.o[i].y);
            }
            warps_sync();
            if (warp < 2) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    float4* a = reinterpret_cast<float4*>(&sm.acc[warp][r][16 * i + 4 * c]);
                    const float4 y = *a;
                    t.e[i] = fadd2(t.e[i], make_float2(y.x, y.z));
                    t.o[i] = fadd2(t.o[i], make_float2(y.y, y.w));
                    if (warp == 1) *a = make_float4(t.e[i].x, t.o[i].x, t.e[i].y, t.o[i].y);
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
                    const float o[4] = {t.e[i].x + y.x, t.o[i].x + y.y, t.e[i].y + y.z, t.o[i].y + y.w};
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
                mbar_init(&sm.empty[i], 2);
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
    // the most units of an item: a list's entries, or the blocks that a window can touch and the table hold
    const long long touched = ((long long)window - 1 + kBlk - 1) / kBlk + 1;
    if (kv8_direct_plan(p, blocks ? p.n_list + 1 : (int)(touched < p.c.NB ? touched : p.c.NB)))
        return kv8_direct_launch(p, stream) == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
    const cudaError_t e = p.c.key == ZGCM_BF16
                              ? (f8 ? launch<bf16, ZGCM_E4M3>(p, stream) : launch<bf16, ZGCM_INT8>(p, stream))
                              : (f8 ? launch<__half, ZGCM_E4M3>(p, stream) : launch<__half, ZGCM_INT8>(p, stream));
    return e == cudaSuccess ? ZGCM_OK : ZGCM_ERR_CUDA;
}

}  // extern "C"
