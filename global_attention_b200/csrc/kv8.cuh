// kv8.cuh — the 8-bit block cache (include/zgcm_kv8.h) as its kernels see it.
#pragma once
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "zgcm_kv8.h"

namespace zgcm {

constexpr int kBlk = ZGCM_KV8_BLOCK;         // tokens of a block
constexpr int kBlkBytes = kBlk * kD;         // bytes of one head's codes in a page
constexpr int kKv8MaxBlocks = 16384;         // zgcm_kv8_select: scores of a sequence's blocks in shared memory

struct Kv8 {
    uint8_t* kc;
    uint8_t* vc;
    float* ks;
    float* vs;
    char* kmean;
    char* ktail;
    bf16* vtail;
    const int* table;
    int B, NB, P, Hkv;
    int code, key;   // zgcm_code_type, zgcm_dtype
};

// page of block j of sequence b, or -1 when the table holds a number outside the cache
__device__ __forceinline__ int kv8_page(const Kv8& c, int b, int j) {
    const int p = c.table[(size_t)b * c.NB + (j < c.NB ? j : j % c.NB)];   // a ring's blocks alone pay for the division
    return (unsigned)p < (unsigned)c.P ? p : -1;
}

// the value of a 16-bit type's bits
template <typename T> __device__ __forceinline__ float from_bits(uint32_t b);
template <> __device__ __forceinline__ float from_bits<bf16>(uint32_t b) { return __uint_as_float(b << 16); }
template <> __device__ __forceinline__ float from_bits<__half>(uint32_t b) {
    return __half2float(__ushort_as_half((unsigned short)b));
}

// checks of a cache; ZGCM_OK with *out filled
int kv8_check(const zgcm_kv8_cache* c, Kv8* out);

}  // namespace zgcm
