// int4.cuh -- writing the INT4 cache's rows, and widening its codes, shared by
// its kernels (the arithmetic is explained at the head of attention_int4.cu).
#pragma once
#include <stdint.h>

#include "attention.cuh"
#include "common.cuh"

namespace fp8kv {

__device__ __forceinline__ uint32_t hfma2(uint32_t a, uint32_t b, uint32_t c) {
    uint32_t r;
    asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
    return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// The four codes of each half word of z times the scales of s (f16x2, one per
// half word) over 4: v[i] = the i-th codes' values n s / 4.
struct Scale2 {
    uint32_t s, c256, c16;      // s / 4, -264 s / 4, -24 s / 4
};
__device__ __forceinline__ Scale2 scale2(uint32_t s) {
    return {hmul2(s, 0x34003400u), hmul2(s, 0xd420d420u), hmul2(s, 0xc600c600u)};
}
// (z & mask) | base as one instruction: written with the operators it becomes
// two, 39 arithmetic-logic operations for 32 codes instead of 24.
__device__ __forceinline__ uint32_t and_or(uint32_t z, uint32_t mask, uint32_t base) {
    uint32_t r;
    asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(r) : "r"(z), "r"(mask), "r"(base));
    return r;
}
__device__ __forceinline__ void widen4(uint32_t z, const Scale2& k, uint32_t (&v)[4]) {
    const uint32_t x = z << 2, y = z >> 6;
    v[0] = hfma2(and_or(x, 0x003c003cu, 0x5c005c00u), k.s, k.c256);
    v[1] = hfma2(and_or(x, 0x03c003c0u, 0x4c004c00u), k.s, k.c16);
    v[2] = hfma2(and_or(y, 0x003c003cu, 0x5c005c00u), k.s, k.c256);
    v[3] = hfma2(and_or(y, 0x03c003c0u, 0x4c004c00u), k.s, k.c16);
}

// One block of 16 elements of K and of V: 8 code bytes and one scale byte each.
struct Int4Block {
    uint2 k, v;
    uint8_t ks, vs;
    Int4Block() = default;
    __device__ __forceinline__ Int4Block(uint4 k0, uint4 k1, uint4 v0, uint4 v1, float kc, float vc) {
        k = int4_encode16(k0, k1, kc, ks);
        v = int4_encode16(v0, v1, vc, vs);
    }
    // into row `off` of (page, head) of the caches
    __device__ __forceinline__ void store(uint8_t* __restrict__ k_cache, uint8_t* __restrict__ v_cache, int64_t page,
                                          int off, int h, int Hkv, int page_size, int block) const {
        const int64_t base = (page * Hkv + h) * page_size * kInt4RowBytes;
        const int64_t code = base + off * kInt4CodeBytes + block * 8;
        const int64_t scale = base + page_size * kInt4CodeBytes + off * kInt4ScaleBytes + block;
        *reinterpret_cast<uint2*>(k_cache + code) = k;
        *reinterpret_cast<uint2*>(v_cache + code) = v;
        k_cache[scale] = ks;
        v_cache[scale] = vs;
    }
};

}  // namespace fp8kv
