// common.cuh -- device helpers shared by the fp8kv kernels (sm_103a).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <atomic>
#include <utility>

#include "../../include/fp8kv.h"

namespace fp8kv {

// Device status word of this translation unit (bits FP8KV_DEV_*); each .cu
// file has its own copy and a host reader, OR-ed by fp8kv_device_status.
static __device__ unsigned int g_status;

__device__ __forceinline__ void flag(unsigned int bits) { atomicOr(&g_status, bits); }

// ------------------------------------------------------------------ E4M3

// Two fp32 values -> two E4M3FN codes (lo in bits 0..7, hi in bits 8..15):
// round to nearest even, saturating to +-448 (infinities included) by the
// hardware conversion; NaN inputs become 0x7F with their own sign bit.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    uint32_t out = r;
    uint32_t bl = __float_as_uint(lo), bh = __float_as_uint(hi);
    if ((bl & 0x7fffffffu) > 0x7f800000u) out = (out & 0xff00u) | 0x7fu | ((bl >> 24) & 0x80u);
    if ((bh & 0x7fffffffu) > 0x7f800000u) out = (out & 0x00ffu) | ((0x7fu | ((bh >> 24) & 0x80u)) << 8);
    return out;
}

// Two E4M3 codes (bits 0..15) -> f16x2, exact (every E4M3 value is an f16).
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint32_t codes) {
    uint32_t r;
    uint16_t c = (uint16_t)codes;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
    return r;
}

// Two E4M3 codes (bits 0..15) -> two fp32 values, exact.
__device__ __forceinline__ void e4m3x2_to_f32x2(uint32_t codes, float& lo, float& hi) {
    const uint32_t h = e4m3x2_to_f16x2(codes);
    lo = __half2float(__ushort_as_half((unsigned short)(h & 0xffffu)));
    hi = __half2float(__ushort_as_half((unsigned short)(h >> 16)));
}

// f16x2 -> two E4M3 codes (bits 0..7 from the low half), round to nearest
// even, saturating; no NaN sign fix-up (for operands, not stored bytes).
__device__ __forceinline__ uint32_t f16x2_to_e4m3x2(uint32_t h) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f16x2 %0, %1;" : "=h"(r) : "r"(h));
    return r;
}

__device__ __forceinline__ float2 f16x2_to_f32x2(uint32_t h) {
    return make_float2(__half2float(__ushort_as_half((unsigned short)(h & 0xffffu))),
                       __half2float(__ushort_as_half((unsigned short)(h >> 16))));
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t sub_f16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Eight bf16 values (one 16-byte chunk) -> eight E4M3 codes of x / scale,
// each with one fp32 IEEE division (the cache-insert encoding).
__device__ __forceinline__ uint2 e4m3_encode8(uint4 x, float scale) {
    uint2 o;
    o.x = e4m3x2(__fdiv_rn(bf16_lo(x.x), scale), __fdiv_rn(bf16_hi(x.x), scale)) |
          (e4m3x2(__fdiv_rn(bf16_lo(x.y), scale), __fdiv_rn(bf16_hi(x.y), scale)) << 16);
    o.y = e4m3x2(__fdiv_rn(bf16_lo(x.z), scale), __fdiv_rn(bf16_hi(x.z), scale)) |
          (e4m3x2(__fdiv_rn(bf16_lo(x.w), scale), __fdiv_rn(bf16_hi(x.w), scale)) << 16);
    return o;
}

// ------------------------------------------------------------------ INT4
//
// A page of one head of an INT4 cache: page_size rows of 64 code bytes, then
// page_size rows of 8 scale bytes (include/fp8kv.h).
constexpr int kInt4CodeBytes = 64, kInt4ScaleBytes = 8, kInt4RowBytes = kInt4CodeBytes + kInt4ScaleBytes;

// 16 bf16 values (one block) -> 8 bytes of 4-bit codes and the E4M3 scale
// code, with the tensor scale c and fp32 roundings throughout:
//     s = max(e4m3(amax / (7 c)), 2^-9),  n = clamp(rint(x * (1 / (s c))), -7, 7)
// The maximum is taken over the bit patterns, where NaN is above infinity: a
// NaN anywhere makes the block's scale NaN (and its codes n = 0).
__device__ __forceinline__ uint2 int4_encode16(uint4 a, uint4 b, float c, uint8_t& scale_code) {
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t m2 = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, w[i] & 0x7fff7fffu);
    const float amax = __uint_as_float(max(m2 & 0xffffu, m2 >> 16) << 16);
    const float r = __fdiv_rn(amax, __fmul_rn(7.0f, c));
    const uint32_t sc = max(e4m3x2(r, 0.0f) & 0xffu, 1u);       // >= 2^-9; NaN is 0x7f
    scale_code = (uint8_t)sc;
    if (sc == 0x7fu) return make_uint2(0x88888888u, 0x88888888u);
    float s, unused;
    e4m3x2_to_f32x2(sc, s, unused);
    const float inv = __frcp_rn(__fmul_rn(s, c));
    // n + 8 in the low mantissa bits of 2^23 + 8 + n (the addition rounds to
    // the nearest integer, ties to even); the words' sum of 16^e times those
    // bits is the codes' word plus 16^e times 2^23's bits, 0xfb000000 in all
    uint32_t o[2];
    auto codes = [&](bool clamp) {
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t acc = 0;
#pragma unroll
            for (int e = 7; e >= 0; --e) {
                const uint32_t x = w[4 * u + (e >> 1)];
                float t = __fmul_rn(e & 1 ? bf16_hi(x) : bf16_lo(x), inv);
                if (clamp) t = fminf(fmaxf(t, -7.0f), 7.0f);
                acc = acc * 16u + __float_as_uint(__fadd_rn(t, 8388616.0f));
            }
            o[u] = acc - 0xfb000000u;
        }
    };
    // A scale that was rounded to a normal E4M3 number, without saturating, is
    // at least amax / (7 c) / (1 + 2^-4): |x inv| stays below 7.44, which rounds
    // to 7, and the clamps (a third of the instructions) can go.
    if (sc >= 8u && r <= 448.0f) codes(false);
    else codes(true);
    return make_uint2(o[0], o[1]);
}

__device__ __forceinline__ uint32_t prmt(uint32_t a, uint32_t b, uint32_t sel) {
    uint32_t r;
    asm("prmt.b32 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(sel));
    return r;
}

// 2^x on the special-function unit (the hardware ex2 instruction).
__device__ __forceinline__ float ex2(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// Pairs of fp32 values in one 64-bit register, for the packed fma and add.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ void unpack2(uint64_t v, float& lo, float& hi) {
    asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v));
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// One thread of the (converged) warp, the same one every time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{ .reg .pred p; elect.sync _|p, 0xffffffff; selp.u32 %0, 1, 0, p; }" : "=r"(r));
    return r != 0;
}

// ------------------------------------------------------------ tensor core

// D += A * B, m16n8k16, fp32 accumulate; A row-major, B column-major.
__device__ __forceinline__ void mma_f16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// D = A * B, m16n8k16.
__device__ __forceinline__ void mma_f16_zero(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.0f));
}

// D += A * B, m16n8k32, E4M3 x E4M3, fp32 accumulate; A row-major, B
// column-major; each register holds four consecutive k elements.
__device__ __forceinline__ void mma_e4m3(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
    asm(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// ------------------------------------------------------ mbarrier and TMA

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void fence_barrier_init() {
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes)
                 : "memory");
}

__device__ __forceinline__ uint64_t globaltimer() {
    uint64_t t;
    asm volatile("mov.u64 %0, %globaltimer;" : "=l"(t));
    return t;
}

// Wait for the phase with parity `phase` of an mbarrier to complete.  Gives up
// after `limit_ns` of wall time (2 s unless a caller asks otherwise; sets
// FP8KV_DEV_WAIT_TIMEOUT and returns false) so a broken pipeline can never
// hang the GPU.
__device__ __forceinline__ bool mbar_wait(uint32_t bar, uint32_t phase, uint64_t limit_ns = 2000000000ull) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    if (ok) return true;
    const uint64_t start = globaltimer();
    while (true) {
        // suspends until the phase completes or 0.5 ms pass: no hot spinning
        asm volatile(
            "{ .reg .pred p; mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3; selp.u32 %0, 1, 0, p; }"
            : "=r"(ok)
            : "r"(bar), "r"(phase), "r"(500000u)
            : "memory");
        if (ok) return true;
        if (globaltimer() - start > limit_ns) {
            flag(FP8KV_DEV_WAIT_TIMEOUT);
            return false;
        }
    }
}

// Non-blocking test: has the phase with parity `phase` of an mbarrier completed?
__device__ __forceinline__ bool mbar_test(uint32_t bar, uint32_t phase) {
    uint32_t ok;
    asm volatile(
        "{ .reg .pred p; mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2; selp.u32 %0, 1, 0, p; }"
        : "=r"(ok)
        : "r"(bar), "r"(phase)
        : "memory");
    return ok != 0;
}

// 3-D tiled TMA load global -> shared, completion counted on `bar` in bytes.
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* tm, int x, int y, int z,
                                            uint32_t bar, uint64_t policy) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4}], [%5], %6;" ::"r"(dst),
        "l"(tm), "r"(x), "r"(y), "r"(z), "r"(bar), "l"(policy)
        : "memory");
}

// Bulk copy of `bytes` (a multiple of 16; both addresses 16-byte aligned)
// from this CTA's shared memory to global memory, tracked as a bulk group.
__device__ __forceinline__ void bulk_store(void* gdst, uint32_t ssrc, uint32_t bytes) {
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(gdst), "r"(ssrc), "r"(bytes)
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
// Wait until every committed bulk group has finished reading shared memory.
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }

__device__ __forceinline__ uint64_t policy_evict_last() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ uint64_t policy_evict_first() {
    uint64_t p;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

// Programmatic dependent launch: let the next kernel in the stream start its
// prologue now; and, before touching any global input, wait until every
// kernel this one depends on has completed and its writes are visible.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap* tm) {
    asm volatile("prefetch.tensormap [%0];" ::"l"(tm) : "memory");
}

}  // namespace fp8kv

// Host-side helpers (api.cu).
namespace fp8kv {
// Counts every kernel launch the library makes (api.cu; fp8kv_launch_count).
void count_launch();

// Launch with programmatic stream serialization: the kernel may start while
// the previous kernel in the stream is finishing; it must call pdl_wait()
// before reading anything that kernel may have written.  cluster_x > 1
// groups that many consecutive CTAs along x into one thread-block cluster.
template <typename... KArgs, typename... Args>
static inline cudaError_t launch_pdl_cluster(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                             cudaStream_t stream, int cluster_x, Args&&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster_x > 1 ? cluster_x : 1;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster_x > 1 ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    if (e == cudaSuccess) count_launch();
    return e;
}

template <typename... KArgs, typename... Args>
static inline cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem,
                                     cudaStream_t stream, Args&&... args) {
    return launch_pdl_cluster(kernel, grid, block, smem, stream, 1, std::forward<Args>(args)...);
}

// Opt in to a kernel's dynamic shared memory, once per device (`done`: a bit for
// each of the first 64; without a lock, as repeating it does no harm), so that
// calls under capture issue no attribute change.
static inline cudaError_t opt_in_smem(std::atomic<uint64_t>& done, const void* kernel, int bytes) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

// ------------------------------------------------ thread-block clusters

// The address of the same shared-memory object in cluster CTA `rank`.
__device__ __forceinline__ uint32_t dsmem_addr(const void* p, int rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
// Bulk copy of `bytes` (a multiple of 16; both addresses 16-byte aligned)
// from this CTA's shared memory to shared memory of a CTA of the cluster
// (`dst`, `mbar`: addresses from dsmem_addr); the copy's bytes complete a
// transaction on that CTA's mbarrier `mbar`.  The source must stay unchanged
// until the receiver has seen the bytes arrive.
__device__ __forceinline__ void bulk_copy_to_cluster(uint32_t dst, uint32_t src, uint32_t bytes, uint32_t mbar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(src), "r"(bytes), "r"(mbar)
                 : "memory");
}
// Split cluster barrier, executed by every thread of every CTA of the
// cluster (warp-aligned): arrive without ordering, then wait (acquire).
// A fence.mbarrier_init before the arrive publishes barrier initialisation.
__device__ __forceinline__ void cluster_arrive_relaxed() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}
// The same, publishing this thread's writes to shared memory.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
// Reads of a cluster CTA's shared memory (addresses from dsmem_addr).
__device__ __forceinline__ uint4 dsmem_ld16(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ float2 dsmem_ld8(uint32_t a) {
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// two ranges of bytes (host)
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

int launch_status();                    // FP8KV_OK or FP8KV_ERR_CUDA after a launch
int num_sms();                          // SM count of the current device
void set_dispatch(const char* text);    // per-thread record of the last dispatch
int status_insert(unsigned int* s, int clear);     // insert.cu
int status_attention(unsigned int* s, int clear);  // attention.cu
int status_attention_int4(unsigned int* s, int clear);  // attention_int4.cu
int status_attention_int4_tc(unsigned int* s, int clear);  // attention_int4_tc.cu
int status_prompt(unsigned int* s, int clear);     // prompt_attention.cu
int status_draft_tree(unsigned int* s, int clear);   // draft_tree.cu
int status_rope_insert(unsigned int* s, int clear);  // rope_insert.cu
int status_verify_tree(unsigned int* s, int clear);  // verify_tree.cu
int status_attention_tree_tc(unsigned int* s, int clear);  // attention_tree_tc.cu

// OR this translation unit's status word into *s, optionally clearing it.
static inline int read_status(unsigned int* s, int clear) {
    unsigned int v = 0;
    if (cudaMemcpyFromSymbol(&v, g_status, sizeof(v)) != cudaSuccess) return FP8KV_ERR_CUDA;
    if (clear) {
        const unsigned int z = 0;
        if (cudaMemcpyToSymbol(g_status, &z, sizeof(z)) != cudaSuccess) return FP8KV_ERR_CUDA;
    }
    *s |= v;
    return FP8KV_OK;
}
}  // namespace fp8kv
