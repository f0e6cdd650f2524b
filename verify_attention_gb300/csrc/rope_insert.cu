// rope_insert.cu -- rotary positions on Q and K, and K and V into the paged
// cache, in one pass over the rows that the projection produced.
//
// With the table row of a token's position, c_k and s_k (k < rot / 2), a pair
// (x_k, y_k) of a head's first rot elements turns by its angle:
//     x' = bf16(fma(x, c, -(y s)))      y' = bf16(fma(y, c, x s))
// the pairs being elements (k, k + rot / 2), or (2 k, 2 k + 1) interleaved; the
// rest of the head stays.  Angles that are scaled for long contexts, and a
// factor on all of them, are in the table.
//
// HBM bounds it: a row of 256 bytes is read and written once, the table row of a
// token is read once for its heads.  A half warp takes one K and V head of a token,
// or QH heads of its Q, a thread four pairs of each (or eight elements behind rot),
// so that position and table row are in registers for all of them and every row's
// load is in flight before the first is needed.  The K blocks are spread over the
// grid, their encoding beside the others' loads (16381 tokens, INT4: 105 us, all K
// blocks first 113).  K rows pass through shared memory, as a thread encodes eight (INT4: sixteen)
// neighbouring elements, whatever the pairs were.
#include "attention.cuh"
#include "common.cuh"
#include "int4.cuh"

namespace fp8kv {

int status_rope_insert(unsigned int* s, int clear) { return read_status(s, clear); }

// Heads of Q a half warp takes: 16381 tokens of 72 + 8 heads, INT4: 2 heads 119 us, 4
// 105 (6.6 TB/s), 8 109.
constexpr int kRopeHeads = 4;

struct RopeParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;       // elements a token
    const int64_t *positions, *slots;
    const float* cos_sin;
    const float *k_scale, *v_scale;
    uint16_t* q_out;
    uint8_t *k_cache, *v_cache;
    int64_t num_slots;
    int max_pos, rot, T, Hq, Hkv, page_size;
    int groups;                 // of QH heads of Q, a token
    unsigned k_blocks, k_every;
};

// A thread's eight elements of a row: runs of four at a and b, which turn as pairs
// (or, PAIRS, hold them as neighbours), or stay.
struct RopeLane {
    int a, b;
    bool turns;
    float c[4], s[4];
    template <bool PAIRS>
    __device__ __forceinline__ static RopeLane at(int i, int rot) {
        RopeLane l;
        l.turns = 8 * i < rot;
        l.a = PAIRS || !l.turns ? 8 * i : 4 * i;
        l.b = PAIRS || !l.turns ? 8 * i + 4 : rot / 2 + 4 * i;
        return l;
    }
    __device__ __forceinline__ void angles(const float* cos_sin, int64_t pos, int rot, int i) {
        if (!turns) return;
        const float* row = cos_sin + pos * rot + 4 * i;
        *reinterpret_cast<float4*>(c) = __ldg(reinterpret_cast<const float4*>(row));
        *reinterpret_cast<float4*>(s) = __ldg(reinterpret_cast<const float4*>(row + rot / 2));
    }
    template <bool PAIRS>
    __device__ __forceinline__ void turn(uint2& xa, uint2& xb) const {
        if (!turns) return;
        const uint32_t w[4] = {xa.x, xa.y, xb.x, xb.y};
        float r[8];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            // pair j: (x, y)
            const uint32_t wx = PAIRS ? w[j] : w[j >> 1], wy = PAIRS ? w[j] : w[2 + (j >> 1)];
            const float x = !PAIRS && (j & 1) ? bf16_hi(wx) : bf16_lo(wx);
            const float y = PAIRS || (j & 1) ? bf16_hi(wy) : bf16_lo(wy);
            r[PAIRS ? 2 * j : j] = __fmaf_rn(x, c[j], -__fmul_rn(y, s[j]));
            r[PAIRS ? 2 * j + 1 : 4 + j] = __fmaf_rn(y, c[j], __fmul_rn(x, s[j]));
        }
        xa = make_uint2(pack_bf16x2(r[0], r[1]), pack_bf16x2(r[2], r[3]));
        xb = make_uint2(pack_bf16x2(r[4], r[5]), pack_bf16x2(r[6], r[7]));
    }
};

template <int DT, bool PAIRS>
__global__ void __launch_bounds__(256) rope_insert_kernel(RopeParams P) {
    constexpr int QH = kRopeHeads;
    __shared__ __align__(16) uint16_t rows[16][128 + 8];
    pdl_launch_dependents();
    const int half = threadIdx.x >> 4, i = threadIdx.x & 15;
    RopeLane lane = RopeLane::at<PAIRS>(i, P.rot);
    pdl_wait();
    // every P.k_every-th block is one of K and V, while there are any
    const unsigned kb = blockIdx.x / P.k_every;
    if (blockIdx.x != kb * P.k_every || kb >= P.k_blocks) {
        // ------------------------------------------------------------------- Q
        const int64_t unit = (int64_t)(blockIdx.x - min(P.k_blocks, kb + 1)) * 16 + half;
        const int64_t t = unit / P.groups;
        if (t >= P.T) return;
        const int h0 = (int)(unit - t * P.groups) * QH;
        const int64_t pos = P.positions[t];
        const uint16_t* src = P.q + t * P.q_stride + h0 * 128;
        uint2 xa[QH], xb[QH];
#pragma unroll
        for (int u = 0; u < QH; ++u) {
            if (h0 + u >= P.Hq) break;
            xa[u] = __ldcs(reinterpret_cast<const uint2*>(src + u * 128 + lane.a));
            xb[u] = __ldcs(reinterpret_cast<const uint2*>(src + u * 128 + lane.b));
        }
        if (pos < 0 || pos >= P.max_pos) return;            // (flagged by the K blocks)
        lane.angles(P.cos_sin, pos, P.rot, i);
        uint16_t* dst = P.q_out + (t * P.Hq + h0) * 128;
#pragma unroll
        for (int u = 0; u < QH; ++u) {
            if (h0 + u >= P.Hq) break;
            lane.turn<PAIRS>(xa[u], xb[u]);
            *reinterpret_cast<uint2*>(dst + u * 128 + lane.a) = xa[u];
            *reinterpret_cast<uint2*>(dst + u * 128 + lane.b) = xb[u];
        }
        return;
    }
    // ------------------------------------------------------------------- K and V
    const int64_t unit = (int64_t)kb * 16 + half;
    const bool in = unit < (int64_t)P.T * P.Hkv;
    const int64_t t = in ? unit / P.Hkv : 0;
    const int h = in ? (int)(unit - t * P.Hkv) : 0;
    // INT4: threads 0-7 take the blocks of K, 8-15 those of V
    const bool v_too = DT != FP8KV_CACHE_INT4 || i >= 8;
    const int64_t pos = P.positions[t], slot = P.slots[t];
    const uint16_t* src = P.k + t * P.k_stride + h * 128;
    uint2 xa = *reinterpret_cast<const uint2*>(src + lane.a), xb = *reinterpret_cast<const uint2*>(src + lane.b);
    const uint4* vrow = reinterpret_cast<const uint4*>(P.v + t * P.v_stride + h * 128);
    uint4 v[2] = {};
    if (DT == FP8KV_CACHE_INT4) {
        if (v_too) {
            v[0] = vrow[2 * (i & 7)];
            v[1] = vrow[2 * (i & 7) + 1];
        }
    } else {
        v[0] = vrow[i];
    }
    const float ks = DT == FP8KV_CACHE_BF16 ? 1.f : *P.k_scale, vs = DT == FP8KV_CACHE_BF16 ? 1.f : *P.v_scale;
    const bool pos_ok = pos >= 0 && pos < P.max_pos;
    if (in && i == 0 && h == 0) {
        if (!pos_ok) flag(FP8KV_DEV_BAD_POSITION);
        else if (slot >= P.num_slots) flag(FP8KV_DEV_BAD_SLOT);
    }
    const bool stores = in && pos_ok && slot >= 0 && slot < P.num_slots;
    if (stores) {
        lane.angles(P.cos_sin, pos, P.rot, i);
        lane.turn<PAIRS>(xa, xb);
        *reinterpret_cast<uint2*>(&rows[half][lane.a]) = xa;
        *reinterpret_cast<uint2*>(&rows[half][lane.b]) = xb;
    }
    __syncwarp();
    if (!stores) return;
    const int64_t page = slot >> (P.page_size == 64 ? 6 : 5);
    const int off = (int)slot & (P.page_size - 1);
    const uint4* krow = reinterpret_cast<const uint4*>(rows[half]);
    if (DT == FP8KV_CACHE_INT4) {
        const int block = i & 7;
        uint8_t sc;
        const uint2 codes = int4_encode16(v_too ? v[0] : krow[2 * block], v_too ? v[1] : krow[2 * block + 1],
                                          v_too ? vs : ks, sc);
        uint8_t* cache = (v_too ? P.v_cache : P.k_cache) + (page * P.Hkv + h) * P.page_size * kInt4RowBytes;
        *reinterpret_cast<uint2*>(cache + off * kInt4CodeBytes + block * 8) = codes;
        cache[P.page_size * kInt4CodeBytes + off * kInt4ScaleBytes + block] = sc;
    } else {
        const int64_t at = ((page * P.Hkv + h) * P.page_size + off) * 128 + 8 * i;
        if (DT == FP8KV_CACHE_E4M3) {
            *reinterpret_cast<uint2*>(P.k_cache + at) = e4m3_encode8(krow[i], ks);
            *reinterpret_cast<uint2*>(P.v_cache + at) = e4m3_encode8(v[0], vs);
        } else {
            *reinterpret_cast<uint4*>(P.k_cache + 2 * at) = krow[i];
            *reinterpret_cast<uint4*>(P.v_cache + 2 * at) = v[0];
        }
    }
}

template <int DT>
static cudaError_t launch_rope(const RopeParams& P, bool pairs, unsigned blocks, cudaStream_t s) {
    auto kern = pairs ? rope_insert_kernel<DT, true> : rope_insert_kernel<DT, false>;
    return launch_pdl(kern, dim3(blocks), dim3(256), 0, s, P);
}

}  // namespace fp8kv

using namespace fp8kv;

extern "C" int fp8kv_rope_insert(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                 int64_t v_stride, const int64_t* positions, const float* cos_sin, int max_pos,
                                 int rot_dim, int interleaved, void* q_out, const int64_t* slot_mapping, int T, int Hq,
                                 int Hkv, int D, const float* k_scale, const float* v_scale, void* k_cache,
                                 void* v_cache, int num_pages, int page_size, int cache_dtype, void* stream) {
    if (T < 0 || Hq <= 0 || Hkv <= 0 || num_pages <= 0 || max_pos <= 0 || rot_dim < 2 || rot_dim > D || rot_dim % 2)
        return FP8KV_ERR_INVALID_ARG;
    if (cache_dtype != FP8KV_CACHE_E4M3 && cache_dtype != FP8KV_CACHE_BF16 && cache_dtype != FP8KV_CACHE_INT4)
        return FP8KV_ERR_INVALID_ARG;
    if (D != 128 || rot_dim % 8 || (page_size != 32 && page_size != 64)) return FP8KV_ERR_UNSUPPORTED;
    if (q_stride < (int64_t)Hq * D || k_stride < (int64_t)Hkv * D || v_stride < (int64_t)Hkv * D || q_stride % 8 ||
        k_stride % 8 || v_stride % 8)
        return FP8KV_ERR_INVALID_ARG;
    if (T == 0) return FP8KV_OK;                                // nothing to do; no pointer is read
    if (!q || !k || !v || !positions || !cos_sin || !q_out || !slot_mapping || !k_cache || !v_cache)
        return FP8KV_ERR_INVALID_ARG;
    if (cache_dtype != FP8KV_CACHE_BF16 && (!k_scale || !v_scale)) return FP8KV_ERR_INVALID_ARG;
    for (const void* p : {q, k, v, (const void*)cos_sin, (const void*)q_out, (const void*)k_cache, (const void*)v_cache})
        if (reinterpret_cast<uintptr_t>(p) & 15) return FP8KV_ERR_INVALID_ARG;
    // rows are read while others are written
    const size_t out_bytes = (size_t)T * Hq * D * 2, k_row = (size_t)Hkv * D * 2;
    if (overlap(q_out, out_bytes, q, (size_t)(T - 1) * q_stride * 2 + (size_t)Hq * D * 2) ||
        overlap(q_out, out_bytes, k, (size_t)(T - 1) * k_stride * 2 + k_row) ||
        overlap(q_out, out_bytes, v, (size_t)(T - 1) * v_stride * 2 + k_row))
        return FP8KV_ERR_INVALID_ARG;
    RopeParams P;
    P.q = (const uint16_t*)q;
    P.k = (const uint16_t*)k;
    P.v = (const uint16_t*)v;
    P.q_stride = q_stride;
    P.k_stride = k_stride;
    P.v_stride = v_stride;
    P.positions = positions;
    P.slots = slot_mapping;
    P.cos_sin = cos_sin;
    P.k_scale = k_scale;
    P.v_scale = v_scale;
    P.q_out = (uint16_t*)q_out;
    P.k_cache = (uint8_t*)k_cache;
    P.v_cache = (uint8_t*)v_cache;
    P.num_slots = (int64_t)num_pages * page_size;
    P.max_pos = max_pos;
    P.rot = rot_dim;
    P.T = T;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.page_size = page_size;
    P.groups = (Hq + kRopeHeads - 1) / kRopeHeads;
    const int64_t k_blocks = ((int64_t)T * Hkv + 15) / 16, blocks = k_blocks + ((int64_t)T * P.groups + 15) / 16;
    if (blocks > 0x7fffffff) return FP8KV_ERR_UNSUPPORTED;
    P.k_blocks = (unsigned)k_blocks;
    P.k_every = (unsigned)(blocks / k_blocks);
    const cudaError_t e = cache_dtype == FP8KV_CACHE_E4M3   ? launch_rope<FP8KV_CACHE_E4M3>(P, interleaved != 0, (unsigned)blocks, (cudaStream_t)stream)
                          : cache_dtype == FP8KV_CACHE_BF16 ? launch_rope<FP8KV_CACHE_BF16>(P, interleaved != 0, (unsigned)blocks, (cudaStream_t)stream)
                                                            : launch_rope<FP8KV_CACHE_INT4>(P, interleaved != 0, (unsigned)blocks, (cudaStream_t)stream);
    return e == cudaSuccess ? FP8KV_OK : (cudaGetLastError(), FP8KV_ERR_CUDA);
}
