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
// token is read once for its heads.  A half warp takes HEADS heads of one token,
// a thread four pairs of each (or eight elements behind rot), so that the table,
// the slot and the position are in registers for all of them and their loads
// are in flight together.  K rows then pass through shared memory: a thread
// encodes eight (INT4: sixteen) neighbouring elements, whatever the pairs were.
#include "attention.cuh"
#include "common.cuh"
#include "int4.cuh"

namespace fp8kv {

int status_rope_insert(unsigned int* s, int clear) { return read_status(s, clear); }

struct RopeParams {
    const uint16_t *q, *k, *v;
    int64_t q_stride, k_stride, v_stride;       // elements a token
    const int64_t *positions, *slots;
    const float* cos_sin;
    const float *k_scale, *v_scale;
    uint16_t* q_out;
    uint8_t *k_cache, *v_cache;
    int64_t num_slots;
    int max_pos, rot, T, Hq, Hkv, page_size, groups;
};

template <int DT, int HEADS, bool PAIRS>
__global__ void __launch_bounds__(256) rope_insert_kernel(RopeParams P) {
    __shared__ __align__(16) uint16_t rows[16][128 + 8];
    pdl_launch_dependents();
    const int half = threadIdx.x >> 4, i = threadIdx.x & 15;
    const int64_t unit = (int64_t)blockIdx.x * 16 + half;
    const int64_t t64 = unit / P.groups;
    const bool in = t64 < P.T;
    const int64_t t = in ? t64 : 0;
    const int h0 = (int)(unit - t64 * P.groups) * HEADS;
    const bool turns = 8 * i < P.rot;
    const int ea = !turns || PAIRS ? 8 * i : 4 * i, eb = !turns || PAIRS ? 8 * i + 4 : P.rot / 2 + 4 * i;
    pdl_wait();
    const int64_t pos = in ? P.positions[t] : 0, slot = in ? P.slots[t] : -1;
    uint2 xa[HEADS], xb[HEADS];
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int h = h0 + u;
        if (!in || h >= P.Hq + P.Hkv) continue;
        const uint16_t* src = h < P.Hq ? P.q + t * P.q_stride + h * 128 : P.k + t * P.k_stride + (h - P.Hq) * 128;
        xa[u] = *reinterpret_cast<const uint2*>(src + ea);
        xb[u] = *reinterpret_cast<const uint2*>(src + eb);
    }
    const bool pos_ok = pos >= 0 && pos < P.max_pos;
    if (!pos_ok && i == 0 && h0 == 0) flag(FP8KV_DEV_BAD_POSITION);
    const bool slot_ok = slot >= 0 && slot < P.num_slots;
    if (in && pos_ok && slot >= P.num_slots && i == 0 && h0 == 0) flag(FP8KV_DEV_BAD_SLOT);
    const bool live = in && pos_ok;
    float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
    if (live && turns) {
        const float* row = P.cos_sin + pos * P.rot + 4 * i;
        c = *reinterpret_cast<const float4*>(row);
        s = *reinterpret_cast<const float4*>(row + P.rot / 2);
    }
    const float cc[4] = {c.x, c.y, c.z, c.w}, ss[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
    for (int u = 0; u < HEADS; ++u) {
        const int h = h0 + u;
        const bool mine = live && h < P.Hq + P.Hkv, is_q = h < P.Hq;
        if (mine && turns) {
            const uint32_t w[4] = {xa[u].x, xa[u].y, xb[u].x, xb[u].y};
            uint32_t o[4];
            if (PAIRS) {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = bf16_lo(w[j]), y = bf16_hi(w[j]);
                    o[j] = pack_bf16x2(__fmaf_rn(x, cc[j], -__fmul_rn(y, ss[j])), __fmaf_rn(y, cc[j], __fmul_rn(x, ss[j])));
                }
            } else {
                float r[8];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float x = j & 1 ? bf16_hi(w[j >> 1]) : bf16_lo(w[j >> 1]);
                    const float y = j & 1 ? bf16_hi(w[2 + (j >> 1)]) : bf16_lo(w[2 + (j >> 1)]);
                    r[j] = __fmaf_rn(x, cc[j], -__fmul_rn(y, ss[j]));
                    r[4 + j] = __fmaf_rn(y, cc[j], __fmul_rn(x, ss[j]));
                }
#pragma unroll
                for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(r[2 * j], r[2 * j + 1]);
            }
            xa[u] = make_uint2(o[0], o[1]);
            xb[u] = make_uint2(o[2], o[3]);
        }
        if (mine && is_q) {
            uint16_t* dst = P.q_out + (t * P.Hq + h) * 128;
            *reinterpret_cast<uint2*>(dst + ea) = xa[u];
            *reinterpret_cast<uint2*>(dst + eb) = xb[u];
        }
        // K: the row in order through shared memory (the loop is uniform over
        // the half warp; its two halves may disagree, so the whole warp meets)
        const bool stores = mine && !is_q && slot_ok;
        if (!__any_sync(0xffffffffu, stores)) continue;
        if (stores) {
            *reinterpret_cast<uint2*>(&rows[half][ea]) = xa[u];
            *reinterpret_cast<uint2*>(&rows[half][eb]) = xb[u];
        }
        __syncwarp();
        if (stores) {
            const int hk = h - P.Hq;
            const int64_t page = slot / P.page_size;
            const int off = (int)(slot - page * P.page_size);
            const uint4* vrow = reinterpret_cast<const uint4*>(P.v + t * P.v_stride + hk * 128);
            const uint4* krow = reinterpret_cast<const uint4*>(rows[half]);
            if (DT == FP8KV_CACHE_INT4) {
                // threads 0-7: the blocks of K, 8-15: those of V
                const bool is_k = i < 8;
                const int block = i & 7;
                const uint4 x0 = is_k ? krow[2 * block] : vrow[2 * block], x1 = is_k ? krow[2 * block + 1] : vrow[2 * block + 1];
                uint8_t sc;
                const uint2 codes = int4_encode16(x0, x1, is_k ? *P.k_scale : *P.v_scale, sc);
                uint8_t* cache = (is_k ? P.k_cache : P.v_cache) + (page * P.Hkv + hk) * P.page_size * kInt4RowBytes;
                *reinterpret_cast<uint2*>(cache + off * kInt4CodeBytes + block * 8) = codes;
                cache[P.page_size * kInt4CodeBytes + off * kInt4ScaleBytes + block] = sc;
            } else {
                const int64_t at = ((page * P.Hkv + hk) * P.page_size + off) * 128 + 8 * i;
                if (DT == FP8KV_CACHE_E4M3) {
                    *reinterpret_cast<uint2*>(P.k_cache + at) = e4m3_encode8(krow[i], *P.k_scale);
                    *reinterpret_cast<uint2*>(P.v_cache + at) = e4m3_encode8(vrow[i], *P.v_scale);
                } else {
                    *reinterpret_cast<uint4*>(P.k_cache + 2 * at) = krow[i];
                    *reinterpret_cast<uint4*>(P.v_cache + 2 * at) = vrow[i];
                }
            }
        }
        __syncwarp();
    }
}

template <int DT>
static cudaError_t launch_rope(const RopeParams& P, bool pairs, int heads, int64_t blocks, cudaStream_t s) {
    auto kern = pairs ? (heads == 4 ? rope_insert_kernel<DT, 4, true> : rope_insert_kernel<DT, 1, true>)
                      : (heads == 4 ? rope_insert_kernel<DT, 4, false> : rope_insert_kernel<DT, 1, false>);
    return launch_pdl(kern, dim3((unsigned)blocks), dim3(256), 0, s, P);
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
    if (q == q_out) return FP8KV_ERR_INVALID_ARG;
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
    const int heads = (int64_t)T * (Hq + Hkv) > 16 * 8 * (int64_t)num_sms() ? 4 : 1;
    P.groups = (Hq + Hkv + heads - 1) / heads;
    const int64_t blocks = ((int64_t)T * P.groups + 15) / 16;
    if (blocks > 0x7fffffff) return FP8KV_ERR_UNSUPPORTED;
    const cudaError_t e = cache_dtype == FP8KV_CACHE_E4M3   ? launch_rope<FP8KV_CACHE_E4M3>(P, interleaved != 0, heads, blocks, (cudaStream_t)stream)
                          : cache_dtype == FP8KV_CACHE_BF16 ? launch_rope<FP8KV_CACHE_BF16>(P, interleaved != 0, heads, blocks, (cudaStream_t)stream)
                                                            : launch_rope<FP8KV_CACHE_INT4>(P, interleaved != 0, heads, blocks, (cudaStream_t)stream);
    return e == cudaSuccess ? FP8KV_OK : (cudaGetLastError(), FP8KV_ERR_CUDA);
}
