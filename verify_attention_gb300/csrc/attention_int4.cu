// attention_int4.cu -- paged decode / verifier attention over a cache held in
// 4 bits (FP8KV_CACHE_INT4, include/fp8kv.h): per 16 elements an E4M3 scale s
// and integers n in [-7, 7], value n s c with the tensor scale c.
//
// What bounds it: a row is 72 bytes, K and V of one token and head 144 for 256
// elements, so one SM's share of the HBM rate brings about 42 elements a cycle
// and the instructions that widen them count.  Widening is exact and costs one
// logic operation and one fma for two elements: the code n + 8 becomes the low
// mantissa bits of the f16 values 256 + code or 16 + code (bits 2..5 or 6..9
// of the half word), and fma(v, s, -264 s) or fma(v, s, -24 s) is n s exactly
// (264 s and 24 s have at most 10 significant bits, n s at most 7).  Two
// shifts serve the eight codes of a word.  The tensor scales are applied to
// the logits and to the output.
//
// One CTA per (partition, KV head x tile of 16 query rows, sequence).  Its
// warps take chunks of 32 keys in turn, each with its own ring of chunks
// filled by cp.async (no producer, no barriers), and run both products on
// mma.sync m16n8k16 (rows x keys, f16 in, fp32 out), online softmax in the
// log2 domain; they merge through shared memory at the end.  Order of the
// fragments: in Q.K^T a thread's B elements are 32 dimensions of one key (16
// code bytes); in P.V they are the 16 dimensions of one scale block of four
// keys.  Both are contiguous in a row, and the key order inside a group of
// eight, key = 4 (n & 1) + (n >> 1) for column n, makes the eight-byte V reads
// free of bank conflicts.
#include <stdio.h>

#include "attention.cuh"
#include "common.cuh"
#include "int4.cuh"

namespace fp8kv {

int status_attention_int4(unsigned int* s, int clear) { return read_status(s, clear); }

namespace i4 {

constexpr int STAGES = 4;                               // chunks of a warp's ring
constexpr int CK = 32;                                  // keys per chunk
constexpr int OFF_V = CK * kInt4CodeBytes;              // K codes, V codes, K scales, V scales
constexpr int OFF_KS = 2 * CK * kInt4CodeBytes;
constexpr int OFF_VS = OFF_KS + CK * kInt4ScaleBytes;
constexpr int STAGE_BYTES = OFF_VS + CK * kInt4ScaleBytes;   // 4608
constexpr float GROW = 4.0f, BIAS = 11.0f;              // see the softmax
constexpr int MERGE_STRIDE = 132;                       // floats per merged row: 128 of O, max, sum
// the rings; after them, in the same bytes, the warps' merged rows and (in a
// cluster) the CTA's
template <int WARPS>
constexpr int SMEM = WARPS * STAGES * STAGE_BYTES;
static_assert((12 + 1) * 16 * MERGE_STRIDE * 4 <= SMEM<12> && (4 + 1) * 16 * MERGE_STRIDE * 4 <= SMEM<4>,
              "merge area exceeds the rings");

// 16 bytes from src + SRC to shared memory at dst + DST (zeros when bytes = 0)
template <int DST, int SRC>
__device__ __forceinline__ void cp16(uint32_t dst, const uint8_t* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0 + %3], [%1 + %4], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes), "n"(DST), "n"(SRC)
                 : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// Where this lane's 16-byte pieces of a chunk go in a stage: K rows at their
// column position (see the key order above), V rows with the 16-byte units
// exchanged on keys 2 and 3 of 4.  Piece u of lane l is row (l >> 2) + 8 u.
struct Lanes {
    uint32_t k, v, s;
};
__device__ __forceinline__ Lanes lane_places(int lane) {
    const int row = lane >> 2, ch = lane & 3;
    return {(uint32_t)((((row & 3) << 1) | (row >> 2)) * 64 + ch * 16),
            (uint32_t)(OFF_V + row * 64 + ((ch ^ (row & 2)) << 4)), (uint32_t)(OFF_KS + lane * 16)};
}

// Issue the copies of the chunk at key_in_page of page `page` into a stage.
// Pages outside the pool read as zeros.
template <int PS>
__device__ __forceinline__ void issue_chunk(uint32_t stage, const Lanes& at, const AttnParams& P, int page, int hk,
                                            int key_in_page, int lane) {
    const bool valid = page >= 0 && page < P.num_pages;
    const int bytes = valid ? 16 : 0;
    const int64_t base = valid ? ((int64_t)page * P.Hkv + hk) * (PS * kInt4RowBytes) : 0;
    const int64_t code = base + key_in_page * kInt4CodeBytes + lane * 16;
    const uint8_t *kp = P.k_cache + code, *vp = P.v_cache + code;
    const uint8_t* sp = (lane < 16 ? P.k_cache : P.v_cache) + base + PS * kInt4CodeBytes +
                        key_in_page * kInt4ScaleBytes + (lane & 15) * 16;
    cp16<0, 0>(stage + at.k, kp, bytes);
    cp16<512, 512>(stage + at.k, kp, bytes);
    cp16<1024, 1024>(stage + at.k, kp, bytes);
    cp16<1536, 1536>(stage + at.k, kp, bytes);
    cp16<0, 0>(stage + at.v, vp, bytes);
    cp16<512, 512>(stage + at.v, vp, bytes);
    cp16<1024, 1024>(stage + at.v, vp, bytes);
    cp16<1536, 1536>(stage + at.v, vp, bytes);
    cp16<0, 0>(stage + at.s, sp, bytes);
}

// Append: the new tokens of sequence b (length L) at positions lo .. hi - 1 of
// [L - M, L), KV head hk.  Only the CTA that reads them writes them, so no other
// has to be waited for (one sequence of 256 keys: 7.1 us; the append as a launch
// of its own 8.7).
template <int PS>
__device__ __forceinline__ void append(const AttnParams& P, int b, int hk, int L, int lo, int hi, int thread,
                                       int threads) {
    for (int i = thread; i < (hi - lo) * 8; i += threads) {
        const int pos = lo + (i >> 3), block = i & 7;
        const int page = P.block_table[(int64_t)b * P.mpps + pos / PS];
        if (page < 0 || page >= P.num_pages) {
            if (block == 0) flag(FP8KV_DEV_BAD_SLOT);
            continue;
        }
        const int64_t src = ((((int64_t)b * P.M + (pos - (L - P.M))) * P.Hkv + hk) * 8 + block) * 2;
        const uint4 *k = (const uint4*)P.k_new + src, *v = (const uint4*)P.v_new + src;
        Int4Block(k[0], k[1], v[0], v[1], *P.k_scale, *P.v_scale)
            .store(P.k_cache, P.v_cache, page, pos % PS, hk, P.Hkv, PS, block);
    }
}

// WARPS = 12, one CTA per SM, or 4, three CTAs per SM (168 registers a thread).
// CL: the partitions of a (sequence, KV head) are a thread-block cluster and
// merge their rows from each other's shared memory (one sequence of 4000 keys:
// 11.2 us; partials through memory and a reduce kernel 13.7).
template <int PS, int WARPS, bool CL>
__global__ void __launch_bounds__(WARPS * 32, 12 / WARPS) paged_attention_int4_kernel(AttnParams P) {
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int THREADS = WARPS * 32;
    const int rt = blockIdx.y % P.NT;
    int split = blockIdx.x, hk = blockIdx.y / P.NT, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int g = lane >> 2, t = lane & 3;
    pdl_launch_dependents();
    pdl_wait();
    if (P.lpt_order) {
        // CTA i: KV head i mod Hkv of the slot of rank i / Hkv, longest first
        const int lin = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
        const int q = P.lpt_order[lin / P.Hkv];
        if (q < 0) return;
        hk = lin % P.Hkv;
        b = q / P.num_splits;
        split = q % P.num_splits;
    }
    // what does not depend on the length is read beside it: q, and the first
    // page id, right unless a window moves the partition (256 keys: 6.5 us
    // without, 6.4 with)
    const int32_t* table = P.block_table + (int64_t)b * P.mpps;
    constexpr int CPP = PS / CK;                        // chunks per page
    const int guess_at = min(split * P.split_pages + warp / CPP, P.mpps - 1), guess = table[guess_at];
    const int R0 = rt * 16;
    uint4 qw[2][4];
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
        const int r = R0 + g + 8 * hr, m = min(r, P.R - 1) / P.G;
        const uint4* src = (const uint4*)(P.q + (((int64_t)b * P.M + m) * P.Hq + hk * P.G + min(r, P.R - 1) % P.G) * 128) + 4 * t;
#pragma unroll
        for (int u = 0; u < 4; ++u) qw[hr][u] = r < P.R ? src[u] : make_uint4(0, 0, 0, 0);
    }
    const float ks = *P.k_scale;
    const int L = P.seq_lens[b];
    if (L < P.M || L > P.max_seq_len || (L + PS - 1) / PS > P.mpps) {
        if (threadIdx.x == 0 && split == 0 && blockIdx.y == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
        return;
    }
    // partitions are cut from the keys that any of the R rows sees
    const int lo0 = (P.window_left >= 0) ? max(0, L - P.M - P.window_left) : 0;
    const int first_page = lo0 / PS, last_page = (L - 1) / PS;
    const int nsplit_b = (last_page - first_page + P.split_pages) / P.split_pages;
    if (nsplit_b > P.num_splits) {   // cannot happen when L <= max_seq_len; never index past the plan
        if (threadIdx.x == 0 && split == 0 && blockIdx.y == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
        return;
    }
    if (split >= nsplit_b) return;
    const int page_begin = first_page + split * P.split_pages;
    const int n_pages = min(P.split_pages, last_page + 1 - page_begin);
    const int key_begin = page_begin * PS;
    const int n_chunks = (min(n_pages * PS, L - key_begin) + CK - 1) / CK;
    const int32_t* bt = table + page_begin;
    const uint32_t ring = smem_u32(smem) + warp * STAGES * STAGE_BYTES;

    // append: this partition's new tokens, before its copies read them
    const int app_lo = max(L - P.M, key_begin), app_hi = min(L, key_begin + n_pages * PS);
    if (P.k_new && app_lo < app_hi) {                   // uniform over the CTA
        append<PS>(P, b, hk, L, app_lo, app_hi, threadIdx.x, THREADS);
        __syncthreads();
    }

    // this warp's chunks: warp, warp + WARPS, ...; their page ids are read one
    // round ahead of the copies
    const Lanes places = lane_places(lane);
    int next = warp;
    int page = next < n_chunks ? (page_begin + next / CPP == guess_at ? guess : bt[next / CPP]) : -1;
    auto issue = [&](int slot) {
        if (next < n_chunks) {
            const int cur = page, at = next;
            next += WARPS;
            page = next < n_chunks ? bt[next / CPP] : -1;
            issue_chunk<PS>(ring + slot * STAGE_BYTES, places, P, cur, hk, (at % CPP) * CK, lane);
        }
        cp_commit();
    };
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) issue(s);

    // ---- rows g and g + 8 of the tile: positions, Q fragments
    int pr[2], lor[2];
    float mult[2];
    uint32_t qa[8][4];
    {
        float qf[2][32];
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            const int r = R0 + g + 8 * hr;
            const int m = min(r, P.R - 1) / P.G;
            pr[hr] = L - P.M + m;
            lor[hr] = (P.window_left >= 0) ? max(0, pr[hr] - P.window_left) : 0;
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                const uint32_t ww[4] = {qw[hr][u].x, qw[hr][u].y, qw[hr][u].z, qw[hr][u].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    qf[hr][8 * u + 2 * e] = bf16_lo(ww[e]);
                    qf[hr][8 * u + 2 * e + 1] = bf16_hi(ww[e]);
                }
            }
            // a power of two that puts the row maximum in [2^4, 2^5): the f16
            // copy of q is then exact down to 2^-18 of the row maximum, and
            // q . (n s) stays below 128 * 2^5 * 7 * 448 < 2^24
            float amax = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j) amax = fmaxf(amax, fabsf(qf[hr][j]));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
            int e = 4;
            const uint32_t ab = __float_as_uint(amax);
            if (amax > 0.f && ((ab >> 23) & 0xff) != 0xff) {
                const int be = (int)((ab >> 23) & 0xff);
                e = be ? be - 127 : -127;
            }
            const int sh = max(-120, min(120, 4 - e));
            // (the sign of sm_scale goes into q: the row maximum is taken before
            // the multiplication below)
            const float scale = copysignf(ldexpf(1.0f, sh), P.sm_scale);
#pragma unroll
            for (int j = 0; j < 32; ++j) qf[hr][j] *= scale;
            mult[hr] = fmaxf(4.0f * ks * fabsf(P.sm_scale) * 1.4426950408889634f * ldexpf(1.0f, -sh), 1e-37f);
        }
        // word w of a key's 16 code bytes holds dims 8w .. 8w + 7 of the 32;
        // widen4 pairs dim f with f + 4, f = 0..3, and fills two k-steps
#pragma unroll
        for (int w = 0; w < 4; ++w) {
#pragma unroll
            for (int f = 0; f < 4; ++f) {
                qa[2 * w + (f >> 1)][2 * (f & 1)] = pack_f16x2(qf[0][8 * w + f], qf[0][8 * w + f + 4]);
                qa[2 * w + (f >> 1)][2 * (f & 1) + 1] = pack_f16x2(qf[1][8 * w + f], qf[1][8 * w + f + 4]);
            }
        }
    }
    // bounds of the warp's rows, to skip the masks on interior chunks
    int pmin = min(pr[0], pr[1]), lomax = max(lor[0], lor[1]);
#pragma unroll
    for (int off = 4; off <= 16; off <<= 1) {
        pmin = min(pmin, __shfl_xor_sync(0xffffffffu, pmin, off));
        lomax = max(lomax, __shfl_xor_sync(0xffffffffu, lomax, off));
    }

    float o[16][4];
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
    float mrow[2] = {-INFINITY, -INFINITY}, lrow[2] = {0.f, 0.f};

    int slot = 0, fill = STAGES - 1;
#pragma unroll 1
    for (int c = warp; c < n_chunks; c += WARPS) {
        cp_wait<STAGES - 2>();
        __syncwarp();                                   // every lane's copies of this chunk; reads of the last one done
        issue(fill);
        fill = fill + 1 == STAGES ? 0 : fill + 1;
        const int cur_slot = slot;
        const uint8_t* st = smem + (warp * STAGES + slot) * STAGE_BYTES;
        slot = slot + 1 == STAGES ? 0 : slot + 1;
        const int k0 = key_begin + c * CK;

        // ---- S = Q K^T
        float sacc[4][4];
        uint32_t kw[4][4];
        Scale2 sc[4][2];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint4 x = *(const uint4*)(st + (8 * j + g) * 64 + 16 * t);
            kw[j][0] = x.x;
            kw[j][1] = x.y;
            kw[j][2] = x.z;
            kw[j][3] = x.w;
            const int key = 8 * j + 4 * (g & 1) + (g >> 1);
            const uint32_t s2 = e4m3x2_to_f16x2(*(const uint16_t*)(st + OFF_KS + key * 8 + 2 * t));
            sc[j][0] = scale2(prmt(s2, s2, 0x1010));
            sc[j][1] = scale2(prmt(s2, s2, 0x3232));
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
            uint32_t v[4][4];
#pragma unroll
            for (int j = 0; j < 4; ++j) widen4(kw[j][w], sc[j][w >> 1], v[j]);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (w == 0) mma_f16_zero(sacc[j], qa[0], v[j][0], v[j][1]);
                else mma_f16(sacc[j], qa[2 * w], v[j][0], v[j][1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) mma_f16(sacc[j], qa[2 * w + 1], v[j][2], v[j][3]);
        }
        // ---- masks, online softmax in log2 units (s mult)
        if ((k0 + CK - 1 > pmin) || (k0 < lomax)) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int key = k0 + 8 * j + 4 * (e & 1) + t;
                    if (key > pr[e >> 1] || key < lor[e >> 1]) sacc[j][e] = -INFINITY;
                }
        }
        // O is rescaled only when a row's maximum grows by more than 2^GROW
        float tmax[2];
        bool grow = false;
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            float x = max3(sacc[0][2 * hr], sacc[0][2 * hr + 1], sacc[1][2 * hr]);
            x = max3(x, sacc[1][2 * hr + 1], sacc[2][2 * hr]);
            x = max3(x, sacc[2][2 * hr + 1], sacc[3][2 * hr]);
            x = fmaxf(x, sacc[3][2 * hr + 1]);
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
            x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
            tmax[hr] = x * mult[hr];
            grow |= tmax[hr] > mrow[hr] + GROW;             // (the first visible keys too: mrow = -inf)
        }
        if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
                const float mnew = fmaxf(mrow[hr], tmax[hr]);
                const float alpha = mrow[hr] == -INFINITY ? 1.f : ex2(mrow[hr] - mnew);
                mrow[hr] = mnew;
                lrow[hr] *= alpha;
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    o[i][2 * hr] *= alpha;
                    o[i][2 * hr + 1] *= alpha;
                }
            }
        }
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
            // weights as 2^11 times 2^(x - m), at most 2^15: f16 then keeps 11
            // bits of every weight down to 2^-25 of the largest
            const float neg = (mrow[hr] == -INFINITY) ? 0.f : BIAS - mrow[hr];
            float sum = 0.f;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                sacc[j][2 * hr] = ex2(fmaf(sacc[j][2 * hr], mult[hr], neg));
                sacc[j][2 * hr + 1] = ex2(fmaf(sacc[j][2 * hr + 1], mult[hr], neg));
                sum += sacc[j][2 * hr] + sacc[j][2 * hr + 1];
            }
            lrow[hr] += sum;
        }
        // ---- O += P V.  Keys that no row sees (behind the end, before the
        // first window) get scale 0: whatever their bytes are, 0 reaches O
        if (k0 + CK > L || k0 < lo0) {
            __syncwarp();
            if (k0 + lane >= L || k0 + lane < lo0)
                *(uint2*)(smem + (warp * STAGES + cur_slot) * STAGE_BYTES + OFF_VS + lane * 8) = make_uint2(0u, 0u);
            __syncwarp();
        }
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
            uint32_t pa[4];
            pa[0] = pack_f16x2(sacc[2 * kk][0], sacc[2 * kk][1]);
            pa[1] = pack_f16x2(sacc[2 * kk][2], sacc[2 * kk][3]);
            pa[2] = pack_f16x2(sacc[2 * kk + 1][0], sacc[2 * kk + 1][1]);
            pa[3] = pack_f16x2(sacc[2 * kk + 1][2], sacc[2 * kk + 1][3]);
            uint32_t w[4][2];                           // keys 16 kk + {0, 4, 8, 12} + t, block g
            Scale2 sc[2];
#pragma unroll
            for (int pr2 = 0; pr2 < 2; ++pr2) {
                uint32_t by[2];
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int key = 16 * kk + 8 * pr2 + 4 * e + t;
                    const uint2 x = *(const uint2*)(st + OFF_V + key * 64 + ((((g >> 1) ^ (key & 2))) << 4) + (g & 1) * 8);
                    w[2 * pr2 + e][0] = x.x;
                    w[2 * pr2 + e][1] = x.y;
                    by[e] = st[OFF_VS + key * 8 + g];
                }
                sc[pr2] = scale2(e4m3x2_to_f16x2(by[0] | (by[1] << 8)));
            }
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    uint32_t va[4], vb[4];
                    widen4(prmt(w[0][i], w[1][i], h ? 0x7632 : 0x5410), sc[0], va);
                    widen4(prmt(w[2][i], w[3][i], h ? 0x7632 : 0x5410), sc[1], vb);
#pragma unroll
                    for (int f = 0; f < 4; ++f) mma_f16(o[8 * i + 4 * h + f], pa, va[f], vb[f]);
                }
            }
        }
    }
    cp_wait<0>();

    // ---- merge the warps' (max, sum, O): n-tile i, column n -> dim 16 n + i
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
        lrow[hr] += __shfl_xor_sync(0xffffffffu, lrow[hr], 1);
        lrow[hr] += __shfl_xor_sync(0xffffffffu, lrow[hr], 2);
    }
    __syncthreads();                                    // every ring is consumed
    float* merge = (float*)smem;
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
        float* dst = merge + (warp * 16 + g + 8 * hr) * MERGE_STRIDE;
#pragma unroll
        for (int i = 0; i < 16; i += 4) {
            *(float4*)(dst + 32 * t + i) =
                make_float4(o[i][2 * hr], o[i + 1][2 * hr], o[i + 2][2 * hr], o[i + 3][2 * hr]);
            *(float4*)(dst + 32 * t + 16 + i) =
                make_float4(o[i][2 * hr + 1], o[i + 1][2 * hr + 1], o[i + 2][2 * hr + 1], o[i + 3][2 * hr + 1]);
        }
        if (t == 0) {
            dst[128] = mrow[hr];
            dst[129] = lrow[hr];
        }
    }
    __syncthreads();
    const float vs = 4.0f * *P.v_scale;
    const int rows = min(16, P.R - R0), nw = min(WARPS, n_chunks);
    for (int item = threadIdx.x; item < rows * 32; item += THREADS) {
        const int r = item >> 5, d4 = (item & 31) * 4;
        float mstar = -INFINITY;
        for (int w = 0; w < nw; ++w) mstar = fmaxf(mstar, merge[(w * 16 + r) * MERGE_STRIDE + 128]);
        float l = 0.f;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        if (mstar != -INFINITY) {
            for (int w = 0; w < nw; ++w) {
                const float* src = merge + (w * 16 + r) * MERGE_STRIDE;
                const float wt = ex2(src[128] - mstar);
                l += wt * src[129];
                const float4 v4 = *(const float4*)(src + d4);
                acc.x += wt * v4.x;
                acc.y += wt * v4.y;
                acc.z += wt * v4.z;
                acc.w += wt * v4.w;
            }
        } else {
            // no key with a number for a score: no visible key at all (l = 0), or
            // NaN scores only, which the maximum passes over but the sum holds.
            // Those must not look like no key where partitions are combined:
            // they go on with the maximum 0 (a NaN key as the last partition's
            // only one would otherwise leave a finite output)
            for (int w = 0; w < nw; ++w) l += merge[(w * 16 + r) * MERGE_STRIDE + 129];
            if (l != l) mstar = 0.f;
        }
        const int m = (R0 + r) / P.G, hq = hk * P.G + (R0 + r) % P.G;
        const int64_t row_idx = ((int64_t)b * P.M + m) * P.Hq + hq;
        if (nsplit_b == 1) {
            const float f = vs / l;
            *(uint2*)(P.out + row_idx * 128 + d4) =
                make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
        } else if (CL) {
            float* dst = merge + (WARPS * 16 + r) * MERGE_STRIDE;
            *(float4*)(dst + d4) = acc;
            if (d4 == 0) *(float2*)(dst + 128) = make_float2(mstar, l);
        } else {
            // partial: f16 of 4 O / l (|x| <= 7 * 448) beside its (max, sum); a
            // row with no visible key here has l = 0: weight 0, values 0
            const float f = l > 0.f ? 4.0f / l : 0.f;
            *(uint2*)((uint16_t*)P.ws_o + (row_idx * P.num_splits + split) * 128 + d4) =
                make_uint2(pack_f16x2(acc.x * f, acc.y * f), pack_f16x2(acc.z * f, acc.w * f));
            if (d4 == 0) *(float2*)(P.ws_ml + (row_idx * P.num_splits + split) * 2) = make_float2(mstar, l);
        }
    }
    if (CL && nsplit_b > 1) {
        // (CTAs of the cluster without keys have returned: the barriers count
        // those that have not)
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        for (int item = split * THREADS + threadIdx.x; item < rows * 32; item += nsplit_b * THREADS) {
            const int r = item >> 5, d4 = (item & 31) * 4;
            const float* at = merge + (WARPS * 16 + r) * MERGE_STRIDE;
            float2 a[8];
            uint4 x[8];
            float top = -INFINITY, l = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= nsplit_b) break;
                a[j] = dsmem_ld8(dsmem_addr(at + 128, j));
                x[j] = dsmem_ld16(dsmem_addr(at + d4, j));
                top = fmaxf(top, a[j].x);
            }
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j >= nsplit_b) break;
                const float w = a[j].x == -INFINITY ? 0.f : ex2(a[j].x - top);
                l += w * a[j].y;
                acc.x += w * __uint_as_float(x[j].x);
                acc.y += w * __uint_as_float(x[j].y);
                acc.z += w * __uint_as_float(x[j].z);
                acc.w += w * __uint_as_float(x[j].w);
            }
            const int m = (R0 + r) / P.G, hq = hk * P.G + (R0 + r) % P.G;
            const float f = vs / l;
            *(uint2*)(P.out + (((int64_t)b * P.M + m) * P.Hq + hq) * 128 + d4) =
                make_uint2(pack_bf16x2(acc.x * f, acc.y * f), pack_bf16x2(acc.z * f, acc.w * f));
        }
        __syncwarp();
        cluster_arrive();                               // no shared memory goes before all have read
        cluster_wait();
    }
}

template <int PS, int WARPS, bool CL>
static int launch(const AttnParams& P, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    auto kern = paged_attention_int4_kernel<PS, WARPS, CL>;
    if (opt_in_smem(done, (const void*)kern, SMEM<WARPS>) != cudaSuccess) return (cudaGetLastError(), FP8KV_ERR_CUDA);
    const dim3 grid(P.num_splits, P.Hkv * P.NT, P.B);
    const cudaError_t e = launch_pdl_cluster(kern, grid, dim3(WARPS * 32), SMEM<WARPS>, s, P.cluster, P);
    return e == cudaSuccess ? FP8KV_OK : (cudaGetLastError(), FP8KV_ERR_CUDA);
}

}  // namespace i4

void int4_clusters(int (&count)[9]) {
    static std::atomic<int> known[64][9];                   // [device][n]: 1 + count
    int dev = 0;
    for (int n = 0; n < 9; ++n) count[n] = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev >= 64) return;
    for (int n = 2; n < 9; ++n) {
        int k = known[dev][n].load(std::memory_order_relaxed);
        if (!k) {
            auto kern = i4::paged_attention_int4_kernel<32, 12, true>;
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(n);
            cfg.blockDim = dim3(12 * 32);
            cfg.dynamicSmemBytes = i4::SMEM<12>;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = n;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int most = 0;
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, i4::SMEM<12>) != cudaSuccess ||
                cudaOccupancyMaxActiveClusters(&most, kern, &cfg) != cudaSuccess) {
                cudaGetLastError();
                most = 0;                                   // no clusters
            }
            k = 1 + most;
            known[dev][n].store(k, std::memory_order_relaxed);
        }
        count[n] = k - 1;
    }
}

int launch_attention_int4(const AttnParams& P, cudaStream_t s, char* text, size_t text_bytes) {
    if ((int64_t)P.Hkv * P.NT > 65535) return FP8KV_ERR_UNSUPPORTED;
    if (P.cluster > 1 && (P.cluster > 8 || P.cluster != P.num_splits || P.NT > 1 || P.lpt_order || P.KW != 12))
        return FP8KV_ERR_UNSUPPORTED;
    // Small CTAs, three to an SM, where there are enough of them: one's set-up
    // and merge run beside the others' keys (64 sequences, 2048 CTAs: 384 us
    // against 405); few of them would leave the SMs part empty (one sequence of
    // 131072 keys, 152 CTAs: 106 us against 49).
    const bool small = P.KW == 4, ps32 = P.page_size == 32;
    const int rc = P.cluster > 1 ? (ps32 ? i4::launch<32, 12, true>(P, s) : i4::launch<64, 12, true>(P, s))
                   : small       ? (ps32 ? i4::launch<32, 4, false>(P, s) : i4::launch<64, 4, false>(P, s))
                                 : (ps32 ? i4::launch<32, 12, false>(P, s) : i4::launch<64, 12, false>(P, s));
    if (rc) return rc;
    snprintf(text, text_bytes,
             "paged_attention_int4_mma<ps=%d> rows=%d row_tiles=%d splits=%d split_tokens=%d grid=%dx%dx%d threads=%d "
             "cluster=%d reduce=%d order=%s",
             P.page_size, P.R, P.NT, P.num_splits, P.split_pages * P.page_size, P.num_splits, P.Hkv * P.NT, P.B,
             small ? 128 : 384, P.cluster > 1 ? P.cluster : 1, P.num_splits > 1 && P.cluster <= 1 ? 1 : 0,
             P.lpt_order ? "longest_first" : "grid");
    return FP8KV_OK;
}

}  // namespace fp8kv
