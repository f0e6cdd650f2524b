// prompt_attention.cu -- causal attention of whole prompts: packed sequences of
// different lengths, grouped heads, an optional sliding window, bf16 rows as
// the projection wrote them (no cache in between).  (The pages have no
// counterpart; the masks are those of fp8kv_paged_attention.)
//
// What bounds it: 4 * 128 operations for each visible (row, key) pair, on the
// tensor cores; the K and V tiles come from L2.  One CTA computes two tiles of
// 128 rows against the same K and V tiles: while the softmax of one tile runs,
// the tensor cores work on the other.
//
// Rows.  The G query heads of a KV head are packed: row r of a tile is position
// r / G, head r % G, NP = 128 / G positions a tile (126 rows for G = 9).  The
// rows of a tile then see nearly the same keys, so a diagonal or a window edge
// costs little more than the keys it holds, and short prompts fill a tile.
//
// One CTA, 11 warps:
//   warp 0     TMA: Q once, then K and V tiles of 128 keys through a ring of
//              five 32 KiB slots; allocates and frees the tensor memory
//   warp 1     issues the MMAs (one thread): per key tile P.V of the previous
//              tile and Q.K^T of this one, for the first row tile, then for
//              the second; S = Q.K^T from shared memory, O += P.V with P from
//              tensor memory
//   warps 2-5  softmax of the first row tile, one row per thread (warp w holds
//   warps 6-9  ... of the second      TMEM lanes 32 (w % 4) ...)
//   warp 10    zeroes the V rows of the first and last key tile that no row of
//              the CTA sees (they may hold another sequence's values, or
//              none): whatever is there, 0 * V reaches no output
// Online softmax in the log2 domain; O is rescaled only when a row's maximum
// grows by more than 2^8 (the weights stay below 2^8, sums are fp32).  P is
// rounded to bf16, V's type, as the MMA needs both alike: 2^-9 of each weight,
// the size of the output's own rounding.
// TMEM columns: S/P of the two row tiles 0-127, 128-255 (P over the first half
// of its S), O 256-383, 384-511.
#include <stdio.h>

#include <mutex>
#include <set>

#include "attention.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace fp8kv {

int status_prompt(unsigned int* s, int clear) { return read_status(s, clear); }

namespace prompt {

constexpr int NK = 128;                         // keys per tile
constexpr int SLOT = NK * 256;                  // 32 KiB: two blocks of 128 rows x 64 dims (128-byte swizzled)
constexpr int HALF = SLOT / 2;
constexpr int SLOTS = 5;
constexpr int WARPS = 11, THREADS = WARPS * 32;
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
constexpr int SMEM = 2 * SLOT + SLOTS * SLOT + 1024 + 512;

enum {
    B_Q = 0,
    B_FULL = 1,
    B_EMPTY = B_FULL + SLOTS,
    B_S = B_EMPTY + SLOTS,                      // per row tile: S ready
    B_P = B_S + 2,                              // per row tile and half: 64 columns of P ready
    B_O = B_P + 4,                              // per row tile: O final
    B_RAW = B_O + 2,                            // first / last V tile loaded, to be cleaned
    B_STAGE = B_RAW + 2,                        // per row tile: output rows staged
    B_IDLE = B_STAGE + 2,
    B_COUNT
};

struct Params {
    const int32_t* cu;          // [B + 1]
    uint16_t* out;              // [T][Hq][128]
    int B, T, Hq, Hkv, G, NP, window_left, max_seq_len;
    float scale_log2;           // sm_scale * log2(e)
};

// bf16 operands: format code 1 for A and B.
constexpr uint32_t ID_QK = idesc(128, NK, false) | (1u << 7) | (1u << 10);
constexpr uint32_t ID_PV = idesc(128, 128, true) | (1u << 7) | (1u << 10);

__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{ .reg .pred p; setp.ne.b32 p, %4, 0; "
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p; }" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* tm, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tm),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

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

// Position of K and V tiles in the ring, in the order of their use:
// K0 K1 V0 K2 V1 ... K(n-1) V(n-2) V(n-1).
__device__ __forceinline__ int k_item(int j) { return j == 0 ? 0 : 2 * j - 1; }
__device__ __forceinline__ int v_item(int j, int n) { return j == n - 1 ? 2 * n - 1 : 2 * j + 2; }

__global__ void __launch_bounds__(THREADS, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                            Params P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* qs = smem;                                     // two row tiles of 32 KiB
    uint8_t* ring = smem + 2 * SLOT;
    uint64_t* bars = (uint64_t*)(ring + SLOTS * SLOT);
    uint32_t* tmem_slot = (uint32_t*)(bars + B_COUNT);
    int* where = (int*)(tmem_slot + 1);                     // sequence start, length, first position
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int hk = blockIdx.x;
    const int rows = P.G * P.NP;                            // used rows of a tile
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        mbar_init(bar(B_Q), 1);
        for (int i = 0; i < SLOTS; ++i) {
            mbar_init(bar(B_FULL + i), 1);
            mbar_init(bar(B_EMPTY + i), 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_S + i), 1);
            mbar_init(bar(B_O + i), 1);
            mbar_init(bar(B_RAW + i), 1);
        }
        for (int i = 0; i < 4; ++i) mbar_init(bar(B_P + i), 4);
        for (int i = 0; i < 2; ++i) mbar_init(bar(B_STAGE + i), 4);
        mbar_init(bar(B_IDLE), 1);
        fence_barrier_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        if (lane == 0) {
            prefetch_tensormap(&tm_q);
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
            prefetch_tensormap(&tm_o);
        }
    }
    // rows behind G * NP take part in the MMAs: zeros there keep them finite
    for (int i = threadIdx.x; i < 2 * 2 * (128 - rows) * 8; i += THREADS) {
        const int c = i & 7, r = rows + (i >> 3) % (128 - rows), blk = (i >> 3) / (128 - rows);
        *(uint4*)(qs + blk * HALF + r * 128 + c * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
    pdl_wait();
    if (warp == 10) {
        // Pair x (two row tiles, 2 NP positions) of the whole launch, the last
        // ones first: sequence b owns the indices from cu[b] / (2 NP) + b on,
        // at least as many as it has pairs, so the largest b whose first index
        // is at most x is found by a 32-way search, without a scan.
        const int PP = 2 * P.NP, x = (int)(gridDim.y - 1 - blockIdx.y);
        int lo = 0, hi = P.B;
        while (hi - lo > 1) {
            const int step = (hi - lo + 31) / 32, at = lo + lane * step;
            const uint32_t m = __ballot_sync(0xffffffffu, at < hi && P.cu[min(at, P.B)] / PP + at <= x);
            lo += m ? (31 - __clz(m)) * step : 0;
            hi = min(hi, lo + step);
        }
        const int s0 = P.cu[lo], s1 = P.cu[lo + 1];
        const bool good = s0 >= 0 && s1 >= s0 && s1 <= P.T && s1 - s0 <= P.max_seq_len;
        const int p0 = (x - (s0 / PP + lo)) * PP;
        if (lane == 0) {
            where[0] = s0;
            where[1] = good && p0 >= 0 && p0 < s1 - s0 ? s1 - s0 : 0;   // 0: nothing to do
            where[2] = p0;
            if (hk == 0 && x < P.B) {                       // every sequence's bounds are looked at once
                const int c0 = P.cu[x], c1 = P.cu[x + 1];
                if (c0 < 0 || c1 < c0 || c1 > P.T || c1 - c0 > P.max_seq_len) flag(FP8KV_DEV_BAD_SEQ_LEN);
            }
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    const int t0 = where[0], len = where[1], p0 = where[2];
    // per row tile i: positions p0 + i NP ..., keys [klo, khi] that its rows
    // see, key tiles [jlo, jhi)
    const int n_tiles_rows = len == 0 ? 0 : (p0 + P.NP < len ? 2 : 1);
    auto key_lo = [&](int i) { return P.window_left >= 0 ? max(0, p0 + i * P.NP - P.window_left) : 0; };
    auto key_hi = [&](int i) { return min(len - 1, p0 + (i + 1) * P.NP - 1); };
    const int j0 = key_lo(0) / NK, j1 = len ? key_hi(max(n_tiles_rows - 1, 0)) / NK + 1 : 0;
    const int n = j1 - j0;                                  // key tiles of the CTA
    const int jlo1 = key_lo(1) / NK, jhi0 = len ? key_hi(0) / NK + 1 : 0;
    // key tiles of row tile i, counted from j0: [lo_of(i), hi_of(i))
    auto lo_of = [&](int i) { return i ? jlo1 - j0 : 0; };
    auto hi_of = [&](int i) { return i ? (n_tiles_rows == 2 ? n : lo_of(1)) : jhi0 - j0; };
    // V rows that no row of the CTA sees, in the first and the last key tile:
    // such a V tile lands on a barrier of its own, for warp 10, which clears
    // those rows and then arrives on the slot's barrier
    const int see_lo = key_lo(0), see_hi = len ? key_hi(n_tiles_rows - 1) : 0;
    const bool clean_first = j0 * NK < see_lo, clean_last = j1 * NK - 1 > see_hi;
    auto cleaned = [&](int j) { return (j == n - 1 && clean_last) || (j == 0 && clean_first); };
    bool ok = true;

    if (n_tiles_rows == 0) {
        // no rows here
    } else if (warp == 0) {
        // ------------------------------------------------------------ loads
        if (lane == 0) {
            uint64_t keep;                                  // K and V are read by many CTAs, Q by one
            asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
            mbar_expect_tx(bar(B_Q), n_tiles_rows * 2 * rows * 128);
            for (int i = 0; i < n_tiles_rows; ++i)
                for (int h = 0; h < 2; ++h)
                    tma_load_3d(smem_u32(qs + i * SLOT + h * HALF), &tm_q, 64 * h, hk * P.G, t0 + p0 + i * P.NP,
                                bar(B_Q), policy_evict_first());
            int done = 0, raw = 0;
            for (int it = 0; it < 2 * n && ok; ++it) {
                // item -> tile: K0, then K(j), V(j - 1) in turn, V(n - 1) last
                const bool is_k = it == 0 || ((it & 1) && it != 2 * n - 1);
                const int j = it == 0 ? 0 : (it == 2 * n - 1 ? n - 1 : ((it & 1) ? (it + 1) / 2 : it / 2 - 1));
                const int s = it % SLOTS, use = it / SLOTS;
                if (use > 0) ok = mbar_wait(bar(B_EMPTY + s), (use - 1) & 1);
                if (!ok) break;
                const uint32_t full = !is_k && cleaned(j) ? bar(B_RAW + (j == n - 1)) : bar(B_FULL + s);
                mbar_expect_tx(full, SLOT);
                for (int h = 0; h < 2; ++h)
                    tma_load_3d(smem_u32(ring + s * SLOT + h * HALF), is_k ? &tm_k : &tm_v, 64 * h, hk,
                                t0 + (j0 + j) * NK, full, keep);
                done = it + 1;
                if (full != bar(B_FULL + s)) raw |= 1 << (j == n - 1);
            }
            // never leave with copies into this CTA's shared memory in flight
            mbar_wait(bar(B_Q), 0);
            for (int e = 0; e < 2; ++e)
                if (raw >> e & 1) mbar_wait(bar(B_RAW + e), 0);
            for (int it = max(0, done - SLOTS); it < done; ++it) mbar_wait(bar(B_FULL + it % SLOTS), (it / SLOTS) & 1);
        }
        __syncwarp();
    } else if (warp == 1) {
        // --------------------------------------------------------- MMA issue
        if (lane == 0) {
            ok = mbar_wait(bar(B_Q), 0);
            for (int j = 0; j <= n && ok; ++j) {
                for (int i = 0; i < n_tiles_rows && ok; ++i) {
                    if (j >= 1 && j - 1 >= lo_of(i) && j - 1 < hi_of(i)) {
                        // O_i += P_i(j - 1) V(j - 1)
                        const int vi = v_item(j - 1, n), c = j - 1 - lo_of(i);
                        ok = mbar_wait(bar(B_FULL + vi % SLOTS), (vi / SLOTS) & 1);
                        const uint32_t vt = smem_u32(ring + (vi % SLOTS) * SLOT);
                        for (int h = 0; h < 2 && ok; ++h) {
                            ok = mbar_wait(bar(B_P + 2 * i + h), c & 1);
                            if (!ok) break;
                            fence_after();
#pragma unroll
                            for (int kk = 4 * h; kk < 4 * h + 4; ++kk)
                                mma_f16_ts(tmem + TM_O + 128 * i, tmem + TM_S + 128 * i + 8 * kk,
                                           sdesc(vt + kk * 2048, HALF, 1024), ID_PV, (c > 0 || kk > 0));
                        }
                        if (ok && j - 1 == hi_of(i) - 1) mma_commit(bar(B_O + i));
                    }
                    if (ok && j < n && j >= lo_of(i) && j < hi_of(i)) {
                        // S_i = Q_i K(j)^T (over P_i(j - 1), which the MMAs above have read)
                        const int ki = k_item(j);
                        ok = mbar_wait(bar(B_FULL + ki % SLOTS), (ki / SLOTS) & 1);
                        if (!ok) break;
                        fence_after();
                        const uint32_t kt = smem_u32(ring + (ki % SLOTS) * SLOT), qt = smem_u32(qs + i * SLOT);
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks) {
                            const uint32_t off = (ks >> 2) * HALF + (ks & 3) * 32;
                            mma_f16_ss(tmem + TM_S + 128 * i, sdesc(qt + off, 16, 1024), sdesc(kt + off, 16, 1024),
                                       ID_QK, ks > 0);
                        }
                        mma_commit(bar(B_S + i));
                    }
                }
                // the slots this step has read, once its MMAs are complete
                if (ok && j < n) mma_commit(bar(B_EMPTY + k_item(j) % SLOTS));
                if (ok && j >= 1) mma_commit(bar(B_EMPTY + v_item(j - 1, n) % SLOTS));
            }
            // nothing the tensor cores still run may outlive the TMEM allocation
            mma_commit(bar(B_IDLE));
            mbar_wait(bar(B_IDLE), 0);
        }
        __syncwarp();
    } else if (warp == 10) {
        // ----------------------------------------------- V rows nobody sees
        for (int e = 0; e < 2; ++e) {
            const int j = e ? n - 1 : 0;
            if (!cleaned(j) || (e == 0 && j == n - 1)) continue;
            const int vi = v_item(j, n), k0 = (j0 + j) * NK;
            ok = mbar_wait(bar(B_RAW + e), 0);
            if (!__all_sync(0xffffffffu, ok)) break;
            uint8_t* vt = ring + (vi % SLOTS) * SLOT;
            const int a = max(0, min(NK, see_lo - k0)), z = max(0, min(NK, see_hi + 1 - k0));
            for (int i = lane; i < NK * 8; i += 32) {       // rows [0, a) and [z, 128)
                const int r = i >> 3;
                if (r >= a && r < z) continue;
                *(uint4*)(vt + i * 16) = make_uint4(0, 0, 0, 0);
                *(uint4*)(vt + HALF + i * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_FULL + vi % SLOTS));
        }
    } else if ((warp - 2) >> 2 < n_tiles_rows) {
        // ----------------------------------------------------------- softmax
        const int i = (warp - 2) >> 2, wq = warp & 3;
        const int r = wq * 32 + lane;
        const int base = p0 + i * P.NP;                     // first position of the row tile
        const int pos = base + min(r, rows - 1) / P.G;
        const int lo_r = P.window_left >= 0 ? max(0, pos - P.window_left) : 0;
        // the warp's bounds: key tiles inside them need no mask
        const int pmin = base + min(wq * 32, rows - 1) / P.G;
        const int plast = base + min(wq * 32 + 31, rows - 1) / P.G;
        const int lomax = P.window_left >= 0 ? max(0, plast - P.window_left) : 0;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t s_col = lanes + TM_S + 128 * i, o_col = lanes + TM_O + 128 * i;
        const float mult = P.scale_log2;
        const int a = lo_of(i), z = hi_of(i);
        float m_run = -INFINITY, l_run = 0.f;
#pragma unroll 1
        for (int j = a; j < z; ++j) {
            const int k0 = (j0 + j) * NK;
            ok = mbar_wait(bar(B_S + i), (j - a) & 1);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            fence_after();
            uint32_t sv[4][32];
#pragma unroll
            for (int c = 0; c < 4; ++c) tmem_ld_x32(s_col + 32 * c, sv[c]);
            tmem_wait_ld();
            if (k0 + NK - 1 > pmin || k0 < lomax) {
                // visible columns [c0, c1) of this row
                const int c0 = lo_r - k0, c1 = pos - k0 + 1;
#pragma unroll
                for (int c = 0; c < 4; ++c)
#pragma unroll
                    for (int u = 0; u < 32; ++u)
                        if (32 * c + u < c0 || 32 * c + u >= c1) sv[c][u] = 0xff800000u;   // -inf
            }
            float m4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                m4[c] = __uint_as_float(sv[c][0]);
#pragma unroll
                for (int u = 1; u < 32; ++u) m4[c] = fmaxf(m4[c], __uint_as_float(sv[c][u]));
            }
            const float tmax = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3])) * mult;
            const bool grow = m_run != -INFINITY && tmax > m_run + 8.0f;
            if (__any_sync(0xffffffffu, grow)) {
                // S(j) ready means that P.V of the tiles before is complete
                const float alpha = grow ? ex2(m_run - tmax) : 1.0f;
#pragma unroll 1
                for (int c = 0; c < 128; c += 32) {
                    uint32_t ov[32];
                    tmem_ld_x32(o_col + c, ov);
                    tmem_wait_ld();
#pragma unroll
                    for (int u = 0; u < 32; ++u) ov[u] = __float_as_uint(__uint_as_float(ov[u]) * alpha);
                    tmem_st_x32(o_col + c, ov);
                }
                tmem_wait_st();
                if (grow) {
                    l_run *= alpha;
                    m_run = tmax;
                }
            }
            if (m_run == -INFINITY) m_run = tmax;
            const float neg = m_run == -INFINITY ? 0.f : -m_run;
            const uint64_t mult2 = pack2(mult, mult), neg2 = pack2(neg, neg);
            uint64_t sum2 = 0;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                uint32_t pw[16];
#pragma unroll
                for (int u = 0; u < 16; ++u) {
                    float x0, x1;
                    unpack2(fma2(pack2(__uint_as_float(sv[c][2 * u]), __uint_as_float(sv[c][2 * u + 1])), mult2, neg2),
                            x0, x1);
                    x0 = ex2(x0);
                    x1 = ex2(x1);
                    sum2 = add2(sum2, pack2(x0, x1));
                    pw[u] = pack_bf16x2(x0, x1);
                }
                tmem_st_x16(s_col + 16 * c, pw);
                if (c & 1) {                                // 64 columns of P: their MMAs may start
                    tmem_wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_P + 2 * i + (c >> 1)));
                }
            }
            float s0, s1;
            unpack2(sum2, s0, s1);
            l_run += s0 + s1;
        }
        // ---------------------------------------------------------- epilogue
        if (ok) ok = mbar_wait(bar(B_O + i), 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok) {
            fence_after();
            const float inv = 1.0f / l_run;
            const bool whole = base + P.NP <= len;          // every used row is one of the sequence
            uint8_t* stage = qs + i * SLOT;                 // Q of this tile is consumed
            const bool live = r < rows && base + r / P.G < len;
            uint16_t* dst = P.out + ((int64_t)(t0 + pos) * P.Hq + hk * P.G + min(r, rows - 1) % P.G) * 128;
#pragma unroll 1
            for (int c = 0; c < 128; c += 32) {
                uint32_t ov[32];
                tmem_ld_x32(o_col + c, ov);
                tmem_wait_ld();
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    uint32_t w[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        w[e] = pack_bf16x2(__uint_as_float(ov[8 * v4 + 2 * e]) * inv,
                                           __uint_as_float(ov[8 * v4 + 2 * e + 1]) * inv);
                    const uint4 q4 = make_uint4(w[0], w[1], w[2], w[3]);
                    if (whole)
                        *(uint4*)(stage + (c >> 6) * HALF + r * 128 + (((((c & 63) >> 3) + v4) ^ (r & 7)) << 4)) = q4;
                    else if (live)
                        *(uint4*)(dst + c + 8 * v4) = q4;
                }
            }
            if (whole) {
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_STAGE + i));
                if (warp == 2 + 4 * i && lane == 0 && mbar_wait(bar(B_STAGE + i), 0)) {
                    for (int h = 0; h < 2; ++h)
                        tma_store_3d(&tm_o, smem_u32(stage + h * HALF), 64 * h, hk * P.G, t0 + base);
                    bulk_commit();
                    bulk_wait_read();
                }
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
    }
}

}  // namespace prompt
}  // namespace fp8kv

using namespace fp8kv;

static bool al16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

extern "C" int fp8kv_prompt_attention(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v,
                                      int64_t v_stride, const int32_t* cu_seqlens, int B, int T, int max_seq_len,
                                      int Hq, int Hkv, int D, float sm_scale, int window_left, void* out,
                                      void* stream) {
    if (B < 0 || T < 0 || max_seq_len < 0 || Hq <= 0 || Hkv <= 0 || Hq % Hkv || window_left < -1)
        return FP8KV_ERR_INVALID_ARG;
    if (!(sm_scale > 0.0f) || !(sm_scale <= 3.0e38f)) return FP8KV_ERR_INVALID_ARG;
    if (D != 128 || Hq / Hkv > 128 || Hkv > 65535) return FP8KV_ERR_UNSUPPORTED;
    for (int64_t st : {q_stride - (int64_t)Hq * 128, k_stride - (int64_t)Hkv * 128, v_stride - (int64_t)Hkv * 128})
        if (st < 0 || st % 8 || st > (1ll << 32)) return FP8KV_ERR_INVALID_ARG;
    const int G = Hq / Hkv, NP = 128 / G;
    const int64_t pairs = (int64_t)T / (2 * NP) + B;
    if (pairs > 65535) return FP8KV_ERR_UNSUPPORTED;
    if (B == 0 || T == 0) return FP8KV_OK;                      // nothing to do; no pointer is read
    if (!q || !k || !v || !cu_seqlens || !out) return FP8KV_ERR_INVALID_ARG;
    if (!al16(q) || !al16(k) || !al16(v) || !al16(out)) return FP8KV_ERR_INVALID_ARG;
    CUtensorMap tq, tk, tv, to;
    if (!rows_map(&tq, q, Hq, q_stride, T, G, NP) || !rows_map(&tk, k, Hkv, k_stride, T, 1, prompt::NK) ||
        !rows_map(&tv, v, Hkv, v_stride, T, 1, prompt::NK) || !rows_map(&to, out, Hq, (int64_t)Hq * 128, T, G, NP))
        return FP8KV_ERR_CUDA;
    {
        static std::mutex mu;
        static std::set<int> done;
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess) return FP8KV_ERR_CUDA;
        std::lock_guard<std::mutex> lock(mu);
        if (!done.count(dev)) {
            if (cudaFuncSetAttribute(prompt::prompt_attention_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     prompt::SMEM) != cudaSuccess)
                return FP8KV_ERR_CUDA;
            done.insert(dev);
        }
    }
    prompt::Params P = {};
    P.cu = cu_seqlens;
    P.out = (uint16_t*)out;
    P.B = B;
    P.T = T;
    P.Hq = Hq;
    P.Hkv = Hkv;
    P.G = G;
    P.NP = NP;
    P.window_left = window_left;
    P.max_seq_len = max_seq_len;
    P.scale_log2 = sm_scale * 1.4426950408889634f;
    const dim3 grid((unsigned)Hkv, (unsigned)pairs);
    const cudaError_t e = launch_pdl(prompt::prompt_attention_kernel, grid, dim3(prompt::THREADS), prompt::SMEM,
                                     (cudaStream_t)stream, tq, tk, tv, to, P);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return FP8KV_ERR_CUDA;
    }
    char text[256];
    snprintf(text, sizeof text, "prompt_attention_tc rows=2x%d positions=2x%d grid=%dx%d threads=%d", G * NP, NP, Hkv,
             (int)pairs, prompt::THREADS);
    set_dispatch(text);
    return FP8KV_OK;
}
