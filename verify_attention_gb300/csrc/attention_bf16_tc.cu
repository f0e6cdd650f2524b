// attention_bf16_tc.cu -- trees of drafted tokens (more than 16 rows per KV head)
// over the BF16 cache on the 5th-generation tensor cores.
//
// K and V are operands as they are stored: TMA brings a (page, head) as two boxes
// of 64 dims, whose 128-byte rows with the 128-byte swizzle are the K-major operand
// of S = Q.K^T and the MN-major operand of O += P.V, so nothing is widened or
// copied on the way.  Q and P (softmax weights rounded to bf16) are in tensor
// memory, accumulators are fp32.
//
// What bounds it: a tile of 128 keys is 64 KiB of pages, 2900 cycles of one SM's
// share of the HBM rate, and its two products with 128 rows are 1024 cycles of the
// tensor cores.  With several row tiles (64 nodes x 9 heads: 5) each reads the keys
// again, from L2.
//
// One CTA per (partition, row tile x KV head, sequence), 12 warps:
//   warp 0       TMA producer (tiles of 128 keys into a ring of three stages)
//   warp 1       issues S = Q.K^T, into two S buffers in turn
//   warp 2       issues O += P.V
//   warp 3       zeroes V rows that no row of the tile sees (behind the sequence's
//                end, before its first window): whatever is stored there, 0 times
//                it must not reach the output
//   warps 4-11   softmax: warps 4+q and 8+q share TMEM lane quarter q (32 rows, one
//                a thread) and split the tile's 128 key columns; O is rescaled when
//                a row's maximum grows by more than 2^8
// One sequence in 2 to 8 partitions of one row tile: those of a KV head are a
// thread-block cluster, and each CTA merges its share of the rows from the others'
// shared memory.
// TMEM columns: Q 0-63, S/P 2 x 128 (64-319), O 320-447.
#include <stdio.h>

#include "attention.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace fp8kv {

int status_attention_bf16_tc(unsigned int* s, int clear) { return read_status(s, clear); }

namespace b16tc {

constexpr int NK = 128;                                 // keys per tile
constexpr int STAGES = 3;
constexpr int HALF = NK * 128;                          // a block of 64 dims
constexpr int STG_BYTES = 4 * HALF;                     // K: two blocks, V: two blocks
constexpr int XCH_BYTES = 3 * 2 * 128 * 4;              // [tile parity 0, parity 1, row sums][half][row]
constexpr int SMEM = STAGES * STG_BYTES + XCH_BYTES + 1024 + 512;
// epilogue, in the ring (free once the last tile is consumed): half rows, fp32 or
// bf16, padded against bank conflicts; behind them (max, sum) of the rows
constexpr int EPI_STRIDE = 272;
static_assert(2 * 128 * EPI_STRIDE + 128 * 8 <= STAGES * STG_BYTES, "epilogue staging exceeds the stage ring");
constexpr uint32_t TM_Q = 0, TM_S = 64, TM_O = 320, TM_COLS = 512;
constexpr int WARPS = 12, THREADS = WARPS * 32, kMaxCluster = 8;
constexpr float GROW = 8.0f;

enum {
    B_STG_FULL = 0,
    B_STG_EMPTY = B_STG_FULL + STAGES,
    B_S_FULL = B_STG_EMPTY + STAGES,
    B_P_FULL = B_S_FULL + 2,
    B_S_EMPTY = B_P_FULL + 2,                           // per S buffer: P.V of the P over it complete
    B_O_DONE = B_S_EMPTY + 2,
    B_O_FINAL = B_O_DONE + 1,
    B_Q_READY = B_O_FINAL + 1,
    B_IDLE = B_Q_READY + 1,
    B_PAIR = B_IDLE + 1,                                // per TMEM lane quarter: its two softmax warps
    B_CLEAN = B_PAIR + 4,                               // V rows of the first, the last tile zeroed
    B_COUNT = B_CLEAN + 2
};
static_assert(B_COUNT * 8 + 16 <= 512, "barrier area");

constexpr uint32_t BF16 = (1u << 7) | (1u << 10);       // A and B format of kind::f16

template <int PS, bool CL>     // CL: the partitions are a cluster
__global__ void __launch_bounds__(THREADS, 1) attention_bf16_tc_kernel(const __grid_constant__ CUtensorMap tm_k,
                                                                      const __grid_constant__ CUtensorMap tm_v,
                                                                      AttnParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stg = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    float* xch = (float*)(stg + STAGES * STG_BYTES);    // [parity][half][row]
    uint64_t* bars = (uint64_t*)((uint8_t*)xch + XCH_BYTES);
    uint32_t* tmem_slot = (uint32_t*)(bars + B_COUNT);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    // the row tiles of one head are neighbours in launch order and share its pages in L2
    const int RT = (P.R + 127) >> 7;
    const int rt = blockIdx.y % RT, split = blockIdx.x, hk = blockIdx.y / RT, b = blockIdx.z;
    const int R0 = rt * 128, RL = min(128, P.R - R0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            int count = 1;
            if (i >= B_STG_EMPTY && i < B_S_FULL) count = 3;    // Q.K^T, P.V, warp 3
            if (i >= B_P_FULL && i < B_S_EMPTY) count = 8;
            if (i == B_Q_READY) count = 8;
            if (i == B_IDLE) count = 2;
            if (i >= B_PAIR && i < B_CLEAN) count = 2;
            mbar_init(bar(i), count);
        }
        fence_barrier_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        if (lane == 0) {
            prefetch_tensormap(&tm_k);
            prefetch_tensormap(&tm_v);
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    const int L = P.seq_lens[b];
    bool run = !(L < P.M || L > P.max_seq_len || (L + PS - 1) / PS > P.mpps);   // uniform over the CTA
    if (!run && threadIdx.x == 0 && split == 0 && blockIdx.y == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
    const int lo0 = (P.window_left >= 0) ? max(0, L - P.M - P.window_left) : 0;
    const int first_page = lo0 / PS, last_page = (L - 1) / PS;
    const int nsplit_b = (last_page - first_page + P.split_pages) / P.split_pages;
    if (run && nsplit_b > P.num_splits) {
        if (threadIdx.x == 0 && split == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
        run = false;
    }
    const bool combine = CL && run && nsplit_b > 1;
    if (split >= nsplit_b) run = false;
    const int page_begin = first_page + split * P.split_pages;
    const int n_pages = min(P.split_pages, last_page + 1 - page_begin);
    constexpr int PPT = NK / PS;                            // pages per tile
    const int n_tiles = (n_pages + PPT - 1) / PPT;
    const int k_begin = page_begin * PS;
    // V rows of tile t to be zeroed: those outside [zlo, zhi)
    auto zlo_of = [&](int t) { return max(0, lo0 - (k_begin + t * NK)); };
    auto zhi_of = [&](int t) { return min(NK, L - (k_begin + t * NK)); };
    auto dirty = [&](int t) { return (t == 0 && zlo_of(t) > 0) || (t == n_tiles - 1 && zhi_of(t) < NK); };
    bool ok = true;

    if (!run) {
        // no keys of this sequence fall in this partition (or bad input)
    } else if (warp == 0) {
        // ---------------------------------------------------------- producer
        // lane 4 p + j: box j (K dims 0-63, 64-127, V likewise) of page p of the tile
        const uint64_t policy = policy_evict_first();
        const int32_t* bt = P.block_table + (int64_t)b * P.mpps + page_begin;
        const int p = lane >> 2, box = lane & 3;
        int issued = 0;
        int next = p < PPT && p < n_pages ? bt[p] : 0;
        for (int t = 0; t < n_tiles; ++t) {
            const int s = t % STAGES, use = t / STAGES, phys = next, at = t * PPT + p;
            const bool mine = p < PPT && at < n_pages;
            next = p < PPT && at + PPT < n_pages ? bt[at + PPT] : 0;
            if (use > 0) ok = mbar_wait(bar(B_STG_EMPTY + s), (use - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            if (lane == 0) mbar_expect_tx(bar(B_STG_FULL + s), min(PPT, n_pages - t * PPT) * PS * 512);
            __syncwarp();
            if (mine)
                tma_load_3d(smem_u32(stg + s * STG_BYTES + box * HALF + p * PS * 128), box < 2 ? &tm_k : &tm_v,
                            64 * (box & 1), hk * PS, phys, bar(B_STG_FULL + s), policy);
            __syncwarp();
            issued = t + 1;
        }
        // never leave with copies into this CTA's shared memory in flight
        for (int t = max(0, issued - STAGES); t < issued; ++t) mbar_wait(bar(B_STG_FULL + t % STAGES), (t / STAGES) & 1);
        __syncwarp();
    } else if (warp == 1 || warp == 2) {
        // ------------------------------------------------------ MMA issue
        constexpr uint32_t ID_QK = idesc(128, NK, false) | BF16, ID_PV = idesc(128, 128, true) | BF16;
        const bool leader = elect_one();
        if (warp == 1) {
            const uint32_t k_lo = desc_lo(smem_u32(stg), 16);
            ok = mbar_wait(bar(B_Q_READY), 0);
            for (int t = 0; t < n_tiles; ++t) {
                const int s = t % STAGES, sb = t & 1;
                if (ok) ok = mbar_wait(bar(B_STG_FULL + s), (t / STAGES) & 1);
                if (ok && t >= 2) ok = mbar_wait(bar(B_S_EMPTY + sb), ((t >> 1) - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fence_after();
                if (leader) {
#pragma unroll
                    for (int ks = 0; ks < 8; ++ks)
                        mma_ts(tmem + TM_S + 128 * sb, tmem + TM_Q + 8 * ks,
                               k_lo + ((s * STG_BYTES + (ks >> 2) * HALF + (ks & 3) * 32) >> 4), ID_QK, ks > 0);
                    mma_commit(bar(B_S_FULL + sb));
                    mma_commit(bar(B_STG_EMPTY + s));
                }
                __syncwarp();
            }
        } else {
            const uint32_t v_lo = desc_lo(smem_u32(stg + 2 * HALF), HALF);
            for (int t = 0; t < n_tiles; ++t) {
                const int s = t % STAGES, sb = t & 1;
                ok = mbar_wait(bar(B_STG_FULL + s), (t / STAGES) & 1);
                if (ok && dirty(t)) ok = mbar_wait(bar(B_CLEAN + (t > 0)), 0);
                if (ok) ok = mbar_wait(bar(B_P_FULL + sb), (t >> 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fence_after();
                if (leader) {
#pragma unroll
                    for (int kk = 0; kk < NK / 16; ++kk)
                        mma_ts(tmem + TM_O, tmem + TM_S + 128 * sb + 8 * kk, v_lo + ((s * STG_BYTES + kk * 2048) >> 4),
                               ID_PV, t > 0 || kk > 0);
                    mma_commit(bar(B_O_DONE));
                    mma_commit(bar(B_S_EMPTY + sb));
                    mma_commit(bar(B_STG_EMPTY + s));
                    if (t == n_tiles - 1) mma_commit(bar(B_O_FINAL));
                }
                __syncwarp();
            }
        }
        // nothing the tensor cores still run may outlive the TMEM allocation
        if (leader) mma_commit(bar(B_IDLE));
        __syncwarp();
        mbar_wait(bar(B_IDLE), 0);
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------- V rows without a reader
        for (int t = 0; t < n_tiles; ++t) {
            const int s = t % STAGES;
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_STG_FULL + s), (t / STAGES) & 1));
            if (!ok) break;
            if (dirty(t)) {
                const int zlo = zlo_of(t), zhi = zhi_of(t);
                uint8_t* v = stg + s * STG_BYTES + 2 * HALF;
                for (int i = lane; i < NK * 16; i += 32) {
                    const int r = i >> 4;
                    if (r < zlo || r >= zhi) *(uint4*)(v + ((i >> 3) & 1) * HALF + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_CLEAN + (t > 0)));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_STG_EMPTY + s));
        }
    } else {
        // ------------------------------------------------------------ softmax
        const int wq = warp & 3, half = (warp - 4) >> 2;
        const int r = wq * 32 + lane;
        const bool active = wq * 32 < RL;                   // the quarter holds at least one real row
        const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
        const int rr = R0 + min(r, RL - 1);                 // the row of the (b, hk) block
        const int m = rr / P.G, base = L - P.M;
        const int64_t row_idx = ((int64_t)b * P.M + m) * P.Hq + hk * P.G + rr % P.G;
        const bool pad = r >= RL;                           // rows past M x G: Q = 0
        const uint64_t word = tree_word(P, b, m);
        {
            const uint4* src = (const uint4*)(P.q + row_idx * 128) + 8 * half;
            uint32_t qw[32];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint4 w = pad ? make_uint4(0, 0, 0, 0) : src[u];
                qw[4 * u] = w.x;
                qw[4 * u + 1] = w.y;
                qw[4 * u + 2] = w.z;
                qw[4 * u + 3] = w.w;
            }
            // (the sign of sm_scale goes into q: the row maximum is taken before
            // the multiplication)
            if (P.sm_scale < 0.f)
#pragma unroll
                for (int u = 0; u < 32; ++u) qw[u] ^= 0x80008000u;
            tmem_st_x32(lane_base + TM_Q + 32 * half, qw);
            tmem_wait_st();
        }
        const float mult = fmaxf(fabsf(P.sm_scale) * 1.4426950408889634f, 1e-37f);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_Q_READY));
        const TreeRow tr = tree_row(P, b, m, word, base);
        int lomax = tr.lo;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) lomax = max(lomax, __shfl_xor_sync(0xffffffffu, lomax, off));
        float m_run = -INFINITY, l_run = 0.f;               // l_run: this half's columns only
        for (int t = 0; t < n_tiles; ++t) {
            const int sb = t & 1;
            ok = mbar_wait(bar(B_S_FULL + sb), (t >> 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
            fence_after();
            if (active) {
                const uint32_t scol = lane_base + TM_S + sb * 128 + 64 * half;
                const int k0 = k_begin + t * NK + 64 * half;   // first key of this half
                uint32_t sv[64];
                tmem_ld_x64(scol, sv);
                tmem_wait_ld();
                if (k0 + 63 >= base || k0 < lomax) {
                    const uint64_t vis = tree_sees64(tr, k0, base);
                    const uint32_t vis_lo = (uint32_t)vis, vis_hi = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        sv[j] = (((j < 32 ? vis_lo : vis_hi) >> (j & 31)) & 1u) ? sv[j] : 0xff800000u;   // -inf
                }
                float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                for (int j = 0; j < 64; j += 8) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
                        m4[c] = max3(m4[c], __uint_as_float(sv[j + c]), __uint_as_float(sv[j + 4 + c]));
                }
                xch[(sb * 2 + half) * 128 + r] = max3(m4[0], m4[1], fmaxf(m4[2], m4[3]));
                // exchange with the partner warp (phase t of the pair barrier)
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_PAIR + wq));
                ok = mbar_wait(bar(B_PAIR + wq), t & 1);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                const float tmax = fmaxf(xch[sb * 256 + r], xch[sb * 256 + 128 + r]) * mult;
                const bool rescale = (m_run != -INFINITY) && (tmax > m_run + GROW);
                if (__any_sync(0xffffffffu, rescale)) {
                    // O holds P.V up to tile t - 1: wait for it, then rescale this half
                    ok = mbar_wait(bar(B_O_DONE), (t - 1) & 1);
                    if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                    fence_after();
                    const float alpha = rescale ? ex2(m_run - tmax) : 1.0f;
#pragma unroll 1
                    for (int c = 0; c < 64; c += 32) {
                        uint32_t ov[32];
                        tmem_ld_x32(lane_base + TM_O + 64 * half + c, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
                        tmem_st_x32(lane_base + TM_O + 64 * half + c, ov);
                    }
                    tmem_wait_st();
                    if (rescale) {
                        l_run *= alpha;
                        m_run = tmax;
                    }
                }
                if (m_run == -INFINITY) m_run = tmax;
                // P = 2^(s mult - m) as bf16 (masked keys are -inf and give 0); both
                // halves' S reads are complete (pair barrier above)
                const float neg = (m_run == -INFINITY) ? 0.f : -m_run;
                const uint64_t mult2 = pack2(mult, mult), neg2 = pack2(neg, neg);
                uint64_t sum2 = 0;
                uint32_t pw[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float p0, p1;
                    unpack2(fma2(pack2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), mult2, neg2), p0, p1);
                    p0 = ex2(p0);
                    p1 = ex2(p1);
                    sum2 = add2(sum2, pack2(p0, p1));
                    pw[j] = pack_bf16x2(p0, p1);
                }
                tmem_st_x32(lane_base + TM_S + sb * 128 + 32 * half, pw);
                float s0, s1;
                unpack2(sum2, s0, s1);
                l_run += s0 + s1;
                tmem_wait_st();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P_FULL + sb));
        }
        // ------------------------------------------------------------ epilogue
        if (ok) ok = mbar_wait(bar(B_O_FINAL), 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && active) {
            fence_after();
            // row sums of both halves: phase n_tiles of the pair barrier
            xch[(4 + half) * 128 + r] = l_run;
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_PAIR + wq));
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_PAIR + wq), n_tiles & 1));
        }
        if (ok && active) {
            const float l_tot = xch[4 * 128 + r] + xch[5 * 128 + r];
            // (NaN scores only, which the maximum passes over: with the maximum 0
            // their NaN sum still counts where partitions are combined)
            if (m_run == -INFINITY && l_tot != l_tot) m_run = 0.f;
            const bool direct = nsplit_b == 1, zero = word == 0 || l_tot == 0.f;
            const float f = direct ? 1.0f / l_tot : 1.0f;
            // direct: bf16 of O / l; partial: fp32 O beside its (max, sum).  The half
            // row goes through the free ring to one bulk copy
            uint8_t* row_stage = stg + (half * 128 + r) * EPI_STRIDE;
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                uint32_t ov[32];
                tmem_ld_x32(lane_base + TM_O + 64 * half + c, ov);
                tmem_wait_ld();
                if (direct) {
                    uint4* dst = (uint4*)(row_stage + c * 2);
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = zero ? 0u
                                        : pack_bf16x2(__uint_as_float(ov[8 * v4 + 2 * j]) * f,
                                                      __uint_as_float(ov[8 * v4 + 2 * j + 1]) * f);
                        dst[v4] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                } else {
                    uint4* dst = (uint4*)(row_stage + c * 4);
#pragma unroll
                    for (int v4 = 0; v4 < 8; ++v4)
                        dst[v4] = make_uint4(ov[4 * v4], ov[4 * v4 + 1], ov[4 * v4 + 2], ov[4 * v4 + 3]);
                }
            }
            if (combine) {
                // stays here: the cluster's CTAs read it below
                if (half == 0) *(float2*)(stg + 2 * 128 * EPI_STRIDE + r * 8) = make_float2(m_run, l_tot);
            } else if (!pad) {
                fence_proxy_async();        // the staged row, written by this thread, to the bulk copy
                if (direct)
                    bulk_store(P.out + row_idx * 128 + 64 * half, smem_u32(row_stage), 128);
                else
                    bulk_store(P.ws_o + (row_idx * P.num_splits + split) * 128 + 64 * half, smem_u32(row_stage), 256);
                bulk_commit();
                bulk_wait_read();
                if (!direct && half == 0)
                    *(float2*)(P.ws_ml + (row_idx * P.num_splits + split) * 2) = make_float2(m_run, l_tot);
            }
        }
    }

    if (CL) {
        // ------------------------------------------------- cluster combine
        // rank = partition; each CTA merges every nsplit_b-th row, 32 threads a row:
        // O = sum_p w_p O_p / sum_p w_p l_p, w_p = 2^(m_p - m*)
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (combine && run) {
            for (int row = split + nsplit_b * warp; row < RL; row += nsplit_b * WARPS) {
                const uint8_t* at = stg + ((lane >> 4) * 128 + row) * EPI_STRIDE + (lane & 15) * 16;
                float2 a[kMaxCluster];
                uint4 x[kMaxCluster];
                float top = -INFINITY, den = 0.f, acc[4] = {};
#pragma unroll
                for (int j = 0; j < kMaxCluster; ++j) {
                    a[j] = make_float2(-INFINITY, 0.f);
                    if (j >= nsplit_b) continue;
                    a[j] = dsmem_ld8(dsmem_addr(stg + 2 * 128 * EPI_STRIDE + row * 8, j));
                    x[j] = dsmem_ld16(dsmem_addr(at, j));
                    top = fmaxf(top, a[j].x);
                }
#pragma unroll
                for (int j = 0; j < kMaxCluster; ++j) {
                    if (j >= nsplit_b) continue;
                    const float w = a[j].x == -INFINITY ? 0.f : ex2(a[j].x - top);
                    den += w * a[j].y;
                    acc[0] += w * __uint_as_float(x[j].x);
                    acc[1] += w * __uint_as_float(x[j].y);
                    acc[2] += w * __uint_as_float(x[j].z);
                    acc[3] += w * __uint_as_float(x[j].w);
                }
                const int m = (R0 + row) / P.G;
                const int64_t idx = ((int64_t)b * P.M + m) * P.Hq + hk * P.G + (R0 + row) % P.G;
                const float f = 1.0f / den;
                uint2 o2 = make_uint2(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f));
                if (den == 0.f || tree_word(P, b, m) == 0) o2 = make_uint2(0u, 0u);
                *(uint2*)(P.out + idx * 128 + 4 * lane) = o2;
            }
        }
        __syncwarp();
        cluster_arrive();                               // no shared memory goes before all have read
        cluster_wait();
    }
    // ---------------------------------------------------------------- teardown
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
    }
}

}  // namespace b16tc

int launch_attention_bf16_tc(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& P, cudaStream_t s,
                             char* text, size_t text_bytes) {
    const int RT = (P.R + 127) / 128;
    if (!P.tree || P.R <= 16 || (int64_t)RT * P.Hkv > 65535 || (P.split_pages * P.page_size) % b16tc::NK)
        return FP8KV_ERR_UNSUPPORTED;
    if (P.cluster > 1 && (P.cluster > b16tc::kMaxCluster || P.cluster != P.num_splits || RT > 1))
        return FP8KV_ERR_UNSUPPORTED;
    static std::atomic<uint64_t> done[2][2];                // [page size][cluster]
    const bool cl = P.cluster > 1;
    auto kern = P.page_size == 32
                    ? (cl ? b16tc::attention_bf16_tc_kernel<32, true> : b16tc::attention_bf16_tc_kernel<32, false>)
                    : (cl ? b16tc::attention_bf16_tc_kernel<64, true> : b16tc::attention_bf16_tc_kernel<64, false>);
    if (opt_in_smem(done[P.page_size == 64][cl], (const void*)kern, b16tc::SMEM) != cudaSuccess)
        return (cudaGetLastError(), FP8KV_ERR_CUDA);
    const dim3 grid(P.num_splits, P.Hkv * RT, P.B);
    const cudaError_t e = launch_pdl_cluster(kern, grid, dim3(b16tc::THREADS), b16tc::SMEM, s, P.cluster, tk, tv, P);
    if (e != cudaSuccess) return (cudaGetLastError(), FP8KV_ERR_CUDA);
    snprintf(text, text_bytes,
             "attention_bf16_tc<ps=%d> rows=%d row_tiles=%d splits=%d split_tokens=%d grid=%dx%dx%d threads=%d "
             "cluster=%d reduce=%d order=grid",
             P.page_size, P.R, RT, P.num_splits, P.split_pages * P.page_size, P.num_splits, P.Hkv * RT, P.B,
             b16tc::THREADS, cl ? P.cluster : 1, P.num_splits > 1 && !cl ? 1 : 0);
    return FP8KV_OK;
}

}  // namespace fp8kv
