// attention_int4_tc.cu -- verifier rows (more than 16 per KV head) over the INT4
// cache on the 5th-generation tensor cores.
//
// What bounds it: a tile of 128 keys is 18 KiB of pages, 800 cycles of one SM's
// share of the HBM rate; its two products with 128 rows are 1024 cycles of the
// tensor cores; and widened to f16 its K and V are written to shared memory
// once and read once by the tensor cores (with Q in tensor memory), which with
// the pages themselves is 164 KiB, 1300 cycles of shared-memory bandwidth.
// That last figure is the bound.
//
// The values n s / 4 are exact in f16 (attention_int4.cu); within groups of
// eight dimensions they are stored in the order 0 4 1 5 2 6 3 7 in which the
// codes of a word widen, Q likewise, and the output is put back in order when
// it is written.  Q rows are scaled by a power of two into f16's range.
//
// One CTA per (partition, row tile x KV head, sequence), 20 warps:
//   warp 0           loads pages (bulk copies of the codes and of the scales of
//                    a (page, head)) into a ring of 128-key stages
//   warp 1           issues S = Q.K^T of the half tiles (64 keys) u = 0, 1, ...,
//                    into three S buffers in turn
//   warp 2           issues O += P(u).V
//   warps 4-7, 8-11  softmax of the even and of the odd half tiles, a row per
//                    thread (warps 4+q and 8+q: TMEM lane quarter q).  Each of
//                    the two keeps its own maximum, sum and O, merged at the
//                    end, so that they never wait for each other.  (One softmax
//                    over whole tiles, the maximum exchanged through shared
//                    memory, took 2800 cycles a tile; two with one S buffer
//                    each, which idle while their next product runs, 2600.)  O
//                    is rescaled when a row's maximum grows by more than 2^4;
//                    the weights are held as 2^11 times 2^(x - m), at most
//                    2^15, so that f16 keeps 11 bits of every weight down to
//                    2^-25 of the largest.
//   warps 12-19      widen K and V into swizzled f16 tiles (five warps took 3700
//                    cycles a tile).  New tokens (append) are encoded by these
//                    warps, a block of 16 elements a thread, written to the cache
//                    and, so that no load has to wait for that, over their rows
//                    of the staged pages (512 keys: 10.3 us; loads that wait 13.4,
//                    an append kernel before this one 12.7).
// At most 8 partitions in one wave of CTAs: those of a (sequence, KV head) are a
// thread-block cluster, and each CTA merges its share of the rows from the
// others' shared memory (12 rows x 9 heads, 512 keys: 8.9 us; partials through
// memory and a reduce kernel 10.3).
// TMEM columns: Q 0-63, S/P 3 x 64 (64-255), O 256-383, 384-511.
#include <stdio.h>

#include "attention.cuh"
#include "common.cuh"
#include "int4.cuh"
#include "tcgen05.cuh"

namespace fp8kv {

int status_attention_int4_tc(unsigned int* s, int clear) { return read_status(s, clear); }

namespace i4tc {

constexpr int NK = 128;                                 // keys per tile
constexpr int STAGES = 5;
constexpr int OFF_V = NK * kInt4CodeBytes;              // of a stage: K codes, V codes, K scales, V scales
constexpr int OFF_KS = 2 * NK * kInt4CodeBytes;
constexpr int OFF_VS = OFF_KS + NK * kInt4ScaleBytes;
constexpr int STAGE_BYTES = OFF_VS + NK * kInt4ScaleBytes;
constexpr int KBUFS = 2, VBUFS = 2;                     // widened tiles
constexpr int BUF = NK * 256, HALF = BUF / 2;           // two blocks of 128 keys x 64 dims (128-byte swizzled)
constexpr int XCH_BYTES = 2 * 128 * 8;                  // (max, sum) of [half][row]
constexpr int SMEM = (KBUFS + VBUFS) * BUF + STAGES * STAGE_BYTES + XCH_BYTES + 1024 + 512;
constexpr int EPI_STRIDE = 144;                         // staged half row (128 bytes), padded against bank conflicts
constexpr int kMaxCluster = 8;
static_assert(2 * 128 * EPI_STRIDE + 128 * 8 <= (KBUFS + VBUFS) * BUF, "epilogue staging exceeds the widened tiles");
constexpr uint32_t TM_Q = 0, TM_S = 64, TM_O = 256, TM_COLS = 512;
constexpr int WARPS = 20, THREADS = WARPS * 32, CONV_WARPS = 8;
// registers: 640 x 96 at launch = 128 x (3 x 72 + 2 x 128) after the split
constexpr int REGS_SERVICE = 72, REGS_SOFTMAX = 128;
static_assert(128 * (3 * REGS_SERVICE + 2 * REGS_SOFTMAX) <= THREADS * 96, "register split above the launch's share");
constexpr float GROW = 4.0f, BIAS = 11.0f;              // see the head of the file

enum {
    B_STG_FULL = 0,
    B_STG_EMPTY = B_STG_FULL + STAGES,
    B_K_FULL = B_STG_EMPTY + STAGES,
    B_K_EMPTY = B_K_FULL + KBUFS,
    B_V_FULL = B_K_EMPTY + KBUFS,
    B_V_EMPTY = B_V_FULL + VBUFS,
    B_S = B_V_EMPTY + VBUFS,                            // per softmax half and its tile mod 3: S ready
    B_P = B_S + 6,                                      // ... P written
    B_S_EMPTY = B_P + 6,                                // per S buffer: P.V of the P over it complete
    B_PV = B_S_EMPTY + 3,                               // per half: its last P.V complete
    B_O = B_PV + 2,                                     // per half: O final
    B_Q_READY = B_O + 2,
    B_IDLE = B_Q_READY + 1,
    B_PAIR = B_IDLE + 1,                                // per TMEM lane quarter: its two softmax warps
    B_APP = B_PAIR + 4,                                 // new tokens written over a staged tile
    B_COUNT = B_APP + 1
};
static_assert(B_COUNT * 8 + 16 <= 512, "barrier area");

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(src), "r"(bytes), "r"(bar)
                 : "memory");
}

// 32 codes (16 bytes, two blocks), widened into four 16-byte units of shared
// memory at `at[u]` + off.
template <int OFF>
__device__ __forceinline__ void widen_chunk(const uint32_t (&at)[4], uint4 codes, uint32_t scales) {
    const uint32_t s2 = e4m3x2_to_f16x2(scales);
    const Scale2 sa = scale2(prmt(s2, s2, 0x1010)), sb = scale2(prmt(s2, s2, 0x3232));
    const uint32_t w[4] = {codes.x, codes.y, codes.z, codes.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        uint32_t v[4];
        widen4(w[u], u < 2 ? sa : sb, v);
        asm volatile("st.shared.v4.b32 [%0 + %5], {%1, %2, %3, %4};" ::"r"(at[u]), "r"(v[0]), "r"(v[1]), "r"(v[2]),
                     "r"(v[3]), "n"(OFF)
                     : "memory");
    }
}

template <int PS, bool CL>     // CL: the partitions are a cluster
__global__ void __launch_bounds__(THREADS, 1) attention_int4_tc_kernel(AttnParams P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* kbuf = smem;                                   // KBUFS x 32 KiB
    uint8_t* vbuf = kbuf + KBUFS * BUF;                     // VBUFS x 32 KiB
    uint8_t* stg = vbuf + VBUFS * BUF;                      // STAGES x 18 KiB
    float* xch = (float*)(stg + STAGES * STAGE_BYTES);
    uint64_t* bars = (uint64_t*)((uint8_t*)xch + XCH_BYTES);
    uint32_t* tmem_slot = (uint32_t*)(bars + B_COUNT);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int RT = (P.R + 127) >> 7;
    const int rt = blockIdx.y % RT;
    int split = blockIdx.x, hk = blockIdx.y / RT, b = blockIdx.z;
    const int R0 = rt * 128, RL = min(128, P.R - R0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            int count = 1;
            if ((i >= B_STG_EMPTY && i < B_K_EMPTY) || (i >= B_V_FULL && i < B_V_EMPTY)) count = CONV_WARPS;
            if (i >= B_P && i < B_S_EMPTY) count = 4;
            if (i == B_Q_READY) count = 8;
            if (i >= B_IDLE && i < B_APP) count = 2;
            if (i == B_APP) count = CONV_WARPS;
            mbar_init(bar(i), count);
        }
        fence_barrier_init();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(TM_COLS)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    bool have_work = true;
    if (P.lpt_order) {
        // CTA i: KV head i mod Hkv of the slot of rank i / Hkv, longest first
        const int lin = blockIdx.x + gridDim.x * (blockIdx.y + gridDim.y * blockIdx.z);
        const int q = P.lpt_order[lin / P.Hkv];
        hk = lin % P.Hkv;
        if (q < 0) {
            have_work = false;
        } else {
            b = q / P.num_splits;
            split = q % P.num_splits;
        }
    }
    // the first page ids, right unless a window moves the partition, are read
    // beside the length
    constexpr int PPT = NK / PS;                            // pages per tile
    int guess_at = -1, guess = -1;
    if (warp == 0) {
        guess_at = min(split * P.split_pages + ((lane >> 2) & (PPT - 1)), P.mpps - 1);
        guess = P.block_table[(int64_t)b * P.mpps + guess_at];
    }
    // so are the new tokens: block ct % 8 of token ct / 8 (at most 16)
    const int ct = threadIdx.x - 12 * 32;
    const bool has_new = P.k_new && ct >= 0 && ct < P.M * 8;
    uint4 nk[2] = {}, nv[2] = {};
    if (has_new) {
        const int64_t src = ((((int64_t)b * P.M + (ct >> 3)) * P.Hkv + hk) * 8 + (ct & 7)) * 2;
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            nk[u] = ((const uint4*)P.k_new)[src + u];
            nv[u] = ((const uint4*)P.v_new)[src + u];
        }
    }
    const int L = P.seq_lens[b];
    const bool seq_ok = !(L < P.M || L > P.max_seq_len || (L + PS - 1) / PS > P.mpps);
    bool run = seq_ok && have_work;                         // uniform over the CTA
    if (!seq_ok && !P.lpt_order && threadIdx.x == 0 && split == 0 && blockIdx.y == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
    // keys visible to any row of the tile: from the first row's window start
    // to the last row's position (row r is query m = r / G at L - M + m)
    const int hi0 = L - P.M + (R0 + RL - 1) / P.G;
    const int lo0 = (P.window_left >= 0) ? max(0, L - P.M + R0 / P.G - P.window_left) : 0;
    const int first_page = lo0 / PS, last_page = hi0 / PS;
    const int nsplit_b = (last_page - first_page + P.split_pages) / P.split_pages;
    if (run && nsplit_b > P.num_splits) {
        if (threadIdx.x == 0 && split == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
        run = false;
    }
    if (split >= nsplit_b) run = false;
    const int page_begin = first_page + split * P.split_pages;
    const int n_pages = min(P.split_pages, last_page + 1 - page_begin);
    const int n_tiles = (n_pages + PPT - 1) / PPT;
    const int k_begin = page_begin * PS;
    // append: the tiles that hold new tokens ([L - M, L) within the partition)
    const int app_lo = max(L - P.M, k_begin), app_hi = min(L, k_begin + n_pages * PS);
    const bool appends = P.k_new && app_lo < app_hi;
    const int app_t0 = appends ? (app_lo - k_begin) / NK : 1 << 30, app_t1 = appends ? (app_hi - 1 - k_begin) / NK : -1;
    bool ok = true;

    if (!run) {
        // no keys of this sequence fall in this partition (or bad input)
    } else if (warp >= 4 && warp < 12) {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REGS_SOFTMAX));
        // ------------------------------------------------------------ softmax
        const int wq = warp & 3, half = (warp - 4) >> 2;
        const int r = wq * 32 + lane;
        const bool active = wq * 32 < RL;                   // the quarter holds at least one real row
        const uint32_t lane_base = tmem + ((uint32_t)(wq * 32) << 16);
        const int rr = R0 + min(r, RL - 1);                 // the row of the (b, hk) block
        const int m = rr / P.G;
        const int p_r = L - P.M + m;
        const int lo_r = (P.window_left >= 0) ? max(0, p_r - P.window_left) : 0;
        const int64_t row_idx = ((int64_t)b * P.M + m) * P.Hq + hk * P.G + rr % P.G;
        const float vs = 4.0f * *P.v_scale;
        const bool pad = r >= RL;                           // rows past M x G: Q = 0
        float mult;
        {
            // this half's 64 dims of the row, times a power of two that puts
            // the row maximum (of all 128) in [2^4, 2^5), as f16 into TMEM
            const uint4* src = (const uint4*)(P.q + row_idx * 128) + 8 * half;
            uint32_t qh[32];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint4 w = pad ? make_uint4(0, 0, 0, 0) : src[u];
                qh[4 * u] = w.x;
                qh[4 * u + 1] = w.y;
                qh[4 * u + 2] = w.z;
                qh[4 * u + 3] = w.w;
            }
            uint32_t am = 0;
#pragma unroll
            for (int u = 0; u < 32; ++u) am = max_bf16x2(am, qh[u] & 0x7fff7fffu);
            xch[half * 128 + r] = fmaxf(bf16_lo(am), bf16_hi(am));
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_PAIR + wq));
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_PAIR + wq), 0));
            const float amax = fmaxf(xch[r], xch[128 + r]);
            int e = 4;
            const uint32_t ab = __float_as_uint(amax);
            if (amax > 0.f && ((ab >> 23) & 0xff) != 0xff) {
                const int be = (int)((ab >> 23) & 0xff);
                e = be ? be - 127 : -127;
            }
            const int sh = max(-120, min(120, 4 - e));
            // (the sign of sm_scale goes into q: the row maximum is taken before
            // the multiplication)
            const float scale = copysignf(ldexpf(1.0f, sh), P.sm_scale);
            mult = fmaxf(4.0f * *P.k_scale * fabsf(P.sm_scale) * 1.4426950408889634f * ldexpf(1.0f, -sh), 1e-37f);
            uint32_t qf[32];
#pragma unroll
            for (int u = 0; u < 8; ++u) {                   // dims 8u .. + 7 in the order 0 4 1 5 2 6 3 7
                const uint32_t* x = qh + 4 * u;
                qf[4 * u] = pack_f16x2(bf16_lo(x[0]) * scale, bf16_lo(x[2]) * scale);
                qf[4 * u + 1] = pack_f16x2(bf16_hi(x[0]) * scale, bf16_hi(x[2]) * scale);
                qf[4 * u + 2] = pack_f16x2(bf16_lo(x[1]) * scale, bf16_lo(x[3]) * scale);
                qf[4 * u + 3] = pack_f16x2(bf16_hi(x[1]) * scale, bf16_hi(x[3]) * scale);
            }
            tmem_st_x32(lane_base + TM_Q + 32 * half, qf);
            tmem_wait_st();
        }
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_Q_READY));

        int pmin = p_r, lomax = lo_r, pmax = p_r, lomin = lo_r;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            pmin = min(pmin, __shfl_xor_sync(0xffffffffu, pmin, off));
            lomax = max(lomax, __shfl_xor_sync(0xffffffffu, lomax, off));
            pmax = max(pmax, __shfl_xor_sync(0xffffffffu, pmax, off));
            lomin = min(lomin, __shfl_xor_sync(0xffffffffu, lomin, off));
        }
        // this half's maximum and sum
        float m_run = -INFINITY, l_run = 0.f;
        const uint32_t o_col = lane_base + TM_O + 128 * half;
        for (int t = 0; t < n_tiles && ok; ++t) {
            const uint32_t s_col = lane_base + TM_S + 64 * ((2 * t + half) % 3);
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_S + 3 * half + t % 3), (t / 3) & 1));
            if (!ok) break;
            fence_after();
            const int k0 = k_begin + t * NK + 64 * half;    // first key of this half
            if (!active || k0 > pmax || k0 + 63 < lomin) {
                // no row of this warp sees any key of it: P = 0
                uint32_t zero[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) zero[j] = 0u;
                tmem_st_x32(s_col, zero);
            } else {
                uint32_t sv[64];
                tmem_ld_x64(s_col, sv);
                tmem_wait_ld();
                if (k0 + 63 > pmin || k0 < lomax) {
                    // this row's visible columns of the half as bits
                    const int jlo = max(0, lo_r - k0), jhi = min(64, p_r - k0 + 1);
                    const uint64_t below_hi = jhi <= 0 ? 0ull : (jhi >= 64 ? ~0ull : (1ull << jhi) - 1);
                    const uint64_t below_lo = jlo >= 64 ? ~0ull : (1ull << jlo) - 1;
                    const uint64_t vis = below_hi & ~below_lo;
                    const uint32_t vis_lo = (uint32_t)vis, vis_hi = (uint32_t)(vis >> 32);
#pragma unroll
                    for (int j = 0; j < 64; ++j)
                        sv[j] = (((j < 32 ? vis_lo : vis_hi) >> (j & 31)) & 1u) ? sv[j] : 0xff800000u;   // -inf
                }
                float m4[4];
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    m4[c] = max3(__uint_as_float(sv[c]), __uint_as_float(sv[c + 4]), __uint_as_float(sv[c + 8]));
#pragma unroll
                    for (int u = c + 12; u < 60; u += 8)
                        m4[c] = max3(m4[c], __uint_as_float(sv[u]), __uint_as_float(sv[u + 4]));
                    m4[c] = fmaxf(m4[c], __uint_as_float(sv[60 + c]));
                }
                const float tmax = max3(m4[0], m4[1], fmaxf(m4[2], m4[3])) * mult;
                const bool rescale = (m_run != -INFINITY) && (tmax > m_run + GROW);
                if (__any_sync(0xffffffffu, rescale)) {
                    // O holds P.V up to tile t - 1 (t > 0: m_run was set): wait for it
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(B_PV + half), (t - 1) & 1));
                    if (!ok) break;
                    fence_after();
                    const float alpha = rescale ? ex2(m_run - tmax) : 1.0f;
#pragma unroll 1
                    for (int c = 0; c < 128; c += 32) {
                        uint32_t ov[32];
                        tmem_ld_x32(o_col + c, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int j = 0; j < 32; ++j) ov[j] = __float_as_uint(__uint_as_float(ov[j]) * alpha);
                        tmem_st_x32(o_col + c, ov);
                    }
                    tmem_wait_st();
                    if (rescale) {
                        l_run *= alpha;
                        m_run = tmax;
                    }
                }
                if (m_run == -INFINITY) m_run = tmax;
                // P = 2^(s mult - m + 11) as f16 (masked keys are -inf and give 0)
                const float neg = (m_run == -INFINITY) ? 0.f : BIAS - m_run;
                const uint64_t mult2 = pack2(mult, mult), neg2 = pack2(neg, neg);
                uint64_t sum2 = 0;
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t pw[16];
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        float p0, p1;
                        unpack2(fma2(pack2(__uint_as_float(sv[32 * c + 2 * j]), __uint_as_float(sv[32 * c + 2 * j + 1])),
                                     mult2, neg2),
                                p0, p1);
                        p0 = ex2(p0);
                        p1 = ex2(p1);
                        sum2 = add2(sum2, pack2(p0, p1));
                        pw[j] = pack_f16x2(p0, p1);
                    }
                    tmem_st_x16(s_col + 16 * c, pw);
                }
                float sum0, sum1;
                unpack2(sum2, sum0, sum1);
                l_run += sum0 + sum1;
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + 3 * half + t % 3));
        }
        // ------------------------------------------------------------ epilogue
        // both halves' O and (max, sum); this thread merges 64 dims of its row
        for (int h = 0; h < 2; ++h)
            if (ok) ok = mbar_wait(bar(B_O + h), 0);
        const bool combine = CL && nsplit_b > 1;
        float2* ml = (float2*)xch;
        float2* ml_all = (float2*)(kbuf + 2 * 128 * EPI_STRIDE);    // (max, sum) of the staged rows
        ml[half * 128 + r] = make_float2(m_run, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PAIR + wq));
        if (ok) ok = mbar_wait(bar(B_PAIR + wq), 1);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && active) {
            fence_after();
            const float2 a = ml[r], z = ml[128 + r];
            const float m_tot = fmaxf(a.x, z.x);
            const float wa = a.x == -INFINITY ? 0.f : ex2(a.x - m_tot), wz = z.x == -INFINITY ? 0.f : ex2(z.x - m_tot);
            const float l_tot = a.y * wa + z.y * wz;
            const bool direct = nsplit_b == 1;
            // direct: bf16 of 4 v_scale O / l; partial: f16 of 4 O / l (|x| <=
            // 7 * 448) beside its (max, sum); a row with no visible key here
            // has l = 0: weight 0, values 0
            const float f = direct ? vs / l_tot : (l_tot > 0.f ? 4.0f / l_tot : 0.f);
            const float fa = wa * f, fz = wz * f;
            // the half row goes through shared memory (the widened tiles are
            // free) to one bulk copy
            uint8_t* row_stage = kbuf + (half * 128 + r) * EPI_STRIDE;
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                uint32_t oa[32], oz[32];
                tmem_ld_x32(lane_base + TM_O + 64 * half + c, oa);
                tmem_ld_x32(lane_base + TM_O + 128 + 64 * half + c, oz);
                tmem_wait_ld();
                uint4* dst = (uint4*)(row_stage + c * 2);
#pragma unroll
                for (int v4 = 0; v4 < 4; ++v4) {
                    float x[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        x[i] = __uint_as_float(oa[8 * v4 + i]) * fa + __uint_as_float(oz[8 * v4 + i]) * fz;
                    // columns 0 4 1 5 2 6 3 7 back in order
                    dst[v4] = direct ? make_uint4(pack_bf16x2(x[0], x[2]), pack_bf16x2(x[4], x[6]),
                                                  pack_bf16x2(x[1], x[3]), pack_bf16x2(x[5], x[7]))
                                     : make_uint4(pack_f16x2(x[0], x[2]), pack_f16x2(x[4], x[6]),
                                                  pack_f16x2(x[1], x[3]), pack_f16x2(x[5], x[7]));
                }
            }
            if (combine) {
                // stays here: the cluster's CTAs read it below
                if (half == 0) ml_all[r] = make_float2(m_tot, l_tot);
            } else if (r < RL) {
                fence_proxy_async();        // the staged row, written by this thread, to the bulk copy
                if (direct)
                    bulk_store(P.out + row_idx * 128 + 64 * half, smem_u32(row_stage), 128);
                else
                    bulk_store((uint16_t*)P.ws_o + (row_idx * P.num_splits + split) * 128 + 64 * half,
                               smem_u32(row_stage), 128);
                bulk_commit();
                bulk_wait_read();
                if (!direct && half == 0)
                    *(float2*)(P.ws_ml + (row_idx * P.num_splits + split) * 2) = make_float2(m_tot, l_tot);
            }
        }
        if (CL) {
            __syncwarp();
            cluster_arrive();
            cluster_wait();
        }
        if (combine) {
            // the partitions of this KV head are a cluster (rank = partition):
            // each merges every nsplit_b-th row, 16 threads a row
            const int c = threadIdx.x & 15;
            for (int row = split + nsplit_b * ((threadIdx.x - 128) >> 4); row < RL; row += 16 * nsplit_b) {
                const uint8_t* at = kbuf + ((c >> 3) * 128 + row) * EPI_STRIDE + (c & 7) * 16;
                float2 a[kMaxCluster];
                float top = -INFINITY, den = 0.f, acc[8] = {};
#pragma unroll
                for (int j = 0; j < kMaxCluster; ++j) {
                    a[j] = j < nsplit_b ? dsmem_ld8(dsmem_addr(ml_all + row, j)) : make_float2(-INFINITY, 0.f);
                    top = fmaxf(top, a[j].x);
                }
#pragma unroll
                for (int j = 0; j < kMaxCluster; ++j) {
                    if (j >= nsplit_b) break;
                    const uint4 x = dsmem_ld16(dsmem_addr(at, j));
                    const float w = a[j].x == -INFINITY ? 0.f : ex2(a[j].x - top) * a[j].y;
                    const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
                    den += w;
#pragma unroll
                    for (int u = 0; u < 4; ++u) {
                        const float2 f = f16x2_to_f32x2(xs[u]);
                        acc[2 * u] += w * f.x;
                        acc[2 * u + 1] += w * f.y;
                    }
                }
                const float f = 0.25f * vs / den;
                const int64_t idx = ((int64_t)b * P.M + row / P.G) * P.Hq + hk * P.G + row % P.G;
                *(uint4*)(P.out + idx * 128 + 8 * c) =
                    make_uint4(pack_bf16x2(acc[0] * f, acc[1] * f), pack_bf16x2(acc[2] * f, acc[3] * f),
                               pack_bf16x2(acc[4] * f, acc[5] * f), pack_bf16x2(acc[6] * f, acc[7] * f));
            }
        }
    } else {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REGS_SERVICE));
        if (warp == 0) {
            // ---------------------------------------------------------- producer
            // lane 4 p + k: copy k (K codes, V codes, K scales, V scales) of page p
            // of the tile; a page id outside the pool reads as zeros
            const int32_t* bt = P.block_table + (int64_t)b * P.mpps + page_begin;
            const int p = lane >> 2, kind = lane & 3;
            const uint8_t* cache = kind & 1 ? P.v_cache : P.k_cache;
            const uint32_t bytes = kind < 2 ? PS * kInt4CodeBytes : PS * kInt4ScaleBytes;
            const uint32_t off = (kind == 0 ? 0 : kind == 1 ? OFF_V : kind == 2 ? OFF_KS : OFF_VS) + p * bytes;
            int issued = 0;
            int next = p < PPT && p < n_pages ? (page_begin + p == guess_at ? guess : bt[p]) : -1;
            for (int t = 0; t < n_tiles; ++t) {
                const int s = t % STAGES, use = t / STAGES, page = next, at = t * PPT + p;
                const bool mine = p < PPT && at < n_pages;
                next = p < PPT && at + PPT < n_pages ? bt[at + PPT] : -1;
                if (use > 0) ok = mbar_wait(bar(B_STG_EMPTY + s), (use - 1) & 1);
                if (!__all_sync(0xffffffffu, ok)) break;
                uint8_t* dst = stg + s * STAGE_BYTES + off;
                const bool valid = mine && page >= 0 && page < P.num_pages;
                if (mine && !valid) {
                    for (uint32_t i = 0; i < bytes; i += 16) *(uint4*)(dst + i) = make_uint4(0, 0, 0, 0);
                    fence_proxy_async();                        // before a later tile's copy over them
                }
                uint32_t total = valid ? bytes : 0;
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
                __syncwarp();                                   // every lane's zeros, before the arrival (the shuffles
                                                                // order no memory)
                if (lane == 0) mbar_expect_tx(bar(B_STG_FULL + s), total);
                __syncwarp();
                if (valid)
                    bulk_load(smem_u32(dst),
                              cache + ((int64_t)page * P.Hkv + hk) * (PS * kInt4RowBytes) +
                                  (kind < 2 ? 0 : PS * kInt4CodeBytes),
                              bytes, bar(B_STG_FULL + s));
                issued = t + 1;
            }
            // never leave with copies into this CTA's shared memory in flight
            for (int t = max(0, issued - STAGES); t < issued; ++t) mbar_wait(bar(B_STG_FULL + t % STAGES), (t / STAGES) & 1);
            __syncwarp();
        } else if (warp == 1 || warp == 2) {
            // ------------------------------------------------------ MMA issue
            constexpr uint32_t ID_QK = idesc(128, NK / 2, false), ID_PV = idesc(128, 128, true);
            const bool leader = elect_one();
            const int n_half = 2 * n_tiles;
            if (warp == 1) {
                // S(u) = Q K^T; the K buffer is free once the second half has read it
                const uint32_t k_lo = desc_lo(smem_u32(kbuf), 16);
                ok = mbar_wait(bar(B_Q_READY), 0);
                for (int u = 0; u < n_half; ++u) {
                    const int t = u >> 1, h = u & 1, tb = t % KBUFS, sb = u % 3;
                    if (ok && h == 0) ok = mbar_wait(bar(B_K_FULL + tb), (t / KBUFS) & 1);
                    if (ok && u >= 3) ok = mbar_wait(bar(B_S_EMPTY + sb), (u / 3 - 1) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    fence_after();
                    if (leader) {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(tmem + TM_S + 64 * sb, tmem + TM_Q + 8 * ks,
                                   k_lo + ((tb * BUF + h * (64 * 128) + (ks >> 2) * HALF + (ks & 3) * 32) >> 4), ID_QK,
                                   ks > 0);
                        mma_commit(bar(B_S + 3 * h + t % 3));
                        if (h == 1) mma_commit(bar(B_K_EMPTY + tb));
                    }
                    __syncwarp();
                }
            } else {
                // O += P(u) V
                const uint32_t v_lo = desc_lo(smem_u32(vbuf), HALF);
                for (int u = 0; u < n_half; ++u) {
                    const int t = u >> 1, h = u & 1, vb = t % VBUFS, sb = u % 3;
                    if (h == 0) ok = mbar_wait(bar(B_V_FULL + vb), (t / VBUFS) & 1);
                    if (ok) ok = mbar_wait(bar(B_P + 3 * h + t % 3), (t / 3) & 1);
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) break;
                    fence_after();
                    if (leader) {
#pragma unroll
                        for (int kk = 0; kk < 4; ++kk)
                            mma_ts(tmem + TM_O + 128 * h, tmem + TM_S + 64 * sb + 8 * kk,
                                   v_lo + ((vb * BUF + h * (64 * 128) + kk * 2048) >> 4), ID_PV, t > 0 || kk > 0);
                        mma_commit(bar(B_PV + h));
                        mma_commit(bar(B_S_EMPTY + sb));
                        if (h == 1) mma_commit(bar(B_V_EMPTY + vb));
                        if (t == n_tiles - 1) mma_commit(bar(B_O + h));
                    }
                    __syncwarp();
                }
            }
            // nothing the tensor cores still run may outlive the TMEM allocation
            if (leader) mma_commit(bar(B_IDLE));
            __syncwarp();
            mbar_wait(bar(B_IDLE), 0);
            __syncwarp();
        } else if (warp >= 12) {
            // ---------------------------------------------------------- widening
            // items of (key, 32 dims); eight lanes cover four keys x two chunks,
            // which keeps the 16-byte stores free of bank conflicts.  A warp has
            // 16 keys: 8 (cw + 8 u) + ..., u = 0, 1
            const int cw = warp - 12;
            const int r0 = 8 * cw + ((lane >> 1) & 3) + 4 * (lane >> 4), cc = (lane & 1) + 2 * ((lane >> 3) & 1);
            // where the four 16-byte units of row r0's chunk go in a tile
            // (swizzled by the row; row r0 + 64 is 8 KiB further)
            uint32_t at[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
                at[u] = smem_u32(kbuf) + (cc >> 1) * HALF + r0 * 128 + (((4 * (cc & 1) + u) ^ (r0 & 7)) << 4);
            uint4 kc[2], vc[2];
            uint32_t ksc[2], vsc[2];
            auto load_k = [&](int t) {
                const uint8_t* src = stg + (t % STAGES) * STAGE_BYTES;
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = r0 + 64 * u;
                    kc[u] = *(const uint4*)(src + r * 64 + cc * 16);
                    ksc[u] = *(const uint16_t*)(src + OFF_KS + r * 8 + 2 * cc);
                }
            };
            auto load_v = [&](int t) {
                const uint8_t* src = stg + (t % STAGES) * STAGE_BYTES;
                // keys outside every row's range get V scale 0: whatever their
                // bytes are, zeros reach the output
                const int k0 = k_begin + t * NK;
                const int zlo = lo0 - k0, zhi = min(min(NK, (n_pages - t * PPT) * PS), hi0 + 1 - k0);
#pragma unroll
                for (int u = 0; u < 2; ++u) {
                    const int r = r0 + 64 * u;
                    vc[u] = *(const uint4*)(src + OFF_V + r * 64 + cc * 16);
                    vsc[u] = *(const uint16_t*)(src + OFF_VS + r * 8 + 2 * cc);
                    if (r < zlo || r >= zhi) vsc[u] = 0;
                }
            };
            // this thread's new block: its row of the partition, or none
            Int4Block fresh;
            int fresh_row = -1;
            if (appends && has_new && L - P.M + (ct >> 3) >= app_lo && L - P.M + (ct >> 3) < app_hi) {
                const int pos = L - P.M + (ct >> 3), page = P.block_table[(int64_t)b * P.mpps + pos / PS];
                fresh = Int4Block(nk[0], nk[1], nv[0], nv[1], *P.k_scale, *P.v_scale);
                if (page >= 0 && page < P.num_pages) {
                    fresh_row = pos - k_begin;
                    fresh.store(P.k_cache, P.v_cache, page, pos % PS, hk, P.Hkv, PS, ct & 7);
                } else if ((ct & 7) == 0) {
                    flag(FP8KV_DEV_BAD_SLOT);
                }
            }
            // the new rows of tile t over its stage
            auto patch = [&](int t) {
                uint8_t* dst = stg + (t % STAGES) * STAGE_BYTES;
                const int r = fresh_row - t * NK;
                if (fresh_row >= 0 && r >= 0 && r < NK) {
                    *(uint2*)(dst + r * 64 + 8 * (ct & 7)) = fresh.k;
                    *(uint2*)(dst + OFF_V + r * 64 + 8 * (ct & 7)) = fresh.v;
                    dst[OFF_KS + r * 8 + (ct & 7)] = fresh.ks;
                    dst[OFF_VS + r * 8 + (ct & 7)] = fresh.vs;
                    fence_proxy_async();                        // before the stage's next load
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_APP));
                ok = __all_sync(0xffffffffu, mbar_wait(bar(B_APP), (t - app_t0) & 1));
            };
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_STG_FULL), 0));
            if (ok && app_t0 == 0) patch(0);
            if (ok) {
                load_k(0);
                load_v(0);
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_STG_EMPTY));           // the stage is in registers
            }
            for (int t = 0; t < n_tiles && ok; ++t) {
                // K of this tile, then the next stage's K on its way while V of
                // this tile is widened
                const int tb = t % KBUFS, vb = t % VBUFS, s1 = (t + 1) % STAGES;
                if (t >= KBUFS) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_K_EMPTY + tb), (t / KBUFS - 1) & 1));
                if (!ok) break;
                uint32_t to[4];
#pragma unroll
                for (int u = 0; u < 4; ++u) to[u] = at[u] + tb * BUF;
                widen_chunk<0>(to, kc[0], ksc[0]);
                widen_chunk<64 * 128>(to, kc[1], ksc[1]);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_K_FULL + tb));
                if (t + 1 < n_tiles) {
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(B_STG_FULL + s1), ((t + 1) / STAGES) & 1));
                    if (ok && t + 1 >= app_t0 && t + 1 <= app_t1) patch(t + 1);
                    if (!ok) break;
                    load_k(t + 1);
                }
                if (t >= VBUFS) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_V_EMPTY + vb), (t / VBUFS - 1) & 1));
                if (!ok) break;
#pragma unroll
                for (int u = 0; u < 4; ++u) to[u] = at[u] + (KBUFS + vb) * BUF;
                widen_chunk<0>(to, vc[0], vsc[0]);
                widen_chunk<64 * 128>(to, vc[1], vsc[1]);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_V_FULL + vb));
                if (t + 1 < n_tiles) {
                    load_v(t + 1);
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_STG_EMPTY + s1));
                }
            }
        }
    }

    // ---------------------------------------------------------------- teardown
    if (CL) {
        // every warp of the cluster takes part in both barriers: the one before
        // the rows are merged, and this one, before any shared memory goes
        __syncwarp();
        if (!run || warp < 4 || warp >= 12) {
            cluster_arrive();
            cluster_wait();
        }
        cluster_arrive();
        cluster_wait();
    }
    fence_before();
    __syncthreads();
    if (warp == 0) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(TM_COLS) : "memory");
    }
}

}  // namespace i4tc

int launch_attention_int4_tc(const AttnParams& P, cudaStream_t s, char* text, size_t text_bytes) {
    const int RT = (P.R + 127) / 128;
    if (P.cluster > 1 && (P.cluster > i4tc::kMaxCluster || P.cluster != P.num_splits || RT > 1 || P.lpt_order))
        return FP8KV_ERR_UNSUPPORTED;
    if ((P.split_pages * P.page_size) % i4tc::NK || (int64_t)RT * P.Hkv > 65535) return FP8KV_ERR_UNSUPPORTED;
    static std::atomic<uint64_t> done[2][2];                // [page size][cluster]
    auto kern = P.page_size == 32
                    ? (P.cluster > 1 ? i4tc::attention_int4_tc_kernel<32, true> : i4tc::attention_int4_tc_kernel<32, false>)
                    : (P.cluster > 1 ? i4tc::attention_int4_tc_kernel<64, true> : i4tc::attention_int4_tc_kernel<64, false>);
    if (opt_in_smem(done[P.page_size == 64][P.cluster > 1], (const void*)kern, i4tc::SMEM) != cudaSuccess)
        return (cudaGetLastError(), FP8KV_ERR_CUDA);
    const dim3 grid(P.num_splits, P.Hkv * RT, P.B);
    const cudaError_t e = launch_pdl_cluster(kern, grid, dim3(i4tc::THREADS), i4tc::SMEM, s, P.cluster, P);
    if (e != cudaSuccess) {
        cudaGetLastError();
        return FP8KV_ERR_CUDA;
    }
    snprintf(text, text_bytes,
             "attention_int4_tc<ps=%d> rows=%d row_tiles=%d splits=%d split_tokens=%d grid=%dx%dx%d threads=%d cluster=%d "
             "reduce=%d order=%s",
             P.page_size, P.R, RT, P.num_splits, P.split_pages * P.page_size, P.num_splits, P.Hkv * RT, P.B,
             i4tc::THREADS, P.cluster > 1 ? P.cluster : 1, P.num_splits > 1 && P.cluster <= 1 ? 1 : 0, P.lpt_order ? "longest_first" : "grid");
    return FP8KV_OK;
}

}  // namespace fp8kv
