// attention_tree_tc.cu -- trees of drafted tokens (more than 16 rows per KV head)
// over the E4M3 and the BF16 cache on the 5th-generation tensor cores.
//
// K is an operand as it is stored: TMA brings a (page, head) in rows of 128 bytes with
// the 128-byte swizzle, the K-major operand of S = Q.K^T.  So is V over a BF16 cache,
// as the MN-major operand of O += P.V; E4M3 V is widened (exactly) to f16 tiles.  Q is
// bf16, or split into two E4M3 terms, q 2^sh = Q_hi + Q_lo with the row maximum in
// [128, 256): exact for elements within 2^-10 of the row maximum, the others are off by
// at most 2^-17 of it.  Softmax weights are bf16, or f16 as 2^11 times 2^(x - m), at
// most 2^15, which keeps 11 bits down to 2^-25 of the largest.  Accumulators are fp32.
//
// What bounds it: a tile of 128 keys is 32 or 64 KiB of pages, 1400 or 2900 cycles of
// one SM's share of the HBM rate (long BF16 batches: 64 trees of 12 nodes, up to 32768
// keys, 772 us, 5.7 TB/s).  Its two products with 128 rows are 1032 cycles of the
// tensor cores, the way of a tile from its scores over the weights to the end of its
// second product some 2000, so what counts is how much of it runs side by side:
//   - the two softmax groups take half tiles (64 keys), each with its own maximum,
//     sum, O, S and P, merged at the end, and never wait for each other (E4M3, both on
//     one tile, its maximum exchanged through shared memory: 1.24 us a tile);
//   - S is read into registers at once, and the next one computed meanwhile;
//   - three threads issue the products (BF16: 0.80 us a tile; both halves' P.V by one
//     thread, which then is busy for 1300 cycles a tile, 0.86);
//   - BF16 stages of K and of V come and go by themselves (before: 0.89).
// BF16 takes 0.78 us a tile, E4M3 0.89 (64 trees of 12 nodes, up to 32768 keys: 495
// us): a softmax warp's way through a half tile (the wait for S 130 cycles, reading it
// 140, the maximum 240, the exponentials 700, P 140) with the products' between them;
// the widening of V has to stay below that (addresses computed for each chunk, and its
// halves exchanged after they were widened: 1.07; eight warps for it instead of four, as
// it was then: 1.20).
//
// One CTA per (partition, row tile x KV head, sequence):
//   warp 0       TMA producer (tiles of 128 keys into rings of K and V stages); BF16: of
//                K, warp 12 of V
//   warp 1       issues S = Q.K^T of both halves of a tile (a product of 128 x 64 x 16
//                takes 55 cycles to issue, one of 128 x 128 x 16 64)
//   warps 2, 3   issue O += P.V of the even and of the odd half tiles
//   warps 4-7, 8-11  softmax of the even and of the odd half tiles, a row a thread
//                (warps 4+q and 8+q: TMEM lane quarter q); O is rescaled when a row's
//                maximum grows by more than 2^GROW
//   warps 12-15  E4M3: widen V; with tokens to append they encode those, one 8-element
//                chunk a thread, and write them over their rows of the staged tile and
//                into the f16 tile, the cache afterwards
//   warp 13      BF16: zeroes V rows that no row of the tile sees (behind the sequence's
//                end, before its first window, padding nodes): whatever is stored there, 0
//                times it must not reach the output (E4M3: they are widened as zeros)
// One sequence in 2 to 8 partitions: those of a KV head and row tile are a
// thread-block cluster, and each CTA merges its share of the rows from the others'
// shared memory.
// TMEM columns: Q 0-63, S 64-127, 128-191, P 192-223, 224-255, O 256-383, 384-511.
#include <stdio.h>

#include "attention.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace fp8kv {

int status_attention_tree_tc(unsigned int* s, int clear) { return read_status(s, clear); }

namespace ttc {

constexpr int NK = 128;                                 // keys per tile
constexpr int HALF = NK * 128;                          // a block of rows of 128 bytes: 128 E4M3 or 64 bf16 dims
constexpr int VBUFS = 2, VBUF = 2 * HALF;               // E4M3: V widened to f16, two blocks of 64 dims
constexpr int kMaxStages = 4;
template <bool FP8>
struct Cfg {
    static constexpr int STAGES = FP8 ? kMaxStages : 3;
    static constexpr int STG = (FP8 ? 1 : 2) * HALF;    // of K, or of V
    static constexpr int OFF_V = STAGES * STG;          // V stages behind K's
    static constexpr int WARPS = FP8 ? 16 : 14, THREADS = 32 * WARPS, CONV = FP8 ? 4 : 1;
    static constexpr int RING = 2 * STAGES * STG;
    static constexpr int SMEM = RING + (FP8 ? VBUFS * VBUF : 0) + 3 * 2 * 128 * 4 + 1024 + 512;
};
// epilogue, in the ring (free once the last tile is consumed): half rows, f16, bf16 or
// fp32, padded against bank conflicts; behind them (max, sum) of the rows
constexpr int EPI_STRIDE = 272;
static_assert(2 * 128 * EPI_STRIDE + 128 * 8 <= Cfg<true>::RING && Cfg<true>::RING <= Cfg<false>::RING,
              "epilogue staging exceeds the stage ring");
constexpr uint32_t TM_Q = 0, TM_S = 64, TM_P = 192, TM_O = 256, TM_COLS = 512;
constexpr int kMaxCluster = 8;

enum {
    B_K_FULL = 0,                                       // stages of K and of V
    B_K_EMPTY = B_K_FULL + kMaxStages,
    B_W_FULL = B_K_EMPTY + kMaxStages,
    B_W_EMPTY = B_W_FULL + kMaxStages,
    B_V_FULL = B_W_EMPTY + kMaxStages,                  // E4M3: widened V
    B_V_EMPTY = B_V_FULL + VBUFS,
    B_S = B_V_EMPTY + VBUFS,                            // per half: S ready
    B_S_READ = B_S + 2,                                 // ... S read
    B_P = B_S_READ + 2,                                 // ... P written
    B_PV = B_P + 2,                                     // ... its last P.V complete
    B_O = B_PV + 2,                                     // per half: O final
    B_Q_READY = B_O + 2,
    B_IDLE = B_Q_READY + 1,
    B_PAIR = B_IDLE + 1,                                // per TMEM lane quarter: its two softmax warps
    B_CLEAN = B_PAIR + 4,                               // BF16: V rows of the first, the last, the last but one tile zeroed
    B_PATCH = B_CLEAN + 3,                              // appended K rows written over a staged tile, one barrier for
                                                        // each of the (at most two) tiles that hold any
    B_COUNT = B_PATCH + 2
};
static_assert(B_COUNT * 8 + 16 + Cfg<true>::CONV * 8 <= 512, "barrier area");

template <int PS, bool FP8, bool CL>     // CL: the partitions are a cluster
__global__ void __launch_bounds__(Cfg<FP8>::THREADS, 1) attention_tree_tc_kernel(
    const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v, AttnParams P) {
    using C = Cfg<FP8>;
    constexpr int STAGES = C::STAGES;
    constexpr float GROW = FP8 ? 4.0f : 8.0f, BIAS = FP8 ? 11.0f : 0.0f;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* stg = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* vbuf = stg + C::RING;                          // E4M3: VBUFS f16 tiles
    float* xch = (float*)(vbuf + (FP8 ? VBUFS * VBUF : 0)); // (max, sum) of [half][row]; of q, its maximum
    uint64_t* bars = (uint64_t*)((uint8_t*)xch + 3 * 2 * 128 * 4);
    uint32_t* tmem_slot = (uint32_t*)(bars + B_COUNT);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    // the row tiles of one head are neighbours in launch order and share its pages in L2
    const int RT = (P.R + 127) >> 7;
    const int rt = blockIdx.y % RT;
    int split = blockIdx.x, hk = blockIdx.y / RT, b = blockIdx.z;
    const int R0 = rt * 128, RL = min(128, P.R - R0);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    pdl_launch_dependents();
    if (threadIdx.x == 0) {
        // (as a loop: 64 trees of 12 nodes and 4096 keys, E4M3, 190 us instead of 184)
#pragma unroll
        for (int i = 0; i < B_COUNT; ++i) {
            int count = 1;
            // V's readers: the widening warps, or P.V of both halves and warp 13
            if (i >= B_W_EMPTY && i < B_V_FULL) count = FP8 ? C::CONV : 3;
            if (i >= B_V_FULL && i < B_V_EMPTY) count = C::CONV;
            if (i >= B_V_EMPTY && i < B_S) count = 2;
            if (i >= B_S_READ && i < B_PV) count = 4;
            if (i == B_Q_READY) count = 8;
            if (i == B_IDLE) count = 3;
            if (i >= B_PAIR && i < B_CLEAN) count = 2;
            if (i >= B_PATCH) count = C::CONV;
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
    const bool loads = warp == 0 || (!FP8 && warp == 12);
    int guess_at = -1, guess = 0;
    if (loads) {
        guess_at = min(split * P.split_pages + (lane / 2 & (PPT - 1)), P.mpps - 1);
        guess = P.block_table[(int64_t)b * P.mpps + guess_at];
    }
    // so are the new tokens: a widening thread's first item (chunk ct % 16 of token
    // ct / 16) when the partition starts at or before the first of them
    const int ct = (warp - 12) * 32 + lane;
    const bool converts = warp >= (FP8 ? 12 : 13);
    uint4 first_k = make_uint4(0, 0, 0, 0), first_v = first_k;
    if (FP8 && P.k_new && converts && ct < P.M * 16) {
        const int64_t src = (((int64_t)b * P.M + (ct >> 4)) * P.Hkv + hk) * 16 + (ct & 15);
        first_k = ((const uint4*)P.k_new)[src];
        first_v = ((const uint4*)P.v_new)[src];
    }
    const int L = P.seq_lens[b];
    const bool seq_ok = !(L < P.M || L > P.max_seq_len || (L + PS - 1) / PS > P.mpps);
    bool run = seq_ok && have_work;                         // uniform over the CTA
    if (!seq_ok && !P.lpt_order && threadIdx.x == 0 && split == 0 && blockIdx.y == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
    // every row tile spans the keys from the first node's window to the end
    const int lo0 = (P.window_left >= 0) ? max(0, L - P.M - P.window_left) : 0;
    const int first_page = lo0 / PS, last_page = (L - 1) / PS;
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
    // (E4M3: in shared memory, each widening warp its own, none of the widening loop's
    // registers)
    const uint64_t holes = !FP8 && (warp == 2 || warp == 3 || converts) ? tree_holes(P, b, lane) : 0;
    uint64_t* warp_holes = bars + B_COUNT + 2 + (warp - 12);
    // V rows of tile t without a reader: those outside [zlo, zhi), and padding nodes
    // (the nodes are in the last two tiles of a partition, if it has any)
    auto zlo_of = [&](int t) { return max(0, lo0 - (k_begin + t * NK)); };
    auto zhi_of = [&](int t) { return min(NK, L - (k_begin + t * NK)); };
    auto holes_in = [&](int t) { return holes && k_begin + t * NK + NK > L - P.M; };
    auto dirty = [&](int t) {
        return !FP8 && ((t == 0 && zlo_of(t) > 0) || (t == n_tiles - 1 && zhi_of(t) < NK) || holes_in(t));
    };
    auto clean = [&](int t) { return B_CLEAN + (t == 0 ? 0 : t == n_tiles - 1 ? 1 : 2); };
    // append: the new tokens in this partition, and the tiles that hold them
    const int app_lo = max(L - P.M, k_begin), app_hi = min(L, k_begin + n_pages * PS);
    const bool appends = FP8 && P.k_new && run && app_lo < app_hi;
    const int app_t0 = appends ? (app_lo - k_begin) / NK : 1 << 30, app_t1 = appends ? (app_hi - 1 - k_begin) / NK : -1;
    bool ok = true;

    if (!run) {
        // no keys of this sequence fall in this partition (or bad input)
    } else if (loads) {
        // ---------------------------------------------------------- producer
        // Lane 2 p + j: copy j of page p of the tile.  E4M3: K and V; BF16: dims 0-63
        // and 64-127 of K (warp 0) or of V (warp 12): a stage of K is free long before
        // the V of its tile, and the loads of one do not wait for the other's
        const uint64_t policy = policy_evict_first();
        const int32_t* bt = P.block_table + (int64_t)b * P.mpps + page_begin;
        const int p = lane / 2, j = lane & 1;
        const bool is_k = FP8 ? j == 0 : warp == 0;
        const int full = is_k ? B_K_FULL : B_W_FULL;
        uint8_t* ring = stg + (is_k ? 0 : C::OFF_V) + (FP8 ? 0 : j * HALF) + p * PS * 128;
        int issued = 0;
        int next = p < PPT && p < n_pages ? (page_begin + p == guess_at ? guess : bt[p]) : 0;
        for (int t = 0; t < n_tiles; ++t) {
            const int s = t % STAGES, use = t / STAGES, phys = next, at = t * PPT + p;
            const bool mine = p < PPT && at < n_pages;
            next = p < PPT && at + PPT < n_pages ? bt[at + PPT] : 0;
            if (use > 0) {
                if (FP8 || warp == 0) ok = mbar_wait(bar(B_K_EMPTY + s), (use - 1) & 1);
                if (ok && (FP8 || warp != 0)) ok = mbar_wait(bar(B_W_EMPTY + s), (use - 1) & 1);
            }
            if (!__all_sync(0xffffffffu, ok)) break;
            const uint32_t bytes = min(PPT, n_pages - t * PPT) * PS * (FP8 ? 128 : 256);
            if (lane == 0 || (FP8 && lane == 1)) mbar_expect_tx(bar(full + s), bytes);
            __syncwarp();
            if (mine)
                tma_load_3d(smem_u32(ring + s * C::STG), is_k ? &tm_k : &tm_v, FP8 ? 0 : 64 * j, hk * PS, phys,
                            bar(full + s), policy);
            __syncwarp();
            issued = t + 1;
        }
        // never leave with copies into this CTA's shared memory in flight
        for (int t = max(0, issued - STAGES); t < issued; ++t) mbar_wait(bar(full + t % STAGES), (t / STAGES) & 1);
        __syncwarp();
    } else if (warp < 4) {
        // ------------------------------------------------------ MMA issue
        constexpr uint32_t BF16 = FP8 ? 0 : (1u << 7) | (1u << 10);      // A and B format of kind::f16
        constexpr uint32_t ID_QK = idesc(128, NK, false) | BF16, ID_PV = idesc(128, 128, true) | BF16;
        const bool leader = elect_one();
        if (warp == 1) {
            // both halves of a tile at once
            ok = mbar_wait(bar(B_Q_READY), 0);
            for (int t = 0; t < n_tiles; ++t) {
                const int s = t % STAGES;
                if (ok) ok = mbar_wait(bar(B_K_FULL + s), (t / STAGES) & 1);
                if (ok && t >= app_t0 && t <= app_t1) ok = mbar_wait(bar(B_PATCH + (t - app_t0)), 0);
                for (int h = 0; h < 2; ++h)
                    if (ok && t > 0) ok = mbar_wait(bar(B_S_READ + h), (t - 1) & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fence_after();
                if (leader) {
                    const uint32_t k = smem_u32(stg + s * C::STG);
                    if (FP8) {
#pragma unroll
                        for (int ks = 0; ks < 4; ++ks) {
                            const uint64_t bd = sdesc(k + ks * 32, 16, 1024);
                            mma_f8_ts(tmem + TM_S, tmem + TM_Q + 8 * ks, bd, ID_QK, ks > 0);
                            mma_f8_ts(tmem + TM_S, tmem + TM_Q + 32 + 8 * ks, bd, ID_QK, 1);
                        }
                    } else {
#pragma unroll
                        for (int ks = 0; ks < 8; ++ks)
                            mma_ts(tmem + TM_S, tmem + TM_Q + 8 * ks, desc_lo(k + (ks >> 2) * HALF + (ks & 3) * 32, 16), ID_QK,
                                   ks > 0);
                    }
                    mma_commit(bar(B_S));
                    mma_commit(bar(B_S + 1));
                    mma_commit(bar(B_K_EMPTY + s));
                }
                __syncwarp();
            }
        } else {
            const int h = warp - 2;
            for (int t = 0; t < n_tiles; ++t) {
                const int s = t % STAGES, vb = t % VBUFS;
                ok = FP8 ? mbar_wait(bar(B_V_FULL + vb), (t / VBUFS) & 1) : mbar_wait(bar(B_W_FULL + s), (t / STAGES) & 1);
                if (ok && dirty(t)) ok = mbar_wait(bar(clean(t)), 0);
                if (ok) ok = mbar_wait(bar(B_P + h), t & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                fence_after();
                if (leader) {
                    const uint32_t v = smem_u32(FP8 ? vbuf + vb * VBUF : stg + C::OFF_V + s * C::STG) + h * (64 * 128);
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        mma_ts(tmem + TM_O + 128 * h, tmem + TM_P + 32 * h + 8 * kk, desc_lo(v + kk * 2048, HALF), ID_PV,
                               t > 0 || kk > 0);
                    mma_commit(bar(B_PV + h));
                    mma_commit(FP8 ? bar(B_V_EMPTY + vb) : bar(B_W_EMPTY + s));
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
    } else if (converts && !FP8) {
        // ------------------------------------------------- V rows without a reader
        for (int t = 0; t < n_tiles; ++t) {
            const int s = t % STAGES;
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_W_FULL + s), (t / STAGES) & 1));
            if (!ok) break;
            if (dirty(t)) {
                const int zlo = zlo_of(t), zhi = zhi_of(t), node0 = L - P.M - (k_begin + t * NK);
                uint8_t* v = stg + C::OFF_V + s * C::STG;
                for (int i = lane; i < NK * 16; i += 32) {
                    const int r = i >> 4;
                    if (r < zlo || r >= zhi || tree_hole(holes, r, node0))
                        *(uint4*)(v + ((i >> 3) & 1) * HALF + r * 128 + (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(clean(t)));
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_W_EMPTY + s));
        }
    } else if (converts) {
        // ---------------------------------------------------------- V widening
        // 128 keys x 8 chunks of 16 E4M3 values -> two 64-dim blocks of 128 x 128 bytes
        // of f16; keys outside every row's range become zeros
        constexpr int CONV_THREADS = 32 * C::CONV;
        const int n_app = appends ? app_hi - app_lo : 0;
        const float ksc = appends ? *P.k_scale : 1.f, vsc = appends ? *P.v_scale : 1.f;
        // the new tokens' codes: 8-element chunk it % 16 of token it / 16
        auto app_item = [&](int it, uint2& kc, uint2& vc, int& pos, int& chunk) {
            pos = app_lo + (it >> 4);
            chunk = it & 15;
            const int64_t src = (((int64_t)b * P.M + (pos - (L - P.M))) * P.Hkv + hk) * 16 + chunk;
            const bool have = it == ct && app_lo == L - P.M && ct < P.M * 16;        // loaded before the length
            kc = e4m3_encode8(have ? first_k : ((const uint4*)P.k_new)[src], ksc);
            vc = e4m3_encode8(have ? first_v : ((const uint4*)P.v_new)[src], vsc);
        };
        // (a token on a page outside the pool is not written: its row stays the zeros of
        // the staged page)
        auto held = [&](int it, int pos, int page) {
            if (it != ct) page = P.block_table[(int64_t)b * P.mpps + pos / PS];
            return page >= 0 && page < P.num_pages;
        };
        // this thread's first item is kept, and its page id
        uint2 kc0 = make_uint2(0, 0), vc0 = kc0;
        int pos0 = -1, chunk0 = 0, page0 = -1;
        if (ct < n_app * 16) {
            page0 = P.block_table[(int64_t)b * P.mpps + (app_lo + (ct >> 4)) / PS];
            app_item(ct, kc0, vc0, pos0, chunk0);
        }
        if (const uint64_t w = tree_holes(P, b, lane); lane == 0) *warp_holes = w;
        __syncwarp();
        for (int t = 0; t < n_tiles; ++t) {
            const int s = t % STAGES, vb = t % VBUFS;
            ok = mbar_wait(bar(B_W_FULL + s), (t / STAGES) & 1);
            const int k0 = k_begin + t * NK;
            const bool patched = t >= app_t0 && t <= app_t1;
            if (patched) ok = ok && mbar_wait(bar(B_K_FULL + s), (t / STAGES) & 1);
            if (patched && __all_sync(0xffffffffu, ok)) {
                // the new rows of K over the staged tile, before its Q.K^T
                uint8_t* kst = stg + s * C::STG;
                for (int it = ct; it < n_app * 16; it += CONV_THREADS) {
                    uint2 kc = kc0, vc = vc0;
                    int pos = pos0, chunk = chunk0;
                    if (it != ct) app_item(it, kc, vc, pos, chunk);
                    const int r = pos - k0;
                    if (r >= 0 && r < NK && held(it, pos, page0))
                        *(uint2*)(kst + r * 128 + ((((chunk >> 1) ^ r) & 7) << 4) + (chunk & 1) * 8) = kc;
                }
                fence_proxy_async();                        // for the tensor cores' read of K
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_PATCH + (t - app_t0)));
            }
            if (ok && t >= VBUFS) ok = mbar_wait(bar(B_V_EMPTY + vb), ((t / VBUFS) - 1) & 1);
            if (!__all_sync(0xffffffffu, ok)) break;
            // rows [nlo, nhi) hold new tokens: their staged V may be old
            const int nlo = patched ? max(0, app_lo - k0) : 0, nhi = patched ? min(NK, app_hi - k0) : 0;
            const int zlo = zlo_of(t), zhi = zhi_of(t);
            // chunk c of rows r0 + (CONV_THREADS / 8) u, in two halves
            const int r0 = ct >> 3, c = ct & 7, c16 = 2 * (c & 3);
            const bool low = c < 4;
            const uint8_t* src = stg + C::OFF_V + s * C::STG + r0 * 128 + (((c ^ r0) & 7) << 4);
            uint8_t* dst = vbuf + vb * VBUF;
            constexpr int PER = NK * 8 / CONV_THREADS;      // chunks a thread
            static_assert(!FP8 || CONV_THREADS % 64 == 0 && PER * CONV_THREADS == NK * 8, "a row's swizzle is that of row r0");
            // the order of the two stores alternates so that each quarter warp covers all
            // 32 banks
            uint8_t* first = dst + (c >> 2) * HALF + r0 * 128 + (((c16 + !low) ^ r0) & 7) * 16;
            uint8_t* second = dst + (c >> 2) * HALF + r0 * 128 + (((c16 + low) ^ r0) & 7) * 16;
            uint2 cf[PER], cg[PER];
            const uint8_t *sf = src + (low ? 0 : 8), *sg = src + (low ? 8 : 0);
            const bool whole = zlo <= 0 && k0 + NK <= L - P.M;     // (no nodes)
            if (whole) {
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    cf[u] = *(const uint2*)(sf + u * CONV_THREADS * 16);
                    cg[u] = *(const uint2*)(sg + u * CONV_THREADS * 16);
                }
            } else {
                const uint64_t holes = *warp_holes;
#pragma unroll
                for (int u = 0; u < PER; ++u) {
                    const int r = r0 + CONV_THREADS / 8 * u;
                    const bool in = r >= zlo && r < zhi && !tree_hole(holes, k0 + r, L - P.M);
                    cf[u] = in ? *(const uint2*)(sf + u * CONV_THREADS * 16) : make_uint2(0, 0);
                    cg[u] = in ? *(const uint2*)(sg + u * CONV_THREADS * 16) : make_uint2(0, 0);
                }
            }
#pragma unroll
            for (int u = 0; u < PER; ++u) {
                const int r = r0 + CONV_THREADS / 8 * u;
                if (r >= nlo && r < nhi) continue;
                *(uint4*)(first + u * CONV_THREADS * 16) =
                    make_uint4(e4m3x2_to_f16x2(cf[u].x), e4m3x2_to_f16x2(cf[u].x >> 16), e4m3x2_to_f16x2(cf[u].y),
                               e4m3x2_to_f16x2(cf[u].y >> 16));
                *(uint4*)(second + u * CONV_THREADS * 16) =
                    make_uint4(e4m3x2_to_f16x2(cg[u].x), e4m3x2_to_f16x2(cg[u].x >> 16), e4m3x2_to_f16x2(cg[u].y),
                               e4m3x2_to_f16x2(cg[u].y >> 16));
            }
            if (patched) {
                for (int it = ct; it < n_app * 16; it += CONV_THREADS) {
                    uint2 kc = kc0, vc = vc0;
                    int pos = pos0, chunk = chunk0;
                    if (it != ct) app_item(it, kc, vc, pos, chunk);
                    const int r = pos - k0, c = chunk >> 1;
                    if (r < 0 || r >= NK) continue;
                    if (tree_hole(*warp_holes, pos, L - P.M) || !held(it, pos, page0)) vc = make_uint2(0, 0);
                    *(uint4*)(dst + (c >> 2) * HALF + r * 128 + ((((2 * (c & 3) + (chunk & 1)) ^ r) & 7) << 4)) =
                        make_uint4(e4m3x2_to_f16x2(vc.x), e4m3x2_to_f16x2(vc.x >> 16), e4m3x2_to_f16x2(vc.y),
                                   e4m3x2_to_f16x2(vc.y >> 16));
                }
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(bar(B_W_EMPTY + s));
                mbar_arrive(bar(B_V_FULL + vb));
            }
        }
        // the new tokens into the cache
        for (int it = ct; it < n_app * 16; it += CONV_THREADS) {
            uint2 kc = kc0, vc = vc0;
            int pos = pos0, chunk = chunk0, page = page0;
            if (it != ct) {
                app_item(it, kc, vc, pos, chunk);
                page = P.block_table[(int64_t)b * P.mpps + pos / PS];
            }
            if (page < 0 || page >= P.num_pages) {
                if (chunk == 0) flag(FP8KV_DEV_BAD_SLOT);
                continue;
            }
            const int64_t dst = (((int64_t)page * P.Hkv + hk) * PS + pos % PS) * 128 + chunk * 8;
            *(uint2*)(P.k_cache + dst) = kc;
            *(uint2*)(P.v_cache + dst) = vc;
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
        float mult = fabsf(P.sm_scale) * 1.4426950408889634f;
        {
            // this half's 64 dims of the row; the sign of sm_scale goes into q, as the
            // row maximum is taken before the multiplication
            const uint4* src = (const uint4*)(P.q + row_idx * 128) + 8 * half;
            const uint32_t sign = P.sm_scale < 0.f ? 0x80008000u : 0u;
            uint32_t qw[32];
#pragma unroll
            for (int u = 0; u < 8; ++u) {
                const uint4 w = pad ? make_uint4(0, 0, 0, 0) : src[u];
                qw[4 * u] = w.x ^ sign;
                qw[4 * u + 1] = w.y ^ sign;
                qw[4 * u + 2] = w.z ^ sign;
                qw[4 * u + 3] = w.w ^ sign;
            }
            if (FP8) {
                // two E4M3 terms, each half's dims behind the other's; the row maximum is
                // that of both halves
                float* qmax = xch + 2 * 2 * 128;
                uint32_t am = 0;
#pragma unroll
                for (int u = 0; u < 32; ++u) am = max_bf16x2(am, qw[u] & 0x7fff7fffu);
                qmax[half * 128 + r] = fmaxf(bf16_lo(am), bf16_hi(am));
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_PAIR + wq));
                ok = __all_sync(0xffffffffu, mbar_wait(bar(B_PAIR + wq), 0));
                const float amax = fmaxf(qmax[r], qmax[128 + r]);
                int e = 7;
                const uint32_t ab = __float_as_uint(amax);
                if (amax > 0.f && ((ab >> 23) & 0xff) != 0xff) {
                    const int be = (int)((ab >> 23) & 0xff);
                    e = be ? be - 127 : -127;
                }
                const int sh = max(-100, min(100, 7 - e));
                const float scale = ldexpf(1.0f, sh);
                mult *= *P.k_scale * ldexpf(1.0f, -sh);
                uint32_t hw[16], lw[16];
#pragma unroll
                for (int k = 0; k < 16; ++k) {
                    uint32_t h2[2], l2[2];
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t x = qw[2 * k + i];
                        const uint32_t q16 = pack_f16x2(bf16_lo(x) * scale, bf16_hi(x) * scale);
                        h2[i] = f16x2_to_e4m3x2(q16);
                        l2[i] = f16x2_to_e4m3x2(sub_f16x2(q16, e4m3x2_to_f16x2(h2[i])));
                    }
                    hw[k] = h2[0] | (h2[1] << 16);
                    lw[k] = l2[0] | (l2[1] << 16);
                }
                tmem_st_x16(lane_base + TM_Q + 16 * half, hw);
                tmem_st_x16(lane_base + TM_Q + 32 + 16 * half, lw);
            } else {
                tmem_st_x32(lane_base + TM_Q + 32 * half, qw);
            }
            tmem_wait_st();
        }
        mult = fmaxf(mult, 1e-37f);
        fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_Q_READY));
        const TreeRow tr = tree_row(P, b, m, word, base);
        int lomax = tr.lo;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) lomax = max(lomax, __shfl_xor_sync(0xffffffffu, lomax, off));
        // this half's maximum and sum
        float m_run = -INFINITY, l_run = 0.f;
        const uint32_t o_col = lane_base + TM_O + 128 * half, s_col = lane_base + TM_S + 64 * half;
        const uint32_t p_col = lane_base + TM_P + 32 * half;
        for (int t = 0; t < n_tiles && ok; ++t) {
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_S + half), t & 1));
            if (!ok) break;
            fence_after();
            const int k0 = k_begin + t * NK + 64 * half;    // first key of this half
            if (!active || k0 >= L) {
                // no row of this warp sees any key of it: P = 0
                if (lane == 0) mbar_arrive(bar(B_S_READ + half));
                if (t > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_PV + half), (t - 1) & 1));
                if (!ok) break;
                fence_after();
                uint32_t zero[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) zero[j] = 0u;
                tmem_st_x32(p_col, zero);
            } else {
                uint32_t sv[64];
                tmem_ld_x64(s_col, sv);
                tmem_wait_ld();
                // S is in registers: the next product may go over it
                fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_S_READ + half));
                if (k0 + 63 >= base || k0 < lomax) {
                    const uint64_t vis = tree_sees64(tr, k0, base);
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
                // P = 2^(s mult - m + BIAS) (masked keys are -inf and give 0)
                const float neg = (m_run == -INFINITY) ? 0.f : BIAS - m_run;
                const uint64_t mult2 = pack2(mult, mult), neg2 = pack2(neg, neg);
                // P.V of tile t - 1 has read P (the wait behind the exponentials: 3% slower over BF16)
                if (t > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_PV + half), (t - 1) & 1));
                if (!ok) break;
                fence_after();
                uint64_t sum2 = 0;
                uint32_t pw[32];
#pragma unroll
                for (int j = 0; j < 32; ++j) {
                    float p0, p1;
                    unpack2(fma2(pack2(__uint_as_float(sv[2 * j]), __uint_as_float(sv[2 * j + 1])), mult2, neg2), p0, p1);
                    p0 = ex2(p0);
                    p1 = ex2(p1);
                    sum2 = add2(sum2, pack2(p0, p1));
                    pw[j] = FP8 ? pack_f16x2(p0, p1) : pack_bf16x2(p0, p1);
                }
                tmem_st_x32(p_col, pw);
                float sum0, sum1;
                unpack2(sum2, sum0, sum1);
                l_run += sum0 + sum1;
            }
            tmem_wait_st();
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_P + half));
        }
        // ------------------------------------------------------------ epilogue
        // both halves' O and (max, sum); this thread merges 64 dims of its row
        for (int h = 0; h < 2; ++h)
            if (ok) ok = mbar_wait(bar(B_O + h), 0);
        const bool direct = nsplit_b == 1, combine = CL && !direct;
        float2* ml = (float2*)xch;
        float2* ml_all = (float2*)(stg + 2 * 128 * EPI_STRIDE);     // (max, sum) of the staged rows
        ml[half * 128 + r] = make_float2(m_run, l_run);
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_PAIR + wq));
        if (ok) ok = mbar_wait(bar(B_PAIR + wq), FP8 ? 1 : 0);
        ok = __all_sync(0xffffffffu, ok);
        if (ok && active) {
            fence_after();
            const float2 a = ml[r], z = ml[128 + r];
            float m_tot = fmaxf(a.x, z.x);
            const float wa = a.x == -INFINITY ? 0.f : ex2(a.x - m_tot), wz = z.x == -INFINITY ? 0.f : ex2(z.x - m_tot);
            // (a half without a key with a number for a score has weight 0, but its
            // sum, NaN if it saw NaN scores, counts)
            const float l_tot = (a.x == -INFINITY ? a.y : a.y * wa) + (z.x == -INFINITY ? z.y : z.y * wz);
            if (m_tot == -INFINITY && l_tot != l_tot) m_tot = 0.f;
            const bool zero = direct && (word == 0 || l_tot == 0.f);
            // direct: bf16 of v_scale O / l; partial, E4M3: f16 of O / l in code units
            // (|x| <= 448), BF16: fp32 of O (its values can exceed f16), beside its
            // (max, sum); a row with no visible key here has l = 0: weight 0, values 0
            const float f = direct ? (FP8 ? *P.v_scale : 1.0f) / l_tot : FP8 ? (l_tot > 0.f ? 1.0f / l_tot : 0.f) : 1.0f;
            const float fa = wa * f, fz = wz * f;
            // the half row goes through the free ring to one bulk copy
            uint8_t* row_stage = stg + (half * 128 + r) * EPI_STRIDE;
#pragma unroll 1
            for (int c = 0; c < 64; c += 32) {
                uint32_t oa[32], oz[32];
                tmem_ld_x32(lane_base + TM_O + 64 * half + c, oa);
                tmem_ld_x32(lane_base + TM_O + 128 + 64 * half + c, oz);
                tmem_wait_ld();
                float x[32];
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    x[i] = zero ? 0.f : __uint_as_float(oa[i]) * fa + __uint_as_float(oz[i]) * fz;
                if (!FP8 && !direct) {
                    uint4* dst = (uint4*)(row_stage + c * 4);
#pragma unroll
                    for (int v4 = 0; v4 < 8; ++v4)
                        dst[v4] = make_uint4(__float_as_uint(x[4 * v4]), __float_as_uint(x[4 * v4 + 1]),
                                             __float_as_uint(x[4 * v4 + 2]), __float_as_uint(x[4 * v4 + 3]));
                } else {
                    uint4* dst = (uint4*)(row_stage + c * 2);
#pragma unroll
                    for (int v4 = 0; v4 < 4; ++v4) {
                        uint32_t w[4];
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            w[j] = direct ? pack_bf16x2(x[8 * v4 + 2 * j], x[8 * v4 + 2 * j + 1])
                                          : pack_f16x2(x[8 * v4 + 2 * j], x[8 * v4 + 2 * j + 1]);
                        dst[v4] = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
            }
            if (combine) {
                // stays here: the cluster's CTAs read it below
                if (half == 0) ml_all[r] = make_float2(m_tot, l_tot);
            } else if (!pad) {
                fence_proxy_async();        // the staged row, written by this thread, to the bulk copy
                if (direct)
                    bulk_store(P.out + row_idx * 128 + 64 * half, smem_u32(row_stage), 128);
                else if (FP8)
                    bulk_store((uint16_t*)P.ws_o + (row_idx * P.num_splits + split) * 128 + 64 * half, smem_u32(row_stage), 128);
                else
                    bulk_store(P.ws_o + (row_idx * P.num_splits + split) * 128 + 64 * half, smem_u32(row_stage), 256);
                bulk_commit();
                bulk_wait_read();
                if (!direct && half == 0)
                    *(float2*)(P.ws_ml + (row_idx * P.num_splits + split) * 2) = make_float2(m_tot, l_tot);
            }
        }
    }

    if (CL) {
        // ------------------------------------------------- cluster combine
        // rank = partition; each CTA merges every nsplit_b-th row, 32 threads a row.
        // BF16: O = sum_p w_p O_p / sum_p w_p l_p, w_p = 2^(m_p - m*); E4M3: O =
        // v_scale sum_p w_p l_p (O_p / l_p) / sum_p w_p l_p
        __syncwarp();
        cluster_arrive();
        cluster_wait();
        if (run && nsplit_b > 1) {
            const float vs = FP8 ? *P.v_scale : 1.0f;
            for (int row = split + nsplit_b * warp; row < RL; row += nsplit_b * C::WARPS) {
                // this lane's four dims of the row in every partition's staging
                const uint8_t* at = stg + ((lane >> 4) * 128 + row) * EPI_STRIDE + (lane & 15) * (FP8 ? 8 : 16);
                float2 a[kMaxCluster];
                uint4 x[kMaxCluster];
                float top = -INFINITY, den = 0.f, acc[4] = {};
#pragma unroll
                for (int j = 0; j < kMaxCluster; ++j) {
                    a[j] = make_float2(-INFINITY, 0.f);
                    if (j >= nsplit_b) continue;
                    a[j] = dsmem_ld8(dsmem_addr(stg + 2 * 128 * EPI_STRIDE + row * 8, j));
                    if (FP8) {
                        const float2 y = dsmem_ld8(dsmem_addr(at, j));
                        x[j].x = __float_as_uint(y.x);
                        x[j].y = __float_as_uint(y.y);
                    } else {
                        x[j] = dsmem_ld16(dsmem_addr(at, j));
                    }
                    top = fmaxf(top, a[j].x);
                }
#pragma unroll
                for (int j = 0; j < kMaxCluster; ++j) {
                    if (j >= nsplit_b) continue;
                    const float e = a[j].x == -INFINITY ? 0.f : ex2(a[j].x - top), w = FP8 ? e * a[j].y : e;
                    den += e * a[j].y;
                    if (FP8) {
                        const float2 y0 = f16x2_to_f32x2(x[j].x), y1 = f16x2_to_f32x2(x[j].y);
                        acc[0] += w * y0.x;
                        acc[1] += w * y0.y;
                        acc[2] += w * y1.x;
                        acc[3] += w * y1.y;
                    } else {
                        acc[0] += w * __uint_as_float(x[j].x);
                        acc[1] += w * __uint_as_float(x[j].y);
                        acc[2] += w * __uint_as_float(x[j].z);
                        acc[3] += w * __uint_as_float(x[j].w);
                    }
                }
                const int m = (R0 + row) / P.G;
                const int64_t idx = ((int64_t)b * P.M + m) * P.Hq + hk * P.G + (R0 + row) % P.G;
                const float f = vs / den;
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

template <int PS, bool FP8, bool CL>
static cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& P, dim3 grid, cudaStream_t s) {
    static std::atomic<uint64_t> done{0};
    auto kern = attention_tree_tc_kernel<PS, FP8, CL>;
    const cudaError_t e = opt_in_smem(done, (const void*)kern, Cfg<FP8>::SMEM);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kern, grid, dim3(Cfg<FP8>::THREADS), Cfg<FP8>::SMEM, s, P.cluster, tk, tv, P);
}
template <int PS, bool FP8>
static cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& P, dim3 grid, cudaStream_t s) {
    return P.cluster > 1 ? launch<PS, FP8, true>(tk, tv, P, grid, s) : launch<PS, FP8, false>(tk, tv, P, grid, s);
}

}  // namespace ttc

int launch_attention_tree_tc(const CUtensorMap& tk, const CUtensorMap& tv, const AttnParams& P, bool fp8,
                             cudaStream_t s, char* text, size_t text_bytes) {
    const int RT = (P.R + 127) / 128;
    if (!P.tree || P.R <= 16 || (int64_t)RT * P.Hkv > 65535 || (P.split_pages * P.page_size) % ttc::NK || P.scale_stride)
        return FP8KV_ERR_UNSUPPORTED;
    if (P.cluster > 1 && (P.cluster > ttc::kMaxCluster || P.cluster != P.num_splits || P.lpt_order))
        return FP8KV_ERR_UNSUPPORTED;
    if ((P.k_new && (!fp8 || RT > 1)) || (P.lpt_order && RT > 1)) return FP8KV_ERR_UNSUPPORTED;
    const dim3 grid(P.num_splits, P.Hkv * RT, P.B);
    const bool p32 = P.page_size == 32;
    const cudaError_t e = fp8 ? (p32 ? ttc::launch<32, true>(tk, tv, P, grid, s) : ttc::launch<64, true>(tk, tv, P, grid, s))
                              : (p32 ? ttc::launch<32, false>(tk, tv, P, grid, s) : ttc::launch<64, false>(tk, tv, P, grid, s));
    if (e != cudaSuccess) return (cudaGetLastError(), FP8KV_ERR_CUDA);
    snprintf(text, text_bytes,
             "attention_tree_tc<ps=%d,%s> rows=%d row_tiles=%d splits=%d split_tokens=%d grid=%dx%dx%d threads=%d "
             "cluster=%d reduce=%d order=%s",
             P.page_size, fp8 ? "e4m3" : "bf16", P.R, RT, P.num_splits, P.split_pages * P.page_size, P.num_splits,
             P.Hkv * RT, P.B, fp8 ? ttc::Cfg<true>::THREADS : ttc::Cfg<false>::THREADS, P.cluster > 1 ? P.cluster : 1,
             P.num_splits > 1 && P.cluster <= 1 ? 1 : 0, P.lpt_order ? "longest_first" : "grid");
    return FP8KV_OK;
}

}  // namespace fp8kv
