// prompt_attention.cu -- causal attention of whole prompts: packed sequences of
// different lengths, grouped heads, an optional sliding window, bf16 rows as
// the projection wrote them (no cache in between).  (The pages have no
// counterpart; the masks are those of fp8kv_paged_attention.)
//
// What bounds it: 4 * 128 operations for each visible (row, key) pair, on the
// tensor cores; the K and V tiles come from L2.  A work item is a pair of row
// tiles of 128 rows against the same K and V tiles: while the softmax of one
// tile runs, the tensor cores work on the other.
//
// Rows.  The G query heads of a KV head are packed: row r of a tile is position
// r / G, head r % G, NP = 128 / G positions a tile (126 rows for G = 9).  The
// rows of a tile then see nearly the same keys, so a diagonal or a window edge
// costs little more than the keys it holds, and short prompts fill a tile.
//
// Items.  The grid has one CTA per item; a resident CTA (one per SM) goes on
// with the items of CTAs that have not started, which it cancels
// (clusterlaunchcontrol), so that loads, set-up and output of one item overlap
// the products of another, without a counter in memory.  Items are handed out
// as SMs come free, the last sequence first and within a sequence from its end,
// where the rows see the most keys.  Twelve warps:
//   warp 0      loads by TMA: Q of each row tile once it is free, K and V tiles
//               of 128 keys through a ring of four 32 KiB slots; allocates and
//               frees the tensor memory
//   warps 1, 2  issue the MMAs of the first and of the second row tile: per key
//               tile Q.K^T, then P.V.  (One warp for both left the tensor cores
//               idle 60% of the time: a wait or a commit takes it 40 to 100
//               cycles, eight MMAs run 512.)
//   warp 3      schedules: the next item, where its rows lie, into a queue; and
//               zeroes the V rows of an item's last key tile that none of its
//               rows sees (they may hold another sequence's values): whatever
//               is there, 0 * V reaches no output
//   warps 4-7   softmax and output of the first row tile, one row per thread
//   warps 8-11  ... of the second         (warp w: TMEM lanes 32 (w % 4) ...)
// Online softmax in the log2 domain over halves of a key tile, whose P.V starts
// while the other half is exponentiated; O is rescaled only when a row's
// maximum grows by more than 2^8 (the weights stay below 2^8, sums are fp32).
// P is rounded to bf16, V's type, as the MMA needs both alike: at most 2^-8 of
// each weight, the size of the output's own rounding.
// TMEM columns: S/P of the two row tiles 0-127, 128-255 (P over the first half
// of its S), O 256-383, 384-511.
#include <stdio.h>

#include "attention.cuh"
#include "common.cuh"
#include "tcgen05.cuh"

namespace fp8kv {

int status_prompt(unsigned int* s, int clear) { return read_status(s, clear); }

namespace prompt {

constexpr int NK = 128;                         // keys per tile
constexpr int SLOT = NK * 256;                  // 32 KiB: two blocks of 128 rows x 64 dims (128-byte swizzled)
constexpr int HALF = SLOT / 2;
constexpr int SLOTS = 4;
constexpr int WARPS = 12, THREADS = WARPS * 32;
constexpr int QUEUE = 4;                        // items in the queue
constexpr uint32_t TM_S = 0, TM_O = 256, TM_COLS = 512;
constexpr int SMEM = 2 * SLOT + SLOTS * SLOT + SLOT + 1024 + 512;    // Q, ring, output tile

enum {
    B_Q = 0,                                    // per row tile: Q loaded
    B_QE = B_Q + 2,                             // ... read by its last Q.K^T
    B_FULL = B_QE + 2,
    B_EMPTY = B_FULL + SLOTS,
    B_S = B_EMPTY + SLOTS,                      // per row tile: S ready
    B_P = B_S + 2,                              // per row tile and half: 64 columns of P ready
    B_H = B_P + 4,                              // per row tile: P.V of the first half complete
    B_O = B_H + 2,                              // per row tile: O final
    B_OE = B_O + 2,                             // ... and read
    B_STAGED = B_OE + 2,                        // per row tile: output tile written
    B_STAGE = B_STAGED + 2,                     // ... the staging tile is this row tile's to write
    B_TURN = B_STAGE + 2,                       // per row tile: its MMA warp's turn
    B_RAW = B_TURN + 2,                         // per slot: an item's last V tile loaded, to be cleaned
    B_ITEM = B_RAW + SLOTS,                     // per queue entry: written
    B_TAKEN = B_ITEM + QUEUE,                   // ... read by every role
    B_NEXT = B_TAKEN + QUEUE,                   // answer of a cancel request
    B_IDLE = B_NEXT + 1,                        // per MMA warp: nothing outstanding
    B_COUNT = B_IDLE + 2
};
constexpr int ROLES = 1 + 2 + 8;                // readers of a queue entry: load, MMA, softmax warps

struct Params {
    const int32_t* cu;          // [B + 1]
    uint16_t* out;              // [T][Hq][128]
    int B, T, Hq, Hkv, G, NP, window_left, max_seq_len;
    float scale_log2;           // sm_scale * log2(e)
};

// bf16 operands: format code 1 for A and B.
constexpr uint32_t ID_QK = idesc(128, NK, false) | (1u << 7) | (1u << 10);
constexpr uint32_t ID_QK_HALF = idesc(128, NK / 2, false) | (1u << 7) | (1u << 10);
constexpr uint32_t ID_PV = idesc(128, 128, true) | (1u << 7) | (1u << 10);

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* tm, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(tm),
                 "r"(src), "r"(x), "r"(y), "r"(z)
                 : "memory");
}

// Ask for a CTA of this grid that has not started to be cancelled; the answer
// (16 bytes) arrives at `resp` and on `mbar`.
__device__ __forceinline__ void cancel_request(uint32_t resp, uint32_t mbar) {
    asm volatile("clusterlaunchcontrol.try_cancel.async.shared::cta.mbarrier::complete_tx::bytes.b128 [%0], [%1];" ::"r"(resp),
                 "r"(mbar)
                 : "memory");
}
// The cancelled CTA's index, or false when there was none left.
__device__ __forceinline__ bool cancel_answer(uint32_t resp, int& x, int& y) {
    uint32_t ok, a = 0, b = 0;
    asm volatile(
        "{ .reg .b128 h; .reg .pred p; .reg .b32 z, u; ld.shared.b128 h, [%3]; "
        "clusterlaunchcontrol.query_cancel.is_canceled.pred.b128 p, h; selp.u32 %0, 1, 0, p; "
        "@p clusterlaunchcontrol.query_cancel.get_first_ctaid.v4.b32.b128 {%1, %2, z, u}, h; }"
        : "=r"(ok), "+r"(a), "+r"(b)
        : "r"(resp)
        : "memory");
    x = (int)a;
    y = (int)b;
    return ok != 0;
}

// An item: rows p0 .. of the sequence of `len` tokens from token t0 on, KV head
// hk; len = 0 ends the queue.  Key tiles are counted from the first key that
// any of its rows sees (see_lo).
struct Item {
    int t0, len, p0, hk;
    int tiles, n;               // row tiles (1 or 2), key tiles
    int see_lo, see_hi;         // keys that any row sees
    int lo1, hi0;               // first key of row tile 1, last key of row tile 0
    __device__ __forceinline__ Item(int4 e, const Params& P) : t0(e.x), len(e.y), p0(e.z), hk(e.w) {
        const int wl = P.window_left, last = len - 1;
        tiles = p0 + P.NP < len ? 2 : 1;
        see_lo = wl >= 0 ? max(0, p0 - wl) : 0;
        see_hi = min(last, p0 + tiles * P.NP - 1);
        n = (see_hi - see_lo) / NK + 1;
        hi0 = min(last, p0 + P.NP - 1);
        lo1 = wl >= 0 ? max(0, p0 + P.NP - wl) : 0;
    }
    __device__ __forceinline__ int key_lo(int i) const { return i ? lo1 : see_lo; }
    __device__ __forceinline__ int key_hi(int i) const { return i ? see_hi : hi0; }
    __device__ __forceinline__ int first(int i) const { return (key_lo(i) - see_lo) / NK; }
    __device__ __forceinline__ int last(int i) const { return (key_hi(i) - see_lo) / NK; }
    // every used row of row tile i is one of the sequence
    __device__ __forceinline__ bool whole(int i, int NP) const { return p0 + (i + 1) * NP <= len; }
    // keys k .. k + 63: does any row of row tile i see one of them?
    __device__ __forceinline__ bool live(int i, int k) const { return k <= key_hi(i) && k + NK / 2 > key_lo(i); }
    // the last V tile has rows that none of the item's rows sees: it lands on
    // its slot's second barrier, for warp 3, which clears those rows and then
    // arrives on the slot's first (one barrier for all slots would take the
    // loads of two short items at once)
    __device__ __forceinline__ bool cleaned() const { return n * NK > see_hi - see_lo + 1; }
};

__global__ void __launch_bounds__(THREADS, 1)
    prompt_attention_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const __grid_constant__ CUtensorMap tm_o,
                            const Params P) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = (uint8_t*)(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t* qs = smem;                                     // two row tiles of 32 KiB
    uint8_t* ring = smem + 2 * SLOT;
    uint8_t* stage = ring + SLOTS * SLOT;                   // an output tile of 32 KiB
    int4* queue = (int4*)(stage + SLOT);
    int4* answer = queue + QUEUE;
    uint64_t* bars = (uint64_t*)(answer + 1);
    uint32_t* tmem_slot = (uint32_t*)(bars + B_COUNT);
    static_assert((QUEUE + 1) * 16 + B_COUNT * 8 + 4 <= 512, "shared memory behind the ring");
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rows = P.G * P.NP;                            // used rows of a tile
    pdl_launch_dependents();

    if (threadIdx.x == 0) {
        for (int i = 0; i < B_COUNT; ++i) {
            int count = 1;
            if ((i >= B_P && i < B_P + 4) || (i >= B_OE && i < B_STAGED + 2)) count = 4;    // softmax warps
            if (i >= B_EMPTY && i < B_EMPTY + SLOTS) count = 2;                         // MMA warps
            if (i >= B_TAKEN && i < B_TAKEN + QUEUE) count = ROLES;
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
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait();
    bool ok = true;
    // the queue's next entry (every role reads every entry, in order); false
    // after the last one
    int taken = 0;
    auto next_item = [&](int4& e) -> bool {
        const int s = taken % QUEUE;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(B_ITEM + s), (taken / QUEUE) & 1));
        if (!ok) return false;
        e = queue[s];
        ++taken;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(B_TAKEN + s));
        return e.y != 0;
    };

    if (warp == 0) {
        // ------------------------------------------------------------ loads
        uint64_t keep;                                      // K and V are read by many CTAs, Q by one
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(keep));
        const uint64_t once = policy_evict_first();
        int4 e;
        int done = 0, q_use[2] = {0, 0};
        uint32_t raw_now = 0, raw_odd = 0;                  // slots that hold a tile to be cleaned; slots with an odd number of such
        while (next_item(e)) {
            const Item it(e, P);
            if (lane == 0) {
                auto load_q = [&](int i) {
                    if (q_use[i] > 0) ok = mbar_wait(bar(B_QE + i), (q_use[i] - 1) & 1);
                    if (!ok) return;
                    mbar_expect_tx(bar(B_Q + i), 2 * rows * 128);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(smem_u32(qs + i * SLOT + h * HALF), &tm_q, 64 * h, it.hk * P.G,
                                    it.t0 + it.p0 + i * P.NP, bar(B_Q + i), once);
                    ++q_use[i];
                };
                load_q(0);
                for (int u = 0; u < 2 * it.n && ok; ++u) {  // K(0) V(0) K(1) V(1) ...
                    const int j = u >> 1, s = done % SLOTS, use = done / SLOTS;
                    if (use > 0) ok = mbar_wait(bar(B_EMPTY + s), (use - 1) & 1);
                    if (!ok) break;
                    uint32_t full = bar(B_FULL + s);
                    raw_now &= ~(1u << s);
                    if (u == 2 * it.n - 1 && it.cleaned()) {
                        full = bar(B_RAW + s);
                        raw_now |= 1u << s;
                        raw_odd ^= 1u << s;
                    }
                    mbar_expect_tx(full, SLOT);
                    for (int h = 0; h < 2; ++h)
                        tma_load_3d(smem_u32(ring + s * SLOT + h * HALF), u & 1 ? &tm_v : &tm_k, 64 * h, it.hk,
                                    it.t0 + it.see_lo + j * NK, full, keep);
                    ++done;
                    if (u == 0 && it.tiles == 2) load_q(1);
                }
            }
            ok = __shfl_sync(0xffffffffu, ok, 0);
            if (!ok) break;
        }
        if (lane == 0) {
            // never leave with copies into this CTA's shared memory in flight
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (q_use[i]) mbar_wait(bar(B_Q + i), (q_use[i] - 1) & 1);
            }
            for (int u = max(0, done - SLOTS); u < done; ++u) {
                const int t = u % SLOTS;
                if (raw_now >> t & 1) mbar_wait(bar(B_RAW + t), (raw_odd >> t & 1) ^ 1);
                else mbar_wait(bar(B_FULL + t), (u / SLOTS) & 1);
            }
        }
        __syncwarp();
    } else if (warp < 3) {
        // ------------------------------------- MMA issue of row tile i = warp - 1
        const int i = warp - 1;
        const bool leader = elect_one();
        const uint32_t s_col = tmem + TM_S + 128 * i, o_col = tmem + TM_O + 128 * i;
        const uint32_t q_lo = desc_lo(smem_u32(qs + i * SLOT), 16);
        const uint32_t k_lo0 = desc_lo(smem_u32(ring), 16), v_lo0 = desc_lo(smem_u32(ring), HALF);
        int slot = 0, phase = 0;                            // the ring's next item
        auto advance = [&]() {
            if (++slot == SLOTS) {
                slot = 0;
                phase ^= 1;
            }
        };
        int tile = 0, items = 0, turns = 0;                 // key tiles and items of this row tile, steps of both, so far
        int4 e;
        while (next_item(e)) {
            const Item it(e, P);
            const bool mine = i < it.tiles;
            const int jf = mine ? it.first(i) : 0, jl = mine ? it.last(i) : -1;
            if (mine) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(B_Q + i), items & 1));
                ++items;
            }
            int v_slot = 0, v_phase = 0;
            bool v_live[2] = {false, false};                // halves of the key tile before that some row sees
            for (int j = 0; j <= it.n && ok; ++j) {
                const bool pv = j - 1 >= jf && j - 1 <= jl, qk = j >= jf && j <= jl && j < it.n;
                // The two warps issue in turn, P.V and Q.K^T of one row tile
                // behind those of the other: left alone they fall into step,
                // both tiles' softmax at once and the tensor cores idle
                // meanwhile (8192 tokens: 905 us, in turn 744).  What a step needs is
                // waited for before its turn (881 us where it was not), and the
                // turn ends behind Q.K^T (earlier: 793 to 813 us instead of 724).
                if (j > 0) ok = mbar_wait(bar(B_FULL + v_slot), v_phase);
                if (ok && j < it.n) ok = mbar_wait(bar(B_FULL + slot), phase);
                // O of the previous item has been read
                if (ok && pv && j - 1 == jf && items > 1) ok = mbar_wait(bar(B_OE + i), items & 1);
                if (ok && pv) ok = mbar_wait(bar(B_P + 2 * i), tile & 1);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                if (i == 1 || turns > 0) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_TURN + i), (i == 1 ? turns : turns - 1) & 1));
                if (!ok) break;
                ++turns;
                fence_after();
                if (pv) {
                    // O += P(j - 1) V(j - 1)
                    const uint32_t v_lo = v_lo0 + v_slot * (SLOT >> 4);
                    if (leader) {
                        if (v_live[0]) {
#pragma unroll
                            for (int kk = 0; kk < 4; ++kk)
                                mma_ts(o_col, s_col + 8 * kk, v_lo + kk * (2048 >> 4), ID_PV, j - 1 > jf || kk > 0);
                        }
                        mma_commit(bar(B_H + i));
                    }
                    __syncwarp();
                    ok = __all_sync(0xffffffffu, mbar_wait(bar(B_P + 2 * i + 1), tile & 1));
                    fence_after();
                    if (leader && ok) {
                        if (v_live[1]) {
#pragma unroll
                            for (int kk = 4; kk < 8; ++kk)
                                mma_ts(o_col, s_col + 8 * kk, v_lo + kk * (2048 >> 4), ID_PV,
                                       j - 1 > jf || kk > 4 || v_live[0]);
                        }
                        mma_commit(bar(B_EMPTY + v_slot));
                        if (j - 1 == jl) mma_commit(bar(B_O + i));
                    }
                    __syncwarp();
                    ++tile;
                } else if (j > 0 && leader) {
                    mbar_arrive(bar(B_EMPTY + v_slot));
                }
                if (qk) {
                    // S = Q K(j)^T, over P(j - 1), which the MMAs above have read
                    const int k0 = it.see_lo + j * NK;
                    v_live[0] = it.live(i, k0);
                    v_live[1] = it.live(i, k0 + NK / 2);
                    if (leader && ok) {
                        // both halves, or the one that some row sees
                        const bool both = v_live[0] && v_live[1];
                        const int h = v_live[0] ? 0 : 1;
                        const uint32_t k_lo = k_lo0 + slot * (SLOT >> 4) + h * (64 * 128 >> 4);
#pragma unroll
                        for (int kk = 0; kk < 8; ++kk) {
                            const uint32_t off = ((kk >> 2) * HALF + (kk & 3) * 32) >> 4;
                            mma_ss(s_col + 64 * h, q_lo + off, k_lo + off, both ? ID_QK : ID_QK_HALF, kk > 0);
                        }
                        mma_commit(bar(B_S + i));
                    }
                }
                if (leader) {
                    mbar_arrive(bar(B_TURN + 1 - i));
                    if (qk) {
                        mma_commit(bar(B_EMPTY + slot));
                        if (j == jl) mma_commit(bar(B_QE + i));
                    } else if (j < it.n) {
                        mbar_arrive(bar(B_EMPTY + slot));
                    }
                }
                __syncwarp();
                if (j < it.n) {
                    advance();
                    v_slot = slot;
                    v_phase = phase;
                    advance();
                }
            }
            if (!ok) break;
        }
        // nothing the tensor cores still run may outlive the TMEM allocation
        if (leader) mma_commit(bar(B_IDLE + i));
        __syncwarp();
        mbar_wait(bar(B_IDLE + i), 0);
        __syncwarp();
    } else if (warp == 3) {
        // ------------------------------------------------- schedule and clean
        // Pair x (2 NP positions) of the launch, the last one first: sequence
        // b owns the indices from cu[b] / (2 NP) + b on, at least as many as it
        // has pairs, so the largest b whose first index is at most x is found
        // by a 32-way search, without a scan.
        const int PP = 2 * P.NP;
        int put = 0, bx = blockIdx.x, by = blockIdx.y;
        auto put_item = [&](int4 e) {
            const int s = put % QUEUE;
            if (put >= QUEUE) ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(B_TAKEN + s), (put / QUEUE - 1) & 1));
            if (lane == 0 && ok) {
                queue[s] = e;
                mbar_arrive(bar(B_ITEM + s));
            }
            __syncwarp();
            ++put;
        };
        int base = 0;
        uint32_t raw_odd = 0;                               // slots with an odd number of tiles cleaned
        auto clean = [&](int4 e) {
            const Item it(e, P);
            base += 2 * it.n;
            if (!it.cleaned()) return;
            const int s = (base - 1) % SLOTS;
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_RAW + s), raw_odd >> s & 1));
            if (!ok) return;
            raw_odd ^= 1u << s;
            const int z = it.see_hi - it.see_lo - (it.n - 1) * NK + 1;
            uint8_t* vt = ring + s * SLOT;
            for (int i = z * 8 + lane; i < NK * 8; i += 32) {   // rows [z, 128)
                *(uint4*)(vt + i * 16) = make_uint4(0, 0, 0, 0);
                *(uint4*)(vt + HALF + i * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_FULL + s));
        };
        // The output tiles of an item, in the order in which they are staged.
        // Both row tiles write one staging tile; this warp gives it to them, a
        // tile at a time, once the copy of the one before has read it.  A row
        // tile's next grant comes behind its last one's tile, so it waits for
        // every phase of its barrier in turn and can miss none.  (Waiting for
        // the other's copies instead, of which it need not see every one, a row
        // tile took an older phase for the one it meant.)
        int sends[2] = {0, 0};
        auto grant = [&](int i) {
            if (lane == 0) mbar_arrive(bar(B_STAGE + i));
        };
        auto send = [&](int4 e) {
            const Item it(e, P);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if (!ok || !it.whole(i, P.NP)) continue;
                if (i == 1) grant(1);
                ok = __all_sync(0xffffffffu, mbar_wait(bar(B_STAGED + i), sends[i] & 1));
                ++sends[i];
                if (lane == 0 && ok) {
                    for (int h = 0; h < 2; ++h)
                        tma_store_3d(&tm_o, smem_u32(stage + h * HALF), 64 * h, it.hk * P.G,
                                     it.t0 + it.p0 + i * P.NP);
                    bulk_commit();
                    bulk_wait_read();
                }
                __syncwarp();
            }
        };
        // every item is put into the queue before the one before it is cleaned
        // and sent: the loads run ahead
        int4 before = make_int4(0, 0, 0, 0);
        bool more = true;
        for (int k = 0; more && ok; ++k) {
            const int x = (int)(gridDim.y - 1) - by, hk = bx;
            // the request for the item after this one is under way meanwhile
            if (lane == 0) {
                fence_proxy_async();                        // the last answer was read before this one is written
                mbar_expect_tx(bar(B_NEXT), 16);
                cancel_request(smem_u32(answer), bar(B_NEXT));
            }
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
            if (lane == 0 && hk == 0 && x < P.B) {          // every sequence's bounds are looked at once
                const int c0 = P.cu[x], c1 = P.cu[x + 1];
                if (c0 < 0 || c1 < c0 || c1 > P.T || c1 - c0 > P.max_seq_len) flag(FP8KV_DEV_BAD_SEQ_LEN);
            }
            if (good && p0 >= 0 && p0 < s1 - s0) {
                const int4 e = make_int4(s0, s1 - s0, p0, hk);
                put_item(e);
                if (ok && before.y) clean(before);
                if (ok && before.y) send(before);
                if (ok && Item(e, P).whole(0, P.NP)) grant(0);
                before = e;
            }
            const bool got = mbar_wait(bar(B_NEXT), k & 1);
            more = __all_sync(0xffffffffu, got && cancel_answer(smem_u32(answer), bx, by));
            __syncwarp();
        }
        if (ok) put_item(make_int4(0, 0, 0, 0));
        if (ok && before.y) clean(before);
        if (ok && before.y) send(before);
    } else {
        // ----------------------------------------------- softmax and output
        const int i = (warp - 4) >> 2, wq = warp & 3;
        const int r = wq * 32 + lane;
        const uint32_t lanes = tmem + ((uint32_t)(wq * 32) << 16);
        const uint32_t s_col = lanes + TM_S + 128 * i, o_col = lanes + TM_O + 128 * i;
        const float mult = P.scale_log2;
        // position of this row and of the warp's first and last within a tile
        const int dpos = min(r, rows - 1) / P.G, head = min(r, rows - 1) % P.G;
        const int dfirst = min(wq * 32, rows - 1) / P.G, dlast = min(wq * 32 + 31, rows - 1) / P.G;
        int s_use = 0, o_use = 0, staged = 0;
        int4 e;
        while (next_item(e)) {
            const Item it(e, P);
            if (i >= it.tiles) continue;
            const int tile0 = it.p0 + i * P.NP, pos = tile0 + dpos;
            const int lo_r = P.window_left >= 0 ? max(0, pos - P.window_left) : 0;
            // halves of key tiles inside these bounds need no mask
            const int pmin = tile0 + dfirst, pmax = min(tile0 + dlast, it.key_hi(i));
            const int lomin = P.window_left >= 0 ? max(0, tile0 + dfirst - P.window_left) : 0;
            const int lomax = P.window_left >= 0 ? max(0, tile0 + dlast - P.window_left) : 0;
            float m_run = -INFINITY, l_run = 0.f;
            const int j_end = it.last(i);
#pragma unroll 1
            for (int j = it.first(i); j <= j_end; ++j) {
                ok = mbar_wait(bar(B_S + i), s_use & 1);
                if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                fence_after();
                const uint64_t mult2 = pack2(mult, mult);
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    const int k0 = it.see_lo + j * NK + 64 * h;
                    if (k0 > pmax || k0 + 63 < lomin) {
                        // no row of the warp sees a key of this half: P = 0
                        // (and no MMA reads it when no row of the tile does)
                        if (it.live(i, k0)) {
                            uint32_t zero[32];
#pragma unroll
                            for (int u = 0; u < 32; ++u) zero[u] = 0;
                            tmem_st_x32(s_col + 32 * h, zero);
                            tmem_wait_st();
                            fence_before();
                        }
                        __syncwarp();
                        if (lane == 0) mbar_arrive(bar(B_P + 2 * i + h));
                        continue;
                    }
                    uint32_t sv[64];
                    tmem_ld_x64(s_col + 64 * h, sv);
                    tmem_wait_ld();
                    if (k0 + 63 > pmin || k0 < lomax) {
                        // this row's visible columns of the half as bits
                        const int c0 = max(0, lo_r - k0), c1 = min(64, pos - k0 + 1);
                        const uint64_t below1 = c1 <= 0 ? 0ull : (c1 >= 64 ? ~0ull : (1ull << c1) - 1);
                        const uint64_t below0 = c0 >= 64 ? ~0ull : (1ull << c0) - 1;
                        const uint64_t see = below1 & ~below0;
                        const uint32_t see0 = (uint32_t)see, see1 = (uint32_t)(see >> 32);
#pragma unroll
                        for (int u = 0; u < 64; ++u)
                            sv[u] = ((u < 32 ? see0 : see1) >> (u & 31)) & 1u ? sv[u] : 0xff800000u;   // -inf
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
                    const bool grow = m_run != -INFINITY && tmax > m_run + 8.0f;
                    if (__any_sync(0xffffffffu, grow)) {
                        // S(j) ready means that P.V of the tiles before is
                        // complete; the first half's of this one is waited for
                        if (h == 1) {
                            ok = mbar_wait(bar(B_H + i), s_use & 1);
                            if (!__all_sync(0xffffffffu, ok)) { ok = false; break; }
                            fence_after();
                        }
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
                    const uint64_t neg2 = pack2(neg, neg);
                    uint64_t sum2[2] = {0, 0};
                    uint32_t pw[32];
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        float x0, x1;
                        unpack2(fma2(pack2(__uint_as_float(sv[2 * u]), __uint_as_float(sv[2 * u + 1])), mult2, neg2),
                                x0, x1);
                        x0 = ex2(x0);
                        x1 = ex2(x1);
                        sum2[u & 1] = add2(sum2[u & 1], pack2(x0, x1));
                        pw[u] = pack_bf16x2(x0, x1);
                    }
                    tmem_st_x32(s_col + 32 * h, pw);
                    float s0, s1;
                    unpack2(add2(sum2[0], sum2[1]), s0, s1);
                    l_run += s0 + s1;
                    tmem_wait_st();
                    fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(bar(B_P + 2 * i + h));
                }
                // (complete before the next S; waited for so that no phase of the
                // barrier is missed, here, where it delays nothing: between S and
                // its softmax it cost 8192 tokens 753 us instead of 724)
                if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(B_H + i), s_use & 1));
                if (!ok) break;
                ++s_use;
            }
            // ------------------------------------------------------ output
            if (ok) ok = mbar_wait(bar(B_O + i), o_use & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            ++o_use;
            fence_after();
            const float inv = 1.0f / l_run;
            uint32_t w[64];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                uint32_t ov[64];
                tmem_ld_x64(o_col + 64 * c, ov);
                tmem_wait_ld();
#pragma unroll
                for (int u = 0; u < 32; ++u)
                    w[32 * c + u] =
                        pack_bf16x2(__uint_as_float(ov[2 * u]) * inv, __uint_as_float(ov[2 * u + 1]) * inv);
            }
            // O is in registers: the next item's first P.V may overwrite it
            fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(B_OE + i));
            // A whole tile goes out as one tensor copy from shared memory (warp
            // 3), so that the next item's first key tiles do not wait behind
            // stores (3100 of an item's 17000 cycles, 16384 tokens, 512-key
            // window).  The two row tiles share the staging tile, in order:
            // warp 3 gives it to each once the copy before its own has read it.
            // A sequence's last tile, with rows behind its end, is stored row
            // by row.
            if (it.whole(i, P.NP)) {
                ok = __all_sync(0xffffffffu, mbar_wait(bar(B_STAGE + i), staged & 1));
                if (!ok) break;
                ++staged;
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    *(uint4*)(stage + (c >> 3) * HALF + r * 128 + (((c ^ r) & 7) << 4)) =
                        make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
                fence_proxy_async();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar(B_STAGED + i));
            } else if (r < rows && pos < it.len) {
                uint4* dst = (uint4*)(P.out + ((int64_t)(it.t0 + pos) * P.Hq + it.hk * P.G + head) * 128);
#pragma unroll
                for (int c = 0; c < 16; ++c) dst[c] = make_uint4(w[4 * c], w[4 * c + 1], w[4 * c + 2], w[4 * c + 3]);
            }
            __syncwarp();
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
    static std::atomic<uint64_t> done{0};
    if (opt_in_smem(done, (const void*)prompt::prompt_attention_kernel, prompt::SMEM) != cudaSuccess)
        return (cudaGetLastError(), FP8KV_ERR_CUDA);
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
