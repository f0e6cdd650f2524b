// verify_tree.cu -- which drafted tokens of a tree stand, from the target's and
// the drafter's probabilities and given random numbers, and the token after them.
//
// At node n, w is what is left of the target's distribution p_n and S its weight
// (w = p_n, S = 1 to begin with).  A child with token x, drawn from q_n, stands
// when u S q_n(x) < w(x) and w(x) > 0; otherwise
//     w <- (w - S q_n)+,   S <- sum w
// (a drafter without probabilities: q_n is 1 at x, so w(x) <- 0 and S <- S - w(x)).
// Behind the last node that stands, the next token is the first whose running sum
// of w exceeds u_0 times the sum of w.  The tokens are then distributed as if the
// target had drawn them one by one.
//
// What has to be read is a node's token in its parent's rows, for all nodes at
// once, and the vocabulary only where a child fell and a sibling follows, and for
// the last draw: one row of p and of q for a chain.  A thread-block cluster takes
// a sequence, each CTA a part of the vocabulary, each warp a run of it: a pass
// leaves a sum per warp, which locate the run that holds the drawn token, and only
// that run is read again.
//
// Whole numbers come out, so sums have to be good to far less than the smallest
// probability: a border that moves by e flips a draw with probability e times the
// number of tokens.  FP64 would bound the pass (2 additions a clock and SM: five
// times the time of the HBM reads; a first form with it in the scans took 17.8 us
// for one sequence of 131072 tokens, this one 6).  The weights, the sums and the prefixes are
// pairs of fp32 instead, hi + lo with the rounding error of each step in lo (the
// two-sum and two-product of Dekker and Knuth): at most 2^-45 of a weight a fall, 2^-44
// of a sum a token that is added to it.
#include "attention.cuh"
#include "common.cuh"

namespace fp8kv {

int status_verify_tree(unsigned int* s, int clear) { return read_status(s, clear); }

// Small CTAs, three or four an SM: while one waits for its cluster others add (64 trees
// of 100003 tokens, drawn: 38 us in CTAs of 512 threads, two an SM).  Two an SM where a
// chunk is 256 bf16 tokens of p and q, for their registers (30.2 us; three 33.2).
constexpr int kVerifyThreads = 256, kVerifyWarps = kVerifyThreads / 32, kVerifyMaxCluster = 16;

struct VerifyParams {
    const void *p, *q;
    int64_t p_stride, q_stride;                 // elements from one node's row to the next's
    const int32_t *tokens, *parents;
    const float* uniforms;
    int32_t *out_tokens, *num_tokens, *path;
    int B, M, V, cluster;
};

// A pair of fp32 that stands for hi + lo.
struct F2 {
    float hi, lo;
};

// a + b = s + e exactly
__device__ __forceinline__ F2 two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), x = __fsub_rn(s, a);
    return {s, __fadd_rn(__fsub_rn(a, __fsub_rn(s, x)), __fsub_rn(b, x))};
}
// the same for |a| >= |b|, or a = 0
__device__ __forceinline__ F2 fast_two_sum(float a, float b) {
    const float s = __fadd_rn(a, b);
    return {s, __fsub_rn(b, __fsub_rn(s, a))};
}
__device__ __forceinline__ F2 two_prod(float a, float b) {
    const float p = __fmul_rn(a, b);
    return {p, __fmaf_rn(a, b, -p)};
}
__device__ __forceinline__ F2 operator+(F2 a, F2 b) {
    const F2 s = two_sum(a.hi, b.hi);
    return fast_two_sum(s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo)));
}
__device__ __forceinline__ F2 operator-(F2 a, F2 b) { return a + F2{-b.hi, -b.lo}; }
__device__ __forceinline__ F2 operator*(F2 a, F2 b) {
    const F2 p = two_prod(a.hi, b.hi);
    return fast_two_sum(p.hi, __fadd_rn(p.lo, __fmaf_rn(a.hi, b.lo, __fmul_rn(a.lo, b.hi))));
}
__device__ __forceinline__ bool operator>(F2 a, F2 b) { return __fadd_rn(__fsub_rn(a.hi, b.hi), __fsub_rn(a.lo, b.lo)) > 0.f; }
__device__ __forceinline__ F2 shfl(F2 a, int lane) {
    return {__shfl_sync(0xffffffffu, a.hi, lane), __shfl_sync(0xffffffffu, a.lo, lane)};
}
// lane l < N: the sum of lanes 0 .. l
template <int N>
__device__ __forceinline__ F2 warp_scan(F2 a, int lane) {
#pragma unroll
    for (int o = 1; o < N; o <<= 1) {
        const F2 b = {__shfl_up_sync(0xffffffffu, a.hi, o), __shfl_up_sync(0xffffffffu, a.lo, o)};
        const F2 c = a + b;
        if (lane >= o) a = c;
    }
    return a;
}
// every lane: the sum of its N, the same for all (both sides of an exchange get the
// same sum and error; hi goes on without waiting for lo, which is joined at the end)
template <int N>
__device__ __forceinline__ F2 warp_total(F2 a) {
#pragma unroll
    for (int o = N / 2; o >= 1; o >>= 1) {
        const F2 b = {__shfl_xor_sync(0xffffffffu, a.hi, o), __shfl_xor_sync(0xffffffffu, a.lo, o)};
        const F2 s = two_sum(a.hi, b.hi);
        a = {s.hi, __fadd_rn(s.lo, __fadd_rn(a.lo, b.lo))};
    }
    return fast_two_sum(a.hi, a.lo);
}
// Of runs with the sums `run` that end at `end`: the first whose end exceeds t
// (should the roundings leave none: the last that holds anything; -1: none does).
__device__ __forceinline__ int locate(F2 run, F2 end, F2 t) {
    const unsigned some = __ballot_sync(0xffffffffu, run.hi > 0.f);
    const unsigned over = __ballot_sync(0xffffffffu, run.hi > 0.f && end > t);
    return over ? __ffs(over) - 1 : 31 - __clz(some);
}
__device__ __forceinline__ F2 before_lane(F2 scan, int at, F2 base) {
    const F2 left = shfl(scan, max(at, 1) - 1);
    return at > 0 ? base + left : base;
}

// The weights of a node's row after k children fell: step j takes w to (w a_j -
// b_j q)+, a_j a power of two that keeps the weights near 1 and b_j = S a_j.
struct __align__(16) VerifyStep {
    float a, bh, bl, unused;
};

// (Negative, zero and NaN: nothing left.  The differences are exact by the short sum:
// where the first operand is the smaller one, either nothing is left, or they are
// within a factor of two of each other and the difference itself is exact.  Little may
// be left of hi then, and lo be the larger one: the pair is put in order, as the next
// step and whoever asks for hi > 0 expect it.  The short sum is exact there too: d.hi is
// a multiple of the last places of both operands, lo at most a few of them, so d.hi is
// one of lo's last place.)
__device__ __forceinline__ F2 step_weight(F2 w, float q, VerifyStep s) {
    const float th = __fmul_rn(s.bh, q), tl = __fmaf_rn(s.bl, q, __fmaf_rn(s.bh, q, -th));
    const F2 d = fast_two_sum(__fmul_rn(w.hi, s.a), -th);
    const F2 left = fast_two_sum(d.hi, __fadd_rn(d.lo, __fmaf_rn(w.lo, s.a, -tl)));
    return {fmaxf(left.hi, 0.f), left.hi > 0.f ? left.lo : 0.f};
}
// a node's first step: S = 1, so w - q, exactly
__device__ __forceinline__ F2 first_step(float p, float q) {
    const F2 d = fast_two_sum(p, -q);
    return {fmaxf(d.hi, 0.f), d.hi > 0.f ? d.lo : 0.f};
}

template <typename T>
__device__ __forceinline__ float prob(T x);
template <>
__device__ __forceinline__ float prob<float>(float x) {
    return x;
}
template <>
__device__ __forceinline__ float prob<uint16_t>(uint16_t x) {
    return __uint_as_float((uint32_t)x << 16);
}

// N elements of 16 bytes as fp32
__device__ __forceinline__ void widen(uint4 x, float (&f)[4]) {
    f[0] = __uint_as_float(x.x);
    f[1] = __uint_as_float(x.y);
    f[2] = __uint_as_float(x.z);
    f[3] = __uint_as_float(x.w);
}
__device__ __forceinline__ void widen(uint4 x, float (&f)[8]) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
}

// One row as groups of 16 bytes: group g holds elements N g - skew .. + N - 1, those
// outside [0, V) as zeros.
template <typename T>
struct Row {
    static constexpr int N = 16 / sizeof(T);
    const T* at;                // element -skew
    int skew, V;
    bool aligned;               // on a 16-byte boundary
    __device__ __forceinline__ Row(const T* row, int skew_, int V_)
        : at(row - skew_), skew(skew_), V(V_), aligned((reinterpret_cast<uintptr_t>(row - skew_) & 15) == 0) {}
    __device__ __forceinline__ uint4 load(int g) const {
        const int first = N * g - skew;
        if (aligned && first >= 0 && first + N <= V) return __ldg(reinterpret_cast<const uint4*>(at) + g);
        uint32_t w[4] = {};
#pragma unroll
        for (int i = 0; i < N; ++i)
            if (first + i >= 0 && first + i < V) {
                const T x = at[(int64_t)N * g + i];
                if constexpr (N == 4) w[i] = __float_as_uint(x);
                else w[i >> 1] |= (uint32_t)x << (16 * (i & 1));
            }
        return {w[0], w[1], w[2], w[3]};
    }
};

// What a CTA tells the others of a pass: its sum, and where its walk stands.  Every
// CTA walks by itself and all read the same inputs; should those change during the
// call the walks may part, and no CTA may then wait for one, or send to one, that has
// gone.  All see the same words, so all stop at the same pass.
struct __align__(16) VerifyPart {
    F2 sum;
    int walk, unused;
};
__device__ __forceinline__ void send_part(uint32_t to, uint32_t mbar, F2 v, int walk) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(to),
                 "r"(__float_as_uint(v.hi)), "r"(__float_as_uint(v.lo)), "r"(walk), "r"(0), "r"(mbar)
                 : "memory");
}

enum { PASS_SUM = 1, PASS_DRAW = 2, PASS_ROW = 3, PASS_STOP = 4 };

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads, !DRAFT ? 4 : sizeof(T) == 4 ? 3 : 2) verify_tree_kernel(VerifyParams P) {
    constexpr int N = Row<T>::N, U = DRAFT && N == 4 ? 2 : 16 / N;      // groups a lane has in flight of a row
    __shared__ int tok[64], fallen[64], path[64];
    __shared__ float un[64], pw[64], qw[64];
    __shared__ unsigned kids[64][2], stands[2];         // bits: a node's children; nodes that stand as first children
    __shared__ VerifyStep steps[64];
    __shared__ F2 warp_sum[2][kVerifyWarps];            // of the warps' runs; of the parts of one of them
    __shared__ VerifyPart parts[2][kVerifyMaxCluster];
    __shared__ __align__(8) uint64_t bars[2];
    __shared__ F2 s_t, s_base;
    __shared__ int s_cur, s_fallen, s_state, s_depth, s_warp;
    pdl_launch_dependents();
    const int C = P.cluster, rank = blockIdx.x % C, b = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, M = P.M, V = P.V;
    const T* p_rows = (const T*)P.p + (int64_t)b * M * P.p_stride;
    const T* q_rows = (const T*)P.q + (int64_t)b * M * P.q_stride;
    if (tid < 64) kids[tid][0] = kids[tid][1] = 0;
    if (tid == 0) {
        mbar_init(smem_u32(&bars[0]), 1);
        mbar_init(smem_u32(&bars[1]), 1);
        fence_barrier_init();
    }
    __syncthreads();
    if (C > 1) cluster_arrive_relaxed();                    // waited for before anything is sent
    pdl_wait();
    if (tid < 64) {
        // a node's token in its parent's rows: the walk below reads no memory
        const int64_t i = (int64_t)b * M + tid;
        int pa = -1, x = 0;
        float u = 0.f, w = 0.f, q = 1.f;
        if (tid < M) {
            if (tid) pa = P.parents[i];
            x = P.tokens[i];
            u = P.uniforms[i];
        }
        if (pa < -1 || pa >= tid || (pa >= 0 && (x < 0 || x >= V))) {
            if (tid && rank == 0) flag(FP8KV_DEV_BAD_TREE);
            pa = -1;
        }
        if (pa >= 0) {
            w = prob(p_rows[pa * P.p_stride + x]);
            if (DRAFT) q = prob(q_rows[pa * P.q_stride + x]);
            atomicOr(&kids[pa][tid >> 5], 1u << lane);
        }
        w = fmaxf(w, 0.f);                                  // (NaN: 0)
        q = fmaxf(q, 0.f);
        tok[tid] = x;
        un[tid] = u;
        pw[tid] = w;
        qw[tid] = q;
        // u q < w, exactly
        const F2 uq = two_prod(u, q);
        const unsigned yes = __ballot_sync(0xffffffffu, w > 0.f && (uq.hi < w || (uq.hi == w && uq.lo < 0.f)));
        if (lane == 0) stands[warp] = yes;
        if (tid == 0) {
            s_cur = s_depth = s_fallen = 0;
            path[0] = 0;
        }
    }
    if (C > 1) cluster_wait();
    __syncthreads();

    // warp 0's (every lane the same): the children not yet looked at, and S
    uint64_t rest = (uint64_t)kids[0][1] << 32 | kids[0][0];
    F2 S = {1.f, 0.f};
    int passes = 0, state = 0;
    bool valid = true;
    while (true) {
        if (warp == 0 && state != PASS_ROW) {
            // ---- the walk, to the next pass: one for S of the current node, or the
            // last draw (from the node's own row, should nothing be left of it)
            int cur = s_cur, k = s_fallen, depth = s_depth;
            state = PASS_DRAW;
            const uint64_t first = (uint64_t)stands[1] << 32 | stands[0];
            while (rest) {
                const int m = __ffsll(rest) - 1;
                rest &= rest - 1;
                const int x = tok[m];
                F2 w = {pw[m], 0.f};
                bool yes = (first >> m) & 1;
                if (k > 0) {
                    const float qx = qw[m];
#pragma unroll 1
                    for (int j = 0; j < k; ++j) {
                        if (DRAFT) w = step_weight(w, qx, steps[j]);
                        else if (fallen[j] == x) w = {0.f, 0.f};
                    }
                    yes = w.hi > 0.f && w > two_prod(un[m], qx) * S;
                }
                if (yes) {
                    cur = m;
                    ++depth;
                    if (lane == 0) path[depth] = m;
                    rest = (uint64_t)kids[m][1] << 32 | kids[m][0];
                    k = 0;
                    S = {1.f, 0.f};
                    continue;
                }
                __syncwarp();
                if (DRAFT) {
                    // S a power of two away from [1, 2)
                    const int e = S.hi > 0.f ? min(max(127 - (int)(__float_as_uint(S.hi) >> 23), -120), 120) : 0;
                    const float a = __uint_as_float((unsigned)(127 + e) << 23);
                    if (lane == 0) steps[k] = {a, S.hi * a, S.lo * a, 0.f};
                } else {
                    if (lane == 0) fallen[k] = x;
                    S = S - w;
                }
                __syncwarp();
                ++k;
                if (DRAFT && rest) {
                    state = PASS_SUM;
                    break;
                }
            }
            if (lane == 0) {
                s_cur = cur;
                s_fallen = k;
                s_depth = depth;
                s_state = state;
            }
        }
        __syncthreads();
        state = s_state;
        const int cur = s_cur, k = state == PASS_ROW ? 0 : s_fallen;
        const T* p_row = p_rows + (int64_t)cur * P.p_stride;
        const T* q_row = q_rows + (int64_t)cur * P.q_stride;
        // groups of 16 bytes, cut at the boundaries of p's row (q's may be others)
        const int skew = (int)((reinterpret_cast<uintptr_t>(p_row) & 15) / sizeof(T));
        const Row<T> pr(p_row, skew, V), qr(q_row, skew, V);
        const int groups = (V + skew + N - 1) / N;
        const int per_warp = ((groups + C * kVerifyWarps - 1) / (C * kVerifyWarps) + 31) & ~31;
        // what is left of a group
        auto weigh = [&](uint4 x, uint4 y, int g, float (&hi)[N], float (&lo)[N]) {
            widen(x, hi);
            if (DRAFT) {
                float qf[N];
                widen(y, qf);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    qf[i] = fmaxf(qf[i], 0.f);
                    const F2 w = first_step(hi[i], qf[i]);  // (k = 0: q is 0 here)
                    hi[i] = w.hi;
                    lo[i] = w.lo;
                }
#pragma unroll 1
                for (int j = 1; j < k; ++j) {
                    const VerifyStep s = steps[j];
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const F2 w = step_weight({hi[i], lo[i]}, qf[i], s);
                        hi[i] = w.hi;
                        lo[i] = w.lo;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    hi[i] = fmaxf(hi[i], 0.f);
                    lo[i] = 0.f;
                }
#pragma unroll 1
                for (int j = 0; j < k; ++j) {
                    const int at = fallen[j] - (N * g - skew);
#pragma unroll
                    for (int i = 0; i < N; ++i)
                        if (at == i) hi[i] = 0.f;
                }
            }
        };
        // ---- stage 0: every warp's run of the row.  Behind the last pass, the CTA
        // that holds the token goes on to stage 1: the run that holds it, a part a
        // warp, and the warp of that part to stage 2: the token
        int begin = (rank * kVerifyWarps + warp) * per_warp, end = min(groups, begin + per_warp);
        F2 t = {0.f, 0.f}, run = {0.f, 0.f};                // the draw; the sum of the tokens before `begin`
        int token = -1;
        bool done = false;
        for (int stage = 0; stage < 3; ++stage) {
            auto fetch = [&](int g, uint4& x, uint4& y) {
                x = y = {};
                if (g < end) {
                    x = pr.load(g);
                    if (DRAFT && k > 0) y = qr.load(g);
                }
            };
            if (stage == 2) {
                // the token whose running sum exceeds t
                for (int g = begin; g < end; g += 32) {
                    uint4 x, y;
                    float hi[N], lo[N];
                    fetch(g + lane, x, y);
                    weigh(x, y, g + lane, hi, lo);
                    F2 mine = {0.f, 0.f};
#pragma unroll
                    for (int i = 0; i < N; ++i) mine = mine + F2{hi[i], lo[i]};
                    const F2 scan = warp_scan<32>(mine, lane);
                    F2 upto = before_lane(scan, lane, run);
                    int top = -1, pick = -1;
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        upto = upto + F2{hi[i], lo[i]};
                        if (hi[i] > 0.f) {
                            top = N * (g + lane) - skew + i;
                            if (pick < 0 && upto > t) pick = top;
                        }
                    }
                    const unsigned over = __ballot_sync(0xffffffffu, pick >= 0);
                    const unsigned some = __ballot_sync(0xffffffffu, top >= 0);
                    // (none, by the roundings of the sums: the last that holds anything)
                    if (over | some)
                        token = __shfl_sync(0xffffffffu, over ? pick : top, over ? __ffs(over) - 1 : 31 - __clz(some));
                    if (over) break;
                    run = run + shfl(scan, 31);
                }
                break;
            }
            F2 acc = {0.f, 0.f}, odd = {0.f, 0.f};           // two, for their latency
            auto add = [&](uint4 x, uint4 y, int g) {
                float hi[N], lo[N];
                weigh(x, y, g, hi, lo);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    F2& to = i & 1 ? odd : acc;
                    const F2 s = two_sum(to.hi, hi[i]);
                    to = {s.hi, __fadd_rn(to.lo, DRAFT ? __fadd_rn(s.lo, lo[i]) : s.lo)};
                }
            };
            // lo grows by up to 2^-24 of the sum a token: it is put back into place every four
            // to eight tokens of a sum, so that a token's rounding of lo stays below 2^-44 of
            // the sum (by the end only: 2^-24 of a lo that grows with the tokens)
            auto in_order = [&] {
                acc = fast_two_sum(acc.hi, acc.lo);
                odd = fast_two_sum(odd.hi, odd.lo);
            };
            // whole chunks of 32 groups, the next U on their way (64 trees, drawn: 46 us with
            // their loads behind branches that look at the row's ends); the others, and
            // all where q lies differently from p, one by one (`!both ||` beside qr.aligned would
            // spare passes that read no q: 64 trees, drawn: 30.8 us instead of 30.1)
            int g = begin;
            const int whole = min(end, qr.aligned ? (V + skew) / N : 0) - 31;
            if (g == 0 && skew && g < end) {
                uint4 x, y;
                fetch(lane, x, y);
                add(x, y, lane);
                g = 32;
                in_order();
            }
            if (g < whole) {
                const bool both = DRAFT && k > 0;
                int left = (whole - g + 31) >> 5;
                const uint4 *px = reinterpret_cast<const uint4*>(pr.at) + g + lane,
                            *py = reinterpret_cast<const uint4*>(qr.at) + g + lane;
                uint4 x[U], y[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    x[u] = y[u] = {};
                    if (u < left) x[u] = __ldg(px + 32 * u);
                    if (both && u < left) y[u] = __ldg(py + 32 * u);
                }
#pragma unroll 1
                for (; left > 0; left -= U, px += 32 * U, py += 32 * U) {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (u >= left) break;
                        const uint4 xu = x[u], yu = y[u];
                        if (u + U < left) x[u] = __ldg(px + 32 * (u + U));
                        if (both && u + U < left) y[u] = __ldg(py + 32 * (u + U));
                        add(xu, yu, g + lane);
                        g += 32;
                    }
                    in_order();
                }
            }
#pragma unroll 1
            for (; g < end; g += 32) {
                uint4 x, y;
                fetch(g + lane, x, y);
                add(x, y, g + lane);
                in_order();
            }
            // ---- the sums of the warps
            acc = acc + odd;
            acc = warp_total<32>(acc);
            if (lane == 0) warp_sum[stage][warp] = acc;
            __syncthreads();
            if (stage == 1) {
                const F2 part = lane < kVerifyWarps ? warp_sum[1][lane] : F2{0.f, 0.f};
                const F2 scan = warp_scan<kVerifyWarps>(part, lane);
                const int at = locate(part, run + scan, t);
                run = before_lane(scan, at, run);
                if (warp != at) break;
                continue;                                   // stage 2, of the same run
            }
            // ---- stage 0: the parts of the CTAs, every one to every one, in two
            // places in turn (one that is a pass ahead does not overwrite what
            // another still reads)
            const int turn = passes & 1;
            VerifyPart* got = parts[turn];
            if (warp == 0) {
                const F2 mine = lane < kVerifyWarps ? warp_sum[0][lane] : F2{0.f, 0.f};
                const F2 all = shfl(warp_total<kVerifyWarps>(mine), 0);
                const int walk = cur | k << 8 | state << 16;
                bool ok = true;
                if (C == 1) {
                    if (lane == 0) got[0] = {all, walk, 0};
                    __syncwarp();
                } else {
                    if (lane == 0) mbar_expect_tx(smem_u32(&bars[turn]), C * (int)sizeof(VerifyPart));
                    if (lane < C) send_part(dsmem_addr(&got[rank], lane), dsmem_addr(&bars[turn], lane), all, walk);
                    ok = __all_sync(0xffffffffu, mbar_wait(smem_u32(&bars[turn]), (passes >> 1) & 1));
                }
                const F2 part = lane < C ? got[lane].sum : F2{0.f, 0.f};
                ok &= !__any_sync(0xffffffffu, lane < C && got[lane].walk != walk);
                const F2 total = shfl(warp_total<kVerifyMaxCluster>(part), 0);
                S = total;
                int next = state, in = -1;
                if (!ok) {
                    next = PASS_STOP;
                } else if (state != PASS_SUM) {
                    if (total.hi > 0.f && total.hi <= 3.4e38f) {
                        // the draw: the CTA and the warp's run that hold the token
                        // whose running sum exceeds t
                        t = F2{un[0], 0.f} * total;
                        const F2 scan = warp_scan<kVerifyMaxCluster>(part, lane);
                        const int owner = locate(part, scan, t);
                        if (owner == rank) {
                            const F2 base = before_lane(scan, owner, {0.f, 0.f});
                            const F2 upto = warp_scan<kVerifyWarps>(mine, lane);
                            in = locate(mine, base + upto, t);
                            run = before_lane(upto, in, base);
                        }
                    } else if (state == PASS_DRAW && !(total.hi > 0.f)) {
                        next = PASS_ROW;
                    } else {
                        next = PASS_ROW + PASS_STOP;        // no token to draw
                    }
                }
                if (lane == 0) {
                    s_t = t;
                    s_base = run;
                    s_warp = in;
                    s_state = next;
                }
            }
            ++passes;
            __syncthreads();
            const int next = s_state;
            if (next == PASS_STOP) {
                if (rank == 0 && tid == 0) flag(FP8KV_DEV_BAD_TREE);
                return;
            }
            valid = next != PASS_ROW + PASS_STOP;
            done = !valid || (state != PASS_SUM && next == state);
            state = next;
            if (!done || s_warp < 0) break;
            t = s_t;
            run = s_base;
            const int r0 = (rank * kVerifyWarps + s_warp) * per_warp, r1 = min(groups, r0 + per_warp);
            const int share = ((r1 - r0 + kVerifyWarps - 1) / kVerifyWarps + 31) & ~31;
            begin = min(r0 + warp * share, r1);
            end = min(begin + share, r1);
        }
        if (done) {
            const int depth = s_depth;
            if (token >= 0 && lane == 0) P.out_tokens[(int64_t)b * M + depth] = token;
            if (rank == 0 && tid < M) {
                const int64_t i = (int64_t)b * M + tid;
                P.path[i] = tid <= depth ? path[tid] : -1;
                if (tid != depth || !valid) P.out_tokens[i] = tid < depth ? tok[path[tid + 1]] : -1;
                if (tid == 0) {
                    P.num_tokens[b] = valid ? depth + 1 : depth;
                    if (!valid) flag(FP8KV_DEV_BAD_PROBS);
                }
            }
            break;
        }
        __syncthreads();                                    // before warp 0 writes the walk's state again
    }
}

}  // namespace fp8kv

using namespace fp8kv;

// Opt in to clusters of 16, once per device (as opt_in_smem).
static cudaError_t allow_cluster16(std::atomic<uint64_t>& done, const void* kernel) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (done.load(std::memory_order_relaxed) & bit) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

extern "C" int fp8kv_verify_tree(const void* target_probs, int64_t target_stride, const void* draft_probs,
                                 int64_t draft_stride, int prob_dtype, const int32_t* tokens, const int32_t* parents,
                                 const float* uniforms, int B, int M, int V, int32_t* out_tokens, int32_t* num_tokens,
                                 int32_t* path, void* stream) {
    if (B < 0 || M < 1 || V < 1) return FP8KV_ERR_INVALID_ARG;
    if (prob_dtype != FP8KV_PROBS_FP32 && prob_dtype != FP8KV_PROBS_BF16) return FP8KV_ERR_INVALID_ARG;
    if (M > FP8KV_TREE_MAX_NODES || V > (1 << 30)) return FP8KV_ERR_UNSUPPORTED;
    if (target_stride < V || (draft_probs && draft_stride < V)) return FP8KV_ERR_INVALID_ARG;
    if (B == 0) return FP8KV_OK;                                // nothing to do; no pointer is read
    if (!target_probs || !tokens || !parents || !uniforms || !out_tokens || !num_tokens || !path)
        return FP8KV_ERR_INVALID_ARG;
    const bool f32 = prob_dtype == FP8KV_PROBS_FP32;
    const uintptr_t size = f32 ? 4 : 2;
    if (reinterpret_cast<uintptr_t>(target_probs) % size || reinterpret_cast<uintptr_t>(draft_probs) % size)
        return FP8KV_ERR_INVALID_ARG;
    // sequences write their outputs while others still read
    const size_t row_bytes = (size_t)B * M * 4, len_bytes = (size_t)B * 4;
    const size_t p_bytes = ((size_t)((int64_t)B * M - 1) * target_stride + V) * size;
    const size_t q_bytes = draft_probs ? ((size_t)((int64_t)B * M - 1) * draft_stride + V) * size : 0;
    for (const void* in : {(const void*)tokens, (const void*)parents, (const void*)uniforms}) {
        if (overlap(num_tokens, len_bytes, in, row_bytes)) return FP8KV_ERR_INVALID_ARG;
        // (a sequence's own row is read before it is written)
        for (const void* rows : {(const void*)out_tokens, (const void*)path})
            if (rows != in && overlap(rows, row_bytes, in, row_bytes)) return FP8KV_ERR_INVALID_ARG;
    }
    for (const void* rows : {(const void*)out_tokens, (const void*)path})
        if (overlap(rows, row_bytes, target_probs, p_bytes) || overlap(rows, row_bytes, draft_probs, q_bytes) ||
            overlap(rows, row_bytes, num_tokens, len_bytes))
            return FP8KV_ERR_INVALID_ARG;
    if (overlap(out_tokens, row_bytes, path, row_bytes) || overlap(num_tokens, len_bytes, target_probs, p_bytes) ||
        overlap(num_tokens, len_bytes, draft_probs, q_bytes))
        return FP8KV_ERR_INVALID_ARG;
    VerifyParams P;
    P.p = target_probs;
    // (chosen drafts: p's own rows stand for q's, which nothing reads, so that they lie
    // alike and the kernel's whole chunks are taken)
    P.q = draft_probs ? draft_probs : target_probs;
    P.p_stride = target_stride;
    P.q_stride = draft_probs ? draft_stride : target_stride;
    P.tokens = tokens;
    P.parents = parents;
    P.uniforms = uniforms;
    P.out_tokens = out_tokens;
    P.num_tokens = num_tokens;
    P.path = path;
    P.B = B;
    P.M = M;
    P.V = V;
    // CTAs a sequence: clusters of 16 (not portable, but one fits every GPC) down to 1
    // as the batch grows, with some 500 CTAs, about what fits at once, and a few
    // thousand tokens each.  (131072 tokens, chosen drafts: 5.6 us in 16 CTAs, 7.6 in
    // 8, 32 in one; 64 trees of 100003, drawn: 31.8 us in 8 CTAs each, 46.5 in 4, 32.8 in
    // 16, chosen 15.5, 21.0, 18.4; 8 such trees 13.2 in 16, 16.8 in 8.)
    const int most = 512;
    int c = 1;
    while (c < kVerifyMaxCluster && (int64_t)B * c * 2 <= most && V / (2 * c) >= 2048) c *= 2;
    if ((int64_t)B * c > 0x7fffffff) return FP8KV_ERR_UNSUPPORTED;
    P.cluster = c;
    auto kern = f32 ? (draft_probs ? verify_tree_kernel<float, true> : verify_tree_kernel<float, false>)
                    : (draft_probs ? verify_tree_kernel<uint16_t, true> : verify_tree_kernel<uint16_t, false>);
    static std::atomic<uint64_t> done[2][2];
    if (c > 8 && allow_cluster16(done[f32][draft_probs != nullptr], (const void*)kern) != cudaSuccess)
        return (cudaGetLastError(), FP8KV_ERR_CUDA);
    const cudaError_t e =
        launch_pdl_cluster(kern, dim3((unsigned)(B * c)), dim3(kVerifyThreads), 0, (cudaStream_t)stream, c, P);
    return e == cudaSuccess ? FP8KV_OK : (cudaGetLastError(), FP8KV_ERR_CUDA);
}
