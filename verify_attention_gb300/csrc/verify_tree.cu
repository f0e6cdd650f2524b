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
// number of tokens.  The FP64 units would bound the pass (two additions a token
// are five times the time of the HBM reads).  The weights and the sums are pairs
// of fp32 instead, hi + lo with the rounding error of each step in lo (the
// two-sum and two-product of Dekker and Knuth): 2^-46 of the weight a step.
#include "attention.cuh"
#include "common.cuh"

namespace fp8kv {

int status_verify_tree(unsigned int* s, int clear) { return read_status(s, clear); }

constexpr int kVerifyThreads = 512, kVerifyWarps = kVerifyThreads / 32, kVerifyMaxCluster = 8;

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

// The weights of a node's row after k children fell: step j takes w to (w a_j -
// b_j q)+, a_j a power of two that keeps the weights near 1 and b_j = S a_j.
struct VerifyStep {
    float a, bh, bl;
};

__device__ __forceinline__ F2 step_weight(F2 w, float q, VerifyStep s) {
    const float th = __fmul_rn(s.bh, q), tl = __fmaf_rn(s.bl, q, __fmaf_rn(s.bh, q, -th));
    const F2 d = two_sum(__fmul_rn(w.hi, s.a), -th);
    const float lo = __fadd_rn(d.lo, __fsub_rn(__fmul_rn(w.lo, s.a), tl));
    const float hi = __fadd_rn(d.hi, lo);
    // (negative, zero and NaN: nothing left)
    return hi > 0.f ? F2{hi, __fsub_rn(lo, __fsub_rn(hi, d.hi))} : F2{0.f, 0.f};
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

// One row as groups of N elements on 16-byte boundaries: group g holds elements
// N g - skew .. + N - 1, those outside [0, V) as zeros.
template <typename T>
struct Row {
    static constexpr int N = 16 / sizeof(T);
    const T* at;                // element -skew, on a 16-byte boundary
    int skew, V;
    __device__ __forceinline__ Row(const T* row, int skew_, int V_) : at(row - skew_), skew(skew_), V(V_) {}
    __device__ __forceinline__ void load(int g, bool aligned, float (&f)[N]) const {
        const int first = N * g - skew;
        if (aligned && first >= 0 && first + N <= V) {
            widen(__ldg(reinterpret_cast<const uint4*>(at + (int64_t)N * g)), f);
        } else {
#pragma unroll
            for (int i = 0; i < N; ++i) f[i] = first + i >= 0 && first + i < V ? prob(at[(int64_t)N * g + i]) : 0.f;
        }
    }
};

__device__ __forceinline__ double dsmem_ld_f64(uint32_t a) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(a) : "memory");
    return v;
}

template <typename T, bool DRAFT>
__global__ void __launch_bounds__(kVerifyThreads) verify_tree_kernel(VerifyParams P) {
    constexpr int N = Row<T>::N, UNROLL = 4;
    __shared__ int par[64], tok[64], fallen[64], path[64];
    __shared__ float up[64], pw[64], qw[64];
    __shared__ VerifyStep steps[64];
    __shared__ double warp_sum[kVerifyWarps], cta_sum[2], sums[kVerifyMaxCluster];
    __shared__ int s_cur, s_fallen, s_state, s_depth;
    pdl_launch_dependents();
    const int C = P.cluster, rank = blockIdx.x % C, b = blockIdx.x / C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, M = P.M, V = P.V;
    const T* p_rows = (const T*)P.p + (int64_t)b * M * P.p_stride;
    const T* q_rows = (const T*)P.q + (int64_t)b * M * P.q_stride;
    pdl_wait();
    if (tid < M) {
        // a node's token in its parent's rows: the walk below reads no memory
        const int64_t i = (int64_t)b * M + tid;
        int pa = tid ? P.parents[i] : -1;
        const int x = P.tokens[i];
        up[tid] = P.uniforms[i];
        if (pa < -1 || pa >= tid || (pa >= 0 && (x < 0 || x >= V))) {
            if (tid) {
                if (rank == 0) flag(FP8KV_DEV_BAD_TREE);
                pa = -1;
            }
        }
        par[tid] = pa;
        tok[tid] = x;
        pw[tid] = pa >= 0 ? prob(p_rows[pa * P.p_stride + x]) : 0.f;
        qw[tid] = DRAFT && pa >= 0 ? prob(q_rows[pa * P.q_stride + x]) : 1.f;
    }
    if (tid == 0) {
        s_cur = s_depth = s_fallen = 0;
        path[0] = 0;
    }
    __syncthreads();

    // the walk's state, thread 0's: the next node to look at, S, the weight's
    // scale (a power of two)
    int m = 1;
    double S = 1.0;
    int passes = 0;
    // states: 1 a pass for S of the current node, 2 the last draw, 3 the last draw
    // from the node's own row (nothing was left of it)
    while (true) {
        if (tid == 0) {
            int cur = s_cur, k = s_fallen, depth = s_depth, state = 2;
            for (; m < M; ++m) {
                if (par[m] != cur) continue;
                const int x = tok[m];
                double w = fmax((double)pw[m], 0.0);
                const double qx = fmax((double)qw[m], 0.0);
                if (DRAFT) {
                    for (int j = 0; j < k; ++j)
                        w = fmax(w * steps[j].a - ((double)steps[j].bh + (double)steps[j].bl) * qx, 0.0);
                } else {
                    for (int j = 0; j < k; ++j)
                        if (fallen[j] == x) w = 0.0;
                }
                if (w > 0.0 && (double)up[m] * S * qx < w) {
                    cur = m;
                    path[++depth] = m;
                    k = 0;
                    S = 1.0;
                    continue;
                }
                if (DRAFT) {
                    // (a step's factor from S as it was for this child)
                    int e = 0;
                    if (S > 0.0) e = min(max(-ilogb(S), -120), 120);
                    const double bs = ldexp(S, e);
                    const float bh = (float)bs;
                    steps[k] = {ldexpf(1.0f, e), bh, (float)(bs - (double)bh)};
                } else {
                    fallen[k] = x;
                    S -= w;
                }
                ++k;
                if (DRAFT) {
                    int sib = m + 1;
                    while (sib < M && par[sib] != cur) ++sib;
                    if (sib < M) {
                        m = sib;
                        state = 1;
                        break;
                    }
                }
            }
            s_cur = cur;
            s_fallen = k;
            s_depth = depth;
            s_state = state;
        }
        __syncthreads();
        int state = s_state, k = s_fallen;
        const int cur = s_cur;
        const T* p_row = p_rows + (int64_t)cur * P.p_stride;
        const T* q_row = q_rows + (int64_t)cur * P.q_stride;
        // groups of 16 bytes, cut at the boundaries of p's row; q's only if they are its own too
        const int skew = (int)((reinterpret_cast<uintptr_t>(p_row) & 15) / sizeof(T));
        const bool q_aligned = DRAFT && (int)((reinterpret_cast<uintptr_t>(q_row) & 15) / sizeof(T)) == skew;
        const Row<T> pr(p_row, skew, V), qr(q_row, skew, V);
        const int groups = (V + skew + N - 1) / N;
        const int per_warp = ((groups + C * kVerifyWarps - 1) / (C * kVerifyWarps) + 31) & ~31;
        double total = 0.0;
        for (int attempt = 0;; ++attempt) {
            if (state == 3) k = 0;
            // what is left of group g
            auto weights = [&](int g, const float (&pf)[N], const float (&qf)[N], F2 (&w)[N]) {
#pragma unroll
                for (int i = 0; i < N; ++i) w[i] = {fmaxf(pf[i], 0.f), 0.f};
                if (DRAFT) {
                    for (int j = 0; j < k; ++j) {
                        const VerifyStep s = steps[j];
#pragma unroll
                        for (int i = 0; i < N; ++i) w[i] = step_weight(w[i], fmaxf(qf[i], 0.f), s);
                    }
                } else {
                    const int first = N * g - skew;
                    for (int j = 0; j < k; ++j) {
                        const unsigned at = (unsigned)(fallen[j] - first);
                        if (at < (unsigned)N) {
#pragma unroll
                            for (int i = 0; i < N; ++i)
                                if (at == (unsigned)i) w[i] = {0.f, 0.f};
                        }
                    }
                }
            };
            // the sum of a warp's run
            auto run_begin = [&](int r, int w) { return (r * kVerifyWarps + w) * per_warp; };
            const int g0 = run_begin(rank, warp), g1 = min(groups, g0 + per_warp);
            F2 acc = {0.f, 0.f};
            for (int g = g0; g < g1; g += 32 * UNROLL) {
                float pf[UNROLL][N], qf[UNROLL][N];
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    const int at = g + 32 * u + lane;
#pragma unroll
                    for (int i = 0; i < N; ++i) pf[u][i] = qf[u][i] = 0.f;
                    if (at < g1) {
                        pr.load(at, true, pf[u]);
                        if (DRAFT && k > 0) qr.load(at, q_aligned, qf[u]);
                    }
                }
#pragma unroll
                for (int u = 0; u < UNROLL; ++u) {
                    F2 w[N];
                    weights(g + 32 * u + lane, pf[u], qf[u], w);
#pragma unroll
                    for (int i = 0; i < N; ++i) {
                        const F2 s = two_sum(acc.hi, w[i].hi);
                        acc.hi = s.hi;
                        acc.lo = __fadd_rn(acc.lo, __fadd_rn(s.lo, w[i].lo));
                    }
                }
            }
            double sum = (double)acc.hi + (double)acc.lo;
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) warp_sum[warp] = sum;
            __syncthreads();
            if (tid == 0) {
                double s = 0.0;
                for (int w = 0; w < kVerifyWarps; ++w) s += warp_sum[w];
                cta_sum[passes & 1] = s;
            }
            // (two places in turn: a CTA that is a pass ahead does not overwrite
            // a sum that another still reads)
            if (C > 1) {
                __syncthreads();
                cluster_arrive();
                cluster_wait();
                if (tid < C) sums[tid] = dsmem_ld_f64(dsmem_addr(&cta_sum[passes & 1], tid));
            } else if (tid == 0) {
                sums[0] = cta_sum[passes & 1];
            }
            ++passes;
            __syncthreads();
            total = 0.0;
            for (int r = 0; r < C; ++r) total += sums[r];
            if (state == 2 && !(total > 0.0)) {
                state = 3;
                __syncthreads();                            // warp_sum and sums are written again
                continue;
            }
            if (state == 1) break;
            // ---- the draw: the CTA, the warp's run and the token whose running
            // sum exceeds t
            const double t = (double)up[0] * total;
            const bool valid = total > 0.0 && total <= 1.7e308;
            double before = 0.0;
            int owner = 0;
            for (int r = 0; r < C; ++r) {
                if (sums[r] > 0.0) owner = r;
                if (before + sums[r] > t) break;
                if (r + 1 < C) before += sums[r];
            }
            const int depth = s_depth;
            if (rank == 0) {
                for (int i = tid; i < M; i += kVerifyThreads) {
                    P.path[(int64_t)b * M + i] = i <= depth ? path[i] : -1;
                    if (i != depth || !valid)
                        P.out_tokens[(int64_t)b * M + i] = i < depth ? tok[path[i + 1]] : -1;
                }
                if (tid == 0) {
                    P.num_tokens[b] = valid ? depth + 1 : depth;
                    if (!valid) flag(FP8KV_DEV_BAD_PROBS);
                }
            }
            if (valid && rank == owner) {
                double base = 0.0;
                for (int r = 0; r < owner; ++r) base += sums[r];
                int w_at = 0;
                double w_base = base;
                for (int w = 0; w < kVerifyWarps; ++w) {
                    if (warp_sum[w] > 0.0) {
                        w_at = w;
                        w_base = base;
                    }
                    if (base + warp_sum[w] > t) break;
                    base += warp_sum[w];
                }
                if (warp == w_at) {
                    int last = -1, found = -1;                  // tokens
                    double run = w_base;
                    for (int g = g0; g < g1 && found < 0; g += 32) {
                        float pf[N], qf[N];
                        F2 w[N];
#pragma unroll
                        for (int i = 0; i < N; ++i) pf[i] = qf[i] = 0.f;
                        if (g + lane < g1) {
                            pr.load(g + lane, true, pf);
                            if (DRAFT && k > 0) qr.load(g + lane, q_aligned, qf);
                        }
                        weights(g + lane, pf, qf, w);
                        double mine = 0.0;
                        int top = -1;
#pragma unroll
                        for (int i = 0; i < N; ++i) {
                            mine += (double)w[i].hi + (double)w[i].lo;
                            if (w[i].hi > 0.f) top = N * (g + lane) - skew + i;
                        }
                        double incl = mine;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const double x = __shfl_up_sync(0xffffffffu, incl, o);
                            if (lane >= o) incl += x;
                        }
                        const uint32_t has = __ballot_sync(0xffffffffu, top >= 0);
                        const uint32_t over = __ballot_sync(0xffffffffu, top >= 0 && run + incl > t);
                        if (over) {
                            const int l = __ffs(over) - 1;
                            int pick = top;
                            double at = run + incl - mine;
#pragma unroll
                            for (int i = N - 1; i >= 0; --i) {
                                // the first element past t: the last one that the loop, backwards, finds past it
                                double upto = at;
#pragma unroll
                                for (int j = 0; j <= i; ++j) upto += (double)w[j].hi + (double)w[j].lo;
                                if (w[i].hi > 0.f && upto > t) pick = N * (g + lane) - skew + i;
                            }
                            found = __shfl_sync(0xffffffffu, pick, l);
                        } else if (has) {
                            last = __shfl_sync(0xffffffffu, top, 31 - __clz(has));
                        }
                        run += __shfl_sync(0xffffffffu, incl, 31);
                    }
                    // (a running sum that its roundings leave below t at the end of
                    // the run: its last token with a weight)
                    if (lane == 0) P.out_tokens[(int64_t)b * M + depth] = found >= 0 ? found : last;
                }
            }
            break;
        }
        if (state != 1) break;
        if (tid == 0) S = total;
        // thread 0 goes on with the walk; the sums are written again behind its barrier
        __syncthreads();
    }
    if (C > 1) {
        // no shared memory goes before every CTA has read the sums
        __syncwarp();
        cluster_arrive();
        cluster_wait();
    }
}

}  // namespace fp8kv

using namespace fp8kv;

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
    VerifyParams P;
    P.p = target_probs;
    P.q = draft_probs;
    P.p_stride = target_stride;
    P.q_stride = draft_stride;
    P.tokens = tokens;
    P.parents = parents;
    P.uniforms = uniforms;
    P.out_tokens = out_tokens;
    P.num_tokens = num_tokens;
    P.path = path;
    P.B = B;
    P.M = M;
    P.V = V;
    // CTAs a sequence: as many as keep the SMs busy, each with a few thousand tokens at least
    int c = 1;
    while (c < kVerifyMaxCluster && (int64_t)B * c * 2 <= 2 * num_sms() && V / (2 * c) >= 2048) c *= 2;
    if ((int64_t)B * c > 0x7fffffff) return FP8KV_ERR_UNSUPPORTED;
    P.cluster = c;
    auto kern = f32 ? (draft_probs ? verify_tree_kernel<float, true> : verify_tree_kernel<float, false>)
                    : (draft_probs ? verify_tree_kernel<uint16_t, true> : verify_tree_kernel<uint16_t, false>);
    const cudaError_t e =
        launch_pdl_cluster(kern, dim3((unsigned)(B * c)), dim3(kVerifyThreads), 0, (cudaStream_t)stream, c, P);
    return e == cudaSuccess ? FP8KV_OK : (cudaGetLastError(), FP8KV_ERR_CUDA);
}
