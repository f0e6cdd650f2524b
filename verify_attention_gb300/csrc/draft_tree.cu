// draft_tree.cu -- what a step of speculative decoding over a tree of drafted
// tokens needs beside its attention: the tree's ancestors, positions and cache
// slots before it, and the accepted path's cache rows moved together after it.
#include <algorithm>

#include "attention.cuh"
#include "common.cuh"

namespace fp8kv {

int status_draft_tree(unsigned int* s, int clear) { return read_status(s, clear); }

// ---------------------------------------------------------------- metadata
//
// Ancestors by pointer doubling: with word(m) = {m} and up(m) = m's parent,
//     word(m) |= word(up(m)),  up(m) = up(up(m))
// holds after i rounds the 2^i nodes from m upwards, so six rounds cover any
// path of 64.  A node without a valid parent points at itself; one whose word
// lacks node 0 after that hangs from no root and is padding.
//
// One warp a sequence, nodes m and m + 32 on lane m: no shared memory, no
// barrier.  Launch latency bounds it (one sequence of 12 nodes), or for a large
// batch the 32 bytes a node that it has to move.
__global__ void __launch_bounds__(128) tree_metadata_kernel(const int32_t* __restrict__ parents,
                                                            const int32_t* __restrict__ seq_lens,
                                                            const int32_t* __restrict__ block_table, int mpps, int B,
                                                            int M, int num_pages, int page_size, int max_seq_len,
                                                            uint64_t* __restrict__ mask, int64_t* __restrict__ positions,
                                                            int64_t* __restrict__ slots) {
    pdl_launch_dependents();
    pdl_wait();
    const int b = (blockIdx.x * blockDim.x + threadIdx.x) >> 5, lane = threadIdx.x & 31;
    if (b >= B) return;
    const int L = seq_lens[b];
    const bool seq_ok = L >= M && L <= max_seq_len && (L + page_size - 1) / page_size <= mpps;
    if (!seq_ok && lane == 0) flag(FP8KV_DEV_BAD_SEQ_LEN);
    int up[2], page[2];
    uint64_t word[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = lane + 32 * h;
        const int p = m > 0 && m < M ? parents[(int64_t)b * M + m] : 0;
        // (read beside the parent: the slot needs it only for nodes of the tree)
        page[h] = seq_ok && m < M ? block_table[(int64_t)b * mpps + (L - M + m) / page_size] : 0;
        const bool ok = p >= 0 && p < m;
        if (m > 0 && m < M && !ok && p != -1) flag(FP8KV_DEV_BAD_TREE);
        up[h] = ok ? p : m;
        word[h] = 1ull << m;
    }
#pragma unroll
    for (int round = 0; round < 6; ++round) {
        uint64_t add[2];
        int next[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const uint64_t w0 = __shfl_sync(0xffffffffu, word[0], up[h] & 31);
            const uint64_t w1 = __shfl_sync(0xffffffffu, word[1], up[h] & 31);
            const int u0 = __shfl_sync(0xffffffffu, up[0], up[h] & 31);
            const int u1 = __shfl_sync(0xffffffffu, up[1], up[h] & 31);
            add[h] = up[h] < 32 ? w0 : w1;
            next[h] = up[h] < 32 ? u0 : u1;
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            word[h] |= add[h];
            up[h] = next[h];
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        const int m = lane + 32 * h;
        if (m >= M) continue;
        const bool node = seq_ok && (word[h] & 1ull);
        const int64_t i = (int64_t)b * M + m;
        int64_t slot = -1;
        if (node) {
            if (page[h] >= 0 && page[h] < num_pages)
                slot = (int64_t)page[h] * page_size + (L - M + m) % page_size;
            else
                flag(FP8KV_DEV_BAD_SLOT);
        }
        mask[i] = node ? word[h] : 0ull;
        positions[i] = seq_ok ? L - M + (node ? __popcll(word[h]) - 1 : 0) : 0;
        slots[i] = slot;
    }
}

// --------------------------------------------------------------- kept path
//
// Row i of the kept path comes from row path[i] >= i of the same sequence and
// the path ascends, so a thread that owns one 16-byte column of the rows can
// move them in order: no source is overwritten before it has been read, and no
// thread waits for another.  The rows of a batch are read before they are
// written, which keeps as many loads in flight.
//
// One CTA per (sequence, one or a few layers): the path, the page ids and with them
// every row's byte offset are looked up once, for K and V and all heads.  HBM bounds a
// large call, the launch and three dependent reads (length, page, row) a small
// one.
constexpr int kKeepBatch = 8;

struct KeepParams {
    uint8_t* k[kMaxLayers];
    uint8_t* v[kMaxLayers];
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* path;
    int32_t* new_seq_lens;
    int mpps, M, Hkv, num_pages, page_size, max_seq_len;
    int n_layers, per_cta;      // layers
};

// A row of the path in a cache: where its page begins, and its place in the page.
struct KeepRow {
    int64_t page;               // bytes
    int off;                    // rows
};

// Moves column `at` of `n` rows whose pages hold rows of UNIT bytes there.
template <typename V, int UNIT>
__device__ __forceinline__ void move_rows(uint8_t* cache, const KeepRow* src, const KeepRow* dst, int n, int64_t at) {
    for (int i0 = 0; i0 < n; i0 += kKeepBatch) {
        V x[kKeepBatch];
#pragma unroll
        for (int i = 0; i < kKeepBatch; ++i)
            if (i0 + i < n) x[i] = *reinterpret_cast<const V*>(cache + src[i0 + i].page + src[i0 + i].off * UNIT + at);
#pragma unroll
        for (int i = 0; i < kKeepBatch; ++i)
            if (i0 + i < n) *reinterpret_cast<V*>(cache + dst[i0 + i].page + dst[i0 + i].off * UNIT + at) = x[i];
    }
}

template <int DT>
__global__ void __launch_bounds__(256) keep_path_kernel(const __grid_constant__ KeepParams P) {
    constexpr int ROW = DT == FP8KV_CACHE_BF16 ? 256 : DT == FP8KV_CACHE_E4M3 ? 128 : kInt4RowBytes;
    __shared__ KeepRow src[64], dst[64];
    __shared__ int moves;
    pdl_launch_dependents();
    pdl_wait();
    const int b = blockIdx.x, layer0 = blockIdx.y * P.per_cta, layers = min(P.per_cta, P.n_layers - layer0);
    const int tid = threadIdx.x;
    if (tid < 32) {
        // lanes: rows tid and tid + 32 of the path
        const int L = P.seq_lens[b];
        const bool seq_ok = L >= P.M && L <= P.max_seq_len && (L + P.page_size - 1) / P.page_size <= P.mpps;
        int node[2], len[2];
        bool good = true;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = tid + 32 * h;
            node[h] = i < P.M ? P.path[(int64_t)b * P.M + i] : -1;
            len[h] = __popc(__ballot_sync(0xffffffffu, node[h] >= 0));
        }
        const int n = len[0] + len[1];
        // rows 0 .. n - 1 hold ascending nodes < M that begin with the root, the rest none
        const int before0 = __shfl_up_sync(0xffffffffu, node[0], 1), last0 = __shfl_sync(0xffffffffu, node[0], 31);
        const int up1 = __shfl_up_sync(0xffffffffu, node[1], 1), before1 = tid ? up1 : last0;
        good &= tid < n ? (tid ? node[0] > before0 : node[0] == 0) && node[0] < P.M : node[0] < 0;
        good &= tid + 32 < n ? node[1] > before1 && node[1] < P.M : node[1] < 0;
        const bool path_ok = __all_sync(0xffffffffu, good) && n > 0;
        if (tid == 0 && layer0 == 0) {
            if (!seq_ok) flag(FP8KV_DEV_BAD_SEQ_LEN);
            else if (!path_ok) flag(FP8KV_DEV_BAD_TREE);
            P.new_seq_lens[b] = seq_ok && path_ok ? L - P.M + n : L;
        }
        int put = 0;
        const int32_t* table = P.block_table + (int64_t)b * P.mpps;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int i = tid + 32 * h;
            const bool wants = seq_ok && path_ok && i < n && node[h] != i;      // (the others are where they belong)
            bool move = false;
            KeepRow from = {}, to = {};
            if (wants) {
                const int ps = L - P.M + node[h], pd = L - P.M + i;
                const int gs = table[ps / P.page_size], gd = table[pd / P.page_size];
                move = gs >= 0 && gs < P.num_pages && gd >= 0 && gd < P.num_pages;
                if (!move && layer0 == 0) flag(FP8KV_DEV_BAD_SLOT);
                const int64_t page_bytes = (int64_t)P.Hkv * P.page_size * ROW;
                from = {gs * page_bytes, ps % P.page_size};
                to = {gd * page_bytes, pd % P.page_size};
            }
            const uint32_t vote = __ballot_sync(0xffffffffu, move);
            if (move) {
                const int at = put + __popc(vote & ((1u << tid) - 1));
                src[at] = from;
                dst[at] = to;
            }
            put += __popc(vote);
        }
        if (tid == 0) moves = put;
    }
    __syncthreads();
    const int n = moves;
    if (n == 0) return;
    const int64_t head_bytes = (int64_t)P.page_size * ROW;
    if (DT == FP8KV_CACHE_INT4) {
        // per head four columns of 16 code bytes and one of 8 scale bytes
        for (int i = tid; i < layers * 2 * P.Hkv * 5; i += blockDim.x) {
            const int c = i % 5, h = i / 5 % P.Hkv, kv = i / 5 / P.Hkv;
            uint8_t* cache = (kv & 1 ? P.v : P.k)[layer0 + (kv >> 1)];
            if (c < 4) move_rows<uint4, kInt4CodeBytes>(cache, src, dst, n, h * head_bytes + c * 16);
            else move_rows<uint2, kInt4ScaleBytes>(cache, src, dst, n, h * head_bytes + P.page_size * kInt4CodeBytes);
        }
    } else {
        constexpr int C = ROW / 16;
        for (int i = tid; i < layers * 2 * P.Hkv * C; i += blockDim.x) {
            const int c = i % C, h = i / C % P.Hkv, kv = i / C / P.Hkv;
            uint8_t* cache = (kv & 1 ? P.v : P.k)[layer0 + (kv >> 1)];
            move_rows<uint4, ROW>(cache, src, dst, n, h * head_bytes + c * 16);
        }
    }
}

}  // namespace fp8kv

using namespace fp8kv;

extern "C" int fp8kv_tree_metadata(const int32_t* parents, const int32_t* seq_lens, const int32_t* block_table,
                                   int max_pages_per_seq, int max_seq_len, int B, int M, int num_pages, int page_size,
                                   uint64_t* tree_mask, int64_t* positions, int64_t* slot_mapping, void* stream) {
    if (B < 0 || M < 1 || num_pages <= 0 || max_pages_per_seq <= 0) return FP8KV_ERR_INVALID_ARG;
    if (M > FP8KV_TREE_MAX_NODES || (page_size != 32 && page_size != 64)) return FP8KV_ERR_UNSUPPORTED;
    if (max_seq_len < M || (int64_t)max_seq_len > (int64_t)max_pages_per_seq * page_size) return FP8KV_ERR_INVALID_ARG;
    if (B == 0) return FP8KV_OK;                                // nothing to do; no pointer is read
    if (!parents || !seq_lens || !block_table || !tree_mask || !positions || !slot_mapping) return FP8KV_ERR_INVALID_ARG;
    // sequences write their outputs while others still read
    const size_t nodes = (size_t)B * M, row_bytes = nodes * 8;
    const void* outs[3] = {tree_mask, positions, slot_mapping};
    for (int i = 0; i < 3; ++i) {
        if (overlap(outs[i], row_bytes, parents, nodes * 4) || overlap(outs[i], row_bytes, seq_lens, (size_t)B * 4) ||
            overlap(outs[i], row_bytes, block_table, (size_t)B * max_pages_per_seq * 4) ||
            overlap(outs[i], row_bytes, outs[(i + 1) % 3], row_bytes))
            return FP8KV_ERR_INVALID_ARG;
    }
    // a small batch: one sequence an SM, so that no warp waits for another's loads
    const int warps = B <= num_sms() ? 1 : 4;
    const cudaError_t e =
        launch_pdl(tree_metadata_kernel, dim3((unsigned)((B + warps - 1) / warps)), dim3(32 * warps), 0,
                   (cudaStream_t)stream, parents, seq_lens, block_table, max_pages_per_seq, B, M, num_pages, page_size,
                   max_seq_len, tree_mask, positions, slot_mapping);
    return e == cudaSuccess ? FP8KV_OK : (cudaGetLastError(), FP8KV_ERR_CUDA);
}

extern "C" int fp8kv_cache_keep_path(void* const* k_caches, void* const* v_caches, int n_layers, int cache_dtype,
                                     const int32_t* block_table, int max_pages_per_seq, const int32_t* seq_lens,
                                     int max_seq_len, const int32_t* path, int B, int M, int Hkv, int D, int num_pages,
                                     int page_size, int32_t* new_seq_lens, void* stream) {
    if (B < 0 || M < 1 || Hkv <= 0 || n_layers < 1 || num_pages <= 0 || max_pages_per_seq <= 0)
        return FP8KV_ERR_INVALID_ARG;
    if (cache_dtype != FP8KV_CACHE_E4M3 && cache_dtype != FP8KV_CACHE_BF16 && cache_dtype != FP8KV_CACHE_INT4)
        return FP8KV_ERR_INVALID_ARG;
    if (D != 128 || (page_size != 32 && page_size != 64) || M > FP8KV_TREE_MAX_NODES || n_layers > kMaxLayers ||
        Hkv > 65535)
        return FP8KV_ERR_UNSUPPORTED;
    if (max_seq_len < M || (int64_t)max_seq_len > (int64_t)max_pages_per_seq * page_size) return FP8KV_ERR_INVALID_ARG;
    if (B == 0) return FP8KV_OK;                                // nothing to do; no pointer is read
    if (!k_caches || !v_caches || !block_table || !seq_lens || !path || !new_seq_lens) return FP8KV_ERR_INVALID_ARG;
    // the lengths, the paths and the table are read while the new lengths are written
    const size_t len_bytes = (size_t)B * 4;
    if (overlap(new_seq_lens, len_bytes, seq_lens, len_bytes) ||
        overlap(new_seq_lens, len_bytes, path, len_bytes * M) ||
        overlap(new_seq_lens, len_bytes, block_table, len_bytes * max_pages_per_seq))
        return FP8KV_ERR_INVALID_ARG;
    KeepParams P;
    uintptr_t at[2 * kMaxLayers];
    for (int i = 0; i < n_layers; ++i) {
        P.k[i] = (uint8_t*)k_caches[i];
        P.v[i] = (uint8_t*)v_caches[i];
        at[2 * i] = reinterpret_cast<uintptr_t>(P.k[i]);
        at[2 * i + 1] = reinterpret_cast<uintptr_t>(P.v[i]);
        if (!P.k[i] || !P.v[i] || ((at[2 * i] | at[2 * i + 1]) & 15)) return FP8KV_ERR_INVALID_ARG;
    }
    // rows of a cache that is there twice would move twice
    const int row_bytes = cache_dtype == FP8KV_CACHE_BF16 ? 256 : cache_dtype == FP8KV_CACHE_E4M3 ? 128 : kInt4RowBytes;
    const uintptr_t cache_bytes = (uintptr_t)num_pages * Hkv * page_size * row_bytes;
    std::sort(at, at + 2 * n_layers);
    for (int i = 1; i < 2 * n_layers; ++i)
        if (at[i] - at[i - 1] < cache_bytes) return FP8KV_ERR_INVALID_ARG;
    P.block_table = block_table;
    P.seq_lens = seq_lens;
    P.path = path;
    P.new_seq_lens = new_seq_lens;
    P.mpps = max_pages_per_seq;
    P.M = M;
    P.Hkv = Hkv;
    P.num_pages = num_pages;
    P.page_size = page_size;
    P.max_seq_len = max_seq_len;
    auto kern = cache_dtype == FP8KV_CACHE_E4M3   ? keep_path_kernel<FP8KV_CACHE_E4M3>
                : cache_dtype == FP8KV_CACHE_BF16 ? keep_path_kernel<FP8KV_CACHE_BF16>
                                                  : keep_path_kernel<FP8KV_CACHE_INT4>;
    const int items = 2 * Hkv * (cache_dtype == FP8KV_CACHE_E4M3 ? 8 : cache_dtype == FP8KV_CACHE_BF16 ? 16 : 5);
    P.n_layers = n_layers;
    // a CTA takes several layers where there are more CTAs than fit at once, up to two
    // columns a thread (64 sequences, 48 layers: one KV head of E4M3 5.7 us with a layer a
    // CTA, 2.9 with 3; 8 heads of INT4 11.1, 9.7), and twice the threads where few CTAs
    // leave room for them (one layer, BF16: 2.2 us, 2.7 with 128; 64 sequences, 48 layers
    // 13.6, 11.3 with 128)
    const int64_t ctas = (int64_t)B * n_layers;
    P.per_cta = (int)std::max<int64_t>(1, std::min<int64_t>((ctas + 8 * num_sms() - 1) / (8 * num_sms()),
                                                            std::min((255 + items) / items, n_layers)));
    const int threads = items * P.per_cta > 128 && ctas <= 4 * num_sms() ? 256 : 128;
    const cudaError_t e =
        launch_pdl(kern, dim3((unsigned)B, (unsigned)((n_layers + P.per_cta - 1) / P.per_cta)), dim3(threads), 0, (cudaStream_t)stream, P);
    return e == cudaSuccess ? FP8KV_OK : (cudaGetLastError(), FP8KV_ERR_CUDA);
}
