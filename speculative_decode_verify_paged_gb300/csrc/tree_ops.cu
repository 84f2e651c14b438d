// Drafted trees: the tables of a step's trees (spec_attn_build_tree), the accepted
// path of each (spec_attn_accept_tree), and the move of its keys and values into
// place (spec_attn_move_kv).
//
// Tables.  A thread a node walks up its parents in shared memory, depth steps: a tree
// of 64 nodes has some 8 levels, the largest chain 1024.  Up to 256 nodes the words of
// its mask are registers (NW of them; with one word at a time, written as the walk
// leaves it, 256 trees of 255 nodes took 4.8 us, 3.1 like this); beyond, ancestors
// having lower places, the words come out from high to low, each written once.
//
// Accepted path.  Whether a child would be taken depends on its own parent only, so
// every node tests itself at once and the lowest child that passes is kept for each
// parent (a minimum in shared memory: its order does not matter).  One thread then
// follows the children, a shared-memory read a step.
//
// Move.  A path ascends, path[i] >= i, so step i writes a place that no later step
// reads: path[k] >= k > i for k > i.  A thread owns 16 bytes of every key of one (layer,
// KV head, K or V) and takes the steps in order, several loads ahead of their stores;
// no two threads touch the same bytes and nothing waits for another.
//
// Bound.  Each is a launch and a short chain of dependent loads (in a graph: tables of
// 8 trees of 64 nodes 1.8 us, of 256 trees of 255 3.1; accepted paths 2.0 and 2.3; the
// move of 8 trees' paths 2.6, of 32 trees' in 8 layers of d 256 3.1).
#include <cuda_runtime.h>
#include <limits.h>
#include <stdint.h>

#include "../../include/spec_attn.h"
#include "common.cuh"
#include "overlap.h"

namespace spec_attn {
namespace {

constexpr unsigned int kDevBadTree = SPEC_ATTN_DEV_BAD_TREE;

struct TreeParams {
    const int32_t* parents;
    const int32_t* seq_lens;
    const int32_t* q_indptr;
    const long long* draft;      // accept
    const long long* target;
    int32_t* positions;          // tables
    uint32_t* row_mask;
    int32_t* path;               // accept
    int32_t* accept_lens;
    long long* next_tokens;
    int32_t* ctx_lens;
    unsigned int* status;
    int num_reqs, total_rows, max_w, words, window, sinks, path_stride;
    int whole;                   // row_mask is aligned for 16-byte stores
};

struct TreeReq {
    int row0, w, len;
};
// A request's rows and length; false (and a status bit, by one thread) where they cannot be.
__device__ __forceinline__ bool tree_request(const TreeParams& p, int r, TreeReq& q) {
    const int row0 = p.q_indptr[r], row1 = p.q_indptr[r + 1];
    q.len = p.seq_lens[r];
    q.row0 = row0;
    q.w = 0;
    if (row0 < 0 || row1 < row0 || row1 > p.total_rows || row1 - row0 > p.max_w) {
        if (threadIdx.x == 0) atomicOr(p.status, kDevBadWindow);
        return false;
    }
    if (q.len < row1 - row0) {
        if (threadIdx.x == 0) atomicOr(p.status, kDevBadSeqLen);
        return false;
    }
    q.w = row1 - row0;
    return true;
}

// A node's parent, -1 (and a status bit) where it is no earlier node.
__device__ __forceinline__ int tree_parent(const TreeParams& p, int row0, int i) {
    const int v = p.parents[row0 + i];
    if (v >= -1 && v < i) return v;
    atomicOr(p.status, kDevBadTree);
    return -1;
}

template <int NW>
__global__ void build_tree_kernel(const TreeParams p) {
    extern __shared__ int parent[];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int r = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    // rows of no request, shared by all CTAs (none where the last window is below 0: they might be another request's)
    const int last = p.num_reqs ? p.q_indptr[p.num_reqs - 1] : 0, end = p.q_indptr[p.num_reqs];
    for (long long row = end < max(last, 0) ? p.total_rows : end + (long long)r * threads + tid; row < p.total_rows;
         row += (long long)gridDim.x * threads) {
        p.positions[row] = 0;
        for (int k = 0; k < p.words; ++k) p.row_mask[row * p.words + k] = 0;
    }
    TreeReq q;
    if (r == p.num_reqs || !tree_request(p, r, q)) return;
    for (int i = tid; i < q.w; i += threads) parent[i] = tree_parent(p, q.row0, i);
    __syncthreads();
    const int ctx = q.len - q.w;
    for (int i = tid; i < q.w; i += threads) {
        int depth = 0;
        if (p.window > 0)            // (which ancestors count depends on the node's own depth)
            for (int j = parent[i]; j >= 0; j = parent[j]) ++depth;
        uint32_t* out = p.row_mask + (long long)(q.row0 + i) * p.words;
        int above = 0;               // levels from the node up to j
        auto counts = [&] { return p.window == 0 || above < p.window || ctx + depth - above < p.sinks; };
        if constexpr (NW > 0) {
            uint32_t words[NW] = {};
            for (int j = i; j >= 0; j = parent[j], ++above) {
                const uint32_t bit = counts() ? 1u << (j & 31) : 0u;
#pragma unroll
                for (int k = 0; k < NW; ++k) words[k] |= j >> 5 == k ? bit : 0u;
            }
            if (p.words == NW && p.whole) {
#pragma unroll
                for (int k = 0; k < NW; k += 4)
                    *reinterpret_cast<uint4*>(out + k) = make_uint4(words[k], words[k + 1], words[k + 2], words[k + 3]);
            } else {
#pragma unroll
                for (int k = 0; k < NW; ++k)
                    if (k < p.words) out[k] = words[k];
                for (int k = NW; k < p.words; ++k) out[k] = 0;
            }
        } else {
            int at = p.words - 1;    // the word being made; those above are written
            uint32_t word = 0;
            for (int j = i; j >= 0; j = parent[j], ++above) {
                for (; at > j >> 5; --at, word = 0) out[at] = word;
                if (counts()) word |= 1u << (j & 31);
            }
            for (; at >= 0; --at, word = 0) out[at] = word;
        }
        p.positions[q.row0 + i] = ctx + above - 1;
    }
}

__global__ void accept_tree_kernel(const TreeParams p) {
    extern __shared__ long long target[];      // [max_w], then the children [max_w]
    int* child = reinterpret_cast<int*>(target + p.max_w);
    __shared__ int s_accepted;
    pdl_wait_primary();
    pdl_launch_dependents();
    const int r = blockIdx.x, tid = threadIdx.x, threads = blockDim.x;
    TreeReq q;
    const bool ok = tree_request(p, r, q);
    int32_t* path = p.path + (long long)r * p.path_stride;
    for (int i = tid; i < q.w; i += threads) {
        target[i] = p.target[q.row0 + i];
        child[i] = INT_MAX;
    }
    __syncthreads();
    for (int i = tid; i < q.w; i += threads) {
        const long long token = p.draft[q.row0 + i];
        const int up = tree_parent(p, q.row0, i);
        if (up >= 0 && token == target[up]) atomicMin(&child[up], i);
    }
    __syncthreads();
    if (tid == 0) {
        int n = 0, last = 0;
        for (int j = q.w > 0 ? 0 : INT_MAX; j != INT_MAX && n < p.path_stride; j = child[j]) {
            path[n++] = j;
            last = j;
        }
        s_accepted = n;
        p.accept_lens[r] = n;
        p.next_tokens[r] = n > 0 ? target[last] : -1;
        p.ctx_lens[r] = ok ? q.len - q.w + n : q.len;
    }
    __syncthreads();
    for (int i = s_accepted + tid; i < p.path_stride; i += threads) path[i] = -1;
}

constexpr int kMoveLayers = 64;                // of one launch: their addresses are kernel parameters
constexpr int kMoveThreads = 256;
constexpr int kMoveSteps = 256;                // places in shared memory at a time
constexpr int kMoveAhead = 8;                  // steps loaded before the first of them is stored

struct MoveParams {
    unsigned char* pool[2][kMoveLayers];       // K, V
    unsigned char* scales[2][kMoveLayers];
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* q_indptr;
    const int32_t* path;
    const int32_t* accept_lens;
    unsigned int* status;
    int num_kv_heads, page_shift, num_pages, bt_stride, path_stride;
    long long max_seq_len, kv_page_stride, scale_page_stride;
};

template <class T>
__device__ __forceinline__ void move_column(unsigned char* base, long long page_stride, int row_bytes,
                                            const int* src, const int* dst, int n, int page_shift) {
    // base: this thread's bytes of slot 0 of page 0; a place is page << page_shift | slot, -1: leave it
    const int mask = (1 << page_shift) - 1;
    auto at = [&](int place) {
        return reinterpret_cast<T*>(base + (long long)(place >> page_shift) * page_stride + (long long)(place & mask) * row_bytes);
    };
    for (int i0 = 0; i0 < n; i0 += kMoveAhead) {
        T x[kMoveAhead];
#pragma unroll
        for (int k = 0; k < kMoveAhead; ++k)
            if (i0 + k < n && src[i0 + k] >= 0) x[k] = *at(src[i0 + k]);
#pragma unroll
        for (int k = 0; k < kMoveAhead; ++k)
            if (i0 + k < n && src[i0 + k] >= 0) *at(dst[i0 + k]) = x[k];
    }
}

template <int D, bool FP4>
__global__ void __launch_bounds__(kMoveThreads) move_kv_kernel(const __grid_constant__ MoveParams p) {
    constexpr int kRow = FP4 ? D / 2 : D * 2;              // bytes of a key's row in a pool
    constexpr int kPieces = kRow / 16 + (FP4 ? 1 : 0);     // 16 bytes each; the scales' row is the last
    __shared__ int src[kMoveSteps], dst[kMoveSteps];
    pdl_wait_primary();
    pdl_launch_dependents();
    const int r = blockIdx.y, layer = blockIdx.z, tid = threadIdx.x;
    const int row0 = p.q_indptr[r], row1 = p.q_indptr[r + 1], len = p.seq_lens[r], n = p.accept_lens[r];
    const int w = row1 - row0, ctx = len - w;
    const int32_t* path = p.path + (long long)r * p.path_stride;
    unsigned int bad = 0;
    if (row0 < 0 || row1 < row0) bad = kDevBadWindow;
    else if (len < w || len > p.max_seq_len || len > (long long)p.bt_stride << p.page_shift) bad = kDevBadSeqLen;
    else if (n < 0 || n > p.path_stride || n > w) bad = kDevBadTree;
    bool wrong = false;
    if (!bad)
        for (int i = tid; i < n; i += kMoveThreads) {
            const int v = path[i];
            wrong |= v < 0 || v >= w || (i > 0 && v <= path[i - 1]);
        }
    if (__syncthreads_or(wrong)) bad = kDevBadTree;
    if (bad) {
        if (tid == 0 && blockIdx.x == 0 && layer == 0) atomicOr(p.status, bad);
        return;
    }
    const int unit = blockIdx.x * kMoveThreads + tid;
    const int piece = unit % kPieces, head = unit / kPieces % p.num_kv_heads, is_v = unit / kPieces / p.num_kv_heads;
    const int32_t* table = p.block_table + (long long)r * p.bt_stride;
    for (int base = 0; base < n; base += kMoveSteps) {
        const int m = min(n - base, kMoveSteps);
        __syncthreads();
        for (int i = tid; i < m; i += kMoveThreads) {
            const int from = ctx + path[base + i], to = ctx + base + i, mask = (1 << p.page_shift) - 1;
            int s = -1, t = -1;
            if (from != to) {
                const int pf = table[from >> p.page_shift], pt = table[to >> p.page_shift];
                if (pf >= 0 && pf < p.num_pages && pt >= 0 && pt < p.num_pages) {
                    s = pf << p.page_shift | (from & mask);
                    t = pt << p.page_shift | (to & mask);
                } else {
                    atomicOr(p.status, kDevBadPage);
                }
            }
            src[i] = s;
            dst[i] = t;
        }
        __syncthreads();
        if (is_v > 1) continue;
        if (!FP4 || piece < kRow / 16) {
            unsigned char* at = p.pool[is_v][layer] + (long long)head * kRow * (1 << p.page_shift) + piece * 16;
            move_column<uint4>(at, p.kv_page_stride, kRow, src, dst, m, p.page_shift);
        } else {
            constexpr int kScales = D / 16;
            unsigned char* at = p.scales[is_v][layer] + (long long)head * kScales * (1 << p.page_shift);
            if constexpr (kScales == 4) move_column<uint32_t>(at, p.scale_page_stride, kScales, src, dst, m, p.page_shift);
            else if constexpr (kScales == 8) move_column<uint2>(at, p.scale_page_stride, kScales, src, dst, m, p.page_shift);
            else move_column<uint4>(at, p.scale_page_stride, kScales, src, dst, m, p.page_shift);
        }
    }
}

template <class... Args>
cudaError_t launch(void (*kernel)(Args...), dim3 grid, int threads, size_t smem, cudaStream_t stream,
                   const Args&... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...);
}

bool aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// The limits both tree calls share, and the words of a mask row.
int check_tree(const spec_attn_tree_problem* problem, int* words) {
    if (!problem) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_tree_problem& p = *problem;
    if (p.num_reqs < 0 || p.total_rows < 0 || p.max_w < 1 || p.mask_row_words < 0 || p.window_left < 0 ||
        p.sink_keys < 0 || p.reserved != 0)
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_reqs > 65535 || p.max_w > SPEC_ATTN_TREE_MAX_W) return SPEC_ATTN_E_UNSUPPORTED;
    const int need = (p.max_w + 31) / 32;
    *words = p.mask_row_words ? p.mask_row_words : need;
    return *words < need ? SPEC_ATTN_E_INVALID_ARG : SPEC_ATTN_OK;
}

int tree_threads(int max_w) { return max_w > 256 ? 256 : (max_w + 31) / 32 * 32; }

}  // namespace
}  // namespace spec_attn

extern "C" {

int spec_attn_build_tree(const spec_attn_tree_problem* problem, const int32_t* parents, const int32_t* seq_lens,
                         const int32_t* q_indptr, int32_t* positions, int32_t* row_mask, void* workspace,
                         size_t workspace_bytes, spec_attn_stream_t stream) {
    using namespace spec_attn;
    int words = 0;
    const int st = check_tree(problem, &words);
    if (st != SPEC_ATTN_OK) return st;
    const spec_attn_tree_problem& p = *problem;
    if (!q_indptr || !workspace || (p.num_reqs > 0 && !seq_lens) ||
        (p.total_rows > 0 && (!parents || !positions || !row_mask)))
        return SPEC_ATTN_E_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(parents), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(q_indptr), static_cast<const void*>(positions),
                          static_cast<const void*>(row_mask)})
        if (!aligned(x, 4)) return SPEC_ATTN_E_INVALID_ARG;
    if (!aligned(workspace, 256)) return SPEC_ATTN_E_INVALID_ARG;
    if (workspace_bytes < 256) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    const uint64_t rows4 = 4ull * p.total_rows, reqs4 = 4ull * p.num_reqs;
    const ByteRows out[] = {bytes_at(positions, rows4), bytes_at(row_mask, rows4 * words), bytes_at(workspace, 256)};
    const ByteRows in[] = {bytes_at(parents, rows4), bytes_at(seq_lens, reqs4), bytes_at(q_indptr, reqs4 + 4)};
    if (outputs_overlap(out, in)) return SPEC_ATTN_E_INVALID_ARG;
    TreeParams t = {};
    t.parents = parents;
    t.seq_lens = seq_lens;
    t.q_indptr = q_indptr;
    t.positions = positions;
    t.row_mask = reinterpret_cast<uint32_t*>(row_mask);
    t.status = static_cast<unsigned int*>(workspace);
    t.num_reqs = p.num_reqs;
    t.total_rows = p.total_rows;
    t.max_w = p.max_w;
    t.words = words;
    t.window = p.window_left;
    t.sinks = p.sink_keys;
    t.whole = aligned(row_mask, 16);
    void (*const kernel)(const TreeParams) = p.max_w <= 128   ? &build_tree_kernel<4>
                                             : p.max_w <= 256 ? &build_tree_kernel<8>
                                                              : &build_tree_kernel<0>;
    const cudaError_t e = launch(kernel, dim3(p.num_reqs ? static_cast<unsigned>(p.num_reqs) : 1u), tree_threads(p.max_w),
                                 4 * static_cast<size_t>(p.max_w), reinterpret_cast<cudaStream_t>(stream), t);
    return e == cudaSuccess ? SPEC_ATTN_OK : record_cuda_error(e);
}

int spec_attn_accept_tree(const spec_attn_tree_problem* problem, const int32_t* parents, const int64_t* draft_tokens,
                          const int64_t* target_tokens, const int32_t* seq_lens, const int32_t* q_indptr, int32_t* path,
                          int32_t* accept_lens, int64_t* next_tokens, int32_t* ctx_lens, void* workspace,
                          size_t workspace_bytes, spec_attn_stream_t stream) {
    using namespace spec_attn;
    int words = 0;
    const int st = check_tree(problem, &words);
    if (st != SPEC_ATTN_OK) return st;
    const spec_attn_tree_problem& p = *problem;
    if (p.path_stride < 1) return SPEC_ATTN_E_INVALID_ARG;
    if (!workspace || (p.total_rows > 0 && (!parents || !draft_tokens || !target_tokens)) ||
        (p.num_reqs > 0 && (!seq_lens || !q_indptr || !path || !accept_lens || !next_tokens || !ctx_lens)))
        return SPEC_ATTN_E_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(parents), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(q_indptr), static_cast<const void*>(path),
                          static_cast<const void*>(accept_lens), static_cast<const void*>(ctx_lens)})
        if (!aligned(x, 4)) return SPEC_ATTN_E_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(draft_tokens), static_cast<const void*>(target_tokens),
                          static_cast<const void*>(next_tokens)})
        if (!aligned(x, 8)) return SPEC_ATTN_E_INVALID_ARG;
    if (!aligned(workspace, 256)) return SPEC_ATTN_E_INVALID_ARG;
    if (workspace_bytes < 256) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    if (p.num_reqs == 0) return SPEC_ATTN_OK;
    const uint64_t rows4 = 4ull * p.total_rows, reqs4 = 4ull * p.num_reqs;
    // (ctx_lens may be seq_lens, which then meets what ctx_lens meets)
    const bool in_place = ctx_lens == seq_lens;
    const ByteRows out[] = {bytes_at(path, reqs4 * p.path_stride), bytes_at(accept_lens, reqs4),
                            bytes_at(next_tokens, 2 * reqs4), bytes_at(ctx_lens, reqs4), bytes_at(workspace, 256)};
    const ByteRows in[] = {bytes_at(parents, rows4), bytes_at(draft_tokens, 2 * rows4), bytes_at(target_tokens, 2 * rows4),
                           bytes_at(seq_lens, in_place ? 0 : reqs4), bytes_at(q_indptr, reqs4 + 4)};
    if (outputs_overlap(out, in)) return SPEC_ATTN_E_INVALID_ARG;
    TreeParams t = {};
    t.parents = parents;
    t.seq_lens = seq_lens;
    t.q_indptr = q_indptr;
    t.draft = reinterpret_cast<const long long*>(draft_tokens);
    t.target = reinterpret_cast<const long long*>(target_tokens);
    t.path = path;
    t.accept_lens = accept_lens;
    t.next_tokens = reinterpret_cast<long long*>(next_tokens);
    t.ctx_lens = ctx_lens;
    t.status = static_cast<unsigned int*>(workspace);
    t.num_reqs = p.num_reqs;
    t.total_rows = p.total_rows;
    t.max_w = p.max_w;
    t.path_stride = p.path_stride;
    const cudaError_t e = launch(accept_tree_kernel, dim3(static_cast<unsigned>(p.num_reqs)), tree_threads(p.max_w),
                                 12 * static_cast<size_t>(p.max_w), reinterpret_cast<cudaStream_t>(stream), t);
    return e == cudaSuccess ? SPEC_ATTN_OK : record_cuda_error(e);
}

int spec_attn_move_kv(const spec_attn_move_problem* problem, void* const* h_k_pools, void* const* h_v_pools,
                      void* const* h_k_scales, void* const* h_v_scales, const int32_t* block_table,
                      const int32_t* seq_lens, const int32_t* q_indptr, const int32_t* path,
                      const int32_t* accept_lens, void* workspace, size_t workspace_bytes,
                      spec_attn_stream_t stream) {
    using namespace spec_attn;
    if (!problem) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_move_problem& p = *problem;
    if (p.num_reqs < 0 || p.num_layers < 0 || p.num_kv_heads < 1 || p.num_pages < 0 || p.block_table_stride < 0 ||
        p.path_stride < 1 || p.max_seq_len < 0 || p.reserved != 0 ||
        (p.kv_dtype != SPEC_ATTN_KV_BF16 && p.kv_dtype != SPEC_ATTN_KV_NVFP4))
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_reqs > 65535 || p.num_kv_heads > 65535 || p.max_seq_len > INT32_MAX ||
        (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256) ||
        (p.page_size != 16 && p.page_size != 32 && p.page_size != 64) ||
        static_cast<int64_t>(p.block_table_stride) * p.page_size > INT32_MAX ||
        static_cast<int64_t>(p.num_pages) * p.page_size > INT32_MAX)
        return SPEC_ATTN_E_UNSUPPORTED;
    const bool fp4 = p.kv_dtype == SPEC_ATTN_KV_NVFP4;
    const int64_t keys = static_cast<int64_t>(p.num_kv_heads) * p.page_size;
    const int64_t page = keys * (fp4 ? p.head_dim / 2 : p.head_dim * 2), scale_page = keys * (p.head_dim / 16);
    auto bad_stride = [](int64_t stride, int64_t dense) { return stride != 0 && (stride < dense || stride % 16 != 0); };
    if (bad_stride(p.kv_page_stride, page) || (fp4 && bad_stride(p.scale_page_stride, scale_page)))
        return SPEC_ATTN_E_INVALID_ARG;
    if (!workspace || !aligned(workspace, 256)) return SPEC_ATTN_E_INVALID_ARG;
    if (workspace_bytes < 256) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    if (p.num_reqs == 0 || p.num_layers == 0) return SPEC_ATTN_OK;
    if (!h_k_pools || !h_v_pools || (fp4 && (!h_k_scales || !h_v_scales)) || !seq_lens || !q_indptr || !path ||
        !accept_lens || (p.block_table_stride > 0 && !block_table))
        return SPEC_ATTN_E_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(q_indptr), static_cast<const void*>(path),
                          static_cast<const void*>(accept_lens)})
        if (!aligned(x, 4)) return SPEC_ATTN_E_INVALID_ARG;
    const uint64_t reqs4 = 4ull * p.num_reqs, step = static_cast<uint64_t>(p.kv_page_stride ? p.kv_page_stride : page);
    const uint64_t scale_step = static_cast<uint64_t>(p.scale_page_stride ? p.scale_page_stride : scale_page);
    const uint64_t pages = static_cast<uint64_t>(p.num_pages);
    for (int l = 0; l < p.num_layers; ++l) {
        const void* at[] = {h_k_pools[l], h_v_pools[l], fp4 ? h_k_scales[l] : nullptr, fp4 ? h_v_scales[l] : nullptr};
        for (int i = 0; i < (fp4 ? 4 : 2); ++i)
            if ((p.num_pages > 0 && !at[i]) || !aligned(at[i], 16)) return SPEC_ATTN_E_INVALID_ARG;
        const ByteRows out[] = {{at[0], static_cast<uint64_t>(page), step, pages},
                                {at[1], static_cast<uint64_t>(page), step, pages},
                                {at[2], static_cast<uint64_t>(scale_page), scale_step, pages},
                                {at[3], static_cast<uint64_t>(scale_page), scale_step, pages},
                                bytes_at(workspace, 256)};
        const ByteRows in[] = {bytes_at(block_table, reqs4 * p.block_table_stride), bytes_at(seq_lens, reqs4),
                               bytes_at(q_indptr, reqs4 + 4), bytes_at(path, reqs4 * p.path_stride),
                               bytes_at(accept_lens, reqs4)};
        if (outputs_overlap(out, in)) return SPEC_ATTN_E_INVALID_ARG;
    }
    MoveParams m = {};
    m.block_table = block_table;
    m.seq_lens = seq_lens;
    m.q_indptr = q_indptr;
    m.path = path;
    m.accept_lens = accept_lens;
    m.status = static_cast<unsigned int*>(workspace);
    m.num_kv_heads = p.num_kv_heads;
    m.page_shift = p.page_size == 64 ? 6 : p.page_size == 32 ? 5 : 4;
    m.num_pages = p.num_pages;
    m.bt_stride = p.block_table_stride;
    m.path_stride = p.path_stride;
    m.max_seq_len = p.max_seq_len;
    m.kv_page_stride = static_cast<long long>(step);
    m.scale_page_stride = static_cast<long long>(scale_step);
    void (*kernel)(const MoveParams) = nullptr;
    if (p.head_dim == 64) kernel = fp4 ? &move_kv_kernel<64, true> : &move_kv_kernel<64, false>;
    if (p.head_dim == 128) kernel = fp4 ? &move_kv_kernel<128, true> : &move_kv_kernel<128, false>;
    if (p.head_dim == 256) kernel = fp4 ? &move_kv_kernel<256, true> : &move_kv_kernel<256, false>;
    const int pieces = fp4 ? p.head_dim / 32 + 1 : p.head_dim / 8;
    const unsigned ctas = static_cast<unsigned>((2 * p.num_kv_heads * pieces + kMoveThreads - 1) / kMoveThreads);
    for (int l0 = 0; l0 < p.num_layers; l0 += kMoveLayers) {
        const int n = p.num_layers - l0 < kMoveLayers ? p.num_layers - l0 : kMoveLayers;
        for (int l = 0; l < n; ++l) {
            m.pool[0][l] = static_cast<unsigned char*>(h_k_pools[l0 + l]);
            m.pool[1][l] = static_cast<unsigned char*>(h_v_pools[l0 + l]);
            m.scales[0][l] = fp4 ? static_cast<unsigned char*>(h_k_scales[l0 + l]) : nullptr;
            m.scales[1][l] = fp4 ? static_cast<unsigned char*>(h_v_scales[l0 + l]) : nullptr;
        }
        const cudaError_t e = launch(kernel, dim3(ctas, static_cast<unsigned>(p.num_reqs), static_cast<unsigned>(n)),
                                     kMoveThreads, 0, reinterpret_cast<cudaStream_t>(stream), m);
        if (e != cudaSuccess) return record_cuda_error(e);
    }
    return SPEC_ATTN_OK;
}

}  // extern "C"
