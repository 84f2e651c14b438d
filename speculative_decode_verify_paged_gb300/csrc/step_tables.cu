// Step tables (spec_attn_build_tables): seq_lens, q_indptr, the grown block
// table, the free-page stack, and every row's position and cache slot, from
// the requests' lengths alone.  The tables restate what the page "DFlash2
// leaves the paged graph fast path at every c>1 ..." (section "Scope") has the
// attention read: one shared paged pool, a batched block table, per-request
// seq_lens and P x (1+k) query rows; the page "perf(dflash): widen the verify
// window past the compact graph's four-row limit" (section "What changed")
// gives the rule for a rejected tail: it is dropped by length alone.
//
// With held = ceil(prev / ps), need = ceil((ctx + W) / ps), new = max(0, need -
// held) and ret = max(0, held - need), three exclusive sums over the requests
// (of W, new and ret) place everything: rows, the pages requests take and the
// pages they give back.  The stack after the returns is C = S[0..F) ++ returned;
// pop k is C[F + R - 1 - k].  C need never exist: its part past F is read
// from the returning rows' own table entries, which nobody writes (a row
// either grows or shrinks), reads of S stay below F and writes of S start at F.
// So every output can be written in parallel with no order between CTAs.
//
// Work split: each CTA makes the three sums itself (the lengths are a few KB
// and come from L2) and then takes its share of rows, taken pages and returned
// pages by a binary search in its shared-memory copy.  One kernel, no
// grid-wide wait.  Rows are dealt from the first CTA on and pages from the last,
// so that the two chains of dependent loads run in different CTAs (512
// requests: 6.4 us with both in turn, 5.0 like this, 4.3 with 256 threads a CTA
// instead of 512).  A thread takes one row:
// four adjacent ones, with wider stores, are four searches in turn where
// windows are short (8.8 us).  Where seq_lens or free_count overwrite an
// input, the CTA that finishes last (a ticket in the workspace) writes them,
// after every CTA has read.
//
// Bound: the chain of dependent memory round trips (lengths, sums, table entry,
// stack entry) behind the launch, not bytes: 8 requests with 72 rows 2.7 us, 512
// requests with 512 to 4608 rows 3.4 to 4.3, 61 prompts with 262144 rows 5.1 (3.2 MB
// written); in place, with the ticket, 3.5 (8 requests) and 4.5 (512).  From some
// thousand requests on the sums themselves, which every CTA makes: 2048 requests
// 6.2 us, 4096 9.9, 16384 28.
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/spec_attn.h"
#include "common.cuh"

namespace spec_attn {
namespace {

constexpr int kTabThreads = 1024;         // at most
constexpr int kTabWarps = kTabThreads / 32;
constexpr int kTabAdjacent = 8;

struct Sums {
    long long w, n, t;   // window rows, new pages, returned pages
};

__device__ __forceinline__ Sums add(const Sums& a, const Sums& b) { return {a.w + b.w, a.n + b.n, a.t + b.t}; }

// One request, checked; a bad one counts nothing and sets bits.
struct TabReq {
    int ctx, w, held, need;
};
__device__ __forceinline__ TabReq tab_request(const TablesParams& p, int r, unsigned int& bad) {
    TabReq q;
    q.ctx = p.ctx_lens[r];
    q.w = p.window_lens[r];
    const int prev = p.prev_seq_lens[r];
    const long long cap = (long long)p.bt_stride << p.page_shift;
    const long long round = (1 << p.page_shift) - 1;
    if (q.w < 0 || q.w > p.max_w) {
        bad |= kDevBadWindow;
        q.w = 0;
    }
    const long long len = (long long)q.ctx + q.w;
    if (q.ctx < 0 || q.ctx > prev || prev > cap || len > cap || len > p.max_seq_len) {
        bad |= kDevBadSeqLen;
        q.ctx = q.w = q.held = q.need = 0;
        return q;
    }
    q.held = (int)((prev + round) >> p.page_shift);
    q.need = (int)((len + round) >> p.page_shift);
    return q;
}

// The last r in [0, n) with a[r] <= x, for x in [a[0], a[n]): the request x falls to.
__device__ __forceinline__ int owner(const int32_t* a, int n, int x) {
    int lo = 0, hi = n;   // a[lo] <= x < a[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (a[mid] <= x) lo = mid;
        else hi = mid;
    }
    return lo;
}

__global__ void __launch_bounds__(kTabThreads) tables_kernel(const TablesParams p) {
    extern __shared__ int32_t tab_smem[];
    const int P = p.num_reqs;
    int32_t* s_row = tab_smem;             // [P + 1] exclusive sums, the total last
    int32_t* s_new = s_row + P + 1;
    int32_t* s_ret = s_new + P + 1;
    __shared__ Sums s_warp[kTabWarps];
    __shared__ long long s_held[kTabWarps];
    __shared__ unsigned int s_bad[kTabWarps];
    __shared__ int s_last;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, threads = blockDim.x, warps = threads >> 5;
    pdl_wait_primary();
    pdl_launch_dependents();

    // ---- the three sums.  A thread takes `per` requests: adjacent ones, summed in its registers, or (many) every 32nd
    // of its warp's, read side by side but scanned over the warp again for each (16384 requests: 28 us, 45 with
    // adjacent ones; 512: 4.2 us adjacent, 4.9 side by side)
    const int per = (P + threads - 1) / threads;
    const bool adjacent = per <= kTabAdjacent;
    const int r0 = adjacent ? tid * per : warp * 32 * per + lane, step = adjacent ? 1 : 32;
    const int F = *p.prev_free_count;
    unsigned int bad = 0;
    auto counts = [&](int r, long long& held) -> Sums {
        if (r >= P) return {0, 0, 0};
        const TabReq q = tab_request(p, r, bad);
        held += q.held;
        return {q.w, max(0, q.need - q.held), max(0, q.held - q.need)};
    };
    auto scan = [&](const Sums& mine) {   // inclusive, over the warp
        Sums inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const Sums up = {__shfl_up_sync(kFullMask, inc.w, o), __shfl_up_sync(kFullMask, inc.n, o),
                             __shfl_up_sync(kFullMask, inc.t, o)};
            if (lane >= o) inc = add(inc, up);
        }
        return inc;
    };
    Sums mine = {0, 0, 0};
    long long held = 0;
#pragma unroll 4
    for (int k = 0; k < per; ++k) mine = add(mine, counts(r0 + step * k, held));
    const Sums inc = scan(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        held += __shfl_xor_sync(kFullMask, held, o);
        bad |= __shfl_xor_sync(kFullMask, bad, o);
    }
    if (lane == 31) {
        s_warp[warp] = inc;
        s_held[warp] = held;
        s_bad[warp] = bad;
    }
    __syncthreads();
    Sums base = {0, 0, 0}, total = {0, 0, 0};
    held = 0;
    bad = 0;
    for (int k = 0; k < warps; ++k) {
        if (k < warp) base = add(base, s_warp[k]);
        total = add(total, s_warp[k]);
        held += s_held[k];
        bad |= s_bad[k];
    }
    if (total.w > p.max_rows) bad |= kDevBadWindow;
    if (F < 0 || F + held > p.num_pages) bad |= kDevBadFreeList;
    else if (total.n > F + total.t) bad |= kDevOutOfPages;
    const bool ok = bad == 0;   // the same in every thread of every CTA
    const int R = (int)total.t, N = (int)total.n, rows = ok ? (int)total.w : 0;
    const int F2 = ok ? F + R - N : F;
    if (ok) {
        // (every sum fits 32 bits: rows <= max_rows, pages <= num_pages)
        auto put = [&](int r, const Sums& at) {
            if (r >= P) return;
            s_row[r] = (int)at.w;
            s_new[r] = (int)at.n;
            s_ret[r] = (int)at.t;
        };
        if (adjacent) {
            Sums at = add(base, {inc.w - mine.w, inc.n - mine.n, inc.t - mine.t});
            for (int k = 0; k < per; ++k) {
                put(r0 + k, at);
                if (k + 1 < per) at = add(at, counts(r0 + k, held));
            }
        } else {
            Sums at = base;
            for (int k = 0; k < per; ++k) {
                const Sums one = counts(r0 + 32 * k, held), all = scan(one);
                put(r0 + 32 * k, add(at, {all.w - one.w, all.n - one.n, all.t - one.t}));
                at = add(at, {__shfl_sync(kFullMask, all.w, 31), __shfl_sync(kFullMask, all.n, 31),
                              __shfl_sync(kFullMask, all.t, 31)});
            }
        }
        if (tid == 0) {
            s_row[P] = rows;
            s_new[P] = N;
            s_ret[P] = R;
        }
    } else if (blockIdx.x == 0 && tid == 0) {
        atomicOr(p.status, bad);
    }
    __syncthreads();

    // (unsigned: an index may pass 2^31 on its last step)
    const unsigned g0 = blockIdx.x * threads + tid, gn = gridDim.x * threads;
    // pages are dealt from the last CTA on: those there have no rows, and the two chains of loads run side by side
    const unsigned p0 = (gridDim.x - 1 - blockIdx.x) * threads + tid;
    unsigned int sick = 0;
    auto entry = [&](int r, int j) -> int32_t* { return p.block_table + (size_t)r * p.bt_stride + j; };
    auto returned = [&](int i) {   // the i-th page given back
        const int r = owner(s_ret, P, i);
        return *entry(r, tab_request(p, r, sick).need + (i - s_ret[r]));
    };
    auto taken = [&](int k) {      // the k-th page handed out
        const int c = F + R - 1 - k;
        const int page = c < F ? p.free_pages[c] : returned(c - F);
        if (page < 0 || page >= p.num_pages) sick |= kDevBadPage;
        return page;
    };

    // ---- rows: position and slot
    for (unsigned row = g0; row < (unsigned)p.max_rows; row += gn) {
        int pos = 0;
        long long slot = -1;
        if (row < (unsigned)rows) {
            const int r = owner(s_row, P, (int)row);
            const TabReq q = tab_request(p, r, sick);
            pos = q.ctx + ((int)row - s_row[r]);
            const int j = pos >> p.page_shift;
            const int page = j < q.held ? *entry(r, j) : taken(s_new[r] + (j - q.held));
            if (page < 0 || page >= p.num_pages) sick |= kDevBadPage;
            else slot = ((long long)page << p.page_shift) + (pos & ((1 << p.page_shift) - 1));
        }
        p.positions[row] = pos;
        p.slot_map[row] = slot;
    }
    if (ok) {
        // ---- pages handed out, and what is left of the returned ones on the stack
        for (unsigned k = p0; k < (unsigned)N; k += gn) {
            const int r = owner(s_new, P, (int)k);
            *entry(r, tab_request(p, r, sick).held + ((int)k - s_new[r])) = taken((int)k);
        }
        for (unsigned i = p0; i < (unsigned)max(0, F2 - F); i += gn) {
            const int page = returned((int)i);
            if (page < 0 || page >= p.num_pages) sick |= kDevBadPage;
            p.free_pages[F + i] = page;
        }
    }
    for (unsigned r = g0; r <= (unsigned)P; r += gn) p.q_indptr[r] = ok ? s_row[r] : 0;
    if (sick) atomicOr(p.status, sick);

    // ---- the state that may overwrite an input
    bool last = true;
    if (p.in_place) {
        __syncthreads();
        if (tid == 0) {
            __threadfence();
            s_last = atomicAdd(p.status + 1, 1u) == gridDim.x - 1;
            if (s_last) p.status[1] = 0;
        }
        __syncthreads();
        last = s_last != 0;
    }
    if (last) {
        const unsigned first = p.in_place ? tid : g0, stride = p.in_place ? threads : gn;
        for (unsigned r = first; r < (unsigned)P; r += stride)
            p.seq_lens[r] = ok ? p.ctx_lens[r] + p.window_lens[r] : p.prev_seq_lens[r];
        if (first == 0) *p.free_count = F2;
    }
}

// The three sums of each request, and their totals.
constexpr size_t tab_smem_bytes(int reqs) { return 3 * (static_cast<size_t>(reqs) + 1) * sizeof(int32_t); }
static_assert(tab_smem_bytes(SPEC_ATTN_TABLES_MAX_REQS) + 4096 <= 232448, "shared memory of a CTA, static part included");

}  // namespace

cudaError_t tables_launch(const TablesParams& p, cudaStream_t stream) {
    const size_t smem = tab_smem_bytes(p.num_reqs);
    if (smem > 46 * 1024) {   // (2 KB are static)
        // The limit belongs to the kernel, not to this launch: one constant for every size, so that no call lowers it
        // under another thread's launch or under a node of a graph.
        const cudaError_t e = cudaFuncSetAttribute(tables_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   static_cast<int>(tab_smem_bytes(SPEC_ATTN_TABLES_MAX_REQS)));
        if (e != cudaSuccess) return e;
    }
    // (each CTA sums all requests: more threads for many, less to synchronise for few)
    const int threads = p.num_reqs <= 256 * kTabAdjacent ? 256 : kTabThreads;
    // a thread a row and one for each page that the rows may take, as many as the 152 SMs hold
    const long long pages = (p.max_rows >> p.page_shift) + (long long)p.num_reqs + 1;
    const long long ctas = ((long long)p.max_rows + threads - 1) / threads + (pages + threads - 1) / threads;
    const long long most = 152 * 1024 / threads;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(ctas < most ? ctas : most));
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tables_kernel, p);
}

}  // namespace spec_attn

namespace {

bool tab_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// [a, a + na) and [b, b + nb) bytes overlap
bool overlap(const void* a, size_t na, const void* b, size_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return na && nb && x < y + nb && y < x + na;
}

}  // namespace

extern "C" int spec_attn_build_tables(const spec_attn_tables_problem* problem, const int32_t* ctx_lens,
                                      const int32_t* window_lens, const int32_t* prev_seq_lens,
                                      const int32_t* prev_free_count, int32_t* free_pages, int32_t* block_table,
                                      int32_t* seq_lens, int32_t* q_indptr, int32_t* free_count, int32_t* positions,
                                      int64_t* slot_map, void* workspace, size_t workspace_bytes,
                                      spec_attn_stream_t stream) {
    using namespace spec_attn;
    if (!problem) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_tables_problem& p = *problem;
    if (p.num_reqs < 0 || p.max_rows < 0 || p.num_pages < 0 || p.block_table_stride < 0 || p.max_w < 1 ||
        p.max_seq_len < 0)
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_reqs > SPEC_ATTN_TABLES_MAX_REQS || p.max_seq_len > INT32_MAX) return SPEC_ATTN_E_UNSUPPORTED;
    if (p.page_size != 16 && p.page_size != 32 && p.page_size != 64) return SPEC_ATTN_E_UNSUPPORTED;
    if (static_cast<int64_t>(p.block_table_stride) * p.page_size > INT32_MAX) return SPEC_ATTN_E_UNSUPPORTED;
    if (!prev_free_count || !q_indptr || !free_count || !workspace) return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_reqs > 0 && (!ctx_lens || !window_lens || !prev_seq_lens || !seq_lens)) return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_reqs > 0 && p.block_table_stride > 0 && !block_table) return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_pages > 0 && !free_pages) return SPEC_ATTN_E_INVALID_ARG;
    if (p.max_rows > 0 && (!positions || !slot_map)) return SPEC_ATTN_E_INVALID_ARG;
    for (const void* q : {static_cast<const void*>(ctx_lens), static_cast<const void*>(window_lens),
                          static_cast<const void*>(prev_seq_lens), static_cast<const void*>(prev_free_count),
                          static_cast<const void*>(free_pages), static_cast<const void*>(block_table),
                          static_cast<const void*>(seq_lens), static_cast<const void*>(q_indptr),
                          static_cast<const void*>(free_count), static_cast<const void*>(positions)})
        if (!tab_aligned(q, 4)) return SPEC_ATTN_E_INVALID_ARG;
    if (!tab_aligned(slot_map, 8) || !tab_aligned(workspace, 256)) return SPEC_ATTN_E_INVALID_ARG;
    if (workspace_bytes < 256) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    // outputs: seq_lens may be an input length array and free_count its input; nothing else overlaps
    const size_t P4 = 4 * static_cast<size_t>(p.num_reqs);
    struct Range { const void* p; size_t n; };
    const Range in[] = {{ctx_lens, P4}, {window_lens, P4}, {prev_seq_lens, P4}, {prev_free_count, 4}};
    const Range out[] = {{free_pages, 4 * static_cast<size_t>(p.num_pages)},
                         {block_table, P4 * static_cast<size_t>(p.block_table_stride)},
                         {seq_lens, P4}, {q_indptr, P4 + 4}, {free_count, 4},
                         {positions, 4 * static_cast<size_t>(p.max_rows)},
                         {slot_map, 8 * static_cast<size_t>(p.max_rows)}, {workspace, 256}};
    for (size_t i = 0; i < sizeof(out) / sizeof(out[0]); ++i) {
        for (size_t j = 0; j < i; ++j)
            if (overlap(out[i].p, out[i].n, out[j].p, out[j].n)) return SPEC_ATTN_E_INVALID_ARG;
        for (const Range& r : in) {
            const bool same = (out[i].p == seq_lens && (r.p == prev_seq_lens || r.p == ctx_lens) && r.p == seq_lens) ||
                              (out[i].p == free_count && r.p == prev_free_count && r.p == free_count);
            if (!same && overlap(out[i].p, out[i].n, r.p, r.n)) return SPEC_ATTN_E_INVALID_ARG;
        }
    }
    TablesParams t = {};
    t.ctx_lens = ctx_lens;
    t.window_lens = window_lens;
    t.prev_seq_lens = prev_seq_lens;
    t.prev_free_count = prev_free_count;
    t.free_pages = free_pages;
    t.block_table = block_table;
    t.seq_lens = seq_lens;
    t.q_indptr = q_indptr;
    t.free_count = free_count;
    t.positions = positions;
    t.slot_map = reinterpret_cast<long long*>(slot_map);
    t.status = static_cast<unsigned int*>(workspace);
    t.num_reqs = p.num_reqs;
    t.max_rows = p.max_rows;
    t.page_shift = p.page_size == 64 ? 6 : p.page_size == 32 ? 5 : 4;
    t.num_pages = p.num_pages;
    t.bt_stride = p.block_table_stride;
    t.max_w = p.max_w;
    t.max_seq_len = p.max_seq_len;
    t.in_place = seq_lens == prev_seq_lens || seq_lens == ctx_lens || free_count == prev_free_count;
    const cudaError_t e = tables_launch(t, reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_ATTN_OK : record_cuda_error(e);
}
