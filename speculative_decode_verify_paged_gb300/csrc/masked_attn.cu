// Attention over the paged cache under tree masks and under a sliding window with
// sinks (spec_attn_run_masked), windows of any width.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>

#include "../../include/spec_attn.h"
#include "common.cuh"
#include "overlap.h"

namespace spec_attn {
namespace {

struct MaskedParams {
    const uint16_t* q;
    const unsigned char* k_pool;
    const unsigned char* v_pool;
    const uint8_t* k_scales;
    const uint8_t* v_scales;
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* q_indptr;
    const uint32_t* row_mask;   // trees
    const int32_t* positions;   // trees with a window
    uint16_t* o;
    float* lse;
    unsigned int* status;
    int num_reqs, total_rows, max_w, num_q_heads, num_kv_heads, group;
    int page_shift;             // log2(page_size)
    int num_pages, bt_stride, tree, window, sinks, mask_words;
    long long max_seq_len, kv_page_stride, scale_page_stride;
    float score_scale_log2;     // sm_scale * log2(e) [* k_gscale]
    float out_scale;            // 1 or v_gscale
};

// A warp for each (window row, query head): the row's keys one after another.
template <int D, bool FP4>
__global__ void __launch_bounds__(128) masked_attn_kernel(const MaskedParams p) {
    constexpr int E = D / 32;   // elements a lane
    pdl_wait_primary();
    pdl_launch_dependents();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int m = blockIdx.x * 4 + warp, kvh = blockIdx.y, r = blockIdx.z;
    ReqInfo ri;
    if (!load_request(p.seq_lens, p.q_indptr, r, p.max_w, p.total_rows, p.max_seq_len, p.bt_stride << p.page_shift, 64,
                      threadIdx.x == 0 && blockIdx.x == 0 && kvh == 0 ? p.status : nullptr, ri))
        return;
    const int i = m / p.group;
    if (i >= ri.w) return;
    const size_t at = (size_t)(ri.row0 + i) * p.num_q_heads + kvh * p.group + m % p.group;
    float q[E], acc[E];
    for (int e = 0; e < E; ++e) {
        q[e] = bf16_bits_to_float(p.q[at * D + lane * E + e]);
        acc[e] = 0.f;
    }
    int pos = ri.ctx + i;
    if (p.tree) pos = p.window ? max(ri.ctx, p.positions[ri.row0 + i]) : ri.ctx;
    // first key of the window, beside the sinks (a tree's own keys are the mask's alone)
    int first = p.window ? max(0, pos - p.window + 1) : 0;
    if (p.tree) first = min(first, ri.ctx);
    const int end = p.tree ? ri.len : pos + 1;
    float mx = -INFINITY, l = 0.f;
    auto value = [&](const unsigned char* pool, const uint8_t* scales, int page, int slot, int e) {
        const size_t row = (size_t)kvh << p.page_shift | slot;
        if (!FP4) return bf16_bits_to_float(reinterpret_cast<const uint16_t*>(pool + page * p.kv_page_stride)[row * D + e]);
        const uint32_t c = (pool + page * p.kv_page_stride)[row * (D / 2) + e / 2];
        return e2m1_to_float(e & 1 ? c >> 4 : c & 15) *
               e4m3_to_float((scales + page * p.scale_page_stride)[row * (D / 16) + e / 16]);
    };
    for (int j = 0; j < end; ++j) {
        if (j >= p.sinks && j < first) {
            j = first;
            if (j >= end) break;
        }
        if (p.tree && j >= ri.ctx) {
            const int b = j - ri.ctx;
            if (!(p.row_mask[(size_t)(ri.row0 + i) * p.mask_words + (b >> 5)] >> (b & 31) & 1)) continue;
        }
        int page = p.block_table[(size_t)r * p.bt_stride + (j >> p.page_shift)];
        if (page < 0 || page >= p.num_pages) {
            if (lane == 0) atomicOr(p.status, kDevBadPage);
            page = 0;
        }
        const int slot = j & ((1 << p.page_shift) - 1);
        float s = 0.f;
        for (int e = 0; e < E; ++e) s = fmaf(q[e], value(p.k_pool, p.k_scales, page, slot, lane * E + e), s);
        for (int o = 16; o; o >>= 1) s += __shfl_xor_sync(kFullMask, s, o);
        s *= p.score_scale_log2;
        const float mn = fmaxf(mx, s), ref = fabsf(mn) == INFINITY ? 0.f : mn;
        const float a = mn > mx ? exp2f(mx - ref) : 1.f, w = exp2f(s - ref);
        mx = mn;
        l = l * a + w;
        for (int e = 0; e < E; ++e)
            acc[e] = fmaf(w, value(p.v_pool, p.v_scales, page, slot, lane * E + e), acc[e] * a);
    }
    const float inv = l == 0.f ? 0.f : p.out_scale / l;
    for (int e = 0; e < E; ++e) p.o[at * D + lane * E + e] = float_to_bf16_bits(acc[e] * inv);
    if (p.lse && lane == 0) p.lse[at] = (mx + log2f(l)) * kLn2;
}

bool masked_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace spec_attn

struct spec_attn_masked_plan {
    spec_attn_masked_problem prob;
    int device;
    float sm_scale;
};

extern "C" {

int spec_attn_masked_plan_create(const spec_attn_masked_problem* problem, spec_attn_masked_plan** out,
                                 size_t* workspace_bytes) {
    if (!out) return SPEC_ATTN_E_INVALID_ARG;
    *out = nullptr;
    if (!problem) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_masked_problem& p = *problem;
    if (p.num_reqs < 0 || p.total_q_rows < 0 || p.max_w < 1 || p.num_q_heads <= 0 || p.num_kv_heads <= 0 ||
        p.num_q_heads % p.num_kv_heads != 0 || p.head_dim <= 0 || p.page_size <= 0 || p.num_pages < 0 ||
        (p.num_reqs > 0 && p.num_pages < 1) || p.block_table_stride < 0 || p.force_splits < 0 || p.window_left < 0 ||
        p.sink_keys < 0 || p.mask_row_words < 0 || p.max_seq_len < 0 || (p.tree != 0 && p.tree != 1) ||
        (p.kv_dtype != SPEC_ATTN_KV_BF16 && p.kv_dtype != SPEC_ATTN_KV_NVFP4) || !(p.sm_scale >= 0.f) ||
        std::isinf(p.sm_scale))
        return SPEC_ATTN_E_INVALID_ARG;
    if ((p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256) ||
        (p.page_size != 16 && p.page_size != 32 && p.page_size != 64) ||
        p.num_q_heads / p.num_kv_heads > SPEC_ATTN_MAX_GROUP || p.num_reqs > 65535 || p.num_kv_heads > 65535 ||
        p.total_q_rows > (1 << 30) || p.max_seq_len > INT32_MAX ||
        static_cast<int64_t>(p.block_table_stride) * p.page_size > INT32_MAX ||
        static_cast<int64_t>(p.num_pages) * p.page_size > INT32_MAX)
        return SPEC_ATTN_E_UNSUPPORTED;
    const int words = static_cast<int>((static_cast<int64_t>(p.max_w) + 31) / 32);
    if (p.tree && p.mask_row_words != 0 && p.mask_row_words < words) return SPEC_ATTN_E_INVALID_ARG;
    const bool fp4 = p.kv_dtype == SPEC_ATTN_KV_NVFP4;
    const int64_t keys = static_cast<int64_t>(p.num_kv_heads) * p.page_size;
    const int64_t page = keys * (fp4 ? p.head_dim / 2 : p.head_dim * 2), scale_page = keys * (p.head_dim / 16);
    auto bad_stride = [](int64_t stride, int64_t dense) { return stride != 0 && (stride < dense || stride % 16 != 0); };
    if (bad_stride(p.kv_page_stride, page) || (fp4 && bad_stride(p.scale_page_stride, scale_page)))
        return SPEC_ATTN_E_INVALID_ARG;
    int dev = 0;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return spec_attn::record_cuda_error(e);
    spec_attn_masked_plan* plan = new (std::nothrow) spec_attn_masked_plan();
    if (!plan) return SPEC_ATTN_E_INVALID_ARG;
    plan->prob = p;
    if (p.kv_page_stride == 0) plan->prob.kv_page_stride = page;
    if (p.scale_page_stride == 0) plan->prob.scale_page_stride = scale_page;
    if (p.mask_row_words == 0) plan->prob.mask_row_words = words;
    plan->device = dev;
    plan->sm_scale = p.sm_scale > 0.f ? p.sm_scale : 1.0f / std::sqrt(static_cast<float>(p.head_dim));
    if (workspace_bytes) *workspace_bytes = 256;
    *out = plan;
    return SPEC_ATTN_OK;
}

int spec_attn_masked_plan_destroy(spec_attn_masked_plan* plan) {
    delete plan;
    return SPEC_ATTN_OK;
}

int spec_attn_run_masked(const spec_attn_masked_plan* plan, const void* q, const void* k_pool, const void* v_pool,
                         const void* k_scales, const void* v_scales, float k_gscale, float v_gscale,
                         const int32_t* block_table, const int32_t* seq_lens, const int32_t* q_indptr,
                         const int32_t* row_mask, const int32_t* positions, void* o, float* lse, void* workspace,
                         size_t workspace_bytes, spec_attn_stream_t stream) {
    using namespace spec_attn;
    if (!plan) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_masked_problem& p = plan->prob;
    const bool fp4 = p.kv_dtype == SPEC_ATTN_KV_NVFP4;
    if (!workspace || !masked_aligned(workspace, 256)) return SPEC_ATTN_E_INVALID_ARG;
    if (workspace_bytes < 256) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    if (p.num_reqs == 0 || p.total_q_rows == 0) return SPEC_ATTN_OK;
    if (!q || !o || !k_pool || !v_pool || (fp4 && (!k_scales || !v_scales)) || !seq_lens || !q_indptr ||
        (p.block_table_stride > 0 && !block_table) || (p.tree && !row_mask) || (p.tree && p.window_left > 0 && !positions))
        return SPEC_ATTN_E_INVALID_ARG;
    for (const void* x : {q, k_pool, v_pool, static_cast<const void*>(o), fp4 ? k_scales : nullptr, fp4 ? v_scales : nullptr})
        if (!masked_aligned(x, 16)) return SPEC_ATTN_E_INVALID_ARG;
    for (const void* x : {static_cast<const void*>(block_table), static_cast<const void*>(seq_lens),
                          static_cast<const void*>(q_indptr), static_cast<const void*>(row_mask),
                          static_cast<const void*>(positions), static_cast<const void*>(lse)})
        if (!masked_aligned(x, 4)) return SPEC_ATTN_E_INVALID_ARG;
    const uint64_t rows = static_cast<uint64_t>(p.total_q_rows), heads = rows * p.num_q_heads, reqs4 = 4ull * p.num_reqs;
    const uint64_t keys = static_cast<uint64_t>(p.num_kv_heads) * p.page_size, pages = static_cast<uint64_t>(p.num_pages);
    const uint64_t page = keys * (fp4 ? p.head_dim / 2 : p.head_dim * 2), scale_page = fp4 ? keys * (p.head_dim / 16) : 0;
    const uint64_t step = static_cast<uint64_t>(p.kv_page_stride), scale_step = static_cast<uint64_t>(p.scale_page_stride);
    const ByteRows out[] = {bytes_at(o, 2 * heads * p.head_dim), bytes_at(lse, 4 * heads), bytes_at(workspace, 256)};
    const ByteRows in[] = {bytes_at(q, 2 * heads * p.head_dim), {k_pool, page, step, pages}, {v_pool, page, step, pages},
                           {k_scales, scale_page, scale_step, pages}, {v_scales, scale_page, scale_step, pages},
                           bytes_at(block_table, reqs4 * p.block_table_stride), bytes_at(seq_lens, reqs4),
                           bytes_at(q_indptr, reqs4 + 4), bytes_at(row_mask, p.tree ? 4 * rows * p.mask_row_words : 0),
                           bytes_at(positions, p.tree && p.window_left ? 4 * rows : 0)};
    if (outputs_overlap(out, in)) return SPEC_ATTN_E_INVALID_ARG;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record_cuda_error(e);
    if (dev != plan->device) return SPEC_ATTN_E_INVALID_ARG;

    MaskedParams m = {};
    m.q = static_cast<const uint16_t*>(q);
    m.k_pool = static_cast<const unsigned char*>(k_pool);
    m.v_pool = static_cast<const unsigned char*>(v_pool);
    m.k_scales = static_cast<const uint8_t*>(k_scales);
    m.v_scales = static_cast<const uint8_t*>(v_scales);
    m.block_table = block_table;
    m.seq_lens = seq_lens;
    m.q_indptr = q_indptr;
    m.row_mask = reinterpret_cast<const uint32_t*>(row_mask);
    m.positions = positions;
    m.o = static_cast<uint16_t*>(o);
    m.lse = lse;
    m.status = static_cast<unsigned int*>(workspace);
    m.num_reqs = p.num_reqs;
    m.total_rows = p.total_q_rows;
    m.max_w = p.max_w;
    m.num_q_heads = p.num_q_heads;
    m.num_kv_heads = p.num_kv_heads;
    m.group = p.num_q_heads / p.num_kv_heads;
    m.page_shift = p.page_size == 64 ? 6 : p.page_size == 32 ? 5 : 4;
    m.num_pages = p.num_pages;
    m.bt_stride = p.block_table_stride;
    m.tree = p.tree;
    m.window = p.window_left;
    m.sinks = p.sink_keys;
    m.mask_words = p.mask_row_words;
    m.max_seq_len = p.max_seq_len;
    m.kv_page_stride = p.kv_page_stride;
    m.scale_page_stride = p.scale_page_stride;
    m.score_scale_log2 = plan->sm_scale * 1.4426950408889634f * (fp4 ? k_gscale : 1.f);
    m.out_scale = fp4 ? v_gscale : 1.f;
    void (*kernel)(const MaskedParams) = nullptr;
    if (p.head_dim == 64) kernel = fp4 ? &masked_attn_kernel<64, true> : &masked_attn_kernel<64, false>;
    if (p.head_dim == 128) kernel = fp4 ? &masked_attn_kernel<128, true> : &masked_attn_kernel<128, false>;
    if (p.head_dim == 256) kernel = fp4 ? &masked_attn_kernel<256, true> : &masked_attn_kernel<256, false>;
    const int64_t per_req = static_cast<int64_t>(std::min(p.max_w, p.total_q_rows)) * m.group;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>((per_req + 3) / 4), static_cast<unsigned>(p.num_kv_heads),
                       static_cast<unsigned>(p.num_reqs));
    cfg.blockDim = dim3(128);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, m);
    return e == cudaSuccess ? SPEC_ATTN_OK : record_cuda_error(e);
}

}  // extern "C"
