// Norm and rotation of q and k in one pass (spec_attn_norm_rope), and the same
// pass writing K and V into the paged cache (spec_attn_norm_rope_append): what
// a verify layer does between its projections and the attention.  The cache
// side restates the page "perf(dflash): widen the verify window past the
// compact graph's four-row limit", section "What changed": the window's rows
// go into the cache before it attends.
//
//   y_e = x_e w_e / sqrt(mean x^2 + eps);  (a, b) -> (a cos t - b sin t, a sin t + b cos t)
//
// fp32 throughout, one rounding to bf16 at the end (for an NVFP4 cache K is
// quantised from that bf16 value, so that the cache bytes do not depend on
// whether this kernel or spec_attn_append_kv wrote them).
//
// Angles.  t / 2 pi = position x f with f turns per position.  The plan holds
// frac(f) as a 64-bit fixed-point fraction, and its product with the position
// modulo 2^64 is the angle modulo one turn, exact for every 32-bit position
// (the fraction itself is within 2^-53 f of the double it came from).  As a
// signed fraction it is rounded once to fp32, for sincospi.
//
// Layout.  A head of d elements is taken by d / 16 adjacent lanes, 16 elements
// each in two 16-byte pieces: with half-split pairs the pieces at l and l +
// rot / 16, so that a rotation needs no exchange between lanes; otherwise
// pieces 2 l and 2 l + 1.  A warp iteration is 512 elements: 2, 4 or 8 heads.  A
// warp takes one row (or a segment of its heads): its lanes compute the row's
// cos and sin once, two or four pairs each, and share them through shared
// memory; every lane then keeps its 8 pairs in registers over the row's heads,
// and its weights for the whole launch.
//
// Loads run kAhead iterations ahead of the arithmetic, across heads, kinds and
// rows, as asynchronous copies of whole 1 KB iterations into a ring of the
// warp's own.  Where a lane's two pieces are not 128-byte runs across lanes
// (interleaved pairs, heads rotated in part), the results go back to the slot
// and leave in the order of memory: 16-byte stores 32 bytes apart cost twice the
// L2 requests.  The next row's positions and slot are asked for a row ahead.  (With the loads in registers, two or four
// heads at a time, each warp waited out a memory round trip a batch: 16384 rows
// x 40 heads x 128 took 58.7 us, 8192 x 32 x 256 into the cache 52.7 us.)
// CTAs stay resident and step over the rows, so the frequencies are copied from
// the kernel parameters to shared memory once per CTA, before the programmatic
// wait.
//
// Bound: HBM (2 bytes read and 2 written an element) for long inputs; launch
// and two dependent memory round trips for a window.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/spec_attn.h"
#include "common.cuh"
#include "nvfp4_quant.cuh"
#include "sm100.cuh"

namespace spec_attn {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;
constexpr int kAhead = 8;               // warp iterations whose loads are in flight (a power of two)
constexpr int kResident = 2;            // CTAs an SM holds (128 registers a thread)

// 16 bytes into shared memory, not through L1 (in place, this kernel writes what it reads).
__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&x)[16], int at) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[at + 2 * i] = __uint_as_float(w[i] << 16);
        x[at + 2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

__device__ __forceinline__ uint4 pack8(const float (&x)[16], int at) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[at + 2 * i], x[at + 2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

struct NrShared {
    uint4 ring[kNrWarps][kAhead][64];              // [iteration]: 512 elements of adjacent heads, in order
    unsigned long long turns[kMaxPairs];
    float cs[kNrWarps][2][kMaxPairs];              // cos and sin of the warp's row
    uint8_t axis[kMaxPairs];
};

enum Kind { kQ = 0, kK = 1, kV = 2 };

template <int D, bool APPEND, bool FP4>
struct Row {
    static constexpr int kLanes = D / 16;          // lanes of a head
    static constexpr int kHeads = 32 / kLanes;     // heads of a warp iteration

    const NormRopeParams& p;
    NrShared& sh;
    int warp, lane, l, sub;                        // l: lane within the head; sub: head within the iteration
    int ea, eb;                                    // first elements of the two pieces
    bool turn;                                     // this lane's pairs rotate
    bool relay;                                    // results leave through the ring
    float qw[16], kw[16];
    float c[8], s[8];
    int row;
    long long slot;
    int pos[kMaxPairs / 32];                       // of the row to come, this lane's pairs
    long long next_slot;

    // head of the iteration's 16-byte piece lane + 32 j, in memory order
    __device__ __forceinline__ int head_of(int it, int j) const {
        return it * kHeads + j * (kHeads / 2) + lane / (D / 8);
    }

    // ---- loads: the warp's items from `item` on, iteration by iteration
    unsigned items, step, item;                    // item: (row, segment)
    int load_row, load_it, load_end;               // of the item being loaded
    unsigned loads, uses;                          // iterations asked for and used so far

    __device__ __forceinline__ void split(unsigned i, int& r, int& it0, int& it1) const {
        if (p.segs == 1) {
            r = (int)i;
            it0 = 0;
            it1 = p.iters_q + p.iters_k + p.iters_v;
        } else {
            r = (int)(i / (unsigned)p.segs);
            it0 = (int)(i % (unsigned)p.segs) * p.iters_per_seg;
            it1 = min(it0 + p.iters_per_seg, p.iters_q + p.iters_k + p.iters_v);
        }
    }
    __device__ __forceinline__ void load_next() {
        if (item < items) {
            const int it = load_it;
            const bool is_q = it < p.iters_q, is_k = it < p.iters_q + p.iters_k;
            const int i = is_q ? it : is_k ? it - p.iters_q : it - p.iters_q - p.iters_k;   // of its kind
            const int H = is_q ? p.num_q_heads : p.num_kv_heads;
            const uint16_t* src = is_q ? p.q : is_k ? p.k : p.v;
            src += (size_t)load_row * (is_q ? p.q_row_stride : is_k ? p.k_row_stride : p.v_row_stride) + i * 512;
            const uint32_t dst = sm100::smem_addr(sh.ring[warp][loads % kAhead]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (head_of(i, j) < H) copy16(dst + (lane + 32 * j) * 16, src + (lane + 32 * j) * 8);
            ++loads;
            if (++load_it == load_end) {
                item += step;
                if (item < items) split(item, load_row, load_it, load_end);
            }
        }
        copies_commit();                           // (one group a call, empty ones too)
    }

    // ---- a row's positions and slot, asked for a row ahead
    __device__ __forceinline__ void ask(unsigned i) {
        if (i >= items) return;
        int r, it0, it1;
        split(i, r, it0, it1);
        if (APPEND) next_slot = p.slot_map[r];
#pragma unroll
        for (int k = 0; k < kMaxPairs / 32; ++k) {
            const int j = lane + 32 * k;
            if (j < p.rot_dim / 2) pos[k] = p.positions[(size_t)sh.axis[j] * p.pos_stride + r];
        }
    }
    __device__ __forceinline__ void take() {
        slot = next_slot;
        float* cs = sh.cs[warp][0];
        __syncwarp();
#pragma unroll
        for (int k = 0; k < kMaxPairs / 32; ++k) {
            const int j = lane + 32 * k;
            if (j < p.rot_dim / 2) {
                // the angle in turns, modulo one: -1/2 .. 1/2
                const unsigned long long u = sh.turns[j] * (unsigned long long)(long long)pos[k];
                float sn, cn;
                sincospif((float)(long long)u * 1.0842021724855044e-19f, &sn, &cn);   // 2^-63: in half turns
                cs[j] = cn * p.rot_scale;
                cs[kMaxPairs + j] = sn * p.rot_scale;
            }
        }
        __syncwarp();
        if (turn) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const float4 cv = *reinterpret_cast<const float4*>(cs + 8 * l + 4 * i);
                const float4 sv = *reinterpret_cast<const float4*>(cs + kMaxPairs + 8 * l + 4 * i);
                c[4 * i] = cv.x; c[4 * i + 1] = cv.y; c[4 * i + 2] = cv.z; c[4 * i + 3] = cv.w;
                s[4 * i] = sv.x; s[4 * i + 1] = sv.y; s[4 * i + 2] = sv.z; s[4 * i + 3] = sv.w;
            }
        }
    }

    __device__ __forceinline__ void rotate(float& a, float& b, int j) const {
        const float t = a;
        a = t * c[j] - b * s[j];
        b = t * s[j] + b * c[j];
    }

    // Warp iterations [it0, it1) of one kind; a row that is skipped is only drained from the ring.
    template <int KIND>
    __device__ __forceinline__ void heads(int it0, int it1, bool skip) {
        const int H = KIND == kQ ? p.num_q_heads : p.num_kv_heads;
        const bool norm = KIND == kQ ? p.q_weight != nullptr : p.k_weight != nullptr;
        // (V is copied: whichever pieces; an NVFP4 block is the pieces 2 l and 2 l + 1)
        const int a = KIND == kV ? 16 * l : ea, b = KIND == kV ? 16 * l + 8 : eb;
#pragma unroll 1
        for (int it = it0; it < it1; ++it) {
            copies_wait<kAhead - 1>();
            __syncwarp();                          // every lane's copies are in
            uint4* ring = sh.ring[warp][uses % kAhead];
            ++uses;
            const int pa = (sub * D + a) / 8, pb = (sub * D + b) / 8;
            uint4 va = ring[pa], vb = ring[pb];
            if (skip) {                            // uniform over the warp
                __syncwarp();
                load_next();
                continue;
            }
            const int h = it * kHeads + sub;
            if (KIND != kV) {
                float x[16];
                unpack8(va, x, 0);
                unpack8(vb, x, 8);
                if (norm) {
                    float ss = 0.f;
#pragma unroll
                    for (int e = 0; e < 16; ++e) ss = fmaf(x[e], x[e], ss);
#pragma unroll
                    for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
                    const float r = rsqrtf(ss * (1.0f / D) + p.eps);
#pragma unroll
                    for (int e = 0; e < 16; ++e) x[e] *= r * (KIND == kQ ? qw[e] : kw[e]);
                }
                if (turn) {
                    if (p.interleaved) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) rotate(x[2 * j], x[2 * j + 1], j);
                    } else {
#pragma unroll
                        for (int j = 0; j < 8; ++j) rotate(x[j], x[8 + j], j);
                    }
                }
                va = pack8(x, 0);
                vb = pack8(x, 8);
            }
            if (KIND == kV ? !FP4 : relay || (APPEND && FP4 && KIND == kK)) {
                if (KIND != kV) {
                    ring[pa] = va;
                    ring[pb] = vb;
                    __syncwarp();
                }
                if (!(FP4 && KIND == kK)) {        // pieces lane and lane + 32, in the order of memory
                    va = ring[lane];
                    vb = ring[lane + 32];
                } else {                           // whole blocks of 16
                    va = ring[(sub * D + 16 * l) / 8];
                    vb = ring[(sub * D + 16 * l) / 8 + 1];
                }
            }
            __syncwarp();                          // the slot is free
            load_next();
            // (in_order: the lane holds pieces lane and lane + 32, else its own two of head h)
            const bool in_order = KIND == kV || relay;
            if constexpr (KIND == kQ || !APPEND) {
                uint16_t* dst = KIND == kQ ? p.q_out + (size_t)row * p.q_out_row_stride
                                           : p.k_out + (size_t)row * p.k_out_row_stride;
                if (in_order) {
                    dst += it * 512;
                    if (head_of(it, 0) < H) sm100::st_global_v4(dst + lane * 8, va);
                    if (head_of(it, 1) < H) sm100::st_global_v4(dst + (lane + 32) * 8, vb);
                } else if (h < H) {
                    sm100::st_global_v4(dst + (size_t)h * D + a, va);
                    sm100::st_global_v4(dst + (size_t)h * D + b, vb);
                }
            } else {
                // row `at` of the page, for the slot's place in head g
                const long long page = slot >> p.page_shift;
                const int in_page = (int)(slot & ((1 << p.page_shift) - 1));
                auto at = [&](int g) { return ((size_t)g << p.page_shift) + in_page; };
                unsigned char* pool = (KIND == kK ? p.k_pool : p.v_pool) + page * p.kv_page_stride;
                if constexpr (!FP4) {
                    if (in_order) {
                        const int e = lane % (D / 8) * 16;      // bytes into the head's row
                        const int g0 = head_of(it, 0), g1 = head_of(it, 1);
                        if (g0 < H) sm100::st_global_v4(pool + at(g0) * (2 * D) + e, va);
                        if (g1 < H) sm100::st_global_v4(pool + at(g1) * (2 * D) + e, vb);
                    } else if (h < H) {
                        sm100::st_global_v4(pool + at(h) * (2 * D) + 2 * a, va);
                        sm100::st_global_v4(pool + at(h) * (2 * D) + 2 * b, vb);
                    }
                } else if (h < H) {
                    uint32_t c0, c1, sb;
                    nvfp4_block(va, vb, KIND == kK ? p.k_gscale : p.v_gscale, c0, c1, sb);
                    st_global_v2(pool + at(h) * (D / 2) + l * 8, c0, c1);
                    uint8_t* sc = (KIND == kK ? p.k_scales : p.v_scales) + page * p.scale_page_stride;
                    sc[at(h) * (D / 16) + l] = static_cast<uint8_t>(sb);
                }
            }
        }
    }
};

__device__ __forceinline__ void load_weights(const float* w, int a, int b, float (&out)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float4 f = make_float4(1.f, 1.f, 1.f, 1.f);
        if (w) f = __ldg(reinterpret_cast<const float4*>(w + (i < 2 ? a : b)) + (i & 1));
        out[4 * i] = f.x; out[4 * i + 1] = f.y; out[4 * i + 2] = f.z; out[4 * i + 3] = f.w;
    }
}

template <int D, bool APPEND, bool FP4>
__global__ void __launch_bounds__(kNrThreads, kResident) norm_rope_kernel(const __grid_constant__ NormRopeParams p) {
    using R = Row<D, APPEND, FP4>;
    extern __shared__ __align__(16) unsigned char nr_smem[];
    NrShared& sh = *reinterpret_cast<NrShared*>(nr_smem);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid < p.rot_dim / 2) {
        sh.turns[tid] = p.turns[tid];
        sh.axis[tid] = p.axis[tid];
    }
    __syncthreads();
    pdl_wait_primary();
    pdl_launch_dependents();

    R t{p, sh};
    t.warp = warp;
    t.lane = lane;
    t.l = lane % R::kLanes;
    t.sub = lane / R::kLanes;
    const int nr = p.rot_dim / 16;                 // lanes of a head that rotate
    t.turn = t.l < nr;
    const bool halves = t.turn && !p.interleaved;
    t.relay = p.interleaved || p.rot_dim < D;
    t.ea = halves ? 8 * t.l : 16 * t.l;
    t.eb = halves ? 8 * (t.l + nr) : 16 * t.l + 8;
    t.items = (unsigned)p.num_rows * (unsigned)p.segs;
    t.step = gridDim.x * kNrWarps;
    t.item = blockIdx.x * kNrWarps + warp;
    t.loads = t.uses = 0;
    t.slot = t.next_slot = 0;
    const unsigned first = t.item;
    if (first >= t.items) return;
    t.split(first, t.load_row, t.load_it, t.load_end);
    t.ask(first);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) t.load_next();
    load_weights(p.q_weight, t.ea, t.eb, t.qw);
    load_weights(p.k_weight, t.ea, t.eb, t.kw);
    const int q1 = p.iters_q, k1 = q1 + p.iters_k;
    for (unsigned i = first; i < t.items; i += t.step) {
        int it0, it1;
        t.split(i, t.row, it0, it1);
        t.take();
        t.ask(i + t.step);
        bool skip = false;
        if (APPEND) {
            skip = t.slot < 0 || t.slot >= p.num_slots;      // a padded row, or a bad slot
            if (t.slot >= p.num_slots && lane == 0) atomicOr(p.status, kDevBadPage);
        }
        t.template heads<kQ>(min(it0, q1), min(it1, q1), skip);
        t.template heads<kK>(max(it0, q1) - q1, min(it1, k1) - q1, skip);
        if (APPEND) t.template heads<kV>(max(it0, k1) - k1, it1 - k1, skip);
    }
}

template <int D>
cudaError_t launch_d(const NormRopeParams& p, bool append, int kv_dtype, dim3 grid, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kNrThreads);
    cfg.dynamicSmemBytes = sizeof(NrShared);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (!append) return cudaLaunchKernelEx(&cfg, &norm_rope_kernel<D, false, false>, p);
    return kv_dtype ? cudaLaunchKernelEx(&cfg, &norm_rope_kernel<D, true, true>, p)
                    : cudaLaunchKernelEx(&cfg, &norm_rope_kernel<D, true, false>, p);
}

template <int D>
cudaError_t prepare_d() {
    const void* kernels[3] = {reinterpret_cast<const void*>(&norm_rope_kernel<D, false, false>),
                              reinterpret_cast<const void*>(&norm_rope_kernel<D, true, false>),
                              reinterpret_cast<const void*>(&norm_rope_kernel<D, true, true>)};
    for (const void* k : kernels) {
        const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(NrShared));
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

cudaError_t norm_rope_prepare(int head_dim) {
    return head_dim == 64 ? prepare_d<64>() : head_dim == 128 ? prepare_d<128>() : prepare_d<256>();
}

cudaError_t norm_rope_launch(NormRopeParams& p, int head_dim, bool append, int kv_dtype, int num_sms,
                             cudaStream_t stream) {
    const int per = 512 / head_dim;                // heads of a warp iteration
    p.iters_q = (p.num_q_heads + per - 1) / per;
    p.iters_k = (p.num_kv_heads + per - 1) / per;
    p.iters_v = append ? p.iters_k : 0;
    const int iters = p.iters_q + p.iters_k + p.iters_v;
    // Segments of a row: few rows are cut into as many as there are warps for, others so that the last
    // round of the resident warps is not mostly idle.  A segment costs its iterations and about one more
    // for its cos and sin.  (5001 rows x 14 iterations on 2432 warps: 3 rounds of 15, or 5 of 8 in halves.)
    const long long resident = (long long)num_sms * kResident * kNrWarps;
    const long long most = std::max<long long>(1, std::min<long long>(iters, resident / std::max(p.num_rows, 1)));
    long long best = -1, best_per = iters;
    for (long long k = 0; k <= 8; ++k) {
        const long long s = k == 0 ? most : std::min<long long>(k, iters);
        const long long per_seg = (iters + s - 1) / s, segs = (iters + per_seg - 1) / per_seg;
        const long long rounds = (p.num_rows * segs + resident - 1) / resident;
        const long long cost = rounds * (per_seg + 1);
        if (best < 0 || cost < best) {
            best = cost;
            best_per = per_seg;
        }
    }
    p.iters_per_seg = (int)best_per;
    p.segs = (int)((iters + best_per - 1) / best_per);
    long long ctas = ((long long)p.num_rows * p.segs + kNrWarps - 1) / kNrWarps;
    if (ctas > (long long)num_sms * kResident) ctas = (long long)num_sms * kResident;
    const dim3 grid(static_cast<unsigned>(ctas));
    switch (head_dim) {
        case 64: return launch_d<64>(p, append, kv_dtype, grid, stream);
        case 128: return launch_d<128>(p, append, kv_dtype, grid, stream);
        case 256: return launch_d<256>(p, append, kv_dtype, grid, stream);
        default: return cudaErrorInvalidValue;
    }
}

}  // namespace spec_attn

struct spec_attn_norm_rope_plan {
    spec_attn_norm_rope_problem prob;
    int device;
    int num_sms;
    spec_attn::NormRopeParams params;   // everything but the call's own pointers
};

namespace {

bool nr_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

bool row_stride(int64_t given, int heads, int d, long long* out) {
    const int64_t dense = static_cast<int64_t>(heads) * d;
    *out = given ? given : dense;
    return given == 0 || (given >= dense && given % 8 == 0);
}

// Checks shared by the two calls; fills the call's own part of the parameters.
int prepare_call(const spec_attn_norm_rope_plan* plan, int32_t num_rows, const void* q, const void* k,
                 const float* q_weight, const float* k_weight, const int32_t* positions, void* q_out,
                 spec_attn::NormRopeParams* out) {
    const spec_attn_norm_rope_problem& p = plan->prob;
    if (p.num_q_heads > 0 && (!q || !q_out || !nr_aligned(q, 16) || !nr_aligned(q_out, 16)))
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_kv_heads > 0 && (!k || !nr_aligned(k, 16))) return SPEC_ATTN_E_INVALID_ARG;
    if (!nr_aligned(q_weight, 16) || !nr_aligned(k_weight, 16)) return SPEC_ATTN_E_INVALID_ARG;
    if (p.rot_dim > 0 && (!positions || !nr_aligned(positions, 4))) return SPEC_ATTN_E_INVALID_ARG;
    int dev = -1;
    const cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return spec_attn::record_cuda_error(e);
    if (dev != plan->device) return SPEC_ATTN_E_INVALID_ARG;
    *out = plan->params;
    out->q = static_cast<const uint16_t*>(q);
    out->k = static_cast<const uint16_t*>(k);
    out->q_weight = q_weight;
    out->k_weight = k_weight;
    out->positions = positions;
    out->pos_stride = num_rows;
    out->q_out = static_cast<uint16_t*>(q_out);
    out->num_rows = num_rows;
    return SPEC_ATTN_OK;
}

}  // namespace

extern "C" {

int spec_attn_norm_rope_plan_create(const spec_attn_norm_rope_problem* problem, const double* h_inv_freq,
                                    const uint8_t* h_pair_axis, spec_attn_norm_rope_plan** out) {
    if (!out) return SPEC_ATTN_E_INVALID_ARG;
    *out = nullptr;
    if (!problem) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_norm_rope_problem& p = *problem;
    if (p.num_q_heads < 0 || p.num_kv_heads < 0 || p.num_q_heads + static_cast<int64_t>(p.num_kv_heads) < 1)
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_q_heads > 4096 || p.num_kv_heads > 4096) return SPEC_ATTN_E_UNSUPPORTED;
    if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256)
        return p.head_dim > 0 ? SPEC_ATTN_E_UNSUPPORTED : SPEC_ATTN_E_INVALID_ARG;
    if (p.rot_dim < 0 || p.rot_dim > p.head_dim) return SPEC_ATTN_E_INVALID_ARG;
    if (p.rot_dim % 16 != 0) return SPEC_ATTN_E_UNSUPPORTED;
    if ((p.interleaved != 0 && p.interleaved != 1) || p.reserved != 0) return SPEC_ATTN_E_INVALID_ARG;
    if (p.num_axes < 1 || p.num_axes > 4) return SPEC_ATTN_E_INVALID_ARG;
    if (!(p.eps >= 0.f) || std::isinf(p.eps) || !std::isfinite(p.rot_scale)) return SPEC_ATTN_E_INVALID_ARG;
    if (p.rot_dim > 0 && !h_inv_freq) return SPEC_ATTN_E_INVALID_ARG;
    spec_attn::NormRopeParams c;
    std::memset(&c, 0, sizeof(c));
    if (!row_stride(p.q_row_stride, p.num_q_heads, p.head_dim, &c.q_row_stride) ||
        !row_stride(p.k_row_stride, p.num_kv_heads, p.head_dim, &c.k_row_stride) ||
        !row_stride(p.v_row_stride, p.num_kv_heads, p.head_dim, &c.v_row_stride) ||
        !row_stride(p.q_out_row_stride, p.num_q_heads, p.head_dim, &c.q_out_row_stride) ||
        !row_stride(p.k_out_row_stride, p.num_kv_heads, p.head_dim, &c.k_out_row_stride))
        return SPEC_ATTN_E_INVALID_ARG;
    for (int j = 0; j < p.rot_dim / 2; ++j) {
        const double w = h_inv_freq[j];
        if (!(w >= 0.0) || !(w < 1048576.0)) return SPEC_ATTN_E_INVALID_ARG;
        if (h_pair_axis && h_pair_axis[j] >= p.num_axes) return SPEC_ATTN_E_INVALID_ARG;
        const double turns = w / 6.283185307179586476925286766559;
        const double frac = turns - std::floor(turns);
        // below 1 by construction; 2^64 x frac is exact, its last bits are below the double's
        c.turns[j] = static_cast<unsigned long long>(std::ldexp(frac, 64));
        c.axis[j] = h_pair_axis ? h_pair_axis[j] : 0;
    }
    if (p.page_size != 0) {
        if (p.kv_dtype != SPEC_ATTN_KV_BF16 && p.kv_dtype != SPEC_ATTN_KV_NVFP4) return SPEC_ATTN_E_INVALID_ARG;
        if (p.page_size != 16 && p.page_size != 32 && p.page_size != 64)
            return p.page_size > 0 ? SPEC_ATTN_E_UNSUPPORTED : SPEC_ATTN_E_INVALID_ARG;
        if (p.num_pages < 1 || p.num_kv_heads < 1) return SPEC_ATTN_E_INVALID_ARG;
        const bool fp4 = p.kv_dtype == SPEC_ATTN_KV_NVFP4;
        const int64_t dense = static_cast<int64_t>(p.num_kv_heads) * p.page_size * (fp4 ? p.head_dim / 2 : 2 * p.head_dim);
        const int64_t dense_sc = static_cast<int64_t>(p.num_kv_heads) * p.page_size * (p.head_dim / 16);
        if (p.kv_page_stride != 0 && (p.kv_page_stride < dense || p.kv_page_stride % 16 != 0))
            return SPEC_ATTN_E_INVALID_ARG;
        if (fp4 && p.scale_page_stride != 0 && (p.scale_page_stride < dense_sc || p.scale_page_stride % 16 != 0))
            return SPEC_ATTN_E_INVALID_ARG;
        c.kv_page_stride = p.kv_page_stride ? p.kv_page_stride : dense;
        c.scale_page_stride = p.scale_page_stride ? p.scale_page_stride : dense_sc;
        c.page_shift = p.page_size == 64 ? 6 : p.page_size == 32 ? 5 : 4;
        c.num_slots = static_cast<long long>(p.num_pages) * p.page_size;
    }
    c.num_q_heads = p.num_q_heads;
    c.num_kv_heads = p.num_kv_heads;
    c.rot_dim = p.rot_dim;
    c.interleaved = p.interleaved;
    c.eps = p.eps;
    c.rot_scale = p.rot_scale == 0.f ? 1.f : p.rot_scale;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess) e = spec_attn::norm_rope_prepare(p.head_dim);
    if (e != cudaSuccess) return spec_attn::record_cuda_error(e);
    spec_attn_norm_rope_plan* plan = new (std::nothrow) spec_attn_norm_rope_plan();
    if (!plan) return SPEC_ATTN_E_INVALID_ARG;
    plan->prob = p;
    plan->device = dev;
    plan->num_sms = sms;
    plan->params = c;
    *out = plan;
    return SPEC_ATTN_OK;
}

int spec_attn_norm_rope_plan_destroy(spec_attn_norm_rope_plan* plan) {
    delete plan;
    return SPEC_ATTN_OK;
}

int spec_attn_norm_rope(const spec_attn_norm_rope_plan* plan, int32_t num_rows, const void* q, const void* k,
                        const float* q_weight, const float* k_weight, const int32_t* positions, void* q_out,
                        void* k_out, spec_attn_stream_t stream) {
    if (!plan || num_rows < 0) return SPEC_ATTN_E_INVALID_ARG;
    if (num_rows == 0) return SPEC_ATTN_OK;
    const spec_attn_norm_rope_problem& p = plan->prob;
    spec_attn::NormRopeParams c;
    const int st = prepare_call(plan, num_rows, q, k, q_weight, k_weight, positions, q_out, &c);
    if (st != SPEC_ATTN_OK) return st;
    if (p.num_kv_heads > 0 && (!k_out || !nr_aligned(k_out, 16))) return SPEC_ATTN_E_INVALID_ARG;
    // in place only where every element is written where it was read
    if ((q_out == q && c.q_out_row_stride != c.q_row_stride) || (k_out == k && k && c.k_out_row_stride != c.k_row_stride))
        return SPEC_ATTN_E_INVALID_ARG;
    c.k_out = static_cast<uint16_t*>(k_out);
    const cudaError_t e = spec_attn::norm_rope_launch(c, p.head_dim, false, 0, plan->num_sms,
                                                      reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_ATTN_OK : spec_attn::record_cuda_error(e);
}

int spec_attn_norm_rope_append(const spec_attn_norm_rope_plan* plan, int32_t num_rows, const void* q,
                               const void* k, const void* v, const float* q_weight, const float* k_weight,
                               const int32_t* positions, const int64_t* slot_map, void* q_out, void* k_pool,
                               void* v_pool, void* k_scales, void* v_scales, float k_gscale, float v_gscale,
                               void* workspace, size_t workspace_bytes, spec_attn_stream_t stream) {
    if (!plan || num_rows < 0 || plan->prob.page_size == 0) return SPEC_ATTN_E_INVALID_ARG;
    if (num_rows == 0) return SPEC_ATTN_OK;
    const spec_attn_norm_rope_problem& p = plan->prob;
    spec_attn::NormRopeParams c;
    const int st = prepare_call(plan, num_rows, q, k, q_weight, k_weight, positions, q_out, &c);
    if (st != SPEC_ATTN_OK) return st;
    if (q_out == q && q && c.q_out_row_stride != c.q_row_stride) return SPEC_ATTN_E_INVALID_ARG;
    if (!v || !nr_aligned(v, 16) || !slot_map || !nr_aligned(slot_map, 8) || !k_pool || !v_pool ||
        !nr_aligned(k_pool, 16) || !nr_aligned(v_pool, 16) || !workspace || !nr_aligned(workspace, 256))
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.kv_dtype == SPEC_ATTN_KV_NVFP4) {
        if (!k_scales || !v_scales || !nr_aligned(k_scales, 16) || !nr_aligned(v_scales, 16))
            return SPEC_ATTN_E_INVALID_ARG;
        if (!(k_gscale > 0.f) || !(v_gscale > 0.f) || std::isinf(k_gscale) || std::isinf(v_gscale))
            return SPEC_ATTN_E_INVALID_ARG;
    }
    if (workspace_bytes < 256) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    c.v = static_cast<const uint16_t*>(v);
    c.slot_map = reinterpret_cast<const long long*>(slot_map);
    c.k_pool = static_cast<unsigned char*>(k_pool);
    c.v_pool = static_cast<unsigned char*>(v_pool);
    c.k_scales = static_cast<uint8_t*>(k_scales);
    c.v_scales = static_cast<uint8_t*>(v_scales);
    c.k_gscale = k_gscale;
    c.v_gscale = v_gscale;
    c.status = static_cast<unsigned int*>(workspace);
    const cudaError_t e = spec_attn::norm_rope_launch(c, p.head_dim, true, p.kv_dtype, plan->num_sms,
                                                      reinterpret_cast<cudaStream_t>(stream));
    return e == cudaSuccess ? SPEC_ATTN_OK : spec_attn::record_cuda_error(e);
}

}  // extern "C"
