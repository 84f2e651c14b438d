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
// signed fraction it is rounded to fp32 for sincospi, and the part that this
// leaves out (up to 9e-8 radians, as much as the functions' own error) turns
// the result once more to first order.
//
// Layout.  A head of d elements is taken by d / 16 adjacent lanes, 16 elements
// each in two 16-byte pieces: with half-split pairs the pieces at l and l +
// rot / 16, so that a rotation needs no exchange between lanes; otherwise
// pieces 2 l and 2 l + 1.  A warp iteration is 512 elements: 2, 4 or 8 heads.  The
// launch's iterations are dealt out in even runs, one a resident warp (whole
// rows would leave the last round mostly idle: 4097 rows on 2432 warps).  At
// each row the lanes compute its cos and sin, two or four pairs each, and share
// them through shared memory; every lane then keeps its 8 pairs in registers
// over the row's heads.
//
// Loads run kAhead iterations ahead of the arithmetic, across heads, kinds and
// rows, as asynchronous copies of whole 1 KB iterations into a ring of the
// warp's own.  Where a lane's two pieces are not 128-byte runs across lanes
// (interleaved pairs, heads rotated in part), the results go back to the slot
// and leave in the order of memory: 16-byte stores 32 bytes apart cost twice the
// L2 requests.  The next row's positions and slot are asked for a row ahead.
// (With the loads in registers, two or four heads at a time, each warp waited
// out a memory round trip a batch: 16384 rows x 40 heads x 128 took 58.7 us,
// now 55.5; 8192 x 32 x 256 into the cache 52.7, now 45.4.  Rings of 4, 8 or 16
// iterations and three CTAs an SM were no faster.)
// CTAs stay resident and step over the rows, so the frequencies are copied from
// the kernel parameters to shared memory once per CTA, before the programmatic
// wait.
//
// Bound: HBM (2 bytes read and 2 written an element) for long inputs, 6.0 and
// 5.9 TB/s of algorithmic bytes in the two cases above (87 to 89 % of a copy);
// launch and two dependent memory round trips for a window (3.0 us for one row
// and for 72 into the cache, 3.5 into an NVFP4 cache).  Into an NVFP4 cache 4097
// rows of 24/4 heads x 256 take 26.3 us, bytes alone 18 (bf16: 24.0 and 20); no
// unit is full: issue slots 59 % of the cycles that an SM is active, integer pipe
// 35, FMA 32, shared memory 60, HBM 33 % of the launch.  The 16 warps of an SM
// wait for their own last instruction, for shared memory and, twice as often as
// with a bf16 cache, for instructions to arrive; SMs are active 83 % of the time.
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>

#include "../../include/spec_attn.h"
#include "common.cuh"
#include "nvfp4_quant.cuh"
#include "overlap.h"
#include "sm100.cuh"

namespace spec_attn {
namespace {

constexpr int kNrThreads = 256;
constexpr int kNrWarps = kNrThreads / 32;
constexpr int kAhead = 3;               // warp iterations whose loads are in flight
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

// A lane's 16 elements as pairs (A_j, B_j), j < 8, two j to a register pair: the
// two pieces (half-split), or the even and the odd elements (interleaved).
struct Pairs {
    uint64_t a[4], b[4];
};
__device__ __forceinline__ uint64_t lows(uint32_t v, uint32_t w) { return pack2(v << 16, w << 16); }
__device__ __forceinline__ uint64_t highs(uint32_t v, uint32_t w) { return pack2(v & 0xFFFF0000u, w & 0xFFFF0000u); }
__device__ __forceinline__ Pairs unpack16(const uint4& va, const uint4& vb, bool interleaved) {
    const uint32_t u[4] = {va.x, va.y, va.z, va.w}, w[4] = {vb.x, vb.y, vb.z, vb.w};
    Pairs x;
    if (interleaved) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            x.a[i] = lows(u[2 * i], u[2 * i + 1]);
            x.b[i] = highs(u[2 * i], u[2 * i + 1]);
            x.a[2 + i] = lows(w[2 * i], w[2 * i + 1]);
            x.b[2 + i] = highs(w[2 * i], w[2 * i + 1]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            x.a[i] = pack2(u[i] << 16, u[i] & 0xFFFF0000u);
            x.b[i] = pack2(w[i] << 16, w[i] & 0xFFFF0000u);
        }
    }
    return x;
}
__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ void pack16(const Pairs& x, bool interleaved, uint4& va, uint4& vb) {
    uint32_t u[4], w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 a = unpack2(x.a[i]), b = unpack2(x.b[i]);
        if (interleaved) {
            (i < 2 ? u : w)[2 * (i & 1)] = bf16x2(a.x, b.x);
            (i < 2 ? u : w)[2 * (i & 1) + 1] = bf16x2(a.y, b.y);
        } else {
            u[i] = bf16x2(a.x, a.y);
            w[i] = bf16x2(b.x, b.y);
        }
    }
    va = make_uint4(u[0], u[1], u[2], u[3]);
    vb = make_uint4(w[0], w[1], w[2], w[3]);
}

struct NrShared {
    uint4 ring[kNrWarps][kAhead][64];              // [iteration]: 512 elements of adjacent heads, in order
    ulonglong2 w[2][64];                           // weights of q and k, four a lane: [four][lane of the head]
    unsigned long long turns[kMaxPairs];
    float cs[kNrWarps][2][kMaxPairs];              // cos and sin of the warp's row
    uint8_t axis[kMaxPairs];
};

enum Kind { kQ = 0, kK = 1, kV = 2 };
enum Mode { kWhole, kPart, kInterleaved };   // half-split pairs over the whole head or part of it, pairs side by side

template <int D, bool APPEND, bool FP4>
struct Row {
    static constexpr int kLanes = D / 16;          // lanes of a head
    static constexpr int kHeads = 32 / kLanes;     // heads of a warp iteration

    const NormRopeParams& p;
    NrShared& sh;
    int warp, lane, l, sub;                        // l: lane within the head; sub: head within the iteration
    int ea, eb;                                    // first elements of the two pieces
    bool turn;                                     // this lane's pairs rotate
    float c[8], s[8];                              // cos and sin of the lane's pairs
    int row;
    long long slot;
    int pos[kMaxPairs / 32];                       // of the row to come, this lane's pairs
    long long next_slot;

    // head of the iteration's 16-byte piece lane + 32 j, in memory order
    __device__ __forceinline__ int head_of(int it, int j) const {
        return it * kHeads + j * (kHeads / 2) + lane / (D / 8);
    }

    // ---- the warp's run of iterations, `left` of them from iteration `it` of row `row` on; the loads' own copy of it
    struct Run {
        int row, it, end;                          // [it, end): the run's part of the row
        long long left;                            // beyond this row
        __device__ __forceinline__ void start(long long from, long long count, int iters) {
            row = (int)(from / iters);
            it = (int)(from % iters);
            left = count;
            trim(iters);
        }
        __device__ __forceinline__ void trim(int iters) {
            end = (int)min((long long)iters, it + left);
            left -= end - it;
        }
        __device__ __forceinline__ bool next(int iters) {
            if (left == 0) return false;
            ++row;
            it = 0;
            trim(iters);
            return true;
        }
    };
    Run load;
    int iters;                                     // of a row
    bool more;                                     // loads left to ask for
    int load_slot, use_slot;                       // ring
    const uint16_t* load_at;                       // this lane's first piece of the next iteration
    int load_head, load_heads;                     // its head, and the heads of its kind
    int load_left;                                 // iterations left of the kind

    // the row's iterations of one kind, from load.it on
    __device__ __forceinline__ void load_kind() {
        const int q1 = p.iters_q, k1 = q1 + p.iters_k, it = load.it;
        const int base = it < q1 ? 0 : it < k1 ? q1 : k1;
        const int stop = min(load.end, it < q1 ? q1 : it < k1 ? k1 : load.end);
        const uint16_t* src = it < q1 ? p.q : it < k1 ? p.k : p.v;
        src += (size_t)load.row * (it < q1 ? p.q_row_stride : it < k1 ? p.k_row_stride : p.v_row_stride);
        load_at = src + (it - base) * 512 + lane * 8;
        load_head = head_of(it - base, 0);
        load_heads = it < q1 ? p.num_q_heads : p.num_kv_heads;
        load_left = stop - it;
        load.it = stop;
    }
    __device__ __forceinline__ void load_next() {
        if (more) {
            const uint32_t dst = sm100::smem_addr(&sh.ring[warp][load_slot][lane]);
            if (load_head < load_heads) copy16(dst, load_at);
            if (load_head + kHeads / 2 < load_heads) copy16(dst + 512, load_at + 256);
            load_at += 512;
            load_head += kHeads;
            load_slot = load_slot + 1 == kAhead ? 0 : load_slot + 1;
            if (--load_left == 0) {
                if (load.it == load.end) more = load.next(iters);
                if (more) load_kind();
            }
        }
        copies_commit();                           // (one group a call, empty ones too)
    }
    __device__ __forceinline__ uint4* arrived() {
        copies_wait<kAhead - 1>();
        __syncwarp();                              // every lane's copies are in
        uint4* r = sh.ring[warp][use_slot];
        use_slot = use_slot + 1 == kAhead ? 0 : use_slot + 1;
        return r;
    }

    // ---- a row's positions and slot, asked for a row ahead
    __device__ __forceinline__ void ask(int r) {
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
                const long long v = (long long)u;
                const float top = (float)v;
                // what rounding the angle to fp32 left out, in radians, turns (cos, sin) by itself
                const float rest = (float)(v - __float2ll_rz(top)) * 3.4061215800865545e-19f;   // 2^-63 pi
                float sn, cn;
                sincospif(top * 1.0842021724855044e-19f, &sn, &cn);                             // 2^-63: in half turns
                cs[j] = fmaf(-rest, sn, cn) * p.rot_scale;
                cs[kMaxPairs + j] = fmaf(rest, cn, sn) * p.rot_scale;
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

    // w: the kind's weights in shared memory, in the lane's order (nullptr: no norm); ALL: every lane's pairs turn
    template <bool ALL>
    __device__ __forceinline__ void norm_rotate(Pairs& x, const ulonglong2* w) const {
        if (w) {
            uint64_t s0 = 0, s1 = 0;               // two fp32 zeros each
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                s0 = fma2(x.a[i], x.a[i], s0);
                s1 = fma2(x.b[i], x.b[i], s1);
            }
            const float2 st = unpack2(add2(s0, s1));
            float ss = st.x + st.y;
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(kFullMask, ss, o);
            const float r = rsqrtf(ss * (1.0f / D) + p.eps);
            const uint64_t r2 = pack2(r, r);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const ulonglong2 wa = w[i * kLanes + l], wb = w[(2 + i) * kLanes + l];
                x.a[2 * i] = mul2(x.a[2 * i], mul2(r2, wa.x));
                x.a[2 * i + 1] = mul2(x.a[2 * i + 1], mul2(r2, wa.y));
                x.b[2 * i] = mul2(x.b[2 * i], mul2(r2, wb.x));
                x.b[2 * i + 1] = mul2(x.b[2 * i + 1], mul2(r2, wb.y));
            }
        }
        if (ALL || turn) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float2 a = unpack2(x.a[i]), b = unpack2(x.b[i]);
                x.a[i] = pack2(a.x * c[2 * i] - b.x * s[2 * i], a.y * c[2 * i + 1] - b.y * s[2 * i + 1]);
                x.b[i] = pack2(a.x * s[2 * i] + b.x * c[2 * i], a.y * s[2 * i + 1] + b.y * c[2 * i + 1]);
            }
        }
    }

    // Warp iterations [it0, it1) of one kind.
    template <int KIND>
    __device__ __forceinline__ void heads(int it0, int it1, bool skip) {
        if (it0 >= it1) return;                    // (every branch here is uniform over the warp)
        if (skip) {                                // the row is only drained from the ring
            for (int it = it0; it < it1; ++it) {
                arrived();
                load_next();
            }
        } else if (KIND == kV) {
            loop<KIND, kWhole>(it0, it1);
        } else if (p.interleaved) {
            loop<KIND, kInterleaved>(it0, it1);
        } else if (p.rot_dim < D) {
            loop<KIND, kPart>(it0, it1);
        } else {
            loop<KIND, kWhole>(it0, it1);
        }
    }
    template <int KIND, int MODE>
    __device__ __forceinline__ void loop(int it0, int it1) {
        constexpr bool kCache = APPEND && KIND != kQ;
        constexpr bool kQuant = kCache && FP4;     // blocks of 16 adjacent elements: the pieces 2 l and 2 l + 1
        const int H = KIND == kQ ? p.num_q_heads : p.num_kv_heads;
        const ulonglong2* w = (KIND == kQ ? p.q_weight : p.k_weight) ? &sh.w[KIND == kQ ? 0 : 1][0] : nullptr;
        constexpr bool interleaved = MODE == kInterleaved;
        // where the lane's two results go: its own pieces of head it * kHeads + sub, or (in order) the
        // iteration's pieces lane and lane + 32
        constexpr bool in_order = !kQuant && (KIND == kV || MODE != kWhole);
        const int pa = (sub * D + ea) / 8, pb = (sub * D + eb) / 8;             // in the ring, read
        const int oa = kQuant ? (sub * D + 16 * l) / 8 : in_order ? lane : pa;  // and sent
        const int ob = kQuant ? oa + 1 : in_order ? lane + 32 : pb;
        int h0 = it0 * kHeads + oa / (D / 8), h1 = it0 * kHeads + ob / (D / 8);
        unsigned char *d0, *d1;                    // (quantised: codes, scales)
        size_t inc0, inc1;
        if constexpr (!kCache) {
            uint16_t* out = KIND == kQ ? p.q_out + (size_t)row * p.q_out_row_stride
                                       : p.k_out + (size_t)row * p.k_out_row_stride;
            d0 = reinterpret_cast<unsigned char*>(out + it0 * 512 + oa * 8);
            d1 = reinterpret_cast<unsigned char*>(out + it0 * 512 + ob * 8);
            inc0 = inc1 = 1024;
        } else {
            const long long page = slot >> p.page_shift;
            const int in_page = (int)(slot & ((1 << p.page_shift) - 1));
            unsigned char* pool = (KIND == kK ? p.k_pool : p.v_pool) + page * p.kv_page_stride;
            auto at = [&](int g) { return ((size_t)g << p.page_shift) + in_page; };   // head g's row of the page
            const size_t rows = (size_t)kHeads << p.page_shift;
            if constexpr (!kQuant) {
                d0 = pool + at(h0) * (2 * D) + oa % (D / 8) * 16;
                d1 = pool + at(h1) * (2 * D) + ob % (D / 8) * 16;
                inc0 = inc1 = rows * (2 * D);
            } else {
                d0 = pool + at(h0) * (D / 2) + l * 8;
                d1 = (KIND == kK ? p.k_scales : p.v_scales) + page * p.scale_page_stride + at(h0) * (D / 16) + l;
                inc0 = rows * (D / 2);
                inc1 = rows * (D / 16);
            }
        }
#pragma unroll 1
        for (int it = it0; it < it1; ++it) {
            uint4* ring = arrived();
            uint4 va, vb;
            if (KIND == kV) {
                va = ring[oa];
                vb = ring[ob];
            } else {
                va = ring[pa];
                vb = ring[pb];
                Pairs x = unpack16(va, vb, interleaved);
                norm_rotate<MODE == kWhole>(x, w);
                pack16(x, interleaved, va, vb);
                if (kQuant || in_order) {
                    ring[pa] = va;
                    ring[pb] = vb;
                    __syncwarp();
                    va = ring[oa];
                    vb = ring[ob];
                }
            }
            __syncwarp();                          // the slot is free
            load_next();
            if constexpr (!kQuant) {
                if (h0 < H) sm100::st_global_v4(d0, va);
                if (h1 < H) sm100::st_global_v4(d1, vb);
            } else if (h0 < H) {
                uint32_t c0, c1, sb;
                nvfp4_block(va, vb, KIND == kK ? p.k_gscale : p.v_gscale, c0, c1, sb);
                st_global_v2(d0, c0, c1);
                *d1 = static_cast<uint8_t>(sb);
            }
            d0 += inc0;
            d1 += inc1;
            h0 += kHeads;
            h1 += kHeads;
        }
    }
};

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
    t.ea = halves ? 8 * t.l : 16 * t.l;
    t.eb = halves ? 8 * (t.l + nr) : 16 * t.l + 8;
    // the launch's iterations in even runs, one a warp (a run begins and ends within a row)
    t.iters = p.iters_q + p.iters_k + p.iters_v;
    const long long total = (long long)p.num_rows * t.iters, warps = (long long)gridDim.x * kNrWarps;
    const long long me = (long long)blockIdx.x * kNrWarps + warp;
    const long long from = total * me / warps, count = total * (me + 1) / warps - from;
    t.load_slot = t.use_slot = 0;
    t.slot = t.next_slot = 0;
    // the weights, fours of one kind of pair (A, A, B, B) for each lane of a head, as unpack16 lays out its elements
    for (int u = tid; u < 2 * 4 * R::kLanes; u += kNrThreads) {
        const int kind = u / (4 * R::kLanes), f = u / R::kLanes % 4, l = u % R::kLanes;
        const float* w = kind ? p.k_weight : p.q_weight;
        if (!w) continue;
        const bool hv = l < nr && !p.interleaved;
        const int ea = hv ? 8 * l : 16 * l, eb = hv ? 8 * (l + nr) : 16 * l + 8;
        float x[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int j = 4 * (f & 1) + i;         // pair of the lane
            x[i] = p.interleaved ? w[16 * l + 2 * j + (f >> 1)] : w[(f < 2 ? ea : eb) + j];
        }
        sh.w[kind][f * R::kLanes + l] = make_ulonglong2(pack2(x[0], x[1]), pack2(x[2], x[3]));
    }
    __syncthreads();
    if (count == 0) return;
    typename R::Run run;
    run.start(from, count, t.iters);
    t.load = run;
    t.more = true;
    t.load_kind();
    t.ask(run.row);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) t.load_next();
    const int q1 = p.iters_q, k1 = q1 + p.iters_k;
    do {
        t.row = run.row;
        t.take();
        if (run.left > 0) t.ask(run.row + 1);
        bool skip = false;
        if (APPEND) {
            skip = t.slot < 0 || t.slot >= p.num_slots;      // a padded row, or a bad slot
            if (t.slot >= p.num_slots && lane == 0) atomicOr(p.status, kDevBadPage);
        }
        t.template heads<kQ>(min(run.it, q1), min(run.end, q1), skip);
        t.template heads<kK>(max(run.it, q1) - q1, min(run.end, k1) - q1, skip);
        if (APPEND) t.template heads<kV>(max(run.it, k1) - k1, run.end - k1, skip);
    } while (run.next(t.iters));
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
    // as many warps as there are iterations, up to those resident
    const long long total = (long long)p.num_rows * (p.iters_q + p.iters_k + p.iters_v);
    long long ctas = (total + kNrWarps - 1) / kNrWarps;
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
    if (!nr_aligned(q_weight, 4) || !nr_aligned(k_weight, 4)) return SPEC_ATTN_E_INVALID_ARG;
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

// `n` rows of `heads` heads, `stride` elements apart.
spec_attn::ByteRows rows_of(const void* p, int heads, int d, long long stride, int n) {
    return {p, 2ull * heads * d, 2ull * stride, static_cast<uint64_t>(n)};
}
// An input that is also the output in its place is looked at as that output.
const void* unless_in_place(const void* in, const void* out) { return in == out ? nullptr : in; }

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
    if ((q_out == q && q && c.q_out_row_stride != c.q_row_stride) ||
        (k_out == k && k && c.k_out_row_stride != c.k_row_stride))
        return SPEC_ATTN_E_INVALID_ARG;
    using spec_attn::bytes_at;
    const uint64_t w4 = 4ull * p.head_dim;
    const spec_attn::ByteRows out[] = {rows_of(q_out, p.num_q_heads, p.head_dim, c.q_out_row_stride, num_rows),
                                       rows_of(k_out, p.num_kv_heads, p.head_dim, c.k_out_row_stride, num_rows)};
    const spec_attn::ByteRows in[] = {
        rows_of(unless_in_place(q, q_out), p.num_q_heads, p.head_dim, c.q_row_stride, num_rows),
        rows_of(unless_in_place(k, k_out), p.num_kv_heads, p.head_dim, c.k_row_stride, num_rows),
        bytes_at(q_weight, w4), bytes_at(k_weight, w4),
        bytes_at(positions, p.rot_dim ? 4ull * p.num_axes * num_rows : 0)};
    if (spec_attn::outputs_overlap(out, in)) return SPEC_ATTN_E_INVALID_ARG;
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
    using spec_attn::bytes_at;
    const bool fp4 = p.kv_dtype == SPEC_ATTN_KV_NVFP4;
    const uint64_t w4 = 4ull * p.head_dim, slots = static_cast<uint64_t>(p.num_kv_heads) * p.page_size;
    const uint64_t page = slots * (fp4 ? p.head_dim / 2 : 2 * p.head_dim), scales = fp4 ? slots * (p.head_dim / 16) : 0;
    const uint64_t pages = static_cast<uint64_t>(p.num_pages);
    const spec_attn::ByteRows out[] = {
        rows_of(q_out, p.num_q_heads, p.head_dim, c.q_out_row_stride, num_rows),
        {k_pool, page, static_cast<uint64_t>(c.kv_page_stride), pages},
        {v_pool, page, static_cast<uint64_t>(c.kv_page_stride), pages},
        {k_scales, scales, static_cast<uint64_t>(c.scale_page_stride), pages},
        {v_scales, scales, static_cast<uint64_t>(c.scale_page_stride), pages},
        bytes_at(workspace, 256)};
    const spec_attn::ByteRows in[] = {
        rows_of(unless_in_place(q, q_out), p.num_q_heads, p.head_dim, c.q_row_stride, num_rows),
        rows_of(k, p.num_kv_heads, p.head_dim, c.k_row_stride, num_rows),
        rows_of(v, p.num_kv_heads, p.head_dim, c.v_row_stride, num_rows),
        bytes_at(q_weight, w4), bytes_at(k_weight, w4),
        bytes_at(positions, p.rot_dim ? 4ull * p.num_axes * num_rows : 0), bytes_at(slot_map, 8ull * num_rows)};
    if (spec_attn::outputs_overlap(out, in)) return SPEC_ATTN_E_INVALID_ARG;
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
