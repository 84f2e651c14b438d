// Cross attention of query rows to an encoder's states (spec_attn_run_cross) on
// 5th-generation tensor cores: dense K and V rows, a range of them for each
// request, every query row of the request seeing the whole range.
//
//   s_j = sm_scale <q, k_j>,  O = sum_j softmax(s)_j v_j,  LSE = ln sum_j exp(s_j)
//
// in one sweep with a running maximum and sum per row (base 2, fp32; P is
// rounded to bf16 for the second product, the sum adds the unrounded weights).
// A request with no states gets O = 0 and LSE = -inf.
//
// One CTA = (NQ query tiles of 128 rows) x (one KV head) x (a split of the
// request's states).  A tile holds wt = 128 / G whole window rows with their G
// heads, so K and V are read once for the G heads.  NQ = 2 (d = 128, launches of
// many tiles): the two tiles share every K and V tile, one tile's products
// running under the other tile's softmax.  Scores have two buffers of 64
// columns a tile or more, so S_{t+1} is made while the softmax works on S_t and
// the only chain from tile to tile is the softmax itself.  (One buffer of 128
// columns runs the first product at its full rate, 64 instead of 96 clocks for
// 128 states and 16 elements, but S_{t+1} then waits for softmax and P V of tile
// t: 451 us where two of 64 take 376.  A row's scores in halves for two threads:
// 443 us, the exchange of their maxima costs more than it saves.)
//
// Warp roles:
//   warp 0      the query tiles, then K and V tiles in turn, by TMA into one ring
//               of slots (64 rows each, 128-byte swizzled, chunk-major).
//   warps 1, 2  issue the products, one elected thread each.  NQ = 2: warp 1 + i
//               issues S_{t+1} and then P_t V_t of tile i.  NQ = 1: warp 1 issues
//               S = Q K^T and warp 2 O += P V, so that a late K tile holds no P V back.
//   warp 3      owns tensor memory.
//   warps 4-7 (and 8-11 for the second tile)   softmax, a row a thread, and the
//               epilogue.  In the last tile they also zero the V rows past the range's
//               end (what lies there may be anything, and 0 x NaN is NaN).
//
// TMEM columns: O tiles [0, NQ d), then two or four S buffers of 64 columns a
// tile, P (bf16 pairs) in the first half of its S buffer.
//
// Every wait is bounded; on time-out the CTA sets the device-status bit, drains
// its copies and products, frees its tensor memory and leaves.
//
// Splits: where the tiles alone would leave SMs idle, each request's states are
// cut into up to 8 ranges, whose CTAs form a cluster.  Each leaves its
// normalised rows in fp32 with their log-sum-exp in its own shared memory, and
// after a cluster barrier every CTA combines a share of the rows, in a fixed
// order, from its peers' shared memory: no partial goes to global memory and no
// second kernel follows.
//
// Bound.  Long prompts: the tensor cores, 1280 clocks for two tiles and 64 states
// at d = 128 (S runs at two thirds of its rate at 64 columns, its operands
// coming from shared memory) of 1350 measured: two requests of 4096 x 4096,
// 32/8 heads x 128, 376 us (1460 TFLOP/s), 24/4 x 256 580 us (1420).  At d = 64
// no unit is full (16/8 heads, the same rows: 162 us, 850 TFLOP/s; of a launch the
// tensor pipe is busy 58 %, the issue slots 50, the exponentials' pipe 35): each
// score takes half the products that it takes at d = 128, and with two query
// tiles an SM the chain from scores over maximum, exponentials and P to the next
// product shows.  At d = 256 the copies: TMA
// brings 42 bytes a clock into an SM, 1560 clocks for a tile's 64 KB (products
// 1280).  Single tokens and windows of large batches: HBM (64 tokens over 400 to
// 1601 states, 24/4 x 256: 48 us, 5.5 TB/s).  Few short windows: the chain of
// launch, first tile, some 0.45 us for each further tile of a split (load, maximum,
// exponentials and store of 64 scores by one thread), staging and combination:
// 8 windows of 9 rows over 1500 states 12.6 us.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <algorithm>
#include <cmath>
#include <new>
#include <type_traits>

#include "../../include/spec_attn.h"
#include "common.cuh"
#include "overlap.h"
#include "sm100.cuh"
#include "tc_common.cuh"

namespace spec_attn {
namespace {

using namespace sm100;
using namespace tcc;

constexpr int kM = 128;
constexpr int kMaxRing = 12;
constexpr int kMaxSorted = 256;          // requests put in order by one CTA's threads
constexpr int kMaxSplits = 8;            // CTAs of a cluster that any GPU schedules
constexpr float kCrossRescale = 8.0f;   // log2 units: O is rescaled when a row's maximum grows by more

constexpr int kBN = 64;                 // states a tile

// DEEP (one tile, d <= 128): the launch has no more CTAs than SMs, and a CTA
// takes the whole SM (12 slots and four S buffers; 9 rows x 32/8 heads x 128 over
// 1500 states for 8 requests: 12.8 us, 14.8 with the half-SM layout); otherwise
// two CTAs share it, one's start, end and waits under the other's work (64
// single tokens over 1601 states: 69.9 us, 80.4 with one CTA an SM).  d = 256
// and two tiles always take the whole SM.
template <int D, int NQ, bool DEEP>
struct CrossLayout {
    static_assert(NQ == 1 || D == 128, "two O tiles and four S buffers fit 512 columns up to d = 128");
    static constexpr int kChunks = D / 64;
    static constexpr int kQBytes = kM * D * 2;             // one query tile
    static constexpr int kTileBytes = kBN * D * 2;         // one K or V tile
    static constexpr int kAux = 2048;
    static constexpr int kCtas = DEEP ? 1 : 2;
    // S buffers of a tile (a power of two): two, or four for a lone tile with the SM to itself, whose
    // S_{t+1} then does not wait for P V of tile t - 1
    static constexpr int kBufShift = NQ == 1 && DEEP ? 2 : 1;
    static constexpr int kBufs = 1 << kBufShift;
    static constexpr int kNeed = NQ * (D + kBufs * kBN);
    static constexpr uint32_t kCols = kNeed <= 256 ? 256u : 512u;   // allocated: a power of two
    static_assert(kNeed <= 512 && kCols * kCtas <= 512, "tensor memory");
    // first column of buffer b of tile i
    __host__ __device__ static constexpr int s_col(int i, int b) { return NQ * D + (kBufs * i + b) * kBN; }
    // The ring.  NQ = 1: a slot a tile, K_t and V_t in turn, each let go as soon as
    // it has been read.  NQ = 2: a slot holds K_t and V_t, filled and let go
    // together: one barrier to wait on and one commit less for each of the
    // products, whose issue is what bounds long prompts.
    static constexpr int kSlotTiles = NQ;
    static constexpr int kSlotBytes = kSlotTiles * kTileBytes;
    static constexpr int kMax = DEEP ? 232448 : 232448 / 2 - 1024;   // 227 KB a CTA, 228 KB an SM (1 KB of each CTA reserved)
    static constexpr int kFit = (kMax - 1024 - kAux - NQ * kQBytes) / kSlotBytes;
    static constexpr int kRing = kFit > kMaxRing ? kMaxRing : kFit;
    static constexpr int kSmem = 1024 + kAux + NQ * kQBytes + kRing * kSlotBytes;
    static_assert(kRing >= 4, "tiles ahead of the ones in use");
    // S may lead P V by as many tiles as it has buffers.  An odd ring puts K_t where V of tile
    // t - (ring + 1) / 2 was, and that V has to be gone before its slot's next phase is waited for
    // (a wait two phases ahead would take the older one for it).
    static constexpr int kLead = (NQ == 2 || kBufs <= (kRing + 1) / 2) ? kBufs : (kRing + 1) / 2;
    // P V barriers in use: one a slot (NQ = 2), or one an S buffer and at least four
    static constexpr int kPv = NQ == 2 ? kRing : 4;
    // the epilogue's fp32 rows, 16 bytes apart beyond their length (no bank conflict), and their log-sum-exps
    static constexpr int kRowFloats = D + 4;
    static_assert(NQ * kM * (kRowFloats + 1) * 4 <= NQ * kQBytes + kRing * kSlotBytes, "epilogue staging");
    static constexpr int kThreads = 128 + NQ * 128;
};

struct CrossAux {
    uint64_t full[kMaxRing];
    uint64_t empty[kMaxRing];           // NQ = 1
    uint64_t pv_done[2][kMaxRing];      // P_t V_t of tile i done: O, P_t's buffer and (NQ = 2) the slot; by t mod ring
    uint64_t q_full[2];
    uint64_t s_full[2][4];              // [tile][buffer] scores written
    uint64_t p_full[2][4];              // P written over them (four softmax warps)
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
    int request;                        // longest-first order: the CTA's request
    int lens[kMaxSorted];
};
static_assert(sizeof(CrossAux) <= 2048, "aux region");

// Bounded wait of a whole warp; the clock is read only when the phase is still open.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, volatile int* abort) {
    if (__all_sync(kFullMask, mbar_try_wait(bar, parity))) return true;
    return warp_wait(bar, parity, abort);
}

// A shared-memory matrix descriptor is its high word, the same for every tile of
// one kind, and a low word that a constant step moves along the tile: the
// issuing thread adds to one register instead of building 64 bits each time.
__device__ __forceinline__ uint32_t desc_lo(uint32_t saddr, uint32_t lbo_bytes) {
    return ((saddr >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);   // (in a cluster the address has the rank above bit 23)
}
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);   // 8-row groups 1024 B apart, version 1, 128-byte swizzle
// Products and commits are issued by the one thread whose `go` is set, under a
// predicate: the whole warp runs the issuing loop and its waits.  (With the loop
// in a branch of one thread, each wait cost the next product 200 clocks: 8 + 4
// instructions with a wait before each kind took 1053 clocks, and 621 like this.)
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate,
                                          uint32_t go) {
    asm volatile(
        "{\n\t.reg .pred p, g;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 g, %6, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@g tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(kDescHi), "r"(go)
        : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate,
                                          uint32_t go) {
    asm volatile(
        "{\n\t.reg .pred p, g;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 g, %6, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@g tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(kDescHi), "r"(go)
        : "memory");
}
__device__ __forceinline__ void commit_if(uint64_t* bar, uint32_t go) {
    asm volatile(
        "{\n\t.reg .pred g;\n\t"
        "setp.ne.b32 g, %1, 0;\n\t"
        "@g tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_addr(bar)),
        "r"(go)
        : "memory");
}
__device__ __forceinline__ uint32_t elected() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r;
}

// Thread-block cluster: all threads of all its CTAs (those that left count as
// arrived), and shared memory of the CTA of a given rank.
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ uint32_t peer_addr(uint32_t saddr, uint32_t rank) {
    uint32_t d;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(saddr), "r"(rank));
    return d;
}
__device__ __forceinline__ float4 ld_peer_v4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}
__device__ __forceinline__ float ld_peer(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

// The request's rows and states, checked.
struct CrossReq {
    int row0, w, start, len;
};
__device__ __forceinline__ bool cross_request(const CrossParams& p, int r, unsigned int* status, CrossReq& q) {
    const int row0 = p.q_indptr[r], row1 = p.q_indptr[r + 1];
    q.start = p.kv_start[r];
    q.len = p.kv_len[r];
    q.row0 = row0;
    if (row0 < 0 || row1 < row0 || row1 > p.total_rows || row1 - row0 > p.max_rows) {
        if (status) atomicOr(status, kDevBadWindow);
        return false;
    }
    q.w = row1 - row0;
    if (q.len < 0 || q.len > p.max_kv_len || q.start < 0 || (long long)q.start + q.len > p.total_kv) {
        if (status) atomicOr(status, kDevBadSeqLen);
        return false;
    }
    return q.w > 0;
}

template <int D, int NQ, bool DEEP>
__global__ void __launch_bounds__(CrossLayout<D, NQ, DEEP>::kThreads, CrossLayout<D, NQ, DEEP>::kCtas)
cross_attn_kernel(const CrossParams p, const __grid_constant__ CUtensorMap tmq, const __grid_constant__ CUtensorMap tmk,
                  const __grid_constant__ CUtensorMap tmv) {
    using L = CrossLayout<D, NQ, DEEP>;
    constexpr int BN = kBN, PV = L::kPv, RING = L::kRing, SH = L::kBufShift, NB = L::kBufs;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int tile = blockIdx.x / p.max_splits, split = blockIdx.x % p.max_splits;   // (split: the rank in the cluster)
    const int kvh = blockIdx.y;
    int r = blockIdx.z;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    CrossAux* aux = reinterpret_cast<CrossAux*>(smem);
    unsigned char* sQ = smem + L::kAux;
    unsigned char* ring = sQ + NQ * L::kQBytes;
    volatile int* abort = &aux->abort;

    if (tid == 0) {
        for (int s = 0; s < RING; ++s) {
            mbar_init(&aux->full[s], 1);
            mbar_init(&aux->empty[s], 1);
        }
        for (int i = 0; i < NQ; ++i) {
            for (int s = 0; s < PV; ++s) mbar_init(&aux->pv_done[i][s], 1);
            mbar_init(&aux->q_full[i], 1);
            for (int b = 0; b < NB; ++b) {
                mbar_init(&aux->s_full[i][b], 1);
                mbar_init(&aux->p_full[i][b], 4);
            }
        }
        mbar_init(&aux->drain[0], 1);
        mbar_init(&aux->drain[1], 1);
        aux->abort = 0;
        fence_mbarrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (warp == 3) tmem_alloc(&aux->tmem_base, L::kCols);
    // up to here the CTA touched only its own resources, while the previous kernel drains
    pdl_wait_primary();
    pdl_launch_dependents();   // (the next kernel's CTAs set up as these leave their SMs)
    if (p.longest_first) {
        // More CTAs than the GPU holds: the requests with the most states go first, so that the last CTAs to
        // start are short ones.  Each CTA ranks the lengths itself (ties by index).
        if (tid < p.longest_first) aux->lens[tid] = p.kv_len[tid];
        __syncthreads();
        if (tid < p.longest_first) {
            const int mine = aux->lens[tid];
            int rank = 0;
            for (int j = 0; j < p.longest_first; ++j) rank += aux->lens[j] > mine || (aux->lens[j] == mine && j < tid);
            if (rank == blockIdx.z) aux->request = tid;
        }
        __syncthreads();
        r = aux->request;
    }
    CrossReq q;
    const bool reporter = tid == 0 && blockIdx.x == 0 && kvh == 0;
    bool active = cross_request(p, r, reporter ? p.status : nullptr, q);
    const int lo = tile * NQ * p.wt;               // first window row of the CTA
    const int nsplits = active ? max(1, (q.len + p.keys_per_split - 1) / p.keys_per_split) : 0;
    active = active && lo < q.w && split < nsplits;
    const int G = p.group;
    const int nact = (NQ == 2 && lo + p.wt < q.w) ? 2 : 1;
    const int rows = min(q.w - lo, NQ * p.wt) * G; // query rows of the CTA, wt * G of them in its first tile
    const int key_lo = split * p.keys_per_split;
    const int key_hi = min(key_lo + p.keys_per_split, q.len);
    const int T = active ? (key_hi - key_lo + BN - 1) / BN : 0;
    const int tail = key_hi - (key_lo + (T - 1) * BN);     // states of the last tile
    // row m of the CTA: its place in O and LSE
    auto place = [&](int m) { return (size_t)(q.row0 + lo + m / G) * p.num_q_heads + kvh * G + m % G; };
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = aux->tmem_base;
    float* stage = reinterpret_cast<float*>(sQ);           // (epilogue)
    float* stage_lse = stage + NQ * kM * L::kRowFloats;
    if (T == 0) {                                  // no work, or no states
        if (active) {
            for (int u = tid; u < rows * (D / 8); u += L::kThreads) {
                const size_t at = place(u / (D / 8));
                st_global_v4(p.o + at * D + u % (D / 8) * 8, make_uint4(0u, 0u, 0u, 0u));
                if (u % (D / 8) == 0 && p.lse) p.lse[at] = -INFINITY;
            }
        }
        __syncwarp();
        if (warp == 3) tmem_dealloc(tmem, L::kCols);
        return;
    }

    if (warp == 0) {
        // ------------------------------------------------------------ copies
        int issued = 0;
        if (lane == 0) {
            const uint32_t qbytes = static_cast<uint32_t>(L::kChunks * 128 * G * p.wt);
            for (int i = 0; i < nact; ++i) {
                mbar_arrive_expect_tx(&aux->q_full[i], qbytes);
                for (int c = 0; c < L::kChunks; ++c)
                    tma_load_3d(sQ + i * L::kQBytes + c * (kM * 128), &tmq, c * 64, kvh * G, q.row0 + lo + i * p.wt,
                                &aux->q_full[i]);
            }
        }
        __syncwarp();
        auto load_tile = [&](unsigned char* dst, const CUtensorMap* map, int t, uint64_t* bar) {
            for (int c = 0; c < L::kChunks; ++c)
                tma_load_3d(dst + c * (BN * 128), map, c * 64, kvh, q.start + key_lo + t * BN, bar);
        };
        for (int n = 0; n < (NQ == 2 ? T : 2 * T); ++n) {
            const int slot = n % RING;
            const uint32_t gone = ((n / RING) - 1) & 1;
            if (n >= RING) {
                if (NQ == 1 && !wait_warp(&aux->empty[slot], gone, abort)) break;
                if (NQ == 2 && !(wait_warp(&aux->pv_done[0][slot], gone, abort) &&
                                 (nact == 1 || wait_warp(&aux->pv_done[1][slot], gone, abort))))
                    break;
            }
            if (lane == 0) {
                unsigned char* dst = ring + slot * L::kSlotBytes;
                mbar_arrive_expect_tx(&aux->full[slot], L::kSlotBytes);
                if (NQ == 2) {
                    load_tile(dst, &tmk, n, &aux->full[slot]);
                    load_tile(dst + L::kTileBytes, &tmv, n, &aux->full[slot]);
                } else {
                    load_tile(dst, (n & 1) ? &tmv : &tmk, n >> 1, &aux->full[slot]);
                }
            }
            __syncwarp();
            issued = n + 1;
        }
        if (*abort && lane == 0) {
            for (int n = max(0, issued - RING); n < issued; ++n) {
                volatile int go_on = 0;
                mbar_wait(&aux->full[n % RING], (n / RING) & 1, &go_on, kDrainLimit);
            }
            volatile int no_abort = 0;
            for (int i = 0; i < nact; ++i) mbar_wait(&aux->q_full[i], 0, &no_abort, kDrainLimit);
        }
        __syncwarp();
    } else if (warp == 1 || (warp == 2 && (NQ == 1 || nact == 2))) {
        // ------------------------------------------------------------ products
        const uint32_t go = elected();
        constexpr uint32_t idesc_s = idesc_bf16_f32(kM, BN, 0, 0);
        constexpr uint32_t idesc_o = idesc_bf16_f32(kM, D, 0, 1);
        const int i = NQ == 2 ? warp - 1 : 0;
        const uint32_t q_lo = desc_lo(smem_addr(sQ + i * L::kQBytes), 16);
        const uint32_t k_lo0 = desc_lo(smem_addr(ring), 16), v_lo0 = desc_lo(smem_addr(ring), BN * 128);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, abort); };
        // the ring slots of K_t and V_t, and the slot t mod ring, stepped along with the parity of their phase
        struct Step {
            int size, slot;
            uint32_t par;
            __device__ __forceinline__ void by(int n) {
                slot += n;
                if (slot >= size) {
                    slot -= size;
                    par ^= 1;
                }
            }
        };
        Step ks = {RING, 0, 0}, vs = {RING, NQ == 1 ? 1 : 0, 0};
        Step done = {PV, 0, 0}, before = {PV, 0, 0};   // (before: t - lead of the next S)
        // S_t, once K_t is here and the P that sat in S_t's buffer has been read
        auto do_s = [&](int t) {
            const int b = t & (NB - 1);
            if (t >= L::kLead) {
                if (!wait(&aux->pv_done[i][before.slot], before.par)) return false;
                before.by(1);
            }
            if (!wait(&aux->full[ks.slot], ks.par)) return false;
            tc_fence_after();
            const uint32_t k_lo = k_lo0 + ks.slot * (L::kSlotBytes >> 4), d_tmem = tmem + L::s_col(i, b);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const int c = kk >> 2, sub = kk & 3;
                mma_ss_lo(d_tmem, q_lo + c * (kM * 128 >> 4) + sub * 2, k_lo + c * (BN * 128 >> 4) + sub * 2, idesc_s,
                          kk > 0, go);
            }
            commit_if(&aux->s_full[i][b], go);
            if (NQ == 1) commit_if(&aux->empty[ks.slot], go);
            ks.by(NQ == 1 ? 2 : 1);
            return true;
        };
        // O += P_t V_t, once both are here (NQ = 2: V_t came with K_t)
        auto do_pv = [&](int t) {
            const int b = t & (NB - 1);
            if (NQ == 1 && !wait(&aux->full[vs.slot], vs.par)) return false;
            if (!wait(&aux->p_full[i][b], (t >> SH) & 1)) return false;
            tc_fence_after();
            const uint32_t v_lo = v_lo0 + (vs.slot * L::kSlotBytes + (NQ - 1) * L::kTileBytes) / 16;
            const uint32_t p_tmem = tmem + L::s_col(i, b);
            const int steps = t == T - 1 ? (tail + 15) / 16 : BN / 16;
#pragma unroll
            for (int kk = 0; kk < BN / 16; ++kk)
                if (kk < steps) mma_ts_lo(tmem + i * D, p_tmem + kk * 8, v_lo + kk * (2048 >> 4), idesc_o, t > 0 || kk > 0, go);
            commit_if(&aux->pv_done[i][done.slot], go);
            if (NQ == 1) commit_if(&aux->empty[vs.slot], go);
            vs.by(NQ == 1 ? 2 : 1);
            done.by(1);
            return true;
        };
        bool ok = true;
        if (NQ == 2 || warp == 1) ok = wait(&aux->q_full[i], 0);
        if (NQ == 2) {
            ok = ok && do_s(0);
            for (int t = 0; t < T && ok; ++t) ok = (t + 1 == T || do_s(t + 1)) && do_pv(t);
        } else if (warp == 1) {
            for (int t = 0; t < T && ok; ++t) ok = do_s(t);
        } else {
            for (int t = 0; t < T && ok; ++t) ok = do_pv(t);
        }
        // every product this thread issued completes before the memory is released
        uint64_t* drain = &aux->drain[warp - 1];
        commit_if(drain, go);
        volatile int no_abort = 0;
        mbar_wait(drain, 0, &no_abort, kDrainLimit);
        __syncwarp();
    } else if (warp >= 4 && (warp < 8 || nact == 2)) {
        // ------------------------------------------------------------ softmax and epilogue
        const int i = warp >= 8 ? 1 : 0;                   // tile
        const int m = (warp & 3) * 32 + lane;              // row of the tile
        const uint32_t lane_tmem = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int wrow = lo + i * p.wt + m / G;            // window row
        const bool valid = m < p.wt * G && wrow < q.w;
        // a warp without rows leaves its scores as they are: they weigh on no other row
        const bool live = __any_sync(kFullMask, valid);
        const float sc = p.score_scale_log2;
        float m_ref = -INFINITY, l_sum = 0.f;
        bool ok = true;
        const uint64_t sc2 = pack2(sc, sc);
        for (int t = 0; t < T; ++t) {
            const int b = t & (NB - 1);
            if (!(ok = wait_warp(&aux->s_full[i][b], (t >> SH) & 1, abort))) break;
            tc_fence_after();
            const uint32_t s_tmem = lane_tmem + L::s_col(i, b);
            if (live) {
                __syncwarp();
                float sv[BN];
                tmem_ld32(s_tmem, *reinterpret_cast<float(*)[32]>(sv));
                tmem_ld32(s_tmem + 32, *reinterpret_cast<float(*)[32]>(sv + 32));
                tmem_wait_ld();
                if (t == T - 1 && tail < BN) {
#pragma unroll
                    for (int c = 0; c < BN; ++c) sv[c] = c < tail ? sv[c] : -INFINITY;
                }
                float mx4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
                for (int c = 4; c < BN; c += 8) {   // (three-way maxima)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx4[k] = fmaxf(fmaxf(mx4[k], sv[c + k]), c + 4 < BN ? sv[c + 4 + k] : mx4[k]);
                }
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sc;
                // the reference moves at the first tile, and when the maximum outgrows it
                const bool need = mx > m_ref + kCrossRescale;
                const float ref = need ? mx : m_ref;
                const float alpha = need ? fast_exp2(m_ref - ref) : 1.f;   // (0 at the first tile)
                // (an infinite reference is not subtracted: inf - inf would hide in the sum what the scores were.  Plus
                // infinity makes the sum and with it the log-sum-exp infinite, and O, times 1 / inf, NaN.)
                const float nref = fabsf(ref) == INFINITY ? 0.f : -ref;
                const uint64_t nref2 = pack2(nref, nref);
                uint32_t pk[BN / 2];
                uint64_t ps[2] = {0, 0};   // two fp32 zeros each
#pragma unroll
                for (int c = 0; c < BN; c += 2) {
                    const float2 x = unpack2(fma2(pack2(sv[c], sv[c + 1]), sc2, nref2));
                    const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                    ps[(c >> 1) & 1] = add2(ps[(c >> 1) & 1], pack2(p0, p1));
                    const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
                    pk[c >> 1] = *reinterpret_cast<const uint32_t*>(&h2);
                }
                const float2 psum = unpack2(add2(ps[0], ps[1]));
                l_sum = l_sum * alpha + (psum.x + psum.y);
                m_ref = ref;
                if (t > 0 && __any_sync(kFullMask, valid && need)) {
                    // every earlier P V has to be in
                    if (!(ok = wait_warp(&aux->pv_done[i][(t - 1) % PV], ((t - 1) / PV) & 1, abort))) break;
                    tc_fence_after();
                    __syncwarp();
#pragma unroll 1
                    for (int ch = 0; ch < D / 32; ++ch) {
                        float ov[32];
                        tmem_ld32(lane_tmem + i * D + ch * 32, ov);
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < 32; ++e) ov[e] *= alpha;
                        tmem_st32(lane_tmem + i * D + ch * 32, ov);
                    }
                }
                tmem_st32u(s_tmem, pk);
                tmem_wait_st();
            }
            if (t == T - 1 && (tail & 15) != 0) {
                // The slot's earlier tile was consumed before these scores could be made, so the parity
                // names this phase.  Both tiles' warps write the same zeros.
                constexpr int C8 = L::kChunks * 8;         // 16-byte pieces of a row
                const int n = NQ == 2 ? T - 1 : 2 * T - 1, rows = ((tail + 15) & ~15) - tail;
                if (!(ok = wait_warp(&aux->full[n % RING], (n / RING) & 1, abort))) break;
                const uint32_t v_addr = smem_addr(ring + (n % RING) * L::kSlotBytes + (NQ - 1) * L::kTileBytes);
                for (int u = m; u < rows * C8; u += 128)
                    st_shared_v4(v_addr + ((u % C8) >> 3) * (BN * 128) + (tail + u / C8) * 128 + (u & 7) * 16,
                                 make_uint4(0u, 0u, 0u, 0u));
                fence_proxy_async_smem();
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&aux->p_full[i][b]);
        }
        // both tiles' products are done: the query tiles and the ring are free
        for (int j = 0; j < NQ; ++j)
            if (ok && j < nact) ok = wait_warp(&aux->pv_done[j][(T - 1) % PV], ((T - 1) / PV) & 1, abort);
        tc_fence_after();
        if (ok) {
            float* row = stage + (i * p.wt * G + m) * L::kRowFloats;   // (rows past the tile's wt * G are not written)
            // (scores of minus infinity throughout: no weight, which the other splits' rows outweigh)
            const float inv = nsplits > 1 && l_sum == 0.f ? 0.f : 1.f / l_sum;
            if (live) {
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ++ch) {
                    float ov[32];
                    tmem_ld32(lane_tmem + i * D + ch * 32, ov);
                    tmem_wait_ld();
                    if (valid) {
#pragma unroll
                        for (int e = 0; e < 32; e += 4)
                            *reinterpret_cast<float4*>(row + ch * 32 + e) =
                                make_float4(ov[e] * inv, ov[e + 1] * inv, ov[e + 2] * inv, ov[e + 3] * inv);
                    }
                    __syncwarp();   // the next load takes the whole warp at once
                }
            }
            if (valid) stage_lse[i * p.wt * G + m] = m_ref + log2f(l_sum);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 3) {
        tc_fence_after();
        tmem_dealloc(tmem, L::kCols);
    }
    if (tid == 0 && *abort) atomicOr(p.status, kDevWaitTimeout);
    // ---------------------------------------------------------------- rows out
    auto pair = [](float lo, float hi) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t*>(&h);
    };
    if (nsplits == 1) {
        if (*abort) return;
        constexpr int C8 = D / 8;
        for (int u = tid; u < rows * C8; u += L::kThreads) {
            const int m = u / C8, c = u % C8;
            const float4* src = reinterpret_cast<const float4*>(stage + m * L::kRowFloats + c * 8);
            const float4 a = src[0], b = src[1];
            st_global_v4(p.o + place(m) * D + c * 8, make_uint4(pair(a.x, a.y), pair(a.z, a.w), pair(b.x, b.y), pair(b.z, b.w)));
            if (c == 0 && p.lse) p.lse[place(m)] = stage_lse[m] * kLn2;
        }
        return;
    }
    __syncwarp();
    cluster_sync();                                // every split's rows are in its shared memory
    if (!*abort) {
        auto combine = [&](auto most) {
            constexpr int N = decltype(most)::value;
            // Every load of a unit is on its way before the first is used, and each CTA begins with its own
            // rows: were all to begin with rank 0, they would queue at one SM.  Units of 4 elements: with 8, half
            // the threads had none (16 rows of 32/8 heads x 128 over 4096 states in 8 splits 12.6 us, now 11.0).
            constexpr int C4 = D / 4;
            uint32_t rows_at[N], lse_at[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int from = split + k < nsplits ? split + k : split + k - nsplits;
                rows_at[k] = peer_addr(smem_addr(stage), k < nsplits ? from : split);
                lse_at[k] = peer_addr(smem_addr(stage_lse), k < nsplits ? from : split);
            }
            for (int u = split * L::kThreads + tid; u < rows * C4; u += nsplits * L::kThreads) {
                const int m = u / C4, c = u % C4;
                float ls[N];
                float4 x[N];
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    ls[k] = ld_peer(lse_at[k] + m * 4);
                    x[k] = ld_peer_v4(rows_at[k] + (m * L::kRowFloats + c * 4) * 4);
                }
                // (N is the least of 2, 4 and 8 that holds the splits: those past the middle may not be there, and a
                // weight of 0 would not take out a row that holds infinity)
                auto here = [&](int k) { return k <= N / 2 || k < nsplits; };
                float mx = ls[0], sum = 0.f;
#pragma unroll
                for (int k = 1; k < N; ++k)
                    if (here(k)) mx = fmaxf(mx, ls[k]);
                const float ref = fabsf(mx) == INFINITY ? 0.f : mx;   // (as in the softmax)
                float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int k = 0; k < N; ++k) {
                    if (!here(k)) break;
                    const float w = fast_exp2(ls[k] - ref);
                    a.x = fmaf(w, x[k].x, a.x); a.y = fmaf(w, x[k].y, a.y);
                    a.z = fmaf(w, x[k].z, a.z); a.w = fmaf(w, x[k].w, a.w);
                    sum += w;
                }
                const float inv = 1.f / sum;
                *reinterpret_cast<uint2*>(p.o + place(m) * D + c * 4) =
                    make_uint2(pair(a.x * inv, a.y * inv), pair(a.z * inv, a.w * inv));
                if (c == 0 && p.lse) p.lse[place(m)] = (mx + log2f(sum)) * kLn2;
            }
        };
        if (nsplits <= 2) combine(std::integral_constant<int, 2>());
        else if (nsplits <= 4) combine(std::integral_constant<int, 4>());
        else combine(std::integral_constant<int, kMaxSplits>());
    }
    __syncwarp();
    cluster_sync();                                // no CTA leaves while its rows are being read
}

using CrossKernel = void (*)(const CrossParams, const CUtensorMap, const CUtensorMap, const CUtensorMap);

// What a launch of (d, query tiles a CTA) needs.
struct CrossVariant {
    CrossKernel kernel;
    int threads, smem, ctas;   // ctas: on one SM
};
template <int D, int NQ, bool DEEP>
CrossVariant variant_of() {
    using L = CrossLayout<D, NQ, DEEP>;
    return {&cross_attn_kernel<D, NQ, DEEP>, L::kThreads, L::kSmem, L::kCtas};
}
CrossVariant cross_variant(int d, int nq, bool deep) {
    if (d == 256) return variant_of<256, 1, true>();
    if (nq == 2) return variant_of<128, 2, true>();
    if (d == 64) return deep ? variant_of<64, 1, true>() : variant_of<64, 1, false>();
    return deep ? variant_of<128, 1, true>() : variant_of<128, 1, false>();
}

PFN_cuTensorMapEncodeTiled_v12000 cross_encode_fn() {
    static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        const bool ok = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                                         &q) == cudaSuccess &&
                        q == cudaDriverEntryPointSuccess;
        return ok ? reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr) : nullptr;
    }();
    return fn;
}

// Rows [rows, heads, d] bf16, row_stride elements apart, as (element, head, row); box = 64 elements x
// box_heads x box_rows, 128-byte swizzle, rows past the end zero-filled.
bool encode_rows(CUtensorMap* map, const void* t, int rows, int heads, int d, long long row_stride, int box_heads,
                 int box_rows) {
    auto fn = cross_encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)row_stride * 2};
    cuuint32_t box[3] = {64, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(t), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace
}  // namespace spec_attn

struct spec_attn_cross_plan {
    spec_attn_cross_problem prob;
    int device;
    int num_sms;
    int nq;
    int wt;
    int tiles;
    int keys_per_split;
    int max_splits;
    float sm_scale;
    spec_attn::CrossVariant variant;
};

namespace {

constexpr int32_t kMaxCrossRows = 1 << 30;

bool cross_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

// Clusters of `size` CTAs that the GPU holds at once: a cluster stays within one group of SMs (GPC), so CTAs that would
// fit singly may not fit as clusters (16 clusters of 8 on 152 SMs: 25.4 us where 16 of 6 take 20.6).
int resident_clusters(const spec_attn::CrossVariant& v, int size, int num_sms) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(size));
    cfg.blockDim = dim3(static_cast<unsigned>(v.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(v.smem);
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(size);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, v.kernel, &cfg) != cudaSuccess || n < 1) {
        cudaGetLastError();
        n = std::max(1, num_sms / size);
    }
    return n * v.ctas;   // (counted at one CTA an SM for kernels with tensor memory)
}

// States a split takes (a multiple of the tile).
int choose_split(const spec_attn_cross_problem& p, int max_rows, int max_len, const spec_attn_cross_plan& plan) {
    const spec_attn::CrossVariant deep = spec_attn::cross_variant(p.head_dim, plan.nq, true);
    const spec_attn::CrossVariant shared = spec_attn::cross_variant(p.head_dim, plan.nq, false);
    const int64_t units = (static_cast<int64_t>(max_len) + spec_attn::kBN - 1) / spec_attn::kBN;
    const int64_t ctas = static_cast<int64_t>(plan.tiles) * p.num_kv_heads * p.num_reqs;
    // Model (us, measured): a CTA has a start and an end, a time for each tile of 64 states (longer beside another CTA
    // with many rows), and with splits the cluster's barriers and the exchange of its rows; the states come from HBM
    // at best at its rate.
    const double rows = std::min(max_rows, plan.nq * plan.wt) * (p.num_q_heads / p.num_kv_heads);
    const double fixed = 3.0, cluster = 1.0 + rows * p.head_dim / 6e3;
    const bool whole = plan.nq == 2 || p.head_dim == 256;
    const double tile_alone = whole ? 0.8 : 0.43, tile_shared = whole ? 0.8 : (p.head_dim == 64 ? 0.3 : 0.45) * (1.0 + rows / 128.0);
    const double hbm = static_cast<double>(p.num_reqs) * max_len * p.num_kv_heads * p.head_dim * 4.0 / 6.5e6;
    double best = 1e300;
    int64_t best_u = units < 1 ? 1 : units;
    for (int64_t s = 1; s <= units && s <= spec_attn::kMaxSplits; ++s) {
        const int64_t u = (units + s - 1) / s, splits = (units + u - 1) / u;
        if (splits < s) continue;                  // (as an earlier s)
        const bool alone = ctas * splits <= plan.num_sms;
        const spec_attn::CrossVariant& v = alone ? deep : shared;
        const int64_t at_once = splits == 1 ? static_cast<int64_t>(plan.num_sms) * v.ctas
                                            : resident_clusters(v, static_cast<int>(splits), plan.num_sms);
        const int64_t waves = (ctas + at_once - 1) / at_once;
        const double cta = fixed + static_cast<double>(u) * (alone ? tile_alone : tile_shared) + (splits > 1 ? cluster : 0.0);
        const double cost = std::max(static_cast<double>(waves) * cta, hbm + fixed);
        if (cost < best * 0.98) {
            best = cost;
            best_u = u;
        }
    }
    return static_cast<int>(best_u * spec_attn::kBN);
}

}  // namespace

extern "C" {

int spec_attn_cross_plan_create(const spec_attn_cross_problem* problem, spec_attn_cross_plan** out,
                                size_t* workspace_bytes) {
    if (!out) return SPEC_ATTN_E_INVALID_ARG;
    *out = nullptr;
    if (!problem) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_cross_problem& p = *problem;
    if (p.num_reqs < 0 || p.total_q_rows < 0 || p.max_q_rows < 1 || p.num_q_heads <= 0 || p.num_kv_heads <= 0 ||
        p.num_q_heads % p.num_kv_heads != 0 || p.head_dim <= 0 || p.total_kv_rows < 0 || p.max_kv_len < 0 ||
        p.force_splits < 0 || !(p.sm_scale >= 0.f) || std::isinf(p.sm_scale))
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.head_dim != 64 && p.head_dim != 128 && p.head_dim != 256) return SPEC_ATTN_E_UNSUPPORTED;
    const int G = p.num_q_heads / p.num_kv_heads;
    if (p.force_splits > spec_attn::kMaxSplits || G > SPEC_ATTN_MAX_GROUP || p.num_reqs > 65535 || p.num_kv_heads > 65535)
        return SPEC_ATTN_E_UNSUPPORTED;
    // (2^30 rows of the smallest head are 128 GiB of K: a limit that keeps every index of the kernel in 32 bits)
    if (p.total_q_rows > kMaxCrossRows || p.total_kv_rows > kMaxCrossRows) return SPEC_ATTN_E_UNSUPPORTED;
    const int64_t dense = static_cast<int64_t>(p.num_kv_heads) * p.head_dim;
    if (p.kv_row_stride != 0 && (p.kv_row_stride < dense || p.kv_row_stride % 8 != 0)) return SPEC_ATTN_E_INVALID_ARG;
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return spec_attn::record_cuda_error(e);
    spec_attn_cross_plan* plan = new (std::nothrow) spec_attn_cross_plan();
    if (!plan) return SPEC_ATTN_E_INVALID_ARG;
    plan->prob = p;
    if (p.kv_row_stride == 0) plan->prob.kv_row_stride = dense;
    // bounds beyond the rows there are (INT32_MAX for "any") size nothing
    const int max_rows = std::max(1, std::min(p.max_q_rows, p.total_q_rows));
    const int max_len = std::min(p.max_kv_len, p.total_kv_rows);
    plan->device = dev;
    plan->num_sms = sms;
    plan->sm_scale = p.sm_scale > 0.f ? p.sm_scale : 1.0f / std::sqrt(static_cast<float>(p.head_dim));
    plan->wt = 128 / G;
    // Two query tiles a CTA read K and V once for both, but make half as many CTAs: for d = 128, where one-tile CTAs
    // would not fit the SMs at once (32/8 heads x 128: 377 instead of 401 us at 4096 x 4096 for two requests, 18.8
    // instead of 19.6 at 1000 x 1000; below, 17.5 instead of 26 us with one tile at 2 x 200 x 1500).  At d = 64 two
    // one-tile CTAs an SM are faster throughout (16/8 heads, 4096 x 4096, two requests: 162 instead of 190 us).
    const int64_t one_tile = (static_cast<int64_t>(max_rows) + plan->wt - 1) / plan->wt * p.num_kv_heads * p.num_reqs;
    plan->nq = p.head_dim == 128 && max_rows > plan->wt && one_tile > sms ? 2 : 1;
    plan->tiles = static_cast<int>((static_cast<int64_t>(max_rows) + plan->nq * plan->wt - 1) / (plan->nq * plan->wt));
    for (const bool deep : {true, false}) {
        const spec_attn::CrossVariant v = spec_attn::cross_variant(p.head_dim, plan->nq, deep);
        e = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
        if (e != cudaSuccess) {
            delete plan;
            return spec_attn::record_cuda_error(e);
        }
    }
    if (p.force_splits > 0) {
        const int64_t units = (static_cast<int64_t>(max_len) + spec_attn::kBN - 1) / spec_attn::kBN;
        const int64_t u = (units + p.force_splits - 1) / p.force_splits;
        plan->keys_per_split = static_cast<int>((u < 1 ? 1 : u) * spec_attn::kBN);
    } else {
        plan->keys_per_split = choose_split(p, max_rows, max_len, *plan);
    }
    plan->max_splits = max_len == 0 ? 1 : (max_len - 1) / plan->keys_per_split + 1;
    if (static_cast<int64_t>(plan->tiles) * plan->max_splits > INT32_MAX) {
        delete plan;
        return SPEC_ATTN_E_UNSUPPORTED;
    }
    plan->variant = spec_attn::cross_variant(
        p.head_dim, plan->nq, static_cast<int64_t>(plan->tiles) * plan->max_splits * p.num_kv_heads * p.num_reqs <= sms);
    if (workspace_bytes) *workspace_bytes = 256;
    *out = plan;
    return SPEC_ATTN_OK;
}

int spec_attn_cross_plan_destroy(spec_attn_cross_plan* plan) {
    delete plan;
    return SPEC_ATTN_OK;
}

int spec_attn_run_cross(const spec_attn_cross_plan* plan, const void* q, const void* k, const void* v,
                        const int32_t* q_indptr, const int32_t* kv_start, const int32_t* kv_len, void* o, float* lse,
                        void* workspace, size_t workspace_bytes, spec_attn_stream_t stream_handle) {
    using namespace spec_attn;
    if (!plan) return SPEC_ATTN_E_INVALID_ARG;
    const spec_attn_cross_problem& p = plan->prob;
    if (p.num_reqs == 0 || p.total_q_rows == 0) return SPEC_ATTN_OK;
    if (!q || !o || !q_indptr || !kv_start || !kv_len || !workspace || !cross_aligned(q, 16) || !cross_aligned(o, 16) ||
        !cross_aligned(q_indptr, 4) || !cross_aligned(kv_start, 4) || !cross_aligned(kv_len, 4) ||
        !cross_aligned(lse, 4) || !cross_aligned(workspace, 256))
        return SPEC_ATTN_E_INVALID_ARG;
    if (p.total_kv_rows > 0 && (!k || !v || !cross_aligned(k, 16) || !cross_aligned(v, 16)))
        return SPEC_ATTN_E_INVALID_ARG;
    if (workspace_bytes < 256) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    const uint64_t heads = static_cast<uint64_t>(p.total_q_rows) * p.num_q_heads, reqs4 = 4ull * p.num_reqs;
    const uint64_t state = 2ull * p.num_kv_heads * p.head_dim, step = 2ull * p.kv_row_stride;
    const uint64_t states = static_cast<uint64_t>(p.total_kv_rows);
    const ByteRows out[] = {bytes_at(o, 2 * heads * p.head_dim), bytes_at(lse, 4 * heads), bytes_at(workspace, 256)};
    const ByteRows in[] = {bytes_at(q, 2 * heads * p.head_dim), {k, state, step, states}, {v, state, step, states},
                           bytes_at(q_indptr, reqs4 + 4), bytes_at(kv_start, reqs4), bytes_at(kv_len, reqs4)};
    if (outputs_overlap(out, in)) return SPEC_ATTN_E_INVALID_ARG;
    int dev = -1;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return record_cuda_error(e);
    if (dev != plan->device) return SPEC_ATTN_E_INVALID_ARG;

    CrossParams c = {};
    c.q_indptr = q_indptr;
    c.kv_start = kv_start;
    c.kv_len = kv_len;
    c.o = static_cast<uint16_t*>(o);
    c.lse = lse;
    c.status = static_cast<unsigned int*>(workspace);
    c.total_rows = p.total_q_rows;
    c.max_rows = p.max_q_rows;
    c.num_q_heads = p.num_q_heads;
    c.group = p.num_q_heads / p.num_kv_heads;
    c.wt = plan->wt;
    c.max_splits = plan->max_splits;
    // (one request, or all CTAs at once: nothing to order)
    const int64_t ctas = static_cast<int64_t>(plan->tiles) * plan->max_splits * p.num_kv_heads * p.num_reqs;
    c.longest_first = p.num_reqs > 1 && p.num_reqs <= kMaxSorted &&
                              ctas > static_cast<int64_t>(plan->num_sms) * plan->variant.ctas
                          ? p.num_reqs
                          : 0;
    c.total_kv = p.total_kv_rows;
    c.max_kv_len = p.max_kv_len;
    c.keys_per_split = plan->keys_per_split;
    c.score_scale_log2 = plan->sm_scale * 1.4426950408889634f;

    CUtensorMap maps[3] = {};
    auto encode = [&] {
        return encode_rows(&maps[0], q, p.total_q_rows, p.num_q_heads, p.head_dim,
                           static_cast<long long>(p.num_q_heads) * p.head_dim, c.group, c.wt) &&
               encode_rows(&maps[1], k, p.total_kv_rows, p.num_kv_heads, p.head_dim, p.kv_row_stride, 1, kBN) &&
               encode_rows(&maps[2], v, p.total_kv_rows, p.num_kv_heads, p.head_dim, p.kv_row_stride, 1, kBN);
    };
    // (with no state rows at all no copy is made: the maps stay empty)
    if (p.total_kv_rows > 0 && !encode()) {
        // a thread's first CUDA call has no context to encode in yet: bind the device's and try once more
        e = cudaSetDevice(dev);
        if (e != cudaSuccess) return record_cuda_error(e);
        if (!encode()) return SPEC_ATTN_E_INVALID_ARG;
    }
    cudaStream_t stream = reinterpret_cast<cudaStream_t>(stream_handle);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan->tiles * plan->max_splits), static_cast<unsigned>(p.num_kv_heads),
                       static_cast<unsigned>(p.num_reqs));
    cfg.blockDim = dim3(static_cast<unsigned>(plan->variant.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(plan->variant.smem);
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan->max_splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = plan->max_splits > 1 ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, plan->variant.kernel, c, maps[0], maps[1], maps[2]);
    if (e != cudaSuccess) return record_cuda_error(e);
    return SPEC_ATTN_OK;
}

}  // extern "C"
