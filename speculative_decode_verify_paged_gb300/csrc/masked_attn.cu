// Attention over the paged cache under tree masks and under a sliding window with
// sinks (spec_attn_run_masked), windows of any width, bf16 or NVFP4 caches, on
// 5th-generation tensor cores.
//
//   s_j = sm_scale <q, k_j>,  O = sum_j softmax(s)_j v_j,  LSE = ln sum_j exp(s_j)
//
// over the keys a row sees, in one sweep with a running maximum and sum per row
// (base 2, fp32; the weights are rounded to 16 bits for the second product, the sum
// adds them unrounded).
//
// One CTA = (NQ query tiles of 128 rows) x (one KV head) x (a split of the keys).  A
// tile holds 128 / G whole window rows with their G heads, so K and V are read once
// for the G heads; NQ = 2 (d = 128) shares every K and V tile between two query tiles,
// one's products under the other's softmax.  The plan takes the query tiles and the
// splits by a model of the call's time (choose_split).
//
// Keys.  The pages a CTA's rows can see are at most two runs: the sinks' and those
// from its first row's window on.  They are walked as one list of pages, 64 keys a
// tile; pages between the runs are never touched, and only the tile with the seam
// has keys of both.  A row's mask of a tile is 64 bits made from its bounds (lowest
// key of its window, sinks, its own key) and, where the tile reaches into a tree's
// window, two words of its mask row, fetched before the scores are waited for.
// Tiles that every row of a warp sees whole skip it.  V rows that no row of the CTA may
// see are zeroed in shared memory (what lies there may be anything, and 0 x NaN is
// NaN); masked scores are replaced, so K may hold anything there.
//
// Warp roles:
//   warp 0      the query tiles, then the K tiles, by TMA, 128-byte swizzle.  NVFP4:
//               codes by TMA and scales by plain asynchronous copies into a raw ring.
//   warps 1, 2  issue the products, one elected thread each.  NQ = 2: warp 1 + i
//               issues S_{t+1} and then P_t V_t of tile i.  NQ = 1: warp 1 issues
//               S = Q K^T and warp 2 O += P V.
//   warp 3      owns tensor memory; the V tiles.
//   warps 4-7   softmax, a row a thread, and epilogue; 8-11 the same for the second
//               query tile, or for every other key tile of the only one (kStreams).
//   NVFP4: the warps behind them decode K and V into fp16 operand tiles (8 warps at
//               d 256, 4 otherwise, in teams that take the tiles in turn); query rows
//               and weights are fp16 too.
//
// Tensor memory: O tiles [0, NQ d), two or four S buffers of 64 columns a tile, P in the
// first half of its S buffer, and where there is room (one tile, the SM to itself) the
// query tile, which frees its shared memory and doubles the first product's rate.
//
// Epilogue.  Rows wait in shared memory so that they leave in memory order, 16 bytes a
// thread: as bf16 where the CTA's row is the result, else in fp32.
//
// Splits.  Up to 8 of them form a cluster: each leaves its normalised rows in fp32 with
// their log-sum-exps in its own shared memory, and after a cluster barrier every CTA
// combines a share of the rows from its peers' shared memory.  More leave their rows
// in the workspace as fp16 of the row's largest element, or of 2^-126 if that is larger (off
// by at most 2^-12 of it), and a second kernel joins them.  Both in an order that the split
// fixes.
//
// Bound, with times of a launch in a graph.  A tile of 64 keys takes 0.44 us at d 64,
// 0.52 at d 128 (two query tiles: 0.71 for both), 0.75-0.80 at d 256; NVFP4 0.47, 0.53,
// 0.80; a launch starts and ends in 5-8 us beside its tiles.  At d 256 bf16 the copies
// bound it: 64 KB a tile at 43 bytes a clock into an SM (48 nodes over 64K keys 75 us; in
// long loops of calls 79-81, the power limit).
// At d 128 two query tiles keep the tensor cores busy for 1280 of 1490 clocks (a prompt
// of 2049 rows under a window of 2048: 67 us, 1.7 rounds of CTAs taking 2).  NVFP4 is bound
// by the chain scores, softmax, P V beside the decoders (4 trees of 32 nodes over 16384
// keys of d 256: 64 us).  One token of a request reads at 91 % of a copy's rate (64 of
// them under a window of 4096: 153 us).
//
// Every wait is bounded; on time-out the CTA sets the device-status bit, drains its
// copies and products, frees its tensor memory and leaves.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_runtime.h>
#include <float.h>
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
constexpr int kBN = 64;                 // keys a tile
constexpr int kMaxRing = 14;
constexpr int kMaxRaw = 8;
// requests put in order by one CTA's threads, a multiple of 32 (tokens over 100-12000 keys of d 256: 256 of them 238-241 us in
// whatever order they come; 257 as they come 237 to 278)
constexpr int kMaxSorted = 256;
constexpr int kMaxCluster = 8;          // CTAs of a cluster that any GPU schedules
constexpr int kJoinBatch = 16;          // splits whose rows a joining thread has on their way at once (8: 19 splits 15.5 us, not 13.4)
constexpr float kRescale = 8.0f;        // log2 units: O is rescaled when a row's maximum grows by more

struct MaskedParams {
    const int32_t* block_table;
    const int32_t* seq_lens;
    const int32_t* q_indptr;
    const uint32_t* row_mask;   // trees
    const int32_t* positions;   // trees with a window
    uint16_t* o;
    float* lse;
    unsigned int* status;
    float2* ws_ls;              // partials: per split and (row, head): (log2 of the sum, largest |element|, at least FLT_MIN)
    uint16_t* ws_o;             //   and the row's elements over it, fp16
    int total_rows, max_w, num_q_heads, group;
    int page_shift;             // log2(page_size)
    int num_pages, bt_stride, tree, window, sinks, mask_words;
    int wt;                     // window rows of a query tile: 128 / group
    int cta_rows;               // window rows of a CTA: wt, or twice that
    int tiles;                  // CTAs' shares of the widest window
    int tiles_per_split;        // key tiles
    int max_splits;
    int cluster;                // the splits of a CTA's rows form a cluster
    int longest_first;          // requests to put in order of length (0: as they come)
    int test_stall;             // testing: no K is copied
    const uint8_t* k_scales;    // NVFP4
    const uint8_t* v_scales;
    long long scale_page_stride;
    long long max_seq_len;
    float score_scale_log2;     // sm_scale * log2(e) [* k_gscale]
    float out_scale;            // 1 or v_gscale
};

// The pages that window rows [lo, lo + cta_rows) of a request can see, as one list: the sinks' pages, then those from
// `first` on.
struct Span {
    int hi;              // keys from here on are seen by no row
    int base;            // first key of the first row's window
    int first;           // its page
    int sink_pages;
    int pages;
    int tiles;
};
__device__ __forceinline__ Span span_of(const MaskedParams& p, const ReqInfo& ri, int lo) {
    Span s;
    const int per_tile = 64 >> p.page_shift;
    s.hi = p.tree ? ri.len : ri.ctx + min(ri.w, lo + p.cta_rows);
    s.base = p.window ? max(0, ri.ctx + (p.tree ? 0 : lo) - p.window + 1) : 0;
    s.first = s.base >> p.page_shift;
    s.sink_pages = p.window ? min(p.sinks ? ((p.sinks - 1) >> p.page_shift) + 1 : 0, s.first) : 0;
    s.pages = s.sink_pages + ((s.hi - 1) >> p.page_shift) + 1 - s.first;
    s.tiles = (s.pages + per_tile - 1) / per_tile;
    return s;
}

// The keys of a tile's columns: key a + c for columns c < seam, key b + c from there on.
struct Columns {
    int a, b, seam;
    uint64_t low;        // columns before the seam
};
__device__ __forceinline__ uint64_t low_bits(int n) { return n <= 0 ? 0ull : n >= 64 ? ~0ull : (1ull << n) - 1; }
__device__ __forceinline__ Columns columns_of(const Span& s, int page_shift, int tile) {
    Columns c;
    const int v = tile << (6 - page_shift);                // the tile's first page in the list
    if (v >= s.sink_pages) {
        c.a = c.seam = 0;
        c.b = (v - s.sink_pages + s.first) << page_shift;
    } else {
        c.a = v << page_shift;
        c.seam = min(64, (s.sink_pages - v) << page_shift);
        c.b = (s.first << page_shift) - c.seam;
    }
    c.low = low_bits(c.seam);
    return c;
}
// columns whose key is below x
__device__ __forceinline__ uint64_t below(const Columns& c, int x) {
    const uint64_t b = low_bits(x - c.b);
    return c.seam == 0 ? b : (low_bits(x - c.a) & c.low) | (b & ~c.low);
}
// The tiles [lo, hi) of the list that lie within the keys [from, to), behind the seam.  (Made once: the columns of every
// tile and their comparison took 290 of a tile's 1150 clocks.)
struct Tiles {
    int lo, hi;
    __device__ __forceinline__ bool has(int t) const { return t >= lo && t < hi; }
};
__device__ __forceinline__ Tiles tiles_within(const Span& s, int page_shift, int from, int to) {
    const int origin = (s.first - s.sink_pages) << page_shift;     // tile t starts at key origin + 64 t
    const int seam = (s.sink_pages + (64 >> page_shift) - 1) >> (6 - page_shift);
    return {max(seam, (max(from - origin, 0) + kBN - 1) / kBN), to - origin < kBN ? 0 : (to - origin) / kBN};
}
// columns that some row of the CTA may see
__device__ __forceinline__ uint64_t live_columns(const MaskedParams& p, const Span& s, const Columns& c) {
    uint64_t m = below(c, s.hi);
    if (p.window) m &= ~below(c, s.base) | below(c, p.sinks);
    return m;
}

// NVFP4 raw slot: the codes and scales of a tile's 16-key units, K then V.  Codes land on 128-byte boundaries, so a unit's
// scales (d bytes) take at least 128.
template <int D>
struct MaskedRaw {
    static constexpr int kCodes = 16 * D / 2;
    static constexpr int kScales = D < 128 ? 128 : D;
    static constexpr int kKS = 4 * kCodes;                 // offsets inside a slot
    static constexpr int kVC = kKS + 4 * kScales;
    static constexpr int kVS = kVC + 4 * kCodes;
    static constexpr int kSlot = 8 * (kCodes + kScales);
};

// DEEP (d <= 128, one query tile, bf16): the launch has no more CTAs than SMs, and a CTA takes the whole SM; otherwise two
// CTAs share it, one's start, end and waits under the other's work.  d = 256, two tiles and NVFP4 always take the whole SM.
template <int D, bool FP4, int NQ, bool DEEP>
struct MaskedLayout {
    static_assert(NQ == 1 || (D == 128 && DEEP && !FP4), "two O tiles and four S buffers fit 512 columns at d = 128");
    static_assert(DEEP || (!FP4 && D <= 128), "half an SM");
    static constexpr int kChunks = D / 64;
    static constexpr int kQBytes = kM * D * 2;             // one query tile
    static constexpr int kTileBytes = kBN * D * 2;         // one K or V tile
    static constexpr int kAux = 2048;
    static constexpr int kCtas = DEEP ? 1 : 2;
    // Key streams: two softmax warpgroups take the query tile's key tiles in turn, each with an O tile and a running
    // maximum and sum of its own, and their rows are joined at the end.  A lone group is bound by its chain of latencies
    // (barrier, scores, maximum, exponentials, weights, barrier: 950 clocks a tile, of them 350 exponentials).
    static constexpr int kStreams = NQ == 1 && DEEP && D <= 128 ? 2 : 1;
    static constexpr int kGroups = NQ * kStreams;          // softmax warpgroups, and O tiles
    // Layout of a bf16 tile: unit-major, a unit 16 keys, [unit][chunk][16 keys][128 bytes], so that a copy takes a whole unit
    // of V (4 KB at d = 128).  K comes 8 keys a copy, [8 keys' group][chunk][8][128 bytes]: its groups then have one stride
    // and S is a product of 64 columns.  (K in units of 16, S in two products of 32 columns: four copies less a tile, but
    // 1080 clocks of products instead of 640, and 64 single tokens under a window of 4096 took 165 us, not 156.  At d = 64
    // a unit is both.)  Decoded tiles are chunk-major, [chunk][64 keys][128 bytes].
    static constexpr bool kEightK = !FP4 && D >= 128;
    static constexpr bool kUnitV = !FP4;
    static constexpr int kUnit = 16 * D * 2;
    // At d = 256 a chain bounds a tile: scores, softmax, P V, and the next scores into the buffer that P V has read.  P is
    // handed over in halves there, so that P V begins under the second half's exponentials (a tile 0.84 -> 0.79 us, NVFP4
    // 0.85 -> 0.79).
    static constexpr bool kHalves = D == 256;
    static constexpr bool kQT = NQ == 1 && DEEP && (kStreams == 1 || D == 64);   // the query tile in tensor memory
    // S buffers of a tile (a power of two); with four, S_{t+1} does not wait for P V of tile t - 1
    static constexpr int kBufShift = NQ == 1 && DEEP && D <= 128 ? 2 : 1;
    static constexpr int kBufs = 1 << kBufShift;
    static constexpr int kQCol = kGroups * D + NQ * kBufs * kBN;
    static constexpr int kNeed = kQCol + (kQT ? D / 2 : 0);
    static constexpr uint32_t kCols = kNeed <= 256 ? 256u : 512u;   // allocated: a power of two
    static_assert(kNeed <= 512 && kCols * kCtas <= 512, "tensor memory");
    // first column of buffer b of query tile i
    __host__ __device__ static constexpr int s_col(int i, int b) { return kGroups * D + (kBufs * i + b) * kBN; }
    // The ring.  NQ = 1: a slot a tile, each let go as soon as it has been read, the first kRingK slots for K and the rest
    // for V (their producers run apart: a slot that both filled in turn could be a phase further than the one that waits
    // for it can tell).  NQ = 2: a slot holds K_t and V_t, filled and let go together.  A query tile bound for tensor memory
    // lands in the last two V slots.
    static constexpr int kSlotBytes = NQ * kTileBytes;
    static constexpr int kQSmem = kQT ? 0 : NQ * kQBytes;
    static constexpr int kMax = DEEP ? 232448 : 232448 / 2 - 1024;   // 227 KB a CTA, 228 KB an SM (1 KB of each CTA reserved)
    static constexpr int kFit = (kMax - 1024 - kAux - kQSmem) / kSlotBytes;
    static constexpr int kRing = FP4 ? (D == 256 ? 4 : 6) : kFit > kMaxRing ? kMaxRing : kFit;
    static_assert(kRing >= 4, "tiles ahead of the ones in use");
    static constexpr int kRingK = NQ == 2 ? kRing : (kRing + 1) / 2, kRingV = NQ == 2 ? kRing : kRing / 2;
    __host__ __device__ static constexpr int k_slot(int t) { return t % kRingK; }
    __host__ __device__ static constexpr int v_slot(int t) { return NQ == 2 ? t % kRing : kRingK + t % kRingV; }
    static constexpr int kRawFit = (kMax - 1024 - kAux - kQSmem - kRing * kSlotBytes) / MaskedRaw<D>::kSlot;
    static constexpr int kRaw = !FP4 ? 0 : kRawFit > kMaxRaw ? kMaxRaw : kRawFit & ~1;   // (even: a slot is one team's of two)
    static constexpr int kTail = kRing * kSlotBytes + kRaw * MaskedRaw<D>::kSlot;   // ring and raw ring, adjacent
    static constexpr int kSmem = 1024 + kAux + kQSmem + kTail;
    static constexpr int kLead = kBufs;                    // tiles by which S leads P V at most
    static_assert(FP4 || kRingV >= kLead, "V of tile t - kRingV was here when S_t is made");
    // P V barriers in use: one a slot (NQ = 2), or one an S buffer and at least four
    static constexpr int kPv = NQ == 2 ? kRing : 4;
    // the epilogue's rows (fp32, or bytes of bf16), 16 bytes apart beyond their length (no bank conflict), their log2 sums and
    // largest elements
    static constexpr int kRowFloats = D + 4, kRow16 = D * 2 + 16;
    static_assert(kGroups * kM * (kRowFloats + 2) * 4 <= kQSmem + kTail, "epilogue staging");
    // NVFP4: two teams of decoding warps for K and two for V take the tiles in turn.  (What a tile takes a team is mostly
    // waits, stores and the fence behind them, 800 clocks: two teams of a warp at d 128 0.53 us a tile, one of two 0.60.)
    static constexpr int kTeam = D == 256 ? 2 : 1;         // warps of a team
    static constexpr int kDecoder0 = 4 + 4 * kGroups;      // the first of them: K's, then as many of V's
    static constexpr int kThreads = 128 + kGroups * 128 + (FP4 ? 4 * kTeam * 32 : 0);
};

struct MaskedAux {
    uint64_t full[kMaxRing];
    uint64_t empty[kMaxRing];           // NQ = 1
    uint64_t pv_done[2][kMaxRing];      // P_t V_t of tile i done: O, P_t's buffer and (NQ = 2) the slot; by t mod kPv
    uint64_t q_full[2];
    uint64_t q_ready;                   // the query tile is in tensor memory, or converted (four softmax warps)
    uint64_t s_full[2][4];              // [tile][buffer] scores written
    uint64_t p_full[2][4];              // P written over them (four softmax warps)
    uint64_t p_half[2];                 // its first 32 keys (kHalves)
    uint64_t raw_full[kMaxRaw];
    uint64_t raw_empty[kMaxRaw];        // the decoding warps of a tile's K and V
    uint64_t drain[2];
    uint32_t tmem_base;
    int abort;
    // longest-first order: requests of each class of lengths, the class and the place in it of the CTA's, its members, and
    // the CTA's
    int classes[64];
    int chosen_class, chosen_place, request;
    uint32_t members[kMaxSorted / 32];
};
static_assert(sizeof(MaskedAux) <= 2048, "aux region");

// 16 bytes to shared memory, and an arrival on `bar` once this thread's copies so far are there (counted in its initial
// count).
__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_addr(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void prefetch_l1(const void* at) { asm volatile("prefetch.global.L1 [%0];" ::"l"(at)); }
__device__ __forceinline__ void cp_async_wait_all() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Four e4m3 scales (a word's bytes), each as a pair of equal fp16.
__device__ __forceinline__ void e4m3x4_pairs_f16x2(uint32_t w, uint32_t (&s2)[4]) {
    uint32_t lo, hi;
    asm("{ .reg .b16 a, b; mov.b32 {a, b}, %2; cvt.rn.f16x2.e4m3x2 %0, a; cvt.rn.f16x2.e4m3x2 %1, b; }"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
    s2[0] = __byte_perm(lo, 0, 0x1010);
    s2[1] = __byte_perm(lo, 0, 0x3232);
    s2[2] = __byte_perm(hi, 0, 0x1010);
    s2[3] = __byte_perm(hi, 0, 0x3232);
}

// A decoding team's work on a tile: the K or V codes of the raw slot into the fp16 operand tile, chunk-major, 128-byte
// swizzle; columns that no row may see as zeros.  A unit is one key's 64 elements (32 code bytes, 4 scales, one 128-byte
// row); eight consecutive keys run side by side, so that the row stores hit distinct banks.  A thread's keys lie a constant
// apart: with the passes unrolled every address is a constant off one of a few registers (a tile of d 256 0.92 -> 0.85 us).
template <int D, int Threads>
__device__ __forceinline__ void decode_tile(const unsigned char* codes, const unsigned char* scales, unsigned char* tile,
                                            uint64_t live, int dt) {
    using R = MaskedRaw<D>;
    constexpr int CPK = D / 64, kRows = Threads / CPK;   // rows a pass: multiples of 16, so that passes differ by constants
    const int j0 = dt / (8 * CPK) * 8 + (dt & 7), c = (dt >> 3) % CPK, unit = j0 >> 4, sl = j0 & 15;
    const unsigned char* kr = codes + unit * R::kCodes + sl * (D / 2);
    const int w0_at = raw_code_chunk<D>(sl, 2 * c) * 16, w1_at = raw_code_chunk<D>(sl, 2 * c + 1) * 16;
    const unsigned char* sr = scales + unit * R::kScales + sl * (D / 16) + c * 4;
    unsigned char* row = tile + c * (kBN * 128) + j0 * 128;
    int at[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) at[q] = (q ^ (j0 & 7)) << 4;
    const bool whole = live == ~0ull;
#pragma unroll
    for (int i = 0; i < kBN / kRows; ++i) {
        constexpr int kUnits = kRows / 16;
        if (whole || (live >> (j0 + i * kRows) & 1)) {
            const uint4 w0 = *reinterpret_cast<const uint4*>(kr + i * kUnits * R::kCodes + w0_at);
            const uint4 w1 = *reinterpret_cast<const uint4*>(kr + i * kUnits * R::kCodes + w1_at);
            const uint32_t sc4 = *reinterpret_cast<const uint32_t*>(sr + i * kUnits * R::kScales);
            const uint32_t words[8] = {w0.x, w0.y, w0.z, w0.w, w1.x, w1.y, w1.z, w1.w};
            uint32_t s2[4];
            e4m3x4_pairs_f16x2(sc4, s2);
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                uint4 x;
                e2m1x8_f16(words[q], s2[q >> 1], x.x, x.y, x.z, x.w);
                *reinterpret_cast<uint4*>(row + i * kRows * 128 + at[q]) = x;
            }
        } else {
#pragma unroll
            for (int q = 0; q < 8; ++q)
                *reinterpret_cast<uint4*>(row + i * kRows * 128 + at[q]) = make_uint4(0u, 0u, 0u, 0u);
        }
    }
}

template <int D, bool FP4, int NQ, bool DEEP>
__global__ void __launch_bounds__(MaskedLayout<D, FP4, NQ, DEEP>::kThreads, MaskedLayout<D, FP4, NQ, DEEP>::kCtas)
masked_attn_kernel(const __grid_constant__ MaskedParams p, const __grid_constant__ CUtensorMap tmq,
                   const __grid_constant__ CUtensorMap tmk, const __grid_constant__ CUtensorMap tmv) {
    using L = MaskedLayout<D, FP4, NQ, DEEP>;
    using R = MaskedRaw<D>;
    constexpr int PV = L::kPv, RING = L::kRing, SH = L::kBufShift, NB = L::kBufs, KS = L::kStreams;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int split = blockIdx.x % p.max_splits;
    const int tile = p.tiles - 1 - blockIdx.x / p.max_splits;     // (a chain's last rows see the most keys)
    const int kvh = blockIdx.y;
    int r = blockIdx.z;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* smem = reinterpret_cast<unsigned char*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                           ~static_cast<uintptr_t>(1023));
    MaskedAux* aux = reinterpret_cast<MaskedAux*>(smem);
    unsigned char* ring = smem + L::kAux + L::kQSmem;
    unsigned char* raw = ring + RING * L::kSlotBytes;
    unsigned char* sQ = L::kQT ? ring + (RING - 2) * L::kTileBytes : smem + L::kAux;
    volatile int* abort = &aux->abort;

    if (tid == 0) {
        for (int s = 0; s < RING; ++s) {
            mbar_init(&aux->full[s], FP4 ? L::kTeam : NQ);
            mbar_init(&aux->empty[s], 1);
        }
        for (int s = 0; s < L::kRaw; ++s) {
            mbar_init(&aux->raw_full[s], 2 + 64);          // codes by either producer, scales by all their lanes
            mbar_init(&aux->raw_empty[s], 2 * L::kTeam);
        }
        for (int i = 0; i < NQ; ++i) {
            for (int s = 0; s < PV; ++s) mbar_init(&aux->pv_done[i][s], 1);
            mbar_init(&aux->q_full[i], 1);
            for (int b = 0; b < NB; ++b) {
                mbar_init(&aux->s_full[i][b], 1);
                mbar_init(&aux->p_full[i][b], 4);
            }
        }
        mbar_init(&aux->q_ready, 4);
        mbar_init(&aux->p_half[0], 4);
        mbar_init(&aux->p_half[1], 4);
        mbar_init(&aux->drain[0], 1);
        mbar_init(&aux->drain[1], 1);
        aux->abort = 0;
        fence_mbarrier_init();
        fence_proxy_async_smem();
        tma_prefetch_desc(&tmq);
        tma_prefetch_desc(&tmk);
        tma_prefetch_desc(&tmv);
    }
    if (tid < 64) aux->classes[tid] = 0;
    if (warp == 3) tmem_alloc(&aux->tmem_base, L::kCols);
    // up to here the CTA touched only its own resources, while the previous kernel drains
    pdl_wait_primary();
    if (p.longest_first) {
        // More CTAs than the GPU holds: the requests with the most keys go first, so that the last CTAs to start are
        // short ones.  Each CTA picks its own: the lengths are counted in classes, two a power of two, and a class's
        // requests go by index.  (Every length ranked against every other took 3.6 us a CTA for 250 requests.  Finer
        // classes put neighbours of one length side by side, and CTAs that start and end together wait together: 250
        // tokens over 50-900 keys 107 us, not 102.)
        const int limit = p.window ? p.window : INT_MAX;
        int mine = -1;
        __syncthreads();                                   // the counts are zero
        if (tid < p.longest_first) {
            prefetch_l1(p.q_indptr + tid);
            const int len = min(p.seq_lens[tid], limit);
            mine = len <= 0 ? 0 : static_cast<int>(__float_as_uint(static_cast<float>(len)) >> 22) - 253;   // 1 .. 63
            atomicAdd(&aux->classes[mine], 1);
        }
        __syncthreads();
        if (warp == 0) {                                   // a lane two classes, the longest first
            const int first = 63 - 2 * lane, c0 = aux->classes[first], c1 = aux->classes[first - 1], sum = c0 + c1;
            int upto = sum;
#pragma unroll
            for (int s = 1; s < 32; s <<= 1) {
                const int x = __shfl_up_sync(kFullMask, upto, s);
                if (lane >= s) upto += x;
            }
            const int place = static_cast<int>(blockIdx.z) - (upto - sum);
            if (place >= 0 && place < sum) {
                aux->chosen_class = place < c0 ? first : first - 1;
                aux->chosen_place = place < c0 ? place : place - c0;
            }
        }
        __syncthreads();
        const uint32_t among = __ballot_sync(kFullMask, mine == aux->chosen_class);
        if (lane == 0 && warp < kMaxSorted / 32) aux->members[warp] = among;
        __syncthreads();
        if (mine == aux->chosen_class) {
            int before = __popc(among & ((1u << lane) - 1));
            for (int k = 0; k < warp; ++k) before += __popc(aux->members[k]);
            if (before == aux->chosen_place) aux->request = tid;
        }
        __syncthreads();
        r = aux->request;
    }
    ReqInfo ri;
    const bool reporter = tid == 0 && blockIdx.x == 0 && kvh == 0;
    bool active = load_request(p.seq_lens, p.q_indptr, r, p.max_w, p.total_rows, p.max_seq_len,
                               p.bt_stride << p.page_shift, kBN, reporter ? p.status : nullptr, ri);
    const int lo = tile * p.cta_rows;                      // first window row of the CTA
    active = active && lo < ri.w;
    Span span = {};
    int nsplits = 0, T = 0;
    const int t0 = split * p.tiles_per_split;              // its key tiles: T from here on
    if (active) {
        span = span_of(p, ri, lo);
        nsplits = (span.tiles + p.tiles_per_split - 1) / p.tiles_per_split;
        T = min(p.tiles_per_split, span.tiles - t0);
        active = T > 0;
    }
    // The split's pages, 32 at a time in the producers' lanes.  The first are asked for here, so that they come while the CTA
    // meets; only entries of the request's pages are read: a table may end with the last of them.  (Without a window they could
    // be asked for beside the lengths, a round trip earlier, whatever they hold: one tile of d 128 5.08 us, not 5.16.)
    const int32_t* const table = p.block_table + (size_t)r * p.bt_stride;
    const int v0 = t0 << (6 - p.page_shift);               // the split's first page in the list
    const int pages = min(span.pages - v0, T << (6 - p.page_shift));
    auto fetch = [&](int k) {
        if (k >= pages) return 0;
        const int v = v0 + k;
        return ld_volatile_i32(table + (v < span.sink_pages ? v : v - span.sink_pages + span.first));
    };
    int early0 = 0, early1 = 0;
    if (active && (warp == 0 || warp == 3)) {
        early0 = fetch(lane);
        early1 = fetch(32 + lane);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    // The next kernel's CTAs set up as these leave their SMs.  (Not before this CTA has its tensor memory: theirs would
    // hold it while they wait for this grid.)
    pdl_launch_dependents();
    const uint32_t tmem = aux->tmem_base;
    if (!active) {                                         // uniform across the CTA
        if (warp == 3) tmem_dealloc(tmem, L::kCols);
        return;
    }
    const int G = p.group;
    const int nact = (NQ == 2 && lo + p.wt < ri.w) ? 2 : 1;
    const int rows = min(ri.w - lo, p.cta_rows) * G;       // query rows of the CTA, wt * G of them in its first tile
    // products of P V take whole 16-key steps: those of the request's last tile end with its keys
    int last_steps = kBN / 16;
    if (t0 + T == span.tiles) {
        const Columns c = columns_of(span, p.page_shift, t0 + T - 1);
        last_steps = (64 - __clzll(static_cast<long long>(live_columns(p, span, c))) + 15) / 16;
    }
    // row m of the CTA: its place in O and LSE
    // (m / G by its rounded-up reciprocal in 2^-16, exact below 2^12 for G <= 16)
    const unsigned by_g = (65536u + G - 1) / G;
    auto place = [&](unsigned m) {
        const unsigned w = m * by_g >> 16;
        return (size_t)(ri.row0 + lo + w) * p.num_q_heads + kvh * G + (m - w * G);
    };
    auto pair = [](float x, float y) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    };
    // Rows wait in shared memory to leave in memory order: of one stream and one split as bf16 already, otherwise in fp32.
    const bool rounded = KS == 1 && nsplits == 1;
    float* stage = reinterpret_cast<float*>(smem + L::kAux);   // (epilogue)
    float* stage_lse = stage + L::kGroups * kM * L::kRowFloats;
    float* stage_max = stage_lse + L::kGroups * kM;

    if (warp == 0 || warp == 3) {
        // ------------------------------------------------------------ copies: K by warp 0, V by warp 3
        const bool is_v = warp == 3;
        const int todo = p.test_stall && !is_v ? 0 : T;
        int issued = 0;
        const int shift = p.page_shift, per_tile = 64 >> shift;
        auto checked = [&](int k, int page) {
            if (k >= pages || (page >= 0 && page < p.num_pages)) return k < pages ? page : 0;
            atomicOr(p.status, kDevBadPage);
            return 0;
        };
        int cur = early0, next = early1, batch = 0;        // (the next 32 on their way)
        if (warp == 0 && lane == 0) {
            const uint32_t qbytes = static_cast<uint32_t>(L::kChunks * 128 * G * p.wt);
            for (int i = 0; i < nact; ++i) {
                mbar_arrive_expect_tx(&aux->q_full[i], qbytes);
                for (int c = 0; c < L::kChunks; ++c)
                    tma_load_3d(sQ + i * L::kQBytes + c * (kM * 128), &tmq, c * 64, kvh * G, ri.row0 + lo + i * p.wt,
                                &aux->q_full[i]);
            }
        }
        __syncwarp();
        cur = checked(lane, cur);
        auto turn = [&](int k) {                           // k: first page of the tile
            if (k >> 5 == batch) return;
            batch = k >> 5;
            cur = checked(32 * batch + lane, next);
            next = fetch(32 * (batch + 1) + lane);
        };
        if constexpr (FP4) {
            for (int t = 0; t < todo; ++t) {
                const int slot = t % L::kRaw, k = t * per_tile;
                if (t >= L::kRaw && !wait_warp(&aux->raw_empty[slot], ((t / L::kRaw) - 1) & 1, abort)) break;
                turn(k);
                const int units = min(4, min(per_tile, pages - k) << (shift - 4));   // of 16 keys
                uint64_t* bar = &aux->raw_full[slot];
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(units * R::kCodes));
                unsigned char* dst = raw + slot * R::kSlot + (is_v ? R::kVC : 0);
                // The scales, d bytes a unit, by plain asynchronous copies: the copy engine takes some 85 clocks a box whatever
                // its size, and 16 of them a tile were what bound it (d 64 and 128: 0.70 us a tile).
                constexpr int kPieces = D / 16;            // of a unit
#pragma unroll
                for (int x = 0; x < (4 * kPieces + 31) / 32; ++x) {
                    const int piece = x * 32 + lane, u = piece / kPieces, sub = u & ((1 << (shift - 4)) - 1);
                    const int page = __shfl_sync(kFullMask, cur, (k & 31) + (min(u, 3) >> (shift - 4)));
                    if (u < units)
                        cp_async_16(dst + R::kKS + u * R::kScales + piece % kPieces * 16,
                                    (is_v ? p.v_scales : p.k_scales) + page * p.scale_page_stride +
                                        ((((long long)kvh << shift) + sub * 16) * (D / 16) + piece % kPieces * 16));
                }
                cp_async_arrive(bar);
                const int pp = lane & 3, sub = pp & ((1 << (shift - 4)) - 1);
                const int page = __shfl_sync(kFullMask, cur, (k & 31) + (pp >> (shift - 4)));
                __syncwarp();
                if (lane < units) tma_load_4d(dst + pp * R::kCodes, is_v ? &tmv : &tmk, 0, sub * 16, kvh, page, bar);
                __syncwarp();
                issued = t + 1;
            }
        } else {
            // A copy a lane: unit pp of V, the same or half of it of K.  (About 90 clocks a copy and 200 a tile, whatever the
            // sizes; the whole warp issuing them one by one is no faster, and prefetches to L2 are slower.)
            const int halves = !is_v && L::kEightK ? 1 : 0, copies = 4 << halves, pp = lane >> halves;
            const int sub = (pp & ((1 << (shift - 4)) - 1)) * 16 + (lane & halves) * 8, turn_of = min(pp, 3) >> (shift - 4);
            const int first = is_v ? L::v_slot(0) : 0, end = first + (is_v ? L::kRingV : L::kRingK);
            unsigned char* const to = ring + (NQ == 2 && is_v ? L::kTileBytes : 0) + lane * (L::kUnit >> halves);
            const CUtensorMap* const map = is_v ? &tmv : &tmk;
            int slot = first, k = 0;
            uint32_t gone = 1;                             // parity of the phase that lets the slot go (none in the first lap)
            for (int t = 0; t < todo; ++t, k += per_tile) {
                if (t >= end - first) {
                    if (NQ == 1 && !wait_warp(&aux->empty[slot], gone, abort)) break;
                    if (NQ == 2 && !(wait_warp(&aux->pv_done[0][slot], gone, abort) &&
                                     (nact == 1 || wait_warp(&aux->pv_done[1][slot], gone, abort))))
                        break;
                }
                // (the query tile has to leave the last two slots first)
                if (L::kQT && is_v && t == L::kRingV - 2 && !wait_warp(&aux->q_ready, 0, abort)) break;
                turn(k);
                const int page = __shfl_sync(kFullMask, cur, (k & 31) + turn_of);
                const int units = k + per_tile <= pages ? 4 : (pages - k) << (shift - 4);   // of 16 keys
                uint64_t* const bar = &aux->full[slot];
                // (the bytes may come before they are expected: the phase stays open until this arrival)
                if (lane == 0) mbar_arrive_expect_tx(bar, static_cast<uint32_t>(units * L::kUnit));
                if (lane < copies && pp < units) tma_load_5d(to + slot * L::kSlotBytes, map, 0, sub, 0, kvh, page, bar);
                __syncwarp();
                issued = t + 1;
                if (++slot == end) {
                    slot = first;
                    gone ^= 1;
                }
            }
        }
        if (FP4) cp_async_wait_all();
        if (*abort && lane == 0) {
            // every copy in flight lands before the CTA's shared memory goes away
            volatile int no_abort = 0;
            const int ahead = FP4 ? L::kRaw : is_v ? L::kRingV : L::kRingK;
            for (int t = max(0, issued - ahead); t < issued; ++t)
                mbar_wait(FP4 ? &aux->raw_full[t % ahead] : &aux->full[is_v ? L::v_slot(t) : L::k_slot(t)], (t / ahead) & 1,
                          &no_abort, kDrainLimit);
            for (int i = 0; i < nact; ++i) mbar_wait(&aux->q_full[i], 0, &no_abort, kDrainLimit);
        }
        __syncwarp();
    } else if (warp == 1 || (warp == 2 && (NQ == 1 || nact == 2))) {
        // ------------------------------------------------------------ products
        const uint32_t go = elected();
        constexpr uint32_t idesc_s = FP4 ? idesc_f16_f32(kM, kBN, 0, 0) : idesc_bf16_f32(kM, kBN, 0, 0);
        constexpr int kGroup = L::kEightK ? L::kUnit / 2 : 1024;                       // from 8 keys of K to the next
        constexpr uint32_t k_hi = kGroup >> 4 | (kDescHi & ~0x3FFFu);
        constexpr int kChunkStep = (L::kEightK ? 1024 : kBN * 128) >> 4;
        constexpr int kVStep = (L::kUnitV ? L::kUnit : 2048) >> 4;                     // 16 keys of V further
        constexpr uint32_t idesc_o = FP4 ? idesc_f16_f32(kM, D, 0, 1) : idesc_bf16_f32(kM, D, 0, 1);
        const int i = NQ == 2 ? warp - 1 : 0;
        const uint32_t q_lo = desc_lo(smem_addr(sQ + i * L::kQBytes), 16);
        const uint32_t k_lo0 = desc_lo(smem_addr(ring), 16), v_lo0 = desc_lo(smem_addr(ring), L::kUnitV ? 2048 : kBN * 128);
        auto wait = [&](uint64_t* bar, uint32_t parity) { return wait_warp(bar, parity, abort); };
        // the ring slots of K_t and V_t, and the slot t mod kPv, stepped along with the parity of their phase
        struct Step {
            int first, end, slot;
            uint32_t par;
            __device__ __forceinline__ void next() {
                if (++slot == end) {
                    slot = first;
                    par ^= 1;
                }
            }
        };
        Step ks = {0, L::kRingK, 0, 0}, vs = {L::v_slot(0), L::v_slot(0) + L::kRingV, L::v_slot(0), 0};
        Step done = {0, PV, 0, 0}, before = {0, PV, 0, 0};   // (before: t - lead of the next S)
        // S_t, once K_t is here and the P that sat in S_t's buffer has been read
        auto do_s = [&](int t) {
            const int b = t & (NB - 1);
            if (t >= L::kLead) {
                if (!wait(&aux->pv_done[i][before.slot], before.par)) return false;
                before.next();
            }
            if (!wait(&aux->full[ks.slot], ks.par)) return false;
            tc_fence_after();
            const uint32_t k_lo = k_lo0 + ks.slot * (L::kSlotBytes >> 4), d_tmem = tmem + L::s_col(i, b);
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
                const uint32_t k_at = k_lo + (kk >> 2) * kChunkStep + (kk & 3) * 2;
                if (L::kQT) mma_ts_lo(d_tmem, tmem + L::kQCol + kk * 8, k_at, idesc_s, kk > 0, go, k_hi);
                else mma_ss_lo(d_tmem, q_lo + (kk >> 2) * (kM * 128 >> 4) + (kk & 3) * 2, k_at, idesc_s, kk > 0, go, k_hi);
            }
            commit_if(&aux->s_full[i][b], go);
            if (NQ == 1) commit_if(&aux->empty[ks.slot], go);
            ks.next();
            return true;
        };
        // O += P_t V_t, once both are here (NQ = 2: V_t came with K_t)
        auto do_pv = [&](int t) {
            const int b = t & (NB - 1);
            if (NQ == 1 && !wait(&aux->full[vs.slot], vs.par)) return false;
            if (!wait(L::kHalves ? &aux->p_half[b] : &aux->p_full[i][b], (t >> SH) & 1)) return false;
            tc_fence_after();
            const uint32_t v_lo = v_lo0 + (vs.slot * L::kSlotBytes + (NQ - 1) * L::kTileBytes) / 16;
            const uint32_t p_tmem = tmem + L::s_col(i, b), o_tmem = tmem + (KS == 2 ? t & 1 : i) * D;
            const int steps = t == T - 1 ? last_steps : kBN / 16;
#pragma unroll
            for (int kk = 0; kk < kBN / 16; ++kk) {
                if (L::kHalves && kk == kBN / 32) {
                    if (!wait(&aux->p_full[i][b], (t >> SH) & 1)) return false;
                    tc_fence_after();
                }
                if (kk < steps) mma_ts_lo(o_tmem, p_tmem + kk * 8, v_lo + kk * kVStep, idesc_o, t >= KS || kk > 0, go);
            }
            commit_if(&aux->pv_done[i][done.slot], go);
            if (NQ == 1) commit_if(&aux->empty[vs.slot], go);
            vs.next();
            done.next();
            return true;
        };
        bool ok = true;
        if (NQ == 2 || warp == 1) ok = wait(L::kQT || FP4 ? &aux->q_ready : &aux->q_full[i], 0);
        tc_fence_after();
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
    } else if (FP4 && warp >= L::kDecoder0) {
        // ------------------------------------------------------------ NVFP4: K and V into operand tiles
        const bool is_v = warp >= L::kDecoder0 + 2 * L::kTeam;
        const Tiles whole = tiles_within(span, p.page_shift, span.base, span.hi);
        for (int t = warp / L::kTeam & 1; t < T; t += 2) {
            const int slot = is_v ? L::v_slot(t) : L::k_slot(t), lap = t / (is_v ? L::kRingV : L::kRingK), rs = t % max(1, L::kRaw);
            const uint64_t live = whole.has(t0 + t) ? ~0ull : live_columns(p, span, columns_of(span, p.page_shift, t0 + t));
            if (!wait_warp(&aux->raw_full[rs], (t / max(1, L::kRaw)) & 1, abort)) break;
            if (lap > 0 && !wait_warp(&aux->empty[slot], (lap - 1) & 1, abort)) break;
            // (the query tile has to leave the last two slots first)
            if (L::kQT && is_v && t >= L::kRingV - 2 && t < L::kRingV && !wait_warp(&aux->q_ready, 0, abort)) break;
            const unsigned char* src = raw + rs * R::kSlot;
            decode_tile<D, L::kTeam * 32>(src + (is_v ? R::kVC : 0), src + (is_v ? R::kVS : R::kKS), ring + slot * L::kTileBytes,
                                          live, tid & (L::kTeam * 32 - 1));
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&aux->full[slot]);
                mbar_arrive(&aux->raw_empty[rs]);
            }
        }
    } else if (warp >= 4 && (warp < 8 || nact == 2 || KS == 2)) {
        // ------------------------------------------------------------ softmax and epilogue
        const int g = warp >= 8 ? 1 : 0;                   // group: a query tile's, or a key stream's
        const int i = NQ == 2 ? g : 0;                     // query tile
        const int m = (warp & 3) * 32 + lane;              // row of the tile
        const uint32_t lane_tmem = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const int wrow = lo + i * p.wt + m / G;            // window row
        const bool valid = m < p.wt * G && wrow < ri.w;
        // a warp without rows leaves its scores as they are: they weigh on no other row
        const bool live = __any_sync(kFullMask, valid);
        bool ok = true;
        if (L::kQT && g == 0) {
            // the query row into tensor memory, two elements a column; NVFP4: as fp16 (saturating; exact for magnitudes of
            // 2^-14 to 65504).  Rows that are none are zeros.
            if ((ok = wait_warp(&aux->q_full[0], 0, abort))) {
                const uint32_t row = smem_addr(sQ) + m * 128;
#pragma unroll 1
                for (int c = 0; c < L::kChunks; ++c) {
                    uint32_t w[32];
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        uint4 v = make_uint4(0u, 0u, 0u, 0u);
                        if (valid) v = ld_shared_v4(row + c * (kM * 128) + ((q ^ (m & 7)) << 4));
                        w[4 * q + 0] = FP4 ? bf16x2_to_f16x2_sat(v.x) : v.x;
                        w[4 * q + 1] = FP4 ? bf16x2_to_f16x2_sat(v.y) : v.y;
                        w[4 * q + 2] = FP4 ? bf16x2_to_f16x2_sat(v.z) : v.z;
                        w[4 * q + 3] = FP4 ? bf16x2_to_f16x2_sat(v.w) : v.w;
                    }
                    __syncwarp();
                    tmem_st32u(lane_tmem + L::kQCol + c * 32, w);
                }
                tmem_wait_st();
                fence_proxy_async_smem();                  // (the slots are written by copies next)
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&aux->q_ready);
            }
        }
        if (FP4 && !L::kQT && g == 0) {
            // the query row to fp16 in its place (as above)
            if ((ok = wait_warp(&aux->q_full[0], 0, abort))) {
                const uint32_t row = smem_addr(sQ) + m * 128;
#pragma unroll 1
                for (int c = 0; c < L::kChunks; ++c) {
#pragma unroll
                    for (int q = 0; q < 8; ++q) {
                        const uint32_t at = row + c * (kM * 128) + ((q ^ (m & 7)) << 4);
                        const uint4 v = valid ? ld_shared_v4(at) : make_uint4(0u, 0u, 0u, 0u);
                        st_shared_v4(at, make_uint4(bf16x2_to_f16x2_sat(v.x), bf16x2_to_f16x2_sat(v.y),
                                                    bf16x2_to_f16x2_sat(v.z), bf16x2_to_f16x2_sat(v.w)));
                    }
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&aux->q_ready);
            }
        }
        // the row's bounds: context keys from `from` (or below the sinks) to `to`
        int to = INT_MAX, from = 0;
        const uint32_t* mask_row = nullptr;
        if (valid) {
            const int row = ri.row0 + wrow;
            int pos = ri.ctx + wrow;
            if (p.tree) {
                pos = p.window ? max(ri.ctx, p.positions[row]) : ri.ctx;
                mask_row = p.row_mask + (size_t)row * p.mask_words;
            }
            to = p.tree ? ri.ctx : pos + 1;
            if (p.window) from = max(0, pos - p.window + 1);
            if (p.tree) from = min(from, ri.ctx);
        }
        // tiles that every row of the warp sees whole
        const Tiles whole = tiles_within(span, p.page_shift, max(span.base, __reduce_max_sync(kFullMask, from)),
                                         min(span.hi, __reduce_min_sync(kFullMask, to)));
        const float sc = p.score_scale_log2;
        float m_ref = -INFINITY, l_sum = 0.f;
        const uint64_t sc2 = pack2(sc, sc);
        for (int t = KS == 2 ? g : 0; t < T && ok; t += KS) {
            const int b = t & (NB - 1);
            uint64_t sees = ~0ull, dead = 0;
            if (!whole.has(t0 + t)) {
                const Columns col = columns_of(span, p.page_shift, t0 + t);
                if (valid) {
                    sees = below(col, to);
                    if (p.window) sees &= ~below(col, from) | below(col, p.sinks);
                    const int off = col.b - ri.ctx;        // the window's key at column 0, or how many context keys precede it
                    if (p.tree && off > -kBN) {
                        const int o = max(off, 0), at = o >> 5, n = p.mask_words;
                        const uint32_t w0 = at < n ? mask_row[at] : 0u, w1 = at + 1 < n ? mask_row[at + 1] : 0u;
                        const uint32_t w2 = at + 2 < n ? mask_row[at + 2] : 0u;
                        uint64_t bits = static_cast<uint64_t>(__funnelshift_r(w1, w2, o & 31)) << 32 |
                                        __funnelshift_r(w0, w1, o & 31);
                        if (off < 0) bits <<= -off;
                        sees |= bits & ~col.low & below(col, ri.len);
                    }
                }
                if (!FP4) dead = ~live_columns(p, span, col) & low_bits((t == T - 1 ? last_steps : kBN / 16) * 16);
            }
            const uint32_t s_tmem = lane_tmem + L::s_col(i, b);
            if (!(ok = wait_warp(&aux->s_full[i][b], (t >> SH) & 1, abort))) break;
            tc_fence_after();
            if (!FP4 && dead) {
                // V rows that no row of the CTA may see.  (P V of tile t - lead is done, or S_t could not have been made, and with
                // it the slot's earlier tile was here: the parity names this phase.  Both tiles' warps write the same zeros.)
                constexpr int C8 = L::kChunks * 8;         // 16-byte pieces of a row
                const int slot = L::v_slot(t);
                if (!(ok = wait_warp(&aux->full[slot], (t / L::kRingV) & 1, abort))) break;
                const uint32_t v_addr = smem_addr(ring + slot * L::kSlotBytes + (NQ - 1) * L::kTileBytes);
                for (int u = m; u < kBN * C8; u += 128)
                    if ((dead >> (u / C8)) & 1)
                        st_shared_v4(v_addr + (u / C8 >> 4) * L::kUnit + ((u % C8) >> 3) * 2048 + (u / C8 & 15) * 128 + (u & 7) * 16,
                                     make_uint4(0u, 0u, 0u, 0u));
                fence_proxy_async_smem();
            }
            // what the warp has stored, and the V rows it has zeroed, before its arrival
            auto hand_over = [&](uint64_t* bar) {
                if (live) tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(bar);
            };
            if (live) {
                __syncwarp();
                float sv[kBN];
                tmem_ld32(s_tmem, *reinterpret_cast<float(*)[32]>(sv));
                tmem_ld32(s_tmem + 32, *reinterpret_cast<float(*)[32]>(sv + 32));
                tmem_wait_ld();
                if (!__all_sync(kFullMask, sees == ~0ull)) {
                    const uint32_t s0 = static_cast<uint32_t>(sees), s1 = static_cast<uint32_t>(sees >> 32);
#pragma unroll
                    for (int c = 0; c < 32; ++c) {
                        sv[c] = s0 >> c & 1 ? sv[c] : -INFINITY;
                        sv[32 + c] = s1 >> c & 1 ? sv[32 + c] : -INFINITY;
                    }
                }
                float mx4[4] = {sv[0], sv[1], sv[2], sv[3]};
#pragma unroll
                for (int c = 4; c < kBN; c += 8) {   // (three-way maxima)
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        mx4[k] = fmaxf(fmaxf(mx4[k], sv[c + k]), c + 4 < kBN ? sv[c + 4 + k] : mx4[k]);
                }
                const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * sc;
                // the reference moves at the first key seen, and when the maximum outgrows it
                const bool need = mx > m_ref + kRescale;
                const float ref = need ? mx : m_ref;
                const float alpha = need ? fast_exp2(m_ref - ref) : 1.f;   // (0 at the first)
                // (an infinite reference is not subtracted: inf - inf would hide in the sum what the scores were.  Plus
                // infinity makes the sum and with it the log-sum-exp infinite, and O, times 1 / inf, NaN.)
                const float nref = fabsf(ref) == INFINITY ? 0.f : -ref;
                const uint64_t nref2 = pack2(nref, nref);
                // (beside a row's 64 scores, 128 registers a thread leave room for 8 columns without spills)
                constexpr int kCols = FP4 && L::kHalves ? 8 : 32;
                auto rescale = [&] {
                    if (t < KS || !__any_sync(kFullMask, valid && need)) return true;
                    // every earlier P V of the O tile has to be in
                    if (!wait_warp(&aux->pv_done[i][(t - KS) % PV], ((t - KS) / PV) & 1, abort)) return false;
                    tc_fence_after();
                    __syncwarp();
#pragma unroll 1
                    for (int ch = 0; ch < D / kCols; ++ch) {
                        uint32_t ov[kCols];
                        const uint32_t at = lane_tmem + g * D + ch * kCols;
                        if constexpr (kCols == 8) tmem_ld8u(at, ov);
                        else tmem_ld32(at, reinterpret_cast<float(&)[kCols]>(ov));
                        tmem_wait_ld();
#pragma unroll
                        for (int e = 0; e < kCols; ++e) ov[e] = __float_as_uint(__uint_as_float(ov[e]) * alpha);
                        if constexpr (kCols == 8) tmem_st8u(at, ov);
                        else tmem_st32u(at, ov);
                    }
                    return true;
                };
                if (L::kHalves && !(ok = rescale())) break;
                uint32_t pk[kBN / 2];
                uint64_t ps[2] = {0, 0};   // two fp32 zeros each
#pragma unroll
                for (int c = 0; c < kBN; c += 2) {
                    if (L::kHalves && c == kBN / 2) {
                        tmem_st16u(s_tmem, pk);
                        hand_over(&aux->p_half[b]);
                        __syncwarp();
                    }
                    const float2 x = unpack2(fma2(pack2(sv[c], sv[c + 1]), sc2, nref2));
                    const float p0 = fast_exp2(x.x), p1 = fast_exp2(x.y);
                    ps[(c >> 1) & 1] = add2(ps[(c >> 1) & 1], pack2(p0, p1));
                    if constexpr (FP4) {
                        pk[c >> 1] = pack_half2(p0, p1);
                    } else {
                        const __nv_bfloat162 h2 = __floats2bfloat162_rn(p0, p1);
                        pk[c >> 1] = *reinterpret_cast<const uint32_t*>(&h2);
                    }
                }
                const float2 psum = unpack2(add2(ps[0], ps[1]));
                l_sum = l_sum * alpha + (psum.x + psum.y);
                m_ref = ref;
                if (!L::kHalves && !(ok = rescale())) break;
                if (L::kHalves) tmem_st16u(s_tmem + 16, pk + 16);
                else tmem_st32u(s_tmem, pk);
            } else if (L::kHalves) {
                hand_over(&aux->p_half[b]);
            }
            hand_over(&aux->p_full[i][b]);
        }
        // every product is done: the query tiles and the ring are free.  (A stream that does not have the last tile waits
        // for its own first: P V is done in order, so that the last one's parity names its phase.)
        if (KS == 2 && ok && T >= 2 && (T - 1 - g) % 2 != 0)
            ok = wait_warp(&aux->pv_done[i][(T - 2) % PV], ((T - 2) / PV) & 1, abort);
        for (int j = 0; j < NQ; ++j)
            if (ok && j < nact) ok = wait_warp(&aux->pv_done[j][(T - 1) % PV], ((T - 1) / PV) & 1, abort);
        tc_fence_after();
        const int sr = (KS == 2 ? g * kM : i * p.wt * G) + m;       // (rows past the tile's wt * G are not written)
        float* row = stage + sr * L::kRowFloats;
        if (KS == 2) {                                     // the streams' maxima and sums meet behind their rows' elements
            if (ok) *reinterpret_cast<float2*>(row + D) = make_float2(m_ref, l_sum);
            named_barrier_sync(1, 2 * kM);
        }
        if (ok) {
            unsigned char* row16 = reinterpret_cast<unsigned char*>(stage) + sr * L::kRow16;
            float inv, lse;
            if (KS == 2) {
                const float2 other = *reinterpret_cast<const float2*>(stage + (sr ^ kM) * L::kRowFloats + D);
                const float mx = fmaxf(m_ref, other.x), ref = fabsf(mx) == INFINITY ? 0.f : mx;   // (as in the softmax)
                const float own = fast_exp2(m_ref - ref), sum = fmaf(l_sum, own, other.y * fast_exp2(other.x - ref));
                inv = sum == 0.f ? 0.f : own * (p.out_scale / sum);
                lse = mx + log2f(sum);
            } else {
                inv = l_sum == 0.f ? 0.f : p.out_scale / l_sum;
                lse = m_ref + log2f(l_sum);
            }
            float most = 0.f;
            if (live) {
#pragma unroll 1
                for (int ch = 0; ch < D / 32; ch += 2) {
                    float ov[64];
                    tmem_ld32(lane_tmem + g * D + ch * 32, *reinterpret_cast<float(*)[32]>(ov));
                    tmem_ld32(lane_tmem + g * D + ch * 32 + 32, *reinterpret_cast<float(*)[32]>(ov + 32));
                    tmem_wait_ld();
                    if (KS == 2 && g >= T) {               // (a stream without tiles: its O tile was never written)
#pragma unroll
                        for (int e = 0; e < 64; ++e) ov[e] = 0.f;
                    }
                    if (valid && rounded) {
#pragma unroll
                        for (int e = 0; e < 64; e += 8)
                            *reinterpret_cast<uint4*>(row16 + (ch * 32 + e) * 2) =
                                make_uint4(pair(ov[e] * inv, ov[e + 1] * inv), pair(ov[e + 2] * inv, ov[e + 3] * inv),
                                           pair(ov[e + 4] * inv, ov[e + 5] * inv), pair(ov[e + 6] * inv, ov[e + 7] * inv));
                    } else if (valid) {
#pragma unroll
                        for (int e = 0; e < 64; e += 4) {
                            const float4 x = make_float4(ov[e] * inv, ov[e + 1] * inv, ov[e + 2] * inv, ov[e + 3] * inv);
                            if (KS == 1) most = fmaxf(fmaxf(most, fmaxf(fabsf(x.x), fabsf(x.y))), fmaxf(fabsf(x.z), fabsf(x.w)));
                            *reinterpret_cast<float4*>(row + ch * 32 + e) = x;
                        }
                    }
                    __syncwarp();   // the next load takes the whole warp at once
                }
            }
            if (valid) {
                stage_lse[sr] = lse;
                if (KS == 1) stage_max[sr] = most;
            }
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
    const bool clustered = p.cluster && nsplits > 1;
    if (rounded) {
        if (!*abort) {
            constexpr int C8 = D / 8, kAtOnce = 4;
            const int pieces = rows * C8;
            for (int u0 = tid; u0 < pieces; u0 += kAtOnce * L::kThreads) {
                uint4 x[kAtOnce];
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int u = u0 + k * L::kThreads;
                    if (u < pieces)
                        x[k] = *reinterpret_cast<const uint4*>(reinterpret_cast<const unsigned char*>(stage) +
                                                               u / C8 * L::kRow16 + u % C8 * 16);
                }
#pragma unroll
                for (int k = 0; k < kAtOnce; ++k) {
                    const int u = u0 + k * L::kThreads, m = u / C8, c = u % C8;
                    if (u >= pieces) break;
                    const size_t at = place(m);
                    st_global_v4(p.o + at * D + c * 8, x[k]);
                    if (c == 0 && p.lse) p.lse[at] = stage_lse[m] * kLn2;
                }
            }
        }
    } else if (!*abort && !(clustered && KS == 1)) {
        constexpr int C8 = D / 8, kAtOnce = 4;             // pieces of 8 elements; a thread's loads before its first store
        const size_t part = (size_t)split * p.total_rows * p.num_q_heads;
        const int pieces = rows * C8;
        for (int u0 = tid; u0 < pieces; u0 += kAtOnce * L::kThreads) {
            float4 a[kAtOnce], b[kAtOnce];
            float lse[kAtOnce];
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int u = u0 + k * L::kThreads, m = u / C8, c = u % C8;
                if (u >= pieces) break;
                const float4* src = reinterpret_cast<const float4*>(stage + m * L::kRowFloats + c * 8);
                // (a piece is two 16-byte words; every other four lanes take the second first, so that eight lanes' reads hit
                // distinct banks)
                const int first = c >> 2 & 1;
                a[k] = src[first];
                b[k] = src[first ^ 1];
                lse[k] = stage_lse[m];
                if (KS == 2) {
                    const float4* other = src + kM * L::kRowFloats / 4;
                    const float4 a1 = other[first], b1 = other[first ^ 1];
                    a[k] = make_float4(a[k].x + a1.x, a[k].y + a1.y, a[k].z + a1.z, a[k].w + a1.w);
                    b[k] = make_float4(b[k].x + b1.x, b[k].y + b1.y, b[k].z + b1.z, b[k].w + b1.w);
                }
                if (first) {
                    const float4 x = a[k];
                    a[k] = b[k];
                    b[k] = x;
                }
            }
#pragma unroll
            for (int k = 0; k < kAtOnce; ++k) {
                const int u = u0 + k * L::kThreads, m = u / C8, c = u % C8;
                if (u >= pieces) break;
                if (clustered) {                           // (the rows stay here for the cluster)
                    float4* to = reinterpret_cast<float4*>(stage + m * L::kRowFloats + c * 8);
                    to[0] = a[k];
                    to[1] = b[k];
                    continue;
                }
                const size_t at = place(m);
                if (nsplits == 1) {
                    st_global_v4(p.o + at * D + c * 8, make_uint4(pair(a[k].x, a[k].y), pair(a[k].z, a[k].w),
                                                                  pair(b[k].x, b[k].y), pair(b[k].z, b[k].w)));
                    if (c == 0 && p.lse) p.lse[at] = lse[k] * kLn2;
                } else {
                    // the row's largest element; of two streams' joined row, whose parts may cancel, by the lanes that hold it
                    float most = KS == 2 ? 0.f : stage_max[m];
                    if (KS == 2) {
                        most = fmaxf(fmaxf(fmaxf(fabsf(a[k].x), fabsf(a[k].y)), fmaxf(fabsf(a[k].z), fabsf(a[k].w))),
                                     fmaxf(fmaxf(fabsf(b[k].x), fabsf(b[k].y)), fmaxf(fabsf(b[k].z), fabsf(b[k].w))));
                        // (a row's C8 pieces are in as many neighbouring lanes, which go on or leave together)
                        const unsigned lanes = static_cast<unsigned>(low_bits(C8)) << (lane & ~(C8 - 1));
#pragma unroll
                        for (int x = 1; x < C8; x <<= 1) most = fmaxf(most, __shfl_xor_sync(lanes, most, x));
                    }
                    // (at least the smallest normal number: its reciprocal is finite, where 1 / 2^-129 would make infinities of
                    // the row's elements and NaN of its zeros)
                    most = fmaxf(most, FLT_MIN);
                    const float s = 1.f / most;
                    st_global_v4(p.ws_o + (part + at) * D + c * 8,
                                 make_uint4(pack_half2(a[k].x * s, a[k].y * s), pack_half2(a[k].z * s, a[k].w * s),
                                            pack_half2(b[k].x * s, b[k].y * s), pack_half2(b[k].z * s, b[k].w * s)));
                    if (c == 0) p.ws_ls[part + at] = make_float2(lse[k], most);
                }
            }
        }
    }
    if (!clustered) return;
    __syncwarp();
    cluster_sync();                                        // every split's rows are in its shared memory
    if (!*abort) {
        auto combine = [&](auto most) {
            constexpr int N = decltype(most)::value, C4 = D / 4;
            // Every load of a unit is on its way before the first is used, and each CTA begins with its own rows.
            uint32_t rows_at[N], lse_at[N];
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const int rank = split + k < nsplits ? split + k : split + k - nsplits;
                rows_at[k] = peer_addr(smem_addr(stage), k < nsplits ? rank : split);
                lse_at[k] = peer_addr(smem_addr(stage_lse), k < nsplits ? rank : split);
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
                // (N is the least of 2, 4 and 8 that holds the splits: those past the middle may not be there)
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
                const float inv = sum == 0.f ? 0.f : 1.f / sum;
                *reinterpret_cast<uint2*>(p.o + place(m) * D + c * 4) =
                    make_uint2(pair(a.x * inv, a.y * inv), pair(a.z * inv, a.w * inv));
                if (c == 0 && p.lse) p.lse[place(m)] = (mx + log2f(sum)) * kLn2;
            }
        };
        if (nsplits <= 2) combine(std::integral_constant<int, 2>());
        else if (nsplits <= 4) combine(std::integral_constant<int, 4>());
        else combine(std::integral_constant<int, kMaxCluster>());
    }
    __syncwarp();
    cluster_sync();                                        // no CTA leaves while its rows are being read
}

// Joins the splits' rows: O = sum_s 2^(lse_s - lse) O_s, in split order.  A thread an 8-element piece of a (row, head).
template <int D>
__global__ void __launch_bounds__(256) masked_join_kernel(const __grid_constant__ MaskedParams p) {
    constexpr int C8 = D / 8, kBatch = kJoinBatch;
    pdl_wait_primary();
    pdl_launch_dependents();
    ReqInfo ri;
    if (!load_request(p.seq_lens, p.q_indptr, blockIdx.y, p.max_w, p.total_rows, p.max_seq_len,
                      p.bt_stride << p.page_shift, kBN, nullptr, ri))
        return;
    const long long u = (long long)blockIdx.x * 256 + threadIdx.x;
    const int wrow = static_cast<int>(u / (p.num_q_heads * C8));
    if (wrow >= ri.w) return;
    const Span s = span_of(p, ri, wrow / p.cta_rows * p.cta_rows);
    const int n = (s.tiles + p.tiles_per_split - 1) / p.tiles_per_split;
    if (n == 1) return;
    const size_t at = (size_t)ri.row0 * p.num_q_heads + u / C8, step = (size_t)p.total_rows * p.num_q_heads;
    const int c = static_cast<int>(u % C8);
    float acc[8] = {}, mx = -INFINITY, sum = 0.f;
    for (int s0 = 0; s0 < n; s0 += kBatch) {
        float2 ls[kBatch];
        uint4 x[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (s0 + k >= n) break;
            ls[k] = p.ws_ls[at + (s0 + k) * step];
            x[k] = *reinterpret_cast<const uint4*>(p.ws_o + (at + (s0 + k) * step) * D + c * 8);
        }
        float m2 = mx;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (s0 + k < n) m2 = fmaxf(m2, ls[k].x);
        const float ref = fabsf(m2) == INFINITY ? 0.f : m2;   // (as in the softmax)
        const float a = m2 > mx ? fast_exp2(mx - ref) : 1.f;
        sum *= a;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= a;
        mx = m2;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (s0 + k >= n) break;
            const float w = fast_exp2(ls[k].x - ref), ws = w * ls[k].y;
            sum += w;
            const uint32_t h[4] = {x[k].x, x[k].y, x[k].z, x[k].w};
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const float2 f = unpack_half2(h[e]);
                acc[2 * e] = fmaf(ws, f.x, acc[2 * e]);
                acc[2 * e + 1] = fmaf(ws, f.y, acc[2 * e + 1]);
            }
        }
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    uint32_t out[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(acc[2 * e] * inv, acc[2 * e + 1] * inv);
        out[e] = *reinterpret_cast<const uint32_t*>(&h);
    }
    st_global_v4(p.o + at * D + c * 8, make_uint4(out[0], out[1], out[2], out[3]));
    if (c == 0 && p.lse) p.lse[at] = (mx + log2f(sum)) * kLn2;
}

using MaskedKernel = void (*)(const MaskedParams, const CUtensorMap, const CUtensorMap, const CUtensorMap);
using JoinKernel = void (*)(const MaskedParams);

// What a launch of (d, cache type, query tiles a CTA) needs.
struct MaskedVariant {
    MaskedKernel kernel;
    int threads, smem, ctas;   // ctas: on one SM
    int keys_k;                // keys of a copy of K (bf16)
    int streams;               // key streams
};
template <int D, bool FP4, int NQ, bool DEEP>
MaskedVariant variant_of() {
    using L = MaskedLayout<D, FP4, NQ, DEEP>;
    return {&masked_attn_kernel<D, FP4, NQ, DEEP>, L::kThreads, L::kSmem, L::kCtas, L::kEightK ? 8 : 16, L::kStreams};
}
MaskedVariant masked_variant(int d, bool fp4, int nq, bool deep) {
    if (fp4) return d == 64 ? variant_of<64, true, 1, true>() : d == 128 ? variant_of<128, true, 1, true>() : variant_of<256, true, 1, true>();
    if (d == 256) return variant_of<256, false, 1, true>();
    if (nq == 2) return variant_of<128, false, 2, true>();
    if (d == 64) return deep ? variant_of<64, false, 1, true>() : variant_of<64, false, 1, false>();
    return deep ? variant_of<128, false, 1, true>() : variant_of<128, false, 1, false>();
}

PFN_cuTensorMapEncodeTiled_v12000 masked_encode_fn() {
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

bool encode(CUtensorMap* map, CUtensorMapDataType type, int rank, const void* at, const cuuint64_t* dims,
            const cuuint64_t* strides, const cuuint32_t* box, CUtensorMapSwizzle swizzle) {
    auto fn = masked_encode_fn();
    const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    return fn && fn(map, type, static_cast<cuuint32_t>(rank), const_cast<void*>(at), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Q [rows, Hq, d] bf16 as (element, head, row); box = 64 elements x G heads x wt rows.
bool encode_q(CUtensorMap* map, const void* q, int rows, int hq, int d, int group, int wt) {
    const cuuint64_t dims[] = {(cuuint64_t)d, (cuuint64_t)hq, (cuuint64_t)rows};
    const cuuint64_t strides[] = {(cuuint64_t)d * 2, (cuuint64_t)d * 2 * hq};
    const cuuint32_t box[] = {64, (cuuint32_t)group, (cuuint32_t)wt};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, q, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// A bf16 pool as (64 elements, slot, 64-element chunk, head, page); box = `keys` keys of a head with all their chunks.
bool encode_units(CUtensorMap* map, const void* pool, const spec_attn_masked_problem& p, int keys) {
    const cuuint64_t row = (cuuint64_t)p.head_dim * 2, ps = (cuuint64_t)p.page_size, chunks = (cuuint64_t)p.head_dim / 64;
    const cuuint64_t dims[] = {64, ps, chunks, (cuuint64_t)p.num_kv_heads, (cuuint64_t)p.num_pages};
    const cuuint64_t strides[] = {row, 128, row * ps, (cuuint64_t)p.kv_page_stride};
    const cuuint32_t box[] = {64, (cuuint32_t)keys, (cuuint32_t)chunks, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 5, pool, dims, strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// An NVFP4 code pool as (byte, slot, head, page); box = a head's codes of 16 keys, swizzled 128/64/32 bytes for d = 256/128/64
// (the row is d/2 bytes).
bool encode_codes(CUtensorMap* map, const void* pool, const spec_attn_masked_problem& p) {
    const cuuint64_t row = (cuuint64_t)p.head_dim / 2, ps = (cuuint64_t)p.page_size;
    const cuuint64_t dims[] = {row, ps, (cuuint64_t)p.num_kv_heads, (cuuint64_t)p.num_pages};
    const cuuint64_t strides[] = {row, row * ps, (cuuint64_t)p.kv_page_stride};
    const cuuint32_t box[] = {(cuuint32_t)row, 16, 1, 1};
    const CUtensorMapSwizzle sw = p.head_dim == 256   ? CU_TENSOR_MAP_SWIZZLE_128B
                                  : p.head_dim == 128 ? CU_TENSOR_MAP_SWIZZLE_64B
                                                      : CU_TENSOR_MAP_SWIZZLE_32B;
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, pool, dims, strides, box, sw);
}

bool masked_aligned(const void* p, size_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

}  // namespace
}  // namespace spec_attn

struct spec_attn_masked_plan {
    spec_attn_masked_problem prob;
    int device;
    int num_sms;
    int nq;
    int wt;
    int tiles;
    int tiles_per_split;
    int max_splits;
    int longest_first;
    int test_stall;
    float sm_scale;
    size_t workspace_bytes;
    spec_attn::MaskedVariant variant;
};

namespace {

// Clusters of `size` CTAs that the GPU holds at once (a cluster stays within one group of SMs).
int64_t resident_clusters(const spec_attn::MaskedVariant& v, int size, int num_sms) {
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
    return static_cast<int64_t>(n) * v.ctas;   // (counted at one CTA an SM for kernels with tensor memory)
}

struct MaskedChoice {
    double cost;
    int tiles_per_split;
};

// Key tiles a split takes with nq query tiles a CTA, of `units` at most (and `mean` of it over the CTAs: a prompt's rows see
// half its own keys), and a figure (us) to rank the choices by: a CTA has a start and an end that grow with its rows, and a
// time for each tile of 64 keys (longer beside another CTA with many rows); splits add their combination, in the cluster or by a
// second kernel; the keys come from HBM at best at its rate.  Its parts were fitted to measurements; as a prediction it is up
// to a third too high (64 tokens under a window of 4096 200 us, measured 152), in part since all lengths count as the longest.
MaskedChoice choose_split(const spec_attn_masked_problem& p, int64_t units, double mean, int rows, int nq, int num_sms) {
    const bool fp4 = p.kv_dtype == SPEC_ATTN_KV_NVFP4;
    const spec_attn::MaskedVariant deep = spec_attn::masked_variant(p.head_dim, fp4, nq, true);
    const spec_attn::MaskedVariant shared = spec_attn::masked_variant(p.head_dim, fp4, nq, false);
    const int group = p.num_q_heads / p.num_kv_heads, wt = nq * (128 / group), d = p.head_dim;
    const int64_t ctas = static_cast<int64_t>((rows - 1) / wt + 1) * p.num_kv_heads * p.num_reqs;
    const double cta_rows = std::min(rows, wt) * group, part = cta_rows * d / 16384.0;
    const bool whole = nq == 2 || fp4 || d == 256;
    const double fixed_alone = nq == 2 ? 12.0 : 4.3 + (fp4 ? 2.4 : 2.0) * part, cluster = 1.1 + 1.1 * part;
    const double fixed_shared = whole ? fixed_alone : fixed_alone + 3.5 * part * part;
    const double tile_alone = nq == 2    ? 0.71
                              : d == 256 ? 0.79
                              : fp4      ? (d == 64 ? 0.47 : 0.53)
                              : d == 64  ? 0.44
                                         : 0.46 + 0.12 * part;
    const double tile_shared = whole ? tile_alone : (d == 64 ? 0.33 : 0.42) * (1.0 + cta_rows / 128.0);
    const double hbm = static_cast<double>(p.num_reqs) * units * 64 * p.num_kv_heads * (fp4 ? d * 1.125 : d * 4.0) / 6.2e6;
    MaskedChoice best = {1e300, static_cast<int>(units)};
    for (int64_t s = 1; s <= units && s <= 128; ++s) {
        const int64_t u = (units + s - 1) / s, splits = (units + u - 1) / u;
        if (splits < s) continue;                  // (as an earlier s)
        const bool alone = ctas * splits <= num_sms;
        const spec_attn::MaskedVariant& v = alone ? deep : shared;
        const int64_t slots = static_cast<int64_t>(num_sms) * v.ctas;
        const int64_t at_once = splits == 1                        ? slots
                                : splits <= spec_attn::kMaxCluster ? resident_clusters(v, static_cast<int>(splits), num_sms)
                                                                   : std::max<int64_t>(1, slots / splits);
        const double waves = std::ceil(static_cast<double>(ctas) * (splits > 1 ? mean : 1.0) / static_cast<double>(at_once));
        const double tiles = static_cast<double>(u) * (splits == 1 && waves > 1.0 ? mean : 1.0);
        const double cta = alone ? fixed_alone + tiles * tile_alone : fixed_shared + tiles * tile_shared;
        const int64_t batches = (splits + spec_attn::kJoinBatch - 1) / spec_attn::kJoinBatch;
        const double join = splits == 1                        ? 0.0
                            : splits <= spec_attn::kMaxCluster ? cluster
                                                               : 2.1 + 0.95 * batches + static_cast<double>(splits) * p.num_reqs * rows * p.num_q_heads * d * 4.0 / 1e7;
        // (HBM's time and the SMs' overlap, not wholly)
        const double inside = waves * cta, outside = hbm + fixed_alone;
        const double cost = std::max(inside, outside) + 0.3 * std::min(inside, outside) + join;
        if (cost < best.cost * 0.98) best = {cost, static_cast<int>(u)};
    }
    return best;
}

}  // namespace

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
    int dev = 0, sms = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return spec_attn::record_cuda_error(e);
    spec_attn_masked_plan* plan = new (std::nothrow) spec_attn_masked_plan();
    if (!plan) return SPEC_ATTN_E_INVALID_ARG;
    plan->prob = p;
    if (p.kv_page_stride == 0) plan->prob.kv_page_stride = page;
    if (p.scale_page_stride == 0) plan->prob.scale_page_stride = scale_page;
    if (p.mask_row_words == 0) plan->prob.mask_row_words = words;
    plan->device = dev;
    plan->num_sms = sms;
    plan->sm_scale = p.sm_scale > 0.f ? p.sm_scale : 1.0f / std::sqrt(static_cast<float>(p.head_dim));
    // bounds beyond the rows and pages there are (INT32_MAX for "any") size nothing
    const int rows = std::max(1, std::min(p.max_w, p.total_q_rows));
    const int64_t max_len = std::max<int64_t>(1, std::min(p.max_seq_len, static_cast<int64_t>(p.block_table_stride) * p.page_size));
    plan->wt = 128 / (p.num_q_heads / p.num_kv_heads);
    // most key tiles of a CTA of `reach` window rows (as span_of counts them)
    auto most_tiles = [&](int cta_rows) {
        int64_t pages = (max_len + p.page_size - 1) / p.page_size;
        if (p.window_left > 0) {
            const int64_t reach = static_cast<int64_t>(p.window_left) - 1 + (p.tree ? rows : std::min(rows, cta_rows));
            pages = std::min(pages, (static_cast<int64_t>(p.sink_keys) + p.page_size - 1) / p.page_size + reach / p.page_size + 2);
        }
        return (pages * p.page_size + spec_attn::kBN - 1) / spec_attn::kBN;
    };
    const double mean = p.tree || p.window_left > 0 ? 1.0 : 1.0 - 0.5 * std::min(1.0, static_cast<double>(rows) / max_len);
    // Two query tiles a CTA (d = 128, bf16) read K and V once for both, but make half as many CTAs: the model decides.
    spec_attn::MaskedVariant v;
    MaskedChoice best = {1e300, 1};
    plan->nq = 1;
    for (int nq = 1; nq <= (p.head_dim == 128 && !fp4 && rows > plan->wt ? 2 : 1); ++nq) {
        for (const bool deep : {true, false}) {
            v = spec_attn::masked_variant(p.head_dim, fp4, nq, deep);
            e = cudaFuncSetAttribute(v.kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, v.smem);
            if (e != cudaSuccess) {
                delete plan;
                return spec_attn::record_cuda_error(e);
            }
        }
        const MaskedChoice c = choose_split(p, most_tiles(nq * plan->wt), mean, rows, nq, sms);
        if (c.cost < best.cost) {
            best = c;
            plan->nq = nq;
        }
    }
    const int cta_rows = plan->nq * plan->wt;
    const int64_t units = most_tiles(cta_rows);
    plan->tiles = (rows - 1) / cta_rows + 1;
    plan->tiles_per_split = p.force_splits > 0 ? static_cast<int>((units + p.force_splits - 1) / p.force_splits) : best.tiles_per_split;
    plan->max_splits = static_cast<int>((units - 1) / plan->tiles_per_split) + 1;
    if (static_cast<int64_t>(plan->tiles) * plan->max_splits > INT32_MAX) {
        delete plan;
        return SPEC_ATTN_E_UNSUPPORTED;
    }
    const int64_t ctas = static_cast<int64_t>(plan->tiles) * plan->max_splits * p.num_kv_heads * p.num_reqs;
    plan->variant = spec_attn::masked_variant(p.head_dim, fp4, plan->nq, ctas <= sms);
    // Longest first: where the CTAs come in rounds.  It takes a CTA 0.4 us and more and shortens the last round's tail, so not
    // for many rounds of short CTAs (64 tokens over 1-3000 keys 78 -> 71 us, 250 over 50-900 keys 91 -> 102), and not beyond
    // kMaxSorted requests.
    const int64_t at_once = static_cast<int64_t>(sms) * plan->variant.ctas;
    plan->longest_first = p.num_reqs > 1 && p.num_reqs <= spec_attn::kMaxSorted && ctas > at_once &&
                                  plan->tiles_per_split * at_once >= 8 * ctas
                              ? p.num_reqs
                              : 0;
    // partials: the pairs of every split, then their elements (a multiple of 256 bytes each)
    const size_t pairs = static_cast<size_t>(plan->max_splits) * p.total_q_rows * p.num_q_heads;
    plan->workspace_bytes = 256 + (plan->max_splits > spec_attn::kMaxCluster ? (pairs * 8 + 255) / 256 * 256 + pairs * p.head_dim * 2 : 0);
    if (workspace_bytes) *workspace_bytes = plan->workspace_bytes;
    *out = plan;
    return SPEC_ATTN_OK;
}

int spec_attn_masked_plan_destroy(spec_attn_masked_plan* plan) {
    delete plan;
    return SPEC_ATTN_OK;
}

int spec_attn_masked_plan_get_info(const spec_attn_masked_plan* plan, spec_attn_masked_plan_info* info) {
    if (!plan || !info) return SPEC_ATTN_E_INVALID_ARG;
    *info = {};
    info->query_tiles = plan->nq;
    info->key_streams = plan->variant.streams;
    info->ctas_per_sm = plan->variant.ctas;
    info->tiles_per_split = plan->tiles_per_split;
    info->max_splits = plan->max_splits;
    info->join = plan->max_splits == 1 ? 0 : plan->max_splits <= spec_attn::kMaxCluster ? 1 : 2;
    info->longest_first = plan->longest_first > 0;
    info->grid_x = plan->tiles * plan->max_splits;
    info->grid_y = plan->prob.num_kv_heads;
    info->grid_z = plan->prob.num_reqs;
    info->block_threads = plan->variant.threads;
    info->smem_bytes = plan->variant.smem;
    info->num_sms = plan->num_sms;
    info->workspace_bytes = plan->workspace_bytes;
    return SPEC_ATTN_OK;
}

int spec_attn_masked_plan_set_test_stall(spec_attn_masked_plan* plan, int stall) {
    if (!plan || (stall != 0 && stall != 1)) return SPEC_ATTN_E_INVALID_ARG;
    plan->test_stall = stall;
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
    if (workspace_bytes < plan->workspace_bytes) return SPEC_ATTN_E_WORKSPACE_TOO_SMALL;
    if (p.num_reqs == 0 || p.total_q_rows == 0) return SPEC_ATTN_OK;
    if (!q || !o || !k_pool || !v_pool || (fp4 && (!k_scales || !v_scales)) || !seq_lens || !q_indptr ||
        (p.block_table_stride > 0 && !block_table) || (p.tree && !row_mask) || (p.tree && p.window_left > 0 && !positions))
        return SPEC_ATTN_E_INVALID_ARG;
    if (fp4 && (!(k_gscale > 0.f) || !(v_gscale > 0.f) || std::isinf(k_gscale) || std::isinf(v_gscale)))
        return SPEC_ATTN_E_INVALID_ARG;
    // (the scale of the scores in base 2: as 0 or infinity it would make NaN of masked and of zero scores)
    const float score_scale = plan->sm_scale * 1.4426950408889634f * (fp4 ? k_gscale : 1.f);
    if (!(score_scale > 0.f) || std::isinf(score_scale)) return SPEC_ATTN_E_INVALID_ARG;
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
    const ByteRows out[] = {bytes_at(o, 2 * heads * p.head_dim), bytes_at(lse, 4 * heads), bytes_at(workspace, plan->workspace_bytes)};
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
    m.block_table = block_table;
    m.seq_lens = seq_lens;
    m.q_indptr = q_indptr;
    m.row_mask = reinterpret_cast<const uint32_t*>(row_mask);
    m.positions = positions;
    m.o = static_cast<uint16_t*>(o);
    m.lse = lse;
    m.status = static_cast<unsigned int*>(workspace);
    const size_t pairs = static_cast<size_t>(plan->max_splits) * rows * p.num_q_heads;
    m.ws_ls = reinterpret_cast<float2*>(static_cast<unsigned char*>(workspace) + 256);
    m.ws_o = reinterpret_cast<uint16_t*>(static_cast<unsigned char*>(workspace) + 256 + (pairs * 8 + 255) / 256 * 256);
    m.total_rows = p.total_q_rows;
    m.max_w = p.max_w;
    m.num_q_heads = p.num_q_heads;
    m.group = p.num_q_heads / p.num_kv_heads;
    m.page_shift = p.page_size == 64 ? 6 : p.page_size == 32 ? 5 : 4;
    m.num_pages = p.num_pages;
    m.bt_stride = p.block_table_stride;
    m.tree = p.tree;
    m.window = p.window_left;
    m.sinks = p.sink_keys;
    m.mask_words = p.mask_row_words;
    m.wt = plan->wt;
    m.cta_rows = plan->nq * plan->wt;
    m.tiles = plan->tiles;
    m.tiles_per_split = plan->tiles_per_split;
    m.max_splits = plan->max_splits;
    m.cluster = plan->max_splits > 1 && plan->max_splits <= kMaxCluster;
    m.longest_first = plan->longest_first;
    m.test_stall = plan->test_stall;
    m.k_scales = static_cast<const uint8_t*>(k_scales);
    m.v_scales = static_cast<const uint8_t*>(v_scales);
    m.scale_page_stride = p.scale_page_stride;
    m.max_seq_len = p.max_seq_len;
    m.score_scale_log2 = score_scale;
    m.out_scale = fp4 ? v_gscale : 1.f;

    CUtensorMap maps[3] = {};
    auto encode_all = [&] {
        return encode_q(&maps[0], q, p.total_q_rows, p.num_q_heads, p.head_dim, m.group, plan->wt) &&
               (fp4 ? encode_codes(&maps[1], k_pool, p) : encode_units(&maps[1], k_pool, p, plan->variant.keys_k)) &&
               (fp4 ? encode_codes(&maps[2], v_pool, p) : encode_units(&maps[2], v_pool, p, 16));
    };
    if (!encode_all()) {
        // a thread's first CUDA call has no context to encode in yet: bind the device's and try once more
        e = cudaSetDevice(dev);
        if (e != cudaSuccess) return record_cuda_error(e);
        if (!encode_all()) return SPEC_ATTN_E_INVALID_ARG;
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(plan->tiles * plan->max_splits), static_cast<unsigned>(p.num_kv_heads),
                       static_cast<unsigned>(p.num_reqs));
    cfg.blockDim = dim3(static_cast<unsigned>(plan->variant.threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(plan->variant.smem);
    cfg.stream = reinterpret_cast<cudaStream_t>(stream);
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(plan->max_splits);
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = m.cluster ? 2 : 1;
    e = cudaLaunchKernelEx(&cfg, plan->variant.kernel, m, maps[0], maps[1], maps[2]);
    if (e != cudaSuccess) return record_cuda_error(e);
    if (plan->max_splits > kMaxCluster) {
        const JoinKernel join = p.head_dim == 64    ? &masked_join_kernel<64>
                                : p.head_dim == 128 ? &masked_join_kernel<128>
                                                    : &masked_join_kernel<256>;
        const int64_t pieces = static_cast<int64_t>(std::min(p.max_w, p.total_q_rows)) * p.num_q_heads * (p.head_dim / 8);
        cfg.gridDim = dim3(static_cast<unsigned>((pieces + 255) / 256), static_cast<unsigned>(p.num_reqs));
        cfg.blockDim = dim3(256);
        cfg.dynamicSmemBytes = 0;   // (numAttrs is 1 here: the splits were no cluster)
        e = cudaLaunchKernelEx(&cfg, join, m);
        if (e != cudaSuccess) return record_cuda_error(e);
    }
    return SPEC_ATTN_OK;
}

}  // extern "C"
