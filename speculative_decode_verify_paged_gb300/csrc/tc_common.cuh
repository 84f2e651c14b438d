// Device helpers of the tensor-core kernels: bounded mbarrier waits, products
// issued under a predicate, the block-table load, NVFP4 decode by the hardware
// converts, and the drain of copies in flight.
#pragma once

#include <limits.h>
#include <stdint.h>

#include <cuda_fp16.h>

#include "common.cuh"
#include "sm100.cuh"

namespace spec_attn {
namespace tcc {

using namespace sm100;

// A 32-bit global load the compiler keeps in program order (not sunk past later loads).
__device__ __forceinline__ int ld_volatile_i32(const int32_t* p) {
    int v;
    asm volatile("ld.global.nc.s32 %0, [%1];" : "=r"(v) : "l"(p));
    return v;
}

constexpr long long kWaitLimit = 2000000000LL;   // ~1 s of SM cycles
constexpr long long kDrainLimit = 200000000LL;
constexpr int kPageListCap = 64;                 // page ids staged in shared memory at a time (2 per lane)
constexpr int kNoPrefetch = INT_MIN;             // the producer fetches its first page ids itself

// Warp-uniform bounded wait (all 32 lanes leave together).
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort) {
    const long long t0 = clock64();
    while (true) {
        const bool ok = mbar_try_wait(bar, parity);
        if (__all_sync(kFullMask, ok)) return true;
        const bool give_up = (*abort != 0) || (clock64() - t0 > kWaitLimit);
        if (__any_sync(kFullMask, give_up)) {
            *abort = 1;
            return false;
        }
    }
}

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
// `b_hi`: the high word of B's descriptor.
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc, bool accumulate,
                                          uint32_t go, uint32_t b_hi = kDescHi) {
    asm volatile(
        "{\n\t.reg .pred p, g;\n\t.reg .b64 a, b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 g, %6, 0;\n\t"
        "mov.b64 a, {%1, %5};\n\t"
        "mov.b64 b, {%2, %7};\n\t"
        "@g tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(kDescHi), "r"(go), "r"(b_hi)
        : "memory");
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc, bool accumulate,
                                          uint32_t go, uint32_t b_hi = kDescHi) {
    asm volatile(
        "{\n\t.reg .pred p, g;\n\t.reg .b64 b;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "setp.ne.b32 g, %6, 0;\n\t"
        "mov.b64 b, {%2, %5};\n\t"
        "@g tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate ? 1 : 0), "r"(b_hi), "r"(go)
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

// Position of 16-byte code chunk ch (of D / 32) within key sl's row of a page's
// codes in the raw ring.  The TMA copies them with the 128/64/32-byte swizzle
// of d = 256/128/64 (16-byte chunk index XOR address bits 7..9), which places
// one chunk of 8 consecutive keys in 8 different 16-byte bank groups.
template <int D>
__device__ __forceinline__ int raw_code_chunk(int sl, int ch) {
    return D == 256 ? (ch ^ (sl & 7)) : D == 128 ? (ch ^ ((sl >> 1) & 3)) : (ch ^ ((sl >> 2) & 1));
}

// Decode of NVFP4 K/V into fp16 MMA operands.  cvt.rn.f16x2.e2m1x2 turns one
// code byte (two e2m1 values, the low nibble into the low half) into an fp16
// pair and cvt.rn.f16x2.e4m3x2 one scale byte into (s, s); the products (at most
// 5 significant bits, magnitudes 2^-10 .. 2688) are exact in fp16.
__device__ __forceinline__ uint32_t e4m3_pair_f16x2(uint32_t byte) {
    uint32_t d;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(d) : "h"(static_cast<unsigned short>(byte * 0x0101u)));
    return d;
}
// 8 e2m1 codes (one 32-bit word) times the fp16 scale pair s2, as 4 fp16 pairs.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t s2, uint32_t& o0, uint32_t& o1, uint32_t& o2,
                                           uint32_t& o3) {
    uint32_t a0, a1, a2, a3;
    asm("{ .reg .b8 b0, b1, b2, b3; mov.b32 {b0, b1, b2, b3}, %4; "
        "cvt.rn.f16x2.e2m1x2 %0, b0; cvt.rn.f16x2.e2m1x2 %1, b1; "
        "cvt.rn.f16x2.e2m1x2 %2, b2; cvt.rn.f16x2.e2m1x2 %3, b3; }"
        : "=r"(a0), "=r"(a1), "=r"(a2), "=r"(a3)
        : "r"(w));
    const __half2 s = *reinterpret_cast<const __half2*>(&s2);
    __half2 h;
    h = __hmul2(*reinterpret_cast<const __half2*>(&a0), s); o0 = *reinterpret_cast<const uint32_t*>(&h);
    h = __hmul2(*reinterpret_cast<const __half2*>(&a1), s); o1 = *reinterpret_cast<const uint32_t*>(&h);
    h = __hmul2(*reinterpret_cast<const __half2*>(&a2), s); o2 = *reinterpret_cast<const uint32_t*>(&h);
    h = __hmul2(*reinterpret_cast<const __half2*>(&a3), s); o3 = *reinterpret_cast<const uint32_t*>(&h);
}

template <int NSLOT>
__device__ __forceinline__ void drain_copies(uint64_t* full, int issued) {
    // let every copy still in flight land before the CTA's shared memory goes away
    for (int t = max(0, issued - NSLOT); t < issued; ++t) {
        volatile int no_abort = 0;
        mbar_wait(&full[t % NSLOT], (t / NSLOT) & 1, &no_abort, kDrainLimit);
    }
}

}  // namespace tcc
}  // namespace spec_attn
