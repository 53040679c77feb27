// Parts of the persistent tensor-core kernels (mx_linear.cu, linear_tc.cu): election, bounded waits and what follows one
// that runs out, rings, copies and commits of pairs of blocks.
#pragma once

#include "ptx.cuh"
#include "tc.cuh"

namespace lora {

// One lane of a full warp, the same at every call.  The tensor-core and copy instructions take
// their operands from uniform registers.  So the copying and issuing warps run their loops and
// waits as whole warps, whose counters the compiler then keeps there, and elect a lane around
// the instructions alone.  Measured: an MMA of N = 16 issued every 59 clocks behind `lane == 0`, every 38 (its
// own time) behind an election; with the loop inside the elected branch each stage of four still cost
// about 470 clocks of register moves.
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

// A kernel's bounded waits.  The first that runs out says so in `stop`, a word of the block's shared memory (of both
// blocks' where a pair works together): every wait that goes on ends too, and the teardown, which all warps reach, lets what
// is under way come to rest before the block goes.
struct Bound {
    uint32_t stop;
    unsigned limit;   // tries
    int32_t *status;
};
__device__ __forceinline__ uint32_t stopped(uint32_t stop) {
    uint32_t r;
    asm volatile("ld.relaxed.cluster.shared::cta.u32 %0, [%1];\n" : "=r"(r) : "r"(stop));
    return r;
}
// Wait of a whole warp, uniform for all its lanes: for warps that copy and issue.
__device__ __forceinline__ bool uniform_wait(uint32_t bar, unsigned parity, const Bound &w, bool &failed) {
    if (__all_sync(FULL, mbar_try<false>(bar, parity))) return true;
    for (unsigned it = 1; it < w.limit && !__any_sync(FULL, stopped(w.stop)); ++it)
        if (__all_sync(FULL, mbar_try<false>(bar, parity))) return true;
    failed = true;
    return false;
}
// The same, lane by lane: for warps that move scales and sums.  As a uniform_wait theirs took 1 x 4096 x 4096 5.46 -> 5.56 us
// and 8192 x 4096 x 4096 in MXFP4 65.8 -> 69.0.
__device__ __forceinline__ bool lanes_wait(uint32_t bar, unsigned parity, const Bound &w, bool &failed) {
    bool ok = false;
    for (unsigned it = 0; it < w.limit; ++it) {
        if ((ok = mbar_try<false>(bar, parity))) break;
        if (stopped(w.stop)) break;
    }
    ok = __all_sync(FULL, ok);
    if (!ok) failed = true;
    return ok;
}
// A warp's part has ended: after a wait of its own that ran out, or that another's stopped.  first: the pair's first rank.
template <bool PAIR>
__device__ __forceinline__ void leave(const Bound &w, bool failed, uint32_t first = 0) {
    if (failed && elect_one()) {
        atomicOr(w.status, LORA_DEV_TIMEOUT);
        if (PAIR) {
#pragma unroll
            for (uint32_t k = 0; k < 2; ++k)
                asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;\n" ::"r"(map_rank(w.stop, first + k)) : "memory");
        } else {
            asm volatile("st.relaxed.cluster.shared::cta.u32 [%0], 1;\n" ::"r"(w.stop) : "memory");
        }
    }
}
// Wait of the teardown after a wait that ran out: for copies and products in flight, which end by themselves.
__device__ __forceinline__ void rest_wait(uint32_t bar, unsigned parity) {
    for (unsigned it = 0; it < 1024 && !__all_sync(FULL, mbar_try<false>(bar, parity)); ++it) {}
}
__device__ __forceinline__ void mbar_complete_tx(uint32_t bar, unsigned bytes) {   // as a copy of so many bytes would
    asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;\n" ::"r"(bar), "r"(bytes) : "memory");
}

// arrival on a barrier of a block of the cluster (address mapped with map_rank); it orders tensor
// memory only (through the tcgen05 fences), so it needs no release
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// A place in a ring of n slots, after so many uses of slots: the next slot and the parity of its use.  Kept by
// counting: an integer division costs as much as the MMAs of a stage.
struct Ring {
    int slot, n;
    unsigned uses, parity;
    __device__ explicit Ring(int n_, unsigned used = 0) : slot((int)(used % (unsigned)n_)), n(n_), uses(used), parity(used / (unsigned)n_ & 1u) {}
    __device__ void next() {
        ++uses;
        if (++slot == n) slot = 0, parity ^= 1u;
    }
    __device__ bool reused() const { return uses >= (unsigned)n; }
};

__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {   // address mapped with map_rank
    asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(addr), "f"(v) : "memory");
}

// The last use of each slot of a ring, up to r, is complete on the slots' barriers.
__device__ __forceinline__ void drain_ring(Ring r, uint32_t full) {
    for (int j = 0; j < r.n; ++j, r.next())   // oldest first: parity ^ 1 is that of the slot's last use
        if (r.reused()) rest_wait(full + 8u * (uint32_t)r.slot, r.parity ^ 1u);
}

// box copy whose bytes count on a barrier of either block of the pair
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// arrival on the barrier at this offset in both blocks once the MMAs issued so far are done; first: the pair's first rank
__device__ __forceinline__ void tc_commit_pair(uint32_t bar, uint32_t first = 0) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
        "h"((uint16_t)(3u << first))
        : "memory");
}
// 32 consecutive fp32 columns of this thread's tensor-memory lane
__device__ __forceinline__ void tc_ld32(uint32_t taddr, uint32_t *r) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, "
        "[%32];\n"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr)
        : "memory");
}

__host__ __device__ constexpr uint32_t pow2_cols(uint32_t c) {
    return c <= 32 ? 32 : c <= 64 ? 64 : c <= 128 ? 128 : c <= 256 ? 256 : 512;
}

}  // namespace lora
