// Base product over microscaled operands, y = X W^T (contract: lora_delta.h),
// on the block-scaled tensor-core kinds: operands stay in 8 or 4 bits all the
// way into tcgen05.mma, which multiplies each product by its two blocks' scales
// and accumulates in fp32 in tensor memory.
//
//   X MXFP8, W MXFP4   kind::mxf8f6f4, K = 32 (one scale) per instruction; W's 4-bit
//                      elements arrive in shared memory in 8-bit cells (the map's packed4 form)
//   X MXFP4, W MXFP4   kind::mxf4, K = 64 (two scales) per instruction, packed
//
// Both kinds see rows of 128 bytes with 128-byte swizzle and step 32 bytes per instruction,
// four to a box: 128 columns of K (MXFP8) or 256 (MXFP4).  Scales lie in tensor memory as the
// MMA wants them: lane r, one column per 32 rows, a byte per block, the same in all four 32-lane partitions;
// the storage's 512-byte tile (128 rows x 4 blocks, 16 bytes for rows r, r+32, r+64, r+96) is a
// lane's four columns.  Warps put them there with tcgen05.st: tcgen05.cp would do it from shared
// memory, but waits in line with the MMAs (six copies a stage of the pair kernel below: 1003 us
// at 8192 x 8192 x 28672 in 4 bits, 845 without).
//
// Two kernels, for few and many rows of x; which one: launch_linear.
#include "mx.cuh"
#include "ptx.cuh"
#include "tc.cuh"

#include <algorithm>
#include <cstdlib>
#include <mutex>
#include <type_traits>

namespace lora {

namespace {

enum { MX_A8 = 0, MX_A4 = 1 };   // x in MXFP8 / MXFP4

struct MxLinArgs {   // a call, as the launchers take it
    const uint8_t *sw, *sx;
    void *y;
    int64_t ld_y;
    int T, d_out;
    int n_kt;      // scale tiles along k: padded columns / 128
    int n_stage;   // ring stages of k
    int32_t *status;
    unsigned limit;   // tries of a bounded wait
    int stall;        // test hook (STALL_*)
};
// The role that waits for what never comes, of LORA_DEBUG_STALL; every other wait is then short too.
enum { STALL_MMA = 1, STALL_SCALES = 2, STALL_COPY = 3, STALL_SUMS = 4, STALL_COPY_FIRST = 5 };

template <int KIND>
__host__ __device__ constexpr int mx_tiles_per_stage() { return KIND == MX_A8 ? 1 : 2; }
__host__ __device__ constexpr uint32_t pow2_cols(uint32_t c) {
    return c <= 32 ? 32 : c <= 64 ? 64 : c <= 128 ? 128 : c <= 256 ? 256 : 512;
}

// Instruction descriptor of the block-scaled kinds: scale ids at [4,6) (B) and
// [29,31) (A), element types at [7,10) (A) and [10,13) (B), N >> 3 at [17,23),
// e8m0 scales at 23, M >> 4 at [24,29).  Element codes: kind::mxf8f6f4 e4m3 0,
// e2m1 5; kind::mxf4 e2m1 1.
__device__ constexpr uint32_t mx_idesc(int a_type, int b_type, int M, int N) {
    return ((uint32_t)a_type << 7) | ((uint32_t)b_type << 10) | ((uint32_t)(N >> 3) << 17) | (1u << 23) |
           ((uint32_t)(M >> 4) << 24);
}
__device__ constexpr uint32_t mx_sf_ids(uint32_t id) { return (id << 4) | (id << 29); }

#define MX_MMA(group, kind)                                                                                         \
    asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"                                                  \
                 "tcgen05.mma.cta_group::" group ".kind::" kind " [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::"r"(d), \
                 "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)                                             \
                 : "memory")
// PAIR: cta_group::2, two blocks of a cluster on one tile
template <int KIND, bool PAIR>
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t acc) {
    if (KIND == MX_A8 && !PAIR) MX_MMA("1", "mxf8f6f4.block_scale.scale_vec::1X");
    if (KIND == MX_A8 && PAIR) MX_MMA("2", "mxf8f6f4.block_scale.scale_vec::1X");
    if (KIND == MX_A4 && !PAIR) MX_MMA("1", "mxf4.block_scale.scale_vec::2X");
    if (KIND == MX_A4 && PAIR) MX_MMA("2", "mxf4.block_scale.scale_vec::2X");
}
#undef MX_MMA
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
// A warp's part has ended: after a wait of its own that ran out, or that another's stopped.
template <bool PAIR>
__device__ __forceinline__ void leave(const Bound &w, bool failed) {
    if (failed && elect_one()) {
        atomicOr(w.status, LORA_DEV_TIMEOUT);
        if (PAIR) {
#pragma unroll
            for (uint32_t k = 0; k < 2; ++k)
                asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;\n" ::"r"(map_rank(w.stop, k)) : "memory");
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

// 16 bytes to four columns of this thread's tensor-memory lane
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint4 v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// arrival on a barrier of a block of the cluster (address mapped with map_rank); it orders tensor
// memory only (through the tcgen05 fences), so it needs no release
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// The MMAs of one ring stage: n_tiles scale tiles (128 columns of K each) of operands
// at a, b (shared memory) whose scales lie at columns sa, sb of tensor memory,
// four (sb_cols) columns a tile.
template <int KIND, bool PAIR>
__device__ __forceinline__ void mx_stage_mmas(uint32_t d, uint32_t a, uint32_t b, uint32_t sa, uint32_t sb, int sb_cols,
                                              int n_tiles, uint32_t idesc, bool first) {
    const uint64_t da = desc_sw128(a), db = desc_sw128(b);
    if (KIND == MX_A8) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mx_mma<KIND, PAIR>(d, da + 2 * k, db + 2 * k, idesc | mx_sf_ids(k), sa, sb, first && k == 0 ? 0u : 1u);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < 2 * n_tiles)
                mx_mma<KIND, PAIR>(d, da + 2 * k, db + 2 * k, idesc | mx_sf_ids(2 * (k & 1)), sa + 4 * (k >> 1),
                                   sb + sb_cols * (k >> 1), first && k == 0 ? 0u : 1u);
    }
}

template <bool BF16>
__device__ __forceinline__ void y_store(void *y, int64_t at, float v) {
    if (BF16) static_cast<__nv_bfloat16 *>(y)[at] = __float2bfloat16_rn(v);
    else static_cast<float *>(y)[at] = v;
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
// Every other row from `from` of a block's `to` rows: the S partial sums at
// [source][row of own][128 features], in order, to y.
template <int S, typename Y>
__device__ __forceinline__ void sum_rows(Y *y, int64_t ld, uint32_t red, int own, int from, int to) {
#pragma unroll 4
    for (int j = from; j < to; j += 2) {
        float v[S];
#pragma unroll
        for (int k = 0; k < S; ++k) v[k] = __uint_as_float(lds32(red + (uint32_t)(k * own + j) * 512u));
        float t = v[0];
#pragma unroll
        for (int k = 1; k < S; ++k) t += v[k];
        store_elem(y + j * ld, t);
    }
}

// The last use of each slot of a ring, up to r, is complete on the slots' barriers.
__device__ __forceinline__ void drain_ring(Ring r, uint32_t full) {
    for (int j = 0; j < r.n; ++j, r.next())   // oldest first: parity ^ 1 is that of the slot's last use
        if (r.reused()) rest_wait(full + 8u * (uint32_t)r.slot, r.parity ^ 1u);
}

// ---------------------------------------------------------------- few rows
// A cluster takes 128 MT output features (the MMA's M side: W's rows, which a small
// batch reads once) x BN rows of x (its N side, any multiple of 16 up to 192), each of its S
// blocks over 1 / S of k; persistent, cluster c takes tiles c, c + clusters, ....
// A ring slot holds KT scale tiles of k (128 columns each): two, or one where wide x tiles would leave too few
// slots.  Roles: one warp copies W and its scales, one x and its, one issues MMAs, four move scales from
// shared to tensor memory, eight take the finished
// accumulator.  There are two: one tile's sums are stored while the next one's products go on; or, MT = 2, one for each
// 128 features, which reads x once for both and may leave a block one tile in place of two (256 x 4096 x 14336 22.3 -> 20.5
// us; tiles of the height that spreads the features evenly over all SMs took the same time).  S > 1 only where every
// cluster has one tile: its blocks then add their partial sums, in block order, through distributed shared memory: each owns
// 1 / S of the rows, and gets the others' sums by plain stores between cluster barriers (st.async, which counts every
// 16 bytes on a barrier, took 1.4 us per 16 rows).  They land behind the ring (few rows) or, once every
// block's products are done, in it.
//
// Bound: from about 130 rows on, each SM's copies into shared memory (257 x 14336 x 4096 22.4 us: 34 KB of W and x per 128
// columns).  For few rows not settled: 64 x 4096 x 28672 moves its 66 MB in 18.8 us (3.5 TB/s, 55 % of HBM's measured
// rate), with x in MXFP4, when the same bytes of W arrive packed in place of 8-bit cells, in 15.7 (4.2).  So HBM is
// not the bound of the first: its 64-byte rows of W are, or the filling of the cells (the two were not timed apart).  What
// a warp does per slot counts as much: a stage of the MMA warp with a barrier for each 128
// columns and one for its scales took 1200 clocks per 256 columns, the products 320.
// warp 0 copies W, 1 MMAs, 2-5 scales, 6-9 and 11-14 sums and stores (every other 16 rows), 10 copies x
constexpr int FEW_THREADS = 480;
constexpr int FEW_STAGES = 12;
constexpr int FEW_ROWS = 192;         // widest BN
constexpr size_t MX_MAX_SMEM = 226 * 1024;

struct MxFewArgs {
    CUtensorMap tmW, tmX;
    const uint8_t *sw, *sx;
    void *y;
    int64_t ld_y;
    int T, d_out, n_kt, n_ks;   // k in scale tiles and in ring slots
    int bn, nt, tiles;          // rows of a tile, row tiles, all tiles
    int bands, x_bands, w_bands;   // 128-row bands of x scales one tile may touch; that x and W have
    int stages, split_log2;     // ring depth; blocks of a cluster
    int own_red;                // the partial sums' place is behind the ring
    int32_t *status;
    unsigned limit;
    int stall;
};

// A slot: W (16 KB a box: a scale tile of MXFP8's k, two of MXFP4's) of each 128 features, x, then the scales of W's
// and of x's bands (KT tiles each)
template <int KIND>
__host__ __device__ constexpr int mx_boxes(int kt) { return KIND == MX_A8 ? kt : kt / 2; }
template <int KIND>
__host__ __device__ constexpr uint32_t few_x_at(int kt, int mt) { return 16384u * mt * mx_boxes<KIND>(kt); }
template <int KIND>
__host__ __device__ constexpr uint32_t few_sf_at(int kt, int mt, int bn) { return (16384u * mt + 128u * bn) * mx_boxes<KIND>(kt); }
template <int KIND>
__host__ __device__ constexpr uint32_t few_slot_bytes(int kt, int mt, int bn, int bands) {
    return (few_sf_at<KIND>(kt, mt, bn) + (mt + bands) * kt * MX_TILE_BYTES + 1023u) & ~1023u;
}
__host__ __device__ constexpr uint32_t few_sf_cols(int kt, int mt, int bn) { return kt * (4 * mt + (bn > 128 ? 8 : 4)); }

template <int KIND, int KT, int MT, typename Y>
__global__ void __launch_bounds__(FEW_THREADS, 1) mx_linear_few_kernel(const __grid_constant__ MxFewArgs a) {
    extern __shared__ __align__(1024) unsigned char mx_sm[];
    __shared__ uint32_t tmem_sm;
    __shared__ __align__(8) uint64_t bars[3 * FEW_STAGES + 5];
    __shared__ uint32_t stop_sm, used_sm[6];   // ring uses of the warps that copy W and x and move scales
    constexpr int BOXES = mx_boxes<KIND>(KT);
    const int warp = __shfl_sync(FULL, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t slot_bytes = few_slot_bytes<KIND>(KT, MT, a.bn, a.bands), sf_at = few_sf_at<KIND>(KT, MT, a.bn);
    const uint32_t base = (smem_u32(mx_sm) + 1023u) & ~1023u, red = base + (a.own_red ? (uint32_t)a.stages * slot_bytes : 0u);
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(FEW_STAGES + s); };
    auto sf_full = [&](int s) { return bar(2 * FEW_STAGES + s); };
    auto acc_full = [&](int b) { return bar(3 * FEW_STAGES + b); };
    auto acc_empty = [&](int b) { return bar(3 * FEW_STAGES + 2 + b); };
    const uint32_t rest = bar(3 * FEW_STAGES + 4);   // completes in the teardown after a wait that ran out, else never
    const Bound bound{smem_u32(&stop_sm), a.limit, a.status};
    const int S = 1 << a.split_log2, rank = (int)blockIdx.x & (S - 1);   // clusters are S consecutive blocks
    const int c0 = (int)blockIdx.x >> a.split_log2, clusters = (int)gridDim.x >> a.split_log2;
    const int k_lo = a.n_ks * rank >> a.split_log2, k_hi = a.n_ks * (rank + 1) >> a.split_log2;
    const uint32_t acc_cols = ((uint32_t)a.bn + 31u) & ~31u, xc = a.bn > 128 ? 8u : 4u;
    const uint32_t sf_cols = few_sf_cols(KT, MT, a.bn), tmem_cols = pow2_cols(2 * acc_cols + (uint32_t)a.stages * sf_cols);
    bool failed = false;

    // a warp's place: tile t (m0, n0: its first feature and row)
    int t, m0, n0;
    auto place = [&](int tile) {
        t = tile;
        const int mi = a.nt == 1 ? t : t / a.nt;
        m0 = mi * 128 * MT, n0 = (t - mi * a.nt) * a.bn;
    };
    auto next_tile = [&]() { place(t + clusters); };
    place(c0);
    Ring ring(a.stages);

    if (warp == 0) {
        for (int i = lane; i < 3 * FEW_STAGES + 5; i += 32) {
            // full: both copying warps and the four scale warps; sf_full: both; acc_empty: eight warps
            const bool six = i < FEW_STAGES, two = i >= 2 * FEW_STAGES && i < 3 * FEW_STAGES;
            const bool eight = i >= 3 * FEW_STAGES + 2 && i < 3 * FEW_STAGES + 4;
            mbar_init(bar(i), six ? 6 : two ? 2 : eight ? 8 : 1);
        }
        if (lane == 0) stop_sm = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        if (lane == 0) prefetch_tmap(&a.tmW);
        __syncwarp();
        asm volatile("bar.sync 1, 64;\nbar.arrive 2, %0;\n" ::"n"(FEW_THREADS) : "memory");
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_sm)),
                     "r"(tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    } else if (warp == 10) {
        if (lane == 0) prefetch_tmap(&a.tmX);
        __syncwarp();
        asm volatile("bar.sync 1, 64;\nbar.arrive 2, %0;\n" ::"n"(FEW_THREADS) : "memory");
    }
    uint32_t tmem = 0;
    if (warp != 0 && warp != 10) {   // the copying warps go ahead: barriers are enough for them
        tc_fence_before();
        asm volatile("bar.sync 2, %0;\n" ::"n"(FEW_THREADS) : "memory");
        tc_fence_after();
        tmem = __shfl_sync(FULL, tmem_sm, 0);
    }
    if (S > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");   // this block's barriers are set
    const uint32_t sf = tmem + 2 * acc_cols;
    pdl_next();
    pdl_wait();   // all warps: none of the bounded waits below runs while the kernel before this one does

    const int64_t band = (int64_t)a.n_kt * MX_TILE_BYTES;   // scale bytes of 128 rows
    if (warp == 0) {   // W and its scales
        if (a.stall == STALL_COPY_FIRST) uniform_wait(rest, 0, bound, failed);
        for (; t < a.tiles && !failed; next_tile()) {
            const uint8_t *sw = a.sw + m0 / 128 * band;
            // features past the last band: any scales will do
            const int64_t sw1 = MT == 2 && m0 / 128 + 1 < a.w_bands ? band : 0;
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                const uint32_t b = full(ring.slot), sb = sf_full(ring.slot), slot = base + (uint32_t)ring.slot * slot_bytes;
                if (ring.reused() && !uniform_wait(empty(ring.slot), ring.parity ^ 1u, bound, failed)) break;
                if (elect_one()) {
                    const uint32_t n = (uint32_t)min(KT, a.n_kt - KT * k) * MX_TILE_BYTES;
                    const uint8_t *p = sw + (int64_t)k * KT * MX_TILE_BYTES;
                    // packed4 boxes count packed bytes; a box past k's end arrives as zeros that no MMA reads
                    mbar_expect_tx(b, (KIND == MX_A8 ? 8192u : 16384u) * (BOXES * MT));
#pragma unroll
                    for (int u = 0; u < MT; ++u)
#pragma unroll
                        for (int x = 0; x < BOXES; ++x)
                            tma_2d(slot + 16384u * (BOXES * u + x), &a.tmW, (BOXES * k + x) * 128, m0 + 128 * u, b);
                    mbar_expect_tx(sb, MT * n);
                    bulk_g2s(slot + sf_at, p, n, sb);
                    if (MT == 2) bulk_g2s(slot + sf_at + KT * MX_TILE_BYTES, p + sw1, n, sb);
                }
            }
        }
        if (elect_one()) used_sm[0] = ring.uses;
    } else if (warp == 10) {   // x and its scales
        if (a.stall == STALL_COPY) uniform_wait(rest, 0, bound, failed);
        const uint32_t x_bytes = (uint32_t)a.bn * 128u;
        for (; t < a.tiles && !failed; next_tile()) {
            const int xb = n0 / 128, nb = min(a.bands, a.x_bands - xb);
            const uint8_t *sx = a.sx + xb * band;
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                const uint32_t b = full(ring.slot), sb = sf_full(ring.slot), slot = base + (uint32_t)ring.slot * slot_bytes;
                if (ring.reused() && !uniform_wait(empty(ring.slot), ring.parity ^ 1u, bound, failed)) break;
                if (elect_one()) {
                    const uint32_t n = (uint32_t)min(KT, a.n_kt - KT * k) * MX_TILE_BYTES;
                    const uint8_t *p = sx + (int64_t)k * KT * MX_TILE_BYTES;
                    mbar_expect_tx(b, x_bytes * BOXES);
#pragma unroll
                    for (int x = 0; x < BOXES; ++x)
                        tma_2d(slot + few_x_at<KIND>(KT, MT) + x_bytes * x, &a.tmX, (BOXES * k + x) * 128, n0, b);
                    mbar_expect_tx(sb, (uint32_t)nb * n);
                    for (int i = 0; i < nb; ++i) bulk_g2s(slot + sf_at + (uint32_t)((MT + i) * KT) * MX_TILE_BYTES, p + i * band, n, sb);
                }
            }
        }
        if (elect_one()) used_sm[1] = ring.uses;
    } else if (warp == 1) {
        const uint32_t idesc = KIND == MX_A8 ? mx_idesc(5, 0, 128, a.bn) : mx_idesc(1, 1, 128, a.bn);
        const uint32_t x_bytes = (uint32_t)a.bn * 128u;
        int n = 0;
        if (a.stall == STALL_MMA) uniform_wait(rest, 0, bound, failed);
        for (; t < a.tiles && !failed; next_tile(), ++n) {
            const int b = MT == 2 ? 0 : n & 1;
            if (MT == 2) {
                if (n >= 1 && !(uniform_wait(acc_empty(0), (unsigned)(n - 1) & 1u, bound, failed) &&
                                uniform_wait(acc_empty(1), (unsigned)(n - 1) & 1u, bound, failed)))
                    break;
            } else if (n >= 2 && !uniform_wait(acc_empty(b), (unsigned)(n / 2 - 1) & 1u, bound, failed)) {
                break;
            }
            const uint32_t d = tmem + (uint32_t)b * acc_cols;
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                const uint32_t slot = base + (uint32_t)ring.slot * slot_bytes, ta = sf + sf_cols * (uint32_t)ring.slot;
                const int tiles = min(KT, a.n_kt - KT * k);
                if (!uniform_wait(full(ring.slot), ring.parity, bound, failed)) break;
                tc_fence_after();
                if (elect_one()) {
#pragma unroll
                    for (int u = 0; u < MT; ++u)
#pragma unroll
                        for (int x = 0; x < BOXES; ++x)
                            if (KIND == MX_A4 || x < tiles)
                                mx_stage_mmas<KIND, false>(d + acc_cols * u, slot + 16384u * (BOXES * u + x),
                                                           slot + few_x_at<KIND>(KT, MT) + x_bytes * x, ta + 4 * (KT * u + x),
                                                           ta + 4 * KT * MT + xc * x, (int)xc, tiles, idesc, k == k_lo && x == 0);
                    tc_commit(empty(ring.slot));
                }
            }
            if (elect_one()) {
                tc_commit(acc_full(b));
                if (MT == 2) tc_commit(acc_full(1));
            }
        }
    } else if (warp < 6) {
        const uint32_t dst = sf + ((uint32_t)(32 * (warp & 3)) << 16);
        if (a.stall == STALL_SCALES && warp == 2) uniform_wait(rest, 0, bound, failed);
        for (; t < a.tiles && !failed; next_tile()) {
            // W: lane r gets the 16 bytes of rows r, r + 32, r + 64, r + 96.  x: the tile's rows may start
            // anywhere in a band; column g, lane r: row n0 + 32 g + r
            const int xb = n0 / 128, last = min(a.bands, a.x_bands - xb) - 1;
            uint32_t at[8];   // where column g's scales of k tile 0 lie in a slot
#pragma unroll
            for (int g = 0; g < 8; ++g) {
                const int row = n0 + 32 * g + lane, band = min(row / 128 - xb, last);
                at[g] = sf_at + (uint32_t)((MT + band) * KT) * MX_TILE_BYTES + (uint32_t)(row % 32 * 16 + row / 32 % 4 * 4);
            }
            for (int k = k_lo; k < k_hi; ++k, ring.next()) {
                if (!uniform_wait(sf_full(ring.slot), ring.parity, bound, failed)) break;
                tc_fence_after();   // earlier MMAs read these columns (their commit let the scales' copy go ahead)
                const uint32_t slot = base + (uint32_t)ring.slot * slot_bytes, to = dst + sf_cols * (uint32_t)ring.slot;
#pragma unroll
                for (int i = 0; i < KT; ++i) {   // a tile past k's end is old data that no MMA reads
                    const uint32_t src = slot + i * MX_TILE_BYTES;
#pragma unroll
                    for (int u = 0; u < MT; ++u)
                        tmem_st4(to + 4 * (KT * u + i), lds128(src + sf_at + u * (KT * MX_TILE_BYTES) + 16 * lane));
                    tmem_st4(to + 4 * KT * MT + xc * i, make_uint4(lds32(src + at[0]), lds32(src + at[1]), lds32(src + at[2]),
                                                              lds32(src + at[3])));
                    if (xc == 8)
                        tmem_st4(to + 4 * KT * MT + xc * i + 4, make_uint4(lds32(src + at[4]), lds32(src + at[5]),
                                                                      lds32(src + at[6]), lds32(src + at[7])));
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (elect_one()) mbar_arrive(full(ring.slot));
            }
        }
        if (elect_one()) used_sm[warp] = ring.uses;
    } else {
        const int q = warp & 3, f = 32 * q + lane;   // this thread's output feature of the tile
        const int half = 16 * (warp > 10);           // its first row; then every other 16
        const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
        if (S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");   // every block's barriers are set
        // n counts accumulators: tile by tile, or the two of a tile
        for (int n = 0; t < a.tiles && !failed; ++n) {
            const int b = n & 1, rows = min(a.bn, a.T - n0), m = m0 + (MT == 2 ? 128 * b : 0) + f;
            const uint32_t src_acc = acc + (uint32_t)b * acc_cols;
            const bool there = m < a.d_out;
            Y *y = static_cast<Y *>(a.y) + (int64_t)n0 * a.ld_y + m;
            const bool stall = a.stall == STALL_SUMS && warp == 6;
            // S > 1: on to the exchange all the same, which every block of the cluster takes part in
            if (!lanes_wait(stall ? rest : acc_full(b), (unsigned)(n / 2) & 1u, bound, failed) && S == 1) break;
            tc_fence_after();
            if (S == 1) {
                for (int c = half; c < rows; c += 32) {
                    float d[16];
                    tc_ld16(src_acc + c, d);
                    tc_wait_ld();
                    Y *p = y + c * a.ld_y;
#pragma unroll
                    for (int j = 0; j < 16; ++j, p += a.ld_y)
                        if (there && c + j < rows) store_elem(p, d[j]);
                }
            } else {
                // rows of a block: a power of two up to 16, or a multiple of 16, so that 16 rows' owners follow from
                // shifts or are one
                const int fair = (rows + S - 1) >> a.split_log2, own_log2 = fair <= 1 ? 0 : 32 - __clz(min(fair, 16) - 1);
                const int own = fair <= 16 ? 1 << own_log2 : (fair + 15) & ~15;
                const uint32_t mine = red + (uint32_t)(rank * own * 128 + f) * 4u;   // [source][row][feature]
                if (!a.own_red) cluster_sync_all();   // every block's products are done with its ring
                for (int c = half; c < rows; c += 32) {
                    float d[16];
                    tc_ld16(src_acc + c, d);
                    if (own >= 16) {
                        const int to = c / own;
                        const uint32_t at = map_rank(mine, (uint32_t)to) + (uint32_t)(c - to * own) * 512u;
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < rows) st_cluster(at + 512u * i, d[i]);
                    } else {
                        tc_wait_ld();
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (c + i < rows)
                                st_cluster(map_rank(mine, (uint32_t)(c + i) >> own_log2) + 512u * (i & (own - 1)), d[i]);
                    }
                }
                cluster_sync_all();
                if (there) {
                    const int to = min(own, rows - rank * own);
                    Y *p = y + (int64_t)(rank * own) * a.ld_y;
                    if (S == 2) sum_rows<2>(p, a.ld_y, red + 4u * f, own, half >> 4, to);
                    else if (S == 4) sum_rows<4>(p, a.ld_y, red + 4u * f, own, half >> 4, to);
                    else sum_rows<8>(p, a.ld_y, red + 4u * f, own, half >> 4, to);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty(b));
            if (MT == 1 || b == 1) next_tile();
        }
    }
    // ---------------------------------------------------------------- teardown
    __syncwarp();
    leave<false>(bound, failed);
    if (S > 1 && (warp < 6 || warp == 10)) {   // the barriers that the other warps wait at
        asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
        if (!a.own_red) cluster_sync_all();
        cluster_sync_all();
    }
    tc_fence_before();
    __syncthreads();
    if (stop_sm) {
        // A wait ran out: the other warps stopped where they were.  Each that arrives on the ring's barriers makes up for the
        // uses that the warps ahead of it began (at most one a slot: none is begun before all are done with the slot's
        // last one), which then complete as their copies land; the copying warps, whose block's memory these go to, see them land.
        const unsigned begun = max(used_sm[0], used_sm[1]);
        const bool copies = warp == 0 || warp == 10;
        if (copies || (warp >= 2 && warp < 6)) {
            Ring r(a.stages, used_sm[warp == 10 ? 1 : warp]);
            for (; r.uses < begun; r.next())
                if (elect_one()) {
                    mbar_arrive(full(r.slot));
                    if (copies) mbar_arrive(sf_full(r.slot));
                }
            if (copies) drain_ring(r, sf_full(0)), drain_ring(r, full(0));
        }
        if (warp == 1) {   // the products read this memory and tensor memory
            if (elect_one()) tc_commit(rest);
            rest_wait(rest, 0);
        }
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(tmem_cols) : "memory");
    }
}

// Blocks along k and clusters of them, by the time they would take: a scale tile of k costs a block `one`, bound by
// its latency or its operands' way into shared memory, or `more` where every SM streams; an exchange of partial sums
// 0.95 us for each doubling of S and 12 ns a row; all 3 us and 8 ns a row and accumulator besides.  Measured (us, S = 1, 2,
// 4): 1 x 4096 x 4096 7.7, 6.0, 5.5; 64 x 4096 x 4096 9.0, 7.9, 7.1; 64 x 1024 x 4096 4.7, 5.6, 5.4;
// 257 x 14336 x 4096 25.7, 22.5.  MT = 1 / 2, MXFP8: 1 x 4096 x 28672 15.8 / 16.1, 64 rows 18.6 / 18.8, 128 rows 24.2 / 22.4,
// 256 x 4096 x 14336 22.3 / 20.5, 64 x 4096 x 50000 27.3 / 34.2; MXFP4: 14.7 / 14.1, 16.0 / 15.6, 17.7 / 17.4, 15.0 / 13.9,
// 23.5 / 26.9.
struct FewPlan {
    int split_log2 = 0, clusters = 1;
    int64_t ns = 0;
};
template <int KIND, int KT, int MT, typename Y>
int few_plan(const MxFewArgs &a, int dev, FewPlan *out) {
    // clusters resident at once: a property of the device and the kernel, asked for once
    static std::mutex mu;
    static int fit[64][4] = {};   // 1 + clusters of 1, 2, 4, 8
    std::lock_guard<std::mutex> lock(mu);
    int *f = fit[dev & 63];
    auto kernel = mx_linear_few_kernel<KIND, KT, MT, Y>;
    if (!f[0]) {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MX_MAX_SMEM);
        for (int i = 3; i >= 0 && e == cudaSuccess; --i) {   // f[0] last: it marks the table as filled
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(1u << i);
            cfg.blockDim = dim3(FEW_THREADS);
            cfg.dynamicSmemBytes = MX_MAX_SMEM;
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = 1u << i;
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            int n = 0;
            e = cudaOccupancyMaxActiveClusters(&n, kernel, &cfg);
            if (e == cudaSuccess) f[i] = 1 + n;
        }
        if (e != cudaSuccess) return cuda_rc(e);
    }
    const bool a8 = KIND == MX_A8;
    const int one = a8 ? std::max(180, 110 + 12 * a.bn / 10) : std::max(150, 90 + 66 * a.bn / 100);
    const int more = MT == 2 ? (a8 ? 410 + a.bn : 345 + a.bn / 2) : (a8 ? 195 + a.bn * 7 / 8 : 190 + a.bn / 4);
    int64_t best = -1;
    for (int i = 0; i < (MT == 2 ? 1 : 4); ++i) {
        const int s = 1 << i, n = std::min(a.tiles, i ? f[i] - 1 : std::max(1, f[i] - 1));
        if (s > a.n_ks || (i && n < a.tiles)) break;
        const int64_t rounds = (a.tiles + n - 1) / n, kt_ns = MT == 2 || rounds > 1 ? more : one;
        const int64_t cost = rounds * ((a.n_ks + s - 1) / s) * KT * kt_ns + (i ? 950 * i + 12 * a.bn : 0);
        if (best < 0 || cost < best) best = cost, out->split_log2 = i, out->clusters = n;
    }
    out->ns = best + 3000 + 8 * a.bn * MT;
    return LORA_OK;
}

template <int KIND, int KT, int MT>
void few_tiles(MxFewArgs &a) {
    a.n_ks = (a.n_kt + KT - 1) / KT;
    a.tiles = (a.w_bands + MT - 1) / MT * a.nt;
}
template <int KIND, int KT, int MT, typename Y>
int launch_few_as(MxFewArgs &a, const FewPlan &plan, cudaStream_t st) {
    few_tiles<KIND, KT, MT>(a);
    a.split_log2 = plan.split_log2;
    const int acc_cols = (a.bn + 31) / 32 * 32;
    a.own_red = a.bn <= 32;
    const size_t room = MX_MAX_SMEM - 1024 - (plan.split_log2 && a.own_red ? (size_t)(2 * a.bn + 16) * 512 : 0);
    a.stages = (int)std::min<size_t>(FEW_STAGES, room / few_slot_bytes<KIND>(KT, MT, a.bn, a.bands));
    a.stages = std::min(a.stages, (512 - 2 * acc_cols) / (int)few_sf_cols(KT, MT, a.bn));
    // all of the shared memory: one block an SM (two might wait for each other's tensor memory)
    return launch_after(mx_linear_few_kernel<KIND, KT, MT, Y>, dim3((unsigned)(plan.clusters << plan.split_log2)), FEW_THREADS,
                        MX_MAX_SMEM, 1u << plan.split_log2, st, a);
}

// A shape of the tiles and what it would take.
struct FewShape {
    int bn = 0, nt = 0, mt = 0;
    FewPlan plan;
};
// Scale tiles of a slot: two while three slots fit, else one (MXFP8: KT = 1 from 145 rows on; 257 x 14336 x 4096
// 23.7 us with one, 22.3 with two).
template <int KIND>
constexpr int few_kt(bool wide, int mt) { return KIND == MX_A4 || (mt == 1 && !wide) ? 2 : 1; }
inline bool few_wide(int bn) { return bn > 144; }

template <int KIND, bool WIDE, typename Y>
int few_consider(MxFewArgs &a, int dev, FewShape *best) {
    constexpr int KT1 = few_kt<KIND>(WIDE, 1), KT2 = few_kt<KIND>(WIDE, 2);
    auto keep = [&](const FewPlan &p, int mt) {
        if (!best->mt || p.ns < best->plan.ns) best->bn = a.bn, best->nt = a.nt, best->mt = mt, best->plan = p;
    };
    FewPlan p;
    few_tiles<KIND, KT1, 1>(a);
    int rc = few_plan<KIND, KT1, 1, Y>(a, dev, &p);
    if (rc != LORA_OK) return rc;
    keep(p, 1);
    if (a.tiles > p.clusters && a.bn <= 128) {   // blocks with a second tile, and room for four slots
        few_tiles<KIND, KT2, 2>(a);
        rc = few_plan<KIND, KT2, 2, Y>(a, dev, &p);
        if (rc != LORA_OK) return rc;
        keep(p, 2);
    }
    return LORA_OK;
}
template <int KIND, bool WIDE, typename Y>
int few_run(MxFewArgs &a, const FewShape &s, cudaStream_t st) {
    constexpr int KT1 = few_kt<KIND>(WIDE, 1), KT2 = few_kt<KIND>(WIDE, 2);
    return s.mt == 2 ? launch_few_as<KIND, KT2, 2, Y>(a, s.plan, st) : launch_few_as<KIND, KT1, 1, Y>(a, s.plan, st);
}

// The call on this kernel unless it would take longer than limit_ns (*took = 0 then).
template <int KIND, typename Y>
int launch_few(const MxLinArgs &l, const lora_mx *x, const lora_mx *w, int dev, int64_t limit_ns, int *took, cudaStream_t st) {
    MxFewArgs a{};
    a.sw = l.sw, a.sx = l.sx, a.y = l.y, a.ld_y = l.ld_y, a.T = l.T, a.d_out = l.d_out, a.n_kt = l.n_kt;
    a.x_bands = (l.T + 127) / 128, a.w_bands = (l.d_out + 127) / 128;
    a.status = l.status, a.limit = l.limit, a.stall = l.stall;
    auto shape = [&](int nt) {   // row tiles of equal height, a multiple of 16
        a.bn = ((l.T + nt - 1) / nt + 15) / 16 * 16;
        a.nt = (l.T + a.bn - 1) / a.bn;
        a.bands = std::min(a.x_bands, a.nt == 1 ? (a.bn + 127) / 128 : (a.bn + 126) / 128 + 1);
    };
    FewShape best;
    const int least = (l.T + FEW_ROWS - 1) / FEW_ROWS;
    for (int nt = least; nt <= least + 2; ++nt) {   // the fewest row tiles, or a little more that fill the SMs better
        shape(nt);
        const int rc = few_wide(a.bn) ? few_consider<KIND, true, Y>(a, dev, &best) : few_consider<KIND, false, Y>(a, dev, &best);
        if (rc != LORA_OK) return rc;
        if (a.bn <= 64) break;
    }
    *took = best.plan.ns <= limit_ns;
    if (!*took) return LORA_OK;
    shape(best.nt);
    const uint64_t xb = (uint64_t)mx_row_bytes(x->format, x->cols), wb = (uint64_t)mx_row_bytes(w->format, w->cols);
    int rc = tensor_map_mx(&a.tmW, w->q, wb, (uint64_t)l.d_out, wb, 128, KIND == MX_A8);
    if (rc == LORA_OK) rc = tensor_map_mx(&a.tmX, x->q, xb, (uint64_t)l.T, xb, (uint32_t)a.bn, false);
    if (rc != LORA_OK) return rc;
    return few_wide(a.bn) ? few_run<KIND, true, Y>(a, best, st) : few_run<KIND, false, Y>(a, best, st);
}

// ---------------------------------------------------------------- many rows
// A pair of blocks (a cluster, cta_group::2) takes 256 rows of x (M) x 256 output
// features (N): each block loads its own 128 rows of x and 128 of W's rows, the
// tensor cores share the halves, so a block moves 32 KB of a stage for 256 x 256 x 32
// bytes of products, half of what two 128 x 256 tiles would.  At the 4-bit rate that
// is 64 bytes a clock and SM from L2: the reason for the pair.  8192 x 8192 x 28672 in 4 bits: 715 us (5.4 PFLOP/s) in a short
// burst, 838 us steady at about 1500 MHz under the power cap, 657 us on zeros.  Persistent: pair p
// takes tiles p, p + pairs, ... of bands of 16 x tiles, x's tiles fastest: concurrent pairs share W's rows and few enough
// of x's to find both in the nearer half of L2 (8192 x 8192 x 28672 in MXFP8, steady 1570 -> 1455 us;
// 8192 x 4096 x 4096 in MXFP4 68.4 -> 66.0).
// The fp32 accumulator (256 columns) is drained to registers by eight warps in one
// go, the next tile's products start, and the rows are stored meanwhile.
constexpr int BIG_THREADS = 448;      // warp 0 copies, warp 1 MMAs, warps 2-5 scales, warps 6-13 epilogue
constexpr int BIG_STAGES = 6;
constexpr int BIG_BAND = 16;

struct MxBigArgs {
    CUtensorMap tmX, tmW;
    const uint8_t *sx, *sw;
    int x_bands, w_bands;   // 128-row bands of x and W
    void *y;
    int64_t ld_y;
    int T, d_out, n_kt, n_stage;
    int mt, nt, tiles;    // 256-row tiles of x, of W; all
    int vec;          // y rows allow 16-byte stores
    int32_t *status;
    unsigned limit;
    int stall;
};

template <int KIND>
__host__ __device__ constexpr uint32_t big_slot_bytes() {   // x rows, W rows, x scales, W scales (two bands)
    return 32768u + 3u * MX_TILE_BYTES * mx_tiles_per_stage<KIND>();
}
// rounded up to the 1 KB the swizzle's atoms ask for
template <int KIND>
__host__ __device__ constexpr uint32_t big_slot_stride() { return (big_slot_bytes<KIND>() + 1023u) & ~1023u; }

// box copy whose bytes count on a barrier of either block of the pair
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, "
        "{%2, %3}], [%4];\n" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
// arrival on the barrier at this offset in both blocks once the MMAs issued so far are done
__device__ __forceinline__ void tc_commit_pair(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n" ::"r"(bar),
        "h"((uint16_t)3)
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

template <int KIND, bool BF16>
__global__ void __launch_bounds__(BIG_THREADS, 1) mx_linear_big_kernel(const __grid_constant__ MxBigArgs a) {
    extern __shared__ __align__(1024) unsigned char mx_sm[];
    __shared__ uint32_t tmem_sm;
    __shared__ __align__(8) uint64_t bars[4 * BIG_STAGES + 3];
    __shared__ uint32_t stop_sm, used_sm;   // used_sm: ring uses that this block's copies have begun
    constexpr int TPS = mx_tiles_per_stage<KIND>();
    constexpr uint32_t SLOT = big_slot_stride<KIND>();
    constexpr uint32_t SF_COLS = 12 * TPS;   // one stage's scales: 4 columns a tile for x, 8 for W
    constexpr uint32_t TX = 2u * (KIND == MX_A8 ? 16384u + 8192u : 32768u);   // packed4 boxes count packed bytes
    const int warp = __shfl_sync(FULL, (int)threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(mx_sm) + 1023u) & ~1023u;
    const int rank = (int)cluster_rank();
    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    auto full = [&](int s) { return smem_u32(&bars[s]); };                  // the leader's counts both blocks' bytes
    auto empty = [&](int s) { return smem_u32(&bars[BIG_STAGES + s]); };
    auto sf_full = [&](int s) { return smem_u32(&bars[2 * BIG_STAGES + s]); };    // this block's scales have landed
    auto sf_ready = [&](int s) { return smem_u32(&bars[3 * BIG_STAGES + s]); };   // the leader's: both blocks' are in tensor memory
    const uint32_t acc_full = smem_u32(&bars[4 * BIG_STAGES]), acc_empty = smem_u32(&bars[4 * BIG_STAGES + 1]);
    const uint32_t rest = smem_u32(&bars[4 * BIG_STAGES + 2]);   // completes in the teardown after a wait that ran out, else never
    const Bound bound{smem_u32(&stop_sm), a.limit, a.status};

    if (threadIdx.x == 0) {
        for (int s = 0; s < BIG_STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
            mbar_init(sf_full(s), 1);
            mbar_init(sf_ready(s), 8);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 16);   // the leader's: 8 epilogue warps of each block
        mbar_init(rest, 1);
        stop_sm = 0;
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        prefetch_tmap(&a.tmX);
        prefetch_tmap(&a.tmW);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(smem_u32(&tmem_sm))
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();   // the pair's barriers and tensor memory are ready
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(FULL, tmem_sm, 0), sf = tmem + 256;
    bool failed = false;
    pdl_next();
    pdl_wait();   // all warps: none of the bounded waits below runs while the kernel before this one does
    auto place = [&](int t, int &mi, int &ni) {   // of tile t
        const int per = BIG_BAND * a.nt, band = t / per, left = t - band * per, high = min(BIG_BAND, a.mt - band * BIG_BAND);
        ni = left / high;
        mi = band * BIG_BAND + left - ni * high;
    };

    if (warp == 0) {
        Ring ring(BIG_STAGES);
        if (a.stall == (rank ? STALL_COPY : STALL_COPY_FIRST)) uniform_wait(rest, 0, bound, failed);
        for (int t = pair; t < a.tiles && !failed; t += pairs) {
            int mi, ni;
            place(t, mi, ni);
            const int m0 = mi * 256 + 128 * rank, nb = 2 * ni;   // nb: first 128-row band of W
            // bands past the last hold rows that no result uses: any scales will do
            const uint8_t *sx = a.sx + (int64_t)min(m0 / 128, a.x_bands - 1) * a.n_kt * MX_TILE_BYTES;
            const uint8_t *sw0 = a.sw + (int64_t)nb * a.n_kt * MX_TILE_BYTES;
            const uint8_t *sw1 = a.sw + (int64_t)min(nb + 1, a.w_bands - 1) * a.n_kt * MX_TILE_BYTES;
            for (int i = 0; i < a.n_stage; ++i, ring.next()) {
                const int s = ring.slot;
                if (ring.reused() && !uniform_wait(empty(s), ring.parity ^ 1u, bound, failed)) break;
                const uint32_t slot = base + (uint32_t)s * SLOT, bar = map_rank(full(s), 0);
                const uint32_t sfs = slot + 32768u, sb = (uint32_t)min(TPS, a.n_kt - i * TPS) * MX_TILE_BYTES;
                if (elect_one()) {
                    if (rank == 0) mbar_expect_tx(full(s), TX);
                    tma_2d_pair(slot, &a.tmX, i * 128, m0, bar);
                    tma_2d_pair(slot + 16384u, &a.tmW, i * 128, (nb + rank) * 128, bar);
                    const int64_t off = (int64_t)i * TPS * MX_TILE_BYTES;
                    mbar_expect_tx(sf_full(s), 3 * sb);
                    bulk_g2s(sfs, sx + off, sb, sf_full(s));
                    bulk_g2s(sfs + TPS * MX_TILE_BYTES, sw0 + off, sb, sf_full(s));
                    bulk_g2s(sfs + 2 * TPS * MX_TILE_BYTES, sw1 + off, sb, sf_full(s));
                }
            }
        }
        if (elect_one()) used_sm = ring.uses;
    } else if (warp == 1) {
        if (rank == 0) {
            constexpr uint32_t idesc = KIND == MX_A8 ? mx_idesc(0, 5, 256, 256) : mx_idesc(1, 1, 256, 256);
            Ring ring(BIG_STAGES);
            int n = 0;
            if (a.stall == STALL_MMA) uniform_wait(rest, 0, bound, failed);
            for (int t = pair; t < a.tiles && !failed; t += pairs, ++n) {
                if (n > 0 && !uniform_wait(acc_empty, (unsigned)(n - 1) & 1u, bound, failed)) break;
                tc_fence_after();
                for (int i = 0; i < a.n_stage; ++i, ring.next()) {
                    const int s = ring.slot;
                    if (!uniform_wait(sf_ready(s), ring.parity, bound, failed) ||
                        !uniform_wait(full(s), ring.parity, bound, failed))
                        break;
                    tc_fence_after();
                    const uint32_t slot = base + (uint32_t)s * SLOT;
                    const uint32_t ta = sf + SF_COLS * (uint32_t)s, tb = ta + 4 * TPS;
                    const int tiles = min(TPS, a.n_kt - i * TPS);
                    if (elect_one()) {
                        mx_stage_mmas<KIND, true>(tmem, slot, slot + 16384u, ta, tb, 8, tiles, idesc, i == 0);
                        tc_commit_pair(empty(s));
                    }
                }
                if (elect_one()) tc_commit_pair(acc_full);
            }
        }
    } else if (warp < 6) {
        // The scales of a stage from shared to tensor memory: lane r of each of the four
        // partitions gets the 16 bytes of rows r, r + 32, r + 64, r + 96.  The slot's columns are free
        // once its shared memory is: both were read by the same MMAs.
        const uint32_t dst = sf + ((uint32_t)(32 * (warp & 3)) << 16);
        int it = 0;
        if (a.stall == STALL_SCALES && rank == 1 && warp == 2) uniform_wait(rest, 0, bound, failed);
        for (int t = pair; t < a.tiles && !failed; t += pairs)
            for (int i = 0; i < a.n_stage; ++i, ++it) {
                const int s = it % BIG_STAGES;
                if (!lanes_wait(sf_full(s), (unsigned)(it / BIG_STAGES) & 1u, bound, failed)) break;
                tc_fence_after();   // earlier MMAs read these columns (their commit let the scales' copy go ahead)
                const uint32_t src = base + (uint32_t)s * SLOT + 32768u + 16u * lane, to = dst + SF_COLS * (uint32_t)s;
#pragma unroll
                for (int k = 0; k < TPS; ++k) {   // a tile past k's end is old data that no MMA reads
                    tmem_st4(to + 4 * k, lds128(src + k * MX_TILE_BYTES));
                    tmem_st4(to + 4 * TPS + 8 * k, lds128(src + (TPS + k) * MX_TILE_BYTES));
                    tmem_st4(to + 4 * TPS + 8 * k + 4, lds128(src + (2 * TPS + k) * MX_TILE_BYTES));
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(map_rank(sf_ready(s), 0));
            }
    } else {
        const int q = warp & 3, half = (warp - 6) >> 2;
        const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + 128u * half;
        const uint32_t release = map_rank(acc_empty, 0);
        int n = 0;
        if (a.stall == STALL_SUMS && rank == 1 && warp == 6) uniform_wait(rest, 0, bound, failed);
        for (int t = pair; t < a.tiles && !failed; t += pairs, ++n) {
            if (!lanes_wait(acc_full, (unsigned)n & 1u, bound, failed)) break;
            tc_fence_after();
            int mi, ni;
            place(t, mi, ni);
            const int64_t row = (int64_t)mi * 256 + 128 * rank + 32 * q + lane, col = (int64_t)ni * 256 + 128 * half;
            auto drained = [&] {   // this warp's part of the accumulator is in registers
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster(release);
            };
            const int64_t n = row < a.T ? a.d_out - col : 0;   // columns to store
            if (!a.vec) {   // rows of y off 16-byte steps: element by element, straight from tensor memory
#pragma unroll 1
                for (int c = 0; c < 128; c += 16) {
                    float v[16];
                    tc_ld16(acc + c, v);
                    tc_wait_ld();
                    if (c + 16 >= 128) drained();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        if (c + j < n) y_store<BF16>(a.y, row * a.ld_y + col + c + j, v[j]);
                }
            } else if (BF16) {
                uint32_t d[64];   // 128 columns
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint32_t r[32];
                    tc_ld32(acc + 32 * c, r);
                    tc_wait_ld();
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        d[16 * c + j] = pack_bf16x2(__uint_as_float(r[2 * j]), __uint_as_float(r[2 * j + 1]));
                }
                drained();
                uint4 *y = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.y) + row * a.ld_y + col);
#pragma unroll
                for (int c = 0; c < 16; ++c)
                    if (8 * c < n) y[c] = make_uint4(d[4 * c], d[4 * c + 1], d[4 * c + 2], d[4 * c + 3]);
            } else {
#pragma unroll 1
                for (int h = 0; h < 2; ++h) {
                    uint32_t d[64];
                    tc_ld32(acc + 64 * h, d);
                    tc_ld32(acc + 64 * h + 32, d + 32);
                    tc_wait_ld();
                    if (h == 1) drained();
                    uint4 *y = reinterpret_cast<uint4 *>(static_cast<float *>(a.y) + row * a.ld_y + col + 64 * h);
#pragma unroll
                    for (int c = 0; c < 16; ++c)
                        if (64 * h + 4 * c < n) y[c] = make_uint4(d[4 * c], d[4 * c + 1], d[4 * c + 2], d[4 * c + 3]);
                }
            }
        }
    }
    // ---------------------------------------------------------------- teardown
    __syncwarp();
    leave<true>(bound, failed);
    tc_fence_before();
    cluster_sync_all();
    if (stop_sm) {   // a wait ran out: in both blocks, which stopped where they were
        if (warp == 0) {
            Ring r(BIG_STAGES, used_sm);
            drain_ring(r, sf_full(0));
            if (rank == 0) {
                // The leader's barriers count both blocks' bytes.  The uses that one block has begun and the other not (at
                // most one a slot) complete with the bytes of that one.
                uint32_t other;
                asm volatile("ld.shared::cluster.u32 %0, [%1];\n" : "=r"(other) : "r"(map_rank(smem_u32(&used_sm), 1)) : "memory");
                for (uint32_t k = other; k < r.uses; ++k)
                    if (elect_one()) mbar_complete_tx(full((int)(k % BIG_STAGES)), TX / 2);
                for (; r.uses < other; r.next())
                    if (elect_one()) mbar_expect_tx(full(r.slot), TX / 2);
                drain_ring(r, full(0));
            }
        } else if (warp == 1) {   // the products read both blocks' memory and tensor memory
            if (rank == 0 && elect_one()) tc_commit_pair(rest);
            rest_wait(rest, 0);
        }
        cluster_sync_all();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
    }
}

template <int KIND, bool BF16>
int launch_big(const MxLinArgs &l, const lora_mx *x, const lora_mx *w, int sms, cudaStream_t st) {
    MxBigArgs a{};
    const uint64_t xb = (uint64_t)mx_row_bytes(x->format, x->cols), wb = (uint64_t)mx_row_bytes(w->format, w->cols);
    int rc = tensor_map_mx(&a.tmX, x->q, xb, (uint64_t)l.T, xb, 128, false);
    if (rc == LORA_OK) rc = tensor_map_mx(&a.tmW, w->q, wb, (uint64_t)l.d_out, wb, 128, KIND == MX_A8);
    if (rc != LORA_OK) return rc;
    a.sx = l.sx, a.sw = l.sw, a.x_bands = (l.T + 127) / 128, a.w_bands = (l.d_out + 127) / 128;
    a.y = l.y, a.ld_y = l.ld_y, a.T = l.T, a.d_out = l.d_out, a.n_kt = l.n_kt, a.n_stage = l.n_stage;
    a.mt = (l.T + 255) / 256;
    a.nt = (l.d_out + 255) / 256;
    a.tiles = a.mt * a.nt;
    a.vec = mx_vec(l.y, l.ld_y, l.d_out, BF16 ? 2 : 4);
    a.status = l.status, a.limit = l.limit, a.stall = l.stall;
    auto kernel = mx_linear_big_kernel<KIND, BF16>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MX_MAX_SMEM);
    if (e != cudaSuccess) return cuda_rc(e);
    // all of the shared memory: one block an SM, as its tensor memory asks for
    return launch_after(kernel, dim3((unsigned)(2 * std::min(a.tiles, sms / 2))), BIG_THREADS, MX_MAX_SMEM, 2, st, a);
}

// Few rows or many, by the time each would take.  The pair kernel: 4.5 us, and per round of its 256 x 256 tiles 3.5 us
// and 310 (MXFP8) or 165 ns a scale tile of k.  Measured, us few / many, MXFP8 then MXFP4: 128 x 4096 x 28672 22.9 / 32.1,
// 17.3 / 23.9; 256 x 4096 x 28672 38.5 / 32.3, 24.8 / 24.0; 256 x 14336 x 4096 21.7 / 39.1, 14.9 / 23.4;
// 512 x 14336 x 4096 34.2 / 40.2, 20.6 / 24.1; 768 x 14336 x 4096 45.8 / 43.5 (few rows taken), 27.1 / 25.4;
// 768 x 4096 x 4096 16.2 / 17.3, 10.8 / 12.2; 1024 x 14336 x 1024 21.0 / 38.8, 14.4 / 23.0.
template <int KIND, typename Y>
int launch_linear(const MxLinArgs &a, const lora_mx *x, const lora_mx *w, int dev, int sms, cudaStream_t st) {
    const int64_t tiles = (int64_t)((a.T + 255) / 256) * ((a.d_out + 255) / 256), pairs = std::max(1, sms / 2);
    const int64_t many_ns = 4500 + (tiles + pairs - 1) / pairs * (3500 + (int64_t)a.n_kt * (KIND == MX_A8 ? 310 : 165));
    int took = 0;
    const int rc = launch_few<KIND, Y>(a, x, w, dev, many_ns, &took, st);
    if (rc != LORA_OK || took) return rc;
    return launch_big<KIND, std::is_same<Y, __nv_bfloat16>::value>(a, x, w, sms, st);
}

}  // namespace

}  // namespace lora

extern "C" {

int lora_mx_linear(void *y, int64_t ld_y, const lora_mx *x, const lora_mx *w, int32_t T, lora_dtype dtype,
                   int32_t *status, void *stream) {
    using namespace lora;
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    if (T < 0 || T > LORA_MAX_ROWS) return LORA_ERR_SHAPE;
    int rc = check_mx(x, T);
    if (rc == LORA_OK) rc = check_mx(w, 1);
    if (rc != LORA_OK) return rc;
    if (w->format != LORA_MXFP4) return LORA_ERR_DTYPE;
    if (x->cols != w->cols || ld_y < w->rows) return LORA_ERR_SHAPE;
    if (!status) return LORA_ERR_NULL;
    if (T == 0) return LORA_OK;
    if (!y) return LORA_ERR_NULL;
    MxLinArgs a{};
    a.sw = w->scales, a.sx = x->scales, a.y = y, a.ld_y = ld_y, a.T = T, a.d_out = w->rows;
    a.n_kt = (int)(mx_padded(x->cols) / MX_TILE_COLS);
    a.status = status;
    const char *stall = std::getenv("LORA_DEBUG_STALL");   // test hook: the waits of one role run out, after a short while
    a.stall = stall ? std::atoi(stall) : 0;
    a.limit = a.stall ? 64 : WAIT_LIMIT;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_rc(e);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool a8 = x->format == LORA_MXFP8;
    a.n_stage = a8 ? a.n_kt : (a.n_kt + 1) / 2;
    if (dtype == LORA_BF16)
        return a8 ? launch_linear<MX_A8, __nv_bfloat16>(a, x, w, dev, sms, st)
                  : launch_linear<MX_A4, __nv_bfloat16>(a, x, w, dev, sms, st);
    return a8 ? launch_linear<MX_A8, float>(a, x, w, dev, sms, st) : launch_linear<MX_A4, float>(a, x, w, dev, sms, st);
}

}  // extern "C"
