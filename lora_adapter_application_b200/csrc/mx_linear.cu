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
// four to a ring stage: 128 columns of K (MXFP8) or 256 (MXFP4).  The storage's
// 512-byte scale tile (128 rows x 4 blocks, 16 bytes for rows r, r+32, r+64,
// r+96) is what tcgen05.cp.32x128b.warpx4 spreads over tensor memory as the
// MMA wants it: lane r, one column per 32 rows, a byte per block.
#include "mx.cuh"
#include "ptx.cuh"
#include "tc.cuh"

#include <algorithm>
#include <mutex>

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
    int y_bf16;
    int32_t *status;
};

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
// One lane of a full warp, the same at every call.  The tensor-core and copy instructions want
// warp-uniform operands: behind this test the compiler knows that one lane runs and
// issues them in a few cycles; behind `lane == 0` each takes about 60 (measured: 59 against 38
// clocks an MMA of N = 16, 49 against 3 a commit).
__device__ __forceinline__ bool elect_one() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}\n" : "=r"(p));
    return p != 0;
}

// 16 bytes to four columns of this thread's tensor-memory lane
__device__ __forceinline__ void tmem_st4(uint32_t taddr, uint4 v) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1,%2,%3,%4};\n" ::"r"(taddr), "r"(v.x), "r"(v.y), "r"(v.z),
                 "r"(v.w)
                 : "memory");
}
__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;\n" ::: "memory"); }
// 8 bytes into the shared memory of a block of the cluster, counted on its barrier (see st_async_f4)
__device__ __forceinline__ void st_async_f2(uint32_t addr, float a, float b, uint32_t bar) {
    asm volatile("st.async.shared::cluster.mbarrier::complete_tx::bytes.v2.f32 [%0], {%1,%2}, [%3];\n" ::"r"(addr), "f"(a),
                 "f"(b), "r"(bar)
                 : "memory");
}
// arrival on a barrier of a block of the cluster (address mapped with map_rank); it orders tensor
// memory only (through the tcgen05 fences), so it needs no release
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(bar) : "memory");
}

// This thread's 16 columns of its feature f to the blocks that own them (block r: 16 / S columns from
// r * 16 / S), at [source][feature][column] of their buffer, counted on their barrier.
__device__ __forceinline__ void send_chunk(const float *d, uint32_t buf, uint32_t bar, int S, int rank, int f) {
    if (S == 8) {
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const uint32_t to = map_rank(buf + (uint32_t)((rank * 128 + f) * 8), (uint32_t)r), tb = map_rank(bar, (uint32_t)r);
            st_async_f2(to, d[2 * r], d[2 * r + 1], tb);
        }
    } else {
#pragma unroll
        for (int g = 0; g < 4; ++g) {   // four columns at a time: all of one owner
            const int share = 16 / S, r = 4 * g / share;
            const uint32_t to = map_rank(buf + (uint32_t)((rank * 128 + f) * share + 4 * g - r * share) * 4u, (uint32_t)r);
            st_async_f4(to, d[4 * g], d[4 * g + 1], d[4 * g + 2], d[4 * g + 3], map_rank(bar, (uint32_t)r));
        }
    }
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
template <class Args>
__device__ __forceinline__ void y_store(const Args &a, int64_t row, int64_t col, float v) {
    if (a.y_bf16) y_store<true>(a.y, row * a.ld_y + col, v);
    else y_store<false>(a.y, row * a.ld_y + col, v);
}

// A place in a ring of n slots: the slot and the parity of its current use.  Kept by counting: a
// single thread's integer division costs as much as the MMAs of a stage.
struct Ring {
    int slot = 0, n;
    unsigned parity = 0;
    int64_t count = 0;   // uses so far
    __device__ explicit Ring(int n_) : n(n_) {}
    __device__ void next() {
        ++count;
        if (++slot == n) slot = 0, parity ^= 1u;
    }
    __device__ bool reused() const { return count >= n; }
};

// after a failed wait: the copies that a thread has under way into a ring land before its block goes
__device__ __forceinline__ void drain_ring(Ring r, uint32_t full) {
    for (int j = 0; j < r.n; ++j, r.next())   // oldest first: parity ^ 1 is that of the slot's last use
        for (unsigned w = 0; r.reused() && w < 1024 && !mbar_try<false>(full + 8u * (uint32_t)r.slot, r.parity ^ 1u); ++w) {}
}

// ---------------------------------------------------------------- few rows
// A cluster takes 128 output features (the MMA's M side: W's rows, which a small
// batch reads once) x BN rows of x (its N side, any multiple of 16 up to 192), each of its S
// blocks over 1 / S of k; persistent, cluster c takes tiles c, c + clusters, ....
// k goes in blocks of 256 columns (two scale tiles).  Roles: one thread copies W into a ring of up to
// FEW_STAGES slots, one copies x into it and scales into FEW_SF slots, one issues MMAs,
// four warps move scales from shared to tensor memory, four take the finished
// accumulator (two of them, so the next tile's products overlap) and add the S
// partial sums, in block order, through distributed shared memory: 16 columns at a
// time, block r owning 16 / S of them, sent as st.async counted on the receiver's barrier
// (four buffers: a block sends chunk i + 1 after reading chunk i - 1, which every block sent
// after reading chunk i - 3; so a buffer's last chunk has been read everywhere when its next is sent).
//
// Bound: W's bytes from HBM (64 rows, 4096 -> 28672: 66 MB), or, per SM, filling shared memory.
constexpr int FEW_THREADS = 352;      // warp 0 copies W, 1 MMAs, 2-5 scales, 6-9 sums and stores, 10 copies x and scales
constexpr int FEW_STAGES = 12;
constexpr int FEW_SF = 8;
constexpr int FEW_XCH = 4;            // exchange buffers of 8 KB
constexpr int FEW_ROWS = 192;         // widest BN
constexpr size_t MX_MAX_SMEM = 226 * 1024;

struct MxFewArgs {
    CUtensorMap tmW, tmX;
    const uint8_t *sw, *sx;
    void *y;
    int64_t ld_y;
    int T, d_out, n_kt, n_kb;   // k in scale tiles (128) and in blocks of two
    int bn, nt, tiles;          // rows of a tile, row tiles, all tiles
    int bands, x_bands;         // 128-row bands of x scales one tile may touch; that x has
    int stages, sf_slots, split;
    int y_bf16;
    int32_t *status;
};

template <int KIND>
__global__ void __launch_bounds__(FEW_THREADS, 1) mx_linear_few_kernel(const __grid_constant__ MxFewArgs a) {
    extern __shared__ __align__(1024) unsigned char mx_sm[];
    __shared__ uint32_t tmem_sm;
    __shared__ __align__(8) uint64_t bars[2 * FEW_STAGES + 3 * FEW_SF + 4 + FEW_XCH];
    constexpr int SUBS = KIND == MX_A8 ? 2 : 1;   // ring stages of a k block
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t slot_bytes = 16384u + (uint32_t)a.bn * 128u, sf_bytes = (uint32_t)(1 + a.bands) * 2 * MX_TILE_BYTES;
    const uint32_t base = (smem_u32(mx_sm) + 1023u) & ~1023u;
    const uint32_t sf_base = base + (uint32_t)a.stages * slot_bytes, red = sf_base + (uint32_t)a.sf_slots * sf_bytes;
    auto bar = [&](int i) { return smem_u32(&bars[i]); };
    auto full = [&](int s) { return bar(s); };
    auto empty = [&](int s) { return bar(FEW_STAGES + s); };
    auto sf_full = [&](int s) { return bar(2 * FEW_STAGES + s); };
    auto sf_ready = [&](int s) { return bar(2 * FEW_STAGES + FEW_SF + s); };
    auto sf_empty = [&](int s) { return bar(2 * FEW_STAGES + 2 * FEW_SF + s); };
    auto acc_full = [&](int b) { return bar(2 * FEW_STAGES + 3 * FEW_SF + b); };
    auto acc_empty = [&](int b) { return bar(2 * FEW_STAGES + 3 * FEW_SF + 2 + b); };
    auto xch = [&](int b) { return bar(2 * FEW_STAGES + 3 * FEW_SF + 4 + b); };
    const int S = a.split, rank = S > 1 ? (int)cluster_rank() : 0;
    const int c0 = (int)blockIdx.x / S, clusters = (int)gridDim.x / S;
    const int kb_lo = (int)((int64_t)a.n_kb * rank / S), kb_hi = (int)((int64_t)a.n_kb * (rank + 1) / S);
    const uint32_t acc_cols = ((uint32_t)a.bn + 31u) & ~31u, xc = a.bn > 128 ? 8u : 4u, sf_cols = 8u + 2u * xc;
    const uint32_t tmem_cols = pow2_cols(2 * acc_cols + (uint32_t)a.sf_slots * sf_cols);
    bool failed = false;

    // a warp's place: tile t (m0, n0: its first feature and row), k block kb, stage sub of the block
    int t = c0, m0 = c0 / a.nt * 128, n0 = c0 % a.nt * a.bn, kb = kb_lo, sub = 0;
    Ring ring(a.stages), sfr(a.sf_slots);
    auto next_tile = [&]() {
        t += clusters;
        m0 = t / a.nt * 128, n0 = t % a.nt * a.bn;
    };

    if (warp == 0) {
        for (int i = lane; i < 2 * FEW_STAGES + 3 * FEW_SF + 4 + FEW_XCH; i += 32) {
            const bool two = i < FEW_STAGES;                                                // full: both copying warps
            const bool four = (i >= 2 * FEW_STAGES + FEW_SF && i < 2 * FEW_STAGES + 2 * FEW_SF) ||      // sf_ready
                              (i >= 2 * FEW_STAGES + 3 * FEW_SF + 2 && i < 2 * FEW_STAGES + 3 * FEW_SF + 4);   // acc_empty
            mbar_init(bar(i), two ? 2 : four ? 4 : 1);
        }
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        if (lane == 0) prefetch_tmap(&a.tmW);
    } else if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_sm)),
                     "r"(tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    } else if (warp == 10) {
        if (lane == 0) prefetch_tmap(&a.tmX);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (S > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");   // this block's barriers are set
    const uint32_t tmem = tmem_sm, sf = tmem + 2 * acc_cols;

    if (warp == 0) {
        if (elect_one()) {
            for (; t < a.tiles && !failed; next_tile())
                for (kb = kb_lo; kb < kb_hi && !failed; ++kb)
                    for (sub = 0; sub < min(SUBS, a.n_kt - 2 * kb); ++sub, ring.next()) {
                        const int s = ring.slot;
                        if (ring.reused() && !mbar_wait(empty(s), ring.parity ^ 1u, a.status, failed)) break;
                        mbar_expect_tx(full(s), KIND == MX_A8 ? 8192u : 16384u);   // packed4 boxes count packed bytes
                        tma_2d(base + (uint32_t)s * slot_bytes, &a.tmW, (SUBS * kb + sub) * 128, m0, full(s));
                    }
            if (failed) drain_ring(ring, full(0));
        }
        __syncwarp();
    } else if (warp == 10) {
        if (elect_one()) {
            for (; t < a.tiles && !failed; next_tile()) {
                const int xb = n0 / 128, nb = min(a.bands, a.x_bands - xb);
                for (kb = kb_lo; kb < kb_hi && !failed; ++kb, sfr.next()) {
                    const int l = sfr.slot, tiles = min(2, a.n_kt - 2 * kb);
                    if (sfr.reused() && !mbar_wait(sf_empty(l), sfr.parity ^ 1u, a.status, failed)) break;
                    const uint32_t dst = sf_base + (uint32_t)l * sf_bytes, n = (uint32_t)tiles * MX_TILE_BYTES;
                    mbar_expect_tx(sf_full(l), (uint32_t)(1 + nb) * n);
                    bulk_g2s(dst, a.sw + ((int64_t)(m0 / 128) * a.n_kt + 2 * kb) * MX_TILE_BYTES, n, sf_full(l));
                    for (int b = 0; b < nb; ++b)
                        bulk_g2s(dst + (uint32_t)(1 + b) * 2 * MX_TILE_BYTES,
                                 a.sx + ((int64_t)(xb + b) * a.n_kt + 2 * kb) * MX_TILE_BYTES, n, sf_full(l));
                    for (sub = 0; sub < min(SUBS, tiles); ++sub, ring.next()) {
                        const int s = ring.slot;
                        if (ring.reused() && !mbar_wait(empty(s), ring.parity ^ 1u, a.status, failed)) break;
                        mbar_expect_tx(full(s), (uint32_t)a.bn * 128u);
                        tma_2d(base + (uint32_t)s * slot_bytes + 16384u, &a.tmX, (SUBS * kb + sub) * 128, n0, full(s));
                    }
                }
            }
            if (failed) drain_ring(sfr, sf_full(0)), drain_ring(ring, full(0));
        }
        __syncwarp();
    } else if (warp == 1) {
        if (elect_one()) {
            const uint32_t idesc = KIND == MX_A8 ? mx_idesc(5, 0, 128, a.bn) : mx_idesc(1, 1, 128, a.bn);
            int n = 0;
            for (; t < a.tiles && !failed; next_tile(), ++n) {
                const int b = n & 1;
                if (n >= 2 && !mbar_wait(acc_empty(b), (unsigned)(n / 2 - 1) & 1u, a.status, failed)) break;
                const uint32_t d = tmem + (uint32_t)b * acc_cols;
                for (kb = kb_lo; kb < kb_hi && !failed; ++kb, sfr.next()) {
                    const int l = sfr.slot, tiles = min(2, a.n_kt - 2 * kb);
                    if (!mbar_wait(sf_ready(l), sfr.parity, a.status, failed)) break;
                    const uint32_t ta = sf + sf_cols * (uint32_t)l, tb = ta + 8;
                    for (sub = 0; sub < min(SUBS, tiles); ++sub, ring.next()) {
                        const int s = ring.slot;
                        if (!mbar_wait(full(s), ring.parity, a.status, failed)) break;
                        tc_fence_after();
                        const uint32_t slot = base + (uint32_t)s * slot_bytes;
                        mx_stage_mmas<KIND, false>(d, slot, slot + 16384u, ta + 4 * sub, tb + xc * sub, (int)xc, tiles, idesc,
                                                   kb == kb_lo && sub == 0);
                        tc_commit(empty(s));
                    }
                    tc_commit(sf_empty(l));
                }
                tc_commit(acc_full(b));
            }
        }
        __syncwarp();
    } else if (warp < 6) {
        const uint32_t dst = sf + ((uint32_t)(32 * (warp & 3)) << 16);
        for (; t < a.tiles && !failed; next_tile()) {
            const int xb = n0 / 128, last = min(a.bands, a.x_bands - xb) - 1;
            for (kb = kb_lo; kb < kb_hi; ++kb, sfr.next()) {
                const int l = sfr.slot;
                if (!warp_wait(sf_full(l), sfr.parity, a.status, failed)) break;
                const uint32_t src = sf_base + (uint32_t)l * sf_bytes, to = dst + sf_cols * (uint32_t)l;
#pragma unroll
                for (int k = 0; k < 2; ++k) {   // a tile past k's end is old data that no MMA reads
                    // W: lane r gets the 16 bytes of rows r, r + 32, r + 64, r + 96
                    tmem_st4(to + 4 * k, lds128(src + k * MX_TILE_BYTES + 16 * lane));
                    // x: the tile's rows start anywhere in a band; column g, lane r: row n0 + 32 g + r
                    for (uint32_t g = 0; g < xc; g += 4) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int row = n0 + 32 * (int)(g + i) + lane, band = min(row / 128 - xb, last);
                            w[i] = lds32(src + (uint32_t)(1 + band) * 2 * MX_TILE_BYTES + k * MX_TILE_BYTES +
                                         (uint32_t)(row % 32 * 16 + row / 32 % 4 * 4));
                        }
                        tmem_st4(to + 8 + xc * k + g, make_uint4(w[0], w[1], w[2], w[3]));
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(sf_ready(l));
            }
        }
    } else {
        const int q = warp & 3, f = 32 * q + lane;   // this thread's output feature of the tile
        const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16);
        if (S > 1) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");   // every block's barriers are set
        const int share = 16 / S;
        int n = 0;
        uint32_t chunk = 0, sent = 0;
        for (; t < a.tiles && !failed; next_tile(), ++n) {
            const int b = n & 1;
            const int64_t m = m0 + f;
            if (!warp_wait(acc_full(b), (unsigned)(n / 2) & 1u, a.status, failed)) break;
            tc_fence_after();
            const int rows = min(a.bn, a.T - n0);
            const uint32_t src_acc = acc + (uint32_t)b * acc_cols;
            if (S == 1) {
                for (int c = 0; c < rows; c += 16) {
                    float d[16];
                    tc_ld16(src_acc + c, d);
                    tc_wait_ld();
                    if (m < a.d_out)
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (c + j < rows) y_store(a, n0 + c + j, m, d[j]);
                }
            } else {
                auto send = [&](int c) {
                    float d[16];
                    tc_ld16(src_acc + c, d);
                    tc_wait_ld();
                    const uint32_t p = sent++ & (FEW_XCH - 1);
                    if (threadIdx.x == 192) mbar_expect_tx(xch((int)p), 8192);
                    send_chunk(d, red + p * 8192u, xch((int)p), S, rank, f);
                };
                send(0);
                for (int c = 0; c < rows; c += 16) {
                    if (c + 16 < rows) send(c + 16);
                    const uint32_t p = chunk & (FEW_XCH - 1), buf = red + p * 8192u;
                    if (!warp_wait(xch((int)p), chunk / FEW_XCH & 1u, a.status, failed)) break;
                    ++chunk;
                    if (m < a.d_out)
                        for (int j = 0; j < share; ++j) {
                            const int row = c + rank * share + j;
                            if (row >= rows) break;
                            float v = 0.f;
                            for (int src = 0; src < S; ++src)
                                v += __uint_as_float(lds32(buf + (uint32_t)(((src * 128 + f) * share + j) * 4)));
                            y_store(a, n0 + row, m, v);
                        }
                }
                if (failed) break;
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(acc_empty(b));
        }
    }
    // ---------------------------------------------------------------- teardown
    // A block may go once it has all its chunks: nothing more is sent to it.  After a failed wait that
    // is not known: the block stays until what is under way has landed and its peers have left or failed too.
    __syncwarp();
    tc_fence_before();
    if (__syncthreads_or(failed) && S > 1) {
        for (int i = 0; i < 100; ++i) __nanosleep(1000);
        __syncwarp();
        if (warp < 6 || warp == 10) asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
        cluster_sync_all();
    }
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(tmem_cols) : "memory");
    }
}

// Blocks along k, clusters of them that fit the device at once, and the time they would take (in k blocks
// a block goes through, a tile's fixed cost counted as TILE_COST of them).
struct FewPlan {
    int split = 1, clusters = 1;
};
template <int KIND>
int few_plan(int tiles, int n_kb, int dev, FewPlan *out) {
    // clusters resident at once: a property of the device and the kernel, asked for once
    static std::mutex mu;
    static int fit[64][4] = {};
    constexpr int TILE_COST = 3;
    std::lock_guard<std::mutex> lock(mu);
    int *f = fit[dev & 63];
    auto kernel = mx_linear_few_kernel<KIND>;
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
            if (e == cudaSuccess) f[i] = std::max(1, n);
        }
        if (e != cudaSuccess) return cuda_rc(e);
    }
    int64_t best = -1;
    for (int i = 0; i < 4; ++i) {
        const int s = 1 << i, n = std::min(tiles, f[i]);
        if (s > n_kb) break;
        const int64_t cost = (int64_t)((tiles + n - 1) / n) * ((n_kb + s - 1) / s + (i ? TILE_COST : 0));
        if (best < 0 || cost < best) best = cost, out->split = s, out->clusters = n;
    }
    return LORA_OK;
}

template <int KIND>
int launch_few(const MxLinArgs &l, const lora_mx *x, const lora_mx *w, int dev, cudaStream_t st) {
    MxFewArgs a{};
    const uint64_t xb = (uint64_t)mx_row_bytes(x->format, x->cols), wb = (uint64_t)mx_row_bytes(w->format, w->cols);
    a.nt = (l.T + FEW_ROWS - 1) / FEW_ROWS;
    a.bn = ((l.T + a.nt - 1) / a.nt + 15) / 16 * 16;
    a.nt = (l.T + a.bn - 1) / a.bn;
    const int mt = (l.d_out + 127) / 128;
    a.tiles = mt * a.nt;
    int rc = tensor_map_mx(&a.tmW, w->q, wb, (uint64_t)l.d_out, wb, 128, KIND == MX_A8);
    if (rc == LORA_OK) rc = tensor_map_mx(&a.tmX, x->q, xb, (uint64_t)l.T, xb, (uint32_t)a.bn, false);
    if (rc != LORA_OK) return rc;
    a.sw = l.sw, a.sx = l.sx, a.y = l.y, a.ld_y = l.ld_y, a.T = l.T, a.d_out = l.d_out, a.n_kt = l.n_kt;
    a.n_kb = (l.n_kt + 1) / 2;
    a.x_bands = (l.T + 127) / 128;
    a.bands = std::min(a.x_bands, a.nt == 1 ? (a.bn + 127) / 128 : (a.bn + 126) / 128 + 1);
    a.y_bf16 = l.y_bf16;
    a.status = l.status;
    FewPlan plan;
    rc = few_plan<KIND>(a.tiles, a.n_kb, dev, &plan);
    if (rc != LORA_OK) return rc;
    a.split = plan.split;
    const uint32_t acc_cols = ((uint32_t)a.bn + 31u) & ~31u, sf_cols = a.bn > 128 ? 24u : 16u;
    a.sf_slots = std::min(FEW_SF, (int)((512 - 2 * acc_cols) / sf_cols));
    const size_t slot = 16384 + (size_t)a.bn * 128, sf = (size_t)a.sf_slots * (1 + a.bands) * 2 * MX_TILE_BYTES;
    a.stages = (int)std::min<size_t>(FEW_STAGES, (MX_MAX_SMEM - 1024 - sf - (plan.split > 1 ? FEW_XCH * 8192 : 0)) / slot);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(plan.split * plan.clusters));
    cfg.blockDim = dim3(FEW_THREADS);
    cfg.dynamicSmemBytes = MX_MAX_SMEM;   // one block an SM: two might wait for each other's tensor memory
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)plan.split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, mx_linear_few_kernel<KIND>, a);
    return cuda_rc(e != cudaSuccess ? e : cudaGetLastError());
}

// ---------------------------------------------------------------- many rows
// A pair of blocks (a cluster, cta_group::2) takes 256 rows of x (M) x 256 output
// features (N): each block loads its own 128 rows of x and 128 of W's rows, the
// tensor cores share the halves, so a block moves 32 KB of a stage for 256 x 256 x 32
// bytes of products, half of what two 128 x 256 tiles would.  At the 4-bit rate that
// is 64 bytes a clock and SM from L2: the reason for the pair.  Persistent: pair p
// takes tiles p, p + pairs, ..., x's tiles fastest (concurrent pairs share W's rows and keep x in L2).
// The fp32 accumulator (256 columns) is drained to registers by eight warps in one
// go, the next tile's products start, and the rows are stored meanwhile.
constexpr int BIG_THREADS = 448;      // warp 0 copies, warp 1 MMAs, warps 2-5 scales, warps 6-13 epilogue
constexpr int BIG_STAGES = 6;

struct MxBigArgs {
    CUtensorMap tmX, tmW;
    const uint8_t *sx, *sw;
    int x_bands, w_bands;   // 128-row bands of x and W
    void *y;
    int64_t ld_y;
    int T, d_out, n_kt, n_stage;
    int mt, tiles;    // 256-row tiles of x; all tiles
    int vec;          // y rows allow 16-byte stores
    int32_t *status;
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
    __shared__ __align__(8) uint64_t bars[4 * BIG_STAGES + 2];
    constexpr int TPS = mx_tiles_per_stage<KIND>();
    constexpr uint32_t SLOT = big_slot_stride<KIND>();
    constexpr uint32_t SF_COLS = 12 * TPS;   // one stage's scales: 4 columns a tile for x, 8 for W
    constexpr uint32_t TX = 2u * (KIND == MX_A8 ? 16384u + 8192u : 32768u);   // packed4 boxes count packed bytes
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(mx_sm) + 1023u) & ~1023u;
    const int rank = (int)cluster_rank();
    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    auto full = [&](int s) { return smem_u32(&bars[s]); };                  // the leader's counts both blocks' bytes
    auto empty = [&](int s) { return smem_u32(&bars[BIG_STAGES + s]); };
    auto sf_full = [&](int s) { return smem_u32(&bars[2 * BIG_STAGES + s]); };    // this block's scales have landed
    auto sf_ready = [&](int s) { return smem_u32(&bars[3 * BIG_STAGES + s]); };   // the leader's: both blocks' are in tensor memory
    const uint32_t acc_full = smem_u32(&bars[4 * BIG_STAGES]), acc_empty = smem_u32(&bars[4 * BIG_STAGES + 1]);

    if (threadIdx.x == 0) {
        for (int s = 0; s < BIG_STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
            mbar_init(sf_full(s), 1);
            mbar_init(sf_ready(s), 8);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 16);   // the leader's: 8 epilogue warps of each block
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
    const uint32_t tmem = tmem_sm, sf = tmem + 256;
    bool failed = false;

    if (warp == 0) {
        if (elect_one()) {
            int it = 0;
            for (int t = pair; t < a.tiles && !failed; t += pairs) {
                const int m0 = (t % a.mt) * 256 + 128 * rank, nb = t / a.mt * 2;   // nb: first 128-row band of W
                // bands past the last hold rows that no result uses: any scales will do
                const uint8_t *sx = a.sx + (int64_t)min(m0 / 128, a.x_bands - 1) * a.n_kt * MX_TILE_BYTES;
                const uint8_t *sw0 = a.sw + (int64_t)nb * a.n_kt * MX_TILE_BYTES;
                const uint8_t *sw1 = a.sw + (int64_t)min(nb + 1, a.w_bands - 1) * a.n_kt * MX_TILE_BYTES;
                for (int i = 0; i < a.n_stage; ++i, ++it) {
                    const int s = it % BIG_STAGES;
                    if (it >= BIG_STAGES && !mbar_wait(empty(s), (unsigned)(it / BIG_STAGES - 1) & 1u, a.status, failed))
                        break;
                    const uint32_t slot = base + (uint32_t)s * SLOT, bar = map_rank(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), TX);
                    tma_2d_pair(slot, &a.tmX, i * 128, m0, bar);
                    tma_2d_pair(slot + 16384u, &a.tmW, i * 128, (nb + rank) * 128, bar);
                    const uint32_t sfs = slot + 32768u, sb = (uint32_t)min(TPS, a.n_kt - i * TPS) * MX_TILE_BYTES;
                    const int64_t off = (int64_t)i * TPS * MX_TILE_BYTES;
                    mbar_expect_tx(sf_full(s), 3 * sb);
                    bulk_g2s(sfs, sx + off, sb, sf_full(s));
                    bulk_g2s(sfs + TPS * MX_TILE_BYTES, sw0 + off, sb, sf_full(s));
                    bulk_g2s(sfs + 2 * TPS * MX_TILE_BYTES, sw1 + off, sb, sf_full(s));
                }
            }
            // after a failed wait: both blocks' copies under way land before the pair goes
            for (int j = failed ? max(0, it - BIG_STAGES) : it; j < it; ++j) {
                const unsigned par = (unsigned)(j / BIG_STAGES) & 1u;
                for (unsigned w = 0; w < 1024 && !mbar_try<false>(sf_full(j % BIG_STAGES), par); ++w) {}
                for (unsigned w = 0; rank == 0 && w < 1024 && !mbar_try<false>(full(j % BIG_STAGES), par); ++w) {}
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = KIND == MX_A8 ? mx_idesc(0, 5, 256, 256) : mx_idesc(1, 1, 256, 256);
            int it = 0, n = 0;
            for (int t = pair; t < a.tiles && !failed; t += pairs, ++n) {
                if (n > 0 && !mbar_wait<true>(acc_empty, (unsigned)(n - 1) & 1u, a.status, failed)) break;
                tc_fence_after();
                for (int i = 0; i < a.n_stage; ++i, ++it) {
                    const int s = it % BIG_STAGES;
                    if (!mbar_wait(full(s), (unsigned)(it / BIG_STAGES) & 1u, a.status, failed) ||
                        !mbar_wait(sf_ready(s), (unsigned)(it / BIG_STAGES) & 1u, a.status, failed))
                        break;
                    tc_fence_after();
                    const uint32_t slot = base + (uint32_t)s * SLOT;
                    const uint32_t ta = sf + SF_COLS * (uint32_t)s, tb = ta + 4 * TPS;
                    const int tiles = min(TPS, a.n_kt - i * TPS);
                    mx_stage_mmas<KIND, true>(tmem, slot, slot + 16384u, ta, tb, 8, tiles, idesc, i == 0);
                    tc_commit_pair(empty(s));
                }
                tc_commit_pair(acc_full);
            }
        }
        __syncwarp();
    } else if (warp < 6) {
        // The scales of a stage from shared to tensor memory: lane r of each of the four
        // partitions gets the 16 bytes of rows r, r + 32, r + 64, r + 96.  The slot's columns are free
        // once its shared memory is: both were read by the same MMAs.
        const uint32_t dst = sf + ((uint32_t)(32 * (warp & 3)) << 16);
        int it = 0;
        for (int t = pair; t < a.tiles && !failed; t += pairs)
            for (int i = 0; i < a.n_stage; ++i, ++it) {
                const int s = it % BIG_STAGES;
                if (!warp_wait(sf_full(s), (unsigned)(it / BIG_STAGES) & 1u, a.status, failed)) break;
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
        for (int t = pair; t < a.tiles; t += pairs, ++n) {
            if (!warp_wait(acc_full, (unsigned)n & 1u, a.status, failed)) break;
            tc_fence_after();
            const int64_t row = (int64_t)(t % a.mt) * 256 + 128 * rank + 32 * q + lane;
            const int64_t col = (int64_t)(t / a.mt) * 256 + 128 * half;
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
    tc_fence_before();
    cluster_sync_all();
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
    a.tiles = a.mt * ((l.d_out + 255) / 256);
    a.vec = mx_vec(l.y, l.ld_y, l.d_out, BF16 ? 2 : 4);
    a.status = l.status;
    auto kernel = mx_linear_big_kernel<KIND, BF16>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MX_MAX_SMEM);
    if (e != cudaSuccess) return cuda_rc(e);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(2 * std::min(a.tiles, sms / 2)));
    cfg.blockDim = dim3(BIG_THREADS);
    cfg.dynamicSmemBytes = MX_MAX_SMEM;   // one block an SM, by its tensor memory
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = 2;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
    return cuda_rc(e != cudaSuccess ? e : cudaGetLastError());
}

template <int KIND>
int launch_linear(const MxLinArgs &a, const lora_mx *x, const lora_mx *w, int dev, int sms, cudaStream_t st) {
    if (a.T > 512) return a.y_bf16 ? launch_big<KIND, true>(a, x, w, sms, st) : launch_big<KIND, false>(a, x, w, sms, st);
    return launch_few<KIND>(a, x, w, dev, st);
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
    a.y_bf16 = dtype == LORA_BF16;
    a.status = status;
    int dev = 0, sms = 148;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e != cudaSuccess) return cuda_rc(e);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (x->format == LORA_MXFP8) {
        a.n_stage = a.n_kt;
        return launch_linear<MX_A8>(a, x, w, dev, sms, st);
    }
    a.n_stage = (a.n_kt + 1) / 2;
    return launch_linear<MX_A4>(a, x, w, dev, sms, st);
}

}  // extern "C"
