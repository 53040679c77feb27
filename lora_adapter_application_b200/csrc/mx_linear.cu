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

struct MxLinArgs {
    CUtensorMap tmW, tmX;
    const uint8_t *sw, *sx;
    void *y;
    int64_t ld_y;
    int T, d_out;
    int n_kt;      // scale tiles along k: padded columns / 128
    int n_stage;   // ring stages of k
    int stages;    // ring depth
    int split;     // blocks along k (a cluster)
    int y_bf16;
    int32_t *status;
};

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
// One 512-byte scale tile to four columns of tensor memory, in all four 32-lane
// partitions.  The matrix descriptor: no swizzle, 8-row x 16-byte core matrices 128
// bytes apart.
template <bool PAIR>
__device__ __forceinline__ void mx_scales_to_tmem(uint32_t taddr, uint32_t smem) {
    const uint64_t desc = (uint64_t)((smem >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
    if (PAIR) asm volatile("tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
    else asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}

// The MMAs of one ring stage: n_tiles scale tiles (128 columns of K each) of operands
// at a, b (shared memory) whose scales lie at columns sa, sb of tensor memory,
// four (SB_COLS) columns a tile.
template <int KIND, bool PAIR, int SB_COLS>
__device__ __forceinline__ void mx_stage_mmas(uint32_t d, uint32_t a, uint32_t b, uint32_t sa, uint32_t sb, int n_tiles,
                                              uint32_t idesc, bool first) {
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
                                   sb + SB_COLS * (k >> 1), first && k == 0 ? 0u : 1u);
    }
}

__device__ __forceinline__ void y_store(const MxLinArgs &a, int64_t row, int64_t col, float v) {
    if (a.y_bf16) static_cast<__nv_bfloat16 *>(a.y)[row * a.ld_y + col] = __float2bfloat16_rn(v);
    else static_cast<float *>(a.y)[row * a.ld_y + col] = v;
}

// ---------------------------------------------------------------- few rows
// A block takes 128 output features (the MMA's M side: W's rows) and BN rows of x
// (its N side), over 1 / split of k; the blocks of a cluster share a tile and
// add their partial sums, in block order, through distributed shared memory.
constexpr int SMALL_THREADS = 128;

template <int KIND>
__host__ __device__ constexpr int mx_tiles_per_stage() { return KIND == MX_A8 ? 1 : 2; }
template <int KIND, int BN>
__host__ __device__ constexpr uint32_t small_slot_bytes() {
    return 16384u + BN * 128u + 2u * MX_TILE_BYTES * mx_tiles_per_stage<KIND>();
}
constexpr uint32_t pow2_cols(uint32_t c) { return c <= 32 ? 32 : c <= 64 ? 64 : c <= 128 ? 128 : c <= 256 ? 256 : 512; }
constexpr int MX_MAX_STAGES = 12;
constexpr size_t MX_MAX_SMEM = 226 * 1024;
// Shared memory a block takes at least, in proportion to its share of the SM's
// 512 tensor-memory columns: whatever blocks of these kernels meet on an SM, their
// columns fit.  A block that had to wait for columns could wait for a block whose cluster
// waits for it.
constexpr size_t tmem_share(uint32_t cols) {
    return cols >= 512 ? MX_MAX_SMEM : (size_t)cols * (228 * 1024 / 512) - 1024;
}

template <int KIND, int BN>
__global__ void __launch_bounds__(SMALL_THREADS) mx_linear_small_kernel(const __grid_constant__ MxLinArgs a) {
    extern __shared__ __align__(1024) unsigned char mx_sm[];
    __shared__ uint32_t tmem_sm;
    __shared__ __align__(8) uint64_t bars[2 * MX_MAX_STAGES + 1];
    constexpr int TPS = mx_tiles_per_stage<KIND>();
    constexpr uint32_t SLOT = small_slot_bytes<KIND, BN>();
    constexpr uint32_t SF_COLS = 8 * TPS;   // tensor-memory columns of one stage's scales
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const uint32_t base = (smem_u32(mx_sm) + 1023u) & ~1023u;
    const uint32_t red = base + (uint32_t)a.stages * SLOT;
    auto full = [&](int s) { return smem_u32(&bars[s]); };
    auto empty = [&](int s) { return smem_u32(&bars[MX_MAX_STAGES + s]); };
    const uint32_t done = smem_u32(&bars[2 * MX_MAX_STAGES]);
    const int rank = a.split > 1 ? (int)cluster_rank() : 0;
    const int m0 = (int)blockIdx.y * 128, n0 = (int)blockIdx.z * BN;
    const int k_lo = (int)((int64_t)a.n_stage * rank / a.split), k_hi = (int)((int64_t)a.n_stage * (rank + 1) / a.split);
    const int n = k_hi - k_lo;
    const uint32_t tmem_cols = pow2_cols(BN + SF_COLS * (uint32_t)a.stages);

    if (tid == 0) {
        for (int s = 0; s < a.stages; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        prefetch_tmap(&a.tmW);
        prefetch_tmap(&a.tmX);
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(smem_u32(&tmem_sm)),
                     "r"(tmem_cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (a.split > 1) asm volatile("barrier.cluster.arrive.release.aligned;\n" ::: "memory");   // the peers have started
    const uint32_t tmem = tmem_sm, sf = tmem + BN;
    bool failed = false;

    if (warp == 0) {
        if (lane == 0) {
            const uint8_t *sw = a.sw + (int64_t)(m0 / 128) * a.n_kt * MX_TILE_BYTES;
            const uint8_t *sx = a.sx + (int64_t)(n0 / 128) * a.n_kt * MX_TILE_BYTES;
            int i = 0;
            for (; i < n; ++i) {
                const int s = i % a.stages;
                if (i >= a.stages && !mbar_wait(empty(s), (unsigned)(i / a.stages - 1) & 1u, a.status, failed)) break;
                const uint32_t slot = base + (uint32_t)s * SLOT, sfs = slot + 16384u + BN * 128u;
                const int kt = (k_lo + i) * TPS;
                const uint32_t sb = (uint32_t)min(TPS, a.n_kt - kt) * MX_TILE_BYTES;
                // packed4 boxes count their packed bytes (measured)
                mbar_expect_tx(full(s), (KIND == MX_A8 ? 8192u : 16384u) + BN * 128u + 2 * sb);
                tma_2d(slot, &a.tmW, (k_lo + i) * 128, m0, full(s));
                tma_2d(slot + 16384u, &a.tmX, (k_lo + i) * 128, n0, full(s));
                bulk_g2s(sfs, sw + (int64_t)kt * MX_TILE_BYTES, sb, full(s));
                bulk_g2s(sfs + TPS * MX_TILE_BYTES, sx + (int64_t)kt * MX_TILE_BYTES, sb, full(s));
            }
            // after a failed wait: the copies under way land before the block goes
            for (int j = failed ? max(0, i - a.stages) : i; j < i; ++j)
                for (unsigned t = 0; t < 1024 && !mbar_try<false>(full(j % a.stages), (unsigned)(j / a.stages) & 1u); ++t) {}
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0) {
            constexpr uint32_t idesc = KIND == MX_A8 ? mx_idesc(5, 0, 128, BN) : mx_idesc(1, 1, 128, BN);
            for (int i = 0; i < n; ++i) {
                const int s = i % a.stages;
                if (!mbar_wait(full(s), (unsigned)(i / a.stages) & 1u, a.status, failed)) break;
                tc_fence_after();
                const uint32_t slot = base + (uint32_t)s * SLOT, sfs = slot + 16384u + BN * 128u;
                const uint32_t ta = sf + SF_COLS * (uint32_t)s, tb = ta + 4 * TPS;
                const int tiles = min(TPS, a.n_kt - (k_lo + i) * TPS);
                for (int t = 0; t < tiles; ++t) {
                    mx_scales_to_tmem<false>(ta + 4 * t, sfs + t * MX_TILE_BYTES);
                    mx_scales_to_tmem<false>(tb + 4 * t, sfs + (TPS + t) * MX_TILE_BYTES);
                }
                mx_stage_mmas<KIND, false, 4>(tmem, slot, slot + 16384u, ta, tb, tiles, idesc, i == 0);
                tc_commit(empty(s));
            }
            tc_commit(done);
        }
        __syncwarp();
    }
    const bool ok = warp_wait(done, 0, a.status, failed);
    tc_fence_after();

    const int f = 32 * warp + lane;   // this thread's output feature of the tile
    const uint32_t acc = tmem + ((uint32_t)(32 * warp) << 16);
    if (a.split == 1) {
#pragma unroll 1
        for (int c = 0; c < BN; c += 16) {
            if (n0 + c >= a.T) break;
            float d[16];
            tc_ld16(acc + c, d);
            tc_wait_ld();
            if (ok && m0 + f < a.d_out)
#pragma unroll
                for (int j = 0; j < 16; ++j)
                    if (n0 + c + j < a.T) y_store(a, n0 + c + j, m0 + f, d[j]);
        }
    } else {
        // column c of the tile goes to block c / share, at [source][c % share][feature]
        const int share = BN / a.split;
        asm volatile("barrier.cluster.wait.acquire.aligned;\n" ::: "memory");
#pragma unroll 1
        for (int c = 0; c < BN; c += 16) {
            float d[16];
            tc_ld16(acc + c, d);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int to = (c + j) / share, at = (c + j) - to * share;
                const uint32_t p = map_rank(red + (uint32_t)(((rank * share + at) * 128 + f) * 4), (uint32_t)to);
                asm volatile("st.shared::cluster.f32 [%0], %1;\n" ::"r"(p), "f"(d[j]) : "memory");
            }
        }
        cluster_sync_all();
        if (ok && m0 + f < a.d_out)
            for (int j = 0; j < share; ++j) {
                const int row = n0 + rank * share + j;
                if (row >= a.T) break;
                float v = 0.f;
                for (int src = 0; src < a.split; ++src)
                    v += __uint_as_float(lds32(red + (uint32_t)(((src * share + j) * 128 + f) * 4)));
                y_store(a, row, m0 + f, v);
            }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem), "r"(tmem_cols) : "memory");
    }
}

template <int KIND, int BN>
int launch_small(MxLinArgs &a, int sms, cudaStream_t st) {
    const int mt = (a.d_out + 127) / 128, nt = (a.T + BN - 1) / BN;
    const int64_t tiles = (int64_t)mt * nt;
    a.split = 1;
    while (a.split < 8 && tiles * a.split * 2 <= sms && a.n_stage >= 2 * a.split * 2) a.split *= 2;
    const uint32_t slot = small_slot_bytes<KIND, BN>(), red = a.split > 1 ? 128u * BN * 4u : 0u;
    const uint32_t room = 220u * 1024u - red - 1024u;
    int stages = (int)(room / slot);
    const int tm = (512 - BN) / (8 * mx_tiles_per_stage<KIND>());
    stages = std::min(std::min(stages, MX_MAX_STAGES), std::min(tm, std::max(1, (a.n_stage + a.split - 1) / a.split)));
    a.stages = stages;
    const size_t smem = std::max<size_t>((size_t)stages * slot + red + 1024,
                                         tmem_share(pow2_cols(BN + 8 * mx_tiles_per_stage<KIND>() * stages)));
    auto kernel = mx_linear_small_kernel<KIND, BN>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)MX_MAX_SMEM);
    if (e != cudaSuccess) return cuda_rc(e);
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)a.split, (unsigned)mt, (unsigned)nt);
    cfg.blockDim = dim3(SMALL_THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)a.split;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, kernel, a);
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
constexpr int BIG_THREADS = 320;      // warp 0 copies, warp 1 MMAs, warps 2-9 epilogue
constexpr int BIG_STAGES = 6;

struct MxBigArgs {
    CUtensorMap tmX, tmW, tmSx, tmSw;
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
    __shared__ __align__(8) uint64_t bars[2 * BIG_STAGES + 2];
    constexpr int TPS = mx_tiles_per_stage<KIND>();
    constexpr uint32_t SLOT = big_slot_stride<KIND>();
    constexpr uint32_t SF_COLS = 12 * TPS;   // one stage's scales: 4 columns a tile for x, 8 for W
    constexpr uint32_t TX = 2u * ((KIND == MX_A8 ? 16384u + 8192u : 32768u) + 3u * MX_TILE_BYTES * TPS);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t base = (smem_u32(mx_sm) + 1023u) & ~1023u;
    const int rank = (int)cluster_rank();
    const int pair = (int)blockIdx.x >> 1, pairs = (int)gridDim.x >> 1;
    auto full = [&](int s) { return smem_u32(&bars[s]); };                  // the leader's counts both blocks' bytes
    auto empty = [&](int s) { return smem_u32(&bars[BIG_STAGES + s]); };
    const uint32_t acc_full = smem_u32(&bars[2 * BIG_STAGES]), acc_empty = smem_u32(&bars[2 * BIG_STAGES + 1]);

    if (threadIdx.x == 0) {
        for (int s = 0; s < BIG_STAGES; ++s) {
            mbar_init(full(s), 1);
            mbar_init(empty(s), 1);
        }
        mbar_init(acc_full, 1);
        mbar_init(acc_empty, 16);   // the leader's: 8 epilogue warps of each block
        asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
        prefetch_tmap(&a.tmX);
        prefetch_tmap(&a.tmW);
        prefetch_tmap(&a.tmSx);
        prefetch_tmap(&a.tmSw);
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
        if (lane == 0) {
            int it = 0;
            for (int t = pair; t < a.tiles && !failed; t += pairs) {
                const int m0 = (t % a.mt) * 256 + 128 * rank, nb = t / a.mt * 2;   // nb: first 128-row band of W
                for (int i = 0; i < a.n_stage; ++i, ++it) {
                    const int s = it % BIG_STAGES;
                    if (it >= BIG_STAGES && !mbar_wait(empty(s), (unsigned)(it / BIG_STAGES - 1) & 1u, a.status, failed))
                        break;
                    const uint32_t slot = base + (uint32_t)s * SLOT, bar = map_rank(full(s), 0);
                    if (rank == 0) mbar_expect_tx(full(s), TX);
                    tma_2d_pair(slot, &a.tmX, i * 128, m0, bar);
                    tma_2d_pair(slot + 16384u, &a.tmW, i * 128, (nb + rank) * 128, bar);
                    tma_2d_pair(slot + 32768u, &a.tmSx, 0, m0 / 128 * a.n_kt + i * TPS, bar);
                    tma_2d_pair(slot + 32768u + TPS * MX_TILE_BYTES, &a.tmSw, 0, nb * a.n_kt + i * TPS, bar);
                    tma_2d_pair(slot + 32768u + 2 * TPS * MX_TILE_BYTES, &a.tmSw, 0, (nb + 1) * a.n_kt + i * TPS, bar);
                }
            }
            // after a failed wait: both blocks' copies under way land before the pair goes
            for (int j = failed && rank == 0 ? max(0, it - BIG_STAGES) : it; j < it; ++j)
                for (unsigned w = 0; w < 1024 && !mbar_try<false>(full(j % BIG_STAGES), (unsigned)(j / BIG_STAGES) & 1u); ++w) {}
        }
        __syncwarp();
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            constexpr uint32_t idesc = KIND == MX_A8 ? mx_idesc(0, 5, 256, 256) : mx_idesc(1, 1, 256, 256);
            int it = 0, n = 0;
            for (int t = pair; t < a.tiles && !failed; t += pairs, ++n) {
                if (n > 0 && !mbar_wait<true>(acc_empty, (unsigned)(n - 1) & 1u, a.status, failed)) break;
                tc_fence_after();
                for (int i = 0; i < a.n_stage; ++i, ++it) {
                    const int s = it % BIG_STAGES;
                    if (!mbar_wait(full(s), (unsigned)(it / BIG_STAGES) & 1u, a.status, failed)) break;
                    tc_fence_after();
                    const uint32_t slot = base + (uint32_t)s * SLOT, sfs = slot + 32768u;
                    const uint32_t ta = sf + SF_COLS * (uint32_t)s, tb = ta + 4 * TPS;
                    const int tiles = min(TPS, a.n_kt - i * TPS);
                    for (int k = 0; k < tiles; ++k) {
                        mx_scales_to_tmem<true>(ta + 4 * k, sfs + k * MX_TILE_BYTES);
                        mx_scales_to_tmem<true>(tb + 8 * k, sfs + (TPS + k) * MX_TILE_BYTES);
                        mx_scales_to_tmem<true>(tb + 8 * k + 4, sfs + (2 * TPS + k) * MX_TILE_BYTES);
                    }
                    mx_stage_mmas<KIND, true, 8>(tmem, slot, slot + 16384u, ta, tb, tiles, idesc, i == 0);
                    tc_commit_pair(empty(s));
                }
                tc_commit_pair(acc_full);
            }
        }
        __syncwarp();
    } else {
        const int q = warp & 3, half = (warp - 2) >> 2;
        const uint32_t acc = tmem + ((uint32_t)(32 * q) << 16) + 128u * half;
        const uint32_t release = map_rank(acc_empty, 0);
        int n = 0;
        for (int t = pair; t < a.tiles; t += pairs, ++n) {
            if (!warp_wait(acc_full, (unsigned)n & 1u, a.status, failed)) break;
            tc_fence_after();
            uint32_t d[128];
#pragma unroll
            for (int c = 0; c < 4; ++c) tc_ld32(acc + 32 * c, d + 32 * c);
            tc_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0)
                asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];\n" ::"r"(release) : "memory");
            const int64_t row = (int64_t)(t % a.mt) * 256 + 128 * rank + 32 * q + lane;
            const int col = t / a.mt * 256 + 128 * half;
            if (row < a.T) {
                if (BF16) {
                    __nv_bfloat16 *y = static_cast<__nv_bfloat16 *>(a.y) + row * a.ld_y + col;
#pragma unroll
                    for (int c = 0; c < 128; c += 8) {
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(d[c + j]);
                        if (a.vec) store8<true>(y + c, a.d_out - col - c, v);
                        else store8<false>(y + c, a.d_out - col - c, v);
                    }
                } else {
                    float *y = static_cast<float *>(a.y) + row * a.ld_y + col;
#pragma unroll
                    for (int c = 0; c < 128; c += 8) {
                        float v[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j) v[j] = __uint_as_float(d[c + j]);
                        if (a.vec) store8<true>(y + c, a.d_out - col - c, v);
                        else store8<false>(y + c, a.d_out - col - c, v);
                    }
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
    const uint64_t x_bands = (uint64_t)(l.T + 127) / 128, w_bands = (uint64_t)(l.d_out + 127) / 128;
    constexpr int TPS = mx_tiles_per_stage<KIND>();
    int rc = tensor_map_mx(&a.tmX, x->q, xb, (uint64_t)l.T, xb, 128, false);
    if (rc == LORA_OK) rc = tensor_map_mx(&a.tmW, w->q, wb, (uint64_t)l.d_out, wb, 128, KIND == MX_A8);
    if (rc == LORA_OK) rc = tensor_map_mx_scales(&a.tmSx, x->scales, x_bands * l.n_kt, TPS);
    if (rc == LORA_OK) rc = tensor_map_mx_scales(&a.tmSw, w->scales, w_bands * l.n_kt, TPS);
    if (rc != LORA_OK) return rc;
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
int launch_linear(MxLinArgs &a, const lora_mx *x, const lora_mx *w, int sms, cudaStream_t st) {
    const uint64_t xb = (uint64_t)mx_row_bytes(x->format, x->cols), wb = (uint64_t)mx_row_bytes(w->format, w->cols);
    if (a.T > 512) return a.y_bf16 ? launch_big<KIND, true>(a, x, w, sms, st) : launch_big<KIND, false>(a, x, w, sms, st);
    const uint32_t bn = a.T <= 16 ? 16 : a.T <= 32 ? 32 : a.T <= 64 ? 64 : 128;
    int rc = tensor_map_mx(&a.tmW, w->q, wb, (uint64_t)a.d_out, wb, 128, KIND == MX_A8);
    if (rc == LORA_OK) rc = tensor_map_mx(&a.tmX, x->q, xb, (uint64_t)a.T, xb, bn, false);
    if (rc != LORA_OK) return rc;
    switch (bn) {
        case 16: return launch_small<KIND, 16>(a, sms, st);
        case 32: return launch_small<KIND, 32>(a, sms, st);
        case 64: return launch_small<KIND, 64>(a, sms, st);
        default: return launch_small<KIND, 128>(a, sms, st);
    }
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
        return launch_linear<MX_A8>(a, x, w, sms, st);
    }
    a.n_stage = (a.n_kt + 1) / 2;
    return launch_linear<MX_A4>(a, x, w, sms, st);
}

}  // extern "C"
