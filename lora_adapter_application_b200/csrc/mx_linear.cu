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

template <int KIND>
__device__ __forceinline__ void mx_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sa, uint32_t sb,
                                       uint32_t acc) {
    if (KIND == MX_A8)
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf8f6f4.block_scale.scale_vec::1X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %6, 0;\n\t"
            "tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}\n" ::
                "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(sa), "r"(sb), "r"(acc)
            : "memory");
}
// One 512-byte scale tile to four columns of tensor memory, in all four 32-lane
// partitions.  The matrix descriptor: no swizzle, 8-row x 16-byte core matrices 128
// bytes apart.
__device__ __forceinline__ void mx_scales_to_tmem(uint32_t taddr, uint32_t smem) {
    const uint64_t desc = (uint64_t)((smem >> 4) & 0x3FFFu) | (1ull << 16) | ((uint64_t)(128 >> 4) << 32) | (1ull << 46);
    asm volatile("tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n" ::"r"(taddr), "l"(desc) : "memory");
}

// The MMAs of one ring stage: n_tiles scale tiles (128 columns of K each) of operands
// at a, b (shared memory) whose scales lie at columns sa, sb of tensor memory.
template <int KIND>
__device__ __forceinline__ void mx_stage_mmas(uint32_t d, uint32_t a, uint32_t b, uint32_t sa, uint32_t sb, int sb_cols,
                                              int n_tiles, uint32_t idesc, bool first) {
    const uint64_t da = desc_sw128(a), db = desc_sw128(b);
    if (KIND == MX_A8) {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            mx_mma<KIND>(d, da + 2 * k, db + 2 * k, idesc | mx_sf_ids(k), sa, sb, first && k == 0 ? 0u : 1u);
    } else {
#pragma unroll
        for (int k = 0; k < 4; ++k)
            if (k < 2 * n_tiles)
                mx_mma<KIND>(d, da + 2 * k, db + 2 * k, idesc | mx_sf_ids(2 * (k & 1)), sa + 4 * (k >> 1),
                             sb + sb_cols * (k >> 1), first && k == 0 ? 0u : 1u);
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
                    mx_scales_to_tmem(ta + 4 * t, sfs + t * MX_TILE_BYTES);
                    mx_scales_to_tmem(tb + 4 * t, sfs + (TPS + t) * MX_TILE_BYTES);
                }
                mx_stage_mmas<KIND>(tmem, slot, slot + 16384u, ta, tb, 4, tiles, idesc, i == 0);
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

template <int KIND>
int launch_linear(MxLinArgs &a, const lora_mx *x, const lora_mx *w, int sms, cudaStream_t st) {
    const uint64_t xb = (uint64_t)mx_row_bytes(x->format, x->cols), wb = (uint64_t)mx_row_bytes(w->format, w->cols);
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
