// The dense products of fp32 data (contract: lora_linear and lora_expert_linear in lora_delta.h), on the ordinary
// arithmetic units: fp32 products, no tf32; any stride and alignment.
//
//   few rows    a warp takes two features (gated: one of each half) x eight rows, its lanes split k: W is read once for
//               eight rows, bound by HBM (1 x 14336 x 4096 38.3 us = 6.1 TB/s; 1 x 4096 x 4096 14.2)
//   many rows   a block takes a tile of rows x features, 8 x 4 or 4 x 4 sums a thread, both operands through shared memory;
//               bound by the arithmetic units, at 60 % of their 128 multiply-adds a clock and SM (4096^3 3.2 ms = 43 TFLOP/s,
//               where torch's matrix product takes 2.4), few tiles by latency (333 x 1003 x 777 35 us, with rows in
//               16-byte steps 29)
#include "linear.cuh"
#include "ptx.cuh"

#include <algorithm>

namespace lora {

namespace {

// y of one element from its sums
template <bool GATED>
__device__ __forceinline__ void finish(const LinArgs &a, int64_t row, int e, int c, float z, float up) {
    const float *bias = static_cast<const float *>(a.bias), *add = static_cast<const float *>(a.addend);
    if (bias) {
        z += bias[(int64_t)e * a.n_w + c];
        if (GATED) up += bias[(int64_t)e * a.n_w + a.d_out + c];
    }
    if (add) {
        z += add[row * a.ld_a + c];
        if (GATED) up += add[row * a.ld_a + a.d_out + c];
    }
    activate<false, 1>(a.act, &z);
    if (GATED) z *= up;
    if (a.residual) z += static_cast<const float *>(a.residual)[row * a.ld_r + c];
    static_cast<float *>(a.y)[row * a.ld_y + c] = z;
}

// Rows of a block: positions q0 .. q0 + cnt - 1 of expert e.  false: the block has none.
struct Rows {
    int e, q0, cnt;
};
__device__ __forceinline__ bool block_rows(const LinArgs &a, int tile, int rows, int *pre, int *part, Rows *out) {
    if (!a.perm) {
        out->e = 0, out->q0 = tile * rows, out->cnt = min(rows, a.T - out->q0);
        return true;
    }
    count_tiles(a.seg_start, a.N, rows, pre, nullptr, part);
    if (tile >= pre[a.N]) return false;
    const int e = expert_of(pre, a.N, tile);
    out->e = e;
    out->q0 = a.seg_start[e] + (tile - pre[e]) * rows;
    out->cnt = min(rows, a.seg_start[e + 1] - out->q0);
    return true;
}

// four elements at p, of which `n` exist (vec: all or none of them do, 16-byte aligned)
__device__ __forceinline__ void load4(const float *p, int n, bool vec, float *v) {
    if (vec) {
        const float4 f = n > 0 ? *reinterpret_cast<const float4 *>(p) : make_float4(0, 0, 0, 0);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : 0.f;
    }
}

// ---------------------------------------------------------------- few rows
constexpr int DOT_ROWS = 8, DOT_FEATURES = 2, DOT_WARPS = 8;

template <bool GATED>
__global__ void __launch_bounds__(32 * DOT_WARPS) linear_dot_kernel(const LinArgs a, int vec, int row_tiles) {
    __shared__ int pre[LORA_MAX_EXPERTS + 1], part[32];
    pdl_next();
    pdl_wait();
    Rows r;
    const int block = (int)blockIdx.x / row_tiles;   // row tiles of the same features beside each other
    if (!block_rows(a, (int)blockIdx.x - block * row_tiles, DOT_ROWS, pre, part, &r)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int COLS = GATED ? DOT_FEATURES / 2 : DOT_FEATURES;   // of y, a warp
    const int c0 = (block * DOT_WARPS + warp) * COLS;
    if (c0 >= a.d_out) return;
    const float *w = static_cast<const float *>(a.w) + (int64_t)r.e * a.n_w * a.ld_w;
    const float *wp[DOT_FEATURES], *xp[DOT_ROWS];
    int slot[DOT_ROWS];
#pragma unroll
    for (int f = 0; f < DOT_FEATURES; ++f) {   // features past the last read the last one's row
        const int c = min(c0 + f % COLS, a.d_out - 1) + f / COLS * a.d_out;
        wp[f] = w + (int64_t)c * a.ld_w;
    }
#pragma unroll
    for (int i = 0; i < DOT_ROWS; ++i) {   // rows past the last read the last one
        const int q = r.q0 + min(i, r.cnt - 1);
        slot[i] = a.perm ? a.perm[q] : q;
        xp[i] = static_cast<const float *>(a.x) + (int64_t)(a.perm ? slot[i] / a.x_div : q) * a.ld_x;
    }
    float acc[DOT_ROWS][DOT_FEATURES] = {};
    constexpr int STEPS = 4;   // of 128 columns, whose W is under way at once
    for (int k0 = 4 * lane; k0 < a.d_in; k0 += 128 * STEPS) {
        float wv[STEPS][DOT_FEATURES][4];
#pragma unroll
        for (int s = 0; s < STEPS; ++s)
#pragma unroll
            for (int f = 0; f < DOT_FEATURES; ++f) load4(wp[f] + (k0 + 128 * s), a.d_in - k0 - 128 * s, vec, wv[s][f]);
#pragma unroll
        for (int i = 0; i < DOT_ROWS; ++i) {
            if (i >= r.cnt) break;
#pragma unroll
            for (int s = 0; s < STEPS; ++s) {
                float xv[4];
                load4(xp[i] + (k0 + 128 * s), a.d_in - k0 - 128 * s, vec, xv);
#pragma unroll
                for (int f = 0; f < DOT_FEATURES; ++f)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][f] = fmaf(wv[s][f][j], xv[j], acc[i][f]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < DOT_ROWS; ++i) {
        if (i >= r.cnt) break;
#pragma unroll
        for (int f = 0; f < DOT_FEATURES; ++f)
#pragma unroll
            for (int d = 16; d; d /= 2) acc[i][f] += __shfl_xor_sync(FULL, acc[i][f], d);
    }
    // lane 4 i + f finishes column f of row i
#pragma unroll
    for (int i = 0; i < DOT_ROWS; ++i)
#pragma unroll
        for (int f = 0; f < COLS; ++f)
            if (lane == 4 * i + f && i < r.cnt && c0 + f < a.d_out)
                finish<GATED>(a, slot[i], r.e, c0 + f, acc[i][f], GATED ? acc[i][COLS + f] : 0.f);
}

// --------------------------------------------------------------- many rows
// BM rows x BN features of W (gated: BN / 2 of each half), TM x TN sums a thread, KG groups of threads that take a part of each
// k tile each (where tiles are few: more warps on an SM) and add their sums at the end, in order; k in tiles of TILE_K that cp.async brings into
// a ring of STAGES: 16 bytes a copy, or 4 where rows are off 16-byte steps.  Rows lie TILE_K + 4 floats apart: a thread reads four
// k of a row at once, eight neighbours eight rows of W in eight different bank groups.  A thread's features are BN / TN
// apart, so a gated tile's gate and up sums of a column meet in one thread, and neighbours store neighbouring columns.
// two fused multiply-adds in one instruction, each rounded as its own
__device__ __forceinline__ void fma2(uint64_t &acc, uint64_t x, uint64_t w) {
    asm("fma.rn.f32x2 %0, %1, %2, %0;\n" : "+l"(acc) : "l"(x), "l"(w));
}
__device__ __forceinline__ float sum2(uint64_t v) {
    return __uint_as_float((uint32_t)v) + __uint_as_float((uint32_t)(v >> 32));
}

template <bool GATED, int BM, int BN, int TM, int TN, int KG, int TILE_K, int STAGES, int BLOCKS>
__global__ void __launch_bounds__(KG * (BM / TM) * (BN / TN), BLOCKS) linear_tile_kernel(const LinArgs a, int vec) {
    constexpr int GROUP = (BM / TM) * (BN / TN), THREADS = KG * GROUP, ROWS = BM + BN, TX = BN / TN, H = BN / 2, TILE_LD = TILE_K + 4;
    static_assert(TN % 2 == 0 && TX % 8 == 0 && GROUP % 32 == 0 && BM / TM % 4 == 0, "gate and up in one thread, whole warps");
    extern __shared__ __align__(16) float lin_tiles[];   // [STAGES][ROWS][TILE_LD]
    __shared__ int pre[LORA_MAX_EXPERTS + 1], part[32];
    __shared__ const float *src[ROWS];   // rows of x, then of W
    pdl_next();
    pdl_wait();
    Rows r;
    if (!block_rows(a, (int)blockIdx.x, BM, pre, part, &r)) return;
    constexpr int COLS = GATED ? H : BN;                    // columns of y of this block
    const int c0 = (int)blockIdx.y * COLS, tid = threadIdx.x;
    // a warp is 8 threads along the features x 4 along the rows: 8 + 4 rows of 16 bytes a step where 16 + 2 would be more
    const int group = tid / GROUP, g_warp = tid % GROUP / 32, tx = tid % 8 + g_warp % (TX / 8) * 8, ty = tid % 32 / 8 + g_warp / (TX / 8) * 4;
    for (int i = tid; i < ROWS; i += THREADS) {   // rows past the last read the last one
        if (i < BM) {
            const int q = r.q0 + min(i, r.cnt - 1);
            src[i] = static_cast<const float *>(a.x) + (int64_t)(a.perm ? a.perm[q] / a.x_div : q) * a.ld_x;
        } else {
            const int f = i - BM, c = GATED ? min(c0 + f % H, a.d_out - 1) + f / H * a.d_out : min(c0 + f, a.d_out - 1);
            src[i] = static_cast<const float *>(a.w) + ((int64_t)r.e * a.n_w + c) * a.ld_w;
        }
    }
    __syncthreads();
    const int n_k = (a.d_in + TILE_K - 1) / TILE_K;
    auto fetch = [&](int k) {
        if (k < n_k) {
            const uint32_t to = smem_u32(lin_tiles + (k % STAGES) * ROWS * TILE_LD);
            if (vec) {
#pragma unroll 4
                for (int i = tid; i < ROWS * (TILE_K / 4); i += THREADS) {
                    const int row = i / (TILE_K / 4), c = i % (TILE_K / 4) * 4, col = k * TILE_K + c;
                    const bool in = col < a.d_in;   // d_in is a multiple of 4
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;\n" ::"r"(to + (uint32_t)(row * TILE_LD + c) * 4u),
                                 "l"(src[row] + (in ? col : 0)), "r"(in ? 16 : 0)
                                 : "memory");
                }
            } else {
#pragma unroll 4
                for (int i = tid; i < ROWS * TILE_K; i += THREADS) {
                    const int row = i / TILE_K, c = i % TILE_K, col = k * TILE_K + c;
                    const bool in = col < a.d_in;
                    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;\n" ::"r"(to + (uint32_t)(row * TILE_LD + c) * 4u),
                                 "l"(src[row] + (in ? col : 0)), "r"(in ? 4 : 0)
                                 : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;\n" ::: "memory");
    };
    uint64_t acc[TM][TN] = {};   // pairs of sums, of the even and the odd k
#pragma unroll
    for (int k = 0; k < STAGES - 1; ++k) fetch(k);
    for (int k = 0; k < n_k; ++k) {
        asm volatile("cp.async.wait_group %0;\n" ::"n"(STAGES - 2) : "memory");
        __syncthreads();   // tile k is there for all, and all are done with tile k - 1, whose place the next one takes
        fetch(k + STAGES - 1);
        const float *xs = lin_tiles + (k % STAGES) * ROWS * TILE_LD + group * (TILE_K / KG), *ws = xs + BM * TILE_LD;
#pragma unroll 4
        for (int kk = 0; kk < TILE_K / KG; kk += 4) {
            ulonglong2 xf[TM], wf[TN];
#pragma unroll
            for (int i = 0; i < TM; ++i) xf[i] = *reinterpret_cast<const ulonglong2 *>(xs + (ty + i * (BM / TM)) * TILE_LD + kk);
#pragma unroll
            for (int j = 0; j < TN; ++j) wf[j] = *reinterpret_cast<const ulonglong2 *>(ws + (tx + j * TX) * TILE_LD + kk);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) fma2(acc[i][j], xf[i].x, wf[j].x);
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) fma2(acc[i][j], xf[i].y, wf[j].y);
        }
    }
    float sum[TM][TN];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) sum[i][j] = sum2(acc[i][j]);
    if (KG > 1) {
        static_assert((KG - 1) * GROUP * TM * TN <= STAGES * ROWS * TILE_LD, "the groups' sums fit the ring");
        asm volatile("cp.async.wait_all;\n" ::: "memory");
        __syncthreads();   // all are done with the ring
        if (group > 0)
#pragma unroll
            for (int i = 0; i < TM * TN; ++i) lin_tiles[((group - 1) * TM * TN + i) * GROUP + tid % GROUP] = sum[i / TN][i % TN];
        __syncthreads();
        if (group > 0) return;
        for (int g = 0; g < KG - 1; ++g)
#pragma unroll
            for (int i = 0; i < TM * TN; ++i) sum[i / TN][i % TN] += lin_tiles[(g * TM * TN + i) * GROUP + tid];
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int at = ty + i * (BM / TM);
        if (at >= r.cnt) continue;
        const int64_t row = a.perm ? a.perm[r.q0 + at] : r.q0 + at;
#pragma unroll
        for (int j = 0; j < (GATED ? TN / 2 : TN); ++j) {
            const int c = c0 + tx + j * TX;
            if (c < a.d_out) finish<GATED>(a, row, r.e, c, sum[i][j], GATED ? sum[i][TN / 2 + j] : 0.f);
        }
    }
}

template <bool GATED, int BM, int BN, int TM, int TN, int KG, int TILE_K, int STAGES, int BLOCKS>
int launch_tile(const LinArgs &a, int vec, int row_tiles, cudaStream_t st) {
    constexpr int COLS = GATED ? BN / 2 : BN;
    constexpr size_t SMEM = (size_t)STAGES * (BM + BN) * (TILE_K + 4) * sizeof(float);
    auto kernel = linear_tile_kernel<GATED, BM, BN, TM, TN, KG, TILE_K, STAGES, BLOCKS>;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)SMEM);
    if (e != cudaSuccess) return cuda_rc(e);
    return launch_after(kernel, dim3(row_tiles, (a.d_out + COLS - 1) / COLS), KG * (BM / TM) * (BN / TN), SMEM, 0, st, a, vec);
}

template <bool GATED>
int launch_as(const LinArgs &a, int sms, cudaStream_t st) {
    const int vec = (a.d_in & 3) == 0 && (a.ld_x & 3) == 0 && (a.ld_w & 3) == 0 && mx_aligned(a.x, 16) && mx_aligned(a.w, 16);
    // row tiles that a grouping may have: whole ones, and a last one for each expert that has rows
    auto row_tiles = [&](int rows) { return a.perm ? a.T / rows + std::min(a.N, a.T) : (a.T + rows - 1) / rows; };
    const int per_group = a.perm ? (a.T + a.N - 1) / a.N : a.T;
    // Few rows a group, by the mean, which is what the host knows (us, few-row kernel / 32 x 64 tiles): 8 x 4096 x 4096 50 / 90, 16 76 / 87,
    // 32 127 / 87; over wide outputs the tiles win earlier, 12 x 4096 x 14336 160 / 176, 16 211 / 173.  The mean counts experts
    // without rows: of 1024 experts (512 -> 256) 8192 slots spread evenly take 777 / 432, with 90 % of them in four 697 / 350.
    if (per_group <= 2 * DOT_ROWS) {
        const int cols = DOT_WARPS * DOT_FEATURES / (GATED ? 2 : 1);
        const int tiles = row_tiles(DOT_ROWS);   // a few thousand of them at most, and 65536 blocks of features
        return launch_after(linear_dot_kernel<GATED>, dim3(tiles * ((a.d_out + cols - 1) / cols)), 32 * DOT_WARPS, 0, 0, st, a, vec, tiles);
    }
    // the largest tile that gives every SM one (us on 32 x 64 / 64 x 64 / 128 x 64: 64 x 4096 x 4096 87 / 149 / 278, 64 x 4096 x 9472
    // 172 / 149 / 321, 64 x 4096 x 14336 341 / 264 / 533, 128 x 4096 x 4096 172 / 227 / 273, 256 x 4096 x 4096 341 / 263 / 420,
    // 512 x 4096 x 4096 597 / 508 / 490, 1024 x 2048 x 2048 317 / 263 / 251, 333 x 1003 x 777 35 / 70 / 94).
    // Two blocks of 256 threads share an SM, for the four registers that this spills: with one, 64 x 4096 x 14336, a
    // wave and a half of tiles, takes 295 us, and 512 x 4096 x 4096 508 instead of 487.
    auto tiles = [&](int bm, int bn) { return (int64_t)row_tiles(bm) * ((a.n_w + bn - 1) / bn); };
    if (per_group > 64 && tiles(128, 64) >= sms) return launch_tile<GATED, 128, 64, 8, 4, 1, 32, 3, 2>(a, vec, row_tiles(128), st);
    if (per_group > 32 && tiles(64, 64) >= sms) return launch_tile<GATED, 64, 64, 8, 4, 2, 32, 3, 2>(a, vec, row_tiles(64), st);
    return launch_tile<GATED, 32, 64, 4, 4, 4, 64, 3, 1>(a, vec, row_tiles(32), st);
}

}  // namespace

int launch_linear_simt(const LinArgs &a, bool gated, int sms, cudaStream_t st) {
    return gated ? launch_as<true>(a, sms, st) : launch_as<false>(a, sms, st);
}

}  // namespace lora
