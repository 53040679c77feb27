// The dense products on the ordinary arithmetic units (contract: lora_linear and lora_expert_linear in
// lora_delta.h): fp32 data, whose products stay in fp32 (no tf32), and bf16 data
// that TMA cannot take (rows off 16-byte steps).
//
//   few rows    a warp takes four features (gated: two of each half) x eight rows, its lanes split k: W is read once for
//               eight rows, bound by HBM
//   many rows   a block of 256 threads takes a tile of rows x features, 8 x 8 or 4 x 4 sums a thread, both
//               operands through shared memory, the next k step's loads in flight meanwhile
#include "linear.cuh"

#include <algorithm>

namespace lora {

namespace {

// y of one element from its sums, fp32 until the one rounding
template <typename E, bool GATED>
__device__ __forceinline__ void finish(const LinArgs &a, int64_t row, int e, int c, float z, float up) {
    const E *bias = static_cast<const E *>(a.bias), *add = static_cast<const E *>(a.addend), *res = static_cast<const E *>(a.residual);
    if (bias) {
        z += load_elem(bias + (int64_t)e * a.n_w + c);
        if (GATED) up += load_elem(bias + (int64_t)e * a.n_w + a.d_out + c);
    }
    if (add) {
        z += load_elem(add + row * a.ld_a + c);
        if (GATED) up += load_elem(add + row * a.ld_a + a.d_out + c);
    }
    activate<sizeof(E) == 2, 1>(a.act, &z);
    if (GATED) z *= up;
    if (res) z += load_elem(res + row * a.ld_r + c);
    store_elem(static_cast<E *>(a.y) + row * a.ld_y + c, z);
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
    count_tiles(a.seg_start, a.N, rows, pre, part);
    if (tile >= pre[a.N]) return false;
    const int e = expert_of(pre, a.N, tile);
    out->e = e;
    out->q0 = a.seg_start[e] + (tile - pre[e]) * rows;
    out->cnt = min(rows, a.seg_start[e + 1] - out->q0);
    return true;
}

// four elements at p, of which `n` exist (vec: all or none of a group do, 16 or 8-byte aligned)
__device__ __forceinline__ void load4(const float *p, int n, bool vec, float *v) {
    if (vec) {
        const float4 f = n > 0 ? *reinterpret_cast<const float4 *>(p) : make_float4(0, 0, 0, 0);
        v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? p[i] : 0.f;
    }
}
__device__ __forceinline__ void load4(const __nv_bfloat16 *p, int n, bool vec, float *v) {
    if (vec) {
        const uint2 u = n > 0 ? *reinterpret_cast<const uint2 *>(p) : make_uint2(0, 0);
        v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] = i < n ? __bfloat162float(p[i]) : 0.f;
    }
}

// ---------------------------------------------------------------- few rows
constexpr int DOT_ROWS = 8, DOT_FEATURES = 4, DOT_WARPS = 8;

template <typename E, bool GATED>
__global__ void __launch_bounds__(32 * DOT_WARPS) linear_dot_kernel(const LinArgs a, int vec) {
    __shared__ int pre[MAX_EXPERTS + 1], part[32];
    pdl_next();
    pdl_wait();
    Rows r;
    if (!block_rows(a, (int)blockIdx.x, DOT_ROWS, pre, part, &r)) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    constexpr int COLS = GATED ? DOT_FEATURES / 2 : DOT_FEATURES;   // of y, a warp
    const int c0 = ((int)blockIdx.y * DOT_WARPS + warp) * COLS;
    if (c0 >= a.d_out) return;
    const E *w = static_cast<const E *>(a.w) + (int64_t)r.e * a.n_w * a.ld_w;
    const E *wp[DOT_FEATURES], *xp[DOT_ROWS];
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
        xp[i] = static_cast<const E *>(a.x) + (int64_t)(a.perm ? slot[i] / a.x_div : q) * a.ld_x;
    }
    float acc[DOT_ROWS][DOT_FEATURES] = {};
#pragma unroll 2
    for (int k = 4 * lane; k < a.d_in; k += 128) {
        const int n = a.d_in - k;
        float wv[DOT_FEATURES][4], xv[4];
#pragma unroll
        for (int f = 0; f < DOT_FEATURES; ++f) load4(wp[f] + k, n, vec, wv[f]);
#pragma unroll
        for (int i = 0; i < DOT_ROWS; ++i) {
            if (i >= r.cnt) break;
            load4(xp[i] + k, n, vec, xv);
#pragma unroll
            for (int f = 0; f < DOT_FEATURES; ++f)
#pragma unroll
                for (int j = 0; j < 4; ++j) acc[i][f] = fmaf(wv[f][j], xv[j], acc[i][f]);
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
                finish<E, GATED>(a, slot[i], r.e, c0 + f, acc[i][f], GATED ? acc[i][COLS + f] : 0.f);
}

// --------------------------------------------------------------- many rows
// BM rows x BN features of W (gated: BN / 2 of each half), TM x TN sums a thread; K steps of 16.
// Threads lie BN / TN along the features.  A thread's features are TN / 2 apart in halves of the tile: its first
// half and the same of the second, so a gated tile's gate and up sums of a column meet in one thread.
constexpr int TILE_K = 16;

template <typename E, bool GATED, int BM, int BN, int TM, int TN>
__global__ void __launch_bounds__(256) linear_tile_kernel(const LinArgs a, int vec) {
    static_assert((BM / TM) * (BN / TN) == 256 && TN % 4 == 0 && TM % 4 == 0, "256 threads");
    __shared__ int pre[MAX_EXPERTS + 1], part[32];
    __shared__ __align__(16) float xs[2][TILE_K][BM + 4], ws[2][TILE_K][BN + 4];
    pdl_next();
    pdl_wait();
    Rows r;
    if (!block_rows(a, (int)blockIdx.x, BM, pre, part, &r)) return;
    constexpr int H = BN / 2, TH = TN / 2;
    constexpr int COLS = GATED ? H : BN;                    // columns of y of this block
    const int c0 = (int)blockIdx.y * COLS, tid = threadIdx.x;
    const int tx = tid % (BN / TN), ty = tid / (BN / TN);
    // tile feature f is W's row w_row(f); those past the last read the last one
    auto w_row = [&](int f) {
        return GATED ? min(c0 + f % H, a.d_out - 1) + f / H * a.d_out : min(c0 + f, a.d_out - 1);
    };
    constexpr int LX = BM * TILE_K / 4 / 256 > 0 ? BM * TILE_K / 4 / 256 : 1, LW = BN * TILE_K / 4 / 256;
    static_assert(BM * TILE_K / 4 % 256 == 0 && LW * 256 * 4 == BN * TILE_K, "whole loads");
    const E *xp[LX], *wp[LW];
    const int kq = tid % 4 * 4;   // this thread's four columns of a k step
#pragma unroll
    for (int i = 0; i < LX; ++i) {
        const int q = r.q0 + min(tid / 4 + 64 * i, r.cnt - 1);
        xp[i] = static_cast<const E *>(a.x) + (int64_t)(a.perm ? a.perm[q] / a.x_div : q) * a.ld_x + kq;
    }
#pragma unroll
    for (int i = 0; i < LW; ++i)
        wp[i] = static_cast<const E *>(a.w) + ((int64_t)r.e * a.n_w + w_row(tid / 4 + 64 * i)) * a.ld_w + kq;
    float xv[LX][4], wv[LW][4], acc[TM][TN] = {};
    auto fetch = [&](int k) {
#pragma unroll
        for (int i = 0; i < LX; ++i) load4(xp[i] + k, a.d_in - k - kq, vec, xv[i]);
#pragma unroll
        for (int i = 0; i < LW; ++i) load4(wp[i] + k, a.d_in - k - kq, vec, wv[i]);
    };
    auto put = [&](int b) {
#pragma unroll
        for (int i = 0; i < LX; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) xs[b][kq + j][tid / 4 + 64 * i] = xv[i][j];
#pragma unroll
        for (int i = 0; i < LW; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) ws[b][kq + j][tid / 4 + 64 * i] = wv[i][j];
    };
    fetch(0);
    put(0);
    __syncthreads();
    int b = 0;
    for (int k = 0; k < a.d_in; k += TILE_K, b ^= 1) {
        const bool more = k + TILE_K < a.d_in;
        if (more) fetch(k + TILE_K);
#pragma unroll
        for (int kk = 0; kk < TILE_K; ++kk) {
            float xf[TM], wf[TN];
#pragma unroll
            for (int i = 0; i < TM; i += 4)   // rows in groups of four, BM / (TM / 4) apart
                *reinterpret_cast<float4 *>(xf + i) = *reinterpret_cast<const float4 *>(&xs[b][kk][ty * 4 + i / 4 * (BM / (TM / 4))]);
            if (TH % 4 == 0) {
#pragma unroll
                for (int j = 0; j < TN; j += 4)
                    *reinterpret_cast<float4 *>(wf + j) =
                        *reinterpret_cast<const float4 *>(&ws[b][kk][j / TH * H + tx * TH + j % TH]);
            } else {
#pragma unroll
                for (int j = 0; j < TN; j += 2)
                    *reinterpret_cast<float2 *>(wf + j) =
                        *reinterpret_cast<const float2 *>(&ws[b][kk][j / TH * H + tx * TH + j % TH]);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TN; ++j) acc[i][j] = fmaf(xf[i], wf[j], acc[i][j]);
        }
        if (more) put(b ^ 1);
        __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int at = ty * 4 + i / 4 * (BM / (TM / 4)) + i % 4;
        if (at >= r.cnt) continue;
        const int64_t row = a.perm ? a.perm[r.q0 + at] : r.q0 + at;
#pragma unroll
        for (int j = 0; j < (GATED ? TH : TN); ++j) {
            const int c = c0 + j / TH * H + tx * TH + j % TH;
            if (c < a.d_out) finish<E, GATED>(a, row, r.e, c, acc[i][j], GATED ? acc[i][TH + j] : 0.f);
        }
    }
}

template <typename E, bool GATED>
int launch_as(const LinArgs &a, int sms, cudaStream_t st) {
    const int vec = (a.d_in & 3) == 0 && (a.ld_x & 3) == 0 && (a.ld_w & 3) == 0 && mx_aligned(a.x, 4 * sizeof(E)) &&
                    mx_aligned(a.w, 4 * sizeof(E));
    // row tiles that a grouping may have: whole ones, and a last one for each expert that has rows
    auto row_tiles = [&](int rows) { return a.perm ? a.T / rows + std::min(a.N, a.T) : (a.T + rows - 1) / rows; };
    const int per_group = a.perm ? (a.T + a.N - 1) / a.N : a.T;
    const int halves = GATED ? 2 : 1;
    if (per_group <= 2 * DOT_ROWS) {
        const int cols = DOT_WARPS * DOT_FEATURES / halves;
        return launch_after(linear_dot_kernel<E, GATED>, dim3(row_tiles(DOT_ROWS), (a.d_out + cols - 1) / cols), 32 * DOT_WARPS, 0, 0,
                            st, a, vec);
    }
    const int64_t big = (int64_t)row_tiles(128) * ((a.n_w + 127) / 128);
    if (per_group > 64 && big >= sms)
        return launch_after(linear_tile_kernel<E, GATED, 128, 128, 8, 8>,
                            dim3(row_tiles(128), (a.d_out + 128 / halves - 1) / (128 / halves)), 256, 0, 0, st, a, vec);
    return launch_after(linear_tile_kernel<E, GATED, 64, 64, 4, 4>, dim3(row_tiles(64), (a.d_out + 64 / halves - 1) / (64 / halves)),
                        256, 0, 0, st, a, vec);
}

}  // namespace

int launch_linear_simt(const LinArgs &a, bool bf16, bool gated, int sms, cudaStream_t st) {
    if (bf16) return gated ? launch_as<__nv_bfloat16, true>(a, sms, st) : launch_as<__nv_bfloat16, false>(a, sms, st);
    return gated ? launch_as<float, true>(a, sms, st) : launch_as<float, false>(a, sms, st);
}

}  // namespace lora
