// Row operators around a microscaled base: quantise, read back, and the
// root-mean-square norm with the residual's sum whose rows leave in the data's
// type and, optionally, microscaled.  Contracts: lora_delta.h.
//
// All three stream rows once and are bound by HBM: norm 8192 x 8192 bf16 with residual and MXFP8 copy 95 us (6.4 TB/s),
// quantize 28672 x 8192 to MXFP4 91 us (6.5), dequantize 92 us (6.4); one row of 4096 2.2 us.  A lane holds 8 consecutive
// columns (one 16-byte bf16 access), so 4 lanes hold a scale's block of 32 and a
// warp 256 columns = two scale tiles; the block's largest magnitude takes two
// shuffles, the tile's four scale bytes two more.
#include "mx.cuh"

#include <algorithm>

namespace lora {

namespace {

constexpr int ROWS_THREADS = 256;

// The rows a warp takes at once: r, r + 32, r + 64, r + 96 of a 128-row band (J = 4), whose
// scale words are neighbours (16 bytes of a tile), or one row (J = 1: small matrices, more warps).
// Grid: groups of 256 columns (a warp each), rows within 32 (or 128), bands.
struct RowItem {
    int64_t row;   // the first row
    int c0;        // the first column
};
__device__ __forceinline__ RowItem row_item() {
    return RowItem{(int64_t)blockIdx.z * MX_TILE_ROWS + blockIdx.y,
                   (int)(blockIdx.x * (ROWS_THREADS / 32) + (threadIdx.x >> 5)) * 256};
}

template <typename E, bool FP4, bool VEC, int J>
__global__ void __launch_bounds__(ROWS_THREADS)
    mx_quantize_kernel(unsigned char *q, uint8_t *scales, const E *x, int64_t ld_x, int T, int cols) {
    using Raw = typename RawOf<E>::type;
    const int lane = threadIdx.x & 31, pad = (int)mx_padded(cols);
    const int64_t row_bytes = FP4 ? pad / 2 : pad;
    const RowItem it = row_item();
    pdl_next();
    pdl_wait();
    if (it.c0 >= pad) return;
    Raw u[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t row = it.row + 32 * j;
        const E *p = x + (row < T ? row : 0) * ld_x;
        const int n = row < T ? cols : 0;
        if (VEC) {
            load8<true>(p, it.c0, n, lane, u[j]);
        } else {   // 8 neighbours one by one: the lines they share come from L1
            float v[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = it.c0 + 8 * lane + i < n ? load_elem(p + it.c0 + 8 * lane + i) : 0.f;
            raw_round(v, u[j]);
        }
    }
    if constexpr (J == 1) {
        float v[8];
        raw_values(u[0], v);
        mx_emit<FP4>(q + it.row * row_bytes, scales, it.row, it.c0, pad, lane, it.row < T, v, mx_top(u[0]));
    } else {
        // Four rows: lane s of a block's four finds row s's largest magnitude, its code and factor, and stores its scale (a byte;
        // the rows' 4 words lie side by side).  Each row's own way through mx_emit: 28672 x 8192 bf16 to MXFP4 106 us, 91 so.
        uint32_t m[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) m[j] = mx_top(u[j]);
        const int s = lane & 3, col = it.c0 + 8 * lane;
        const bool odd = s & 1, high = s & 2;
        const uint32_t m0 = max(high ? m[2] : m[0], __shfl_xor_sync(FULL, high ? m[0] : m[2], 2));
        const uint32_t m1 = max(high ? m[3] : m[1], __shfl_xor_sync(FULL, high ? m[1] : m[3], 2));
        const uint32_t code = mx_code<FP4>(max(odd ? m1 : m0, __shfl_xor_sync(FULL, odd ? m0 : m1, 1)));
        const float inverse = mx_inverse(code);
        if (it.row + 32 * s < T && col < pad)
            scales[mx_scale_word(it.row, col >> 7, pad / MX_TILE_COLS) + 4 * s + ((col >> 5) & 3)] = (uint8_t)code;
        const bool nans = __any_sync(FULL, code == 255u);
#pragma unroll
        for (int j = 0; j < J; ++j) {
            const int64_t row = it.row + 32 * j;
            const float inv = __shfl_sync(FULL, inverse, j, 4);
            float v[8];
            raw_values(u[j], v);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= inv;
            if (nans && inv == 0.f)   // elements of a NaN block: zeros
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = 0.f;
            if (row < T && col < pad) {
                if (FP4) *reinterpret_cast<uint32_t *>(q + row * row_bytes + (col >> 1)) = mx_pack_e2m1(v);
                else *reinterpret_cast<uint2 *>(q + row * row_bytes + col) = mx_pack_e4m3(v);
            }
        }
    }
}

template <typename E, bool FP4, bool VEC, int J>
__global__ void __launch_bounds__(ROWS_THREADS)
    mx_dequantize_kernel(E *out, int64_t ld_out, const unsigned char *q, const uint8_t *scales, int T, int cols) {
    __shared__ __align__(16) float turn[VEC ? 1 : ROWS_THREADS * 8];
    const int lane = threadIdx.x & 31, pad = (int)mx_padded(cols);
    const int64_t row_bytes = FP4 ? pad / 2 : pad;
    const RowItem it = row_item();
    const int col = it.c0 + 8 * lane;
    pdl_next();
    pdl_wait();
    uint2 e[J];
    uint32_t code[J];
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t row = it.row + 32 * j;
        e[j] = make_uint2(0, 0), code[j] = 0;
        if (row < T && col < cols) {
            const unsigned char *p = q + row * row_bytes;
            if (FP4) e[j].x = *reinterpret_cast<const uint32_t *>(p + (col >> 1));
            else e[j] = *reinterpret_cast<const uint2 *>(p + col);
            code[j] = scales[mx_scale_word(row, col >> 7, pad / MX_TILE_COLS) + ((col >> 5) & 3)];
        }
    }
#pragma unroll
    for (int j = 0; j < J; ++j) {
        const int64_t row = it.row + 32 * j;
        if (row >= T) break;
        float v[8];
        if (FP4) mx_unpack_e2m1(e[j].x, v);
        else mx_unpack_e4m3(e[j], v);
        const float s = mx_scale(code[j]);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= s;
        if (!VEC) rows_to_lanes(v, turn + (VEC ? 0 : (threadIdx.x >> 5) * 256), lane);
        typename RawOf<E>::type u;
        raw_round(v, u);
        store8<VEC>(out + row * ld_out, it.c0, cols, lane, u);
    }
}

struct NormArgs {
    void *h;
    int64_t ld_h;
    const void *x;
    int64_t ld_x;
    const void *residual;
    int64_t ld_r;
    void *sum;
    int64_t ld_s;
    const void *weight;
    float eps;
    int T, d;
    unsigned char *q;
    uint8_t *scales;
};

enum { NORM_NO_Q = 0, NORM_FP8 = 1, NORM_FP4 = 2 };

// One row per TPR threads.  V > 0: the row stays in registers (V * 8 columns a
// thread, as the type holds them: r is rounded to it) between the sum of squares and the scaling; V = 0: longer rows, read a
// second time (from the stored sum where there is a residual).
template <typename E, int V, int Q, bool VEC, bool RES>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ NormArgs a, int tpr) {
    __shared__ float part[32];
    extern __shared__ __align__(16) float turn[];   // 256 floats a warp where !VEC && Q
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = threadIdx.x % tpr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    pdl_next();
    pdl_wait();
    if (row >= a.T) return;   // whole warps; only blocks of one warp per row hold several rows
    const E *x = static_cast<const E *>(a.x) + row * a.ld_x;
    const E *res = RES ? static_cast<const E *>(a.residual) + row * a.ld_r : nullptr;
    E *sum = RES ? static_cast<E *>(a.sum) + row * a.ld_s : nullptr;
    const int pad = (int)mx_padded(a.d), end = Q ? pad : a.d;   // columns the warps walk over
    using Raw = typename RawOf<E>::type;
    Raw keep[V > 0 ? V : 1];
    float ss = 0.f;
    auto first = [&](int c0, Raw &u, const Raw &res_u) {   // the warp's (summed) 256 columns at c0
        float v[8];
        raw_values(u, v);
        if (RES) {
            float r[8];
            raw_values(res_u, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] += r[i];
            raw_round(v, u);
            store8<VEC>(sum, c0, a.d, lane, u);
            raw_values(u, v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    };
    const int w0 = 8 * (t - lane), step = 8 * tpr;   // the warp's first columns, and from one to the next
    if (V > 0) {
        Raw r[RES && V > 0 ? V : 1];
#pragma unroll
        for (int k = 0; k < V; ++k) {   // every load first
            load8<VEC>(x, w0 + k * step, a.d, lane, keep[k]);
            if (RES) load8<VEC>(res, w0 + k * step, a.d, lane, r[RES ? k : 0]);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) first(w0 + k * step, keep[k], r[RES ? k : 0]);
    } else {
        for (int c0 = w0; c0 < a.d; c0 += step) {
            Raw r;
            load8<VEC>(x, c0, a.d, lane, keep[0]);
            if (RES) load8<VEC>(res, c0, a.d, lane, r);
            first(c0, keep[0], r);
        }
    }
#pragma unroll
    for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
    if (tpr > 32) {
        if (lane == 0) part[warp] = ss;
        __syncthreads();
        ss = lane < tpr / 32 ? part[lane] : 0.f;
#pragma unroll
        for (int o = 16; o; o >>= 1) ss += __shfl_xor_sync(FULL, ss, o);
    }
    const float rstd = 1.f / sqrtf(ss / (float)a.d + a.eps);
    E *h = a.h ? static_cast<E *>(a.h) + row * a.ld_h : nullptr;
    const E *w = static_cast<const E *>(a.weight);
    auto second = [&](int c0, Raw &u) {
        Raw g;
        load8<VEC>(w, c0, a.d, lane, g);
        float v[8], gv[8];
        raw_values(u, v);
        raw_values(g, gv);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = v[i] * rstd * gv[i];
        raw_round(v, u);
        if (h) store8<VEC>(h, c0, a.d, lane, u);
        if (Q) {   // of the rounded row: the base product sees what the adapters see
            raw_values(u, v);
            if (!VEC) lanes_to_rows(v, turn + warp * 256, lane);
            if (c0 + 256 > a.d)   // columns past the row's end are zeros, which 0 * rstd need not be
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c0 + 8 * lane + i >= a.d) v[i] = 0.f;
            mx_emit<Q == NORM_FP4>(a.q + row * (Q == NORM_FP4 ? pad / 2 : pad), a.scales, row, c0, pad, lane, true, v, mx_top(v));
        }
    };
    if (V > 0) {
#pragma unroll
        for (int k = 0; k < V; ++k)
            if (w0 + k * step < end) second(w0 + k * step, keep[k]);
    } else {
        for (int c0 = w0; c0 < end; c0 += step) {
            load8<VEC>(RES ? sum : x, c0, a.d, lane, keep[0]);
            second(c0, keep[0]);
        }
    }
}

template <typename E, int V, int Q, bool VEC>
int norm_launch_res(const NormArgs &a, int tpr, unsigned blocks, int threads, cudaStream_t st) {
    const size_t smem = !VEC && Q ? (size_t)threads * 32 : 0;
    if (a.residual) return launch_after(rms_norm_kernel<E, V, Q, VEC, true>, dim3(blocks), (unsigned)threads, smem, 0, st, a, tpr);
    return launch_after(rms_norm_kernel<E, V, Q, VEC, false>, dim3(blocks), (unsigned)threads, smem, 0, st, a, tpr);
}

template <typename E, int Q, bool VEC>
int norm_launch(const NormArgs &a, int sms, cudaStream_t st) {
    const int64_t vecs = (mx_padded(a.d) + 7) / 8;   // 8-column groups of a row
    const bool many = a.T >= 4 * sms;
    // Few rows: one group a thread, the shortest way through one row.  Many rows: four a thread (loads in
    // flight), but not more than a warp's share of a short row; rows past the registers of 1024
    // threads are read twice, the second time from L2.  So are, where there are many, rows whose registers would
    // leave an SM one block of 1024 threads: bf16 2048 x 28672 67 us in blocks of 512 against 83 us, fp32 as fast
    // either way; rows off 16-byte steps from 2048 columns on (fp32 4000 x 9001 116 us in blocks of 256, 198 us).
    int v = many && VEC ? 4 : 1;
    while (v > 1 && 32 * (v / 2) >= vecs) v /= 2;
    while (v < 4 && vecs > (int64_t)v * 1024) v *= 2;
    int64_t tpr = 32;
    while (tpr < 1024 && tpr * v < vecs) tpr *= 2;
    if (tpr * v < vecs || (many && VEC && sizeof(E) == 2 && vecs > 4 * 512)) v = 0, tpr = 512;
    if (many && !VEC && vecs > 256) v = 0, tpr = vecs > 2048 ? 512 : 256;
    const int threads = (int)std::max<int64_t>(tpr, tpr == 32 ? 128 : tpr);
    const int rows = threads / (int)tpr;
    const unsigned blocks = (unsigned)((a.T + rows - 1) / rows);
    switch (v) {
        case 1: return norm_launch_res<E, 1, Q, VEC>(a, (int)tpr, blocks, threads, st);
        case 2: return norm_launch_res<E, 2, Q, VEC>(a, (int)tpr, blocks, threads, st);
        case 4: return norm_launch_res<E, 4, Q, VEC>(a, (int)tpr, blocks, threads, st);
        default: return norm_launch_res<E, 0, Q, VEC>(a, (int)tpr, blocks, threads, st);
    }
}

template <typename E>
int norm_dispatch(const NormArgs &a, int q, bool vec, int sms, cudaStream_t st) {
    if (q == NORM_NO_Q) return vec ? norm_launch<E, NORM_NO_Q, true>(a, sms, st) : norm_launch<E, NORM_NO_Q, false>(a, sms, st);
    if (q == NORM_FP8) return vec ? norm_launch<E, NORM_FP8, true>(a, sms, st) : norm_launch<E, NORM_FP8, false>(a, sms, st);
    return vec ? norm_launch<E, NORM_FP4, true>(a, sms, st) : norm_launch<E, NORM_FP4, false>(a, sms, st);
}

// Rows of a warp: four where that still gives every SM 32 warps.
struct RowGrid {
    dim3 grid;
    bool four;
};
RowGrid row_grid(int64_t T, int64_t cols) {
    const int64_t groups = (mx_padded(cols) + 255) / 256, per = ROWS_THREADS / 32, bands = (T + MX_TILE_ROWS - 1) / MX_TILE_ROWS;
    RowGrid g;
    g.four = groups * T / 4 >= 148 * 32;
    g.grid = dim3((unsigned)((groups + per - 1) / per), (unsigned)std::min<int64_t>(T, g.four ? 32 : 128), (unsigned)bands);
    return g;
}

template <typename E, bool FP4, bool VEC>
int quantize_launch_vec(const lora_mx *m, const E *x, int64_t ld_x, int T, cudaStream_t st) {
    const RowGrid g = row_grid(T, m->cols);
    auto kernel = g.four ? mx_quantize_kernel<E, FP4, VEC, 4> : mx_quantize_kernel<E, FP4, VEC, 1>;
    return launch_after(kernel, g.grid, ROWS_THREADS, 0, 0, st, static_cast<unsigned char *>(m->q), m->scales, x, ld_x, T, m->cols);
}
template <typename E, bool FP4>
int quantize_launch(const lora_mx *m, const void *x, int64_t ld_x, int T, bool vec, cudaStream_t st) {
    return vec ? quantize_launch_vec<E, FP4, true>(m, static_cast<const E *>(x), ld_x, T, st)
               : quantize_launch_vec<E, FP4, false>(m, static_cast<const E *>(x), ld_x, T, st);
}

template <typename E, bool FP4, bool VEC>
int dequantize_launch_vec(const lora_mx *m, E *out, int64_t ld_out, int T, cudaStream_t st) {
    const RowGrid g = row_grid(T, m->cols);
    auto kernel = g.four ? mx_dequantize_kernel<E, FP4, VEC, 4> : mx_dequantize_kernel<E, FP4, VEC, 1>;
    return launch_after(kernel, g.grid, ROWS_THREADS, 0, 0, st, out, ld_out, static_cast<const unsigned char *>(m->q), m->scales, T,
                        m->cols);
}
template <typename E, bool FP4>
int dequantize_launch(const lora_mx *m, void *out, int64_t ld_out, int T, bool vec, cudaStream_t st) {
    return vec ? dequantize_launch_vec<E, FP4, true>(m, static_cast<E *>(out), ld_out, T, st)
               : dequantize_launch_vec<E, FP4, false>(m, static_cast<E *>(out), ld_out, T, st);
}

}  // namespace

int check_mx(const lora_mx *m, int64_t rows) {
    if (!m) return LORA_ERR_NULL;
    if (m->format != LORA_MXFP8 && m->format != LORA_MXFP4) return LORA_ERR_DTYPE;
    if (m->rows < 0 || m->rows > LORA_MX_MAX || m->cols < 1 || m->cols > LORA_MX_MAX || m->rows < rows)
        return LORA_ERR_SHAPE;
    if (m->rows == 0) return LORA_OK;
    if (!m->q || !m->scales) return LORA_ERR_NULL;
    if (!mx_aligned(m->q, LORA_MX_ALIGN) || !mx_aligned(m->scales, LORA_MX_ALIGN)) return LORA_ERR_ALIGN;
    return LORA_OK;
}

}  // namespace lora

extern "C" {

int64_t lora_mx_row_bytes(int32_t format, int32_t cols) {
    if ((format != LORA_MXFP8 && format != LORA_MXFP4) || cols < 1 || cols > LORA_MX_MAX) return 0;
    return lora::mx_row_bytes(format, cols);
}

int64_t lora_mx_scale_bytes(int32_t rows, int32_t cols) {
    if (rows < 0 || rows > LORA_MX_MAX || cols < 1 || cols > LORA_MX_MAX) return 0;
    const int64_t bands = ((int64_t)rows + lora::MX_TILE_ROWS - 1) / lora::MX_TILE_ROWS;
    return bands * (lora::mx_padded(cols) / lora::MX_TILE_COLS) * lora::MX_TILE_BYTES;
}

int lora_mx_quantize(const lora_mx *q, const void *x, int64_t ld_x, int32_t T, lora_dtype dtype, void *stream) {
    using namespace lora;
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    if (T < 0) return LORA_ERR_SHAPE;
    const int rc = check_mx(q, T);
    if (rc != LORA_OK) return rc;
    if (ld_x < q->cols) return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!x) return LORA_ERR_NULL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool fp4 = q->format == LORA_MXFP4, vec = mx_vec(x, ld_x, q->cols, dtype == LORA_BF16 ? 2 : 4);
    if (dtype == LORA_BF16)
        return fp4 ? quantize_launch<__nv_bfloat16, true>(q, x, ld_x, T, vec, st)
                   : quantize_launch<__nv_bfloat16, false>(q, x, ld_x, T, vec, st);
    return fp4 ? quantize_launch<float, true>(q, x, ld_x, T, vec, st) : quantize_launch<float, false>(q, x, ld_x, T, vec, st);
}

int lora_mx_dequantize(void *out, int64_t ld_out, const lora_mx *q, int32_t T, lora_dtype dtype, void *stream) {
    using namespace lora;
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    if (T < 0) return LORA_ERR_SHAPE;
    const int rc = check_mx(q, T);
    if (rc != LORA_OK) return rc;
    if (ld_out < q->cols) return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!out) return LORA_ERR_NULL;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const bool fp4 = q->format == LORA_MXFP4, vec = mx_vec(out, ld_out, q->cols, dtype == LORA_BF16 ? 2 : 4);
    if (dtype == LORA_BF16)
        return fp4 ? dequantize_launch<__nv_bfloat16, true>(q, out, ld_out, T, vec, st)
                   : dequantize_launch<__nv_bfloat16, false>(q, out, ld_out, T, vec, st);
    return fp4 ? dequantize_launch<float, true>(q, out, ld_out, T, vec, st) : dequantize_launch<float, false>(q, out, ld_out, T, vec, st);
}

int lora_rms_norm(void *h, int64_t ld_h, const void *x, int64_t ld_x, const void *residual, int64_t ld_r,
                  void *residual_out, int64_t ld_ro, const void *weight, float eps, int32_t T, int32_t d,
                  const lora_mx *q, lora_dtype dtype, void *stream) {
    using namespace lora;
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    if (T < 0 || T > LORA_MAX_ROWS || d < 1 || d > LORA_MX_MAX || !(eps >= 0.f)) return LORA_ERR_SHAPE;
    if (!h && !q) return LORA_ERR_NULL;
    if (!residual != !residual_out) return LORA_ERR_NULL;
    if (h && h == residual_out) return LORA_ERR_SHAPE;
    if (ld_x < d || (h && ld_h < d) || (residual && (ld_r < d || ld_ro < d))) return LORA_ERR_SHAPE;
    if (q) {
        const int rc = check_mx(q, T);
        if (rc != LORA_OK) return rc;
        if (q->cols != d) return LORA_ERR_SHAPE;
    }
    if (T == 0) return LORA_OK;
    if (!x || !weight) return LORA_ERR_NULL;
    NormArgs a{};
    a.h = h, a.ld_h = ld_h, a.x = x, a.ld_x = ld_x, a.residual = residual, a.ld_r = ld_r;
    a.sum = residual_out, a.ld_s = ld_ro, a.weight = weight, a.eps = eps, a.T = T, a.d = d;
    if (q) a.q = static_cast<unsigned char *>(q->q), a.scales = q->scales;
    const int es = dtype == LORA_BF16 ? 2 : 4;
    bool vec = mx_vec(x, ld_x, d, es) && mx_aligned(weight, 16) && (!h || mx_vec(h, ld_h, d, es));
    if (residual) vec = vec && mx_vec(residual, ld_r, d, es) && mx_vec(residual_out, ld_ro, d, es);
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int form = !q ? NORM_NO_Q : q->format == LORA_MXFP4 ? NORM_FP4 : NORM_FP8;
    return dtype == LORA_BF16 ? norm_dispatch<__nv_bfloat16>(a, form, vec, sms, st) : norm_dispatch<float>(a, form, vec, sms, st);
}

}  // extern "C"
