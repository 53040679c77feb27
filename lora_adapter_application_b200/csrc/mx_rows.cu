// Row operators around a microscaled base: quantise, read back, and the
// root-mean-square norm with the residual's sum whose rows leave in the data's
// type and, optionally, microscaled.  Contracts: lora_delta.h.
//
// All three stream rows once and are bound by HBM.  A lane holds 8 consecutive
// columns (one 16-byte bf16 access), so 4 lanes hold a scale's block of 32 and a
// warp 256 columns = two scale tiles; the block's largest magnitude takes two
// shuffles, the tile's four scale bytes two more.
#include "mx.cuh"

#include <algorithm>

namespace lora {

namespace {

constexpr int ROWS_THREADS = 256;

// The rows a warp takes at once: r, r + 32, r + 64, r + 96 of a 128-row band,
// whose scale words are neighbours (16 bytes of a tile).  Small matrices have
// fewer of them; row R of a band of height h is there if R < h.
struct RowItem {
    int64_t band;   // first row of the 128-row band
    int r;          // row within 32
    int64_t group;  // 256-column group
};
__device__ __forceinline__ RowItem row_item(int64_t item, int r_count, int64_t groups) {
    RowItem it;
    it.group = item % groups;
    const int64_t rest = item / groups;
    it.r = (int)(rest % r_count);
    it.band = rest / r_count * MX_TILE_ROWS;
    return it;
}

template <typename E, bool FP4, bool VEC>
__global__ void __launch_bounds__(ROWS_THREADS)
    mx_quantize_kernel(unsigned char *q, uint8_t *scales, const E *x, int64_t ld_x, int T, int cols, int r_count,
                       int64_t items) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (ROWS_THREADS / 32) + (threadIdx.x >> 5);
    if (item >= items) return;
    const int64_t pad = mx_padded(cols), groups = (pad + 255) / 256, n_kt = pad / MX_TILE_COLS;
    const int64_t row_bytes = FP4 ? pad / 2 : pad;
    const RowItem it = row_item(item, r_count, groups);
    const int64_t col = it.group * 256 + lane * 8;
    float v[4][8];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t row = it.band + it.r + 32 * j;
        load8<VEC>(x + (row < T ? row : 0) * ld_x + col, row < T ? cols - col : 0, v[j]);
    }
    uint32_t word[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) word[j] = mx_scale_warp<FP4>(v[j]);
    if (col >= pad) return;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t row = it.band + it.r + 32 * j;
        if (row < T) {
            mx_store8<FP4>(q + row * row_bytes, col, v[j]);
            if ((lane & 15) == 0)
                *reinterpret_cast<uint32_t *>(scales + mx_scale_word(row, col >> 7, n_kt)) = word[j];
        }
    }
}

template <typename E, bool FP4, bool VEC>
__global__ void __launch_bounds__(ROWS_THREADS)
    mx_dequantize_kernel(E *out, int64_t ld_out, const unsigned char *q, const uint8_t *scales, int T, int cols,
                         int r_count, int64_t items) {
    const int lane = threadIdx.x & 31;
    const int64_t item = (int64_t)blockIdx.x * (ROWS_THREADS / 32) + (threadIdx.x >> 5);
    if (item >= items) return;
    const int64_t pad = mx_padded(cols), groups = (pad + 255) / 256, n_kt = pad / MX_TILE_COLS;
    const int64_t row_bytes = FP4 ? pad / 2 : pad;
    const RowItem it = row_item(item, r_count, groups);
    const int64_t col = it.group * 256 + lane * 8;
    if (col >= cols) return;
    uint2 e[4];
    uint32_t code[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t row = it.band + it.r + 32 * j;
        if (row < T) {
            const unsigned char *p = q + row * row_bytes;
            if (FP4) e[j].x = *reinterpret_cast<const uint32_t *>(p + (col >> 1));
            else e[j] = *reinterpret_cast<const uint2 *>(p + col);
            code[j] = scales[mx_scale_word(row, col >> 7, n_kt) + ((col >> 5) & 3)];
        }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int64_t row = it.band + it.r + 32 * j;
        if (row < T) {
            float v[8];
            if (FP4) mx_unpack_e2m1(e[j].x, v);
            else mx_unpack_e4m3(e[j], v);
            const float s = mx_scale(code[j]);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] *= s;
            store8<VEC>(out + row * ld_out + col, cols - col, v);
        }
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
// thread) between the sum of squares and the scaling; V = 0: longer rows, read a
// second time (from the stored sum where there is a residual).
template <typename E, int V, int Q, bool VEC, bool RES>
__global__ void __launch_bounds__(1024) rms_norm_kernel(const __grid_constant__ NormArgs a, int tpr) {
    __shared__ float part[32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int t = threadIdx.x % tpr;
    const int64_t row = (int64_t)blockIdx.x * (blockDim.x / tpr) + threadIdx.x / tpr;
    if (row >= a.T) return;   // whole warps; only blocks of one warp per row hold several rows
    const E *x = static_cast<const E *>(a.x) + row * a.ld_x;
    const E *res = RES ? static_cast<const E *>(a.residual) + row * a.ld_r : nullptr;
    E *sum = RES ? static_cast<E *>(a.sum) + row * a.ld_s : nullptr;
    const int64_t pad = mx_padded(a.d);
    const int64_t end = Q ? pad : a.d;   // columns the warps walk over
    float keep[V > 0 ? V : 1][8];
    float ss = 0.f;
    auto first = [&](int64_t c, float *v) {   // the row's (summed) 8 columns at c
        const int64_t n = a.d - c;
        load8<VEC>(x + c, n, v);
        if (RES) {
            float r[8];
            load8<VEC>(res + c, n, r);
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = round_to(x, v[i] + r[i]);
            store8<VEC>(sum + c, n, v);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss = fmaf(v[i], v[i], ss);
    };
    if (V > 0) {
#pragma unroll
        for (int k = 0; k < V; ++k) first(8 * ((int64_t)t + (int64_t)k * tpr), keep[k]);
    } else {
        for (int64_t c = 8 * t; c < a.d; c += 8 * (int64_t)tpr) first(c, keep[0]);
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
    auto second = [&](int64_t c, float *v) {
        const int64_t n = a.d - c;
        float g[8];
        load8<VEC>(w + c, n, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = round_to(x, v[i] * rstd * g[i]);
        if (h) store8<VEC>(h + c, n, v);
        if (Q) {   // of the rounded row: the base product sees what the adapters see
            const uint32_t word = mx_scale_warp<Q == NORM_FP4>(v);
            if (c < pad) {
                mx_store8<Q == NORM_FP4>(a.q + row * (Q == NORM_FP4 ? pad / 2 : pad), c, v);
                if ((lane & 15) == 0)
                    *reinterpret_cast<uint32_t *>(a.scales + mx_scale_word(row, c >> 7, pad / MX_TILE_COLS)) = word;
            }
        }
    };
    if (V > 0) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int64_t c = 8 * ((int64_t)t + (int64_t)k * tpr);
            if (c - 8 * lane < end) second(c, keep[k]);   // the whole warp: its first column
        }
    } else {
        for (int64_t c = 8 * t; c - 8 * lane < end; c += 8 * (int64_t)tpr) {
            load8<VEC>((RES ? sum : x) + c, a.d - c, keep[0]);
            second(c, keep[0]);
        }
    }
}

template <typename E, int V, int Q, bool VEC>
void norm_launch_res(const NormArgs &a, int tpr, unsigned blocks, int threads, cudaStream_t st) {
    if (a.residual) rms_norm_kernel<E, V, Q, VEC, true><<<blocks, threads, 0, st>>>(a, tpr);
    else rms_norm_kernel<E, V, Q, VEC, false><<<blocks, threads, 0, st>>>(a, tpr);
}

template <typename E, int Q, bool VEC>
void norm_launch(const NormArgs &a, int sms, cudaStream_t st) {
    const int64_t vecs = (mx_padded(a.d) + 7) / 8;   // 8-column groups of a row
    // Many rows: four groups a thread (one warp of loads in flight per row); few
    // rows: one group a thread, the shortest way through one row.
    int v = a.T >= 4 * sms ? 4 : 1;
    while (v < 4 && vecs > (int64_t)v * 1024) v *= 2;
    int64_t tpr = 32;
    while (tpr < 1024 && tpr * v < vecs) tpr *= 2;
    if (tpr * v < vecs) v = 0;
    const int threads = (int)std::max<int64_t>(tpr, tpr == 32 ? 128 : tpr);
    const int rows = threads / (int)tpr;
    const unsigned blocks = (unsigned)((a.T + rows - 1) / rows);
    switch (v) {
        case 1: norm_launch_res<E, 1, Q, VEC>(a, (int)tpr, blocks, threads, st); break;
        case 2: norm_launch_res<E, 2, Q, VEC>(a, (int)tpr, blocks, threads, st); break;
        case 4: norm_launch_res<E, 4, Q, VEC>(a, (int)tpr, blocks, threads, st); break;
        default: norm_launch_res<E, 0, Q, VEC>(a, (int)tpr, blocks, threads, st);
    }
}

template <typename E>
void norm_dispatch(const NormArgs &a, int q, bool vec, int sms, cudaStream_t st) {
    if (q == NORM_NO_Q) vec ? norm_launch<E, NORM_NO_Q, true>(a, sms, st) : norm_launch<E, NORM_NO_Q, false>(a, sms, st);
    else if (q == NORM_FP8) vec ? norm_launch<E, NORM_FP8, true>(a, sms, st) : norm_launch<E, NORM_FP8, false>(a, sms, st);
    else vec ? norm_launch<E, NORM_FP4, true>(a, sms, st) : norm_launch<E, NORM_FP4, false>(a, sms, st);
}

struct RowGrid {
    int r_count;
    int64_t items;
    unsigned blocks;
};
RowGrid row_grid(int64_t T, int64_t cols) {
    RowGrid g;
    const int64_t groups = (mx_padded(cols) + 255) / 256, bands = (T + MX_TILE_ROWS - 1) / MX_TILE_ROWS;
    g.r_count = (int)std::min<int64_t>(T, 32);
    g.items = bands * g.r_count * groups;
    g.blocks = (unsigned)((g.items + ROWS_THREADS / 32 - 1) / (ROWS_THREADS / 32));
    return g;
}

template <typename E, bool FP4>
void quantize_launch(const lora_mx *m, const void *x, int64_t ld_x, int T, bool vec, cudaStream_t st) {
    const RowGrid g = row_grid(T, m->cols);
    auto *q = static_cast<unsigned char *>(m->q);
    auto *p = static_cast<const E *>(x);
    if (vec) mx_quantize_kernel<E, FP4, true><<<g.blocks, ROWS_THREADS, 0, st>>>(q, m->scales, p, ld_x, T, m->cols, g.r_count, g.items);
    else mx_quantize_kernel<E, FP4, false><<<g.blocks, ROWS_THREADS, 0, st>>>(q, m->scales, p, ld_x, T, m->cols, g.r_count, g.items);
}

template <typename E, bool FP4>
void dequantize_launch(const lora_mx *m, void *out, int64_t ld_out, int T, bool vec, cudaStream_t st) {
    const RowGrid g = row_grid(T, m->cols);
    auto *q = static_cast<const unsigned char *>(m->q);
    auto *p = static_cast<E *>(out);
    if (vec) mx_dequantize_kernel<E, FP4, true><<<g.blocks, ROWS_THREADS, 0, st>>>(p, ld_out, q, m->scales, T, m->cols, g.r_count, g.items);
    else mx_dequantize_kernel<E, FP4, false><<<g.blocks, ROWS_THREADS, 0, st>>>(p, ld_out, q, m->scales, T, m->cols, g.r_count, g.items);
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
        fp4 ? quantize_launch<__nv_bfloat16, true>(q, x, ld_x, T, vec, st)
            : quantize_launch<__nv_bfloat16, false>(q, x, ld_x, T, vec, st);
    else
        fp4 ? quantize_launch<float, true>(q, x, ld_x, T, vec, st)
            : quantize_launch<float, false>(q, x, ld_x, T, vec, st);
    return cuda_rc(cudaGetLastError());
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
        fp4 ? dequantize_launch<__nv_bfloat16, true>(q, out, ld_out, T, vec, st)
            : dequantize_launch<__nv_bfloat16, false>(q, out, ld_out, T, vec, st);
    else
        fp4 ? dequantize_launch<float, true>(q, out, ld_out, T, vec, st)
            : dequantize_launch<float, false>(q, out, ld_out, T, vec, st);
    return cuda_rc(cudaGetLastError());
}

int lora_rms_norm(void *h, int64_t ld_h, const void *x, int64_t ld_x, const void *residual, int64_t ld_r,
                  void *residual_out, int64_t ld_ro, const void *weight, float eps, int32_t T, int32_t d,
                  const lora_mx *q, lora_dtype dtype, void *stream) {
    using namespace lora;
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    if (T < 0 || T > LORA_MAX_ROWS || d < 1 || d > LORA_MX_MAX || !(eps >= 0.f)) return LORA_ERR_SHAPE;
    if (!h && !q) return LORA_ERR_NULL;
    if (!residual != !residual_out) return LORA_ERR_NULL;
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
    if (dtype == LORA_BF16) norm_dispatch<__nv_bfloat16>(a, form, vec, sms, st);
    else norm_dispatch<float>(a, form, vec, sms, st);
    return cuda_rc(cudaGetLastError());
}

}  // extern "C"
