// Before and after the experts' products (contracts: lora_expert_route and
// lora_expert_sum in lora_delta.h).
#include "linear.cuh"

#include <algorithm>

namespace lora {

namespace {

// ------------------------------------------------------------------ route
// A warp takes a token; its lanes hold the logits, expert 32 i + lane in key[i], as whole numbers that order as the logits
// do, 0 for those that cannot be chosen.  A pick is one warp reduction in hardware for bf16 logits, whose 16 bits share a
// key with the expert's complement (the largest key is the first expert's of the largest logit), two for fp32: the largest
// key, and the first expert that holds it.  The weights come from the picks' logits, so that ids depend on comparisons
// alone.  Bound: latency (1 token: 2.2 us), then instructions, of which a pick costs about 35 (8192 x 256 bf16, 8 picks: 9.2 us,
// issue slots 60 % busy; fp32 11.3).
constexpr int ROUTE_WARPS = 4;

__device__ __forceinline__ uint32_t order_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.f);   // -0 as 0: the two tie
    return !(l > -INFINITY) ? 0u : u >> 31 ? ~u : u | 0x80000000u;   // -infinity and NaN: never chosen
}
__device__ __forceinline__ float key_value(uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7fffffffu : ~k); }
// e^(l - m), 1 where both are infinite
__device__ __forceinline__ float exp_below(float l, float m) { return l == m ? 1.f : expf(l - m); }

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int d = 16; d; d /= 2) v += __shfl_xor_sync(FULL, v, d);
    return v;
}

template <typename E, int VPL>
__global__ void __launch_bounds__(32 * ROUTE_WARPS) route_kernel(int32_t *ids, float *weights, const E *logits, int64_t ld, int T,
                                                                 int n, int k, int sigmoid, int renorm, float scale) {
    constexpr bool SHARED_KEY = sizeof(E) == 2;
    pdl_next();
    pdl_wait();
    const int t = (int)blockIdx.x * ROUTE_WARPS + (int)(threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (t >= T) return;
    const E *row = logits + t * ld;
    // the logit of a key: its high 16 bits, the rest as order_key leaves it for a bf16 value
    auto value = [](uint32_t key) { return key_value(SHARED_KEY ? (key & 0xffff0000u) | (key >> 31 ? 0u : 0xffffu) : key); };
    uint32_t key[VPL], top = 0;   // top: the largest of this lane's
#pragma unroll
    for (int i = 0; i < VPL; ++i) {
        key[i] = 32 * i + lane < n ? order_key(load_elem(row + 32 * i + lane)) : 0u;
        if (SHARED_KEY && key[i]) key[i] = (key[i] & 0xffff0000u) | (0xffffu ^ (uint32_t)(32 * i + lane));
        top = max(top, key[i]);
    }
    const float most = value(__reduce_max_sync(FULL, top));   // of no use where no expert is open: then nothing is chosen
    float all = 0.f;
    if (!sigmoid && !renorm) {   // the softmax's sum over all experts
#pragma unroll
        for (int i = 0; i < VPL; ++i)
            if (key[i]) all += exp_below(value(key[i]), most);
        all = warp_sum(all);
    }
    uint32_t my_key = 0;   // lane j: the j-th pick
    int my_id = -1;
    for (int j = 0; j < k; ++j) {
        const uint32_t best = __reduce_max_sync(FULL, top);
        if (best == 0) break;
        int id;
        if (SHARED_KEY) {
            id = (int)(0xffffu ^ (best & 0xffffu));
        } else {
            int at = VPL;
#pragma unroll
            for (int i = VPL - 1; i >= 0; --i)
                if (key[i] == best) at = i;
            id = (int)__reduce_min_sync(FULL, at < VPL ? (unsigned)(32 * at + lane) : 0xffffffffu);
        }
        if (lane == j) my_key = best, my_id = id;
        if ((id & 31) == lane) {
            top = 0;
#pragma unroll
            for (int i = 0; i < VPL; ++i) {
                if (i == id >> 5) key[i] = 0;
                top = max(top, key[i]);
            }
        }
    }
    const float l = value(my_key);
    float w = 0.f;
    if (my_id >= 0) {
        if (!sigmoid) {
            w = exp_below(l, most);
        } else {
            // 1 / (1 + e^-l) = e^min(l, 0) / (1 + e^-|l|); where only the ratios matter, over e^min(most, 0), so that
            // logits far below 0 leave a sum that is not 0
            const float up = renorm ? exp_below(fminf(l, 0.f), fminf(most, 0.f)) : expf(fminf(l, 0.f));
            w = up / (1.f + expf(-fabsf(l)));
        }
    }
    if (renorm) all = warp_sum(w);
    if (sigmoid && !renorm) all = 1.f;
    if (lane < k) {
        ids[(int64_t)t * k + lane] = my_id;
        weights[(int64_t)t * k + lane] = my_id >= 0 ? w / all * scale : 0.f;
    }
}

template <typename E>
int launch_route(int32_t *ids, float *weights, const void *logits, int64_t ld, int T, int n, int k, int sigmoid, int renorm,
                 float scale, cudaStream_t st) {
    const dim3 grid((unsigned)((T + ROUTE_WARPS - 1) / ROUTE_WARPS));
    const E *l = static_cast<const E *>(logits);
    auto go = [&](auto kernel) { return launch_after(kernel, grid, 32 * ROUTE_WARPS, 0, 0, st, ids, weights, l, ld, T, n, k, sigmoid, renorm, scale); };
    if (n <= 64) return go(route_kernel<E, 2>);
    if (n <= 128) return go(route_kernel<E, 4>);
    if (n <= 256) return go(route_kernel<E, 8>);
    if (n <= 512) return go(route_kernel<E, 16>);
    return go(route_kernel<E, 32>);
}

// -------------------------------------------------------------------- sum
// A warp takes 256 columns of a few tokens, eight a lane (VEC: 16-byte accesses; else 32 columns apart), and adds the slots'
// rows in slot order, then the residual, fp32, one rounding: ahead of the rows a residual, larger than they are, would have
// every sum rounded at its size (33 x 8 x 2048 in fp32, four times a row: 7.0e-8 off the value for 2.6e-8).  The tokens' ids
// and weights come in one load of the warp, ahead of all; four rows' loads are in flight at a time.  Bound: HBM (8192 x 4 x
// 4096 with a residual 64.1 us, 96 % of the measured copy rate; with a block for each token 68.0).
constexpr int SUM_WARPS = 4, SUM_TOKENS = 4;

template <typename E, bool VEC>
__global__ void __launch_bounds__(32 * SUM_WARPS) sum_kernel(E *y, int64_t ld_y, const E *x, int64_t ld_x, const int32_t *ids,
                                                             const float *weights, int n, int T, int k, int tokens, int d, const E *res,
                                                             int64_t ld_r) {
    pdl_next();
    pdl_wait();
    using Raw = typename RawOf<E>::type;
    const int64_t t0 = (int64_t)blockIdx.x * tokens;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c0 = ((int)blockIdx.y * SUM_WARPS + warp) * 256;   // the warp's 256 columns
    if (c0 >= d) return;
    const int here = min(tokens, (int)(T - t0));
    // tokens * k <= 32, or one token of up to 32 slots: lane l has slot l
    const int my_id = lane < here * k ? ids[t0 * k + lane] : -1;
    const float my_w = lane < here * k ? weights[t0 * k + lane] : 0.f;
    for (int i = 0; i < here; ++i) {
        const int64_t t = t0 + i;
        float acc[8], v[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] = -0.f;   // -0: added to a residual of -0 it leaves it so
        Raw r;
        for (int j = 0; j < k; j += 4) {
            Raw u[4];
            float w[4];
            bool there[4];
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                const int at = min(i * k + j + s, 31);
                const int id = __shfl_sync(FULL, my_id, at);
                w[s] = __shfl_sync(FULL, my_w, at);
                there[s] = j + s < k && id >= 0 && id < n;
                // the rows of slots without an expert hold nothing of use: not read
                if (there[s]) load8<VEC>(x + (t * k + j + s) * ld_x, c0, d, lane, u[s]);
            }
            // beside the last rows; behind them where halves are packed two to a register, which each waits for its load
            if (VEC && res && j + 4 >= k) load8<VEC>(res + t * ld_r, c0, d, lane, r);
#pragma unroll
            for (int s = 0; s < 4; ++s)
                if (there[s]) {
                    raw_values(u[s], v);
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[c] = fmaf(w[s], v[c], acc[c]);
                }
        }
        if (res) {
            if (!VEC) load8<VEC>(res + t * ld_r, c0, d, lane, r);
            raw_values(r, v);
        } else {
#pragma unroll
            for (int c = 0; c < 8; ++c) v[c] = 0.f;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) acc[c] += v[c];
        Raw u;
        raw_round(acc, u);
        store8<VEC>(y + t * ld_y, c0, d, lane, u);
    }
}

template <typename E>
int launch_sum(void *y, int64_t ld_y, const void *x, int64_t ld_x, const int32_t *ids, const float *weights, int n, int T, int k,
               int d, const void *res, int64_t ld_r, cudaStream_t st) {
    const bool vec = mx_vec(x, ld_x, d, sizeof(E)) && mx_vec(y, ld_y, d, sizeof(E)) && (!res || mx_vec(res, ld_r, d, sizeof(E)));
    // several tokens a warp only where many: a block of one token lives mostly for the latency of its ids (us, one / several, bf16:
    // 1024 x 4 x 4096 10.2 / 10.9, 4096 34.0 / 33.2, 8192 68.0 / 63.7; 1024 x 2 x 512 2.2 / 3.9, 16384 19.1 / 15.3; not worth it at
    // eight slots, 4096 x 8 x 2048 27.8 / 30.9, 16384 99 / 102; fp32 within 3 % from 4096 on, at 512
    // columns 4096 x 2 6.8 / 7.2, 8192 13.0 / 13.8, 16384 25.0 / 23.8)
    const int tokens = T >= 4096 ? std::max(1, std::min(SUM_TOKENS, 32 / k)) : 1;
    const dim3 grid((unsigned)((T + tokens - 1) / tokens), (unsigned)((d + 256 * SUM_WARPS - 1) / (256 * SUM_WARPS)));
    return launch_after(vec ? sum_kernel<E, true> : sum_kernel<E, false>, grid, 32 * SUM_WARPS, 0, 0, st, static_cast<E *>(y), ld_y,
                        static_cast<const E *>(x), ld_x, ids, weights, n, T, k, tokens, d, static_cast<const E *>(res), ld_r);
}

}  // namespace

}  // namespace lora

extern "C" {

int lora_expert_route(int32_t *ids, float *weights, const void *logits, int64_t ld, int32_t T, int32_t n_experts, int32_t k,
                      int32_t score, int32_t renormalize, float scale, lora_dtype dtype, void *stream) {
    using namespace lora;
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    if (T < 0 || T > LORA_MAX_ROWS || n_experts < 1 || n_experts > LORA_MAX_EXPERTS || k < 1 || k > LORA_MAX_TOPK || k > n_experts ||
        ld < n_experts || (score != LORA_SCORE_SOFTMAX && score != LORA_SCORE_SIGMOID))
        return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!ids || !weights || !logits) return LORA_ERR_NULL;
    if (!mx_aligned(ids, 4) || !mx_aligned(weights, 4) || !mx_aligned(logits, dtype == LORA_BF16 ? 2 : 4)) return LORA_ERR_ALIGN;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    const int sigmoid = score == LORA_SCORE_SIGMOID, renorm = renormalize != 0;
    return dtype == LORA_BF16 ? launch_route<__nv_bfloat16>(ids, weights, logits, ld, T, n_experts, k, sigmoid, renorm, scale, st)
                              : launch_route<float>(ids, weights, logits, ld, T, n_experts, k, sigmoid, renorm, scale, st);
}

int lora_expert_sum(void *y, int64_t ld_y, const void *x, int64_t ld_x, const int32_t *ids, const float *weights,
                    int32_t n_experts, int32_t T, int32_t k, int32_t d, const void *residual, int64_t ld_r, lora_dtype dtype,
                    void *stream) {
    using namespace lora;
    if (dtype != LORA_BF16 && dtype != LORA_FP32) return LORA_ERR_DTYPE;
    if (T < 0 || T > LORA_MAX_ROWS || n_experts < 1 || n_experts > LORA_MAX_EXPERTS || k < 1 || k > LORA_MAX_TOPK || d < 1 ||
        d > LORA_MX_MAX || ld_y < d || ld_x < d || (residual && ld_r < d))
        return LORA_ERR_SHAPE;
    if (T == 0) return LORA_OK;
    if (!y || !x || !ids || !weights) return LORA_ERR_NULL;
    const uintptr_t es = dtype == LORA_BF16 ? 2 : 4;
    if (!mx_aligned(y, es) || !mx_aligned(x, es) || !mx_aligned(residual, es) || !mx_aligned(ids, 4) || !mx_aligned(weights, 4))
        return LORA_ERR_ALIGN;
    if (y == x || (y == residual && ld_y != ld_r)) return LORA_ERR_SHAPE;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return dtype == LORA_BF16 ? launch_sum<__nv_bfloat16>(y, ld_y, x, ld_x, ids, weights, n_experts, T, k, d, residual, ld_r, st)
                              : launch_sum<float>(y, ld_y, x, ld_x, ids, weights, n_experts, T, k, d, residual, ld_r, st);
}

}  // extern "C"
