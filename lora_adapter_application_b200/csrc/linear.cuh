// What the dense products share (lora_linear, lora_expert_linear): the call's
// parameters, the epilogue's arithmetic and the way from a row tile to its expert.
#pragma once

#include "mx.cuh"

namespace lora {

// A call, as the kernels take it.  Rows: of a plain product, 0..T-1 of x and y.  Of the experts', position q of the grouping
// is slot perm[q] (a row of y) and row perm[q] / x_div of x; expert e has positions seg_start[e] .. seg_start[e + 1] - 1.
struct LinArgs {
    void *y;
    const void *x, *w;
    const void *bias, *addend, *residual;   // NULL: none
    int64_t ld_y, ld_x, ld_w, ld_a, ld_r;
    int T, d_in, d_out;   // d_out: columns of y; W has n_w rows (gated: the gate's d_out, then the up projection's)
    int n_w;
    int act;
    const int32_t *perm, *seg_start;   // experts, else NULL
    int N, x_div;
    int32_t *status;
};

// ------------------------------------------------------------------ epilogue
// silu and both gelus as quotients or products without cancellation: z / (1 + e^-z) and z erfc(-z / sqrt 2) / 2 keep their
// relative accuracy where z is far below 0, which z (1 + erf) / 2 and z (1 + tanh) / 2 lose.
// FAST (results rounded to bf16, off by up to 2^-8 of themselves): the approximate base-2 exponential and reciprocal; for fp32
// results the accurate functions.  The exponential multiplies its argument's rounding by the argument u (silu: u = z), so both
// are within (9 + 3.2 |u|) 2^-23 of the value.  With exponential and reciprocal rounded exactly, silu is off by 2^-19.9 at worst
// for |z| <= 20, the tanh form of gelu by as much up to |z| = 3, then by more, where the value goes to 0: 2^-15.8 at z = -9.8
// (a value of 1e-35).
template <bool FAST>
__device__ __forceinline__ float over_one_plus_exp(float z, float u) {   // z / (1 + e^-u)
    if (!FAST) return z / (1.f + expf(-u));
    float e, r;   // where e^-u passes fp32's range, the quotient is z times 0
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(-1.4426950408889634f * u));
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(r) : "f"(1.f + e));
    return z * r;
}
// z Phi(z) = z erfc(-z / sqrt 2) / 2.  For a = |z| / sqrt 2: erfc(a) = t e^(-a^2 + g(t)), t = 1 / (1 + a / 2), the form of Press
// et al., Numerical Recipes (error function, Chebyshev fit).  g is a polynomial of degree 9 of our own: least squares to
// ln(erfc(a) e^(a^2) / t) in 64 bits on the 4000 Chebyshev nodes of t in [2/17, 1] (a in [0, 15]), weights of the squares started
// at 1 and 200 times multiplied by each node's error (Lawson's iteration), which leaves the largest error smallest: 6.3e-8; then
// in powers of t, times log2 e, rounded to fp32: 1.9e-7 (1.6 units of 2^-23, at a = 0.04).  In all within (8 + z^2) 2^-23 of the
// value, z^2 from the rounding of the exponent.  A third of the instructions of erfcf: 4126 x 1024 x 13536 with this activation 201 -> 140 us.
__device__ __forceinline__ float gelu_fast(float z) {
    float t, e;
    asm("rcp.approx.ftz.f32 %0, %1;\n" : "=f"(t) : "f"(fmaf(fabsf(z), 0.35355339059327376f, 1.f)));
    float g = 0.23579010367393494f;
    g = fmaf(g, t, -1.1268246173858643f);
    g = fmaf(g, t, 2.006770372390747f);
    g = fmaf(g, t, -1.4504882097244263f);
    g = fmaf(g, t, 0.24917496740818024f);
    g = fmaf(g, t, -0.189505934715271f);
    g = fmaf(g, t, 0.11389805376529694f);
    g = fmaf(g, t, 0.5447050333023071f);
    g = fmaf(g, t, 1.4422062635421753f);
    g = fmaf(g, t, -1.8257261514663696f);
    asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(e) : "f"(fmaf(-0.72134752044448170f * z, z, g)));
    const float h = 0.5f * fminf(z, 1e30f) * (t * e);   // the smaller of the two parts (0 where z is infinite)
    return z < 0.f ? h : z - h;
}
template <bool FAST, int N>
__device__ __forceinline__ void activate(int act, float *z) {
    switch (act) {
        case LORA_ACT_SILU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = over_one_plus_exp<FAST>(z[i], z[i]);
            break;
        case LORA_ACT_GELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = FAST ? gelu_fast(z[i]) : 0.5f * z[i] * erfcf(-0.70710678118654752f * z[i]);
            break;
        case LORA_ACT_GELU_TANH:   // (1 + tanh u) / 2 = 1 / (1 + e^-2u), u = sqrt(2 / pi) (z + 0.044715 z^3)
#pragma unroll
            for (int i = 0; i < N; ++i)
                z[i] = over_one_plus_exp<FAST>(z[i], 1.5957691216057308f * (z[i] + 0.044715f * z[i] * z[i] * z[i]));
            break;
        case LORA_ACT_RELU:
#pragma unroll
            for (int i = 0; i < N; ++i) z[i] = z[i] < 0.f ? 0.f : z[i];   // NaN stays
            break;
        default: break;
    }
}

// ------------------------------------------------------------------ experts
// Row tiles (rows positions each) of experts before e, for e in 0..N, to pre[0..N] in shared memory, by a whole block, and
// seg_start to start[0..N] (may be NULL); part: 32 words of shared memory.  Ends with the block's barrier.
__device__ __forceinline__ void count_tiles(const int32_t *seg_start, int N, int rows, int *pre, int *start, int *part) {
    const int per = (N + (int)blockDim.x - 1) / (int)blockDim.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int lo = min(N, (int)threadIdx.x * per), hi = min(N, lo + per);
    int sum = 0;
    for (int e = lo; e < hi; ++e) sum += (seg_start[e + 1] - seg_start[e] + rows - 1) / rows;
    int up = sum;
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        const int v = __shfl_up_sync(FULL, up, d);
        if (lane >= d) up += v;
    }
    if (lane == 31) part[warp] = up;
    __syncthreads();
    int at = up - sum;
    for (int w = 0; w < warp; ++w) at += part[w];
    if (threadIdx.x == 0) {
        pre[0] = 0;
        if (start) start[0] = seg_start[0];
    }
    for (int e = lo; e < hi; ++e) {
        at += (seg_start[e + 1] - seg_start[e] + rows - 1) / rows;
        pre[e + 1] = at;
        if (start) start[e + 1] = seg_start[e + 1];
    }
    __syncthreads();
}
// The expert of row tile t: the last e with pre[e] <= t (t < pre[N]), from e on (pre[e] <= t), by a whole warp: 32 to a look.
__device__ __forceinline__ int expert_of(const int *pre, int N, int t, int e = 0) {
    const int lane = threadIdx.x & 31;
    for (;;) {
        const unsigned before = __ballot_sync(FULL, e + 1 + lane <= N && pre[e + 1 + lane] <= t);
        e += __popc(before);
        if (before != FULL) return e;
    }
}

// tmaps.cu
int tensor_map_rows(CUtensorMap *out, const void *base, uint64_t inner, uint64_t rows, uint64_t row_stride,
                    uint32_t box_rows);

// linear_tc.cu: bf16, any stride and alignment; x_rows: rows that x has
int launch_linear_tc(const LinArgs &a, int64_t x_rows, bool gated, int dev, cudaStream_t st);

// linear_simt.cu: fp32, any stride and alignment
int launch_linear_simt(const LinArgs &a, bool gated, int sms, cudaStream_t st);

}  // namespace lora
