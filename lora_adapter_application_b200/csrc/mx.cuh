// Microscaled storage (lora_mx): element and scale conversions, scale
// addressing and the argument checks shared by the kernels that read or write
// it.  Formats: OCP Microscaling v1.0, MXFP8 (e4m3) and MXFP4 (e2m1), blocks of
// 32 elements along a row with one e8m0 scale.
#pragma once

#include "kernels.cuh"

#include <cuda_fp16.h>

namespace lora {

constexpr int MX_BLOCK = 32;         // elements of one scale
constexpr int MX_TILE_ROWS = 128;    // rows of one scale tile
constexpr int MX_TILE_COLS = 128;    // columns (4 blocks) of one scale tile
constexpr int MX_TILE_BYTES = 512;

// columns of a stored row, padding included
__host__ __device__ constexpr int64_t mx_padded(int64_t cols) {
    return (cols + MX_TILE_COLS - 1) / MX_TILE_COLS * MX_TILE_COLS;
}
__host__ __device__ constexpr int64_t mx_row_bytes(int format, int64_t cols) {
    return format == LORA_MXFP4 ? mx_padded(cols) / 2 : mx_padded(cols);
}

// Byte of the first of a row's four scales in tile column kt (the 4 blocks of
// columns 128 kt .. 128 kt + 127); tiles of one 128-row band run along k.
__host__ __device__ constexpr int64_t mx_scale_word(int64_t row, int64_t kt, int64_t n_kt) {
    return ((row / MX_TILE_ROWS) * n_kt + kt) * MX_TILE_BYTES + (row % 32) * 16 + (row / 32 % 4) * 4;
}

// The scale code of a block from the bits of its largest magnitude: the
// exponent of that magnitude less the format's own largest exponent, not below
// 2^-127.  The bit patterns of magnitudes order as the magnitudes do, with infinity and NaN on
// top: such a block gets the e8m0 NaN (255) and reads back as NaN as a whole.
template <bool FP4>
__device__ __forceinline__ uint32_t mx_code(uint32_t amax_bits) {
    if (amax_bits >= 0x7f800000u) return 255u;
    const int e = (int)(amax_bits >> 23) - (FP4 ? 2 : 8);
    return (uint32_t)max(e, 0);
}
// 2^(127 - code): the factor that brings a block onto its format's grid.  Codes
// of finite blocks end at 252, so the factor is a normal number and the product exact.
// 0 for the NaN code (its elements are stored as zeros).
__device__ __forceinline__ float mx_inverse(uint32_t code) {
    return code == 255u ? 0.f : __uint_as_float((254u - code) << 23);
}
// 2^(code - 127), NaN for 255
__device__ __forceinline__ float mx_scale(uint32_t code) {
    return __uint_as_float(code == 255u ? 0x7fffffffu : code ? code << 23 : 0x00400000u);
}

// 8 scaled elements to storage, round-to-nearest-even, saturating
__device__ __forceinline__ uint2 mx_pack_e4m3(const float *v) {
    uint2 r;
    asm("{\n\t.reg .b16 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 a, %3, %2;\n\tcvt.rn.satfinite.e4m3x2.f32 b, %5, %4;\n\t"
        "cvt.rn.satfinite.e4m3x2.f32 c, %7, %6;\n\tcvt.rn.satfinite.e4m3x2.f32 d, %9, %8;\n\t"
        "mov.b32 %0, {a, b};\n\tmov.b32 %1, {c, d};\n\t}\n"
        : "=r"(r.x), "=r"(r.y)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
__device__ __forceinline__ uint32_t mx_pack_e2m1(const float *v) {
    uint32_t r;
    asm("{\n\t.reg .b8 a, b, c, d;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
        "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\tcvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
        "mov.b32 %0, {a, b, c, d};\n\t}\n"
        : "=r"(r)
        : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
    return r;
}
__device__ __forceinline__ void mx_half2(uint32_t h, float *v) {
    const __half2 x = *reinterpret_cast<__half2 *>(&h);
    v[0] = __low2float(x);
    v[1] = __high2float(x);
}
// 8 stored elements to fp32 (exact), without their scale
__device__ __forceinline__ void mx_unpack_e4m3(uint2 q, float *v) {
    uint32_t h[4];
    asm("{\n\t.reg .b16 a, b, c, d;\n\tmov.b32 {a, b}, %4;\n\tmov.b32 {c, d}, %5;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t"
        "cvt.rn.f16x2.e4m3x2 %2, c;\n\tcvt.rn.f16x2.e4m3x2 %3, d;\n\t}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q.x), "r"(q.y));
#pragma unroll
    for (int i = 0; i < 4; ++i) mx_half2(h[i], v + 2 * i);
}
__device__ __forceinline__ void mx_unpack_e2m1(uint32_t q, float *v) {
    uint32_t h[4];
    asm("{\n\t.reg .b8 a, b, c, d;\n\tmov.b32 {a, b, c, d}, %4;\n\t"
        "cvt.rn.f16x2.e2m1x2 %0, a;\n\tcvt.rn.f16x2.e2m1x2 %1, b;\n\t"
        "cvt.rn.f16x2.e2m1x2 %2, c;\n\tcvt.rn.f16x2.e2m1x2 %3, d;\n\t}\n"
        : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
        : "r"(q));
#pragma unroll
    for (int i = 0; i < 4; ++i) mx_half2(h[i], v + 2 * i);
}

// Largest magnitude of 8 elements as fp32 bits, from their raw form (bf16: two to a
// word, compared as 16-bit integers).
__device__ __forceinline__ uint32_t mx_top(const uint4 &u) {
    const uint32_t m = __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu));
    return max(m << 16, m & 0xffff0000u);
}
struct Raw32 {   // 8 fp32 elements
    uint4 a, b;
};
__device__ __forceinline__ uint32_t mx_top(const Raw32 &u) {
    const uint32_t k = 0x7fffffffu;
    const uint32_t m = max(max(u.a.x & k, u.a.y & k), max(u.a.z & k, u.a.w & k));
    return max(m, max(max(u.b.x & k, u.b.y & k), max(u.b.z & k, u.b.w & k)));
}
__device__ __forceinline__ void raw_values(const uint4 &u, float *v) {
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void raw_values(const Raw32 &u, float *v) {
    v[0] = __uint_as_float(u.a.x), v[1] = __uint_as_float(u.a.y), v[2] = __uint_as_float(u.a.z), v[3] = __uint_as_float(u.a.w);
    v[4] = __uint_as_float(u.b.x), v[5] = __uint_as_float(u.b.y), v[6] = __uint_as_float(u.b.z), v[7] = __uint_as_float(u.b.w);
}
// fp32 values rounded to the raw form
__device__ __forceinline__ void raw_round(const float *v, uint4 &u) {
    u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void raw_round(const float *v, Raw32 &u) {
    u.a = make_uint4(__float_as_uint(v[0]), __float_as_uint(v[1]), __float_as_uint(v[2]), __float_as_uint(v[3]));
    u.b = make_uint4(__float_as_uint(v[4]), __float_as_uint(v[5]), __float_as_uint(v[6]), __float_as_uint(v[7]));
}
template <typename E>
struct RawOf {
    using type = uint4;
};
template <>
struct RawOf<float> {
    using type = Raw32;
};

// A warp works on 256 consecutive columns of a row from c0 (a multiple of 256), 8 per lane.
//   VEC   lane l holds columns c0 + 8 l ..: 16-byte accesses, a scale's block is 4 lanes
//   else  lane l holds columns c0 + 32 i + l: rows that 16-byte accesses do not suit (8 neighbours a lane, one
//         by one, took twice as long in the norm)
template <bool VEC>
__device__ __forceinline__ void load8(const __nv_bfloat16 *row, int c0, int cols, int lane, uint4 &u) {
    if (VEC) {
        u = c0 + 8 * lane < cols ? *reinterpret_cast<const uint4 *>(row + c0 + 8 * lane) : make_uint4(0, 0, 0, 0);
    } else {
        uint32_t w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i)
            w[i] = c0 + 32 * i + lane < cols ? __bfloat16_as_ushort(row[c0 + 32 * i + lane]) : 0u;
        u = make_uint4(w[0] | w[1] << 16, w[2] | w[3] << 16, w[4] | w[5] << 16, w[6] | w[7] << 16);
    }
}
template <bool VEC>
__device__ __forceinline__ void load8(const float *row, int c0, int cols, int lane, Raw32 &u) {
    if (VEC) {
        const uint4 z = make_uint4(0, 0, 0, 0);
        const bool there = c0 + 8 * lane < cols;
        const uint4 *p = reinterpret_cast<const uint4 *>(row + c0 + 8 * lane);
        u.a = there ? p[0] : z;
        u.b = there ? p[1] : z;
    } else {
        float v[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = c0 + 32 * i + lane < cols ? row[c0 + 32 * i + lane] : 0.f;
        raw_round(v, u);
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(__nv_bfloat16 *row, int c0, int cols, int lane, const uint4 &u) {
    if (VEC) {
        if (c0 + 8 * lane < cols) *reinterpret_cast<uint4 *>(row + c0 + 8 * lane) = u;
    } else {
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + 32 * i + lane < cols)
                row[c0 + 32 * i + lane] = __ushort_as_bfloat16((unsigned short)(w[i >> 1] >> (16 * (i & 1))));
    }
}
template <bool VEC>
__device__ __forceinline__ void store8(float *row, int c0, int cols, int lane, const Raw32 &u) {
    if (VEC) {
        if (c0 + 8 * lane < cols) {
            uint4 *p = reinterpret_cast<uint4 *>(row + c0 + 8 * lane);
            p[0] = u.a;
            p[1] = u.b;
        }
    } else {
        float v[8];
        raw_values(u, v);
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c0 + 32 * i + lane < cols) row[c0 + 32 * i + lane] = v[i];
    }
}

// Elements c0 + 32 i + lane of the warp's lanes to c0 + 8 lane + i and back, through
// 256 floats of shared memory of its own.
__device__ __forceinline__ void lanes_to_rows(float *v, float *sm, int lane) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) sm[32 * i + lane] = v[i];
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(v + i) = *reinterpret_cast<const float4 *>(sm + 8 * lane + i);
}
__device__ __forceinline__ void rows_to_lanes(float *v, float *sm, int lane) {
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; i += 4) *reinterpret_cast<float4 *>(sm + 8 * lane + i) = *reinterpret_cast<const float4 *>(v + i);
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = sm[32 * i + lane];
}

// The warp's 256 columns, microscaled, to a stored row q and the scales of its row r; a lane holds
// columns c0 + 8 lane .. (v, fp32, and their largest magnitude's bits m).
// pad: the stored columns; there: the row exists (whole warps take part either way).
template <bool FP4>
__device__ __forceinline__ void mx_emit(unsigned char *q, uint8_t *scales, int64_t r, int c0, int pad, int lane, bool there,
                                        float *v, uint32_t m) {
    m = max(m, __shfl_xor_sync(FULL, m, 1));
    m = max(m, __shfl_xor_sync(FULL, m, 2));
    const uint32_t code = mx_code<FP4>(m);
    const float inv = mx_inverse(code);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] *= inv;
    if (__any_sync(FULL, code == 255u) && code == 255u)   // elements of a NaN block: zeros
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = 0.f;
    uint32_t word = code << (8 * ((lane >> 2) & 3));
    word |= __shfl_xor_sync(FULL, word, 4);
    word |= __shfl_xor_sync(FULL, word, 8);
    const int col = c0 + 8 * lane;
    if (there && col < pad) {
        if (FP4) *reinterpret_cast<uint32_t *>(q + (col >> 1)) = mx_pack_e2m1(v);
        else *reinterpret_cast<uint2 *>(q + col) = mx_pack_e4m3(v);
        if ((lane & 15) == 0) *reinterpret_cast<uint32_t *>(scales + mx_scale_word(r, col >> 7, pad / MX_TILE_COLS)) = word;
    }
}
__device__ __forceinline__ uint32_t mx_top(const float *v) {
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
    return m;
}

// Programmatic dependent launch: a kernel launched by launch_after may be set up while the one before it on
// the stream ends.  pdl_wait: everything before it on the stream has completed and is visible (ahead of any access to
// memory that other kernels use).  pdl_next: the next kernel's blocks may come, once every block of this one has said
// so or ended (they then wait in their own pdl_wait).
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;\n" ::: "memory"); }
__device__ __forceinline__ void pdl_next() { asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory"); }

template <typename... P, typename... A>
int launch_after(void (*kernel)(P...), dim3 grid, unsigned threads, size_t smem, unsigned cluster, cudaStream_t st, A... args) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2] = {};
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<P>(args)...);
    return cuda_rc(e != cudaSuccess ? e : cudaGetLastError());
}

// tmaps.cu: a map over the bytes of a microscaled matrix's q
int tensor_map_mx(CUtensorMap *out, const void *base, uint64_t inner, uint64_t rows, uint64_t pitch,
                  uint32_t box_rows, bool packed4);


// mx_rows.cu: LORA_OK, or what is wrong with a microscaled matrix of at least `rows` rows
int check_mx(const lora_mx *m, int64_t rows);

inline bool mx_aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }
// rows of ld elements of es bytes at p allow 16-byte accesses to 8-column groups of `cols` columns
inline bool mx_vec(const void *p, int64_t ld, int64_t cols, int es) {
    return mx_aligned(p, 16) && (cols & 7) == 0 && (ld * es) % 16 == 0;
}

}  // namespace lora
