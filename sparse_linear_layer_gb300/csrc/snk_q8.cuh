// 8-bit matrices with scales: device helpers shared by the kernels that write
// them (snk_q8.cu, snk_norm.cu) and by the sparse products that read them.
//
// A matrix [rows, cols] is held as one byte per element and one fp32 scale per
// group of consecutive columns of a row (32, 64, 128 or 256 columns; 0: the
// whole row); element (r, c) stands for scale * code.  For a group with
// largest magnitude m and a format whose largest code is Q (127 or 448):
//     scale = m / Q,   code = round_half_even(y * (Q / m)) on the code grid.
// Both quotients are IEEE fp32 divisions, so codes do not depend on the kernel
// that wrote them.  m < 2^-100 gives scale 0 and codes 0 (Q / m would
// overflow); an inf or NaN in the group gives scale NaN and codes 0, so every
// value of the group reads as NaN.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "snk_internal.cuh"

namespace snk {

constexpr int kQTile = 256;               // elements of a row that one warp holds, 8 per lane
constexpr float kQTiny = 7.888609052e-31f;   // 2^-100

// ---- element types -----------------------------------------------------------
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
template <typename T>
__device__ __forceinline__ T from_f32(float x);
template <>
__device__ __forceinline__ float from_f32<float>(float x) { return x; }
template <>
__device__ __forceinline__ __half from_f32<__half>(float x) { return __float2half_rn(x); }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// Two values from / to a packed pair of 16-bit elements (low half first).
template <typename T>
__device__ __forceinline__ float2 unpack2(uint32_t w);
template <>
__device__ __forceinline__ float2 unpack2<__half>(uint32_t w) {
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <>
__device__ __forceinline__ float2 unpack2<__nv_bfloat16>(uint32_t w) {
    return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <typename T>
__device__ __forceinline__ uint32_t pack2(float2 f);
template <>
__device__ __forceinline__ uint32_t pack2<__half>(float2 f) {
    const __half2 h = __floats2half2_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t pack2<__nv_bfloat16>(float2 f) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(f.x, f.y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// Eight fp32 values of a lane, worked on two at a time (one instruction for a
// pair's addition, product or fused product).
struct F8 {
    float2 p[4];
    __device__ __forceinline__ float at(int j) const { return (j & 1) ? p[j >> 1].y : p[j >> 1].x; }
    __device__ __forceinline__ void set(int j, float x) {
        if (j & 1) p[j >> 1].y = x;
        else p[j >> 1].x = x;
    }
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = make_float2(0.f, 0.f);
    }
    __device__ __forceinline__ void add(const F8& o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __fadd2_rn(p[i], o.p[i]);
    }
    __device__ __forceinline__ void mul(const F8& o) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __fmul2_rn(p[i], o.p[i]);
    }
    __device__ __forceinline__ void mul(float x) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __fmul2_rn(p[i], make_float2(x, x));
    }
    // this += a * b
    __device__ __forceinline__ void fma(const F8& a, const F8& b) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = __ffma2_rn(a.p[i], b.p[i], p[i]);
    }
    // rounded to T and back
    template <typename T>
    __device__ __forceinline__ void round() {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
            for (int i = 0; i < 4; ++i) p[i] = unpack2<T>(pack2<T>(p[i]));
        }
    }
};

// Eight consecutive elements; p is 32-byte aligned for fp32 (one 256-bit
// access) and 16-byte aligned for the 16-bit types (one 128-bit access).
__device__ __forceinline__ void load8(const float* q, F8& v) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v.p[0].x), "=f"(v.p[0].y), "=f"(v.p[1].x), "=f"(v.p[1].y), "=f"(v.p[2].x), "=f"(v.p[2].y),
                   "=f"(v.p[3].x), "=f"(v.p[3].y)
                 : "l"(q)
                 : "memory");
}
__device__ __forceinline__ void store8(float* q, const F8& v) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(q), "f"(v.p[0].x), "f"(v.p[0].y),
                 "f"(v.p[1].x), "f"(v.p[1].y), "f"(v.p[2].x), "f"(v.p[2].y), "f"(v.p[3].x), "f"(v.p[3].y)
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void unpack8(const uint4& w, F8& v) {
    v.p[0] = unpack2<T>(w.x);
    v.p[1] = unpack2<T>(w.y);
    v.p[2] = unpack2<T>(w.z);
    v.p[3] = unpack2<T>(w.w);
}
template <typename T>
__device__ __forceinline__ void load8(const T* q, F8& v) {
    static_assert(sizeof(T) == 2, "16-bit element");
    unpack8<T>(*reinterpret_cast<const uint4*>(q), v);
}
template <typename T>
__device__ __forceinline__ void store8(T* q, const F8& v) {
    static_assert(sizeof(T) == 2, "16-bit element");
    *reinterpret_cast<uint4*>(q) = make_uint4(pack2<T>(v.p[0]), pack2<T>(v.p[1]), pack2<T>(v.p[2]), pack2<T>(v.p[3]));
}

// ---- tiles -------------------------------------------------------------------
// A warp's tile is kQTile consecutive columns of a row.  VEC (cols a multiple of
// 8, aligned rows): lane l holds columns 8 l .. 8 l + 7 of the tile; else columns
// 32 j + l, so that every access of the warp is contiguous at any alignment.
// Pointers are to the lane's first element; `left` is how many of the tile's
// columns lie in the row (0 or less: none).  Columns past the row's end read as
// zero and are not written.
template <bool VEC>
__device__ __forceinline__ int lane_col(int lane) { return VEC ? 8 * lane : lane; }
template <typename T, bool VEC>
__device__ __forceinline__ void load_tile(const T* p, int left, int lane, F8& v) {
    if constexpr (VEC) {
        if (left < kQTile) v.clear();
        if (8 * lane < left) load8(p, v);
    } else if (left >= kQTile) {   // a whole tile: no tests
#pragma unroll
        for (int j = 0; j < 8; ++j) v.set(j, to_f32(p[32 * j]));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) v.set(j, 32 * j + lane < left ? to_f32(p[32 * j]) : 0.f);
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_tile(T* p, int left, int lane, const F8& v) {
    if constexpr (VEC) {
        if (8 * lane < left) store8(p, v);
    } else if (left >= kQTile) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[32 * j] = from_f32<T>(v.at(j));
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (32 * j + lane < left) p[32 * j] = from_f32<T>(v.at(j));
    }
}
// x + residual rounded to T, as fp32, of a lane's 8 elements.  16-bit types add
// in pairs; the sum of two such values has one rounding either way (where their
// exponents are so far apart that fp32 would round, too, the larger is the sum).
template <typename T>
__device__ __forceinline__ uint32_t add2(uint32_t a, uint32_t b);
template <>
__device__ __forceinline__ uint32_t add2<__half>(uint32_t a, uint32_t b) {
    const __half2 h = __hadd2(*reinterpret_cast<const __half2*>(&a), *reinterpret_cast<const __half2*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}
template <>
__device__ __forceinline__ uint32_t add2<__nv_bfloat16>(uint32_t a, uint32_t b) {
    const __nv_bfloat162 h =
        __hadd2(*reinterpret_cast<const __nv_bfloat162*>(&a), *reinterpret_cast<const __nv_bfloat162*>(&b));
    return *reinterpret_cast<const uint32_t*>(&h);
}

// ---- quantisation ------------------------------------------------------------
struct QScale {
    float scale, inv;
};
// scale = m / top and inv = top / m, both rounded to nearest: a quotient q = a y
// from the reciprocal y, corrected once by its remainder, fma(fma(-b, q, a), y, q)
// (Markstein, "Computation of elementary functions on the IBM RISC System/6000
// processor", 1990); y of the constant is exact to half a unit, that of m / 4 (so
// that it is a normal number for every finite m) is the approximate reciprocal
// with one Newton step.  Equal to IEEE division for every m from 2^-100 on, and
// without its branches, which cost GELU's training batch 5 of 60 us.
__device__ __forceinline__ QScale q_scale(float m, int format) {
    const float top = format == SNK_Q8_INT8 ? 127.f : 448.f;
    const float yt = format == SNK_Q8_INT8 ? 1.f / 127.f : 1.f / 448.f;
    float s = m * yt;
    s = fmaf(fmaf(-top, s, m), yt, s);
    const float m4 = 0.25f * m, top4 = 0.25f * top;
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(m4));
    y = fmaf(fmaf(-m4, y, 1.f), y, y);
    float i = top4 * y;
    i = fmaf(fmaf(-m4, i, top4), y, i);
    const bool big = !(m <= 3.4028235e38f);   // inf or NaN
    const bool ok = m >= kQTiny && !big;
    return QScale{ok ? s : (big ? __int_as_float(0x7fc00000) : 0.f), ok ? i : 0.f};
}
// max(m, |a|, |b|), NaN if any is.
__device__ __forceinline__ float max_abs(float m, float a, float b) {
    float r;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(m), "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float amax8(const F8& v, float m = 0.f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) m = max_abs(m, v.p[i].x, v.p[i].y);
    return m;
}
// Over the warp, of non-negative values (NaN's bits are above infinity's).
__device__ __forceinline__ float warp_amax(float m) {
    return __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m) & 0x7fffffffu));
}

// Codes of four scaled values, the first in the lowest byte.
// int8: adding 1.5 * 2^23 rounds to the nearest integer, half to even, and
// leaves its two's complement in the low byte (|v| <= 127 (1 + 2^-22)).
__device__ __forceinline__ uint32_t q_codes4(float2 a, float2 b, int format) {
    uint32_t r;
    if (format == SNK_Q8_INT8) {
        const float2 half = make_float2(12582912.f, 12582912.f);
        const float2 x = __fadd2_rn(a, half), y = __fadd2_rn(b, half);
        r = __byte_perm(__byte_perm(__float_as_uint(x.x), __float_as_uint(x.y), 0x0040),
                        __byte_perm(__float_as_uint(y.x), __float_as_uint(y.y), 0x0040), 0x5410);
    } else {
        asm("{ .reg .b16 lo, hi;\n cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n"
            " mov.b32 %0, {lo, hi}; }"
            : "=r"(r)
            : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
    }
    return r;
}
__device__ __forceinline__ uint8_t q_code(float v, int format) {
    if (format == SNK_Q8_INT8) return (uint8_t)__float_as_uint(__fadd_rn(v, 12582912.f));
    return __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
}
// Codes of a lane's 8 values 32 columns apart, scaled by inv[j] (0: code 0).
__device__ __forceinline__ void store_codes32(uint8_t* p, int left, int lane, const F8& v, const float (&inv)[8],
                                              int format) {
    uint8_t c[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        // (the product is rounded before q_code's addition: not one fused product)
        c[j] = q_code(__fmul_rn(v.at(j), inv[j]), format);
        if (inv[j] == 0.f) c[j] = 0;
    }
    if (left >= kQTile) {
#pragma unroll
        for (int j = 0; j < 8; ++j) p[32 * j] = c[j];
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
            if (32 * j + lane < left) p[32 * j] = c[j];
    }
}
__device__ __forceinline__ float q_value(uint8_t code, int format) {
    if (format == SNK_Q8_INT8) return __uint_as_float(0x4B000000u | (code ^ 0x80u)) - 8388736.f;
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}
// The values of four codes (first in the lowest byte).  int8: the code plus
// 128 as the low byte of 2^23's mantissa, minus (2^23 + 128): exact.
__device__ __forceinline__ void q_values4(uint32_t w, int format, float2& a, float2& b) {
    if (format == SNK_Q8_INT8) {
        w ^= 0x80808080u;
        const float2 off = make_float2(-8388736.f, -8388736.f);
        a = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540)),
                                   __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541))), off);
        b = __fadd2_rn(make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7542)),
                                   __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7543))), off);
    } else {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        a = __half22float2(__half2(lo));
        b = __half22float2(__half2(hi));
    }
}

// Where a matrix's codes and scales go.
struct Q8Out {
    uint8_t* codes;    // [rows, cols]
    float* scales;     // [rows, n_groups]
    int format;
    int gshift;        // log2(group); 31: one group per row
    int64_t n_groups;
};
__device__ __forceinline__ float q_at(const Q8In& q, int64_t r, int64_t c) {
    return q_value(__ldg(q.codes + r * q.cols + c), q.format) * __ldg(q.scales + r * q.n_groups + (c >> q.gshift));
}
__device__ __forceinline__ float SrcQ8::at(int64_t r, int64_t c) const { return q_at(q, r, c); }

// Write the codes of a lane's 8 columns under one scale (VEC).  inv = 0 (a
// group held as zeros, or with an inf or NaN) gives codes 0.
__device__ __forceinline__ void store_codes(uint8_t* p, F8 v, float inv, int format) {
    v.mul(inv);
    uint2 w = make_uint2(q_codes4(v.p[0], v.p[1], format), q_codes4(v.p[2], v.p[3], format));
    if (inv == 0.f) w = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(p) = w;
}

// Quantise a tile whose groups lie inside it (gshift 5..8): codes at the lane's
// position, scales from the tile's first one on.
template <bool VEC>
__device__ __forceinline__ void pack_tile_groups(int format, int gshift, uint8_t* codes, float* scales, int left,
                                                 int lane, const F8& v) {
    if constexpr (VEC) {
        float m = amax8(v);
        // lanes of a group: 4, 8, 16 or 32
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 2));
        if (gshift > 5) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 4));
        if (gshift > 6) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 8));
        if (gshift > 7) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, 16));
        const QScale s = q_scale(m, format);
        if (8 * lane < left) {
            if (((8 * lane) & ((1 << gshift) - 1)) == 0) scales[(8 * lane) >> gshift] = s.scale;
            store_codes(codes, v, s.inv, format);
        }
    } else {
        float m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = warp_amax(v.at(j));
#pragma unroll
        for (int b = 0; b < 3; ++b) {
            if (gshift > 5 + b) {
                float u[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) u[j] = max_nan(m[j], m[j ^ (1 << b)]);
#pragma unroll
                for (int j = 0; j < 8; ++j) m[j] = u[j];
            }
        }
        // lanes 4 j .. 4 j + 3 work out the scale of the j-th 32 columns
        float mine = m[0];
#pragma unroll
        for (int j = 1; j < 8; ++j) mine = (lane >> 2) == j ? m[j] : mine;
        const QScale s = q_scale(mine, format);
        const int c = 32 * (lane >> 2);
        if ((lane & 3) == 0 && (c & ((1 << gshift) - 1)) == 0 && c < left) scales[c >> gshift] = s.scale;
        float inv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) inv[j] = __shfl_sync(0xffffffffu, s.inv, 4 * j);
        store_codes32(codes, left, lane, v, inv, format);
    }
}
// Quantise a tile under its row's scale.
template <bool VEC>
__device__ __forceinline__ void pack_tile_row(int format, uint8_t* codes, int left, int lane, const F8& v, float inv) {
    if constexpr (VEC) {
        if (8 * lane < left) store_codes(codes, v, inv, format);
    } else {
        const float each[8] = {inv, inv, inv, inv, inv, inv, inv, inv};
        store_codes32(codes, left, lane, v, each, format);
    }
}
// The values of a tile; scales points to its first one (gshift 31: the row's).
template <bool VEC>
__device__ __forceinline__ void load_values(int format, int gshift, const uint8_t* codes, const float* scales,
                                            int left, int lane, F8& v) {
    if constexpr (VEC) {
        if (left < kQTile) v.clear();
        if (8 * lane < left) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(codes));
            const float s = __ldg(scales + ((8 * lane) >> gshift));
            q_values4(w.x, format, v.p[0], v.p[1]);
            q_values4(w.y, format, v.p[2], v.p[3]);
            v.mul(s);
        }
    } else {
        // lane j < 8 holds the scale of the j-th 32 columns
        const float mine = lane < 8 && 32 * lane < left ? __ldg(scales + ((32 * lane) >> gshift)) : 0.f;
        uint8_t c[8];
        if (left >= kQTile) {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = __ldg(codes + 32 * j);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) c[j] = 32 * j + lane < left ? __ldg(codes + 32 * j) : (uint8_t)0;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) v.set(j, q_value(c[j], format) * __shfl_sync(0xffffffffu, mine, j));
    }
}

// ---- rows over several warps ---------------------------------------------------
// ONE: every warp of a block has a row of its own; else the block's W warps share
// one row and meet on the block's barrier.  (Several rows of several warps in one
// block would need named barriers chosen at run time: the compiler then reserves
// all 16 of a block, and an SM, which has 64, holds 4 blocks.)
constexpr int kRowsPerBlock = 8;   // ONE
template <bool ONE>
struct RowSlot {
    int W, slots, slot, w, lane;
    __device__ __forceinline__ RowSlot() {
        const int warp = threadIdx.x >> 5, warps = blockDim.x >> 5;
        W = ONE ? 1 : warps;
        slots = ONE ? warps : 1;
        slot = ONE ? warp : 0;
        w = ONE ? 0 : warp;
        lane = threadIdx.x & 31;
    }
    __device__ __forceinline__ int64_t first_row() const { return (int64_t)blockIdx.x * slots + slot; }
    // Sum over the row, the same in every thread: lanes by a shuffle tree,
    // warps in order.  `red` holds 32 floats; two calls on the same `red` need
    // another barrier between them.
    __device__ __forceinline__ float sum(float x, float* red) const {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if constexpr (!ONE) {
            if (lane == 0) red[w] = x;
            __syncthreads();
            x = 0.f;
            for (int i = 0; i < W; ++i) x += red[i];
        }
        return x;
    }
    // Largest of non-negative values over the row, NaN if any is.
    __device__ __forceinline__ float max_of(float m, float* red) const {
        m = warp_amax(m);
        if constexpr (!ONE) {
            if (lane == 0) red[w] = m;
            __syncthreads();
            m = 0.f;
            for (int i = 0; i < W; ++i) m = max_nan(m, red[i]);
        }
        return m;
    }
};

// Warps per row W and tiles per warp K for rows of `tiles` tiles: up to `one`
// tiles (at most 4) one warp holds the row; else a warp holds one tile, or two of
// rows of more than 32.
struct RowShape {
    int W, K;
    bool one() const { return W == 1; }
    int slots() const { return W == 1 ? kRowsPerBlock : 1; }
    int threads() const { return 32 * W * slots(); }
};
inline RowShape row_shape(int64_t tiles, int one) {
    if (tiles <= one) return RowShape{1, (int)tiles};
    const int K = tiles <= 32 ? 1 : 2;
    return RowShape{(int)ceil_div(tiles, K), K};
}
constexpr int64_t kRegisterTiles = 64;   // longer rows are read again for each step

// ---- rows in flight -------------------------------------------------------------
// A block that walks many rows copies the tiles of its next row into shared
// memory while it works on this one (cp.async).  Every thread copies what it will
// read itself, so no barrier is needed, only the thread's own wait.  Unit u (16
// bytes) of a stage lies at (u * blockDim + thread) * 16.
template <typename T>
struct Ring {
    static constexpr int kUnits = (int)sizeof(T) / 2;   // 16-byte units of a lane's 8 elements
    // (.ca: the two halves of a lane's 32 bytes of fp32 are two copies of the
    // same sector, the second of which hits L1)
    static __device__ __forceinline__ void copy(uint4* stage, int unit, const T* p, int left, int lane) {
        const int n = 8 * lane < left ? 16 : 0;
        const char* src = reinterpret_cast<const char*>(n ? p : p - 8 * lane);   // read only when n > 0
#pragma unroll
        for (int h = 0; h < kUnits; ++h)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(
                             stage + (unit * kUnits + h) * blockDim.x + threadIdx.x)),
                         "l"(src + 16 * h), "r"(n)
                         : "memory");
    }
    static __device__ __forceinline__ void read(const uint4* stage, int unit, F8& v) {
        if constexpr (sizeof(T) == 4) {
            const uint4 a = stage[(2 * unit) * blockDim.x + threadIdx.x];
            const uint4 b = stage[(2 * unit + 1) * blockDim.x + threadIdx.x];
            v.p[0] = make_float2(__uint_as_float(a.x), __uint_as_float(a.y));
            v.p[1] = make_float2(__uint_as_float(a.z), __uint_as_float(a.w));
            v.p[2] = make_float2(__uint_as_float(b.x), __uint_as_float(b.y));
            v.p[3] = make_float2(__uint_as_float(b.z), __uint_as_float(b.w));
        } else {
            unpack8<T>(stage[unit * blockDim.x + threadIdx.x], v);
        }
    }
    // the sum of two units, rounded to T
    static __device__ __forceinline__ void read_sum(const uint4* stage, int unit, int other, F8& v) {
        if constexpr (sizeof(T) == 4) {
            F8 t;
            read(stage, unit, v);
            read(stage, other, t);
            v.add(t);
        } else {
            const uint4 a = stage[unit * blockDim.x + threadIdx.x], b = stage[other * blockDim.x + threadIdx.x];
            unpack8<T>(make_uint4(add2<T>(a.x, b.x), add2<T>(a.y, b.y), add2<T>(a.z, b.z), add2<T>(a.w, b.w)), v);
        }
    }
};
__device__ __forceinline__ void ring_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void ring_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// ---- host side -----------------------------------------------------------------
inline bool q8_group_ok(int group) { return group == 0 || group == 32 || group == 64 || group == 128 || group == 256; }
inline int q8_gshift(int group) { return group == 0 ? 31 : group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : 8; }
inline int64_t q8_groups(int64_t cols, int group) { return group == 0 ? 1 : ceil_div(cols, group); }
inline bool q8_aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t elt_size(int dtype) { return dtype == SNK_F32 ? 4 : 2; }

}  // namespace snk
