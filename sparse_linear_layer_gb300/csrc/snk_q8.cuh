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

// Eight consecutive elements; p is 32-byte aligned for fp32 (one 256-bit
// access) and 16-byte aligned for the 16-bit types (one 128-bit access).
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    asm volatile("ld.global.v8.f32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7])
                 : "l"(p)
                 : "memory");
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
    asm volatile("st.global.v8.f32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "f"(v[0]), "f"(v[1]), "f"(v[2]),
                 "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
}
template <typename T>
__device__ __forceinline__ void load8(const T* p, float (&v)[8]) {
    static_assert(sizeof(T) == 2, "16-bit element");
    uint4 w;
    asm volatile("ld.global.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "l"(p) : "memory");
    const T* h = reinterpret_cast<const T*>(&w);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = to_f32(h[j]);
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float (&v)[8]) {
    static_assert(sizeof(T) == 2, "16-bit element");
    uint4 w;
    T* h = reinterpret_cast<T*>(&w);
#pragma unroll
    for (int j = 0; j < 8; ++j) h[j] = from_f32<T>(v[j]);
    *reinterpret_cast<uint4*>(p) = w;
}

// ---- tiles -------------------------------------------------------------------
// A warp's tile is kQTile consecutive columns from c0.  VEC (cols a multiple
// of 8 and aligned rows): lane l holds columns c0 + 8 l .. + 7; else columns
// c0 + 32 j + l, so that every access of the warp is contiguous at any
// alignment.  Columns past the row's end read as zero and are not written.
template <bool VEC>
__device__ __forceinline__ int64_t tile_col(int64_t c0, int lane, int j) {
    return VEC ? c0 + 8 * lane + j : c0 + 32 * j + lane;
}
template <typename T, bool VEC>
__device__ __forceinline__ void load_tile(const T* row, int64_t c0, int64_t cols, int lane, float (&v)[8]) {
    if constexpr (VEC) {
        if (c0 + 8 * lane < cols) {
            load8(row + c0 + 8 * lane, v);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 32 * j + lane;
            v[j] = c < cols ? to_f32(row[c]) : 0.f;
        }
    }
}
template <typename T, bool VEC>
__device__ __forceinline__ void store_tile(T* row, int64_t c0, int64_t cols, int lane, const float (&v)[8]) {
    if constexpr (VEC) {
        if (c0 + 8 * lane < cols) store8(row + c0 + 8 * lane, v);
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 32 * j + lane;
            if (c < cols) row[c] = from_f32<T>(v[j]);
        }
    }
}

// ---- quantisation ------------------------------------------------------------
struct QScale {
    float scale, inv;
};
// From the bit pattern of the group's largest magnitude (NaN's is above
// infinity's, so it also marks a group that holds one).
__device__ __forceinline__ QScale q_scale(uint32_t amax_bits, float top) {
    const float m = __uint_as_float(amax_bits);
    if (amax_bits >= 0x7f800000u) return QScale{__int_as_float(0x7fc00000), 0.f};
    if (m < kQTiny) return QScale{0.f, 0.f};
    return QScale{__fdiv_rn(m, top), __fdiv_rn(top, m)};
}
__device__ __forceinline__ float q_top(int format) { return format == SNK_Q8_INT8 ? 127.f : 448.f; }

// Codes of four values scaled by inv, the first in the lowest byte.
// int8: adding 1.5 * 2^23 rounds to the nearest integer, half to even, and
// leaves its two's complement in the low byte (|v| <= 127 (1 + 2^-22)).
__device__ __forceinline__ uint32_t q_codes4(float a, float b, float c, float d, float inv, int format) {
    if (inv == 0.f) return 0u;
    if (format == SNK_Q8_INT8) {
        constexpr float kRound = 12582912.f;
        const uint32_t x = __float_as_uint(__fadd_rn(__fmul_rn(a, inv), kRound));
        const uint32_t y = __float_as_uint(__fadd_rn(__fmul_rn(b, inv), kRound));
        const uint32_t z = __float_as_uint(__fadd_rn(__fmul_rn(c, inv), kRound));
        const uint32_t w = __float_as_uint(__fadd_rn(__fmul_rn(d, inv), kRound));
        return __byte_perm(__byte_perm(x, y, 0x0040), __byte_perm(z, w, 0x0040), 0x5410);
    }
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a * inv, b * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c * inv, d * inv), __NV_SATFINITE, __NV_E4M3);
    return lo | (hi << 16);
}
__device__ __forceinline__ float q_value(uint8_t code, int format) {
    if (format == SNK_Q8_INT8) return (float)(int8_t)code;
    return __half2float(__half(__nv_cvt_fp8_to_halfraw(code, __NV_E4M3)));
}
// The values of four codes (first in the lowest byte).  int8: the code plus
// 128 as the low byte of 2^23's mantissa, minus (2^23 + 128): exact.
__device__ __forceinline__ void q_values4(uint32_t w, int format, float* v) {
    if (format == SNK_Q8_INT8) {
        w ^= 0x80808080u;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + j)) - 8388736.f;
    } else {
        const __half2_raw lo = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w & 0xffffu), __NV_E4M3);
        const __half2_raw hi = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> 16), __NV_E4M3);
        const float2 a = __half22float2(__half2(lo)), b = __half22float2(__half2(hi));
        v[0] = a.x;
        v[1] = a.y;
        v[2] = b.x;
        v[3] = b.y;
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

// Write a tile's codes under one scale.
template <bool VEC>
__device__ __forceinline__ void store_codes(uint8_t* row, int64_t c0, int64_t cols, int lane, const float (&v)[8],
                                            const float (&inv)[VEC ? 1 : 8], int format) {
    if constexpr (VEC) {
        if (c0 + 8 * lane < cols) {
            uint2 w;
            w.x = q_codes4(v[0], v[1], v[2], v[3], inv[0], format);
            w.y = q_codes4(v[4], v[5], v[6], v[7], inv[0], format);
            *reinterpret_cast<uint2*>(row + c0 + 8 * lane) = w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 32 * j + lane;
            if (c < cols) row[c] = (uint8_t)q_codes4(v[j], 0.f, 0.f, 0.f, inv[j], format);
        }
    }
}

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }
// The largest magnitude of a tile over the whole warp, as bits.
__device__ __forceinline__ uint32_t tile_amax(const float (&v)[8]) {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
    return __reduce_max_sync(0xffffffffu, m);
}

// Quantise a tile whose groups lie inside it (gshift 5..8) and write codes and
// scales of matrix row `r`.
template <bool VEC>
__device__ __forceinline__ void pack_tile_groups(const Q8Out& q, int64_t r, int64_t c0, int64_t cols, int lane,
                                                 const float (&v)[8]) {
    const float top = q_top(q.format);
    float* srow = q.scales + r * q.n_groups;
    if constexpr (VEC) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[j]));
        const int lanes = 1 << (q.gshift - 3);   // lanes of a group
        for (int o = 1; o < lanes; o <<= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        const QScale s = q_scale(m, top);
        const int64_t c = c0 + 8 * lane;
        if ((lane & (lanes - 1)) == 0 && c < cols) srow[c >> q.gshift] = s.scale;
        const float inv[1] = {s.inv};
        store_codes<VEC>(q.codes + r * cols, c0, cols, lane, v, inv, q.format);
    } else {
        uint32_t m[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) m[j] = __reduce_max_sync(0xffffffffu, abs_bits(v[j]));
#pragma unroll
        for (int b = 0; b < 3; ++b) {
            if (q.gshift > 5 + b) {
                uint32_t t[8];
#pragma unroll
                for (int j = 0; j < 8; ++j) t[j] = max(m[j], m[j ^ (1 << b)]);
#pragma unroll
                for (int j = 0; j < 8; ++j) m[j] = t[j];
            }
        }
        float inv[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const QScale s = q_scale(m[j], top);
            inv[j] = s.inv;
            const int64_t c = c0 + 32 * j;
            if (lane == 0 && (c & ((1 << q.gshift) - 1)) == 0 && c < cols) srow[c >> q.gshift] = s.scale;
        }
        store_codes<VEC>(q.codes + r * cols, c0, cols, lane, v, inv, q.format);
    }
}
// Quantise a tile under its row's scale.
template <bool VEC>
__device__ __forceinline__ void pack_tile_row(const Q8Out& q, int64_t r, int64_t c0, int64_t cols, int lane,
                                              const float (&v)[8], float inv_row) {
    float inv[VEC ? 1 : 8];
#pragma unroll
    for (int j = 0; j < (VEC ? 1 : 8); ++j) inv[j] = inv_row;
    store_codes<VEC>(q.codes + r * cols, c0, cols, lane, v, inv, q.format);
}
// The values of a tile.
template <bool VEC>
__device__ __forceinline__ void load_values(const Q8In& q, int64_t r, int64_t c0, int lane, float (&v)[8]) {
    const uint8_t* row = q.codes + r * q.cols;
    const float* srow = q.scales + r * q.n_groups;
    if constexpr (VEC) {
        const int64_t c = c0 + 8 * lane;
        if (c < q.cols) {
            const uint2 w = __ldg(reinterpret_cast<const uint2*>(row + c));
            const float s = __ldg(srow + (c >> q.gshift));
            q_values4(w.x, q.format, v);
            q_values4(w.y, q.format, v + 4);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] *= s;
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.f;
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int64_t c = c0 + 32 * j + lane;
            v[j] = c < q.cols ? q_value(__ldg(row + c), q.format) * __ldg(srow + (c >> q.gshift)) : 0.f;
        }
    }
}

// ---- rows over several warps ---------------------------------------------------
// A block holds `slots` rows at a time, W warps each; the warps of a slot meet
// on a named barrier of their own (1 + slot), so slots never wait for one another.
struct RowSlot {
    int W, slot, w, lane;
    __device__ __forceinline__ explicit RowSlot(int warps_per_row) : W(warps_per_row) {
        const int warp = threadIdx.x >> 5;
        slot = warp / W;
        w = warp - slot * W;
        lane = threadIdx.x & 31;
    }
    __device__ __forceinline__ void sync() const {
        if (W > 1) asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(W * 32) : "memory");
        else __syncwarp();
    }
    // Sum over the row, the same in every thread: lanes by a shuffle tree,
    // warps in order.  `red` holds 32 floats per slot; two calls on the same
    // `red` need another sync between them.
    __device__ __forceinline__ float sum(float x, float* red) const {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        if (W == 1) return x;
        if (lane == 0) red[slot * 32 + w] = x;
        sync();
        x = 0.f;
        for (int i = 0; i < W; ++i) x += red[slot * 32 + i];
        return x;
    }
    // Largest value over the row (already equal within the warp).
    __device__ __forceinline__ uint32_t max_of(uint32_t m, uint32_t* red) const {
        if (W == 1) return m;
        if (lane == 0) red[slot * 32 + w] = m;
        sync();
        m = 0;
        for (int i = 0; i < W; ++i) m = max(m, red[slot * 32 + i]);
        return m;
    }
};
constexpr int kMaxSlots = 8;

// ---- host side -----------------------------------------------------------------
inline bool q8_group_ok(int group) { return group == 0 || group == 32 || group == 64 || group == 128 || group == 256; }
inline int q8_gshift(int group) { return group == 0 ? 31 : group == 32 ? 5 : group == 64 ? 6 : group == 128 ? 7 : 8; }
inline int64_t q8_groups(int64_t cols, int group) { return group == 0 ? 1 : ceil_div(cols, group); }
inline bool q8_aligned(const void* p, uintptr_t a) { return ((uintptr_t)p & (a - 1)) == 0; }
inline size_t elt_size(int dtype) { return dtype == SNK_F32 ? 4 : 2; }

}  // namespace snk
