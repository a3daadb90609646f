// 8-bit activation checkpoints: pack (with or without GELU), unpack, and
// GELU's gradient from a packed input.
//
//     pack        codes, scales of y = x  or  y = gelu(x)   (and of x itself)
//     unpack      x = scale * code
//     GELU grad   dh = da * (Phi(h) + h phi(h)),  h = scale * code
//
// Every element is read and written once, so the memory system bounds them.
// A warp holds 256 consecutive elements of a row (8 per lane): a group of
// 32..256 columns never leaves its warp, and its largest magnitude is a few
// shuffles.  A scale for the whole row needs the row's largest magnitude
// before the first code: the row then stays in registers over W warps
// (k_pack_row), up to 16384 columns; longer rows are read twice (k_pack_long).
//
// Measured, 16384 x 3072 fp32 in groups of 128: GELU with its checkpoint, E4M3, 51 us
// (6.0 TB/s; issue slots 80% busy: two quantisations and GELU per element); GELU's
// gradient from int8 codes 67 us (6.8 TB/s, the rate of a copy).  4096 x 10000 fp32 to
// int8 and back 65 us (6.3 TB/s).
#include <algorithm>

#include "snk_q8.cuh"

namespace snk {
namespace {

// Phi(-|x|) and exp(-x^2 / 2) of two values, from nax = -|x|.  The form of
// Abramowitz and Stegun, Handbook of Mathematical Functions, 7.1.26: erfc(z) =
// (c1 t + ... + cn t^n) exp(-z^2), t = 1 / (1 + p z), z >= 0; here with n = 6, p =
// 0.39 and coefficients fitted to 8.3e-9 (weighted least squares, iterated towards
// equal errors; the five printed terms are off by 1.5e-7 in exact arithmetic).  z =
// |x| / sqrt(2), the c_i are halved, and the exponential also serves the gradient.
// Evaluated in fp32 the tail is within 2.0e-7, worst near x = 0 (3 units of its last
// place there); over normal inputs GELU's relative error is 3.3e-8 and its slope's
// 6.1e-8 (root mean squares; 4.0e-8 with erff and expf).  With those the arithmetic,
// not the bytes, set GELU's time: the gradient at 16384 x 3072 took 128 us for 67.
__device__ __forceinline__ float2 both(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 neg_abs(float2 x) {
    return make_float2(__uint_as_float(__float_as_uint(x.x) | 0x80000000u),
                       __uint_as_float(__float_as_uint(x.y) | 0x80000000u));
}
__device__ __forceinline__ float2 normal_tail(float2 nax, float2& e) {
    const float2 d = __ffma2_rn(nax, both(-0.39f * 0.70710678f), both(1.f));
    const float2 z = __fmul2_rn(__fmul2_rn(nax, nax), both(-0.72134752f));   // -x^2 / 2 in powers of 2
    float2 t;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.x) : "f"(d.x));
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(t.y) : "f"(d.y));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(z.x));
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(z.y));
    float2 p = __ffma2_rn(t, both(0.5f * -0.2275369323f), both(0.5f * 0.8866635814f));
    p = __ffma2_rn(t, p, both(0.5f * -0.6353989968f));
    p = __ffma2_rn(t, p, both(0.5f * 0.6495583633f));
    p = __ffma2_rn(t, p, both(0.5f * 0.09138882993f));
    p = __ffma2_rn(t, p, both(0.5f * 0.2353251529f));
    return __fmul2_rn(__fmul2_rn(p, t), e);
}
// x Phi(x) = max(x, 0) - |x| Phi(-|x|)
__device__ __forceinline__ void gelu(F8& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = v.p[i], nax = neg_abs(x);
        float2 e;
        const float2 q = normal_tail(nax, e);
        v.p[i] = __ffma2_rn(nax, q, make_float2(fmaxf(x.x, 0.f), fmaxf(x.y, 0.f)));
    }
}
// Phi(x) + x phi(x)
__device__ __forceinline__ void gelu_slope(F8& v) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 x = v.p[i];
        float2 e;
        const float2 q = normal_tail(neg_abs(x), e);
        const float2 phi = make_float2(x.x >= 0.f ? 1.f - q.x : q.x, x.y >= 0.f ? 1.f - q.y : q.y);
        v.p[i] = __ffma2_rn(__fmul2_rn(x, both(0.39894228f)), e, phi);
    }
}

struct PackArgs {
    const void* x;
    int64_t rows, cols;
    int act;       // 1: gelu(x) is packed
    Q8Out out;     // what is packed
    Q8Out keep;    // x itself (codes null: not kept)
};

// A warp's tile of a flat grid over matrices of `tpr` tiles per row: its row, its
// first column, and the columns of it that lie in the row.  Few tiles per warp:
// the registers of more cost more warps than their loads in flight gain (GELU's
// gradient at 16384 x 3072 takes 70 us with 1, 79 with 2, 115 with 4).
struct FlatTile {
    int64_t e0;    // the tile's first element
    int64_t s0;    // its first scale
    int left;
};
// ROWS false: the matrix is one row (its rows are whole groups).
// (U tiles side by side count as one.)
template <bool ROWS, int U = 1>
__device__ __forceinline__ FlatTile flat_tile(uint32_t i, uint32_t tpr, int64_t cols, int64_t n_groups, int gshift) {
    constexpr int W = U * kQTile;
    if constexpr (!ROWS) {
        const int64_t e0 = (int64_t)i * W, left = cols - e0;
        return FlatTile{e0, gshift == 31 ? 0 : ((int64_t)i * U) << (8 - gshift), (int)min((int64_t)W, left)};
    }
    const uint32_t r = i / tpr, c0 = (i - r * tpr) * W;
    return FlatTile{(int64_t)r * cols + c0, (int64_t)r * n_groups + (c0 >> gshift), min(W, (int)cols - (int)c0)};
}

// Groups of 32..256 columns: tiles are independent of one another.
// Two tiles side by side per warp share their addresses (GELU's training batch 58 ->
// 51 us; a third is no gain).
template <typename T, bool VEC, bool ROWS, int U>
__global__ void __launch_bounds__(256) k_pack_groups(const PackArgs a, uint32_t tiles, uint32_t tpr) {
    const uint32_t i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= tiles) return;
    const int lane = threadIdx.x & 31;
    const FlatTile t = flat_tile<ROWS, U>(i, tpr, a.cols, a.out.n_groups, a.out.gshift);
    const int64_t e = t.e0 + lane_col<VEC>(lane);
    F8 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
        load_tile<T, VEC>((const T*)a.x + e + u * kQTile, t.left - u * kQTile, lane, v[u]);
    const int gs = a.out.gshift;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int left = t.left - u * kQTile;
        const int64_t sc = t.s0 + (u << (8 - gs));
        if (a.keep.codes)
            pack_tile_groups<VEC>(a.keep.format, gs, a.keep.codes + e + u * kQTile, a.keep.scales + sc, left, lane, v[u]);
        if (a.act) gelu(v[u]);
        pack_tile_groups<VEC>(a.out.format, gs, a.out.codes + e + u * kQTile, a.out.scales + sc, left, lane, v[u]);
    }
}

// One scale per row: the row in the registers of W warps, K tiles each.
template <typename T, bool VEC, int K, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kRowsPerBlock : 1024) k_pack_row(const PackArgs a) {
    __shared__ float red[2][32];
    const RowSlot<ONE> rs;
    const int64_t r = rs.first_row();
    if (r >= a.rows) return;
    const int c0 = rs.w * K * kQTile;
    const int64_t e = r * a.cols + c0 + lane_col<VEC>(rs.lane);
    const int left = (int)a.cols - c0;
    F8 v[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        load_tile<T, VEC>((const T*)a.x + e + k * kQTile, left - k * kQTile, rs.lane, v[k]);
    auto pack = [&](const Q8Out& q, float* rd) {
        float m = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) m = amax8(v[k], m);
        const QScale s = q_scale(rs.max_of(m, rd), q.format);
        if (rs.w == 0 && rs.lane == 0) q.scales[r] = s.scale;
#pragma unroll
        for (int k = 0; k < K; ++k)
            pack_tile_row<VEC>(q.format, q.codes + e + k * kQTile, left - k * kQTile, rs.lane, v[k], s.inv);
    };
    if (a.keep.codes) pack(a.keep, red[0]);
    if (a.act) {
#pragma unroll
        for (int k = 0; k < K; ++k) gelu(v[k]);
    }
    pack(a.out, red[1]);
}

// One scale per row, rows of more than 16384 columns: a block of 32 warps
// reads the row once for its magnitudes and once for its codes.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) k_pack_long(const PackArgs a) {
    __shared__ float red[2][32];
    const RowSlot<false> rs;
    const int64_t r = blockIdx.x;
    float mk = 0.f, mo = 0.f;
    for (int64_t c0 = rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        F8 v;
        load_tile<T, VEC>((const T*)a.x + r * a.cols + c0 + lane_col<VEC>(rs.lane), (int)(a.cols - c0), rs.lane, v);
        mk = amax8(v, mk);
        if (a.act) {
            gelu(v);
            mo = amax8(v, mo);
        } else {
            mo = mk;
        }
    }
    const QScale sk = q_scale(rs.max_of(mk, red[0]), a.keep.format);
    const QScale so = q_scale(rs.max_of(mo, red[1]), a.out.format);
    if (threadIdx.x == 0) {
        if (a.keep.codes) a.keep.scales[r] = sk.scale;
        a.out.scales[r] = so.scale;
    }
    for (int64_t c0 = rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        const int64_t e = r * a.cols + c0 + lane_col<VEC>(rs.lane);
        const int left = (int)(a.cols - c0);
        F8 v;
        load_tile<T, VEC>((const T*)a.x + e, left, rs.lane, v);
        if (a.keep.codes) pack_tile_row<VEC>(a.keep.format, a.keep.codes + e, left, rs.lane, v, sk.inv);
        if (a.act) gelu(v);
        pack_tile_row<VEC>(a.out.format, a.out.codes + e, left, rs.lane, v, so.inv);
    }
}

// unpack (GRAD false: x = scale * code) and GELU's gradient (GRAD: x = da
// times the slope at scale * code).  One tile per warp (see FlatTile).
template <typename T, bool VEC, bool GRAD, bool ROWS>
__global__ void __launch_bounds__(256) k_unpack(const Q8In q, const T* da, T* x, uint32_t tiles, uint32_t tpr) {
    const uint32_t i = blockIdx.x * 8 + (threadIdx.x >> 5);
    if (i >= tiles) return;
    const int lane = threadIdx.x & 31;
    const FlatTile t = flat_tile<ROWS>(i, tpr, q.cols, q.n_groups, q.gshift);
    const int64_t e = t.e0 + lane_col<VEC>(lane);
    F8 v, g;
    if constexpr (GRAD) load_tile<T, VEC>(da + e, t.left, lane, g);
    load_values<VEC>(q.format, q.gshift, q.codes + e, q.scales + t.s0, t.left, lane, v);
    if constexpr (GRAD) {
        gelu_slope(v);
        v.mul(g);
    }
    store_tile<T, VEC>(x + e, t.left, lane, v);
}

// dst[c * bp + beta] = row beta's value at column c, 0 for beta >= b: four rows
// per thread, so a store covers 16 bytes (or all of a narrower tile).
template <int BP>
__global__ void __launch_bounds__(256) k_q8_transposed(const Q8In q, int b, float* __restrict__ dst) {
    constexpr int R = BP < 4 ? BP : 4;
    const int64_t items = q.cols * (BP / R);
    for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < items;
         i += (int64_t)gridDim.x * blockDim.x) {
        const int qb = (int)(i / q.cols);
        const int64_t c = i - (int64_t)qb * q.cols;
        float v[R];
#pragma unroll
        for (int t = 0; t < R; ++t) v[t] = qb * R + t < b ? q_at(q, qb * R + t, c) : 0.f;
        float* d = dst + c * BP + qb * R;
        if constexpr (R == 4) *reinterpret_cast<float4*>(d) = make_float4(v[0], v[1], v[2], v[3]);
        else if constexpr (R == 2) *reinterpret_cast<float2*>(d) = make_float2(v[0], v[1]);
        else *d = v[0];
    }
}

template <typename T, bool VEC>
int launch_pack(const PackArgs& a, int group, cudaStream_t s) {
    const int64_t tpr = ceil_div(a.cols, kQTile);
    if (group != 0) {
        const int U = a.cols > kQTile ? 2 : 1;
        const int64_t per_row = ceil_div(a.cols, U * kQTile), tiles = a.rows * per_row;
        if (tiles > INT32_MAX) return SNK_ERR_LIMIT;
        auto fn = U == 1 ? k_pack_groups<T, VEC, true, 1>
                  : a.rows == 1 ? k_pack_groups<T, VEC, false, 2>
                                : k_pack_groups<T, VEC, true, 2>;
        fn<<<(unsigned)ceil_div(tiles, 8), 256, 0, s>>>(a, (uint32_t)tiles, (uint32_t)per_row);
    } else if (tpr <= kRegisterTiles) {
        const RowShape f = row_shape(tpr, a.rows <= 256 ? 1 : 4);
        const unsigned grid = (unsigned)ceil_div(a.rows, f.slots()), threads = f.threads();
        switch (f.K + (f.one() ? 2 : 0)) {
            case 1: k_pack_row<T, VEC, 1, false><<<grid, threads, 0, s>>>(a); break;
            case 2: k_pack_row<T, VEC, 2, false><<<grid, threads, 0, s>>>(a); break;
            case 3: k_pack_row<T, VEC, 1, true><<<grid, threads, 0, s>>>(a); break;
            case 4: k_pack_row<T, VEC, 2, true><<<grid, threads, 0, s>>>(a); break;
            case 5: k_pack_row<T, VEC, 3, true><<<grid, threads, 0, s>>>(a); break;
            default: k_pack_row<T, VEC, 4, true><<<grid, threads, 0, s>>>(a); break;
        }
    } else {
        k_pack_long<T, VEC><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

bool pack_vec(const PackArgs& a, int dtype) {
    return a.cols % 8 == 0 && q8_aligned(a.x, dtype == SNK_F32 ? 32 : 16) && q8_aligned(a.out.codes, 8) &&
           q8_aligned(a.keep.codes, 8);
}

int run_pack(PackArgs a, int dtype, int group, cudaStream_t s) {
    if (a.rows == 0) return SNK_OK;
    if (a.rows > INT32_MAX || a.cols > INT32_MAX) return SNK_ERR_LIMIT;
    // whole groups: the matrix is one long row of groups, whatever its width
    if (group != 0 && a.cols % group == 0 && a.rows * a.cols <= INT64_MAX / 2) {
        a.cols *= a.rows;
        a.rows = 1;
    }
    const bool vec = pack_vec(a, dtype);
    switch (dtype) {
        case SNK_F32: return vec ? launch_pack<float, true>(a, group, s) : launch_pack<float, false>(a, group, s);
        case SNK_F16: return vec ? launch_pack<__half, true>(a, group, s) : launch_pack<__half, false>(a, group, s);
        default:
            return vec ? launch_pack<__nv_bfloat16, true>(a, group, s) : launch_pack<__nv_bfloat16, false>(a, group, s);
    }
}

template <typename T, bool GRAD>
int launch_unpack(Q8In q, int64_t rows, int group, const void* da, void* x, cudaStream_t s) {
    if (rows > INT32_MAX || q.cols > INT32_MAX) return SNK_ERR_LIMIT;
    if (group != 0 && q.cols % group == 0) {
        q.cols *= rows;
        rows = 1;
    }
    const int64_t tpr = ceil_div(q.cols, kQTile), tiles = rows * tpr;
    if (tiles > INT32_MAX) return SNK_ERR_LIMIT;
    const uintptr_t al = sizeof(T) == 4 ? 32 : 16;
    const bool vec = q.cols % 8 == 0 && q8_aligned(q.codes, 8) && q8_aligned(x, al) && q8_aligned(da, al);
    const unsigned grid = (unsigned)ceil_div(tiles, 8);
    auto fn = vec ? (rows == 1 ? k_unpack<T, true, GRAD, false> : k_unpack<T, true, GRAD, true>)
                  : (rows == 1 ? k_unpack<T, false, GRAD, false> : k_unpack<T, false, GRAD, true>);
    fn<<<grid, 256, 0, s>>>(q, (const T*)da, (T*)x, (uint32_t)tiles, (uint32_t)tpr);
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

// Shape, type and pointer checks shared by the calls.
bool bad_common(const void* x, int dtype, int64_t rows, int64_t cols, int format, int group, const void* codes,
                const float* scales) {
    if (rows < 0 || cols < 1 || dtype < SNK_F32 || dtype > SNK_BF16) return true;
    if ((format != SNK_Q8_INT8 && format != SNK_Q8_E4M3) || !q8_group_ok(group)) return true;
    if (rows == 0) return false;
    return !x || !codes || !scales || !q8_aligned(x, elt_size(dtype)) || !q8_aligned(scales, 4);
}

Q8Out q8_out(void* codes, float* scales, int format, int group, int64_t cols) {
    return Q8Out{(uint8_t*)codes, scales, format, q8_gshift(group), q8_groups(cols, group)};
}

}  // namespace

int launch_q8_rows(const Q8In& q, int64_t b, float* dst, cudaStream_t s) {
    const int group = q.gshift == 31 ? 0 : 1 << q.gshift;
    return launch_unpack<float, false>(q, b, group, nullptr, dst, s);
}

int launch_q8_transposed(const Q8In& q, int b, int bp, float* dst, int num_sms, cudaStream_t s) {
    const int64_t items = q.cols * std::max(1, bp / 4);
    const unsigned grid = (unsigned)std::min<int64_t>(ceil_div(items, 256), (int64_t)num_sms * 8);
    switch (bp) {
        case 1: k_q8_transposed<1><<<grid, 256, 0, s>>>(q, b, dst); break;
        case 2: k_q8_transposed<2><<<grid, 256, 0, s>>>(q, b, dst); break;
        case 4: k_q8_transposed<4><<<grid, 256, 0, s>>>(q, b, dst); break;
        case 8: k_q8_transposed<8><<<grid, 256, 0, s>>>(q, b, dst); break;
        case 16: k_q8_transposed<16><<<grid, 256, 0, s>>>(q, b, dst); break;
        case 32: k_q8_transposed<32><<<grid, 256, 0, s>>>(q, b, dst); break;
        default: k_q8_transposed<64><<<grid, 256, 0, s>>>(q, b, dst); break;
    }
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

}  // namespace snk

using namespace snk;

extern "C" {

int snk_q8_pack(const void* x, int dtype, int64_t rows, int64_t cols, int format, int group, void* codes,
                float* scales, void* stream) {
    if (bad_common(x, dtype, rows, cols, format, group, codes, scales)) return SNK_ERR_ARG;
    PackArgs a{x, rows, cols, 0, q8_out(codes, scales, format, group, cols), Q8Out{}};
    return run_pack(a, dtype, group, (cudaStream_t)stream);
}

int snk_gelu_q8(const void* x, int dtype, int64_t rows, int64_t cols, int format, int group, void* codes,
                float* scales, void* kept_codes, float* kept_scales, void* stream) {
    if (bad_common(x, dtype, rows, cols, format, group, codes, scales)) return SNK_ERR_ARG;
    if (!kept_codes != !kept_scales || !q8_aligned(kept_scales, 4)) return SNK_ERR_ARG;
    PackArgs a{x, rows, cols, 1, q8_out(codes, scales, format, group, cols),
               q8_out(kept_codes, kept_scales, format, group, cols)};
    return run_pack(a, dtype, group, (cudaStream_t)stream);
}

int snk_q8_unpack(const void* codes, const float* scales, int64_t rows, int64_t cols, int format, int group, void* x,
                  int dtype, void* stream) {
    if (bad_common(x, dtype, rows, cols, format, group, codes, scales)) return SNK_ERR_ARG;
    if (rows == 0) return SNK_OK;
    const Q8In q{(const uint8_t*)codes, scales, format, q8_gshift(group), q8_groups(cols, group), cols};
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case SNK_F32: return launch_unpack<float, false>(q, rows, group, nullptr, x, s);
        case SNK_F16: return launch_unpack<__half, false>(q, rows, group, nullptr, x, s);
        default: return launch_unpack<__nv_bfloat16, false>(q, rows, group, nullptr, x, s);
    }
}

int snk_gelu_backward_q8(const void* da, int dtype, const void* codes, const float* scales, int64_t rows,
                         int64_t cols, int format, int group, void* dh, void* stream) {
    if (bad_common(da, dtype, rows, cols, format, group, codes, scales)) return SNK_ERR_ARG;
    if (rows == 0) return SNK_OK;
    if (!dh || !q8_aligned(dh, elt_size(dtype))) return SNK_ERR_ARG;
    const Q8In q{(const uint8_t*)codes, scales, format, q8_gshift(group), q8_groups(cols, group), cols};
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case SNK_F32: return launch_unpack<float, true>(q, rows, group, da, dh, s);
        case SNK_F16: return launch_unpack<__half, true>(q, rows, group, da, dh, s);
        default: return launch_unpack<__nv_bfloat16, true>(q, rows, group, da, dh, s);
    }
}

}  // extern "C"
