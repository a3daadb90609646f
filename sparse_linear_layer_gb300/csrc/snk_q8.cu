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
// (k_pack_row), up to 32768 columns; longer rows are read twice (k_pack_long).
#include <algorithm>

#include "snk_q8.cuh"

namespace snk {
namespace {

__device__ __forceinline__ float gelu(float x) { return 0.5f * x * (1.f + erff(x * 0.70710678f)); }
__device__ __forceinline__ float gelu_slope(float x) {
    return 0.5f * (1.f + erff(x * 0.70710678f)) + x * 0.39894228f * expf(-0.5f * x * x);
}

struct PackArgs {
    const void* x;
    int64_t rows, cols;
    int act;       // 1: gelu(x) is packed
    Q8Out out;     // what is packed
    Q8Out keep;    // x itself (codes null: not kept)
};

// Groups of 32..256 columns: a warp takes kU tiles at a time, independent of
// one another.
constexpr int kU = 4;
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) k_pack_groups(const PackArgs a, uint32_t tiles, uint32_t tpr) {
    const int lane = threadIdx.x & 31;
    const uint32_t t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kU;
    float v[kU][8];
    int64_t r[kU], c0[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const uint32_t t = t0 + u;
        r[u] = t / tpr;
        c0[u] = (int64_t)(t - (uint32_t)r[u] * tpr) * kQTile;
        if (t < tiles) load_tile<T, VEC>((const T*)a.x + r[u] * a.cols, c0[u], a.cols, lane, v[u]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        if (t0 + u >= tiles) break;
        if (a.keep.codes) pack_tile_groups<VEC>(a.keep, r[u], c0[u], a.cols, lane, v[u]);
        if (a.act) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[u][j] = gelu(v[u][j]);
        }
        pack_tile_groups<VEC>(a.out, r[u], c0[u], a.cols, lane, v[u]);
    }
}

// One scale per row: the row in the registers of W warps, K tiles each.
template <typename T, bool VEC, int K>
__global__ void __launch_bounds__(1024) k_pack_row(const PackArgs a, int W, int slots) {
    __shared__ uint32_t red[2][kMaxSlots * 32];
    const RowSlot rs(W);
    const int64_t r = (int64_t)blockIdx.x * slots + rs.slot;
    if (r >= a.rows) return;
    float v[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
        load_tile<T, VEC>((const T*)a.x + r * a.cols, (int64_t)(k * W + rs.w) * kQTile, a.cols, rs.lane, v[k]);
    auto pack = [&](const Q8Out& q, uint32_t* rd) {
        uint32_t m = 0;
#pragma unroll
        for (int k = 0; k < K; ++k) m = max(m, tile_amax(v[k]));
        const QScale s = q_scale(rs.max_of(m, rd), q_top(q.format));
        if (rs.w == 0 && rs.lane == 0) q.scales[r] = s.scale;
#pragma unroll
        for (int k = 0; k < K; ++k)
            pack_tile_row<VEC>(q, r, (int64_t)(k * W + rs.w) * kQTile, a.cols, rs.lane, v[k], s.inv);
    };
    if (a.keep.codes) pack(a.keep, red[0]);
    if (a.act) {
#pragma unroll
        for (int k = 0; k < K; ++k)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = gelu(v[k][j]);
    }
    pack(a.out, red[1]);
}

// One scale per row, rows of more than 32768 columns: a block of 32 warps
// reads the row once for its magnitudes and once for its codes.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) k_pack_long(const PackArgs a) {
    __shared__ uint32_t red[2][32];
    const RowSlot rs(32);
    const int64_t r = blockIdx.x;
    const T* x = (const T*)a.x + r * a.cols;
    uint32_t mk = 0, mo = 0;
    for (int64_t c0 = (int64_t)rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        float v[8];
        load_tile<T, VEC>(x, c0, a.cols, rs.lane, v);
        mk = max(mk, tile_amax(v));
        if (a.act) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = gelu(v[j]);
            mo = max(mo, tile_amax(v));
        } else {
            mo = mk;
        }
    }
    const QScale sk = q_scale(rs.max_of(mk, red[0]), q_top(a.keep.format));
    const QScale so = q_scale(rs.max_of(mo, red[1]), q_top(a.out.format));
    if (threadIdx.x == 0) {
        if (a.keep.codes) a.keep.scales[r] = sk.scale;
        a.out.scales[r] = so.scale;
    }
    for (int64_t c0 = (int64_t)rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        float v[8];
        load_tile<T, VEC>(x, c0, a.cols, rs.lane, v);
        if (a.keep.codes) pack_tile_row<VEC>(a.keep, r, c0, a.cols, rs.lane, v, sk.inv);
        if (a.act) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = gelu(v[j]);
        }
        pack_tile_row<VEC>(a.out, r, c0, a.cols, rs.lane, v, so.inv);
    }
}

// unpack (GRAD false: x = scale * code) and GELU's gradient (GRAD: x = da
// times the slope at scale * code), kU tiles per warp.
template <typename T, bool VEC, bool GRAD>
__global__ void __launch_bounds__(256) k_unpack(const Q8In q, const T* da, T* x, uint32_t tiles, uint32_t tpr) {
    const int lane = threadIdx.x & 31;
    const uint32_t t0 = (blockIdx.x * 8 + (threadIdx.x >> 5)) * kU;
    float v[kU][8], g[GRAD ? kU : 1][8];
    int64_t r[kU], c0[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        const uint32_t t = t0 + u;
        r[u] = t / tpr;
        c0[u] = (int64_t)(t - (uint32_t)r[u] * tpr) * kQTile;
        if (t < tiles) {
            load_values<VEC>(q, r[u], c0[u], lane, v[u]);
            if constexpr (GRAD) load_tile<T, VEC>(da + r[u] * q.cols, c0[u], q.cols, lane, g[u]);
        }
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
        if (t0 + u >= tiles) break;
        if constexpr (GRAD) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[u][j] = g[u][j] * gelu_slope(v[u][j]);
        }
        store_tile<T, VEC>(x + r[u] * q.cols, c0[u], q.cols, lane, v[u]);
    }
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
        const int64_t tiles = a.rows * tpr;
        if (tiles > INT32_MAX) return SNK_ERR_LIMIT;
        k_pack_groups<T, VEC><<<(unsigned)ceil_div(tiles, 8 * kU), 256, 0, s>>>(a, (uint32_t)tiles, (uint32_t)tpr);
    } else if (tpr <= 128) {
        // few rows: one tile per warp, for the shortest time of a row
        const bool short_rows = tpr <= 8 || (a.rows <= 256 && tpr <= 32);
        const int K = short_rows ? 1 : 4;
        const int W = (int)ceil_div(tpr, K), slots = std::max(1, std::min(kMaxSlots, 8 / W));
        const unsigned grid = (unsigned)ceil_div(a.rows, slots);
        if (K == 1) k_pack_row<T, VEC, 1><<<grid, slots * W * 32, 0, s>>>(a, W, slots);
        else k_pack_row<T, VEC, 4><<<grid, slots * W * 32, 0, s>>>(a, W, slots);
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
    const unsigned grid = (unsigned)ceil_div(tiles, 8 * kU);
    if (vec)
        k_unpack<T, true, GRAD><<<grid, 256, 0, s>>>(q, (const T*)da, (T*)x, (uint32_t)tiles, (uint32_t)tpr);
    else
        k_unpack<T, false, GRAD><<<grid, 256, 0, s>>>(q, (const T*)da, (T*)x, (uint32_t)tiles, (uint32_t)tpr);
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
