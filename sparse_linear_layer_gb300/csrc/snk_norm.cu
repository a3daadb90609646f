// Root-mean-square norm with the residual's addition and an 8-bit output, and
// its gradient.
//
//     r = x + residual (rounded to the element type, written as `total`)
//     rstd = 1 / sqrt(mean(r^2) + eps)
//     y = r * rstd * gain  ->  codes and scales
//
//     n = r * rstd
//     dx = rstd * (gain dy - n * mean(gain dy n)) + dtotal
//     dgain = sum over the rows of dy n
//
// Bound by the memory system: every element is read once and written once.  A
// row stays in the registers of W warps (K tiles of 256 columns each) from its
// load to its last store; the only exchanges are the row's sum of squares (or
// the gradient's dot product) and, for one scale per row, its largest
// magnitude.  All sums are fp32: a lane adds at most 8 K squares, lanes are
// added by a tree, warps in order.  Rows of more than 32768 columns are read
// again for each step (k_norm_long, k_norm_grad_long).
//
// The gain's gradient needs a sum over the rows.  A block walks rows
// blockIdx, + grid, ... and keeps the sums of its columns in registers; they go
// to one scratch row per block, which k_dgain_sum adds in block order, so the
// result does not depend on timing.
#include <algorithm>

#include "snk_q8.cuh"

namespace snk {
namespace {

struct NormArgs {
    const void* x;
    const void* residual;   // null: r = x, and total is not written
    const float* gain;
    int64_t rows, cols;
    float eps;
    void* total;
    float* rstd;
    Q8Out out;
};

template <typename T, bool VEC, int K>
__global__ void __launch_bounds__(1024) k_norm(const NormArgs a, int W, int slots) {
    __shared__ float red[kMaxSlots * 32];
    __shared__ uint32_t redm[kMaxSlots * 32];
    const RowSlot rs(W);
    const int64_t r = (int64_t)blockIdx.x * slots + rs.slot;
    if (r >= a.rows) return;
    const int64_t off = r * a.cols;
    float v[K][8];
    float ss = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k)
        load_tile<T, VEC>((const T*)a.x + off, (int64_t)(k * W + rs.w) * kQTile, a.cols, rs.lane, v[k]);
    if (a.residual) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t c0 = (int64_t)(k * W + rs.w) * kQTile;
            float t[8];
            load_tile<T, VEC>((const T*)a.residual + off, c0, a.cols, rs.lane, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[k][j] = to_f32(from_f32<T>(v[k][j] + t[j]));
            store_tile<T, VEC>((T*)a.total + off, c0, a.cols, rs.lane, v[k]);
        }
    }
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) ss = fmaf(v[k][j], v[k][j], ss);
    ss = rs.sum(ss, red);
    const float rstd = __frsqrt_rn(__fdiv_rn(ss, (float)a.cols) + a.eps);
    if (rs.w == 0 && rs.lane == 0) a.rstd[r] = rstd;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int64_t c0 = (int64_t)(k * W + rs.w) * kQTile;
        float g[8];
        load_tile<float, VEC>(a.gain, c0, a.cols, rs.lane, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[k][j] = v[k][j] * rstd * g[j];
        if (a.out.gshift < 31) pack_tile_groups<VEC>(a.out, r, c0, a.cols, rs.lane, v[k]);
        else m = max(m, tile_amax(v[k]));
    }
    if (a.out.gshift < 31) return;
    const QScale s = q_scale(rs.max_of(m, redm), q_top(a.out.format));
    if (rs.w == 0 && rs.lane == 0) a.out.scales[r] = s.scale;
#pragma unroll
    for (int k = 0; k < K; ++k)
        pack_tile_row<VEC>(a.out, r, (int64_t)(k * W + rs.w) * kQTile, a.cols, rs.lane, v[k], s.inv);
}

// Rows of any length: a block of 32 warps, the row read once for each step.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) k_norm_long(const NormArgs a) {
    __shared__ float red[32];
    __shared__ uint32_t redm[32];
    const RowSlot rs(32);
    const int64_t r = blockIdx.x, off = r * a.cols;
    // the summed row is re-read by the thread that wrote it
    const T* src = a.residual ? (const T*)a.total + off : (const T*)a.x + off;
    float ss = 0.f;
    for (int64_t c0 = (int64_t)rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        float v[8];
        load_tile<T, VEC>((const T*)a.x + off, c0, a.cols, rs.lane, v);
        if (a.residual) {
            float t[8];
            load_tile<T, VEC>((const T*)a.residual + off, c0, a.cols, rs.lane, t);
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = to_f32(from_f32<T>(v[j] + t[j]));
            store_tile<T, VEC>((T*)a.total + off, c0, a.cols, rs.lane, v);
        }
        float part = 0.f;
#pragma unroll
        for (int j = 0; j < 8; ++j) part = fmaf(v[j], v[j], part);
        ss += part;
    }
    ss = rs.sum(ss, red);
    const float rstd = __frsqrt_rn(__fdiv_rn(ss, (float)a.cols) + a.eps);
    if (threadIdx.x == 0) a.rstd[r] = rstd;
    auto normed = [&](int64_t c0, float (&v)[8]) {
        float g[8];
        load_tile<T, VEC>(src, c0, a.cols, rs.lane, v);
        load_tile<float, VEC>(a.gain, c0, a.cols, rs.lane, g);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = v[j] * rstd * g[j];
    };
    uint32_t m = 0;
    for (int64_t c0 = (int64_t)rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        float v[8];
        normed(c0, v);
        if (a.out.gshift < 31) pack_tile_groups<VEC>(a.out, r, c0, a.cols, rs.lane, v);
        else m = max(m, tile_amax(v));
    }
    if (a.out.gshift < 31) return;
    const QScale s = q_scale(rs.max_of(m, redm), q_top(a.out.format));
    if (threadIdx.x == 0) a.out.scales[r] = s.scale;
    for (int64_t c0 = (int64_t)rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        float v[8];
        normed(c0, v);
        pack_tile_row<VEC>(a.out, r, c0, a.cols, rs.lane, v, s.inv);
    }
}

struct NormGradArgs {
    const float* dy;
    const void* total;
    const float* rstd;
    const float* gain;
    const void* dtotal;   // or null
    int64_t rows, cols;
    void* dx;
    float* part;          // [gridDim.x][cols], or null: no gain gradient
};

template <typename T, bool VEC, int K>
__global__ void __launch_bounds__(K == 1 ? 1024 : 512) k_norm_grad(const NormGradArgs a, int W, int slots) {
    extern __shared__ float cols_sm[];                    // [W * K * 256] when slots > 1
    __shared__ float red[2][kMaxSlots * 32];
    const RowSlot rs(W);
    float acc[K][8];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[k][j] = 0.f;
    int turn = 0;
    for (int64_t r = (int64_t)blockIdx.x * slots + rs.slot; r < a.rows; r += (int64_t)gridDim.x * slots, turn ^= 1) {
        const int64_t off = r * a.cols;
        const float rstd = __ldg(a.rstd + r);
        float g[K][8], n[K][8], add[K][8];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t c0 = (int64_t)(k * W + rs.w) * kQTile;
            load_tile<float, VEC>(a.dy + off, c0, a.cols, rs.lane, g[k]);
            load_tile<T, VEC>((const T*)a.total + off, c0, a.cols, rs.lane, n[k]);
            if (a.dtotal) load_tile<T, VEC>((const T*)a.dtotal + off, c0, a.cols, rs.lane, add[k]);
        }
        float dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            float w[8];
            load_tile<float, VEC>(a.gain, (int64_t)(k * W + rs.w) * kQTile, a.cols, rs.lane, w);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                n[k][j] *= rstd;
                acc[k][j] = fmaf(g[k][j], n[k][j], acc[k][j]);
                g[k][j] *= w[j];
                dot = fmaf(g[k][j], n[k][j], dot);
            }
        }
        // two turns share no `red`, so a warp still reading this turn's sums
        // is past them before anyone writes there again
        dot = __fdiv_rn(rs.sum(dot, red[turn]), (float)a.cols);
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[k][j] = rstd * (g[k][j] - n[k][j] * dot);
                if (a.dtotal) g[k][j] += add[k][j];
            }
            store_tile<T, VEC>((T*)a.dx + off, (int64_t)(k * W + rs.w) * kQTile, a.cols, rs.lane, g[k]);
        }
    }
    if (!a.part) return;
    // the slots' sums in slot order
    float* dst = a.part + (int64_t)blockIdx.x * a.cols;
    for (int s = 0; s < slots; ++s) {
        if (rs.slot == s) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int t = k * W + rs.w;
                if (s > 0) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) acc[k][j] += cols_sm[t * kQTile + j * 32 + rs.lane];
                }
                if (s + 1 < slots) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) cols_sm[t * kQTile + j * 32 + rs.lane] = acc[k][j];
                } else {
                    store_tile<float, VEC>(dst, (int64_t)t * kQTile, a.cols, rs.lane, acc[k]);
                }
            }
        }
        if (slots > 1) __syncthreads();
    }
}

// Rows of any length; the gain's partial sums live in the block's scratch row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) k_norm_grad_long(const NormGradArgs a) {
    __shared__ float red[2][32];
    const RowSlot rs(32);
    float* dst = a.part ? a.part + (int64_t)blockIdx.x * a.cols : nullptr;
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
        const int64_t off = r * a.cols;
        const float rstd = __ldg(a.rstd + r);
        const bool first = r == blockIdx.x;
        auto load = [&](int64_t c0, float (&g)[8], float (&n)[8]) {
            load_tile<float, VEC>(a.dy + off, c0, a.cols, rs.lane, g);
            load_tile<T, VEC>((const T*)a.total + off, c0, a.cols, rs.lane, n);
#pragma unroll
            for (int j = 0; j < 8; ++j) n[j] *= rstd;
        };
        float dot = 0.f;
        for (int64_t c0 = (int64_t)rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
            float g[8], n[8], w[8];
            load(c0, g, n);
            load_tile<float, VEC>(a.gain, c0, a.cols, rs.lane, w);
            float part = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) part = fmaf(g[j] * w[j], n[j], part);
            dot += part;
            if (dst) {
                float d[8];
                if (first) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) d[j] = 0.f;
                } else {
                    load_tile<float, VEC>(dst, c0, a.cols, rs.lane, d);
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) d[j] = fmaf(g[j], n[j], d[j]);
                store_tile<float, VEC>(dst, c0, a.cols, rs.lane, d);
            }
        }
        dot = __fdiv_rn(rs.sum(dot, red[turn]), (float)a.cols);
        for (int64_t c0 = (int64_t)rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
            float g[8], n[8], w[8], add[8];
            load(c0, g, n);
            load_tile<float, VEC>(a.gain, c0, a.cols, rs.lane, w);
            if (a.dtotal) load_tile<T, VEC>((const T*)a.dtotal + off, c0, a.cols, rs.lane, add);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                g[j] = rstd * (g[j] * w[j] - n[j] * dot);
                if (a.dtotal) g[j] += add[j];
            }
            store_tile<T, VEC>((T*)a.dx + off, c0, a.cols, rs.lane, g);
        }
    }
}

// dgain[c] = the blocks' partial sums of column c: 32 threads take every 32nd
// of them, a tree adds the 32.
__global__ void __launch_bounds__(1024) k_dgain_sum(const float* __restrict__ part, int n, int64_t cols,
                                                    float* __restrict__ dgain) {
    __shared__ float sm[32][33];
    const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + x;
    float t = 0.f;
    if (c < cols)
        for (int i = y; i < n; i += 32) t += part[(int64_t)i * cols + c];
    sm[y][x] = t;
    __syncthreads();
    t = sm[x][y];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    const int64_t cc = (int64_t)blockIdx.x * 32 + y;
    if (x == 0 && cc < cols) dgain[cc] = t;
}

template <typename T, bool VEC>
int launch_norm(const NormArgs& a, cudaStream_t s) {
    const int64_t tpr = ceil_div(a.cols, kQTile);
    if (tpr <= 128) {
        const bool short_rows = tpr <= 2 || (a.rows <= 256 && tpr <= 32);
        const int K = short_rows ? 1 : 4;
        const int W = (int)ceil_div(tpr, K), slots = std::max(1, std::min(kMaxSlots, 8 / W));
        const unsigned grid = (unsigned)ceil_div(a.rows, slots);
        if (K == 1) k_norm<T, VEC, 1><<<grid, slots * W * 32, 0, s>>>(a, W, slots);
        else k_norm<T, VEC, 4><<<grid, slots * W * 32, 0, s>>>(a, W, slots);
    } else {
        k_norm_long<T, VEC><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

// Blocks of the gradient kernel: a scratch row each.
constexpr int kGradBlocks = 304;

template <typename T, bool VEC>
int launch_norm_grad(const NormGradArgs& a, float* dgain, cudaStream_t s) {
    const int64_t tpr = ceil_div(a.cols, kQTile);
    int64_t grid;
    if (tpr <= 64) {
        const bool k1 = tpr <= 2 || a.rows <= 152;
        const int K = k1 && tpr <= 32 ? 1 : 4;
        const int W = (int)ceil_div(tpr, K), slots = std::max(1, std::min(kMaxSlots, 8 / W));
        grid = std::min<int64_t>(kGradBlocks, ceil_div(a.rows, slots));
        const size_t smem = slots > 1 ? (size_t)W * K * kQTile * sizeof(float) : 0;
        if (K == 1) k_norm_grad<T, VEC, 1><<<(unsigned)grid, slots * W * 32, smem, s>>>(a, W, slots);
        else k_norm_grad<T, VEC, 4><<<(unsigned)grid, slots * W * 32, smem, s>>>(a, W, slots);
    } else {
        grid = std::min<int64_t>(kGradBlocks, a.rows);
        k_norm_grad_long<T, VEC><<<(unsigned)grid, 1024, 0, s>>>(a);
    }
    if (cudaGetLastError() != cudaSuccess) return SNK_ERR_CUDA;
    if (dgain) {
        k_dgain_sum<<<(unsigned)ceil_div(a.cols, 32), 1024, 0, s>>>(a.part, (int)grid, a.cols, dgain);
        if (cudaGetLastError() != cudaSuccess) return SNK_ERR_CUDA;
    }
    return SNK_OK;
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

int snk_rmsnorm_q8(const void* x, const void* residual, int dtype, const float* gain, int64_t rows, int64_t cols,
                   float eps, int format, int group, void* codes, float* scales, void* total, float* rstd,
                   void* stream) {
    if (rows < 0 || cols < 1 || dtype < SNK_F32 || dtype > SNK_BF16 || !(eps > 0.f)) return SNK_ERR_ARG;
    if ((format != SNK_Q8_INT8 && format != SNK_Q8_E4M3) || !q8_group_ok(group)) return SNK_ERR_ARG;
    if (rows == 0) return SNK_OK;
    const size_t e = elt_size(dtype);
    if (!x || !gain || !codes || !scales || !rstd || !residual != !total) return SNK_ERR_ARG;
    if (!q8_aligned(x, e) || !q8_aligned(residual, e) || !q8_aligned(total, e) || !q8_aligned(gain, 4) ||
        !q8_aligned(scales, 4) || !q8_aligned(rstd, 4))
        return SNK_ERR_ARG;
    if (rows > INT32_MAX || cols > INT32_MAX) return SNK_ERR_LIMIT;
    const NormArgs a{x, residual, gain, rows, cols, eps, total, rstd,
                     Q8Out{(uint8_t*)codes, scales, format, q8_gshift(group), q8_groups(cols, group)}};
    const uintptr_t al = dtype == SNK_F32 ? 32 : 16;
    const bool vec = cols % 8 == 0 && q8_aligned(x, al) && q8_aligned(residual, al) && q8_aligned(total, al) &&
                     q8_aligned(gain, 32) && q8_aligned(codes, 8);
    cudaStream_t s = (cudaStream_t)stream;
    switch (dtype) {
        case SNK_F32: return vec ? launch_norm<float, true>(a, s) : launch_norm<float, false>(a, s);
        case SNK_F16: return vec ? launch_norm<__half, true>(a, s) : launch_norm<__half, false>(a, s);
        default: return vec ? launch_norm<__nv_bfloat16, true>(a, s) : launch_norm<__nv_bfloat16, false>(a, s);
    }
}

int64_t snk_rmsnorm_backward_scratch(int64_t rows, int64_t cols) {
    if (rows < 1 || cols < 1) return 0;
    return std::min<int64_t>(rows, kGradBlocks) * ((cols + 7) & ~(int64_t)7) * (int64_t)sizeof(float);
}

int snk_rmsnorm_backward(const float* dy, const void* total, int dtype, const float* rstd, const float* gain,
                         const void* dtotal, int64_t rows, int64_t cols, void* dx, float* dgain, void* scratch,
                         void* stream) {
    if (rows < 0 || cols < 1 || dtype < SNK_F32 || dtype > SNK_BF16) return SNK_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (!q8_aligned(dgain, 4)) return SNK_ERR_ARG;
    if (rows == 0) {
        // a sum over no rows
        if (dgain && cudaMemsetAsync(dgain, 0, (size_t)cols * sizeof(float), s) != cudaSuccess) return SNK_ERR_CUDA;
        return SNK_OK;
    }
    const size_t e = elt_size(dtype);
    if (!dy || !total || !rstd || !gain || !dx || (dgain && !scratch)) return SNK_ERR_ARG;
    if (!q8_aligned(dy, 4) || !q8_aligned(total, e) || !q8_aligned(rstd, 4) || !q8_aligned(gain, 4) ||
        !q8_aligned(dtotal, e) || !q8_aligned(dx, e) || !q8_aligned(scratch, 32))
        return SNK_ERR_ARG;
    if (rows > INT32_MAX || cols > INT32_MAX) return SNK_ERR_LIMIT;
    const NormGradArgs a{dy, total, rstd, gain, dtotal, rows, cols, dx, dgain ? (float*)scratch : nullptr};
    const uintptr_t al = dtype == SNK_F32 ? 32 : 16;
    const bool vec = cols % 8 == 0 && q8_aligned(dy, 32) && q8_aligned(total, al) && q8_aligned(dtotal, al) &&
                     q8_aligned(dx, al) && q8_aligned(gain, 32);
    switch (dtype) {
        case SNK_F32: return vec ? launch_norm_grad<float, true>(a, dgain, s) : launch_norm_grad<float, false>(a, dgain, s);
        case SNK_F16: return vec ? launch_norm_grad<__half, true>(a, dgain, s) : launch_norm_grad<__half, false>(a, dgain, s);
        default:
            return vec ? launch_norm_grad<__nv_bfloat16, true>(a, dgain, s)
                       : launch_norm_grad<__nv_bfloat16, false>(a, dgain, s);
    }
}

}  // extern "C"
