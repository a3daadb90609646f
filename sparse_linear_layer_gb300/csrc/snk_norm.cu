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
// added by a tree, warps in order.  Rows of more than 16384 columns are read
// again for each step (k_norm_long, k_norm_grad_long).
//
// Measured: 32768 x 768 bf16 to E4M3 in groups of 128 with a residual, 33 us (5.4 TB/s
// of the bytes it has to move; issue slots 61% busy, 80 registers), its gradient 49 us (5.1
// TB/s; latency of the row's exchange, 64 registers).  One row of 768: 2.1 us.
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
    float inv_cols;         // 1 / cols
    float eps;
    void* total;
    float* rstd;
    Q8Out out;
};

// 1 / sqrt(x): the approximate one and a Newton step, within an ulp.
__device__ __forceinline__ float inv_sqrt(float x) {
    float y;
    asm("rsqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
    const float h = 0.5f * y;
    const float e = fmaf(-x * y, h, 0.5f);
    return isfinite(e) ? fmaf(y, e, y) : y;
}

// The sum of a lane's 8 values.
__device__ __forceinline__ float sum8(const F8& v) {
    const float2 h = __fadd2_rn(__fadd2_rn(v.p[0], v.p[1]), __fadd2_rn(v.p[2], v.p[3]));
    return h.x + h.y;
}

// From the row in v (r = x + residual, rounded): its norm's codes and scales.
// gain, codes: at the lane's first element of the row; scales: the first scale of
// the warp's first tile; left: the columns from that tile on.
template <bool VEC, int K, bool ONE>
__device__ __forceinline__ void norm_row(const NormArgs& a, const RowSlot<ONE>& rs, F8 (&v)[K], const float* gain,
                                         uint8_t* codes, float* scales, float* rstd_out, int left, float* red,
                                         float* redm) {
    F8 sq;
    sq.clear();
#pragma unroll
    for (int k = 0; k < K; ++k) sq.fma(v[k], v[k]);
    const float ss = rs.sum(sum8(sq), red);
    const float rstd = inv_sqrt(fmaf(ss, a.inv_cols, a.eps));
    if (rs.w == 0 && rs.lane == 0) *rstd_out = rstd;
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        F8 g;
        load_tile<float, VEC>(gain + k * kQTile, left - k * kQTile, rs.lane, g);
        v[k].mul(rstd);
        v[k].mul(g);
        if (a.out.gshift < 31)
            pack_tile_groups<VEC>(a.out.format, a.out.gshift, codes + k * kQTile, scales + ((k * kQTile) >> a.out.gshift),
                                  left - k * kQTile, rs.lane, v[k]);
        else
            m = amax8(v[k], m);
    }
    if (a.out.gshift < 31) return;
    const QScale s = q_scale(rs.max_of(m, redm), a.out.format);
    if (rs.w == 0 && rs.lane == 0) *scales = s.scale;
#pragma unroll
    for (int k = 0; k < K; ++k)
        pack_tile_row<VEC>(a.out.format, codes + k * kQTile, left - k * kQTile, rs.lane, v[k], s.inv);
}

// One row per slot, straight from memory: rows that are not aligned, calls of
// too few rows to keep any in flight, and rows over many warps.
template <typename T, bool VEC, int K, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kRowsPerBlock : 1024) k_norm(const NormArgs a) {
    __shared__ float red[32], redm[32];
    const RowSlot<ONE> rs;
    const int64_t r = rs.first_row();
    if (r >= a.rows) return;
    const int c0 = rs.w * K * kQTile, left = (int)a.cols - c0, c = c0 + lane_col<VEC>(rs.lane);
    const int64_t e = r * a.cols + c;
    F8 v[K];
#pragma unroll
    for (int k = 0; k < K; ++k)
        load_tile<T, VEC>((const T*)a.x + e + k * kQTile, left - k * kQTile, rs.lane, v[k]);
    if (a.residual) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            F8 t;
            load_tile<T, VEC>((const T*)a.residual + e + k * kQTile, left - k * kQTile, rs.lane, t);
            v[k].add(t);
            v[k].template round<T>();
            store_tile<T, VEC>((T*)a.total + e + k * kQTile, left - k * kQTile, rs.lane, v[k]);
        }
    }
    norm_row<VEC, K, ONE>(a, rs, v, a.gain + c, a.out.codes + e, a.out.scales + r * a.out.n_groups + (c0 >> a.out.gshift),
                          a.rstd + r, left, red, redm);
}

// Many aligned rows: each slot walks rows, the next row's tiles in flight.
template <typename T, int K, bool ONE>
__global__ void __launch_bounds__(ONE ? 32 * kRowsPerBlock : 1024, ONE ? 3 : 1) k_norm_ring(const NormArgs a) {
    extern __shared__ uint4 ring[];
    // two turns use two halves: a warp may still be reading this row's sums
    // when another is at the next row's
    __shared__ float red[2][32], redm[2][32];
    const RowSlot<ONE> rs;
    const int units = (a.residual ? 2 : 1) * K * Ring<T>::kUnits;
    const int c0 = rs.w * K * kQTile, left = (int)a.cols - c0, c = c0 + 8 * rs.lane;
    const int64_t step = (int64_t)gridDim.x * rs.slots;
    auto request = [&](int64_t r, int stage) {
        if (r < a.rows) {
            uint4* st = ring + stage * units * blockDim.x;
            const int64_t e = r * a.cols + c;
#pragma unroll
            for (int k = 0; k < K; ++k) {
                Ring<T>::copy(st, k, (const T*)a.x + e + k * kQTile, left - k * kQTile, rs.lane);
                if (a.residual)
                    Ring<T>::copy(st, K + k, (const T*)a.residual + e + k * kQTile, left - k * kQTile, rs.lane);
            }
        }
        ring_commit();
    };
    int64_t r = rs.first_row();
    request(r, 0);
    for (int turn = 0; r < a.rows; r += step, turn ^= 1) {
        request(r + step, turn ^ 1);
        ring_wait<1>();
        const uint4* st = ring + turn * units * blockDim.x;
        const int64_t e = r * a.cols + c;
        F8 v[K];
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if (a.residual) {
                Ring<T>::read_sum(st, k, K + k, v[k]);
                store_tile<T, true>((T*)a.total + e + k * kQTile, left - k * kQTile, rs.lane, v[k]);
            } else {
                Ring<T>::read(st, k, v[k]);
            }
        }
        norm_row<true, K, ONE>(a, rs, v, a.gain + c, a.out.codes + e,
                               a.out.scales + r * a.out.n_groups + (c0 >> a.out.gshift), a.rstd + r, left, red[turn],
                               redm[turn]);
    }
}

// Rows of any length: a block of 32 warps, the row read once for each step.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) k_norm_long(const NormArgs a) {
    __shared__ float red[32], redm[32];
    const RowSlot<false> rs;
    const int64_t r = blockIdx.x, row = r * a.cols;
    const int lc = lane_col<VEC>(rs.lane);
    // the summed row is re-read by the thread that wrote it
    const T* src = a.residual ? (const T*)a.total : (const T*)a.x;
    float ss = 0.f;
    for (int64_t c0 = rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        const int left = (int)(a.cols - c0);
        F8 v, sq;
        load_tile<T, VEC>((const T*)a.x + row + c0 + lc, left, rs.lane, v);
        if (a.residual) {
            F8 u;
            load_tile<T, VEC>((const T*)a.residual + row + c0 + lc, left, rs.lane, u);
            v.add(u);
            v.template round<T>();
            store_tile<T, VEC>((T*)a.total + row + c0 + lc, left, rs.lane, v);
        }
        sq.clear();
        sq.fma(v, v);
        ss += sum8(sq);
    }
    ss = rs.sum(ss, red);
    const float rstd = inv_sqrt(fmaf(ss, a.inv_cols, a.eps));
    if (threadIdx.x == 0) a.rstd[r] = rstd;
    auto normed = [&](int64_t c0, int left, F8& v) {
        F8 g;
        load_tile<T, VEC>(src + row + c0 + lc, left, rs.lane, v);
        load_tile<float, VEC>(a.gain + c0 + lc, left, rs.lane, g);
        v.mul(rstd);
        v.mul(g);
    };
    float m = 0.f;
    for (int64_t c0 = rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        const int left = (int)(a.cols - c0);
        F8 v;
        normed(c0, left, v);
        if (a.out.gshift < 31)
            pack_tile_groups<VEC>(a.out.format, a.out.gshift, a.out.codes + row + c0 + lc,
                                  a.out.scales + r * a.out.n_groups + (c0 >> a.out.gshift), left, rs.lane, v);
        else
            m = amax8(v, m);
    }
    if (a.out.gshift < 31) return;
    const QScale s = q_scale(rs.max_of(m, redm), a.out.format);
    if (threadIdx.x == 0) a.out.scales[r] = s.scale;
    for (int64_t c0 = rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
        const int left = (int)(a.cols - c0);
        F8 v;
        normed(c0, left, v);
        pack_tile_row<VEC>(a.out.format, a.out.codes + row + c0 + lc, left, rs.lane, v, s.inv);
    }
}

struct NormGradArgs {
    const float* dy;
    const void* total;
    const float* rstd;
    const float* gain;
    const void* dtotal;   // or null
    int64_t rows, cols;
    float inv_cols;       // 1 / cols
    void* dx;
    float* part;          // [gridDim.x][cols], or null: no gain gradient
};

// A slot walks rows; with RING (aligned rows) the next row's tiles are in flight.
template <typename T, bool VEC, int K, bool ONE, bool RING>
__global__ void __launch_bounds__(ONE ? 32 * kRowsPerBlock : 1024)
    k_norm_grad(const NormGradArgs a) {
    // RING: two stages of the rows; then, for ONE, [K * 256] column sums
    extern __shared__ uint4 ring[];
    __shared__ float red[2][32];
    const RowSlot<ONE> rs;
    constexpr int U4 = Ring<float>::kUnits, UT = RING ? Ring<T>::kUnits : 0;
    const int units = K * (U4 + (a.dtotal ? 2 : 1) * UT);
    const int c0 = rs.w * K * kQTile, left = (int)a.cols - c0, c = c0 + lane_col<VEC>(rs.lane);
    const int64_t step = (int64_t)gridDim.x * rs.slots;
    auto request = [&](int64_t r, int stage) {
        if constexpr (RING) {
            if (r < a.rows) {
                uint4* st = ring + stage * units * blockDim.x;
                uint4* st_t = st + K * U4 * blockDim.x;
                const int64_t e = r * a.cols + c;
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    const int l = left - k * kQTile;
                    Ring<float>::copy(st, k, a.dy + e + k * kQTile, l, rs.lane);
                    Ring<T>::copy(st_t, k, (const T*)a.total + e + k * kQTile, l, rs.lane);
                    if (a.dtotal) Ring<T>::copy(st_t, K + k, (const T*)a.dtotal + e + k * kQTile, l, rs.lane);
                }
            }
            ring_commit();
        }
    };
    F8 acc[K];
#pragma unroll
    for (int k = 0; k < K; ++k) acc[k].clear();
    int64_t r = rs.first_row();
    request(r, 0);
    float rstd_next = r < a.rows ? __ldg(a.rstd + r) : 0.f;
    for (int turn = 0; r < a.rows; r += step, turn ^= 1) {
        request(r + step, turn ^ 1);
        const float rstd = rstd_next;
        if (r + step < a.rows) rstd_next = __ldg(a.rstd + r + step);
        const int64_t e = r * a.cols + c;
        const uint4* st = nullptr;
        const uint4* st_t = nullptr;
        if constexpr (RING) {
            ring_wait<1>();
            st = ring + turn * units * blockDim.x;
            st_t = st + K * U4 * blockDim.x;
        }
        F8 g[K], n[K], add[RING ? 1 : K];
        if constexpr (!RING) {
#pragma unroll
            for (int k = 0; k < K; ++k) {
                const int l = left - k * kQTile;
                load_tile<float, VEC>(a.dy + e + k * kQTile, l, rs.lane, g[k]);
                load_tile<T, VEC>((const T*)a.total + e + k * kQTile, l, rs.lane, n[k]);
                if (a.dtotal) load_tile<T, VEC>((const T*)a.dtotal + e + k * kQTile, l, rs.lane, add[k]);
            }
        }
        F8 dots;
        dots.clear();
#pragma unroll
        for (int k = 0; k < K; ++k) {
            if constexpr (RING) {
                Ring<float>::read(st, k, g[k]);
                Ring<T>::read(st_t, k, n[k]);
            }
            F8 w;
            load_tile<float, VEC>(a.gain + c + k * kQTile, left - k * kQTile, rs.lane, w);
            n[k].mul(rstd);
            acc[k].fma(g[k], n[k]);
            g[k].mul(w);
            dots.fma(g[k], n[k]);
        }
        // two turns share no `red`, so a warp still reading this turn's sums
        // is past them before anyone writes there again
        const float mean = rs.sum(sum8(dots), red[turn]) * a.inv_cols;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            n[k].mul(-mean);
            g[k].add(n[k]);
            g[k].mul(rstd);
            if (a.dtotal) {
                if constexpr (RING) Ring<T>::read(st_t, K + k, add[0]);
                g[k].add(add[RING ? 0 : k]);
            }
            store_tile<T, VEC>((T*)a.dx + e + k * kQTile, left - k * kQTile, rs.lane, g[k]);
        }
    }
    if (!a.part) return;
    float* dst = a.part + blockIdx.x * a.cols + c;
    if constexpr (!ONE) {
#pragma unroll
        for (int k = 0; k < K; ++k) store_tile<float, VEC>(dst + k * kQTile, left - k * kQTile, rs.lane, acc[k]);
    } else {
        // the warps' sums in warp order
        float* cols_sm = reinterpret_cast<float*>(ring + (RING ? 2 * units * blockDim.x : 0)) + rs.lane;
        for (int s = 0; s < rs.slots; ++s) {
            if (rs.slot == s) {
#pragma unroll
                for (int k = 0; k < K; ++k) {
                    float* mine = cols_sm + k * kQTile;
                    if (s > 0) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) acc[k].set(j, acc[k].at(j) + mine[j * 32]);
                    }
                    if (s + 1 < rs.slots) {
#pragma unroll
                        for (int j = 0; j < 8; ++j) mine[j * 32] = acc[k].at(j);
                    } else {
                        store_tile<float, VEC>(dst + k * kQTile, left - k * kQTile, rs.lane, acc[k]);
                    }
                }
            }
            __syncthreads();
        }
    }
}

// Few rows, in one launch and without scratch: block r < row_blocks computes row r of
// dx; the blocks after them take 32 columns of dgain each, their warps sharing the
// rows, from dy and total again (which L2 then holds).  Where dx is total itself, dgain's
// blocks are a launch of their own before the rows': nothing orders the blocks of one
// launch, and these read what the rows' blocks write over.  Up to 256 rows and 2^20
// elements: beyond, the second reading costs more than a launch (229 x 1152 bf16: 5.1
// us against 6.4 in two launches; 500 x 1000: 9.0 against 5.4).
inline bool few_rows(int64_t rows, int64_t cols) {
    return rows <= 256 && rows * cols <= (1 << 20) && cols <= kRegisterTiles * kQTile;
}
template <typename T, bool VEC, int K>
__global__ void __launch_bounds__(1024) k_norm_grad_few(const NormGradArgs a, unsigned row_blocks, float* __restrict__ dgain) {
    __shared__ float red[32][33];
    const RowSlot<false> rs;
    if (blockIdx.x >= row_blocks) {
        const int64_t c = (int64_t)(blockIdx.x - row_blocks) * 32 + rs.lane;
        float t = 0.f;
        if (c < a.cols) {
#pragma unroll 8
            for (int64_t r = rs.w; r < a.rows; r += rs.W)
                t = fmaf(__ldg(a.dy + r * a.cols + c),
                         to_f32(static_cast<const T*>(a.total)[r * a.cols + c]) * __ldg(a.rstd + r), t);
        }
        red[rs.w][rs.lane] = t;
        __syncthreads();
        if (rs.w == 0 && c < a.cols) {
            for (int i = 1; i < rs.W; ++i) t += red[i][rs.lane];
            dgain[c] = t;
        }
        return;
    }
    const int c0 = rs.w * K * kQTile, left = (int)a.cols - c0, c = c0 + lane_col<VEC>(rs.lane);
    const int64_t e = (int64_t)blockIdx.x * a.cols + c;
    const float rstd = __ldg(a.rstd + blockIdx.x);
    F8 g[K], n[K], add[K], dots;
    dots.clear();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int l = left - k * kQTile;
        load_tile<float, VEC>(a.dy + e + k * kQTile, l, rs.lane, g[k]);
        load_tile<T, VEC>((const T*)a.total + e + k * kQTile, l, rs.lane, n[k]);
        if (a.dtotal) load_tile<T, VEC>((const T*)a.dtotal + e + k * kQTile, l, rs.lane, add[k]);
        F8 w;
        load_tile<float, VEC>(a.gain + c + k * kQTile, l, rs.lane, w);
        n[k].mul(rstd);
        g[k].mul(w);
        dots.fma(g[k], n[k]);
    }
    const float mean = rs.sum(sum8(dots), red[0]) * a.inv_cols;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        n[k].mul(-mean);
        g[k].add(n[k]);
        g[k].mul(rstd);
        if (a.dtotal) g[k].add(add[k]);
        store_tile<T, VEC>((T*)a.dx + e + k * kQTile, left - k * kQTile, rs.lane, g[k]);
    }
}

// Rows of any length; the gain's partial sums live in the block's scratch row.
template <typename T, bool VEC>
__global__ void __launch_bounds__(1024) k_norm_grad_long(const NormGradArgs a) {
    __shared__ float red[2][32];
    const RowSlot<false> rs;
    const int lc = lane_col<VEC>(rs.lane);
    int turn = 0;
    for (int64_t r = blockIdx.x; r < a.rows; r += gridDim.x, turn ^= 1) {
        const float rstd = __ldg(a.rstd + r);
        const bool first = r == blockIdx.x;
        const int64_t row = r * a.cols;
        auto load = [&](int64_t c0, int left, F8& g, F8& n, F8& w) {
            load_tile<float, VEC>(a.dy + row + c0 + lc, left, rs.lane, g);
            load_tile<T, VEC>((const T*)a.total + row + c0 + lc, left, rs.lane, n);
            load_tile<float, VEC>(a.gain + c0 + lc, left, rs.lane, w);
            n.mul(rstd);
        };
        float dot = 0.f;
        for (int64_t c0 = rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
            const int left = (int)(a.cols - c0);
            F8 g, n, w, d;
            load(c0, left, g, n, w);
            if (a.part) {
                float* dst = a.part + blockIdx.x * a.cols + c0 + lc;
                d.clear();
                if (!first) load_tile<float, VEC>(dst, left, rs.lane, d);
                d.fma(g, n);
                store_tile<float, VEC>(dst, left, rs.lane, d);
            }
            d.clear();
            g.mul(w);
            d.fma(g, n);
            dot += sum8(d);
        }
        const float mean = rs.sum(dot, red[turn]) * a.inv_cols;
        for (int64_t c0 = rs.w * kQTile; c0 < a.cols; c0 += 32 * kQTile) {
            const int left = (int)(a.cols - c0);
            F8 g, n, w;
            load(c0, left, g, n, w);
            g.mul(w);
            n.mul(-mean);
            g.add(n);
            g.mul(rstd);
            if (a.dtotal) {
                load_tile<T, VEC>((const T*)a.dtotal + row + c0 + lc, left, rs.lane, w);
                g.add(w);
            }
            store_tile<T, VEC>((T*)a.dx + row + c0 + lc, left, rs.lane, g);
        }
    }
}

// dgain[c] = the blocks' partial sums of column c.  C columns per block: 1024 / C
// threads share a column's n sums, a shuffle tree adds theirs.  8 columns (one
// sector) where there are many sums per column, so that a thread has few loads
// one after another; else 32.
template <int C>
__global__ void __launch_bounds__(1024) k_dgain_sum(const float* __restrict__ part, int n, int64_t cols,
                                                    float* __restrict__ dgain) {
    constexpr int Y = 1024 / C;
    __shared__ float sm[Y][C + 1];
    const int x = threadIdx.x % C, y = threadIdx.x / C, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * C + x;
    float t = 0.f;
    if (c < cols) {
#pragma unroll 10
        for (int i = y; i < n; i += Y) t += part[(int64_t)i * cols + c];
    }
    sm[y][x] = t;
    __syncthreads();
    if (warp < C) {
        t = 0.f;
#pragma unroll
        for (int k = lane; k < Y; k += 32) t += sm[k][warp];
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        const int64_t cw = (int64_t)blockIdx.x * C + warp;
        if (lane == 0 && cw < cols) dgain[cw] = t;
    }
}

template <typename F>
bool allow_smem(F fn, size_t bytes) {
    return bytes <= 32 * 1024 ||   // the kernels have static arrays beside it
           cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) == cudaSuccess;
}

constexpr size_t kSmSmem = 227 * 1024;   // shared memory of an SM that blocks can take
constexpr int64_t kSms = 152;

// Blocks of the kernel that an SM holds at once.
template <typename F>
int64_t blocks_per_sm(F fn, int threads, size_t smem) {
    int n = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, fn, threads, smem) != cudaSuccess) cudaGetLastError();
    return std::max(1, n);
}

template <typename T, bool VEC, int K, bool ONE>
int launch_norm_k(const NormArgs& a, const RowShape& f, cudaStream_t s) {
    const int threads = f.threads();
    if constexpr (VEC) {
        const size_t smem = (size_t)2 * (a.residual ? 2 : 1) * K * Ring<T>::kUnits * 16 * threads;
        // Rows in flight pay for one warp's rows and for two tiles per warp (768
        // bf16 columns: 33 us a training batch against 39; 10000: 33 against
        // 54), not for one tile per warp (5000 fp32 columns: 48 against 41),
        // given rows for more than one turn of every slot and room for two stages.
        if ((ONE || K == 2) && smem <= kSmSmem - 8192 && a.rows >= 2 * kSms * f.slots()) {
            auto fn = k_norm_ring<T, K, ONE>;
            if (!allow_smem(fn, smem)) return SNK_ERR_CUDA;
            const int64_t bps = blocks_per_sm(fn, threads, smem);
            const int64_t turns = ceil_div(a.rows, kSms * bps * f.slots());
            fn<<<(unsigned)ceil_div(a.rows, turns * f.slots()), threads, smem, s>>>(a);
            return SNK_OK;
        }
    }
    k_norm<T, VEC, K, ONE><<<(unsigned)ceil_div(a.rows, f.slots()), threads, 0, s>>>(a);
    return SNK_OK;
}

template <typename T, bool VEC>
int launch_norm(const NormArgs& a, cudaStream_t s) {
    const int64_t tpr = ceil_div(a.cols, kQTile);
    int st = SNK_OK;
    if (tpr <= kRegisterTiles) {
        // few rows: one tile per warp, for the shortest time of a row; unaligned
        // ones too (their 8 accesses per tile want warps, not registers)
        const RowShape f = row_shape(tpr, VEC && a.rows > 256 ? 3 : 1);
        if (!f.one()) {
            st = f.K == 1 ? launch_norm_k<T, VEC, 1, false>(a, f, s) : launch_norm_k<T, VEC, 2, false>(a, f, s);
        } else if constexpr (VEC) {
            st = f.K == 1   ? launch_norm_k<T, VEC, 1, true>(a, f, s)
                 : f.K == 2 ? launch_norm_k<T, VEC, 2, true>(a, f, s)
                            : launch_norm_k<T, VEC, 3, true>(a, f, s);
        } else {
            st = launch_norm_k<T, VEC, 1, true>(a, f, s);
        }
    } else {
        k_norm_long<T, VEC><<<(unsigned)a.rows, 1024, 0, s>>>(a);
    }
    return st != SNK_OK || cudaGetLastError() == cudaSuccess ? st : SNK_ERR_CUDA;
}

// Most blocks of the gradient kernel: a scratch row each.
constexpr int64_t kGradBlocks = 8 * kSms;

template <typename T, bool VEC, int K, bool ONE>
int launch_norm_grad_k(const NormGradArgs& a, const RowShape& f, int64_t* grid, cudaStream_t s) {
    const int threads = f.threads();
    const size_t sums = ONE ? (size_t)K * kQTile * sizeof(float) : 0;
    auto blocks = [&](int64_t bps) {   // blocks of equally many rows
        const int64_t turns = ceil_div(a.rows, std::min<int64_t>(kGradBlocks / kSms, bps) * kSms * f.slots());
        return ceil_div(a.rows, turns * f.slots());
    };
    if constexpr (VEC) {
        const size_t smem = (size_t)2 * K * (2 + (a.dtotal ? 2 : 1) * Ring<T>::kUnits) * 16 * threads + sums;
        if (smem <= kSmSmem - 8192 && a.rows >= 2 * kSms * f.slots()) {
            auto fn = k_norm_grad<T, true, K, ONE, true>;
            if (!allow_smem(fn, smem)) return SNK_ERR_CUDA;
            *grid = blocks(blocks_per_sm(fn, threads, smem));
            fn<<<(unsigned)*grid, threads, smem, s>>>(a);
            return SNK_OK;
        }
    }
    auto fn = k_norm_grad<T, VEC, K, ONE, false>;
    *grid = blocks(blocks_per_sm(fn, threads, sums));
    fn<<<(unsigned)*grid, threads, sums, s>>>(a);
    return SNK_OK;
}

template <typename T, bool VEC>
int launch_norm_grad(const NormGradArgs& a, float* dgain, cudaStream_t s) {
    const int64_t tpr = ceil_div(a.cols, kQTile);
    int64_t grid = 0;
    int st = SNK_OK;
    if (few_rows(a.rows, a.cols)) {
        // 8 or 32 warps at least, for the blocks of dgain
        const RowShape f = row_shape(tpr, 1);
        const unsigned threads = 32 * std::max(a.rows > 64 ? 32 : 8, f.W);
        const unsigned rows = (unsigned)a.rows, sums = dgain ? (unsigned)ceil_div(a.cols, 32) : 0;
        auto fn = f.K == 1 ? k_norm_grad_few<T, VEC, 1> : k_norm_grad_few<T, VEC, 2>;
        if (sums && a.dx == a.total) {
            fn<<<sums, threads, 0, s>>>(a, 0, dgain);
            fn<<<rows, threads, 0, s>>>(a, rows, dgain);
        } else {
            fn<<<rows + sums, threads, 0, s>>>(a, rows, dgain);
        }
        return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
    }
    if (tpr <= kRegisterTiles) {
        // one tile per warp (768 bf16 columns: 50 us a training batch, against 57
        // with the row's three in one warp, whose registers leave 16 warps per SM)
        const RowShape f = row_shape(tpr, 1);
        if (f.one()) st = launch_norm_grad_k<T, VEC, 1, true>(a, f, &grid, s);
        else if (f.K == 1) st = launch_norm_grad_k<T, VEC, 1, false>(a, f, &grid, s);
        else st = launch_norm_grad_k<T, VEC, 2, false>(a, f, &grid, s);
    } else {
        grid = std::min<int64_t>(2 * kSms, a.rows);
        k_norm_grad_long<T, VEC><<<(unsigned)grid, 1024, 0, s>>>(a);
    }
    if (st != SNK_OK || cudaGetLastError() != cudaSuccess) return SNK_ERR_CUDA;
    if (dgain) {
        if (grid > 320) k_dgain_sum<8><<<(unsigned)ceil_div(a.cols, 8), 1024, 0, s>>>(a.part, (int)grid, a.cols, dgain);
        else k_dgain_sum<32><<<(unsigned)ceil_div(a.cols, 32), 1024, 0, s>>>(a.part, (int)grid, a.cols, dgain);
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
    const NormArgs a{x, residual, gain, rows, cols, 1.f / (float)cols, eps, total, rstd,
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
    if (rows < 1 || cols < 1 || few_rows(rows, cols)) return 0;
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
    if (!dy || !total || !rstd || !gain || !dx) return SNK_ERR_ARG;
    if (dgain && !scratch && snk_rmsnorm_backward_scratch(rows, cols) > 0) return SNK_ERR_ARG;
    if (!q8_aligned(dy, 4) || !q8_aligned(total, e) || !q8_aligned(rstd, 4) || !q8_aligned(gain, 4) ||
        !q8_aligned(dtotal, e) || !q8_aligned(dx, e) || !q8_aligned(scratch, 32))
        return SNK_ERR_ARG;
    if (rows > INT32_MAX || cols > INT32_MAX) return SNK_ERR_LIMIT;
    const NormGradArgs a{dy, total, rstd, gain, dtotal, rows, cols, 1.f / (float)cols, dx, dgain ? (float*)scratch : nullptr};
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
