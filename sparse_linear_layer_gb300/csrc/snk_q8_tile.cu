// 8-bit forms of a matrix that need tiles of 128 x 128: codes with scales along the
// columns and, transposed, along the rows (what the three products of a dense layer's
// training step take), the column sums, and codes with one scale for each block.
//
// A block of threads takes a tile: its values go into shared memory once, rows are packed
// on the way in, columns from there.  Bound by memory: every element is read once and
// written as one byte per form.
#include <algorithm>

#include "snk_q8.cuh"

namespace snk {
namespace {

constexpr int kTile = 128;
constexpr int kTileThreads = 256;

struct TileArgs {
    const void* x;
    int64_t rows, cols;
    int64_t tiles_r, tiles_c;
    uint8_t *codes, *codes_t;      // [rows, cols] at stride ld; [cols, rows] at stride ld_t; either may be null
    int64_t ld, ld_t;
    float *scales, *scales_t;      // [rows, tiles_c]; [cols, tiles_r]; blocks: [tiles_r, tiles_c]; [tiles_c, tiles_r]
    float* part;                   // [tiles_r, cols] sums of the tile's columns, or null
};

// Pitch of a tile's row in shared memory: columns lie in different banks.
template <typename T>
constexpr int kPitch = sizeof(T) == 4 ? kTile + 1 : kTile + 2;
template <typename T>
constexpr int kTileSmem = kTile * kPitch<T> * (int)sizeof(T);

// BLOCKS: one scale for the whole tile.  VEC: rows are read four columns a lane.
template <typename T, bool BLOCKS, bool VEC>
__global__ void __launch_bounds__(kTileThreads) k_q8_tile(const TileArgs a) {
    extern __shared__ __align__(16) unsigned char tile_raw[];
    T* sm = reinterpret_cast<T*>(tile_raw);
    __shared__ float most_s[kTileThreads];
    __shared__ float sums_s[kTile];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    for (int64_t id = blockIdx.x; id < a.tiles_r * a.tiles_c; id += gridDim.x) {
        const int64_t tr = id / a.tiles_c, tc = id - tr * a.tiles_c;
        const int64_t r0 = tr * kTile, c0 = tc * kTile;
        const int nr = (int)min((int64_t)kTile, a.rows - r0), nc = (int)min((int64_t)kTile, a.cols - c0);
        const T* x = static_cast<const T*>(a.x) + r0 * a.cols + c0;
        float most = 0.f;
        // ---- in: a warp's 16 rows, 8 in flight
#pragma unroll
        for (int b = 0; b < 2; ++b) {
            float v[8][4];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = warp * 16 + b * 8 + i;
                if (VEC) {
                    const int c = 4 * lane;
                    if (r < nr && c < nc) {   // (columns come in fours)
                        if constexpr (sizeof(T) == 4) {
                            const float4 f = __ldg(reinterpret_cast<const float4*>(x + r * a.cols + c));
                            v[i][0] = f.x;
                            v[i][1] = f.y;
                            v[i][2] = f.z;
                            v[i][3] = f.w;
                        } else {
                            const uint2 w = __ldg(reinterpret_cast<const uint2*>(x + r * a.cols + c));
                            const float2 p = unpack2<T>(w.x), q = unpack2<T>(w.y);
                            v[i][0] = p.x;
                            v[i][1] = p.y;
                            v[i][2] = q.x;
                            v[i][3] = q.y;
                        }
                    } else {
                        v[i][0] = v[i][1] = v[i][2] = v[i][3] = 0.f;
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j) v[i][j] = r < nr && lane + 32 * j < nc ? to_f32(x[r * a.cols + lane + 32 * j]) : 0.f;
                }
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = warp * 16 + b * 8 + i;
                float m = max_abs(max_abs(0.f, v[i][0], v[i][1]), v[i][2], v[i][3]);
#pragma unroll
                for (int j = 0; j < 4; ++j) sm[r * kPitch<T> + (VEC ? 4 * lane + j : lane + 32 * j)] = from_f32<T>(v[i][j]);
                if constexpr (BLOCKS) {
                    most = max_nan(most, m);
                } else if (a.codes) {
                    m = warp_amax(m);
                    const QScale q = q_scale(m, SNK_Q8_E4M3);
                    if (r < nr) {
                        uint8_t* out = a.codes + (r0 + r) * a.ld + c0;
                        uint32_t w = q_codes4(make_float2(__fmul_rn(v[i][0], q.inv), __fmul_rn(v[i][1], q.inv)),
                                              make_float2(__fmul_rn(v[i][2], q.inv), __fmul_rn(v[i][3], q.inv)), SNK_Q8_E4M3);
                        if (q.inv == 0.f) w = 0;
                        if (VEC) {
                            if (4 * lane < nc) *reinterpret_cast<uint32_t*>(out + 4 * lane) = w;
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (lane + 32 * j < nc) out[lane + 32 * j] = (uint8_t)(w >> (8 * j));
                        }
                        if (lane == 0) a.scales[(r0 + r) * a.tiles_c + tc] = q.scale;
                    }
                }
            }
        }
        QScale block{0.f, 0.f};
        if constexpr (BLOCKS) {
            most = warp_amax(most);
            if (lane == 0) most_s[warp] = most;
            __syncthreads();
            most = most_s[lane & 7];
            most = warp_amax(most);
            block = q_scale(most, SNK_Q8_E4M3);
            if (t == 0) {
                if (a.scales) a.scales[tr * a.tiles_c + tc] = block.scale;
                if (a.scales_t) a.scales_t[tc * a.tiles_r + tr] = block.scale;
            }
            if (a.codes) {
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    const int r = warp * 16 + i;
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        v[j] = __fmul_rn(to_f32(sm[r * kPitch<T> + (VEC ? 4 * lane + j : lane + 32 * j)]), block.inv);
                    uint32_t w = q_codes4(make_float2(v[0], v[1]), make_float2(v[2], v[3]), SNK_Q8_E4M3);
                    if (block.inv == 0.f) w = 0;
                    if (r < nr) {
                        uint8_t* out = a.codes + (r0 + r) * a.ld + c0;
                        if (VEC) {
                            if (4 * lane < nc) *reinterpret_cast<uint32_t*>(out + 4 * lane) = w;
                        } else {
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                if (lane + 32 * j < nc) out[lane + 32 * j] = (uint8_t)(w >> (8 * j));
                        }
                    }
                }
            }
        } else {
            __syncthreads();
        }
        // ---- out along the rows: a thread has half of a column
        if (a.codes_t || a.part) {
            const int c = t & (kTile - 1), h = t >> 7;
            const T* col = sm + (h * 64) * kPitch<T> + c;
            QScale q = block;
            if (!BLOCKS || a.part) {
                float m = 0.f, s = 0.f;
#pragma unroll 8
                for (int i = 0; i < 64; i += 2) {
                    const float u = to_f32(col[i * kPitch<T>]), v = to_f32(col[(i + 1) * kPitch<T>]);
                    m = max_abs(m, u, v);
                    s += u + v;
                }
                if constexpr (!BLOCKS) {
                    most_s[t] = m;
                    if (h) sums_s[c] = s;
                    __syncthreads();
                    q = q_scale(max_nan(m, most_s[t ^ kTile]), SNK_Q8_E4M3);
                    if (!h && c < nc) {
                        if (a.codes_t) a.scales_t[(c0 + c) * a.tiles_r + tr] = q.scale;
                        if (a.part) a.part[tr * a.cols + c0 + c] = s + sums_s[c];
                    }
                }
            }
            if (a.codes_t && c < nc) {
                uint8_t* out = a.codes_t + (c0 + c) * a.ld_t + r0 + h * 64;
                const int left = nr - h * 64;
#pragma unroll
                for (int b = 0; b < 64; b += 32) {
                    uint32_t w[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const T* p = col + (b + 4 * k) * kPitch<T>;
                        w[k] = q_codes4(make_float2(__fmul_rn(to_f32(p[0]), q.inv), __fmul_rn(to_f32(p[kPitch<T>]), q.inv)),
                                        make_float2(__fmul_rn(to_f32(p[2 * kPitch<T>]), q.inv),
                                                    __fmul_rn(to_f32(p[3 * kPitch<T>]), q.inv)),
                                        SNK_Q8_E4M3);
                        if (q.inv == 0.f) w[k] = 0;
                    }
                    if (b + 32 <= left && ((uintptr_t)(out + b) & 31) == 0) {
                        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(out + b), "r"(w[0]), "r"(w[1]),
                                     "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                                     : "memory");
                    } else {
#pragma unroll
                        for (int k = 0; k < 32; ++k)
                            if (b + k < left) out[b + k] = (uint8_t)(w[k >> 2] >> (8 * (k & 3)));
                    }
                }
            }
        }
        __syncthreads();   // the tile and the exchanged maxima are free
    }
}

// sums[c] = the parts of column c, in order.
__global__ void __launch_bounds__(256) k_q8_sums(const float* __restrict__ part, int64_t tiles, int64_t cols, float* __restrict__ sums) {
    __shared__ float sm[8][33];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols)
        for (int64_t i = warp; i < tiles; i += 8) s += __ldg(part + i * cols + c);
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sm[i][lane];
        sums[c] = s;
    }
}

template <typename T, bool BLOCKS, bool VEC>
int launch_tile(const TileArgs& a, cudaStream_t s) {
    auto* f = k_q8_tile<T, BLOCKS, VEC>;
    if (cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kTileSmem<T>) != cudaSuccess) {
        cudaGetLastError();
        return SNK_ERR_CUDA;
    }
    const unsigned blocks = (unsigned)std::min<int64_t>(a.tiles_r * a.tiles_c, 1 << 20);
    f<<<blocks, kTileThreads, kTileSmem<T>, s>>>(a);
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}
template <typename T>
int launch_tile(const TileArgs& a, bool blocks, cudaStream_t s) {
    const bool vec = a.cols % 4 == 0 && ((uintptr_t)a.x & (4 * sizeof(T) - 1)) == 0 &&
                     (!a.codes || (a.ld % 4 == 0 && ((uintptr_t)a.codes & 3) == 0));
    if (blocks) return vec ? launch_tile<T, true, true>(a, s) : launch_tile<T, true, false>(a, s);
    return vec ? launch_tile<T, false, true>(a, s) : launch_tile<T, false, false>(a, s);
}
int run_tile(const TileArgs& a, int dtype, bool blocks, cudaStream_t s) {
    switch (dtype) {
        case SNK_F32: return launch_tile<float>(a, blocks, s);
        case SNK_F16: return launch_tile<__half>(a, blocks, s);
        default: return launch_tile<__nv_bfloat16>(a, blocks, s);
    }
}

int bad_tiles(const void* x, int dtype, int64_t rows, int64_t cols, const void* codes, int64_t ld, const float* scales,
              const void* codes_t, int64_t ld_t, const float* scales_t) {
    if (dtype < SNK_F32 || dtype > SNK_BF16 || rows < 0 || cols < 1) return SNK_ERR_ARG;
    if (rows >= INT32_MAX || cols >= INT32_MAX) return SNK_ERR_LIMIT;
    auto off = [](const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; };
    if (!codes != !scales || !codes_t != !scales_t || (codes && ld < cols) || (codes_t && ld_t < rows) ||
        off(x, dtype == SNK_F32 ? 4 : 2) || off(scales, 4) || off(scales_t, 4))
        return SNK_ERR_ARG;
    return SNK_OK;
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

int64_t snk_q8_pack_both_scratch(int64_t rows, int64_t cols) {
    return rows < 1 || cols < 1 || rows >= INT32_MAX || cols >= INT32_MAX ? 0 : 4 * ceil_div(rows, kTile) * cols;
}

int snk_q8_pack_both(const void* x, int dtype, int64_t rows, int64_t cols, void* codes, int64_t ld, float* scales, void* codes_t,
                     int64_t ld_t, float* scales_t, float* sums, void* scratch, void* stream) {
    if (int st = bad_tiles(x, dtype, rows, cols, codes, ld, scales, codes_t, ld_t, scales_t); st != SNK_OK) return st;
    if (((uintptr_t)sums & 3) || ((uintptr_t)scratch & 3)) return SNK_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0)
        return !sums || cudaMemsetAsync(sums, 0, (size_t)cols * 4, s) == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
    if (!x || (sums && !scratch)) return SNK_ERR_ARG;
    if (!codes && !codes_t && !sums) return SNK_OK;
    const TileArgs a{x, rows, cols, ceil_div(rows, kTile), ceil_div(cols, kTile), static_cast<uint8_t*>(codes),
                     static_cast<uint8_t*>(codes_t), ld, ld_t, scales, scales_t, sums ? static_cast<float*>(scratch) : nullptr};
    if (int st = run_tile(a, dtype, false, s); st != SNK_OK || !sums) return st;
    k_q8_sums<<<(unsigned)ceil_div(cols, 32), 256, 0, s>>>(a.part, a.tiles_r, cols, sums);
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

int snk_q8_pack_blocks(const void* w, int dtype, int64_t rows, int64_t cols, void* codes, int64_t ld, float* scales,
                       void* codes_t, int64_t ld_t, float* scales_t, void* stream) {
    if (int st = bad_tiles(w, dtype, rows, cols, codes, ld, scales, codes_t, ld_t, scales_t); st != SNK_OK) return st;
    if (rows == 0 || (!codes && !codes_t)) return SNK_OK;
    if (!w) return SNK_ERR_ARG;
    const TileArgs a{w, rows, cols, ceil_div(rows, kTile), ceil_div(cols, kTile), static_cast<uint8_t*>(codes),
                     static_cast<uint8_t*>(codes_t), ld, ld_t, scales, scales_t, nullptr};
    return run_tile(a, dtype, true, (cudaStream_t)stream);
}

}  // extern "C"
