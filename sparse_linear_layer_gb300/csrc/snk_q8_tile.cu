// 8-bit forms of a matrix that need tiles of 128 x 128: codes with scales along the
// columns and, transposed, along the rows (what the three products of a dense layer's
// training step take), the column sums, and codes with one scale for each block.
//
// A block of threads takes a tile: its values go into shared memory once, rows and columns are
// packed from there.  Bound by memory: every element is read once and
// written as one byte per form.
//
// A wait for a tile that runs out (kTcWaitCycles) leaves NaN, in the scales and sums of what
// the waiting thread reads of this tile and of all that follow.  The thread that brings the tiles
// then brings no more, so that nothing comes to a place whose last copy may still be on its way,
// and waits at its end, with kTcDrainCycles, for the copies that it has started.
#include <algorithm>
#include <type_traits>

#include "snk_q8.cuh"
#include "snk_tcgen.cuh"

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

// How a tile comes in: by TMA, the next one while this one is worked on (16-bit types; of
// 32-bit ones a block holds one, and two blocks take turns on an SM), or, where rows are not
// whole 16-byte chunks, by plain loads.
enum TileLoad { kTileTma, kTilePlain };
template <typename T, TileLoad LOAD>
constexpr int kTileBuffers = LOAD == kTileTma && sizeof(T) == 2 ? 2 : 1;
// The tiles, and a tile's codes along the rows (turned there, so that a column's 128 bytes leave
// together: as 32-byte stores of 32 columns the training step's packs took 2.3 times as long).
template <typename T, TileLoad LOAD>
constexpr int kTileSmem = kTile * kTile * (kTileBuffers<T, LOAD> * (int)sizeof(T) + 1) + 128;

// BLOCKS: one scale for the whole tile.
template <typename T, bool BLOCKS, TileLoad LOAD>
__global__ void __launch_bounds__(kTileThreads, 2) k_q8_tile(const __grid_constant__ CUtensorMap map, const TileArgs a) {
    // along the rows, a thread takes a word (CW columns) of RT rows; every access to the tile is then
    // of consecutive words by the lanes of a warp
    constexpr int CW = 4 / (int)sizeof(T), WORDS = kTile / CW, RT = kTile * WORDS / kTileThreads;
    constexpr int BUFS = kTileBuffers<T, LOAD>, BYTES = kTile * kTile * (int)sizeof(T);
    extern __shared__ __align__(128) unsigned char tile_raw[];
    unsigned char* tiles = tile_raw + ((128 - (smem_u32(tile_raw) & 127)) & 127);
    unsigned char* turned = tiles + BUFS * BYTES;   // [column][16-byte chunk of rows, exclusive-or (column / CW) % 8]
    __shared__ float most_s[CW][kTileThreads], sums_s[CW][kTileThreads];
    __shared__ uint64_t full[BUFS];
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t n_tiles = a.tiles_r * a.tiles_c;
    after_previous();
    let_next_start();
    auto fetch = [&](int64_t id, int b) {
        const int64_t tr = id / a.tiles_c, tc = id - tr * a.tiles_c;
        mbar_expect_tx(&full[b], BYTES);
        tma_load_2d(tiles + b * BYTES, &map, (int)(tc * kTile), (int)(tr * kTile), &full[b]);
    };
    if constexpr (LOAD == kTileTma) {
        if (t == 0) {
            for (int b = 0; b < BUFS; ++b) mbar_init(&full[b], 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            for (int b = 0; b < BUFS; ++b)
                if (blockIdx.x + (int64_t)b * gridDim.x < n_tiles) fetch(blockIdx.x + (int64_t)b * gridDim.x, b);
        }
        __syncthreads();
    }
    int buf = 0;
    uint32_t parity = 0;
    bool ok = true;     // no wait of this thread's has run out
    int64_t lost = 0;   // else the tile that it waited for
    for (int64_t id = blockIdx.x; id < n_tiles; id += gridDim.x) {
        const int64_t tr = id / a.tiles_c, tc = id - tr * a.tiles_c;
        const int64_t r0 = tr * kTile, c0 = tc * kTile;
        const int nr = (int)min((int64_t)kTile, a.rows - r0), nc = (int)min((int64_t)kTile, a.cols - c0);
        T* sm = reinterpret_cast<T*>(tiles + buf * BYTES);
        float most = 0.f;
        if constexpr (LOAD == kTileTma) {
            if (ok && !mbar_wait(&full[buf], parity)) {
                ok = false;
                lost = id;
            }
        } else {
            const T* x = static_cast<const T*>(a.x) + r0 * a.cols + c0;
#pragma unroll 4
            for (int r = warp; r < kTile; r += kTileThreads / 32) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sm[r * kTile + lane + 32 * j] = r < nr && lane + 32 * j < nc ? x[r * a.cols + lane + 32 * j] : from_f32<T>(0.f);
            }
            __syncthreads();
        }
        if (!ok) most = __int_as_float(0x7fc00000);
        // ---- along the columns: a warp's 16 rows, four columns a lane
        uint8_t* row_codes = a.codes + r0 * a.ld + c0 + 4 * lane;
        const bool words = a.ld % 4 == 0 && ((uintptr_t)a.codes & 3) == 0 && 4 * lane + 4 <= nc;
        auto read4 = [&](int r, float2& p, float2& q) {
            if constexpr (sizeof(T) == 4) {
                const float4 f = *reinterpret_cast<const float4*>(sm + r * kTile + 4 * lane);
                p = make_float2(f.x, f.y);
                q = make_float2(f.z, f.w);
            } else {
                const uint2 w = *reinterpret_cast<const uint2*>(sm + r * kTile + 4 * lane);
                p = unpack2<T>(w.x);
                q = unpack2<T>(w.y);
            }
        };
        auto write4 = [&](int r, float2 p, float2 q, float inv) {
            const float2 i2 = make_float2(inv, inv);
            uint32_t w = q_codes4(__fmul2_rn(p, i2), __fmul2_rn(q, i2), SNK_Q8_E4M3);
            if (inv == 0.f) w = 0;
            if (r >= nr) return;
            uint8_t* out = row_codes + r * a.ld;
            if (words) {
                *reinterpret_cast<uint32_t*>(out) = w;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (4 * lane + j < nc) out[j] = (uint8_t)(w >> (8 * j));
            }
        };
        if constexpr (BLOCKS) {
#pragma unroll 4
            for (int i = 0; i < 16; ++i) {
                float2 p, q;
                read4(warp * 16 + i, p, q);
                most = max_abs(max_abs(most, p.x, p.y), q.x, q.y);
            }
        } else if (a.codes) {
            // lane i (and i + 16) finds the scale of row i, once for the warp's 16 rows
            float m = 0.f;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float2 p, q;
                read4(warp * 16 + i, p, q);
                const float r = warp_amax(max_abs(max_abs(most, p.x, p.y), q.x, q.y));
                if ((lane & 15) == i) m = r;
            }
            const QScale s = q_scale(m, SNK_Q8_E4M3);
            if (lane < 16 && warp * 16 + lane < nr) a.scales[(r0 + warp * 16 + lane) * a.tiles_c + tc] = s.scale;
#pragma unroll
            for (int i = 0; i < 16; ++i) {
                float2 p, q;
                read4(warp * 16 + i, p, q);
                write4(warp * 16 + i, p, q, __shfl_sync(0xffffffffu, s.inv, i));
            }
        }
        QScale block{0.f, 0.f};
        if constexpr (BLOCKS) {
            most = warp_amax(most);
            if (lane == 0) most_s[0][warp] = most;
            __syncthreads();
            most = most_s[0][lane & 7];
            most = warp_amax(most);
            block = q_scale(most, SNK_Q8_E4M3);
            if (t == 0) {
                if (a.scales) a.scales[tr * a.tiles_c + tc] = block.scale;
                if (a.scales_t) a.scales_t[tc * a.tiles_r + tr] = block.scale;
            }
            if (a.codes) {
#pragma unroll 4
                for (int i = 0; i < 16; ++i) {
                    float2 p, q;
                    read4(warp * 16 + i, p, q);
                    write4(warp * 16 + i, p, q, block.inv);
                }
            }
        }
        // ---- along the rows
        if (a.codes_t || a.part) {
            const int word = t % WORDS, h = t / WORDS;   // rows h RT .. + RT - 1
            const uint32_t* col = reinterpret_cast<const uint32_t*>(sm) + h * RT * WORDS + word;
            uint32_t raw[RT];
#pragma unroll
            for (int i = 0; i < RT; ++i) raw[i] = col[i * WORDS];
            auto value = [&](int i, int k) {
                if constexpr (CW == 1) return __uint_as_float(raw[i]);
                else return k ? unpack2<T>(raw[i]).y : unpack2<T>(raw[i]).x;
            };
            QScale q[CW];
#pragma unroll
            for (int k = 0; k < CW; ++k) q[k] = block;
            if constexpr (!BLOCKS) {
#pragma unroll
                for (int k = 0; k < CW; ++k) {
                    float m = ok ? 0.f : __int_as_float(0x7fc00000), s = 0.f;
#pragma unroll
                    for (int i = 0; i < RT; i += 2) m = max_abs(m, value(i, k), value(i + 1, k));
                    if (a.part) {
#pragma unroll
                        for (int i = 0; i < RT; i += 2) s += value(i, k) + value(i + 1, k);
                    }
                    most_s[k][t] = m;
                    sums_s[k][t] = s;
                }
                __syncthreads();
#pragma unroll
                for (int k = 0; k < CW; ++k) {
                    float m = 0.f, s = 0.f;
#pragma unroll
                    for (int u = word; u < kTileThreads; u += WORDS) {
                        m = max_nan(m, most_s[k][u]);
                        s += sums_s[k][u];
                    }
                    q[k] = q_scale(m, SNK_Q8_E4M3);
                    const int c = word * CW + k;
                    if (h == 0 && c < nc) {
                        if (a.codes_t) a.scales_t[(c0 + c) * a.tiles_r + tr] = q[k].scale;
                        if (a.part) a.part[tr * a.cols + c0 + c] = m == m ? s : m;   // (a wait ran out, or a value is NaN)
                    }
                }
            }
            if (a.codes_t) {
#pragma unroll
                for (int k = 0; k < CW; ++k) {
                    unsigned char* out = turned + (word * CW + k) * kTile;
#pragma unroll
                    for (int b = 0; b < RT; b += 16) {
                        uint32_t w[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int r = b + 4 * i;
                            const float2 i2 = make_float2(q[k].inv, q[k].inv);
                            w[i] = q_codes4(__fmul2_rn(make_float2(value(r, k), value(r + 1, k)), i2),
                                            __fmul2_rn(make_float2(value(r + 2, k), value(r + 3, k)), i2), SNK_Q8_E4M3);
                            if (q[k].inv == 0.f) w[i] = 0;
                        }
                        *reinterpret_cast<uint4*>(out + 16 * (((h * RT + b) / 16) ^ (word & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
                    }
                }
                __syncthreads();
                uint8_t* to = a.codes_t + c0 * a.ld_t + r0;
                if (a.ld_t % 16 == 0 && ((uintptr_t)a.codes_t & 15) == 0) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int c = (t + kTileThreads * i) >> 3, chunk = t & 7;
                        const unsigned char* from = turned + c * kTile + 16 * (chunk ^ ((c / CW) & 7));
                        if (c >= nc || 16 * chunk >= nr) continue;
                        if (16 * chunk + 16 <= nr) {
                            *reinterpret_cast<uint4*>(to + c * a.ld_t + 16 * chunk) = *reinterpret_cast<const uint4*>(from);
                        } else {
                            for (int k = 0; k < nr - 16 * chunk; ++k) to[c * a.ld_t + 16 * chunk + k] = from[k];
                        }
                    }
                } else {
                    for (int c = warp; c < nc; c += kTileThreads / 32) {
#pragma unroll
                        for (int r = lane; r < kTile; r += 32)
                            if (r < nr) to[c * a.ld_t + r] = turned[c * kTile + 16 * ((r >> 4) ^ ((c / CW) & 7)) + (r & 15)];
                    }
                }
            }
        }
        __syncthreads();   // the tile and the exchanged maxima are free
        if constexpr (LOAD == kTileTma) {
            if (t == 0 && ok && id + (int64_t)BUFS * gridDim.x < n_tiles) fetch(id + (int64_t)BUFS * gridDim.x, buf);
            if (++buf == BUFS) {
                buf = 0;
                parity ^= 1;
            }
        }
    }
    if constexpr (LOAD == kTileTma) {
        if (t == 0 && !ok) {
            for (int b = 0; b < BUFS && lost < n_tiles; ++b, lost += gridDim.x) {
                const uint32_t j = (uint32_t)((lost - blockIdx.x) / gridDim.x);   // the block's how manieth
                mbar_wait(&full[j % BUFS], (j / BUFS) & 1, kTcDrainCycles);
            }
        }
    }
}

// sums[c] = the parts of column c, in order.
__global__ void __launch_bounds__(256) k_q8_sums(const float* __restrict__ part, int64_t tiles, int64_t cols, float* __restrict__ sums) {
    __shared__ float sm[8][33];
    after_previous();
    let_next_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t c = (int64_t)blockIdx.x * 32 + lane;
    float s = 0.f;
    if (c < cols)
#pragma unroll 8
        for (int64_t i = warp; i < tiles; i += 8) s += __ldg(part + i * cols + c);
    sm[warp][lane] = s;
    __syncthreads();
    if (warp == 0 && c < cols) {
#pragma unroll
        for (int i = 1; i < 8; ++i) s += sm[i][lane];
        sums[c] = s;
    }
}

template <typename T, bool BLOCKS, TileLoad LOAD>
int launch_tile(const CUtensorMap& map, const TileArgs& a, int num_sms, cudaStream_t s) {
    constexpr auto f = k_q8_tile<T, BLOCKS, LOAD>;
    if (!allow_smem<f>(kTileSmem<T, LOAD>)) return SNK_ERR_CUDA;
    const unsigned blocks = (unsigned)std::min<int64_t>(a.tiles_r * a.tiles_c, 2 * num_sms);
    return launch_after(f, blocks, kTileThreads, kTileSmem<T, LOAD>, 1, s, map, a);
}
template <typename T>
int launch_tile(const TileArgs& a, bool blocks, cudaStream_t s) {
    const int n = device_sms();
    if (n < 1) return SNK_ERR_CUDA;
    CUtensorMap map = {};
    if (a.cols * sizeof(T) % 16 || ((uintptr_t)a.x & 15))
        return blocks ? launch_tile<T, true, kTilePlain>(map, a, n, s) : launch_tile<T, false, kTilePlain>(map, a, n, s);
    EncodeTiledFn fn = encoder();
    const CUtensorMapDataType type = sizeof(T) == 4                     ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
                                     : std::is_same<T, __half>::value ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                                        : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;
    cuuint64_t dims[2] = {(cuuint64_t)a.cols, (cuuint64_t)a.rows}, strides[1] = {(cuuint64_t)a.cols * sizeof(T)};
    cuuint32_t box[2] = {kTile, kTile}, estr[2] = {1, 1};
    if (!fn || fn(&map, type, 2, const_cast<void*>(a.x), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return SNK_ERR_CUDA;
    return blocks ? launch_tile<T, true, kTileTma>(map, a, n, s) : launch_tile<T, false, kTileTma>(map, a, n, s);
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
    return launch_after(k_q8_sums, (unsigned)ceil_div(cols, 32), 256, 0, 1, s, a.part, a.tiles_r, cols, sums);
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
