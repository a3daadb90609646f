// Products of a layer with few stored entries and an 8-bit X of many rows.
//
// The batch-tiled kernels take 64 rows at a time and give every SM a share of the
// entries; with a few thousand entries such a share is a handful, and each tile
// pays for its staging, its chunk tables and two launches (1023 x 1240 at 99%, b =
// 361: 120 us in six tiles).  Here the work is cut the other way, up to 256 batch
// rows at a time, on the transposed codes xt[c][rows], one byte each:
//   forward          a block per row of W and 128 batch rows; its 8 warps take runs
//                    of up to 32 of the row's entries, a lane 4 batch rows (one
//                    word of codes per entry)
//   weight gradient  a warp per 8 entries; the row's dY values stay in registers
//                    while the row lasts, a lane holding 4 batch rows of each 128
// Sums are fp32: a run's terms, then runs in order, then warps in order (forward);
// 8 terms per lane and a shuffle tree (weight gradient).
// Bound by launches and L2 latency: the codes are in * rows bytes.  Times beside
// those of the other paths stand at light_layer.
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <type_traits>

#include "snk_q8.cuh"

namespace snk {
namespace {

constexpr int kLightRows = 256;     // batch rows per pass, at most
constexpr int kLightWarps = 8;
constexpr int kLightEntries = 8;    // per warp of the weight gradient

// xt[c * cb + r] = code (r, c) and st[g * cb + r] = scale (r, g) for r < rows, zero
// up to cb.  Tiles of 32 rows x 128 columns.
__global__ void __launch_bounds__(256) k_light_x(const Q8In q, int rows, int cb, uint8_t* __restrict__ xt,
                                                 float* __restrict__ st) {
    __shared__ __align__(16) uint8_t tile[32][132];
    const int tx = threadIdx.x & 31, ty = threadIdx.x >> 5;
    const int64_t n = q.cols, c0 = (int64_t)blockIdx.x * 128;
    const int r0 = blockIdx.y * 32;
    const bool words = n % 4 == 0 && ((uintptr_t)q.codes & 3) == 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int r = r0 + ty + 8 * i;
        const int64_t c = c0 + 4 * tx;
        uint32_t w = 0;
        if (r < rows && c < n) {
            const uint8_t* p = q.codes + (int64_t)r * n + c;
            if (words) {
                w = __ldg(reinterpret_cast<const uint32_t*>(p));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (c + j < n) w |= (uint32_t)__ldg(p + j) << (8 * j);
            }
        }
        *reinterpret_cast<uint32_t*>(&tile[ty + 8 * i][4 * tx]) = w;
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        const int64_t c = c0 + ty + 8 * i;
        if (c < n && r0 + tx < cb) xt[c * cb + r0 + tx] = tile[tx][ty + 8 * i];
    }
    const int64_t groups = q.n_groups * cb;
    const int64_t id = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 256 + threadIdx.x;
    for (int64_t i = id; i < groups; i += (int64_t)gridDim.x * gridDim.y * 256) {
        const int64_t g = i / cb;
        const int r = (int)(i - g * cb);
        st[i] = r < rows ? __ldg(q.scales + (int64_t)r * q.n_groups + g) : 0.f;
    }
}

struct LightArgs {
    const int32_t* row_ptr;
    const int32_t* rows_of;   // row of each entry
    const int32_t* cols;
    const float* val;
    const uint8_t* xt;
    const float* st;
    int format, gshift, rows, cb;
    int64_t nnz, out_f;
    const float* bias;   // forward
    float* Y;            // [rows, out]
    const float* dY;     // weight gradient: [rows, out]
    float* dW;
    int accumulate;
    int64_t b_all;       // with db: the rows of the whole batch, from dY on
    float* db;           // or null
    unsigned blocks;     // blocks of the weight gradient; db's follow
};

// Values of 4 batch rows of column c from their codes (group scales applied unless
// ROW).
template <bool ROW>
__device__ __forceinline__ void light_decode(const LightArgs& a, uint32_t w, int c, int r, float2& x, float2& y) {
    q_values4(w, a.format, x, y);
    if constexpr (!ROW) {
        const float4 s = __ldg(reinterpret_cast<const float4*>(a.st + (int64_t)(c >> a.gshift) * a.cb + r));
        x = __fmul2_rn(x, make_float2(s.x, s.y));
        y = __fmul2_rn(y, make_float2(s.z, s.w));
    }
}
template <bool ROW>
__device__ __forceinline__ void light_values(const LightArgs& a, int c, int r, float2& x, float2& y) {
    light_decode<ROW>(a, __ldg(reinterpret_cast<const uint32_t*>(a.xt + (int64_t)c * a.cb + r)), c, r, x, y);
}

template <bool ROW>
__global__ void __launch_bounds__(32 * kLightWarps) k_light_forward(const LightArgs a) {
    __shared__ float4 part[kLightWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t o = blockIdx.x;
    const int r = blockIdx.y * 128 + 4 * lane;
    const int k0 = __ldg(a.row_ptr + o), k1 = __ldg(a.row_ptr + o + 1);
    const int r_in = r < a.cb ? r : 0;   // (lanes past cb read rows 0..3; their sums are not used)
    float2 tx = make_float2(0.f, 0.f), ty = tx;
    const int run = min(32, (k1 - k0 + kLightWarps - 1) / kLightWarps);
    for (int kb = k0 + warp * run; kb < k1; kb += kLightWarps * run) {
        const int n = min(run, k1 - kb);
        const int c_mine = lane < n ? __ldg(a.cols + kb + lane) : 0;
        const float w_mine = lane < n ? __ldg(a.val + kb + lane) : 0.f;
        float2 sx = make_float2(0.f, 0.f), sy = sx;
        // the codes (and scales) of 8 entries, or of 4 at a run's end, in flight
        // together; entries past the run read column 0 and are left out of the sum
        // (one at a time at the end: 67 us for 35 on rows as rank^-1.2, 1023 x 1240
        // at 99%, b = 361)
        auto take = [&](auto count, int i) {
            constexpr int N = decltype(count)::value;
            float2 x[N], y[N];
#pragma unroll
            for (int u = 0; u < N; ++u)
                light_values<ROW>(a, __shfl_sync(0xffffffffu, c_mine, i + u), r_in, x[u], y[u]);
#pragma unroll
            for (int u = 0; u < N; ++u) {
                const float w = __shfl_sync(0xffffffffu, w_mine, i + u);
                if (i + u < n) {
                    sx = __ffma2_rn(x[u], make_float2(w, w), sx);
                    sy = __ffma2_rn(y[u], make_float2(w, w), sy);
                }
            }
        };
        int i = 0;
        for (; n - i > 4; i += 8) take(std::integral_constant<int, 8>{}, i);
        if (i < n) take(std::integral_constant<int, 4>{}, i);
        tx = __fadd2_rn(tx, sx);
        ty = __fadd2_rn(ty, sy);
    }
    part[warp][lane] = make_float4(tx.x, tx.y, ty.x, ty.y);
    __syncthreads();
    // thread t < 128: batch row 128 blockIdx.y + t
    const int t = threadIdx.x, row = blockIdx.y * 128 + t;
    if (t < 128 && row < a.rows) {
        float y = 0.f;
#pragma unroll
        for (int i = 0; i < kLightWarps; ++i) y += reinterpret_cast<const float*>(&part[i][0])[t];
        // a row with no entries is its bias, whatever the scale
        if (ROW) y = k0 < k1 ? y * __ldg(a.st + row) : 0.f;
        a.Y[(int64_t)row * a.out_f + o] = y + (a.bias ? __ldg(a.bias + o) : 0.f);
    }
}

template <bool ROW>
__global__ void __launch_bounds__(256) k_light_weight(const LightArgs a) {
    const int lane = threadIdx.x & 31;
    if (blockIdx.x >= a.blocks) {   // db: 32 columns, the warps sharing the rows
        __shared__ float sm[8][33];
        const int y = threadIdx.x >> 5;
        const int64_t c = (int64_t)(blockIdx.x - a.blocks) * 32 + lane;
        float t = 0.f;
        if (c < a.out_f) {
            for (int64_t i0 = y; i0 < a.b_all; i0 += 256) {   // 32 terms to a running sum
                float u = 0.f;
                const int64_t i1 = min(a.b_all, i0 + 256);
#pragma unroll 8
                for (int64_t i = i0; i < i1; i += 8) u += __ldg(a.dY + i * a.out_f + c);
                t += u;
            }
        }
        sm[y][lane] = t;
        __syncthreads();
        if (y == 0 && c < a.out_f) {
            for (int i = 1; i < 8; ++i) t += sm[i][lane];
            a.db[c] = t;
        }
        return;
    }
    const int64_t e0 = ((int64_t)blockIdx.x * 8 + (threadIdx.x >> 5)) * kLightEntries;
    if (e0 >= a.nnz) return;
    const int n = (int)min((int64_t)kLightEntries, a.nnz - e0);
    constexpr int G = kLightRows / 128;
    const int c_mine = lane < n ? __ldg(a.cols + e0 + lane) : 0;
    const int r_mine = lane < n ? __ldg(a.rows_of + e0 + lane) : 0;
    // the codes of all entries are in flight together
    uint32_t w[kLightEntries][G];
#pragma unroll
    for (int i = 0; i < kLightEntries; ++i) {
        const int c = __shfl_sync(0xffffffffu, c_mine, i);
#pragma unroll
        for (int g = 0; g < G; ++g) {
            const int b0 = 128 * g + 4 * lane;
            w[i][g] = b0 < a.cb ? __ldg(reinterpret_cast<const uint32_t*>(a.xt + (int64_t)c * a.cb + b0)) : 0u;
        }
    }
    int row = -1;
    float2 dx[G], dy[G];
    float mine = 0.f;
#pragma unroll
    for (int i = 0; i < kLightEntries; ++i) {
        if (i < n) {
            const int r = __shfl_sync(0xffffffffu, r_mine, i);
            if (r != row) {
                row = r;
#pragma unroll
                for (int g = 0; g < G; ++g) {
                    const int b0 = 128 * g + 4 * lane;
                    float v[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        v[j] = b0 + j < a.rows ? __ldg(a.dY + (int64_t)(b0 + j) * a.out_f + r) : 0.f;
                        if (ROW && b0 + j < a.rows) v[j] *= __ldg(a.st + b0 + j);
                    }
                    dx[g] = make_float2(v[0], v[1]);
                    dy[g] = make_float2(v[2], v[3]);
                }
            }
            const int c = __shfl_sync(0xffffffffu, c_mine, i);
            float2 s = make_float2(0.f, 0.f);
#pragma unroll
            for (int g = 0; g < G; ++g) {
                const int b0 = 128 * g + 4 * lane;
                if (b0 < a.cb) {
                    float2 x, y;
                    light_decode<ROW>(a, w[i][g], c, b0, x, y);
                    s = __ffma2_rn(dy[g], y, __ffma2_rn(dx[g], x, s));
                }
            }
            float t = s.x + s.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane == i) mine = t;
        }
    }
    if (lane < n) a.dW[e0 + lane] = a.accumulate ? a.dW[e0 + lane] + mine : mine;
}

// The transposed codes and scales of batch rows [r0, r0 + rows), in the handle's
// operand space (256 bytes per column of the larger dimension): cb rows of codes
// for each column and, for group scales, cb scales for each group.
int light_operand(Layer* L, const Q8In& q, int64_t r0, int rows, LightArgs* a, cudaStream_t s) {
    a->rows = rows;
    a->cb = (int)ceil_div(rows, 32) * 32;
    a->format = q.format;
    a->gshift = q.gshift;
    uint8_t* base = reinterpret_cast<uint8_t*>(L->xt);
    a->xt = base;
    // (a scale per row needs no table)
    float* st = reinterpret_cast<float*>(base + (int64_t)L->in_f * a->cb);
    const Q8In qr = q.from_row(r0);
    Q8In src = qr;
    if (q.gshift == 31) {
        a->st = qr.scales;
        src.n_groups = 0;
    } else {
        a->st = st;
    }
    k_light_x<<<dim3((unsigned)ceil_div(L->in_f, 128), (unsigned)(a->cb / 32)), 256, 0, s>>>(src, rows, a->cb, base, st);
    a->row_ptr = L->row_ptr;
    a->rows_of = L->r;
    a->cols = L->c;
    a->val = L->v;
    a->nnz = L->nnz;
    a->out_f = L->out_f;
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

// Batch rows that fit there, a multiple of 32 (at least 192: a group has 32 columns
// or more, and the layer 64).
int64_t pass_rows(const Layer* L, const Q8In& q) {
    const int64_t table = q.gshift == 31 ? 0 : q.n_groups * (int64_t)sizeof(float);
    const int64_t space = std::max(L->out_f, L->in_f) * kMaxBatchTile * (int64_t)sizeof(float);
    return std::min<int64_t>(kLightRows, space / (L->in_f + table) / 32 * 32);
}
// Rows of the next pass where `left` are left: what no longer fits one pass but two of
// 128 runs as two of 128 (1000 x 3000 at 90% with groups, forward of 256 rows: 192 + 64
// take 61 us, the second pass costs as much as one of 128).
int64_t next_pass(int64_t step, int64_t left) {
    if (left <= step) return left;
    return step >= 128 && left <= 256 ? 128 : step;
}

}  // namespace

// More than one 64-row tile, and few enough entries (measured, us, this path
// against the others): forward, 1000 x 1000 at 90%, b = 128: 10 against 48; 5000 x
// 5000 at 99.5%, b = 128: 16 against 27; 3000 x 1000 at 90% (300,000 entries), b = 70:
// 18 against 18, with group scales 23 against 19 (24 against 22 at b = 96, 3072 x 768
// 20 against 30: more entries from there).  Weight gradient, 768 x 3072 at
// 99%, b = 128: 11 against 30; 500 x 500 at 80% (50,000 entries), b = 70: 12 against
// 14; 1000 x 1000 at 90% (100,000), b = 70: 17 against 15.  Where the tensor cores
// take the layer, whose time hardly grows with the batch, the work is limited too.
bool light_layer(const Layer* L, const Q8In& q, int64_t b, bool weight) {
    if (L->nnz == 0 || b <= 64 || L->in_f < 64) return false;
    const bool tc = tc_eligible(L, q, b, weight);
    if (L->nnz > (weight ? 65536 : (b >= 96 || q.gshift == 31) ? 400000 : 131072)) return false;
    const char* f = getenv("SNK_LARGE_BATCH");   // forces one of the other two
    if (f && (strcmp(f, "on") == 0 || strcmp(f, "off") == 0)) return false;
    return !tc || L->nnz * b <= (weight ? 16000000 : 80000000);
}

int light_forward(Layer* L, const Q8In& q, int64_t b, const float* bias, float* Y, cudaStream_t s) {
    const int64_t step = pass_rows(L, q);
    for (int64_t r0 = 0, rows; r0 < b; r0 += rows) {
        rows = next_pass(step, b - r0);
        LightArgs a{};
        if (int st = light_operand(L, q, r0, (int)rows, &a, s); st != SNK_OK) return st;
        a.bias = bias;
        a.Y = Y + r0 * L->out_f;
        const dim3 grid((unsigned)L->out_f, (unsigned)ceil_div(rows, 128));
        if (q.gshift == 31) k_light_forward<true><<<grid, 32 * kLightWarps, 0, s>>>(a);
        else k_light_forward<false><<<grid, 32 * kLightWarps, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SNK_ERR_CUDA;
    }
    return SNK_OK;
}

int light_weight(Layer* L, const Q8In& q, const float* dY, int64_t b, float* dW, float* db, cudaStream_t s) {
    const int64_t step = pass_rows(L, q);
    for (int64_t r0 = 0, rows; r0 < b; r0 += rows) {
        rows = next_pass(step, b - r0);
        LightArgs a{};
        if (int st = light_operand(L, q, r0, (int)rows, &a, s); st != SNK_OK) return st;
        a.dY = dY + r0 * L->out_f;
        a.dW = dW;
        a.accumulate = r0 > 0;
        a.blocks = (unsigned)ceil_div(L->nnz, 8 * kLightEntries);
        a.db = r0 == 0 ? db : nullptr;
        a.b_all = b;
        const unsigned grid = a.blocks + (a.db ? (unsigned)ceil_div(L->out_f, 32) : 0);
        if (q.gshift == 31) k_light_weight<true><<<grid, 256, 0, s>>>(a);
        else k_light_weight<false><<<grid, 256, 0, s>>>(a);
        if (cudaGetLastError() != cudaSuccess) return SNK_ERR_CUDA;
    }
    return SNK_OK;
}

}  // namespace snk
