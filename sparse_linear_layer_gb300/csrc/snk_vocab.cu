// Softmax cross entropy over a large vocabulary, loss and gradients, without the logits.
//
//   z = x W^T,  lse_r = log sum_v exp z_rv,  loss_r = lse_r - z_r,t(r)
//   dz_rv = g_r (exp(z_rv - lse_r) - [v = t(r)]),  dx = dz W,  dW = dz^T x
//
// x [rows, cols] and W [vocab, cols] are bf16 or fp16, everything else fp32.  A row whose
// target is `ignore` takes no part: its loss and dx are zero, and neither its x nor its
// upstream gradient reaches dW, whatever they hold.
//
// Four products (snk_dense.cuh), all tiles of 256 logits by 128 or 256 rows:
//   LseEpilogue    z, and for each row and half tile its largest logit and the sum of
//                  exp(z - largest): 8 bytes leave the SM for 128 logits; k_vocab_finish
//                  joins them and takes z_r,t as a dot product of its own
//   GradEpilogue   z once more, dz rounded to 16 bits for a piece of the vocabulary
//   SumEpilogue    dx += dz W over the piece, fp32, in ranges of kSumStages stages
//   StoreEpilogue  the piece's rows of dW = dz^T x, complete, turns of kSumStages stages
// The gradient's rows are gathered first (k_vocab_rows): the rows that count, side by
// side, zeros up to a whole tile; ignored rows then cost nothing, and the count stays on
// the device.  dz is held as c_r 2^13 (p - [v = t]), rounded to 16 bits, so that probabilities
// down to 2^-27 stay normal fp16 numbers.  For a sum or a mean c_r = 1 and the upstream gradient
// multiplies the finished products: the largest term of most rows, p - 1 with p small, then
// lies just below a power of two, where a rounding costs least, and not wherever g puts it (the
// gradients' errors against 64 bits are 1.00 to 1.17 of those of fp32 sums rounded to the same
// type, fp16 batches of 8192 rows 1.01; with a power of two near g in its place draws of 1.5 were seen).  For losses that go out
// row by row c_r = g_r / G, G the power of two next to the largest |g|.
#include <algorithm>

#include "snk_dense.cuh"

namespace snk {
namespace {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kGatherRows = 256;    // rows per block of k_vocab_rows at most
constexpr float kDzScale = 8192.f;  // 2^13
// Stages of an accumulator's turn in the loss: 64 MMA steps, whose additions truncate, towards
// zero. At 4096 columns one accumulator leaves the mean loss off by 1.2e-6 of it, turns of 32
// stages by 6e-7, of 16 by 2.9e-7 (768 columns, one turn: 1.7e-7); one accumulator and dual tiles
// would take 858 us for 2867 x 4096 x 65536, these take 946.  (Logits three times as large as there, 768 columns: 1.0e-6.)
constexpr int kTurnStages = 16;
// Stages that an accumulator adds at most in the gradients' products: 1024 MMA steps, 16384 rows of dW or
// columns of the vocabulary in dx.  What truncation takes off a sum of terms of one sign: 1.7e-4 of it
// after 256 stages, 3.5e-4 after 1024 (dW of 65536 rows in fp16: error 4.2e-4 where one rounding of the
// exact result is 2.2e-4; so 2.4e-4).  More rows of dW and wider rows' logits therefore take turns, and
// dx has ranges of K: 8192 x 768 -> 50257 1.3% of the step, 32768 rows 8%; 128 stages would take 4% and 8% for
// errors within 2% of a rounding's instead of 12%.
constexpr int kSumStages = 256;

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}
__device__ __forceinline__ float nan_f() { return __int_as_float(0x7fc00000); }

// ---- epilogues ------------------------------------------------------------------

struct LseEpilogue {
    struct Args {
        float2* part;    // [2 n_nt][ld]: largest logit (times log2 e) and sum of 2^(z log2 e - largest)
        int64_t ld;
        int64_t vocab;
    };
    template <class Source>
    __device__ static void run(const Args& a, const DenseTile& t, const Source& from) {
        const int lim = (int)min((int64_t)t.cols, a.vocab - t.col);   // (may be negative: nothing here)
        float m = __int_as_float(0xff800000), s = 0.f;
#pragma unroll
        for (int c = 0; c < kDenseN / 2; c += 32) {
            if (c >= lim) break;
            float v[32];
            from.get(c, t, v);
            if (c + 32 > lim) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (c + j >= lim) v[j] = __int_as_float(0xff800000);
            }
            float cm = m;
#pragma unroll
            for (int j = 0; j < 32; j += 2) cm = fmaxf(cm, fmaxf(v[j] * kLog2e, v[j + 1] * kLog2e));
            const float base = cm == __int_as_float(0xff800000) ? 0.f : cm;   // (all of them -inf: sums stay 0)
            float s0 = s * exp2_fast(m - base), s1 = 0.f, s2 = 0.f, s3 = 0.f;
#pragma unroll
            for (int j = 0; j < 32; j += 4) {
                s0 += exp2_fast(fmaf(v[j], kLog2e, -base));
                s1 += exp2_fast(fmaf(v[j + 1], kLog2e, -base));
                s2 += exp2_fast(fmaf(v[j + 2], kLog2e, -base));
                s3 += exp2_fast(fmaf(v[j + 3], kLog2e, -base));
            }
            s = (s0 + s1) + (s2 + s3);
            m = cm;
        }
        a.part[(int64_t)(2 * t.nt + t.half) * a.ld + t.row] = make_float2(m, s);
    }
};

// Eight fp32 values as 16-bit ones, and the 32-byte store of sixteen.
template <typename T>
__device__ __forceinline__ uint32_t two(float a, float b) { return pack2<T>(make_float2(a, b)); }
__device__ __forceinline__ void store32(void* p, const uint32_t (&w)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                 "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
}

// What dz is multiplied by, and the products of dz.
struct GradScale {
    const uint32_t* most;     // bits of the largest finite |g_r|
    const float* uniform;     // the upstream gradient of all rows, or null
    // Row by row: in() = 2^13 / G = 2^(139 - e), G the power of two above the largest finite |g|, e that one's
    // biased exponent (|g| < 2^(e - 126)), and out() = 2^(e - 139).  From e = 13 on both are normal numbers, for all
    // finite g; below (|g| < 2^-114) in() stays at 2^126, and |g in()| < 2^12.
    __device__ __forceinline__ uint32_t exponent() const { return max(__ldg(most) >> 23, 13u); }
    __device__ __forceinline__ float in() const { return uniform ? kDzScale : __uint_as_float((266 - exponent()) << 23); }
    __device__ __forceinline__ float out() const {
        return uniform ? __ldg(uniform) * (1.f / kDzScale) : __uint_as_float((exponent() - 12) << 23);
    }
};

template <typename T>
struct GradEpilogue {
    struct Args {
        T* dz;                    // [rows, ld]
        int64_t ld;
        int64_t width;            // columns of the piece that exist
        int64_t first;            // vocabulary index of its first column
        const float* lse2;        // [rows] log2 e times lse
        const float* g;           // [rows] factor of the row
        const int64_t* target;    // [rows]
        GradScale scale;
    };
    template <class Source>
    __device__ static void run(const Args& a, const DenseTile& t, const Source& from) {
        float c = 0.f, l2 = 0.f;
        int64_t at = -1;
        if (t.row < t.rows) {
            c = a.g[t.row] * a.scale.in();
            l2 = a.lse2[t.row];
            at = a.target[t.row] - a.first - t.col;
        }
        const int lim = (int)min((int64_t)t.cols, a.width - t.col);
        const int top = (int)min((int64_t)t.cols, a.ld - t.col);   // a multiple of 16
        T* out = a.dz + t.row * a.ld + t.col;
#pragma unroll
        for (int b = 0; b < kDenseN / 2; b += 32) {
            if (b >= top) break;
            float v[32];
            from.get(b, t, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = c * exp2_fast(fmaf(v[j], kLog2e, -l2));
            if (at >= b && at < b + 32) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (at == b + j) v[j] -= c;
            }
            if (b + 32 > lim) {
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (b + j >= lim) v[j] = 0.f;
            }
            if (t.row >= t.rows) {   // (its x is zero, but exp may overflow beside c = 0)
#pragma unroll
                for (int j = 0; j < 32; ++j) v[j] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = two<T>(v[j + 2 * i], v[j + 2 * i + 1]);
                if (b + j < top) store32(out + b + j, w);
            }
        }
    }
};

struct SumEpilogue {
    struct Args {
        float* slab;       // [splits][rows, ld]
        int64_t rows, ld;
        int add;           // to what is there
    };
    template <class Source>
    __device__ static void run(const Args& a, const DenseTile& t, const Source& from) {
        const int lim = (int)min((int64_t)t.cols, a.ld - t.col);   // (a multiple of 8)
        float* out = a.slab + ((int64_t)t.split * a.rows + t.row) * a.ld + t.col;
#pragma unroll
        for (int b = 0; b < kDenseN / 2; b += 32) {
            if (b >= lim) break;
            float v[32];
            from.get(b, t, v);
#pragma unroll
            for (int j = 0; j < 32; j += 8) {
                if (b + j < lim) {
                    F8 f;
#pragma unroll
                    for (int i = 0; i < 8; ++i) f.set(i, v[j + i]);
                    if (a.add) {
                        F8 o;
                        load8(out + b + j, o);
                        f.add(o);
                    }
                    store8(out + b + j, f);
                }
            }
        }
    }
};

template <typename T>
struct StoreEpilogue {
    struct Args {
        T* out;                  // [width, cols]
        int64_t width, cols;     // (cols a multiple of 8)
        GradScale scale;
        int vec;                 // elements per store: 16 or 8, by the rows' alignment
    };
    template <class Source>
    __device__ static void run(const Args& a, const DenseTile& t, const Source& from) {
        const int lim = t.row < a.width ? (int)min((int64_t)t.cols, a.cols - t.col) : 0;
        const float scale = a.scale.out();
        T* out = a.out + t.row * a.cols + t.col;
        const int top = (int)min((int64_t)t.cols, a.cols - t.col);   // the same in all lanes
#pragma unroll
        for (int b = 0; b < kDenseN / 2; b += 32) {
            if (b >= top) break;
            float v[32];
            from.get(b, t, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= scale;
#pragma unroll
            for (int j = 0; j < 32; j += 16) {
                uint32_t w[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i] = two<T>(v[j + 2 * i], v[j + 2 * i + 1]);
                if (a.vec == 16 && b + j + 16 <= lim) {
                    store32(out + b + j, w);
                } else {   // (lim is a multiple of 8 too)
                    if (b + j < lim) *reinterpret_cast<uint4*>(out + b + j) = make_uint4(w[0], w[1], w[2], w[3]);
                    if (b + j + 8 < lim) *reinterpret_cast<uint4*>(out + b + j + 8) = make_uint4(w[4], w[5], w[6], w[7]);
                }
            }
        }
    }
};

// ---- rows that count --------------------------------------------------------------

struct RowsArgs {
    const void* x;
    const int64_t* target;
    int64_t ignore;
    int64_t rows, cols, vocab, ld, padded;   // padded: rows of the gathered matrix
    void* xc;                         // [padded, ld] the rows that count, then zeros
    int32_t* index;                   // [rows] of the gathered row: its row of x
    int32_t* at;                      // [rows] of the row of x: its gathered row, or -1
    int64_t* tc;                      // [rows] its target
    int32_t* count;                   // how many
    // forward: what ignored rows get
    float* loss;                      // null: none
    float* lse_zero;
    // backward: upstream gradient, lse
    const float* lse;                 // [rows]
    const float* dloss;               // [rows] (reduction 0) or [1]
    int reduction;
    int per_block;                    // rows of a block
    float* lse2;                      // [rows]
    float* g;                         // [rows]
    uint32_t* most;                   // cleared before; the largest finite |g|'s bits
    float* uniform;                   // reductions 1, 2: the upstream gradient of every row (g is then 1)
};
// A block takes a.per_block rows; how many count before it and in all it finds out by itself:
// targets are 8 bytes a row, and the more rows there are the more a block takes (gather_rows), so
// that all blocks together read 4096 rows' worth for each row at most.
template <typename T>
__global__ void __launch_bounds__(256) k_vocab_rows(const RowsArgs a) {
    __shared__ int before_s[8], all_s[8], list[kGatherRows];
    __shared__ int mine_s;
    after_previous();
    let_next_start();
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int64_t r0 = (int64_t)blockIdx.x * a.per_block;
    int before = 0, all = 0;
#pragma unroll 4
    for (int64_t r = t; r < a.rows; r += 256) {
        const bool in = __ldg(a.target + r) != a.ignore;
        all += in;
        before += in && r < r0;
    }
    before = __reduce_add_sync(0xffffffffu, before);
    all = __reduce_add_sync(0xffffffffu, all);
    if (lane == 0) {
        before_s[warp] = before;
        all_s[warp] = all;
    }
    __syncthreads();
    before = all = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        before += before_s[i];
        all += all_s[i];
    }
    if (warp == 0) {   // this block's rows, in order
        int n = 0;
        uint32_t most = 0;
        for (int i = 0; i < a.per_block; i += 32) {
            const int64_t r = i + lane < a.per_block ? r0 + i + lane : a.rows;
            const int64_t tg = r < a.rows ? a.target[r] : a.ignore;
            const bool in = r < a.rows && tg != a.ignore;
            const uint32_t mask = __ballot_sync(0xffffffffu, in);
            const int k = n + __popc(mask & ((1u << lane) - 1));
            if (in) {
                list[k] = i + lane;
                const int64_t to = before + k;
                a.index[to] = (int32_t)r;
                a.tc[to] = tg;
                if (a.g) {
                    float g = a.reduction == 0 ? a.dloss[r] : 1.f;
                    if (tg < 0 || tg >= a.vocab) g = nan_f();
                    a.g[to] = g;
                    a.lse2[to] = a.lse[r] * kLog2e;
                    const uint32_t bits = __float_as_uint(g) & 0x7fffffffu;
                    if (bits < 0x7f800000u) most = max(most, bits);
                }
            }
            if (r < a.rows) {
                a.at[r] = in ? before + k : -1;
                if (!in && a.loss) a.loss[r] = 0.f;
                if (!in && a.lse_zero) a.lse_zero[r] = 0.f;
            }
            n += __popc(mask);
        }
        if (a.g) {
            most = __reduce_max_sync(0xffffffffu, most);
            if (lane == 0 && most) atomicMax(a.most, most);   // (a maximum: the same in any order)
        }
        if (lane == 0) {
            mine_s = n;
            if (blockIdx.x == 0) {
                *a.count = all;
                if (a.g && a.reduction) *a.uniform = all == 0 ? 0.f : (a.reduction == 2 ? a.dloss[0] / (float)all : a.dloss[0]);
            }
        }
    }
    __syncthreads();
    const int mine = mine_s;
    T* xc = static_cast<T*>(a.xc);
    const T* x = static_cast<const T*>(a.x);
    for (int k = warp; k < mine; k += 8) {
        const T* from = x + (r0 + list[k]) * a.cols;
        T* to = xc + (before + k) * a.ld;
        if (a.ld == a.cols) {   // whole 16-byte chunks
            const int64_t n16 = a.ld / 8;
#pragma unroll 4
            for (int64_t c = lane; c < n16; c += 32) reinterpret_cast<uint4*>(to)[c] = __ldg(reinterpret_cast<const uint4*>(from) + c);
        } else {
            for (int64_t c = lane; c < a.ld / 8; c += 32)
                reinterpret_cast<uint4*>(to)[c] = padded_chunk(reinterpret_cast<const uint8_t*>(from), 2 * a.cols, c);
        }
    }
    // zeros from the last row that counts up to the last tile that holds one
    const int64_t end = min(a.padded, (int64_t)((all + 255) / 256) * 256);
    uint4* z = reinterpret_cast<uint4*>(xc + (int64_t)all * a.ld);
    const int64_t nz = (end - all) * (a.ld / 8);
    for (int64_t i = (int64_t)blockIdx.x * 256 + t; i < nz; i += (int64_t)gridDim.x * 256) z[i] = make_uint4(0, 0, 0, 0);
}

// ---- the loss from its partial sums -------------------------------------------------

struct FinishArgs {
    const float2* part;     // [slots][ld]
    int64_t ld;
    int slots;
    const void *x, *w;      // rows of x: gathered ones (ldx), of w: [vocab, cols]
    int64_t cols, ldx, vocab;
    const int64_t* target;  // of the gathered rows
    const int32_t* index;   // null: row r itself
    const int32_t* count;   // null: `rows` of them
    int64_t rows;
    int64_t ignore;
    float *loss, *lse;      // [rows of x]; loss null: only its sum
    int reduction;
    int per_block;          // rows of a block, a power of two up to 8 (its warps)
    float* sums;            // [2 blocks]: sum of losses, number of rows that count
    int32_t* arrived;
    float* out;             // reduction 1, 2: [1]
};
template <typename T>
__global__ void __launch_bounds__(256) k_vocab_finish(const FinishArgs a) {
    __shared__ float2 sm[256];
    __shared__ float row_loss[8];
    __shared__ int row_in[8];
    __shared__ bool last;
    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int R = a.per_block, W = 256 / R;   // threads of a row
    const int64_t r0 = (int64_t)blockIdx.x * R;
    // The target's logit, a warp's row each, before the wait for the product: what it reads was
    // complete when that product's own wait ended, and the blocks start on processors that have had
    // their last tile (1 x 768 -> 50257 19.0 us without, 17.8 so; 333 x 1000 -> 32003 40.4 and 38.1).
    const int64_t n = a.count ? (int64_t)*a.count : a.rows, c = r0 + warp;
    int64_t tg = a.ignore, to = c;
    float z = 0.f;
    if (warp < R && c < n) {
        tg = a.target[c];
        if (a.index) to = a.index[c];
        if (tg != a.ignore && tg >= 0 && tg < a.vocab) {
            const T* x = static_cast<const T*>(a.x) + c * a.ldx;
            const T* w = static_cast<const T*>(a.w) + tg * a.cols;
            float d0 = 0.f, d1 = 0.f;
            if ((a.cols & 7) == 0) {   // (rows are whole 16-byte chunks)
                F8 sum;
                sum.clear();
#pragma unroll 4
                for (int64_t j = 8 * lane; j < a.cols; j += 256) {
                    F8 p, q;
                    load8(x + j, p);
                    load8(w + j, q);
                    sum.fma(p, q);
                }
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    d0 += sum.p[i].x;
                    d1 += sum.p[i].y;
                }
            } else {
                for (int64_t j = lane; j < a.cols; j += 32) d0 = fmaf(to_f32(x[j]), to_f32(w[j]), d0);
            }
            z = d0 + d1;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        }
    }
    after_previous();
    let_next_start();
    const int i = t & (R - 1);
    const float inf = __int_as_float(0x7f800000);
    {
        float m = -inf, s = 0.f;
        if (r0 + i < n) {
#pragma unroll 4
            for (int k = t / R; k < a.slots; k += W) {
                const float2 p = __ldcg(a.part + (int64_t)k * a.ld + r0 + i);
                const float top = fmaxf(m, p.x), base = top == -inf ? 0.f : top;
                s = s * exp2_fast(m - base) + p.y * exp2_fast(p.x - base);
                m = top;
            }
        }
        sm[t] = make_float2(m, s);
    }
    __syncthreads();
    for (int w = W / 2; w > 0; w >>= 1) {   // neighbours of a row are R apart
        if (t < w * R) {
            const float2 p = sm[t], q = sm[t + w * R];
            const float top = fmaxf(p.x, q.x), base = top == -inf ? 0.f : top;
            sm[t] = make_float2(top, p.y * exp2_fast(p.x - base) + q.y * exp2_fast(q.x - base));
        }
        __syncthreads();
    }
    if (warp < R && lane == 0) {
        float loss = 0.f;
        if (c < n) {
            float l = 0.f;
            if (tg != a.ignore) {
                l = kLn2 * sm[warp].x + logf(sm[warp].y);
                loss = tg >= 0 && tg < a.vocab ? l - z : nan_f();
            }
            if (a.loss) a.loss[to] = loss;
            if (a.lse) a.lse[to] = l;
        }
        row_loss[warp] = loss;
        row_in[warp] = c < n && tg != a.ignore;
    }
    if (a.reduction == 0) return;
    __syncthreads();
    if (t == 0) {
        float s = 0.f;
        int in = 0;
        for (int k = 0; k < R; ++k) {
            s += row_loss[k];
            in += row_in[k];
        }
        a.sums[2 * blockIdx.x] = s;
        a.sums[2 * blockIdx.x + 1] = (float)in;   // (at most 8)
        __threadfence();
        last = atomicAdd(a.arrived, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!last) return;
    // the last block adds all of them, in an order of their own
    __threadfence();
    float s = 0.f;
    int64_t in = 0;
    for (int64_t b = t; b < gridDim.x; b += 256) {
        s += __ldcg(a.sums + 2 * b);
        in += (int64_t)__ldcg(a.sums + 2 * b + 1);
    }
    double* ds = reinterpret_cast<double*>(sm);   // (256 x 8 bytes, no longer needed)
    __shared__ int counts[256];
    ds[t] = (double)s;
    counts[t] = (int)in;
    __syncthreads();
    for (int w = 128; w > 0; w >>= 1) {
        if (t < w) {
            ds[t] += ds[t + w];
            counts[t] += counts[t + w];
        }
        __syncthreads();
    }
    if (t == 0) *a.out = (float)(a.reduction == 2 ? ds[0] / (double)counts[0] : ds[0]);
}

// dx of every row of x from the slabs; ignored rows zero. WARPS: how many warps share the slabs of an
// element (many slabs of few rows: one thread's chain of loads would be the call's longest part).
template <typename T, int WARPS>
__global__ void __launch_bounds__(256) k_vocab_dx(const float* __restrict__ slab, int splits, int64_t stride, int64_t ld,
                                                  const int32_t* __restrict__ at, const GradScale by, int64_t rows, int64_t cols,
                                                  T* __restrict__ dx) {
    __shared__ F8 part[WARPS > 1 ? WARPS : 1][WARPS > 1 ? 32 : 1];
    after_previous();
    let_next_start();
    const float scale = by.out();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, first = WARPS > 1 ? warp : 0;
    constexpr int E = WARPS > 1 ? 32 : 256;   // elements (of 8 columns) of a block
    const int64_t n8 = ld / 8, n = rows * n8;
    for (int64_t i0 = (int64_t)blockIdx.x * E; i0 < n; i0 += (int64_t)gridDim.x * E) {
        const int64_t i = i0 + (WARPS > 1 ? lane : (int)threadIdx.x);
        const bool in = i < n;
        const int64_t r = in ? i / n8 : 0, c = in ? (i - r * n8) * 8 : 0;
        const int k = in ? __ldg(at + r) : -1;
        F8 f;
        f.clear();
        if (k >= 0) {
            const float* p = slab + (int64_t)k * ld + c;
#pragma unroll 4
            for (int s = first; s < splits; s += WARPS) {
                F8 o;
                load8(p + s * stride, o);
                f.add(o);
            }
        }
        if constexpr (WARPS > 1) {
            part[warp][lane] = f;
            __syncthreads();
            if (warp == 0) {
#pragma unroll
                for (int w = 1; w < WARPS; ++w) f.add(part[w][lane]);
            }
            __syncthreads();
        }
        if (!in || first > 0) continue;
        if (k >= 0) f.mul(scale);   // (an ignored row stays zero whatever the scale is)
        T* out = dx + r * cols + c;
        if (ld == cols) {
            store8(out, f);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (c + j < cols) out[j] = from_f32<T>(f.at(j));
        }
    }
}

// ---- host -----------------------------------------------------------------------------

int64_t up(int64_t n, int64_t m) { return ceil_div(n, m) * m; }
// Rows of a block of k_vocab_rows: few, so that the copies spread (8192 x 768: 64 rows 21 us, 16 rows 10),
// but not more than 4096 blocks that all read all targets until a block has its most.
int gather_rows(int64_t rows) { return (int)std::min<int64_t>(kGatherRows, std::max<int64_t>(16, up(ceil_div(rows, 4096), 16))); }

// A product's tile and ranges of K: the form whose waves take least by this account.  A stage
// takes its MMAs (us as measured, fewer columns than 128 at the same cost) or, where all SMs are
// busy, the bytes that they all fetch for it from the L2 (12.5 TB/s as measured); a tile has a
// microsecond beside its stages; a range's sums are written and read.
struct Form {
    int cg = 1, bn = 256, splits = 1;
    bool dual = false;
    int rows() const { return 128 * cg * (dual ? 2 : 1); }   // of a tile
};
// m x n over n_k stages; rows: of A that a tile loads; width: multiples of it (per CTA of a pair)
// are possible as tile widths; most: ranges of K at most; sums: bytes of one range's sums; dual: us that
// a dual tile has beside its stages (0: no dual tiles), its epilogue's time; longest: stages of a range at most.
Form pick_form(int64_t m, int64_t n, int64_t n_k, int rows, int width, int most, double sums, int num_sms, double dual,
               int64_t longest = INT64_MAX) {
    Form best;
    double least = 1e30;
    auto look = [&](const Form& f0, double mmas, double fixed) {
        Form f = f0;
        const int64_t tiles = ceil_div(m, f.rows()) * ceil_div(n, f.bn), units = num_sms / f.cg;
        for (f.splits = (int)std::max<int64_t>(1, ceil_div(n_k, longest)); f.splits <= most && (f.splits == 1 || n_k / f.splits >= 8); ++f.splits) {
            const double busy = (double)std::min(units, tiles * f.splits) * f.cg;
            const double stage = std::max(mmas, (rows * (f.dual ? 2 : 1) + f.bn / f.cg) * 128 * busy / 12.5e6);
            const double t = (double)ceil_div(tiles * f.splits, units) * ((double)ceil_div(n_k, f.splits) * stage + fixed) +
                             f.splits * sums / 3.3e6;
            if (t < 0.99 * least) {
                least = t;
                best = f;
            }
        }
    };
    Form f;
    if (m > 256 && dual > 0 && 256 % (2 * width) == 0) {
        f.cg = 2;
        f.dual = true;
        look(f, 0.62, dual);
        f.dual = false;
    }
    for (f.cg = m > 128 ? 2 : 1; f.cg >= 1; --f.cg) {
        const int step = std::max(32, width * f.cg);
        for (f.bn = 256; f.bn >= std::max(64, step); f.bn -= step) look(f, f.cg == 2 ? 0.34 : std::max(0.18, 0.36 * f.bn / 256), 1.0);
    }
    return best;
}

// The scratch of a call, in order; take() hands out 256-byte aligned pieces.
struct Scratch {
    char* base;
    int64_t used = 0;
    explicit Scratch(void* p) : base(static_cast<char*>(p)) {}
    template <typename T>
    T* take(int64_t n) {
        T* p = reinterpret_cast<T*>(base + used);
        used += up(n * (int64_t)sizeof(T), 256);
        return p;
    }
};

struct Shape {
    int64_t rows, cols, vocab, ld, padded;   // ld: columns in whole 16-byte chunks
    Shape(int64_t r, int64_t c, int64_t v) : rows(r), cols(c), vocab(v), ld(up(c, 8)), padded(up(r, 256)) {}
    bool pads() const { return ld != cols; }
    int tile_rows() const { return (int)std::min<int64_t>(kDenseM, up(rows, 8)); }   // that a row tile loads
};

struct ForwardPlan {
    bool gather;
    Form form;
    int n_nt, per_block, blocks;
    void *xc, *wc;
    int32_t *index, *at, *count, *arrived;
    int64_t* tc;
    float2* part;
    float* sums;
    int64_t bytes;
    ForwardPlan(const Shape& h, int num_sms, void* scratch) {
        form = pick_form(h.rows, h.vocab, ceil_div(h.cols, 64), h.tile_rows(), 32, 1, 0, num_sms,
                         ceil_div(h.ld, kDenseK) <= kTurnStages ? 2 : 0);
        // one row tile is one row tile whatever is left out: it reads x itself (333 x 1000 -> 32003, a dual
        // tile: 31.8 us, with its rows gathered 38.0; 200 x 768 -> 32003 18.7 and 22.4)
        gather = h.rows > form.rows() || h.pads();
        n_nt = (int)ceil_div(h.vocab, form.bn);
        per_block = 1;
        while (per_block < 8 && ceil_div(h.rows, per_block) > num_sms) per_block *= 2;
        blocks = (int)ceil_div(h.rows, per_block);
        Scratch s(scratch);
        count = s.take<int32_t>(2);
        arrived = count + 1;
        index = s.take<int32_t>(gather ? h.rows : 0);
        at = s.take<int32_t>(gather ? h.rows : 0);
        tc = s.take<int64_t>(gather ? h.rows : 0);
        xc = s.take<uint16_t>(gather ? h.padded * h.ld : 0);
        wc = s.take<uint16_t>(h.pads() ? h.vocab * h.ld : 0);
        part = s.take<float2>((int64_t)2 * n_nt * h.padded);
        sums = s.take<float>(2 * (int64_t)blocks);
        bytes = s.used;
    }
};

// Columns of the vocabulary whose dz is held at a time.
constexpr int64_t kPieceBytes = 512ll << 20;
constexpr int kRangesMost = 64;   // of K, in dx

struct BackwardPlan {
    Form z, x, w;
    bool z_turns, w_turns;
    int64_t piece;
    void *xc, *wc, *dz;
    int32_t *index, *at, *count;
    uint32_t* most;
    float* uniform;
    int64_t* tc;
    float *lse2, *g, *slab;
    int64_t bytes;
    BackwardPlan(const Shape& h, int num_sms, void* scratch) {
        const int64_t whole = up(h.vocab, 256);
        piece = std::max<int64_t>(256, std::min({whole, kPieceBytes / (2 * h.padded) / 256 * 256, (int64_t)kRangesMost * kSumStages * kDenseK}));
        piece = up(ceil_div(whole, ceil_div(whole, piece)), 256);   // equal ones
        z_turns = ceil_div(h.ld, kDenseK) > kSumStages;
        w_turns = ceil_div(h.rows, kDenseK) > kSumStages;
        z = pick_form(h.rows, piece, ceil_div(h.cols, 64), h.tile_rows(), 32, 1, 0, num_sms, z_turns ? 0 : 4.5);
        x = pick_form(h.rows, h.ld, piece / 64, h.tile_rows(), 64, kRangesMost, 8.0 * h.rows * h.ld, num_sms, 2, kSumStages);
        w = pick_form(piece, h.ld, ceil_div(h.rows, 64), kDenseM, 64, 1, 0, num_sms, w_turns ? 0 : 2);
        Scratch s(scratch);
        count = s.take<int32_t>(4);
        most = reinterpret_cast<uint32_t*>(count + 1);
        uniform = reinterpret_cast<float*>(count + 2);
        index = s.take<int32_t>(h.rows);
        at = s.take<int32_t>(h.rows);
        tc = s.take<int64_t>(h.rows);
        lse2 = s.take<float>(h.rows);
        g = s.take<float>(h.rows);
        xc = s.take<uint16_t>(h.padded * h.ld);
        wc = s.take<uint16_t>(h.pads() ? h.vocab * h.ld : 0);
        dz = s.take<uint16_t>(h.padded * piece);
        slab = s.take<float>((int64_t)x.splits * h.padded * h.ld);
        bytes = s.used;
    }
};

DenseArgs dense_args(const Form& f, bool bf16, bool a_mn, bool b_mn, int64_t m, int64_t n, int64_t k, int a_rows = kDenseM) {
    DenseArgs a = {};
    a.n_mt = (int)ceil_div(m, f.rows());
    a.n_nt = (int)ceil_div(n, f.bn);
    a.bn = f.bn;
    a.a_rows = a_rows;
    a.stages = dense_stages(f.cg, f.dual ? 2 * a_rows : a_rows, f.bn);
    a.m_held = up(m, 256);
    a.splits = f.splits;
    a.K = k;
    a.idesc = dense_idesc(bf16, a_mn, b_mn, 128 * f.cg, f.bn);
    a.group = 16 / f.cg;
    return a;
}
template <bool A_MN, bool B_MN, bool TURNS, class Epilogue>
int launch_form(const Form& f, const CUtensorMap& ma, const CUtensorMap& mb, const DenseArgs& a, const typename Epilogue::Args& e, int num_sms,
           cudaStream_t s) {
    if constexpr (!TURNS) {
        if (f.dual) return dense_launch<2, A_MN, B_MN, false, true, Epilogue>(ma, mb, a, e, num_sms, s);
    }
    return f.cg == 2 ? dense_launch<2, A_MN, B_MN, TURNS, false, Epilogue>(ma, mb, a, e, num_sms, s)
                     : dense_launch<1, A_MN, B_MN, TURNS, false, Epilogue>(ma, mb, a, e, num_sms, s);
}
// (turn_stages 0: one accumulator for all of K)
template <bool A_MN, bool B_MN, class Epilogue>
int launch(const Form& f, const CUtensorMap& ma, const CUtensorMap& mb, const DenseArgs& a, const typename Epilogue::Args& e, int num_sms,
           cudaStream_t s) {
    return a.turn_stages ? launch_form<A_MN, B_MN, true, Epilogue>(f, ma, mb, a, e, num_sms, s)
                         : launch_form<A_MN, B_MN, false, Epilogue>(f, ma, mb, a, e, num_sms, s);
}

int pad_weight(const Shape& h, const void* w, void* wc, cudaStream_t s) {
    return launch_after(k_pad_rows, (unsigned)std::min<int64_t>(ceil_div(h.vocab * ceil_div(h.ld, 256), 8), 1 << 20), 256, 0, 1, s,
                        static_cast<const uint8_t*>(w), 2 * h.cols, static_cast<uint8_t*>(wc), h.vocab, 2 * h.cols, 2 * h.ld);
}

template <typename T>
int forward(const Shape& h, const void* x, const void* w, const int64_t* target, int64_t ignore, int reduction, float* loss,
            float* lse, void* scratch, int num_sms, cudaStream_t s) {
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    ForwardPlan p(h, num_sms, scratch);
    float* row_loss = reduction == 0 ? loss : nullptr;
    if (p.gather) {
        RowsArgs r = {};
        r.x = x;
        r.target = target;
        r.ignore = ignore;
        r.rows = h.rows;
        r.cols = h.cols;
        r.vocab = h.vocab;
        r.ld = h.ld;
        r.padded = h.padded;
        r.per_block = gather_rows(h.rows);
        r.xc = p.xc;
        r.index = p.index;
        r.at = p.at;
        r.tc = p.tc;
        r.count = p.count;
        r.loss = row_loss;
        r.lse_zero = lse;
        if (int st = launch_after(k_vocab_rows<T>, (unsigned)ceil_div(h.rows, r.per_block), 256, 0, 1, s, r); st != SNK_OK) return st;
    }
    const void* wt = w;
    if (h.pads()) {
        if (int st = pad_weight(h, w, p.wc, s); st != SNK_OK) return st;
        wt = p.wc;
    }
    CUtensorMap ma, mb;
    const void* xt = p.gather ? p.xc : x;
    const int a_rows = h.tile_rows();
    if (!dense_map(&ma, xt, bf, h.ld, p.gather ? h.padded : h.rows, h.ld, a_rows) ||
        !dense_map(&mb, wt, bf, h.ld, h.vocab, h.ld, p.form.bn / p.form.cg))
        return SNK_ERR_CUDA;
    DenseArgs a = dense_args(p.form, bf, false, false, h.rows, h.vocab, h.ld, a_rows);
    a.rows = p.gather ? p.count : nullptr;
    a.zero = p.arrived;
    const LseEpilogue::Args ea{p.part, h.padded, h.vocab};
    if (ceil_div(h.ld, kDenseK) > kTurnStages) a.turn_stages = kTurnStages;
    if (int st = launch<false, false, LseEpilogue>(p.form, ma, mb, a, ea, num_sms, s); st != SNK_OK) return st;
    FinishArgs f = {};
    f.part = p.part;
    f.ld = h.padded;
    f.slots = 2 * p.n_nt;
    f.x = xt;
    f.w = w;
    f.cols = h.cols;
    f.ldx = p.gather ? h.ld : h.cols;
    f.vocab = h.vocab;
    f.target = p.gather ? p.tc : target;
    f.index = p.gather ? p.index : nullptr;
    f.count = p.gather ? p.count : nullptr;
    f.rows = h.rows;
    f.ignore = ignore;
    f.loss = row_loss;
    f.lse = lse;
    f.reduction = reduction;
    f.per_block = p.per_block;
    f.sums = p.sums;
    f.arrived = p.arrived;
    f.out = loss;
    return launch_after(k_vocab_finish<T>, (unsigned)p.blocks, 256, 0, 1, s, f);
}

template <typename T>
int backward(const Shape& h, const BackwardPlan& p, const void* wt, int reduction, void* dx, void* dw, int num_sms, cudaStream_t s) {
    const GradScale scale{p.most, reduction ? p.uniform : nullptr};
    constexpr bool bf = std::is_same<T, __nv_bfloat16>::value;
    CUtensorMap mx, mx_t, mz, mz_t;   // _t: read along the rows
    if (!dense_map(&mx, p.xc, bf, h.ld, h.padded, h.ld, h.tile_rows()) || !dense_map(&mx_t, p.xc, bf, h.ld, h.padded, h.ld, 64))
        return SNK_ERR_CUDA;
    for (int64_t v0 = 0; v0 < h.vocab; v0 += p.piece) {
        const int64_t width = std::min(p.piece, h.vocab - v0);
        const T* wp = static_cast<const T*>(wt) + v0 * h.ld;
        CUtensorMap mw, mw_t;
        // (dz's columns behind the piece's width are not written everywhere: they read as zeros)
        if (!dense_map(&mw, wp, bf, h.ld, width, h.ld, p.z.bn / p.z.cg) || !dense_map(&mw_t, wp, bf, h.ld, width, h.ld, 64) ||
            !dense_map(&mz, p.dz, bf, width, h.padded, p.piece, h.tile_rows()) ||
            !dense_map(&mz_t, p.dz, bf, width, h.padded, p.piece, 64))
            return SNK_ERR_CUDA;
        DenseArgs a = dense_args(p.z, bf, false, false, h.rows, width, h.ld, h.tile_rows());   // dz of the piece
        a.rows = p.count;
        if (p.z_turns) a.turn_stages = kSumStages;
        const typename GradEpilogue<T>::Args eg{static_cast<T*>(p.dz), p.piece, width, v0, p.lse2, p.g, p.tc, scale};
        if (int st = launch<false, false, GradEpilogue<T>>(p.z, mx, mw, a, eg, num_sms, s); st != SNK_OK) return st;
        if (dx) {
            a = dense_args(p.x, bf, false, true, h.rows, h.ld, width, h.tile_rows());
            a.rows = p.count;
            const SumEpilogue::Args es{p.slab, h.padded, h.ld, v0 > 0};
            if (int st = launch_form<false, true, false, SumEpilogue>(p.x, mz, mw_t, a, es, num_sms, s); st != SNK_OK) return st;
        }
        if (dw) {
            // Rows that are not whole 16-byte chunks go over the weight's padded copy, of which this piece has
            // been read, and from there side by side (20 x 1001 -> 50257, written from the tiles by 2 bytes: 557 us).
            T* end = static_cast<T*>(dw) + v0 * h.cols;
            T* out = h.pads() ? static_cast<T*>(p.wc) + v0 * h.ld : end;
            a = dense_args(p.w, bf, true, true, width, h.ld, h.rows);
            a.rows = p.count;
            a.rows_k = 1;
            if (p.w_turns) a.turn_stages = kSumStages;
            const int vec = h.ld % 16 == 0 && ((uintptr_t)out & 31) == 0 ? 16 : 8;
            const typename StoreEpilogue<T>::Args eo{out, width, h.ld, scale, vec};
            if (int st = launch<true, true, StoreEpilogue<T>>(p.w, mz_t, mx_t, a, eo, num_sms, s); st != SNK_OK) return st;
            if (h.pads()) {
                const int64_t blocks = std::min<int64_t>(ceil_div(width * h.cols, 2048), 1 << 20);
                if (int st = launch_after(k_join_rows, (unsigned)blocks, 256, 0, 1, s, reinterpret_cast<const uint16_t*>(out), h.ld,
                                          reinterpret_cast<uint16_t*>(end), width, h.cols);
                    st != SNK_OK)
                    return st;
            }
        }
    }
    if (dx) {
        const int64_t n = h.rows * (h.ld / 8);
        T* out = static_cast<T*>(dx);
        return p.x.splits > 8 ? launch_after(k_vocab_dx<T, 8>, (unsigned)std::min<int64_t>(ceil_div(n, 32), 64 * num_sms), 256, 0, 1, s,
                                             p.slab, p.x.splits, h.padded * h.ld, h.ld, p.at, scale, h.rows, h.cols, out)
                              : launch_after(k_vocab_dx<T, 1>, (unsigned)std::min<int64_t>(ceil_div(n, 256), 16 * num_sms), 256, 0, 1, s,
                                             p.slab, p.x.splits, h.padded * h.ld, h.ld, p.at, scale, h.rows, h.cols, out);
    }
    return SNK_OK;
}

template <typename T>
int backward_rows(const Shape& h, const BackwardPlan& p, const void* x, const void* w, const int64_t* target, int64_t ignore,
                  const float* lse, const float* dloss, int reduction, void* dx, void* dw, int num_sms, cudaStream_t s) {
    if (cudaMemsetAsync(p.most, 0, 4, s) != cudaSuccess) {
        cudaGetLastError();
        return SNK_ERR_CUDA;
    }
    RowsArgs r = {};
    r.x = x;
    r.target = target;
    r.ignore = ignore;
    r.rows = h.rows;
    r.cols = h.cols;
    r.vocab = h.vocab;
    r.ld = h.ld;
    r.padded = h.padded;
    r.per_block = gather_rows(h.rows);
    r.xc = p.xc;
    r.index = p.index;
    r.at = p.at;
    r.tc = p.tc;
    r.count = p.count;
    r.lse = lse;
    r.dloss = dloss;
    r.reduction = reduction;
    r.lse2 = p.lse2;
    r.g = p.g;
    r.most = p.most;
    r.uniform = p.uniform;
    if (int st = launch_after(k_vocab_rows<T>, (unsigned)ceil_div(h.rows, r.per_block), 256, 0, 1, s, r); st != SNK_OK) return st;
    const void* wt = w;
    if (h.pads()) {
        if (int st = pad_weight(h, w, p.wc, s); st != SNK_OK) return st;
        wt = p.wc;
    }
    return backward<T>(h, p, wt, reduction, dx, dw, num_sms, s);
}

bool unaligned(const void* p, uintptr_t n) { return p && ((uintptr_t)p & (n - 1)); }
// 1: bad, 2: too large
int bad_shape(int dtype, int64_t rows, int64_t cols, int64_t vocab, int reduction) {
    if ((dtype != SNK_F16 && dtype != SNK_BF16) || rows < 0 || cols < 1 || vocab < 1 || reduction < 0 || reduction > 2)
        return SNK_ERR_ARG;
    const int64_t lim = INT32_MAX - 512;
    if (rows > lim || cols > lim || vocab > lim) return SNK_ERR_LIMIT;
    // tiles are counted in 32 bits
    if ((double)ceil_div(rows, 128) * (double)ceil_div(vocab, 64) * 2 > 2.0e9 ||
        (double)ceil_div(vocab, 128) * (double)ceil_div(cols, 64) > 2.0e9 ||
        (double)ceil_div(rows, 128) * (double)ceil_div(cols, 64) * 512 > 2.0e9)
        return SNK_ERR_LIMIT;
    return SNK_OK;
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

int64_t snk_vocab_loss_scratch(int64_t rows, int64_t cols, int64_t vocab, int backward) {
    if (rows < 1 || bad_shape(SNK_BF16, rows, cols, vocab, 0) != SNK_OK) return 0;
    const int n = device_sms();
    if (n < 1) return 0;
    const Shape h(rows, cols, vocab);
    return backward ? BackwardPlan(h, n, nullptr).bytes : ForwardPlan(h, n, nullptr).bytes;
}

int snk_vocab_loss(const void* x, const void* weight, int dtype, const int64_t* target, int64_t ignore, int64_t rows,
                   int64_t cols, int64_t vocab, int reduction, float* loss, float* lse, void* scratch, void* stream) {
    if (int st = bad_shape(dtype, rows, cols, vocab, reduction); st != SNK_OK) return st;
    if (!weight || unaligned(weight, 16) || unaligned(x, 16) || unaligned(target, 8) || unaligned(loss, 4) || unaligned(lse, 4) ||
        unaligned(scratch, 256))
        return SNK_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {
        if (reduction == 0) return SNK_OK;
        if (!loss) return SNK_ERR_ARG;
        // the sum of no rows is 0, their mean NaN (all bits set is one)
        return cudaMemsetAsync(loss, reduction == 1 ? 0 : 0xff, 4, s) == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
    }
    if (!x || !target || !loss || !scratch) return SNK_ERR_ARG;
    const int n = device_sms();
    if (n < 1) return SNK_ERR_CUDA;
    const Shape h(rows, cols, vocab);
    return dtype == SNK_F16
               ? forward<__half>(h, x, weight, target, ignore, reduction, loss, lse, scratch, n, s)
               : forward<__nv_bfloat16>(h, x, weight, target, ignore, reduction, loss, lse, scratch, n, s);
}

int snk_vocab_loss_backward(const void* x, const void* weight, int dtype, const int64_t* target, int64_t ignore,
                            const float* lse, const float* dloss, int64_t rows, int64_t cols, int64_t vocab, int reduction,
                            void* dx, void* dweight, void* scratch, void* stream) {
    if (int st = bad_shape(dtype, rows, cols, vocab, reduction); st != SNK_OK) return st;
    if (!weight || unaligned(weight, 16) || unaligned(x, 16) || unaligned(target, 8) || unaligned(lse, 4) ||
        unaligned(dloss, 4) || unaligned(dx, 16) || unaligned(dweight, 16) || unaligned(scratch, 256))
        return SNK_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (rows == 0) {
        if (!dweight) return SNK_OK;
        return cudaMemsetAsync(dweight, 0, (size_t)(vocab * cols * 2), s) == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
    }
    if (!x || !target || !lse || !dloss || !scratch) return SNK_ERR_ARG;
    if (!dx && !dweight) return SNK_OK;
    const int n = device_sms();
    if (n < 1) return SNK_ERR_CUDA;
    const Shape h(rows, cols, vocab);
    const BackwardPlan p(h, n, scratch);
    return dtype == SNK_F16
               ? backward_rows<__half>(h, p, x, weight, target, ignore, lse, dloss, reduction, dx, dweight, n, s)
               : backward_rows<__nv_bfloat16>(h, p, x, weight, target, ignore, lse, dloss, reduction, dx, dweight, n, s);
}

}  // extern "C"
