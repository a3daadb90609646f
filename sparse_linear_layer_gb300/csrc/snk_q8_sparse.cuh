// The batch-tiled products on an 8-bit X: the chunk-walk SpMM (snk_spmm.cuh) and the
// row-order weight gradient (snk_sddmm.cuh) with the codes themselves as the operand.
//
//     Y[beta, o] = s_beta * sum_k w_k q[beta, c_k] + bias
//     dW_k       = sum_beta (s_beta dY[beta, r_k]) q[beta, c_k]
//
// With one scale per row, as written here, the scale leaves the sum (forward) or goes
// into dY (weight gradient), so an entry reads BP bytes of the transposed codes where
// the fp32 operand has 4 BP:
// a tile of 16 columns at in = 10000 then fits shared memory (160 KB), and a wider
// one, gathered through L1, moves a quarter of the bytes.  A lane decodes the codes
// of up to 16 batch columns itself, 4 per instruction word, exactly (see
// q_values4), and accumulates in fp32.  int8 codes are kept with their sign bit
// flipped in the transposed operand, which is the form the decoding starts from.
// Groups within a row have a scale per (row, group) instead: a table of them, groups x
// BP, follows the transposed codes, an entry reads its column's BP scales from it and
// multiplies the decoded values.  That pays up to 16 columns; wider tiles, layers
// of few entries per column, and the forward of one or two wide rows, run on the fp32
// kernels (q8_codes_tile).
//
// Measured at 10000 x 10000, 90%, int8, a scale per row, batch 1/4/8/16/32: forward
// 16/20/25/36/68 us (from an fp32 copy of the tile 17/25/43/69/103), weight gradient
// 17/20/29/48/90 (23/29/54/88/108); 64 rows forward 102 (134), weight gradient at 95%, where
// the tensor cores do not take it, 85 (118).  In groups of 128, batch 4/8/16: forward
// 21/29/45, weight gradient 27/38/66.  At 64 rows 56% of the issue slots are busy (6.6
// warp instructions per entry, the decoding); the rest is the latency of the words
// gathered through L1 and L2.
#pragma once

#include "snk_q8.cuh"
#include "snk_sddmm.cuh"
#include "snk_spmm.cuh"

namespace snk {

template <int FMT>
__device__ __forceinline__ constexpr uint32_t code_flip() {
    return FMT == SNK_Q8_INT8 ? 0x80808080u : 0u;
}

// dst[c * BP + beta] = code (beta, c), its sign bit flipped for int8, the code of
// 0 for b <= beta < BP.  Items of 4 rows x 4 columns, row groups fastest, so that
// the stores of neighbouring threads are contiguous.
template <int BP, int FMT>
__device__ __forceinline__ void stage_codes(uint8_t* dst, const uint8_t* __restrict__ src, int64_t n, int b, int tid,
                                            int nthreads) {
    constexpr uint32_t F = code_flip<FMT>();
    constexpr int QB = BP < 4 ? 1 : BP / 4, R = BP < 4 ? BP : 4;
    const bool words = n % 4 == 0 && ((uintptr_t)src & 3) == 0;
    const int64_t groups = (n + 3) / 4, items = groups * QB;
    for (int64_t i = tid; i < items; i += nthreads) {
        const int64_t g = i / QB;
        const int r0 = (int)(i - g * QB) * 4;
        uint32_t w[R];
#pragma unroll
        for (int r = 0; r < R; ++r) {
            w[r] = 0;
            if (r0 + r < b) {
                const uint8_t* p = src + (int64_t)(r0 + r) * n + 4 * g;
                if (words) {
                    w[r] = __ldg(reinterpret_cast<const uint32_t*>(p));
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (4 * g + j < n) w[r] |= (uint32_t)__ldg(p + j) << (8 * j);
                }
            }
            w[r] ^= F;
        }
        uint8_t* d = dst + 4 * g * BP + r0;
        if constexpr (BP == 1) {
            if (4 * g + 3 < n) {
                *reinterpret_cast<uint32_t*>(d) = w[0];
            } else {
                for (int j = 0; 4 * g + j < n; ++j) d[j] = (uint8_t)(w[0] >> (8 * j));
            }
        } else if constexpr (BP == 2) {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * g + j < n)
                    *reinterpret_cast<uint16_t*>(d + 2 * j) =
                        (uint16_t)(((w[0] >> (8 * j)) & 0xffu) | (((w[1] >> (8 * j)) & 0xffu) << 8));
        } else {
            const uint32_t a0 = __byte_perm(w[0], w[1], 0x5140), a1 = __byte_perm(w[2], w[3], 0x5140);
            const uint32_t a2 = __byte_perm(w[0], w[1], 0x7362), a3 = __byte_perm(w[2], w[3], 0x7362);
            const uint32_t o[4] = {__byte_perm(a0, a1, 0x5410), __byte_perm(a0, a1, 0x7632),
                                   __byte_perm(a2, a3, 0x5410), __byte_perm(a2, a3, 0x7632)};
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (4 * g + j < n) *reinterpret_cast<uint32_t*>(d + j * BP) = o[j];
        }
    }
}

// dst[g * BP + beta] = scale (beta, g), 0 for b <= beta < BP.
template <int BP>
__device__ __forceinline__ void stage_scales(float* dst, const float* __restrict__ src, int64_t groups, int b, int tid,
                                             int nthreads) {
    for (int64_t i = tid; i < groups * BP; i += nthreads) {
        const int beta = (int)(i % BP);
        dst[i] = beta < b ? __ldg(src + beta * groups + i / BP) : 0.f;
    }
}

// scales null: the codes only
template <int BP, int FMT>
__global__ void k_codes_transposed(const uint8_t* __restrict__ src, int64_t n, int b, uint8_t* __restrict__ dst,
                                   const float* __restrict__ scales, int64_t groups, int64_t table) {
    const int tid = blockIdx.x * blockDim.x + threadIdx.x, nthreads = gridDim.x * blockDim.x;
    stage_codes<BP, FMT>(dst, src, n, b, tid, nthreads);
    if (scales) stage_scales<BP>(reinterpret_cast<float*>(dst + table), scales, groups, b, tid, nthreads);
}

// Lane layout: a lane holds up to 16 batch columns of an entry (8 at BP = 16, which
// is faster there: 10000^2, 90%: forward 38 -> 35 us, dW 48 -> 45; at BP = 64 8
// columns take 120 and 176 us against 100 and 139).  Loading the next block's words
// before decoding this one's was slower throughout (registers).
template <int B, int FMT, bool GROUPED>
struct TileQ {
    using Elem = uint8_t;
    using DwArgs = SddmmQ8Args;
    static constexpr int BP = B;
    static constexpr int VEC = B < 8 ? B : (B <= 16 ? 8 : 16);
    static constexpr int LPE = B / VEC;
    static constexpr int GPW = kWarp / LPE;
    static constexpr int WORDS = VEC < 4 ? 1 : VEC / 4;
    struct Dy {
        float2 p[(VEC + 1) / 2];
        __device__ __forceinline__ void set(int j, float x) {
            if (j & 1) p[j >> 1].y = x;
            else p[j >> 1].x = x;
        }
    };
    __host__ __device__ static constexpr int beta(int sub, int j) { return sub * VEC + j; }
    // the codes, and with group scales a table [groups][B] of them
    template <class Args>
    __host__ __device__ static size_t codes_bytes(const Args& a) {
        return ((size_t)columns(a) * B + 15) & ~(size_t)15;
    }
    template <class Args>
    __host__ __device__ static size_t bytes(const Args& a) {
        return codes_bytes(a) + (GROUPED ? ((size_t)a.groups * B * sizeof(float) + 15) & ~(size_t)15 : 0);
    }

    // pair i of a word's 4 values
    __device__ __forceinline__ static float2 pair(uint32_t w, int i) {
        if constexpr (FMT == SNK_Q8_INT8) {
            const float2 x = make_float2(__uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540 + 2 * i)),
                                         __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7541 + 2 * i)));
            return __fadd2_rn(x, make_float2(-8388736.f, -8388736.f));
        } else {
            return __half22float2(
                __half2(__nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(i ? w >> 16 : w & 0xffffu), __NV_E4M3)));
        }
    }
    __device__ __forceinline__ static float one(uint32_t code) {
        if constexpr (FMT == SNK_Q8_INT8) return __uint_as_float(0x4B000000u | code) - 8388736.f;
        else return q_value((uint8_t)code, FMT);
    }
    // the lane's codes of operand row idx
    template <bool SMEM>
    __device__ __forceinline__ static void load(const uint8_t* xsrc, int idx, int sub, uint32_t (&w)[WORDS]) {
        const uint8_t* p = xsrc + (size_t)idx * B + sub * VEC;
        if constexpr (VEC == 1) {
            w[0] = SMEM ? *p : __ldg(p);
        } else if constexpr (VEC == 2) {
            w[0] = SMEM ? *reinterpret_cast<const uint16_t*>(p) : __ldg(reinterpret_cast<const uint16_t*>(p));
        } else if constexpr (VEC == 4) {
            w[0] = SMEM ? *reinterpret_cast<const uint32_t*>(p) : __ldg(reinterpret_cast<const uint32_t*>(p));
        } else if constexpr (VEC == 8) {
            const uint2 t = SMEM ? *reinterpret_cast<const uint2*>(p) : __ldg(reinterpret_cast<const uint2*>(p));
            w[0] = t.x;
            w[1] = t.y;
        } else {
            const uint4 t = SMEM ? *reinterpret_cast<const uint4*>(p) : __ldg(reinterpret_cast<const uint4*>(p));
            w[0] = t.x;
            w[1] = t.y;
            w[2] = t.z;
            w[3] = t.w;
        }
    }
    // the lane's scales of operand row idx
    template <bool SMEM, class Args>
    __device__ __forceinline__ static void load_scales(const Args& a, const uint8_t* xsrc, int idx, int sub,
                                                       float2 (&s)[(VEC + 1) / 2]) {
        const float* p = reinterpret_cast<const float*>(xsrc + a.table) + (size_t)(idx >> a.gshift) * B + sub * VEC;
        if constexpr (VEC == 1) {
            s[0].x = SMEM ? *p : __ldg(p);
        } else if constexpr (VEC == 2) {
            s[0] = SMEM ? *reinterpret_cast<const float2*>(p) : __ldg(reinterpret_cast<const float2*>(p));
        } else {
#pragma unroll
            for (int t = 0; t < VEC / 4; ++t) {
                const float4 v = SMEM ? reinterpret_cast<const float4*>(p)[t] : __ldg(reinterpret_cast<const float4*>(p) + t);
                s[2 * t] = make_float2(v.x, v.y);
                s[2 * t + 1] = make_float2(v.z, v.w);
            }
        }
    }
    template <bool SMEM>
    __device__ __forceinline__ static void axpy(const SpmmArgs& a, const uint8_t* xsrc, int idx, int sub, float wt,
                                                float (&acc)[VEC]) {
        uint32_t w[WORDS];
        load<SMEM>(xsrc, idx, sub, w);
        float2 sc[(VEC + 1) / 2];
        if constexpr (GROUPED) load_scales<SMEM>(a, xsrc, idx, sub, sc);
        if constexpr (VEC == 1) {
            acc[0] = fmaf(wt, GROUPED ? one(w[0]) * sc[0].x : one(w[0]), acc[0]);
        } else {
#pragma unroll
            for (int t = 0; t < VEC; t += 2) {
                float2 x = pair(w[t / 4], (t >> 1) & 1);
                if constexpr (GROUPED) x = __fmul2_rn(x, sc[t >> 1]);
                const float2 r = __ffma2_rn(x, make_float2(wt, wt), make_float2(acc[t], acc[t + 1]));
                acc[t] = r.x;
                acc[t + 1] = r.y;
            }
        }
    }
    template <bool SMEM>
    __device__ __forceinline__ static float dot(const SddmmQ8Args& a, const uint8_t* xsrc, int idx, int sub,
                                                const Dy& d) {
        uint32_t w[WORDS];
        load<SMEM>(xsrc, idx, sub, w);
        float2 sc[(VEC + 1) / 2];
        if constexpr (GROUPED) load_scales<SMEM>(a, xsrc, idx, sub, sc);
        if constexpr (VEC == 1) {
            return d.p[0].x * (GROUPED ? one(w[0]) * sc[0].x : one(w[0]));
        } else {
            float2 p = make_float2(0.f, 0.f);
#pragma unroll
            for (int t = 0; t < VEC; t += 2) {
                float2 x = pair(w[t / 4], (t >> 1) & 1);
                if constexpr (GROUPED) x = __fmul2_rn(x, sc[t >> 1]);
                p = __ffma2_rn(x, d.p[t >> 1], p);
            }
            return p.x + p.y;
        }
    }
    // from a transposed copy, if there is one (kStageCopy), else from the codes
    template <class Args>
    __device__ __forceinline__ static void stage(uint8_t* xs, const Args& a, int tid, int nthreads) {
        if (!a.xt) {
            stage_codes<B, FMT>(xs, a.codes, columns(a), a.b, tid, nthreads);
            if constexpr (GROUPED)
                stage_scales<B>(reinterpret_cast<float*>(xs + a.table), a.scales, a.groups, a.b, tid, nthreads);
            return;
        }
        constexpr int U = 6;   // loads in flight per thread
        const uint4* src = static_cast<const uint4*>(a.xt);
        uint4* dst = reinterpret_cast<uint4*>(xs);
        const int n = (int)(bytes(a) / 16);
        for (int i0 = tid; i0 < n; i0 += U * nthreads) {
            uint4 v[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * nthreads < n) v[u] = __ldg(src + i0 + u * nthreads);
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (i0 + u * nthreads < n) dst[i0 + u * nthreads] = v[u];
        }
    }
    __host__ __device__ static int64_t columns(const SpmmArgs& a) { return a.n_src; }
    __host__ __device__ static int64_t columns(const SddmmQ8Args& a) { return a.in_f; }
    // an output of a row of W with no entries is its bias, whatever the scale
    __device__ __forceinline__ static float out(const SpmmArgs& a, int beta, float sum, bool empty) {
        if constexpr (GROUPED) return sum;
        return empty ? 0.f : sum * __ldg(a.scales + beta);
    }
    __device__ __forceinline__ static float dy(const SddmmQ8Args& a, int beta, int r) {
        const float d = __ldg(a.dY + (int64_t)beta * a.out_f + r);
        return GROUPED ? d : d * __ldg(a.scales + beta);
    }
};

template <typename F>
static int q8_smem(F fn, size_t smem) {
    if (smem > 40 * 1024 &&
        cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess)
        return SNK_ERR_CUDA;
    return SNK_OK;
}

// From this size on, the codes are transposed once by a kernel of their own and
// every block copies the result with 16-byte accesses; below it every block
// transposes them itself and the launch is saved (forward, 10000 x 16 at 99%:
// 23.6 -> 14.6 us).
constexpr size_t kStageCopy = 48 * 1024;

template <int BP, int FMT, bool GROUPED>
static int q8_forward_bp(Layer* L, SpmmArgs a, cudaStream_t s) {
    using TL = TileQ<BP, FMT, GROUPED>;
    a.table = (int64_t)TL::codes_bytes(a);
    const size_t slots = spmm_slot_bytes<BP, false>();
    const size_t smem = TL::bytes(a) + slots;
    uint8_t* xt = reinterpret_cast<uint8_t*>(L->xt);
    const bool fits = smem <= (size_t)L->max_smem && a.idx16;
    a.xt = nullptr;
    if (!fits || TL::bytes(a) >= kStageCopy) {
        k_codes_transposed<BP, FMT><<<L->num_sms * 4, 256, 0, s>>>(a.codes, a.n_src, a.b, xt,
                                                                  GROUPED ? a.scales : nullptr, a.groups, a.table);
        a.xt = xt;
    }
    if (fits) {
        auto fn = k_spmm<TL, false, true>;
        if (q8_smem(fn, smem) != SNK_OK) return SNK_ERR_CUDA;
        fn<<<a.n_blocks, kThreads, smem, s>>>(a);
    } else {
        if (a.idx16) {
            k_spmm<TL, false, false, true><<<a.n_blocks, kThreads, slots, s>>>(a);
        } else {
            k_spmm<TL, false, false, false><<<a.n_blocks, kThreads, slots, s>>>(a);
        }
    }
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

template <int BP, int FMT, bool GROUPED>
static int q8_weight_bp(Layer* L, SddmmQ8Args a, cudaStream_t s) {
    using TL = TileQ<BP, FMT, GROUPED>;
    a.table = (int64_t)TL::codes_bytes(a);
    const size_t smem = TL::bytes(a);
    uint8_t* xt = reinterpret_cast<uint8_t*>(L->xt);
    const bool fits = smem <= (size_t)L->max_smem && a.col16;
    a.xt = nullptr;
    if (!fits || smem >= kStageCopy) {
        k_codes_transposed<BP, FMT><<<L->num_sms * 4, 256, 0, s>>>(a.codes, a.in_f, a.b, xt,
                                                                  GROUPED ? a.scales : nullptr, a.groups, a.table);
        a.xt = xt;
    }
    if (fits) {
        auto fn = k_sddmm<TL, true>;
        if (q8_smem(fn, smem) != SNK_OK) return SNK_ERR_CUDA;
        fn<<<a.n_blocks, kThreads, smem, s>>>(a);
    } else {
        if (a.col16) k_sddmm<TL, false, true><<<a.n_blocks, kThreads, 0, s>>>(a);
        else k_sddmm<TL, false, false><<<a.n_blocks, kThreads, 0, s>>>(a);
    }
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

// One batch tile (a.b rows; codes, scales, groups and gshift set); a translation unit
// per format and kind of scale.
template <int FMT, bool GROUPED>
int q8_forward_tile(Layer* L, const SpmmArgs& a, int bp, cudaStream_t s);
template <int FMT, bool GROUPED>
int q8_weight_tile(Layer* L, const SddmmQ8Args& a, int bp, cudaStream_t s);

#define SNK_Q8_ROW_TILES(FMT)                                                                       \
    template <>                                                                                     \
    int q8_forward_tile<FMT, false>(Layer * L, const SpmmArgs& a, int bp, cudaStream_t s) {         \
        switch (bp) {                                                                               \
            case 1: return q8_forward_bp<1, FMT, false>(L, a, s);                                   \
            case 2: return q8_forward_bp<2, FMT, false>(L, a, s);                                   \
            case 4: return q8_forward_bp<4, FMT, false>(L, a, s);                                   \
            case 8: return q8_forward_bp<8, FMT, false>(L, a, s);                                   \
            case 16: return q8_forward_bp<16, FMT, false>(L, a, s);                                 \
            case 32: return q8_forward_bp<32, FMT, false>(L, a, s);                                 \
            default: return q8_forward_bp<64, FMT, false>(L, a, s);                                 \
        }                                                                                           \
    }                                                                                               \
    template <>                                                                                     \
    int q8_weight_tile<FMT, false>(Layer * L, const SddmmQ8Args& a, int bp, cudaStream_t s) {         \
        switch (bp) {                                                                               \
            case 1: return q8_weight_bp<1, FMT, false>(L, a, s);                                    \
            case 2: return q8_weight_bp<2, FMT, false>(L, a, s);                                    \
            case 4: return q8_weight_bp<4, FMT, false>(L, a, s);                                    \
            case 8: return q8_weight_bp<8, FMT, false>(L, a, s);                                    \
            case 16: return q8_weight_bp<16, FMT, false>(L, a, s);                                  \
            case 32: return q8_weight_bp<32, FMT, false>(L, a, s);                                  \
            default: return q8_weight_bp<64, FMT, false>(L, a, s);                                  \
        }                                                                                           \
    }
// (q8_codes_tile)
#define SNK_Q8_GROUP_TILES(FMT)                                                                     \
    template <>                                                                                     \
    int q8_forward_tile<FMT, true>(Layer * L, const SpmmArgs& a, int bp, cudaStream_t s) {          \
        switch (bp) {                                                                               \
            case 1: return q8_forward_bp<1, FMT, true>(L, a, s);                                    \
            case 2: return q8_forward_bp<2, FMT, true>(L, a, s);                                    \
            case 4: return q8_forward_bp<4, FMT, true>(L, a, s);                                    \
            case 8: return q8_forward_bp<8, FMT, true>(L, a, s);                                    \
            default: return q8_forward_bp<16, FMT, true>(L, a, s);                                  \
        }                                                                                           \
    }                                                                                               \
    template <>                                                                                     \
    int q8_weight_tile<FMT, true>(Layer * L, const SddmmQ8Args& a, int bp, cudaStream_t s) {          \
        switch (bp) {                                                                               \
            case 1: return q8_weight_bp<1, FMT, true>(L, a, s);                                     \
            case 2: return q8_weight_bp<2, FMT, true>(L, a, s);                                     \
            case 4: return q8_weight_bp<4, FMT, true>(L, a, s);                                     \
            case 8: return q8_weight_bp<8, FMT, true>(L, a, s);                                     \
            default: return q8_weight_bp<16, FMT, true>(L, a, s);                                   \
        }                                                                                           \
    }

}  // namespace snk
