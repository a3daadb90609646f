// The row-order weight-gradient kernel, for an fp32 X (snk_sddmm.cu, which
// describes it) and for an 8-bit one (snk_q8_sparse.cuh).  A tile type TL says how
// a lane reads its batch columns (as in snk_spmm.cuh):
//   stage()      the transposed X into shared memory
//   dy()         a value of dY as the lane multiplies it
//   Dy           the lane's values of a row of dY
//   dot<SMEM>()  the lane's share of an entry's dot product
//   DwArgs       the kernel's arguments
#pragma once

#include <type_traits>

#include "snk_device.cuh"

namespace snk {

struct SddmmArgs {
    const int32_t* col;     // canonical column indices
    const uint16_t* col16;  // the same as 16-bit, zero padded (shared-memory path)
    const int32_t* row_ptr; // [out+1]
    const int4* cdesc;      // [n_blocks * kWarpsPerBlock] (k0, k1, first row, end row)
    int64_t nnz, out_f, in_f;
    int b;                  // batch columns of this tile
    int n_blocks;
    const float* X;         // [b, in] (tile)
    const void* xt;         // [in][BP] (global path)
    const float* dY;        // [b, out] (tile)
    float* dW;              // [nnz]
    bool accumulate;        // add to dW (later batch tiles)
    const float* dY_all;    // [b_all, out] for db, or null
    int64_t b_all;
    float* db;              // [out] or null
};
// With an 8-bit X.
struct SddmmQ8Args : SddmmArgs {
    explicit SddmmQ8Args(const SddmmArgs& a) : SddmmArgs(a) {}
    const float* scales = nullptr;    // [b, groups]
    const uint8_t* codes = nullptr;   // [b, in]
    int64_t groups = 0;     // groups of a row
    int64_t table = 0;      // byte offset of the transposed scales in the operand
    int gshift = 0;         // log2 of a group's columns
};

// The fp32 X.  How long a kernel's argument block is changes what the compiler spills:
// with the 8-bit fields in it 16 columns in shared memory are slower (3000 x 3000 at 80%:
// 23.1 us against 22.4) and 32 and 64 faster (8000 x 800 at 80%, 64: 37.5 against 39.3),
// so those alone have them.
template <int B>
struct DwTileF32 : Tile<B> {
    using TL = Tile<B>;
    using Elem = float;
    using DwArgs = std::conditional_t<(B >= 32), SddmmQ8Args, SddmmArgs>;
    static constexpr int BP = B;
    struct Dy {
        float v[TL::VEC];
        __device__ __forceinline__ void set(int j, float x) { v[j] = x; }
    };
    __device__ __forceinline__ static void stage(float* xs, const SddmmArgs& a, int tid, int nthreads) {
        stage_transposed<B>(xs, a.X, a.in_f, a.b, a.in_f, tid, nthreads);
    }
    __device__ __forceinline__ static float dy(const SddmmArgs& a, int beta, int r) {
        return __ldg(a.dY + (int64_t)beta * a.out_f + r);
    }
    template <bool SMEM>
    __device__ __forceinline__ static float dot(const SddmmArgs&, const float* xsrc, int idx, int sub, const Dy& d) {
        float x[TL::VEC];
        if constexpr (SMEM) TL::load(xsrc + idx * B, sub, x);
        else TL::ldg(xsrc + idx * B, sub, x);
        float p = 0.f;
#pragma unroll
        for (int t = 0; t < TL::VEC; ++t) p = fmaf(d.v[t], x[t], p);
        return p;
    }
};

template <class TL>
__device__ __forceinline__ void load_dy_row(const typename TL::DwArgs& a, int r, int sub, typename TL::Dy& d) {
#pragma unroll
    for (int j = 0; j < TL::VEC; ++j) {
        const int beta = TL::beta(sub, j);
        d.set(j, beta < a.b ? TL::dy(a, beta, r) : 0.f);
    }
}

// One warp per chunk; the chunk's column indices stream as flat blocks of
// 4*GPW entries held in D+1 register slots (D blocks in flight while one is
// consumed; the slot loop is unrolled so slot indices are constants).  The dY
// values of the current row are in registers and the next row's are
// requested one row ahead.
template <class TL, bool SMEM, bool I16 = SMEM && SNK_IDX16>
__global__ void __launch_bounds__(kThreads, 1) k_sddmm(const typename TL::DwArgs a) {
    using Elem = typename TL::Elem;
    constexpr int VEC = TL::VEC, LPE = TL::LPE, GPW = TL::GPW, BP = TL::BP;
    constexpr uint32_t BLK = 4 * GPW;
    constexpr int D = BP <= 2 ? SNK_PIPE_DW_NARROW : ((BP == 4 || SMEM) ? SNK_PIPE_DW : SNK_PIPE_DW_WIDE);
    constexpr int NS = D + 1;
    extern __shared__ float4 smem4[];
    Elem* xs = reinterpret_cast<Elem*>(smem4);

    const int lane = threadIdx.x & 31;
    const int grp = lane / LPE;
    const int sub = lane % LPE;
    const uint32_t nnz = (uint32_t)a.nnz;
    const int4 cd = a.cdesc[blockIdx.x * kWarpsPerBlock + (threadIdx.x >> 5)];
    const uint32_t k0 = (uint32_t)cd.x, k1 = (uint32_t)cd.y;
    const uint32_t base_first = k0 & ~3u;
    IdxBlk<I16> ib[NS];
    auto issue = [&](int s, uint32_t blk0) {
        const uint32_t base = blk0 + 4 * grp;
        if constexpr (I16) ib[s].load(a.col16, base);
        else ib[s].load(a.col, base, nnz);
    };
    SegWindow win{cd.z, cd.w - cd.z, 0, 0u, 0.f};
    if (k0 < k1) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if (base_first + s * BLK < k1) issue(s, base_first + s * BLK);
        win.load(0, lane, a.row_ptr, nullptr);
    }
    if (a.db) {
        // bias gradient over the whole batch, sequential in batch order
        for (int64_t o = blockIdx.x * (int64_t)kThreads + threadIdx.x; o < a.out_f;
             o += (int64_t)gridDim.x * kThreads) {
            float sacc = 0.f;
            for (int64_t beta = 0; beta < a.b_all; ++beta) sacc += a.dY_all[beta * a.out_f + o];
            a.db[o] = sacc;
        }
    }
    if constexpr (SMEM) {
        TL::stage(xs, a, threadIdx.x, kThreads);
        __syncthreads();
    }
    if (k0 >= k1) return;  // no entries in this chunk (rows without entries need no output)
    const Elem* xsrc = SMEM ? xs : static_cast<const Elem*>(a.xt);

    const int r_begin = win.r_begin;
    int i = 0;
    uint32_t rs = win.bnd(0, lane, a.row_ptr, nullptr), re = win.bnd(1, lane, a.row_ptr, nullptr);
    typename TL::Dy dyr, dyn;
    load_dy_row<TL>(a, r_begin, sub, dyr);
#pragma unroll
    for (int j = 0; j < VEC; ++j) dyn.set(j, 0.f);
    if (win.nrows > 1) load_dy_row<TL>(a, r_begin + 1, sub, dyn);

    auto consume = [&](int s, uint32_t blk0) {
        const uint32_t base = blk0 + 4 * grp;
        const uint32_t blk_end = min(blk0 + BLK, k1);
        float res[4] = {0.f, 0.f, 0.f, 0.f};
        const bool interior = rs <= blk0 && k0 <= blk0 && blk0 + BLK < re && blk0 + BLK <= k1;
        while (true) {
            if (interior) {
                // every entry of the block belongs to the current row, which
                // continues past the block
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    float p = TL::template dot<SMEM>(a, xsrc, ib[s].get(j), sub, dyr);
#pragma unroll
                    for (int o = 1; o < LPE; o <<= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
                    res[j] = p;
                }
                break;
            }
            const uint32_t lo_k = max(max(rs, k0), blk0), hi_k = min(re, blk_end);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint32_t k = base + j;
                const bool ok = k >= lo_k && k < hi_k;
                float p = TL::template dot<SMEM>(a, xsrc, ok ? ib[s].get(j) : 0, sub, dyr);
#pragma unroll
                for (int o = 1; o < LPE; o <<= 1) p += __shfl_xor_sync(0xffffffffu, p, o);
                if (ok) res[j] = p;
            }
            if (min(re, k1) > blk_end) break;  // row continues in the next block
            if (++i >= win.nrows) break;
            rs = re;
            re = win.bnd(i + 1, lane, a.row_ptr, nullptr);
            dyr = dyn;
            if (i + 1 < win.nrows) load_dy_row<TL>(a, r_begin + i + 1, sub, dyn);
            if (rs >= blk_end) break;
        }
        if (sub == 0) {
            if (base >= k0 && base + 3 < k1) {
                float4 v = make_float4(res[0], res[1], res[2], res[3]);
                float4* dst = reinterpret_cast<float4*>(a.dW + base);
                if (a.accumulate) {
                    const float4 o4 = *dst;
                    v.x += o4.x;
                    v.y += o4.y;
                    v.z += o4.z;
                    v.w += o4.w;
                }
                *dst = v;
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t k = base + j;
                    if (k >= k0 && k < k1) a.dW[k] = a.accumulate ? a.dW[k] + res[j] : res[j];
                }
            }
        }
    };

    for (uint32_t base0 = base_first; base0 < k1; base0 += NS * BLK) {
#pragma unroll
        for (int s = 0; s < NS; ++s) {
            const uint32_t blk0 = base0 + s * BLK;
            if (blk0 < k1) {
                consume(s, blk0);
                if (blk0 + NS * BLK < k1) issue(s, blk0 + NS * BLK);
            }
        }
    }
}

}  // namespace snk
