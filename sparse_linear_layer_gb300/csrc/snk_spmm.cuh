// The chunk-walk SpMM kernel, for an fp32 operand (snk_spmm.cu, which describes
// it) and for an 8-bit one (snk_q8_sparse.cuh).  A tile type TL says how a lane
// reads its batch columns of one stored entry's operand row:
//   BP, VEC, LPE, GPW, beta()   the lane layout (Tile in snk_device.cuh)
//   Elem                        the operand's element
//   stage()                     the transposed operand into shared memory
//   axpy<SMEM>()                acc += w * (the lane's values of a row)
//   out()                       an output from its sum
#pragma once

#include "snk_device.cuh"

namespace snk {

struct SpmmArgs {
    const float* val;        // stored values, canonical order
    const int32_t* perm;     // column-order -> canonical slot (transposed product) or null
    const int32_t* idx;      // operand index per stored entry (col, or row in column order)
    const uint16_t* idx16;   // the same as 16-bit, zero padded (shared-memory path)
    const int32_t* seg_ptr;  // [n_seg+1]
    const int4* cdesc;       // [n_blocks * kWarpsPerBlock] (k0, k1, first seg, end seg)
    const BlockDesc* bdesc;  // [n_blocks]
    const int32_t* bnd;      // [n_blocks+1] first entry of each block
    int64_t nnz;
    int64_t n_seg;           // output length per batch row
    int64_t n_src;           // operand length per batch row
    int b;                   // batch columns of this tile (<= BP)
    int n_blocks;
    const float* X;          // [b, n_src] row-major
    const void* xt;          // [n_src][BP] transposed copy (global-memory path)
    const float* scales;     // 8-bit operand: [b, groups], its scales
    const uint8_t* codes;    // and its codes [b, n_src]
    int64_t groups;          // groups of a row
    int gshift;              // log2 of their columns
    int64_t table;           // byte offset of the transposed scales in the operand
    const float* bias;       // [n_seg] or null
    float* Y;                // [b, n_seg] row-major
    float* part;             // [n_blocks][2][BP] cross-block partial sums
    int32_t* cnt;            // [n_seg] arrival counters
    // column sweep of the transposed product (k_sweep only)
    const int4* sw_blk;      // per block: two records
    const int2* sw_col;      // per block and column: (first virtual lane, lanes)
    const int4* sw_lane;     // per virtual lane: (first quad, quad stride, first entry, end entry)
    float* sw_gpart;         // partials of virtual lanes beyond the block's threads
    const int* sw_split;     // [boundary][lane] resume quad of each lane at each table boundary
    int64_t sw_nlane;        // lanes per boundary in sw_split
    int sw_rows;             // operand rows staged per phase (a multiple of 4)
    int sw_phases;           // phases of this launch
    int sw_stride;           // table boundaries per phase of this launch
};

// A segment cut by a chunk boundary, whose partial sum this warp stored in
// its shared-memory slot (0: the segment entered the chunk from before,
// 1: it starts in the chunk and leaves it).
struct Pending {
    int r;
    uint32_t rs, re;
};

// Shared memory: [transposed operand (shared-memory path)][partials
// [warps][2][BP]][segment ids [warps][2]].
template <bool GATHER>
struct SpmmShape {
    static constexpr int kNT = GATHER ? kThreadsDx : kThreads;
    static constexpr int kW = kNT / kWarp;
};
template <int BP, bool GATHER>
__host__ __device__ constexpr size_t spmm_slot_bytes() {
    return (size_t)SpmmShape<GATHER>::kW * 2 * BP * sizeof(float) +
           (size_t)SpmmShape<GATHER>::kW * 2 * sizeof(int);
}
__host__ __device__ inline size_t operand_floats(int64_t n_src, int bp) {
    return ((size_t)n_src * bp + 3) & ~(size_t)3;
}

// The fp32 operand.
template <int B>
struct TileF32 : Tile<B> {
    using TL = Tile<B>;
    using Elem = float;
    static constexpr int BP = B;
    __host__ __device__ static size_t bytes(const SpmmArgs& a) { return operand_floats(a.n_src, B) * sizeof(float); }
    __device__ __forceinline__ static void stage(float* xs, const SpmmArgs& a, int tid, int nthreads) {
        stage_transposed<B>(xs, a.X, a.n_src, a.b, a.n_src, tid, nthreads);
    }
    template <bool SMEM>
    __device__ __forceinline__ static void axpy(const SpmmArgs&, const float* xsrc, int idx, int sub, float w,
                                                float (&acc)[TL::VEC]) {
        float x[TL::VEC];
        if constexpr (SMEM) TL::load(xsrc + idx * B, sub, x);
        else TL::ldg(xsrc + idx * B, sub, x);
#pragma unroll
        for (int t = 0; t < TL::VEC; ++t) acc[t] = fmaf(w, x[t], acc[t]);
    }
    __device__ __forceinline__ static float out(const SpmmArgs&, int, float sum, bool) { return sum; }
};

// Finish one output segment: reduce the per-lane partial sums across the
// warp's groups; write the result, or, for a segment cut by a chunk boundary,
// store this warp's partial in its shared slot.
template <class TL>
__device__ __forceinline__ void finish_segment(const SpmmArgs& a, float (&acc)[TL::VEC],
                                               int r, uint32_t rs, uint32_t re, uint32_t k0,
                                               uint32_t k1, float bo, int lane, int sub,
                                               float* my_slots, Pending (&pend)[2]) {
    constexpr int VEC = TL::VEC, LPE = TL::LPE, BP = TL::BP;
#pragma unroll
    for (int o = LPE; o < kWarp; o <<= 1) {
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] += __shfl_xor_sync(0xffffffffu, acc[j], o);
    }
    if (rs >= k0 && re <= k1) {
        if (lane < LPE) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) {
                const int beta = TL::beta(sub, j);
                if (beta < a.b) a.Y[(int64_t)beta * a.n_seg + r] = TL::out(a, beta, acc[j], rs == re) + bo;
            }
        }
    } else {
        const int slot = (rs < k0) ? 0 : 1;
        if (lane < LPE) {
#pragma unroll
            for (int j = 0; j < VEC; ++j) my_slots[slot * BP + sub * VEC + j] = acc[j];
        }
        pend[slot] = Pending{r, rs, re};
    }
#pragma unroll
    for (int j = 0; j < VEC; ++j) acc[j] = 0.f;
}

// A segment cut between blocks: store this block's partial, count the
// arrival, and let the last arriving block add the partials of the non-empty
// blocks first..last in block order (the first block's is in its slot 1).
template <class TL>
__device__ __noinline__ void cross_block(const SpmmArgs& a, int r, int slot,
                                         const float (&sum)[TL::VEC], int first, int last,
                                         int n_contrib, int lane, int sub) {
    constexpr int VEC = TL::VEC, LPE = TL::LPE, BP = TL::BP;
    if (lane < LPE) {
        float* my = a.part + ((int64_t)blockIdx.x * 2 + slot) * BP + sub * VEC;
#pragma unroll
        for (int j = 0; j < VEC; ++j) my[j] = sum[j];
    }
    __threadfence();
    __syncwarp();
    int old = 0;
    if (lane == 0) old = atomicAdd(a.cnt + r, 1);
    old = __shfl_sync(0xffffffffu, old, 0);
    if (old != n_contrib - 1) return;
    __threadfence();
    if (lane < LPE) {
        float tot[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) tot[j] = 0.f;
        for (int c = first; c <= last; ++c) {
            if (__ldg(a.bnd + c + 1) == __ldg(a.bnd + c)) continue;
            const float* pp = a.part + ((int64_t)c * 2 + (c == first ? 1 : 0)) * BP + sub * VEC;
#pragma unroll
            for (int j = 0; j < VEC; ++j) tot[j] += __ldcg(pp + j);
        }
        const float bo = a.bias ? __ldg(a.bias + r) : 0.f;
#pragma unroll
        for (int j = 0; j < VEC; ++j) {
            const int beta = TL::beta(sub, j);
            if (beta < a.b) a.Y[(int64_t)beta * a.n_seg + r] = TL::out(a, beta, tot[j], false) + bo;
        }
    }
    if (lane == 0) a.cnt[r] = 0;
}

// After the block barrier: the warp where a cut segment starts adds the
// partials of the following warps that continue it (warp order) and writes
// the result, unless the segment leaves the block; warp 0 does the same for
// the segment that entered the block from before.  Segments that cross a
// block boundary continue in cross_block.
template <class TL, int W>
__device__ __forceinline__ void block_combine(const SpmmArgs& a, const float* sp, const int* srow,
                                              const Pending (&pend)[2], int warp, int lane,
                                              int sub) {
    constexpr int VEC = TL::VEC, LPE = TL::LPE, BP = TL::BP;
    if (pend[1].r < 0 && !(warp == 0 && pend[0].r >= 0)) return;
    const BlockDesc bd = a.bdesc[blockIdx.x];
#pragma unroll
    for (int which = 1; which >= 0; --which) {
        const int slot = which;
        if (slot == 0 && warp != 0) continue;
        const int r = pend[slot].r;
        if (r < 0) continue;
        float sum[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j)
            sum[j] = lane < LPE ? sp[(warp * 2 + slot) * BP + sub * VEC + j] : 0.f;
        for (int w2 = warp + 1; w2 < W && srow[w2 * 2] == r; ++w2) {
#pragma unroll
            for (int j = 0; j < VEC; ++j)
                if (lane < LPE) sum[j] += sp[(w2 * 2) * BP + sub * VEC + j];
        }
        const bool ends_here = pend[slot].re <= (uint32_t)bd.k1;
        if (slot == 1) {
            if (ends_here) {
                if (lane < LPE) {
                    const float bo = a.bias ? __ldg(a.bias + r) : 0.f;
#pragma unroll
                    for (int j = 0; j < VEC; ++j) {
                        const int beta = TL::beta(sub, j);
                        if (beta < a.b) a.Y[(int64_t)beta * a.n_seg + r] = TL::out(a, beta, sum[j], false) + bo;
                    }
                }
            } else {
                cross_block<TL>(a, r, 1, sum, blockIdx.x, bd.tail_last, bd.n_tail, lane, sub);
            }
        } else {
            if (ends_here)
                cross_block<TL>(a, r, 0, sum, bd.head_first, blockIdx.x, bd.n_head, lane, sub);
            else
                cross_block<TL>(a, r, 0, sum, bd.head_first, bd.tail_last,
                                bd.n_head + bd.n_tail - 1, lane, sub);
        }
    }
}

// One warp per chunk.  The chunk's entries [k0, k1) are streamed as a flat
// sequence of blocks of 4*GPW entries from the multiple of 4 at or below k0
// (each group of LPE lanes owns 4 consecutive entries of a block).  Blocks
// sit in D+1 register slots: while block j is consumed, blocks j+1 .. j+D
// are in flight (and, for the transposed product, the values of blocks
// j+1 .. j+G are being gathered).  The loop over slots is unrolled so every slot index
// is a compile-time constant.  A block inside one segment is consumed
// without masks; a block that straddles segment or chunk boundaries is
// consumed once per segment it touches, with masks.
template <class TL, bool GATHER, bool SMEM, bool I16 = SMEM && SNK_IDX16>
__global__ void __launch_bounds__(SpmmShape<GATHER>::kNT, 1) k_spmm(const SpmmArgs a) {
    constexpr int NT = SpmmShape<GATHER>::kNT;
    constexpr int W = SpmmShape<GATHER>::kW;
    using Elem = typename TL::Elem;
    constexpr int VEC = TL::VEC, LPE = TL::LPE, GPW = TL::GPW, BP = TL::BP;
    constexpr uint32_t BLK = 4 * GPW;
    constexpr int D = GATHER ? (BP == 16 ? SNK_PIPE_DX16 : SNK_PIPE_DX) : (BP == 1 ? SNK_PIPE_FWD_NARROW : SNK_PIPE_FWD);
    constexpr int NS = D + 1;
    // blocks whose values are gathered ahead of the consumed one (the
    // permutation of a block arrives NS - G blocks before its gather)
    constexpr int G = GATHER ? (SNK_GATHER_LEAD < D ? SNK_GATHER_LEAD : D) : 0;
    extern __shared__ float4 smem4[];
    Elem* xs = reinterpret_cast<Elem*>(smem4);
    float* sp = reinterpret_cast<float*>(reinterpret_cast<char*>(smem4) + (SMEM ? TL::bytes(a) : 0));
    int* srow = reinterpret_cast<int*>(sp + W * 2 * BP);

    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const int grp = lane / LPE;
    const int sub = lane % LPE;
    const uint32_t nnz = (uint32_t)a.nnz;
    const int4 cd = a.cdesc[blockIdx.x * W + warp];
    const uint32_t k0 = (uint32_t)cd.x, k1 = (uint32_t)cd.y;
    const uint32_t base_first = k0 & ~3u;
    float* my_slots = sp + warp * 2 * BP;

    IdxBlk<I16> ib[NS];
    float wb[NS][4];
    int pb[NS][4];
    auto issue = [&](int s, uint32_t blk0) {
        const uint32_t base = blk0 + 4 * grp;
        if constexpr (I16) ib[s].load(a.idx16, base);
        else ib[s].load(a.idx, base, nnz);
        if constexpr (GATHER) padded4(a.perm, base, pb[s]);
        else stream4(a.val, base, nnz, wb[s]);
    };
    // The value gather hits L1 when another entry of the same row (in the
    // block's column range) brought its sector in, so it goes through L1;
    // except with a 4-column operand in shared memory (160 KB at out =
    // 10000), where the L1 left is small and caching the gathered sectors
    // only in L2 is faster (measured: 56 against 60 us at 10000^2, 90%).
    constexpr bool kGatherL2Only = SMEM && BP == 4;
    auto gather = [&](int s, uint32_t blk0) {
        const uint32_t base = blk0 + 4 * grp;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            wb[s][j] = (base + j < k1) ? (kGatherL2Only ? __ldcg(a.val + pb[s][j]) : __ldg(a.val + pb[s][j])) : 0.f;
    };

    // Everything that only depends on the chunk is requested before the
    // operand staging: the first blocks of the stream and the first window of
    // segment starts (and biases).
    if (k0 < k1) {
#pragma unroll
        for (int s = 0; s < NS; ++s)
            if (base_first + s * BLK < k1) issue(s, base_first + s * BLK);
    }
    SegWindow win{cd.z, cd.w - cd.z, 0, 0u, 0.f};
    if (win.nrows > 0) win.load(0, lane, a.seg_ptr, a.bias);
    if constexpr (SMEM) TL::stage(xs, a, threadIdx.x, NT);
    __syncthreads();
    const Elem* xsrc = SMEM ? xs : static_cast<const Elem*>(a.xt);

    Pending pend[2] = {Pending{-1, 0u, 0u}, Pending{-1, 0u, 0u}};
    if (win.nrows > 0) {
        if constexpr (GATHER) {
#pragma unroll
            for (int s = 0; s < G; ++s)
                if (k0 < k1 && base_first + s * BLK < k1) gather(s, base_first + s * BLK);
        }
        const int r_begin = win.r_begin;
        int i = 0;
        uint32_t rs = win.bnd(0, lane, a.seg_ptr, a.bias), re = win.bnd(1, lane, a.seg_ptr, a.bias);
        float acc[VEC];
#pragma unroll
        for (int j = 0; j < VEC; ++j) acc[j] = 0.f;

        auto consume = [&](int s, uint32_t blk0) {
            const uint32_t base = blk0 + 4 * grp;
            if (rs <= blk0 && k0 <= blk0 && blk0 + BLK < re && blk0 + BLK <= k1) {
                // interior block: every entry belongs to the current segment,
                // which continues past the block
#pragma unroll
                for (int j = 0; j < 4; ++j) TL::template axpy<SMEM>(a, xsrc, ib[s].get(j), sub, wb[s][j], acc);
                return;
            }
            const uint32_t blk_end = min(blk0 + BLK, k1);
            while (true) {
                const uint32_t lo_k = max(max(rs, k0), blk0), hi_k = min(re, blk_end);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t k = base + j;
                    if (k >= lo_k && k < hi_k) TL::template axpy<SMEM>(a, xsrc, ib[s].get(j), sub, wb[s][j], acc);
                }
                if (min(re, k1) > blk_end) break;  // segment continues in the next block
                finish_segment<TL>(a, acc, r_begin + i, rs, re, k0, k1, win.bias_of(i), lane, sub,
                                   my_slots, pend);
                if (++i >= win.nrows) break;
                rs = re;
                re = win.bnd(i + 1, lane, a.seg_ptr, a.bias);
                if (rs >= blk_end) break;
            }
        };

        if (k0 < k1) {
            for (uint32_t base0 = base_first; base0 < k1; base0 += NS * BLK) {
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const uint32_t blk0 = base0 + s * BLK;
                    if (blk0 < k1) {
                        if constexpr (GATHER) {
                            if (blk0 + G * BLK < k1) gather((s + G) % NS, blk0 + G * BLK);
                        }
                        consume(s, blk0);
                        if (blk0 + NS * BLK < k1) issue(s, blk0 + NS * BLK);
                    }
                }
            }
        }
        // segments that start at the end of the chunk (empty here)
        while (i < win.nrows) {
            finish_segment<TL>(a, acc, r_begin + i, rs, re, k0, k1, win.bias_of(i), lane, sub,
                               my_slots, pend);
            if (++i >= win.nrows) break;
            rs = re;
            re = win.bnd(i + 1, lane, a.seg_ptr, a.bias);
        }
    }
    if (lane == 0) {
        srow[warp * 2 + 0] = pend[0].r;
        srow[warp * 2 + 1] = pend[1].r;
    }
    __syncthreads();
    block_combine<TL, W>(a, sp, srow, pend, warp, lane, sub);
}

}  // namespace snk
