// Dense products of 8-bit matrices, y = A B^T + bias, on the tensor cores.
//
// A [M, K] and B [N, K] are E4M3 codes with fp32 scales: A's one for each 128 columns of
// a row, B's the same or one for each 128 x 128 block:
//     y_mn = sum_g sa[m, g] sb[n or n / 128, g] (sum_{k in group g} a_mk b_nk) + bias_n
// Products of two codes are exact in fp32; the sum of a group is the tensor cores' (four
// MMA steps of 32 columns), the sum over groups is fp32 with rounding, in order.  Since a
// scale changes every 128 columns, an accumulator lasts one group: two or more of them in
// TMEM take turns, and while the tensor cores fill one the
// epilogue warps multiply another by its scales into registers.
//
// k_q8_dense has the same parts as k_dense (snk_dense.cuh): a stage is one group, 128
// bytes of a row.  k_q8_rows is for up to 16 rows of A, where the codes of B are read
// once and nothing else counts.
#include <algorithm>
#include <type_traits>

#include "snk_dense.cuh"

namespace snk {
namespace {

// Threads as in k_dense; with 216 registers for the sums' threads instead of 232 some spilled
// (8192 x 10000 x 10000 639 us against 612).  With 232 the two kernels of 128 columns spill 12 and 24 bytes, those of
// row scales and 256 columns 4, the others nothing.
constexpr int kQ8Threads = kDenseThreads;
constexpr int kQ8RoleRegs = 40, kQ8SumRegs = 232;
static_assert(shares_fit(kQ8RoleRegs, kQ8SumRegs), "the shares come out of the launch's registers");

struct Q8DenseArgs {
    int64_t M, N;
    int n_g;               // groups along K
    int n_mt, n_nt, splits, group;
    int a_rows, stages;
    uint32_t idesc;
    const float* sa;       // [M, n_g]
    const float* sb;       // [N, n_g] or [ceil(N / 128), n_g]
    const float* bias;     // [N] or null
    void* y;               // [M, N]
    int dtype;
    int vec;               // rows of y (slab) are aligned to 16 bytes: TMA writes them, by map_y
    float* slab;           // splits > 1: [splits][M, N] sums without bias
};

template <int CG>
__device__ __forceinline__ void q8_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}
// ROWS: scales of A's and B's rows, [groups][rows] in the call's scratch, come with the
// stages, into a ring of their own: an epilogue warp reads those of a group after the
// stage of that group may have been filled again, but never as late as the ring is long (it
// frees an accumulator, of which there are up to 4, before it reads the last of them, and TMA
// is up to 8 stages ahead of the MMAs).
constexpr int kScaleSlots = 16;

// A lane's row of a box, 128 bytes with the 128-byte swizzle, and the box's way out.
template <typename T>
__device__ __forceinline__ void put_box(unsigned char* box, int lane, const float (&v)[Turn<T>::kCols]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(v[4 * i + k]);
            else w[k] = pack2<T>(make_float2(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]));
        }
        *reinterpret_cast<uint4*>(box + lane * 128 + 16 * (i ^ (lane & 7))) = make_uint4(w[0], w[1], w[2], w[3]);
    }
}
__device__ __forceinline__ void store_box(const void* box, const CUtensorMap* map, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(map), "r"(x),
                 "r"(y), "r"(z), "r"(smem_u32(box))
                 : "memory");
}

// First of the n groups of a range of K, in 32 bits (n < 2^24, at most 16 splits): 64-bit divisions
// took each tile's start about 0.25 us (32768 x 768 -> 2304: 72 us, now 68).
__device__ __forceinline__ int range_first(int n, int split, int splits) {
    return splits == 1 ? n * split : (int)((uint32_t)n * (uint32_t)split / (uint32_t)splits);
}

// What an epilogue warp's outputs go through: boxes of 32 rows by 128 bytes, two for a pair; one for a CTA
// by itself, whose stages need the room (64 x 768 -> 50257: 17.3 us with two boxes and two stages).
constexpr int out_bytes(int cg) { return cg == 2 ? 2 * 4096 : 5 * 1024; }
static_assert(kTurnBytes <= out_bytes(1) && kTurnBytes <= out_bytes(2), "the other way out uses the same memory");
constexpr int kQ8Smem = 227 * 1024 - 4096;   // (beside the static part)
// Stages: what fits beside the outputs and the scales' ring, 4 for a pair (5 were slower), and an even
// number: each issuing thread then keeps to its own half of the ring and sees every phase of its
// barriers (known by their parity only, a phase may not be waited for while an earlier one is
// open).  a_rows as in dense_stages.
constexpr int kQ8Stages = 8;
inline int q8_stages(int cg, int bn, int a_rows, bool by_rows) {
    const int room = kQ8Smem - 1024 - kDenseEpilogueWarps * out_bytes(cg) - (by_rows ? kScaleSlots * (kDenseM + bn) * 4 : 0) -
                     (kDenseM - a_rows) * 128;
    return cg == 2 ? 4 : std::min(kQ8Stages, room / ((a_rows + bn) * 128)) & ~1;
}

template <int CG, int BN, bool ROWS>
__global__ void __launch_bounds__(kQ8Threads, 1)
    k_q8_dense(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
               const __grid_constant__ CUtensorMap map_sa, const __grid_constant__ CUtensorMap map_sb,
               const __grid_constant__ CUtensorMap map_y, const Q8DenseArgs a) {
    constexpr int S = kQ8Stages;
    constexpr int HC = BN / 2;    // columns of an epilogue warp
    constexpr int HB = BN / CG;   // rows of B that a CTA loads
    constexpr int kUnroll = ROWS ? 2 : 1;   // (8192^3: with row scales 566 us without, with blocks 757 with)
    constexpr int kOutBytes = out_bytes(CG), BOXES = kOutBytes / 4096;
    constexpr int NB = BN == 256 ? 2 : 4;   // accumulators (an even number, as the stages)
    extern __shared__ __align__(1024) unsigned char q8_raw[];
    unsigned char* sm = q8_raw + ((1024 - (smem_u32(q8_raw) & 1023)) & 1023);
    // outputs of each epilogue warp; ROWS: scales [kScaleSlots][kDenseM + BN]; stages
    unsigned char* turn = sm;
    float* scales = reinterpret_cast<float*>(turn + kDenseEpilogueWarps * kOutBytes);
    unsigned char* stages = turn + kDenseEpilogueWarps * kOutBytes + (ROWS ? kScaleSlots * (kDenseM + BN) * 4 : 0);
    const int a_bytes = a.a_rows * 128, stage = a_bytes + HB * 128;
    const uint32_t stage_tx = (uint32_t)(stage + (ROWS ? (kDenseM + BN) * 4 : 0));   // with its scales
    __shared__ uint64_t full[S], empty[S], accf[NB], acce[NB], fin[2], sink[NB];
    __shared__ PairEnd peer;
    __shared__ uint32_t tmem_base;

    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int rank = CG == 1 ? 0 : (int)cluster_rank();
    if (t == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < NB; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&acce[i], kDenseEpilogueWarps * CG);
            mbar_init(&sink[i], kSinkCount);
        }
        mbar_init(&fin[0], 1);
        mbar_init(&fin[1], 1);
        mbar_init(&peer.bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    if (warp == 3) tmem_alloc<CG>(&tmem_base, 512);
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    const uint32_t tmem = tmem_base;
    after_previous();
    let_next_start();
    const int items = a.n_mt * a.n_nt * a.splits;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;

    if (warp < 4) {
        fewer_registers<kQ8RoleRegs>();
        if (warp == 0 && lane == 0) {
            bool ok = true, used = false;   // used: every slot has been filled once
            Stages r(a.stages);
            uint32_t w = 0;   // groups loaded
            for (int id = first; id < items && ok; id += step) {
                const DenseItem it = DenseItem::of(id, a.n_mt, a.n_nt, a.splits, a.group);
                const int g0 = range_first(a.n_g, it.split, a.splits), g1 = range_first(a.n_g, it.split + 1, a.splits);
                const int m0 = (it.mt * CG + rank) * kDenseM, n0 = it.nt * BN + rank * HB;
                for (int g = g0; g < g1; ++g, ++w) {
                    const int s = r.slot;
                    if (used && !mbar_wait(&empty[s], r.parity ^ 1)) {
                        ok = false;
                        break;
                    }
                    unsigned char* sa = stages + s * stage;
                    unsigned char* sb = sa + a_bytes;
                    if (rank == 0) mbar_expect_tx(&full[s], stage_tx * CG);
                    const uint32_t bar = CG == 1 ? smem_u32(&full[s]) : first_cta(&full[s]);
                    dense_load<CG>(sa, &map_a, g * 128, m0, bar);
                    dense_load<CG>(sb, &map_b, g * 128, n0, bar);
                    if constexpr (ROWS) {
                        float* at = scales + (w % kScaleSlots) * (kDenseM + BN);
                        dense_load<CG>(at, &map_sa, m0, g, bar);
                        dense_load<CG>(at + kDenseM, &map_sb, it.nt * BN, g, bar);
                    }
                    r.next();
                    used |= r.slot == 0;
                }
            }
            land_all<CG>(full, fin, peer, rank, w, a.stages, stage_tx);
        }
        // Two threads issue, one the even groups and one the odd ones: a group takes the tensor
        // cores 512 cycles, but its thread 1000 (issue blocks while they are busy, and two
        // waits and two commits add what they take even when nothing is to be waited for).
        if ((warp == 1 || warp == 2) && lane == 0 && rank == 0) {
            const uint32_t mine = warp - 1;
            bool ok = true;
            Stages r(a.stages);
            uint32_t w = 0;   // groups done
            for (int id = first; id < items && ok; id += step) {
                const DenseItem it = DenseItem::of(id, a.n_mt, a.n_nt, a.splits, a.group);
                const int g0 = range_first(a.n_g, it.split, a.splits), g1 = range_first(a.n_g, it.split + 1, a.splits);
                for (int g = g0; g < g1; ++g, ++w, r.next()) {
                    if ((w & 1) != mine) continue;
                    const int s = r.slot, ab = (int)(w % NB);
                    if (!mbar_wait(&full[s], r.parity) || (w >= NB && !mbar_wait(&acce[ab], (w / NB - 1) & 1))) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint32_t sa = smem_u32(stages + s * stage), sb = sa + a_bytes;
#pragma unroll
                    for (int kk = 0; kk < 4; ++kk)
                        q8_mma<CG>(tmem + ab * BN, desc_sw128(sa + kk * 32), desc_sw128(sb + kk * 32), a.idesc, kk > 0 ? 1u : 0u);
                    dense_commit<CG>(&accf[ab]);
                    dense_commit<CG>(&empty[s]);
                }
            }
            dense_commit<CG>(&fin[mine]);
        }
    } else {
        more_registers<kQ8SumRegs>();
        const int half = warp >= 8 ? 1 : 0, quarter = warp & 3;
        const uint32_t lanes = tmem + half * HC + ((uint32_t)(quarter * 32) << 16);
        uint32_t base = CG == 1 ? smem_u32(acce) : first_cta(acce);
        bool ok = true;
        uint32_t w = 0;   // groups done
        for (int id = first; id < items; id += step) {
            const DenseItem it = DenseItem::of(id, a.n_mt, a.n_nt, a.splits, a.group);
            const int g0 = range_first(a.n_g, it.split, a.splits), g1 = range_first(a.n_g, it.split + 1, a.splits);
            const int64_t row = (int64_t)(it.mt * CG + rank) * kDenseM + quarter * 32 + lane;
            const int64_t col = (int64_t)it.nt * BN + half * HC;
            // rows and columns outside the matrix read the last ones' scales and are not stored
            const float* pa = a.sa + min(row, a.M - 1) * a.n_g;
            const float* pb = a.sb + (min(col, a.N - 1) >> 7) * a.n_g;
            float2 acc[HC / 2];
#pragma unroll
            for (int j = 0; j < HC / 2; ++j) acc[j] = make_float2(0.f, 0.f);
            float na = 0.f, nb = 0.f;   // the next group's scales
            if (!ROWS && g0 < g1) {
                na = __ldg(pa + g0);
                nb = __ldg(pb + g0);
            }
#pragma unroll kUnroll
            for (int g = g0; g < g1; ++g, ++w) {
                const int ab = (int)(w % NB);
                float s = na * nb;
                if (!ROWS && g + 1 < g1) {
                    na = __ldg(pa + g + 1);
                    nb = __ldg(pb + g + 1);
                }
                const float* at = scales + (w % kScaleSlots) * (kDenseM + BN);
                const float* sbp = at + kDenseM + half * HC;
                if (ok && !mbar_wait(&accf[ab], (w / NB) & 1)) {
                    ok = false;
                    base = smem_u32(sink);
                }
                if constexpr (ROWS) {
                    ok = __all_sync(0xffffffffu, ok);
                    if (!ok) base = smem_u32(sink);
                } else {   // (the lanes agree on ok at the end: 8192^3 416 -> 396 us; what lane 0, which gives back, has
                    __syncwarp();   // waited for is there for all)
                }
                tc_fence_after();
                if constexpr (ROWS) s = at[quarter * 32 + lane];
                const uint32_t ta = lanes + ab * BN;
                uint32_t r[2][32];   // the next 32 columns are read while these are added
                tmem_ld32_async(ta, r[0]);
#pragma unroll
                for (int c = 0; c < HC; c += 32) {
                    tmem_wait_ld();
                    if (c + 32 < HC) {
                        tmem_ld32_async(ta + c + 32, r[(c / 32 + 1) & 1]);
                    } else {   // all read: the accumulator is free before its last columns are added
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) give_back<CG>(base + 8 * ab);
                    }
                    const uint32_t(&u)[32] = r[(c / 32) & 1];
#pragma unroll
                    for (int j = 0; j < 32; j += 4) {
                        float2 f0 = make_float2(s, s), f1 = f0;
                        if constexpr (ROWS) {
                            const float4 b4 = *reinterpret_cast<const float4*>(sbp + c + j);
                            f0 = __fmul2_rn(f0, make_float2(b4.x, b4.y));
                            f1 = __fmul2_rn(f1, make_float2(b4.z, b4.w));
                        }
                        float2 &x = acc[(c + j) / 2], &y = acc[(c + j) / 2 + 1];
                        x = __ffma2_rn(make_float2(__uint_as_float(u[j]), __uint_as_float(u[j + 1])), f0, x);
                        y = __ffma2_rn(make_float2(__uint_as_float(u[j + 2]), __uint_as_float(u[j + 3])), f1, y);
                    }
                }
            }
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) {
                base = smem_u32(sink);
#pragma unroll
                for (int j = 0; j < HC / 2; ++j) acc[j] = make_float2(__int_as_float(0x7fc00000), __int_as_float(0x7fc00000));
            }
            const int64_t row0 = row - lane;
            const int rows = (int)max((int64_t)0, min((int64_t)32, a.M - row0)), cols = (int)min((int64_t)HC, a.N - col);
            unsigned char* buf = turn + (warp - 4) * kOutBytes;
            if (a.vec && lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");   // the last tile's boxes have left
            __syncwarp();
            auto store = [&](auto* y, const float* bias) {
                using T = typename std::remove_pointer<decltype(y)>::type;
                constexpr int E = Turn<T>::kCols;
                y += row0 * a.N + col;
#pragma unroll
                for (int c = 0; c < HC; c += E) {
                    if (c < cols) {
                        float v[E];
#pragma unroll
                        for (int j = 0; j < E; ++j) v[j] = c + j >= HC ? 0.f : ((j & 1) ? acc[(c + j) / 2 % (HC / 2)].y : acc[(c + j) / 2 % (HC / 2)].x);
                        if (bias && c + E <= cols && HC >= E && ((uintptr_t)(bias + col) & 15) == 0) {
#pragma unroll
                            for (int j = 0; j < E; j += 4) {
                                const float4 b4 = __ldg(reinterpret_cast<const float4*>(bias + col + c + j));
                                v[j] += b4.x;
                                v[j + 1] += b4.y;
                                v[j + 2] += b4.z;
                                v[j + 3] += b4.w;
                            }
                        } else if (bias) {
#pragma unroll
                            for (int j = 0; j < E; ++j)
                                if (c + j < cols) v[j] += __ldg(bias + col + c + j);
                        }
                        if (E <= HC && a.vec) {
                            // the writes leave while the next tile's groups are added
                            unsigned char* box = buf + (c / E % BOXES) * 4096;
                            if (c >= BOXES * E) {   // the box's last content has left
                                if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(BOXES - 1) : "memory");
                                __syncwarp();
                            }
                            put_box<T>(box, lane, v);
                            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                            __syncwarp();
                            if (lane == 0) {
                                if (rows > 0) store_box(box, &map_y, (int)(col + c), (int)row0, it.split);
                                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
                            }
                        } else {
                            Turn<T>::put(buf, lane, v);
                            Turn<T>::flush(buf, lane, y + c, a.N, rows, cols - c, a.vec);
                        }
                    }
                }
            };
            if (a.splits > 1) store(a.slab + it.split * a.M * a.N, nullptr);
            else if (a.dtype == SNK_F32) store(static_cast<float*>(a.y), a.bias);
            else if (a.dtype == SNK_F16) store(static_cast<__half*>(a.y), a.bias);
            else store(static_cast<__nv_bfloat16*>(a.y), a.bias);
        }
        if (a.vec && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    }
    if (warp == 3) wait_for_mmas(fin);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();
    tc_fence_after();
    if (warp == 3) tmem_free<CG>(tmem, 512);
}
// Scales [rows, n_g] of A (even blocks) or B (odd ones) as [n_g][padded], zeros behind the rows.
__global__ void __launch_bounds__(256) k_q8_scales(const float* __restrict__ sa, int64_t M, int64_t padded_m, float* __restrict__ ta,
                                                   const float* __restrict__ sb, int64_t N, int64_t padded_n, float* __restrict__ tb,
                                                   int n_g) {
    __shared__ float sm[32][33];
    after_previous();
    let_next_start();
    const bool second = blockIdx.x & 1;
    const float* src = second ? sb : sa;
    float* dst = second ? tb : ta;
    const int64_t rows = second ? N : M, padded = second ? padded_n : padded_m;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t tiles_g = (n_g + 31) / 32, tiles = padded / 32 * tiles_g;
    for (int64_t id = blockIdx.x >> 1; id < tiles; id += gridDim.x >> 1) {
        const int64_t r0 = id / tiles_g * 32;
        const int g0 = (int)(id % tiles_g) * 32;
#pragma unroll
        for (int i = warp; i < 32; i += 8) sm[i][lane] = r0 + i < rows && g0 + lane < n_g ? __ldg(src + (r0 + i) * n_g + g0 + lane) : 0.f;
        __syncthreads();
#pragma unroll
        for (int i = warp; i < 32; i += 8)
            if (g0 + i < n_g) dst[(int64_t)(g0 + i) * padded + r0 + lane] = sm[lane][i];
        __syncthreads();
    }
}

// The sum of the splits' parts, in order, and the bias; V outputs a thread: 4 where rows are whole fours
// and still fill the device (with the product: 2304 x 768 over 32768 tokens, 5 parts, 79.1 -> 77.0 us;
// 512 x 8192 -> 2048 17.8 -> 15.9; 300 x 300, 16 parts, 15.2 by ones and 19.8 by fours).
template <typename T, int V>
__global__ void __launch_bounds__(256) k_q8_join(const float* __restrict__ slab, int splits, int64_t M, int64_t N,
                                                 const float* __restrict__ bias, T* __restrict__ y) {
    const int64_t n = M * N;
    after_previous();   // (the next kernel started beside it cost 0.5 to 2 us)
    for (int64_t i = V * ((int64_t)blockIdx.x * 256 + threadIdx.x); i < n; i += V * (int64_t)gridDim.x * 256) {
        float v[V] = {};
#pragma unroll 4
        for (int s = 0; s < splits; ++s) {
            if constexpr (V == 4) {
                const float4 p = __ldg(reinterpret_cast<const float4*>(slab + s * n + i));
                v[0] += p.x;
                v[1] += p.y;
                v[2] += p.z;
                v[3] += p.w;
            } else {
                v[0] += __ldg(slab + s * n + i);
            }
        }
        if (bias) {
            const int64_t c = i % N;
#pragma unroll
            for (int j = 0; j < V; ++j) v[j] += __ldg(bias + c + j);
        }
        if constexpr (V == 1) {
            y[i] = from_f32<T>(v[0]);
        } else if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float4*>(y + i) = make_float4(v[0], v[1], v[2], v[3]);
        } else {
            *reinterpret_cast<uint2*>(y + i) = make_uint2(pack2<T>(make_float2(v[0], v[1])), pack2<T>(make_float2(v[2], v[3])));
        }
    }
}

// ---- few rows ---------------------------------------------------------------------
// Up to 16 rows of A: the call reads B's codes once, N K bytes, and little else, so it is
// bound by memory and, for small layers, by latency (one row, 2304 x 768: 1.8 us; 50257 x 768:
// 9 us, 4.3 TB/s).  A warp takes 16 rows of B and some
// of the groups; the block's warps share the groups and are added through shared memory.
// The products are mma.sync m16n8k32 (B's rows as its 16, A's as its 8): a dot product
// does not care for the order of its columns, so each lane takes 16 consecutive bytes of
// its two rows of B and of its row of A, 64 columns for four lanes, as the operands of two
// MMAs.
constexpr int kRowsMax = 16;
constexpr int kRowsWarps = 8;

__device__ __forceinline__ void mma_e4m3(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// 16 codes of a row from column k on, zeros from K on (what lies there is not read).
__device__ __forceinline__ uint4 load16(const uint8_t* row, int64_t k, int64_t K) {
    if (k + 16 <= K) return __ldg(reinterpret_cast<const uint4*>(row + k));
    uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < 15; ++i)
        if (k + i < K) w[i >> 2] |= (uint32_t)row[k + i] << (8 * (i & 3));
    return make_uint4(w[0], w[1], w[2], w[3]);
}

struct Q8RowsArgs {
    const uint8_t *a, *b;
    int64_t lda, ldb;      // multiples of 16
    int64_t M, N, K;
    int n_g;
    const float *sa, *sb;
    const float* bias;
    void* y;
    int blocks_b;          // B's scales are of 128 x 128 blocks
};
// NT: tiles of 8 rows of A.
template <int NT, typename T>
__global__ void __launch_bounds__(32 * kRowsWarps, NT == 1 ? 4 : 2) k_q8_rows(const Q8RowsArgs a) {
    __shared__ float part[kRowsWarps][16][8 * NT + 1];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, q = lane & 3, r = lane >> 2;
    after_previous();
    let_next_start();
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t nr0 = n0 + r, nr1 = n0 + r + 8;
    const uint8_t* b0 = a.b + min(nr0, a.N - 1) * a.ldb;
    const uint8_t* b1 = a.b + min(nr1, a.N - 1) * a.ldb;
    float acc[NT][4];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) acc[i][j] = 0.f;
    for (int g = warp; g < a.n_g; g += kRowsWarps) {
        float d[NT][4];
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[i][j] = 0.f;
        uint4 w0[2], w1[2], x[NT][2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const int64_t k = (int64_t)g * 128 + h * 64 + q * 16;
            w0[h] = load16(b0, k, a.K);
            w1[h] = load16(b1, k, a.K);
#pragma unroll
            for (int i = 0; i < NT; ++i) x[i][h] = load16(a.a + min((int64_t)(8 * i + r), a.M - 1) * a.lda, k, a.K);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < NT; ++i) {
                mma_e4m3(d[i], w0[h].x, w1[h].x, w0[h].y, w1[h].y, x[i][h].x, x[i][h].y);
                mma_e4m3(d[i], w0[h].z, w1[h].z, w0[h].w, w1[h].w, x[i][h].z, x[i][h].w);
            }
        // d[i]: rows r, r + 8 of B; rows 8 i + 2 q, + 1 of A
        const float s0 = a.blocks_b ? __ldg(a.sb + (n0 >> 7) * a.n_g + g) : __ldg(a.sb + min(nr0, a.N - 1) * a.n_g + g);
        const float s1 = a.blocks_b ? s0 : __ldg(a.sb + min(nr1, a.N - 1) * a.n_g + g);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const int m = 8 * i + 2 * q;
            const float t0 = m < a.M ? __ldg(a.sa + (int64_t)m * a.n_g + g) : 0.f;
            const float t1 = m + 1 < a.M ? __ldg(a.sa + (int64_t)(m + 1) * a.n_g + g) : 0.f;
            acc[i][0] = fmaf(d[i][0], s0 * t0, acc[i][0]);
            acc[i][1] = fmaf(d[i][1], s0 * t1, acc[i][1]);
            acc[i][2] = fmaf(d[i][2], s1 * t0, acc[i][2]);
            acc[i][3] = fmaf(d[i][3], s1 * t1, acc[i][3]);
        }
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        part[warp][r][8 * i + 2 * q] = acc[i][0];
        part[warp][r][8 * i + 2 * q + 1] = acc[i][1];
        part[warp][r + 8][8 * i + 2 * q] = acc[i][2];
        part[warp][r + 8][8 * i + 2 * q + 1] = acc[i][3];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * 8 * NT; i += 32 * kRowsWarps) {
        const int n = i & 15, m = i >> 4;
        if (n0 + n < a.N && m < a.M) {
            float v = 0.f;
#pragma unroll
            for (int k = 0; k < kRowsWarps; ++k) v += part[k][n][m];
            if (a.bias) v += __ldg(a.bias + n0 + n);
            static_cast<T*>(a.y)[m * a.N + n0 + n] = from_f32<T>(v);
        }
    }
}

// ---- host ------------------------------------------------------------------------------

int64_t up(int64_t n, int64_t m) { return ceil_div(n, m) * m; }

// Scales [n_g][padded] in boxes of one group and `box` rows.
bool scales_map(CUtensorMap* map, const float* base, int64_t padded, int n_g, int box_rows) {
    EncodeTiledFn fn = encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)padded, (cuuint64_t)n_g};
    cuuint64_t strides[1] = {(cuuint64_t)padded * 4};
    cuuint32_t box[2] = {(cuuint32_t)box_rows, 1u};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, const_cast<float*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
// y (or each split's sums) in boxes of 32 rows by 128 bytes.
bool out_map(CUtensorMap* map, void* base, int dtype, int64_t rows, int64_t cols, int splits) {
    EncodeTiledFn fn = encoder();
    if (!fn) return false;
    const int e = dtype == SNK_F32 ? 4 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)cols, (cuuint64_t)rows, (cuuint64_t)splits};
    cuuint64_t strides[2] = {(cuuint64_t)cols * e, (cuuint64_t)(rows * cols) * e};
    cuuint32_t box[3] = {(cuuint32_t)(128 / e), 32u, 1u};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map,
              dtype == SNK_F32   ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32
              : dtype == SNK_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16,
              3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
bool q8_map(CUtensorMap* map, const uint8_t* base, int64_t len, int64_t rows, int64_t ld, int box_rows) {
    EncodeTiledFn fn = encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)len, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld};
    cuuint32_t box[2] = {128u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<uint8_t*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Q8Plan {
    bool rows;               // k_q8_rows
    bool copy_a, copy_b;
    int cg, bn, n_mt, n_nt, splits;
    int64_t ld;              // of the copies
    uint8_t *a, *b;
    float* slab;
    int64_t padded_m, padded_n;   // scales by rows: their transposed copies' rows
    float *ta, *tb;
    int64_t bytes;
    Q8Plan(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, bool blocks, int num_sms, void* scratch) {
        copy_a = lda % 16 != 0;
        copy_b = ldb % 16 != 0;
        ld = up(K, 16);
        const int n_g = (int)ceil_div(K, 128);
        // The tile and the ranges of K whose waves take least. Times in us as measured where all SMs are busy (full
        // waves of tiles, K = 512 to 16384): of a group, with scales of blocks and of rows; of a tile beside its groups; of
        // joining ranges and their sums, written and read: 8 bytes at 8 TB/s from the L2 (2304 x 768 over 32768: 5 ranges
        // 77 us, 2 ranges 87), at half of it where they do not stay there.  A CTA by itself with 256 columns is bound by
        // the L2's bytes (0.8 for all SMs), by its own accumulators where few are busy.  Over 62 shapes (17 to
        // 16384 rows) times both kinds of scales the form so chosen takes 1% more than the best one, 19% at most.
        struct Form {
            int cg, bn;
            double blocks, rows;
        };
        constexpr Form forms[] = {{2, 256, 0.44, 0.60}, {1, 256, 0.50, 0.75}, {1, 128, 0.36, 0.41}, {1, 64, 0.30, 0.335}};
        double best = 1e30;
        for (const Form& f : forms) {
            if (f.cg == 2 && M <= 128) continue;
            const int64_t mt = ceil_div(M, 128 * f.cg), nt = ceil_div(N, f.bn), units = num_sms / f.cg;
            for (int sp = 1; sp <= 16 && (sp == 1 || n_g / sp >= 4); ++sp) {
                const double waves = (double)ceil_div(mt * nt * sp, units), busy = std::min(1.0, (double)(mt * nt * sp) / (double)units);
                const double group = std::max(blocks ? f.blocks : f.rows, f.cg == 1 && f.bn == 256 ? 0.8 * busy : 0.0);
                const double t = waves * ((double)ceil_div(n_g, sp) * group + 1.5) +
                                 (sp > 1 ? 2.0 + (4.0 * sp * M * N < 64e6 ? 1e-6 : 2e-6) * sp * M * N : 0.0);
                if (t < best) {
                    best = t;
                    cg = f.cg;
                    bn = f.bn;
                    splits = sp;
                }
            }
        }
        // Few rows: B's codes once by mma.sync, by the waves of its blocks (4 to an SM, 2 with two tiles of rows) and the
        // rounds of a block's warps over the groups.  us, W from memory, blocks' scales, this and the tiles: 8 rows
        // 768 -> 2304 1.8 and 4.4, 4096 -> 4096 6.6 and 10.3, 768 -> 50257 12.0 and 13.4, 12288 -> 8192 21.0 and 23.9, 10000 -> 10000
        // 29.9 and 24.4; 16 rows 4096 -> 4096 7.4 and 10.6, 768 -> 50257 19.2 and 14.0.  Tiles take 2 us beside the account
        // above, 4 with the turning of rows' scales.
        const double few = 1.3 + (M <= 8 ? 1.5 : 1.35) * (double)ceil_div(ceil_div(N, 16), (M <= 8 ? 4 : 2) * num_sms) *
                                     (double)ceil_div(n_g, kRowsWarps);
        rows = M <= kRowsMax && few <= best + (blocks ? 2.0 : 4.0);
        if (rows) splits = 1;
        n_mt = (int)ceil_div(M, 128 * cg);
        n_nt = (int)ceil_div(N, bn);
        char* p = static_cast<char*>(scratch);
        int64_t used = 0;
        auto take = [&](int64_t n) {
            char* q = p + used;
            used += up(n, 256);
            return q;
        };
        a = reinterpret_cast<uint8_t*>(take(copy_a ? M * ld : 0));
        b = reinterpret_cast<uint8_t*>(take(copy_b ? N * ld : 0));
        slab = reinterpret_cast<float*>(take(splits > 1 ? 4 * splits * M * N : 0));
        padded_m = up(M, 128 * cg);
        padded_n = up(N, bn);
        const bool turn = !rows && !blocks;
        ta = reinterpret_cast<float*>(take(turn ? 4 * n_g * padded_m : 0));
        tb = reinterpret_cast<float*>(take(turn ? 4 * n_g * padded_n : 0));
        bytes = used;
    }
};

template <int CG, int BN, bool ROWS>
int launch_dense(const CUtensorMap (&m)[5], const Q8DenseArgs& a, int num_sms, cudaStream_t s) {
    constexpr auto f = k_q8_dense<CG, BN, ROWS>;
    if (!allow_smem<f>(kQ8Smem)) return SNK_ERR_CUDA;
    const int64_t items = (int64_t)a.n_mt * a.n_nt * a.splits;
    return launch_after(f, (unsigned)(CG * std::min<int64_t>(items, num_sms / CG)), kQ8Threads, kQ8Smem, CG, s, m[0], m[1], m[2], m[3],
                        m[4], a);
}
template <bool ROWS>
int launch_dense(const Q8Plan& p, const CUtensorMap (&m)[5], const Q8DenseArgs& a, int num_sms, cudaStream_t s) {
    if (p.cg == 2) return launch_dense<2, 256, ROWS>(m, a, num_sms, s);
    if (p.bn == 256) return launch_dense<1, 256, ROWS>(m, a, num_sms, s);
    if (p.bn == 128) return launch_dense<1, 128, ROWS>(m, a, num_sms, s);
    return launch_dense<1, 64, ROWS>(m, a, num_sms, s);
}
template <typename T>
int launch_rows(const Q8RowsArgs& r, cudaStream_t s) {
    const unsigned blocks = (unsigned)ceil_div(r.N, 16);
    return r.M <= 8 ? launch_after(k_q8_rows<1, T>, blocks, 32 * kRowsWarps, 0, 1, s, r)
                    : launch_after(k_q8_rows<2, T>, blocks, 32 * kRowsWarps, 0, 1, s, r);
}
template <typename T>
int launch_join(const Q8Plan& p, int64_t M, int64_t N, const float* bias, void* y, int num_sms, cudaStream_t s) {
    const bool fours = N % 4 == 0 && ((uintptr_t)y & (4 * sizeof(T) - 1)) == 0 && M * N >= 2048 * num_sms;
    const unsigned blocks = (unsigned)std::min<int64_t>(ceil_div(M * N, fours ? 1024 : 256), (fours ? 32 : 8) * num_sms);
    return launch_after(fours ? k_q8_join<T, 4> : k_q8_join<T, 1>, blocks, 256, 0, 1, s, p.slab, p.splits, M, N, bias, static_cast<T*>(y));
}

int bad_product(int64_t M, int64_t N, int64_t K) {
    if (M < 0 || N < 1 || K < 1) return SNK_ERR_ARG;
    const int64_t lim = INT32_MAX - 512;
    if (M > lim || N > lim || K > lim || (double)ceil_div(M, 128) * (double)ceil_div(N, 64) > 1.0e9) return SNK_ERR_LIMIT;
    return SNK_OK;
}

}  // namespace
}  // namespace snk

using namespace snk;

extern "C" {

int64_t snk_q8_matmul_scratch(int64_t M, int64_t N, int64_t K, int64_t lda, int64_t ldb, int b_blocks) {
    if (M < 1 || bad_product(M, N, K) != SNK_OK) return 0;
    const int n = device_sms();
    return n < 1 ? 0 : Q8Plan(M, N, K, lda, ldb, b_blocks, n, nullptr).bytes;
}

int snk_q8_matmul(const void* a, int64_t lda, const float* a_scales, const void* b, int64_t ldb, const float* b_scales,
                  int b_blocks, int64_t M, int64_t N, int64_t K, const float* bias, void* y, int dtype, void* scratch,
                  void* stream) {
    if (int st = bad_product(M, N, K); st != SNK_OK) return st;
    if (dtype < SNK_F32 || dtype > SNK_BF16 || lda < K || ldb < K) return SNK_ERR_ARG;
    auto off = [](const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) != 0; };
    if (!b || !b_scales || off(a, 16) || off(b, 16) || off(a_scales, 4) || off(b_scales, 4) || off(bias, 4) ||
        off(y, dtype == SNK_F32 ? 4 : 2) || off(scratch, 256))
        return SNK_ERR_ARG;
    if (M == 0) return SNK_OK;
    if (!a || !a_scales || !y) return SNK_ERR_ARG;
    const int n = device_sms();
    if (n < 1) return SNK_ERR_CUDA;
    const Q8Plan p(M, N, K, lda, ldb, b_blocks, n, scratch);
    if (p.bytes > 0 && !scratch) return SNK_ERR_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    auto copy = [&](const void* src, int64_t ld, uint8_t* dst, int64_t rows) {
        return launch_after(k_pad_rows, (unsigned)std::min<int64_t>(ceil_div(rows * ceil_div(p.ld, 512), 8), 1 << 20), 256, 0, 1, s, static_cast<const uint8_t*>(src),
                            ld, dst, rows, K, p.ld);
    };
    const uint8_t *pa = static_cast<const uint8_t*>(a), *pb = static_cast<const uint8_t*>(b);
    if (p.copy_a) {
        if (int st = copy(a, lda, p.a, M); st != SNK_OK) return st;
        pa = p.a;
        lda = p.ld;
    }
    if (p.copy_b) {
        if (int st = copy(b, ldb, p.b, N); st != SNK_OK) return st;
        pb = p.b;
        ldb = p.ld;
    }
    const int n_g = (int)ceil_div(K, 128);
    if (p.rows) {
        const Q8RowsArgs r{pa, pb, lda, ldb, M, N, K, n_g, a_scales, b_scales, bias, y, b_blocks};
        return dtype == SNK_F32 ? launch_rows<float>(r, s) : dtype == SNK_F16 ? launch_rows<__half>(r, s) : launch_rows<__nv_bfloat16>(r, s);
    }
    CUtensorMap m[5];
    const int a_rows = (int)std::min<int64_t>(kDenseM, up(M, 8));
    if (!q8_map(&m[0], pa, K, M, lda, a_rows) || !q8_map(&m[1], pb, K, N, ldb, p.bn / p.cg)) return SNK_ERR_CUDA;
    m[2] = m[3] = m[4] = m[0];
    if (!b_blocks) {
        if (!scales_map(&m[2], p.ta, p.padded_m, n_g, kDenseM) || !scales_map(&m[3], p.tb, p.padded_n, n_g, p.bn)) return SNK_ERR_CUDA;
        const int64_t tiles = std::max(p.padded_m, p.padded_n) / 32 * ceil_div(n_g, 32);
        if (int st = launch_after(k_q8_scales, 2 * (unsigned)std::min<int64_t>(tiles, 16 * n), 256, 0, 1, s, a_scales, M, p.padded_m, p.ta,
                                  b_scales, N, p.padded_n, p.tb, n_g);
            st != SNK_OK)
            return st;
    }
    Q8DenseArgs q = {};
    q.M = M;
    q.N = N;
    q.n_g = n_g;
    q.a_rows = a_rows;
    q.stages = q8_stages(p.cg, p.bn, a_rows, !b_blocks);
    q.n_mt = p.n_mt;
    q.n_nt = p.n_nt;
    q.splits = p.splits;
    q.group = 16 / p.cg;
    q.idesc = (1u << 4) | ((uint32_t)(p.bn >> 3) << 17) | ((uint32_t)((128 * p.cg) >> 4) << 24);   // fp32; E4M3, K-major
    q.sa = a_scales;
    q.sb = b_scales;
    q.bias = bias;
    q.y = y;
    q.dtype = dtype;
    q.slab = p.slab;
    const int e = p.splits > 1 || dtype == SNK_F32 ? 4 : 2;
    const uintptr_t base = (uintptr_t)(p.splits > 1 ? (void*)p.slab : y) | (uintptr_t)(N * e);
    q.vec = (base & 15) == 0;
    if (q.vec && !out_map(&m[4], p.splits > 1 ? p.slab : y, p.splits > 1 ? SNK_F32 : dtype, M, N, p.splits)) return SNK_ERR_CUDA;
    const int st = b_blocks ? launch_dense<false>(p, m, q, n, s) : launch_dense<true>(p, m, q, n, s);
    if (st != SNK_OK || p.splits == 1) return st;
    return dtype == SNK_F32   ? launch_join<float>(p, M, N, bias, y, n, s)
           : dtype == SNK_F16 ? launch_join<__half>(p, M, N, bias, y, n, s)
                              : launch_join<__nv_bfloat16>(p, M, N, bias, y, n, s);
}

}  // extern "C"
