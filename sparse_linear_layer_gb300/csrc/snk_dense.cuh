// Dense products of 16-bit matrices on the tensor cores: D = A B^T tile by tile, with
// the epilogue as a type.  Used by the vocabulary loss (snk_vocab.cu).
//
// A is [M, K] and B [N, K], each stored along K (rows of the matrix, "K-major") or along
// its own dimension ("MN-major": the matrix lies transposed in memory); either way TMA
// brings 128-byte wide boxes with the 128-byte swizzle.  A tile is 128 CG rows by `bn`
// columns, CG the CTAs that share it: a pair (CG = 2) runs one MMA of 256 rows over both
// SMs, each holding its 128 rows of A and half of B's columns, so that B crosses the L2
// once per pair.  Persistent CTAs, twelve warps:
//   warp 0     TMA loads into a ring of stages (64 columns of K each);
//   warps 1, 2 issue the MMAs (a thread each, of the pair's first CTA), one the even
//              accumulator turns and one the odd ones;
//   warp 3     owns the TMEM allocation, two accumulators of up to 256 columns that take turns;
//   warps 4-11 the epilogue: warp w reads the TMEM lanes 32 (w % 4) .. + 31 and, by
//              w < 8 or not, the first or second half of the columns.
// Every wait is bounded (kTcWaitCycles). A producer or an issuing thread whose wait ran out
// stops; an epilogue warp whose wait ran out writes NaN for that tile and all that it still has,
// and gives no accumulator back any more (it arrives on the sink): arrivals are only counted, and one too many would
// stand for a warp that still reads. The others then run out too. No CTA ends before its copies
// have landed (land_all) and its MMAs are done (fin), whoever stopped.
#pragma once

#include "snk_q8.cuh"
#include "snk_tcgen.cuh"

namespace snk {

constexpr int kDenseM = 128;             // rows of a tile per CTA (TMEM lanes)
constexpr int kDenseN = 256;             // columns of a tile at most
constexpr int kDenseK = 64;              // columns of K per stage: 128 bytes
// Four warps of roles and eight of the epilogue, whose threads may keep 128 sums; registers as launched
// (168 a thread) and as redistributed (with 40 and 232 the dual tiles' roles spill: dW of 100 x 768 -> 50257 37.5 us, 34.7 without).
constexpr int kDenseThreads = 384;
constexpr int kRoleRegs = 48, kSumRegs = 224;
constexpr bool shares_fit(int role, int sum) { return 128 * role + 256 * sum <= kDenseThreads * 168; }
static_assert(shares_fit(kRoleRegs, kSumRegs), "the shares come out of the launch's registers");
template <int R>
__device__ __forceinline__ void fewer_registers() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(R)); }
template <int R>
__device__ __forceinline__ void more_registers() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(R)); }
constexpr int kDenseEpilogueWarps = 8;
constexpr int kDenseBoxBytes = 64 * 128;   // an MN-major box: 64 rows of K, 64 columns
constexpr int kDenseStages = 8;          // at most
constexpr int kDenseStageRoom = 192 * 1024;
constexpr int kDenseSmem = kDenseStageRoom + 1024;

struct DenseArgs {
    int n_mt, n_nt;        // tiles
    int bn;                // columns of a tile
    int a_rows;            // rows of A that a CTA loads of a tile: 128, or fewer where there is one tile of fewer
    int stages;
    int splits;            // ranges of K, each an item of its own
    int turn_stages;       // k_dense<.., TURNS>: stages that an accumulator adds at most
    int64_t K;
    uint32_t idesc;
    const int32_t* rows;   // on the device: the rows of A (rows_k = 0) or the length of K (1) that count; null: all
    int rows_k;
    int group;             // row tiles that sweep the columns together (L2 reuse)
    int64_t m_held;        // rows that the output has memory for: those behind them are not handed to the epilogue
    int32_t* zero;         // a word that the first CTA clears, or null
};

// The item of an index: row tile, column tile, range of K.
struct DenseItem {
    int mt, nt, split;
    __device__ __forceinline__ static DenseItem of(int id, int n_mt, int n_nt, int splits, int group) {
        DenseItem t;
        const int tiles = n_mt * n_nt;
        t.split = splits == 1 ? 0 : id / tiles;
        id -= t.split * tiles;
        const int gsz = group * n_nt;
        const int first = (id / gsz) * group;
        const int gm = min(n_mt - first, group);
        t.mt = first + (id % gsz) % gm;
        t.nt = (id % gsz) / gm;
        return t;
    }
};

// Stages that fit: A's rows (what the MMA reads behind them is another operand's, for rows
// that nobody reads) and B's.
inline int dense_stages(int cg, int a_rows, int bn) {
    const int bytes = (a_rows + bn / cg) * 128, room = kDenseStageRoom - (a_rows < kDenseM ? kDenseM - a_rows : 0) * 128;
    return room / bytes < kDenseStages ? room / bytes : kDenseStages;
}

// kind::f16 instruction descriptor: D fp32, A and B fp16 (0) or bf16 (1).
inline uint32_t dense_idesc(bool bf16, bool a_mn, bool b_mn, int m, int n) {
    return (1u << 4) | ((uint32_t)bf16 << 7) | ((uint32_t)bf16 << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(n >> 3) << 17) | ((uint32_t)(m >> 4) << 24);
}
// Shared-memory descriptor of an MN-major operand with the 128-byte swizzle: atoms of 64
// elements by 8 rows of K, 1024 bytes apart along K, boxes of 64 elements 8 KB apart.
__device__ __forceinline__ uint64_t desc_mn128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFF) >> 4) | ((uint64_t)(kDenseBoxBytes >> 4) << 16) |
           ((uint64_t)(1024 >> 4) << 32) | ((uint64_t)1 << 46) | ((uint64_t)2 << 61);
}
template <int CG>
__device__ __forceinline__ void dense_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if constexpr (CG == 1)
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
    else
        asm volatile(
            "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
            " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
            "l"(a), "l"(b), "r"(idesc), "r"(acc)
            : "memory");
}

// ---- pairs of CTAs -------------------------------------------------------------
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of the pair's first CTA's copy of a shared-memory object.
__device__ __forceinline__ uint32_t first_cta(const void* p) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(smem_u32(p)));
    return r;
}
// An epilogue warp gives accumulators back by arriving at `base` + 8 times the accumulator's number; after a wait that ran
// out base is that of the CTA's sink, barriers that nobody waits for (a test of `ok` at each arrival instead cost the
// 8-bit product 2%).
constexpr int kSinkCount = 1 << 19;
// (relaxed: what the arrival orders are accumulator reads, by tcgen05.fence; a release at
// cluster scope waits for all of the warp's memory accesses first, spills and scales among
// them, and was a third of the 8-bit product's stall cycles)
__device__ __forceinline__ void mbar_arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
template <int CG>
__device__ __forceinline__ void give_back(uint32_t bar) {
    if constexpr (CG == 1) asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
    else mbar_arrive_cluster(bar);
}
// The MMAs issued so far arrive on the barrier, in both CTAs of a pair.
template <int CG>
__device__ __forceinline__ void dense_commit(uint64_t* bar) {
    if constexpr (CG == 1)
        mma_commit(bar);
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
                smem_u32(bar)),
            "h"((uint16_t)3)
            : "memory");
}
// All MMAs of an issuing thread, whether it has stopped or not, arrive on fin; the TMEM's owner
// waits for both threads' before it gives the memory back (each of them ends after a few
// bounded waits).
__device__ __forceinline__ void wait_for_mmas(uint64_t (&fin)[2]) {
#pragma unroll 1
    for (int i = 0; i < 2; ++i) mbar_wait(&fin[i], 0, 4 * kTcDrainCycles);
}
// What the second CTA's producer tells the first one at its end, in the first one's memory.
struct PairEnd {
    uint64_t bar;      // one arrival
    uint32_t issued;   // stages that it has loaded
};
// Every copy of the stages that the CTA (pair) has loaded has landed.  Called by each producer at its end with
// the number of stages that it has loaded; w % stages is stage w's slot, bytes what a CTA loads of a stage.  The
// first CTA's barriers count the copies of both.  Where one CTA stopped earlier than the other (the issuing
// threads have stopped too then, and are waited for first), the stages that only one of them has loaded
// are counted as far as they were loaded.
template <int CG>
__device__ __forceinline__ void land_all(uint64_t* full, uint64_t (&fin)[2], PairEnd& peer, int rank, uint32_t issued, int stages,
                                         uint32_t bytes) {
    uint32_t other = issued;
    if constexpr (CG == 2) {
        if (rank == 1) {
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(first_cta(&peer.issued)), "r"(issued) : "memory");
            asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(first_cta(&peer.bar)) : "memory");
            return;
        }
        bool told = false;
        for (const long long t0 = clock64(); !told && clock64() - t0 < 4 * kTcDrainCycles;) {
            uint32_t ok;
            asm volatile(
                "{ .reg .pred p; mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], 0; selp.u32 %0, 1, 0, p; }"
                : "=r"(ok)
                : "r"(smem_u32(&peer.bar))
                : "memory");
            told = ok;
        }
        if (told) other = *reinterpret_cast<volatile uint32_t*>(&peer.issued);
        if (other != issued) {
            wait_for_mmas(fin);
#pragma unroll 1
            for (uint32_t w = other; w < issued; ++w)
                asm volatile("mbarrier.complete_tx.relaxed.cta.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(&full[w % stages])), "r"(bytes)
                             : "memory");
#pragma unroll 1
            for (uint32_t w = issued; w < other; ++w) mbar_expect_tx(&full[w % stages], bytes);
        }
    }
    const uint32_t end = max(issued, other);
#pragma unroll 1
    for (uint32_t w = end > (uint32_t)stages ? end - stages : 0; w < end; ++w)
        mbar_wait(&full[w % stages], (w / stages) & 1, kTcDrainCycles);
}
// A 2-d box into this CTA's memory, counted on `bar` (of a pair: the first CTA's).
template <int CG>
__device__ __forceinline__ void dense_load(void* dst, const CUtensorMap* map, int x, int y, uint32_t bar) {
    if constexpr (CG == 1)
        asm volatile(
            "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
    else
        asm volatile(
            "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
            " [%0], [%1, {%2, %3}], [%4];" ::"r"(smem_u32(dst)),
            "l"(map), "r"(x), "r"(y), "r"(bar)
            : "memory");
}
template <int CG>
__device__ __forceinline__ void tmem_alloc(uint32_t* at, uint32_t cols) {
    if constexpr (CG == 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    } else {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(at)), "r"(cols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
}
template <int CG>
__device__ __forceinline__ void tmem_free(uint32_t at, uint32_t cols) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
    else
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(at), "r"(cols) : "memory");
}

// What the epilogue gets: 32 lanes of a warp hold 32 rows.
struct DenseTile {
    int64_t row;       // of this lane, in D
    int64_t col;       // first column of this warp's half, in D
    int cols;          // columns of the half
    int mt, nt, half, split;
    bool ok;           // false: a wait ran out, write NaN
    int rows;          // rows of A that count (all of them without a device count)
};
// An epilogue reads its half's columns 32 at a time, c = 0, 32, 64, 96 (constants, in an unrolled
// loop), from the accumulator ...
struct FromTmem {
    uint32_t taddr;   // of the half's first column on the warp's lanes
    bool none;        // no columns of K: zeros
    __device__ __forceinline__ void get(int c, const DenseTile& t, float (&v)[32]) const {
        uint32_t r[32];
        tmem_ld32(taddr + c, r);
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
        if (!t.ok || none) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = t.ok ? 0.f : __int_as_float(0x7fc00000);
        }
    }
};
// ... or from registers, so that the accumulator is free before it is worked on.
struct FromSums {
    const float (&sum)[kDenseN / 2];
    bool none;
    __device__ __forceinline__ void get(int c, const DenseTile& t, float (&v)[32]) const {
#pragma unroll
        for (int j = 0; j < 32; ++j) v[j] = sum[c + j];
        if (!t.ok || none) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = t.ok ? 0.f : __int_as_float(0x7fc00000);
        }
    }
};

// Rows of an epilogue warp's tile, 128 bytes each, turned in shared memory so that a store
// instruction writes 128 contiguous bytes of a row instead of 32 bytes of 32 rows (the
// output of 128 x 256 bf16 took 4900 cycles that way).
constexpr int kTurnPitch = 144;                   // bytes of a row: 16-byte accesses by rows and by columns meet no bank twice
constexpr int kTurnBytes = 32 * kTurnPitch;       // of a warp
template <typename T>
struct Turn {
    static constexpr int kCols = 128 / (int)sizeof(T);
    // lane's row
    __device__ __forceinline__ static void put(unsigned char* buf, int lane, const float (&v)[kCols]) {
        uint4* p = reinterpret_cast<uint4*>(buf + lane * kTurnPitch);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            uint32_t w[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                if constexpr (sizeof(T) == 4) w[k] = __float_as_uint(v[4 * i + k]);
                else w[k] = pack2<T>(make_float2(v[8 * i + 2 * k], v[8 * i + 2 * k + 1]));
            }
            p[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
        __syncwarp();
    }
    // the warp's first `rows` rows, their first `cols` columns, to out (row stride ld); vec: 16-byte
    // aligned rows and whole 16-byte chunks
    __device__ __forceinline__ static void flush(const unsigned char* buf, int lane, T* out, int64_t ld, int rows, int cols, bool vec) {
        if (vec) {
            const int seg = lane & 7;
            if (seg * (16 / (int)sizeof(T)) < cols) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const int r = 4 * i + (lane >> 3);
                    if (r < rows)
                        *reinterpret_cast<uint4*>(reinterpret_cast<char*>(out + r * ld) + 16 * seg) =
                            *reinterpret_cast<const uint4*>(buf + r * kTurnPitch + 16 * seg);
                }
            }
        } else {
#pragma unroll 4
            for (int r = 0; r < rows; ++r) {
                const T* p = reinterpret_cast<const T*>(buf + r * kTurnPitch);
#pragma unroll
                for (int c = 0; c < kCols; c += 32)
                    if (c + lane < cols) out[r * ld + c + lane] = p[c + lane];
            }
        }
        __syncwarp();
    }
};

// Position in a ring of slots: the slot and its phase's parity (counted, not divided:
// the issuing threads pass here for every stage).
struct Stages {
    int n;
    int slot = 0;
    uint32_t parity = 0;
    __device__ explicit Stages(int slots) : n(slots) {}
    __device__ __forceinline__ void next() {
        if (++slot == n) {
            slot = 0;
            parity ^= 1;
        }
    }
    __device__ __forceinline__ void skip(int count) {
        const int laps = (slot + count) / n;
        slot += count - laps * n;
        parity ^= (uint32_t)laps & 1;
    }
};
// Stages by which a dual tile's first accumulator goes ahead of its second at a tile's start (8192 x 768 ->
// 50257, the loss: 391 us before it did, 386 with 1, 380 with 2 or 3, 385 with 4, which is all there are).
constexpr int kDenseLead = 3;

// Epilogue: a type with Args and static __device__ void run(const Args&, const DenseTile&,
// const Source&).  TURNS: the tensor cores' additions truncate, so a long K is shared by
// accumulators, which the epilogue's threads add with rounding in registers.  DUAL: a pair's tile
// is 512 rows, two MMAs of 256 that share B, each with its own accumulator; a stage is then worth
// two for 1.5 times the bytes from the L2, which bound the single tile (12.5 TB/s), and the
// accumulators are drained between tiles instead of beside them.
template <int CG, bool A_MN, bool B_MN, bool TURNS, bool DUAL, class Epilogue>
__global__ void __launch_bounds__(kDenseThreads, 1)
    k_dense(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b, const DenseArgs a,
            const typename Epilogue::Args ea) {
    static_assert(!DUAL || (CG == 2 && !TURNS), "a dual tile is a pair's, and has no accumulator to take turns");
    constexpr int S = kDenseStages, SUBS = DUAL ? 2 : 1;
    extern __shared__ __align__(1024) unsigned char dense_raw[];
    unsigned char* sm = dense_raw + ((1024 - (smem_u32(dense_raw) & 1023)) & 1023);
    __shared__ uint64_t full[S], empty[S], accf[2], acce[2], fin[2], hand[2], sink[2];
    __shared__ PairEnd peer;
    __shared__ uint32_t tmem_base;

    const int t = threadIdx.x, warp = t >> 5, lane = t & 31;
    const int rank = CG == 1 ? 0 : (int)cluster_rank();
    if (t == 0) {
        for (int i = 0; i < S; ++i) {
            mbar_init(&full[i], 1);
            mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&accf[i], 1);
            mbar_init(&acce[i], kDenseEpilogueWarps * CG);
            mbar_init(&fin[i], 1);
            mbar_init(&hand[i], 1);
            mbar_init(&sink[i], kSinkCount);
        }
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
    if (a.zero && blockIdx.x == 0 && t == 0) *a.zero = 0;

    // a device count of rows shortens M or K; each role finds the same items
    int n_mt = a.n_mt, rows = 0x7fffffff;
    int64_t K = a.K;
    if (a.rows) {
        const int n = __ldg(a.rows);
        if (a.rows_k) K = min(K, (int64_t)n);
        else {
            n_mt = min(n_mt, (n + kDenseM * CG * SUBS - 1) / (kDenseM * CG * SUBS));
            rows = n;
        }
    }
    const int n_k = (int)((K + kDenseK - 1) / kDenseK);
    const int items = n_mt * a.n_nt * a.splits;
    const int first = blockIdx.x / CG, step = gridDim.x / CG;
    const int half_b = a.bn / CG;   // rows of B that this CTA loads
    const int a_bytes = a.a_rows * 128, stage = (a.a_rows * SUBS + half_b) * 128;
    const uint32_t tx = (uint32_t)stage * CG;
    // accumulators that share the stages of an item (one at least: an item without stages hands its accumulator on too)
    auto turns_of = [&](int n) { return TURNS ? max(1, (n + a.turn_stages - 1) / a.turn_stages) : 1; };
    // first row of A of a tile's part in this CTA
    auto row_of = [&](int mt, int sub) { return ((mt * SUBS + sub) * CG + rank) * kDenseM; };

    if (warp < 4) {
        fewer_registers<kRoleRegs>();
        if (warp == 0 && lane == 0) {
            bool ok = true, used = false;   // used: every slot has been filled once
            int id = first, left = 0;       // left: stages of the last item that have not been loaded
            Stages r(a.stages);
            for (; id < items && ok; id += step) {
                const DenseItem it = DenseItem::of(id, n_mt, a.n_nt, a.splits, a.group);
                const int k0 = (int)((int64_t)n_k * it.split / a.splits), k1 = (int)((int64_t)n_k * (it.split + 1) / a.splits);
                const int n0 = it.nt * a.bn + rank * half_b;
                for (int k = k0; k < k1; ++k) {
                    const int s = r.slot;
                    if (used && !mbar_wait(&empty[s], r.parity ^ 1)) {
                        ok = false;
                        left = k1 - k;
                        break;
                    }
                    unsigned char* sa = sm + s * stage;
                    unsigned char* sb = sa + SUBS * a_bytes;
                    if (rank == 0) mbar_expect_tx(&full[s], tx);
                    const uint32_t bar = CG == 1 ? smem_u32(&full[s]) : first_cta(&full[s]);
                    const int kc = k * kDenseK;
#pragma unroll
                    for (int sub = 0; sub < SUBS; ++sub) {
                        const int m0 = row_of(it.mt, sub);
                        if constexpr (A_MN) {
                            dense_load<CG>(sa + sub * a_bytes, &map_a, m0, kc, bar);
                            dense_load<CG>(sa + sub * a_bytes + kDenseBoxBytes, &map_a, m0 + 64, kc, bar);
                        } else {
                            dense_load<CG>(sa + sub * a_bytes, &map_a, kc, m0, bar);
                        }
                    }
                    if constexpr (B_MN) {
                        for (int j = 0; j < half_b; j += 64)
                            dense_load<CG>(sb + j * 128, &map_b, n0 + j, kc, bar);
                    } else {
                        dense_load<CG>(sb, &map_b, kc, n0, bar);
                    }
                    r.next();
                    used |= r.slot == 0;
                }
            }
            // (counted afterwards: a counter in the loop spilled registers there)
            uint32_t issued = 0;
            if (a.splits == 1) {
                issued = (uint32_t)((id - first) / step) * (uint32_t)n_k;
            } else {
                for (int i = first; i < id; i += step) {
                    const int split = DenseItem::of(i, n_mt, a.n_nt, a.splits, a.group).split;
                    issued += (uint32_t)((int64_t)n_k * (split + 1) / a.splits - (int64_t)n_k * split / a.splits);
                }
            }
            issued -= (uint32_t)left;
            land_all<CG>(full, fin, peer, rank, issued, a.stages, stage);
        }
        // One thread for all turns left the tensor cores idle for 850 cycles where they changed the
        // accumulator: its waits and commits, with nothing queued behind the last MMA.  The other
        // thread makes its waits beside the last MMAs of a turn.  It is told when to (hand): a
        // barrier's phase is known by its parity only, so nobody may wait for one while an earlier
        // phase of that barrier is still open.  The word comes when all stages but the turn's last
        // have been waited for; the next turn's first stage is then at most the second in the ring
        // that is open, and its accumulators' earlier phases are past.  (A stage is given back after the
        // next one has been waited for, or not at all: the ring does not come around to one that nobody saw.)
        if ((warp == 1 || warp == 2) && lane == 0 && rank == 0) {
            const uint32_t mine = warp - 1;
            bool ok = true;
            Stages r(a.stages);
            uint32_t q = 0;   // accumulators filled, by both threads
            uint32_t u = 0;   // turns
            for (int id = first; id < items && ok; id += step) {
                const DenseItem it = DenseItem::of(id, n_mt, a.n_nt, a.splits, a.group);
                const int i0 = (int)((int64_t)n_k * it.split / a.splits), i1 = (int)((int64_t)n_k * (it.split + 1) / a.splits);
                // a turn's stages: from floor(n turn / turns) on, counted (the product of a long K's stages and its
                // turns passes 32 bits)
                const int turns = turns_of(i1 - i0);
                const int whole = TURNS ? (i1 - i0) / turns : i1 - i0, rest = i1 - i0 - whole * turns;
                int k1 = i0, over = 0;
                for (int turn = 0; turn < turns; ++turn, ++u, q += SUBS) {
                    const int k0 = k1;
                    k1 += whole;
                    if (TURNS && (over += rest) >= turns) {
                        over -= turns;
                        ++k1;
                    }
                    if ((u & 1) != mine) {
                        r.skip(k1 - k0);
                        continue;
                    }
                    const int ab = q & 1;
                    if ((u > 0 && !mbar_wait(&hand[mine], ((u - 1) >> 1) & 1)) ||
                        (q >= 2 && !mbar_wait(&acce[ab], ((q >> 1) - 1) & 1)) || (k0 < k1 && !mbar_wait(&full[r.slot], r.parity))) {
                        ok = false;
                        break;
                    }
                    const uint32_t d = tmem + ab * kDenseN;
                    const int last = max(k0, k1 - 2);
                    if (k0 == k1) {   // nothing to add (no row counts): both accumulators are handed on, so both must be drained
                        if (DUAL && q >= 2 && !mbar_wait(&acce[1], ((q >> 1) - 1) & 1)) ok = false;
                        if (ok) mbar_arrive(&hand[mine ^ 1]);
                    }
                    // the MMAs of a stage with one accumulator; next: another stage's come after them, which is
                    // waited for while the tensor cores are busy (a wait costs a hundred cycles even when there
                    // is nothing to wait for)
                    auto multiply = [&](int s, int sub, bool more, bool next, const Stages& then) {
                        const uint32_t sa = smem_u32(sm + s * stage), so = sa + sub * a_bytes, sb = sa + SUBS * a_bytes;
#pragma unroll
                        for (int kk = 0; kk < kDenseK / 16; ++kk) {
                            // 16 columns of K: 32 bytes along a K-major row, two atoms of an MN-major box
                            const uint64_t da = A_MN ? desc_mn128(so + kk * 2048) : desc_sw128(so + kk * 32);
                            const uint64_t db = B_MN ? desc_mn128(sb + kk * 2048) : desc_sw128(sb + kk * 32);
                            dense_mma<CG>(d + sub * kDenseN, da, db, a.idesc, (more || kk > 0) ? 1u : 0u);
                            if (kk == 1 && next && !mbar_wait(&full[then.slot], then.parity)) ok = false;
                        }
                    };
                    int k = k0;
                    if constexpr (DUAL) {
                        // A tile's first accumulator is drained before its second: its MMAs go ahead with the first
                        // stages.  (accf[0] is told after acce[1] has been waited for: nobody then waits for a
                        // phase of acce[1] while an earlier one is open.)
                        if (q >= 2 && k0 < k1) {
                            const int ahead = min(k1, k0 + min(kDenseLead, a.stages));
                            const Stages begin = r;
#pragma unroll 1
                            for (int sub = 0; sub < 2 && ok; ++sub) {
                                if (sub == 1) {
                                    if (!mbar_wait(&acce[1], ((q >> 1) - 1) & 1)) {
                                        ok = false;
                                        break;
                                    }
                                    if (ahead == k1) dense_commit<CG>(&accf[0]);
                                }
                                r = begin;
#pragma unroll 1
                                for (k = k0; k < ahead && ok; ++k) {
                                    if (sub == 0 && k == last) mbar_arrive(&hand[mine ^ 1]);
                                    tc_fence_after();
                                    const int s = r.slot;
                                    r.next();
                                    multiply(s, sub, k > k0, (k + 1 == ahead) == (sub == 1) && k + 1 < k1, r);
                                    if (sub == 1 && ok) dense_commit<CG>(&empty[s]);
                                }
                            }
                        }
                    }
                    for (; k < k1 && ok; ++k) {
                        if (k == last) mbar_arrive(&hand[mine ^ 1]);
                        tc_fence_after();
                        const int s = r.slot;
                        r.next();
                        multiply(s, 0, k > k0, !DUAL && k + 1 < k1, r);
                        if constexpr (DUAL) {
                            if (k + 1 == k1) dense_commit<CG>(&accf[0]);
                            multiply(s, 1, k > k0, k + 1 < k1, r);
                        }
                        if (ok) dense_commit<CG>(&empty[s]);
                    }
                    if (!ok) break;
                    if (!DUAL || k0 == k1) dense_commit<CG>(&accf[ab]);
                    if constexpr (DUAL) dense_commit<CG>(&accf[1]);
                }
            }
            dense_commit<CG>(&fin[mine]);
        }
    } else {
        more_registers<kSumRegs>();
        const int half = warp >= 8 ? 1 : 0, quarter = warp & 3;
        const int hc = a.bn / 2;
        const uint32_t lanes = tmem + half * hc + ((uint32_t)(quarter * 32) << 16);
        bool ok = true;
        uint32_t q = 0, base = CG == 1 ? smem_u32(acce) : first_cta(acce);
        auto wait = [&] {
            if (ok) ok = mbar_wait(&accf[q & 1], (q >> 1) & 1);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) base = smem_u32(sink);
            tc_fence_after();
            return lanes + (q & 1) * kDenseN;
        };
        auto release = [&] {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) give_back<CG>(base + 8 * (q & 1));
            ++q;
        };
        for (int id = first; id < items; id += step) {
            const DenseItem it = DenseItem::of(id, n_mt, a.n_nt, a.splits, a.group);
            DenseTile tile;
            tile.col = (int64_t)it.nt * a.bn + half * hc;
            tile.cols = hc;
            tile.mt = it.mt;
            tile.nt = it.nt;
            tile.half = half;
            tile.split = it.split;
            const int n = (int)((int64_t)n_k * (it.split + 1) / a.splits) - (int)((int64_t)n_k * it.split / a.splits);
            const bool none = n == 0;   // no columns of K
            tile.rows = rows;
#pragma unroll 1
            for (int sub = 0; sub < SUBS; ++sub) {
                tile.row = row_of(it.mt, sub) + quarter * 32 + lane;
                const bool held = tile.row - lane < a.m_held;
                if constexpr (TURNS || DUAL) {
                    float sum[kDenseN / 2];
                    if constexpr (TURNS) {
#pragma unroll
                        for (int j = 0; j < kDenseN / 2; ++j) sum[j] = 0.f;
                        for (int turn = turns_of(n); turn > 0; --turn) {
                            const uint32_t taddr = wait();
#pragma unroll
                            for (int c = 0; c < kDenseN / 2; c += 32) {
                                if (c < hc) {
                                    uint32_t r[32];
                                    tmem_ld32(taddr + c, r);
#pragma unroll
                                    for (int j = 0; j < 32; ++j) sum[c + j] += __uint_as_float(r[j]);
                                }
                            }
                            release();
                        }
                    } else {   // (tiles of 256 columns)
                        const uint32_t taddr = wait();
                        uint32_t r[kDenseN / 64][32];
#pragma unroll
                        for (int c = 0; c < kDenseN / 2; c += 32) tmem_ld32_async(taddr + c, r[c / 32]);
                        tmem_wait_ld();
                        release();
#pragma unroll
                        for (int c = 0; c < kDenseN / 2; ++c) sum[c] = __uint_as_float(r[c / 32][c % 32]);
                    }
                    tile.ok = ok;
                    if (held) Epilogue::run(ea, tile, FromSums{sum, none});
                } else {
                    const FromTmem source{wait(), none};
                    tile.ok = ok;
                    if (held) Epilogue::run(ea, tile, source);
                    release();
                }
            }
        }
    }
    if (warp == 3) wait_for_mmas(fin);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if constexpr (CG == 2) cluster_sync();   // no barrier or tile of a CTA goes while the other may still touch it
    tc_fence_after();
    if (warp == 3) tmem_free<CG>(tmem, 512);
}

// 16 bytes of a row of any alignment from byte 16 c on, zeros behind its `bytes`: from the five aligned
// words that hold them.  Nothing outside the row's words is read; the first row's start is one of a word.
__device__ __forceinline__ uint4 padded_chunk(const uint8_t* row, int64_t bytes, int64_t c) {
    const int off = (int)((uintptr_t)row & 3);
    const uint32_t* words = reinterpret_cast<const uint32_t*>(row - off) + 4 * c;   // (in front of a row lies the one before it)
    const int64_t left = bytes + off - 16 * c;   // bytes from the first word to the row's end
    uint32_t w[5];
    if (left >= 20) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = __ldg(words + i);
    } else {
        const uint8_t* b = reinterpret_cast<const uint8_t*>(words);
#pragma unroll
        for (int i = 0; i < 5; ++i) {
            w[i] = 0;
            for (int k = 0; k < 4; ++k)
                if (4 * i + k < left) w[i] |= (uint32_t)b[4 * i + k] << (8 * k);
        }
    }
    return make_uint4(__funnelshift_r(w[0], w[1], 8 * off), __funnelshift_r(w[1], w[2], 8 * off),
                      __funnelshift_r(w[2], w[3], 8 * off), __funnelshift_r(w[3], w[4], 8 * off));
}

// Rows of `bytes` bytes, `ld` apart and of any alignment (the first one of 16), to rows of `to` bytes, a
// multiple of 16, with zeros behind: what TMA can read.
static __global__ void __launch_bounds__(256) k_pad_rows(const uint8_t* __restrict__ src, int64_t ld, uint8_t* __restrict__ dst,
                                                         int64_t rows, int64_t bytes, int64_t to) {
    after_previous();
    let_next_start();
    // (a warp takes 32 chunks of a row; chunks of all rows, so that short rows fill the device too)
    const int64_t per_row = (to / 16 + 31) / 32, n = rows * per_row;
    for (int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); id < n; id += (int64_t)gridDim.x * 8) {
        const int64_t r = id / per_row, c = (id - r * per_row) * 32 + (threadIdx.x & 31);
        if (c < to / 16) reinterpret_cast<uint4*>(dst + r * to)[c] = padded_chunk(src + r * ld, bytes, c);
    }
}
// The way back, for rows of 16-bit elements: rows of `cols` elements, ld (more, a multiple of 8) apart and
// aligned, side by side.  A thread writes 8 elements of the whole; they lie in one row mostly, in five
// words of it.
static __global__ void __launch_bounds__(256) k_join_rows(const uint16_t* __restrict__ src, int64_t ld, uint16_t* __restrict__ dst,
                                                          int64_t rows, int64_t cols) {
    after_previous();
    let_next_start();
    const int64_t n = rows * cols, chunks = (n + 7) / 8;
    for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < chunks; q += (int64_t)gridDim.x * 256) {
        int64_t r = 8 * q / cols, c = 8 * q - r * cols;
        if (c + 8 <= cols && 8 * q + 8 <= n) {
            const uint32_t* words = reinterpret_cast<const uint32_t*>(src + r * ld) + c / 2;   // (the fifth ends within ld, as cols < ld)
            const int off = (int)(c & 1) * 16;
            uint32_t w[5];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = __ldg(words + i);
            w[4] = off ? __ldg(words + 4) : 0;
            reinterpret_cast<uint4*>(dst)[q] = make_uint4(__funnelshift_r(w[0], w[1], off), __funnelshift_r(w[1], w[2], off),
                                                          __funnelshift_r(w[2], w[3], off), __funnelshift_r(w[3], w[4], off));
        } else {
            for (int k = 0; k < 8 && 8 * q + k < n; ++k) {
                dst[8 * q + k] = src[r * ld + c];
                if (++c == cols) {
                    c = 0;
                    ++r;
                }
            }
        }
    }
}

// 16-bit [rows][len] at row stride ld (a multiple of 8), in boxes of 64 columns by
// box_rows rows with the 128-byte swizzle; what lies past len or rows reads as zero.
inline bool dense_map(CUtensorMap* map, const void* base, bool bf16, int64_t len, int64_t rows, int64_t ld, int box_rows) {
    EncodeTiledFn fn = encoder();
    if (!fn) return false;
    cuuint64_t dims[2] = {(cuuint64_t)len, (cuuint64_t)rows};
    cuuint64_t strides[1] = {(cuuint64_t)ld * 2};
    cuuint32_t box[2] = {64u, (cuuint32_t)box_rows};
    cuuint32_t estr[2] = {1, 1};
    return fn(map, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<void*>(base), dims,
              strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
              CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Launch: items run by as many CTAs (pairs) as there are SMs (pairs of SMs), or fewer.
template <int CG, bool A_MN, bool B_MN, bool TURNS, bool DUAL, class Epilogue>
int dense_launch(const CUtensorMap& ma, const CUtensorMap& mb, const DenseArgs& a, const typename Epilogue::Args& ea, int num_sms,
                 cudaStream_t s) {
    constexpr auto f = k_dense<CG, A_MN, B_MN, TURNS, DUAL, Epilogue>;
    if (!allow_smem<f>(kDenseSmem)) return SNK_ERR_CUDA;
    const int64_t items = (int64_t)a.n_mt * a.n_nt * a.splits;
    return launch_after(f, (unsigned)(CG * std::min<int64_t>(items, num_sms / CG)), kDenseThreads, kDenseSmem, CG, s, ma, mb, a, ea);
}

}  // namespace snk
