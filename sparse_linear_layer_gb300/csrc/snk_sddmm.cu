// Weight gradient on the support (SDDMM) and the bias gradient.
//
//   "Padded-CSR: A sparse storage format for dynamic sparse training on CPU",
//     sec. 7.1: dL/dW is wanted only at the live slots of W; for each live
//     slot at (i, c) it is the dot product of the dL/dY row i with the X
//     row c, so the dense M x K gradient is never formed.
//   "Beyond Masked Sparsity: SNACK Enables Truly Sparse Neural Networks on
//     GPU", Fig. 1: the backward pass as a sparse outer product over supp(W).
//
//     dW_k  = sum_beta dY[beta, r_k] * X[beta, c_k]     (canonical order)
//     db[o] = sum_beta dY[beta, o]
//
// GB300 design: the same merge-path chunks and lane layout as the SpMM
// kernel, walking the canonical order.  The row index comes from the row
// pointer (no rows[] stream), the dY values of a row sit in registers for
// the whole row, X is staged transposed in shared memory, and the output is
// written with 128-bit stores in the order it is read, so the only HBM
// streams are cols (read) and dW (write).  No entry depends on another, so no
// chunk ever waits for another.
#include "snk_sddmm.cuh"

namespace snk {

// snk_q8_sparse.cuh: one batch tile of an 8-bit X.
template <int FMT, bool GROUPED>
int q8_weight_tile(Layer* L, const SddmmQ8Args& a, int bp, cudaStream_t s);

template <int BP>
__global__ void k_transpose_x(const float* __restrict__ X, int64_t n, int b, float* __restrict__ xt) {
    stage_transposed<BP>(xt, X, n, b, n, blockIdx.x * blockDim.x + threadIdx.x,
                         gridDim.x * blockDim.x);
}

__global__ void k_bias_grad_only(const float* __restrict__ dY, int64_t b, int64_t n,
                                 float* __restrict__ db) {
    for (int64_t o = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; o < n;
         o += (int64_t)gridDim.x * blockDim.x) {
        float sacc = 0.f;
        for (int64_t beta = 0; beta < b; ++beta) sacc += dY[beta * n + o];
        db[o] = sacc;
    }
}

template <int BP>
static int launch_bp(Layer* L, SddmmArgs a, const Q8In* q, cudaStream_t s) {
    const size_t smem = (size_t)a.in_f * BP * sizeof(float);
    const int grid = a.n_blocks;
    using Args = typename DwTileF32<BP>::DwArgs;
    if constexpr (BP >= 8 && SNK_BANDS) {
        // an operand too wide for shared memory: row runs over column bands
        if (smem > (size_t)L->max_smem) {
            bool done = false;
            const int st = band_backward_weight(L, BP, a.X, q, a.dY, a.b, a.dW, a.accumulate, a.dY_all, a.b_all,
                                                a.db, s, &done);
            if (st != SNK_OK || done) return st;
        }
    }
    if (smem <= (size_t)L->max_smem && a.col16) {
        if (q) {
            if (int st = launch_q8_rows(*q, a.b, L->xt, s); st != SNK_OK) return st;
            a.X = L->xt;
        }
        auto fn = k_sddmm<DwTileF32<BP>, true>;
        if (smem > 48 * 1024 &&
            cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) !=
                cudaSuccess)
            return SNK_ERR_CUDA;
        fn<<<grid, kThreads, smem, s>>>(Args(a));
    } else {
        if (q) {
            if (int st = launch_q8_transposed(*q, a.b, BP, L->xt, L->num_sms, s); st != SNK_OK) return st;
        } else {
            k_transpose_x<BP><<<L->num_sms * 4, 256, 0, s>>>(a.X, a.in_f, a.b, L->xt);
        }
        a.xt = L->xt;
        k_sddmm<DwTileF32<BP>, false><<<grid, kThreads, 0, s>>>(Args(a));
    }
    return cudaGetLastError() == cudaSuccess ? SNK_OK : SNK_ERR_CUDA;
}

int launch_backward_weight(Layer* L, const float* X, const Q8In* q, const float* dY, int64_t b, float* dW,
                           float* db, cudaStream_t s) {
    if (L->nnz == 0) {
        if (db) {
            k_bias_grad_only<<<L->num_sms * 4, 256, 0, s>>>(dY, b, L->out_f, db);
            if (cudaGetLastError() != cudaSuccess) return SNK_ERR_CUDA;
        }
        return SNK_OK;
    }
    if (q && light_layer(L, *q, b, true)) return light_weight(L, *q, dY, b, dW, db, s);
    if (q ? tc_eligible(L, *q, b, true) : tc_eligible(L, b))
        return q ? run_tc_sddmm(L, SrcQ8{*q}, dY, b, dW, db, s)
                 : run_tc_sddmm(L, SrcF32{X, L->in_f}, dY, b, dW, db, s);
    SddmmArgs a{};
    a.col = L->c;
    a.col16 = L->c16;
    a.row_ptr = L->row_ptr;
    a.cdesc = L->cdesc_r;
    a.nnz = L->nnz;
    a.out_f = L->out_f;
    a.in_f = L->in_f;
    a.n_blocks = L->n_blocks;
    a.dW = dW;
    a.b_all = b;
    a.dY_all = dY;
    for (int64_t t0 = 0, bt; t0 < b; t0 += bt) {
        bt = q ? q8_tile_rows(*q, b - t0, L->nnz, true) : std::min<int64_t>(kMaxBatchTile, b - t0);
        a.b = (int)bt;
        Q8In qt{};
        if (q) qt = q->from_row(t0);
        else a.X = X + t0 * L->in_f;
        const Q8In* qp = q ? &qt : nullptr;
        a.dY = dY + t0 * L->out_f;
        a.accumulate = t0 > 0;
        a.db = (t0 == 0) ? db : nullptr;
        int st;
        if (q && q8_codes_tile(*q, batch_tile(bt), L->nnz, L->in_f, true)) {
            SddmmQ8Args aq(a);
            aq.codes = qt.codes;
            aq.scales = qt.scales;
            aq.groups = qt.n_groups;
            aq.gshift = qt.gshift;
            const int bp = batch_tile(bt);
            const bool int8 = q->format == SNK_Q8_INT8;
            if (q->gshift == 31)
                st = int8 ? q8_weight_tile<SNK_Q8_INT8, false>(L, aq, bp, s) : q8_weight_tile<SNK_Q8_E4M3, false>(L, aq, bp, s);
            else
                st = int8 ? q8_weight_tile<SNK_Q8_INT8, true>(L, aq, bp, s) : q8_weight_tile<SNK_Q8_E4M3, true>(L, aq, bp, s);
            if (st != SNK_OK) return st;
            continue;
        }
        switch (batch_tile(bt)) {
            case 1: st = launch_bp<1>(L, a, qp, s); break;
            case 2: st = launch_bp<2>(L, a, qp, s); break;
            case 4: st = launch_bp<4>(L, a, qp, s); break;
            case 8: st = launch_bp<8>(L, a, qp, s); break;
            case 16: st = launch_bp<16>(L, a, qp, s); break;
            case 32: st = launch_bp<32>(L, a, qp, s); break;
            default: st = launch_bp<64>(L, a, qp, s); break;
        }
        if (st != SNK_OK) return st;
    }
    return SNK_OK;
}

}  // namespace snk
