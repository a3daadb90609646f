// The batch-tiled products on 8-bit floating-point codes (E4M3) with one scale per row (see
// snk_q8_sparse.cuh).
#include "snk_q8_sparse.cuh"

namespace snk {
SNK_Q8_ROW_TILES(SNK_Q8_E4M3)
}  // namespace snk
