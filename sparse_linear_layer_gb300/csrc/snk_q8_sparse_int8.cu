// The batch-tiled products on int8 codes with one scale per row (see
// snk_q8_sparse.cuh).
#include "snk_q8_sparse.cuh"

namespace snk {
SNK_Q8_ROW_TILES(SNK_Q8_INT8)
}  // namespace snk
