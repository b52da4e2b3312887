#include "moe_block_norm_row.h"

namespace moe {
hipError_t launch_block_norm_row_fp16(const BlockNorm& a, const Runs& runs, const Partials& part, hipStream_t s) { return launch_row<fp16_t>(a, runs, part, s); }
}  // namespace moe
