// Persistent attention kernel over an E4M3 cache with one scale for each 16
// tokens and head, with or without a window (no window: kNoWindow, which
// leaves nothing out).
#include "attn_kernel.cuh"

namespace hpc {

// The plain FP8 form's pipeline shapes: two tiles per stage (eight consumer
// warps), four stages.
using One = AttnVariant<true, 4, 2, 1, true, true>;  // up to 8 query rows per KV head
using Two = AttnVariant<true, 4, 2, 2, true, true>;  // up to 16

AttnConfig attn_config_block(int nb) { return nb == 2 ? Two::config() : One::config(); }

cudaError_t launch_attn_block(int nb, const CUtensorMap &tk, const CUtensorMap &tv,
                             const AttnParams &p, int grid, cudaStream_t s) {
    return nb == 2 ? Two::launch(tk, tv, p, grid, s) : One::launch(tk, tv, p, grid, s);
}

}  // namespace hpc
