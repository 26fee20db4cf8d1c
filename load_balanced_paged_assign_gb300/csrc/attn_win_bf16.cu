// Windowed form of the persistent attention kernel over a BF16 cache: its
// 2 bytes a value leave the warp-level MMAs time enough.  64 requests of 1K to 16K
// tokens, 64 heads on 8, window 4096 and 64 sinks (819 MB): 129 us, 93% of the
// measured copy rate; HBM bounds it.
#include "attn_kernel.cuh"

namespace hpc {

// The plain form's pipeline shapes: one tile per stage, four stages.
using One = AttnVariant<false, 4, 1, 1, true>;  // up to 8 query rows per KV head
using Two = AttnVariant<false, 4, 1, 2, true>;  // up to 16

AttnConfig attn_config_win_bf16(int nb) { return nb == 2 ? Two::config() : One::config(); }

cudaError_t launch_attn_win_bf16(int nb, const CUtensorMap &tk, const CUtensorMap &tv,
                             const AttnParams &p, int grid, cudaStream_t s) {
    return nb == 2 ? Two::launch(tk, tv, p, grid, s) : One::launch(tk, tv, p, grid, s);
}

}  // namespace hpc
