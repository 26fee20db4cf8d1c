// Decode attention over an E4M3 cache with one scale for each 16 tokens and
// head, with or without a window (no window: kNoWindow, which leaves nothing
// out).
#include "attn_tc.cuh"

namespace hpc {

template <int RB, int HEADS>
using Tc = TcVariant<RB, HEADS, true>;

// nb = 1: up to 8 query rows per KV head, 2: up to 16; heads: KV heads of a
// descriptor.
AttnConfig attn_config_block(int nb, int heads) {
    if (heads == 2) return nb == 2 ? Tc<16, 2>::config() : Tc<8, 2>::config();
    return nb == 2 ? Tc<16, 1>::config() : Tc<8, 1>::config();
}

cudaError_t launch_attn_block(int nb, int heads, const CUtensorMap &tk, const CUtensorMap &tv,
                             const AttnParams &p, int grid, cudaStream_t s) {
    if (heads == 2)
        return nb == 2 ? Tc<16, 2>::launch(tk, tv, p, grid, s) : Tc<8, 2>::launch(tk, tv, p, grid, s);
    return nb == 2 ? Tc<16, 1>::launch(tk, tv, p, grid, s) : Tc<8, 1>::launch(tk, tv, p, grid, s);
}

}  // namespace hpc
