// Decode attention over shared prefixes, E4M3 pages.
#include "attn_shared.cuh"

namespace hpc {
namespace {

template <int RB, int HEADS>
using Form = SharedVariant<HPC_KV_FP8_E4M3, TcTail<RB, HEADS, false>>;

}  // namespace

AttnConfig shared_config_e4m3(int nb, int heads) {
    if (heads == 2) return nb == 2 ? Form<16, 2>::config() : Form<8, 2>::config();
    return nb == 2 ? Form<16, 1>::config() : Form<8, 1>::config();
}

cudaError_t launch_shared_e4m3(int nb, int heads, const SharedMaps &m, const AttnParams &t,
                               const HeadArgs &h, int grid, cudaStream_t s) {
    if (heads == 2)
        return nb == 2 ? Form<16, 2>::launch(m, t, h, grid, s)
                       : Form<8, 2>::launch(m, t, h, grid, s);
    return nb == 2 ? Form<16, 1>::launch(m, t, h, grid, s) : Form<8, 1>::launch(m, t, h, grid, s);
}

}  // namespace hpc
