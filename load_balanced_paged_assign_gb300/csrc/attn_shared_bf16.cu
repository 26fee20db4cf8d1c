// Decode attention over shared prefixes, BF16 pages.
#include "attn_shared.cuh"

namespace hpc {
namespace {

// The decode kernel with rings of four stages of one tile, for one and for two blocks of
// query rows (five stages: the same times; two of two tiles: the same or slower).
template <int NB>
struct Tail {
    static constexpr int kStages = 4, kTps = 1;
    using Tr = AttnTraits<false, kStages, kTps, NB>;
    static constexpr int kThreads = Tr::kThreads, kSmemBytes = Tr::kSmemBytes;
    static __device__ __forceinline__ void run(const CUtensorMap &tk, const CUtensorMap &tv,
                                               const AttnParams &t) {
        attn_cta<false, kStages, kTps, NB>(tk, tv, t);
    }
};

using One = SharedVariant<HPC_KV_BF16, Tail<1>>;  // up to 8 query rows per KV head and request
using Two = SharedVariant<HPC_KV_BF16, Tail<2>>;  // up to 16

}  // namespace

AttnConfig shared_config_bf16(int nb) { return nb == 2 ? Two::config() : One::config(); }

cudaError_t launch_shared_bf16(int nb, const SharedMaps &m, const AttnParams &t, const HeadArgs &h,
                               int grid, cudaStream_t s) {
    return nb == 2 ? Two::launch(m, t, h, grid, s) : One::launch(m, t, h, grid, s);
}

}  // namespace hpc
