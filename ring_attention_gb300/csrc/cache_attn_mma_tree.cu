// cache_attn_mma_tree.cu - the few-row cache attention under trees: its instances, compiled on their own.
#include "cache_attn_mma.cuh"

namespace bpa {
namespace cache_mma {

cudaError_t launch_trees(const Work& w, int DP, int DVP, int NT, const CUtensorMap* maps, int rpb, cudaStream_t s) {
    return launch_any<true>(w, DP, DVP, NT, maps, rpb, s);
}

}  // namespace cache_mma
}  // namespace bpa
