// qmv_attn_tc.cu - tree attention of many rows on the tcgen05 tensor cores: the
// kernel k_attn_tc of qmv_attn_tc.cuh.
#include "qmv_attn_tc.cuh"

namespace qmv {
namespace attn {

cudaError_t launch_tree_tc(const AttnCache &c, const TreeArgs &a, cudaStream_t st) {
    return run_tc<false>(c, a, st);
}

}  // namespace attn
}  // namespace qmv
