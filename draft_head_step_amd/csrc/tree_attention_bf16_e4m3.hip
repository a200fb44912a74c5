// Tree attention kernels, bf16_e4m3 (elements, e4m3 cache).
#include "tree_attention_kernels.h"

namespace dspark {
template dspark_status run_tree_attention<0, true>(const TreeAttnArgs&, const AttnPlan&, hipStream_t);
}  // namespace dspark
