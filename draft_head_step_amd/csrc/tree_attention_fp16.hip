// Tree attention kernels, fp16 (elements).
#include "tree_attention_kernels.h"

namespace dspark {
template dspark_status run_tree_attention<1, false>(const TreeAttnArgs&, const AttnPlan&, hipStream_t);
}  // namespace dspark
