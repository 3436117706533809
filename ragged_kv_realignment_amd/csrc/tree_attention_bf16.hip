// Tree attention over bf16 caches (the kernel is in tree_attention.h; a source per
// type so that they compile in parallel).
#include "tree_attention.h"

namespace sd {

hipError_t launch_tree_attention_bf16(const TreeAttnParams &p, hipStream_t s) { return launch_attn_dt<2>(p, s); }

}  // namespace sd
