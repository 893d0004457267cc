// Attention over a prefix that sequences share, few rows: the launch over the groups' prefixes (a translation unit of its own, for the
// build's time).
#include "cb_kv8_few.cuh"

namespace cb {

cudaError_t launch_kv8_few_prefix(const Kv8& c, void* attn_args, cudaStream_t s) {
    AttnArgs& p = *static_cast<AttnArgs*>(attn_args);              // (gets the columns of a piece)
    return c.cfg.head_dim == 128 ? launch_few<128, PREFIX>(c, p, s) : launch_few<64, PREFIX>(c, p, s);
}

}  // namespace cb
