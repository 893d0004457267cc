// Attention over a prefix that sequences share, few rows: the launch over the sequences' own keys (a translation unit of its own, for the
// build's time).
#include "cb_kv8_few.cuh"

namespace cb {

cudaError_t launch_kv8_few_own(const Kv8& c, const void* attn_args, cudaStream_t s) {
    AttnArgs p = *static_cast<const AttnArgs*>(attn_args);
    return c.cfg.head_dim == 128 ? launch_few<128, BESIDE>(c, p, s) : launch_few<64, BESIDE>(c, p, s);
}

}  // namespace cb
