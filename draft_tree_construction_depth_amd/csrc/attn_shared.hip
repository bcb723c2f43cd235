// The attention of a batch that shares its first rows, over 16-bit caches
// (csrc/attention.hpp), a source of its own so that the variants are compiled
// side by side.
#include "verify.hpp"

namespace ddt {

int launch_attn_shared(const AttnParams& ap, const AttnPlan& pl, int dtype, int head_dim,
                     hipStream_t st) {
  return dtype == DDT_BF16 ? launch_attn<__bf16, kAtSame, true>(ap, pl, head_dim, st)
                           : launch_attn<_Float16, kAtSame, true>(ap, pl, head_dim, st);
}

}  // namespace ddt
