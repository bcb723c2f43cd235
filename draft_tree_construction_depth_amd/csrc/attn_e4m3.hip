// The attention over caches of e4m3 codes (csrc/attention.hpp), a source of
// its own so that the variants are compiled side by side.
#include "verify.hpp"

namespace ddt {

int launch_attn_e4m3(const AttnParams& ap, const AttnPlan& pl, int dtype, int head_dim,
                     hipStream_t st) {
  return dtype == DDT_BF16 ? launch_attn<__bf16, kAtE4M3, true>(ap, pl, head_dim, st)
                           : launch_attn<_Float16, kAtE4M3, true>(ap, pl, head_dim, st);
}

}  // namespace ddt
