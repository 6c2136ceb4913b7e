// mla_token_mass for bf16 latents (see mass.cuh).
#include "mass_few.cuh"

namespace mla {

mla_status launch_mass_bf16(const MassParams& p, int lf, int kf, cudaStream_t stream) {
  if (lf == MLA_FMT_BF16 && kf == MLA_FMT_BF16) return launch_mass_pair<MLA_FMT_BF16, MLA_FMT_BF16>(p, stream);
  if (lf == MLA_FMT_BF16 && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_BF16, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_BF16 && kf == MLA_FMT_INT4_SYM) return launch_mass_pair<MLA_FMT_BF16, MLA_FMT_INT4_SYM>(p, stream);
  return MLA_ERR_UNSUPPORTED;
}

}  // namespace mla
