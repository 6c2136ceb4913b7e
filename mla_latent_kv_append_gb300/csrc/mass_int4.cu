// mla_token_mass for 4-bit latents (see mass.cuh).
#include "mass_few.cuh"

namespace mla {

mla_status launch_mass_int4(const MassParams& p, int lf, int kf, cudaStream_t stream) {
  if (lf == MLA_FMT_INT4_ASYM && kf == MLA_FMT_BF16) return launch_mass_pair<MLA_FMT_INT4_ASYM, MLA_FMT_BF16>(p, stream);
  if (lf == MLA_FMT_INT4_ASYM && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT4_ASYM, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_INT4_ASYM && kf == MLA_FMT_INT4_SYM) return launch_mass_pair<MLA_FMT_INT4_ASYM, MLA_FMT_INT4_SYM>(p, stream);
  if (lf == MLA_FMT_INT4_SYM && kf == MLA_FMT_BF16) return launch_mass_pair<MLA_FMT_INT4_SYM, MLA_FMT_BF16>(p, stream);
  if (lf == MLA_FMT_INT4_SYM && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT4_SYM, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_INT4_SYM && kf == MLA_FMT_INT4_SYM) return launch_mass_pair<MLA_FMT_INT4_SYM, MLA_FMT_INT4_SYM>(p, stream);
  return MLA_ERR_UNSUPPORTED;
}

}  // namespace mla
