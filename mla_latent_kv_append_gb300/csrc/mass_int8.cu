// mla_token_mass for INT8 latents in blocks of 16 (see mass.cuh).
#include "mass_few.cuh"

namespace mla {

mla_status launch_mass_int8(const MassParams& p, int lf, int kf, cudaStream_t stream) {
  if (lf == MLA_FMT_INT8_SYM && kf == MLA_FMT_BF16) return launch_mass_pair<MLA_FMT_INT8_SYM, MLA_FMT_BF16>(p, stream);
  if (lf == MLA_FMT_INT8_SYM && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT8_SYM, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_INT8_SYM && kf == MLA_FMT_INT4_SYM) return launch_mass_pair<MLA_FMT_INT8_SYM, MLA_FMT_INT4_SYM>(p, stream);
  return MLA_ERR_UNSUPPORTED;
}

}  // namespace mla
