// mla_token_mass for INT8 latents in other blocks, and with protected channels (see mass.cuh).
#include "mass_few.cuh"

namespace mla {

mla_status launch_mass_int8_blocks(const MassParams& p, int lf, int kf, cudaStream_t stream) {
  if (lf == MLA_FMT_INT8_G8 && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT8_G8, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_INT8_G32 && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT8_G32, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_INT8_G64 && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT8_G64, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_INT8_TOKEN && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT8_TOKEN, MLA_FMT_INT8_SYM>(p, stream);
  if (lf == MLA_FMT_INT8_OUTLIER && kf == MLA_FMT_BF16) return launch_mass_pair<MLA_FMT_INT8_OUTLIER, MLA_FMT_BF16>(p, stream);
  if (lf == MLA_FMT_INT8_OUTLIER && kf == MLA_FMT_INT8_SYM) return launch_mass_pair<MLA_FMT_INT8_OUTLIER, MLA_FMT_INT8_SYM>(p, stream);
  return MLA_ERR_UNSUPPORTED;
}

}  // namespace mla
