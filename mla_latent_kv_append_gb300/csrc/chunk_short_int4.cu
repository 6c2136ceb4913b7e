// The short path of mla_chunk_attention for 4-bit latents (see chunk_short.cuh).
#include "chunk_short.cuh"

namespace mla {

mla_status launch_short_int4(const ChunkParams& p, int lf, int kf, int R, cudaStream_t stream) {
  if (lf == MLA_FMT_INT4_ASYM && kf == MLA_FMT_BF16) return launch_fmt<MLA_FMT_INT4_ASYM, MLA_FMT_BF16>(p, R, stream);
  if (lf == MLA_FMT_INT4_ASYM && kf == MLA_FMT_INT8_SYM) return launch_fmt<MLA_FMT_INT4_ASYM, MLA_FMT_INT8_SYM>(p, R, stream);
  if (lf == MLA_FMT_INT4_ASYM && kf == MLA_FMT_INT4_SYM) return launch_fmt<MLA_FMT_INT4_ASYM, MLA_FMT_INT4_SYM>(p, R, stream);
  if (lf == MLA_FMT_INT4_SYM && kf == MLA_FMT_BF16) return launch_fmt<MLA_FMT_INT4_SYM, MLA_FMT_BF16>(p, R, stream);
  if (lf == MLA_FMT_INT4_SYM && kf == MLA_FMT_INT8_SYM) return launch_fmt<MLA_FMT_INT4_SYM, MLA_FMT_INT8_SYM>(p, R, stream);
  if (lf == MLA_FMT_INT4_SYM && kf == MLA_FMT_INT4_SYM) return launch_fmt<MLA_FMT_INT4_SYM, MLA_FMT_INT4_SYM>(p, R, stream);
  return MLA_ERR_UNSUPPORTED;
}

}  // namespace mla
