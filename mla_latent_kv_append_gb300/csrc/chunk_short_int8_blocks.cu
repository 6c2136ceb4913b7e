// The short path of mla_chunk_attention for INT8 latents in other blocks, and with protected channels (see chunk_short.cuh).
#include "chunk_short.cuh"

namespace mla {

mla_status launch_short_int8_blocks(const ChunkParams& p, int lf, int kf, int R, cudaStream_t stream) {
  if (lf == MLA_FMT_INT8_G8 && kf == MLA_FMT_INT8_SYM) return launch_fmt<MLA_FMT_INT8_G8, MLA_FMT_INT8_SYM>(p, R, stream);
  if (lf == MLA_FMT_INT8_G32 && kf == MLA_FMT_INT8_SYM) return launch_fmt<MLA_FMT_INT8_G32, MLA_FMT_INT8_SYM>(p, R, stream);
  if (lf == MLA_FMT_INT8_G64 && kf == MLA_FMT_INT8_SYM) return launch_fmt<MLA_FMT_INT8_G64, MLA_FMT_INT8_SYM>(p, R, stream);
  if (lf == MLA_FMT_INT8_TOKEN && kf == MLA_FMT_INT8_SYM) return launch_fmt<MLA_FMT_INT8_TOKEN, MLA_FMT_INT8_SYM>(p, R, stream);
  if (lf == MLA_FMT_INT8_OUTLIER && kf == MLA_FMT_BF16) return launch_fmt<MLA_FMT_INT8_OUTLIER, MLA_FMT_BF16>(p, R, stream);
  if (lf == MLA_FMT_INT8_OUTLIER && kf == MLA_FMT_INT8_SYM) return launch_fmt<MLA_FMT_INT8_OUTLIER, MLA_FMT_INT8_SYM>(p, R, stream);
  return MLA_ERR_UNSUPPORTED;
}

}  // namespace mla
