// Many-row attention kernels of views for heads of 64 (attention_chunk.hpp).
#include "attention_chunk.hpp"

namespace qlinear {

QLINEAR_VIEW_LAUNCHER(launch_view_chunk_64) { return attn::launch_chunk_width<64>(c, a, p, part, stream); }

}  // namespace qlinear
