// Many-row attention kernels of views for heads of 128 (attention_chunk.hpp).
#include "attention_chunk.hpp"

namespace qlinear {

QLINEAR_VIEW_LAUNCHER(launch_view_chunk_128) { return attn::launch_chunk_width<128>(c, a, p, part, stream); }

}  // namespace qlinear
