// Few-row attention kernels of views for heads of 64 (attention_few.hpp).
#include "attention_few.hpp"

namespace qlinear {

QLINEAR_VIEW_LAUNCHER(launch_view_few_64) { return attn::launch_few_width<64>(c, a, p, part, stream); }

}  // namespace qlinear
