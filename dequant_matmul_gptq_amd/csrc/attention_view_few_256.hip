// Few-row attention kernels of views for heads of 256 (attention_few.hpp).
#include "attention_few.hpp"

namespace qlinear {

QLINEAR_VIEW_LAUNCHER(launch_view_few_256) { return attn::launch_few_width<256>(c, a, p, part, stream); }

}  // namespace qlinear
