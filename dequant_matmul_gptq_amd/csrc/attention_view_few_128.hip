// Few-row attention kernels of views for heads of 128 (attention_few.hpp).
#include "attention_few.hpp"

namespace qlinear {

QLINEAR_VIEW_LAUNCHER(launch_view_few_128) { return attn::launch_few_width<128>(c, a, p, part, stream); }

}  // namespace qlinear
