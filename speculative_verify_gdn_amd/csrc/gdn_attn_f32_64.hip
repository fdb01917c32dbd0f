// gdn_attn_f32_64.hip -- the window attention for float, head size 64.
#include "gdn_attn_launch.h"

namespace gdn {
namespace attn {

hipError_t launch_f32_64(const AttnArgs& a, hipStream_t s)
{
    using M16 = Cfg<false, 64, 8, 1, 1, 8, 1>;
    using M32 = Cfg<false, 64, 8, 2, 1, 4, 1>;
    using M64 = Cfg<false, 64, 8, 4, 1, 2, 1>;
    using M128 = Cfg<false, 64, 8, 8, 1, 1, 1>;
    return launch_all<false, 64, M16, M32, M64, M128>(a, s);
}

}  // namespace attn
}  // namespace gdn
