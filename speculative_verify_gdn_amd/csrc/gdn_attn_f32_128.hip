// gdn_attn_f32_128.hip -- the window attention for float, head size 128.
#include "gdn_attn_launch.h"

namespace gdn {
namespace attn {

hipError_t launch_f32_128(const AttnArgs& a, hipStream_t s)
{
    using M16 = Cfg<false, 128, 8, 1, 1, 4, 2>;
    using M32 = Cfg<false, 128, 8, 2, 1, 2, 2>;
    using M64 = Cfg<false, 128, 8, 4, 1, 2, 1>;
    using M128 = Cfg<false, 128, 8, 8, 1, 1, 1>;
    return launch_all<false, 128, M16, M32, M64, M128>(a, s);
}

}  // namespace attn
}  // namespace gdn
