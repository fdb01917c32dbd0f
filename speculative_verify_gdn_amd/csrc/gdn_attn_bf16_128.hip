// gdn_attn_bf16_128.hip -- the window attention for bfloat16, head size 128.
#include "gdn_attn_launch.h"

namespace gdn {
namespace attn {

hipError_t launch_bf16_128(const AttnArgs& a, hipStream_t s)
{
    using M16 = Cfg<true, 128, 4, 1, 1, 4, 1>;
    using M32 = Cfg<true, 128, 4, 2, 1, 2, 1>;
    using M64 = Cfg<true, 128, 4, 4, 1, 1, 1>;
    using M128 = Cfg<true, 128, 4, 4, 2, 1, 1>;
    return launch_all<true, 128, M16, M32, M64, M128>(a, s);
}

}  // namespace attn
}  // namespace gdn
