// gdn_attn_bf16_256.hip -- the window attention for bfloat16, head size 256.
#include "gdn_attn_launch.h"

namespace gdn {
namespace attn {

hipError_t launch_bf16_256(const AttnArgs& a, hipStream_t s)
{
    using M16 = Cfg<true, 256, 4, 1, 1, 2, 2>;
    using M32 = Cfg<true, 256, 4, 2, 1, 1, 2>;
    using M64 = Cfg<true, 256, 4, 4, 1, 1, 1>;
    return launch_all<true, 256, M16, M32, M64, void>(a, s);
}

}  // namespace attn
}  // namespace gdn
