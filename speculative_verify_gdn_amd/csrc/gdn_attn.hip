// gdn_attn.hip -- which instance of the window attention runs (gdn_attn_impl.h
// has the kernels), and what workspace it needs.
#include "gdn_attn_launch.h"

namespace gdn {

// 0 where the work lists would have more units than 32 bits count
size_t attn_work_bytes(int B, int K, int Hq, int Hkv, int D, int page_log2, int P, int prefix, bool bf16)
{
    AttnArgs a{};
    a.B = B;
    a.K = K;
    a.Hq = Hq;
    a.Hkv = Hkv;
    a.D = D;
    a.page_log2 = page_log2;
    a.P = P;
    a.prefix = prefix;
    const attn::Pick p = attn::pick(a, bf16);
    return attn::countable(a, p, 8192 / D) ? attn::layout(a, p.blocks, p.MS, p.MO).bytes : 0;
}

hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t s)
{
    if (bf16)
        return a.D == 64 ? attn::launch_bf16_64(a, s) : a.D == 128 ? attn::launch_bf16_128(a, s)
                                                                  : attn::launch_bf16_256(a, s);
    return a.D == 64 ? attn::launch_f32_64(a, s) : a.D == 128 ? attn::launch_f32_128(a, s)
                                                             : attn::launch_f32_256(a, s);
}

}  // namespace gdn
