// gdn_attn_launch.h -- the instances of the window attention and the rule that
// picks among them.
#pragma once

#include "gdn_attn_impl.h"

namespace gdn {
namespace attn {

struct Pick {
    int blocks, MS, MO;  // workgroups, rows of a shared tile (0: no shared list), rows of an own tile
};

// A tile of M rows reads its keys once for up to M rows of a key/value head; rows that are not there cost
// matrix work only.  Own tiles take the smallest size that holds a window's rows (64 single tokens with 4 rows a head
// in tiles of 64 rows: 118 us, of 16: 108); shared ones the largest as soon as there are rows for it (128 windows of 16
// tokens in tiles of 64 rows: 708 us, of 128: 574).
inline Pick pick(const AttnArgs& a, bool bf16)
{
    Pick p;
    const int G = a.Hq / a.Hkv, R = a.K * G;
    p.blocks = bf16 ? 512 : 256;   // two workgroups fit a CU (64 KB of tiles each), one in fp32
    // (128 rows of 256 columns take 50 registers more than there are: 16 nodes over 16411 keys 55 us, in 64 rows 31)
    const int most = bf16 && a.D == 256 ? 64 : 128;
    p.MO = R <= 16 ? 16 : R <= 32 ? 32 : R <= 64 ? 64 : most;
    p.MS = a.prefix == 0 ? 0 : a.B * R <= 64 ? 64 : most;
    return p;
}

// units of the two lists at most: they are counted in 32 bits, and so are the threads of the join
inline bool countable(const AttnArgs& a, const Pick& p, int N)
{
    const long long G = a.Hq / a.Hkv, most = (1ll << 31) - 1;
    const long long own = (long long)a.B * a.Hkv * ((a.K * G + p.MO - 1) / p.MO);
    const long long tiles = (((long long)a.P << a.page_log2) + N - 1) / N + kStartup;
    const long long shared = p.MS ? a.Hkv * ((a.B * a.K * G + p.MS - 1) / p.MS) : 0;
    return own <= most / tiles && shared <= most / tiles && (long long)a.B * a.K * a.Hq * (a.D / 4) <= 2 * most - 1024;
}

hipError_t launch_bf16_64(const AttnArgs& a, hipStream_t s);
hipError_t launch_bf16_128(const AttnArgs& a, hipStream_t s);
hipError_t launch_bf16_256(const AttnArgs& a, hipStream_t s);
hipError_t launch_f32_64(const AttnArgs& a, hipStream_t s);
hipError_t launch_f32_128(const AttnArgs& a, hipStream_t s);
hipError_t launch_f32_256(const AttnArgs& a, hipStream_t s);

// more than the default 64 KB of LDS a workgroup has to be asked for, once for each kernel and device
template <typename K>
hipError_t allow_lds(K kernel, int bytes, unsigned long long& done)
{
    int dev = 0;
    hipError_t e = hipGetDevice(&dev);
    if (e != hipSuccess) return e;
    const unsigned long long bit = 1ull << (dev & 63);
    if (__atomic_load_n(&done, __ATOMIC_RELAXED) & bit) return hipSuccess;
    e = hipFuncSetAttribute(reinterpret_cast<const void*>(kernel), hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == hipSuccess) __atomic_fetch_or(&done, bit, __ATOMIC_RELAXED);
    return e;
}

template <class OW, class SH>
hipError_t launch_one(const AttnArgs& a, const Pick& p, hipStream_t s)
{
    static unsigned long long done = 0;
    constexpr int lds = 2 * OW::STAGE + (int)sizeof(Small);
    auto* kernel = attn_kernel<OW, SH>;
    const hipError_t e = allow_lds(kernel, lds, done);
    if (e != hipSuccess) return e;
    kernel<<<dim3(p.blocks), dim3(OW::THREADS), lds, s>>>(a, p.blocks);
    return hipGetLastError();
}

template <class SH, class M16, class M32, class M64, class M128>
hipError_t launch_with(const AttnArgs& a, const Pick& p, hipStream_t s)
{
    if (p.MO == 16) return launch_one<M16, SH>(a, p, s);
    if (p.MO == 32) return launch_one<M32, SH>(a, p, s);
    if constexpr (!__is_same(M128, void))
        if (p.MO == 128) return launch_one<M128, SH>(a, p, s);
    return launch_one<M64, SH>(a, p, s);
}

template <bool BF16, int D, class M16, class M32, class M64, class M128>
hipError_t launch_all(const AttnArgs& given, hipStream_t s)
{
    AttnArgs a = given;
    const Pick p = pick(a, BF16);
    a.G = a.Hq / a.Hkv;
    a.listed = row_tiles_listed(a, p.MO, p.blocks);
    a.at = layout(a, p.blocks, p.MS, p.MO);
    hipError_t e;
    if (p.MS == 0) {
        e = launch_with<void, M16, M32, M64, M128>(a, p, s);
    } else {
        if constexpr (!__is_same(M128, void))
            e = p.MS == 128 ? launch_with<M128, M16, M32, M64, M128>(a, p, s)
                            : launch_with<M64, M16, M32, M64, M128>(a, p, s);
        else
            e = launch_with<M64, M16, M32, M64, M128>(a, p, s);
    }
    if (e != hipSuccess) return e;
    // 4 columns a thread; where that fills less than half the chip or a sixteenth of it, 4 or 16 threads share them
    // (one token over 60000 keys 19.6 us with 16 and 34.4 with 4; 16 nodes over 16411 keys 31.2 with 4 and 37.9 with 1;
    // above that many columns 4 are slower, 85.0 against 82.6 for 32 windows of 8 and 608 against 574 for 128 of 16)
    const long long units = (long long)a.B * a.K * a.Hq * (D / 4);
    const int split = units <= 16384 ? 16 : units <= 131072 ? 4 : 1;
    const dim3 grid((unsigned)((units * split + kJoin - 1) / kJoin));
    auto* join = split == 16 ? attn_join_kernel<BF16, D, 16> : split == 4 ? attn_join_kernel<BF16, D, 4>
                                                                          : attn_join_kernel<BF16, D, 1>;
    join<<<grid, dim3(kJoin), 0, s>>>(a, p.blocks, p.MS, p.MO, M16::N);
    return hipGetLastError();
}

}  // namespace attn
}  // namespace gdn
