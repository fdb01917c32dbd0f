// gdn_attn.hip -- attention of a verify window over the paged cache (gdn_attn_verify).
//
// The plain form: a workgroup per row (sequence, token, query head).  Its four
// waves take every fourth key; a wave holds q, k and v spread over its lanes,
// sums the dot product across them and keeps the running maximum m, the sum l
// of e^{x-m} and the accumulator of e^{x-m} v.  The four are joined in LDS.
#include "gdn_device.h"
#include "gdn_kv_internal.h"

namespace gdn {
namespace {

// sees: bit i set where window node i is on the path from a root to node t
__device__ __forceinline__ unsigned long long window_mask(const int32_t* parent, int t)
{
    if (!parent) return t == 63 ? ~0ull : (1ull << (t + 1)) - 1;
    unsigned long long m = 0;
    for (int i = t; i >= 0;) {
        m |= 1ull << i;
        const int p = parent[i];
        i = p < i ? p : -1;
    }
    return m;
}

template <bool BF16, int D>
__global__ __launch_bounds__(256) void attn_row_kernel(AttnArgs a)
{
    constexpr int E = D / 64;
    __shared__ float lm[4], ll[4], lo[4][D];
    const int h = blockIdx.x, t = blockIdx.y, b = blockIdx.z;
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int count = a.count ? min(max(a.count[b], 0), a.K) : a.K;
    if (t >= count) return;
    const int hk = h / (a.Hq / a.Hkv);
    const long long len = min((long long)max(a.lens[b], 0), (long long)a.P << a.page_log2);
    const long long end = min(len + count, (long long)a.P << a.page_log2);
    const unsigned long long sees = window_mask(a.parent ? a.parent + (size_t)b * a.K : nullptr, t);
    float q[E], acc[E];
    float m = -INFINITY, l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        q[e] = load1<BF16>(a.q, ((size_t)b * a.K + t) * a.q_stride + (size_t)h * D + e * 64 + lane) * a.scale;
        acc[e] = 0.f;
    }
    for (long long j = w; j < end; j += 4) {
        if (j >= len && !(sees >> (j - len) & 1)) continue;
        const int id = a.table[(size_t)b * a.P + (j >> a.page_log2)];
        if ((unsigned)id >= (unsigned)a.n_pages) continue;
        const size_t at =
            ((((size_t)id * a.Hkv + hk) << a.page_log2) + (size_t)(j & ((1 << a.page_log2) - 1))) * D + lane;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) x = __builtin_fmaf(q[e], load1<BF16>(a.k_pages, at + e * 64), x);
#pragma unroll
        for (int s = 1; s < 64; s <<= 1) x += __shfl_xor(x, s, 64);
        const float mn = fmaxf(m, x), f = m == mn ? 1.f : __expf(m - mn), p = __expf(x - mn);
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = __builtin_fmaf(p, load1<BF16>(a.v_pages, at + e * 64), acc[e] * f);
        m = mn;
    }
    if (lane == 0) lm[w] = m, ll[w] = l;
#pragma unroll
    for (int e = 0; e < E; ++e) lo[w][e * 64 + lane] = acc[e];
    __syncthreads();
    if (w != 0) return;
    float M = -INFINITY, L = 0.f;
    for (int i = 0; i < 4; ++i) M = fmaxf(M, lm[i]);
    float f[4];
    for (int i = 0; i < 4; ++i) {
        f[i] = ll[i] == 0.f ? 0.f : __expf(lm[i] - M);
        L += ll[i] * f[i];
    }
    const size_t row = ((size_t)b * a.K + t) * a.Hq + h;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        float o = 0.f;
        for (int i = 0; i < 4; ++i) o = __builtin_fmaf(lo[i][e * 64 + lane], f[i], o);
        store1<BF16>(a.o, row * D + e * 64 + lane, L == 0.f ? 0.f : o / L);
    }
    if (a.lse && lane == 0) a.lse[row] = L == 0.f ? -INFINITY : M + __logf(L);
}

}  // namespace

size_t attn_work_bytes(int B, int K, int Hq, int Hkv, int D, int page_log2, int P, int prefix, bool bf16) { return 16; }

hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t s)
{
    const dim3 grid(a.Hq, a.K, a.B), block(256);
    if (bf16) {
        if (a.D == 64) attn_row_kernel<true, 64><<<grid, block, 0, s>>>(a);
        else if (a.D == 128) attn_row_kernel<true, 128><<<grid, block, 0, s>>>(a);
        else attn_row_kernel<true, 256><<<grid, block, 0, s>>>(a);
    } else {
        if (a.D == 64) attn_row_kernel<false, 64><<<grid, block, 0, s>>>(a);
        else if (a.D == 128) attn_row_kernel<false, 128><<<grid, block, 0, s>>>(a);
        else attn_row_kernel<false, 256><<<grid, block, 0, s>>>(a);
    }
    return hipGetLastError();
}

}  // namespace gdn
