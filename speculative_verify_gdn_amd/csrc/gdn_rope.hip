// gdn_rope.hip -- rotary positions, the RMS norms of query and key heads, and
// the append of a window's keys and values to the paged cache with both on the
// way (include/gdn.h: gdn_rope, gdn_qk_norm_rope, gdn_kv_append_rope).
//
// One kernel for the three.  With theta_i = position * freqs[i], a pair (a, b) of
// a head becomes (a c - b s, b c + a s), c = m cos theta_i, s = m sin theta_i; with
// weights the head is first x / sqrt(mean x^2 + eps) * w.  It reads every head once
// and writes it once, about 7 operations an element: memory bound, so what
// matters is that the rest stays off the path.
//   - theta is formed in 64 bits from the position and the frequency (no table
//     in memory: at position 2^31 the rounding of theta is 2^-22, a table of
//     that many rows would not fit), reduced to turns and only then rounded to
//     32 bits; a workgroup forms the sines of its tokens once, into LDS, and
//     every head of a token reads them from there.
//   - a group of lanes holds one head, a lane the two 16-byte pieces whose
//     elements are pairs of one another: (j, j + rot/2) for the two halves, the
//     neighbouring pieces for neighbours.  So no element crosses lanes, and the norm is
//     a sum over the group.
//   - where the head goes (dense rows, or a page of the cache) is an offset a
//     token, found while the first heads are on their way.
#include "gdn_device.h"
#include "gdn_window_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTileMax = 16;        // tokens of a workgroup
constexpr int kAngles = 1024;       // sines (and cosines) of a workgroup
constexpr double kInv2Pi = 0.15915494309189533577;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// E elements of one piece as floats
template <bool BF16, int E>
struct Piece {
    float f[E];

    __device__ __forceinline__ void load(const char* p)
    {
        if constexpr (BF16 && E == 8) {
            const uint4 u = *reinterpret_cast<const uint4*>(p);
            const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(w[i]), f[2 * i + 1] = bf16_hi(w[i]);
        } else if constexpr (!BF16 && E == 4) {
            const float4 u = *reinterpret_cast<const float4*>(p);
            f[0] = u.x, f[1] = u.y, f[2] = u.z, f[3] = u.w;
        } else {
            static_assert(E == 1, "pieces are 16 bytes or one element");
            f[0] = load1<BF16>(p, 0);
        }
    }
    __device__ __forceinline__ void store(char* p) const
    {
        if constexpr (BF16 && E == 8) {
            uint32_t w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const bf16x2_t h = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
                w[i] = __builtin_bit_cast(uint32_t, h);
            }
            *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        } else if constexpr (!BF16 && E == 4) {
            *reinterpret_cast<float4*>(p) = make_float4(f[0], f[1], f[2], f[3]);
        } else {
            store1<BF16>(p, 0, f[0]);
        }
    }
};

// sum over aligned groups of 2^log2 lanes
__device__ __forceinline__ float group_sum(float v, int log2)
{
    if (log2 >= 1) v += dpp_mov<kDppQuadXor1>(v);
    if (log2 >= 2) v += dpp_mov<kDppQuadXor2>(v);
    if (log2 >= 3) v += dpp_mov<kDppRowHalfMirror>(v);
    if (log2 >= 4) v += dpp_mov<kDppRowMirror>(v);
    if (log2 >= 5) v += __shfl_xor(v, 16, 64);
    if (log2 >= 6) v += __shfl_xor(v, 32, 64);
    return v;
}

// The depth of node t in its window's tree (parents first; an entry outside [0, i) marks a root), found by a
// whole wave by doubling: a lane holds how far it has come up from its node, and where it stands.
__device__ __forceinline__ int node_depth(const int32_t* parent, int K, int t)
{
    const int lane = threadIdx.x & 63;
    int up = -1;
    if (lane < K) {
        const int p = parent[lane];
        up = p >= 0 && p < lane ? p : -1;
    }
    int depth = up >= 0;
#pragma unroll
    for (int d = 1; d < kKvWindowMax; d <<= 1) {
        const int more = __shfl(depth, max(up, 0), 64), far = __shfl(up, max(up, 0), 64);
        if (up >= 0) {
            depth += more;
            up = far;
        }
    }
    return __shfl(depth, t, 64);
}

// what the heads of a token need to know of it
struct Token {
    long long from[3];  // byte offset of its first head in each part
    long long to[3];    // the same where it goes; below 0: nowhere
};

// E: elements of a piece; NP: pairs of pieces of a lane
template <bool BF16, int E, int NP, bool INTERLEAVED>
__global__ __launch_bounds__(kThreads) void rope_kernel(RopeArgs a)
{
    constexpr int ES = BF16 ? 2 : 4;
    __shared__ Token info[kTileMax];
    __shared__ float cs[kAngles], sn[kAngles];
    __shared__ float weight[2][kRopeHeadMax];

    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const long long tokens = (long long)a.B * a.K;
    const long long first = (long long)blockIdx.x * a.tile;
    const int n = (int)min((long long)a.tile, tokens - first);
    const int half = a.rot >> 1;

    // where each token stands and goes, and its sines: a wave a token, or several where there are few
    const int share = a.tile == 1 ? kWaves : a.tile == 2 ? kWaves / 2 : 1;
    for (int i = wave / share; i < n; i += kWaves / share) {
        const long long tok = first + i;
        const int b = (int)(tok / a.K), t = (int)(tok - (long long)b * a.K);
        const long long len = a.lens ? max(a.lens[b], 0) : 0;
        const bool there = !a.count || t < a.count[b];
        const long long p = a.pos    ? (long long)a.pos[tok]
                            : a.parent ? len + node_depth(a.parent + (size_t)b * a.K, a.K, t)
                                       : len + t;
        const int sub = wave % share;
        for (int j = lane + 64 * sub; j < half; j += 64 * share) {
            const double turns = (double)p * a.freqs[j] * kInv2Pi;
            float s, c;
            sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
            cs[i * half + j] = a.mscale * c;
            sn[i * half + j] = a.mscale * s;
        }
        if (sub == 0 && lane < 3) {
            const RopePart& r = a.part[lane];
            long long to = -1;
            if (there && !r.paged) to = b * r.ys[0] + t * r.ys[1];
            if (there && r.paged) {
                const long long at = len + t, slot = at >> a.g.page_log2;
                const int id = slot < a.P ? a.table[(size_t)b * a.P + slot] : -1;
                if ((unsigned)id < (unsigned)a.g.n_pages)
                    to = ((((long long)id * a.g.Hkv) << a.g.page_log2) + (at & ((1 << a.g.page_log2) - 1))) *
                         a.g.row_bytes;
            }
            info[i].from[lane] = b * r.xs[0] + t * r.xs[1];
            info[i].to[lane] = to;
        }
    }
    for (int s = 0; s < 2; ++s)
        if (a.part[s].w)
            for (int d = threadIdx.x; d < a.D; d += kThreads) weight[s][d] = a.part[s].w[d];
    __syncthreads();

    // the heads: a group of lanes each
    const int h0 = blockIdx.y * a.chunk, nh = min(a.chunk, a.heads - h0);
    const int group = threadIdx.x >> a.lanes_log2, step = kThreads >> a.lanes_log2;
    const int l = threadIdx.x & ((1 << a.lanes_log2) - 1);
    const int pairs = a.D / (2 * E);   // pairs of pieces of a head
    const int turned = half / E;       // those of them that turn
    const float inv_d = 1.0f / (float)a.D;
    for (int r = group; r < n * nh; r += step) {
        const int i = r / nh;
        int h = h0 + r - i * nh, s = 0;
        if (h >= a.part[0].H) {
            h -= a.part[0].H;
            s = 1;
            if (h >= a.part[1].H) {
                h -= a.part[1].H;
                s = 2;
            }
        }
        const RopePart& part = a.part[s];
        const long long to = info[i].to[s];
        if (to < 0) continue;
        const char* x = static_cast<const char*>(part.x) + info[i].from[s] + h * part.xs[2];
        char* y = static_cast<char*>(part.y) + to +
                  h * (part.paged ? (long long)a.g.row_bytes << a.g.page_log2 : part.ys[2]);
        Piece<BF16, E> u[NP], v[NP];
        int at[NP], bt[NP];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int j = l + (k << a.lanes_log2);
            if (INTERLEAVED || j >= turned) at[k] = 2 * j * E, bt[k] = at[k] + E;
            else at[k] = j * E, bt[k] = at[k] + half;
            if (j < pairs) {
                u[k].load(x + at[k] * ES);
                v[k].load(x + bt[k] * ES);
            }
        }
        if (part.w) {
            float q = 0.0f;
#pragma unroll
            for (int k = 0; k < NP; ++k)
                if (l + (k << a.lanes_log2) < pairs) {
#pragma unroll
                    for (int e = 0; e < E; ++e) q = fmaf(u[k].f[e], u[k].f[e], fmaf(v[k].f[e], v[k].f[e], q));
                }
            q = group_sum(q, a.lanes_log2);
            const float z = 1.0f / sqrtf(q * inv_d + a.eps);
#pragma unroll
            for (int k = 0; k < NP; ++k)
                if (l + (k << a.lanes_log2) < pairs) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        u[k].f[e] *= z * weight[s][at[k] + e];
                        v[k].f[e] *= z * weight[s][bt[k] + e];
                    }
                }
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int j = l + (k << a.lanes_log2);
            if (j >= pairs) continue;
            if (part.turned && j < turned) {
                const float *c = cs + i * half + j * E, *d = sn + i * half + j * E;
#pragma unroll
                for (int e = 0; e < E; ++e) {
                    // the pair: element e of both pieces, or elements 2e and 2e+1 of the two pieces in a row
                    float &p = !INTERLEAVED ? u[k].f[e] : 2 * e < E ? u[k].f[2 * e] : v[k].f[2 * e - E];
                    float &q = !INTERLEAVED ? v[k].f[e] : 2 * e + 1 < E ? u[k].f[2 * e + 1] : v[k].f[2 * e + 1 - E];
                    const float p0 = p, q0 = q;
                    p = fmaf(p0, c[e], -(q0 * d[e]));
                    q = fmaf(q0, c[e], p0 * d[e]);
                }
            }
            u[k].store(y + at[k] * ES);
            v[k].store(y + bt[k] * ES);
        }
    }
}

int log2_up(int n)
{
    int l = 0;
    while ((1 << l) < n) ++l;
    return l;
}

template <bool BF16, bool INTERLEAVED>
void launch(RopeArgs& a, hipStream_t s)
{
    constexpr int E = BF16 ? 8 : 4;
    // 16-byte pieces where the turned part is made of whole pairs of them, single elements otherwise
    const bool wide = a.rot % (2 * E) == 0;
    a.lanes_log2 = min(log2_up(a.D / (wide ? 2 * E : 2)), 6);
    a.heads = a.part[0].H + a.part[1].H + a.part[2].H;
    const long long tokens = (long long)a.B * a.K;
    const int half = a.rot / 2, pass = kThreads >> a.lanes_log2;
    a.tile = 1;
    while (a.tile < 4 && tokens / a.tile > 2048 && 2 * a.tile * half <= kAngles) a.tile *= 2;
    const long long tiles = (tokens + a.tile - 1) / a.tile;
    int chunks = (a.heads * a.tile + pass - 1) / pass;   // one head a group of lanes
    while (chunks > 1 && tiles * chunks > 2048) chunks = (chunks + 1) / 2;
    a.chunk = (a.heads + chunks - 1) / chunks;
    const dim3 grid((unsigned)tiles, (a.heads + a.chunk - 1) / a.chunk);
    if (wide) rope_kernel<BF16, E, 1, INTERLEAVED><<<grid, dim3(kThreads), 0, s>>>(a);
    else rope_kernel<BF16, 1, 4, INTERLEAVED><<<grid, dim3(kThreads), 0, s>>>(a);
}

}  // namespace

hipError_t launch_rope(const RopeArgs& args, bool bf16, bool interleaved, hipStream_t s)
{
    RopeArgs a = args;
    if (bf16) interleaved ? launch<true, true>(a, s) : launch<true, false>(a, s);
    else interleaved ? launch<false, true>(a, s) : launch<false, false>(a, s);
    return hipGetLastError();
}

}  // namespace gdn
