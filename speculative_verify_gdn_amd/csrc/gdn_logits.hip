// gdn_logits.hip -- the logits of a verify window adjusted (penalties for tokens
// already seen, biases, grammar masks, temperature) with the best token of each
// node, and the accepted node of a draft tree (include/gdn.h: gdn_logits_adjust,
// gdn_accept_tree).
//
// A logit x of token v behind node t becomes, with n how often v stands in the
// text since `start` and on the path to t, and seen if it stands in the text at all
// or on that path:
//   seen: x > 0 ? x / repetition : x * repetition;   x - frequency n;
//   n > 0: x - presence;   x + bias;   not allowed: -inf;   x / temperature
// One read of the logits and one write: memory bound, if the counts cost
// little.  So a workgroup takes a slice of the vocabulary for the rows of one
// sequence: it walks the history once, counts the tokens of its slice in LDS, and
// marks them in a bit map.  Eight logits whose byte of that map is 0, which is nearly
// all of them, skip the penalties (two correctly rounded divisions among
// them); the others take the long way.
// Every operation is one rounding of 32 bits in the order above, so that equal
// logits stay equal and the best is the lowest of them.
#include "gdn_device.h"
#include "gdn_window_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kSliceMax = 4096;            // tokens of the vocabulary of a workgroup
constexpr uint32_t kSeen = 0x80000000u;    // stands in the text before `start`

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
// 16 bytes at an element's own alignment (rows of an odd length start anywhere)
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

template <bool BF16>
__device__ __forceinline__ void load8(const void* base, size_t at, float* f)
{
    if constexpr (BF16) {
        const u32x4_any_t u = *reinterpret_cast<const u32x4_any_t*>(static_cast<const uint16_t*>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(u[i]), f[2 * i + 1] = bf16_hi(u[i]);
    } else {
        const u32x4_any_t* p = reinterpret_cast<const u32x4_any_t*>(static_cast<const float*>(base) + at);
        const u32x4_any_t u = p[0], v = p[1];
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = __uint_as_float(u[i]), f[4 + i] = __uint_as_float(v[i]);
    }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* base, size_t at, const float* f)
{
    u32x4_any_t u;
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2_t h = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
            u[i] = __builtin_bit_cast(uint32_t, h);
        }
        *reinterpret_cast<u32x4_any_t*>(static_cast<uint16_t*>(base) + at) = u;
    } else {
        u32x4_any_t* p = reinterpret_cast<u32x4_any_t*>(static_cast<float*>(base) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(f[i]);
        p[0] = u;
#pragma unroll
        for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(f[4 + i]);
        p[1] = u;
    }
}

// the larger score, the lower token where they are equal; no token: INT_MAX
struct Best {
    float score;
    int token;

    __device__ __forceinline__ void take(float s, int t)
    {
        if (s > score || (s == score && t < token)) score = s, token = t;
    }
};

__device__ __forceinline__ Best none() { return Best{-__builtin_huge_valf(), 0x7fffffff}; }

__device__ __forceinline__ Best wave_best(Best b)
{
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const float s = __shfl_xor(b.score, d, 64);
        const int t = __shfl_xor(b.token, d, 64);
        b.take(s, t);
    }
    return b;
}

// the nodes on the path root..i as a bit mask, in lane i, by doubling (a whole wave)
__device__ __forceinline__ unsigned long long node_paths(const int32_t* parent, int N)
{
    const int lane = threadIdx.x & 63;
    int up = -1;
    if (lane < N) {
        const int p = parent ? parent[lane] : lane - 1;
        up = p >= 0 && p < lane ? p : -1;
    }
    unsigned long long path = 1ull << lane;
#pragma unroll
    for (int d = 1; d < kKvWindowMax; d <<= 1) {
        const unsigned long long more = __shfl(path, max(up, 0), 64);
        const int far = __shfl(up, max(up, 0), 64);
        if (up >= 0) {
            path |= more;
            up = far;
        }
    }
    return path;
}

__device__ __forceinline__ int clamp_count(const int32_t* count, int b, int K)
{
    return count ? min(max(count[b], 0), K) : K;
}

template <bool XBF16, bool OBF16>
__global__ __launch_bounds__(kThreads) void logits_kernel(LogitsArgs a)
{
    extern __shared__ uint32_t lds[];   // counts, their bit map, and where there are biases their entries
    __shared__ unsigned long long paths[kKvWindowMax], inside_s;
    __shared__ int draft[kKvWindowMax];
    __shared__ Best part[kKvWindowMax][kWaves];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int groups = (a.K + a.rows - 1) / a.rows;
    const int b = blockIdx.y / groups, t0 = (blockIdx.y - b * groups) * a.rows;
    const int t1 = min(t0 + a.rows, clamp_count(a.count, b, a.K));
    if (t0 >= t1) return;
    const int v0 = blockIdx.x * a.slice, nv = min(a.slice, a.V - v0);
    uint32_t *cnt = lds, *bits = lds + a.slice;
    int* entry = reinterpret_cast<int*>(bits + a.slice / 32);
    const bool counted = a.params != nullptr, biased = a.n_bias > 0;

    float rep = 1.0f, presence = 0.0f, frequency = 0.0f, temp = 1.0f;
    if (counted) {
        const float* p = a.params + (size_t)b * 4;
        rep = p[0], presence = p[1], frequency = p[2], temp = p[3];
        if (!(temp > 0.0f)) temp = 1.0f;
    }

    if (counted)
        for (int i = tid; i < a.slice; i += kThreads) cnt[i] = 0;
    if (biased)
        for (int i = tid; i < a.slice; i += kThreads) entry[i] = -1;
    for (int i = tid; i < a.slice / 32; i += kThreads) bits[i] = 0;
    if (wave == 0) {
        // the path to each node, and the drafted tokens of this slice
        const bool drafts = counted && a.tokens;
        unsigned long long path = 0;
        if (drafts) path = node_paths(a.parent ? a.parent + (size_t)b * a.K : nullptr, a.K);
        int u = -1;
        if (drafts && lane < a.K) {
            const int d = a.tokens[(size_t)b * a.K + lane];
            if (d >= v0 && d - v0 < nv) u = d - v0;
        }
        paths[lane] = path;
        draft[lane] = u;
        const unsigned long long inside = __ballot(u >= 0);
        if (lane == 0) inside_s = inside;
    }
    __syncthreads();
    if (counted && a.history) {
        const int32_t* h = a.history + (size_t)b * a.capacity;
        const int len = min(max(a.history_lens[b], 0), a.capacity);
        const int start = a.history_start ? a.history_start[b] : 0;
#pragma unroll 4
        for (int i = tid; i < len; i += kThreads) {
            const int u = h[i] - v0;
            if ((unsigned)u < (unsigned)nv) {
                if (i >= start) atomicAdd(&cnt[u], 1u);
                else atomicOr(&cnt[u], kSeen);
                atomicOr(&bits[u >> 5], 1u << (u & 31));
            }
        }
    }
    if (biased)
        for (int i = tid; i < a.n_bias; i += kThreads) {
            const int u = a.bias_ids[(size_t)b * a.n_bias + i] - v0;
            if ((unsigned)u < (unsigned)nv) {
                atomicMax(&entry[u], i);   // (a token named twice: its last entry)
                atomicOr(&bits[u >> 5], 1u << (u & 31));
            }
        }
    const unsigned long long inside = inside_s;
    if (tid < 64 && (inside >> tid & 1)) atomicOr(&bits[draft[tid] >> 5], 1u << (draft[tid] & 31));
    __syncthreads();

    const unsigned char* touched = reinterpret_cast<const unsigned char*>(bits);
    const float* bias = biased ? a.bias_values + (size_t)b * a.n_bias : nullptr;
    for (int t = t0; t < t1; ++t) {
        const size_t row = (size_t)b * a.K + t;
        // the drafted tokens of this slice on the path to the node count for this row alone
        const unsigned long long mine = paths[t] & inside;
        if (mine) {
            __syncthreads();
            if (tid < 64 && (mine >> tid & 1)) atomicAdd(&cnt[draft[tid]], 1u);
            __syncthreads();
        }
        const size_t x_at = row * a.x_stride + v0, o_at = row * a.out_stride + v0, n_at = row * a.V + v0;
        const unsigned char* allow =
            a.mask ? reinterpret_cast<const unsigned char*>(a.mask + row * ((a.V + 31) / 32) + (v0 >> 5)) : nullptr;
        Best best = none();
        for (int k = tid * 8; k < nv; k += kThreads * 8) {
            const int m = min(8, nv - k);
            float f[8];
            if (m == 8) load8<XBF16>(a.x, x_at + k, f);
            else
                for (int e = 0; e < 8; ++e) f[e] = e < m ? load1<XBF16>(a.x, x_at + k + e) : 0.0f;
            if (touched[k >> 3]) {
                for (int e = 0; e < 8; ++e) {
                    if (e >= m) break;
                    float x = f[e];
                    if (counted) {
                        const uint32_t c = cnt[k + e], n = c & ~kSeen;
                        if (c) x = x > 0.0f ? x / rep : x * rep;
                        if (n) x = (x - frequency * (float)n) - presence;
                    }
                    if (biased && entry[k + e] >= 0) x += bias[entry[k + e]];
                    f[e] = x;
                }
            }
            if (allow) {
                const unsigned char w = allow[k >> 3];
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (!(w >> e & 1)) f[e] = -__builtin_huge_valf();
            }
            if (temp != 1.0f) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] /= temp;
            }
            if (a.out) {
                if (m == 8) store8<OBF16>(a.out, o_at + k, f);
                else
                    for (int e = 0; e < m; ++e) store1<OBF16>(a.out, o_at + k + e, f[e]);
            }
            if (a.best) {
                if (a.noise) {
                    float z[8];
                    if (m == 8) load8<false>(a.noise, n_at + k, z);
                    else
                        for (int e = 0; e < 8; ++e) z[e] = e < m ? a.noise[n_at + k + e] : 0.0f;
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] += z[e];
                }
#pragma unroll
                for (int e = 0; e < 8; ++e)
                    if (e < m && f[e] > best.score) best = Best{f[e], v0 + k + e};
            }
        }
        if (a.best) {
            best = wave_best(best);
            if (lane == 0) part[t - t0][wave] = best;
        }
        if (mine) {
            __syncthreads();
            if (tid < 64 && (mine >> tid & 1)) atomicSub(&cnt[draft[tid]], 1u);
            __syncthreads();   // the next row may look at the counts without a barrier of its own
        }
    }
    if (a.best) {
        __syncthreads();
        if (tid < t1 - t0) {
            Best r = part[tid][0];
#pragma unroll
            for (int w = 1; w < kWaves; ++w) r.take(part[tid][w].score, part[tid][w].token);
            a.work[((size_t)b * a.K + t0 + tid) * a.slices + blockIdx.x] = make_int2(__float_as_int(r.score), r.token);
        }
    }
}

// the best of a row's slices: a wave a row
__global__ __launch_bounds__(kThreads) void logits_best_kernel(LogitsArgs a)
{
    const long long row = (long long)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= (long long)a.B * a.K) return;
    const int b = (int)(row / a.K), t = (int)(row - (long long)b * a.K);
    if (t >= clamp_count(a.count, b, a.K)) return;
    Best best = none();
    for (int i = lane; i < a.slices; i += 64) {
        const int2 w = a.work[row * a.slices + i];
        best.take(__int_as_float(w.x), w.y);
    }
    best = wave_best(best);
    if (lane == 0) a.best[row] = best.token == 0x7fffffff ? -1 : best.token;
}

// ---------------------------------------------------------------- the accepted node
// A wave a sequence, a lane a node: a node is good where its token is the one its parent's row found best (a root:
// the token asked for, or any); it is kept where its whole path is good.
__global__ __launch_bounds__(kThreads) void accept_kernel(AcceptArgs a)
{
    const int b = blockIdx.x * kWaves + (threadIdx.x >> 6), lane = threadIdx.x & 63;
    if (b >= a.B) return;
    const int live = clamp_count(a.count, b, a.K);
    const int32_t* parent = a.parent ? a.parent + (size_t)b * a.K : nullptr;
    const bool node = lane < a.K;
    const int token = node ? a.tokens[(size_t)b * a.K + lane] : -1;
    const int target = node ? a.target[(size_t)b * a.K + lane] : -1;
    const int root = a.root ? a.root[b] : -1;
    int up = -1;
    if (node) {
        const int p = parent ? parent[lane] : lane - 1;
        up = p >= 0 && p < lane ? p : -1;
    }
    const unsigned long long path = node_paths(parent, a.K);
    const int above = __shfl(target, max(up, 0), 64);
    const bool good = lane < live && (up >= 0 ? token >= 0 && token == above : root < 0 || token == root);
    const unsigned long long bad = __ballot(!good);
    // deepest first, then the lowest index
    int rank = (path & bad) == 0 ? __popcll(path) << 6 | (63 - lane) : -1;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) rank = max(rank, __shfl_xor(rank, d, 64));
    const int last = rank < 0 ? -1 : 63 - (rank & 63);
    const unsigned long long kept = rank < 0 ? 0 : __shfl(path, max(last, 0), 64);
    const int next = __shfl(target, max(last, 0), 64);
    if (lane == 0) {
        a.node[b] = last;
        a.next[b] = last >= 0 ? next : root;
    }
    if (a.history) {
        const int len = min(max(a.lens[b], 0), a.capacity);
        const int i = __popcll(kept & ((1ull << lane) - 1));
        if ((kept >> lane & 1) && i < a.capacity - len) a.history[(size_t)b * a.capacity + len + i] = token;
        if (lane == 0) a.lens_out[b] = min(a.capacity - len, (int)__popcll(kept)) + len;
    }
}

// The vocabulary is cut so that a launch has about four workgroups for each of the 256 CUs; a slice of 512 tokens still
// has eight logits for each of 64 lanes.
int slice_of(int B, int V)
{
    int slice = kSliceMax;
    while (slice > 512 && (long long)B * ((V + slice - 1) / slice) < 512) slice /= 2;
    return slice;
}

}  // namespace

int logits_slices(int B, int V)
{
    const int slice = slice_of(B, V);
    return (V + slice - 1) / slice;
}

hipError_t launch_logits(const LogitsArgs& args, bool x_bf16, bool out_bf16, hipStream_t s)
{
    LogitsArgs a = args;
    a.slice = slice_of(a.B, a.V);
    a.slices = (a.V + a.slice - 1) / a.slice;
    a.rows = a.K;
    const dim3 grid(a.slices, a.B * ((a.K + a.rows - 1) / a.rows));
    const size_t lds = ((size_t)a.slice + a.slice / 32 + (a.n_bias > 0 ? a.slice : 0)) * 4;
    if (x_bf16) {
        if (out_bf16) logits_kernel<true, true><<<grid, dim3(kThreads), lds, s>>>(a);
        else logits_kernel<true, false><<<grid, dim3(kThreads), lds, s>>>(a);
    } else {
        if (out_bf16) logits_kernel<false, true><<<grid, dim3(kThreads), lds, s>>>(a);
        else logits_kernel<false, false><<<grid, dim3(kThreads), lds, s>>>(a);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess || !a.best) return e;
    const long long rows = (long long)a.B * a.K;
    logits_best_kernel<<<dim3((unsigned)((rows + kWaves - 1) / kWaves)), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_accept(const AcceptArgs& a, hipStream_t s)
{
    accept_kernel<<<dim3((a.B + kWaves - 1) / kWaves), dim3(kThreads), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
