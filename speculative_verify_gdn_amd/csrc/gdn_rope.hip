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
//   - a group of lanes holds one head, a lane two 16-byte pieces of it: for the
//     two halves those whose elements are pairs of one another, for neighbours
//     any two, taken half the turned part (or half the head, where not all of it turns)
//     apart so that the lanes of a group lie side by side.  So no element crosses lanes, and the norm is a sum over the group.
//   - where the head goes (dense rows, or a page of the cache) is an offset a
//     token.
// Measured: 16384 tokens of 48 heads of 128 (bf16, into the cache, 403 MB) 77.1 us, 5.2 TB/s; 8193 of 40
// heads of 128 (fp32, normed, 336 MB) 66.0 us; 16384 of 32 (bf16, 268 MB) 51.5 us: 97 to 100% of a copy of the same
// bytes.  1024 tokens in trees of 16, 32 heads of 256 (34 MB) 10.5 us: a workgroup's chain of reads, 9 us from its
// start to its last store.  Of these only a page id needs another read (the length); the others are waited for one by one
// as they stand: the norms' weights before the tokens' lengths, counts and parents, those each alone, the parts' places
// (arguments indexed by lane, so read like data) before the angles, and again before each head.  Heads asked for before
// that chain, or a head ahead, took longer in every case (waves then hold more registers, or reads come back in an order
// that the chain waits for).
#include "gdn_device.h"
#include "gdn_window_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;
constexpr int kTileMax = 32;        // tokens of a workgroup
constexpr int kAngles = 1024;       // sines (and cosines) of a workgroup
constexpr long long kGridX = 1 << 23;   // workgroups in x (a launch's threads there stay below 2^32)
// Reads of more than this go past the caches (tokens of 32 heads of 256, by their number: 2048, 33.5 MB read, 17.9 us past
// them and 14.7 through them; 4096 31.1 and 31.8; 8192 59.5 and 61.4).
constexpr long long kStreamBytes = 48 << 20;
constexpr long long kNowhere = 1LL << 62;   // (no position: a token that is not there)
constexpr double kInv2Pi = 0.15915494309189533577;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// E elements of one piece, 16 or 8 bytes or a single one: as they lie in memory, and as floats
template <bool BF16, int E, bool STREAM>
struct Piece {
    static constexpr int kWords = E * (BF16 ? 2 : 4) / 4;   // (a single bf16: 0)
    static_assert(kWords == 4 || kWords == 2 || E == 1, "a piece is 16 or 8 bytes or one element");
    typedef uint32_t words_t __attribute__((ext_vector_type(E == 1 ? 1 : kWords)));
    words_t raw;

    __device__ __forceinline__ void load(const char* p)
    {
        if constexpr (E == 1 && BF16) raw[0] = *reinterpret_cast<const uint16_t*>(p);
        else if constexpr (STREAM) raw = __builtin_nontemporal_load(reinterpret_cast<const words_t*>(p));
        else raw = *reinterpret_cast<const words_t*>(p);
    }
    __device__ __forceinline__ void floats(float* f) const
    {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = i & 1 ? bf16_hi(raw[i >> 1]) : bf16_lo(raw[i >> 1]);
        } else {
#pragma unroll
            for (int i = 0; i < E; ++i) f[i] = __uint_as_float(raw[i]);
        }
    }
    // as it came, to the bit (a conversion makes a signalling NaN a quiet one)
    __device__ __forceinline__ void keep(char* p) const
    {
        if constexpr (E == 1 && BF16) *reinterpret_cast<uint16_t*>(p) = (uint16_t)raw[0];
        else if constexpr (STREAM) __builtin_nontemporal_store(raw, reinterpret_cast<words_t*>(p));
        else *reinterpret_cast<words_t*>(p) = raw;
    }
    static __device__ __forceinline__ void store(char* p, const float* f)
    {
        if constexpr (E == 1) {
            store1<BF16>(p, 0, f[0]);
        } else {
            words_t w;
#pragma unroll
            for (int i = 0; i < kWords; ++i) {
                if constexpr (BF16) {
                    const bf16x2_t h = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
                    w[i] = __builtin_bit_cast(uint32_t, h);
                } else {
                    w[i] = __float_as_uint(f[i]);
                }
            }
            if constexpr (STREAM) __builtin_nontemporal_store(w, reinterpret_cast<words_t*>(p));
            else *reinterpret_cast<words_t*>(p) = w;
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
// whole wave by doubling: a lane holds how far it has come up from its node, and where it stands.  parent: lane i's is
// that of node i.
__device__ __forceinline__ int node_depth(int parent, int K, int t)
{
    const int lane = threadIdx.x & 63;
    int up = lane < K && parent >= 0 && parent < lane ? parent : -1;
    int depth = up >= 0;
    for (int d = 1; d < K; d <<= 1) {
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

// kPart: neighbours of heads that turn in part.  Their pieces turn or not each for itself, so that any whole number of
// pieces may turn, and the two of a lane are half the head apart: accesses of whole lines.  (16384 tokens of 32 heads of
// 80, bf16, 40 elements turned: 46 us, in pieces of half the size 76; 110304 of 4 heads of 128, 32 turned: 51.5 and 56.5.  With
// whole heads it has more registers to hold than there are: 16384 of 32 heads of 128, 54.5 and 51.4.)
enum Pairs { kHalves, kNeighbours, kPart };

// E: elements of a piece; NP: pairs of pieces of a lane; STREAM: past the caches; LANES: the tokens are looked after by a
// lane each, not by a wave
template <bool BF16, int E, int NP, Pairs PAIRS, bool STREAM, bool LANES>
__device__ __forceinline__ void rope_heads(const RopeArgs& a)
{
    constexpr int ES = BF16 ? 2 : 4;
    constexpr int PE = E > 1 ? E / 2 : 1;   // pairs within a piece (neighbours)
    __shared__ Token info[kTileMax];
    __shared__ long long where[LANES ? kTileMax : 1];
    __shared__ float cs[kAngles], sn[kAngles];
    __shared__ float weight[2][kRopeHeadMax];

    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t tokens = (uint32_t)a.B * a.K, first = (blockIdx.x + blockIdx.z * gridDim.x) * a.tile;
    if (first >= tokens) return;
    if constexpr (LANES || STREAM)   // (many workgroups) done where none of the tokens is there
        if (a.count) {
            const uint32_t b = first / (uint32_t)a.K, t = first - b * a.K;
            if (t + a.tile <= (uint32_t)a.K && (int)t >= a.count[b]) return;
        }
    const int n = (int)min((uint32_t)a.tile, tokens - first);
    const int half = a.rot >> 1;

    // the norms' weights are asked for first
    float w[2][kRopeHeadMax / kThreads];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < kRopeHeadMax / kThreads; ++i) {
            const int d = threadIdx.x + i * kThreads;
            w[s][i] = a.part[s].w && d < a.D ? a.part[s].w[d] : 0.0f;
        }

    // A group of lanes holds a head; lane l of it the pieces l and l + turned of the part that turns, or l and l +
    // (pairs - turned) of the rest; kPart: l and l + pairs of the head.
    const int h0 = blockIdx.y * a.chunk, nh = min(a.chunk, a.heads - h0);
    const int group = threadIdx.x >> a.lanes_log2, step = kThreads >> a.lanes_log2;
    const int l = threadIdx.x & ((1 << a.lanes_log2) - 1);
    const int pairs = a.D / (2 * E);   // pairs of pieces of a head
    const int turned = half / E;       // those of them that turn
    int at[NP], bt[NP];                // this lane's, in elements from the head's start
#pragma unroll
    for (int k = 0; k < NP; ++k) {
        const int j = l + (k << a.lanes_log2);
        if (PAIRS == kPart) at[k] = j * E, bt[k] = (j + pairs) * E;
        else if (PAIRS == kNeighbours && E == 1 && j < turned) at[k] = 2 * j, bt[k] = 2 * j + 1;
        else if (j < turned) at[k] = j * E, bt[k] = at[k] + half;
        else at[k] = a.rot + (j - turned) * E, bt[k] = at[k] + (pairs - turned) * E;
    }
    // the r-th head of the workgroup: of which token and part, and which of the part's heads
    struct Head {
        int i, s, h;
    };
    auto head_of = [&](int r) {
        const int i = r / nh;
        Head x{i, 0, h0 + r - i * nh};
        if (x.h >= a.part[0].H) {
            x.h -= a.part[0].H;
            x.s = 1;
            if (x.h >= a.part[1].H) {
                x.h -= a.part[1].H;
                x.s = 2;
            }
        }
        return x;
    };
    Piece<BF16, E, STREAM> u[NP], v[NP];
    auto load = [&](const char* x) {
#pragma unroll
        for (int k = 0; k < NP; ++k)
            if (l + (k << a.lanes_log2) < pairs) {
                u[k].load(x + at[k] * ES);
                v[k].load(x + bt[k] * ES);
            }
    };
    // the byte offset of a sequence's place `at` in a plane of the cache, below 0: it has no page
    auto page_of = [&](int b, long long at) -> long long {
        const long long slot = at >> a.g.page_log2;
        const int id = slot < a.P ? a.table[(size_t)b * a.P + slot] : -1;
        if ((unsigned)id >= (unsigned)a.g.n_pages) return -1;
        return ((((long long)id * a.g.Hkv) << a.g.page_log2) + (at & ((1 << a.g.page_log2) - 1))) * a.g.row_bytes;
    };
    // the i-th token of the workgroup, token t of sequence b, in a part
    auto place = [&](int i, int part, int b, int t, bool there, long long page_at) {
        const RopePart& r = a.part[part];
        info[i].from[part] = b * r.xs[0] + t * r.xs[1];
        info[i].to[part] = !there ? -1 : r.paged ? page_at : b * r.ys[0] + t * r.ys[1];
    };
    // the sine and cosine of its pair j
    auto angle = [&](int i, int j, long long p, double freq) {
        const double turns = (double)p * freq * kInv2Pi;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        cs[i * half + j] = a.mscale * c;
        sn[i * half + j] = a.mscale * s;
    };
    if constexpr (LANES) {   // a lane a token, then its pairs side by side with those of other tokens
        const int j = threadIdx.x & ((1 << a.half_log2) - 1);
        const double freq = j < half ? a.freqs[j] : 0.0;
        if (threadIdx.x < n) {
            const int i = threadIdx.x;
            const uint32_t tok = first + i;
            const int b = (int)(tok / (uint32_t)a.K), t = (int)(tok - (uint32_t)b * a.K);
            const long long len = a.lens ? max(a.lens[b], 0) : 0;
            const bool there = !a.count || t < a.count[b];
            where[i] = !there ? kNowhere : a.pos ? (long long)a.pos[tok] : len + t;
            const long long page_at = a.table ? page_of(b, len + t) : -1;
#pragma unroll
            for (int part = 0; part < 3; ++part) place(i, part, b, t, there, page_at);
        }
        __syncthreads();
        if (j < half)
            for (int i = threadIdx.x >> a.half_log2; i < n; i += kThreads >> a.half_log2)
                if (where[i] != kNowhere) angle(i, j, where[i], freq);
    } else {   // a wave a token, or several waves where there are fewer tokens
        const int share = max(kWaves / a.tile, 1), sub = wave % share;
        for (int i = wave / share; i < n; i += kWaves / share) {
            const uint32_t tok = first + i;
            const int b = (int)(tok / (uint32_t)a.K), t = (int)(tok - (uint32_t)b * a.K);
            const int32_t parent = a.parent && lane < a.K ? a.parent[(size_t)b * a.K + lane] : -1;
            const int j0 = lane + 64 * sub;
            const double freq = j0 < half ? a.freqs[j0] : 0.0;
            const long long len = a.lens ? max(a.lens[b], 0) : 0;
            const bool there = !a.count || t < a.count[b];
            if (sub == 0) {
                const long long page_at = a.table ? page_of(b, len + t) : -1;
                if (lane < 3) place(i, lane, b, t, there, page_at);
            }
            const long long p = a.pos      ? (long long)a.pos[tok]
                                : a.parent ? len + node_depth(parent, a.K, t)
                                           : len + t;
            for (int j = j0; j < half; j += 64 * share) angle(i, j, p, j == j0 ? freq : a.freqs[j]);
        }
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int i = 0; i < kRopeHeadMax / kThreads; ++i)
            if (a.part[s].w) weight[s][threadIdx.x + i * kThreads] = w[s][i];
    __syncthreads();

    const float inv_d = 1.0f / (float)a.D;
    for (int r = group; r < n * nh; r += step) {
        const Head x = head_of(r);
        const RopePart& part = a.part[x.s];
        const long long to = info[x.i].to[x.s];
        if (to < 0) continue;
        load(static_cast<const char*>(part.x) + info[x.i].from[x.s] + x.h * part.xs[2]);
        float f[NP][E], g[NP][E];
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            u[k].floats(f[k]);
            v[k].floats(g[k]);
        }
        char* y = static_cast<char*>(part.y) + to +
                  x.h * (part.paged ? (long long)a.g.row_bytes << a.g.page_log2 : part.ys[2]);
        if (part.w) {
            float q = 0.0f;
#pragma unroll
            for (int k = 0; k < NP; ++k)
                if (l + (k << a.lanes_log2) < pairs) {
#pragma unroll
                    for (int e = 0; e < E; ++e) q = fmaf(f[k][e], f[k][e], fmaf(g[k][e], g[k][e], q));
                }
            q = group_sum(q, a.lanes_log2);
            const float z = 1.0f / sqrtf(q * inv_d + a.eps);
#pragma unroll
            for (int k = 0; k < NP; ++k)
                if (l + (k << a.lanes_log2) < pairs) {
#pragma unroll
                    for (int e = 0; e < E; ++e) {
                        f[k][e] *= z * weight[x.s][at[k] + e];
                        g[k][e] *= z * weight[x.s][bt[k] + e];
                    }
                }
        }
#pragma unroll
        for (int k = 0; k < NP; ++k) {
            const int j = l + (k << a.lanes_log2);
            if (j >= pairs) continue;
            // (the second piece turns only where the first does)
            const bool tu = part.turned && (PAIRS == kPart ? at[k] < a.rot : j < turned);
            const bool tv = PAIRS == kPart ? part.turned && bt[k] < a.rot : tu;
            if (!tu && !part.w) {
                u[k].keep(y + at[k] * ES);
                v[k].keep(y + bt[k] * ES);
                continue;
            }
            auto turn = [](float& p, float& q, float c, float s) {
                const float p0 = p, q0 = q;
                p = fmaf(p0, c, -(q0 * s));
                q = fmaf(q0, c, p0 * s);
            };
            const float *c = cs + x.i * half, *s = sn + x.i * half;
            if constexpr (PAIRS == kHalves || E == 1) {   // the pair: an element of each piece
                if (tu)
#pragma unroll
                    for (int e = 0; e < E; ++e) turn(f[k][e], g[k][e], c[j * E + e], s[j * E + e]);
            } else if constexpr (PAIRS == kNeighbours) {   // the two pieces turn by themselves
                if (tu)
#pragma unroll
                    for (int e = 0; e < PE; ++e) {
                        const int i = j * PE + e, m = (turned + j) * PE + e;
                        turn(f[k][2 * e], f[k][2 * e + 1], c[i], s[i]);
                        turn(g[k][2 * e], g[k][2 * e + 1], c[m], s[m]);
                    }
            } else {
                if (tu)
#pragma unroll
                    for (int e = 0; e < PE; ++e) turn(f[k][2 * e], f[k][2 * e + 1], c[j * PE + e], s[j * PE + e]);
                if (tv)
#pragma unroll
                    for (int e = 0; e < PE; ++e)
                        turn(g[k][2 * e], g[k][2 * e + 1], c[(pairs + j) * PE + e], s[(pairs + j) * PE + e]);
            }
            Piece<BF16, E, STREAM>::store(y + at[k] * ES, f[k]);
            if (PAIRS == kPart && !tv && !part.w) v[k].keep(y + bt[k] * ES);
            else Piece<BF16, E, STREAM>::store(y + bt[k] * ES, g[k]);
        }
    }
}

// Eight waves a SIMD: with six (ten registers more) the large windows took 3 to 6% longer.  For it the bf16 kernels keep
// registers in memory: 8 bytes a lane with kPart, 12 to 20 element by element.
template <bool BF16, Pairs PAIRS, bool STREAM, bool LANES>
__global__ __launch_bounds__(kThreads, 8) void rope_kernel(RopeArgs a)
{
    rope_heads<BF16, BF16 ? 8 : 4, 1, PAIRS, STREAM, LANES>(a);
}

// Pieces of 8 bytes, and element by element: for turned parts that no whole pieces (halves: pairs of them) of 16 bytes make
// up (16384 tokens of 32 heads of 96, bf16, halves: 24 elements of each turned 74 us, 22 197).
template <bool BF16, int E, int NP, Pairs PAIRS, bool LANES>
__global__ __launch_bounds__(kThreads, 8) void rope_narrow_kernel(RopeArgs a)
{
    rope_heads<BF16, E, NP, PAIRS, false, LANES>(a);
}

template <bool BF16, bool INTERLEAVED, bool LANES>
void launch(const RopeArgs& a, int e, bool stream, dim3 grid, hipStream_t s)
{
    constexpr int E = BF16 ? 8 : 4;
    constexpr Pairs kWhole = INTERLEAVED ? kNeighbours : kHalves, kSome = INTERLEAVED ? kPart : kHalves;
    const dim3 block(kThreads);
    if constexpr (BF16 || !INTERLEAVED)   // (neighbours in fp32 fill 8 bytes by themselves)
        if (e == 1) {
            rope_narrow_kernel<BF16, 1, 4, kWhole, LANES><<<grid, block, 0, s>>>(a);
            return;
        }
    if (e < E) rope_narrow_kernel<BF16, E / 2, BF16 ? 1 : 2, kSome, LANES><<<grid, block, 0, s>>>(a);
    else if (INTERLEAVED && a.rot < a.D)
        stream ? rope_kernel<BF16, kSome, true, LANES><<<grid, block, 0, s>>>(a)
               : rope_kernel<BF16, kSome, false, LANES><<<grid, block, 0, s>>>(a);
    else
        stream ? rope_kernel<BF16, kWhole, true, LANES><<<grid, block, 0, s>>>(a)
               : rope_kernel<BF16, kWhole, false, LANES><<<grid, block, 0, s>>>(a);
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
    const int whole = INTERLEAVED ? 1 : 2;   // pieces that the turned part has to be made of
    const int e = a.rot % (whole * E) == 0 ? E : a.rot % (whole * E / 2) == 0 ? E / 2 : 1;   // elements of a piece
    a.lanes_log2 = min(log2_up(a.D / (2 * e)), 6);
    a.heads = a.part[0].H + a.part[1].H + a.part[2].H;
    const long long tokens = (long long)a.B * a.K;
    const int half = a.rot / 2, pass = kThreads >> a.lanes_log2;
    // Tokens of a workgroup: as many as give its groups a head each (tokens of 6 heads of 64, 65536 of them: 100 us with
    // one a workgroup, 43 with four), and three where there are many workgroups left (4096 x 4 tokens of 32 heads of 128:
    // 58.6 us with one, 52.1 with four; 8192 of 32 heads of 256: 56.3 with one, 57.2 with two).
    a.tile = 1;
    while (2 * a.tile <= kTileMax && 2 * a.tile * half <= kAngles &&
           ((a.tile * a.heads < pass && tokens / (2 * a.tile) >= 1024) ||
            (a.tile * a.heads < 3 * pass && tokens / (2 * a.tile) >= 2048)))
        a.tile *= 2;
    const long long tiles = (tokens + a.tile - 1) / a.tile;
    // A head a group, and several for each where that makes more workgroups than four a CU (128 windows of 16 tokens of 32
    // heads of 256: 14.8 us, with one head a group 16.8).
    int chunks = (a.heads * a.tile + pass - 1) / pass;
    while (chunks > 1 && tiles * chunks > 1024) chunks = (chunks + 1) / 2;
    a.chunk = (a.heads + chunks - 1) / chunks;
    const dim3 grid((unsigned)min(tiles, kGridX), (a.heads + a.chunk - 1) / a.chunk, (unsigned)((tiles + kGridX - 1) / kGridX));
    a.half_log2 = log2_up(half);
    // Past the caches go accesses of whole lines, or of runs of 64 bytes and at least 128: parts of lines are joined in the
    // caches (13278 tokens of 30 heads of 128, bf16, 32 elements turned: 69 us past them, 53 through them; 40562 of 24 of 64
    // 74 and 58; but 16384 of 32 of 256, 64 turned, runs of 64 and 192, 45.8 and 48.7).
    const int es = BF16 ? 2 : 4, run = (INTERLEAVED ? a.D / 2 : half) * es, rest = INTERLEAVED ? 0 : (a.D - a.rot) / 2 * es;
    const bool stream = (long long)tokens * a.heads * a.D * es > kStreamBytes && (run | rest) % 64 == 0 && max(run, rest) >= 128;
    // A lane a token where a workgroup has more of them than waves (110304 tokens of 4 heads of 96: 67 us with a wave a token,
    // 48 with a lane); the depth in a tree takes a wave.
    if (a.tile > kWaves && (a.pos || !a.parent)) launch<BF16, INTERLEAVED, true>(a, e, stream, grid, s);
    else launch<BF16, INTERLEAVED, false>(a, e, stream, grid, s);
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
