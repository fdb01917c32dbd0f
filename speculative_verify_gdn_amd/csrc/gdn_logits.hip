// gdn_logits.hip -- the logits of a verify window adjusted (penalties for tokens
// already seen, biases, grammar masks, temperature) with the best token of each
// node, and the accepted node of a draft tree (include/gdn.h: gdn_logits_adjust,
// gdn_accept_tree).
//
// A logit x of token v behind node t becomes, with n how often v stands in the
// text since `start` and on the path to t, and seen if it stands in the text at all
// or on that path:
//   seen: x (x > 0 ? 1 / repetition : repetition);   n > 0: x - (frequency n + presence);
//   x + bias;   x (1 / temperature);   not allowed: -inf
// One read of the logits and one write: memory bound, if the counts cost
// little.  So a workgroup takes a slice of the vocabulary for some rows of one
// sequence: it walks the text once, counts the tokens of its slice in LDS (16
// bits each, 16 KB for 8192 tokens), and then streams; a lane knows which of its tokens have a
// count or a bias, and looks up those alone.
// Every operation is one rounding of 32 bits in the order above, so that equal
// logits stay equal and the best is the lowest of them.  The reciprocals of repetition and temperature are formed once a
// workgroup, each rounded: a product with one is off by up to two half steps where a division is by one, and a division
// is about ten vector instructions for each logit, in a stream whose vector instructions issue in 0.83 of the time.
//
// Measured: 64 rows of 131072, fp32, with noise and output (101 MB) 22.4 us, of which the stream 19.6 (5.1 TB/s);
// 32 ragged windows of 8 rows of 131072, bf16, masks, biases and texts of 4000 (78 MB)
// 20.8 to 23.6 us box to box: the counting and what it makes the stream look up take 2 us each, joining the best 2.5, a workgroup's reads before its
// stream 3; without texts, biases, masks and best 14.0.
// With the logits of the counted tokens left to a second kernel (a hash table a sequence) the stream was 1 us shorter, and
// that kernel's scattered reads and writes took 13.
#include "gdn_device.h"
#include "gdn_window_internal.h"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2_t __attribute__((ext_vector_type(2)));
// 16 bytes at an element's own alignment (rows of an odd length start anywhere)
typedef uint32_t u32x4_any_t __attribute__((ext_vector_type(4), aligned(2)));

// eight values as they lie in memory
template <bool BF16>
struct Raw8 {
    u32x4_any_t u[BF16 ? 1 : 2];

    __device__ __forceinline__ void load(const void* row, int at)
    {
        const char* p = static_cast<const char*>(row) + (size_t)at * (BF16 ? 2 : 4);
#pragma unroll
        for (int i = 0; i < (BF16 ? 1 : 2); ++i) u[i] = reinterpret_cast<const u32x4_any_t*>(p)[i];
    }
    // of a row of fewer than eight: the last one again and again
    __device__ __forceinline__ void load_few(const void* row, int V)
    {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int at = min(e, V - 1);
            if constexpr (BF16) {
                const uint32_t h = static_cast<const uint16_t*>(row)[at];
                u[0][e >> 1] = e & 1 ? u[0][e >> 1] | h << 16 : h;
            } else {
                u[e >> 2][e & 3] = static_cast<const uint32_t*>(row)[at];
            }
        }
    }
    __device__ __forceinline__ void floats(float* f) const
    {
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 4; ++i) f[2 * i] = bf16_lo(u[0][i]), f[2 * i + 1] = bf16_hi(u[0][i]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(u[i >> 2][i & 3]);
        }
    }
};

// the last m < 8 of eight to the front
__device__ __forceinline__ void to_front(float* f, int m)
{
#pragma unroll
    for (int d = 4; d; d >>= 1)
        if ((8 - m) & d) {
#pragma unroll
            for (int e = 0; e + d < 8; ++e) f[e] = f[e + d];
        }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* row, int at, const float* f)
{
    char* p = static_cast<char*>(row) + (size_t)at * (BF16 ? 2 : 4);
    u32x4_any_t u;
    if constexpr (BF16) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const bf16x2_t h = {(__bf16)f[2 * i], (__bf16)f[2 * i + 1]};
            u[i] = __builtin_bit_cast(uint32_t, h);
        }
        __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any_t*>(p));
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = __float_as_uint(f[4 * h + i]);
            __builtin_nontemporal_store(u, reinterpret_cast<u32x4_any_t*>(p) + h);
        }
    }
}

// the largest over a wave (NaN is passed over)
__device__ __forceinline__ float wave_max(float v)
{
    v = fmaxf(v, dpp_mov<kDppQuadXor1>(v));
    v = fmaxf(v, dpp_mov<kDppQuadXor2>(v));
    v = fmaxf(v, dpp_mov<kDppRowHalfMirror>(v));
    v = fmaxf(v, dpp_mov<kDppRowMirror>(v));
    v = fmaxf(v, __shfl_xor(v, 16, 64));
    return fmaxf(v, __shfl_xor(v, 32, 64));
}

// A score and its token as one number: the larger score is the larger number, the lower token where they are equal; 0
// is none.  (Scores that are NaN or -inf have none.)
__device__ __forceinline__ unsigned long long key_of(float score, int token)
{
    const uint32_t u = __float_as_uint(score + 0.0f);   // (-0 is 0)
    const uint32_t up = u & 0x80000000u ? ~u : u | 0x80000000u;
    return (unsigned long long)up << 32 | (0xffffffffu - (uint32_t)token);
}

__device__ __forceinline__ int token_of(unsigned long long key)
{
    return key ? (int)(0xffffffffu - (uint32_t)key) : -1;
}

// the smallest over a wave
__device__ __forceinline__ int wave_min(int v)
{
    auto with = [&](int u) { v = min(v, u); };
    with(__builtin_amdgcn_update_dpp(0, v, kDppQuadXor1, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(0, v, kDppQuadXor2, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(0, v, kDppRowHalfMirror, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(0, v, kDppRowMirror, 0xF, 0xF, false));
    with(__shfl_xor(v, 16, 64));
    with(__shfl_xor(v, 32, 64));
    return v;
}

// the largest over a wave of numbers without a sign
__device__ __forceinline__ uint32_t wave_most(uint32_t v)
{
    auto with = [&](int u) { v = max(v, (uint32_t)u); };
    with(__builtin_amdgcn_update_dpp(0, (int)v, kDppQuadXor1, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(0, (int)v, kDppQuadXor2, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(0, (int)v, kDppRowHalfMirror, 0xF, 0xF, false));
    with(__builtin_amdgcn_update_dpp(0, (int)v, kDppRowMirror, 0xF, 0xF, false));
    with(__shfl_xor((int)v, 16, 64));
    with(__shfl_xor((int)v, 32, 64));
    return v;
}

// the sums of the lanes up to each
__device__ __forceinline__ int wave_sums(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xF, 0xF, false);   // within a row: 1, 2, 4, 8 lanes before
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xF, 0xF, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xA, 0xF, false);   // rows 1 and 3: the last of the row before
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xC, 0xF, false);   // rows 2 and 3: the last of row 1
    return v;
}

// the node above lane's of a tree (parent: its entry) or of a chain, below 0: none
__device__ __forceinline__ int node_above(const int32_t* parent, int N)
{
    const int lane = threadIdx.x & 63;
    if (lane >= N) return -1;
    const int p = parent ? parent[lane] : lane - 1;
    return p >= 0 && p < lane ? p : -1;
}

// the nodes on the path root..i as a bit mask, in lane i, from the node above each, by doubling (a whole wave)
__device__ __forceinline__ unsigned long long node_paths(int up, int N)
{
    unsigned long long path = 1ull << (threadIdx.x & 63);
    for (int d = 1; d < N; d <<= 1) {
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

// What a thread reads of a row: eight logits, their noise and whether they are allowed.  Eight that would pass the
// row's end are its last eight instead (to_front): no load depends on a lane's place.
template <bool XBF16, bool NOISE>
struct Row8 {
    Raw8<XBF16> x;
    Raw8<false> z;
    uint32_t allow;
};

// where a row starts: its logits, its noise and its mask
template <bool XBF16, bool NOISE>
struct Rows {
    const char* x;
    const float* z;
    const uint8_t* allow;
    int V, allow_bytes;
    size_t x_step;

    __device__ __forceinline__ Rows(const LogitsArgs& a, size_t row)
        : V(a.V), allow_bytes((a.V + 31) / 32 * 4), x_step(a.x_stride * (XBF16 ? 2 : 4))
    {
        x = static_cast<const char*>(a.x) + row * x_step;
        z = NOISE ? a.noise + row * a.V : nullptr;
        allow = a.mask ? reinterpret_cast<const uint8_t*>(a.mask) + row * allow_bytes : nullptr;
    }
    __device__ __forceinline__ void next()
    {
        x += x_step;
        if constexpr (NOISE) z += V;
        if (allow) allow += allow_bytes;
    }
    __device__ __forceinline__ void load(Row8<XBF16, NOISE>& r, int v) const
    {
        if (V >= 8) {
            r.x.load(x, min(v, V - 8));
            if constexpr (NOISE) r.z.load(z, min(v, V - 8));
        } else {
            r.x.load_few(x, V);
            if constexpr (NOISE) r.z.load_few(z, V);
        }
        if (allow) r.allow = allow[min(v >> 3, allow_bytes - 1)];
    }
};

struct Params {
    float rep, less, presence, frequency, cool;   // less, cool: the reciprocals of repetition and temperature

    __device__ __forceinline__ Params(const float* p, int b)
        : rep(1.0f), less(1.0f), presence(0.0f), frequency(0.0f), cool(1.0f)
    {
        if (!p) return;
        p += (size_t)b * 4;
        rep = p[0], less = 1.0f / rep, presence = p[1], frequency = p[2];
        if (p[3] >= 0x1p-126f) cool = 1.0f / p[3];
    }
};

// f where bit e of `bits` is set, -inf elsewhere
__device__ __forceinline__ float only(float f, uint32_t bits, int e)
{
    const int m = __builtin_amdgcn_sbfe((int)bits, e, 1);
    return __int_as_float(__builtin_amdgcn_bitop3_b32(__float_as_int(f), (int)0xff800000, m, 0xe4));   // m ? f : -inf
}

// What is known of the tokens of a slice, in LDS: their counts, and whether they stand in the text before `start` or have
// a bias; a bit map of the drafted ones.  Narrow: 16 bits a token (14 of the count, one for a bias, one for the text before
// `start`), and a list of the slice's biases; a token with a bias has its place in that list instead, and its count
// there.  Long, for texts that may be of more than 16000 tokens: the same, and such a text is counted in parts, between
// which counts of 3000 and more go to a list of their own (all but one).  Wide: 32 bits a token, and a bias's entry for
// each; where that list could overflow or the biases are more than two a thread.  (64 rows of 131072, fp32, texts of
// 1000: 20.1 us wide, 18.5 narrow; of 15000 36.5 and 25.0.)
constexpr int kStep = kThreads * 4;   // tokens of a text that a workgroup reads at once
constexpr int kPart = 12 * kStep;     // those of a part (the first has a step more)
constexpr int kMuch = 3000, kNarrowText = 16000;
static_assert(kNarrowText + kKvWindowMax < 1 << 14 && kMuch + kPart + kKvWindowMax < 1 << 14 &&
                  kPart + kStep + kKvWindowMax < 1 << 14, "a count with a window's drafts has 14 bits");
constexpr int kSpills = 128;
constexpr int kLongText = kSpills * (kMuch - 1);
enum Size { kNarrow, kLong, kWide };
constexpr int kNarrowBias = 2 * kThreads;
constexpr int kEach = kNarrowBias / kThreads;   // biases of a thread

template <Size SIZE, int TOKENS>
struct Known {
    static constexpr bool WIDE = SIZE == kWide, LONG = SIZE == kLong;
    static constexpr int kBits = WIDE ? 32 : 16;
    static constexpr uint32_t kCount = (1u << (kBits - 2)) - 1, kBias = 1u << (kBits - 2), kSeen = 1u << (kBits - 1);
    uint32_t cnt[WIDE ? TOKENS : TOKENS / 2];
    uint32_t drafted[TOKENS / 32];
    int entry[WIDE ? TOKENS : 1];
    float bias_value[WIDE ? 1 : kNarrowBias];
    uint32_t bias_cnt[WIDE ? 1 : kNarrowBias / 2];   // (16 bits each)
    uint16_t bias_token[WIDE ? 1 : kNarrowBias];
    int biases[kEach * kWaves];
    int spill_token[LONG ? kSpills : 1];
    uint32_t spill_cnt[LONG ? kSpills : 1];

    __device__ __forceinline__ void clear()
    {
        for (int i = threadIdx.x; i < (int)(sizeof(cnt) / 16); i += kThreads)
            reinterpret_cast<uint4*>(cnt)[i] = make_uint4(0, 0, 0, 0);
        for (int i = threadIdx.x; i < TOKENS / 32; i += kThreads) drafted[i] = 0;
        if constexpr (WIDE)
            for (int i = threadIdx.x; i < TOKENS; i += kThreads) entry[i] = -1;
        if (LONG && threadIdx.x < kSpills) spill_token[threadIdx.x] = -1, spill_cnt[threadIdx.x] = 0;
    }
    static __device__ __forceinline__ void add16(uint32_t* p, int i, int n) { atomicAdd(&p[i >> 1], (uint32_t)n << 16 * (i & 1)); }
    static __device__ __forceinline__ uint16_t& at16(uint32_t* p, int i) { return reinterpret_cast<uint16_t*>(p)[i]; }
    __device__ __forceinline__ void draft(int u) { atomicOr(&drafted[u >> 5], 1u << (u & 31)); }
    __device__ __forceinline__ void add(int u, int n)
    {
        if constexpr (WIDE) atomicAdd(&cnt[u], (uint32_t)n);
        else add16(cnt, u, n);
    }
    // much counted tokens to their list (there are seldom any)
    __device__ __forceinline__ void spill()
    {
        if constexpr (LONG) {
            constexpr int kEights = TOKENS / 8 / kThreads;   // a thread's
            uint32_t most = 0;
#pragma unroll
            for (int r = 0; r < kEights; ++r) {
                const uint4 w = reinterpret_cast<const uint4*>(cnt)[threadIdx.x + r * kThreads];
                for (const uint32_t x : {w.x, w.y, w.z, w.w}) most = max(most, max(x & kCount, x >> 16 & kCount));
            }
            if (most < kMuch) return;
#pragma clang loop unroll(disable)
            for (int i = 0; i < 8 * kEights; ++i) {
                const int u = (threadIdx.x + (i >> 3) * kThreads) * 8 + (i & 7);
                const uint32_t c = at16(cnt, u), n = c & kCount;
                if (n < kMuch) continue;
                at16(cnt, u) = (uint16_t)(c - (n - 1));
                int at = 0;
                for (;;) {
                    const int was = atomicCAS(&spill_token[at], -1, u);
                    if (was == -1 || was == u || at == kSpills - 1) break;
                    ++at;
                }
                atomicAdd(&spill_cnt[at], n - 1);
            }
        }
    }
    // what that list has of a token
    __device__ __forceinline__ uint32_t spilled(int u) const
    {
        if constexpr (LONG)
#pragma clang loop unroll(disable)
            for (int i = 0; i < kSpills && spill_token[i] != -1; ++i)
                if (spill_token[i] == u) return spill_cnt[i];
        return 0;
    }
    __device__ __forceinline__ void mark(int u, uint32_t bit)
    {
        if constexpr (WIDE) atomicOr(&cnt[u], bit);
        else atomicOr(&cnt[u >> 1], bit << 16 * (u & 1));
    }
    // The biases of the slice, in four steps with a barrier between each and the next; narrow: entries tid, tid + kThreads,
    // ... are the thread's, id and value.
    __device__ __forceinline__ void ask_biases(const LogitsArgs& a, int v0, int nv, const int* id, unsigned long long* which)
    {
        const int tid = threadIdx.x;
        if constexpr (!WIDE)
#pragma unroll
            for (int r = 0; r < kEach; ++r) {
                which[r] = __ballot(tid + r * kThreads < a.n_bias && (uint32_t)id[r] - (uint32_t)v0 < (uint32_t)nv);
                if ((tid & 63) == 0) biases[r * kWaves + (tid >> 6)] = (int)__popcll(which[r]);
            }
    }
    __device__ __forceinline__ void take_biases(const LogitsArgs& a, int b, int v0, int nv, const int* id, const float* value,
                                                const unsigned long long* which)
    {
        const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
        if constexpr (WIDE) {
            const int32_t* ids = a.bias_ids + (size_t)b * a.n_bias;
            for (int i = tid; i < a.n_bias; i += kThreads) {
                const uint32_t u = (uint32_t)ids[i] - (uint32_t)v0;
                if (u < (uint32_t)nv) {
                    atomicMax(&entry[u], i);   // (a token named twice: its last entry)
                    mark(u, kBias);
                }
            }
        } else {
#pragma unroll
            for (int r = 0; r < kEach; ++r) {
                int at = (int)__popcll(which[r] & ((1ull << lane) - 1));
#pragma unroll
                for (int i = 0; i < kEach * kWaves; ++i) at += i < r * kWaves + wave ? biases[i] : 0;
                if (which[r] >> lane & 1) {
                    bias_token[at] = (uint16_t)(id[r] - v0);
                    bias_value[at] = value[r];
                }
            }
        }
    }
    // (a token named twice: all of its entries have its count, and its word the last one's place)
    __device__ __forceinline__ int listed() const
    {
        int all = 0;
#pragma unroll
        for (int i = 0; i < kEach * kWaves; ++i) all += biases[i];
        return all;
    }
    __device__ __forceinline__ void count_biases()
    {
        if constexpr (!WIDE)
            for (int i = threadIdx.x, all = listed(); i < all; i += kThreads) at16(bias_cnt, i) = at16(cnt, bias_token[i]);
    }
    __device__ __forceinline__ void place_biases()
    {
        if constexpr (!WIDE)
            for (int i = threadIdx.x, all = listed(); i < all; i += kThreads) {
                const int u = bias_token[i], shift = 16 * (u & 1);
                uint32_t* const word = &cnt[u >> 1];
                const uint32_t mine = kBias | i;
                for (uint32_t was = *word;;) {
                    const uint32_t half = was >> shift & 0xffffu;
                    // (a count has kBias nowhere; with kSeen alone it is no place either)
                    if ((half & kBias) && half > mine) break;
                    const uint32_t now = atomicCAS(word, was, (was & ~(0xffffu << shift)) | mine << shift);
                    if (now == was) break;
                    was = now;
                }
            }
    }
    // n more of a token, once the biases are in place
    __device__ __forceinline__ void add_later(int u, int n)
    {
        if constexpr (!WIDE) {
            const uint32_t c = at16(cnt, u);
            if (c & kBias) {
                add16(bias_cnt, c & (kNarrowBias - 1), n);
                return;
            }
        }
        add(u, n);
    }
    // which of eight tokens from u on need more than the mask and the temperature
    __device__ __forceinline__ uint32_t which(int u) const
    {
        uint32_t some = reinterpret_cast<const uint8_t*>(drafted)[u >> 3];
        if constexpr (WIDE) {
#pragma unroll
            for (int e = 0; e < 8; ++e) some |= min(cnt[u + e], 1u) << e;
        } else {
            uint32_t two = 0;   // bits 0, 2, 4, 6: the even ones; 16, 18, ...: the odd ones
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const u16x2_t w = __builtin_elementwise_min(__builtin_bit_cast(u16x2_t, cnt[(u >> 1) + i]), (u16x2_t){1, 1});
                two |= __builtin_bit_cast(uint32_t, w) << 2 * i;
            }
            some |= (two | two >> 15) & 0xffu;
        }
        return some;
    }
    // what is known of a token: its count with kSeen, and its bias (if it has one)
    __device__ __forceinline__ uint32_t look(const LogitsArgs& a, int b, int u, bool& biased, float& bias) const
    {
        uint32_t c;
        if constexpr (WIDE) c = cnt[u];
        else c = reinterpret_cast<const uint16_t*>(cnt)[u];
        biased = c & kBias;
        if (biased) {
            if constexpr (WIDE) {
                c &= ~kBias;
                bias = a.bias_values[(size_t)b * a.n_bias + entry[u]];
            } else {
                const int i = c & (kNarrowBias - 1);
                c = reinterpret_cast<const uint16_t*>(bias_cnt)[i];
                bias = bias_value[i];
            }
        }
        return c;
    }
};

// The i-th workgroup's sequence and rows t0 to t1, at most a.rows of them; false: there are none.  Windows differ in length;
// where the sequences are few, those with all their rows come first and the shorter ones behind them, so that each CU gets
// about the same number of rows (32 windows of 1 to 8 rows of 131072: 7 to 10 rows a CU where it was 4 to 14, 24.6 to 23.2
// us).
__device__ __forceinline__ bool rows_of(const LogitsArgs& a, int i, int& b, int& t0, int& t1)
{
    if (a.count && a.B <= 64) {
        const int lane = threadIdx.x & 63;
        const int count = lane < a.B ? clamp_count(a.count, lane, a.K) : 0;
        const int full = count / a.rows, rest = count - full * a.rows;
        const int upto = wave_sums(full);   // of this and the sequences before
        const int all = __shfl(upto, 63, 64);
        int g;
        if (i < all) {
            b = (int)__popcll(__ballot(upto <= i));
            g = i - __shfl(upto - full, b, 64);
        } else {
            const unsigned long long rests = __ballot(rest > 0);
            const int rank = (int)__popcll(rests & ((1ull << lane) - 1));
            const unsigned long long it = __ballot(rest > 0 && rank == i - all);
            if (it == 0) return false;
            b = __ffsll((long long)it) - 1;
            g = __shfl(full, b, 64);
        }
        b = __builtin_amdgcn_readfirstlane(b);
        t0 = __builtin_amdgcn_readfirstlane(g * a.rows);
        t1 = min(t0 + a.rows, __builtin_amdgcn_readfirstlane(__shfl(count, b, 64)));
        return true;
    }
    // (a CU gets workgroups that lie a fixed number apart: with the sequences shifted from one g to the next these are of
    // different sequences)
    const int g = i / a.B;
    b = (i - g * a.B + 5 * g) % a.B;
    t0 = g * a.rows;
    t1 = min(t0 + a.rows, clamp_count(a.count, b, a.K));
    return t0 < t1;
}

// 2048 VECTORS tokens of the vocabulary, for some rows of one sequence: a thread has eight of each 2048.
template <int VECTORS, Size SIZE, bool XBF16, bool OBF16, bool NOISE>
__global__ __launch_bounds__(kThreads) void logits_kernel(LogitsArgs a)
{
    constexpr int kTokens = 8 * kThreads * VECTORS;
    constexpr bool WIDE = SIZE == kWide, LONG = SIZE == kLong;
    using K = Known<SIZE, kTokens>;
    __shared__ alignas(16) K known;
    __shared__ unsigned long long best[kKvWindowMax], paths[kKvWindowMax], inside_s;
    __shared__ int draft[kKvWindowMax];

    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    int b, t0, t1;
    if (!rows_of(a, blockIdx.y, b, t0, t1)) return;
    const size_t row0 = (size_t)b * a.K;
    const int v0 = blockIdx.x * kTokens, nv = min(kTokens, a.V - v0);

    // What the counting needs is asked for first: reads come back in their order, and those of the logits take longer
    // (64 rows of 131072, fp32: 22.5 to 22.1 us).
    const bool marks = a.marks, texts = marks && a.params && a.history, drafts = marks && a.params && a.tokens;
    const int32_t* h = a.history + (size_t)b * a.capacity;
    // four tokens of the text from index i on, or its last four where there are fewer behind i
    auto four = [&](int i) { return *reinterpret_cast<const u32x4_any_t*>(h + min(i, a.capacity - 4)); };
    u32x4_any_t text = {0, 0, 0, 0};
    int drafted = -1, above = -1, id[kEach] = {}, len = 0, start = 0;
    float value[kEach] = {};
    bool longer = false;
    if (texts) {
        len = min(max(a.history_lens[b], 0), a.capacity);
        if (a.history_start) start = a.history_start[b];
        longer = LONG && len - max(min(start, len), 0) > kNarrowText;
    }
    if (texts && a.capacity >= 4) text = four(tid * 4);
    if (drafts && wave == kWaves - 1) {
        drafted = lane < a.K ? a.tokens[row0 + lane] : -1;
        above = node_above(a.parent ? a.parent + row0 : nullptr, a.K);
    }
    if constexpr (!WIDE)
#pragma unroll
        for (int r = 0; r < kEach; ++r)
            if (tid + r * kThreads < a.n_bias) {
                id[r] = a.bias_ids[(size_t)b * a.n_bias + tid + r * kThreads];
                value[r] = a.bias_values[(size_t)b * a.n_bias + tid + r * kThreads];
            }

    // the first two vectors of eight are on their way while the text is counted, later ones two ahead
    const int vectors = (nv + 8 * kThreads - 1) / (8 * kThreads);
    Row8<XBF16, NOISE> even, odd;
    Rows<XBF16, NOISE> ahead(a, row0 + t0);
    int ahead_t = t0, ahead_j = 0;
    auto load = [&](Row8<XBF16, NOISE>& r) {
        if (ahead_t < t1) ahead.load(r, v0 + (ahead_j * kThreads + tid) * 8);
        if (++ahead_j == vectors) {
            ahead_j = 0;
            ++ahead_t;
            ahead.next();
        }
    };
    load(even);
    load(odd);
    const Params p(a.params, b);

    unsigned long long inside = 0;
    uint32_t some = 0;   // a byte for each of the thread's vectors: the tokens of which something is known
    if (tid < kKvWindowMax) best[tid] = 0;
    unsigned long long biased_here[kEach];
    if (marks) {
        known.clear();
        if (a.n_bias > 0) known.ask_biases(a, v0, nv, id, biased_here);
    }
    __syncthreads();
    if (marks) {
        if (a.n_bias > 0) known.take_biases(a, b, v0, nv, id, value, biased_here);
        if (texts) {
            auto count = [&](int token, bool since) {
                const uint32_t u = (uint32_t)token - (uint32_t)v0;
                if (u < (uint32_t)nv) {
                    if (since) known.add(u, 1);
                    else known.mark(u, K::kSeen);
                }
            };
            if (a.capacity >= 4) {
                auto count4 = [&](const u32x4_any_t& text, int i) {
                    if (i >= start && i + 4 <= len) {   // (nearly all)
#pragma unroll
                        for (int e = 0; e < 4; ++e) count((int)text[e], true);
                    } else if (i < len) {
                        const int from = min(i, a.capacity - 4);   // (see four)
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (from + e >= i && from + e < len) count((int)text[e], from + e >= start);
                    }
                };
                count4(text, tid * 4);
                // (four reads at a time)
                u32x4_any_t more[4];
                auto ask = [&](int i0) {
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (i0 + r * kStep < len) more[r] = four(i0 + r * kStep + tid * 4);
                };
                for (int i0 = kStep; i0 < len; i0 += 4 * kStep) {
                    ask(i0);
#pragma unroll
                    for (int r = 0; r < 4; ++r)
                        if (i0 + r * kStep < len) count4(more[r], i0 + r * kStep + tid * 4);
                    if (LONG && longer && i0 % kPart == kPart - 3 * kStep) {
                        __syncthreads();
                        known.spill();
                        __syncthreads();
                    }
                }
            } else if (tid < len) {
                count(h[tid], tid >= start);
            }
        }
        if (wave == kWaves - 1) {   // the path to each node, and the drafted tokens of this slice
            const bool here = drafted >= v0 && drafted - v0 < nv;
            paths[lane] = drafts ? node_paths(above, a.K) : 0;
            draft[lane] = drafted - v0;
            if (here) known.draft(drafted - v0);
            const unsigned long long which = __ballot(here);
            if (lane == 0) inside_s = which;
        }
        __syncthreads();
        if (!WIDE && a.n_bias > 0) {
            known.count_biases();
            __syncthreads();
            known.place_biases();
            __syncthreads();
        }
        inside = inside_s;
#pragma unroll
        for (int i = 0; i < VECTORS; ++i) some |= known.which((i * kThreads + tid) * 8) << 8 * i;
    }

    const size_t out_step = a.out_stride * (OBF16 ? 2 : 4);
    char* out = static_cast<char*>(a.out) + (row0 + t0) * out_step;
    int t = t0, j = 0;
    float top = -__builtin_huge_valf();
    int token = 0x7fffffff;
    // the drafted tokens of this slice on the path to the node count for its row alone
    auto drafts_count = [&](int n) {
        const unsigned long long mine = paths[t] & inside;
        if (mine == 0) return;
        __syncthreads();
        if (tid < 64 && (mine >> tid & 1)) known.add_later(draft[tid], n);
        __syncthreads();
    };
    // one vector of eight: the j-th of row t
    auto take = [&](Row8<XBF16, NOISE>& r) {
        const int k = (j * kThreads + tid) * 8, m = min(nv - k, 8);
        const bool whole = m == 8 || a.V < 8;
        const uint32_t allow = a.mask ? r.allow : 0xffu;
        float f[8], z[8];
        r.x.floats(f);
        if constexpr (NOISE) r.z.floats(z);
        load(r);
        if (j == 0 && inside) drafts_count(1);
        if (m > 0) {
            if (!whole) {
                to_front(f, m);
                if constexpr (NOISE) to_front(z, m);
            }
            if (marks) {
                // one known token of each lane at a time: most have none, few have two
                for (uint32_t left = some >> 8 * j & 0xffu; left; left &= left - 1) {
                    const int e = __ffs(left) - 1;
                    bool biased;
                    float bias = 0.0f;
                    const uint32_t c = known.look(a, b, k + e, biased, bias);
                    uint32_t n = c & K::kCount;
                    if (LONG && longer && n) n += known.spilled(k + e);
                    float x = f[0];
#pragma unroll
                    for (int i = 1; i < 8; ++i) x = i == e ? f[i] : x;
                    if (c) x *= x > 0.0f ? p.less : p.rep;
                    if (n) x -= p.frequency * (float)n + p.presence;
                    if (biased) x += bias;
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = i == e ? x : f[i];
                }
            }
#pragma unroll
            for (int e = 0; e < 8; ++e) f[e] *= p.cool;
            if (a.mask) {
#pragma unroll
                for (int e = 0; e < 8; ++e) f[e] = only(f[e], allow, e);
            }
            if (a.out) {
                if (m == 8) {
                    store8<OBF16>(out, v0 + k, f);
                } else {
#pragma unroll
                    for (int e = 0; e < 7; ++e)
                        if (e < m) store1<OBF16>(out, v0 + k + e, f[e]);
                }
            }
            if (a.best) {
                if constexpr (NOISE) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] += z[e];
                }
                if (m < 8) {
#pragma unroll
                    for (int e = 0; e < 8; ++e) f[e] = only(f[e], 0xffu >> (8 - m), e);
                }
                float most = f[0];
#pragma unroll
                for (int e = 1; e < 8; ++e) most = fmaxf(most, f[e]);
                if (most > top) {
                    int e = 7;
#pragma unroll
                    for (int i = 6; i >= 0; --i) e = f[i] == most ? i : e;
                    top = most;
                    token = v0 + k + e;
                }
            }
        }
        if (++j < vectors) return;
        if (a.best) {
            const float most = wave_max(top);
            const int lowest = wave_min(top == most ? token : 0x7fffffff);
            if (lane == 0 && most > -__builtin_huge_valf()) atomicMax(&best[t - t0], key_of(most, lowest));
            top = -__builtin_huge_valf();
        }
        if (inside) drafts_count(-1);
        j = 0;
        ++t;
        out += out_step;
    };
    for (;;) {
        take(even);
        if (t == t1) break;
        take(odd);
        if (t == t1) break;
    }
    if (a.best) {
        __syncthreads();
        if (tid < t1 - t0) a.work[(row0 + t0 + tid) * a.slices + blockIdx.x] = best[tid];
    }
}

// the best of a row's slices: a wave a row
__global__ __launch_bounds__(kThreads) void logits_best_kernel(LogitsArgs a)
{
    const long long row = (long long)blockIdx.x * kWaves + (threadIdx.x >> 6);
    const int lane = threadIdx.x & 63;
    if (row >= (long long)a.B * a.K) return;
    unsigned long long key = 0;
    for (int i = lane; i < a.slices; i += 64) key = max(key, a.work[row * a.slices + i]);
    const uint32_t hi = (uint32_t)(key >> 32), most = wave_most(hi), low = wave_most(hi == most ? (uint32_t)key : 0);
    const int b = (int)(row / a.K), t = (int)(row - (long long)b * a.K);
    if (lane == 0 && t < clamp_count(a.count, b, a.K)) a.best[row] = token_of((unsigned long long)most << 32 | low);
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
    const int up = node_above(parent, a.K);
    const unsigned long long path = node_paths(up, a.K);
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

// Slices of 8192 tokens where they make enough workgroups, of 2048 otherwise (a token of each of 16 sequences over 131072,
// fp32: 9.0 us in large slices, 8.3 in small ones; of 24 10.4 and 10.7; windows of 8 over 32000, bf16, of 16
// sequences: 10.2 and 12.3).
int vectors_of(const LogitsArgs& a)
{
    return (long long)a.B * a.K * ((a.V + 8 * kThreads * 4 - 1) / (8 * kThreads * 4)) >= 384 ? 4 : 1;
}

template <int VECTORS, Size SIZE, bool XBF16, bool OBF16>
void launch(const LogitsArgs& a, dim3 grid, hipStream_t s)
{
    if (a.noise) logits_kernel<VECTORS, SIZE, XBF16, OBF16, true><<<grid, dim3(kThreads), 0, s>>>(a);
    else logits_kernel<VECTORS, SIZE, XBF16, OBF16, false><<<grid, dim3(kThreads), 0, s>>>(a);
}

template <int VECTORS, Size SIZE>
void launch(LogitsArgs& a, bool x_bf16, bool out_bf16, hipStream_t s)
{
    const int slice = 8 * kThreads * VECTORS;
    a.slices = (a.V + slice - 1) / slice;
    // Rows of a workgroup: each walks its sequence's text anew, so few workgroups take many rows: about 1024, and twice that
    // where windows may be short (32 ragged windows of 8 rows of 131072 with texts of 4000: 23.1 us, with half as many
    // workgroups 26.2, with twice as many 27.3; whole windows, 16 of 32 rows of 32000: 20.4 with 1024, 22.5 with 2048, 25.0
    // with 512).
    const long long units = (long long)a.B * a.slices;
    const int groups = (int)min((long long)a.K, max(1LL, (a.count ? 2048 : 1024) / units));
    a.rows = (a.K + groups - 1) / groups;
    const dim3 grid(a.slices, a.B * ((a.K + a.rows - 1) / a.rows));
    if (x_bf16) out_bf16 ? launch<VECTORS, SIZE, true, true>(a, grid, s) : launch<VECTORS, SIZE, true, false>(a, grid, s);
    else out_bf16 ? launch<VECTORS, SIZE, false, true>(a, grid, s) : launch<VECTORS, SIZE, false, false>(a, grid, s);
}

}  // namespace

// (as many as the smallest slices make: the workspace fits whichever are taken)
int logits_slices(int V) { return (V + 8 * kThreads - 1) / (8 * kThreads); }

hipError_t launch_logits(const LogitsArgs& args, bool x_bf16, bool out_bf16, hipStream_t s)
{
    LogitsArgs a = args;
    a.marks = a.n_bias > 0 || (a.params && (a.history || a.tokens));
    const int text = a.params && a.history ? a.capacity : 0;
    const bool many = vectors_of(a) == 4;
    // By the width of the texts' buffer: their lengths are on the device.  (Small slices have room for 32 bits, and no
    // parts to wait for: a row of 131072 with a text of 32000 13.2 us wide, 15.6 long; 8 rows, 100000 34.0 and 43.9; but 64
    // rows, 100000 in large slices 61 us long, 103 wide in small ones; 32 ragged windows of 8, texts of 4000 in rows of
    // 131072 23.5 and 30.7.)
    if (text > kLongText || a.n_bias > kNarrowBias || (text > kNarrowText && !many)) launch<1, kWide>(a, x_bf16, out_bf16, s);
    else if (text > kNarrowText) launch<4, kLong>(a, x_bf16, out_bf16, s);
    else many ? launch<4, kNarrow>(a, x_bf16, out_bf16, s) : launch<1, kNarrow>(a, x_bf16, out_bf16, s);
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
