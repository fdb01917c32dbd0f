// gdn_attn_impl.h -- the window attention over the paged cache (gdn_attn_verify),
// instantiated per type and head size in gdn_attn_{bf16,f32}_{64,128,256}.hip.
//
// Mathematics.  Over any set of keys a row keeps m (a reference for its
// exponents), l = sum e^{x-m} and the vector a = sum e^{x-m} v; sets are joined
// by scaling both to a common m.  So a row's keys can be cut anywhere: the
// pages that all sequences share are read once for the rows of all of them, and
// what is left is cut evenly over the chip.
//
// Work lists.  A unit is one tile of N keys against the M rows of one
// key/value head.  The shared list has an item for each (head, split of the prefix,
// row tile), whose row tiles run through the window tokens of every sequence that
// holds the prefix; the splits are as many as make the items fill the grid best.
// The own list has the units (sequence, head, key tile) in this order, and part i of
// n has the units [i U / n, (i+1) U / n), so the load is even whatever the lengths are;
// a part's row tiles go to neighbouring workgroups (with windows of unequal length
// the row tiles are units of the list instead).  No host knowledge of lengths is
// needed: each workgroup sums them over the sequences by itself.  The workgroups
// take the shared items in their order and the own parts from the last workgroup
// down, so that short lists meet as little as may be.  A run of units of
// one row tile is a piece; a piece leaves (m, l, a) in the workspace and a second
// kernel joins the pieces of each row, except where one piece is all there is.
// Consecutive workgroups sit on one XCD, so that row tiles that read the same keys
// at the same time share its L2: before the row tiles of a key range were
// neighbours, four of five reads of a shared prefix missed it.
//
// A tile.  K and V rows go from memory straight into LDS (16 bytes a lane), one
// tile ahead of the one being worked on.  S^T = K Q^T leaves a query row in the
// lanes with the same lane & 15, 4 keys a register group; e^{x-m} of that layout
// is already the operand of O^T = V^T P^T, and V^T comes out of LDS by the
// transposing 8-byte read.  The 16-byte chunks of a row are permuted by the key's
// low bits so that both kinds of read meet every bank once.
#pragma once

#include "gdn_device.h"
#include "gdn_kv_internal.h"

namespace gdn {
namespace attn {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short bf16x4_t;
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4;

constexpr int kThreads = 512, kWaves = kThreads / 64;
constexpr float kNoMax = -1e37f;   // the reference of a row that has seen no key: finite, so differences are
constexpr float kSlack = 8.0f;     // a reference is kept while no exponent passes it by more than 2^8
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// M rows by N keys over the 8 waves: RW groups of rows x KW groups of keys x DW parts of the output's columns;
// a wave has MW times 16 rows
template <bool BF16_, int D_, int RW_, int KW_, int DW_, int MW_>
struct Cfg {
    static constexpr bool BF16 = BF16_;
    static constexpr int D = D_, RW = RW_, KW = KW_, DW = DW_, MW = MW_;
    static_assert(RW * KW * DW == kWaves, "every wave has a part");
    static constexpr int M = 16 * MW * RW;
    static constexpr int ES = BF16 ? 2 : 4, ROW = D * ES, CH = ROW / 16;
    static constexpr int N = 8192 / D;             // keys a tile: K and V are 32 KB in bf16, 64 KB in fp32
    static constexpr int KF = N / KW / 16;         // 16-key groups of a wave
    static constexpr int DB = D / 16 / DW;         // 16-column groups of a wave's output
    static constexpr int MAT = N * ROW, STAGE = 2 * MAT;
    static constexpr int QC = BF16 ? D / 32 : D / 16;  // registers groups of a row's q
};

// where each 16-byte chunk of a key's row sits: chunk ^ swizzle(key)
template <class C>
__device__ __forceinline__ constexpr int k_swizzle(int key) { return C::CH >= 16 ? (key & 15) : ((key >> 1) & 7); }
template <class C>
__device__ __forceinline__ constexpr int v_swizzle(int key)
{
    if constexpr (!C::BF16) return ((key >> 2) & 3) << 2;
    else return C::CH >= 16 ? (key & 7) << 1 : ((key >> 1) & 3) << 1;
}

// what a sequence asks for
struct Seq {
    int cnt, len, end, start, tiles, rts;
    bool part;
    int units;
};

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b, int N, int M)
{
    Seq s;
    const int cap = a.P << a.page_log2;
    s.cnt = a.count ? min(max(a.count[b], 0), a.K) : a.K;
    s.len = min(max(a.lens[b], 0), cap);
    s.end = (int)min((long long)s.len + s.cnt, (long long)cap);
    s.part = a.prefix > 0 && s.len >= a.prefix && s.cnt > 0;
    s.start = s.part ? a.prefix : 0;
    s.tiles = s.cnt > 0 ? (s.end - s.start + N - 1) / N : 0;
    s.rts = (s.cnt * (a.Hq / a.Hkv) + M - 1) / M;
    s.units = a.Hkv * s.tiles * (a.count ? s.rts : 1);
    return s;
}

// the lists' lengths and cuts, for the joining kernel
struct Head {
    int row_tiles, splits;       // of the shared list
    int own_units, own_parts;
};
struct PlanSeq {
    int own_base;   // own units of the sequences before
    int tok_base;   // window tokens of the prefix-holding sequences before (-1: not one of them)
};

// workspace: Head | PlanSeq[B] | (m, l) of shared rows | of own rows | a of shared rows | of own rows
struct Layout {
    size_t plan, ml_s, ml_o, o_s, o_o, bytes;
};
__host__ __device__ inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
__host__ __device__ inline Layout layout(const AttnArgs& a, int nb, int MS, int MO)
{
    const size_t G = a.Hq / a.Hkv;
    const size_t segs = MS ? a.Hkv * (((size_t)a.B * a.K * G + MS - 1) / MS) : 0;
    const size_t slots_s = MS ? (segs > 2 * (size_t)nb ? segs : 2 * (size_t)nb) : 0;
    const size_t slots_o = nb + (size_t)a.B * a.Hkv * ((a.K * G + MO - 1) / MO);
    Layout w;
    w.plan = up256(sizeof(Head));
    w.ml_s = up256(w.plan + a.B * sizeof(PlanSeq));
    w.ml_o = up256(w.ml_s + slots_s * MS * 8);
    w.o_s = up256(w.ml_o + slots_o * MO * 8);
    w.o_o = w.o_s + slots_s * MS * a.D * 4;
    w.bytes = w.o_o + slots_o * MO * a.D * 4;
    return w;
}

// Part i of n parts of U units has the units floor(U i / n) .. floor(U (i+1) / n) - 1, so unit u is in part
// floor(((u + 1) n - 1) / U).  Both quotients by doubles (an integer division of 64 bits takes ten times as
// long): their numerators are below 2^40 and exact, and half a unit added keeps the rounding of the quotient
// (below 2^31 parts in 2^53) on the right side of every integer.
__device__ __forceinline__ int first_unit(int units, int n, int i)
{
    return (int)(((double)units * i + 0.5) / n);
}
__device__ __forceinline__ int part_of(int units, int n, int u)
{
    return (int)(((double)(u + 1) * n - 0.5) / units);
}
// Into how many splits the prefix goes: for s of them, `segs` heads and row tiles take ceil(segs s / nb) rounds of
// ceil(tiles / s) tiles and about kStartup tiles' time for a piece's first reads and its end.  A lane tries each s;
// there are at most max(segs, 2 nb) items.
constexpr int kStartup = 6;
__device__ __forceinline__ int splits_for(int segs, int tiles, int nb)
{
    const int n = (threadIdx.x & 63) + 1;
    int cost = (segs * n + nb - 1) / nb * ((tiles + n - 1) / n + kStartup);
    if (n > 1 && (n > tiles || segs * n > 2 * nb)) cost = 0x7fffffff;
    int best = n;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int c = __shfl_xor(cost, d, 64), m = __shfl_xor(best, d, 64);
        const bool less = c < cost || (c == cost && m < best);
        cost = less ? c : cost;
        best = less ? m : best;
    }
    return __builtin_amdgcn_readfirstlane(best);
}

// how the own list counts row tiles: with equal windows a unit stands for all RT of them, taken by RT
// neighbouring workgroups; otherwise each is a unit of its own
struct RowTiles {
    int in_list, grouped;
};
__host__ __device__ inline RowTiles row_tiles_of(const AttnArgs& a, int M)
{
    const int rt = (a.K * (a.Hq / a.Hkv) + M - 1) / M;
    return a.count ? RowTiles{rt, 1} : RowTiles{1, rt};
}
// (a list is cut in no more parts than it has units, so that none is empty)
__device__ __forceinline__ int parts_for(int nb, int grouped, int units) { return min(max(nb / grouped, 1), units); }

// ---------------------------------------------------------------- pieces of a tile
// COUNT KB of global memory to LDS: in the i-th, lane l's 16 bytes at base + 1024 i + voff[i] go to
// lds + 1024 i + 16 l (the instruction's offset counts on both sides).  Written as assembly because the
// compiler would otherwise wait for the tile on its way before it reads the tile that is there; nothing
// is returned in registers, and load_wait() below waits for all of them.  (m0 takes the LDS address; one
// wait state between writing it and the load.)
template <int COUNT>
__device__ __forceinline__ void load_lds(uint32_t lds, const uint32_t* voff, const char* base)
{
    static_assert(COUNT == 2 || COUNT == 4, "2 or 4 KB");
    if constexpr (COUNT == 2)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\t"
                     "global_load_lds_dwordx4 %1, %3\n\t"
                     "global_load_lds_dwordx4 %2, %3 offset:1024"
                     :
                     : "s"(lds), "v"(voff[0]), "v"(voff[1]), "s"(base)
                     : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\t"
                     "global_load_lds_dwordx4 %1, %5\n\t"
                     "global_load_lds_dwordx4 %2, %5 offset:1024\n\t"
                     "global_load_lds_dwordx4 %3, %5 offset:2048\n\t"
                     "global_load_lds_dwordx4 %4, %5 offset:3072"
                     :
                     : "s"(lds), "v"(voff[0]), "v"(voff[1]), "v"(voff[2]), "v"(voff[3]), "s"(base)
                     : "memory", "m0");
}

__device__ __forceinline__ void load_wait()
{
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
}

__device__ __forceinline__ void block_barrier()
{
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

__device__ __forceinline__ uint4 lds_read16(uint32_t at)
{
    typedef __attribute__((address_space(3))) const f32x4_t lds_f4;
    return __builtin_bit_cast(uint4, *(lds_f4*)(lds_char*)(uintptr_t)at);
}

__device__ __forceinline__ float lds_read4(uint32_t at)
{
    typedef __attribute__((address_space(3))) const float lds_f1;
    return *(lds_f1*)(lds_char*)(uintptr_t)at;
}

__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }

__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// two floats to bf16 (to nearest), packed
__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    const bf16x2_t h = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, h);
}

// nodes on the path from a root to each node: lane i returns those of node i (called by a whole wave, K <= 64)
__device__ __forceinline__ unsigned long long ancestors(const int32_t* parent, int K)
{
    const int lane = threadIdx.x & 63;
    int up = -1;
    if (lane < K) {
        const int p = parent ? parent[lane] : lane - 1;
        up = p >= 0 && p < lane ? p : -1;
    }
    unsigned long long path = 1ull << lane;
#pragma unroll
    for (int d = 1; d < kKvWindowMax; d <<= 1) {
        const int from = max(up, 0);
        const unsigned long long more = __shfl(path, from, 64);
        const int far = __shfl(up, from, 64);
        if (up >= 0) {
            path |= more;
            up = far;
        }
    }
    return path;
}

// LDS beside the tiles
struct Small {
    int part[kWaves];
    int found_b, found_off;
    int tok_base[kThreads];   // window tokens of the prefix-holding sequences before a thread's own
    int bad_value;
    unsigned long long path[64];
    int tok[132];             // window tokens (b * K + t) of a shared row tile
    float2 ml[kWaves][32];    // (m, l) of the waves' rows, to be joined
};

struct PieceIn {
    const int32_t* row;       // table row
    const int32_t* parent;    // of the sequence, or nullptr
    int h, p0, tiles;         // key/value head, first position, tiles
    int len, end;             // window's first position and the end of what is there
    bool window;              // keys at len.. are seen by their descendants only
};

struct PieceOut {
    bool direct;              // the whole row: o and lse at once
    float* o;                 // [M][D]
    float2* ml;               // [M]
};

// a row of the tile: token b * K + t, t, and the query head of its group; false for a row that is not there
struct RowId {
    int tok, t, g;
    bool live;
};

template <class C, class RowFn>
__device__ __forceinline__ void run_piece(const AttnArgs& a, char* sm, Small& s, const PieceIn& in,
                                          const PieceOut& out, RowFn row_of)
{
    constexpr int MW = C::MW, KF = C::KF, DB = C::DB, QC = C::QC, N = C::N;
    const int lane = threadIdx.x & 63, w = uni(threadIdx.x >> 6);
    const int rw = w % C::RW, kw = (w / C::RW) % C::KW, dw = w / (C::RW * C::KW);
    const int n16 = lane & 15, grp = lane >> 4;
    const int page_mask = (1 << a.page_log2) - 1;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)sm;
    const int G = a.Hq / a.Hkv;

    // ---- the pages: lane i holds slot first + i (a missing one as page 0, flagged), and the 64 slots after
    auto slot_id = [&](int sl, bool& bad) {
        int id = sl < a.P ? in.row[sl] : -1;
        bad = (unsigned)id >= (unsigned)a.n_pages;
        return bad ? 0 : id;
    };
    int first = in.p0 >> a.page_log2;
    bool bad_lane, bad_lane2;
    int ids = slot_id(first + lane, bad_lane), ids2 = slot_id(first + 64 + lane, bad_lane2);
    unsigned long long bad = __ballot(bad_lane), bad2 = __ballot(bad_lane2);

    // ---- tile loads: wave w brings the keys w N/8 .. of K and V, in groups of up to 16 keys (of one page, as a
    // page has 16 at least), a group in runs of CNT KB
    constexpr int WK = N / kWaves, GK = WK < 16 ? WK : 16, KPI = 1024 / C::ROW, NI = GK / KPI, CNT = NI < 4 ? NI : 4;
    const uint32_t page_bytes = ((uint32_t)a.Hkv << a.page_log2) * C::ROW;
    const uint32_t head_off = ((uint32_t)in.h << a.page_log2) * C::ROW;
    const int lkey = lane / C::CH, lch = lane % C::CH;
    // (the i-th KB of a group is i KPI keys on: bits of the key that no other part of it has, so they flip in)
    const int key0 = w * WK + lkey;
    const uint32_t k_off = lkey * C::ROW + ((lch ^ k_swizzle<C>(key0 & 15)) << 4);
    const uint32_t v_off = lkey * C::ROW + ((lch ^ v_swizzle<C>(key0 & 15)) << 4);
    auto issue = [&](int j, int buf) {
        const int pt = in.p0 + j * N;
        int s0 = (pt >> a.page_log2) - first;
        if (s0 >= 64) {
            ids = ids2;
            bad = bad2;
            first += 64;
            s0 -= 64;
            ids2 = slot_id(first + 64 + lane, bad_lane2);
            bad2 = __ballot(bad_lane2);
        }
#pragma unroll
        for (int g = 0; g < WK / GK; ++g) {
            const int key = w * WK + g * GK;
            const uint32_t id = __builtin_amdgcn_readlane(ids, s0 + (key >> a.page_log2));
            const uint64_t off = (uint64_t)id * page_bytes + (head_off + ((pt + key) & page_mask) * C::ROW);
            const uint32_t to = lds0 + buf * C::STAGE + key * C::ROW;
#pragma unroll
            for (int i = 0; i < NI; i += CNT) {
                uint32_t ko[CNT], vo[CNT];
#pragma unroll
                for (int e = 0; e < CNT; ++e) {
                    ko[e] = k_off ^ (k_swizzle<C>((i + e) * KPI) << 4);
                    vo[e] = v_off ^ (v_swizzle<C>((i + e) * KPI) << 4);
                }
                load_lds<CNT>(to + i * 1024, ko, static_cast<const char*>(a.k_pages) + off + i * 1024);
                load_lds<CNT>(to + C::MAT + i * 1024, vo, static_cast<const char*>(a.v_pages) + off + i * 1024);
            }
        }
        const int slots = max(N >> a.page_log2, 1);
        return (unsigned)(bad >> s0) & ((1u << slots) - 1);   // missing pages of the tile
    };
    if (threadIdx.x == 0) s.bad_value = 0;   // (before the first barrier of the loop)
    unsigned miss_next = issue(0, 0);

    // ---- the rows
    // Row r of this lane, formed anew wherever it is asked for: kept, it would take registers through the loop.
    auto row_id = [&](int r) {
        int row = (rw * MW + r) * 16 + (threadIdx.x & 15);
        asm volatile("" : "+v"(row));
        return row_of(row);
    };
    // the window's nodes on the path to each node, for the tiles that need them
    if (in.window && w == 0) s.path[lane] = ancestors(in.parent, a.K);
    float m[MW], l[MW];
    uint4 q[MW][QC];
    const float c = fabsf(a.scale) * kLog2e;
    bool any = false;
    {
        const uint32_t flip = a.scale < 0.f ? (C::BF16 ? 0x80008000u : 0x80000000u) : 0u;  // the sign goes into q
#pragma unroll
        for (int r = 0; r < MW; ++r) {
            const RowId id = row_id(r);
            any |= id.live;
            m[r] = kNoMax;
            l[r] = 0.f;
            const char* qp = static_cast<const char*>(a.q) +
                             ((size_t)id.tok * a.q_stride + (size_t)(in.h * G + id.g) * C::D) * C::ES + grp * 16;
#pragma unroll
            for (int e = 0; e < QC; ++e) {
                uint4 u = make_uint4(0, 0, 0, 0);
                if (id.live) u = *reinterpret_cast<const uint4*>(qp + e * 64);
                q[r][e] = make_uint4(u.x ^ flip, u.y ^ flip, u.z ^ flip, u.w ^ flip);
            }
        }
    }
    const bool alive = __any(any);   // a wave without rows only loads
    f32x4_t o[DB][MW];
#pragma unroll
    for (int d = 0; d < DB; ++d)
#pragma unroll
        for (int r = 0; r < MW; ++r) o[d][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    // LDS addresses of this lane within a tile: chunk c of a row sits at its lane's chunk with the low bits of c
    // flipped in, and further chunks, keys and 16-key groups lie at constant distances
    const int kbase = kw * (N / C::KW);
    const int vkey = C::BF16 ? 4 * grp + (n16 >> 2) : 4 * grp;   // (fp32 adds the register's index)
    const uint32_t k_lane = lds0 + (kbase + n16) * C::ROW + ((grp ^ k_swizzle<C>(n16)) << 4);
    const uint32_t v_lane =
        lds0 + C::MAT + (kbase + vkey) * C::ROW + (dw * DB * 16 * C::ES & ~255) +
        (C::BF16 ? ((((n16 >> 1) & 1) ^ v_swizzle<C>(vkey) ^ (2 * dw * DB & 15)) << 4) + (n16 & 1) * 8
                 : (((n16 >> 2) ^ v_swizzle<C>(vkey)) << 4) + (n16 & 3) * 4);
    static_assert(C::DW == 1 || DB * 16 * C::ES >= 128, "a part starts on a half or whole swizzle group");

    for (int j = 0; j < in.tiles; ++j) {
        const unsigned miss = miss_next;
        load_wait();
        block_barrier();   // every wave's part of this tile is there, and nobody reads the other buffer any more
        if (j + 1 < in.tiles) miss_next = issue(j + 1, (j + 1) & 1);
        char* kt = sm + (j & 1) * C::STAGE;
        char* vt = kt + C::MAT;
        const int pt = in.p0 + j * N;
        const bool masked = miss != 0 || (in.window && pt + N > in.len) || pt + N > in.end;

        // Values nobody may see are cleared where they lie (0 times NaN is NaN), and so are the window's that are
        // not finite: only some rows see them, and get them at the end.
        if (masked) {
            for (int e = threadIdx.x; e < N * C::CH; e += kThreads) {
                const int key = e / C::CH, pos = pt + key;
                uint32_t* v = reinterpret_cast<uint32_t*>(vt + e * 16);
                if (pos >= in.end || (miss >> (key >> a.page_log2) & 1)) {
                    *reinterpret_cast<uint4*>(v) = make_uint4(0, 0, 0, 0);
                } else if (in.window && pos >= in.len) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t u = v[i];
                        uint32_t keep = u;
                        if ((u & 0x7f800000u) == 0x7f800000u) keep &= C::BF16 ? 0xffffu : 0u;
                        if (C::BF16 && (u & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
                        if (keep != u) {
                            v[i] = keep;
                            s.bad_value = 1;
                        }
                    }
                }
            }
            block_barrier();
        }
        if (!alive) continue;

        // opaque, so that the addresses are formed from them in the loop and not kept in dozens of registers
        uint32_t k_at = k_lane + (j & 1) * C::STAGE, v_at = v_lane + (j & 1) * C::STAGE;
        asm volatile("" : "+v"(k_at), "+v"(v_at));

        // ---- S^T = K Q^T
        f32x4_t x[KF][MW];
#pragma unroll
        for (int k = 0; k < KF; ++k)
#pragma unroll
            for (int r = 0; r < MW; ++r) x[k][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int e = 0; e < QC; ++e)
#pragma unroll
            for (int k = 0; k < KF; ++k) {
                const uint4 u = lds_read16((k_at ^ (uint32_t)(((4 * e) & (C::CH - 1) & 15) << 4)) +
                                           (4 * e / 16) * 256 + 16 * k * C::ROW);
#pragma unroll
                for (int r = 0; r < MW; ++r) {
                    if constexpr (C::BF16) {
                        x[k][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, u),
                                                                          __builtin_bit_cast(bf16x8_t, q[r][e]),
                                                                          x[k][r], 0, 0, 0);
                    } else {
                        const uint32_t ua[4] = {u.x, u.y, u.z, u.w};
                        const uint32_t qa[4] = {q[r][e].x, q[r][e].y, q[r][e].z, q[r][e].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            x[k][r] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(ua[i]),
                                                                           __uint_as_float(qa[i]), x[k][r], 0, 0, 0);
                    }
                }
            }

        // ---- weights e^{x-m}
        unsigned seen[MW];   // of a masked tile: a bit for each of this lane's keys
        if (masked) {
#pragma unroll
            for (int r = 0; r < MW; ++r) {
                seen[r] = 0;
                const unsigned long long sees = in.window ? s.path[row_id(r).t & 63] : 0;
#pragma unroll
                for (int k = 0; k < KF; ++k) {
                    const int key = kbase + 16 * k + 4 * grp;
                    // the 4 keys from position pt + key on: committed ones (below len), then the window's by their
                    // bits in `sees`, none from end on and none of a missing page; by shifts and selects only
                    const int rel = pt + key - in.len, left = in.end - (pt + key);
                    const unsigned win = rel > 63 ? 0u : (unsigned)(sees >> (max(rel, 0) & 63));
                    const int old = min(max(-rel, 0), 4);
                    unsigned bits = (win << old | ((1u << old) - 1)) & ((1u << min(max(left, 0), 4)) - 1);
                    bits = (miss >> (key >> a.page_log2) & 1) ? 0u : bits;
                    seen[r] |= bits << (4 * k);
#pragma unroll
                    for (int i = 0; i < 4; ++i) x[k][r][i] = (bits >> i & 1) ? x[k][r][i] : -INFINITY;
                }
            }
        }
#pragma unroll
        for (int r = 0; r < MW; ++r) {
            float t = x[0][r][0];
#pragma unroll
            for (int k = 0; k < KF; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) t = fmaxf(t, x[k][r][i]);
            if (__any(t * c > m[r] + kSlack)) {
                t = fmaxf(t, __shfl_xor(t, 16, 64));
                t = fmaxf(t, __shfl_xor(t, 32, 64));
                // a row moves its reference by its own keys alone, so its bits depend on no other row
                const float mn = t * c > m[r] + kSlack ? t * c : m[r], f = exp2_(m[r] - mn);
                m[r] = mn;
                l[r] *= f;
#pragma unroll
                for (int d = 0; d < DB; ++d) o[d][r] *= f;
            }
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < KF; ++k)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float p = exp2_(__builtin_fmaf(x[k][r][i], c, -m[r]));
                    if (masked) p = (seen[r] >> (4 * k + i) & 1) ? p : 0.f;
                    x[k][r][i] = p;
                    sum += p;
                }
            l[r] += sum;
        }

        // ---- O^T += V^T P^T
        if constexpr (C::BF16) {
            // the weights enter the product in bf16, as v is: half a step of 2^-8 each, unbiased
            auto v_frag = [&](int k, int d) {
                lds_char* at = (lds_char*)(uintptr_t)((v_at ^ (uint32_t)((d & (C::CH / 2 - 1) & 7) << 5)) +
                                                      (d / 8) * 256 + 16 * k * C::ROW);
                return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)at));
            };
            if constexpr (KF == 1) {
                uint2 p[MW];
#pragma unroll
                for (int r = 0; r < MW; ++r)
                    p[r] = make_uint2(pack2(x[0][r][0], x[0][r][1]), pack2(x[0][r][2], x[0][r][3]));
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const bf16x4_t v = __builtin_bit_cast(bf16x4_t, v_frag(0, d));
#pragma unroll
                    for (int r = 0; r < MW; ++r)
                        o[d][r] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(v, __builtin_bit_cast(bf16x4_t, p[r]),
                                                                            o[d][r], 0, 0, 0);
                }
            } else {
#pragma unroll
                for (int k = 0; k < KF; k += 2) {
                    uint4 p[MW];
#pragma unroll
                    for (int r = 0; r < MW; ++r)
                        p[r] = make_uint4(pack2(x[k][r][0], x[k][r][1]), pack2(x[k][r][2], x[k][r][3]),
                                          pack2(x[k + 1][r][0], x[k + 1][r][1]), pack2(x[k + 1][r][2], x[k + 1][r][3]));
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const uint2 v0 = v_frag(k, d), v1 = v_frag(k + 1, d);
                        const bf16x8_t v = __builtin_bit_cast(bf16x8_t, make_uint4(v0.x, v0.y, v1.x, v1.y));
#pragma unroll
                        for (int r = 0; r < MW; ++r)
                            o[d][r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, __builtin_bit_cast(bf16x8_t, p[r]),
                                                                              o[d][r], 0, 0, 0);
                    }
                }
            }
        } else {
#pragma unroll
            for (int k = 0; k < KF; ++k)
#pragma unroll
                for (int d = 0; d < DB; ++d)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float v = lds_read4((v_at ^ (uint32_t)((d & 3) << 6)) + (d / 4) * 256 +
                                                  (16 * k + i) * C::ROW);
#pragma unroll
                        for (int r = 0; r < MW; ++r)
                            o[d][r] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, x[k][r][i], o[d][r], 0, 0, 0);
                    }
        }
    }

    // ---- the four lane groups' sums, then the waves of other keys, in a fixed order
#pragma unroll
    for (int r = 0; r < MW; ++r) {
        l[r] += __shfl_xor(l[r], 16, 64);
        l[r] += __shfl_xor(l[r], 32, 64);
    }
    const bool bad_value = uni(s.bad_value) != 0;
    if (bad_value && alive) {
        unsigned long long sees[MW];
#pragma unroll
        for (int r = 0; r < MW; ++r) sees[r] = s.path[row_id(r).t & 63];
        // a window value that is not finite makes what it makes of the rows that see it
        for (int pos = max(in.p0, in.len); pos < min(in.end, in.p0 + in.tiles * N); ++pos) {
            if (((pos - in.p0) % N) / (N / C::KW) != kw) continue;   // this wave's keys
            bool missing;
            const int page = slot_id(pos >> a.page_log2, missing);
            if (missing) continue;
            const size_t at = ((((size_t)page * a.Hkv + in.h) << a.page_log2) + (pos & page_mask)) * C::D;
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const float4 y = load4<C::BF16>(a.v_pages, at + (dw * DB + d) * 16 + 4 * grp);
                const float ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                for (int r = 0; r < MW; ++r)
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        if ((sees[r] >> (pos - in.len) & 1) && !(fabsf(ya[i]) < INFINITY)) o[d][r][i] += ya[i];
            }
        }
    }
    block_barrier();   // the tiles, and what this piece kept beside them, are done with
    if constexpr (C::KW > 1) {
        constexpr int F = DB * MW;
        float* box = reinterpret_cast<float*>(sm);
        auto at = [&](int k, int f) {
            return reinterpret_cast<f32x4_t*>(box + ((((k - 1) * C::DW + dw) * C::RW + rw) * F + f) * 256 + lane * 4);
        };
        if (kw > 0) {
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int r = 0; r < MW; ++r) *at(kw, d * MW + r) = o[d][r];
            if (grp == 0)
#pragma unroll
                for (int r = 0; r < MW; ++r) s.ml[w][r * 16 + n16] = make_float2(m[r], l[r]);
        }
        block_barrier();
        if (kw == 0) {
#pragma nounroll
            for (int k = 1; k < C::KW; ++k) {
#pragma unroll
                for (int r = 0; r < MW; ++r) {
                    const float2 v = s.ml[w + k * C::RW][r * 16 + n16];
                    const float mn = fmaxf(m[r], v.x), f = exp2_(m[r] - mn), g = exp2_(v.x - mn);
                    m[r] = mn;
                    l[r] = l[r] * f + v.y * g;
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[d][r] = o[d][r] * f + *at(k, d * MW + r) * g;
                }
            }
        }
        block_barrier();   // the next piece's tiles may come
        if (kw > 0) return;
    }
#pragma unroll
    for (int r = 0; r < MW; ++r) {
        const RowId id = row_id(r);
        if (!id.live) continue;
        const int row = (rw * MW + r) * 16 + n16;
        if (out.direct) {
            const size_t at = (size_t)id.tok * a.Hq + in.h * G + id.g;
            const float inv = l[r] == 0.f ? 0.f : 1.f / l[r];
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const f32x4_t y = o[d][r] * inv;
                const size_t e = at * C::D + (dw * DB + d) * 16 + 4 * grp;
                if constexpr (C::BF16) {
                    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.o) + e) =
                        make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
                } else {
                    *reinterpret_cast<f32x4_t*>(static_cast<float*>(a.o) + e) = y;
                }
            }
            if (a.lse && dw == 0 && grp == 0) a.lse[at] = l[r] == 0.f ? -INFINITY : (m[r] + __log2f(l[r])) * kLn2;
        } else {
#pragma unroll
            for (int d = 0; d < DB; ++d)
                *reinterpret_cast<f32x4_t*>(out.o + (size_t)row * C::D + (dw * DB + d) * 16 + 4 * grp) = o[d][r];
            if (dw == 0 && grp == 0) out.ml[row] = make_float2(m[r], l[r]);
        }
    }
}

// exclusive sum over the workgroup's threads, and the total
__device__ __forceinline__ int scan_int(int v, Small& s, int& total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int inc = v;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(inc, d, 64);
        if (lane >= d) inc += u;
    }
    __syncthreads();
    if (lane == 63) s.part[w] = inc;
    __syncthreads();
    int base = 0;
    total = 0;
    for (int i = 0; i < kWaves; ++i) {
        base += i < w ? s.part[i] : 0;
        total += s.part[i];
    }
    return base + inc - v;
}

// SH: the shared list's configuration, or void
template <class OW, class SH>
__global__ __launch_bounds__(kThreads, OW::BF16 ? 4 : 2) void attn_kernel(AttnArgs a, int nb)
{
    // all of LDS is asked for at the launch and starts at 0: the swizzled addresses flip bits below 256
    extern __shared__ __attribute__((aligned(1024))) char sm[];
    Small& s = *reinterpret_cast<Small*>(sm + 2 * OW::STAGE);
    constexpr bool kShared = !__is_same(SH, void);
    const int G = a.Hq / a.Hkv;
    int MS = 0;
    if constexpr (kShared) MS = SH::M;
    const Layout wk = layout(a, nb, MS, OW::M);
    char* work = static_cast<char*>(a.work);

    // ---- the lists' lengths: thread i sums the sequences [b0, b1)
    const int per = (a.B + kThreads - 1) / kThreads;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    int mine = 0, toks = 0;
    for (int b = b0; b < b1; ++b) {
        const Seq q = seq_of(a, b, OW::N, OW::M);
        mine += q.units;
        if (q.part) toks += q.cnt;
    }
    int own;
    const int own_base = scan_int(mine, s, own);
    own = uni(own);
    int tok_total = 0, tok_base = 0;
    int items = 0, row_tiles = 0, key_tiles = 0, splits = 0;
    if constexpr (kShared) {
        tok_base = scan_int(toks, s, tok_total);
        s.tok_base[threadIdx.x] = tok_base;
        tok_total = uni(tok_total);
        row_tiles = (tok_total * G + SH::M - 1) / SH::M;
        key_tiles = (a.prefix + SH::N - 1) / SH::N;
        splits = splits_for(a.Hkv * row_tiles, key_tiles, nb);
        items = a.Hkv * row_tiles * splits;
    }
    const RowTiles rts_of = row_tiles_of(a, OW::M);
    const int own_parts = parts_for(nb, rts_of.grouped, own);
    const int blocks = min(nb, items + own_parts * rts_of.grouped);
    // consecutive workgroups of the lists on one XCD (workgroups are dealt to the 8 XCDs in turn)
    const int per_xcd = (blocks + 7) / 8;
    const int lb = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *reinterpret_cast<Head*>(work) = Head{row_tiles, splits, own, own_parts};
        PlanSeq* plan = reinterpret_cast<PlanSeq*>(work + wk.plan);
        int base = own_base, tok = tok_base;
        for (int b = b0; b < b1; ++b) {
            const Seq q = seq_of(a, b, OW::N, OW::M);
            plan[b] = PlanSeq{base, q.part ? tok : -1};
            base += q.units;
            tok += q.part ? q.cnt : 0;
        }
    }
    if ((int)(blockIdx.x >> 3) >= per_xcd || lb >= blocks) return;

    // the own part: its units [own_u, own_u1), the first in sequence own_b, own_off units into it
    const int own_block = blocks - 1 - lb;
    const bool has_own = own_block < own_parts * rts_of.grouped;
    const int part = own_block / rts_of.grouped, rt_block = own_block - part * rts_of.grouped;
    const int own_u = has_own ? first_unit(own, own_parts, part) : 0;
    const int own_u1 = has_own ? first_unit(own, own_parts, part + 1) : 0;
    if (own_base <= own_u && own_u < own_base + mine) {
        int base = own_base;
        for (int b = b0; b < b1; ++b) {
            const Seq q = seq_of(a, b, OW::N, OW::M);
            if (own_u < base + q.units) {
                s.found_b = b;
                s.found_off = own_u - base;
                break;
            }
            base += q.units;
        }
    }
    __syncthreads();
    const int own_b = uni(s.found_b), own_off = uni(s.found_off);

    if constexpr (kShared) {
        for (int it = lb; it < items; it += blocks) {
            const int hs = it / row_tiles, rt = it - hs * row_tiles, h = hs / splits, sp = hs - h * splits;
            const int k0 = (int)((unsigned)key_tiles * sp / splits), k1 = (int)((unsigned)key_tiles * (sp + 1) / splits);
            // the tile's tokens
            const int r0 = rt * SH::M, t0 = r0 / G;
            const int t1 = min((r0 + SH::M - 1) / G + 1, tok_total);
            __syncthreads();
            int tok = s.tok_base[threadIdx.x];
            const int f0 = min((int)threadIdx.x * per, a.B), f1 = min(f0 + per, a.B);
            for (int b = f0; b < f1 && tok < t1; ++b) {
                const Seq q = seq_of(a, b, OW::N, OW::M);
                if (!q.part) continue;
                for (int t = max(0, t0 - tok); t < q.cnt && tok + t < t1; ++t) s.tok[tok + t - t0] = b * a.K + t;
                tok += q.cnt;
            }
            __syncthreads();
            const int lead = uni(s.tok[0] / a.K);
            PieceIn in{a.table + (size_t)lead * a.P, nullptr, h, k0 * SH::N, k1 - k0, a.prefix, a.prefix, false};
            const size_t slot = it;
            PieceOut out{false, reinterpret_cast<float*>(work + wk.o_s) + slot * SH::M * SH::D,
                         reinterpret_cast<float2*>(work + wk.ml_s) + slot * SH::M};
            run_piece<SH>(a, sm, s, in, out, [&](int r) {
                RowId id{0, 0, 0, false};
                const int t = (r0 + r) / G;
                id.live = t < t1;
                if (id.live) {
                    id.tok = s.tok[t - t0];
                    id.t = id.tok % a.K;
                    id.g = (r0 + r) - t * G;
                }
                return id;
            });
        }
    }

    int b = own_b, off = own_off, u = own_u;
    while (u < own_u1) {
        const Seq q = seq_of(a, b, OW::N, OW::M);
        const int tiles = uni(q.tiles), rts = a.count ? uni(q.rts) : 1;
        if (off >= a.Hkv * rts * tiles) {
            off = 0;
            ++b;
            continue;
        }
        const int seg = off / tiles, k0 = off - seg * tiles;
        const int nt = min(tiles - k0, own_u1 - u);
        const int h = seg / rts, rt_list = seg - h * rts, rt = rt_list + rt_block;
        const size_t slot = ((size_t)part + ((size_t)b * a.Hkv + h) * rts_of.in_list + rt_list) * rts_of.grouped + rt_block;
        PieceIn in{a.table + (size_t)b * a.P, a.parent ? a.parent + (size_t)b * a.K : nullptr, h,
                   uni(q.start) + k0 * OW::N, nt, uni(q.len), uni(q.end), true};
        PieceOut out{uni(q.part) == 0 && nt == tiles, reinterpret_cast<float*>(work + wk.o_o) + slot * OW::M * OW::D,
                     reinterpret_cast<float2*>(work + wk.ml_o) + slot * OW::M};
        const int r0 = rt * OW::M, cnt = uni(q.cnt);
        run_piece<OW>(a, sm, s, in, out, [&](int r) {
            RowId id{0, 0, 0, false};
            const int t = (r0 + r) / G;
            id.live = t < cnt;
            if (id.live) {
                id.tok = b * a.K + t;
                id.t = t;
                id.g = (r0 + r) - t * G;
            }
            return id;
        });
        u += nt;
        off += nt;
    }
}

// ---------------------------------------------------------------- joining
// A thread has 4 columns of a row; SPLIT threads share them, each taking every SPLIT-th piece (few rows have
// many pieces, and then it is the chain of reads that costs), and are joined in LDS in a fixed order.
constexpr int kJoin = 256;

template <bool BF16, int D, int SPLIT>
__global__ __launch_bounds__(kJoin) void attn_join_kernel(AttnArgs a, int nb, int MS, int MO, int N)
{
    constexpr int C4 = D / 4, PER = kJoin / SPLIT, AHEAD = 4;
    __shared__ f32x4_t box[SPLIT > 1 ? kJoin : 1];
    __shared__ float2 box_ml[SPLIT > 1 ? kJoin : 1];
    const int sub = threadIdx.x / PER;
    const long long unit = (long long)blockIdx.x * PER + threadIdx.x % PER;
    const long long row = unit / C4;
    const int c4 = (int)(unit % C4);
    int n_s = 0, n_o = 0;
    size_t at_s = 0, at_o = 0, step_s = 0, step_o = 0;   // first rows in the workspace, rows to the next piece
    const Layout wk = layout(a, nb, MS, MO);
    const char* work = static_cast<const char*>(a.work);
    bool mine = row < (long long)a.B * a.K * a.Hq;
    if (mine) {
        const int G = a.Hq / a.Hkv;
        const int tok = (int)(row / a.Hq), hq = (int)(row - (long long)tok * a.Hq);
        const int b = tok / a.K, t = tok - b * a.K, h = hq / G, g = hq - h * G;
        const Head head = *reinterpret_cast<const Head*>(work);
        const PlanSeq plan = reinterpret_cast<const PlanSeq*>(work + wk.plan)[b];
        const Seq q = seq_of(a, b, N, MO);
        mine = t < q.cnt;
        if (mine && plan.tok_base >= 0) {
            const int r = (plan.tok_base + t) * G + g, rt = r / MS;
            n_s = head.splits;
            at_s = ((size_t)h * head.splits * head.row_tiles + rt) * MS + (r - rt * MS);
            step_s = (size_t)head.row_tiles * MS;
        }
        if (mine && q.tiles > 0) {
            const RowTiles rts_of = row_tiles_of(a, MO);
            const int r = t * G + g, rt = r / MO;
            const int rt_list = a.count ? rt : 0, rt_block = a.count ? 0 : rt;
            const int u = plan.own_base + (h * (a.count ? q.rts : 1) + rt_list) * q.tiles;
            const int p0 = part_of(head.own_units, head.own_parts, u);
            n_o = part_of(head.own_units, head.own_parts, u + q.tiles - 1) - p0 + 1;
            const size_t slot =
                ((size_t)p0 + ((size_t)b * a.Hkv + h) * rts_of.in_list + rt_list) * rts_of.grouped + rt_block;
            at_o = slot * MO + (r - rt * MO);
            step_o = (size_t)rts_of.grouped * MO;
            if (n_o == 1 && !q.part) mine = false;   // written by its one piece
        }
    }
    const float2* ml_s = reinterpret_cast<const float2*>(work + wk.ml_s) + at_s;
    const float2* ml_o = reinterpret_cast<const float2*>(work + wk.ml_o) + at_o;
    const f32x4_t* o_s = reinterpret_cast<const f32x4_t*>(work + wk.o_s) + at_s * C4 + c4;
    const f32x4_t* o_o = reinterpret_cast<const f32x4_t*>(work + wk.o_o) + at_o * C4 + c4;
    const int n = mine ? n_s + n_o : 0;
    float M = kNoMax, L = 0.f;
    f32x4_t acc = {0.f, 0.f, 0.f, 0.f};
    for (int i = sub; i < n; i += SPLIT * AHEAD) {
        float2 v[AHEAD];
        f32x4_t x[AHEAD];
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const int p = i + k * SPLIT;
            v[k] = make_float2(kNoMax, 0.f);
            x[k] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            if (p < n) {
                const bool sh = p < n_s;
                const size_t j = sh ? p * step_s : (p - n_s) * step_o;
                v[k] = (sh ? ml_s : ml_o)[j];
                x[k] = (sh ? o_s : o_o)[j * C4];
            }
        }
        float mn = M;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) mn = fmaxf(mn, v[k].x);
        const float f = exp2_(M - mn);
        M = mn;
        L *= f;
        acc *= f;
#pragma unroll
        for (int k = 0; k < AHEAD; ++k) {
            const float w = exp2_(v[k].x - mn);
            L = __builtin_fmaf(v[k].y, w, L);
            acc += x[k] * w;
        }
    }
    if constexpr (SPLIT > 1) {
        box[threadIdx.x] = acc;
        box_ml[threadIdx.x] = make_float2(M, L);
        __syncthreads();
        if (sub > 0) return;
        for (int k = 1; k < SPLIT; ++k) {
            const float2 v = box_ml[k * PER + threadIdx.x];
            const float mn = fmaxf(M, v.x), f = exp2_(M - mn), w = exp2_(v.x - mn);
            M = mn;
            L = L * f + v.y * w;
            acc = acc * f + box[k * PER + threadIdx.x] * w;
        }
    }
    if (!mine) return;
    const f32x4_t y = acc * (L == 0.f ? 0.f : 1.f / L);
    if constexpr (BF16)
        reinterpret_cast<uint2*>(a.o)[unit] = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
    else
        reinterpret_cast<f32x4_t*>(a.o)[unit] = y;
    if (a.lse && c4 == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
}

}  // namespace attn
}  // namespace gdn
