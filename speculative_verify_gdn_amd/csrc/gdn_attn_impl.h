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
// The own list has the units (sequence, head, key tile) in this order, with
// kStartup empty ones before each head's tiles, and part i of n has the units
// [i U / n, (i+1) U / n), so the load is even whatever the lengths are; a part's row
// tiles go to neighbouring workgroups (with windows of unequal length, or more row
// tiles than there are workgroups, the row tiles are units of the list instead).  No host knowledge of lengths is
// needed: each workgroup sums them over the sequences by itself.  The workgroups
// take the shared items in their order and the own parts from the last workgroup
// down, so that short lists meet as little as may be.  A run of units of
// one row tile is a piece; a piece leaves (m, l, a) in the workspace and a second
// kernel joins the pieces of each row, except where one piece is all there is.
// Consecutive workgroups sit on one XCD, so that row tiles that read the same keys
// at the same time share its L2: before the row tiles of a key range were
// neighbours, four of five reads of a shared prefix missed it.
//
// Rows a wave.  In bf16 4 waves share a workgroup and 2 workgroups a CU, so a wave has 256 registers: enough for 32
// rows (two groups of 16 that use each fragment of K and V twice) up to head size 128.  8 waves of 16 rows read twice
// as much from LDS; with loads that nobody waited for early both came from 600 to 556 us over 128 windows of 16 tokens.
//
// A tile.  K and V rows go from memory straight into LDS (16 bytes a lane), one
// tile ahead of the one being worked on.  S^T = K Q^T leaves a query row in the
// lanes with the same lane & 15, 4 keys a register group; e^{x-m} of that layout
// is already the operand of O^T = V^T P^T, and V^T comes out of LDS by the
// transposing 8-byte read.  The 16-byte chunks of a row are permuted by the key's
// low bits so that both kinds of read meet every bank once.
//
// What bounds it.  Shared tiles of 128 rows and 64 keys of 128: products take 0.46 of a SIMD's busy time and vector work
// (the exponentials) 0.53, one after the other within a wave and only by chance beside the other wave's.  At head size
// 256 a wave has 16 rows, and no unit is busy for more than a third of the time (products 0.23, vector work 0.31, LDS
// 0.26, the loads' 64 bytes a cycle 0.32): it is the chain of its steps that costs, with two waves a SIMD.  Own tiles of
// few rows stream at 6.1 TB/s.
#pragma once

#include "gdn_device.h"
#include "gdn_kv_internal.h"

namespace gdn {
namespace attn {

typedef __attribute__((__vector_size__(4 * sizeof(short)))) short bf16x4_t;
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) char lds_char;
typedef __attribute__((address_space(3))) bf16x4_t lds_bf16x4;

constexpr int kThreads = 512, kWaves = kThreads / 64;   // of a workgroup at most
constexpr float kNoMax = -3.4028234e38f;   // the reference of a row that has seen no key: finite, so that -inf less it is -inf
constexpr float kNoScore = -0x1.fffffcp127f;   // of one that has seen keys, all with a score of -inf: the next above
constexpr float kSlack = 8.0f;     // a reference is kept while no exponent passes it by more than 2^8
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// M rows by N keys over W waves: RW groups of RG x 16 rows x KW groups of keys x DW parts of the output's columns
template <bool BF16_, int D_, int W_, int RW_, int RG_, int KW_, int DW_>
struct Cfg {
    static constexpr bool BF16 = BF16_;
    static constexpr int D = D_, WAVES = W_, THREADS = 64 * W_, RW = RW_, RG = RG_, KW = KW_, DW = DW_;
    static_assert(RW * KW * DW == WAVES && WAVES <= kWaves, "every wave has a part");
    static constexpr int M = 16 * RW * RG;
    static constexpr int ES = BF16 ? 2 : 4, ROW = D * ES, CH = ROW / 16;
    static constexpr int N = 8192 / D;             // keys a tile: K and V are 32 KB in bf16, 64 KB in fp32
    static constexpr int KF = N / KW / 16;         // 16-key groups of a wave
    static constexpr int DB = D / 16 / DW;         // 16-column groups of a wave's output
    static constexpr int MAT = N * ROW, STAGE = 2 * MAT;
    static constexpr int QC = BF16 ? D / 32 : D / 16;  // 16-byte pieces a lane holds of a row's q
    static_assert((KW - 1) * DW * RW * RG * DB * 1024 <= STAGE, "what the waves of other keys leave fits one buffer");
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

// What a piece costs beside its tiles (its first reads, its end), in tiles: cutting by tiles alone left the workgroups
// with many short sequences at work twice as long as the others.
constexpr int kStartup = 6;

// what a sequence asks for
struct Seq {
    int cnt, len, end, start, tiles, rts;
    bool part;
    int segs;        // runs of tiles: (head, row tile) pairs
};

__host__ __device__ __forceinline__ Seq seq_from(const AttnArgs& a, int len, int count, int N, int M)
{
    Seq s;
    const int cap = a.P << a.page_log2;
    s.cnt = min(max(count, 0), a.K);
    s.len = min(max(len, 0), cap);
    s.end = (int)min((long long)s.len + s.cnt, (long long)cap);
    s.part = a.prefix > 0 && s.len >= a.prefix && s.cnt > 0;
    s.start = s.part ? a.prefix : 0;
    s.tiles = s.cnt > 0 ? (s.end - s.start + N - 1) >> __builtin_ctz(N) : 0;   // (N and M are powers of two)
    s.rts = (s.cnt * a.G + M - 1) >> __builtin_ctz(M);
    s.segs = s.tiles > 0 ? a.Hkv * (a.listed ? s.rts : 1) : 0;
    return s;
}

// (by values: a conditional of two lvalues would put the arguments in memory)
__device__ __forceinline__ int count_of(const AttnArgs& a, int b)
{
    int n = a.K;
    if (a.count) n = a.count[b];
    return n;
}

__device__ __forceinline__ Seq seq_of(const AttnArgs& a, int b, int N, int M)
{
    return seq_from(a, a.lens[b], count_of(a, b), N, M);
}

// the lists' lengths and cuts, for the joining kernel
struct Head {
    int row_tiles, splits;       // of the shared list
    int own_units, own_parts, own_extra;
};
struct PlanSeq {
    int own_base;   // own units of the sequences before
    int tok_base;   // window tokens of the prefix-holding sequences before (-1: not one of them)
};

// workspace: Head | PlanSeq[B] | (m, l) of shared rows | of own rows | a of shared rows | of own rows
inline size_t up256(size_t x) { return (x + 255) & ~(size_t)255; }
inline AttnWork layout(const AttnArgs& a, int nb, int MS, int MO)
{
    const size_t G = a.Hq / a.Hkv;
    const size_t segs = MS ? a.Hkv * (((size_t)a.B * a.K * G + MS - 1) / MS) : 0;
    const size_t slots_s = MS ? (segs > 2 * (size_t)nb ? segs : 2 * (size_t)nb) : 0;
    const size_t slots_o = nb + (size_t)a.B * a.Hkv * ((a.K * G + MO - 1) / MO);
    AttnWork w;
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
__host__ __device__ __forceinline__ int first_unit(int units, int n, int i)
{
    return (int)(((double)units * i + 0.5) / n);
}
__host__ __device__ __forceinline__ int part_of(int units, int n, int u)
{
    return (int)(((double)(u + 1) * n - 0.5) / units);
}
// Into how many splits the prefix goes: for s of them, `segs` heads and row tiles take ceil(segs s / nb) rounds of
// ceil(tiles / s) tiles and about kStartup tiles' time for a piece's first reads and its end.  A lane tries each s;
// there are at most max(segs, 2 nb) items.
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

// How the own list counts row tiles: with equal windows a unit stands for all RT of them, taken by RT
// neighbouring workgroups; otherwise each is a unit of its own.  So it is too where there are more of them than the nb
// workgroups, of which some would then have none to take them.
struct RowTiles {
    int in_list, grouped;
};
__host__ __device__ inline int own_row_tiles(const AttnArgs& a, int M) { return (a.K * a.G + M - 1) >> __builtin_ctz(M); }
inline bool row_tiles_listed(const AttnArgs& a, int M, int nb) { return a.count || own_row_tiles(a, M) > nb; }
__host__ __device__ inline RowTiles row_tiles_of(const AttnArgs& a, int M)
{
    const int rt = own_row_tiles(a, M);
    return a.listed ? RowTiles{rt, 1} : RowTiles{1, rt};
}

// The own list of `tiles` tiles in `segs` runs: its units, the empty ones before a run's tiles, and into how many parts
// it is cut (no more than it has units, so that none is empty), each the work of `grouped` of the nb workgroups.
struct OwnList {
    int units, extra, parts, blocks;
};
__host__ __device__ __forceinline__ OwnList own_list_of(const RowTiles& rts, int tiles, int segs, int nb)
{
    OwnList l;
    l.extra = tiles <= nb / rts.grouped ? 0 : kStartup;   // (with a part for every tile there is nothing to even out)
    l.units = tiles + l.extra * segs;
    l.parts = min(max(nb / rts.grouped, 1), l.units);
    l.blocks = l.parts * rts.grouped;
    return l;
}

// ---------------------------------------------------------------- pieces of a tile
__device__ __forceinline__ int uni(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uni_ptr(const char* p)
{
    const uint64_t v = (uint64_t)p;
    return (const char*)((uint64_t)(uint32_t)uni((int)v) | (uint64_t)(uint32_t)uni((int)(v >> 32)) << 32);
}

// COUNT KB of global memory to LDS: in the i-th, lane l's 16 bytes at base + 1024 i + voff[i] go to
// lds + 1024 i + 16 l (the instruction's offset counts on both sides).  Written as assembly because the
// compiler would otherwise wait for the tile on its way before it reads the tile that is there; nothing
// is returned in registers, and load_wait() below waits for all of them.  (m0 takes the LDS address; one
// wait state between writing it and the load.)
template <int COUNT>
__device__ __forceinline__ void load_lds(uint32_t lds, const uint32_t* voff, const char* base)
{
    static_assert(COUNT == 2 || COUNT == 4, "2 or 4 KB");
    lds = uni(lds);
    base = uni_ptr(base);
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
    // by the builtin, which the compiler's own count of outstanding loads sees (vmcnt 0, the other counters free): after
    // a wait in assembly it waited again for the page ids, behind the next tile's loads, which held every tile up for
    // the time of its successor's loads
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt(0x0f70);
    asm volatile("" ::: "memory");
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


__device__ __forceinline__ float exp2_(float x) { return __builtin_amdgcn_exp2f(x); }

// A row's reference is one of its scores times the factor c, m.  Exponents are formed as fma(x, c, -m), one
// instruction; from kFar on as (x - score) c: there the rounding of m, half a step, would grow past what a float's
// exponent holds (2^31 and more gave infinities or no weight at all).  References are joined as m: rounding keeps
// their order, and is off by less than the scores themselves.
constexpr float kFar = 1048576.f;
__device__ __forceinline__ bool is_far(float m) { return fabsf(m) >= kFar && m != kNoMax; }

// 1 / l of a row; without any weight 0 where it has seen no key, and the 0 / 0 of the formula where all its scores are -inf
__device__ __forceinline__ float inverse_of(float l, float m)
{
    return l != 0.f ? 1.f / l : m == kNoMax ? 0.f : __builtin_nanf("");
}

// scores enter the exponentials with a factor above 0: the sign of `scale` goes into q, and for a scale of 0 all of q
__device__ __forceinline__ float factor_of(float scale) { return scale == 0.f ? 1.f : fabsf(scale) * kLog2e; }

// two floats to bf16 (to nearest), packed
__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    const bf16x2_t h = {(__bf16)x, (__bf16)y};
    return __builtin_bit_cast(uint32_t, h);
}

// nodes on the path from a root to each node: lane i has the parent of node i (one that is not below it: a root) and
// gets those of node i (called by a whole wave)
__device__ __forceinline__ unsigned long long ancestors(int parent)
{
    const int lane = threadIdx.x & 63;
    int up = parent >= 0 && parent < lane ? parent : -1;
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
    // what pieces are described from: uniform values, read again where they are needed (in scalar registers they
    // would be spilled to vector registers all through the loop)
    int own_part, rt_block, own_u1, extra;
    int row_tiles, key_tiles, splits, tok_total;
    const char* base[4];                // in the workspace: a of shared and of own rows, their (m, l)
    int bad_value;                      // the number of the last piece that had a window value that is not finite
    int tok_base[kThreads];             // window tokens of the prefix-holding sequences before a thread's own
    int len[kThreads], count[kThreads]; // lengths and windows of the first sequences (all of them, mostly)
    unsigned long long path[2][64];     // the window's nodes on the path to each node, by the piece's number
    int tok[132];                       // window tokens (b * K + t) of a shared row tile
    float far[kWaves][32];              // the scores that references are of, for rows that are far
    float2 ml[kWaves][32];              // (m, l) of the waves' rows, to be joined
};

// where a piece starts: own: sequence b, `off` units into it, unit u of the list; shared: item it
struct Ref {
    int b, off, u, it;
};

// a run of tiles of one row tile
struct Piece {
    int b;                  // whose table row it reads
    int h, p0, tiles;       // key/value head, first position, tiles
    int len, end;           // the window's first position and the end of what is there
    int r0, tok0, tok1;     // rows r0.. of the tokens tok0 .. tok1-1 (row r is of token r / G)
    int slot;               // workspace slot; -1: the rows are whole, o and lse are written at once
};

// The kernel's arguments, loaded anew (the first argument is at the start of their segment): used where the time of
// a scalar load does not count, to keep them out of the registers of the loop.
__device__ __forceinline__ const AttnArgs& args_again()
{
    auto p = __builtin_amdgcn_kernarg_segment_ptr();
    asm volatile("" : "+s"(p));
    return *(const AttnArgs*)p;
}

// inclusive sum over the lanes of a wave, by DPP (row shifts, then the rows' last lanes to the rows after)
__device__ __forceinline__ int wave_scan(int v)
{
    v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
    v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
    return v;
}

// exclusive sum over the workgroup's threads, and the total
template <int WAVES>
__device__ __forceinline__ int scan_int(int v, Small& s, int& total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int inc = wave_scan(v);
    __syncthreads();
    if (lane == 63) s.part[w] = inc;
    __syncthreads();
    int base = 0;
    total = 0;
    for (int i = 0; i < WAVES; ++i) {
        base += i < w ? s.part[i] : 0;
        total += s.part[i];
    }
    return base + inc - v;
}

// which list a piece is of
template <class Config, bool SHARED>
struct ListTag {
    using C = Config;
    static constexpr bool shared = SHARED;
};

template <class C>
__device__ __forceinline__ constexpr int rows_of()
{
    if constexpr (__is_same(C, void)) return 0;
    else return C::RG;
}

// SH: the shared list's configuration, or void
template <class OW, class SH>
__global__ __launch_bounds__(OW::THREADS, 2) void attn_kernel(AttnArgs a, int nb)
{
    // all of LDS is asked for at the launch and starts at 0: the swizzled addresses flip bits below 256
    extern __shared__ __attribute__((aligned(1024))) char sm[];
    Small& s = *reinterpret_cast<Small*>(sm + 2 * OW::STAGE);
    constexpr bool kShared = !__is_same(SH, void);
    constexpr int N = OW::N, QC = OW::QC, ROW = OW::ROW, THREADS = OW::THREADS, WAVES = OW::WAVES;
    using OwnTag = ListTag<OW, false>;
    using SharedTag = ListTag<SH, true>;
    const int lane = threadIdx.x & 63, w = uni(threadIdx.x >> 6);
    const int n16 = lane & 15, grp = lane >> 4;
    const int G = a.G;
    constexpr int RGS = rows_of<SH>(), RGM = OW::RG > RGS ? OW::RG : RGS;
    int MS = 0;
    if constexpr (kShared) {
        static_assert(SH::THREADS == THREADS);
        MS = SH::M;
    }
    char* work = static_cast<char*>(a.work);

    // ---- the lists' lengths: thread i sums the sequences [b0, b1)
    const int per = (a.B + THREADS - 1) / THREADS;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);
    int my_tiles = 0, my_segs = 0, toks = 0;
    for (int b = b0; b < b1; ++b) {
        const int len = a.lens[b], count = count_of(a, b);
        const Seq q = seq_from(a, len, count, N, OW::M);
        my_tiles += q.segs * q.tiles;
        my_segs += q.segs;
        if (q.part) toks += q.cnt;
        if (b < kThreads) {
            s.len[b] = len;
            s.count[b] = count;
        }
    }
    if (threadIdx.x == 0) s.bad_value = 0;
    int own_tiles, own_segs;
    const int tiles_base = scan_int<WAVES>(my_tiles, s, own_tiles), segs_base = scan_int<WAVES>(my_segs, s, own_segs);
    int tok_total = 0, tok_base = 0;
    int items = 0, row_tiles = 0, key_tiles = 0, splits = 0;
    if constexpr (kShared) {
        tok_base = scan_int<WAVES>(toks, s, tok_total);
        s.tok_base[threadIdx.x] = tok_base;
        tok_total = uni(tok_total);
        row_tiles = (tok_total * G + SH::M - 1) / SH::M;
        key_tiles = (a.prefix + N - 1) / N;
        splits = splits_for(a.Hkv * row_tiles, key_tiles, nb);
        items = a.Hkv * row_tiles * splits;
    }
    const RowTiles rts_of = row_tiles_of(a, OW::M);
    const OwnList list = own_list_of(rts_of, uni(own_tiles), uni(own_segs), nb);
    const int extra = list.extra, own = list.units, own_base = tiles_base + extra * segs_base;
    const int mine = my_tiles + extra * my_segs;
    const int own_parts = list.parts;
    const int blocks = min(nb, items + list.blocks);
    // consecutive workgroups of the lists on one XCD (workgroups are dealt to the 8 XCDs in turn)
    const int per_xcd = (blocks + 7) / 8;
    const int lb = (blockIdx.x & 7) * per_xcd + (blockIdx.x >> 3);
    if (blockIdx.x == 0) {
        if (threadIdx.x == 0) *reinterpret_cast<Head*>(work) = Head{row_tiles, splits, own, own_parts, extra};
        PlanSeq* plan = reinterpret_cast<PlanSeq*>(work + a.at.plan);
        int base = own_base, tok = tok_base;
        for (int b = b0; b < b1; ++b) {
            const Seq q = seq_of(a, b, N, OW::M);
            plan[b] = PlanSeq{base, q.part ? tok : -1};
            base += q.segs * (q.tiles + extra);
            tok += q.part ? q.cnt : 0;
        }
    }
    if ((int)(blockIdx.x >> 3) >= per_xcd || lb >= blocks) return;

    // ---- the own part: its units [own_u, own_u1), the first in sequence found_b, found_off units into it
    const int own_block = blocks - 1 - lb;
    const bool has_own = own_block < list.blocks;
    const int own_part = own_block / rts_of.grouped;
    const int own_u = uni(has_own ? first_unit(own, own_parts, own_part) : 0);
    const int own_u1 = uni(has_own ? first_unit(own, own_parts, own_part + 1) : 0);
    if (own_base <= own_u && own_u < own_base + mine) {
        int base = own_base;
        for (int b = b0; b < b1; ++b) {
            const Seq q = seq_of(a, b, N, OW::M);
            const int units = q.segs * (q.tiles + extra);
            if (own_u < base + units) {
                s.found_b = b;
                s.found_off = own_u - base;
                break;
            }
            base += units;
        }
    }
    if (threadIdx.x == 0) {
        s.own_part = own_part;
        s.rt_block = own_block - own_part * rts_of.grouped;
        s.own_u1 = own_u1;
        s.extra = extra;
        s.row_tiles = row_tiles;
        s.key_tiles = key_tiles;
        s.splits = splits;
        s.tok_total = tok_total;
        s.base[0] = work + a.at.o_s;
        s.base[1] = work + a.at.o_o;
        s.base[2] = work + a.at.ml_s;
        s.base[3] = work + a.at.ml_o;
    }
    __syncthreads();

    auto seq_at = [&](int b) {
        int len, count;
        if (b < kThreads) {
            len = uni(s.len[b]);
            count = uni(s.count[b]);
        } else {
            len = uni(args_again().lens[b]);
            count = uni(count_of(args_again(), b));
        }
        return seq_from(args_again(), len, count, N, OW::M);
    };
    // the piece of the own list at a place (it may have no tile) and on past it, or of an item of the shared one
    auto piece_of = [&](auto tag, Ref& r) {
        const AttnArgs& a = args_again();
        const int G = a.G;
        Piece p;
        if constexpr (tag.shared) {
            const int row_tiles = uni(s.row_tiles), key_tiles = uni(s.key_tiles), splits = uni(s.splits);
            const int hs = r.it / row_tiles, rt = r.it - hs * row_tiles, sp = hs % splits;
            const int k0 = (int)((unsigned)key_tiles * sp / splits);
            p.b = uni(s.tok[0]) / a.K;   // (all of the tile's sequences hold the same pages here)
            p.h = hs / splits;
            p.p0 = k0 * N;
            p.tiles = (int)((unsigned)key_tiles * (sp + 1) / splits) - k0;
            p.len = p.end = a.prefix;
            p.r0 = rt * decltype(tag)::C::M;
            p.tok0 = p.r0 / G;
            p.tok1 = min((p.r0 + decltype(tag)::C::M - 1) / G + 1, uni(s.tok_total));
            p.slot = r.it;
        } else {
            const Seq q = seq_at(r.b);
            const RowTiles rts_of = row_tiles_of(a, OW::M);
            const int rt_block = uni(s.rt_block);
            const int extra = uni(s.extra), span = q.tiles + extra, seg = r.off / span, u0 = r.off - seg * span;
            const int u1 = min(span, u0 + uni(s.own_u1) - r.u), k0 = max(u0 - extra, 0);
            const int h = a.listed ? seg / q.rts : seg, rt_list = a.listed ? seg - h * q.rts : 0;
            p.b = r.b;
            p.h = h;
            p.p0 = q.start + k0 * N;
            p.tiles = u1 - extra - k0;
            p.len = q.len;
            p.end = q.end;
            p.r0 = (rt_list + rt_block) * OW::M;
            p.tok0 = 0;
            p.tok1 = q.cnt;
            p.slot = !q.part && p.tiles == q.tiles
                         ? -1
                         : (uni(s.own_part) + (r.b * a.Hkv + h) * rts_of.in_list + rt_list) * rts_of.grouped + rt_block;
            r.u += u1 - u0;
            r.off += u1 - u0;
        }
        return p;
    };

    // ---- the loader, which is one tile ahead of the work and goes on from a piece to the next: lane i holds the
    // page of the slot first + i (a missing one as page 0, flagged), and that of the 64 slots after
    const int page_mask = (1 << a.page_log2) - 1;
    const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_char*)sm;
    const uint32_t page_bytes = ((uint32_t)a.Hkv << a.page_log2) * ROW;
    auto slot_id = [&](const int32_t* row, int sl) { return sl < a.P ? row[sl] : -1; };
    auto is_bad = [&](int id) { return (unsigned)id >= (unsigned)a.n_pages; };
    const int32_t* ld_row = nullptr;   // its table row
    int ld_first = 0, ld_p0 = 0, ids = 0, ids2 = 0, ids_next = 0, ids2_next = 0;
    uint32_t ld_head = 0;
    unsigned long long bad = 0;
    int buf = 0;             // the buffer that the next tile is loaded into
    unsigned miss_next = 0;  // missing pages of the tile loaded last
    auto row_at = [&](int b) { return a.table + (size_t)b * a.P; };
    auto load_ids = [&](const Piece p) {
        const int32_t* row = row_at(p.b);
        const int first = (p.p0 >> a.page_log2) + lane;
        ids_next = slot_id(row, first);
        ids2_next = slot_id(row, first + 64);
    };
    // (loads nothing: a load here, into registers that the loop goes on using, would be waited for behind every tile's)
    auto load_piece = [&](const Piece p) {
        ld_row = row_at(p.b);
        ld_p0 = p.p0;
        ld_first = p.p0 >> a.page_log2;
        ld_head = ((uint32_t)p.h << a.page_log2) * ROW;
        ids = ids_next;
        ids2 = ids2_next;
        bad = __ballot(is_bad(ids));
    };
    // Wave w of W brings the keys w N/W .. of K and V, in groups of up to 16 keys (of one page, as a page has 16 at
    // least), a group in runs of CNT KB; the i-th KB of a group is i KPI keys on: bits of the key that no other part
    // of it has, so they flip into the swizzle.
    constexpr int WK = N / WAVES, GK = WK < 16 ? WK : 16, KPI = 1024 / ROW, NI = GK / KPI, CNT = NI < 4 ? NI : 4;
    const int lkey = lane / OW::CH, lch = lane % OW::CH;
    const uint32_t k_off = lkey * ROW + ((lch ^ k_swizzle<OW>((w * WK + lkey) & 15)) << 4);
    const uint32_t v_off = lkey * ROW + ((lch ^ v_swizzle<OW>((w * WK + lkey) & 15)) << 4);
    auto issue = [&](int j) {
        const int pt = ld_p0 + j * N;
        int s0 = (pt >> a.page_log2) - ld_first;
        if (s0 >= 64) {
            ids = ids2;
            bad = __ballot(is_bad(ids));
            ld_first += 64;
            s0 -= 64;
            ids2 = slot_id(ld_row, ld_first + 64 + lane);
            load_wait();   // here, or it may be waited for where the ways meet again: behind every tile's loads
        }
#pragma unroll
        for (int g = 0; g < WK / GK; ++g) {
            const int key = w * WK + g * GK;
            int id = __builtin_amdgcn_readlane(ids, s0 + (key >> a.page_log2));
            id = is_bad(id) ? 0 : id;
            const uint64_t off = (uint64_t)(uint32_t)id * page_bytes + (ld_head + ((pt + key) & page_mask) * ROW);
            const uint32_t to = lds0 + buf * OW::STAGE + key * ROW;
#pragma unroll
            for (int i = 0; i < NI; i += CNT) {
                uint32_t ko[CNT], vo[CNT];
#pragma unroll
                for (int e = 0; e < CNT; ++e) {
                    ko[e] = k_off ^ (k_swizzle<OW>((i + e) * KPI) << 4);
                    vo[e] = v_off ^ (v_swizzle<OW>((i + e) * KPI) << 4);
                }
                load_lds<CNT>(to + i * 1024, ko, static_cast<const char*>(a.k_pages) + off + i * 1024);
                load_lds<CNT>(to + OW::MAT + i * 1024, vo, static_cast<const char*>(a.v_pages) + off + i * 1024);
            }
        }
        const int slots = max(N >> a.page_log2, 1);
        miss_next = (unsigned)(bad >> s0) & ((1u << slots) - 1);
        buf ^= 1;
    };

    // ---- the rows of a piece
    // Row `row` of the tile: its token b * K + t, t, and the query head of its group.  Formed anew wherever it is
    // asked for: kept, it would take registers through the loop.
    auto row_of = [&](auto tag, const Piece p, int rw, int& tok, int& t, int& g) {
        const AttnArgs& a = args_again();
        const int G = a.G;
        int row = rw * 16 + (threadIdx.x & 15);
        asm volatile("" : "+v"(row));
        const int x = p.r0 - p.tok0 * G + row;   // below 2^17, so the quotient by floats is exact (half an x added)
        const int tx = (int)(((float)x + 0.5f) * __builtin_amdgcn_rcpf((float)G)), ti = p.tok0 + tx;
        const bool live = ti < p.tok1;
        g = live ? x - tx * G : 0;
        tok = !live ? 0 : tag.shared ? s.tok[ti - p.tok0] : p.b * a.K + ti;
        t = !live ? 0 : tag.shared ? 0 : ti;
        return live;
    };
    const float c = factor_of(a.scale);
    uint4 q[RGM][QC];
    bool alive = false;      // a wave without rows only loads
    auto load_q = [&](auto tag, const Piece p) {
        const AttnArgs& a = args_again();
        using C = typename decltype(tag)::C;
        alive = false;
#pragma unroll
        for (int r = 0; r < C::RG; ++r) {
            int tok, t, g;
            const bool live = row_of(tag, p, w % C::RW * C::RG + r, tok, t, g);
            alive |= __any(live);
            const char* qp = static_cast<const char*>(a.q) +
                             ((size_t)tok * a.q_stride + (size_t)(p.h * a.G + g) * OW::D) * OW::ES + grp * 16;
#pragma unroll
            for (int e = 0; e < QC; ++e) {
                q[r][e] = make_uint4(0, 0, 0, 0);
                if (live) q[r][e] = *reinterpret_cast<const uint4*>(qp + e * 64);
            }
        }
    };
    const uint32_t flip = a.scale < 0.f ? (OW::BF16 ? 0x80008000u : 0x80000000u) : 0u;
    const uint32_t keep = a.scale == 0.f ? 0u : ~0u;

    int serial = 0;          // the pieces' numbers
    const bool has_parent = a.parent != nullptr;
    int parent_next = -1;    // (first wave) lane i: the parent of node i in the next piece's window
    auto load_parent = [&](const Piece p) {   // (of own pieces)
        if (w == 0 && p.p0 + p.tiles * N > p.len) {
            const AttnArgs& a = args_again();
            parent_next = -1;
            if (a.parent && lane < a.K) parent_next = a.parent[(size_t)p.b * a.K + lane];
        }
    };

    // Works on the piece at `now`, whose first tile and q are on their way; where `more`, brings the same of the own
    // piece at `next` while it works.
    auto run = [&](auto tag, const Piece p, const bool more, const Piece n) {
        using C = typename decltype(tag)::C;
        constexpr bool window = !tag.shared;
        constexpr int KF = C::KF, DB = C::DB, RG = C::RG;
        const int rw = w % C::RW, kw = (w / C::RW) % C::KW, dw = w / (C::RW * C::KW);
        ++serial;
        if (w == 0) s.path[serial & 1][lane] = has_parent ? ancestors(parent_next) : ~0ull >> (63 - lane);
        if (more) {
            load_ids(n);
            load_parent(n);
        }
        const int p0 = p.p0, tiles = p.tiles, len = p.len, end = p.end;
        float m[RG], l[RG];
        bool far = false;   // a row of this wave is
        f32x4_t o[RG][DB];
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            m[r] = kNoMax;
            l[r] = 0.f;
#pragma unroll
            for (int d = 0; d < DB; ++d) o[r][d] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int e = 0; e < QC; ++e) {
                const uint4 u = q[r][e];
                q[r][e] = make_uint4((u.x ^ flip) & keep, (u.y ^ flip) & keep, (u.z ^ flip) & keep, (u.w ^ flip) & keep);
            }
        }

        // LDS addresses of this lane within a tile: chunk c of a row sits at its lane's chunk with the low bits of c
        // flipped in, and further chunks, keys and 16-key groups lie at constant distances
        const int kbase = kw * (N / C::KW);
        const int vkey = C::BF16 ? 4 * grp + (n16 >> 2) : 4 * grp;   // (fp32 adds the register's index)
        const uint32_t k_lane = lds0 + (kbase + n16) * ROW + ((grp ^ k_swizzle<C>(n16)) << 4);
        const uint32_t v_lane =
            lds0 + C::MAT + (kbase + vkey) * ROW + (dw * DB * 16 * C::ES & ~255) +
            (C::BF16 ? ((((n16 >> 1) & 1) ^ v_swizzle<C>(vkey) ^ (2 * dw * DB & 15)) << 4) + (n16 & 1) * 8
                     : (((n16 >> 2) ^ v_swizzle<C>(vkey)) << 4) + (n16 & 3) * 4);
        static_assert((DB & (DB - 1)) == 0 && (C::BF16 || DB % 4 == 0), "a part's columns do not straddle swizzle groups");

        for (int j = 0; j < tiles; ++j) {
            const unsigned miss = miss_next;
            load_wait();
            block_barrier();   // every wave's part of this tile is there, and nobody reads the other buffer any more
            const int here = buf ^ 1;
            if (j + 1 < tiles) {
                issue(j + 1);
            } else if (more) {
                load_piece(n);
                issue(0);
            }
            char* vt = sm + here * C::STAGE + C::MAT;
            const int pt = p0 + j * N;
            const bool masked = miss != 0 || (window && pt + N > len) || pt + N > end;

            // Values nobody may see are cleared where they lie (0 times NaN is NaN), and so are the window's that are
            // not finite: only some rows see them, and get them at the end.
            if (masked) {
                int e0 = threadIdx.x;
                asm volatile("" : "+v"(e0));
                for (int e = e0; e < N * C::CH; e += THREADS) {
                    const int key = e / C::CH, pos = pt + key;
                    uint32_t* v = reinterpret_cast<uint32_t*>(vt + e * 16);
                    if (pos >= end || (miss >> (key >> a.page_log2) & 1)) {
                        *reinterpret_cast<uint4*>(v) = make_uint4(0, 0, 0, 0);
                    } else if (window && pos >= len) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const uint32_t u = v[i];
                            uint32_t keep = u;
                            if ((u & 0x7f800000u) == 0x7f800000u) keep &= C::BF16 ? 0xffffu : 0u;
                            if (C::BF16 && (u & 0x7f80u) == 0x7f80u) keep &= 0xffff0000u;
                            if (keep != u) {
                                v[i] = keep;
                                s.bad_value = serial;
                            }
                        }
                    }
                }
                block_barrier();
            }
            if (!alive) continue;

            // opaque, so that the addresses are formed from them in the loop and not kept in dozens of registers
            uint32_t k_at = k_lane + here * C::STAGE, v_at = v_lane + here * C::STAGE;
            asm volatile("" : "+v"(k_at), "+v"(v_at));

            // ---- S^T = K Q^T, the reads of a 16-byte column of K (for all keys) ahead of the products with the one
            // before: left to itself the compiler waits for each read right after it
            f32x4_t x[RG][KF];
#pragma unroll
            for (int r = 0; r < RG; ++r)
#pragma unroll
                for (int k = 0; k < KF; ++k) x[r][k] = f32x4_t{0.f, 0.f, 0.f, 0.f};
            uint4 kf[2][KF];
            auto read_k = [&](int e) {
#pragma unroll
                for (int k = 0; k < KF; ++k)
                    kf[e & 1][k] = lds_read16((k_at ^ (uint32_t)(((4 * e) & (C::CH - 1) & 15) << 4)) +
                                              (4 * e / 16) * 256 + 16 * k * ROW);
            };
            read_k(0);
#pragma unroll
            for (int e = 0; e < QC; ++e) {
                if (e + 1 < QC) read_k(e + 1);
                __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                for (int k = 0; k < KF; ++k) {
                    const uint4 u = kf[e & 1][k];
#pragma unroll
                    for (int r = 0; r < RG; ++r) {
                        if constexpr (C::BF16) {
                            x[r][k] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, u),
                                                                              __builtin_bit_cast(bf16x8_t, q[r][e]),
                                                                              x[r][k], 0, 0, 0);
                        } else {
                            const uint32_t ua[4] = {u.x, u.y, u.z, u.w};
                            const uint32_t qa[4] = {q[r][e].x, q[r][e].y, q[r][e].z, q[r][e].w};
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                x[r][k] = __builtin_amdgcn_mfma_f32_16x16x4f32(
                                    __uint_as_float(ua[i]), __uint_as_float(qa[i]), x[r][k], 0, 0, 0);
                        }
                    }
                }
                __builtin_amdgcn_sched_barrier(0);
            }

            // ---- weights e^{x-m}
            if (masked) {
                int key0 = kbase + 4 * grp;
                asm volatile("" : "+v"(key0));   // (what follows is formed here, not kept through the loop)
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    int tok, t, g;
                    row_of(tag, p, rw * RG + r, tok, t, g);
                    const unsigned long long sees = window ? s.path[serial & 1][t & 63] : 0;
#pragma unroll
                    for (int k = 0; k < KF; ++k) {
                        const int key = key0 + 16 * k;
                        // the 4 keys from position pt + key on: committed ones (below len), then the window's by their
                        // bits in `sees`, none from end on and none of a missing page; by shifts and selects only
                        const int rel = pt + key - len, left = end - (pt + key);
                        const unsigned win = rel > 63 ? 0u : (unsigned)(sees >> (max(rel, 0) & 63));
                        const int old = min(max(-rel, 0), 4);
                        unsigned bits = (win << old | ((1u << old) - 1)) & ((1u << min(max(left, 0), 4)) - 1);
                        bits = (miss >> (key >> a.page_log2) & 1) ? 0u : bits;
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[r][k][i] = (bits >> i & 1) ? x[r][k][i] : -INFINITY;
                    }
                }
            }
            float top[RG];
            bool move = false;
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                top[r] = x[r][0][0];
#pragma unroll
                for (int k = 0; k < KF; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) top[r] = fmaxf(top[r], x[r][k][i]);
                move |= top[r] * c > m[r] + kSlack;
            }
            if (__any(move) || far) {
                bool now_far = false;
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    top[r] = fmaxf(top[r], __shfl_xor(top[r], 16, 64));
                    top[r] = fmaxf(top[r], __shfl_xor(top[r], 32, 64));
                    // a row moves its reference by its own keys alone, so its bits depend on no other row
                    const bool up = top[r] * c > m[r] + kSlack || (is_far(m[r]) && top[r] > s.far[w][r * 16 + n16]);
                    const float mn = up ? top[r] * c : m[r], f = exp2_(m[r] - mn);
                    m[r] = mn;
                    if (up) s.far[w][r * 16 + n16] = top[r];
                    now_far |= is_far(mn);
                    l[r] *= f;
#pragma unroll
                    for (int d = 0; d < DB; ++d) o[r][d] *= f;
                }
                far = __any(now_far);
            }
            float mc[RG];
#pragma unroll
            for (int r = 0; r < RG; ++r) mc[r] = m[r];
            if (far) {
#pragma unroll
                for (int r = 0; r < RG; ++r) {
                    const float from = is_far(m[r]) ? s.far[w][r * 16 + n16] : 0.f;
                    mc[r] = is_far(m[r]) ? 0.f : m[r];
#pragma unroll
                    for (int k = 0; k < KF; ++k)
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[r][k][i] -= from;
                }
            }
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                float sum = 0.f;
#pragma unroll
                for (int k = 0; k < KF; ++k)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        x[r][k][i] = exp2_(__builtin_fmaf(x[r][k][i], c, -mc[r]));   // (0 where it is -infinity: c > 0)
                        sum += x[r][k][i];
                    }
                l[r] += sum;
            }

            // ---- O^T += V^T P^T
            if constexpr (C::BF16) {
                // The weights enter the product in bf16, as v is: half a step of 2^-8 each, unbiased (against 64 bits
                // 0.0018 to 0.0023 in all, 0.0017 with weights of 32 bits, of which 0.0017 is the output's own rounding).
                // Weights of 32 bits would be two or three bf16 products in the place of one.
                auto v_frag = [&](int k, int d) {
                    lds_char* at = (lds_char*)(uintptr_t)((v_at ^ (uint32_t)((d & (C::CH / 2 - 1) & 7) << 5)) +
                                                          (d / 8) * 256 + 16 * k * ROW);
                    return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_bf16x4*)at));
                };
                // groups of GV columns' reads, ahead of the products as above
                constexpr int KP = KF == 1 ? 1 : KF / 2, GV = DB < 4 ? DB : DB * RG > 16 ? 2 : 4, NG = KP * DB / GV;
                uint2 vf[2][GV][2];
                auto read_v = [&](int g) {
#pragma unroll
                    for (int i = 0; i < GV; ++i) {
                        const int k = g * GV / DB * 2, d = g * GV % DB + i;
                        vf[g & 1][i][0] = v_frag(k, d);
                        if constexpr (KF > 1) vf[g & 1][i][1] = v_frag(k + 1, d);
                    }
                };
                read_v(0);
                uint4 y[RG][KP];
#pragma unroll
                for (int r = 0; r < RG; ++r)
#pragma unroll
                    for (int k = 0; k < KP; ++k) {
                        y[r][k].x = pack2(x[r][2 * k][0], x[r][2 * k][1]);
                        y[r][k].y = pack2(x[r][2 * k][2], x[r][2 * k][3]);
                        if constexpr (KF > 1) {
                            y[r][k].z = pack2(x[r][2 * k + 1][0], x[r][2 * k + 1][1]);
                            y[r][k].w = pack2(x[r][2 * k + 1][2], x[r][2 * k + 1][3]);
                        }
                    }
#pragma unroll
                for (int g = 0; g < NG; ++g) {
                    if (g + 1 < NG) read_v(g + 1);
                    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
                    for (int i = 0; i < GV; ++i) {
                        const int k = g * GV / DB, d = g * GV % DB + i;
                        const uint2 v0 = vf[g & 1][i][0];
#pragma unroll
                        for (int r = 0; r < RG; ++r) {
                            if constexpr (KF == 1) {
                                o[r][d] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(
                                    __builtin_bit_cast(bf16x4_t, v0),
                                    __builtin_bit_cast(bf16x4_t, make_uint2(y[r][0].x, y[r][0].y)), o[r][d], 0, 0, 0);
                            } else {
                                const uint2 v1 = vf[g & 1][i][1];
                                o[r][d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                                    __builtin_bit_cast(bf16x8_t, make_uint4(v0.x, v0.y, v1.x, v1.y)),
                                    __builtin_bit_cast(bf16x8_t, y[r][k]), o[r][d], 0, 0, 0);
                            }
                        }
                    }
                    __builtin_amdgcn_sched_barrier(0);
                }
            } else {
#pragma unroll
                for (int k = 0; k < KF; ++k)
#pragma unroll
                    for (int d = 0; d < DB; ++d)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float v =
                                lds_read4((v_at ^ (uint32_t)((d & 3) << 6)) + (d / 4) * 256 + (16 * k + i) * ROW);
#pragma unroll
                            for (int r = 0; r < RG; ++r)
                                o[r][d] = __builtin_amdgcn_mfma_f32_16x16x4f32(v, x[r][k][i], o[r][d], 0, 0, 0);
                        }
            }
        }

        // ---- the next piece's q, while this one is put away
        const bool was_alive = alive;
        if (more) load_q(OwnTag{}, n);

        // ---- the four lane groups' sums, then the waves of other keys, in a fixed order
        const AttnArgs& a = args_again();
        const int G = a.G;
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            l[r] += __shfl_xor(l[r], 16, 64);
            l[r] += __shfl_xor(l[r], 32, 64);
        }
        bool none = false;
#pragma unroll
        for (int r = 0; r < RG; ++r) none |= l[r] == 0.f;
        if (was_alive && __any(none)) {
            // no weight: such a row sees nothing of this piece, or only scores of -inf
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                int tok, t, g;
                row_of(tag, p, rw * RG + r, tok, t, g);
                const unsigned long long sees = window ? s.path[serial & 1][t & 63] : 0;
                const int last = min(p.end, p.p0 + p.tiles * N);
                bool some = l[r] != 0.f;
#pragma nounroll
                for (int pos = p.p0, next; pos < last && !__all(some); pos = next) {   // a page after the other
                    next = min(((pos >> a.page_log2) + 1) << a.page_log2, last);
                    if (is_bad(slot_id(row_at(p.b), pos >> a.page_log2))) continue;
                    const int i0 = max(pos - p.len, 0), i1 = next - p.len;   // nodes i0 .. i1-1 of the window
                    some |= pos < p.len || (window && (sees >> i0 & ~0ull >> (64 - (i1 - i0))) != 0);
                }
                if (l[r] == 0.f && some) m[r] = kNoScore;
            }
        }
        if (uni(s.bad_value) == serial && was_alive) {
            // a window value that is not finite makes what it makes of the rows that see it
#pragma unroll
            for (int r = 0; r < RG; ++r) {
                int tok, t, g;
                row_of(tag, p, rw * RG + r, tok, t, g);
                const unsigned long long sees = s.path[serial & 1][t & 63];
#pragma nounroll
                for (int pos = max(p.p0, p.len); pos < min(p.end, p.p0 + p.tiles * N); ++pos) {
                    if (((pos - p.p0) % N) / (N / C::KW) != kw) continue;   // this wave's keys
                    const int page = slot_id(row_at(p.b), pos >> a.page_log2);
                    if (is_bad(page)) continue;
                    const size_t at = ((((size_t)page * a.Hkv + p.h) << a.page_log2) + (pos & page_mask)) * C::D;
#pragma unroll
                    for (int d = 0; d < DB; ++d) {
                        const float4 y = load4<C::BF16>(a.v_pages, at + (dw * DB + d) * 16 + 4 * grp);
                        const float ya[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
                        for (int i = 0; i < 4; ++i)
                            if ((sees >> (pos - p.len) & 1) && !(fabsf(ya[i]) < INFINITY)) o[r][d][i] += ya[i];
                    }
                }
            }
        }
        if constexpr (C::KW > 1) {
            // in the buffer of the last tile (the other one is being filled)
            float* box = reinterpret_cast<float*>(sm + (more ? buf : buf ^ 1) * C::STAGE);
            auto at = [&](int k, int r, int f) {
                return reinterpret_cast<f32x4_t*>(
                    box + (((((k - 1) * C::DW + dw) * C::RW + rw) * RG + r) * DB + f) * 256 + lane * 4);
            };
            block_barrier();   // the tile is done with
            if (kw > 0) {
#pragma unroll
                for (int r = 0; r < RG; ++r) {
#pragma unroll
                    for (int d = 0; d < DB; ++d) *at(kw, r, d) = o[r][d];
                    if (grp == 0) s.ml[w][r * 16 + n16] = make_float2(m[r], l[r]);
                }
            }
            block_barrier();
            if (kw == 0) {
#pragma unroll
                for (int r = 0; r < RG; ++r)
#pragma nounroll
                    for (int k = 1; k < C::KW; ++k) {
                        const float2 v = s.ml[w + k * C::RW][r * 16 + n16];
                        const float mn = fmaxf(m[r], v.x), f = exp2_(m[r] - mn), f2 = exp2_(v.x - mn);
                        m[r] = mn;
                        l[r] = l[r] * f + v.y * f2;
#pragma unroll
                        for (int d = 0; d < DB; ++d) o[r][d] = o[r][d] * f + *at(k, r, d) * f2;
                    }
            }
        }
        if (kw > 0) return;
#pragma unroll
        for (int r = 0; r < RG; ++r) {
            int tok, t, g;
            if (!row_of(tag, p, rw * RG + r, tok, t, g)) continue;
            if (p.slot < 0) {
                const size_t at = (size_t)tok * a.Hq + p.h * G + g;
                const float inv = inverse_of(l[r], m[r]);
#pragma unroll
                for (int d = 0; d < DB; ++d) {
                    const f32x4_t y = o[r][d] * inv;
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
                const size_t row = (size_t)p.slot * C::M + (rw * RG + r) * 16 + n16;
                float* po = reinterpret_cast<float*>(const_cast<char*>(s.base[window])) + row * C::D;
#pragma unroll
                for (int d = 0; d < DB; ++d) *reinterpret_cast<f32x4_t*>(po + (dw * DB + d) * 16 + 4 * grp) = o[r][d];
                if (dw == 0 && grp == 0)
                    reinterpret_cast<float2*>(const_cast<char*>(s.base[2 + window]))[row] = make_float2(m[r], l[r]);
            }
        }
    };

    // the first tile and q of a piece that no other one brought
    auto start = [&](auto tag, const Piece p) {
        load_ids(p);
        load_piece(p);
        issue(0);
        if constexpr (!tag.shared) load_parent(p);
        load_q(tag, p);
    };

    Ref at{uni(s.found_b), uni(s.found_off), own_u, 0};
    // the next own piece that has a tile; false: there is none
    auto next_own = [&](Piece& p) {
        while (at.u < uni(s.own_u1)) {
            const Seq q = seq_at(at.b);
            if (at.off >= q.segs * (q.tiles + uni(s.extra))) {
                at.off = 0;
                ++at.b;
                continue;
            }
            p = piece_of(OwnTag{}, at);
            if (p.tiles > 0) return true;
        }
        return false;
    };
    Piece own_piece{};
    bool more = next_own(own_piece), started = false;
    auto shared_list = [&](const bool then_own) {
        if constexpr (kShared) {
            for (int it = lb; it < items; it += blocks) {
                // the tile's tokens
                const int r0 = it % row_tiles * SH::M, t0 = r0 / G;
                const int t1 = min((r0 + SH::M - 1) / G + 1, tok_total);
                __syncthreads();   // nobody reads the tokens of the item before, nor its last tile
                int tok = s.tok_base[threadIdx.x];
                const int f0 = min((int)threadIdx.x * per, a.B), f1 = min(f0 + per, a.B);
                for (int b = f0; b < f1 && tok < t1; ++b) {
                    const Seq q = seq_of(a, b, N, OW::M);
                    if (!q.part) continue;
                    for (int t = max(0, t0 - tok); t < q.cnt && tok + t < t1; ++t) s.tok[tok + t - t0] = b * a.K + t;
                    tok += q.cnt;
                }
                __syncthreads();
                Ref item{0, 0, 0, it};
                const Piece now = piece_of(SharedTag{}, item);
                start(SharedTag{}, now);
                // (the item after needs the tokens' place for its own, so it is not brought; the own part is)
                started = then_own && more && it + blocks >= items;
                run(SharedTag{}, now, started, own_piece);
            }
        }
    };
    auto own_list = [&] {
        if (more && !started) start(OwnTag{}, own_piece);
#pragma nounroll
        while (more) {
            Piece n{};
            const bool then = next_own(n);
            run(OwnTag{}, own_piece, then, n);
            own_piece = n;
            more = then;
        }
    };
    if constexpr (kShared && OW::BF16 && OW::M <= 32) {
        // Half of the workgroups, one of a CU's two, take the lists the other way round: the shared one is bound by
        // matrix products and vector work, the own one by memory where its tiles have few rows, so that each has the
        // other beside it (64 single tokens behind 32768 shared keys 116 to 108 us; with 64-row own tiles it cost 2-3%).
        const bool own_first = blockIdx.x >> 8 & 1;
#pragma nounroll
        for (int pass = 0; pass < 2; ++pass) {
            if ((pass == 0) != own_first) shared_list(!own_first);
            else own_list();
        }
    } else {
        shared_list(true);
        own_list();
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
    const char* work = static_cast<const char*>(a.work);
    bool mine = row < (long long)a.B * a.K * a.Hq;
    if (mine) {
        const int G = a.G;
        const int tok = (int)row / a.Hq, hq = (int)row - tok * a.Hq;   // (below 2^28 rows)
        const int b = tok / a.K, t = tok - b * a.K, h = hq / G, g = hq - h * G;
        const Head head = *reinterpret_cast<const Head*>(work);
        const PlanSeq plan = reinterpret_cast<const PlanSeq*>(work + a.at.plan)[b];
        const Seq q = seq_of(a, b, N, MO);
        mine = t < q.cnt;
        if (mine && plan.tok_base >= 0) {
            const int r = (plan.tok_base + t) * G + g, rt = r >> __builtin_ctz(MS);
            n_s = head.splits;
            at_s = ((size_t)h * head.splits * head.row_tiles + rt) * MS + (r - rt * MS);
            step_s = (size_t)head.row_tiles * MS;
        }
        if (mine && q.tiles > 0) {
            const RowTiles rts_of = row_tiles_of(a, MO);
            const int r = t * G + g, rt = r >> __builtin_ctz(MO);
            const int rt_list = a.listed ? rt : 0, rt_block = a.listed ? 0 : rt;
            const int u = plan.own_base + (h * (a.listed ? q.rts : 1) + rt_list) * (q.tiles + head.own_extra) + head.own_extra;
            const int p0 = part_of(head.own_units, head.own_parts, u);
            n_o = part_of(head.own_units, head.own_parts, u + q.tiles - 1) - p0 + 1;
            const size_t slot =
                ((size_t)p0 + ((size_t)b * a.Hkv + h) * rts_of.in_list + rt_list) * rts_of.grouped + rt_block;
            at_o = slot * MO + (r - rt * MO);
            step_o = (size_t)rts_of.grouped * MO;
            if (n_o == 1 && !q.part) mine = false;   // written by its one piece
        }
    }
    const float2* ml_s = reinterpret_cast<const float2*>(work + a.at.ml_s) + at_s;
    const float2* ml_o = reinterpret_cast<const float2*>(work + a.at.ml_o) + at_o;
    const f32x4_t* o_s = reinterpret_cast<const f32x4_t*>(work + a.at.o_s) + at_s * C4 + c4;
    const f32x4_t* o_o = reinterpret_cast<const f32x4_t*>(work + a.at.o_o) + at_o * C4 + c4;
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
    const f32x4_t y = acc * inverse_of(L, M);
    if constexpr (BF16)
        reinterpret_cast<uint2*>(a.o)[unit] = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
    else
        reinterpret_cast<f32x4_t*>(a.o)[unit] = y;
    if (a.lse && c4 == 0) a.lse[row] = L == 0.f ? -INFINITY : (M + __log2f(L)) * kLn2;
}

}  // namespace attn
}  // namespace gdn
