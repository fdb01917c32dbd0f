// gdn_kv.hip -- the paged key/value cache: pages taken (reserve), windows
// written (append), cut back to an accepted tree path (rollback), and pages
// freed, forked, compacted and copied (include/gdn.h states each call).
//
// Two kinds of kernel.  Those that decide which page goes where (reserve, fork,
// compact) are one workgroup: their answer is a running count over all pages
// and all sequences, a few kilobytes of int32, and one workgroup needs no
// second launch and no cross-workgroup order; what it costs is the latency of its
// dependent reads, about 0.7 us each (reserve 2.8 to 3.2 us, fork and the plan of a
// compaction 5 us).  Those that move bytes (append, rollback, page
// copies) spread 16-byte pieces over the chip.
#include "gdn_device.h"
#include "gdn_kv_internal.h"

namespace gdn {
namespace {

constexpr int kCtl = 1024;            // threads of a deciding workgroup
constexpr int kCtlWaves = kCtl / 64;
constexpr int kScanPer = 4;           // pages per thread and scan step
constexpr int kScan = kCtl * kScanPer;

__device__ __forceinline__ int clamp_count(const int32_t* count, int b, int K)
{
    return count ? min(max(count[b], 0), K) : K;
}

__device__ __forceinline__ bool held(int id, int n_pages) { return (unsigned)id < (unsigned)n_pages; }

// inclusive sum over the lanes of a wave
__device__ __forceinline__ int wave_scan(int v)
{
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int u = __shfl_up(v, d, 64);
        if (lane >= d) v += u;
    }
    return v;
}

// exclusive sum over the kCtl threads of a deciding workgroup; `total` gets the sum of all.
// Every thread calls it (two barriers); `part` is kCtlWaves words of LDS.
__device__ __forceinline__ int block_scan(int v, int* part, int& total)
{
    const int lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    const int inc = wave_scan(v);
    __syncthreads();  // part may still be read from the scan before
    if (lane == 63) part[w] = inc;
    __syncthreads();
    int base = 0, sum = 0;
#pragma unroll
    for (int i = 0; i < kCtlWaves; ++i) {
        const int p = part[i];
        base += i < w ? p : 0;
        sum += p;
    }
    total = sum;
    return base + inc - v;
}

// The pages in ascending steps of kScan, kScanPer consecutive ones a thread.  The first step (all there is, for most
// pools) is read once, when the kernel starts, and kept; the reads of later ones are repeated.
struct PageScan {
    const int32_t* ref;
    int n;
    int first[kScanPer];

    __device__ __forceinline__ PageScan(const int32_t* r, int n_pages) : ref(r), n(n_pages)
    {
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) {
            const int p = (int)threadIdx.x * kScanPer + i;
            first[i] = p < n ? ref[p] : 1;
        }
    }
    // a bit for each of this thread's pages of the step at `at` whose ref satisfies pred(page, ref)
    template <typename F>
    __device__ __forceinline__ unsigned bits(int at, F pred) const
    {
        unsigned b = 0;
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) {
            const int p = at + (int)threadIdx.x * kScanPer + i;
            if (p < n && pred(p, at == 0 ? first[i] : ref[p])) b |= 1u << i;
        }
        return b;
    }
    __device__ __forceinline__ unsigned free_bits(int at) const
    {
        return bits(at, [](int, int r) { return r == 0; });
    }
    // number of free pages, at most about `enough` (counting stops once it is reached)
    __device__ __forceinline__ int count_free(int enough, int* part) const
    {
        int have = 0;
        for (int at = 0; at < n && have < enough; at += kScan) {
            int step;
            block_scan(__popc(free_bits(at)), part, step);
            have += step;
        }
        return have;
    }
};

// ---------------------------------------------------------------- reserve
// slots of a sequence's window: [s0, s1); false where it asks for nothing or passes the table
__device__ __forceinline__ bool window_of(const KvReserveArgs& a, int lens, int wants, int& s0, int& s1)
{
    const long long len = max(lens, 0), add = wants;
    s0 = s1 = 0;
    if (add <= 0 || ((len + add - 1) >> a.page_log2) >= a.P) return false;
    s0 = (int)(len >> a.page_log2);
    s1 = (int)((len + add - 1) >> a.page_log2) + 1;
    return true;
}

// For up to kCtl sequences and kScan pages: a thread has one sequence and kScanPer pages, which are read once and kept,
// and wants and free pages are numbered in one scan (two rounds of reads in all, 2.8 to 3.1 us for one sequence; the general
// kernel below, with five, takes 4.9).
constexpr int kSlots = 4;   // slots of a window that are kept (more are read again)

__global__ __launch_bounds__(kCtl) void kv_reserve_small_kernel(KvReserveArgs a)
{
    __shared__ int2 part[kCtlWaves];
    __shared__ int ids[kScan];
    const PageScan pages(a.ref, a.n_pages);
    const int b = threadIdx.x, lane = threadIdx.x & 63, w = threadIdx.x >> 6;
    int add = 0, s0 = 0, s1 = 0, need = 0;
    bool any = false;
    unsigned empty = 0;
    int32_t* row = a.table + (size_t)b * a.P;
    if (b < a.B) {
        const int len = a.lens[b];
        add = a.add[b];
        any = window_of(a, len, add, s0, s1);
        int id[kSlots];
#pragma unroll
        for (int i = 0; i < kSlots; ++i) id[i] = s0 + i < s1 ? row[s0 + i] : 0;
#pragma unroll
        for (int i = 0; i < kSlots; ++i)
            if (s0 + i < s1 && !held(id[i], a.n_pages)) empty |= 1u << i;
        need = __popc(empty);
        for (int s = s0 + kSlots; s < s1; ++s) need += !held(row[s], a.n_pages);
        need = min(need, a.n_pages + 1);   // (more is as good, and keeps the sum in 32 bits)
    }
    const unsigned bits = pages.free_bits(0);
    const int inc = wave_scan(need), inc_free = wave_scan(__popc(bits));
    if (lane == 63) part[w] = make_int2(inc, inc_free);
    __syncthreads();
    int base = inc - need, r = inc_free - __popc(bits), have = 0;
#pragma unroll
    for (int i = 0; i < kCtlWaves; ++i) {
        const int2 p = part[i];
        base += i < w ? p.x : 0;
        r += i < w ? p.y : 0;
        have += p.y;
    }
#pragma unroll
    for (int i = 0; i < kScanPer; ++i)
        if (bits >> i & 1) ids[r++] = (int)threadIdx.x * kScanPer + i;
    __syncthreads();
    if (b >= a.B) return;
    const bool fits = any && (need == 0 || base + need <= have);
    a.granted[b] = fits ? add : 0;
    if (!fits || need == 0) return;
    int next = base;
    for (int s = s0; s < s1; ++s) {
        const int i = s - s0;
        if (i < kSlots ? !(empty >> i & 1) : held(row[s], a.n_pages)) continue;
        const int id = ids[next++];
        row[s] = id;
        a.ref[id] = 1;
    }
}

// Any number of them.  Thread i owns a run of consecutive sequences; their wants are numbered by an
// exclusive sum, the free pages by another, and want r takes free page r.
__global__ __launch_bounds__(kCtl) void kv_reserve_kernel(KvReserveArgs a)
{
    __shared__ int part[kCtlWaves];
    __shared__ int ids[kScan];
    const PageScan pages(a.ref, a.n_pages);
    const int per = (a.B + kCtl - 1) / kCtl;
    const int b0 = min((int)threadIdx.x * per, a.B), b1 = min(b0 + per, a.B);

    auto window = [&](int b, int& s0, int& s1) { return window_of(a, a.lens[b], a.add[b], s0, s1); };
    auto need_of = [&](int b, int s0, int s1) {
        int n = 0;
        for (int s = s0; s < s1; ++s) n += !held(a.table[(size_t)b * a.P + s], a.n_pages);
        return n;
    };

    int need = 0;
    for (int b = b0; b < b1; ++b) {
        int s0, s1;
        // more than there are pages is as good as any larger number, and keeps the block's sum in 32 bits
        if (window(b, s0, s1)) need = min(need + min(need_of(b, s0, s1), a.n_pages + 1), a.n_pages + 1);
    }
    int total;
    const int base = block_scan(need, part, total);
    const int have = pages.count_free(total, part);

    // grants, and where this thread's wants end: the first sequence that does not fit stops all later
    // ones that need a page, so the granted wants are ranks base .. last-1
    long long rank = base;
    int last = base;
    for (int b = b0; b < b1; ++b) {
        int s0, s1;
        const bool any = window(b, s0, s1);
        const int n = any ? need_of(b, s0, s1) : 0;
        rank += n;
        const bool fits = any && (n == 0 || rank <= have);
        a.granted[b] = fits ? a.add[b] : 0;
        if (n > 0 && fits) last = (int)rank;
    }

    int b = b0, s = -1, s0 = 0, s1 = 0, next = base, seen = 0;
    for (int at = 0; at < a.n_pages && seen < min(total, have); at += kScan) {
        const unsigned bits = pages.free_bits(at);
        int step, r = block_scan(__popc(bits), part, step);
#pragma unroll
        for (int i = 0; i < kScanPer; ++i)
            if (bits >> i & 1) ids[r++] = at + (int)threadIdx.x * kScanPer + i;
        __syncthreads();
        while (next < last && next < seen + step) {
            if (s < 0) {  // the next sequence's window
                if (!window(b, s0, s1)) {
                    ++b;
                    continue;
                }
                s = s0;
            }
            for (; s < s1 && next < last && next < seen + step; ++s) {
                int32_t* slot = a.table + (size_t)b * a.P + s;
                if (held(*slot, a.n_pages)) continue;
                const int id = ids[next - seen];
                *slot = id;
                a.ref[id] = 1;
                ++next;
            }
            if (s == s1) {
                ++b;
                s = -1;
            }
        }
        seen += step;
    }
}

// ---------------------------------------------------------------- append
// A thread per 16 bytes of one token and head, of both K and V.
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a)
{
    const int b = blockIdx.y;
    const int per_row = a.g.row_bytes >> 4, per_token = a.g.Hkv * per_row;
    const int i = blockIdx.x * 256 + threadIdx.x;
    const int t = i / per_token, c = i - t * per_token;
    if (t >= clamp_count(a.count, b, a.K)) return;
    const long long at = (long long)max(a.lens[b], 0) + t;
    const long long slot = at >> a.g.page_log2;
    if (slot >= a.P) return;
    const int id = a.table[(size_t)b * a.P + slot];
    if (!held(id, a.g.n_pages)) return;
    const int h = c / per_row, x = c - h * per_row;
    const int in_page = (int)(at & ((1 << a.g.page_log2) - 1));
    const size_t to = ((((size_t)id * a.g.Hkv + h) << a.g.page_log2) + in_page) * a.g.row_bytes + (size_t)x * 16;
    const size_t from = ((size_t)b * a.K + t) * a.token_bytes + (size_t)c * 16;
    const uint4 k = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.k) + from);
    const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const char*>(a.v) + from);
    *reinterpret_cast<uint4*>(static_cast<char*>(a.k_pages) + to) = k;
    *reinterpret_cast<uint4*>(static_cast<char*>(a.v_pages) + to) = v;
}

// ---------------------------------------------------------------- rollback
// The nodes on the path root..i as a bit mask, in lane i: by doubling, a lane holding what
// it has found above its node and the node to go on from.  Called by a whole wave.
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

constexpr int kMoveBatch = 8;
constexpr long long kForkAtOnce = 32 * 1024;   // bytes of pages that kv_fork copies in its one workgroup

// what a sequence keeps of its window
struct Kept {
    unsigned long long path;
    long long len;
    // the new length: a length has 31 bits, also where the window reaches past them (wrapped, it would be a slot in
    // front of the row)
    __device__ __forceinline__ long long after() const { return min(len + __popcll(path), 0x7fffffffll); }
};

__device__ __forceinline__ Kept kept_of(const KvRollbackArgs& a, int b)
{
    const int n = a.node[b], live = clamp_count(a.count, b, a.N);
    Kept k;
    k.len = max(a.lens[b], 0);
    // (every lane's path, also where none is kept: parent and node are then read at the same time)
    const unsigned long long path = __shfl(node_paths(a.parent ? a.parent + (size_t)b * a.N : nullptr, a.N), n & 63, 64);
    k.path = n >= 0 && n < live ? path : 0;
    return k;
}

// The table row of a sequence in LDS, read when the kernel starts, beside the lengths and the tree: a read that waits
// for another costs these kernels most (a step of 64 sequences and 8 layers took 23.2 us with the row read after the
// length and again after the moves, and takes 20.5 to 21.5; one layer of one sequence gains less, 5.1 to 5.3 us of 5.4).
// Longer rows are read from memory where they are needed.
constexpr int kRow = 2048;

struct Row {
    const int32_t* row;
    int P;
    const int32_t* staged;   // (nullptr: not staged)

    __device__ __forceinline__ int at(long long slot) const
    {
        if (slot >= P) return -1;
        return staged ? staged[slot] : row[slot];
    }
};

__device__ __forceinline__ Row stage_row(const KvRollbackArgs& a, int b, int32_t* lds)
{
    Row r{a.table + (size_t)b * a.P, a.P, nullptr};
    if (a.P <= kRow) {
        for (int s = threadIdx.x; s < a.P; s += blockDim.x) lds[s] = r.row[s];
        r.staged = lds;
    }
    return r;
}

// Moves the kept tokens of sequence b: this workgroup's threads take the 16-byte pieces first, first + step, .. of
// all planes and heads.  A path's i-th node has an index >= i, so a thread that owns a piece and moves the path in
// order never overwrites what it has yet to read; it reads a batch before it writes it.
__device__ __forceinline__ void move_kept(const KvRollbackArgs& a, const Kept& k, const Row& row, int first, int step)
{
    __shared__ int from_id[kKvWindowMax], to_id[kKvWindowMax], from_row[kKvWindowMax], to_row[kKvWindowMax];
    const int lane = threadIdx.x & 63, kept = __popcll(k.path);
    const int mask = (1 << a.g.page_log2) - 1;
    __syncthreads();   // the row is there
    if (threadIdx.x < 64 && (k.path >> lane & 1)) {
        const int i = __popcll(k.path & ((1ull << lane) - 1));
        const long long from = k.len + lane, to = k.len + i;
        const int f = row.at(from >> a.g.page_log2), t = row.at(to >> a.g.page_log2);
        const bool move = i != lane && held(f, a.g.n_pages) && held(t, a.g.n_pages);
        from_id[i] = move ? f : -1;
        to_id[i] = t;
        from_row[i] = (int)from & mask;
        to_row[i] = (int)to & mask;
    }
    __syncthreads();

    const int per_row = a.g.row_bytes >> 4;
    const int pieces = a.g.planes * a.g.Hkv * per_row;
    const size_t plane = (size_t)a.g.n_pages * ((size_t)a.g.Hkv << a.g.page_log2) * a.g.row_bytes;
    for (int e = first; e < pieces; e += step) {
        const int x = e % per_row, ph = e / per_row;
        const int h = ph % a.g.Hkv, pl = ph / a.g.Hkv;
        char* at = static_cast<char*>(a.pool) + pl * plane + (size_t)x * 16;
        auto addr = [&](int id, int r) {
            return reinterpret_cast<uint4*>(at + ((((size_t)id * a.g.Hkv + h) << a.g.page_log2) + r) * a.g.row_bytes);
        };
        for (int i0 = 0; i0 < kept; i0 += kMoveBatch) {
            uint4 u[kMoveBatch];
#pragma unroll
            for (int j = 0; j < kMoveBatch; ++j)
                if (i0 + j < kept && from_id[i0 + j] >= 0) u[j] = *addr(from_id[i0 + j], from_row[i0 + j]);
#pragma unroll
            for (int j = 0; j < kMoveBatch; ++j)
                if (i0 + j < kept && from_id[i0 + j] >= 0) *addr(to_id[i0 + j], to_row[i0 + j]) = u[j];
        }
    }
}

// Gives back the pages behind what sequence b keeps.
__device__ __forceinline__ void cut_row(const KvRollbackArgs& a, int b, long long after, const Row& row)
{
    const int mask = (1 << a.g.page_log2) - 1;
    for (long long s = ((after + mask) >> a.g.page_log2) + threadIdx.x; s < a.P; s += blockDim.x) {
        const int id = row.at(s);
        if (held(id, a.g.n_pages)) {
            atomicSub(a.ref + id, 1);
            a.table[(size_t)b * a.P + s] = -1;
        }
    }
    if (threadIdx.x == 0) a.lens_out[b] = (int32_t)after;
}

// A workgroup per sequence: every token moved, then the row cut.
__global__ __launch_bounds__(kCtl) void kv_rollback_kernel(KvRollbackArgs a)
{
    __shared__ int32_t lds[kRow];
    const int b = blockIdx.x;
    const Row row = stage_row(a, b, lds);
    const Kept k = kept_of(a, b);
    move_kept(a, k, row, threadIdx.x, blockDim.x);
    __syncthreads();   // (a row that is not staged, and lens, which lens_out may be, have been read)
    cut_row(a, b, k.after(), row);
}

// The two halves on their own, for more planes than a workgroup moves at once: many workgroups a sequence read its
// row, so it may be cut only after the last of them.
__global__ __launch_bounds__(256) void kv_move_kernel(KvRollbackArgs a)
{
    __shared__ int32_t lds[kRow];
    const Row row = stage_row(a, blockIdx.y, lds);
    const Kept k = kept_of(a, blockIdx.y);
    // the new length, for kv_cut_kernel (unless it would overwrite what other workgroups read)
    if (a.lens_out != a.lens && blockIdx.x == 0 && threadIdx.x == 0)
        a.lens_out[blockIdx.y] = (int32_t)k.after();
    move_kept(a, k, row, blockIdx.x * 256 + threadIdx.x, gridDim.x * 256);
}

__global__ __launch_bounds__(64) void kv_cut_kernel(KvRollbackArgs a)
{
    __shared__ int32_t lds[kRow];
    const Row row = stage_row(a, blockIdx.x, lds);
    long long after;
    if (a.lens_out != a.lens) {
        after = a.lens_out[blockIdx.x];
    } else {
        after = kept_of(a, blockIdx.x).after();
    }
    __syncthreads();   // (lens has been read, and the row is there)
    cut_row(a, blockIdx.x, after, row);
}

// ---------------------------------------------------------------- free
__global__ __launch_bounds__(256) void kv_free_kernel(const int32_t* rows, int32_t* lens, int32_t* table, int32_t* ref,
                                                      int B, int P, int n_pages)
{
    const int b = rows[blockIdx.x];
    if (!held(b, B)) return;
    for (int s = threadIdx.x; s < P; s += 256) {
        const int id = atomicExch(table + (size_t)b * P + s, -1);  // a row named twice gives each page back once
        if (held(id, n_pages)) atomicSub(ref + id, 1);
    }
    if (threadIdx.x == 0) lens[b] = 0;
}

// ---------------------------------------------------------------- page copies
// 16-byte pieces of the pages src -> dst of every plane; a workgroup takes
// kCopyPer pieces of a thread at a time and walks on until all are done.  Memory
// bounds it: 900 pages of 32 KB in 4 planes, 118 MB read and as much written, take 58 us from a pool of 7.9 GB
// (4.1 TB/s, a large plain copy reaches 5.2) and 37 to 38 us again and again, when they stay in the last cache.
// Stores past the caches took 36 us in the second case but 40 instead of 38 where 32 copies
// of one page are made, loads past them 40 and 47; 8 pieces a thread or other grids the same.
// Small pages are far from that: a chunk never crosses a page, so 500 pages of 2 KB in 16
// planes, 33 MB read and written, take 23 us (1.4 TB/s).
constexpr int kCopyPer = 4;
constexpr int kCopyChunk = 256 * kCopyPer;   // pieces a workgroup moves in one go
constexpr int kCopyGrid = 256 * 8;           // workgroups that fill the chip
// 1 / chunks and the product are rounded, so a quotient is off by 2^-52 of itself, and half a step from the next integer
constexpr long long kCopyExact = 1LL << 50;

template <typename F>
__device__ __forceinline__ void copy_pages(char* pool, const KvGeom& g, long long n, F pair)
{
    const long long pieces = (long long)(g.page_bytes() >> 4);
    const long long chunks = (pieces + kCopyChunk - 1) / kCopyChunk, all = n * g.planes * chunks;
    const size_t bytes = g.page_bytes();
    const double by_chunks = 1.0 / chunks, by_planes = 1.0 / g.planes;
    for (long long w = blockIdx.x; w < all; w += gridDim.x) {
        // quotients by doubles: exact below kCopyExact, at a tenth of an integer division's time
        const long long r = (long long)(((double)w + 0.5) * by_chunks), c = w - r * chunks;
        const long long i = (long long)(((double)r + 0.5) * by_planes), pl = r - i * g.planes;
        int from, to;
        if (!pair(i, from, to)) continue;
        const uint4* s = reinterpret_cast<const uint4*>(pool + (pl * g.n_pages + from) * bytes);
        uint4* d = reinterpret_cast<uint4*>(pool + (pl * g.n_pages + to) * bytes);
        const long long e = c * kCopyChunk + threadIdx.x;
        uint4 u[kCopyPer];
#pragma unroll
        for (int i = 0; i < kCopyPer; ++i)
            if (e + i * 256 < pieces) u[i] = s[e + i * 256];
#pragma unroll
        for (int i = 0; i < kCopyPer; ++i)
            if (e + i * 256 < pieces) d[e + i * 256] = u[i];
    }
}

int copy_grid(long long n, const KvGeom& g)
{
    const long long chunks = ((long long)(g.page_bytes() >> 4) + kCopyChunk - 1) / kCopyChunk;
    const long long all = n * g.planes * chunks;
    return (int)(all < kCopyGrid ? (all > 0 ? all : 1) : kCopyGrid);
}

__global__ __launch_bounds__(256) void kv_copy_kernel(const int32_t* src, const int32_t* dst, char* pool, int n,
                                                      KvGeom g)
{
    copy_pages(pool, g, n, [&](long long i, int& from, int& to) {
        from = src[i];
        to = dst[i];
        return held(from, g.n_pages) && held(to, g.n_pages) && from != to;
    });
}

// ---------------------------------------------------------------- fork
// Which forks can be made, their new pages, and the rows; with COPY the pages too, by this one workgroup.
template <bool COPY>
__global__ __launch_bounds__(kCtl) void kv_fork_kernel(KvForkArgs a)
{
    __shared__ int from_of[COPY ? kKvForkMax : 1];
    __shared__ int part[kCtlWaves];
    __shared__ int ids[kScan];
    __shared__ int page_of[kKvForkMax];          // -2 refused, -1 no new page, else its rank, then its id
    const PageScan pages(a.ref, a.g.n_pages);
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const int page = 1 << a.g.page_log2;
    auto length = [&](int i) { return max(a.lens[a.src[i]], 0); };

    // can be made, but for the number of free pages: a wave looks over a fork's two rows
    for (int i = wave; i < a.n; i += kCtlWaves) {
        const int src = a.src[i], dst = a.dst[i];
        bool fine = held(src, a.B) && held(dst, a.B) && src != dst;
        bool tail = false;
        if (fine) {
            const long long len = length(i);
            const long long slots = (len + page - 1) >> a.g.page_log2;
            fine = slots <= a.P;
            tail = (len & (page - 1)) != 0;
            bool bad = false;
            for (int s = lane; s < a.P; s += 64) {
                bad |= held(a.table[(size_t)dst * a.P + s], a.g.n_pages);
                bad |= s < slots && !held(a.table[(size_t)src * a.P + s], a.g.n_pages);
            }
            fine = fine && __ballot(bad) == 0;
        }
        if (lane == 0) page_of[i] = !fine ? -2 : (tail ? 0 : -1);
    }
    __syncthreads();
    const int per = (a.n + kCtl - 1) / kCtl;
    const int i0 = min((int)threadIdx.x * per, a.n), i1 = min(i0 + per, a.n);
    int need = 0;
    for (int i = i0; i < i1; ++i) need += page_of[i] == 0;
    int total, rank = block_scan(need, part, total);
    const int have = pages.count_free(total, part);
    for (int i = i0; i < i1; ++i)
        if (page_of[i] == 0) {
            page_of[i] = rank < have ? rank : -2;
            ++rank;
        }
    // ranks to ids
    int next = i0, seen = 0;
    for (int at = 0; at < a.g.n_pages && seen < min(total, have); at += kScan) {
        const unsigned bits = pages.free_bits(at);
        int step, r = block_scan(__popc(bits), part, step);
#pragma unroll
        for (int i = 0; i < kScanPer; ++i)
            if (bits >> i & 1) ids[r++] = at + (int)threadIdx.x * kScanPer + i;
        __syncthreads();
        for (; next < i1; ++next) {
            if (page_of[next] < 0) continue;
            if (page_of[next] >= seen + step) break;
            page_of[next] = ids[page_of[next] - seen];
        }
        seen += step;
    }
    __syncthreads();
    // the rows
    for (int i = wave; i < a.n; i += kCtlWaves) {
        const int id = page_of[i];
        if (lane == 0) a.granted[i] = id != -2;
        if (id == -2) continue;
        const int src = a.src[i], dst = a.dst[i], len = length(i);
        const int full = len >> a.g.page_log2;
        if (COPY && lane == 0) from_of[i] = id >= 0 ? a.table[(size_t)src * a.P + full] : -1;
        for (int s = lane; s < a.P; s += 64) {
            int to = -1;
            if (s < full) {
                to = a.table[(size_t)src * a.P + s];
                if (held(to, a.g.n_pages)) atomicAdd(a.ref + to, 1);
            } else if (s == full && id >= 0) {
                to = id;
                a.ref[id] = 1;
            }
            a.table[(size_t)dst * a.P + s] = to;
        }
        if (lane == 0) a.lens[dst] = len;
    }
    if constexpr (COPY) {
        __syncthreads();
        const size_t bytes = a.g.page_bytes();
        const int pieces = (int)(bytes >> 4), all = a.n * a.g.planes * pieces;   // (at most kForkAtOnce / 16)
        char* pool = static_cast<char*>(a.pool);
        for (int e0 = threadIdx.x; e0 < all; e0 += kCtl * kMoveBatch) {
            uint4 u[kMoveBatch];
            uint4* to[kMoveBatch];
#pragma unroll
            for (int j = 0; j < kMoveBatch; ++j) {
                const int e = e0 + j * kCtl, r = e / pieces, c = e - r * pieces, i = r / a.g.planes, pl = r - i * a.g.planes;
                to[j] = nullptr;
                if (e < all && page_of[i] >= 0 && held(from_of[i], a.g.n_pages)) {
                    char* plane = pool + (size_t)pl * a.g.n_pages * bytes;
                    to[j] = reinterpret_cast<uint4*>(plane + page_of[i] * bytes) + c;
                    u[j] = reinterpret_cast<const uint4*>(plane + from_of[i] * bytes)[c];
                }
            }
#pragma unroll
            for (int j = 0; j < kMoveBatch; ++j)
                if (to[j]) *to[j] = u[j];
        }
    }
}

__global__ __launch_bounds__(256) void kv_fork_copy_kernel(KvForkArgs a)
{
    copy_pages(static_cast<char*>(a.pool), a.g, a.n, [&](long long i, int& from, int& to) {
        const int granted = a.granted[i], src = a.src[i], dst = a.dst[i];
        if (!granted) return false;
        const int len = max(a.lens[src], 0), full = len >> a.g.page_log2;
        if ((len & ((1 << a.g.page_log2) - 1)) == 0 || full >= a.P) return false;
        from = a.table[(size_t)src * a.P + full];
        to = a.table[(size_t)dst * a.P + full];
        return held(from, a.g.n_pages) && held(to, a.g.n_pages);
    });
}

// ---------------------------------------------------------------- compact
// work: [0] moves, then the moves' sources, their destinations, and the new id of every page
__host__ __device__ inline int32_t* compact_from(int32_t* w) { return w + 4; }
__host__ __device__ inline int32_t* compact_to(int32_t* w, int n) { return w + 4 + (n + 1) / 2; }
__host__ __device__ inline int32_t* compact_map(int32_t* w, int n) { return w + 4 + 2 * ((n + 1) / 2); }

// The holes below U and the pages in use above it, both in ascending order.
// There are as many of one as of the other, at most n_pages / 2.
__global__ __launch_bounds__(kCtl) void kv_compact_plan_kernel(KvCompactArgs a)
{
    __shared__ int part[kCtlWaves];
    const int n = a.g.n_pages;
    const PageScan pages(a.ref, n);
    int32_t *from = compact_from(a.work), *to = compact_to(a.work, n), *map = compact_map(a.work, n);
    int used = 0;
    for (int at = 0; at < n; at += kScan) {
        int step;
        block_scan(__popc(pages.bits(at, [](int, int r) { return r > 0; })), part, step);
        used += step;
    }
    int holes = 0, moves = 0;
    for (int at = 0; at < n; at += kScan) {
        // a page is a hole or a move or neither: both counts in one scan, 16 bits each (a step has 4096 pages)
        const unsigned hole = pages.bits(at, [&](int p, int r) { return p < used && !(r > 0); });
        const unsigned move = pages.bits(at, [&](int p, int r) { return p >= used && r > 0; });
        int step;
        const int both = block_scan(__popc(hole) | __popc(move) << 16, part, step);
        int h = holes + (both & 0xffff), m = moves + (both >> 16);
#pragma unroll
        for (int i = 0; i < kScanPer; ++i) {
            const int p = at + (int)threadIdx.x * kScanPer + i;
            if (hole >> i & 1) to[h++] = p;
            if (move >> i & 1) from[m++] = p;
            if (p < n) {
                map[p] = p;
                a.ref_out[p] = p < used && !(hole >> i & 1) ? (at == 0 ? pages.first[i] : a.ref[p]) : 0;
            }
        }
        holes += step & 0xffff;
        moves += step >> 16;
    }
    __syncthreads();
    for (int k = threadIdx.x; k < moves; k += kCtl) {
        map[from[k]] = to[k];
        a.ref_out[to[k]] = a.ref[from[k]];
    }
    if (threadIdx.x == 0) a.work[0] = moves;
}

__global__ __launch_bounds__(256) void kv_compact_kernel(KvCompactArgs a)
{
    const int n = a.g.n_pages;
    const int32_t *from_of = compact_from(a.work), *to_of = compact_to(a.work, n), *map = compact_map(a.work, n);
    for (long long e = (long long)blockIdx.x * 256 + threadIdx.x; e < a.entries; e += (long long)gridDim.x * 256) {
        const int id = a.table[e];
        a.table_out[e] = held(id, n) ? map[id] : id;
    }
    copy_pages(static_cast<char*>(a.pool), a.g, a.work[0], [&](long long i, int& from, int& to) {
        from = from_of[i];
        to = to_of[i];
        return true;
    });
}

}  // namespace

bool kv_copy_countable(long long n, const KvGeom& g)
{
    const long long chunks = ((long long)(g.page_bytes() >> 4) + kCopyChunk - 1) / kCopyChunk;
    return n <= kCopyExact / (g.planes * chunks);
}

size_t kv_compact_words(int n_pages) { return 4 + 2 * (((size_t)n_pages + 1) / 2) + (size_t)n_pages; }

hipError_t launch_kv_reserve(const KvReserveArgs& a, hipStream_t s)
{
    if (a.B <= kCtl && a.n_pages <= kScan)
        kv_reserve_small_kernel<<<dim3(1), dim3(kCtl), 0, s>>>(a);
    else
        kv_reserve_kernel<<<dim3(1), dim3(kCtl), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s)
{
    const long long pieces = (long long)a.K * a.g.Hkv * (a.g.row_bytes >> 4);
    kv_append_kernel<<<dim3((unsigned)((pieces + 255) / 256), a.B), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_rollback(const KvRollbackArgs& a, hipStream_t s)
{
    // One launch up to kCtl pieces a sequence, two above: 16 planes of 64 sequences took 25.6 us in one (64 workgroups
    // with two pieces a thread), 14 us in two; one layer of one sequence takes 5.1 to 5.3 us in one.
    const int pieces = a.g.planes * a.g.Hkv * (a.g.row_bytes >> 4);
    if (pieces <= kCtl) {
        kv_rollback_kernel<<<dim3(a.B), dim3(pieces <= 256 ? 256 : kCtl), 0, s>>>(a);
        return hipGetLastError();
    }
    kv_move_kernel<<<dim3((pieces + 255) / 256, a.B), dim3(256), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    kv_cut_kernel<<<dim3(a.B), dim3(64), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_free(const int32_t* rows, int32_t* lens, int32_t* table, int32_t* ref, int n, int B, int P,
                          int n_pages, hipStream_t s)
{
    kv_free_kernel<<<dim3(n), dim3(256), 0, s>>>(rows, lens, table, ref, B, P, n_pages);
    return hipGetLastError();
}

hipError_t launch_kv_copy(const int32_t* src, const int32_t* dst, void* pool, int n, const KvGeom& g, hipStream_t s)
{
    kv_copy_kernel<<<dim3(copy_grid(n, g)), dim3(256), 0, s>>>(src, dst, static_cast<char*>(pool), n, g);
    return hipGetLastError();
}

hipError_t launch_kv_fork(const KvForkArgs& a, hipStream_t s)
{
    // A few pages are copied by the workgroup that decides, which saves a launch; more bytes than that take one CU
    // longer than a launch of many (a free and a fork of 16 KB 9.2 us against 11.5 with a launch for the copy, 32 KB
    // 10.4 against 12.0, 64 KB 12.5 against 12.1).
    if ((long long)a.n * a.g.planes * (long long)a.g.page_bytes() <= kForkAtOnce) {
        kv_fork_kernel<true><<<dim3(1), dim3(kCtl), 0, s>>>(a);
        return hipGetLastError();
    }
    kv_fork_kernel<false><<<dim3(1), dim3(kCtl), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    kv_fork_copy_kernel<<<dim3(copy_grid(a.n, a.g)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t s)
{
    kv_compact_plan_kernel<<<dim3(1), dim3(kCtl), 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    kv_compact_kernel<<<dim3(copy_grid(a.g.n_pages / 2 + 1, a.g)), dim3(256), 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace gdn
