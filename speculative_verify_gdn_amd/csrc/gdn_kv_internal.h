// gdn_kv_internal.h -- launchers of the paged cache and the window attention
// (gdn_kv.hip, gdn_attn.hip) behind the C ABI of include/gdn.h.  The ABI layer
// validates every argument on the host; ids and lengths that live in device
// memory are bounded by the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace gdn {

constexpr int kKvWindowMax = 64;    // tokens of a window (its ancestor sets are 64-bit masks)
constexpr int kKvForkMax = 4096;    // forks in one call (their new pages' ids are kept in LDS)
constexpr int kKvPagesMax = (1 << 21) - 2;  // 1024 threads' page counts sum within 32 bits
constexpr int kAttnBatchMax = 4096; // sequences of one attention call

// pool geometry shared by the cache calls; a page of one plane is `page_bytes` long
struct KvGeom {
    int planes, n_pages, Hkv, page_log2, row_bytes;  // row_bytes: one token of one head
    __host__ __device__ size_t page_bytes() const { return ((size_t)Hkv << page_log2) * row_bytes; }
};

struct KvReserveArgs {
    const int32_t *lens, *add;
    int32_t *table, *ref, *granted;
    int B, P, n_pages, page_log2;
};

struct KvAppendArgs {
    const void *k, *v;
    size_t token_bytes;  // from one token to the next of k and v
    void *k_pages, *v_pages;
    const int32_t *lens, *count, *table;
    int B, K, P;
    KvGeom g;
};

struct KvRollbackArgs {
    const int32_t *node, *parent, *lens, *count;
    int32_t *table, *ref;
    void* pool;
    int32_t* lens_out;
    int B, N, P;
    KvGeom g;
};

struct KvForkArgs {
    const int32_t *src, *dst;
    int32_t *lens, *table, *ref;
    void* pool;
    int32_t* granted;
    int n, B, P;
    KvGeom g;
};

struct KvCompactArgs {
    const int32_t *table, *ref;
    void* pool;
    int32_t *table_out, *ref_out;
    int32_t* work;  // kv_compact_words(n_pages) words
    long long entries;
    KvGeom g;
};

// where the parts of the attention's workspace start
struct AttnWork {
    size_t plan, ml_s, ml_o, o_s, o_o, bytes;
};

struct AttnArgs {
    const void* q;
    size_t q_stride;  // elements from one token to the next
    const void *k_pages, *v_pages;
    const int32_t *lens, *count, *parent, *table;
    void* o;
    float* lse;
    void* work;
    int B, K, Hq, Hkv, D, page_log2, n_pages, P, prefix;
    float scale;
    // set at the launch: divisions and products that every workgroup would repeat
    int G;       // Hq / Hkv
    int listed;  // row tiles are units of the own list (attn::row_tiles_listed)
    AttnWork at;
};

size_t kv_compact_words(int n_pages);
bool kv_copy_countable(long long n, const KvGeom& g);  // n pages' pieces stay where the copies count them exactly
size_t attn_work_bytes(int B, int K, int Hq, int Hkv, int D, int page_log2, int P, int prefix, bool bf16);

hipError_t launch_kv_reserve(const KvReserveArgs& a, hipStream_t s);
hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t s);
hipError_t launch_kv_rollback(const KvRollbackArgs& a, hipStream_t s);
hipError_t launch_kv_free(const int32_t* rows, int32_t* lens, int32_t* table, int32_t* ref, int n, int B, int P,
                          int n_pages, hipStream_t s);
hipError_t launch_kv_fork(const KvForkArgs& a, hipStream_t s);
hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t s);
hipError_t launch_kv_copy(const int32_t* src, const int32_t* dst, void* pool, int n, const KvGeom& g, hipStream_t s);
hipError_t launch_attn(const AttnArgs& a, bool bf16, hipStream_t s);

}  // namespace gdn
