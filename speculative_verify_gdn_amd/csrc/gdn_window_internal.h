// gdn_window_internal.h -- launchers of what a verify window passes around the
// attention (gdn_rope.hip, gdn_logits.hip) behind the C ABI of include/gdn.h.
// The ABI layer validates every argument on the host; lengths, parents, page
// ids and tokens that live in device memory are bounded by the kernels.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "gdn_kv_internal.h"

namespace gdn {

constexpr int kRopeHeadMax = 512;   // elements of a head of the rotary calls

// queries, keys, values: heads of one token, from a strided source to a strided
// destination (or to the pages of the cache)
struct RopePart {
    const void* x;
    void* y;
    long long xs[3], ys[3];  // bytes from one sequence, token, head to the next (ys unused where paged)
    const float* w;          // norm weights [D] or nullptr
    int H;                   // heads (0: the part is absent)
    int turned;              // the heads are rotated (and normed, with w); else copied
    int paged;               // y is a plane of the cache
};

struct RopeArgs {
    RopePart part[3];
    const int32_t *pos, *lens, *parent, *count, *table;
    const double* freqs;
    int rot;
    float mscale, eps;
    int B, K, D, P;
    KvGeom g;
    // set at the launch
    int heads;       // of all parts together
    int tile;        // tokens of a workgroup
    int chunk;       // heads of a workgroup
    int lanes_log2;  // lanes of one head
    int half_log2;   // lanes of one token's pairs
};

struct LogitsArgs {
    const void* x;
    void* out;
    size_t x_stride, out_stride;  // elements from one row to the next
    int32_t* best;
    const int32_t *history, *history_lens, *history_start;
    const int32_t *tokens, *parent, *count;
    const float* params;
    const int32_t* bias_ids;
    const float* bias_values;
    const uint32_t* mask;
    const float* noise;
    unsigned long long* work;  // [rows][slices] the best of each slice, score and token as one number
    int B, K, V, capacity, n_bias;
    // set at the launch
    int marks;   // some tokens may need more than the mask and the temperature
    int slices;  // of the vocabulary
    int rows;    // rows of a window of a workgroup
};

struct AcceptArgs {
    const int32_t *target, *tokens, *parent, *count, *root;
    int32_t *node, *next, *history;
    const int32_t* lens;
    int32_t* lens_out;
    int B, K, capacity;
};

int logits_slices(int V);   // of the vocabulary, at most

hipError_t launch_rope(const RopeArgs& a, bool bf16, bool interleaved, hipStream_t s);
hipError_t launch_logits(const LogitsArgs& a, bool x_bf16, bool out_bf16, hipStream_t s);
hipError_t launch_accept(const AcceptArgs& a, hipStream_t s);

}  // namespace gdn
