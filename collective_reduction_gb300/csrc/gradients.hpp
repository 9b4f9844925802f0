// Work over many tensors after a gradient allreduce: the launch interface
// between the C ABI (gradients.cpp) and the kernels (gradients.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

// A handle splits every tensor into ranges that a warp each works through.
// Range k of a tensor ends before element (k + 1) item_elems - lead and starts
// where range k - 1 ends: a tensor that begins `lead` elements past an
// alignment boundary (lead < item_elems) has a short first range, and every
// later one starts on a boundary.
struct RangeSplit {
    uint64_t count;
    uint32_t item_elems;
    uint32_t lead;

    __host__ __device__ uint64_t ranges() const {
        return count == 0 ? 0 : (count + lead + item_elems - 1) / item_elems;
    }
    __host__ __device__ uint64_t begin(uint64_t k) const { return k == 0 ? 0 : k * item_elems - lead; }
    __host__ __device__ uint64_t end(uint64_t k) const {
        const uint64_t e = (k + 1) * item_elems - lead;
        return e < count ? e : count;
    }
};

// Ranges start on this boundary of their leading stream (the gradients; for
// AdamW the first moments): a warp's 512-byte loads then cover whole lines.
constexpr uint32_t kRangeAlign = 128;
inline uint32_t lead_elems(const void* p, uint32_t es) {
    return static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p) % kRangeAlign) / es;
}

// Flags: element types of the streams (bit set: bfloat16, else float32), and
// whether a scaled tensor overwrites its own gradients.
constexpr uint32_t kGradBf16 = 1, kOutBf16 = 2, kInPlace = 4, kParamBf16 = 8, kHasCopy = 16;

// A gradient and the tensor that takes it scaled.
struct GradTensor {
    const char* src;
    char* dst;
    RangeSplit split;
    uint32_t flags;
};

// A parameter, its gradient, moments and optional bf16 copy.
struct AdamTensor {
    char* p;
    const char* g;
    float* m;
    float* v;
    char* w;
    RangeSplit split;
    uint32_t flags;
    float decay;  // this tensor's multiple of the weight decay
};

// One range of them.
struct alignas(16) GradItem {
    const char* src;
    char* dst;
    uint32_t count;
    uint32_t flags;
    uint64_t pad;
};

struct alignas(16) AdamItem {
    char* p;
    const char* g;
    float* m;
    float* v;
    char* w;
    uint32_t count;
    uint32_t flags;
    float decay;
    uint32_t pad[3];
};

constexpr int kGradThreads = 256;  // 8 warps, an item each
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kNormCtasPerSm = 3;
constexpr uint32_t kNormLists = 8;
// The cluster that adds up the items' sums
constexpr uint32_t kFinishThreads = 512, kFinishCtas = 8;
// Small sets: one cluster, a range of at most kSmallItemElems to each warp
constexpr int kSmallThreads = 512;
constexpr int kSmallWarps = kSmallThreads / 32;
constexpr int kSmallCtas = 8;
constexpr uint32_t kSmallItems = kSmallWarps * kSmallCtas;
constexpr uint32_t kSmallItemElems = 1024;

inline uint32_t grad_ctas(uint32_t n_items) {
    return n_items <= kGradWarps ? 1 : (n_items + kGradWarps - 1) / kGradWarps;
}

struct NormArgs {
    const GradItem* items;
    uint32_t n_items;
    uint32_t keep_from;     // launch_norm's keep: items before it leave L2 first
    int kind;               // AR_NORM_L2 or AR_NORM_MAX
    uint64_t* partials;     // each item's sum
    uint32_t* drawn;        // items drawn from the counter; 0 between calls
    double pre_scale, max_norm;
    float* result;          // norm, scale, nonfinite, clipped
    uint32_t record_ctas;   // finish: CTAs that write the record: 0 or kFinishCtas
    const uint32_t* first;  // finish: each tensor's first item (n_tensors + 1)
    float* tensor_norms;    // finish: the norms of single tensors
    uint32_t n_tensors;     // finish: their number, or 0
};

struct ScaleArgs {
    const GradItem* items;
    uint32_t n_items;
    uint32_t item_warps;    // warps that share an item: 1, 2, 4 or 8
    uint32_t rounds;        // items that a CTA's warps work through in turn
    bool in_place;          // every item
    const float* result;
};

// What of an update depends on its number.
struct AdamScalars {
    float step_size;           // lr / (1 - beta1^t)
    float inv_bc2;             // 1 / sqrt(1 - beta2^t)
    float lr_decay;            // lr times the weight decay
};

struct AdamArgs {
    const AdamItem* items;
    uint32_t n_items;
    const float* result;       // the norm's record, or null: factor 1
    float beta1, omb1;         // omb: one minus beta, rounded from 64 bits
    float beta2, omb2;
    float eps;
    AdamScalars scalars;
    const AdamScalars* counted;  // null, or where launch_count left them
};

// The scalars of update *steps + 1, and *steps counted up, unless the record
// says that the update is skipped.
struct CountArgs {
    uint64_t* steps;
    const float* lr;           // null: host_lr
    const float* result;
    double host_lr, beta1, beta2, weight_decay;
    AdamScalars* scalars;
};

// Writes the items of n tensors; first[t] is tensor t's first item (n + 1).
cudaError_t launch_items(const GradTensor* tensors, const uint32_t* first, int n, uint32_t n_items, GradItem* items,
                         cudaStream_t st);
cudaError_t launch_items(const AdamTensor* tensors, const uint32_t* first, int n, uint32_t n_items, AdamItem* items,
                         cudaStream_t st);

// Every item's sum, for launch_finish.  keep: the gradients are read again
// after it, last items first; num_sms: the device's.
cudaError_t launch_norm(const NormArgs& a, bool keep, int num_sms, cudaStream_t st);
cudaError_t launch_finish(const NormArgs& a, cudaStream_t st);
cudaError_t launch_scale(const ScaleArgs& a, cudaStream_t st);
// The sums, the record and, with `scale`, the scaling in one launch: at most kSmallItems
// items of at most kSmallItemElems elements.
cudaError_t launch_small(const NormArgs& a, bool scale, cudaStream_t st);
cudaError_t launch_count(const CountArgs& a, cudaStream_t st);
// whole: every stream of every tensor can be read and written in quads.
cudaError_t launch_adamw(const AdamArgs& a, bool whole, cudaStream_t st);

}  // namespace ar
