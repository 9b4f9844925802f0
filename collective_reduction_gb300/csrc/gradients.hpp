// Work over many tensors after a gradient allreduce: the launch interface
// between the C ABI (gradients.cpp) and the kernels (gradients.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>
#include <vector>

#include "ar.h"

namespace ar {

// A range of one tensor that one warp works through.  Every item of a tensor
// but its last holds the handle's item_elems elements, so all start at the
// same place within a 16-byte vector as the tensor does.
struct TensorRange {
    uint32_t tensor;
    uint32_t count;
    uint64_t elem;
};

// The ranges of n tensors in order, none empty; first[t] is the index of
// tensor t's first range (first[n] their number).
void split_tensors(int n, const uint64_t* counts, uint64_t item_elems, std::vector<TensorRange>& ranges,
                   std::vector<uint32_t>& first);

// Item flags: element types of the streams (bit set: bfloat16, else float32),
// and whether a scaled item overwrites its own gradients.
constexpr uint32_t kGradBf16 = 1, kOutBf16 = 2, kInPlace = 4, kParamBf16 = 8, kHasCopy = 16;

// One range of a gradient (src) and of the tensor that takes it scaled (dst).
struct alignas(16) GradItem {
    const char* src;
    char* dst;
    uint32_t count;
    uint32_t flags;
    uint64_t pad;
};

// One range of a parameter, its gradient, moments and optional bf16 copy.
struct alignas(16) AdamItem {
    char* p;
    const char* g;
    float* m;
    float* v;
    char* w;
    uint32_t count;
    uint32_t flags;
    float decay;  // this tensor's multiple of the weight decay
    uint32_t pad[3];
};

constexpr int kGradThreads = 256;                   // 8 warps, an item each at a time
constexpr int kGradWarps = kGradThreads / 32;
constexpr int kNormCtasPerSm = 4;                   // the norm kernel's persistent grid
constexpr int kTensorNormThreads = 512;

// What the norm kernels leave for the host's caller and for the kernels after
// them: the norm, the factor, and two truth values.
struct NormArgs {
    const GradItem* items;
    uint32_t n_items;
    int kind;                // AR_NORM_L2 or AR_NORM_MAX
    uint64_t* cta_partials;  // one per CTA of the grid
    uint64_t* item_partials; // one per item, or null: no norms of single tensors
    uint32_t* counter;       // CTAs done; 0 between calls
    double pre_scale, max_norm;
    float* result;           // 4 floats
};

struct TensorNormArgs {
    const uint64_t* item_partials;
    const uint32_t* first;   // n + 1
    int kind;
    double pre_scale;
    float* norms;            // n
};

struct ScaleArgs {
    const GradItem* items;
    uint32_t n_items;
    const float* result;
};

struct AdamArgs {
    const AdamItem* items;
    uint32_t n_items;
    const float* result;     // the norm's record, or null: factor 1
    float beta1, omb1;       // omb: one minus beta, rounded from 64 bits
    float beta2, omb2;
    float step_size;         // lr / (1 - beta1^t)
    float inv_bc2;           // 1 / sqrt(1 - beta2^t)
    float eps;
    float lr_decay;          // lr times the weight decay
};

// CTAs of the norm kernel's grid for n_items on num_sms SMs.
int norm_grid(uint32_t n_items, int num_sms);
cudaError_t launch_norm(const NormArgs& a, int grid, cudaStream_t st);
cudaError_t launch_tensor_norms(const TensorNormArgs& a, int n_tensors, cudaStream_t st);
cudaError_t launch_scale(const ScaleArgs& a, cudaStream_t st);
cudaError_t launch_adamw(const AdamArgs& a, cudaStream_t st);

}  // namespace ar
