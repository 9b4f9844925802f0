// The output layer's losses: the launch interface between the C ABI
// (outloss.cpp) and the kernels (outloss.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

// Rows and columns that the workspace's arrays are padded to, and the columns
// of one partial softmax statistic.
constexpr uint32_t kLossTile = 256, kStatColumns = 128;
constexpr int kMaxPlanes = 3;
constexpr int32_t kNoId = 0x7FFFFFFF;  // behind the last entry of a sorted list

constexpr uint32_t kLossSms = 152;

// A matrix as `planes` bf16 planes whose sum it is: one plane for bf16 values,
// three for float32 (each the bf16 nearest to what the planes before it left:
// 24 bits in all).
struct Planes {
    uint16_t* p;
    uint64_t plane;  // elements from one plane to the next
    uint64_t pitch;  // ... and from one row to the next
    int planes;
    // null, or where the second and the third plane are instead: in the place of a float32
    // matrix of this pitch, of every kLowGroup columns the second plane's and then the third's
    uint16_t* low = nullptr;
};
constexpr uint32_t kLowGroup = 64;

// What every token has, by its place among the n of the call: its list of ids
// (ascending, kNoId behind the last) with their shares.
struct Lists {
    int32_t* ids;       // n x top
    float* shares;      // n x top; null: every share is 1
    float* entropy;     // sum p log p; NaN for a list that is not valid
    uint32_t* counted;  // whether the token counts
    float* logits;      // the student's logits at the ids, n x top
    int top;
};

// The tokens that count, in order, and what follows from their number.
struct Counted {
    uint32_t* count;
    int32_t* row;  // the token at each place
    float* factor;
};

struct TeacherArgs {
    const void* ids;
    const void* logits;
    uint64_t ids_stride, logits_stride;
    int id_bytes;
    int logits_bf16;
    int k;
    float inv_t;
    uint32_t n, vocab;
    Lists lists;
};

struct RowsArgs {
    const void* targets;  // null: lists.counted says which tokens count
    int target_bytes;
    int64_t ignore;
    uint32_t n, vocab;
    double scale;
    int mean;
    Lists lists;
    Counted rows;
    float* result;     // written here where nothing counts
    uint32_t* ticket;  // of the joins of this call
    // of a call on few tokens (others' are cleared as they are packed): what those that
    // do not count are given; null: none
    float* losses;
    void* grad;
    uint64_t grad_stride;
    int grad_bf16;
    uint32_t width;
};

// Rows of a caller's matrix into planes: row i from row rows.row[i] of src
// (rows.row null: row i), zeros behind the last one up to a tile's end.  Of the n
// tokens those that do not count are given a loss and a gradient of 0.
struct PackArgs {
    const void* src;
    uint64_t stride;
    int bf16;
    uint32_t n, width;  // rows, columns of src; planes have `pitch` columns, zero behind width
    Counted rows;
    Planes out;
    const uint32_t* counted;  // null: no tokens
    float* losses;            // null: none, as below
    void* grad;
    uint64_t grad_stride;
    int grad_bf16;
};

// The counted tokens at places [base, base + n) are a piece; arrays by place
// start at the piece's first.  stats: a place's largest y = z log2(e) / t and sum
// 2^(y - largest) of every kStatColumns columns, `pitch` of them a place.
struct JoinArgs {
    const float2* stats;
    uint64_t pitch;
    uint32_t parts, base, n;
    float c;               // log2(e) / t
    float t2;              // t^2
    Lists lists;
    Counted rows;
    float* losses;         // by token; null: none
    // losses alone: the record, by the last of the CTAs, of kJoinRows places each
    double* sums;
    uint32_t* bad;
    uint32_t *ticket, tickets;
    float* result;
    // with gradients: the piece's logits (overwritten where they are g.low's place) and the place
    // of every loss and logit gradient
    const float* z;
    uint64_t z_pitch;
    uint32_t vocab, columns;  // ..., of a CTA
    uint32_t round;           // zeros in the rows up to a multiple of this
    float* loss;
    Planes g;
};

constexpr uint32_t kJoinRows = 8;

// C = A B^T over k, A's rows and B's rows as planes; a matrix of which k runs
// along the rows of memory is `turned`: element (row, k) lies at [k][row].
struct Operand {
    Planes m;
    bool turned;
    uint64_t rows, cols;  // of the array in memory
};

// Logits of a piece: their statistics and, if z is not null, the logits.
struct LogitArgs {
    float c;
    uint32_t v0;         // the first column's vocabulary entry (stats and z start there)
    bool at_ids;         // whether lists.logits is to be written
    Lists lists;
    const int32_t* row;  // the token at each place
    float2* stats;
    uint64_t stats_pitch;
    float* z;
    uint64_t z_pitch;
};

// Where a product goes: it is scaled, `add` (float32, null: nothing) is added to it, and it is
// stored in `sum` (float32), or if that is null in the caller's rows (row i into
// row[i] if row is not null).  Products of several splits go to parts, a matrix of
// whole tiles each, and are finished by launch_finish; they have no add and sum.
struct OutArgs {
    const float* factor;  // the product times *factor t
    float t;
    const float* add;
    float* sum;
    uint64_t sum_pitch;
    float* parts;
    uint64_t part_pitch;
    void* out;
    uint64_t stride;
    int bf16;
    int accumulate;
    const int32_t* row;
};

struct ProductArgs {
    Operand a, b;
    uint32_t m, n, k;      // rows of A, rows of B, products of a sum
    int count_m, count_k;  // m, k: no more than the counted tokens behind base
    uint32_t base;
    uint32_t run;          // blocks of 64 products that are summed in the tensor cores
    uint32_t splits;       // parts of k
    uint32_t width;        // columns of a tile: a multiple of 32 up to 256
    uint32_t group;        // rows of tiles that are worked on side by side
    const uint32_t* count;
    LogitArgs logit;
    OutArgs out;
    uint32_t* status;
};

// The record of a call with gradients, written beside its last products.
struct RecordArgs {
    const float* loss;  // by place
    Counted rows;
    float* result;      // null: none
};

// Calls of a few tokens, whose time is that of reading the weights: no tiles, no
// packing.  Of the counted tokens those at places [base, base + n), n <= kFewTokens;
// z, stats and g start at the first of them.
constexpr uint32_t kFewTokens = 8, kFewColumns = 64;

struct FewArgs {
    const void *x, *w;
    uint64_t x_stride, w_stride;
    int bf16;
    uint32_t base, n, width, vocab;
    Counted rows;
    // logits
    float c;
    Lists lists;
    float2* stats;
    uint64_t stats_pitch;
    float* z;  // null: the statistics alone
    uint64_t z_pitch;
    // gradients from the logits' (null: not wanted)
    Planes g;
    float t;
    void *grad_x, *grad_w;
    uint64_t grad_x_stride, grad_w_stride;
    int grad_x_bf16, grad_w_bf16, accumulate;
    float* parts;  // of grad_x
    uint64_t room;
    uint32_t entries;  // vocabulary entries of a CTA, a multiple of kFewColumns
};

cudaError_t launch_teacher(const TeacherArgs& a, cudaStream_t st);
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st);
cudaError_t launch_pack(const PackArgs& a, const PackArgs* b, cudaStream_t st);  // b: null, or a second matrix
cudaError_t launch_join(const JoinArgs& a, cudaStream_t st);  // losses alone
cudaError_t launch_grad(const JoinArgs& a, cudaStream_t st);  // losses and the logits' gradients
// What the products' kernels need once on a device before their first launch.
cudaError_t prepare_products();
cudaError_t launch_logits(ProductArgs a, cudaStream_t st);
// One or two products in one launch (and the finish of the first, if it is worth
// splitting: its parts have room for `room` values).
cudaError_t launch_products(const ProductArgs* a, int n, uint64_t room, const RecordArgs& r, cudaStream_t st);

cudaError_t launch_few_logits(const FewArgs& a, cudaStream_t st);
cudaError_t launch_few_gradients(FewArgs a, const RecordArgs& r, cudaStream_t st);

}  // namespace ar
