// The output layer's losses: the launch interface between the C ABI
// (outloss.cpp) and the kernels (outloss.cu).
#pragma once

#include <cuda_runtime.h>

#include <cstdint>

#include "ar.h"

namespace ar {

// Rows and columns that the workspace's arrays are padded to, and the columns
// of one partial softmax statistic.
constexpr uint32_t kLossTile = 256;
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
};

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
};

// Rows of a caller's matrix into planes: row i from row rows.row[i] of src
// (rows.row null: row i), zeros behind the last one up to a tile's end.
struct PackArgs {
    const void* src;
    uint64_t stride;
    int bf16;
    uint32_t n, width;  // rows, columns of src; planes have `pitch` columns, zero behind width
    Counted rows;
    Planes out;
};

// What the tokens that do not count are given.
struct ClearArgs {
    const uint32_t* counted;
    uint32_t n, width;
    float* losses;       // null: none
    void* grad_hidden;   // null: none
    uint64_t stride;
    int bf16;
};

// A token's place's softmax: largest y = z c, and factor / sum 2^(y - max).
struct RowStat {
    float top, inv;
};

struct JoinArgs {
    const float2* stats;  // [tiles][pitch]: largest y, sum 2^(y - largest)
    uint64_t pitch;
    uint32_t tiles, n;
    float c;              // log2(e) / t
    double t;
    Lists lists;
    Counted rows;
    RowStat* stat;        // by place
    float* gain;          // by place: what the shares are multiplied by, factor t
    float* loss;          // by place
    float* losses;        // by token; null: none
};

struct RecordArgs {
    const float* loss;
    Counted rows;
    float* result;
};

// C = A B^T over k, A's rows and B's rows as planes; a matrix of which k runs
// along the rows of memory is `turned`: element (row, k) lies at [k][row].
struct Operand {
    Planes m;
    bool turned;
    uint64_t rows, cols;  // of the array in memory
};

enum LossEpilogue { kLossStats, kLossGrad, kLossOut };

// Columns [v0, v1) of the logits or of their gradient; columns of a piece
// start at 0.
struct LogitArgs {
    uint32_t v0, v1;
    float c;
    Lists lists;
    float2* stats;
    uint64_t stats_pitch;
    const RowStat* stat;
    const float* gain;
    Planes g;
};

// Where a product goes: parts (float32, one of `splits` each, added to if
// `add_parts`), or the caller's rows (row i into row[i] if row is not null).
struct OutArgs {
    float* parts;
    uint64_t part_stride, part_pitch;
    int add_parts;
    void* out;
    uint64_t stride;
    int bf16;
    int accumulate;
    const int32_t* row;
};

struct ProductArgs {
    Operand a, b;
    uint32_t m, n, k;       // rows of A, rows of B, products of a sum
    int count_m, count_k;   // m, k: no more than the tokens that count
    int splits;             // parts of k
    const uint32_t* count;
    LossEpilogue epilogue;
    LogitArgs logit;
    OutArgs out;
    uint32_t* status;
};

struct FinishArgs {
    const float* parts;
    uint64_t part_stride, part_pitch;
    int splits;
    uint32_t n, width;
    Counted rows;
    int by_count;  // n: the tokens that count
    void* out;
    uint64_t stride;
    int bf16;
    int accumulate;
};

cudaError_t launch_teacher(const TeacherArgs& a, cudaStream_t st);
cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st);
cudaError_t launch_pack(const PackArgs& a, cudaStream_t st);
cudaError_t launch_clear(const ClearArgs& a, cudaStream_t st);
cudaError_t launch_join(const JoinArgs& a, cudaStream_t st);
cudaError_t launch_record(const RecordArgs& a, cudaStream_t st);
// What the products' kernels need once on a device before their first launch.
cudaError_t prepare_products();
cudaError_t launch_product(const ProductArgs& a, cudaStream_t st);
cudaError_t launch_finish_parts(const FinishArgs& a, cudaStream_t st);

}  // namespace ar
