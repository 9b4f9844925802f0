// Kernels of the output layer's losses: teacher lists, the tokens that count,
// the products over hidden size, vocabulary and tokens with the softmax in
// their epilogues, and the joins between them.
//
// With z = X W^T, y = z log2(e) / t and a token's shares p over a short list
// of ids, the loss is t^2 (sum p log p - sum p z / t + log sum exp(z / t)) and
// its gradient by z, with the factor f of the record,
//   g = 2^(y - top) / sum 2^(y - top) - p,   dX = f t g W,   dW = f t g^T X.
#include <cuda.h>  // the tensor map's types only: the driver call is resolved at run time

#include <algorithm>
#include <type_traits>

#include "device.cuh"
#include "outloss.hpp"

namespace ar {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
constexpr float kInf = __builtin_huge_valf();
constexpr double kLn2 = 0.69314718055994530942;

__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ uint16_t bf16_of(float x) { return static_cast<uint16_t>(pack_bf16x2(x, 0.f)); }

__device__ __forceinline__ float load_value(const void* p, uint64_t i, int bf16) {
    return bf16 ? bf16_value(static_cast<const uint16_t*>(p)[i]) : static_cast<const float*>(p)[i];
}

// The next bf16 plane of x: the nearest bf16 (a finite x whose nearest would be
// an infinity: towards zero); x keeps what is left, exactly.
__device__ __forceinline__ uint16_t split_plane(float& x) {
    uint16_t b = bf16_of(x);
    if ((b & 0x7FFFu) == 0x7F80u && fabsf(x) < kInf) b -= 1;
    const float v = bf16_value(b);
    x = (b & 0x7F80u) == 0x7F80u ? 0.f : __fsub_rn(x, v);  // an infinity or NaN leaves nothing
    return b;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// ------------------------------------------------------------ lists and rows

constexpr int kTeacherWarps = 4;

// A warp a token: the softmax of its entries, entries of one id added up, sorted
// by id.  The k^2 comparisons of a list stay in shared memory: 17 us for 2048 lists
// of 64, 2% of what follows.
__global__ void __launch_bounds__(32 * kTeacherWarps) teacher_kernel(const __grid_constant__ TeacherArgs a) {
    extern __shared__ char smem[];
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t i = blockIdx.x * kTeacherWarps + warp;
    int32_t* id = reinterpret_cast<int32_t*>(smem) + warp * 2 * a.k;
    float* share = reinterpret_cast<float*>(id + a.k);
    griddep_launch_dependents();
    griddep_wait();
    if (i >= a.n) return;
    bool bad = false;
    float top = -kInf;
    for (int j = lane; j < a.k; j += 32) {
        const uint64_t at = i * a.ids_stride + j;
        const int64_t v = a.id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
        float u = -kInf;
        int32_t x = kNoId;
        if (v >= 0) {
            u = load_value(a.logits, i * a.logits_stride + j, a.logits_bf16);
            if (u != -kInf) {  // NaN stays in
                if (v >= a.vocab) bad = true;
                else x = static_cast<int32_t>(v);
                if (u != u) bad = true;
            }
        }
        id[j] = x;
        share[j] = u;
        if (x != kNoId) top = fmaxf(top, u);
    }
    for (int o = 16; o > 0; o /= 2) top = fmaxf(top, __shfl_xor_sync(kFull, top, o));
    bad = __any_sync(kFull, bad) || top == kInf;
    float sum = 0.f;
    for (int j = lane; j < a.k; j += 32) {
        const bool in = id[j] != kNoId && !bad;
        const float e = in ? expf(__fmul_rn(__fsub_rn(share[j], top), a.inv_t)) : 0.f;
        share[j] = e;
        sum = __fadd_rn(sum, e);
    }
    for (int o = 16; o > 0; o /= 2) sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, o));
    const bool any = __any_sync(kFull, top != -kInf);
    __syncwarp();
    // entries of one id: the first takes the sum, the others go
    for (int b = 0; b < a.k; b += 32) {
        const int j = b + static_cast<int>(lane);
        float s = 0.f;
        bool first = j < a.k && id[j] != kNoId;
        if (first) {
            for (int q = 0; q < a.k; ++q) {
                if (id[q] != id[j]) continue;
                if (q < j) {
                    first = false;
                    break;
                }
                s = __fadd_rn(s, share[q]);
            }
        }
        // a share is overwritten only by its own lane, and only entries before b + 32
        // have gone: those of later ids read none of them
        __syncwarp();
        if (j < a.k) {
            if (first) share[j] = s;
            else share[j] = -1.f;  // marks what has gone; ids stay for the comparisons above
        }
        __syncwarp();
    }
    const uint64_t row = static_cast<uint64_t>(i) * a.lists.top;
    float entropy = 0.f;
    uint32_t kept = 0;
    for (int j = lane; j < a.k; j += 32) {
        if (share[j] < 0.f) continue;
        int place = 0;
        for (int q = 0; q < a.k; ++q) place += share[q] >= 0.f && id[q] < id[j];
        const float p = __fdiv_rn(share[j], sum);
        a.lists.ids[row + place] = id[j];
        a.lists.shares[row + place] = p;
        if (p > 0.f) entropy = __fadd_rn(entropy, __fmul_rn(p, logf(p)));
        ++kept;
    }
    for (int o = 16; o > 0; o /= 2) {
        entropy = __fadd_rn(entropy, __shfl_xor_sync(kFull, entropy, o));
        kept += __shfl_xor_sync(kFull, kept, o);
    }
    for (int j = static_cast<int>(kept + lane); j < a.lists.top; j += 32) {
        a.lists.ids[row + j] = kNoId;
        a.lists.shares[row + j] = 0.f;
    }
    if (lane == 0) {
        a.lists.entropy[i] = bad ? __int_as_float(0x7FC00000) : entropy;
        a.lists.counted[i] = any || bad;
    }
}

constexpr int kRowThreads = 1024;

// One CTA: targets into lists of one id, and the tokens that count in their
// order; every warp has a run of tokens, 32 at a time (14 us for 16384: latency; a
// thread a run of its own took 45).
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ uint32_t sums[32];
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t run = (a.n + kRowThreads - 1) / kRowThreads * 32;
    const uint32_t lo = min(a.n, warp * run), hi = min(a.n, lo + run);
    griddep_launch_dependents();
    griddep_wait();
    uint32_t mine = 0;
#pragma unroll 4
    for (uint32_t i = lo + lane; i - lane < hi; i += 32) {
        bool counts = false;
        if (i < hi) {
            if (a.targets) {
                const int64_t v = a.target_bytes == 8 ? static_cast<const int64_t*>(a.targets)[i]
                                                      : static_cast<const int32_t*>(a.targets)[i];
                counts = v != a.ignore;
                const bool in = v >= 0 && v < a.vocab;
                a.lists.ids[static_cast<uint64_t>(i) * a.lists.top] = counts && in ? static_cast<int32_t>(v) : kNoId;
                a.lists.entropy[i] = counts && !in ? __int_as_float(0x7FC00000) : 0.f;
                a.lists.counted[i] = counts;
            } else {
                counts = a.lists.counted[i];
            }
        }
        mine += __popc(__ballot_sync(kFull, counts));
    }
    if (lane == 0) sums[warp] = mine;
    __syncthreads();
    if (warp == 0) {
        uint32_t s = sums[lane];
        for (int o = 1; o < 32; o *= 2) {
            const uint32_t x = __shfl_up_sync(kFull, s, o);
            if (lane >= static_cast<uint32_t>(o)) s += x;
        }
        sums[lane] = s;
    }
    __syncthreads();
    uint32_t place = warp ? sums[warp - 1] : 0;
#pragma unroll 4
    for (uint32_t i = lo + lane; i - lane < hi; i += 32) {
        const bool counts = i < hi && a.lists.counted[i];
        const uint32_t who = __ballot_sync(kFull, counts);
        if (counts) a.rows.row[place + __popc(who & ((1u << lane) - 1))] = static_cast<int32_t>(i);
        place += __popc(who);
    }
    if (a.losses || a.grad) {  // a few tokens
        __syncthreads();
        for (uint32_t i = 0; i < a.n; ++i) {
            if (a.lists.counted[i]) continue;
            if (a.losses && tid == 0) a.losses[i] = 0.f;
            for (uint32_t c = tid; a.grad && c < a.width; c += kRowThreads) {
                if (a.grad_bf16) static_cast<uint16_t*>(a.grad)[i * a.grad_stride + c] = 0;
                else static_cast<float*>(a.grad)[i * a.grad_stride + c] = 0.f;
            }
        }
    }
    if (tid == 0) {
        const uint32_t n = sums[31];
        const float factor = static_cast<float>(a.mean ? a.scale / (n ? n : 1u) : a.scale);
        *a.rows.count = n;
        *a.rows.factor = factor;
        *a.ticket = 0;
        if (n == 0) {
            a.result[0] = a.result[1] = a.result[2] = 0.f;
            a.result[3] = factor;
        }
    }
}

// Eight values of a row of src, zeros behind its width.
__device__ __forceinline__ void load_eight(const PackArgs& a, uint64_t from, uint32_t c, float (&x)[8]) {
    if (a.bf16) {
        const uint16_t* p = static_cast<const uint16_t*>(a.src) + from + c;
        if (c + 8 <= a.width && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
            const uint4 v = *reinterpret_cast<const uint4*>(p);
            x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
            x[4] = bf_lo(v.z), x[5] = bf_hi(v.z), x[6] = bf_lo(v.w), x[7] = bf_hi(v.w);
            return;
        }
#pragma unroll
        for (uint32_t j = 0; j < 8; ++j) x[j] = c + j < a.width ? bf16_value(p[j]) : 0.f;
        return;
    }
    const float* p = static_cast<const float*>(a.src) + from + c;
    if (c + 8 <= a.width && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const float4 u = *reinterpret_cast<const float4*>(p), v = *reinterpret_cast<const float4*>(p + 4);
        x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w, x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
        return;
    }
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j) x[j] = c + j < a.width ? p[j] : 0.f;
}

// Eight values' next plane.
__device__ __forceinline__ uint4 split_eight(float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t low = split_plane(x[2 * i]), high = split_plane(x[2 * i + 1]);
        w[i] = low | (high << 16);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 pack_eight(const float (&x)[8]) {
    return make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]), pack_bf16x2(x[6], x[7]));
}

// A warp a row (and a token), over the rows up to a tile's end.  Bound by HBM at
// size: 65 MB of odd bf16 rows 26 us, 16384 rows of 1024 15 us.
__device__ __forceinline__ void pack_row(const PackArgs& a, uint64_t r, uint32_t lane) {
    if (a.counted && r < a.n && !a.counted[r]) {
        if (a.losses && lane == 0) a.losses[r] = 0.f;
        if (a.grad)
            for (uint32_t c = lane; c < a.width; c += 32) {
                if (a.grad_bf16) static_cast<uint16_t*>(a.grad)[r * a.grad_stride + c] = 0;
                else static_cast<float*>(a.grad)[r * a.grad_stride + c] = 0.f;
            }
    }
    const uint32_t n = a.rows.row ? *a.rows.count : a.n;
    if (r >= (static_cast<uint64_t>(n) + kLossTile - 1) / kLossTile * kLossTile) return;
    const bool there = r < n;
    const uint64_t from = there ? (a.rows.row ? static_cast<uint64_t>(a.rows.row[r]) : r) * a.stride : 0;
    uint16_t* out = a.out.p + r * a.out.pitch;
#pragma unroll 2
    for (uint32_t c = 8 * lane; c < a.out.pitch; c += 256) {
        float x[8] = {};
        if (there) load_eight(a, from, c, x);
        if (a.out.planes == 1) {
            *reinterpret_cast<uint4*>(out + c) = pack_eight(x);
        } else {
            for (int q = 0; q < a.out.planes; ++q) *reinterpret_cast<uint4*>(out + q * a.out.plane + c) = split_eight(x);
        }
    }
}

// One matrix, or two of which the second begins with CTA `second`.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a, const __grid_constant__ PackArgs b,
                                                   uint32_t second) {
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    if (blockIdx.x < second) pack_row(a, blockIdx.x * 8ull + warp, lane);
    else pack_row(b, (blockIdx.x - second) * 8ull + warp, lane);
}

// ------------------------------------------------------------------- joins

// (top, sum 2^(y - top)) of two parts of a row.  A part of -infinities alone has sum
// 0 and adds nothing; +infinity and NaN make the sum NaN, also where they are all
// that a part has: fmaxf leaves NaN out, so such a part's top is -infinity, and it
// keeps its sum.
__device__ __forceinline__ void join_stat(float& top, float& sum, float top2, float sum2) {
    const float m = fmaxf(top, top2);
    const float low = -kInf;
    const float a = top == low ? sum : __fmul_rn(sum, exp2_fast(__fsub_rn(top, m)));
    const float b = top2 == low ? sum2 : __fmul_rn(sum2, exp2_fast(__fsub_rn(top2, m)));
    top = m;
    sum = __fadd_rn(a, b);
}

// The loss of a place from its softmax statistics, by the lanes of a warp, alike in
// all of them.  With y = z c and shares that add up to 1
//   log sum exp(z / t) - sum p z / t = ln 2 (log2 sum 2^(y - top) + sum p (top - y)),
// whose terms do not cancel, so float32 does.
__device__ __forceinline__ float row_loss(const JoinArgs& a, uint64_t r, uint64_t token, float top, float sum,
                                          uint32_t lane) {
    const uint64_t at = token * a.lists.top;
    float dot = 0.f;  // sum p (top - y)
    for (int j = lane; j < a.lists.top; j += 32) {
        const int32_t id = a.lists.ids[at + j];
        if (id == kNoId) break;  // nothing behind it
        // logits that other CTAs may be overwriting are not read
        const float z = a.z && !a.g.low ? a.z[r * a.z_pitch + id] : a.lists.logits[at + j];
        const float d = -__fmaf_rn(z, a.c, -top);
        const float share = a.lists.shares ? a.lists.shares[at + j] : 1.f;
        if (share != 0.f) dot = __fmaf_rn(share, d, dot);
    }
    for (int o = 16; o > 0; o /= 2) dot = __fadd_rn(dot, __shfl_xor_sync(kFull, dot, o));
    return __fmul_rn(a.t2, __fmaf_rn(static_cast<float>(kLn2), __fadd_rn(log2f(sum), dot), a.lists.entropy[token]));
}

// The statistics of a place by the lanes of a warp, from part `first` on in steps of `step`.
__device__ __forceinline__ void row_stat(const JoinArgs& a, uint64_t r, uint32_t first, uint32_t step, float& top,
                                         float& sum) {
    const float2* at = a.stats + r * a.pitch;
    top = -kInf;
    sum = 0.f;
#pragma unroll 4
    for (uint32_t q = first; q < a.parts; q += step) {
        const float2 s = at[q];
        join_stat(top, sum, s.x, s.y);
    }
    for (int o = 16; o > 0; o /= 2) {
        const float t2 = __shfl_xor_sync(kFull, top, o), s2 = __shfl_xor_sync(kFull, sum, o);
        join_stat(top, sum, t2, s2);  // either order gives the same bits
    }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < kInf; }

// A warp a place.  Every sum has a fixed order; the call's last CTA adds up the
// CTAs' and writes the record.
__global__ void __launch_bounds__(32 * kJoinRows) join_kernel(const __grid_constant__ JoinArgs a) {
    __shared__ double total[kJoinRows];
    __shared__ uint32_t flag[kJoinRows];
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t count = *a.rows.count, m = count > a.base ? min(a.n, count - a.base) : 0;
    const float factor = *a.rows.factor;
    const uint32_t r = blockIdx.x * kJoinRows + warp;
    float loss = 0.f;
    if (r < m) {
        float top, sum;
        row_stat(a, r, lane, 32, top, sum);
        const uint64_t token = a.rows.row[a.base + r];
        loss = row_loss(a, r, token, top, sum, lane);
        if (a.losses && lane == 0) a.losses[token] = loss;
    }
    if (lane == 0) {
        total[warp] = loss;
        flag[warp] = !finite(loss);
    }
    __syncthreads();
    if (tid == 0) {
        double all = 0.0;
        uint32_t any = 0;
        for (uint32_t w = 0; w < kJoinRows; ++w) {
            all += total[w];
            any |= flag[w];
        }
        const uint32_t cta = a.base / kJoinRows + blockIdx.x;
        a.sums[cta] = all;
        a.bad[cta] = any;
        __threadfence();
        flag[0] = atomicAdd(a.ticket, 1u) == a.tickets - 1;
    }
    __syncthreads();
    if (!flag[0] || count == 0) return;
    __threadfence();
    double all = 0.0;
    bool bad = false;
    for (uint32_t k = tid; k < (count + kJoinRows - 1) / kJoinRows; k += 32 * kJoinRows) {
        all += __ldcg(a.sums + k);
        bad = bad || __ldcg(a.bad + k);
    }
    for (int o = 16; o > 0; o /= 2) all += __shfl_down_sync(kFull, all, o);
    bad = __any_sync(kFull, bad);
    __syncthreads();
    if (lane == 0) {
        total[warp] = all;
        flag[warp] = bad;
    }
    __syncthreads();
    if (tid != 0) return;
    all = 0.0;
    uint32_t any = 0;
    for (uint32_t w = 0; w < kJoinRows; ++w) {
        all += total[w];
        any |= flag[w];
    }
    a.result[0] = static_cast<float>(all * factor);
    a.result[1] = static_cast<float>(count);
    a.result[2] = any ? 1.f : 0.f;
    a.result[3] = factor;
}

constexpr int kGradThreads = 256;

// The second plane's value of a row's column; the third's is kLowGroup on.
__device__ __forceinline__ uint16_t* low_place(const Planes& g, uint64_t r, uint32_t v) {
    return g.low + 2 * r * g.pitch + v / kLowGroup * (2 * kLowGroup) + v % kLowGroup;
}

// A CTA a place's `columns` columns: the statistics (of the whole row, in every
// one of its CTAs), then
//   g = 2^(y - top) / sum - share
// from the logits, then the few columns of the row's list.  The factor comes with
// the products' float32 sums: in bf16 a token's largest gradients, near -1, would all
// carry the factor's own rounding.  Bound by HBM: a logit's 4 bytes in and its
// gradient's 2 (float32: 6) out, 6.2 TB/s on cold caches at 4096 x 50001, 7 among the
// other launches.  A row's statistics cost each of its CTAs a round trip, so ranges are
// long: 281 us for 2048 x 128000 in 8192 columns, 247 in 32768.
__global__ void __launch_bounds__(kGradThreads) grad_kernel(const __grid_constant__ JoinArgs a) {
    __shared__ float2 part[kGradThreads / 32];
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t lo = blockIdx.x * a.columns, hi = min(a.vocab, lo + a.columns);
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t count = *a.rows.count, m = count > a.base ? min(a.n, count - a.base) : 0;
    for (uint64_t r = blockIdx.y; r < (m + a.round - 1) / a.round * a.round; r += gridDim.y) {
        const bool in = r < m;
        float top = 0.f, inv = 0.f;
        uint64_t token = 0;
        if (in) {
            float sum;
            row_stat(a, r, tid, kGradThreads, top, sum);
            __syncthreads();  // the row before has been read
            if (lane == 0) part[warp] = make_float2(top, sum);
            __syncthreads();
            top = part[0].x;
            sum = part[0].y;
            for (int w = 1; w < kGradThreads / 32; ++w) join_stat(top, sum, part[w].x, part[w].y);
            token = a.rows.row[a.base + r];
            const float entropy = a.lists.entropy[token];  // NaN: a list that is not valid
            inv = entropy == entropy && sum > 0.f ? __fdiv_rn(1.f, sum) : __int_as_float(0x7FC00000);
            if (blockIdx.x == 0 && warp == 0) {
                const float loss = row_loss(a, r, token, top, sum, lane);
                if (lane == 0) {
                    a.loss[r] = loss;
                    if (a.losses) a.losses[token] = loss;
                }
            }
        }
        const float* z = a.z + r * a.z_pitch;
        uint16_t* g = a.g.p + r * a.g.pitch;
        auto value = [&](float x) { return __fmul_rn(exp2_fast(__fmaf_rn(x, a.c, -top)), inv); };
        // a warp's 256 columns' low planes are their logits' place
        for (uint32_t v = lo + 8 * tid; a.g.low && v - 8 * lane < hi; v += 8 * kGradThreads) {
            float x[8] = {};
            if (in && v < hi) {
                const float4 p = *reinterpret_cast<const float4*>(z + v), q = *reinterpret_cast<const float4*>(z + v + 4);
                x[0] = value(p.x), x[1] = value(p.y), x[2] = value(p.z), x[3] = value(p.w);
                x[4] = value(q.x), x[5] = value(q.y), x[6] = value(q.z), x[7] = value(q.w);
#pragma unroll
                for (uint32_t j = 0; j < 8; ++j)
                    if (v + j >= hi) x[j] = 0.f;
            }
            __syncwarp();
            if (v >= (hi + kLowGroup - 1) / kLowGroup * kLowGroup) continue;
            uint16_t* low = low_place(a.g, r, v);
            *reinterpret_cast<uint4*>(g + v) = split_eight(x);
            *reinterpret_cast<uint4*>(low) = split_eight(x);
            *reinterpret_cast<uint4*>(low + kLowGroup) = split_eight(x);
        }
#pragma unroll 2
        for (uint32_t v = lo + 8 * tid; !a.g.low && v < hi; v += 8 * kGradThreads) {  // the pitch is of whole tiles
            float x[8] = {};
            if (in) {
                const float4 p = *reinterpret_cast<const float4*>(z + v), q = *reinterpret_cast<const float4*>(z + v + 4);
                x[0] = value(p.x), x[1] = value(p.y), x[2] = value(p.z), x[3] = value(p.w);
                x[4] = value(q.x), x[5] = value(q.y), x[6] = value(q.z), x[7] = value(q.w);
            }
            if (a.g.planes == 1) {
                *reinterpret_cast<uint4*>(g + v) = pack_eight(x);
            } else {
                for (int q = 0; q < a.g.planes; ++q) *reinterpret_cast<uint4*>(g + q * a.g.plane + v) = split_eight(x);
            }
        }
        if (!in) continue;  // the whole CTA
        __syncthreads();
        const uint64_t list = token * a.lists.top;
        for (int k = tid; k < a.lists.top; k += kGradThreads) {
            const uint32_t v = static_cast<uint32_t>(a.lists.ids[list + k]);
            if (v < lo || v >= hi) continue;
            const float share = a.lists.shares ? a.lists.shares[list + k] : 1.f;
            if (a.g.low) {
                uint16_t* low = low_place(a.g, r, v);  // the planes' sum is the value
                float x = __fadd_rn(__fadd_rn(bf16_value(low[kLowGroup]), bf16_value(low[0])), bf16_value(g[v]));
                x = __fsub_rn(x, share);
                g[v] = split_plane(x);
                low[0] = split_plane(x);
                low[kLowGroup] = split_plane(x);
                continue;
            }
            float x = __fsub_rn(value(z[v]), share);
            for (int q = 0; q < a.g.planes; ++q) g[q * a.g.plane + v] = split_plane(x);
        }
    }
}

__device__ __forceinline__ void store_out(void* out, uint64_t at, int bf16, int accumulate, float x) {
    if (accumulate) x = __fadd_rn(x, load_value(out, at, bf16));
    if (bf16) static_cast<uint16_t*>(out)[at] = bf16_of(x);
    else static_cast<float*>(out)[at] = x;
}

// ---------------------------------------------------------------- products
//
// C = A B^T on the tensor cores: a pair of CTAs (a cluster of two) works on one
// tile of 256 x 256, each holding 128 rows of A and of B in shared memory and 128
// rows of C in its tensor memory, twice (the epilogue of one tile runs beside the
// products of the next).  Persistent: pairs take tiles in turn.  Warp 0 loads (TMA,
// a ring of blocks of 64 products), warp 1 of the pair's first CTA issues
// the products, warps 4 to 11 are the epilogue: a thread half a row.
//
// The tensor cores cut sums off where float32 would round them.  Products whose
// result is float32 are therefore summed there for a run of blocks only, and runs
// are added up in the epilogue's registers.
//
// Bound by the tensor cores: 256 x 256 is the largest tile whose accumulators fit
// TMEM twice and halves what each CTA loads of B; 64 products a block is a swizzle's
// 128 bytes, six blocks in flight all that shared memory holds beside 32 KB on its way
// out.  4096 tokens of 2048 x 50001: logits 511 us (1.64 PFLOP/s; tensor cores 81%
// busy, the logits' way out takes shared memory's bandwidth), both gradients 846 us
// (1.98 PFLOP/s, 94%).

constexpr int kSide = 256;             // rows and columns of a pair's tile
constexpr int kHalf = kSide / 2;       // ... of A and of B in one CTA
constexpr int kDeep = 64;              // products of a block: 128 bytes of bf16
constexpr uint32_t kStages = 6;        // blocks of A and B (of float32 a plane's) in flight
constexpr uint32_t kOperandBytes = kHalf * kDeep * 2, kStageBytes = 2 * kOperandBytes;
constexpr int kProductThreads = 384, kEpilogueWarp = 4, kEpilogueWarps = 8;
constexpr uint32_t kStagedBytes = 32 * 128;  // of an epilogue warp: 32 rows' part of a result on its way out
constexpr int kTmemColumns = 512;

static_assert(kStages % kMaxPlanes == 0, "a float32 block's stages follow each other");
static_assert(kSide == static_cast<int>(kLossTile) && kHalf == static_cast<int>(kStatColumns),
              "statistics are of an epilogue thread's columns");

// Barriers, in 8-byte words of shared memory.
enum : uint32_t {
    kFullBar = 0,                      // a stage's blocks are there (the pair's; in its first CTA)
    kEmptyBar = kFullBar + kStages,    // ... have been read
    kReadyBar = kEmptyBar + kStages,   // an accumulator is complete
    kFreeBar = kReadyBar + 2,          // ... has been read (in the pair's first CTA)
    kDoneBar = kFreeBar + 2,           // the products issued are complete
    kTmemWord = kDoneBar + 1,
    kBarWords = kTmemWord + 1
};
// (1024: to a swizzle's boundary)
constexpr uint32_t kProductSmem = kStages * kStageBytes + kEpilogueWarps * kStagedBytes + kBarWords * 8 + 1024;

// One or two products in one launch.
struct ProductParams {
    CUtensorMap a[2], b[2];  // of logits a[1] is theirs
    CUtensorMap low[2];      // A's second and third plane, if they are in a float32 matrix's place
    ProductArgs args[2];
    RecordArgs record;
};

// As mbar_wait, without a call: accumulators live in registers across it.
__device__ __forceinline__ bool mbar_wait_here(uint32_t bar, uint32_t parity) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer() - t0 > kWaitNs) return false;
    return true;
}

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// The address of the pair's first CTA's copy of a shared variable.
__device__ __forceinline__ uint32_t in_first(uint32_t addr) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(a) : "r"(addr));
    return a;
}

__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}

// A block of 64 x rows x 1 of a tensor into this CTA's shared memory; its bytes
// count for a barrier of the pair's first CTA.
__device__ __forceinline__ void tma_load(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4}], [%5];" ::"r"(dst),
        "l"(map), "r"(x), "r"(y), "r"(z), "r"(bar)
        : "memory");
}

// The same of a group of columns of a low plane.
__device__ __forceinline__ void tma_load_low(uint32_t dst, const CUtensorMap* map, int plane, int group, int y,
                                             uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, "
        "%4, %5}], [%6];" ::"r"(dst),
        "l"(map), "r"(0), "r"(plane), "r"(group), "r"(y), "r"(bar)
        : "memory");
}

// Shared memory descriptor of a bf16 operand in 128-byte swizzled rows of 64
// values.  Rows along k: eight rows are 1024 bytes.  Turned (rows along the other
// axis): eight values of k are 1024 bytes, the next 64 of the other axis start
// kDeep rows on.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr, bool turned) {
    const uint64_t lead = turned ? kDeep * 128 : 16, stride = 1024;
    return static_cast<uint64_t>((addr >> 4) & 0x3FFF) | ((lead >> 4) << 16) | ((stride >> 4) << 32) |
           (uint64_t(1) << 46) | (uint64_t(2) << 61);
}

// float32 accumulators of bf16 products, M = 256 and N = width over the pair.
__device__ __forceinline__ uint32_t mma_desc(bool a_turned, bool b_turned, uint32_t width) {
    return (1u << 4) | (1u << 7) | (1u << 10) | (a_turned ? 1u << 15 : 0u) | (b_turned ? 1u << 16 : 0u) |
           ((width >> 3) << 17) | (static_cast<uint32_t>(kSide >> 4) << 24);
}

__device__ __forceinline__ void mma(uint32_t tmem, uint64_t a, uint64_t b, uint32_t desc, uint32_t add) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem),
        "l"(a), "l"(b), "r"(desc), "r"(add)
        : "memory");
}

// Arrives at the barrier in both CTAs once the products issued so far are complete.
__device__ __forceinline__ void mma_commit(uint32_t bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}

// 16 columns of the warp's lanes; tmem_wait_ld before their use.
__device__ __forceinline__ void tmem_read16(uint32_t taddr, float* v) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, "
        "[%16];"
        : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]),
          "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15])
        : "r"(taddr)
        : "memory");
}

__device__ __forceinline__ void tmem_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// No use of 16 values read from tensor memory before the wait that precedes this.
__device__ __forceinline__ void tmem_arrived(float* v) {
    asm volatile(""
                 : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]),
                   "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]));
}

// The tiles of a product and the blocks of each.
struct Tiles {
    uint32_t m, blocks, splits, per;  // rows of A, blocks of k, ... of a split
    uint32_t tall, wide, group, total;  // the launch makes sure that total fits
    __device__ __forceinline__ void set(const ProductArgs& a) {
        const uint32_t count = *a.count, left = count > a.base ? count - a.base : 0;
        m = a.count_m ? min(a.m, left) : a.m;
        blocks = ((a.count_k ? min(a.k, left) : a.k) + kDeep - 1) / kDeep;
        tall = (m + kSide - 1) / kSide;
        wide = (a.n + a.width - 1) / a.width;
        group = a.group;
        splits = a.splits;
        per = (blocks + splits - 1) / splits;
        total = tall * wide * splits;
    }
    // Tile t: in each split, groups of `group` rows of tiles, column by column.
    __device__ __forceinline__ void at(uint32_t t, uint32_t& mt, uint32_t& nt, uint32_t& split, uint32_t& lo,
                                       uint32_t& n) const {
        const uint32_t each = tall * wide;
        split = splits == 1 ? 0 : t / each;
        const uint32_t r = t - split * each;
        const uint32_t g = r / (group * wide), rest = r - g * group * wide;
        const uint32_t rows = min(group, tall - g * group);
        nt = rest / rows;
        mt = g * group + rest - nt * rows;
        lo = min(blocks, split * per);
        n = min(blocks, lo + per) - lo;
    }
};

// What each pair works on, alike in every role: the tiles of the first product in
// turn; then the second's, of which the pairs with fewer of the first's take as
// many more as take the same time.
struct Work {
    Tiles tiles[2];
    uint32_t first, pairs, over, early;
    __device__ __forceinline__ void set(const ProductArgs* a, int n, uint32_t pairs_) {
        pairs = pairs_;
        tiles[0].set(a[0]);
        if (n > 1) tiles[1].set(a[1]);
        else tiles[1].total = 0;
        first = tiles[0].total / pairs;
        over = tiles[0].total - first * pairs;
        early = 0;
        const uint64_t cost = n > 1 ? static_cast<uint64_t>(tiles[1].blocks) * a[1].width : 0;
        if (over && cost)
            early = static_cast<uint32_t>(min(static_cast<uint64_t>(tiles[0].per) * a[0].width / cost,
                                              static_cast<uint64_t>(tiles[1].total / (pairs - over))));
    }
    // The pair's i-th tile: of which product, which.
    __device__ __forceinline__ bool pick(uint32_t i, uint32_t pair, uint32_t& which, uint32_t& t) const {
        const uint32_t mine = first + (pair < over);
        which = i >= mine;
        if (!which) {
            t = pair + i * pairs;
            return true;
        }
        const uint32_t j = i - mine, others = pairs - over;  // pairs with fewer of the first product's tiles
        if (pair < over) t = early * others + j * pairs + others + pair;
        else if (j < early) t = j * others + (pair - over);
        else t = early * others + (j - early) * pairs + (pair - over);
        return t < tiles[1].total;
    }
};

// The plane in the q-th of a float32 block's three stages.
__device__ __forceinline__ int plane_at(int q) { return q == 0 ? 1 : q == 1 ? 0 : 2; }

// A row's next id at or behind column v, as its place in the list.
__device__ __forceinline__ int first_id(const int32_t* ids, int top, int32_t v) {
    int lo = 0, hi = top;
    while (lo < hi) {
        const int mid = (lo + hi) / 2;
        if (ids[mid] < v) lo = mid + 1;
        else hi = mid;
    }
    return lo;
}

// One thread's half row of a tile.
struct Place {
    uint64_t row;   // of C
    uint32_t n0;    // first column, and how many there are
    uint32_t cols;
    bool in;
    uint32_t staged;  // the warp's shared memory
    uint32_t lane;
};

// The warp's 32 rows' 128 bytes each, word(0..31) this lane's, to shared memory ...
template <class Word>
__device__ __forceinline__ void stage(const Place& p, Word word) {
    __syncwarp();
#pragma unroll
    for (uint32_t j = 0; j < 8; ++j)
        sts128(p.staged + p.lane * 128 + ((j ^ (p.lane & 7)) << 4),
               make_uint4(word(4 * j), word(4 * j + 1), word(4 * j + 2), word(4 * j + 3)));
    __syncwarp();
}

// ... whose rows' words are then a lane's each,
__device__ __forceinline__ uint32_t staged_word(const Place& p, uint32_t r) {
    return lds32(p.staged + r * 128 + ((p.lane / 4 ^ (r & 7)) << 4) + p.lane % 4 * 4);
}

// or given to use() in 16 bytes by eight lanes a row: whole lines for memory.
template <class Word, class Use>
__device__ __forceinline__ void transposed(const Place& p, Word word, Use use) {
    stage(p, word);
#pragma unroll 4
    for (uint32_t i = 0; i < 8; ++i) {
        const uint32_t r = 4 * i + p.lane / 8, j = p.lane % 8;
        use(r, j, lds128(p.staged + r * 128 + ((j ^ (r & 7)) << 4)));
    }
}

// The same for rows that follow each other `pitch` elements apart, from `to` on (the
// first row's first of these columns): use(address of a row's 16 bytes, they).
template <class T, class Word, class Use>
__device__ __forceinline__ void walked(const Place& p, Word word, T* to, uint64_t pitch, uint32_t rows, Use use) {
    stage(p, word);
    const uint32_t r0 = p.lane / 8, j = p.lane % 8;
    T* q = to + r0 * pitch + j * (16 / sizeof(T));
    const uint64_t step = 4 * pitch;
#pragma unroll
    for (uint32_t i = 0; i < 8; ++i, q += step) {
        const uint4 x = lds128(p.staged + (4 * i + r0) * 128 + ((j ^ (4 * i + r0 & 7)) << 4));
        if (4 * i + r0 < rows) use(q, x);
    }
}

__device__ __forceinline__ float4 floats(uint4 v) {
    return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
}

// Logits: the largest and the sum of a thread's 128 columns, the logits, and those at
// the row's ids (where the gradients' kernel does not find them among the others).
struct LogitTile {
    const LogitArgs& g;
    uint64_t list = 0;
    int next = 0;
    int32_t next_id = kNoId;

    // Before the products are complete: the row's place in its list.
    const CUtensorMap* z_map;

    __device__ __forceinline__ LogitTile(const ProductArgs& a, const Place& p, const CUtensorMap* z_map_)
        : g(a.logit), z_map(z_map_) {
        if (!p.in || !g.at_ids) return;
        list = static_cast<uint64_t>(g.row[p.row]) * g.lists.top;
        next = first_id(g.lists.ids + list, g.lists.top, static_cast<int32_t>(g.v0 + p.n0));
        if (next < g.lists.top) next_id = g.lists.ids[list + next];
    }

    template <int C>
    __device__ __forceinline__ void chunk(const Place& p, float (&z)[32]) {
        const uint32_t c0 = 32 * C;
        if (g.z) {
            // rows behind the last are the workspace's too
            if (p.lane == 0) asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");  // the buffer before
            stage(p, [&](uint32_t j) { return __float_as_uint(z[j]); });
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            __syncwarp();
            if (p.lane == 0) {
                asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(z_map),
                             "r"(static_cast<int>(p.n0 + c0)), "r"(static_cast<int>(p.row)), "r"(p.staged)
                             : "memory");
                asm volatile("cp.async.bulk.commit_group;" ::: "memory");
            }
        }
        if (c0 + 32 > p.cols) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (c0 + j >= p.cols) z[j] = -kInf;
        }
        const int32_t v = static_cast<int32_t>(g.v0 + p.n0 + c0);
        while (next_id < v + 32) {  // a list ends at kNoId, or with its places
            const int at = next_id - v;
            float x = 0.f;
#pragma unroll
            for (int j = 0; j < 32; ++j)
                if (j == at) x = z[j];
            g.lists.logits[list + next] = x;
            ++next;
            next_id = next < g.lists.top ? g.lists.ids[list + next] : kNoId;
        }
    }

    __device__ __forceinline__ void finish(const Place& p, float (&z)[4][32]) {
        chunk<0>(p, z[0]);
        chunk<1>(p, z[1]);
        chunk<2>(p, z[2]);
        chunk<3>(p, z[3]);
        float m[4] = {-kInf, -kInf, -kInf, -kInf}, part[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 32; ++j)
#pragma unroll
            for (int h = 0; h < 4; ++h) m[h] = fmaxf(m[h], z[h][j]);
        // c > 0: the largest y is the largest z's
        const float top = __fmul_rn(fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])), g.c), base = top == -kInf ? 0.f : top;
#pragma unroll
        for (int j = 0; j < 32; ++j)
#pragma unroll
            for (int h = 0; h < 4; ++h) part[h] = __fadd_rn(part[h], exp2_fast(__fmaf_rn(z[h][j], g.c, -base)));
        if (p.in && p.cols)
            g.stats[p.row * g.stats_pitch + p.n0 / kStatColumns] =
                make_float2(top, __fadd_rn(__fadd_rn(part[0], part[1]), __fadd_rn(part[2], part[3])));
    }
};

// Four columns of a row of the caller's matrix.
__device__ __forceinline__ void store_four(const OutArgs& o, uint64_t at, uint32_t cols, float4 x) {
    if (cols >= 4) {
        if (o.bf16) {
            uint16_t* p = static_cast<uint16_t*>(o.out) + at;
            if ((reinterpret_cast<uintptr_t>(p) & 7) == 0) {
                if (o.accumulate) {
                    const uint2 y = *reinterpret_cast<const uint2*>(p);
                    x = make_float4(__fadd_rn(x.x, bf_lo(y.x)), __fadd_rn(x.y, bf_hi(y.x)), __fadd_rn(x.z, bf_lo(y.y)),
                                    __fadd_rn(x.w, bf_hi(y.y)));
                }
                *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w));
                return;
            }
        } else {
            float* p = static_cast<float*>(o.out) + at;
            if ((reinterpret_cast<uintptr_t>(p) & 15) == 0) {
                if (o.accumulate) {
                    const float4 y = *reinterpret_cast<const float4*>(p);
                    x = make_float4(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y), __fadd_rn(x.z, y.z), __fadd_rn(x.w, y.w));
                }
                *reinterpret_cast<float4*>(p) = x;
                return;
            }
        }
    }
    const float v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (uint32_t j = 0; j < 4; ++j)
        if (j < cols) store_out(o.out, at + j, o.bf16, o.accumulate, v[j]);
}

struct OutTile {
    const OutArgs& args;
    uint64_t to = 0;  // this lane's row in the caller's matrix
    float scale;

    __device__ __forceinline__ OutTile(const ProductArgs& a, const Place& p) : args(a.out) {
        scale = __fmul_rn(*args.factor, args.t);
        if (p.in) to = (args.row ? static_cast<uint64_t>(args.row[p.row]) : p.row) * args.stride;
    }

    // Rows off a 16-byte boundary go row by row, a lane a word: lines are written
    // whole but at their ends.  (By 4-byte stores of 16 bytes' lanes, 30 MB of float32
    // rows of 515 took 60 us longer.)
    __device__ __forceinline__ void finish(const Place& p, float (&z)[4][32], float* part) const {
        if (p.cols == 0) return;
        // copies: read through the reference again after every store, they made a tile of
        // 256 x 192 float32 off alignment take 13 us
        OutArgs o;
        o.out = args.out;
        o.add = args.add;
        o.bf16 = args.bf16;
        o.accumulate = args.accumulate;
        o.sum_pitch = args.sum_pitch;
        const uint32_t rows = __popc(__ballot_sync(kFull, p.in));  // the warp's first ones
        const uint64_t row0 = p.row - p.lane;
        float* sum = part ? part : args.sum;
        const uint64_t pitch = part ? args.part_pitch : o.sum_pitch;
        const uintptr_t mine = reinterpret_cast<uintptr_t>(o.out) + (to + p.n0) * (o.bf16 ? 2 : 4);
        const bool aligned = __all_sync(kFull, (mine & 15) == 0 || !p.in), mapped = args.row != nullptr;
        if (!sum && !o.add && o.bf16 && !o.accumulate) {
            // two values a word: 64 columns at a time
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                auto word = [&](uint32_t j) {
                    const float(&x)[32] = z[2 * h + j / 16];
                    return pack_bf16x2(__fmul_rn(x[2 * j % 32], scale), __fmul_rn(x[2 * j % 32 + 1], scale));
                };
                const uint32_t c0 = 64 * h;
                if (c0 >= p.cols) break;
                if (aligned && !mapped && c0 + 64 <= p.cols) {
                    walked(p, word, static_cast<uint16_t*>(o.out) + __shfl_sync(kFull, to, 0) + p.n0 + c0, args.stride, rows,
                           [&](uint16_t* q, uint4 x) { *reinterpret_cast<uint4*>(q) = x; });
                    continue;
                }
                if (aligned && c0 + 64 <= p.cols) {
                    transposed(p, word, [&](uint32_t r, uint32_t j, uint4 x) {
                        uint16_t* q = static_cast<uint16_t*>(o.out) + __shfl_sync(kFull, to, r) + p.n0 + c0 + 8 * j;
                        if (r < rows) *reinterpret_cast<uint4*>(q) = x;
                    });
                    continue;
                }
                stage(p, word);
                const uint32_t c = c0 + 2 * p.lane;
                // a row's address: one addition from row to row where they follow each other
                uint16_t* q = static_cast<uint16_t*>(o.out) + __shfl_sync(kFull, to, 0) + p.n0 + c;
#pragma unroll 4
                for (uint32_t r = 0; r < rows; ++r, q += args.stride) {
                    const uint32_t x = staged_word(p, r), before = __shfl_up_sync(kFull, x, 1);
                    uint16_t* at = mapped ? static_cast<uint16_t*>(o.out) + __shfl_sync(kFull, to, r) + p.n0 + c : q;
                    if ((reinterpret_cast<uintptr_t>(at) & 2) == 0) {
                        if (c + 1 < p.cols) *reinterpret_cast<uint32_t*>(at) = x;
                        else if (c < p.cols) *at = static_cast<uint16_t>(x);
                    } else {
                        // this lane's first value goes with the one before it
                        if (p.lane == 0) *at = static_cast<uint16_t>(x);
                        else if (c < p.cols) *reinterpret_cast<uint32_t*>(at - 1) = (before >> 16) | (x << 16);
                        else if (c - 1 < p.cols) at[-1] = static_cast<uint16_t>(before >> 16);
                        if (p.lane == 31 && c + 1 < p.cols) at[1] = static_cast<uint16_t>(x >> 16);
                    }
                }
            }
            return;
        }
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            const uint32_t c0 = 32 * h;
            auto word = [&](uint32_t j) { return __float_as_uint(__fmul_rn(z[h][j], scale)); };
            if (c0 >= p.cols) break;
            const bool fresh = !o.add && (sum || (!mapped && !o.bf16 && !o.accumulate));
            if (fresh && (sum || (aligned && c0 + 32 <= p.cols))) {
                // float32 as it is, into the workspace (whole tiles there) or the caller's rows
                float* first = sum ? sum + row0 * pitch : static_cast<float*>(o.out) + __shfl_sync(kFull, to, 0);
                walked(p, word, first + p.n0 + c0, sum ? pitch : args.stride, rows,
                       [&](float* q, uint4 x) { *reinterpret_cast<uint4*>(q) = x; });
                continue;
            }
            if (sum || (aligned && c0 + 32 <= p.cols)) {
                transposed(p, word, [&](uint32_t r, uint32_t j, uint4 bits) {
                    const uint32_t c = c0 + 4 * j;
                    const uint64_t at = __shfl_sync(kFull, to, r) + p.n0 + c;
                    if (r >= rows || c >= p.cols) return;
                    float4 x = floats(bits);
                    if (o.add) {
                        const float4 y = *reinterpret_cast<const float4*>(o.add + (row0 + r) * o.sum_pitch + p.n0 + c);
                        x = make_float4(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y), __fadd_rn(x.z, y.z), __fadd_rn(x.w, y.w));
                    }
                    if (sum) *reinterpret_cast<float4*>(sum + (row0 + r) * pitch + p.n0 + c) = x;  // whole tiles there
                    else store_four(o, at, 4, x);
                });
                continue;
            }
            stage(p, word);
            const uint32_t c = c0 + p.lane;
            if (!mapped && !o.add && !o.bf16 && !o.accumulate) {
                float* q = static_cast<float*>(o.out) + __shfl_sync(kFull, to, 0) + p.n0 + c;
                const uint64_t stride = args.stride;
                if (c >= p.cols) continue;
#pragma unroll 8
                for (uint32_t r = 0; r < rows; ++r, q += stride) *q = __uint_as_float(staged_word(p, r));
                continue;
            }
            for (uint32_t r = 0; r < rows; ++r) {
                const uint64_t at = __shfl_sync(kFull, to, r) + p.n0 + c;
                float x = __uint_as_float(staged_word(p, r));
                if (c >= p.cols) continue;
                if (o.add) x = __fadd_rn(x, o.add[(row0 + r) * o.sum_pitch + p.n0 + c]);
                store_out(o.out, at, o.bf16, o.accumulate, x);
            }
        }
    }
};

// The record, by a warp that has nothing else to do.
__device__ void write_record(const RecordArgs& a, uint32_t lane) {
    const uint32_t count = *a.rows.count;
    if (count == 0) return;  // written when the rows were
    double sum = 0.0;
    bool bad = false;
#pragma unroll 4
    for (uint32_t r = lane; r < count; r += 32) {
        const float x = a.loss[r];
        sum += x;
        bad = bad || !finite(x);
    }
    for (int o = 16; o > 0; o /= 2) sum += __shfl_down_sync(kFull, sum, o);
    bad = __any_sync(kFull, bad);
    if (lane != 0) return;
    const float factor = *a.rows.factor;
    a.result[0] = static_cast<float>(sum * factor);
    a.result[1] = static_cast<float>(count);
    a.result[2] = bad ? 1.f : 0.f;
    a.result[3] = factor;
}

// LOGITS: one product of two matrices along k, the softmax's statistics in its
// epilogue.  Otherwise one or two with B turned, into the caller's memory.  A and B
// are of one plane each, of three each (six products a term), or A of three and B of one.
template <bool LOGITS, int kPlanes, int kPlanesB>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kProductThreads, 1)
    product_kernel(const __grid_constant__ ProductParams p, int products) {
    extern __shared__ char raw[];
    __shared__ Work work;
    constexpr bool BT = !LOGITS;
    const uint32_t base = (smem_addr(raw) + 1023) & ~1023u;  // the same in both CTAs
    const uint32_t staged = base + kStages * kStageBytes, bars = staged + kEpilogueWarps * kStagedBytes;
    auto bar = [bars](uint32_t i) { return bars + 8 * i; };
    griddep_launch_dependents();
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32, rank = cluster_rank();
    if (threadIdx.x == 0) {
        for (uint32_t s = 0; s < kStages; ++s) {
            mbar_init(bar(kFullBar + s), 1);
            mbar_init(bar(kEmptyBar + s), 1);
        }
        for (uint32_t b = 0; b < 2; ++b) {
            mbar_init(bar(kReadyBar + b), 1);
            mbar_init(bar(kFreeBar + b), 2 * kEpilogueWarps);
        }
        mbar_init(bar(kDoneBar), 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        for (int i = 0; i < products; ++i) {
            asm volatile("prefetch.tensormap [%0];" ::"l"(&p.a[i]) : "memory");
            asm volatile("prefetch.tensormap [%0];" ::"l"(&p.b[i]) : "memory");
        }
        griddep_wait();
        work.set(p.args, products, gridDim.x / 2);
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(bar(kTmemWord)),
                     "r"(kTmemColumns)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
        tmem_fence_before();
    }
    __syncwarp();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    const uint32_t tmem = lds32(bar(kTmemWord));
    griddep_wait();
    const uint32_t pair = blockIdx.x / 2;
    uint32_t mt, nt, split, lo, n, which, t;
    bool ok = true;
    if (warp == 0 && lane == 0) {
        const uint32_t full0 = in_first(bar(kFullBar));
        uint32_t s = 0, round = 0;
        for (uint32_t j = 0; ok && work.pick(j, pair, which, t); ++j) {
            const ProductArgs& a = p.args[which];
            const CUtensorMap *ma = &p.a[which], *mb = &p.b[which];
            work.tiles[which].at(t, mt, nt, split, lo, n);
            const bool at = !LOGITS && a.a.turned;
            const int m0 = static_cast<int>(mt * kSide + rank * kHalf);
            const int n0 = static_cast<int>(nt * a.width + rank * (a.width / 2));
            for (uint32_t i = 0; i < n && ok; ++i) {
                const int k0 = static_cast<int>((lo + i) * kDeep);
                for (int q = 0; q < kPlanes; ++q) {
                    if (round > 0 && !(ok = mbar_wait_here(bar(kEmptyBar + s), (round - 1) & 1))) break;
                    const int plane = kPlanesB == 1 ? 0 : plane_at(q);
                    const uint32_t full = full0 + 8 * s, to = base + s * kStageBytes;
                    const bool with_b = q < kPlanesB;  // one plane of B: in the first of A's stages
                    if (rank == 0) mbar_expect_tx(bar(kFullBar + s), 2 * (with_b ? kStageBytes : kOperandBytes));
                    if (kPlanes > kPlanesB && q > 0) {
                        if (at) {
                            tma_load_low(to, &p.low[which], q - 1, m0 / kDeep, k0, full);
                            tma_load_low(to + kOperandBytes / 2, &p.low[which], q - 1, m0 / kDeep + 1, k0, full);
                        } else {
                            tma_load_low(to, &p.low[which], q - 1, k0 / kDeep, m0, full);
                        }
                    } else if (at) {
                        tma_load(to, ma, m0, k0, plane, full);
                        tma_load(to + kOperandBytes / 2, ma, m0 + 64, k0, plane, full);
                    } else {
                        tma_load(to, ma, k0, m0, plane, full);
                    }
                    if (with_b && BT) {
                        tma_load(to + kOperandBytes, mb, n0, k0, plane, full);
                        tma_load(to + kOperandBytes + kOperandBytes / 2, mb, n0 + 64, k0, plane, full);
                    } else if (with_b) {
                        tma_load(to + kOperandBytes, mb, k0, n0, plane, full);
                    }
                    if (++s == kStages) s = 0, ++round;
                }
            }
        }
        // the last blocks have been read before the pair's memory goes
        for (uint32_t i = 0; i < kStages; ++i) {
            if (round > 0 && !mbar_wait_here(bar(kEmptyBar + s), (round - 1) & 1)) ok = false;
            if (++s == kStages) s = 0, ++round;
        }
        if (rank == 1 && !mbar_wait_here(bar(kDoneBar), 0)) ok = false;
    } else if (warp == 1 && lane == 0 && rank == 0) {
        uint32_t s = 0, phase = 0, done = 0;
        for (uint32_t i0 = 0; ok && work.pick(i0, pair, which, t); ++i0) {
            const ProductArgs& a = p.args[which];
            work.tiles[which].at(t, mt, nt, split, lo, n);
            const bool turned = !LOGITS && a.a.turned;
            // a descriptor's address is its low bits, in units of 16 bytes
            const uint64_t a0 = operand_desc(base, turned), b0 = operand_desc(base + kOperandBytes, BT);
            const uint32_t desc = mma_desc(turned, BT, a.width), a_step = turned ? 2048 / 16 : 32 / 16, run = a.run;
            for (uint32_t i = 0; i < n && ok; ++done) {
                const uint32_t b = done & 1, acc = tmem + b * kSide;
                if (done >= 2 && !(ok = mbar_wait_here(bar(kFreeBar + b), (done / 2 - 1) & 1))) break;
                tmem_fence_after();
                const uint32_t end = n - i > run ? i + run : n;
                // the products of A's block in one stage and B's in another
                auto multiply = [&](uint32_t sa, uint32_t sb, bool add) {
#pragma unroll
                    for (uint32_t k = 0; k < kDeep / 16; ++k)
                        mma(acc, a0 + (sa * (kStageBytes / 16) + k * a_step),
                            b0 + (sb * (kStageBytes / 16) + k * (BT ? 2048 / 16 : 32 / 16)), desc, add || k > 0);
                };
                auto full = [&](uint32_t stage) {
                    if (!mbar_wait_here(bar(kFullBar + stage), phase)) return false;
                    tmem_fence_after();
                    return true;
                };
                for (uint32_t j = i; j < end; ++j) {
                    if constexpr (kPlanes == 1) {
                        if (!(ok = full(s))) break;
                        multiply(s, s, j > i);
                        mma_commit(bar(kEmptyBar + s));
                    } else if constexpr (kPlanesB == 1) {
                        if (!(ok = full(s))) break;
                        multiply(s, s, j > i);
                        if (!(ok = full(s + 1))) break;
                        multiply(s + 1, s, true);
                        if (!(ok = full(s + 2))) break;
                        multiply(s + 2, s, true);
                        mma_commit(bar(kEmptyBar + s));
                        mma_commit(bar(kEmptyBar + s + 1));
                        mma_commit(bar(kEmptyBar + s + 2));
                    } else {
                        // planes 1, 0, 2: the first one's stage is free for the next block but one
                        // while the others are still read
                        if (!(ok = full(s))) break;
                        multiply(s, s, j > i);
                        if (!(ok = full(s + 1))) break;
                        multiply(s, s + 1, true);
                        multiply(s + 1, s, true);
                        mma_commit(bar(kEmptyBar + s));
                        multiply(s + 1, s + 1, true);
                        if (!(ok = full(s + 2))) break;
                        multiply(s + 1, s + 2, true);
                        multiply(s + 2, s + 1, true);
                        mma_commit(bar(kEmptyBar + s + 1));
                        mma_commit(bar(kEmptyBar + s + 2));
                    }
                    s += kPlanes;
                    if (s == kStages) s = 0, phase ^= 1;
                }
                if (!ok) break;
                mma_commit(bar(kReadyBar + b));
                i = end;
            }
        }
        mma_commit(bar(kDoneBar));
        if (!mbar_wait_here(bar(kDoneBar), 0)) ok = false;
    } else if (!LOGITS && warp == 3 && blockIdx.x == 0) {
        if (p.record.result) write_record(p.record, lane);
    } else if (warp >= kEpilogueWarp) {
        const uint32_t quarter = warp % 4, half = (warp - kEpilogueWarp) / 4;
        const uint32_t lanes = tmem + ((quarter * 32) << 16) + half * kHalf;
        uint32_t done = 0;
        Place at;
        at.staged = staged + (warp - kEpilogueWarp) * kStagedBytes;
        at.lane = lane;
        for (uint32_t i0 = 0; work.pick(i0, pair, which, t); ++i0) {
            const ProductArgs& a = p.args[LOGITS ? 0 : which];
            work.tiles[which].at(t, mt, nt, split, lo, n);
            at.row = static_cast<uint64_t>(mt) * kSide + rank * kHalf + quarter * 32 + lane;
            at.in = at.row < work.tiles[which].m;
            at.n0 = nt * a.width + half * kHalf;
            const uint32_t end = min(a.n, (nt + 1) * a.width);
            at.cols = end > at.n0 ? min(static_cast<uint32_t>(kHalf), end - at.n0) : 0;
            auto tile = [&] {
                if constexpr (LOGITS) return LogitTile(a, at, &p.a[1]);
                else return OutTile(a, at);
            }();
            float z[4][32];
            uint32_t i = 0;
            // a run's accumulators, waited for; its buffer, given back
            auto ready = [&] {
                ok = __all_sync(kFull, mbar_wait_here(bar(kReadyBar + (done & 1)), (done / 2) & 1));
                tmem_fence_after();
                return ok;
            };
            auto release = [&] {
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) arrive_cluster(in_first(bar(kFreeBar + (done & 1))));
                ++done;
                i = n - i > a.run ? i + a.run : n;
            };
            if (n > 0) {
                if (!ready()) break;
#pragma unroll
                for (int h = 0; h < 8; ++h) tmem_read16(lanes + (done & 1) * kSide + 16 * h, z[h / 2] + 16 * (h & 1));
                tmem_wait_ld();
#pragma unroll
                for (int h = 0; h < 8; ++h) tmem_arrived(z[h / 2] + 16 * (h & 1));
                release();
            } else {
#pragma unroll
                for (int h = 0; h < 4; ++h)
#pragma unroll
                    for (int j = 0; j < 32; ++j) z[h][j] = 0.f;
            }
            // 32 columns at a time where registers are left for them (515 float32 tokens'
            // gradients spill: 173 us instead of 167)
            constexpr int kAhead = LOGITS ? 2 : 1;
            while (i < n) {
                if (!ready()) break;
#pragma unroll
                for (int h = 0; h < 8; h += kAhead) {
                    float x[kAhead][16];
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) tmem_read16(lanes + (done & 1) * kSide + 16 * (h + k), x[k]);
                    tmem_wait_ld();
#pragma unroll
                    for (int k = 0; k < kAhead; ++k) {
                        float* to = z[(h + k) / 2] + 16 * ((h + k) & 1);
                        tmem_arrived(x[k]);
#pragma unroll
                        for (int j = 0; j < 16; ++j) to[j] = __fadd_rn(to[j], x[k][j]);
                    }
                }
                release();
            }
            if (!ok) break;
            if constexpr (LOGITS) {
                tile.finish(at, z);
            } else {
                const Tiles& tiles = work.tiles[which];
                const uint64_t part = static_cast<uint64_t>(tiles.tall) * kSide * a.out.part_pitch;
                tile.finish(at, z, tiles.splits > 1 ? a.out.parts + split * part : nullptr);
            }
        }
    }
    // the logits are in memory before the CTA's end
    if (LOGITS && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
    if (!ok) atomicOr(p.args[0].status, 1u);
    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    cluster_sync();
    tmem_fence_after();
    if (warp == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemColumns) : "memory");
}

// A split product's parts, added in their order: four columns a thread.
__global__ void __launch_bounds__(256) finish_kernel(const __grid_constant__ ProductArgs a) {
    griddep_launch_dependents();
    griddep_wait();
    Tiles tiles;
    tiles.set(a);
    const OutArgs& o = a.out;
    const uint64_t stride = static_cast<uint64_t>(tiles.tall) * kSide * o.part_pitch;
    const uint32_t quads = (a.n + 3) / 4;
    const uint64_t all = static_cast<uint64_t>(tiles.m) * quads;
    for (uint64_t i = blockIdx.x * 256ull + threadIdx.x; i < all; i += gridDim.x * 256ull) {
        const uint64_t r = i / quads;
        const uint32_t c = 4 * static_cast<uint32_t>(i - r * quads);
        const float* from = o.parts + r * o.part_pitch + c;
        float4 x = *reinterpret_cast<const float4*>(from);
#pragma unroll 8
        for (uint32_t s = 1; s < tiles.splits; ++s) {
            const float4 y = *reinterpret_cast<const float4*>(from + s * stride);
            x = make_float4(__fadd_rn(x.x, y.x), __fadd_rn(x.y, y.y), __fadd_rn(x.z, y.z), __fadd_rn(x.w, y.w));
        }
        store_four(o, (o.row ? static_cast<uint64_t>(o.row[r]) : r) * o.stride + c, a.n - c, x);
    }
}

using EncodeFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                              const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

// cuTensorMapEncodeTiled through the runtime's driver entry-point query (the
// library links only the static runtime); null if the driver has none.
EncodeFn encode_tiled() {
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q = cudaDriverEntryPointSymbolNotFound;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess) {
            cudaGetLastError();
            return static_cast<EncodeFn>(nullptr);
        }
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// Blocks of 64 columns x 128 rows (turned: 64 rows) of one plane; zeros outside.
// A tile narrower than 256 loads as much and multiplies less.
cudaError_t make_map(const Operand& o, CUtensorMap* map) {
    const EncodeFn encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const int planes = o.m.low ? 1 : o.m.planes;
    const cuuint64_t row = 2 * o.m.pitch, plane = planes > 1 ? 2 * o.m.plane : row;
    const cuuint64_t dims[3] = {o.cols, std::max<uint64_t>(1, o.rows), static_cast<cuuint64_t>(planes)};
    const cuuint64_t strides[2] = {row, plane};
    const cuuint32_t box[3] = {kDeep, static_cast<cuuint32_t>(o.turned ? kDeep : kHalf), 1}, steps[3] = {1, 1, 1};
    static_assert(kDeep == 64, "a block's rows are one swizzle wide, turned or not");
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, o.m.p, dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// The same blocks of the low planes: 64 columns, plane, group of columns, row.  Columns
// behind the last up to a group's end are zeros there.
cudaError_t make_low_map(const Operand& o, CUtensorMap* map) {
    const EncodeFn encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    static_assert(kLowGroup == kDeep, "a group of columns is a block's");
    const cuuint64_t dims[4] = {kDeep, 2, (o.cols + kDeep - 1) / kDeep, std::max<uint64_t>(1, o.rows)};
    const cuuint64_t strides[3] = {2 * kDeep, 4 * kDeep, 4 * o.m.pitch};
    const cuuint32_t box[4] = {kDeep, 1, 1, static_cast<cuuint32_t>(o.turned ? kDeep : kHalf)}, steps[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, o.m.low, dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

// ------------------------------------------------------------- a few tokens
//
// Up to eight tokens: the weights are read (and their gradient written) once by
// plain loads and every sum is a float32 fused multiply-add, for float32 inputs
// without the three planes of the tensor cores.  A CTA's 64 vocabulary entries are
// eight rows of W a warp, 16 bytes of each a lane where rows are aligned, else a
// value; eight rows' loads are in flight together.

constexpr int kFewThreads = 256, kFewRows = kFewColumns / (kFewThreads / 32), kFewDeep = 1024;

// VEC values of a row from i on.
template <bool BF16, int VEC>
__device__ __forceinline__ void few_load(const void* p, uint64_t i, float (&x)[VEC]) {
    if constexpr (VEC == 1) {
        x[0] = load_value(p, i, BF16);
    } else if constexpr (!BF16) {
        const float4 v = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + i);
        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
    } else if constexpr (VEC == 4) {
        const uint2 v = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + i);
        x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
    } else {
        const uint4 v = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(p) + i);
        x[0] = bf_lo(v.x), x[1] = bf_hi(v.x), x[2] = bf_lo(v.y), x[3] = bf_hi(v.y);
        x[4] = bf_lo(v.z), x[5] = bf_hi(v.z), x[6] = bf_lo(v.w), x[7] = bf_hi(v.w);
    }
}

// Where value d of a token lies in shared memory: a lane's VEC values in fours, so
// that a warp's reads of four are of consecutive addresses.
template <int VEC>
__device__ __forceinline__ uint32_t few_place(uint32_t d) {
    if (VEC <= 4) return d;
    return d / 256 * 256 + d % 8 / 4 * 128 + d % 256 / 8 * 4 + d % 4;
}

template <int N>
__device__ __forceinline__ uint32_t few_count(const FewArgs& a) {
    const uint32_t count = *a.rows.count;
    return count > a.base ? min(count - a.base, static_cast<uint32_t>(N)) : 0;
}

template <int N, bool BF16, int VEC>
__global__ void __launch_bounds__(kFewThreads) few_logits_kernel(const __grid_constant__ FewArgs a) {
    __shared__ __align__(16) float xs[N][kFewDeep];
    __shared__ float zs[N][kFewColumns];
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t v0 = blockIdx.x * kFewColumns;
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t count = few_count<N>(a);
    const int32_t* row = a.rows.row + a.base;
    float acc[kFewRows * N] = {};  // row by row
    uint64_t at[kFewRows];
#pragma unroll
    for (int j = 0; j < kFewRows; ++j)  // behind the vocabulary: its last entry, not used
        at[j] = min(v0 + warp * kFewRows + j, a.vocab - 1) * a.w_stride;
    for (uint32_t d0 = 0; d0 < a.width; d0 += kFewDeep) {
        const uint32_t deep = min(static_cast<uint32_t>(kFewDeep), a.width - d0);
        __syncthreads();
        for (uint32_t i = tid; i < N * kFewDeep; i += kFewThreads) {
            const uint32_t r = i / kFewDeep, d = i % kFewDeep;
            if (d < deep) xs[r][few_place<VEC>(d)] = r < count ? load_value(a.x, row[r] * a.x_stride + d0 + d, BF16) : 0.f;
        }
        __syncthreads();
#pragma unroll(VEC == 1 ? 4 : 1)
        for (uint32_t d = VEC * lane; d < deep; d += 32 * VEC) {
            float w[kFewRows][VEC];
#pragma unroll
            for (int j = 0; j < kFewRows; ++j) few_load<BF16, VEC>(a.w, at[j] + d0 + d, w[j]);
#pragma unroll
            for (int i = 0; i < VEC; i += VEC == 1 ? 1 : 4)
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    float x[4];
                    if constexpr (VEC == 1) {
                        x[0] = xs[r][d];
                    } else {
                        const float4 v = *reinterpret_cast<const float4*>(&xs[r][few_place<VEC>(d + i)]);
                        x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
                    }
#pragma unroll
                    for (int q = 0; q < (VEC == 1 ? 1 : 4); ++q)
#pragma unroll
                        for (int j = 0; j < kFewRows; ++j) acc[j * N + r] = __fmaf_rn(w[j][i + q], x[q], acc[j * N + r]);
                }
        }
    }
    // the lanes' sums: each step hands half of the values to the other half of the lanes
    int have = kFewRows * N, first = 0;
#pragma unroll
    for (int o = 16; o > 0; o /= 2) {
        const bool upper = lane & o;
        if (have > 1) {
            have /= 2;
#pragma unroll
            for (int i = 0; i < kFewRows * N / 2; ++i) {
                if (i >= have) break;
                const float give = upper ? acc[i] : acc[i + have], keep = upper ? acc[i + have] : acc[i];
                acc[i] = __fadd_rn(keep, __shfl_xor_sync(kFull, give, o));
            }
            first += upper ? have : 0;
        } else {
            acc[0] = __fadd_rn(acc[0], __shfl_xor_sync(kFull, acc[0], o));
        }
    }
#pragma unroll
    for (int i = 0; i < (N * kFewRows > 32 ? N * kFewRows / 32 : 1); ++i)
        zs[(first + i) % N][warp * kFewRows + (first + i) / N] = acc[i];
    __syncthreads();
    if (warp < count) {
        float top = -kInf, sum = 0.f;
#pragma unroll
        for (uint32_t i = lane; i < kFewColumns; i += 32) {
            if (v0 + i >= a.vocab) break;
            const float z = zs[warp][i];
            if (a.z) a.z[warp * a.z_pitch + v0 + i] = z;
            const float y = __fmul_rn(z, a.c);
            join_stat(top, sum, y, y == -kInf ? 0.f : 1.f);
        }
        for (int o = 16; o > 0; o /= 2) {
            const float t2 = __shfl_xor_sync(kFull, top, o), s2 = __shfl_xor_sync(kFull, sum, o);
            join_stat(top, sum, t2, s2);
        }
        if (lane == 0) a.stats[warp * a.stats_pitch + blockIdx.x] = make_float2(top, sum);
    }
    for (uint32_t k = tid; k < count * a.lists.top; k += kFewThreads) {
        const uint32_t r = k / a.lists.top;
        const uint64_t i = static_cast<uint64_t>(row[r]) * a.lists.top + (k - r * a.lists.top);
        const uint32_t v = static_cast<uint32_t>(a.lists.ids[i]) - v0;
        if (v < kFewColumns) a.lists.logits[i] = zs[r][v];
    }
}

// grad W = f t g^T X of the CTA's entries, and its part of grad X = f t g W: a thread
// four columns (VEC 4: next to each other, else `lanes` apart), `lanes` threads a
// row; the gradients of 64 entries' logits at a time.
template <int N, bool BF16, int VEC>
__global__ void __launch_bounds__(kFewThreads) few_gradients_kernel(const __grid_constant__ FewArgs a, uint32_t lanes,
                                                                    const __grid_constant__ RecordArgs record) {
    constexpr int kAhead = N <= 2 ? 8 : 4;  // rows of W whose loads are in flight
    __shared__ float gs[N][kFewColumns];
    __shared__ float sums[4 * kFewThreads];
    const uint32_t tid = threadIdx.x, tx = tid % lanes, ty = tid / lanes, rows = kFewThreads / lanes;
    const uint32_t c0 = VEC == 4 ? (blockIdx.x * lanes + tx) * 4 : blockIdx.x * 4 * lanes + tx, step = VEC == 4 ? 1 : lanes;
    griddep_launch_dependents();
    griddep_wait();
    if (blockIdx.x == 0 && blockIdx.y == 0 && tid < 32 && record.result) write_record(record, tid);
    const uint32_t count = few_count<N>(a);
    const int32_t* row = a.rows.row + a.base;
    if (count == 0 && a.base > 0) return;  // nothing to add
    const float scale = __fmul_rn(*a.rows.factor, a.t);
    float x[N][4], acc[N][4] = {};
#pragma unroll
    for (int r = 0; r < N; ++r)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const uint32_t c = c0 + j * step;
            x[r][j] = static_cast<uint32_t>(r) < count && c < a.width ? load_value(a.x, row[r] * a.x_stride + c, BF16) : 0.f;
        }
    const uint32_t lo = blockIdx.y * a.entries, hi = min(a.vocab, lo + a.entries);
    for (uint32_t v0 = lo; v0 < hi; v0 += kFewColumns) {
        __syncthreads();
        for (uint32_t i = tid; i < N * kFewColumns; i += kFewThreads) {
            const uint32_t r = i / kFewColumns, v = v0 + i % kFewColumns;
            float g = 0.f;
            if (r < count && v < hi)
                for (int q = a.g.planes - 1; q >= 0; --q)
                    g = __fadd_rn(g, bf16_value(a.g.p[q * a.g.plane + r * a.g.pitch + v]));
            gs[r][i % kFewColumns] = g;
        }
        __syncthreads();
        const uint32_t end = min(hi - v0, kFewColumns);
        for (uint32_t i0 = ty; i0 < end; i0 += kAhead * rows) {
            float w[kAhead][4] = {};
            if (a.grad_x && c0 < a.width) {
#pragma unroll
                for (int k = 0; k < kAhead; ++k) {
                    const uint64_t at = static_cast<uint64_t>(v0 + min(i0 + k * rows, end - 1)) * a.w_stride + c0;
                    if constexpr (VEC == 4) {
                        few_load<BF16, 4>(a.w, at, w[k]);
                    } else {
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            if (c0 + j * step < a.width) w[k][j] = load_value(a.w, at + j * step, BF16);
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const uint32_t i = i0 + k * rows;
                if (i >= end) break;
                float y[4] = {};
#pragma unroll
                for (int r = 0; r < N; ++r) {
                    const float g = gs[r][i];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        y[j] = __fmaf_rn(g, x[r][j], y[j]);
                        acc[r][j] = __fmaf_rn(g, w[k][j], acc[r][j]);
                    }
                }
                if (!a.grad_w || c0 >= a.width) continue;
                const uint64_t to = static_cast<uint64_t>(v0 + i) * a.grad_w_stride + c0;
#pragma unroll
                for (int j = 0; j < 4; ++j) y[j] = __fmul_rn(y[j], scale);
                const bool add = a.accumulate || a.base > 0;
                if (VEC == 4 && add && !a.grad_w_bf16) {
                    const float4 old = *reinterpret_cast<const float4*>(static_cast<const float*>(a.grad_w) + to);
                    y[0] = __fadd_rn(y[0], old.x), y[1] = __fadd_rn(y[1], old.y);
                    y[2] = __fadd_rn(y[2], old.z), y[3] = __fadd_rn(y[3], old.w);
                }
                if (VEC == 4 && !(add && a.grad_w_bf16)) {
                    if (a.grad_w_bf16)
                        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.grad_w) + to) =
                            make_uint2(pack_bf16x2(y[0], y[1]), pack_bf16x2(y[2], y[3]));
                    else
                        *reinterpret_cast<float4*>(static_cast<float*>(a.grad_w) + to) = make_float4(y[0], y[1], y[2], y[3]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        if (c0 + j * step < a.width) store_out(a.grad_w, to + j * step, a.grad_w_bf16, add, y[j]);
                }
            }
        }
    }
    if (!a.grad_x) return;
#pragma unroll
    for (int r = 0; r < N; ++r) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < 4; ++j) sums[j * kFewThreads + tid] = acc[r][j];
        __syncthreads();
        if (ty != 0) continue;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            float s = 0.f;
            for (uint32_t k = 0; k < rows; ++k) s = __fadd_rn(s, sums[j * kFewThreads + k * lanes + tx]);
            if (c0 + j * step < a.width) a.parts[(static_cast<uint64_t>(blockIdx.y) * N + r) * a.width + c0 + j * step] = s;
        }
    }
}

// grad X from its parts, in their order.
__global__ void __launch_bounds__(128) few_finish_kernel(const __grid_constant__ FewArgs a, uint32_t tokens,
                                                         uint32_t splits) {
    griddep_launch_dependents();
    griddep_wait();
    const uint32_t c = blockIdx.x * 128 + threadIdx.x, r = blockIdx.y;
    if (c >= a.width || a.base + r >= *a.rows.count) return;
    const float scale = __fmul_rn(*a.rows.factor, a.t);
    float s = 0.f;
#pragma unroll 8
    for (uint32_t k = 0; k < splits; ++k) s = __fadd_rn(s, a.parts[(static_cast<uint64_t>(k) * tokens + r) * a.width + c]);
    store_out(a.grad_x, a.rows.row[a.base + r] * a.grad_x_stride + c, a.grad_x_bf16, a.accumulate, __fmul_rn(s, scale));
}

template <class... Args>
cudaError_t launch(void (*f)(Args...), dim3 grid, int block, size_t smem, cudaStream_t st, const Args&... a) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = AR_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<Args*>(&a)...};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(f), args);
}

uint32_t ctas(uint64_t n, uint64_t each) { return static_cast<uint32_t>((n + each - 1) / each); }

uint64_t tall_of(const ProductArgs& a) { return (static_cast<uint64_t>(a.m) + kSide - 1) / kSide; }
uint64_t wide_of(const ProductArgs& a) { return (static_cast<uint64_t>(a.n) + a.width - 1) / a.width; }
uint64_t blocks_of(const ProductArgs& a) { return (static_cast<uint64_t>(a.k) + kDeep - 1) / kDeep; }

// Tiles as wide as they divide the columns evenly; rows of tiles side by side: all
// of them while A's rows stay in L2, then eight.  Measured, all against eight: logits
// of 4096 tokens of 2048 x 50001 460 against 468 us (16 MB of A), of 8192 of 4096 x
// 128000 4.49 against 4.48 ms (64 MB); dW of the two (410 MB and 2.1 GB) with its
// logits 1298 against 1204 us and 12.0 against 11.3 ms.
void set_shape(ProductArgs& a) {
    const uint32_t wide = ctas(a.n, kSide);
    a.width = (ctas(a.n, wide) + 31) / 32 * 32;
    const uint64_t tall = std::max<uint64_t>(1, tall_of(a));
    a.group = tall * kSide * a.k * 2 * a.a.m.planes > (64ull << 20) ? 8 : static_cast<uint32_t>(tall);
    a.splits = 1;
}

// Parts of the first product's k: the number that leaves the fullest pair the least
// to do, in columns of blocks, with what the parts cost (8 blocks' time for their
// launch, one for four parts of a tile).  Whole calls of float32 tokens with parts
// and without: 37 of 129 x 2003 40 and 87 us, 300 of 256 x 5003 60 and 180, 515 of
// 515 x 10007 173 and 363.
uint32_t splits_of(const ProductArgs& a, const ProductArgs* second, uint64_t room) {
    const uint64_t pairs = kLossSms / 2, tiles = tall_of(a) * wide_of(a), blocks = blocks_of(a);
    if (tiles == 0 || tiles >= 8 * pairs) return 1;
    const uint64_t passes = a.a.m.planes == 1 ? 1 : a.b.m.planes == 1 ? 3 : 6;
    const uint64_t most = std::min(blocks * passes / 4, room / (tall_of(a) * kSide * a.out.part_pitch));
    const uint64_t other = second ? blocks_of(*second) * second->width : 0;
    const uint64_t others = second ? tall_of(*second) * wide_of(*second) * other : 0;
    uint64_t best = 0;
    uint32_t splits = 0;
    auto look = [&](uint64_t s) {
        if (s > std::max<uint64_t>(1, most)) return;
        const uint64_t each = (blocks + s - 1) / s * a.width;
        const uint64_t even = (tiles * s * each + others) / pairs + other / 2;
        const uint64_t fullest = std::max((tiles * s + pairs - 1) / pairs * each, even);
        const uint64_t cost = fullest * passes + (s > 1 ? (8 + tiles * s / 4) * kSide : 0);
        if (splits == 0 || cost < best) {
            best = cost;
            splits = static_cast<uint32_t>(s);
        }
    };
    for (uint64_t s = 1; s <= 8; ++s) look(s);
    for (uint64_t s = 12; s <= pairs / tiles; s += 4) look(s);
    return splits;
}

}  // namespace

cudaError_t launch_teacher(const TeacherArgs& a, cudaStream_t st) {
    const size_t smem = static_cast<size_t>(kTeacherWarps) * 2 * a.k * 4;
    return launch(teacher_kernel, ctas(a.n, kTeacherWarps), 32 * kTeacherWarps, smem, st, a);
}

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) { return launch(rows_kernel, 1, kRowThreads, 0, st, a); }

cudaError_t launch_pack(const PackArgs& a, const PackArgs* b, cudaStream_t st) {
    const uint32_t first = ctas(a.n, kLossTile) * (kLossTile / 8), more = b ? ctas(b->n, kLossTile) * (kLossTile / 8) : 0;
    return launch(pack_kernel, first + more, 256, 0, st, a, b ? *b : a, first);
}

cudaError_t launch_join(const JoinArgs& a, cudaStream_t st) {
    return launch(join_kernel, ctas(a.n, kJoinRows), 32 * kJoinRows, 0, st, a);
}

cudaError_t launch_grad(const JoinArgs& a0, cudaStream_t st) {
    JoinArgs a = a0;
    const uint32_t rows = ctas(a.n, a.round) * a.round;
    a.columns = 128 * kGradThreads;  // less while a few waves of CTAs are not full
    while (a.columns > 8 * kGradThreads && static_cast<uint64_t>(a.n) * ctas(a.vocab, a.columns) < 16 * kLossSms)
        a.columns /= 2;
    return launch(grad_kernel, dim3(ctas(a.vocab, a.columns), std::min(rows, 32768u)), kGradThreads, 0, st, a);
}

using ProductKernel = void (*)(ProductParams, int);

// By the planes of A and of B.
ProductKernel product_of(bool logits, int a, int b) {
    if (a == 1) return logits ? product_kernel<true, 1, 1> : product_kernel<false, 1, 1>;
    if (b == 1) return product_kernel<false, kMaxPlanes, 1>;
    return logits ? product_kernel<true, kMaxPlanes, kMaxPlanes> : product_kernel<false, kMaxPlanes, kMaxPlanes>;
}

cudaError_t prepare_products() {
    for (const ProductKernel f : {product_of(true, 1, 1), product_of(false, 1, 1), product_of(false, kMaxPlanes, 1),
                                  product_of(true, kMaxPlanes, kMaxPlanes), product_of(false, kMaxPlanes, kMaxPlanes)}) {
        const cudaError_t e = cudaFuncSetAttribute(reinterpret_cast<const void*>(f),
                                                   cudaFuncAttributeMaxDynamicSharedMemorySize, kProductSmem);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

// The piece's logits, 32 rows of 32 columns a store.
cudaError_t make_logit_map(const LogitArgs& g, uint64_t rows, uint64_t columns, CUtensorMap* map) {
    const EncodeFn encode = encode_tiled();
    if (!encode) return cudaErrorNotSupported;
    const cuuint64_t dims[2] = {columns, rows}, strides[1] = {g.z_pitch * 4};
    const cuuint32_t box[2] = {32, 32}, steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 2, g.z, dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                  CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS
               ? cudaSuccess
               : cudaErrorInvalidValue;
}

namespace {

cudaError_t launch_tiles(ProductParams& p, int n, bool logits, cudaStream_t st) {
    uint64_t tiles = 0;
    for (int i = 0; i < n; ++i) {
        const ProductArgs& a = p.args[i];
        cudaError_t e = make_map(a.a, &p.a[i]);
        if (e == cudaSuccess) e = make_map(a.b, &p.b[i]);
        if (e == cudaSuccess && a.a.m.low) e = make_low_map(a.a, &p.low[i]);
        if (e != cudaSuccess) return e;
        tiles += tall_of(a) * wide_of(a) * a.splits;
    }
    if (tiles > 0x7FFFFFFFu) return cudaErrorInvalidValue;  // 2^22 tokens and 2^24 entries make 2^30
    const uint32_t pairs = static_cast<uint32_t>(std::min<uint64_t>(std::max<uint64_t>(1, tiles), kLossSms / 2));
    const ProductKernel f = product_of(logits, p.args[0].a.m.planes, p.args[0].b.m.planes);
    return launch(f, 2 * pairs, kProductThreads, kProductSmem, st, p, n);
}

}  // namespace

cudaError_t launch_logits(ProductArgs a, cudaStream_t st) {
    ProductParams p = {};
    set_shape(a);
    a.width = std::min<uint32_t>(kSide, ctas(a.n, 32) * 32);  // statistics are of whole tiles' halves
    p.args[0] = a;
    if (a.logit.z) {
        const cudaError_t e = make_logit_map(a.logit, tall_of(a) * kSide, wide_of(a) * kSide, &p.a[1]);
        if (e != cudaSuccess) return e;
    }
    return launch_tiles(p, 1, true, st);
}

cudaError_t launch_products(const ProductArgs* a, int n, uint64_t room, const RecordArgs& r, cudaStream_t st) {
    ProductParams p = {};
    p.record = r;
    for (int i = 0; i < n; ++i) {
        p.args[i] = a[i];
        set_shape(p.args[i]);
    }
    if (p.args[0].out.parts) p.args[0].splits = splits_of(p.args[0], n > 1 ? &p.args[1] : nullptr, room);
    const cudaError_t e = launch_tiles(p, n, false, st);
    if (e != cudaSuccess || p.args[0].splits == 1) return e;
    const uint32_t whole = ctas(static_cast<uint64_t>(a[0].m) * ctas(a[0].n, 4), 256);
    return launch(finish_kernel, std::min(std::max(1u, whole), 8 * kLossSms), 256, 0, st, p.args[0]);
}

namespace {

bool aligned(const void* p, uint64_t stride, int es, uint32_t width, uint32_t bytes) {
    return reinterpret_cast<uintptr_t>(p) % bytes == 0 && stride * es % bytes == 0 &&
           static_cast<uint64_t>(width) * es % bytes == 0;
}

template <int N>
cudaError_t few_logits(const FewArgs& a, cudaStream_t st) {
    const bool whole = aligned(a.w, a.w_stride, a.bf16 ? 2 : 4, a.width, 16);
    return launch(a.bf16 ? (whole ? few_logits_kernel<N, true, 8> : few_logits_kernel<N, true, 1>)
                         : (whole ? few_logits_kernel<N, false, 4> : few_logits_kernel<N, false, 1>),
                  ctas(a.vocab, kFewColumns), kFewThreads, 0, st, a);
}

template <int N>
cudaError_t few_gradients(FewArgs a, const RecordArgs& r, cudaStream_t st) {
    uint32_t lanes = 32;
    while (lanes < kFewThreads && 4 * lanes < a.width) lanes *= 2;
    const uint32_t wide = ctas(a.width, 4 * lanes);
    // four CTAs an SM
    const uint32_t most =
        std::min<uint64_t>(std::max(1u, 4 * kLossSms / wide), a.room / (static_cast<uint64_t>(N) * a.width));
    a.entries = ctas(ctas(a.vocab, std::max(1u, most)), kFewColumns) * kFewColumns;
    const uint32_t splits = ctas(a.vocab, a.entries);
    const bool whole = (!a.grad_x || aligned(a.w, a.w_stride, a.bf16 ? 2 : 4, a.width, a.bf16 ? 8 : 16)) &&
                       (!a.grad_w || aligned(a.grad_w, a.grad_w_stride, a.grad_w_bf16 ? 2 : 4, a.width, a.grad_w_bf16 ? 8 : 16)) &&
                       a.width % 4 == 0;
    cudaError_t e = launch(a.bf16 ? (whole ? few_gradients_kernel<N, true, 4> : few_gradients_kernel<N, true, 1>)
                                  : (whole ? few_gradients_kernel<N, false, 4> : few_gradients_kernel<N, false, 1>),
                           dim3(wide, splits), kFewThreads, 0, st, a, lanes, r);
    if (e == cudaSuccess && a.grad_x)
        e = launch(few_finish_kernel, dim3(ctas(a.width, 128), a.n), 128, 0, st, a, static_cast<uint32_t>(N), splits);
    return e;
}

}  // namespace

cudaError_t launch_few_logits(const FewArgs& a, cudaStream_t st) {
    return a.n <= 1   ? few_logits<1>(a, st)
           : a.n <= 2 ? few_logits<2>(a, st)
           : a.n <= 4 ? few_logits<4>(a, st)
                      : few_logits<8>(a, st);
}

cudaError_t launch_few_gradients(FewArgs a, const RecordArgs& r, cudaStream_t st) {
    return a.n <= 1   ? few_gradients<1>(a, r, st)
           : a.n <= 2 ? few_gradients<2>(a, r, st)
           : a.n <= 4 ? few_gradients<4>(a, r, st)
                      : few_gradients<8>(a, r, st);
}

}  // namespace ar
