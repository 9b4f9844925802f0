// Kernels of the output layer's losses: teacher lists, the tokens that count,
// the products over hidden size, vocabulary and tokens with the softmax in
// their epilogues, and the joins between them.
//
// With z = X W^T, y = z log2(e) / t and a token's shares p over a short list
// of ids, the loss is t^2 (sum p log p - sum p z / t + log sum exp(z / t)) and
// its gradient by z, with the factor f of the record,
//   g = f t (2^(y - top) / sum 2^(y - top) - p),   dX = g W,   dW = g^T X.
#include "device.cuh"
#include "outloss.hpp"

namespace ar {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;
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
    if ((b & 0x7FFFu) == 0x7F80u && fabsf(x) < __int_as_float(0x7F800000)) b -= 1;
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
// by id.  The k^2 comparisons of a list stay in shared memory.
__global__ void __launch_bounds__(32 * kTeacherWarps) teacher_kernel(const __grid_constant__ TeacherArgs a) {
    extern __shared__ char smem[];
    const uint32_t warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t i = blockIdx.x * kTeacherWarps + warp;
    int32_t* id = reinterpret_cast<int32_t*>(smem) + warp * 2 * a.k;
    float* share = reinterpret_cast<float*>(id + a.k);
    griddep_wait();
    if (i >= a.n) return;
    bool bad = false;
    float top = -__int_as_float(0x7F800000);
    for (int j = lane; j < a.k; j += 32) {
        const uint64_t at = i * a.ids_stride + j;
        const int64_t v = a.id_bytes == 8 ? static_cast<const int64_t*>(a.ids)[at] : static_cast<const int32_t*>(a.ids)[at];
        float u = -__int_as_float(0x7F800000);
        int32_t x = kNoId;
        if (v >= 0) {
            u = load_value(a.logits, i * a.logits_stride + j, a.logits_bf16);
            if (u != -__int_as_float(0x7F800000)) {  // NaN stays in
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
    bad = __any_sync(kFull, bad) || top == __int_as_float(0x7F800000);
    float sum = 0.f;
    for (int j = lane; j < a.k; j += 32) {
        const bool in = id[j] != kNoId && !bad;
        const float e = in ? expf(__fmul_rn(__fsub_rn(share[j], top), a.inv_t)) : 0.f;
        share[j] = e;
        sum = __fadd_rn(sum, e);
    }
    for (int o = 16; o > 0; o /= 2) sum = __fadd_rn(sum, __shfl_xor_sync(kFull, sum, o));
    const bool any = __any_sync(kFull, top != -__int_as_float(0x7F800000));
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
// order; every thread has a run of tokens.
__global__ void __launch_bounds__(kRowThreads) rows_kernel(const __grid_constant__ RowsArgs a) {
    __shared__ uint32_t sums[32];
    const uint32_t tid = threadIdx.x, lane = tid % 32, warp = tid / 32;
    const uint32_t run = (a.n + kRowThreads - 1) / kRowThreads;
    const uint32_t lo = min(a.n, tid * run), hi = min(a.n, lo + run);
    griddep_wait();
    uint32_t mine = 0;
    for (uint32_t i = lo; i < hi; ++i) {
        uint32_t counts = 0;
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
        mine += counts;
    }
    uint32_t before = mine;
    for (int o = 1; o < 32; o *= 2) {
        const uint32_t x = __shfl_up_sync(kFull, before, o);
        if (lane >= static_cast<uint32_t>(o)) before += x;
    }
    if (lane == 31) sums[warp] = before;
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
    uint32_t place = before - mine + (warp ? sums[warp - 1] : 0);
    for (uint32_t i = lo; i < hi; ++i)
        if (a.lists.counted[i]) a.rows.row[place++] = static_cast<int32_t>(i);
    if (tid == 0) {
        const uint32_t n = sums[31];
        *a.rows.count = n;
        *a.rows.factor = static_cast<float>(a.mean ? a.scale / (n ? n : 1u) : a.scale);
    }
}

// A warp a row, over the rows up to a tile's end.
__global__ void __launch_bounds__(256) pack_kernel(const __grid_constant__ PackArgs a) {
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t r = blockIdx.x * 8ull + threadIdx.x / 32;
    griddep_wait();
    const uint32_t n = a.rows.row ? *a.rows.count : a.n;
    if (r >= (static_cast<uint64_t>(n) + kLossTile - 1) / kLossTile * kLossTile) return;
    const bool there = r < n;
    const uint64_t from = there ? (a.rows.row ? static_cast<uint64_t>(a.rows.row[r]) : r) * a.stride : 0;
    for (uint64_t c = lane; c < a.out.pitch; c += 32) {
        float x = there && c < a.width ? load_value(a.src, from + c, a.bf16) : 0.f;
        for (int q = 0; q < a.out.planes; ++q) a.out.p[q * a.out.plane + r * a.out.pitch + c] = split_plane(x);
    }
}

__global__ void __launch_bounds__(256) clear_kernel(const __grid_constant__ ClearArgs a) {
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t i = blockIdx.x * 8ull + threadIdx.x / 32;
    griddep_wait();
    if (i >= a.n || a.counted[i]) return;
    if (a.losses && lane == 0) a.losses[i] = 0.f;
    if (a.grad_hidden)
        for (uint32_t c = lane; c < a.width; c += 32) {
            if (a.bf16) static_cast<uint16_t*>(a.grad_hidden)[i * a.stride + c] = 0;
            else static_cast<float*>(a.grad_hidden)[i * a.stride + c] = 0.f;
        }
}

// ------------------------------------------------------------------- joins

// (top, sum 2^(y - top)) of two parts of a row; a part of -infinities alone adds
// nothing, +infinity or NaN make the sum NaN.
__device__ __forceinline__ void join_stat(float& top, float& sum, float top2, float sum2) {
    const float m = fmaxf(top, top2);
    const float low = -__int_as_float(0x7F800000);
    const float a = top == low ? 0.f : __fmul_rn(sum, exp2_fast(__fsub_rn(top, m)));
    const float b = top2 == low ? 0.f : __fmul_rn(sum2, exp2_fast(__fsub_rn(top2, m)));
    top = m;
    sum = __fadd_rn(a, b);
}

// A warp a place: the tiles' statistics in a fixed order, the loss.
__global__ void __launch_bounds__(256) join_kernel(const __grid_constant__ JoinArgs a) {
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t r = blockIdx.x * 8ull + threadIdx.x / 32;
    griddep_wait();
    if (r >= *a.rows.count) return;
    const uint64_t i = a.rows.row[r];
    float top = -__int_as_float(0x7F800000), sum = 0.f;
    for (uint32_t q = lane; q < a.tiles; q += 32) {
        const float2 s = a.stats[q * a.pitch + r];
        join_stat(top, sum, s.x, s.y);
    }
    for (int o = 16; o > 0; o /= 2) {
        const float t2 = __shfl_down_sync(kFull, top, o), s2 = __shfl_down_sync(kFull, sum, o);
        join_stat(top, sum, t2, s2);
    }
    double dot = 0.0;  // sum p z
    const uint64_t at = i * a.lists.top;
    for (int k = lane; k < a.lists.top; k += 32) {
        if (a.lists.ids[at + k] == kNoId) continue;
        dot += (a.lists.shares ? static_cast<double>(a.lists.shares[at + k]) : 1.0) * a.lists.logits[at + k];
    }
    for (int o = 16; o > 0; o /= 2) dot += __shfl_down_sync(kFull, dot, o);
    if (lane != 0) return;
    const double lse = (static_cast<double>(top) + log2(static_cast<double>(sum))) * kLn2;
    const float loss = static_cast<float>(a.t * a.t * (static_cast<double>(a.lists.entropy[i]) - dot / a.t + lse));
    const float f = loss == loss ? static_cast<float>(*a.rows.factor * a.t) : loss;  // NaN: the whole row
    a.loss[r] = loss;
    a.gain[r] = f;
    a.stat[r] = {top, __fdiv_rn(f, sum)};
    if (a.losses) a.losses[i] = loss;
}

constexpr int kRecordThreads = 1024;

__global__ void __launch_bounds__(kRecordThreads) record_kernel(const __grid_constant__ RecordArgs a) {
    __shared__ double sums[32];
    __shared__ uint32_t bads[32];
    const uint32_t lane = threadIdx.x % 32, warp = threadIdx.x / 32;
    griddep_wait();
    const uint32_t n = *a.rows.count;
    double sum = 0.0;
    bool bad = false;
    for (uint32_t r = threadIdx.x; r < n; r += kRecordThreads) {
        const float x = a.loss[r];
        bad = bad || !(fabsf(x) < __int_as_float(0x7F800000));
        sum += x;
    }
    bad = __any_sync(kFull, bad);
    for (int o = 16; o > 0; o /= 2) sum += __shfl_down_sync(kFull, sum, o);
    if (lane == 0) {
        sums[warp] = sum;
        bads[warp] = bad;
    }
    __syncthreads();
    if (threadIdx.x != 0) return;
    uint32_t any = 0;
    sum = 0.0;
    for (int w = 0; w < 32; ++w) {
        sum += sums[w];
        any |= bads[w];
    }
    a.result[0] = static_cast<float>(sum * *a.rows.factor);
    a.result[1] = static_cast<float>(n);
    a.result[2] = any ? 1.f : 0.f;
    a.result[3] = *a.rows.factor;
}

__device__ __forceinline__ void store_out(void* out, uint64_t at, int bf16, int accumulate, float x) {
    if (accumulate) x = __fadd_rn(x, load_value(out, at, bf16));
    if (bf16) static_cast<uint16_t*>(out)[at] = bf16_of(x);
    else static_cast<float*>(out)[at] = x;
}

// The parts of a product, added in their order.
__global__ void __launch_bounds__(256) finish_parts_kernel(const __grid_constant__ FinishArgs a) {
    const uint32_t lane = threadIdx.x % 32;
    const uint64_t r = blockIdx.x * 8ull + threadIdx.x / 32;
    griddep_wait();
    if (r >= (a.by_count ? *a.rows.count : a.n)) return;
    const uint64_t to = (a.rows.row ? static_cast<uint64_t>(a.rows.row[r]) : r) * a.stride;
    for (uint32_t c = lane; c < a.width; c += 32) {
        float x = 0.f;
        for (int s = 0; s < a.splits; ++s) x = __fadd_rn(x, a.parts[s * a.part_stride + r * a.part_pitch + c]);
        store_out(a.out, to + c, a.bf16, a.accumulate, x);
    }
}

// ---------------------------------------------------------------- products

constexpr int kSide = 64, kDeep = 16;

__device__ __forceinline__ float operand_value(const Operand& o, uint64_t row, uint64_t k) {
    const uint64_t at = o.turned ? k * o.m.pitch + row : row * o.m.pitch + k;
    float x = 0.f;
    for (int q = o.m.planes - 1; q >= 0; --q) x = __fadd_rn(x, bf16_value(o.m.p[q * o.m.plane + at]));
    return x;
}

template <int EPI>
__global__ void __launch_bounds__(256) product_kernel(const __grid_constant__ ProductArgs a) {
    __shared__ float as[kDeep][kSide + 1], bs[kDeep][kSide + 1], cs[kSide][kSide + 1];
    const uint32_t tid = threadIdx.x, tx = tid % 16, ty = tid / 16;
    griddep_wait();
    const uint32_t count = *a.count;
    const uint32_t m = a.count_m ? min(a.m, count) : a.m, k_all = a.count_k ? min(a.k, count) : a.k;
    const uint32_t wide = (a.n + kLossTile - 1) / kLossTile;
    const uint64_t tall = (static_cast<uint64_t>(a.m) + kLossTile - 1) / kLossTile * (kLossTile / kSide);
    uint64_t b = blockIdx.x;
    const uint64_t m0 = b % tall * kSide;
    b /= tall;
    const uint32_t tile = static_cast<uint32_t>(b % wide), split = static_cast<uint32_t>(b / wide);
    const uint32_t per = (k_all + a.splits - 1) / a.splits;
    const uint32_t k_lo = min(k_all, split * per), k_hi = min(k_all, k_lo + per);
    if (m0 >= (static_cast<uint64_t>(m) + kLossTile - 1) / kLossTile * kLossTile) return;
    float top = -__int_as_float(0x7F800000), sum = 0.f;
    for (uint32_t n0 = tile * kLossTile; n0 < (tile + 1) * kLossTile && n0 < a.n; n0 += kSide) {
        float acc[4][4] = {};
        for (uint32_t k0 = k_lo; k0 < k_hi; k0 += kDeep) {
            for (int q = tid; q < kSide * kDeep; q += 256) {
                const uint32_t ra = a.a.turned ? q % kSide : q / kDeep, ka = a.a.turned ? q / kSide : q % kDeep;
                const uint32_t rb = a.b.turned ? q % kSide : q / kDeep, kb = a.b.turned ? q / kSide : q % kDeep;
                as[ka][ra] = m0 + ra < m && k0 + ka < k_hi ? operand_value(a.a, m0 + ra, k0 + ka) : 0.f;
                bs[kb][rb] = n0 + rb < a.n && k0 + kb < k_hi ? operand_value(a.b, n0 + rb, k0 + kb) : 0.f;
            }
            __syncthreads();
            for (int k = 0; k < kDeep; ++k)
                for (int i = 0; i < 4; ++i)
                    for (int j = 0; j < 4; ++j)
                        acc[i][j] = __fmaf_rn(as[k][ty * 4 + i], bs[k][tx * 4 + j], acc[i][j]);
            __syncthreads();
        }
        for (int i = 0; i < 4; ++i)
            for (int j = 0; j < 4; ++j) cs[ty * 4 + i][tx * 4 + j] = acc[i][j];
        __syncthreads();
        if (tid < kSide) {
            const uint64_t r = m0 + tid;
            const LogitArgs& g = a.logit;
            if (EPI != kLossOut) {
                const uint64_t at = r < m ? static_cast<uint64_t>(a.logit.lists.top) * a.out.row[r] : 0;
                const RowStat st = EPI == kLossGrad && r < m ? g.stat[r] : RowStat{0.f, 0.f};
                for (uint32_t j = 0; j < kSide; ++j) {
                    const uint32_t v = g.v0 + n0 + j;
                    const bool in = r < m && n0 + j < a.n;
                    const float z = cs[tid][j];
                    float share = 0.f;
                    if (in)
                        for (int k = 0; k < g.lists.top; ++k)
                            if (g.lists.ids[at + k] == static_cast<int32_t>(v)) {
                                share = g.lists.shares ? g.lists.shares[at + k] : 1.f;
                                if (EPI == kLossStats) g.lists.logits[at + k] = z;
                            }
                    if (EPI == kLossStats) {
                        if (in) join_stat(top, sum, __fmul_rn(z, g.c), 1.f);
                    } else {
                        float x = 0.f;
                        if (in)
                            x = __fsub_rn(__fmul_rn(exp2_fast(__fmaf_rn(z, g.c, -st.top)), st.inv),
                                          __fmul_rn(share, g.gain[r]));
                        for (int q = 0; q < g.g.planes; ++q)
                            g.g.p[q * g.g.plane + r * g.g.pitch + n0 + j] = split_plane(x);
                    }
                }
            } else if (r < m) {
                for (uint32_t j = 0; j < kSide && n0 + j < a.n; ++j) {
                    if (a.out.parts) {
                        float* p = a.out.parts + split * a.out.part_stride + r * a.out.part_pitch + n0 + j;
                        *p = a.out.add_parts ? __fadd_rn(*p, cs[tid][j]) : cs[tid][j];
                    } else {
                        const uint64_t to = (a.out.row ? static_cast<uint64_t>(a.out.row[r]) : r) * a.out.stride;
                        store_out(a.out.out, to + n0 + j, a.out.bf16, a.out.accumulate, cs[tid][j]);
                    }
                }
            }
        }
        __syncthreads();
    }
    if (EPI == kLossStats && tid < kSide && m0 + tid < m)
        a.logit.stats[(a.logit.v0 / kLossTile + tile) * a.logit.stats_pitch + m0 + tid] = make_float2(top, sum);
}

template <class Args>
cudaError_t launch(void (*f)(Args), const Args& a, uint64_t grid, int block, cudaStream_t st, size_t smem = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(grid));
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = AR_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<Args*>(&a)};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(f), args);
}

}  // namespace

cudaError_t launch_teacher(const TeacherArgs& a, cudaStream_t st) {
    return launch(teacher_kernel, a, (a.n + kTeacherWarps - 1) / kTeacherWarps, 32 * kTeacherWarps, st,
                  static_cast<size_t>(kTeacherWarps) * 2 * a.k * 4);
}

cudaError_t launch_rows(const RowsArgs& a, cudaStream_t st) { return launch(rows_kernel, a, 1, kRowThreads, st); }

cudaError_t launch_pack(const PackArgs& a, cudaStream_t st) {
    return launch(pack_kernel, a, (a.n + kLossTile - 1) / kLossTile * (kLossTile / 8), 256, st);
}

cudaError_t launch_clear(const ClearArgs& a, cudaStream_t st) { return launch(clear_kernel, a, (a.n + 7) / 8, 256, st); }

cudaError_t launch_join(const JoinArgs& a, cudaStream_t st) { return launch(join_kernel, a, (a.n + 7) / 8, 256, st); }

cudaError_t launch_record(const RecordArgs& a, cudaStream_t st) {
    return launch(record_kernel, a, 1, kRecordThreads, st);
}

cudaError_t launch_product(const ProductArgs& a, cudaStream_t st) {
    const uint64_t tall = (static_cast<uint64_t>(a.m) + kLossTile - 1) / kLossTile * (kLossTile / kSide);
    const uint64_t grid = tall * ((a.n + kLossTile - 1) / kLossTile) * a.splits;
    return launch(a.epilogue == kLossStats ? product_kernel<kLossStats>
                                           : (a.epilogue == kLossGrad ? product_kernel<kLossGrad> : product_kernel<kLossOut>),
                  a, grid, 256, st);
}

cudaError_t launch_finish_parts(const FinishArgs& a, cudaStream_t st) {
    return launch(finish_parts_kernel, a, (a.n + 7) / 8, 256, st);
}

}  // namespace ar
