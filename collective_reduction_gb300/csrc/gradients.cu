// Kernels over many tensors after a gradient allreduce: the global norm, the
// scaling by the clip factor, and the AdamW update.  All are bound by HBM at
// size and by launches and one dependent chain when small.
//
// A handle's tables split every tensor into ranges ("items") of equal element
// count; a warp works through one item at a time, so items of tiny tensors
// run beside each other and no barrier stands between items.
#include "device.cuh"
#include "gradients.hpp"

namespace ar {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint4 load128(const char* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ uint2 load64(const char* p) {
    uint2 v;
    asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

__device__ __forceinline__ void store128(char* p, uint4 v) {
    asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                 : "memory");
}

__device__ __forceinline__ void store64(char* p, uint2 v) {
    asm volatile("st.global.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
}

// One element as the bits of a float32.
template <bool BF>
__device__ __forceinline__ uint32_t load_elem(const char* p, uint32_t i) {
    if (BF) {
        uint16_t h;
        asm volatile("ld.global.u16 %0, [%1];" : "=h"(h) : "l"(p + 2ull * i));
        return static_cast<uint32_t>(h) << 16;
    }
    uint32_t w;
    asm volatile("ld.global.u32 %0, [%1];" : "=r"(w) : "l"(p + 4ull * i));
    return w;
}

// bf16 stores round to nearest even, as every bf16 result of the engine does.
template <bool BF>
__device__ __forceinline__ void store_elem(char* p, uint32_t i, float x) {
    if (BF) {
        const uint16_t h = static_cast<uint16_t>(pack_bf16x2(x, 0.f));
        asm volatile("st.global.u16 [%0], %1;" ::"l"(p + 2ull * i), "h"(h) : "memory");
    } else {
        asm volatile("st.global.f32 [%0], %1;" ::"l"(p + 4ull * i), "f"(x) : "memory");
    }
}

// Four elements starting at element i (16 bytes of float32 or 8 of bfloat16).
template <bool BF>
__device__ __forceinline__ float4 load_quad(const char* p, uint32_t i) {
    if (BF) {
        const uint2 w = load64(p + 2ull * i);
        return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
    }
    const uint4 w = load128(p + 4ull * i);
    return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
}

template <bool BF>
__device__ __forceinline__ void store_quad(char* p, uint32_t i, float4 x) {
    if (BF)
        store64(p + 2ull * i, make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w)));
    else
        store128(p + 4ull * i, make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z),
                                          __float_as_uint(x.w)));
}

// Elements before the first whole vector of `bytes` bytes (a power of two).
template <bool BF>
__device__ __forceinline__ uint32_t head_elems(const void* p, uint32_t bytes) {
    const uint32_t off = static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) & (bytes - 1);
    return ((bytes - off) & (bytes - 1)) / (BF ? 2 : 4);
}

// ------------------------------------------------------------------- the norm

// Largest magnitude of a group, as a float32's bits: they order as the
// magnitudes do, an infinity above every finite value, NaN above infinity.
template <bool BF, int U>
__device__ __forceinline__ uint32_t magnitude(const uint4 (&x)[U]) {
    uint32_t m = 0;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            if (BF) m = max(m, (w[k] << 16) & 0x7FFFFFFFu);
            m = max(m, w[k] & (BF ? 0x7FFF0000u : 0x7FFFFFFFu));
        }
    }
    return m;
}

// Sum of squares.  A thread squares and adds up to 32 float32 (64 bfloat16)
// values in float32, then adds that group sum to its float64 accumulator:
// GB300's float64 rate is far too low for an operation per element, and one
// per group costs nothing beside the loads, while long float32 sums would
// lose digits with their length.
//
// Range: squares leave float32's range where the values themselves do not
// (|x| above 1.8e19 or below 1e-19).  A group whose float32 sum is finite and
// at least 2^-100 lost nothing that counts (a square that fell below the
// smallest normal is off by 2^-150 at most).  Any other group is summed again
// from the registers, scaled by the power of two that brings its largest
// value to [1, 2); the float64 accumulator takes the exact scale back out.
// All-zero groups end at the look at the largest value.
struct SumSquares {
    double s = 0.0;

    template <bool BF, int U>
    __device__ __forceinline__ static float group(const uint4 (&x)[U], float f) {
        float a = 0.f, b = 0.f, c = 0.f, d = 0.f;
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
            if (BF) {
                float t;
                t = __fmul_rn(bf_lo(w[0]), f), a = __fmaf_rn(t, t, a);
                t = __fmul_rn(bf_hi(w[0]), f), b = __fmaf_rn(t, t, b);
                t = __fmul_rn(bf_lo(w[1]), f), c = __fmaf_rn(t, t, c);
                t = __fmul_rn(bf_hi(w[1]), f), d = __fmaf_rn(t, t, d);
                t = __fmul_rn(bf_lo(w[2]), f), a = __fmaf_rn(t, t, a);
                t = __fmul_rn(bf_hi(w[2]), f), b = __fmaf_rn(t, t, b);
                t = __fmul_rn(bf_lo(w[3]), f), c = __fmaf_rn(t, t, c);
                t = __fmul_rn(bf_hi(w[3]), f), d = __fmaf_rn(t, t, d);
            } else {
                float t;
                t = __fmul_rn(__uint_as_float(w[0]), f), a = __fmaf_rn(t, t, a);
                t = __fmul_rn(__uint_as_float(w[1]), f), b = __fmaf_rn(t, t, b);
                t = __fmul_rn(__uint_as_float(w[2]), f), c = __fmaf_rn(t, t, c);
                t = __fmul_rn(__uint_as_float(w[3]), f), d = __fmaf_rn(t, t, d);
            }
        }
        return __fadd_rn(__fadd_rn(a, b), __fadd_rn(c, d));
    }

    // false when the group has to be summed again by again()
    template <bool BF, int U>
    __device__ __forceinline__ bool feed(const uint4 (&x)[U]) {
        const float q = group<BF, U>(x, 1.f);
        if (q >= 0x1p-100f && q <= 0x1.fffffep127f) {
            s += static_cast<double>(q);
            return true;
        }
        return q == 0.f && magnitude<BF, U>(x) == 0;
    }

    // The group of vectors q, q + 32, ... below nv, with the scale.
    template <bool BF, int U>
    __device__ __noinline__ static double again(const char* body, uint32_t q, uint32_t nv) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = q + 32 * u < nv ? load128(body + 16ull * (q + 32 * u)) : make_uint4(0, 0, 0, 0);
        const uint32_t top = magnitude<BF, U>(x);
        if (top >= 0x7F800000u) return static_cast<double>(group<BF, U>(x, 1.f));  // an infinity or NaN, as the norm
        const uint32_t e = min(max(top >> 23, 1u), 253u);  // 2^(127 - e) is a normal float32
        const float r = group<BF, U>(x, __uint_as_float((254u - e) << 23));
        const uint64_t back = static_cast<uint64_t>(1023 + 2 * (static_cast<int>(e) - 127)) << 52;
        return static_cast<double>(r) * __longlong_as_double(static_cast<long long>(back));
    }

    __device__ __forceinline__ void one(uint32_t bits) {  // one value, as a float32's bits
        const double d = static_cast<double>(__uint_as_float(bits));
        s = fma(d, d, s);
    }

    __device__ __forceinline__ void add(double d) { s += d; }
    __device__ __forceinline__ void join(uint64_t other) { s += __longlong_as_double(static_cast<long long>(other)); }
    __device__ __forceinline__ uint64_t bits() const {
        return static_cast<uint64_t>(__double_as_longlong(s));
    }
    __device__ __forceinline__ double norm() const { return sqrt(s); }
    __device__ __forceinline__ bool nonfinite() const { return !(s <= 1.7976931348623157e308); }
};

// Largest magnitude; NaN is above everything and so never lost.
struct MaxAbs {
    uint32_t m = 0;

    template <bool BF, int U>
    __device__ __forceinline__ bool feed(const uint4 (&x)[U]) {
        m = max(m, magnitude<BF, U>(x));
        return true;
    }

    template <bool BF, int U>
    __device__ __forceinline__ static uint32_t again(const char*, uint32_t, uint32_t) {
        return 0;
    }

    __device__ __forceinline__ void one(uint32_t bits) { m = max(m, bits & 0x7FFFFFFFu); }
    __device__ __forceinline__ void add(uint32_t d) { m = max(m, d); }
    __device__ __forceinline__ void join(uint64_t other) { m = max(m, static_cast<uint32_t>(other)); }
    __device__ __forceinline__ uint64_t bits() const { return m; }
    __device__ __forceinline__ double norm() const { return static_cast<double>(__uint_as_float(m)); }
    __device__ __forceinline__ bool nonfinite() const { return m >= 0x7F800000u; }
};

template <class Acc>
__device__ __forceinline__ void warp_join(Acc& a) {
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) a.join(__shfl_down_sync(kFull, a.bits(), d));
}

// Joins the accumulators of a CTA of WARPS warps; the result is thread 0's.
template <class Acc, int WARPS>
__device__ __forceinline__ void cta_join(Acc& a, uint64_t* sm) {
    warp_join(a);
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (lane == 0) sm[warp] = a.bits();
    __syncthreads();
    if (warp == 0) {
        Acc b;
        if (lane < WARPS) b.join(sm[lane]);
        warp_join(b);
        a = b;
    }
}

// Lane's share of one item: whole 16-byte vectors, 8 in flight a thread, and
// single elements before the first and after the last.
template <class Acc, bool BF>
__device__ __forceinline__ void norm_item(Acc& acc, const char* src, uint32_t count, uint32_t lane) {
    constexpr uint32_t V = BF ? 8 : 4;
    constexpr int U = 8;
    const uint32_t head = min(count, head_elems<BF>(src, 16));
    const uint32_t nv = (count - head) / V;
    const uint32_t tail = count - head - nv * V;
    const char* body = src + head * (BF ? 2 : 4);
    uint32_t q = lane;
    for (; q + 32 * (U - 1) < nv; q += 32 * U) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = load128(body + 16ull * (q + 32 * u));
        if (!acc.template feed<BF, U>(x)) acc.add(Acc::template again<BF, U>(body, q, nv));
    }
    if (q < nv) {
        uint4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = q + 32 * u < nv ? load128(body + 16ull * (q + 32 * u)) : make_uint4(0, 0, 0, 0);
        if (!acc.template feed<BF, U>(x)) acc.add(Acc::template again<BF, U>(body, q, nv));
    }
    if (lane < head) acc.one(load_elem<BF>(src, lane));
    if (lane < tail) acc.one(load_elem<BF>(src, count - tail + lane));
}

// Every warp sums its items, every CTA its warps, and the CTA that finishes
// last adds the CTAs' sums in their order: which warp takes which item is
// fixed by the grid, so repeated calls give the same bits.
template <class Acc>
__global__ void __launch_bounds__(kGradThreads, kNormCtasPerSm) norm_kernel(const __grid_constant__ NormArgs a) {
    __shared__ uint64_t sm[kGradWarps];
    __shared__ bool last;
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t stride = gridDim.x * kGradWarps;
    griddep_wait();
    griddep_launch_dependents();
    Acc acc;
    for (uint32_t it = blockIdx.x * kGradWarps + (threadIdx.x >> 5); it < a.n_items; it += stride) {
        const GradItem w = a.items[it];
        Acc part;
        if (w.flags & kGradBf16)
            norm_item<Acc, true>(part, w.src, w.count, lane);
        else
            norm_item<Acc, false>(part, w.src, w.count, lane);
        acc.join(part.bits());
        if (a.item_partials) {
            warp_join(part);
            if (lane == 0) a.item_partials[it] = part.bits();
        }
    }
    cta_join<Acc, kGradWarps>(acc, sm);
    if (threadIdx.x == 0) {
        a.cta_partials[blockIdx.x] = acc.bits();
        __threadfence();
        last = atomicInc(a.counter, gridDim.x - 1) == gridDim.x - 1;  // wraps to 0 for the next call
    }
    __syncthreads();
    if (!last) return;
    __threadfence();
    Acc all;
    for (uint32_t i = threadIdx.x; i < gridDim.x; i += kGradThreads) all.join(__ldcg(a.cta_partials + i));
    cta_join<Acc, kGradWarps>(all, sm);
    if (threadIdx.x == 0) {
        const double c = a.pre_scale, norm = c * all.norm();
        const bool bad = all.nonfinite();
        const bool clipped = !bad && norm > a.max_norm;
        a.result[0] = static_cast<float>(norm);
        a.result[1] = static_cast<float>(clipped ? c * (a.max_norm / norm) : c);
        a.result[2] = bad ? 1.f : 0.f;
        a.result[3] = clipped ? 1.f : 0.f;
    }
}

// Norms of single tensors: a CTA adds one tensor's item sums.
template <class Acc>
__global__ void __launch_bounds__(kTensorNormThreads) tensor_norm_kernel(const __grid_constant__ TensorNormArgs a) {
    __shared__ uint64_t sm[kTensorNormThreads / 32];
    griddep_wait();
    griddep_launch_dependents();
    const uint32_t lo = a.first[blockIdx.x], hi = a.first[blockIdx.x + 1];
    Acc acc;
#pragma unroll 8
    for (uint32_t i = lo + threadIdx.x; i < hi; i += kTensorNormThreads) acc.join(a.item_partials[i]);
    cta_join<Acc, kTensorNormThreads / 32>(acc, sm);
    if (threadIdx.x == 0) a.norms[blockIdx.x] = static_cast<float>(a.pre_scale * acc.norm());
}

// ---------------------------------------------------------------- the scaling

// dst = round(f * src) over one item: quads where both sides are whole
// vectors after the same head, else element by element.
template <bool SB, bool DB>
__device__ __forceinline__ void scale_item(const char* src, char* dst, uint32_t count, float f, uint32_t lane) {
    constexpr int U = 8;
    const uint32_t head = min(count, head_elems<DB>(dst, DB ? 8 : 16));
    const uintptr_t s0 = reinterpret_cast<uintptr_t>(src) + head * (SB ? 2 : 4);
    if (s0 % (SB ? 8 : 16) == 0) {
        const uint32_t nq = (count - head) / 4;
        const uint32_t done = head + nq * 4;
        for (uint32_t q = lane; q < nq; q += 32 * U) {
            float4 x[U];
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (q + 32 * u < nq) x[u] = load_quad<SB>(src, head + 4 * (q + 32 * u));
#pragma unroll
            for (int u = 0; u < U; ++u)
                if (q + 32 * u < nq)
                    store_quad<DB>(dst, head + 4 * (q + 32 * u),
                                   make_float4(__fmul_rn(x[u].x, f), __fmul_rn(x[u].y, f), __fmul_rn(x[u].z, f),
                                               __fmul_rn(x[u].w, f)));
        }
        if (lane < head) store_elem<DB>(dst, lane, __fmul_rn(__uint_as_float(load_elem<SB>(src, lane)), f));
        if (done + lane < count)
            store_elem<DB>(dst, done + lane, __fmul_rn(__uint_as_float(load_elem<SB>(src, done + lane)), f));
        return;
    }
    for (uint32_t q = lane; q < count; q += 32 * U) {
        uint32_t x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + 32 * u < count) x[u] = load_elem<SB>(src, q + 32 * u);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + 32 * u < count) store_elem<DB>(dst, q + 32 * u, __fmul_rn(__uint_as_float(x[u]), f));
    }
}

// The items in the reverse of the norm's order: what the norm read last may
// still be in L2.  In place, a factor of exactly 1 leaves nothing to do.
__global__ void __launch_bounds__(kGradThreads) scale_kernel(const __grid_constant__ ScaleArgs a) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    griddep_wait();
    griddep_launch_dependents();
    if (w >= a.n_items) return;
    const GradItem it = a.items[a.n_items - 1 - w];
    const float f = __ldcg(a.result + 1);
    if ((it.flags & kInPlace) && f == 1.f) return;
    const bool sb = it.flags & kGradBf16, db = it.flags & kOutBf16;
    if (sb && db)
        scale_item<true, true>(it.src, it.dst, it.count, f, lane);
    else if (sb)
        scale_item<true, false>(it.src, it.dst, it.count, f, lane);
    else if (db)
        scale_item<false, true>(it.src, it.dst, it.count, f, lane);
    else
        scale_item<false, false>(it.src, it.dst, it.count, f, lane);
}

// ---------------------------------------------------------------------- AdamW

// One element: moments and parameter, in float32.  The decay is subtracted
// with the update (p - (lr wd p + update)), so its small factor is never
// rounded against 1.
__device__ __forceinline__ void adam_one(const AdamArgs& a, float decay, float f, float& p, float g, float& m,
                                         float& v) {
    g = __fmul_rn(g, f);
    m = __fmaf_rn(a.omb1, g, __fmul_rn(a.beta1, m));
    v = __fmaf_rn(__fmul_rn(a.omb2, g), g, __fmul_rn(a.beta2, v));
    const float den = __fmaf_rn(__fsqrt_rn(v), a.inv_bc2, a.eps);
    const float upd = __fmul_rn(a.step_size, __fdiv_rn(m, den));
    p = __fsub_rn(p, __fmaf_rn(decay, p, upd));
}

__device__ __forceinline__ void adam_quad(const AdamArgs& a, float decay, float f, float4& p, float4 g, float4& m,
                                          float4& v) {
    adam_one(a, decay, f, p.x, g.x, m.x, v.x);
    adam_one(a, decay, f, p.y, g.y, m.y, v.y);
    adam_one(a, decay, f, p.z, g.z, m.z, v.z);
    adam_one(a, decay, f, p.w, g.w, m.w, v.w);
}

template <bool PB, bool GB, bool COPY>
__device__ __forceinline__ void adam_elem(const AdamArgs& a, const AdamItem& it, float decay, float f, uint32_t i) {
    char* mp = reinterpret_cast<char*>(it.m);
    char* vp = reinterpret_cast<char*>(it.v);
    float p = __uint_as_float(load_elem<PB>(it.p, i)), m = __uint_as_float(load_elem<false>(mp, i));
    const float g = __uint_as_float(load_elem<GB>(it.g, i));
    float v = __uint_as_float(load_elem<false>(vp, i));
    adam_one(a, decay, f, p, g, m, v);
    store_elem<PB>(it.p, i, p);
    store_elem<false>(mp, i, m);
    store_elem<false>(vp, i, v);
    if (COPY) store_elem<true>(it.w, i, p);
}

template <bool PB, bool GB, bool COPY>
__device__ __forceinline__ void adam_item(const AdamArgs& a, const AdamItem& it, float f, uint32_t lane) {
    constexpr int U = 2;
    const float decay = __fmul_rn(a.lr_decay, it.decay);
    char* mp = reinterpret_cast<char*>(it.m);
    char* vp = reinterpret_cast<char*>(it.v);
    const uint32_t head = min(it.count, head_elems<false>(mp, 16));
    auto whole = [&](const void* p, bool bf) {
        return (reinterpret_cast<uintptr_t>(p) + head * (bf ? 2 : 4)) % (bf ? 8 : 16) == 0;
    };
    if (whole(it.p, PB) && whole(it.g, GB) && whole(vp, false) && (!COPY || whole(it.w, true))) {
        const uint32_t nq = (it.count - head) / 4;
        const uint32_t done = head + nq * 4;
        for (uint32_t q = lane; q < nq; q += 32 * U) {
            float4 p[U], g[U], m[U], v[U];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t i = head + 4 * (q + 32 * u);
                if (q + 32 * u < nq) {
                    g[u] = load_quad<GB>(it.g, i);
                    m[u] = load_quad<false>(mp, i);
                    v[u] = load_quad<false>(vp, i);
                    p[u] = load_quad<PB>(it.p, i);
                }
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const uint32_t i = head + 4 * (q + 32 * u);
                if (q + 32 * u < nq) {
                    adam_quad(a, decay, f, p[u], g[u], m[u], v[u]);
                    store_quad<PB>(it.p, i, p[u]);
                    store_quad<false>(mp, i, m[u]);
                    store_quad<false>(vp, i, v[u]);
                    if (COPY) store_quad<true>(it.w, i, p[u]);
                }
            }
        }
        if (lane < head) adam_elem<PB, GB, COPY>(a, it, decay, f, lane);
        if (done + lane < it.count) adam_elem<PB, GB, COPY>(a, it, decay, f, done + lane);
        return;
    }
    for (uint32_t i = lane; i < it.count; i += 32) adam_elem<PB, GB, COPY>(a, it, decay, f, i);
}

// A warp updates one item.  With a record, nothing is touched when the
// gradients held an infinity or NaN.
__global__ void __launch_bounds__(kGradThreads) adamw_kernel(const __grid_constant__ AdamArgs a) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    griddep_wait();
    griddep_launch_dependents();
    if (w >= a.n_items) return;
    const AdamItem it = a.items[a.n_items - 1 - w];
    float f = 1.f;
    if (a.result) {
        f = __ldcg(a.result + 1);
        if (__ldcg(a.result + 2) != 0.f) return;
    }
    switch (it.flags & (kGradBf16 | kParamBf16 | kHasCopy)) {
        case 0: return adam_item<false, false, false>(a, it, f, lane);
        case kGradBf16: return adam_item<false, true, false>(a, it, f, lane);
        case kHasCopy: return adam_item<false, false, true>(a, it, f, lane);
        case kHasCopy | kGradBf16: return adam_item<false, true, true>(a, it, f, lane);
        case kParamBf16: return adam_item<true, false, false>(a, it, f, lane);
        default: return adam_item<true, true, false>(a, it, f, lane);
    }
}

template <class Args>
cudaError_t launch(void (*f)(Args), const Args& a, uint32_t grid, int block, cudaStream_t st) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = AR_PDL;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    void* args[] = {const_cast<Args*>(&a)};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(f), args);
}

uint32_t ctas(uint32_t n_items) { return (n_items + kGradWarps - 1) / kGradWarps; }

}  // namespace

int norm_grid(uint32_t n_items, int num_sms) {
    const uint32_t most = static_cast<uint32_t>(num_sms) * kNormCtasPerSm, want = ctas(n_items);
    return static_cast<int>(want < 1 ? 1 : want < most ? want : most);
}

cudaError_t launch_norm(const NormArgs& a, int grid, cudaStream_t st) {
    return launch(a.kind == AR_NORM_MAX ? norm_kernel<MaxAbs> : norm_kernel<SumSquares>, a,
                  static_cast<uint32_t>(grid), kGradThreads, st);
}

cudaError_t launch_tensor_norms(const TensorNormArgs& a, int n_tensors, cudaStream_t st) {
    return launch(a.kind == AR_NORM_MAX ? tensor_norm_kernel<MaxAbs> : tensor_norm_kernel<SumSquares>, a,
                  static_cast<uint32_t>(n_tensors), kTensorNormThreads, st);
}

cudaError_t launch_scale(const ScaleArgs& a, cudaStream_t st) {
    return launch(scale_kernel, a, ctas(a.n_items), kGradThreads, st);
}

cudaError_t launch_adamw(const AdamArgs& a, cudaStream_t st) {
    return launch(adamw_kernel, a, ctas(a.n_items), kGradThreads, st);
}

}  // namespace ar
