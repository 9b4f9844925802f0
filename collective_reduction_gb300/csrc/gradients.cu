// Kernels over many tensors after a gradient allreduce: the global norm, the
// scaling by the clip factor, and the AdamW update.  All are bound by HBM at
// size and by launches and one dependent chain when small.  Measured on GB300 in
// a CUDA graph, sets rotating beyond L2; TB/s of the bytes each has to move (a
// copy: 6.77):
//
//   norm    4.3 GB of bf16 581 us (7.4), 25 MB of float32 9.8 us, 35 KB 3.75 us
//   clip    2.7 GB of float32 into other tensors 1144 us (7.0 of its two reads
//           and one write), in place 1154 us, 96 MB 44.8 us, 0.4 MB 5.25 us
//   AdamW   184M float32 parameters, bf16 gradients and copies 737 us (7.0),
//           0.4M float32 parameters 3.85 us
//
// (Called from Python in a loop, where launches overlap, 25 MB takes 8.3 us.)
//
// A handle's tables split every tensor into ranges ("items"); a warp works
// through one item at a time, so items of tiny tensors run beside each other
// and no barrier stands between items.  An item's vectors start on whole
// lines of the leading stream; the elements before and after them, at a
// tensor's ends, go singly.
#include "device.cuh"
#include "gradients.hpp"

namespace ar {
namespace {

constexpr uint32_t kFull = 0xFFFFFFFFu;

// How soon the lines that a load brings in may leave L2: the last ones read in
// their usual turn, the others first.  Not evict_last: such lines stay after
// their reader has gone (reading them again with evict_first or streaming loads
// does not release them) and take their part of L2 from every kernel that
// follows.  Measured: four passes over an 80 MB tensor after a clip of 24 MB
// 60 us, 70 with evict_last (which itself took 0.5 to 5% off norm and AdamW).
__device__ __forceinline__ uint64_t keep_policy(bool last_out) {
    uint64_t p;
    if (last_out)
        asm volatile("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(p));
    else
        asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
    return p;
}

__device__ __forceinline__ uint4 load128(const char* p) {
    uint4 v;
    asm volatile("ld.global.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
    return v;
}

__device__ __forceinline__ uint4 load128(const char* p, uint64_t policy) {
    uint4 v;
    asm volatile("ld.global.L2::cache_hint.v4.u32 {%0, %1, %2, %3}, [%4], %5;"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p), "l"(policy));
    return v;
}

// CS: the line is not used again (streaming)
template <bool CS>
__device__ __forceinline__ uint4 load_vec4(const char* p) {
    if (!CS) return load128(p);
    uint4 v;
    asm volatile("ld.global.cs.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

template <bool CS>
__device__ __forceinline__ uint2 load_vec2(const char* p) {
    uint2 v;
    if (CS)
        asm volatile("ld.global.cs.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    else
        asm volatile("ld.global.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "l"(p));
    return v;
}

template <bool CS>
__device__ __forceinline__ void store_vec4(char* p, uint4 v) {
    if (CS)
        asm volatile("st.global.cs.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
    else
        asm volatile("st.global.v4.u32 [%0], {%1, %2, %3, %4};" ::"l"(p), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                     : "memory");
}

template <bool CS>
__device__ __forceinline__ void store_vec2(char* p, uint2 v) {
    if (CS)
        asm volatile("st.global.cs.v2.u32 [%0], {%1, %2};" ::"l"(p), "r"(v.x), "r"(v.y) : "memory");
    else
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

// Four elements starting at element i: one access of 16 bytes of float32 or 8
// of bfloat16 where `whole` says that they are aligned to it, else four.
template <bool BF, bool CS = false>
__device__ __forceinline__ float4 load_quad(const char* p, uint32_t i, bool whole) {
    if (!whole)
        return make_float4(__uint_as_float(load_elem<BF>(p, i)), __uint_as_float(load_elem<BF>(p, i + 1)),
                           __uint_as_float(load_elem<BF>(p, i + 2)), __uint_as_float(load_elem<BF>(p, i + 3)));
    if (BF) {
        const uint2 w = load_vec2<CS>(p + 2ull * i);
        return make_float4(bf_lo(w.x), bf_hi(w.x), bf_lo(w.y), bf_hi(w.y));
    }
    const uint4 w = load_vec4<CS>(p + 4ull * i);
    return make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
}

template <bool BF, bool CS = false>
__device__ __forceinline__ void store_quad(char* p, uint32_t i, float4 x, bool whole) {
    if (!whole) {
        store_elem<BF>(p, i, x.x), store_elem<BF>(p, i + 1, x.y);
        store_elem<BF>(p, i + 2, x.z), store_elem<BF>(p, i + 3, x.w);
    } else if (BF)
        store_vec2<CS>(p + 2ull * i, make_uint2(pack_bf16x2(x.x, x.y), pack_bf16x2(x.z, x.w)));
    else
        store_vec4<CS>(p + 4ull * i, make_uint4(__float_as_uint(x.x), __float_as_uint(x.y), __float_as_uint(x.z),
                                          __float_as_uint(x.w)));
}

// Whether quads from element i on lie on their alignment.
template <bool BF>
__device__ __forceinline__ bool quad_aligned(const void* p, uint32_t i) {
    return ((static_cast<uint32_t>(reinterpret_cast<uintptr_t>(p)) + i * (BF ? 2 : 4)) & (BF ? 7 : 15)) == 0;
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
// smallest normal is off by 2^-150 at most), and a group of zeros adds none.
// Any other group is loaded and summed again, scaled by the power of two that
// brings its largest value to [1, 2), and the exact scale goes back in in
// float64.  (That path is a function of its own: inlined, it cost the loads
// their registers.)
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
    // The root r and 1 / r.  float64 roots and divisions are long dependent
    // chains here (0.3 us each of a call that takes 4): float32's reciprocal
    // root of s 4^-k in [1, 4) and one Newton step in float64 give 2^-42.
    __device__ __forceinline__ void root(double& r, double& inverse) const {
        if (s == 0.0 || nonfinite()) {
            r = inverse = s;  // the inverse is not used
            return;
        }
        const uint64_t b = bits();
        const int k = (static_cast<int>(b >> 52) - 1023) >> 1;  // s is at least 2^-298: a normal number
        const double t = __longlong_as_double(static_cast<long long>(b - (static_cast<uint64_t>(2 * k) << 52)));
        const double y = rsqrtf(static_cast<float>(t));
        const double z = fma(y, fma(-0.5 * t * y, y, 0.5), y);
        const auto power = [](int e) { return __longlong_as_double(static_cast<long long>(1023 + e) << 52); };
        r = t * z * power(k);
        inverse = z * power(-k);
    }
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
    __device__ __forceinline__ void root(double& r, double& inverse) const {
        r = static_cast<double>(__uint_as_float(m));
        inverse = 1.0 / r;
    }
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

// The record of a norm (and what every element is scaled by).
struct Record {
    float norm, scale, nonfinite, clipped;
};

template <class Acc>
__device__ __forceinline__ Record make_record(const Acc& acc, double c, double max_norm) {
    double r, inverse;
    acc.root(r, inverse);
    const bool bad = acc.nonfinite(), clipped = !bad && c * r > max_norm;
    return {static_cast<float>(c * r), static_cast<float>(clipped ? max_norm * inverse : c), bad ? 1.f : 0.f,
            clipped ? 1.f : 0.f};
}

__device__ __forceinline__ void store_record(float* to, const Record& r) {
    to[0] = r.norm;
    to[1] = r.scale;
    to[2] = r.nonfinite;
    to[3] = r.clipped;
}

// An item's 16-byte vectors and the elements before and after them.
template <bool BF>
struct Vectors {
    static constexpr uint32_t V = BF ? 8 : 4;
    uint32_t head, n, tail;
    const char* body;

    __device__ __forceinline__ Vectors(const char* src, uint32_t count) {
        head = min(count, head_elems<BF>(src, 16));
        n = (count - head) / V;
        tail = count - head - n * V;
        body = src + head * (BF ? 2 : 4);
    }
};

// Lane's share of one item, 8 vectors in flight a thread: at the kernel's 3
// CTAs an SM that keeps 98 KB in flight on each.
template <class Acc, bool BF, bool HINT>
__device__ __forceinline__ void norm_item(Acc& acc, const char* src, uint32_t count, uint32_t lane, uint64_t policy) {
    constexpr int U = 8;
    const Vectors<BF> v(src, count);
    auto load = [&](uint32_t q) { return HINT ? load128(v.body + 16ull * q, policy) : load128(v.body + 16ull * q); };
    for (uint32_t q0 = 0; q0 < v.n; q0 += 32 * U) {
        const uint32_t q = q0 + lane;
        uint4 x[U];
        if (q0 + 32 * U <= v.n) {
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = load(q + 32 * u);
        } else {
#pragma unroll
            for (int u = 0; u < U; ++u) x[u] = q + 32 * u < v.n ? load(q + 32 * u) : make_uint4(0, 0, 0, 0);
        }
        if (!acc.template feed<BF, U>(x)) acc.add(Acc::template again<BF, U>(v.body, q, v.n));
    }
    if (lane < v.head) acc.one(load_elem<BF>(src, lane));
    if (lane < v.tail) acc.one(load_elem<BF>(src, count - v.tail + lane));
}

// Any number of items, on one resident wave of CTAs.  A warp takes an item at a
// time and leaves its sum in the item's place; finish_kernel adds them up in
// their order, so repeated calls give the same bits whichever warp took which.
// More items than warps are dealt to kNormLists lists, and a CTA's warps draw
// from one of them, after a first two items each that are fixed: the SMs do
// not all read at one rate (with equal shares some idled for the last tenth).
// One list would do but for its counter: an item every 3 ns is what one
// address gives out (4.3 GB in ranges of 8192 elements: 897 us with one list,
// 580 with eight).  Fewer items than warps are one list, an item to each of the
// first warps (25 MB in a graph: 9.8 us, 11.6 dealt to eight).  Item and draw are fetched
// one item ahead.
// KEEP: a reader of the gradients follows, in the reverse order.
template <class Acc, bool KEEP>
__global__ void __launch_bounds__(kGradThreads, kNormCtasPerSm) norm_kernel(const __grid_constant__ NormArgs a) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t lists = a.n_items > gridDim.x * kGradWarps ? kNormLists : 1, list = blockIdx.x % lists;
    const uint32_t warps = (gridDim.x - list + lists - 1) / lists * kGradWarps;  // that draw from this list
    uint32_t it = list + lists * (blockIdx.x / lists * kGradWarps + (threadIdx.x >> 5)), next = it + lists * warps;
    GradItem w = {};  // the items are the handle's own and constant: read while the kernel before still runs
    if (it < a.n_items) w = a.items[it];
    griddep_wait();
    griddep_launch_dependents();
    while (it < a.n_items) {
        GradItem ahead = {};
        uint32_t drawn = 0;
        if (next < a.n_items) {
            ahead = a.items[next];
            if (lane == 0) drawn = atomicAdd(a.drawn + 32 * list, 1u);
        }
        Acc acc;
        const uint64_t policy = KEEP ? keep_policy(it >= a.keep_from) : 0;
        if (w.flags & kGradBf16)
            norm_item<Acc, true, KEEP>(acc, w.src, w.count, lane, policy);
        else
            norm_item<Acc, false, KEEP>(acc, w.src, w.count, lane, policy);
        warp_join(acc);
        if (lane == 0) a.partials[it] = acc.bits();
        it = next;
        w = ahead;
        next = list + lists * (2 * warps + __shfl_sync(kFull, drawn, 0));
    }
}

// A CTA's shared memory may be written by others of its cluster only once it has
// started, which nothing but a cluster barrier says: every thread arrives at its
// kernel's start (relaxed: nothing is handed over yet), and cluster_join waits
// for the others before its first store to them, with the loads in between.
__device__ __forceinline__ void cluster_started() {
    asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
}

// The sums of a cluster's CTAs, in their order, through their shared memory:
// thread 0 of every CTA gets the total.  mine: the CTA's sum, in its thread 0.
// Every thread of the cluster has called cluster_started before.
template <class Acc>
__device__ __forceinline__ Acc cluster_join(const Acc& mine, uint64_t* sums, uint32_t ctas, uint32_t rank) {
    __syncwarp();
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    if (threadIdx.x < 32) {
        const uint64_t bits = __shfl_sync(kFull, mine.bits(), 0);
        if (threadIdx.x < ctas) {  // to CTA number `lane`'s shared memory
            uint32_t to;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                         : "=r"(to)
                         : "r"(smem_addr(sums + rank)), "r"(threadIdx.x));
            asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(to), "l"(bits) : "memory");
        }
    }
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    Acc all;
    if (threadIdx.x == 0)
        for (uint32_t c = 0; c < ctas; ++c) all.join(sums[c]);
    return all;
}

// The items' sums to the record (the first record_ctas CTAs, one cluster) and to
// the norms of single tensors (a CTA each, after them).
template <class Acc>
__global__ void __launch_bounds__(kFinishThreads) finish_kernel(const __grid_constant__ NormArgs a) {
    __shared__ uint64_t sm[kFinishThreads / 32], sums[kFinishCtas];
    if (blockIdx.x < a.record_ctas) cluster_started();
    griddep_wait();
    griddep_launch_dependents();
    Acc acc;
    if (blockIdx.x < a.record_ctas) {
#pragma unroll 8
        for (uint32_t i = blockIdx.x * kFinishThreads + threadIdx.x; i < a.n_items; i += kFinishCtas * kFinishThreads)
            acc.join(a.partials[i]);
        cta_join<Acc, kFinishThreads / 32>(acc, sm);
        const Acc all = cluster_join(acc, sums, kFinishCtas, blockIdx.x);
        if (blockIdx.x == 0 && threadIdx.x == 0) store_record(a.result, make_record(all, a.pre_scale, a.max_norm));
        if (blockIdx.x == 0 && threadIdx.x < kNormLists) a.drawn[32 * threadIdx.x] = 0;  // for the next call
        return;
    }
    const uint32_t t = blockIdx.x - a.record_ctas;
    if (t >= a.n_tensors) return;
#pragma unroll 8
    for (uint32_t i = a.first[t] + threadIdx.x; i < a.first[t + 1]; i += kFinishThreads) acc.join(a.partials[i]);
    cta_join<Acc, kFinishThreads / 32>(acc, sm);
    if (threadIdx.x == 0) a.tensor_norms[t] = make_record(acc, a.pre_scale, 0.0).norm;
}

// Small sets: one cluster, an item to a warp, the sums exchanged through the
// CTAs' shared memory; with SCALE the gradients wait in registers for the
// factor: one launch and one read where the general path takes three and two.
// Bound by its chain of latencies: 17 vectors 3.75 us a norm (4.96 with the
// general kernels), 0.4 MB 5.25 us a clip (6.88).
template <class Acc, bool SCALE>
__global__ void __launch_bounds__(kSmallThreads) small_kernel(const __grid_constant__ NormArgs a) {
    __shared__ uint64_t sm[kSmallWarps], sums[kSmallCtas];
    __shared__ float factor;
    cluster_started();
    constexpr int U = kSmallItemElems / 128;  // float32 vectors of a full item, a lane's
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t it = blockIdx.x * kSmallWarps + warp;
    GradItem w = {};
    if (it < a.n_items) w = a.items[it];
    griddep_wait();
    griddep_launch_dependents();
    const bool bf = w.flags & kGradBf16;
    const uint32_t head = bf ? Vectors<true>(w.src, w.count).head : Vectors<false>(w.src, w.count).head;
    const uint32_t n = (w.count - head) / (bf ? 8 : 4), tail = w.count - head - n * (bf ? 8 : 4);
    const char* body = w.src + head * (bf ? 2 : 4);
    uint4 x[U];
    uint32_t edge[2] = {0, 0};
#pragma unroll
    for (int u = 0; u < U; ++u)
        x[u] = lane + 32 * u < n ? load128(body + 16ull * (lane + 32 * u)) : make_uint4(0, 0, 0, 0);
    if (lane < head) edge[0] = bf ? load_elem<true>(w.src, lane) : load_elem<false>(w.src, lane);
    if (lane < tail)
        edge[1] = bf ? load_elem<true>(w.src, w.count - tail + lane) : load_elem<false>(w.src, w.count - tail + lane);
    Acc acc;
    if (bf) {
        if (!acc.template feed<true, U>(x)) acc.add(Acc::template again<true, U>(body, lane, n));
    } else {
        if (!acc.template feed<false, U>(x)) acc.add(Acc::template again<false, U>(body, lane, n));
    }
    if (lane < head) acc.one(edge[0]);
    if (lane < tail) acc.one(edge[1]);
    warp_join(acc);
    if (lane == 0) {
        if (it < a.n_items) a.partials[it] = acc.bits();
        sm[warp] = acc.bits();
    }
    __syncthreads();
    Acc cta;
    if (warp == 0) {
        if (lane < kSmallWarps) cta.join(sm[lane]);
        warp_join(cta);
    }
    const Acc all = cluster_join(cta, sums, gridDim.x, blockIdx.x);
    if (threadIdx.x == 0) {
        const Record r = make_record(all, a.pre_scale, a.max_norm);
        factor = r.scale;
        if (blockIdx.x == 0) store_record(a.result, r);
    }
    if (!SCALE) return;
    __syncthreads();
    const float f = factor;
    if ((w.flags & kInPlace) && f == 1.f) return;
    const bool ob = w.flags & kOutBf16;
    const auto store = [&](uint32_t i, float4 v, bool whole) {
        v = make_float4(__fmul_rn(v.x, f), __fmul_rn(v.y, f), __fmul_rn(v.z, f), __fmul_rn(v.w, f));
        if (ob)
            store_quad<true>(w.dst, i, v, whole);
        else
            store_quad<false>(w.dst, i, v, whole);
    };
    const bool whole = ob ? quad_aligned<true>(w.dst, head) : quad_aligned<false>(w.dst, head);
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t q = lane + 32 * u;
        if (q >= n) continue;
        if (bf) {
            store(head + 8 * q, make_float4(bf_lo(x[u].x), bf_hi(x[u].x), bf_lo(x[u].y), bf_hi(x[u].y)), whole);
            store(head + 8 * q + 4, make_float4(bf_lo(x[u].z), bf_hi(x[u].z), bf_lo(x[u].w), bf_hi(x[u].w)), whole);
        } else {
            store(head + 4 * q, make_float4(__uint_as_float(x[u].x), __uint_as_float(x[u].y), __uint_as_float(x[u].z),
                                            __uint_as_float(x[u].w)), whole);
        }
    }
    const auto store_edge = [&](uint32_t i, uint32_t bits) {
        const float v = __fmul_rn(__uint_as_float(bits), f);
        if (ob)
            store_elem<true>(w.dst, i, v);
        else
            store_elem<false>(w.dst, i, v);
    };
    if (lane < head) store_edge(lane, edge[0]);
    if (lane < tail) store_edge(w.count - tail + lane, edge[1]);
}

// ---------------------------------------------------------------- the scaling

// dst = round(f * src) for n quads of four elements, the source on its
// alignment, the destination too if WHOLE.  (Every x gets a value: one left
// undefined past the end would hold its register through the caller's loop.)
template <bool SB, bool DB, bool WHOLE, int U>
__device__ __forceinline__ void scale_quads(const char* src, char* dst, uint32_t n, float f, uint32_t lane) {
#pragma unroll 1
    for (uint32_t q = lane; q < n; q += 32 * U) {
        const char* from = src + q * (SB ? 8 : 16);
        char* to = dst + q * (DB ? 8 : 16);
        float4 x[U];
#pragma unroll
        for (int u = 0; u < U; ++u)
            x[u] = q + 32 * u < n ? load_quad<SB, true>(from, 128 * u, true) : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (q + 32 * u < n)
                store_quad<DB, true>(to, 128 * u,
                                     make_float4(__fmul_rn(x[u].x, f), __fmul_rn(x[u].y, f), __fmul_rn(x[u].z, f),
                                                 __fmul_rn(x[u].w, f)),
                                     WHOLE);
    }
}

// One of `warps` warps' part of an item; the first also takes the elements
// before and after the quads.
template <bool SB, bool DB>
__device__ __forceinline__ void scale_item(const GradItem& it, float f, uint32_t warp, uint32_t warps, uint32_t lane) {
    const uint32_t head = min(it.count, head_elems<SB>(it.src, SB ? 8 : 16));
    const uint32_t nq = (it.count - head) / 4;
    const uint32_t part = (nq + 32 * warps - 1) / (32 * warps) * 32, at = min(nq, warp * part);
    const char* from = it.src + (head + 4 * at) * (SB ? 2 : 4);
    char* to = it.dst + (head + 4 * at) * (DB ? 2 : 4);
    if (quad_aligned<DB>(to, 0))
        scale_quads<SB, DB, true, 8>(from, to, min(part, nq - at), f, lane);
    else
        scale_quads<SB, DB, false, 4>(from, to, min(part, nq - at), f, lane);
    if (warp != 0) return;
    const uint32_t done = head + nq * 4;
    if (lane < head) store_elem<DB>(it.dst, lane, __fmul_rn(__uint_as_float(load_elem<SB>(it.src, lane)), f));
    if (done + lane < it.count)
        store_elem<DB>(it.dst, done + lane, __fmul_rn(__uint_as_float(load_elem<SB>(it.src, done + lane)), f));
}

// The items in the reverse of the norm's order: the norm leaves its last ones
// in L2.  Loads and stores are streaming (neither is used again), so the
// results do not push out the gradients that wait there.  item_warps warps
// share an item, 4 KB of gradients to each: a clip of 2.7 GB of float32 takes
// 1144 us, 1155 with twice that a warp, 1164 with an item a warp.
// In place, a factor of exactly 1 leaves nothing to do, as for most steps of a
// training that runs well; then the CTAs' starts are what is left, and a CTA
// takes several items in turn: 2.7 GB within the bound 377 us, 451 with an item
// a CTA; scaled it is the slower, 1154 us against 1133.  Into other tensors,
// which are written either way, it is an item a CTA: 1144 us against 1164.
__global__ void __launch_bounds__(kGradThreads, 4) scale_kernel(const __grid_constant__ ScaleArgs a) {
    const uint32_t side = kGradWarps / a.item_warps;  // items side by side in a CTA
    const uint32_t lane = threadIdx.x & 31, warp = threadIdx.x >> 5, part = warp % a.item_warps;
    uint32_t i = blockIdx.x * a.rounds * side + warp / a.item_warps;
    GradItem it = {};
    if (i < a.n_items) it = a.items[a.n_items - 1 - i];
    griddep_wait();
    griddep_launch_dependents();
    const float f = __ldcg(a.result + 1);
    if (a.in_place && f == 1.f) return;
#pragma unroll 1
    for (uint32_t r = 0; r < a.rounds && i < a.n_items; ++r) {
        if (r > 0) it = a.items[a.n_items - 1 - i];
        if (!(it.flags & kInPlace) || f != 1.f) {
            switch (it.flags & (kGradBf16 | kOutBf16)) {
                case 0: scale_item<false, false>(it, f, part, a.item_warps, lane); break;
                case kGradBf16: scale_item<true, false>(it, f, part, a.item_warps, lane); break;
                case kOutBf16: scale_item<false, true>(it, f, part, a.item_warps, lane); break;
                default: scale_item<true, true>(it, f, part, a.item_warps, lane);
            }
        }
        i += side;
    }
}

// ---------------------------------------------------------------------- AdamW

// One element: moments and parameter, in float32.  The decay is subtracted
// with the update (p - (lr wd p + update)), so its small factor is never
// rounded against 1.
__device__ __forceinline__ void adam_one(const AdamArgs& a, const AdamScalars& s, float decay, float f, float& p,
                                         float g, float& m, float& v) {
    g = __fmul_rn(g, f);
    m = __fmaf_rn(a.omb1, g, __fmul_rn(a.beta1, m));
    v = __fmaf_rn(__fmul_rn(a.omb2, g), g, __fmul_rn(a.beta2, v));
    const float den = __fmaf_rn(__fsqrt_rn(v), s.inv_bc2, a.eps);
    const float upd = __fmul_rn(s.step_size, __fdiv_rn(m, den));
    p = __fsub_rn(p, __fmaf_rn(decay, p, upd));
}

__device__ __forceinline__ void adam_quad(const AdamArgs& a, const AdamScalars& s, float decay, float f, float4& p,
                                          float4 g, float4& m, float4& v) {
    adam_one(a, s, decay, f, p.x, g.x, m.x, v.x);
    adam_one(a, s, decay, f, p.y, g.y, m.y, v.y);
    adam_one(a, s, decay, f, p.z, g.z, m.z, v.z);
    adam_one(a, s, decay, f, p.w, g.w, m.w, v.w);
}

template <bool PB, bool GB, bool COPY>
__device__ __forceinline__ void adam_elem(const AdamArgs& a, const AdamScalars& s, const AdamItem& it, float decay,
                                          float f, uint32_t i) {
    char* mp = reinterpret_cast<char*>(it.m);
    char* vp = reinterpret_cast<char*>(it.v);
    float p = __uint_as_float(load_elem<PB>(it.p, i)), m = __uint_as_float(load_elem<false>(mp, i));
    const float g = __uint_as_float(load_elem<GB>(it.g, i));
    float v = __uint_as_float(load_elem<false>(vp, i));
    adam_one(a, s, decay, f, p, g, m, v);
    store_elem<PB>(it.p, i, p);
    store_elem<false>(mp, i, m);
    store_elem<false>(vp, i, v);
    if (COPY) store_elem<true>(it.w, i, p);
}

template <bool PB, bool GB, bool COPY, bool WHOLE>
__device__ __forceinline__ void adam_item(const AdamArgs& a, const AdamScalars& s, const AdamItem& it, float f,
                                          uint32_t lane) {
    constexpr int U = WHOLE ? 2 : 1;
    const float decay = __fmul_rn(s.lr_decay, it.decay);
    char* mp = reinterpret_cast<char*>(it.m);
    char* vp = reinterpret_cast<char*>(it.v);
    const uint32_t head = min(it.count, head_elems<false>(mp, 16));
    const bool pw = WHOLE || quad_aligned<PB>(it.p, head), gw = WHOLE || quad_aligned<GB>(it.g, head);
    const bool vw = WHOLE || quad_aligned<false>(vp, head), ww = WHOLE || (COPY && quad_aligned<true>(it.w, head));
    const uint32_t nq = (it.count - head) / 4;
    const uint32_t done = head + nq * 4;
    for (uint32_t q = lane; q < nq; q += 32 * U) {
        float4 p[U], g[U], m[U], v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = head + 4 * (q + 32 * u);
            if (q + 32 * u < nq) {
                g[u] = load_quad<GB>(it.g, i, gw);
                m[u] = load_quad<false>(mp, i, true);
                v[u] = load_quad<false>(vp, i, vw);
                p[u] = load_quad<PB>(it.p, i, pw);
            }
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t i = head + 4 * (q + 32 * u);
            if (q + 32 * u < nq) {
                adam_quad(a, s, decay, f, p[u], g[u], m[u], v[u]);
                store_quad<PB>(it.p, i, p[u], pw);
                store_quad<false>(mp, i, m[u], true);
                store_quad<false>(vp, i, v[u], vw);
                if (COPY) store_quad<true>(it.w, i, p[u], ww);
            }
        }
    }
    if (lane < head) adam_elem<PB, GB, COPY>(a, s, it, decay, f, lane);
    if (done + lane < it.count) adam_elem<PB, GB, COPY>(a, s, it, decay, f, done + lane);
}

// A warp updates one item; with a record, nothing is touched when the
// gradients held an infinity or NaN.  The items in the reverse of the norm's
// order, whose last gradients may still be in L2.  Bound by HBM.
// WHOLE: every stream moves in quads.  Two quads of each in flight a thread at
// 4 CTAs an SM; a stream off its alignment takes single elements, which need
// more warps instead: one quad, 6 CTAs (whose 40 registers a thread spill a
// few: 16 bytes stored, 104 read).  Measured both ways, norm included: a billion
// float32 parameters 4541 and 4653 us; 122M bf16 parameters whose bf16 gradients
// are packed tight at odd sizes 501 and 440 (457 with 5 CTAs).
template <bool WHOLE>
__global__ void __launch_bounds__(kGradThreads, WHOLE ? 4 : 6) adamw_kernel(const __grid_constant__ AdamArgs a) {
    const uint32_t lane = threadIdx.x & 31;
    const uint32_t w = blockIdx.x * kGradWarps + (threadIdx.x >> 5);
    AdamItem it = {};
    if (w < a.n_items) it = a.items[a.n_items - 1 - w];
    griddep_wait();
    griddep_launch_dependents();
    if (w >= a.n_items) return;
    float f = 1.f;
    if (a.result) {
        f = __ldcg(a.result + 1);
        if (__ldcg(a.result + 2) != 0.f) return;
    }
    AdamScalars s = a.scalars;
    if (a.counted) s = {__ldcg(&a.counted->step_size), __ldcg(&a.counted->inv_bc2), __ldcg(&a.counted->lr_decay)};
    switch (it.flags & (kGradBf16 | kParamBf16 | kHasCopy)) {
        case 0: return adam_item<false, false, false, WHOLE>(a, s, it, f, lane);
        case kGradBf16: return adam_item<false, true, false, WHOLE>(a, s, it, f, lane);
        case kHasCopy: return adam_item<false, false, true, WHOLE>(a, s, it, f, lane);
        case kHasCopy | kGradBf16: return adam_item<false, true, true, WHOLE>(a, s, it, f, lane);
        case kParamBf16: return adam_item<true, false, false, WHOLE>(a, s, it, f, lane);
        default: return adam_item<true, true, false, WHOLE>(a, s, it, f, lane);
    }
}

// x^n for n >= 1, by squaring.
__device__ double power(double x, uint64_t n) {
    double y = 1.0;
    for (; n > 0; n >>= 1, x *= x)
        if (n & 1) y *= x;
    return y;
}

// The number of an update, and what follows from it, on the device: a CUDA
// graph of a training step then counts its replays, and a skipped update is
// not counted.  A thread of one warp and one of another take a moment each;
// float32's reciprocals and a Newton step in float64 stand for its divisions
// and root, whose long chains the update would wait for.
__global__ void __launch_bounds__(64) count_kernel(const __grid_constant__ CountArgs a) {
    griddep_wait();
    griddep_launch_dependents();
    if (a.result && a.result[2] != 0.f) return;
    const uint64_t t = *a.steps + 1;
    if (threadIdx.x == 0) {
        const double lr = a.lr ? static_cast<double>(*a.lr) : a.host_lr;
        const double d = 1.0 - power(a.beta1, t), y = __frcp_rn(static_cast<float>(d));
        a.scalars->step_size = static_cast<float>(lr * fma(y, fma(-d, y, 1.0), y));
        a.scalars->lr_decay = static_cast<float>(lr * a.weight_decay);
    } else if (threadIdx.x == 32) {
        const double d = 1.0 - power(a.beta2, t), y = rsqrtf(static_cast<float>(d));
        a.scalars->inv_bc2 = static_cast<float>(fma(y, fma(-0.5 * d * y, y, 0.5), y));
    }
    __syncthreads();
    if (threadIdx.x == 0) *a.steps = t;
}

// ------------------------------------------------------------------ the items

__device__ __forceinline__ GradItem make_item(const GradTensor& t, uint64_t lo, uint64_t hi) {
    GradItem it = {};
    it.src = t.src + lo * (t.flags & kGradBf16 ? 2 : 4);
    it.dst = t.dst + lo * (t.flags & kOutBf16 ? 2 : 4);
    it.count = static_cast<uint32_t>(hi - lo);
    it.flags = t.flags;
    return it;
}

__device__ __forceinline__ AdamItem make_item(const AdamTensor& t, uint64_t lo, uint64_t hi) {
    AdamItem it = {};
    it.p = t.p + lo * (t.flags & kParamBf16 ? 2 : 4);
    it.g = t.g + lo * (t.flags & kGradBf16 ? 2 : 4);
    it.m = t.m + lo;
    it.v = t.v + lo;
    it.w = t.flags & kHasCopy ? t.w + lo * 2 : nullptr;
    it.count = static_cast<uint32_t>(hi - lo);
    it.flags = t.flags;
    it.decay = t.decay;
    return it;
}

// Once per handle, a thread an item: the tensor whose items hold it, by
// halving, and the item's place in it.
template <class Tensor, class Item>
__global__ void items_kernel(const Tensor* tensors, const uint32_t* first, int n, Item* items) {
    const uint32_t i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= first[n]) return;
    int lo = 0, hi = n;  // first[lo] <= i < first[hi]
    while (hi - lo > 1) {
        const int mid = lo + (hi - lo) / 2;
        if (first[mid] <= i)
            lo = mid;
        else
            hi = mid;
    }
    const Tensor t = tensors[lo];
    const uint32_t k = i - first[lo];
    items[i] = make_item(t, t.split.begin(k), t.split.end(k));
}

template <class Tensor, class Item>
cudaError_t make_items(const Tensor* tensors, const uint32_t* first, int n, uint32_t n_items, Item* items,
                       cudaStream_t st) {
    // (a launch by <<<>>> has its status in the thread's last error, where an earlier call's may still be)
    void* args[] = {&tensors, &first, &n, &items};
    return cudaLaunchKernel(reinterpret_cast<const void*>(&items_kernel<Tensor, Item>), dim3((n_items + 255) / 256),
                            dim3(256), args, 0, st);
}

template <class Args>
cudaError_t launch(void (*f)(Args), const Args& a, uint32_t grid, int block, cudaStream_t st, uint32_t cluster = 0) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(static_cast<unsigned>(block));
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = AR_PDL;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster ? 2 : 1;
    void* args[] = {const_cast<Args*>(&a)};
    return cudaLaunchKernelExC(&cfg, reinterpret_cast<const void*>(f), args);
}

}  // namespace

cudaError_t launch_items(const GradTensor* tensors, const uint32_t* first, int n, uint32_t n_items, GradItem* items,
                         cudaStream_t st) {
    return make_items(tensors, first, n, n_items, items, st);
}

cudaError_t launch_items(const AdamTensor* tensors, const uint32_t* first, int n, uint32_t n_items, AdamItem* items,
                         cudaStream_t st) {
    return make_items(tensors, first, n, n_items, items, st);
}

cudaError_t launch_norm(const NormArgs& a, bool keep, int num_sms, cudaStream_t st) {
    const bool max = a.kind == AR_NORM_MAX;
    const uint32_t wave = static_cast<uint32_t>(num_sms) * kNormCtasPerSm, ctas = grad_ctas(a.n_items);
    return launch(keep ? (max ? norm_kernel<MaxAbs, true> : norm_kernel<SumSquares, true>)
                       : (max ? norm_kernel<MaxAbs, false> : norm_kernel<SumSquares, false>),
                  a, ctas < wave ? ctas : wave, kGradThreads, st);
}

cudaError_t launch_small(const NormArgs& a, bool scale, cudaStream_t st) {
    const bool max = a.kind == AR_NORM_MAX;
    const uint32_t ctas = a.n_items == 0 ? 1 : (a.n_items + kSmallWarps - 1) / kSmallWarps;
    return launch(scale ? (max ? small_kernel<MaxAbs, true> : small_kernel<SumSquares, true>)
                        : (max ? small_kernel<MaxAbs, false> : small_kernel<SumSquares, false>),
                  a, ctas, kSmallThreads, st, ctas);
}

cudaError_t launch_finish(const NormArgs& a, cudaStream_t st) {
    const uint32_t ctas = a.record_ctas + (a.n_tensors + kFinishCtas - 1) / kFinishCtas * kFinishCtas;
    return launch(a.kind == AR_NORM_MAX ? finish_kernel<MaxAbs> : finish_kernel<SumSquares>, a, ctas, kFinishThreads,
                  st, kFinishCtas);
}

cudaError_t launch_scale(const ScaleArgs& a, cudaStream_t st) {
    const uint32_t items = a.rounds * (kGradWarps / a.item_warps);  // of a CTA
    return launch(scale_kernel, a, (a.n_items + items - 1) / items, kGradThreads, st);
}

cudaError_t launch_count(const CountArgs& a, cudaStream_t st) { return launch(count_kernel, a, 1, 64, st); }

cudaError_t launch_adamw(const AdamArgs& a, bool whole, cudaStream_t st) {
    return launch(whole ? adamw_kernel<true> : adamw_kernel<false>, a, grad_ctas(a.n_items), kGradThreads, st);
}

}  // namespace ar
