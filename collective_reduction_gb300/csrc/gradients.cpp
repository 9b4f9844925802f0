// C ABI of the work over many tensors after a gradient allreduce: handles
// that bind the caller's tensors (checked once, their ranges uploaded once)
// and the calls that launch the kernels on them.
#include "gradients.hpp"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <new>
#include <vector>

#include "bufcheck.hpp"

namespace {

constexpr double kFloatMax = 3.4028234e38;
constexpr int kMaxTensors = 1 << 20;
constexpr uint64_t kMaxElems = uint64_t(1) << 40;

// One wave of warps on GB300's 152 SMs: the norm kernel runs 3 CTAs of 8 warps
// on each, the AdamW kernel 4 (off alignment 6: its ranges are sized for 4 all the
// same).  Constants, as a set's ranges follow from its sizes alone, also where no
// device is asked (ar_tensors_lowering).
//
// A set takes as many waves of ranges as full ones would need, and the range is
// what each warp gets then, rounded up to a multiple of the step that is larger.
// The rounding counts where a warp gets one or a few steps: 15 MB of float32
// (one step each) are split into ranges of two, which half of a wave takes, 25 MB
// into 0.83 of a wave, 180 MB (1.004 waves of full ranges) into 1.7.  Measured in a
// graph: a norm of 180 MB 31.9 us, 39.1 in full ranges, where a few warps have two
// and the others wait; one of 25 MB 9.8 us, 15.4 in ranges of one step.  Full: a norm
// of 4.2 GB takes in bf16 583 us in ranges of 12288 elements, 587 and 597 of 8192
// and 16384, in float32 1148 us, 1178 and 1167; AdamW on a billion, the norm
// included, 4541 us in ranges of 512, 4559 and 4575 of 768 and 1024, and on 0.4M
// 3.85 us in ranges of 256, 8.4 of 1024.  An AdamW range is 64 bytes of table: an
// eighth of a byte a parameter.
constexpr uint64_t kNormWave = 152 * ar::kNormCtasPerSm * ar::kGradWarps, kAdamWave = 152 * 4 * ar::kGradWarps;
constexpr uint32_t kGradItemMax = 12288, kAdamItemStep = 256, kAdamItemMax = 512;

uint32_t item_elems(int n, const uint64_t* counts, uint64_t wave, uint32_t step, uint32_t most) {
    uint64_t total = 0;
    for (int t = 0; t < n; ++t) total += counts[t];
    const uint64_t waves = total / (wave * most) + 1;
    return static_cast<uint32_t>((total / (wave * waves) / step + 1) * step);
}
uint32_t grad_item_elems(int n, const uint64_t* counts) {
    return item_elems(n, counts, kNormWave, ar::kSmallItemElems, kGradItemMax);
}
uint32_t adam_item_elems(int n, const uint64_t* counts) {
    return item_elems(n, counts, kAdamWave, kAdamItemStep, kAdamItemMax);
}

// Gradient bytes at the end of a set that may stay in L2 (of 129 MB) after a norm
// that has a bound, the ones before them leaving first: the scaling or the update
// reads the gradients next, last ones first.  Measured without and with, in a
// graph that writes the gradients first (its time included): clipping into other
// tensors 80 MB of float32 87.3 and 88.2 us, 640 MB 703 and 695, 600 MB of bf16 665
// and 654; the norm and AdamW on 160 MB of float32 gradients 296 and 292, on 600 MB of
// bf16 1609 and 1596.
constexpr uint64_t kKeepBytes = 64ull << 20;

ar_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
    cudaGetLastError();  // reported here: not once more by whoever looks at the thread's last error
    return e == cudaErrorMemoryAllocation ? AR_ERR_NOMEM : AR_ERR_CUDA;
}

bool float_dtype(ar_dtype d) { return d == AR_FLOAT32 || d == AR_BFLOAT16; }
int esize(ar_dtype d) { return d == AR_BFLOAT16 ? 2 : 4; }

// The number of tensors, their sizes and element types.
ar_status check_layout(int n, const uint64_t* counts, const ar_dtype* dtypes) {
    if (n < 0 || (n > 0 && (!counts || !dtypes))) return AR_ERR_INVALID_ARG;
    if (n > kMaxTensors) return AR_ERR_UNSUPPORTED;
    uint64_t total = 0;
    for (int t = 0; t < n; ++t) {
        if (dtypes[t] != AR_INT32 && !float_dtype(dtypes[t])) return AR_ERR_INVALID_ARG;
        if (!float_dtype(dtypes[t]) || counts[t] > kMaxElems) return AR_ERR_UNSUPPORTED;
        total += counts[t];
        if (total > kMaxElems) return AR_ERR_UNSUPPORTED;
    }
    return AR_OK;
}

void fill_info(int n, const uint64_t* counts, uint64_t item_elems, size_t items, ar_tensors_info* info) {
    std::memset(info, 0, sizeof(*info));
    info->n_tensors = n;
    for (int t = 0; t < n; ++t) info->elems += counts[t];
    info->n_items = items;
    info->item_elems = item_elems;
}

// Device memory in parts, each on a 256-byte boundary.
struct DeviceMemory {
    char* dev = nullptr;
    size_t bytes = 0;
    size_t part(size_t n) {  // its offset
        const size_t at = bytes;
        bytes += (n + 255) / 256 * 256;
        return at;
    }
    cudaError_t allocate() { return cudaMalloc(&dev, bytes); }
    template <class T>
    T* at(size_t offset) const {
        return reinterpret_cast<T*>(dev + offset);
    }
    ~DeviceMemory() {
        if (dev) cudaFree(dev);
    }
};

// The tensors' first items from their splits; their number, or 0 with *ok
// false when there are more than the kernels index.
template <class Tensor>
uint32_t first_items(const std::vector<Tensor>& tensors, std::vector<uint32_t>& first, bool* ok) {
    uint64_t n = 0;
    first.assign(1, 0);
    for (const Tensor& t : tensors) {
        n += t.split.ranges();
        if (n > 0x7FFFFFFFu) {
            *ok = false;
            return 0;
        }
        first.push_back(static_cast<uint32_t>(n));
    }
    *ok = true;
    return static_cast<uint32_t>(n);
}

// Uploads the tensors and has the device write their items.  All of it is in
// place on return (a copy from pageable memory alone may return before that, and
// the calls may be on streams that do not wait for this one).
template <class Tensor, class Item>
cudaError_t upload_items(const std::vector<Tensor>& tensors, const std::vector<uint32_t>& first, uint32_t* d_first,
                         Item* d_items) {
    const uint32_t n_items = first.back();
    cudaError_t e = cudaMemcpy(d_first, first.data(), first.size() * sizeof(uint32_t), cudaMemcpyHostToDevice);
    Tensor* d_tensors = nullptr;
    if (n_items > 0) {
        if (e == cudaSuccess) e = cudaMalloc(&d_tensors, tensors.size() * sizeof(Tensor));
        if (e == cudaSuccess)
            e = cudaMemcpy(d_tensors, tensors.data(), tensors.size() * sizeof(Tensor), cudaMemcpyHostToDevice);
        if (e == cudaSuccess)
            e = ar::launch_items(d_tensors, d_first, static_cast<int>(tensors.size()), n_items, d_items, nullptr);
    }
    if (e == cudaSuccess) e = cudaStreamSynchronize(nullptr);
    cudaFree(d_tensors);
    return e;
}

// A positive number that float32 holds without losing digits.
bool float_normal(double x) { return x >= 1.17549436e-38 && x <= kFloatMax; }

// Frees a handle when its device has done its work, whichever is current.
template <class Handle>
ar_status destroy(Handle* h) {
    if (!h) return AR_ERR_INVALID_ARG;
    int now = -1;
    cudaError_t e = cudaGetDevice(&now);
    const bool other = e == cudaSuccess && now != h->device;
    if (other) e = cudaSetDevice(h->device);
    if (e == cudaSuccess) e = cudaDeviceSynchronize();
    delete h;
    if (other) cudaSetDevice(now);
    return cuda_status(e);
}

bool on_device(int device) {
    int now = -1;
    return cudaGetDevice(&now) == cudaSuccess && now == device;
}

// A caller's device float array that a call reads or writes.
bool float_buffer(const float* p, uint64_t n, int device) {
    return p && reinterpret_cast<uintptr_t>(p) % sizeof(float) == 0 &&
           ar::device_resident(p, n * sizeof(float), device);
}

}  // namespace

struct ar_grads_s {
    int n = 0, device = 0, num_sms = 0;
    ar_tensors_info info = {};
    uint32_t n_items = 0, keep_from = 0;
    uint32_t least_es = 4;  // bytes of the gradients' smallest element type
    bool in_place = true;   // every tensor is scaled where it is
    DeviceMemory memory;
    const ar::GradItem* items = nullptr;
    const uint32_t* first = nullptr;
    uint64_t* partials = nullptr;
    uint32_t* drawn = nullptr;
};

struct ar_adamw_s {
    int device = 0;
    ar_tensors_info info = {};
    uint32_t n_items = 0;
    bool whole = true;
    DeviceMemory memory;
    const ar::AdamItem* items = nullptr;
    ar::AdamScalars* scalars = nullptr;
};

namespace {

// The norm, and with `clip` the scaling by its record.
ar_status run_norm(ar_grads_s* h, ar_norm_kind kind, double pre_scale, double max_norm, float* result,
                   float* tensor_norms, bool clip, cudaStream_t st) {
    if (!h || (kind != AR_NORM_L2 && kind != AR_NORM_MAX)) return AR_ERR_INVALID_ARG;
    if (!float_normal(pre_scale) || !(max_norm >= 0.0)) return AR_ERR_INVALID_ARG;
    if (!on_device(h->device) || !float_buffer(result, 4, h->device)) return AR_ERR_INVALID_ARG;
    const bool norms = tensor_norms && h->n > 0;
    if (norms && !float_buffer(tensor_norms, h->n, h->device)) return AR_ERR_INVALID_ARG;
    ar::NormArgs a = {};
    a.items = h->items;
    a.n_items = h->n_items;
    a.keep_from = h->keep_from;
    a.kind = kind;
    a.partials = h->partials;
    a.drawn = h->drawn;
    a.pre_scale = pre_scale;
    a.max_norm = max_norm;
    a.result = result;
    a.first = h->first;
    a.tensor_norms = tensor_norms;
    a.n_tensors = norms ? h->n : 0;
    // one cluster holds the whole set (in the smallest ranges: a set in larger
    // ones has enough elements for half a wave of them)
    static_assert(kNormWave / 2 > ar::kSmallItems, "a set of kSmallItems ranges has the smallest ranges");
    const bool small = h->n_items <= ar::kSmallItems;
    a.record_ctas = small ? 0 : ar::kFinishCtas;
    cudaError_t e = small ? ar::launch_small(a, clip, st) : ar::launch_norm(a, max_norm <= kFloatMax, h->num_sms, st);
    if (e == cudaSuccess && (!small || norms)) {
        e = ar::launch_finish(a, st);
        // what would have put the counters back did not start
        if (e != cudaSuccess) cudaMemsetAsync(h->drawn, 0, sizeof(uint32_t) * 32 * ar::kNormLists, st);
    }
    if (e == cudaSuccess && clip && !small) {
        ar::ScaleArgs b = {};
        b.items = h->items;
        b.n_items = h->n_items;
        b.item_warps = 1;
        while (b.item_warps < ar::kGradWarps && b.item_warps * 2 * 4096 <= h->info.item_elems * h->least_es)
            b.item_warps *= 2;  // 4 KB of gradients at least to each
        // in place: several items to a CTA, while 8 waves of CTAs are left
        const uint32_t ctas = h->n_items / (ar::kGradWarps / b.item_warps);
        b.rounds = h->in_place ? std::min(8u, std::max(1u, ctas / (8 * 4 * 152))) : 1;
        b.in_place = h->in_place;
        b.result = result;
        e = ar::launch_scale(b, st);
    }
    return cuda_status(e);
}

bool float_finite(double x) { return x >= 0.0 && x <= kFloatMax; }

bool adam_params_ok(const ar_adamw_params& p) {
    return float_finite(p.lr) && float_finite(p.weight_decay) && float_finite(p.lr * p.weight_decay) &&
           float_normal(p.eps) && p.beta1 >= 0.0 && p.beta1 < 1.0 && p.beta2 >= 0.0 && p.beta2 < 1.0;
}

ar::AdamArgs adam_args(const ar_adamw_s* h, const ar_adamw_params& p, const float* result) {
    ar::AdamArgs a = {};
    a.items = h->items;
    a.n_items = h->n_items;
    a.result = result;
    a.beta1 = static_cast<float>(p.beta1);
    a.omb1 = static_cast<float>(1.0 - p.beta1);
    a.beta2 = static_cast<float>(p.beta2);
    a.omb2 = static_cast<float>(1.0 - p.beta2);
    a.eps = static_cast<float>(p.eps);
    return a;
}

}  // namespace

extern "C" {

ar_status ar_tensors_lowering(int n_tensors, const uint64_t* counts, const ar_dtype* dtypes, ar_tensors_info* out) {
    if (!out) return AR_ERR_INVALID_ARG;
    std::memset(out, 0, sizeof(*out));
    const ar_status s = check_layout(n_tensors, counts, dtypes);
    if (s != AR_OK) return s;
    // every tensor's ranges against its size, for a tensor on a range boundary
    // and for one off it
    const uint32_t e = grad_item_elems(n_tensors, counts);
    bool ok = true;
    uint64_t items = 0;
    for (int t = 0; t < n_tensors; ++t) {
        const uint32_t off = 1 + static_cast<uint32_t>(t) % (ar::kRangeAlign / esize(dtypes[t]) - 1);
        for (const uint32_t lead : {0u, off}) {
            const ar::RangeSplit s{counts[t], e, lead};
            uint64_t next = 0;
            for (uint64_t k = 0; k < s.ranges(); ++k) {
                const uint64_t lo = s.begin(k), hi = s.end(k);
                ok = ok && lo == next && hi > lo && hi - lo <= e && (lo == 0 || (lo + lead) % e == 0);
                next = hi;
            }
            ok = ok && next == counts[t];
            if (lead == 0) items += s.ranges();
        }
    }
    fill_info(n_tensors, counts, e, items, out);
    out->tiling_ok = ok ? 1 : 0;
    return AR_OK;
}

ar_status ar_grads_create(int n_tensors, const uint64_t* counts, const ar_dtype* grad_dtypes, void* const* grads,
                          const ar_dtype* out_dtypes, void* const* outs, ar_grads_t* out) {
    ar::TraceRange trace("ar_grads_create");
    if (!out) return AR_ERR_INVALID_ARG;
    *out = nullptr;
    ar_status s = check_layout(n_tensors, counts, grad_dtypes);
    if (s == AR_OK && outs) s = check_layout(n_tensors, counts, out_dtypes);
    if (s != AR_OK) return s;
    if (n_tensors > 0 && !grads) return AR_ERR_INVALID_ARG;
    ar_grads_s* h = nullptr;
    try {
        h = new ar_grads_s();
        cudaError_t e = cudaGetDevice(&h->device);
        if (e == cudaSuccess) e = cudaDeviceGetAttribute(&h->num_sms, cudaDevAttrMultiProcessorCount, h->device);
        if (e != cudaSuccess) {
            delete h;
            return cuda_status(e);
        }
        std::vector<ar::Span> spans;
        for (int t = 0; t < n_tensors; ++t) {
            const int es = esize(grad_dtypes[t]);
            spans.push_back({grads[t], counts[t] * es, es});
            if (outs && (outs[t] != grads[t] || out_dtypes[t] != grad_dtypes[t]))
                spans.push_back({outs[t], counts[t] * esize(out_dtypes[t]), esize(out_dtypes[t])});
        }
        s = ar::check_spans(spans, h->device);
        if (s != AR_OK) {
            delete h;
            return s;
        }
        const uint32_t elems = grad_item_elems(n_tensors, counts);
        std::vector<ar::GradTensor> tensors;
        for (int t = 0; t < n_tensors; ++t) {
            const ar_dtype gt = grad_dtypes[t], ot = outs ? out_dtypes[t] : gt;
            void* dst = outs ? outs[t] : grads[t];
            if (gt == AR_BFLOAT16) h->least_es = 2;
            h->in_place = h->in_place && (dst == grads[t] || counts[t] == 0);
            const uint32_t flags = (gt == AR_BFLOAT16 ? ar::kGradBf16 : 0) | (ot == AR_BFLOAT16 ? ar::kOutBf16 : 0) |
                                   (dst == grads[t] ? ar::kInPlace : 0);
            tensors.push_back({static_cast<const char*>(grads[t]), static_cast<char*>(dst),
                               {counts[t], elems, ar::lead_elems(grads[t], esize(gt))}, flags});
        }
        std::vector<uint32_t> first;
        bool fits = false;
        h->n = n_tensors;
        h->n_items = first_items(tensors, first, &fits);
        if (!fits) {
            delete h;
            return AR_ERR_UNSUPPORTED;
        }
        // the items that make up the last kKeepBytes
        h->keep_from = h->n_items;
        uint64_t room = kKeepBytes;
        for (int t = n_tensors - 1; t >= 0; --t) {
            const uint64_t bytes = counts[t] * esize(grad_dtypes[t]);
            if (bytes > room) {
                const uint64_t part = room / (elems * esize(grad_dtypes[t])), all = tensors[t].split.ranges();
                h->keep_from -= static_cast<uint32_t>(part < all ? part : all);
                break;
            }
            h->keep_from = first[t];
            room -= bytes;
        }
        const size_t o_items = h->memory.part(sizeof(ar::GradItem) * h->n_items);
        const size_t o_first = h->memory.part(sizeof(uint32_t) * first.size());
        const size_t o_partials = h->memory.part(sizeof(uint64_t) * h->n_items);
        const size_t o_drawn = h->memory.part(sizeof(uint32_t) * 32 * ar::kNormLists);
        e = h->memory.allocate();
        if (e == cudaSuccess) {
            h->items = h->memory.at<ar::GradItem>(o_items);
            h->first = h->memory.at<uint32_t>(o_first);
            h->partials = h->memory.at<uint64_t>(o_partials);
            h->drawn = h->memory.at<uint32_t>(o_drawn);
            e = cudaMemset(h->drawn, 0, sizeof(uint32_t) * 32 * ar::kNormLists);
        }
        if (e == cudaSuccess)
            e = upload_items(tensors, first, h->memory.at<uint32_t>(o_first), h->memory.at<ar::GradItem>(o_items));
        if (e != cudaSuccess) {
            delete h;
            return cuda_status(e);
        }
        fill_info(n_tensors, counts, elems, h->n_items, &h->info);
        h->info.table_bytes = h->memory.bytes;
        h->info.tiling_ok = 1;
        *out = h;
        return AR_OK;
    } catch (const std::bad_alloc&) {
        delete h;
        return AR_ERR_NOMEM;
    }
}

ar_status ar_grads_query(ar_grads_t h, ar_tensors_info* info) {
    if (!h || !info) return AR_ERR_INVALID_ARG;
    *info = h->info;
    return AR_OK;
}

ar_status ar_grads_destroy(ar_grads_t h) { return destroy(h); }

ar_status ar_grad_norm(ar_grads_t h, ar_norm_kind kind, double pre_scale, double max_norm, float* result,
                       float* tensor_norms, void* stream) {
    ar::TraceRange trace("ar_grad_norm");
    return run_norm(h, kind, pre_scale, max_norm, result, tensor_norms, false, static_cast<cudaStream_t>(stream));
}

ar_status ar_grad_clip(ar_grads_t h, ar_norm_kind kind, double pre_scale, double max_norm, float* result,
                       float* tensor_norms, void* stream) {
    ar::TraceRange trace("ar_grad_clip");
    return run_norm(h, kind, pre_scale, max_norm, result, tensor_norms, true, static_cast<cudaStream_t>(stream));
}

ar_status ar_adamw_create(int n_tensors, const uint64_t* counts, const ar_dtype* param_dtypes, void* const* params,
                          const ar_dtype* grad_dtypes, void* const* grads, float* const* exp_avg,
                          float* const* exp_avg_sq, void* const* copies, const float* decay, ar_adamw_t* out) {
    ar::TraceRange trace("ar_adamw_create");
    if (!out) return AR_ERR_INVALID_ARG;
    *out = nullptr;
    ar_status s = check_layout(n_tensors, counts, param_dtypes);
    if (s == AR_OK) s = check_layout(n_tensors, counts, grad_dtypes);
    if (s != AR_OK) return s;
    if (n_tensors > 0 && (!params || !grads || !exp_avg || !exp_avg_sq)) return AR_ERR_INVALID_ARG;
    for (int t = 0; t < n_tensors; ++t) {
        if (copies && param_dtypes[t] != AR_FLOAT32) return AR_ERR_INVALID_ARG;
        if (decay && !(decay[t] >= 0.f && decay[t] <= kFloatMax)) return AR_ERR_INVALID_ARG;
    }
    ar_adamw_s* h = nullptr;
    try {
        h = new ar_adamw_s();
        const cudaError_t e = cudaGetDevice(&h->device);
        if (e != cudaSuccess) {
            delete h;
            return cuda_status(e);
        }
        std::vector<ar::Span> spans;
        for (int t = 0; t < n_tensors; ++t) {
            const int pe = esize(param_dtypes[t]), ge = esize(grad_dtypes[t]);
            spans.push_back({params[t], counts[t] * pe, pe});
            spans.push_back({grads[t], counts[t] * ge, ge});
            spans.push_back({exp_avg[t], counts[t] * 4, 4});
            spans.push_back({exp_avg_sq[t], counts[t] * 4, 4});
            if (copies) spans.push_back({copies[t], counts[t] * 2, 2});
        }
        s = ar::check_spans(spans, h->device);
        if (s != AR_OK) {
            delete h;
            return s;
        }
        const uint32_t elems = adam_item_elems(n_tensors, counts);
        std::vector<ar::AdamTensor> tensors;
        for (int t = 0; t < n_tensors; ++t) {
            const uint32_t pe = esize(param_dtypes[t]), ge = esize(grad_dtypes[t]);
            const uint32_t flags = (pe == 2 ? ar::kParamBf16 : 0) | (ge == 2 ? ar::kGradBf16 : 0) |
                                   (copies ? ar::kHasCopy : 0);
            ar::AdamTensor a = {static_cast<char*>(params[t]), static_cast<const char*>(grads[t]), exp_avg[t],
                                exp_avg_sq[t], copies ? static_cast<char*>(copies[t]) : nullptr,
                                {counts[t], elems, ar::lead_elems(exp_avg[t], 4)}, flags, decay ? decay[t] : 1.f};
            // the first moments' quads start `o` elements in: do the others'?
            const uint64_t o = (16 - reinterpret_cast<uintptr_t>(a.m) % 16) % 16 / 4;
            const auto quads = [o](const void* p, uint32_t es) {
                return (reinterpret_cast<uintptr_t>(p) + o * es) % (4 * es) == 0;
            };
            h->whole = h->whole && (counts[t] == 0 || (quads(a.p, pe) && quads(a.g, ge) && quads(a.v, 4) &&
                                                       (!copies || quads(a.w, 2))));
            tensors.push_back(a);
        }
        std::vector<uint32_t> first;
        bool fits = false;
        h->n_items = first_items(tensors, first, &fits);
        if (!fits) {
            delete h;
            return AR_ERR_UNSUPPORTED;
        }
        const size_t o_items = h->memory.part(sizeof(ar::AdamItem) * h->n_items);
        const size_t o_first = h->memory.part(sizeof(uint32_t) * first.size());
        const size_t o_scalars = h->memory.part(sizeof(ar::AdamScalars));
        cudaError_t up = h->memory.allocate();
        if (up == cudaSuccess)
            up = upload_items(tensors, first, h->memory.at<uint32_t>(o_first), h->memory.at<ar::AdamItem>(o_items));
        if (up != cudaSuccess) {
            delete h;
            return cuda_status(up);
        }
        h->items = h->memory.at<ar::AdamItem>(o_items);
        h->scalars = h->memory.at<ar::AdamScalars>(o_scalars);
        fill_info(n_tensors, counts, elems, h->n_items, &h->info);
        h->info.table_bytes = h->memory.bytes;
        h->info.tiling_ok = 1;
        *out = h;
        return AR_OK;
    } catch (const std::bad_alloc&) {
        delete h;
        return AR_ERR_NOMEM;
    }
}

ar_status ar_adamw_query(ar_adamw_t h, ar_tensors_info* info) {
    if (!h || !info) return AR_ERR_INVALID_ARG;
    *info = h->info;
    return AR_OK;
}

ar_status ar_adamw_destroy(ar_adamw_t h) { return destroy(h); }

ar_status ar_adamw_step(ar_adamw_t h, const ar_adamw_params* p, const float* result, void* stream) {
    ar::TraceRange trace("ar_adamw_step");
    if (!h || !p || p->step < 1 || !adam_params_ok(*p)) return AR_ERR_INVALID_ARG;
    const double t = static_cast<double>(p->step);
    const double bc1 = 1.0 - std::pow(p->beta1, t), bc2 = 1.0 - std::pow(p->beta2, t);
    if (!float_finite(p->lr / bc1)) return AR_ERR_INVALID_ARG;
    if (!on_device(h->device) || (result && !float_buffer(result, 4, h->device))) return AR_ERR_INVALID_ARG;
    if (h->n_items == 0) return AR_OK;
    ar::AdamArgs a = adam_args(h, *p, result);
    a.scalars = {static_cast<float>(p->lr / bc1), static_cast<float>(1.0 / std::sqrt(bc2)),
                 static_cast<float>(p->lr * p->weight_decay)};
    return cuda_status(ar::launch_adamw(a, h->whole, static_cast<cudaStream_t>(stream)));
}

ar_status ar_adamw_step_counted(ar_adamw_t h, const ar_adamw_params* p, uint64_t* steps, const float* lr,
                                const float* result, void* stream) {
    ar::TraceRange trace("ar_adamw_step_counted");
    if (!h || !p || !adam_params_ok(*p)) return AR_ERR_INVALID_ARG;
    if (!on_device(h->device) || !steps || reinterpret_cast<uintptr_t>(steps) % sizeof(uint64_t) != 0 ||
        !ar::device_resident(steps, sizeof(uint64_t), h->device) || (lr && !float_buffer(lr, 1, h->device)) ||
        (result && !float_buffer(result, 4, h->device)))
        return AR_ERR_INVALID_ARG;
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    ar::CountArgs c = {};
    c.steps = steps;
    c.lr = lr;
    c.result = result;
    c.host_lr = p->lr;
    c.beta1 = p->beta1;
    c.beta2 = p->beta2;
    c.weight_decay = p->weight_decay;
    c.scalars = h->scalars;
    cudaError_t e = ar::launch_count(c, st);
    if (e != cudaSuccess || h->n_items == 0) return cuda_status(e);
    ar::AdamArgs a = adam_args(h, *p, result);
    a.counted = h->scalars;
    return cuda_status(ar::launch_adamw(a, h->whole, st));
}

}  // extern "C"
