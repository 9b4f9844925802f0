// C ABI of the work over many tensors after a gradient allreduce: handles
// that bind the caller's tensors (checked once, their ranges uploaded once)
// and the calls that launch the kernels on them.
#include "gradients.hpp"

#include <cmath>
#include <cstring>
#include <new>
#include <stdexcept>

#include "bufcheck.hpp"

namespace ar {

void split_tensors(int n, const uint64_t* counts, uint64_t item_elems, std::vector<TensorRange>& ranges,
                   std::vector<uint32_t>& first) {
    ranges.clear();
    first.assign(1, 0);
    for (int t = 0; t < n; ++t) {
        for (uint64_t at = 0; at < counts[t]; at += item_elems) {
            const uint64_t left = counts[t] - at;
            ranges.push_back({static_cast<uint32_t>(t), static_cast<uint32_t>(left < item_elems ? left : item_elems), at});
        }
        if (ranges.size() > 0x7FFFFFFFu) throw std::length_error("too many ranges");
        first.push_back(static_cast<uint32_t>(ranges.size()));
    }
}

}  // namespace ar

namespace {

constexpr int kMaxTensors = 1 << 20;
constexpr uint64_t kMaxElems = uint64_t(1) << 40;
constexpr uint64_t kGradItemElems = 4096;
constexpr uint64_t kAdamItemElems = 1024;

ar_status cuda_status(cudaError_t e) {
    if (e == cudaSuccess) return AR_OK;
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

struct DeviceBlob {
    std::vector<char> host;
    char* dev = nullptr;
    size_t reserve(size_t bytes) {  // zeroed bytes on a 256-byte boundary; returns their offset
        const size_t off = (host.size() + 255) / 256 * 256;
        host.resize(off + bytes);
        return off;
    }
    template <class T>
    size_t put(const std::vector<T>& v) {
        const size_t off = reserve(v.size() * sizeof(T));
        if (!v.empty()) std::memcpy(host.data() + off, v.data(), v.size() * sizeof(T));
        return off;
    }
    cudaError_t upload() {
        if (host.empty()) host.resize(256);
        cudaError_t e = cudaMalloc(&dev, host.size());
        if (e == cudaSuccess) e = cudaMemcpy(dev, host.data(), host.size(), cudaMemcpyHostToDevice);
        return e;
    }
    template <class T>
    T* at(size_t off) const {
        return reinterpret_cast<T*>(dev + off);
    }
    ~DeviceBlob() {
        if (dev) cudaFree(dev);
    }
};

bool on_device(int device) {
    int now = -1;
    return cudaGetDevice(&now) == cudaSuccess && now == device;
}

// A caller's device float array that a call reads or writes.
bool float_buffer(const float* p, uint64_t n, int device) {
    return p && reinterpret_cast<uintptr_t>(p) % sizeof(float) == 0 && ar::device_resident(p, n * sizeof(float), device);
}

}  // namespace

struct ar_grads_s {
    int n = 0, device = 0, num_sms = 0, grid = 0;
    ar_tensors_info info = {};
    uint32_t n_items = 0;
    DeviceBlob tables;     // items, first ranges, then the workspace below
    const ar::GradItem* items = nullptr;
    const uint32_t* first = nullptr;
    uint64_t* cta_partials = nullptr;
    uint32_t* counter = nullptr;
    uint64_t* item_partials = nullptr;
};

struct ar_adamw_s {
    int device = 0;
    ar_tensors_info info = {};
    uint32_t n_items = 0;
    DeviceBlob tables;
    const ar::AdamItem* items = nullptr;
};

namespace {

ar_status run_norm(ar_grads_s* h, ar_norm_kind kind, double pre_scale, double max_norm, float* result,
                   float* tensor_norms, cudaStream_t st) {
    if (!h || (kind != AR_NORM_L2 && kind != AR_NORM_MAX)) return AR_ERR_INVALID_ARG;
    // a factor below float32's smallest normal would lose its digits
    if (!(pre_scale >= 1.17549436e-38 && pre_scale <= 3.4028234e38) || !(max_norm >= 0.0)) return AR_ERR_INVALID_ARG;
    if (!on_device(h->device) || !float_buffer(result, 4, h->device)) return AR_ERR_INVALID_ARG;
    if (tensor_norms && h->n > 0 && !float_buffer(tensor_norms, h->n, h->device)) return AR_ERR_INVALID_ARG;
    ar::NormArgs a = {};
    a.items = h->items;
    a.n_items = h->n_items;
    a.kind = kind;
    a.cta_partials = h->cta_partials;
    a.item_partials = tensor_norms ? h->item_partials : nullptr;
    a.counter = h->counter;
    a.pre_scale = pre_scale;
    a.max_norm = max_norm;
    a.result = result;
    cudaError_t e = ar::launch_norm(a, h->grid, st);
    if (e == cudaSuccess && tensor_norms && h->n > 0) {
        ar::TensorNormArgs b = {};
        b.item_partials = h->item_partials;
        b.first = h->first;
        b.kind = kind;
        b.pre_scale = pre_scale;
        b.norms = tensor_norms;
        e = ar::launch_tensor_norms(b, h->n, st);
    }
    return cuda_status(e);
}

}  // namespace

extern "C" {

ar_status ar_tensors_lowering(int n_tensors, const uint64_t* counts, const ar_dtype* dtypes, ar_tensors_info* out) {
    if (!out) return AR_ERR_INVALID_ARG;
    std::memset(out, 0, sizeof(*out));
    const ar_status s = check_layout(n_tensors, counts, dtypes);
    if (s != AR_OK) return s;
    try {
        std::vector<ar::TensorRange> R;
        std::vector<uint32_t> first;
        ar::split_tensors(n_tensors, counts, kGradItemElems, R, first);
        fill_info(n_tensors, counts, kGradItemElems, R.size(), out);
        // the ranges against the sizes, apart from the loop that made them
        std::vector<uint64_t> next(n_tensors, 0);
        bool ok = first.size() == static_cast<size_t>(n_tensors) + 1 && first.back() == R.size();
        for (size_t i = 0; i < R.size() && ok; ++i) {
            const ar::TensorRange& r = R[i];
            ok = r.tensor < static_cast<uint32_t>(n_tensors) && r.count > 0 && r.count <= kGradItemElems &&
                 r.elem == next[r.tensor] && i >= first[r.tensor] && i < first[r.tensor + 1] && r.elem % 8 == 0;
            if (ok) next[r.tensor] += r.count;
        }
        for (int t = 0; t < n_tensors && ok; ++t) ok = next[t] == counts[t];
        out->tiling_ok = ok ? 1 : 0;
        return AR_OK;
    } catch (const std::length_error&) {
        return AR_ERR_UNSUPPORTED;
    } catch (const std::bad_alloc&) {
        return AR_ERR_NOMEM;
    }
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
        std::vector<ar::TensorRange> R;
        std::vector<uint32_t> first;
        ar::split_tensors(n_tensors, counts, kGradItemElems, R, first);
        std::vector<ar::GradItem> items;
        items.reserve(R.size());
        for (const ar::TensorRange& r : R) {
            const ar_dtype gt = grad_dtypes[r.tensor], ot = outs ? out_dtypes[r.tensor] : gt;
            void* dst = outs ? outs[r.tensor] : grads[r.tensor];
            ar::GradItem it = {};
            it.src = static_cast<const char*>(grads[r.tensor]) + r.elem * esize(gt);
            it.dst = static_cast<char*>(dst) + r.elem * esize(ot);
            it.count = r.count;
            it.flags = (gt == AR_BFLOAT16 ? ar::kGradBf16 : 0) | (ot == AR_BFLOAT16 ? ar::kOutBf16 : 0) |
                       (dst == grads[r.tensor] ? ar::kInPlace : 0);
            items.push_back(it);
        }
        h->n = n_tensors;
        h->n_items = static_cast<uint32_t>(items.size());
        h->grid = ar::norm_grid(h->n_items, h->num_sms);
        fill_info(n_tensors, counts, kGradItemElems, items.size(), &h->info);
        h->info.tiling_ok = 1;
        const size_t o_items = h->tables.put(items), o_first = h->tables.put(first);
        const size_t o_cta = h->tables.reserve(sizeof(uint64_t) * h->grid), o_counter = h->tables.reserve(256);
        const size_t o_parts = h->tables.reserve(sizeof(uint64_t) * items.size());
        e = h->tables.upload();
        if (e != cudaSuccess) {
            delete h;
            return cuda_status(e);
        }
        h->info.table_bytes = h->tables.host.size();
        h->items = h->tables.at<ar::GradItem>(o_items);
        h->first = h->tables.at<uint32_t>(o_first);
        h->cta_partials = h->tables.at<uint64_t>(o_cta);
        h->counter = h->tables.at<uint32_t>(o_counter);
        h->item_partials = h->tables.at<uint64_t>(o_parts);
        std::vector<char>().swap(h->tables.host);
        *out = h;
        return AR_OK;
    } catch (const std::length_error&) {
        delete h;
        return AR_ERR_UNSUPPORTED;
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

ar_status ar_grads_destroy(ar_grads_t h) {
    if (!h) return AR_ERR_INVALID_ARG;
    const cudaError_t e = cudaDeviceSynchronize();
    delete h;
    return cuda_status(e);
}

ar_status ar_grad_norm(ar_grads_t h, ar_norm_kind kind, double pre_scale, double max_norm, float* result,
                       float* tensor_norms, void* stream) {
    ar::TraceRange trace("ar_grad_norm");
    return run_norm(h, kind, pre_scale, max_norm, result, tensor_norms, static_cast<cudaStream_t>(stream));
}

ar_status ar_grad_clip(ar_grads_t h, ar_norm_kind kind, double pre_scale, double max_norm, float* result,
                       float* tensor_norms, void* stream) {
    ar::TraceRange trace("ar_grad_clip");
    const cudaStream_t st = static_cast<cudaStream_t>(stream);
    const ar_status s = run_norm(h, kind, pre_scale, max_norm, result, tensor_norms, st);
    if (s != AR_OK || h->n_items == 0) return s;
    ar::ScaleArgs a = {};
    a.items = h->items;
    a.n_items = h->n_items;
    a.result = result;
    return cuda_status(ar::launch_scale(a, st));
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
        if (decay && !(decay[t] >= 0.f && decay[t] <= 3.4028234e38f)) return AR_ERR_INVALID_ARG;
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
        std::vector<ar::TensorRange> R;
        std::vector<uint32_t> first;
        ar::split_tensors(n_tensors, counts, kAdamItemElems, R, first);
        std::vector<ar::AdamItem> items;
        items.reserve(R.size());
        for (const ar::TensorRange& r : R) {
            const uint32_t t = r.tensor;
            ar::AdamItem it = {};
            it.p = static_cast<char*>(params[t]) + r.elem * esize(param_dtypes[t]);
            it.g = static_cast<const char*>(grads[t]) + r.elem * esize(grad_dtypes[t]);
            it.m = exp_avg[t] + r.elem;
            it.v = exp_avg_sq[t] + r.elem;
            it.w = copies ? static_cast<char*>(copies[t]) + r.elem * 2 : nullptr;
            it.count = r.count;
            it.flags = (param_dtypes[t] == AR_BFLOAT16 ? ar::kParamBf16 : 0) |
                       (grad_dtypes[t] == AR_BFLOAT16 ? ar::kGradBf16 : 0) | (copies ? ar::kHasCopy : 0);
            it.decay = decay ? decay[t] : 1.f;
            items.push_back(it);
        }
        h->n_items = static_cast<uint32_t>(items.size());
        fill_info(n_tensors, counts, kAdamItemElems, items.size(), &h->info);
        h->info.tiling_ok = 1;
        const size_t o_items = h->tables.put(items);
        const cudaError_t up = h->tables.upload();
        if (up != cudaSuccess) {
            delete h;
            return cuda_status(up);
        }
        h->info.table_bytes = h->tables.host.size();
        h->items = h->tables.at<ar::AdamItem>(o_items);
        std::vector<char>().swap(h->tables.host);
        *out = h;
        return AR_OK;
    } catch (const std::length_error&) {
        delete h;
        return AR_ERR_UNSUPPORTED;
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

ar_status ar_adamw_destroy(ar_adamw_t h) {
    if (!h) return AR_ERR_INVALID_ARG;
    const cudaError_t e = cudaDeviceSynchronize();
    delete h;
    return cuda_status(e);
}

ar_status ar_adamw_step(ar_adamw_t h, const ar_adamw_params* p, const float* result, void* stream) {
    ar::TraceRange trace("ar_adamw_step");
    if (!h || !p) return AR_ERR_INVALID_ARG;
    const auto finite = [](double x) { return x >= 0.0 && x <= 3.4028234e38; };
    if (p->step < 1 || !finite(p->lr) || !finite(p->weight_decay) || !finite(p->lr * p->weight_decay) ||
        !finite(p->eps) || !(p->eps >= 1.17549436e-38) || !(p->beta1 >= 0.0 && p->beta1 < 1.0) ||
        !(p->beta2 >= 0.0 && p->beta2 < 1.0))
        return AR_ERR_INVALID_ARG;
    const double t = static_cast<double>(p->step);
    const double bc1 = 1.0 - std::pow(p->beta1, t), bc2 = 1.0 - std::pow(p->beta2, t);
    if (!finite(p->lr / bc1)) return AR_ERR_INVALID_ARG;
    if (!on_device(h->device) || (result && !float_buffer(result, 4, h->device))) return AR_ERR_INVALID_ARG;
    if (h->n_items == 0) return AR_OK;
    ar::AdamArgs a = {};
    a.items = h->items;
    a.n_items = h->n_items;
    a.result = result;
    a.beta1 = static_cast<float>(p->beta1);
    a.omb1 = static_cast<float>(1.0 - p->beta1);
    a.beta2 = static_cast<float>(p->beta2);
    a.omb2 = static_cast<float>(1.0 - p->beta2);
    a.step_size = static_cast<float>(p->lr / bc1);
    a.inv_bc2 = static_cast<float>(1.0 / std::sqrt(bc2));
    a.eps = static_cast<float>(p->eps);
    a.lr_decay = static_cast<float>(p->lr * p->weight_decay);
    return cuda_status(ar::launch_adamw(a, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
