// binding.cpp -- the Python entry points of the paged operators, in C++: checks
// of shapes, types and devices, allocation of results, and the call of the C ABI
// (include/kda.h).  These calls run once a layer in every decoding step, where the
// host's time is what a small call costs.  Time on the host of a call, through
// ctypes and checks in Python / through this: kda_latent_attn (one sequence, two
// launches) 17.5 / 9.1 us, kda_latent_append (64 tokens, query part) 9.5 / 3.6,
// kda_rope 10.1 / 4.9, kda_pages_copy (3 pages) 6.4 / 3.4.
//
// The library's functions are handed in as addresses (init), so that this module
// goes with whichever libkda_b200.so the package has loaded.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <cmath>
#include <optional>
#include <string>

#include "../../include/kda.h"

namespace py = pybind11;
using at::Tensor;
using OptTensor = std::optional<Tensor>;

namespace {

decltype(&kda_latent_attn) f_attn;
decltype(&kda_latent_attn) f_attn_selftest;
decltype(&kda_latent_append) f_append;
decltype(&kda_rope) f_rope;
decltype(&kda_pages_copy) f_copy;
decltype(&kda_pages_compact) f_compact;
decltype(&kda_last_error_message) f_message;
PyObject *error_type;            // KDAError(status, message)

[[noreturn]] void bad_value(const std::string &what) { throw py::value_error(what); }
[[noreturn]] void bad_type(const std::string &what) { throw py::type_error(what); }

void init(const py::dict &f, const py::object &error) {
    auto address = [&](const char *name) { return f[name].cast<uintptr_t>(); };
    f_attn = reinterpret_cast<decltype(f_attn)>(address("kda_latent_attn"));
    f_attn_selftest = reinterpret_cast<decltype(f_attn_selftest)>(address("kda_selftest_latent_attn"));
    f_append = reinterpret_cast<decltype(f_append)>(address("kda_latent_append"));
    f_rope = reinterpret_cast<decltype(f_rope)>(address("kda_rope"));
    f_copy = reinterpret_cast<decltype(f_copy)>(address("kda_pages_copy"));
    f_compact = reinterpret_cast<decltype(f_compact)>(address("kda_pages_compact"));
    f_message = reinterpret_cast<decltype(f_message)>(address("kda_last_error_message"));
    error_type = error.inc_ref().ptr();
}

std::string str(const Tensor &t) { return c10::str(t.device()); }

// The CUDA device of a call's first tensor.
c10::DeviceIndex device_of(const Tensor &t, const char *who) {
    if (!t.is_cuda()) bad_value(std::string(who) + " needs CUDA tensors (no CPU path)");
    return t.device().index();
}

// A contiguous tensor of the type on that device.
void *on(const Tensor &t, const char *name, c10::DeviceIndex dev, at::ScalarType type) {
    if (!t.is_cuda() || t.device().index() != dev)
        bad_value(std::string(name) + " is on " + str(t) + ", expected cuda:" + std::to_string(dev));
    if (t.scalar_type() != type) bad_type(std::string(name) + " must be " + c10::toString(type) + ", got " + c10::toString(t.scalar_type()));
    if (!t.is_contiguous()) bad_value(std::string(name) + " must be contiguous");
    return t.data_ptr();
}

kda_dtype dtype_of(const Tensor &t) {
    switch (t.scalar_type()) {
        case at::kBFloat16: return KDA_BF16;
        case at::kFloat: return KDA_F32;
        default: return (kda_dtype)-1;      // refused by the library
    }
}

int to_int(int64_t x, const char *what) {
    if (x > INT32_MAX || x < INT32_MIN) bad_value(std::string(what) + " is too large");
    return (int)x;
}

template <typename F, typename... A>
void call(F f, c10::DeviceIndex dev, A... args) {
    kda_status s;
    {
        // (a guard costs a driver call when it changes the device only)
        c10::cuda::OptionalCUDAGuard guard;
        if (c10::cuda::current_device() != dev) guard.set_index(dev);
        // other threads of the program go on, as a launch may wait for room in the queue
        py::gil_scoped_release release;
        s = f(args..., (void *)c10::cuda::getCurrentCUDAStream(dev).stream());
    }
    if (s != KDA_OK) {
        py::tuple what = py::make_tuple((int)s, f_message());
        PyErr_SetObject(error_type, what.ptr());
        throw py::error_already_set();
    }
}

struct Plan {
    const int32_t *table, *lens, *cu;
    int N, pages, page_size, max_pages;
    long long stride;
};

// The cache and its index arrays.
Plan plan(const std::string &who, int64_t T, const Tensor &cache, const Tensor &table, const Tensor &lens, const OptTensor &cu,
          c10::DeviceIndex dev, at::ScalarType type, int64_t dk) {
    if (cache.dim() != 3 || cache.size(2) != dk) bad_value(who + ": cache must be [num_pages, page_size, " + std::to_string(dk) + "]");
    if (!cache.is_cuda() || cache.device().index() != dev || cache.scalar_type() != type)
        bad_type(who + ": cache must be " + c10::toString(type) + " on cuda:" + std::to_string(dev));
    if (cache.stride(2) != 1 || cache.stride(1) != dk) bad_value(who + ": the rows of a page must be contiguous");
    Plan p;
    p.table = (const int32_t *)on(table, "page_table", dev, at::kInt);
    p.lens = (const int32_t *)on(lens, "kv_lens", dev, at::kInt);
    const int64_t N = lens.numel();
    if (table.dim() != 2 || lens.dim() != 1 || table.size(0) != N) bad_value(who + ": page_table must be [num_seqs, max_pages] and kv_lens [num_seqs]");
    p.cu = nullptr;
    if (cu) {
        p.cu = (const int32_t *)on(*cu, "cu_seqlens", dev, at::kInt);
        if (cu->dim() != 1 || cu->numel() != N + 1) bad_value(who + ": cu_seqlens must be [" + std::to_string(N + 1) + "]");
    } else if (N == 0 || T % N) {
        bad_value(who + ": without cu_seqlens the tokens must divide evenly over the sequences");
    }
    p.N = to_int(N, "num_seqs");
    p.pages = to_int(cache.size(0), "num_pages");
    p.page_size = to_int(cache.size(1), "page_size");
    p.max_pages = to_int(table.size(1), "max_pages");
    // (a pool of one page may report any stride; a page repeated by expand() has stride 0, which is no stride to hand
    // on: to the library 0 stands for pages one after the other, which here lie behind the tensor's end)
    if (cache.size(0) > 1 && cache.stride(0) < cache.size(1) * dk) bad_value(who + ": the pages of the cache must not overlap");
    p.stride = cache.size(0) > 1 ? cache.stride(0) : cache.size(1) * dk;
    return p;
}

// f: kda_latent_attn or its self-test
py::tuple attn_by(decltype(f_attn) f, const Tensor &q, const Tensor &cache, const Tensor &table, const Tensor &lens, int64_t dv,
                  const OptTensor &cu, const OptTensor &out_, const OptTensor &lse_, std::optional<double> scale, bool causal) {
    const auto dev = device_of(q, "kda_latent_attn");
    if (q.dim() != 3) bad_value("q must be [T,H,dk]");
    const int64_t T = q.size(0), H = q.size(1), dk = q.size(2);
    const auto type = q.scalar_type();
    const kda_dtype code = dtype_of(q);
    const void *qp = on(q, "q", dev, type);
    const Plan p = plan("kda_latent_attn", T, cache, table, lens, cu, dev, type, dk);
    if (dv < 0) bad_value("dv must not be negative");
    const int vd = to_int(dv, "dv");
    auto shaped = [&](const Tensor &t, const char *name, at::IntArrayRef s) {
        if (t.sizes() != s) bad_value(std::string(name) + " must be " + c10::str(s));
        return t;
    };
    Tensor out = out_ ? shaped(*out_, "out", {T, H, dv}) : at::empty({T, H, dv}, q.options());
    Tensor lse = lse_ ? shaped(*lse_, "lse", {T, H}) : at::empty({T, H}, q.options().dtype(at::kFloat));
    void *op = on(out, "out", dev, type);
    float *lp = (float *)on(lse, "lse", dev, at::kFloat);
    if (T > 0)
        call(f, dev, qp, (const void *)cache.data_ptr(), p.table, p.lens, p.cu, op, lp, to_int(T, "T"), to_int(H, "H"),
             to_int(dk, "dk"), vd, p.N, p.pages, p.page_size, p.max_pages, p.stride,
             (float)(scale ? *scale : 1.0 / std::sqrt((double)dk)), causal ? 0u : (unsigned)KDA_ATTN_FULL, code);
    return py::make_tuple(std::move(out), std::move(lse));
}

py::tuple latent_attn(const Tensor &q, const Tensor &cache, const Tensor &table, const Tensor &lens, int64_t dv,
                      const OptTensor &cu, const OptTensor &out, const OptTensor &lse, std::optional<double> scale, bool causal) {
    return attn_by(f_attn, q, cache, table, lens, dv, cu, out, lse, scale, causal);
}

py::tuple selftest_latent_attn(const Tensor &q, const Tensor &cache, const Tensor &table, const Tensor &lens, int64_t dv,
                               const OptTensor &cu, const OptTensor &out, const OptTensor &lse,
                               std::optional<double> scale, bool causal) {
    return attn_by(f_attn_selftest, q, cache, table, lens, dv, cu, out, lse, scale, causal);
}

void latent_append(const Tensor &kv, const Tensor &cache, const Tensor &table, const Tensor &lens, const OptTensor &q_pe,
                   const OptTensor &q, const OptTensor &freqs, const OptTensor &cu, bool interleaved, double scale) {
    const auto dev = device_of(kv, "kda_latent_append");
    if (kv.dim() != 2) bad_value("kv must be [T,dk]");
    const int64_t T = kv.size(0), dk = kv.size(1);
    const auto type = kv.scalar_type();
    const kda_dtype code = dtype_of(kv);
    if (T > 0 && (kv.stride(1) != 1 || (T > 1 && kv.stride(0) < dk))) bad_value("kv must have contiguous rows, one after the other");
    const Plan p = plan("kda_latent_append", T, cache, table, lens, cu, dev, type, dk);
    int64_t H = 1, rot = 0, ts = 0, hs = 0;
    const float *fp = nullptr;
    const void *pp = nullptr;
    void *qp = nullptr;
    if (freqs) {
        fp = (const float *)on(*freqs, "freqs", dev, at::kFloat);
        rot = 2 * freqs->numel();
    }
    if (q_pe.has_value() != q.has_value()) bad_value("q_pe and q come together");
    if (q_pe) {
        if (q_pe->dim() != 3 || q_pe->size(0) != T || !q_pe->is_cuda() || q_pe->device().index() != dev || q_pe->scalar_type() != type)
            bad_value("q_pe must be [" + std::to_string(T) + ",H,rot], of kv's type and device");
        H = q_pe->size(1);
        if (freqs && q_pe->size(2) != rot) bad_value("q_pe must have " + std::to_string(rot) + " channels, twice as many as freqs");
        rot = q_pe->size(2);
        if (T > 0 && H > 0 && q_pe->stride(2) != 1) bad_value("the heads of q_pe must be contiguous");
        if ((T > 1 && q_pe->stride(0) == 0) || (H > 1 && q_pe->stride(1) == 0)) bad_value("q_pe must not be broadcast");
        if (T > 1) ts = q_pe->stride(0);
        if (H > 1) hs = q_pe->stride(1);
        pp = q_pe->data_ptr();
        qp = on(*q, "q", dev, type);
        if (q->dim() != 3 || q->size(0) != T || q->size(1) != H || q->size(2) != dk)
            bad_value("q must be [" + std::to_string(T) + "," + std::to_string(H) + "," + std::to_string(dk) + "]");
    }
    if (T == 0) return;
    call(f_append, dev, (const void *)kv.data_ptr(), cache.data_ptr(), p.table, p.lens, p.cu, pp, qp, fp, to_int(T, "T"),
         to_int(H, "H"), to_int(dk, "dk"), to_int(rot, "rot"), p.N, p.pages, p.page_size, p.max_pages, p.stride,
         (long long)(T > 1 ? kv.stride(0) : 0), (long long)ts, (long long)hs, interleaved ? (unsigned)KDA_ROPE_INTERLEAVED : 0u,
         (float)scale, code);
}

Tensor rope(const Tensor &x, const Tensor &positions, const Tensor &freqs, const OptTensor &out_, int64_t offset, bool interleaved,
            bool inverse, double scale) {
    const auto dev = device_of(x, "kda_rope");
    if (x.dim() != 3) bad_value("x must be [T,H,d]");
    const int64_t T = x.size(0), H = x.size(1), d = x.size(2);
    const kda_dtype code = dtype_of(x);
    auto stride = [&](const Tensor &t, const char *name) -> long long {
        if (t.numel() && (t.stride(2) != 1 || (H > 1 && t.stride(1) != d))) bad_value(std::string("the heads of ") + name + " must be contiguous");
        if (T <= 1) return H * d;
        if (t.stride(0) == 0) bad_value(std::string(name) + " must not be broadcast");
        return t.stride(0);
    };
    const long long xs = stride(x, "x");
    const auto *pp = (const int32_t *)on(positions, "positions", dev, at::kInt);
    const auto *fp = (const float *)on(freqs, "freqs", dev, at::kFloat);
    if (positions.dim() != 1 || positions.size(0) != T || freqs.dim() != 1)
        bad_value("positions must be [" + std::to_string(T) + "] and freqs [rot / 2]");
    if (out_ && (out_->sizes() != x.sizes() || !out_->is_cuda() || out_->device().index() != dev || out_->scalar_type() != x.scalar_type()))
        bad_value("out must have x's shape, type and device");
    Tensor out = out_ ? *out_ : at::empty({T, H, d}, x.options());
    if (T > 0)
        call(f_rope, dev, (const void *)x.data_ptr(), pp, fp, out.data_ptr(), (long long)T, to_int(H, "H"), to_int(d, "d"),
             to_int(2 * freqs.numel(), "rot"), to_int(offset, "offset"), xs, stride(out, "out"),
             (interleaved ? (unsigned)KDA_ROPE_INTERLEAVED : 0u) | (inverse ? (unsigned)KDA_ROPE_INVERSE : 0u), (float)scale, code);
    return out;
}

struct Pool {
    c10::DeviceIndex dev;
    int planes, pages;
    long long bytes;
};

// A contiguous pool [pages, ...] or [planes, pages, ...].
Pool pool_of(const std::string &who, const Tensor &t, bool planes) {
    Pool p;
    p.dev = device_of(t, who.c_str());
    if (t.dim() < (planes ? 3 : 2) || t.numel() == 0 || !t.is_contiguous())
        bad_value(who + ": the pool must be a contiguous, non-empty [" + (planes ? "planes, " : "") + "pages, ...]");
    p.planes = planes ? to_int(t.size(0), "planes") : 1;
    p.pages = to_int(t.size(planes ? 1 : 0), "pages");
    p.bytes = t.numel() / ((int64_t)p.planes * p.pages) * (int64_t)t.element_size();
    return p;
}

void pages_copy(const Tensor &pool, const Tensor &src, const Tensor &dst, bool planes) {
    const Pool p = pool_of("kda_pages_copy", pool, planes);
    const auto *s = (const int32_t *)on(src, "src", p.dev, at::kInt), *d = (const int32_t *)on(dst, "dst", p.dev, at::kInt);
    if (src.dim() != 1 || dst.dim() != 1 || src.numel() != dst.numel()) bad_value("src and dst must be [n]");
    call(f_copy, p.dev, pool.data_ptr(), s, d, to_int(src.numel(), "n"), p.planes, p.pages, p.bytes);
}

Tensor pages_compact(const Tensor &pool, const Tensor &pages, bool planes, const OptTensor &out_) {
    const Pool p = pool_of("kda_pages_compact", pool, planes);
    const auto *list = (const int32_t *)on(pages, "pages", p.dev, at::kInt);
    if (out_ && out_->sizes() != pages.sizes()) bad_value("out must have the shape of pages");
    Tensor out = out_ ? *out_ : at::empty(pages.sizes(), pages.options());
    auto *names = (int32_t *)on(out, "out", p.dev, at::kInt);
    call(f_compact, p.dev, pool.data_ptr(), list, names, (long long)pages.numel(), p.planes, p.pages, p.bytes);
    return out;
}

}  // namespace

// the torch and Python that this was compiled against (build.py looks for it in the module's bytes)
extern const char built_for[];
const char built_for[] = "\0" KDA_BUILT_FOR;

PYBIND11_MODULE(_paged, m) {
    m.attr("built_for") = built_for + 1;
    m.def("init", &init);
    m.def("latent_attn", &latent_attn);
    m.def("selftest_latent_attn", &selftest_latent_attn);
    m.def("latent_append", &latent_append);
    m.def("rope", &rope);
    m.def("pages_copy", &pages_copy);
    m.def("pages_compact", &pages_compact);
}
