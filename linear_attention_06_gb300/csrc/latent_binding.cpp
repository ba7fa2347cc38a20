// latent_binding.cpp -- the Python side of the kda_latent_* entry points: tensors checked and turned into the
// pointers, sizes, strides and stream that kda.h declares.  Written in C++ because a decode step's calls are short:
// the same checks in Python took 18 us a call, on top of 3 to 6 us for the entry point itself.
//
// The entry points are called through addresses that the package hands over (bind), so the module works on whichever
// build of the library the package has loaded.
#include <ATen/ATen.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/utils/pybind.h>

#include <algorithm>
#include <optional>
#include <sstream>
#include <string>

#include "kda.h"

namespace py = pybind11;

namespace {

constexpr int64_t kLatent = 512, kRope = 64, kHead = 128;
using Opt = std::optional<at::Tensor>;

struct Entry {
    decltype(&kda_latent_append) append = nullptr;
    decltype(&kda_latent_gather) gather = nullptr;
    decltype(&kda_latent_decode) decode = nullptr;
    decltype(&kda_latent_decode_workspace_size) workspace_size = nullptr;
    decltype(&kda_latent_prefill) prefill = nullptr;
} entry;
PyObject* check_status = nullptr;             // check_status(name, status) raises; lives as long as the process

template <typename... T>
std::string text(const T&... x) {
    std::ostringstream s;
    (s << ... << x);
    return s.str();
}

// A tensor argument: its type, shape and device; contiguous unless the call takes its strides.
void* expect(const char* name, const at::Tensor& t, at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex device,
             bool strides = false) {
    if (t.scalar_type() != type) throw py::type_error(text(name, " must be ", type, ", not ", t.scalar_type()));
    if (t.sizes() != shape) throw py::value_error(text(name, " must have shape ", shape, ", not ", t.sizes()));
    if (!t.is_cuda() || t.get_device() != device)
        throw py::value_error(text(name, " must be on cuda:", (int)device, ", not on ", t.device()));
    if (!strides && !t.is_contiguous()) throw py::value_error(text(name, " must be contiguous"));
    return t.data_ptr();
}
void* expect(const char* name, const Opt& t, at::IntArrayRef shape, at::ScalarType type, c10::DeviceIndex device,
             bool strides = false) {
    if (!t) throw py::value_error(text(name, " is needed"));
    return expect(name, *t, shape, type, device, strides);
}

// An argument that the call's shape has no place for: it is refused, not dropped.
void expect_none(const char* name, const Opt& t, const char* why) {
    if (t) throw py::value_error(text(name, " must be None: ", why));
}
constexpr char kNoRope[] = "the cache's rows have no rotated part";

c10::DeviceIndex index_of(const at::Tensor& t) {
    if (!t.is_cuda()) throw py::value_error("tensor arguments must be CUDA tensors");
    return (c10::DeviceIndex)t.get_device();
}

// Elements between consecutive rows of t [..., channels], all its leading axes one run of rows.
int64_t row_stride(const std::string& name, const at::Tensor& t) {
    const int64_t dims = t.dim(), width = t.size(dims - 1);
    if (t.is_contiguous()) return std::max<int64_t>(width, 8);
    if (width > 1 && t.stride(dims - 1) != 1) throw py::value_error(name + ": channels must be contiguous");
    int64_t rows = 1, step = -1;
    for (int64_t d = dims - 2; d >= 0; --d) {
        if (t.size(d) <= 1) continue;
        if (step < 0) {
            step = t.stride(d);
            if (step < width) throw py::value_error(name + ": rows must not overlap");
        } else if (t.stride(d) != step * rows) {
            throw py::value_error(name + ": rows must be evenly spaced");
        }
        rows *= t.size(d);
    }
    return step < 0 ? std::max<int64_t>(width, 8) : step;
}

void check(const char* fn, kda_status st) {
    if (st == KDA_OK) return;
    py::reinterpret_borrow<py::object>(check_status)(fn, (int)st);
    throw py::value_error(text(fn, " failed"));          // not reached: check_status raises
}

kda_stream_t stream_of(c10::DeviceIndex device) {
    return reinterpret_cast<kda_stream_t>(c10::cuda::getCurrentCUDAStream(device).stream());
}

at::Tensor make(at::IntArrayRef shape, at::ScalarType type, const at::Tensor& like) {
    return at::empty(shape, at::TensorOptions().dtype(type).device(like.device()));
}

// The descriptor of a call on a cache and its table, with their addresses.
kda_latent_shape latent_shape(const at::Tensor& cache, const at::Tensor& table, int64_t tokens, int64_t heads,
                              c10::DeviceIndex device) {
    if (cache.dim() != 3 || (cache.size(2) != kLatent && cache.size(2) != kLatent + kRope))
        throw py::value_error(text("cache must be [pages, page_size, ", kLatent, " or ", kLatent + kRope, "], not ", cache.sizes()));
    if (table.dim() != 2) throw py::value_error("block_table must be [N, max_pages]");
    expect("cache", cache, cache.sizes(), at::kBFloat16, device);
    expect("block_table", table, table.sizes(), at::kInt, device);
    const auto most = (int64_t)INT32_MAX;
    if (cache.size(0) > most || cache.size(1) > most || table.size(0) > most || table.size(1) > most || heads > most)
        throw py::value_error("a cache or block_table axis exceeds 2^31 - 1");
    return {(int32_t)table.size(0), tokens, (int32_t)heads, (int32_t)kLatent, (int32_t)(cache.size(2) - kLatent),
            (int32_t)cache.size(1), (int32_t)cache.size(0), (int32_t)table.size(1), KDA_BF16};
}

std::optional<at::Tensor> append(const at::Tensor& latent, const Opt& k_rope, const at::Tensor& cache, const at::Tensor& table,
                                 const at::Tensor& lens, const Opt& inv_freq, bool interleaved, const Opt& q_rope, Opt q_out,
                                 const Opt& cu) {
    const auto dev = index_of(cache);
    const c10::cuda::CUDAGuard guard(dev);
    if (latent.dim() != 2) throw py::value_error("latent must be [T, 512]");
    if (q_rope && q_rope->dim() != 3) throw py::value_error("q_rope must be [T, H, 64]");
    const int64_t T = latent.size(0), H = q_rope ? q_rope->size(1) : 1;
    const kda_latent_shape shape = latent_shape(cache, table, T, H, dev);
    const int64_t n = shape.num_seqs;
    const void* p_latent = expect("latent", latent, {T, kLatent}, at::kBFloat16, dev, true);
    const int64_t latent_step = row_stride("latent", latent);
    const void* p_rope = shape.rope_dim ? expect("k_rope", k_rope, {T, kRope}, at::kBFloat16, dev, true) : nullptr;
    const int64_t rope_step = shape.rope_dim ? row_stride("k_rope", *k_rope) : 0;
    if (!shape.rope_dim) expect_none("k_rope", k_rope, kNoRope);
    if (!q_rope) expect_none("q_rope_out", q_out, "there is no q_rope");
    const void* p_lens = expect("seq_lens", lens, {n}, at::kInt, dev);
    const void* p_freq = inv_freq ? expect("inv_freq", *inv_freq, {kRope / 2}, at::kFloat, dev) : nullptr;
    const void* p_cu = cu ? expect("cu_seqlens", *cu, {n + 1}, at::kInt, dev) : nullptr;
    const void* p_q = nullptr;
    void* p_out = nullptr;
    int64_t q_step = 0, out_step = 0;
    if (q_rope) {
        p_q = expect("q_rope", *q_rope, {T, H, kRope}, at::kBFloat16, dev, true);
        q_step = row_stride("q_rope", *q_rope);
        if (!q_out) q_out = make({T, H, kRope}, at::kBFloat16, cache);
        p_out = expect("q_rope_out", *q_out, {T, H, kRope}, at::kBFloat16, dev, true);
        out_step = row_stride("q_rope_out", *q_out);
    }
    kda_status st;
    {
        py::gil_scoped_release free;
        st = entry.append(&shape, p_latent, latent_step, p_rope, rope_step, static_cast<const float*>(p_freq), interleaved,
                          p_q, q_step, p_out, out_step, static_cast<const int32_t*>(p_cu), static_cast<const int32_t*>(p_lens),
                          static_cast<const int32_t*>(table.data_ptr()), cache.data_ptr(), stream_of(dev));
    }
    check("kda_latent_append", st);
    return q_rope ? q_out : std::nullopt;
}

std::pair<at::Tensor, std::optional<at::Tensor>> gather(const at::Tensor& cache, const at::Tensor& table, const at::Tensor& cu,
                                                        int64_t T, const Opt& starts, Opt latent, Opt k_rope) {
    const auto dev = index_of(cache);
    const c10::cuda::CUDAGuard guard(dev);
    if (T < 0) throw py::value_error("total_tokens must not be negative");
    const kda_latent_shape shape = latent_shape(cache, table, T, 1, dev);
    const int64_t n = shape.num_seqs;
    const void* p_cu = expect("cu_seqlens", cu, {n + 1}, at::kInt, dev);
    const void* p_starts = starts ? expect("starts", *starts, {n}, at::kInt, dev) : nullptr;
    if (!shape.rope_dim) expect_none("k_rope", k_rope, kNoRope);
    if (!latent) {
        expect_none("k_rope", k_rope, "out names no latent to go with it");
        latent = make({T, kLatent}, at::kBFloat16, cache);
        if (shape.rope_dim) k_rope = make({T, kRope}, at::kBFloat16, cache);
    }
    void* p_latent = expect("latent", *latent, {T, kLatent}, at::kBFloat16, dev);
    void* p_rope = shape.rope_dim ? expect("k_rope", k_rope, {T, kRope}, at::kBFloat16, dev) : nullptr;
    kda_status st;
    {
        py::gil_scoped_release free;
        st = entry.gather(&shape, cache.data_ptr(), static_cast<const int32_t*>(table.data_ptr()),
                          static_cast<const int32_t*>(p_cu), static_cast<const int32_t*>(p_starts), p_latent, p_rope,
                          stream_of(dev));
    }
    check("kda_latent_gather", st);
    return {*latent, shape.rope_dim ? k_rope : std::nullopt};
}

std::pair<at::Tensor, std::optional<at::Tensor>> decode(const at::Tensor& q, const Opt& q_rope, const at::Tensor& cache,
                                                        const at::Tensor& table, const at::Tensor& lens, double scale, Opt out,
                                                        Opt lse, bool make_lse, Opt workspace) {
    const auto dev = index_of(cache);
    const c10::cuda::CUDAGuard guard(dev);
    if (q.dim() != 3) throw py::value_error("q_latent must be [N * T, H, 512]");
    const int64_t rows = q.size(0), H = q.size(1);
    const kda_latent_shape shape = latent_shape(cache, table, rows, H, dev);
    const void* p_q = expect("q_latent", q, {rows, H, kLatent}, at::kBFloat16, dev);
    const void* p_r = shape.rope_dim ? expect("q_rope", q_rope, {rows, H, kRope}, at::kBFloat16, dev) : nullptr;
    if (!shape.rope_dim) expect_none("q_rope", q_rope, kNoRope);
    const void* p_lens = expect("seq_lens", lens, {shape.num_seqs}, at::kInt, dev);
    if (!out) out = make({rows, H, kLatent}, at::kBFloat16, cache);
    if (make_lse) lse = make({rows, H}, at::kFloat, cache);
    void* p_out = expect("out", *out, {rows, H, kLatent}, at::kBFloat16, dev);
    void* p_lse = lse ? expect("lse", *lse, {rows, H}, at::kFloat, dev) : nullptr;
    if (!workspace) {
        size_t need = 0;
        check("kda_latent_decode", entry.workspace_size(&shape, &need));
        workspace = make({std::max<int64_t>((int64_t)need, 1)}, at::kByte, cache);
    }
    void* p_ws = expect("workspace", *workspace, workspace->sizes(), at::kByte, dev);
    kda_status st;
    {
        py::gil_scoped_release free;
        st = entry.decode(&shape, p_q, p_r, cache.data_ptr(), static_cast<const int32_t*>(table.data_ptr()),
                          static_cast<const int32_t*>(p_lens), (float)scale, p_out, static_cast<float*>(p_lse), p_ws,
                          (size_t)workspace->numel(), stream_of(dev));
    }
    check("kda_latent_decode", st);
    return {*out, lse};
}

std::pair<at::Tensor, std::optional<at::Tensor>> prefill(const at::Tensor& q, const at::Tensor& k, const at::Tensor& v,
                                                         const Opt& k_rope, double scale, const Opt& cu, const Opt& cu_k,
                                                         std::optional<int64_t> num_seqs, Opt out, Opt lse, bool make_lse) {
    const auto dev = index_of(q);
    const c10::cuda::CUDAGuard guard(dev);
    if (q.dim() != 3 || (q.size(2) != kHead && q.size(2) != kHead + kRope))
        throw py::value_error(text("q must be [T, H, ", kHead, " or ", kHead + kRope, "], not ", q.sizes()));
    if (k.dim() != 3) throw py::value_error("k must be [S, H, 128]");
    const int64_t T = q.size(0), H = q.size(1), dk = q.size(2), S = k.size(0);
    const void* p_q = expect("q", q, {T, H, dk}, at::kBFloat16, dev);
    const void* p_k = expect("k", k, {S, H, kHead}, at::kBFloat16, dev, true);
    const void* p_v = expect("v", v, {S, H, kHead}, at::kBFloat16, dev, true);
    const void* p_r = dk > kHead ? expect("k_rope", k_rope, {S, dk - kHead}, at::kBFloat16, dev) : nullptr;
    if (dk == kHead) expect_none("k_rope", k_rope, "q has no rotated part");
    const int64_t step = row_stride("k", k);
    if (S * H > 1 && step != row_stride("v", v)) throw py::value_error("k and v must have the same row stride");
    int64_t n = num_seqs.value_or(1);
    if (cu) {
        if (cu->dim() != 1 || cu->numel() < 1) throw py::value_error("cu_seqlens must hold N + 1 offsets");
        n = cu->numel() - 1;
    } else if (cu_k) {
        if (cu_k->dim() != 1 || cu_k->numel() < 1) throw py::value_error("cu_seqlens_k must hold N + 1 offsets");
        n = cu_k->numel() - 1;
    }
    if (num_seqs && *num_seqs != n) throw py::value_error(text("num_seqs is ", *num_seqs, ", but the offsets are those of ", n));
    if (n < 0 || n > INT32_MAX || H > INT32_MAX) throw py::value_error("too many sequences or heads");
    const void* p_cu = cu ? expect("cu_seqlens", *cu, {n + 1}, at::kInt, dev) : nullptr;
    // the queries' table serves the keys where there are as many
    const void* p_cu_k = cu_k ? expect("cu_seqlens_k", *cu_k, {n + 1}, at::kInt, dev) : (cu && S == T ? p_cu : nullptr);
    if (!out) out = make({T, H, kHead}, at::kBFloat16, q);
    if (make_lse) lse = make({T, H}, at::kFloat, q);
    void* p_out = expect("out", *out, {T, H, kHead}, at::kBFloat16, dev);
    void* p_lse = lse ? expect("lse", *lse, {T, H}, at::kFloat, dev) : nullptr;
    const kda_shape shape{(int32_t)n, T, (int32_t)H, (int32_t)dk, (int32_t)kHead, KDA_BF16};
    kda_status st;
    {
        py::gil_scoped_release free;
        st = entry.prefill(&shape, S, p_q, p_k, p_v, step, p_r, (float)scale, static_cast<const int32_t*>(p_cu),
                           static_cast<const int32_t*>(p_cu_k), p_out, static_cast<float*>(p_lse), stream_of(dev));
    }
    check("kda_latent_prefill", st);
    return {*out, lse};
}

void bind(py::dict addresses, py::function raise) {
    auto at = [&](const char* name) { return reinterpret_cast<void*>(addresses[name].cast<uintptr_t>()); };
    entry.append = reinterpret_cast<decltype(entry.append)>(at("kda_latent_append"));
    entry.gather = reinterpret_cast<decltype(entry.gather)>(at("kda_latent_gather"));
    entry.decode = reinterpret_cast<decltype(entry.decode)>(at("kda_latent_decode"));
    entry.workspace_size = reinterpret_cast<decltype(entry.workspace_size)>(at("kda_latent_decode_workspace_size"));
    entry.prefill = reinterpret_cast<decltype(entry.prefill)>(at("kda_latent_prefill"));
    check_status = raise.release().ptr();
}

}  // namespace

PYBIND11_MODULE(_latent, m) {
    m.def("bind", &bind);
    m.def("row_stride", &row_stride);
    m.def("append", &append);
    m.def("gather", &gather);
    m.def("decode", &decode);
    m.def("prefill", &prefill);
}
