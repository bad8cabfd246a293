// tkv_torch.cpp -- libtkv's calls on torch tensors, for tkv.py.
//
// A step of decoding makes a few calls of some microseconds each on the GPU, so
// what Python spends on a call's arguments is in the way.  Host time of a call,
// its launches included: append 4.0 us, attend 5.2 (3.9 where its outputs are
// given), read 6.2, evict 10; with the checks in Python and the call through
// ctypes append was 7.6, attend 11.5 and read 10.8.  A call that launches nothing
// takes 0.6 (append) to 1.7 us (attend).
// A wrong argument is a ValueError; what libtkv refuses comes back as its status.
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/utils/pybind.h>

#include <ATen/core/grad_mode.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPGuard.h>
#include <c10/hip/HIPStream.h>

#include <cmath>

#include "../../include/tkv.h"

namespace py = pybind11;
using at::Tensor;
using Maybe = std::optional<Tensor>;

namespace {

#define TKV_CHECK(cond, ...) TORCH_CHECK_VALUE(cond, __VA_ARGS__)

// What a call needs to know of a cache.
struct Cache {
    tkv_cache described;
    Tensor pool;
    int64_t heads, dim, page_tokens;

    Cache(int64_t at, Tensor pool_, int64_t heads_, int64_t dim_, int64_t page_tokens_)
        : described(*reinterpret_cast<const tkv_cache *>(at)), pool(std::move(pool_)), heads(heads_), dim(dim_),
          page_tokens(page_tokens_) {}
};

const char *name_of(at::ScalarType t) {
    switch (t) {
        case at::kHalf: return "float16";
        case at::kBFloat16: return "bfloat16";
        case at::kFloat: return "float32";
        case at::kInt: return "int32";
        case at::kByte: return "uint8";
        default: return c10::toString(t);
    }
}

void on_gpu(const Tensor &t, const char *what, const Cache &c) {
    // nothing here has a backward pass: a gradient that is asked for would be lost without a word
    TKV_CHECK(!(t.requires_grad() && at::GradMode::is_enabled()), what,
              " requires a gradient, and these operators give none: call them under torch.no_grad()");
    TKV_CHECK(t.is_cuda(), what, " must be a GPU tensor");
    TKV_CHECK(t.device() == c.pool.device(), what, " is on ", t.device(), ", the cache on ", c.pool.device());
}

void typed(const Tensor &t, const char *what, at::ScalarType type, const Cache &c) {
    TKV_CHECK(t.scalar_type() == type, what, " must be ", name_of(type), ", not ", name_of(t.scalar_type()));
    on_gpu(t, what, c);
}

tkv_tokens tokens(const Tensor &t, const char *what, int64_t heads, int64_t n_tokens, bool fp32_too, const Cache &c) {
    TKV_CHECK(t.dim() == 3, what, " must be a tensor [tokens, heads, head_dim]");
    int32_t type = 0;
    switch (t.scalar_type()) {
        case at::kHalf: type = TMAP_F16; break;
        case at::kBFloat16: type = TMAP_BF16; break;
        case at::kFloat: type = fp32_too ? TMAP_F32 : 0; break;
        default: break;
    }
    TKV_CHECK(type, what, " must be one of float16, bfloat16", fp32_too ? ", float32" : "");
    on_gpu(t, what, c);
    TKV_CHECK(t.size(2) == c.dim && (heads < 0 || t.size(1) == heads), what, " is ", t.sizes(), ", the cache has ",
              heads < 0 ? std::string("n") : std::to_string(heads), " heads of ", c.dim);
    TKV_CHECK(n_tokens < 0 || t.size(0) == n_tokens, what, " has ", t.size(0), " tokens, not ", n_tokens);
    TKV_CHECK(t.stride(2) == 1 || t.numel() == 0, what, "'s last dimension must be contiguous");
    return {t.data_ptr(), t.stride(0), t.stride(1), type};
}

// A tensor that a call writes: its rows are apart.
void apart(const tkv_tokens &t, const char *what, const Tensor &x) {
    const int64_t n = x.size(0), heads = x.size(1), dim = x.size(2), ts = t.token_stride, hs = t.head_stride;
    TKV_CHECK((n < 2 || ts >= (heads - 1) * hs + dim || heads < 2 || hs >= (n - 1) * ts + dim) &&
                  (n < 2 || ts >= dim) && (heads < 2 || hs >= dim), what, "'s rows overlap: strides ", x.strides(), " of ",
              x.sizes());
}

struct Table {
    const int32_t *data;
    int64_t stride;
    int32_t width;
};

Table table_of(const Tensor &t, const char *what, int64_t n_seq, const Cache &c) {
    typed(t, what, at::kInt, c);
    TKV_CHECK(t.dim() == 2 && t.size(0) == n_seq, what, " must be [", n_seq, ", pages]");
    TKV_CHECK(t.size(1) < 2 || t.stride(1) == 1 || t.numel() == 0, what, "'s rows must be contiguous");
    TKV_CHECK(n_seq < 2 || t.stride(0) >= t.size(1), what, "'s rows must not overlap");
    TKV_CHECK(t.size(1) <= INT32_MAX, what, " is too wide");
    return {t.data_ptr<int32_t>(), n_seq < 2 ? t.size(1) : t.stride(0), (int32_t)t.size(1)};
}

void on_current_device(const Cache &c) {
    const auto current = c10::hip::current_device();
    TKV_CHECK(current == c.pool.get_device(), "the cache is on ", c.pool.device(), ", the current device is ",
              (int)current);
}

struct Batch {
    tkv_batch b;
    int64_t held;  // positions that a row of the table holds
};

Batch batch(const Cache &c, const Tensor &table, const Tensor &lens, const Maybe &starts, int64_t n_tokens,
            std::optional<int64_t> max_new) {
    on_current_device(c);
    typed(lens, "lens", at::kInt, c);
    TKV_CHECK(lens.dim() == 1 && (lens.size(0) < 2 || lens.stride(0) == 1), "lens must be a contiguous vector");
    const int64_t n_seq = lens.size(0);
    TKV_CHECK(n_seq <= INT32_MAX, "too many sequences");
    const Table t = table_of(table, "table", n_seq, c);
    const int32_t *first = nullptr;
    if (starts) {
        typed(*starts, "starts", at::kInt, c);
        TKV_CHECK(starts->dim() == 1 && starts->size(0) == n_seq + 1 && (n_seq == 0 || starts->stride(0) == 1),
                  "starts must be a contiguous vector of sequences + 1");
        first = starts->data_ptr<int32_t>();
    } else {
        TKV_CHECK(n_seq == 0 || n_tokens % n_seq == 0, "without starts, ", n_tokens, " tokens must be a multiple of ",
                  n_seq, " sequences");
    }
    const int64_t most = max_new ? *max_new : starts ? n_tokens : n_seq ? n_tokens / n_seq : 0;
    TKV_CHECK(most <= INT32_MAX, "max_new: a number is out of range");
    return {{t.data, t.stride, lens.data_ptr<int32_t>(), first, n_tokens, (int32_t)n_seq, t.width,
             (int32_t)std::max<int64_t>(most, -1)},
            t.width * c.page_tokens};
}

// The stream of a call's work: the given one, or torch's current.  A given one is
// torch's current one for as long as this lives, so that what the call makes is
// memory of that stream: another stream's may still be in use there by work
// that was queued before the memory was given back.
struct Stream {
    std::optional<c10::hip::HIPStreamGuard> guard;
    Stream(const Cache &c, std::optional<int64_t> given) {
        if (given) {
            on_current_device(c);
            guard.emplace(c10::hip::getStreamFromExternal((hipStream_t)*given, c.pool.device().index()));
        }
    }
    void *handle() const { return (void *)c10::hip::getCurrentHIPStream().stream(); }
};

Tensor made(at::IntArrayRef size, at::ScalarType type, const Cache &c) {
    return at::empty(size, at::TensorOptions().dtype(type).device(c.pool.device()));
}

int do_append(const Cache &c, const Tensor &k, const Tensor &v, const Tensor &table, const Tensor &lens, const Maybe &starts,
           std::optional<int64_t> max_new, std::optional<int64_t> stream) {
    const tkv_tokens kt = tokens(k, "k", c.heads, -1, false, c);
    const int64_t n = k.size(0);
    const tkv_tokens vt = tokens(v, "v", c.heads, n, false, c);
    const Batch b = batch(c, table, lens, starts, n, max_new);
    const Stream on(c, stream);
    return tkv_append(&c.described, &kt, &vt, &b.b, on.handle());
}

py::tuple do_append_rotated(const Cache &c, const Tensor &k, const Tensor &v, const Tensor &table, const Tensor &lens,
                            const Maybe &starts, std::optional<int64_t> max_new, const Tensor &cos_sin,
                            const Maybe &positions, bool neighbours, const Maybe &q, const Maybe &q_out_,
                            std::optional<int64_t> stream) {
    const tkv_tokens kt = tokens(k, "k", c.heads, -1, false, c);
    const int64_t n = k.size(0);
    const tkv_tokens vt = tokens(v, "v", c.heads, n, false, c);
    const Batch b = batch(c, table, lens, starts, n, max_new);
    const Stream on(c, stream);
    tkv_rotation r{};
    typed(cos_sin, "cos_sin", at::kFloat, c);
    TKV_CHECK(cos_sin.dim() == 2, "cos_sin must be a tensor [positions, channels]");
    TKV_CHECK(cos_sin.stride(1) == 1 || cos_sin.numel() == 0, "cos_sin's rows must be contiguous");
    TKV_CHECK(cos_sin.size(1) <= c.dim, "cos_sin turns ", cos_sin.size(1), " channels, the cache has ", c.dim);
    r.cos_sin = cos_sin.data_ptr<float>();
    r.n_positions = cos_sin.size(0);
    r.rot_dim = (int32_t)cos_sin.size(1);
    r.stride = r.n_positions < 2 ? r.rot_dim : cos_sin.stride(0);
    r.neighbours = neighbours;
    if (positions) {
        typed(*positions, "positions", at::kInt, c);
        TKV_CHECK(positions->dim() == 1 && positions->size(0) == n && (n < 2 || positions->stride(0) == 1),
                  "positions must be a contiguous vector of the ", n, " tokens");
        r.positions = positions->data_ptr<int32_t>();
    }
    TKV_CHECK(q || !q_out_, "q_out is only written where q is given");
    Tensor q_out;
    if (q) {
        r.q = tokens(*q, "q", -1, n, false, c);
        TKV_CHECK(q->size(1) > 0 && q->size(1) <= INT32_MAX, "q has no heads, or too many");
        r.q_heads = (int32_t)q->size(1);
        q_out = q_out_ ? *q_out_ : made({n, q->size(1), c.dim}, q->scalar_type(), c);
        r.q_out = tokens(q_out, "q_out", q->size(1), n, false, c);
        apart(r.q_out, "q_out", q_out);
        TKV_CHECK(q_out.scalar_type() == q->scalar_type(), "q_out must be ", name_of(q->scalar_type()));
    }
    const int st = tkv_append_rotated(&c.described, &kt, &vt, &r, &b.b, on.handle());
    return py::make_tuple(st, q ? py::cast(q_out) : py::none());
}

py::tuple do_read(const Cache &c, const Tensor &table, const Tensor &lens, const Maybe &starts,
               std::optional<int64_t> max_new, std::optional<int64_t> n_tokens, at::ScalarType dtype, const Maybe &k_,
               const Maybe &v_, std::optional<int64_t> stream) {
    TKV_CHECK(k_.has_value() == v_.has_value(), "give both k and v, or neither");
    const Stream on(c, stream);
    Tensor k, v;
    if (k_) {
        k = *k_, v = *v_;
    } else {
        TKV_CHECK(n_tokens, "n_tokens is needed where k and v are not given");
        TKV_CHECK(*n_tokens >= 0, "n_tokens is negative");
        k = made({*n_tokens, c.heads, c.dim}, dtype, c);
        v = made({*n_tokens, c.heads, c.dim}, dtype, c);
    }
    const tkv_tokens kt = tokens(k, "k", c.heads, n_tokens.value_or(-1), true, c);
    const tkv_tokens vt = tokens(v, "v", c.heads, k.size(0), true, c);
    apart(kt, "k", k);
    apart(vt, "v", v);
    const Batch b = batch(c, table, lens, starts, k.size(0), max_new);
    const int st = tkv_read(&c.described, &kt, &vt, &b.b, on.handle());
    return py::make_tuple(st, k, v);
}

const float *scores_of(const Tensor &t, const char *what, const Cache &c, int64_t n_seq, int64_t max_len) {
    typed(t, what, at::kFloat, c);
    TKV_CHECK(t.dim() == 3 && t.size(0) == n_seq && t.size(1) == c.heads && t.size(2) >= max_len && t.is_contiguous(),
              what, " must be contiguous [", n_seq, ", ", c.heads, ", at least ", max_len, "], not ", t.sizes());
    return t.data_ptr<float>();
}

int64_t bound(std::optional<int64_t> max_len, int64_t held) {
    const int64_t n = max_len ? std::min(*max_len, held) : held;
    TKV_CHECK(n <= INT32_MAX, "max_len: a number is out of range");
    return std::max<int64_t>(n, -1);
}

py::tuple do_attend(const Cache &c, const Tensor &q, const Tensor &table, const Tensor &lens, const Maybe &starts,
                    std::optional<int64_t> max_new, std::optional<int64_t> max_len, std::optional<double> scale, bool causal,
                    const Maybe &scores, const Maybe &scores_out, const Maybe &out_, const Maybe &lse_, const Maybe &workspace,
                    std::optional<int64_t> stream, std::optional<int64_t> window, int64_t sinks) {
    const Stream on(c, stream);
    TKV_CHECK(window || sinks == 0, "sinks are only apart from the others where a window is given");
    tkv_window seen{};
    if (window) {
        TKV_CHECK(*window >= 1, "window is less than 1");
        TKV_CHECK(sinks >= 0, "sinks is negative");
        seen.window = (int32_t)std::min<int64_t>(*window, INT32_MAX);
        seen.sinks = (int32_t)std::min<int64_t>(sinks, INT32_MAX);
    }
    const tkv_window *const w = window ? &seen : nullptr;
    tkv_attend_args a{};
    a.q = tokens(q, "q", -1, -1, false, c);
    const int64_t n = q.size(0), heads = q.size(1);
    TKV_CHECK(heads <= INT32_MAX, "too many query heads");
    const Tensor out = out_ ? *out_ : made({n, heads, c.dim}, q.scalar_type(), c);
    const Tensor lse = lse_ ? *lse_ : made({n, heads}, at::kFloat, c);
    a.out = tokens(out, "out", heads, n, false, c);
    apart(a.out, "out", out);
    TKV_CHECK(out.scalar_type() == q.scalar_type(), "out must be ", name_of(q.scalar_type()));
    typed(lse, "lse", at::kFloat, c);
    TKV_CHECK(lse.dim() == 2 && lse.size(0) == n && lse.size(1) == heads && lse.is_contiguous(),
              "lse must be contiguous [", n, ", ", heads, "]");
    const Batch b = batch(c, table, lens, starts, n, max_new);
    a.lse = lse.data_ptr<float>();
    a.max_len = (int32_t)bound(max_len, b.held);
    if (scores_out) {
        a.scores_out = const_cast<float *>(scores_of(*scores_out, "scores_out", c, b.b.n_seq, a.max_len));
        a.score_stride = scores_out->size(2);
        if (scores) {
            a.scores_in = scores_of(*scores, "scores", c, b.b.n_seq, a.max_len);
            TKV_CHECK(scores->sizes() == scores_out->sizes(), "scores and scores_out must have one shape");
        }
    } else {
        TKV_CHECK(!scores, "scores are only read where scores_out is given");
    }
    a.q_heads = (int32_t)heads;
    a.scale = (float)(scale ? *scale : 1.0 / std::sqrt((double)c.dim));
    a.causal = causal;
    uint64_t need = 0;
    int st = tkv_attend_window_workspace(&c.described, &a, w, &b.b, &need);
    Tensor room;
    if (st == TMAP_SUCCESS && need) {
        if (workspace) {
            typed(*workspace, "workspace", at::kByte, c);
            TKV_CHECK(workspace->is_contiguous(), "workspace must be contiguous");
            room = *workspace;
        } else {
            room = made({(int64_t)need}, at::kByte, c);
        }
        a.workspace = room.data_ptr();
        a.workspace_bytes = (uint64_t)room.numel();
    }
    if (st == TMAP_SUCCESS) st = tkv_attend_window(&c.described, &a, w, &b.b, on.handle());
    return py::make_tuple(st, out, lse);
}

py::tuple do_evict(const Cache &c, const Tensor &table, const Tensor &lens, const Tensor &scores, int64_t budget,
                int64_t recent, const Tensor &dst_table, std::optional<int64_t> max_len, const Maybe &kept_,
                const Maybe &lens_out_, const Maybe &scores_out_, std::optional<int64_t> stream) {
    const Batch b = batch(c, table, lens, std::nullopt, 0, 0);
    const Stream on(c, stream);
    tkv_evict_args a{};
    a.max_len = (int32_t)bound(max_len, b.held);
    a.scores = scores_of(scores, "scores", c, b.b.n_seq, a.max_len);
    a.score_stride = scores.size(2);
    TKV_CHECK(budget >= 0 && recent >= 0, "budget and recent must not be negative");
    TKV_CHECK(budget <= INT32_MAX && recent <= INT32_MAX, "budget or recent: a number is out of range");
    const auto output = [&](const Maybe &t, const char *what, at::IntArrayRef size, at::ScalarType type) {
        if (!t) return made(size, type, c);
        typed(*t, what, type, c);
        TKV_CHECK(t->sizes() == size && t->is_contiguous(), what, " must be contiguous ", size);
        return *t;
    };
    const int64_t size[3] = {b.b.n_seq, c.heads, budget};
    const Tensor kept = output(kept_, "kept", size, at::kInt);
    const Tensor lens_out = output(lens_out_, "lens_out", {b.b.n_seq}, at::kInt);
    const Tensor scores_out = output(scores_out_, "scores_out", size, at::kFloat);
    const Table t = table_of(dst_table, "dst_table", b.b.n_seq, c);
    a.scores_out = scores_out.data_ptr<float>();
    a.kept = kept.data_ptr<int32_t>();
    a.lens_out = lens_out.data_ptr<int32_t>();
    a.dst_table = t.data;
    a.dst_stride = t.stride;
    a.dst_width = t.width;
    a.budget = (int32_t)budget;
    a.recent = (int32_t)recent;
    const int st = tkv_evict(&c.described, &a, &b.b, on.handle());
    return py::make_tuple(st, kept, lens_out, scores_out);
}

}  // namespace

PYBIND11_MODULE(_tkv, m) {
    py::class_<Cache>(m, "Cache").def(py::init<int64_t, Tensor, int64_t, int64_t, int64_t>());
    m.def("append", torch::wrap_pybind_function(do_append));
    m.def("append_rotated", torch::wrap_pybind_function(do_append_rotated));
    m.def("read", torch::wrap_pybind_function(do_read));
    using py::arg;
    m.def("attend", torch::wrap_pybind_function(do_attend), arg("cache"), arg("q"), arg("table"), arg("lens"), arg("starts"),
          arg("max_new"), arg("max_len"), arg("scale"), arg("causal"), arg("scores"), arg("scores_out"), arg("out"),
          arg("lse"), arg("workspace"), arg("stream"), arg("window") = py::none(), arg("sinks") = 0);
    m.def("evict", torch::wrap_pybind_function(do_evict));
}
