// binding.cpp -- Python entry points of the calls that a decode step makes many of: tensor checks and
// the C call in one native function.
//
// A call launches microseconds of work, and checking and unwrapping ten tensors in Python takes as
// long as the kernels (append of one token: 5.7 us of Python, 2.2 us of ctypes, of 10.9 us in all).
// Here the checks are a few loads each.  Refused arguments raise ValueError before anything is
// launched; the C function's return code goes back to the caller.
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include <algorithm>
#include <sstream>
#include <string>

#include "kvz.h"

namespace {

struct Refused {
    std::string why;
};

std::string shape_of(const at::Tensor &t)
{
    std::ostringstream s;
    s << '(';
    for (int64_t i = 0; i < t.dim(); ++i) s << (i ? ", " : "") << t.size(i);
    s << ')';
    return s.str();
}

const at::Tensor &tensor(PyObject *o, const char *name)
{
    if (!THPVariable_Check(o)) throw Refused{std::string(name) + ": expected a tensor"};
    return THPVariable_Unpack(o);
}

constexpr at::ScalarType kBf16 = at::kBFloat16, kI32 = at::kInt, kI64 = at::kLong, kU8 = at::kByte;

void on_device(const at::Tensor &t, const char *name, int dev)
{
    if (!t.is_cuda()) throw Refused{std::string(name) + ": expected a CUDA tensor"};
    if (t.get_device() != dev)
        throw Refused{std::string(name) + ": expected a tensor on CUDA device " + std::to_string(dev) + ", got device " +
                      std::to_string(t.get_device())};
}

void of_type(const at::Tensor &t, const char *name, at::ScalarType a, at::ScalarType b)
{
    if (t.scalar_type() != a && t.scalar_type() != b)
        throw Refused{std::string(name) + ": expected torch." + (a == kBf16 ? "bfloat16" : a == kI32 ? "int32" : a == kI64 ? "int64" : "uint8") +
                      ", got " + c10::toString(t.scalar_type())};
}

// The data of a contiguous tensor on the call's device.
void *data(const at::Tensor &t, const char *name, int dev, at::ScalarType a, at::ScalarType b)
{
    on_device(t, name, dev);
    of_type(t, name, a, b);
    if (!t.is_contiguous()) throw Refused{std::string(name) + ": expected a contiguous tensor"};
    return t.data_ptr();
}

template <class T>
T *data(PyObject *o, const char *name, int dev, at::ScalarType a, at::ScalarType b)
{
    return static_cast<T *>(data(tensor(o, name), name, dev, a, b));
}

template <class T>
T *data(PyObject *o, const char *name, int dev, at::ScalarType a)
{
    return data<T>(o, name, dev, a, a);
}

// The device of a call: its status tensor's, which has to be the current one.
int device_of(PyObject *status)
{
    const at::Tensor &t = tensor(status, "status");
    if (!t.is_cuda() || t.get_device() != c10::cuda::current_device())
        throw Refused{"status: expected a tensor on the current CUDA device"};
    return t.get_device();
}

kvz_stream_t stream_of(PyObject *o, int dev)
{
    if (o == Py_None) return reinterpret_cast<kvz_stream_t>(c10::cuda::getCurrentCUDAStream(dev).stream());
    const unsigned long long s = PyLong_AsUnsignedLongLong(o);
    if (PyErr_Occurred()) throw Refused{"stream: expected a torch.cuda.Stream"};
    return reinterpret_cast<kvz_stream_t>(s);
}

void dims_of(const at::Tensor &t, const char *name, std::initializer_list<int64_t> want, const char *text)
{
    bool ok = t.dim() == (int64_t)want.size();
    int64_t i = 0;
    for (int64_t w : want) {
        if (ok && w >= 0 && t.size(i) != w) ok = false;
        ++i;
    }
    if (!ok) throw Refused{std::string(name) + ": expected " + text + ", got " + shape_of(t)};
}

int32_t i32(int64_t x, const char *name)
{
    if (x > INT32_MAX) throw Refused{std::string(name) + ": too large"};
    return (int32_t)x;
}

// BF16 [tokens][heads][128] whose heads are contiguous.
struct Heads {
    int32_t heads = 0;
    const void *data = nullptr;
    int64_t token = 0, head = 0;  // strides
};

Heads heads_of(const at::Tensor &t, const char *name, int64_t tokens, int dev)
{
    dims_of(t, name, {tokens, -1, 128}, "[tokens][heads][128]");
    on_device(t, name, dev);
    of_type(t, name, kBf16, kBf16);
    if (t.stride(2) != 1) throw Refused{std::string(name) + ": expected contiguous heads"};
    // a stride nothing steps by may be any number
    return {i32(t.size(1), name), t.data_ptr(), tokens > 1 ? t.stride(0) : 0, t.size(1) > 1 ? t.stride(1) : 0};
}

// Runs f (which throws Refused) and turns its return code into a Python number.
template <class F>
PyObject *guarded(F &&f)
{
    try {
        return PyLong_FromLong(f());
    } catch (const Refused &r) {
        PyErr_SetString(PyExc_ValueError, r.why.c_str());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_ValueError, e.what());
    }
    return nullptr;
}

void count(Py_ssize_t n, Py_ssize_t want)
{
    if (n != want) throw Refused{"wrong number of arguments"};
}

// Norm weights [128] or [heads][128], BF16 or float32, or None.
struct Norm {
    const void *data = nullptr;
    int32_t type = KVZ_OUT_BF16;
    bool per_head = false;
};

Norm norm_of(PyObject *o, const char *name, int64_t heads, int dev)
{
    Norm n;
    if (o == Py_None) return n;
    const at::Tensor &t = tensor(o, name);
    if (t.scalar_type() != at::kFloat && t.scalar_type() != kBf16)
        throw Refused{std::string(name) + ": expected torch.float32 or torch.bfloat16, got " + c10::toString(t.scalar_type())};
    n.per_head = t.dim() == 2;
    if (n.per_head) dims_of(t, name, {heads, 128}, "[128] or [heads][128]");
    else dims_of(t, name, {128}, "[128] or [heads][128]");
    n.type = t.scalar_type() == at::kFloat ? KVZ_OUT_F32 : KVZ_OUT_BF16;
    n.data = data(t, name, dev, t.scalar_type(), t.scalar_type());
    return n;
}

// k, v, slots, raw_pool, status, q, q_out, rope, positions, interleaved, rope_scale, stream, q_norm, k_norm, norm_eps
PyObject *append_tokens(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&] {
        count(n, 15);
        const int dev = device_of(a[4]);
        const bool kv = a[0] != Py_None;
        int64_t T = 0, pages = 0;
        int32_t hkv = 1;
        Heads k, v, q;
        const int32_t *slots = nullptr;
        void *pool = nullptr, *q_out = nullptr;
        if ((a[1] != Py_None) != kv || (a[2] != Py_None) != kv || (a[3] != Py_None) != kv)
            throw Refused{"append_tokens: k, v, slots and raw_pool go together"};
        if (kv) {
            const at::Tensor &kt = tensor(a[0], "k");
            if (kt.dim() != 3) throw Refused{"k: expected [tokens][heads][128], got " + shape_of(kt)};
            T = kt.size(0);
            k = heads_of(kt, "k", T, dev);
            v = heads_of(tensor(a[1], "v"), "v", T, dev);
            hkv = k.heads;
            if (v.heads != hkv) throw Refused{"v: expected " + std::to_string(hkv) + " heads, got " + std::to_string(v.heads)};
            const at::Tensor &pt = tensor(a[3], "raw_pool"), &st = tensor(a[2], "slots");
            dims_of(pt, "raw_pool", {-1, hkv, 2, 16, 128}, "[pages][heads of k][2][16][128]");
            dims_of(st, "slots", {T}, "[tokens]");
            pages = pt.size(0);
            pool = data(pt, "raw_pool", dev, kBf16, kBf16);
            slots = static_cast<const int32_t *>(data(st, "slots", dev, kI32, kI32));
        } else if (a[5] == Py_None) {
            throw Refused{"append_tokens: no tokens (k and q are both None)"};
        }
        if (a[5] != Py_None) {
            const at::Tensor &qt = tensor(a[5], "q"), &ot = tensor(a[6], "q_out");
            if (qt.dim() != 3) throw Refused{"q: expected [tokens][heads][128], got " + shape_of(qt)};
            if (!kv) T = qt.size(0);
            q = heads_of(qt, "q", T, dev);
            if (ot.sizes() != qt.sizes()) throw Refused{"q_out: expected " + shape_of(qt) + ", got " + shape_of(ot)};
            q_out = data(ot, "q_out", dev, kBf16, kBf16);
        } else if (a[6] != Py_None) {
            throw Refused{"q_out without q"};
        }
        int32_t axes = 0, rot = 0;
        const uint64_t *rope = nullptr;
        const int32_t *positions = nullptr;
        if (a[7] != Py_None) {
            const at::Tensor &rt = tensor(a[7], "rope");
            if (a[8] == Py_None) throw Refused{"rope without positions"};
            const at::Tensor &pt = tensor(a[8], "positions");
            dims_of(rt, "rope", {-1, 2}, "a rope_table");
            if ((pt.dim() != 1 && pt.dim() != 2) || pt.size(-1) != T)
                throw Refused{"positions: expected [tokens] or [axes][tokens], got " + shape_of(pt)};
            axes = pt.dim() == 1 ? 1 : i32(pt.size(0), "positions");
            rot = i32(2 * rt.size(0), "rope");
            rope = static_cast<const uint64_t *>(data(rt, "rope", dev, kI64, kI64));
            positions = static_cast<const int32_t *>(data(pt, "positions", dev, kI32, kI32));
        }
        const int interleaved = PyObject_IsTrue(a[9]);
        const double scale = PyFloat_AsDouble(a[10]), eps = PyFloat_AsDouble(a[14]);
        if (interleaved < 0 || PyErr_Occurred())
            throw Refused{"interleaved, rope_scale, norm_eps: expected a truth value and numbers"};
        if ((a[12] != Py_None && a[5] == Py_None) || (a[13] != Py_None && !kv)) throw Refused{"q_norm without q, or k_norm without k"};
        const Norm qn = norm_of(a[12], "q_norm", q.heads, dev), kn = norm_of(a[13], "k_norm", hkv, dev);
        if (qn.data && kn.data && qn.type != kn.type) throw Refused{"q_norm, k_norm: expected weights of one type"};
        const int32_t nflags = (qn.per_head ? KVZ_NORM_Q_PER_HEAD : 0) | (kn.per_head ? KVZ_NORM_K_PER_HEAD : 0);
        uint32_t *status = data<uint32_t>(a[4], "status", dev, kI32, at::kUInt32);
        const kvz_stream_t stream = stream_of(a[11], dev);
        const kvz_dims dims{hkv, 128, 16};
        const int32_t tokens = i32(T, "tokens");
        int rc = 0;
        Py_BEGIN_ALLOW_THREADS;
        rc = kvz_append_tokens_normed(dims, tokens, q.heads, q.data, q.token, q.head, k.data, k.token, k.head, v.data,
                                      v.token, v.head, slots, positions, axes, rope, rot,
                                      interleaved ? KVZ_ROPE_INTERLEAVED : 0u, (float)scale, qn.data, kn.data,
                                      qn.data ? qn.type : kn.type, nflags, (float)eps, q_out, pool, pages, status, stream);
        Py_END_ALLOW_THREADS;
        return rc;
    });
}

// q, group_start, prefix_ids, prefix_lens, prefix_tail, page_ids, seq_lens, tail_page, meta, arena, raw_pool, out,
// status, workspace, stream; the raw call has None for prefix_tail, tail_page, meta and arena
PyObject *prefix_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&] {
        count(n, 15);
        const int dev = device_of(a[12]);
        const bool coded = a[8] != Py_None;
        const at::Tensor &q = tensor(a[0], "q"), &start = tensor(a[1], "group_start"), &pids = tensor(a[2], "prefix_ids");
        const at::Tensor &plens = tensor(a[3], "prefix_lens"), &ids = tensor(a[5], "page_ids"), &lens = tensor(a[6], "seq_lens");
        const at::Tensor &pool = tensor(a[10], "raw_pool"), &out = tensor(a[11], "out"), &ws = tensor(a[13], "workspace");
        dims_of(q, "q", {-1, -1, 128}, "[batch][heads][128]");
        const int64_t B = q.size(0), hq = q.size(1);
        dims_of(plens, "prefix_lens", {-1}, "[groups]");
        const int64_t G = plens.size(0);
        dims_of(start, "group_start", {G + 1}, "[groups + 1]");
        dims_of(pids, "prefix_ids", {G, -1}, "[groups][pages]");
        dims_of(ids, "page_ids", {B, -1}, "[batch][pages]");
        dims_of(lens, "seq_lens", {B}, "[batch]");
        if (out.sizes() != q.sizes()) throw Refused{"out: expected " + shape_of(q) + ", got " + shape_of(out)};
        if (out.scalar_type() != at::kFloat && out.scalar_type() != kBf16)
            throw Refused{std::string("out: expected torch.float32 or torch.bfloat16, got ") + c10::toString(out.scalar_type())};
        dims_of(pool, "raw_pool", {-1, -1, 2, 16, 128}, "[pages][heads][2][16][128]");
        const int64_t hkv = pool.size(1);
        const int32_t type = out.scalar_type() == at::kFloat ? KVZ_OUT_F32 : KVZ_OUT_BF16;
        const void *qp = data(q, "q", dev, kBf16, kBf16);
        const auto *sp = static_cast<const int32_t *>(data(start, "group_start", dev, kI32, kI32));
        const auto *pip = static_cast<const int32_t *>(data(pids, "prefix_ids", dev, kI32, kI32));
        const auto *plp = static_cast<const int32_t *>(data(plens, "prefix_lens", dev, kI32, kI32));
        const auto *ip = static_cast<const int32_t *>(data(ids, "page_ids", dev, kI32, kI32));
        const auto *lp = static_cast<const int32_t *>(data(lens, "seq_lens", dev, kI32, kI32));
        const void *poolp = data(pool, "raw_pool", dev, kBf16, kBf16);
        void *outp = data(out, "out", dev, out.scalar_type(), out.scalar_type());
        void *wsp = data(ws, "workspace", dev, kU8, kU8);
        uint32_t *status = data<uint32_t>(a[12], "status", dev, kI32, at::kUInt32);
        const kvz_stream_t stream = stream_of(a[14], dev);
        const kvz_dims dims{i32(hkv, "raw_pool"), 128, 16};
        const int32_t b = i32(B, "batch"), h = i32(hq, "heads"), g = i32(G, "groups");
        const int32_t pp = i32(pids.size(1), "prefix_ids"), op = i32(ids.size(1), "page_ids");
        const int64_t pages = pool.size(0);
        const size_t bytes = (size_t)ws.numel();
        int rc = 0;
        if (!coded) {
            Py_BEGIN_ALLOW_THREADS;
            rc = kvz_prefix_attention_raw(dims, b, h, qp, g, sp, pip, pp, plp, ip, op, lp, poolp, pages, outp, type, wsp, bytes,
                                          status, stream);
            Py_END_ALLOW_THREADS;
            return rc;
        }
        const at::Tensor &ptail = tensor(a[4], "prefix_tail"), &tail = tensor(a[7], "tail_page"), &meta = tensor(a[8], "meta");
        const at::Tensor &arena = tensor(a[9], "arena");
        dims_of(ptail, "prefix_tail", {G}, "[groups]");
        dims_of(tail, "tail_page", {B}, "[batch]");
        dims_of(meta, "meta", {-1, hkv, 2}, "[pages][heads of raw_pool][2]");
        const auto *ptp = static_cast<const int32_t *>(data(ptail, "prefix_tail", dev, kI32, kI32));
        const auto *tp = static_cast<const int32_t *>(data(tail, "tail_page", dev, kI32, kI32));
        const auto *mp = static_cast<const uint64_t *>(data(meta, "meta", dev, kI64, at::kUInt64));
        const auto *ap = static_cast<const uint8_t *>(data(arena, "arena", dev, kU8, kU8));
        const int64_t meta_pages = meta.size(0);
        const uint64_t arena_bytes = (uint64_t)arena.numel();
        Py_BEGIN_ALLOW_THREADS;
        rc = kvz_prefix_attention(dims, b, h, qp, g, sp, pip, pp, plp, ptp, ip, op, lp, tp, mp, meta_pages, ap, arena_bytes,
                                  poolp, pages, outp, type, wsp, bytes, status, stream);
        Py_END_ALLOW_THREADS;
        return rc;
    });
}

// rows, new_tokens, lens, tables, free_pages, free_count, q_start, seq_lens, page_ids, positions, slots, lens_out,
// free_out, status, stream
PyObject *plan_step(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&] {
        count(n, 15);
        const int dev = device_of(a[13]);
        const char *names[] = {"rows", "new_tokens", "lens", "tables", "free_pages", "free_count", "q_start", "seq_lens",
                               "page_ids", "positions", "slots", "lens_out", "free_out"};
        int32_t *p[13];
        int64_t size[13];
        for (int i = 0; i < 13; ++i) {
            const at::Tensor &t = tensor(a[i], names[i]);
            p[i] = static_cast<int32_t *>(data(t, names[i], dev, kI32, kI32));
            size[i] = t.numel();
        }
        const at::Tensor &tables = tensor(a[3], "tables"), &rows = tensor(a[0], "rows"), &positions = tensor(a[9], "positions");
        dims_of(rows, "rows", {-1}, "[requests]");
        const int64_t B = rows.size(0);
        dims_of(tensor(a[2], "lens"), "lens", {-1}, "[rows]");
        dims_of(tables, "tables", {size[2], -1}, "[rows of lens][pages]");
        dims_of(tensor(a[4], "free_pages"), "free_pages", {-1}, "[pages]");
        dims_of(positions, "positions", {-1}, "[tokens]");
        const int64_t want[13] = {B, B, size[2], size[3], size[4], 1, B + 1, B, B * tables.size(1), size[9], size[9], size[2], 1};
        for (int i = 0; i < 13; ++i)
            if (size[i] != want[i])
                throw Refused{std::string(names[i]) + ": expected " + std::to_string(want[i]) + " values, got " + std::to_string(size[i])};
        // what is written may overlap nothing else, but lens_out and free_out may be lens and free_count
        for (int i : {3, 6, 7, 8, 9, 10, 11, 12})
            for (int j = 0; j < 13; ++j) {
                if (i == j || (i == 11 && j == 2 && p[i] == p[j]) || (i == 12 && j == 5 && p[i] == p[j])) continue;
                if (size[i] && size[j] && p[i] < p[j] + size[j] && p[j] < p[i] + size[i])
                    throw Refused{std::string(names[i]) + " overlaps " + names[j]};
            }
        uint32_t *status = data<uint32_t>(a[13], "status", dev, kI32, at::kUInt32);
        const kvz_stream_t stream = stream_of(a[14], dev);
        const int32_t batch = i32(B, "rows"), tokens = i32(size[9], "positions"), num_rows = i32(size[2], "lens");
        const int32_t width = i32(tables.size(1), "tables"), capacity = i32(size[4], "free_pages");
        int rc = 0;
        Py_BEGIN_ALLOW_THREADS;
        rc = kvz_plan_step(batch, tokens, p[0], p[1], p[2], num_rows, p[3], width, p[4], capacity, p[5], p[6], p[7], p[8], p[9],
                           p[10], p[11], p[12], status, stream);
        Py_END_ALLOW_THREADS;
        return rc;
    });
}

// q, q_start, page_ids, seq_lens, tail_page, meta, arena, raw_pool, window, sinks, out, status, workspace, stream; the raw
// call has None for tail_page, meta and arena
PyObject *chunk_attention(PyObject *, PyObject *const *a, Py_ssize_t n)
{
    return guarded([&] {
        count(n, 14);
        const int dev = device_of(a[11]);
        const bool coded = a[5] != Py_None;
        const at::Tensor &q = tensor(a[0], "q"), &start = tensor(a[1], "q_start"), &ids = tensor(a[2], "page_ids");
        const at::Tensor &lens = tensor(a[3], "seq_lens"), &pool = tensor(a[7], "raw_pool"), &out = tensor(a[10], "out");
        const at::Tensor &ws = tensor(a[12], "workspace");
        dims_of(q, "q", {-1, -1, 128}, "[tokens][heads][128]");
        dims_of(lens, "seq_lens", {-1}, "[batch]");
        const int64_t B = lens.size(0);
        dims_of(start, "q_start", {B + 1}, "[batch + 1]");
        dims_of(ids, "page_ids", {B, -1}, "[batch][pages]");
        if (out.sizes() != q.sizes()) throw Refused{"out: expected " + shape_of(q) + ", got " + shape_of(out)};
        if (out.scalar_type() != at::kFloat && out.scalar_type() != kBf16)
            throw Refused{std::string("out: expected torch.float32 or torch.bfloat16, got ") + c10::toString(out.scalar_type())};
        dims_of(pool, "raw_pool", {-1, -1, 2, 16, 128}, "[pages][heads][2][16][128]");
        const int64_t hkv = pool.size(1);
        const int32_t type = out.scalar_type() == at::kFloat ? KVZ_OUT_F32 : KVZ_OUT_BF16;
        const void *qp = data(q, "q", dev, kBf16, kBf16);
        const auto *sp = static_cast<const int32_t *>(data(start, "q_start", dev, kI32, kI32));
        const auto *ip = static_cast<const int32_t *>(data(ids, "page_ids", dev, kI32, kI32));
        const auto *lp = static_cast<const int32_t *>(data(lens, "seq_lens", dev, kI32, kI32));
        const void *poolp = data(pool, "raw_pool", dev, kBf16, kBf16);
        void *outp = data(out, "out", dev, out.scalar_type(), out.scalar_type());
        void *wsp = data(ws, "workspace", dev, kU8, kU8);
        uint32_t *status = data<uint32_t>(a[11], "status", dev, kI32, at::kUInt32);
        const int64_t window = PyLong_AsLongLong(a[8]), sinks = PyLong_AsLongLong(a[9]);
        if (PyErr_Occurred()) throw Refused{"window, sinks: expected whole numbers"};
        if (window < 0 || sinks < 0) throw Refused{"window, sinks: expected numbers >= 0"};
        const kvz_stream_t stream = stream_of(a[13], dev);
        const kvz_dims dims{i32(hkv, "raw_pool"), 128, 16};
        const int32_t T = i32(q.size(0), "tokens"), hq = i32(q.size(1), "heads"), b = i32(B, "batch");
        const int32_t pages = i32(ids.size(1), "page_ids");
        // (more than any length is no limit)
        const int32_t w = (int32_t)std::min<int64_t>(window, INT32_MAX), k = (int32_t)std::min<int64_t>(sinks, INT32_MAX);
        const int64_t num = pool.size(0);
        const size_t bytes = (size_t)ws.numel();
        int rc = 0;
        if (!coded) {
            Py_BEGIN_ALLOW_THREADS;
            rc = kvz_chunk_attention_raw(dims, T, hq, qp, b, sp, ip, pages, lp, poolp, num, w, k, outp, type, wsp, bytes, status,
                                         stream);
            Py_END_ALLOW_THREADS;
            return rc;
        }
        const at::Tensor &tail = tensor(a[4], "tail_page"), &meta = tensor(a[5], "meta"), &arena = tensor(a[6], "arena");
        dims_of(tail, "tail_page", {B}, "[batch]");
        dims_of(meta, "meta", {-1, hkv, 2}, "[pages][heads of raw_pool][2]");
        const auto *tp = static_cast<const int32_t *>(data(tail, "tail_page", dev, kI32, kI32));
        const auto *mp = static_cast<const uint64_t *>(data(meta, "meta", dev, kI64, at::kUInt64));
        const auto *ap = static_cast<const uint8_t *>(data(arena, "arena", dev, kU8, kU8));
        const int64_t meta_pages = meta.size(0);
        const uint64_t arena_bytes = (uint64_t)arena.numel();
        Py_BEGIN_ALLOW_THREADS;
        rc = kvz_chunk_attention(dims, T, hq, qp, b, sp, ip, pages, lp, tp, mp, meta_pages, ap, arena_bytes, poolp, num, w, k,
                                 outp, type, wsp, bytes, status, stream);
        Py_END_ALLOW_THREADS;
        return rc;
    });
}

PyMethodDef methods[] = {
    {"chunk_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(chunk_attention)), METH_FASTCALL, nullptr},
    {"plan_step", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(plan_step)), METH_FASTCALL, nullptr},
    {"append_tokens", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(append_tokens)), METH_FASTCALL, nullptr},
    {"prefix_attention", reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(prefix_attention)), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
