// The Python side of the single-token calls (moss_enc_gemv_q4,
// moss_enc_kv_append, moss_enc_paged_attn): checks of the tensors, new outputs
// from PyTorch's allocator on the handle's stream, and the call of the C ABI.
//
// These calls run for a few microseconds on the GPU and a decoding step makes
// several per layer, so their way through Python counts: checked and marshalled
// in Python with ctypes, as the other calls are, they took 13 to 18 us of the
// host's time each, here about 4.
#include <Python.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cmath>
#include <optional>

#include "../../include/moss_enc.h"

namespace {

// The C ABI, by address (the library is loaded by the caller).
decltype(&moss_enc_gemv_q4) p_gemv = nullptr;
decltype(&moss_enc_kv_append) p_append = nullptr;
decltype(&moss_enc_paged_attn) p_attn = nullptr;
decltype(&moss_enc_paged_attn_workspace) p_workspace = nullptr;

// What every call gets first: the handle, its stream and its device.
struct Handle {
    moss_enc *h;
    cudaStream_t stream;
    c10::DeviceIndex device;
};

struct Refused {
    const char *why;
};

long long integer(PyObject *o)
{
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    return v;
}

int small(PyObject *o, const char *why)
{
    const long long v = integer(o);
    if (v < INT_MIN || v > INT_MAX) throw Refused{why};
    return (int)v;
}

Handle handle(PyObject *const *args)
{
    return Handle{reinterpret_cast<moss_enc *>(integer(args[0])),
                  reinterpret_cast<cudaStream_t>(integer(args[1])),
                  (c10::DeviceIndex)integer(args[2])};
}

// A tensor argument on the handle's device; null for None where that is allowed.
const at::Tensor *tensor(const Handle &h, PyObject *o, bool none, const char *why)
{
    if (o == Py_None) {
        if (none) return nullptr;
        throw Refused{why};
    }
    if (!THPVariable_Check(o)) throw Refused{why};
    const at::Tensor &t = THPVariable_Unpack(o);
    if (!t.is_cuda() || t.get_device() != h.device) throw Refused{"tensors must be on the handle's CUDA device"};
    return &t;
}

// A new tensor whose memory belongs to the handle's stream.
at::Tensor fresh(const Handle &h, c10::IntArrayRef shape, at::ScalarType type)
{
    const c10::Device dev(c10::DeviceType::CUDA, h.device);
    if (c10::cuda::getCurrentCUDAStream(h.device).stream() == h.stream)
        return at::detail::empty_cuda(shape, type, dev, std::nullopt);
    c10::cuda::CUDAStreamGuard guard(c10::cuda::getStreamFromExternal(h.stream, h.device));
    return at::detail::empty_cuda(shape, type, dev, std::nullopt);
}

PyObject *answer(moss_enc_status st, PyObject *ok)
{
    if (st == MOSS_ENC_OK) return ok;
    Py_XDECREF(ok);
    return PyLong_FromLong(st);  // the caller asks the handle what it was
}

#define CALL_BEGIN                     \
    HANDLE_TH_ERRORS                   \
    try {
#define CALL_END                                      \
    }                                                 \
    catch (const Refused &r)                          \
    {                                                 \
        PyErr_SetString(PyExc_ValueError, r.why);     \
        return nullptr;                               \
    }                                                 \
    END_HANDLE_TH_ERRORS

PyObject *owned(PyObject *given, const at::Tensor &made)
{
    if (given == Py_None) return THPVariable_Wrap(made);
    Py_INCREF(given);
    return given;
}

// gemv_q4(handle, stream, device, x, Bq, Bs, bias, out, epilogue)
PyObject *gemv_q4(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    CALL_BEGIN
    if (n != 9) throw Refused{"gemv_q4 takes nine arguments"};
    const Handle h = handle(args);
    static const char *shapes = "x [M][K] bf16, Bq [N][K/2] uint8, Bs [K/128][N] fp32, contiguous, K a multiple of 128";
    const at::Tensor &x = *tensor(h, args[3], false, shapes), &bq = *tensor(h, args[4], false, shapes);
    const at::Tensor &bs = *tensor(h, args[5], false, shapes);
    const int epilogue = small(args[8], "unsupported epilogue");
    if (x.dim() != 2 || bq.dim() != 2 || bs.dim() != 2 || x.scalar_type() != at::kBFloat16 || bq.scalar_type() != at::kByte ||
        bs.scalar_type() != at::kFloat || !x.is_contiguous() || !bq.is_contiguous() || !bs.is_contiguous())
        throw Refused{shapes};
    const int64_t M = x.size(0), K = x.size(1), N = bq.size(0);
    if (K % 128 != 0 || bq.size(1) * 2 != K || bs.size(0) != K / 128 || bs.size(1) != N || M > INT_MAX || N > INT_MAX || K > INT_MAX)
        throw Refused{shapes};
    const at::Tensor *bias = tensor(h, args[6], true, "bias [N] fp32");
    if (bias && (bias->scalar_type() != at::kFloat || bias->dim() != 1 || bias->size(0) != N || !bias->is_contiguous()))
        throw Refused{"bias [N] fp32"};
    const at::ScalarType type = epilogue == 0 || epilogue == 1 ? at::kBFloat16 : at::kFloat;
    static const char *outs = "out [M][N], contiguous, bf16 (epilogues 0, 1) or fp32 (2, 5); epilogue 2 adds to it";
    const at::Tensor *given = tensor(h, args[7], epilogue != 2, outs);
    at::Tensor made;
    if (!given)
        made = fresh(h, {M, N}, type);
    else if (given->scalar_type() != type || given->dim() != 2 || given->size(0) != M || given->size(1) != N || !given->is_contiguous())
        throw Refused{outs};
    const at::Tensor &out = given ? *given : made;
    const moss_enc_status st = p_gemv(h.h, x.data_ptr(), bq.data_ptr(), static_cast<const float *>(bs.data_ptr()),
                                      bias ? static_cast<const float *>(bias->data_ptr()) : nullptr, out.data_ptr(), (int)M,
                                      (int)N, (int)K, epilogue);
    return answer(st, st == MOSS_ENC_OK ? owned(args[7], made) : nullptr);
    CALL_END
}

// Row stride of x [rows][heads][dim] whose rows are whole; `heads` < 0: any.
int64_t heads_stride(const at::Tensor &x, int64_t rows, int64_t heads, int64_t dim, at::ScalarType type, const char *why)
{
    if (x.dim() != 3 || x.scalar_type() != type || x.size(0) != rows || x.size(2) != dim || (heads >= 0 && x.size(1) != heads) ||
        x.stride(2) != 1 || (x.size(1) > 1 && x.stride(1) != dim))
        throw Refused{why};
    return rows > 1 ? x.stride(0) : x.size(1) * dim;
}

// The 16-bit type of rows that may meet the cache.
int rows_type(const moss_enc_kv_cache *c, const at::Tensor &x, const char *why)
{
    const int t = x.scalar_type() == at::kBFloat16 ? MOSS_ENC_KV_BF16 : x.scalar_type() == at::kHalf ? MOSS_ENC_KV_F16 : -1;
    if (t < 0 || (c->dtype != MOSS_ENC_KV_E4M3 && c->dtype != t)) throw Refused{why};
    return t;
}

bool vector32(const at::Tensor &x, int64_t n)
{
    return x.scalar_type() == at::kInt && x.dim() == 1 && x.size(0) == n && x.is_contiguous();
}

// kv_append(handle, stream, device, cache, k, v, positions, seqs, q, q_out, inv_freq, interleaved)
PyObject *kv_append(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    CALL_BEGIN
    if (n != 12) throw Refused{"kv_append takes twelve arguments"};
    const Handle h = handle(args);
    const moss_enc_kv_cache *c = reinterpret_cast<const moss_enc_kv_cache *>(integer(args[3]));
    static const char *keys = "k and v: [rows][n_kv_heads][head_dim] of the cache's type (bf16 or f16 with an e4m3 cache), the heads of a row together";
    static const char *queries = "q and q_out: [rows][heads][head_dim] of k's type, the heads of a row together";
    static const char *freqs = "inv_freq: fp64 [r / 2], contiguous";
    const at::Tensor &k = *tensor(h, args[4], false, keys), &v = *tensor(h, args[5], false, keys);
    const at::Tensor &positions = *tensor(h, args[6], false, "positions: int32 [rows]");
    const at::Tensor *seqs = tensor(h, args[7], true, "seqs: int32 [rows]"), *q = tensor(h, args[8], true, queries);
    const at::Tensor *q_out = tensor(h, args[9], true, queries), *inv = tensor(h, args[10], true, freqs);
    const int interleaved = PyObject_IsTrue(args[11]);
    if (interleaved < 0) throw python_error();
    if (k.dim() != 3) throw Refused{keys};
    const int64_t rows = k.size(0), dim = c->head_dim;
    moss_enc_kv_rows r{};
    r.dtype = rows_type(c, k, keys);
    const at::ScalarType type = k.scalar_type();
    r.k_stride = heads_stride(k, rows, c->n_kv_heads, dim, type, keys);
    r.v_stride = heads_stride(v, rows, c->n_kv_heads, dim, type, keys);
    if (rows > INT_MAX || !vector32(positions, rows)) throw Refused{"positions: int32 [rows]"};
    if (seqs && !vector32(*seqs, rows)) throw Refused{"seqs: int32 [rows]"};
    if (inv && (inv->scalar_type() != at::kDouble || inv->dim() != 1 || !inv->is_contiguous() || inv->size(0) > INT_MAX / 2))
        throw Refused{freqs};
    at::Tensor made;
    if (q) {
        r.q_stride = heads_stride(*q, rows, -1, dim, type, queries);
        const int64_t heads = q->size(1);
        if (heads > INT_MAX) throw Refused{queries};
        if (!q_out) {
            made = fresh(h, {rows, heads, dim}, type);
            q_out = &made;
        }
        r.q_out_stride = heads_stride(*q_out, rows, heads, dim, type, queries);
        r.n_q_heads = (int)heads;
        if (heads > 0) {
            r.q = q->data_ptr();
            r.q_out = q_out->data_ptr();
        }
    } else if (q_out)
        throw Refused{"q_out needs q"};
    r.k = k.data_ptr();
    r.v = v.data_ptr();
    r.positions = static_cast<const int32_t *>(positions.data_ptr());
    r.seqs = seqs ? static_cast<const int32_t *>(seqs->data_ptr()) : nullptr;
    r.rotary = inv ? 2 * (int)inv->size(0) : 0;
    r.inv_freq = r.rotary ? static_cast<const double *>(inv->data_ptr()) : nullptr;
    r.n_rows = (int)rows;
    r.interleaved = interleaved;
    const moss_enc_status st = p_append(h.h, c, &r);
    if (st != MOSS_ENC_OK) return answer(st, nullptr);
    if (!q) Py_RETURN_NONE;
    return owned(args[9], made);
    CALL_END
}

// paged_attn(handle, stream, device, cache, q, lengths, scale, out, lse, return_lse, max_len, workspace)
PyObject *paged_attn(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    CALL_BEGIN
    if (n != 12) throw Refused{"paged_attn takes twelve arguments"};
    const Handle h = handle(args);
    const moss_enc_kv_cache *c = reinterpret_cast<const moss_enc_kv_cache *>(integer(args[3]));
    static const char *queries = "q: [n_seqs][heads][head_dim] of the cache's type (bf16 or f16 with an e4m3 cache), the heads of a row together";
    static const char *outs = "out: contiguous, of q's shape and type", *sums = "lse: fp32 [n_seqs][heads], contiguous";
    static const char *room = "workspace: uint8, contiguous";
    const at::Tensor &q = *tensor(h, args[4], false, queries), &lengths = *tensor(h, args[5], false, "lengths: int32 [n_seqs]");
    const at::Tensor *out = tensor(h, args[7], true, outs), *lse = tensor(h, args[8], true, sums);
    const at::Tensor *work = tensor(h, args[11], true, room);
    const int return_lse = PyObject_IsTrue(args[9]);
    if (return_lse < 0) throw python_error();
    const int64_t seqs = c->n_seqs, dim = c->head_dim;
    moss_enc_attn a{};
    a.dtype = rows_type(c, q, queries);
    a.q_stride = heads_stride(q, seqs, -1, dim, q.scalar_type(), queries);
    const int64_t heads = q.size(1);
    if (heads > INT_MAX) throw Refused{queries};
    if (!vector32(lengths, seqs)) throw Refused{"lengths: int32 [n_seqs]"};
    a.max_len = small(args[10], "max_len out of range");
    a.n_q_heads = (int)heads;
    a.scale = args[6] == Py_None ? (float)(1.0 / std::sqrt((double)dim)) : (float)PyFloat_AsDouble(args[6]);
    if (PyErr_Occurred()) throw python_error();
    const int64_t need = p_workspace(h.h, c, a.n_q_heads, a.max_len);
    if (need < 0) throw Refused{"the number of query heads must be a multiple of the key heads', max_len not negative"};
    at::Tensor made, made_lse, made_work;
    if (!out) {
        made = fresh(h, {seqs, heads, dim}, q.scalar_type());
        out = &made;
    } else if (out->scalar_type() != q.scalar_type() || out->sizes() != q.sizes() || !out->is_contiguous())
        throw Refused{outs};
    if (lse) {
        if (lse->scalar_type() != at::kFloat || lse->dim() != 2 || lse->size(0) != seqs || lse->size(1) != heads || !lse->is_contiguous())
            throw Refused{sums};
    } else if (return_lse) {
        made_lse = fresh(h, {seqs, heads}, at::kFloat);
        lse = &made_lse;
    }
    if (work) {
        if (work->scalar_type() != at::kByte || !work->is_contiguous()) throw Refused{room};
    } else if (need > 0) {
        made_work = fresh(h, {need}, at::kByte);
        work = &made_work;
    }
    a.q = q.data_ptr();
    a.out = out->data_ptr();
    a.lse = lse ? static_cast<float *>(lse->data_ptr()) : nullptr;
    a.lengths = static_cast<const int32_t *>(lengths.data_ptr());
    a.workspace = work ? work->data_ptr() : nullptr;
    a.workspace_bytes = work ? work->numel() : 0;
    const moss_enc_status st = p_attn(h.h, c, &a);
    if (st != MOSS_ENC_OK) return answer(st, nullptr);
    PyObject *o = owned(args[7], made);
    if (!return_lse || !o) return o;
    PyObject *l = owned(args[8], made_lse);
    PyObject *both = l ? PyTuple_Pack(2, o, l) : nullptr;
    Py_DECREF(o);
    Py_XDECREF(l);
    return both;
    CALL_END
}

// bind(gemv_q4, kv_append, paged_attn, paged_attn_workspace): addresses
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    CALL_BEGIN
    if (n != 4) throw Refused{"bind takes four addresses"};
    p_gemv = reinterpret_cast<decltype(p_gemv)>(integer(args[0]));
    p_append = reinterpret_cast<decltype(p_append)>(integer(args[1]));
    p_attn = reinterpret_cast<decltype(p_attn)>(integer(args[2]));
    p_workspace = reinterpret_cast<decltype(p_workspace)>(integer(args[3]));
    Py_RETURN_NONE;
    CALL_END
}

PyMethodDef methods[] = {
    {"bind", (PyCFunction)(void (*)(void))bind, METH_FASTCALL, nullptr},
    {"gemv_q4", (PyCFunction)(void (*)(void))gemv_q4, METH_FASTCALL, nullptr},
    {"kv_append", (PyCFunction)(void (*)(void))kv_append, METH_FASTCALL, nullptr},
    {"paged_attn", (PyCFunction)(void (*)(void))paged_attn, METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_pycalls", "The single-token calls of moss_enc.", -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pycalls(void) { return PyModule_Create(&module); }
