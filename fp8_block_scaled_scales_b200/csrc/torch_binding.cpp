// The expert-layer and gradient calls, and those around the expert layer, for Python: argument checks, output allocation and the
// call through the C ABI (include/dg.h), in one native function each.  A decode step is a
// chain of calls whose kernels take a few microseconds; done in Python, the checks, three
// allocations and the marshalling of a dozen arguments cost 9 to 17 us a call, here 3 to 8.
//
// Every function takes positional arguments (binding.py has the signatures and their
// documentation), raises ValueError for a tensor of the wrong type, shape, device or layout,
// and binding.DGError for a status that the library returns.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <vector>

#include "../../include/dg.h"

namespace {

using at::Tensor;
using Shape = std::initializer_list<int64_t>;

PyObject *g_error = nullptr;  // binding.DGError

constexpr at::ScalarType kU8 = at::kByte, kF32 = at::kFloat, kBF16 = at::kBFloat16, kI32 = at::kInt;

int64_t blocks(int64_t n) { return (n + 127) / 128; }

const Tensor &tensor(PyObject *o, const char *name) {
    TORCH_CHECK_TYPE(THPVariable_Check(o), name, " must be a tensor");
    return THPVariable_Unpack(o);
}

// The device of a call: its first tensor's, which has to be the current one.
int device_of(const Tensor &t, const char *name, int64_t dims) {
    TORCH_CHECK_VALUE(t.dim() == dims, name, " must have ", dims, " dimensions, not ", t.dim());
    TORCH_CHECK_VALUE(t.is_cuda(), name, " must be a CUDA device tensor");
    const int dev = t.get_device();
    TORCH_CHECK_VALUE(dev == c10::cuda::current_device(), name, " is on cuda:", dev, ", which is not the current device");
    return dev;
}

// Address of a tensor that has to have this type, shape and device, row-major; codes may be
// uint8 or float8_e4m3fn.
void *checked(const Tensor &t, const char *name, at::ScalarType type, at::IntArrayRef shape, int dev) {
    TORCH_CHECK_VALUE(t.scalar_type() == type || (type == kU8 && t.scalar_type() == at::kFloat8_e4m3fn), name,
                      " must be ", type, ", not ", t.scalar_type());
    TORCH_CHECK_VALUE(t.sizes() == shape, name, " must have shape ", shape, ", not ", t.sizes());
    TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == dev, name, " must be on cuda:", dev,
                      ", the current device and that of the other tensors");
    TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous (row-major)");
    return t.data_ptr();
}

template <typename T = void>
T *in(PyObject *o, const char *name, at::ScalarType type, Shape shape, int dev) {
    return static_cast<T *>(checked(tensor(o, name), name, type, shape, dev));
}

template <typename T = void>
T *in_or_null(PyObject *o, const char *name, at::ScalarType type, Shape shape, int dev) {
    return o == Py_None ? nullptr : in<T>(o, name, type, shape, dev);
}

Tensor make(at::ScalarType type, Shape shape, int dev) {
    // what at::empty comes to on a GPU, without the way through the dispatcher
    return Tensor(at::detail::empty_cuda(at::IntArrayRef(shape), type,
                                         c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(dev)), std::nullopt));
}

// The caller's output, checked, or a new one (not filled).
Tensor out(PyObject *o, const char *name, at::ScalarType type, Shape shape, int dev) {
    if (o == Py_None) return make(type, shape, dev);
    const Tensor &t = tensor(o, name);
    checked(t, name, type, shape, dev);
    return t;
}

template <typename T = void>
T *ptr(const Tensor &t) {
    return static_cast<T *>(t.data_ptr());
}

// The stream of a call, made the current one while the call lasts: what the call allocates then
// comes from that stream's own memory, which no work on another stream can still be using, and
// scratch that is freed at the end of the call goes back to it.
class CallStream {
public:
    CallStream(PyObject *stream, int dev) {
        const auto device = static_cast<c10::DeviceIndex>(dev);
        if (stream == Py_None) {
            handle_ = c10::cuda::getCurrentCUDAStream(device).stream();
            return;
        }
        PyObject *h = PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) throw python_error();
        const unsigned long long v = PyLong_AsUnsignedLongLong(h);
        Py_DECREF(h);
        if (PyErr_Occurred()) throw python_error();
        handle_ = reinterpret_cast<cudaStream_t>(v);
        guard_.reset_stream(c10::cuda::getStreamFromExternal(handle_, device));
    }
    operator cudaStream_t() const { return handle_; }

private:
    cudaStream_t handle_;
    c10::cuda::OptionalCUDAStreamGuard guard_;
};

int64_t integer(PyObject *o, const char *name, int64_t least, int64_t most) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw python_error();
    TORCH_CHECK_VALUE(v >= least && v <= most, name, " must lie in [", least, ", ", most, "], not ", v);
    return v;
}

bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw python_error();
    return v != 0;
}

void status(dg_status_t st, const char *what) {
    if (st == DG_OK) return;
    PyObject *e = PyObject_CallFunction(g_error, "is", static_cast<int>(st), what);
    if (e) {
        PyErr_SetObject(g_error, e);
        Py_DECREF(e);
    }
    throw python_error();
}

PyObject *wrap(const Tensor &t) { return THPVariable_Wrap(t); }

template <typename... Ts>
PyObject *wrap_all(const Ts &...ts) {
    PyObject *tuple = PyTuple_New(sizeof...(ts));
    if (!tuple) throw python_error();
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(tuple, i++, wrap(ts)), ...);
    return tuple;
}

constexpr int64_t kIntMax = 0x7FFFFFFF;

// The sorts' outputs follow G and M_max, which no tensor bounds: the library's limits on them
// are looked at before anything is allocated.
void sort_sizes(int64_t G, int64_t M_max, const char *what) {
    if (G < 1 || G > 1024 || M_max > kIntMax / G) status(DG_ERR_SHAPE, what);
}

// Scratch for one call, from the call's stream: an empty tensor where none is needed.
Tensor scratch(int64_t bytes, int dev) { return bytes == 0 ? Tensor() : make(kU8, {bytes}, dev); }

// (topk_ids, G, offsets, row_of_slot, slot_of_row, stream)
PyObject *moe_sort(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &ids = tensor(a[0], "topk_ids");
    const int dev = device_of(ids, "topk_ids", 2);
    const CallStream st(a[5], dev);
    const int64_t T = ids.size(0), k = ids.size(1), G = integer(a[1], "G", 0, kIntMax);
    TORCH_CHECK_VALUE(k <= kIntMax, "topk_ids is too wide");
    const bool wide = ids.scalar_type() == at::kLong;
    void *pi = checked(ids, "topk_ids", wide ? at::kLong : kI32, {T, k}, dev);
    sort_sizes(G, 0, "dg_moe_sort");
    const int64_t S = T * k, cap = a[4] == Py_None ? (S + 127 * std::min(G, S)) / 128 * 128 : tensor(a[4], "slot_of_row").numel();
    const Tensor offsets = out(a[2], "offsets", kI32, {G + 1}, dev);
    const Tensor row = out(a[3], "row_of_slot", kI32, {T, k}, dev);
    const Tensor slot = out(a[4], "slot_of_row", kI32, {cap}, dev);
    const Tensor w = scratch(dg_moe_sort_workspace(T, static_cast<int>(k), static_cast<int>(G)), dev);
    status(dg_moe_sort(pi, wide, T, static_cast<int>(k), static_cast<int>(G), ptr<int32_t>(offsets), ptr<int32_t>(row),
                       ptr<int32_t>(slot), cap, w.defined() ? w.data_ptr() : nullptr, w.defined() ? w.numel() : 0, st),
           "dg_moe_sort");
    return wrap_all(offsets, row, slot);
    END_HANDLE_TH_ERRORS
}

// (topk_ids, G, M_max, masked_m, row_of_slot, slot_of_row, stream)
PyObject *moe_sort_masked(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &ids = tensor(a[0], "topk_ids");
    const int dev = device_of(ids, "topk_ids", 2);
    const CallStream st(a[6], dev);
    const int64_t T = ids.size(0), k = ids.size(1), G = integer(a[1], "G", 0, kIntMax);
    const int64_t M_max = integer(a[2], "M_max", 0, kIntMax);
    TORCH_CHECK_VALUE(k <= kIntMax, "topk_ids is too wide");
    const bool wide = ids.scalar_type() == at::kLong;
    void *pi = checked(ids, "topk_ids", wide ? at::kLong : kI32, {T, k}, dev);
    sort_sizes(G, M_max, "dg_moe_sort_masked");
    const Tensor m = out(a[3], "masked_m", kI32, {G}, dev);
    const Tensor row = out(a[4], "row_of_slot", kI32, {T, k}, dev);
    const Tensor slot = out(a[5], "slot_of_row", kI32, {G * M_max}, dev);
    const Tensor w = scratch(dg_moe_sort_workspace(T, static_cast<int>(k), static_cast<int>(G)), dev);
    status(dg_moe_sort_masked(pi, wide, T, static_cast<int>(k), static_cast<int>(G), ptr<int32_t>(m), ptr<int32_t>(row),
                              ptr<int32_t>(slot), M_max, w.defined() ? w.data_ptr() : nullptr,
                              w.defined() ? w.numel() : 0, st),
           "dg_moe_sort_masked");
    return wrap_all(m, row, slot);
    END_HANDLE_TH_ERRORS
}

// (x, slot_of_row, offsets, k, weights, q, s, stream)
PyObject *moe_dispatch_quantize(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &x = tensor(a[0], "x");
    const int dev = device_of(x, "x", 2);
    const CallStream st(a[7], dev);
    const int64_t T = x.size(0), H = x.size(1), k = integer(a[3], "k", 0, kIntMax);
    const void *px = checked(x, "x", kBF16, {T, H}, dev);
    const int64_t cap = tensor(a[1], "slot_of_row").numel(), G = tensor(a[2], "offsets").numel() - 1;
    TORCH_CHECK_VALUE(G <= kIntMax, "offsets is too long");
    const auto *slot = in<int32_t>(a[1], "slot_of_row", kI32, {cap}, dev);
    const auto *off = in<int32_t>(a[2], "offsets", kI32, {G + 1}, dev);
    const auto *w = in_or_null<float>(a[4], "weights", kF32, {T, k}, dev);
    const Tensor q = out(a[5], "q", kU8, {cap, H}, dev);
    const Tensor s = out(a[6], "s", kF32, {blocks(cap), blocks(H)}, dev);
    const Tensor ws = scratch(dg_moe_dispatch_workspace(T, static_cast<int>(k), H, cap), dev);
    status(dg_moe_dispatch_quantize(px, w, slot, off, T, static_cast<int>(k), H, cap, static_cast<int>(G),
                                    ptr<uint8_t>(q), ptr<float>(s), ws.defined() ? ws.data_ptr() : nullptr,
                                    ws.defined() ? ws.numel() : 0, st),
           "dg_moe_dispatch_quantize");
    return wrap_all(q, s);
    END_HANDLE_TH_ERRORS
}

// (x, slot_of_row, masked_m, k, q, s, stream)
PyObject *moe_dispatch_quantize_masked(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &x = tensor(a[0], "x");
    const int dev = device_of(x, "x", 2);
    const CallStream st(a[6], dev);
    const int64_t T = x.size(0), H = x.size(1), k = integer(a[3], "k", 0, kIntMax);
    const void *px = checked(x, "x", kBF16, {T, H}, dev);
    const int64_t G = tensor(a[2], "masked_m").numel(), rows = tensor(a[1], "slot_of_row").numel();
    TORCH_CHECK_VALUE(G >= 1 && G <= kIntMax && rows % G == 0, "slot_of_row must hold the same number of rows for each of ", G,
                      " experts, not ", rows, " in all");
    const int64_t M_max = rows / G;
    const auto *slot = in<int32_t>(a[1], "slot_of_row", kI32, {rows}, dev);
    const auto *m = in<int32_t>(a[2], "masked_m", kI32, {G}, dev);
    const Tensor q = out(a[4], "q", kU8, {G, M_max, H}, dev);
    const Tensor s = out(a[5], "s", kF32, {G, blocks(M_max), blocks(H)}, dev);
    status(dg_moe_dispatch_quantize_masked(px, slot, m, T, static_cast<int>(k), H, static_cast<int>(G), M_max,
                                           ptr<uint8_t>(q), ptr<float>(s), st),
           "dg_moe_dispatch_quantize_masked");
    return wrap_all(q, s);
    END_HANDLE_TH_ERRORS
}

// y as [rows][H], from two or three dimensions.
const void *rows_of(const Tensor &y, int64_t H, int dev, int64_t &rows) {
    TORCH_CHECK_VALUE(y.dim() == 2 || y.dim() == 3, "y must have 2 or 3 dimensions, not ", y.dim());
    TORCH_CHECK_VALUE(y.size(-1) == H, "y must have ", H, " columns, not ", y.size(-1));
    rows = H ? y.numel() / H : 0;
    return checked(y, "y", kBF16, y.sizes(), dev);
}

// (y, row_of_slot, weights, out, stream)
PyObject *moe_combine(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &y = tensor(a[0], "y"), &row = tensor(a[1], "row_of_slot");
    const int dev = device_of(row, "row_of_slot", 2);
    const CallStream st(a[4], dev);
    const int64_t T = row.size(0), k = row.size(1), H = y.dim() ? y.size(-1) : 0;
    TORCH_CHECK_VALUE(k <= kIntMax, "row_of_slot is too wide");
    int64_t rows;
    const void *py = rows_of(y, H, dev, rows);
    const auto *pr = in<int32_t>(a[1], "row_of_slot", kI32, {T, k}, dev);
    const auto *w = in_or_null<float>(a[2], "weights", kF32, {T, k}, dev);
    const Tensor o = out(a[3], "out", kBF16, {T, H}, dev);
    status(dg_moe_combine(py, w, pr, T, static_cast<int>(k), H, rows, ptr(o), st), "dg_moe_combine");
    return wrap(o);
    END_HANDLE_TH_ERRORS
}

// (dout, y, row_of_slot, dweights, stream)
PyObject *moe_combine_backward(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &dout = tensor(a[0], "dout"), &row = tensor(a[2], "row_of_slot");
    const int dev = device_of(dout, "dout", 2);
    const CallStream st(a[4], dev);
    const int64_t T = dout.size(0), H = dout.size(1);
    TORCH_CHECK_VALUE(row.dim() == 2 && row.size(1) <= kIntMax, "row_of_slot must have 2 dimensions");
    const int64_t k = row.size(1);
    const void *pd = checked(dout, "dout", kBF16, {T, H}, dev);
    int64_t rows;
    const void *py = rows_of(tensor(a[1], "y"), H, dev, rows);
    const auto *pr = in<int32_t>(a[2], "row_of_slot", kI32, {T, k}, dev);
    const Tensor dw = out(a[3], "dweights", kF32, {T, k}, dev);
    status(dg_moe_combine_backward(pd, py, pr, T, static_cast<int>(k), H, rows, ptr<float>(dw), st),
           "dg_moe_combine_backward");
    return wrap(dw);
    END_HANDLE_TH_ERRORS
}

// group_offsets or None: the number of experts and the address
const int32_t *groups(PyObject *o, int dev, int64_t &G) {
    G = 0;
    if (o == Py_None) return nullptr;
    G = tensor(o, "offsets").numel() - 1;
    TORCH_CHECK_VALUE(G >= 1 && G <= kIntMax, "offsets must have G + 1 elements, G at least 1");  // an empty one has no address
    return in<int32_t>(o, "offsets", kI32, {G + 1}, dev);
}

// (h, offsets, checkpoint, q, s, h8, sh, stream)
PyObject *swiglu_quantize(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &h = tensor(a[0], "h");
    const int dev = device_of(h, "h", 2);
    const CallStream st(a[7], dev);
    const int64_t M = h.size(0), F = h.size(1) / 2;
    const bool checkpoint = truth(a[2]);
    TORCH_CHECK_VALUE(checkpoint || (a[5] == Py_None && a[6] == Py_None), "h8 and sh are outputs of checkpoint=True");
    const void *ph = checked(h, "h", kBF16, {M, 2 * F}, dev);
    int64_t G;
    const int32_t *off = groups(a[1], dev, G);
    const Tensor q = out(a[3], "q", kU8, {M, F}, dev);
    const Tensor s = out(a[4], "s", kF32, {blocks(M), blocks(F)}, dev);
    if (!checkpoint) {
        status(dg_swiglu_quantize(ph, off, static_cast<int>(G), M, F, ptr<uint8_t>(q), ptr<float>(s), nullptr, nullptr, st),
               "dg_swiglu_quantize");
        return wrap_all(q, s);
    }
    const Tensor h8 = out(a[5], "h8", kU8, {M, 2 * F}, dev);
    const Tensor sh = out(a[6], "sh", kF32, {2 * F / 128, M}, dev);
    status(dg_swiglu_quantize(ph, off, static_cast<int>(G), M, F, ptr<uint8_t>(q), ptr<float>(s), ptr<uint8_t>(h8),
                              ptr<float>(sh), st),
           "dg_swiglu_quantize");
    return wrap_all(q, s, h8, sh);
    END_HANDLE_TH_ERRORS
}

// (h, masked_m, q, s, stream)
PyObject *swiglu_quantize_masked(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &h = tensor(a[0], "h");
    const int dev = device_of(h, "h", 3);
    const CallStream st(a[4], dev);
    const int64_t G = h.size(0), M = h.size(1), F = h.size(2) / 2;
    TORCH_CHECK_VALUE(G <= kIntMax, "h has too many experts");
    const void *ph = checked(h, "h", kBF16, {G, M, 2 * F}, dev);
    const auto *m = in<int32_t>(a[1], "masked_m", kI32, {G}, dev);
    const Tensor q = out(a[2], "q", kU8, {G, M, F}, dev);
    const Tensor s = out(a[3], "s", kF32, {G, blocks(M), blocks(F)}, dev);
    status(dg_swiglu_quantize_masked(ph, m, static_cast<int>(G), M, F, ptr<uint8_t>(q), ptr<float>(s), st),
           "dg_swiglu_quantize_masked");
    return wrap_all(q, s);
    END_HANDLE_TH_ERRORS
}

// (h8, sh, da, offsets, q, s, stream)
PyObject *swiglu_quantize_backward(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &da = tensor(a[2], "da");
    const int dev = device_of(da, "da", 2);
    const CallStream st(a[6], dev);
    const int64_t M = da.size(0), F = da.size(1);
    const auto *h8 = in<uint8_t>(a[0], "h8", kU8, {M, 2 * F}, dev);
    const auto *sh = in<float>(a[1], "sh", kF32, {2 * F / 128, M}, dev);
    const void *pa = checked(da, "da", kBF16, {M, F}, dev);
    int64_t G;
    const int32_t *off = groups(a[3], dev, G);
    const Tensor q = out(a[4], "q", kU8, {M, 2 * F}, dev);
    const Tensor s = out(a[5], "s", kF32, {blocks(M), blocks(2 * F)}, dev);
    status(dg_swiglu_quantize_backward(h8, sh, pa, off, static_cast<int>(G), M, F, ptr<uint8_t>(q), ptr<float>(s), st),
           "dg_swiglu_quantize_backward");
    return wrap_all(q, s);
    END_HANDLE_TH_ERRORS
}

// (dY, sdY, W, sW, offsets or None, C, stream)
PyObject *dgrad(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &dy = tensor(a[0], "dY"), &w = tensor(a[2], "W");
    const int dev = device_of(dy, "dY", 2);
    const CallStream st(a[6], dev);
    const int64_t M = dy.size(0), N = dy.size(1), K = w.dim() ? w.size(-1) : 0;
    const auto *pd = in<uint8_t>(a[0], "dY", kU8, {M, N}, dev);
    const auto *pa = in<float>(a[1], "sdY", kF32, {blocks(M), blocks(N)}, dev);
    int64_t G;
    const int32_t *off = groups(a[4], dev, G);
    const uint8_t *pw;
    const float *pb;
    if (off) {
        pw = in<uint8_t>(a[2], "W", kU8, {G, N, K}, dev);
        pb = in<float>(a[3], "sW", kF32, {G, blocks(N), blocks(K)}, dev);
    } else {
        pw = in<uint8_t>(a[2], "W", kU8, {N, K}, dev);
        pb = in<float>(a[3], "sW", kF32, {blocks(N), blocks(K)}, dev);
    }
    const Tensor c = out(a[5], "C", kBF16, {M, K}, dev);
    if (off)
        status(dg_fp8_grouped_dgrad_contiguous(pd, pa, pw, pb, ptr(c), off, M, static_cast<int>(G), N, K, st),
               "dg_fp8_grouped_dgrad_contiguous");
    else {
        const Tensor ws = scratch(dg_fp8_dgrad_workspace(M, N, K), dev);
        status(dg_fp8_dgrad_blockscaled(pd, pa, pw, pb, ptr(c), M, N, K, ws.defined() ? ws.data_ptr() : nullptr,
                                        ws.defined() ? ws.numel() : 0, st),
               "dg_fp8_dgrad_blockscaled");
    }
    return wrap(c);
    END_HANDLE_TH_ERRORS
}

// (dY, sdY, X, sX, offsets or None, C, accumulate, BF16 wanted: True, False or None, stream)
PyObject *wgrad(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &dy = tensor(a[0], "dY"), &x = tensor(a[2], "X");
    const int dev = device_of(dy, "dY", 2);
    const CallStream st(a[8], dev);
    const int64_t M = dy.size(0), N = dy.size(1), K = x.dim() ? x.size(-1) : 0;
    const auto *pd = in<uint8_t>(a[0], "dY", kU8, {M, N}, dev);
    const auto *pa = in<float>(a[1], "sdY", kF32, {blocks(M), blocks(N)}, dev);
    const auto *px = in<uint8_t>(a[2], "X", kU8, {M, K}, dev);
    const auto *pb = in<float>(a[3], "sX", kF32, {blocks(M), blocks(K)}, dev);
    int64_t G;
    const int32_t *off = groups(a[4], dev, G);
    const bool accumulate = truth(a[6]);
    TORCH_CHECK_VALUE(!accumulate || a[5] != Py_None, "accumulate needs the gradient C that is added to");
    at::ScalarType type = kF32;
    if (a[7] != Py_None) {
        type = truth(a[7]) ? kBF16 : kF32;
    } else if (a[5] != Py_None) {
        type = tensor(a[5], "C").scalar_type();
        TORCH_CHECK_VALUE(type == kF32 || type == kBF16, "a weight gradient is float32 or bfloat16");
    }
    const Tensor c = off ? out(a[5], "C", type, {G, N, K}, dev) : out(a[5], "C", type, {N, K}, dev);
    if (off)
        status(dg_fp8_grouped_wgrad_contiguous(pd, pa, px, pb, ptr(c), type == kF32, accumulate, off, M,
                                               static_cast<int>(G), N, K, st),
               "dg_fp8_grouped_wgrad_contiguous");
    else {
        const Tensor ws = scratch(dg_fp8_wgrad_workspace(M, N, K), dev);
        status(dg_fp8_wgrad_blockscaled(pd, pa, px, pb, ptr(c), type == kF32, accumulate, M, N, K,
                                        ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, st),
               "dg_fp8_wgrad_blockscaled");
    }
    return wrap(c);
    END_HANDLE_TH_ERRORS
}

float number(PyObject *o, const char *name) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw python_error();
    const float f = static_cast<float>(v);
    TORCH_CHECK_VALUE(f - f == 0.0f, name, " must be finite in float32, not ", v);
    return f;
}

// logits [T][G], float32 or bfloat16
const void *scores(const Tensor &z, const char *name, int dev, bool &bf16) {
    bf16 = z.scalar_type() == kBF16;
    return checked(z, name, bf16 ? kBF16 : kF32, {z.size(0), z.size(1)}, dev);
}

// (logits, k, sigmoid, bias, mask, renormalize, scale, balance, topk_ids, weights, counts, loss, dprob, stream)
PyObject *moe_route(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &z = tensor(a[0], "logits");
    const int dev = device_of(z, "logits", 2);
    const CallStream st(a[13], dev);
    const int64_t T = z.size(0), G = z.size(1), k = integer(a[1], "k", 0, kIntMax);
    bool bf16;
    const void *pz = scores(z, "logits", dev, bf16);
    const auto *bias = in_or_null<float>(a[3], "bias", kF32, {G}, dev);
    const uint8_t *mask = nullptr;
    if (a[4] != Py_None) {
        const Tensor &m = tensor(a[4], "mask");
        mask = static_cast<const uint8_t *>(checked(m, "mask", m.scalar_type() == kU8 ? kU8 : at::kBool, {T}, dev));
    }
    const bool balance = truth(a[7]);
    const dg_route_options_t options = {truth(a[2]) ? DG_SCORE_SIGMOID : DG_SCORE_SOFTMAX, truth(a[5]), number(a[6], "scale")};
    TORCH_CHECK_VALUE(balance || (a[10] == Py_None && a[11] == Py_None && a[12] == Py_None),
                      "counts, loss and dprob are outputs of balance=True");
    // the outputs follow k, which no tensor bounds
    if (G < 1 || G > 1024 || k < 1 || k > 32 || k > G) status(DG_ERR_SHAPE, "dg_moe_route");
    const Tensor ids = out(a[8], "topk_ids", kI32, {T, k}, dev);
    const Tensor w = out(a[9], "weights", kF32, {T, k}, dev);
    if (!balance) {
        status(dg_moe_route(pz, bf16, &options, bias, mask, T, static_cast<int>(G), static_cast<int>(k),
                            ptr<int32_t>(ids), ptr<float>(w), nullptr, nullptr, nullptr, nullptr, 0, st),
               "dg_moe_route");
        return wrap_all(ids, w);
    }
    const Tensor counts = out(a[10], "counts", kI32, {G}, dev);
    const Tensor loss = out(a[11], "loss", kF32, {}, dev);
    const Tensor dprob = out(a[12], "dprob", kF32, {G}, dev);
    const Tensor ws = scratch(dg_moe_route_workspace(T, static_cast<int>(G)), dev);
    status(dg_moe_route(pz, bf16, &options, bias, mask, T, static_cast<int>(G), static_cast<int>(k),
                        ptr<int32_t>(ids), ptr<float>(w), ptr<int32_t>(counts), ptr<float>(loss), ptr<float>(dprob),
                        ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, st),
           "dg_moe_route");
    return wrap_all(ids, w, counts, loss, dprob);
    END_HANDLE_TH_ERRORS
}

// (logits, topk_ids, dweights, dprob, dloss, sigmoid, renormalize, scale, dlogits, stream)
PyObject *moe_route_backward(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Tensor &z = tensor(a[0], "logits"), &ids = tensor(a[1], "topk_ids");
    const int dev = device_of(z, "logits", 2);
    const CallStream st(a[9], dev);
    const int64_t T = z.size(0), G = z.size(1);
    bool bf16;
    const void *pz = scores(z, "logits", dev, bf16);
    TORCH_CHECK_VALUE(ids.dim() == 2 && ids.size(1) <= kIntMax && G <= kIntMax, "topk_ids must have 2 dimensions");
    const int64_t k = ids.size(1);
    const auto *pi = in<int32_t>(a[1], "topk_ids", kI32, {T, k}, dev);
    const auto *dw = in_or_null<float>(a[2], "dweights", kF32, {T, k}, dev);
    const auto *dprob = in_or_null<float>(a[3], "dprob", kF32, {G}, dev);
    const auto *dloss = in_or_null<float>(a[4], "dloss", kF32, {}, dev);
    TORCH_CHECK_VALUE((a[3] == Py_None) == (a[4] == Py_None), "dprob and dloss go together");
    const dg_route_options_t options = {truth(a[5]) ? DG_SCORE_SIGMOID : DG_SCORE_SOFTMAX, truth(a[6]), number(a[7], "scale")};
    const Tensor dz = out(a[8], "dlogits", bf16 ? kBF16 : kF32, {T, G}, dev);
    status(dg_moe_route_backward(pz, bf16, &options, pi, dw, dprob, dloss, T, static_cast<int>(G), static_cast<int>(k),
                                 ptr(dz), st),
           "dg_moe_route_backward");
    return wrap(dz);
    END_HANDLE_TH_ERRORS
}

// The inputs that the norms' calls share: x, weight, y, gate and post_weight of a row width.
struct NormInputs {
    int dev;
    int64_t T, H;
    bool bf16;
    const void *x, *y, *weight, *gate, *post;

    NormInputs(PyObject *x_, const char *name, PyObject *weight_, PyObject *y_, PyObject *gate_, PyObject *post_) {
        const Tensor &t = tensor(x_, name), &w = tensor(weight_, "weight");
        dev = device_of(t, name, 2);
        T = t.size(0), H = t.size(1);
        x = checked(t, name, kBF16, {T, H}, dev);
        bf16 = w.scalar_type() == kBF16;  // the vectors are of one type
        const auto type = bf16 ? kBF16 : kF32;
        weight = checked(w, "weight", type, {H}, dev);
        y = in_or_null(y_, "y", kBF16, {T, H}, dev);
        gate = in_or_null(gate_, "gate", type, {H}, dev);
        post = in_or_null(post_, "post_weight", type, {H}, dev);
        TORCH_CHECK_VALUE(y_ != Py_None || (gate_ == Py_None && post_ == Py_None), "gate and post_weight belong to y");
    }
};

// A new reference to a tensor, or None.
PyObject *wrap_or_none(const Tensor &t) {
    if (t.defined()) return wrap(t);
    Py_RETURN_NONE;
}

template <typename... Ts>
PyObject *wrap_some(const Ts &...ts) {
    PyObject *tuple = PyTuple_New(sizeof...(ts));
    if (!tuple) throw python_error();
    Py_ssize_t i = 0;
    (PyTuple_SET_ITEM(tuple, i++, wrap_or_none(ts)), ...);
    return tuple;
}

// (x, weight, y, gate, post_weight, alpha, eps, n, r, rstd, rstd_y, stream)
PyObject *rmsnorm_residual(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const NormInputs in(a[0], "x", a[1], a[2], a[3], a[4]);
    const CallStream st(a[11], in.dev);
    const dg_norm_options_t options = {number(a[5], "alpha"), number(a[6], "eps"), in.bf16};
    TORCH_CHECK_VALUE(a[2] != Py_None || a[8] == Py_None, "r is x itself without y");
    TORCH_CHECK_VALUE(a[4] != Py_None || a[10] == Py_None, "rstd_y belongs to post_weight");
    const Tensor n = out(a[7], "n", kBF16, {in.T, in.H}, in.dev);
    const Tensor r = a[2] == Py_None ? Tensor() : out(a[8], "r", kBF16, {in.T, in.H}, in.dev);
    const Tensor rstd = out(a[9], "rstd", kF32, {in.T}, in.dev);
    const Tensor rstd_y = a[4] == Py_None ? Tensor() : out(a[10], "rstd_y", kF32, {in.T}, in.dev);
    status(dg_rmsnorm_residual(in.x, in.y, in.weight, in.post, in.gate, &options, in.T, in.H, ptr(n),
                               r.defined() ? ptr(r) : nullptr, ptr<float>(rstd),
                               rstd_y.defined() ? ptr<float>(rstd_y) : nullptr, st),
           "dg_rmsnorm_residual");
    return wrap_some(n, r.defined() ? r : tensor(a[0], "x"), rstd, rstd_y);
    END_HANDLE_TH_ERRORS
}

// (x, weight, y, gate, post_weight, alpha, eps, q, s, r, stream)
PyObject *rmsnorm_residual_quantize(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const NormInputs in(a[0], "x", a[1], a[2], a[3], a[4]);
    const CallStream st(a[10], in.dev);
    const dg_norm_options_t options = {number(a[5], "alpha"), number(a[6], "eps"), in.bf16};
    TORCH_CHECK_VALUE(a[2] != Py_None || a[9] == Py_None, "r is x itself without y");
    const Tensor q = out(a[7], "q", kU8, {in.T, in.H}, in.dev);
    const Tensor s = out(a[8], "s", kF32, {blocks(in.H), in.T}, in.dev);
    const Tensor r = a[2] == Py_None ? Tensor() : out(a[9], "r", kBF16, {in.T, in.H}, in.dev);
    status(dg_rmsnorm_residual_quantize(in.x, in.y, in.weight, in.post, in.gate, &options, in.T, in.H,
                                        ptr<uint8_t>(q), ptr<float>(s), r.defined() ? ptr(r) : nullptr, st),
           "dg_rmsnorm_residual_quantize");
    return wrap_some(q, s, r.defined() ? r : tensor(a[0], "x"));
    END_HANDLE_TH_ERRORS
}

// (dn, r, rstd, weight, dr, y, rstd_y, gate, post_weight, alpha, dx, dy, dweight, dgate, dpost_weight, stream)
PyObject *rmsnorm_residual_backward(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const NormInputs v(a[1], "r", a[3], a[5], a[7], a[8]);
    const CallStream st(a[15], v.dev);
    const int dev = v.dev;
    const int64_t T = v.T, H = v.H;
    const auto type = kBF16;
    const void *dn = checked(tensor(a[0], "dn"), "dn", type, {T, H}, dev);
    const auto *rstd = in<float>(a[2], "rstd", kF32, {T}, dev);
    const void *dr = in_or_null(a[4], "dr", type, {T, H}, dev);
    const auto *rstd_y = in_or_null<float>(a[6], "rstd_y", kF32, {T}, dev);
    const bool has_y = a[5] != Py_None, has_gate = a[7] != Py_None, has_post = a[8] != Py_None;
    TORCH_CHECK_VALUE(has_post == (a[6] != Py_None), "post_weight and rstd_y go together");
    TORCH_CHECK_VALUE((has_y || a[11] == Py_None) && (has_gate || a[13] == Py_None) && (has_post || a[14] == Py_None),
                      "dy, dgate and dpost_weight are outputs where y, gate and post_weight are given");
    const dg_norm_options_t options = {number(a[9], "alpha"), 0.0f, v.bf16};
    const Tensor dx = out(a[10], "dx", type, {T, H}, dev);
    const Tensor dy = has_y ? out(a[11], "dy", type, {T, H}, dev) : Tensor();
    const Tensor dw = out(a[12], "dweight", kF32, {H}, dev);
    const Tensor dg = has_gate ? out(a[13], "dgate", kF32, {H}, dev) : Tensor();
    const Tensor dp = has_post ? out(a[14], "dpost_weight", kF32, {H}, dev) : Tensor();
    const Tensor ws = scratch(dg_rmsnorm_residual_backward_workspace(T, H, has_post, has_gate), dev);
    status(dg_rmsnorm_residual_backward(dn, dr, v.x, rstd, v.y, rstd_y, v.weight, v.post, v.gate, &options, T, H,
                                        ptr(dx), has_y ? ptr(dy) : nullptr, ptr<float>(dw),
                                        has_post ? ptr<float>(dp) : nullptr, has_gate ? ptr<float>(dg) : nullptr,
                                        ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, st),
           "dg_rmsnorm_residual_backward");
    return wrap_some(dx, dy, dw, dg, dp);
    END_HANDLE_TH_ERRORS
}

// A sequence of gradients as the C interface's host arrays; `out` None: in place.  The sequences live as long as
// this does: of an iterable that is neither list nor tuple, nobody else may hold the tensors, and their memory must
// not serve for the call's own outputs and scratch.
class Grads {
public:
    std::vector<void *> in, out;
    std::vector<int64_t> sizes;
    std::vector<uint8_t> bf16;
    int dev = -1;  // the tensors', which has to be the current one
    bool in_place = true;

    // Both are iterated over before either is read: an iterator is Python code, which could change the other one.
    Grads(PyObject *grads, PyObject *outs) : g_(grads, "grads"), o_(outs, "out", true) {
        const Py_ssize_t n = g_.size();
        PyObject *const *const g = g_.items();
        in.reserve(n), sizes.reserve(n), bf16.reserve(n);
        for (Py_ssize_t i = 0; i < n; ++i) {
            const Tensor &t = tensor(g[i], "a gradient");
            if (i == 0) dev = device_of(t, "a gradient", t.dim());
            bf16.push_back(t.scalar_type() == kBF16);
            in.push_back(address(t, "a gradient", bf16.back() ? kBF16 : kF32));
            sizes.push_back(t.numel());
        }
        if (n == 0) dev = c10::cuda::current_device();
        if (outs == Py_None) return;
        in_place = false;
        TORCH_CHECK_VALUE(o_.size() == n, "out must hold ", n, " tensors, not ", o_.size());
        out.reserve(n);
        PyObject *const *const o = o_.items();
        for (Py_ssize_t i = 0; i < n; ++i) {
            const Tensor &t = tensor(o[i], "an output"), &like = THPVariable_Unpack(g[i]);
            out.push_back(address(t, "an output", bf16[i] ? kBF16 : kF32));
            TORCH_CHECK_VALUE(t.sizes() == like.sizes(), "an output must have shape ", like.sizes(), ", not ", t.sizes());
        }
    }

    int64_t count() const { return static_cast<int64_t>(in.size()); }
    void *const *outs() const { return in_place ? nullptr : out.data(); }

    // After the launch, on the call's stream: tensors that only this holds are not given out anew before its work is done.
    void launched() const {
        if (!g_.ours() && !o_.ours()) return;
        const auto stream = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(dev));
        for (const Items *list : {&g_, &o_})
            for (Py_ssize_t i = 0; list->ours() && i < list->size(); ++i)
                c10::cuda::CUDACachingAllocator::recordStream(THPVariable_Unpack(list->items()[i]).storage().data_ptr(), stream);
    }

private:
    // checked() without the shape: a step has hundreds of these.
    void *address(const Tensor &t, const char *name, at::ScalarType type) const {
        TORCH_CHECK_VALUE(t.scalar_type() == type, name, " must be ", type, ", not ", t.scalar_type());
        TORCH_CHECK_VALUE(t.is_cuda() && t.get_device() == dev, name, " must be on cuda:", dev,
                          ", the current device and that of the other tensors");
        TORCH_CHECK_VALUE(t.is_contiguous(), name, " must be contiguous (row-major)");
        return t.unsafeGetTensorImpl()->mutable_data();
    }

    class Items {  // the caller's list or tuple, or a list of what an iterable yields; nothing for an optional None
    public:
        Items(PyObject *o, const char *name, bool optional = false) {
            if (optional && o == Py_None) return;
            TORCH_CHECK_TYPE(!THPVariable_Check(o), name, " must be a sequence of tensors");
            held_ = PySequence_Fast(o, "expected a sequence of tensors");
            if (!held_) throw python_error();
            ours_ = held_ != o;
        }
        ~Items() { Py_XDECREF(held_); }
        Items(const Items &) = delete;
        Items &operator=(const Items &) = delete;
        Py_ssize_t size() const { return held_ ? PySequence_Fast_GET_SIZE(held_) : 0; }
        PyObject *const *items() const { return held_ ? PySequence_Fast_ITEMS(held_) : nullptr; }
        bool ours() const { return ours_; }

    private:
        PyObject *held_ = nullptr;
        bool ours_ = false;
    };
    const Items g_, o_;
};

// (grads, norm, stream)
PyObject *grad_norm(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Grads g(a[0], Py_None);
    const CallStream st(a[2], g.dev);
    const Tensor norm = out(a[1], "norm", kF32, {}, g.dev);
    const Tensor ws = scratch(dg_grad_norm_workspace(g.count()), g.dev);
    status(dg_grad_norm(g.in.data(), g.sizes.data(), g.bf16.data(), g.count(), ptr<float>(norm),
                        ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, st),
           "dg_grad_norm");
    g.launched();
    return wrap(norm);
    END_HANDLE_TH_ERRORS
}

// (grads, norm, max_norm, out, stream)
PyObject *grad_clip(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Grads g(a[0], a[3]);
    const CallStream st(a[4], g.dev);
    const auto *norm = in<float>(a[1], "norm", kF32, {}, g.dev);
    const auto limit = number(a[2], "max_norm");
    status(dg_grad_clip(g.in.data(), g.sizes.data(), g.bf16.data(), g.count(), norm, &limit, g.outs(), st), "dg_grad_clip");
    g.launched();
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// (grads, max_norm, out, norm, stream)
PyObject *clip_grad_norm(PyObject *, PyObject *const *a, Py_ssize_t) {
    HANDLE_TH_ERRORS
    const Grads g(a[0], a[2]);
    const CallStream st(a[4], g.dev);
    const auto limit = number(a[1], "max_norm");
    const Tensor norm = out(a[3], "norm", kF32, {}, g.dev);
    const Tensor ws = scratch(dg_grad_norm_workspace(g.count()), g.dev);
    status(dg_grad_norm_clip(g.in.data(), g.sizes.data(), g.bf16.data(), g.count(), &limit, g.outs(), ptr<float>(norm),
                             ws.defined() ? ws.data_ptr() : nullptr, ws.defined() ? ws.numel() : 0, st),
           "dg_grad_norm_clip");
    g.launched();
    return wrap(norm);
    END_HANDLE_TH_ERRORS
}

// (exception class): what a status is raised as
PyObject *set_error(PyObject *, PyObject *cls) {
    Py_INCREF(cls);
    Py_XDECREF(g_error);
    g_error = cls;
    Py_RETURN_NONE;
}

// A function that takes exactly ARGC positional arguments.
template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t), Py_ssize_t ARGC>
PyObject *counted(PyObject *self, PyObject *const *a, Py_ssize_t n) {
    if (n != ARGC) {
        PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", ARGC, n);
        return nullptr;
    }
    return F(self, a, n);
}

#define DG_METHOD(name, argc) \
    {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(&counted<name, argc>)), METH_FASTCALL, nullptr}

PyMethodDef methods[] = {DG_METHOD(moe_sort, 6),
                         DG_METHOD(moe_sort_masked, 7),
                         DG_METHOD(moe_dispatch_quantize, 8),
                         DG_METHOD(moe_dispatch_quantize_masked, 7),
                         DG_METHOD(moe_combine, 5),
                         DG_METHOD(moe_combine_backward, 5),
                         DG_METHOD(swiglu_quantize, 8),
                         DG_METHOD(swiglu_quantize_masked, 5),
                         DG_METHOD(swiglu_quantize_backward, 7),
                         DG_METHOD(dgrad, 7),
                         DG_METHOD(wgrad, 9),
                         DG_METHOD(moe_route, 14),
                         DG_METHOD(moe_route_backward, 10),
                         DG_METHOD(rmsnorm_residual, 12),
                         DG_METHOD(rmsnorm_residual_quantize, 11),
                         DG_METHOD(rmsnorm_residual_backward, 16),
                         DG_METHOD(grad_norm, 3),
                         DG_METHOD(grad_clip, 5),
                         DG_METHOD(clip_grad_norm, 5),
                         {"set_error", set_error, METH_O, nullptr},
                         {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_dgtorch", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__dgtorch(void) { return PyModule_Create(&module); }
