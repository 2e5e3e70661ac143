// tensor_calls.cpp -- the microscaled tensor calls' plain case, from Python
// straight to the C entry points (module _tensor_calls).
//
// A call for one token's work spends longer in the interpreter than on the
// device, so the plain case (dense operands on the current device, results
// allocated here, the current stream) is checked, allocated and launched
// here.  Every function returns None for anything else, wrong arguments
// included: the caller then goes the long way, which says what is wrong.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <c10/hip/HIPFunctions.h>
#include <c10/hip/HIPStream.h>

#include "lpgemm.h"

namespace {

constexpr int64_t kUnit = 128, kUnitCodes = 64, kUnitScales = 4;

// The device of a plain tensor object on the current device, else -1.
int home(PyObject *o)
{
    if (!THPVariable_CheckExact(o) || !THPVariable_Unpack(o).is_cuda()) return -1;
    const int device = THPVariable_Unpack(o).get_device();
    return device == c10::hip::current_device() ? device : -1;
}

// The tensor of a plain tensor object on `device`, else null.
const at::Tensor *tensor_of(PyObject *o, int device)
{
    if (!THPVariable_CheckExact(o)) return nullptr;
    const at::Tensor &t = THPVariable_Unpack(o);
    return t.is_cuda() && t.get_device() == device && t.layout() == at::kStrided ? &t : nullptr;
}

// Operand of `dim` dimensions: codes and scales; its units per row, or -1.
struct Operand {
    const at::Tensor *codes, *scales;
    int64_t units;
};
bool operand_of(PyObject *codes, PyObject *scales, int64_t dim, int device, Operand *out)
{
    const at::Tensor *c = tensor_of(codes, device), *s = tensor_of(scales, device);
    if (!c || !s || c->dim() != dim || s->dim() != dim || c->scalar_type() != at::kByte || s->scalar_type() != at::kByte ||
        !c->is_contiguous() || !s->is_contiguous())
        return false;
    const int64_t units = c->size(dim - 1) / kUnitCodes;
    if (units * kUnitCodes != c->size(dim - 1) || units * kUnitScales != s->size(dim - 1)) return false;
    for (int64_t i = 0; i + 1 < dim; ++i)
        if (c->size(i) != s->size(i)) return false;
    *out = Operand{c, s, units};
    return true;
}

// Result type of a dtype object (None: bf16).
bool out_type(PyObject *dtype, at::ScalarType *type, lpgemm_out_dtype *code)
{
    *type = dtype == Py_None ? at::kBFloat16 : THPDtype_Check(dtype) ? reinterpret_cast<THPDtype *>(dtype)->scalar_type : at::kByte;
    switch (*type) {
    case at::kFloat: *code = LPGEMM_OUT_F32; return true;
    case at::kBFloat16: *code = LPGEMM_OUT_BF16; return true;
    case at::kHalf: *code = LPGEMM_OUT_F16; return true;
    default: return false;
    }
}

at::Tensor fresh(at::IntArrayRef sizes, at::ScalarType type, const at::Tensor &like)
{
    return at::empty(sizes, at::TensorOptions().dtype(type).device(like.device()));
}

// A call of the library without the interpreter's lock.
template <typename Call>
bool launch(int device, Call call)
{
    const hipStream_t stream = c10::hip::getCurrentHIPStream((c10::DeviceIndex)device).stream();
    PyThreadState *state = PyEval_SaveThread();
    const lpgemm_status status = call(stream);
    PyEval_RestoreThread(state);
    return status == LPGEMM_OK;
}

uint8_t *bytes(const at::Tensor &t) { return static_cast<uint8_t *>(t.data_ptr()); }

PyObject *quantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    if (n != 1) Py_RETURN_NONE;
    const int device = home(args[0]);
    if (device < 0) Py_RETURN_NONE;
    const at::Tensor *x = tensor_of(args[0], device);
    if (!x || x->dim() != 2) Py_RETURN_NONE;
    lpgemm_out_dtype code;
    switch (x->scalar_type()) {
    case at::kFloat: code = LPGEMM_OUT_F32; break;
    case at::kBFloat16: code = LPGEMM_OUT_BF16; break;
    case at::kHalf: code = LPGEMM_OUT_F16; break;
    default: Py_RETURN_NONE;
    }
    const int64_t rows = x->size(0), K = x->size(1), ldx = x->stride(0);
    if ((K > 1 && x->stride(1) != 1) || (rows > 1 && ldx < K)) Py_RETURN_NONE;
    const int64_t units = (K + kUnit - 1) / kUnit;
    const at::Tensor codes = fresh({rows, units * kUnitCodes}, at::kByte, *x), scales = fresh({rows, units * kUnitScales}, at::kByte, *x);
    if (!launch(device, [&](hipStream_t s) { return lpgemm_mxfp4_quantize(x->data_ptr(), code, ldx, bytes(codes), bytes(scales), rows, K, s); }))
        Py_RETURN_NONE;
    PyObject *pair = PyTuple_New(2);
    if (!pair) return nullptr;
    PyTuple_SET_ITEM(pair, 0, THPVariable_Wrap(codes));
    PyTuple_SET_ITEM(pair, 1, THPVariable_Wrap(scales));
    return pair;
    END_HANDLE_TH_ERRORS
}

PyObject *dequantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Operand a;
    at::ScalarType type;
    lpgemm_out_dtype code;
    const int device = n == 4 ? home(args[0]) : -1;
    if (device < 0 || !operand_of(args[0], args[1], 2, device, &a) || !PyLong_CheckExact(args[2]) || !out_type(args[3], &type, &code))
        Py_RETURN_NONE;
    int overflow = 0;
    const int64_t rows = a.codes->size(0), K = PyLong_AsLongLongAndOverflow(args[2], &overflow);
    if (overflow || K < 0 || (K / kUnit + (K % kUnit != 0)) != a.units) Py_RETURN_NONE;
    const at::Tensor y = fresh({rows, K}, type, *a.codes);
    if (!launch(device, [&](hipStream_t s) { return lpgemm_mxfp4_dequantize(bytes(*a.codes), bytes(*a.scales), y.data_ptr(), code, rows, K, s); }))
        Py_RETURN_NONE;
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *product(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Operand a, b;
    at::ScalarType type;
    lpgemm_out_dtype code;
    const int device = n == 5 ? home(args[0]) : -1;
    if (device < 0 || !operand_of(args[0], args[1], 2, device, &a) || !operand_of(args[2], args[3], 2, device, &b) || a.units != b.units ||
        !out_type(args[4], &type, &code))
        Py_RETURN_NONE;
    const int64_t M = a.codes->size(0), N = b.codes->size(0), K = kUnit * a.units;
    const at::Tensor d = fresh({M, N}, type, *a.codes);
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_mxfp4(bytes(*a.codes), bytes(*a.scales), bytes(*b.codes), bytes(*b.scales), d.data_ptr(), code, M, N, K, nullptr, 0, s);
        }))
        Py_RETURN_NONE;
    return THPVariable_Wrap(d);
    END_HANDLE_TH_ERRORS
}

PyObject *grouped(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    Operand a, b;
    at::ScalarType type;
    lpgemm_out_dtype code;
    const int device = n == 7 ? home(args[0]) : -1;
    if (device < 0 || !operand_of(args[0], args[1], 2, device, &a) || !operand_of(args[2], args[3], 3, device, &b) || a.units != b.units ||
        !out_type(args[6], &type, &code))
        Py_RETURN_NONE;
    const at::Tensor *offsets = tensor_of(args[4], device), *rows = nullptr;
    if (args[5] != Py_None && !(rows = tensor_of(args[5], device))) Py_RETURN_NONE;
    const int64_t E = b.codes->size(0), N = b.codes->size(1), T = a.codes->size(0), K = kUnit * a.units;
    for (const at::Tensor *t : {offsets, rows})
        if (t ? t->scalar_type() != at::kInt || t->dim() != 1 || !t->is_contiguous() : t == offsets) Py_RETURN_NONE;
    if (offsets->size(0) != E + 1) Py_RETURN_NONE;
    const int64_t R = rows ? rows->size(0) : T;
    const at::Tensor d = fresh({R, N}, type, *a.codes);
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_mxfp4_grouped(bytes(*a.codes), bytes(*a.scales), T, rows ? static_cast<const int32_t *>(rows->data_ptr()) : nullptr,
                                        bytes(*b.codes), bytes(*b.scales), E, static_cast<const int32_t *>(offsets->data_ptr()), d.data_ptr(),
                                        code, R, N, K, s);
        }))
        Py_RETURN_NONE;
    return THPVariable_Wrap(d);
    END_HANDLE_TH_ERRORS
}

#define LPGEMM_FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"quantize", LPGEMM_FASTCALL(quantize), "(x) -> (codes, scales) or None"},
    {"dequantize", LPGEMM_FASTCALL(dequantize), "(codes, scales, K, dtype) -> values or None"},
    {"product", LPGEMM_FASTCALL(product), "(A, SFA, B, SFB, dtype) -> D or None"},
    {"grouped", LPGEMM_FASTCALL(grouped), "(A, SFA, B, SFB, offsets, rows, dtype) -> D or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", "The microscaled tensor calls' plain case.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&module); }
