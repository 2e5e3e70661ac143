// tensor_calls.cpp -- the float operators' tensor calls' plain case, from Python
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
#include <ATen/ops/as_strided.h>
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

// ---- e4m3 with a scale per block of 128 --------------------------------------
constexpr int64_t kBlock = 128;

int64_t blocks(int64_t n) { return n / kBlock + (n % kBlock != 0); }

const float *floats(const at::Tensor &t) { return static_cast<const float *>(t.data_ptr()); }
const int32_t *ints(const at::Tensor &t) { return static_cast<const int32_t *>(t.data_ptr()); }

// Operand of `dim` dimensions: codes and scales, its units per row, and the rows that
// share a scale (1 where both readings are the same).
struct BlockOperand {
    const at::Tensor *codes, *scales;
    int64_t units, block_rows;
};
bool block_operand(PyObject *codes, PyObject *scales, int64_t dim, int device, BlockOperand *out)
{
    const at::Tensor *c = tensor_of(codes, device), *s = tensor_of(scales, device);
    if (!c || !s || c->dim() != dim || s->dim() != dim || (c->scalar_type() != at::kFloat8_e4m3fn && c->scalar_type() != at::kByte) ||
        s->scalar_type() != at::kFloat || !c->is_contiguous() || !s->is_contiguous())
        return false;
    const int64_t units = c->size(dim - 1) / kBlock, rows = c->size(dim - 2);
    if (units * kBlock != c->size(dim - 1) || units != s->size(dim - 1) || (dim == 3 && c->size(0) != s->size(0))) return false;
    const int64_t block_rows = s->size(dim - 2) == rows ? 1 : kBlock;
    if (block_rows != 1 && s->size(dim - 2) != blocks(rows)) return false;
    *out = BlockOperand{c, s, units, block_rows};
    return true;
}

// Values of a float type the library reads; their code.
bool value_type(const at::Tensor &t, lpgemm_out_dtype *code)
{
    switch (t.scalar_type()) {
    case at::kFloat: *code = LPGEMM_OUT_F32; return true;
    case at::kBFloat16: *code = LPGEMM_OUT_BF16; return true;
    case at::kHalf: *code = LPGEMM_OUT_F16; return true;
    default: return false;
    }
}

// Rows of values [rows, n], dense along the last dimension.
const at::Tensor *rows_of(PyObject *o, int device, lpgemm_out_dtype *code)
{
    const at::Tensor *x = tensor_of(o, device);
    if (!x || x->dim() != 2 || !value_type(*x, code) || (x->size(1) > 1 && x->stride(1) != 1) || (x->size(0) > 1 && x->stride(0) < x->size(1)))
        return nullptr;
    return x;
}

// A contiguous tensor of a type and two sizes.
const at::Tensor *table_of(PyObject *o, int device, at::ScalarType type, int64_t rows, int64_t n)
{
    const at::Tensor *t = tensor_of(o, device);
    return t && t->scalar_type() == type && t->dim() == 2 && t->size(0) == rows && t->size(1) == n && t->is_contiguous() ? t : nullptr;
}

PyObject *pair(const at::Tensor &a, const at::Tensor &b)
{
    PyObject *both = PyTuple_New(2);
    if (!both) return nullptr;
    PyTuple_SET_ITEM(both, 0, THPVariable_Wrap(a));
    PyTuple_SET_ITEM(both, 1, THPVariable_Wrap(b));
    return both;
}

// A Python int; false for anything else.
bool number(PyObject *o, int64_t *out)
{
    int overflow = 0;
    if (!PyLong_CheckExact(o)) return false;
    *out = PyLong_AsLongLongAndOverflow(o, &overflow);
    return overflow == 0;
}

PyObject *block_quantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    lpgemm_out_dtype code;
    int64_t block_rows;
    const int device = n == 3 ? home(args[0]) : -1;
    const at::Tensor *x = device < 0 ? nullptr : rows_of(args[0], device, &code);
    if (!x || !number(args[1], &block_rows) || (block_rows != 1 && block_rows != kBlock) || !PyBool_Check(args[2])) Py_RETURN_NONE;
    const int64_t rows = x->size(0), K = x->size(1), units = blocks(K);
    const at::Tensor codes = fresh({rows, units * kBlock}, at::kFloat8_e4m3fn, *x);
    const at::Tensor scales = fresh({block_rows == 1 ? rows : blocks(rows), units}, at::kFloat, *x);
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_fp8_block_quantize(x->data_ptr(), code, x->stride(0), block_rows, args[2] == Py_True, bytes(codes),
                                             static_cast<float *>(scales.data_ptr()), rows, K, s);
        }))
        Py_RETURN_NONE;
    return pair(codes, scales);
    END_HANDLE_TH_ERRORS
}

PyObject *block_dequantize(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    BlockOperand a;
    at::ScalarType type;
    lpgemm_out_dtype code;
    int64_t K;
    const int device = n == 4 ? home(args[0]) : -1;
    if (device < 0 || !block_operand(args[0], args[1], 2, device, &a) || !number(args[2], &K) || K < 0 || blocks(K) != a.units ||
        !out_type(args[3], &type, &code))
        Py_RETURN_NONE;
    const int64_t rows = a.codes->size(0);
    const at::Tensor y = fresh({rows, K}, type, *a.codes);
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_fp8_block_dequantize(bytes(*a.codes), floats(*a.scales), a.block_rows, y.data_ptr(), code, rows, K, s);
        }))
        Py_RETURN_NONE;
    return THPVariable_Wrap(y);
    END_HANDLE_TH_ERRORS
}

PyObject *block_product(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    BlockOperand a, b;
    at::ScalarType type;
    lpgemm_out_dtype code;
    const int device = n == 5 ? home(args[0]) : -1;
    if (device < 0 || !block_operand(args[0], args[1], 2, device, &a) || !block_operand(args[2], args[3], 2, device, &b) || a.units != b.units ||
        a.block_rows != 1 || !out_type(args[4], &type, &code))
        Py_RETURN_NONE;
    const int64_t M = a.codes->size(0), N = b.codes->size(0), K = kBlock * a.units;
    const at::Tensor d = fresh({M, N}, type, *a.codes);
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_fp8_block(bytes(*a.codes), floats(*a.scales), bytes(*b.codes), floats(*b.scales), b.block_rows, d.data_ptr(), code, M, N, K, s);
        }))
        Py_RETURN_NONE;
    return THPVariable_Wrap(d);
    END_HANDLE_TH_ERRORS
}

PyObject *block_grouped(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    BlockOperand a, b;
    at::ScalarType type;
    lpgemm_out_dtype code;
    const int device = n == 7 ? home(args[0]) : -1;
    if (device < 0 || !block_operand(args[0], args[1], 2, device, &a) || !block_operand(args[2], args[3], 3, device, &b) || a.units != b.units ||
        a.block_rows != 1 || !out_type(args[6], &type, &code))
        Py_RETURN_NONE;
    const at::Tensor *offsets = tensor_of(args[4], device), *rows = nullptr;
    if (args[5] != Py_None && !(rows = tensor_of(args[5], device))) Py_RETURN_NONE;
    const int64_t E = b.codes->size(0), N = b.codes->size(1), T = a.codes->size(0), K = kBlock * a.units;
    for (const at::Tensor *t : {offsets, rows})
        if (t ? t->scalar_type() != at::kInt || t->dim() != 1 || !t->is_contiguous() : t == offsets) Py_RETURN_NONE;
    if (offsets->size(0) != E + 1) Py_RETURN_NONE;
    const int64_t R = rows ? rows->size(0) : T;
    const at::Tensor d = fresh({R, N}, type, *a.codes);
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_fp8_block_grouped(bytes(*a.codes), floats(*a.scales), T, rows ? ints(*rows) : nullptr, bytes(*b.codes), floats(*b.scales),
                                            b.block_rows, E, ints(*offsets), d.data_ptr(), code, R, N, K, s);
        }))
        Py_RETURN_NONE;
    return THPVariable_Wrap(d);
    END_HANDLE_TH_ERRORS
}

// ---- routing and the sum of a token's experts ---------------------------------
PyObject *route(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    lpgemm_out_dtype code;
    const int device = n == 9 ? home(args[0]) : -1;
    const at::Tensor *x = device < 0 ? nullptr : rows_of(args[0], device, &code), *bias = nullptr;
    int64_t top, score, groups, top_groups, group_top;
    if (!x || !number(args[1], &top) || !number(args[2], &score) || !number(args[4], &groups) || !number(args[5], &top_groups) ||
        !number(args[6], &group_top) || !PyBool_Check(args[7]) || !PyFloat_CheckExact(args[8]))
        Py_RETURN_NONE;
    const int64_t T = x->size(0), E = x->size(1);
    if (args[3] != Py_None) {
        bias = tensor_of(args[3], device);
        if (!bias || bias->scalar_type() != at::kFloat || bias->dim() != 1 || bias->size(0) != E || !bias->is_contiguous()) Py_RETURN_NONE;
    }
    for (const int64_t v : {score, groups, top_groups, group_top})
        if (v < 0 || v > INT32_MAX) Py_RETURN_NONE;
    size_t need = 0;
    if (top < 1 || top > LPGEMM_ROUTE_MAX_TOP || lpgemm_route_workspace_size(T, E, &need) != LPGEMM_OK) Py_RETURN_NONE;
    const lpgemm_route_options options{(int32_t)score, (int32_t)top, (int32_t)groups, (int32_t)top_groups, (int32_t)group_top, args[7] == Py_True,
                                       (float)PyFloat_AS_DOUBLE(args[8])};
    const int64_t R = T * top;
    const at::Tensor all = fresh({3 * R + E + 1}, at::kInt, *x), weights = fresh({T, top}, at::kFloat, *x);
    const at::Tensor space = need ? fresh({(int64_t)need}, at::kByte, *x) : at::Tensor();
    int32_t *p = static_cast<int32_t *>(all.data_ptr());
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_route(x->data_ptr(), code, x->stride(0), bias ? floats(*bias) : nullptr, &options, p, static_cast<float *>(weights.data_ptr()),
                                p + 2 * R, p + 3 * R, p + R, T, E, need ? space.data_ptr() : nullptr, need, s);
        }))
        Py_RETURN_NONE;
    PyObject *five = PyTuple_New(5);
    if (!five) return nullptr;
    PyTuple_SET_ITEM(five, 0, THPVariable_Wrap(at::as_strided(all, {T, top}, {top, 1}, 0)));
    PyTuple_SET_ITEM(five, 1, THPVariable_Wrap(weights));
    PyTuple_SET_ITEM(five, 2, THPVariable_Wrap(at::as_strided(all, {R}, {1}, 2 * R)));
    PyTuple_SET_ITEM(five, 3, THPVariable_Wrap(at::as_strided(all, {E + 1}, {1}, 3 * R)));
    PyTuple_SET_ITEM(five, 4, THPVariable_Wrap(at::as_strided(all, {T, top}, {top, 1}, R)));
    return five;
    END_HANDLE_TH_ERRORS
}

PyObject *combine(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    HANDLE_TH_ERRORS
    lpgemm_out_dtype y_code, code;
    at::ScalarType type;
    const int device = n == 5 ? home(args[0]) : -1;
    const at::Tensor *y = device < 0 ? nullptr : tensor_of(args[0], device), *places = device < 0 ? nullptr : tensor_of(args[1], device);
    if (!y || !places || y->dim() != 2 || !y->is_contiguous() || !value_type(*y, &y_code) || places->dim() != 2 || places->scalar_type() != at::kInt ||
        !places->is_contiguous())
        Py_RETURN_NONE;
    const int64_t T = places->size(0), top = places->size(1), R = y->size(0), N = y->size(1);
    if (args[4] == Py_None) {
        type = y->scalar_type();
        code = y_code;
    } else if (!out_type(args[4], &type, &code)) {
        Py_RETURN_NONE;
    }
    const at::Tensor *weights = nullptr, *residual = nullptr;
    if (args[2] != Py_None && !(weights = table_of(args[2], device, at::kFloat, T, top))) Py_RETURN_NONE;
    if (args[3] != Py_None && !(residual = table_of(args[3], device, type, T, N))) Py_RETURN_NONE;
    const at::Tensor out = fresh({T, N}, type, *y);
    if (!launch(device, [&](hipStream_t s) {
            return lpgemm_combine(y->data_ptr(), y_code, R, ints(*places), weights ? floats(*weights) : nullptr, residual ? residual->data_ptr() : nullptr,
                                  out.data_ptr(), code, T, top, N, s);
        }))
        Py_RETURN_NONE;
    return THPVariable_Wrap(out);
    END_HANDLE_TH_ERRORS
}

#define LPGEMM_FASTCALL(f) reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)(void)>(f)), METH_FASTCALL
PyMethodDef methods[] = {
    {"quantize", LPGEMM_FASTCALL(quantize), "(x) -> (codes, scales) or None"},
    {"dequantize", LPGEMM_FASTCALL(dequantize), "(codes, scales, K, dtype) -> values or None"},
    {"product", LPGEMM_FASTCALL(product), "(A, SFA, B, SFB, dtype) -> D or None"},
    {"grouped", LPGEMM_FASTCALL(grouped), "(A, SFA, B, SFB, offsets, rows, dtype) -> D or None"},
    {"block_quantize", LPGEMM_FASTCALL(block_quantize), "(x, block_rows, power_of_two) -> (codes, scales) or None"},
    {"block_dequantize", LPGEMM_FASTCALL(block_dequantize), "(codes, scales, K, dtype) -> values or None"},
    {"block_product", LPGEMM_FASTCALL(block_product), "(A, SFA, B, SFB, dtype) -> D or None"},
    {"block_grouped", LPGEMM_FASTCALL(block_grouped), "(A, SFA, B, SFB, offsets, rows, dtype) -> D or None"},
    {"route", LPGEMM_FASTCALL(route), "(logits, top, score, bias, groups, top_groups, group_top, renormalise, scale) -> five tensors or None"},
    {"combine", LPGEMM_FASTCALL(combine), "(y, places, weights, residual, dtype) -> sums or None"},
    {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_calls", "The float operators' tensor calls' plain case.", -1, methods,
                      nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_calls() { return PyModule_Create(&module); }
