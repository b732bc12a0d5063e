// tensor_args.cpp -- the binding's argument packer (Python module _tensor_args).
//
// A serving operator's smallest call takes 2 us on the GPU.  In Python the checks of
// one tensor (type, device, shape, contiguity, address) take 0.4 us, and packing
// and a foreign call of the argument struct 0.4 more, so that a call of seven tensors
// spent 5 of its 7.8 us there.  call() does them here, on the tensors themselves:
//
//   call(function, layout, names, device, *values) -> the function's return code
//
// function: the address of an int f(const struct ...*); layout: one character
// per field of the struct, in its order and without padding:
//   B F I U   the address of a contiguous bf16, fp32, int32 or uint8 tensor; takes two
//             values, the tensor and its shape (None: any)
//   b f i u   the same, or None for a null pointer; for u also a number of bytes and the handle of a
//             stream of the current device: the address of as many of that stream's, from torch's
//             allocator, which has them back when the call returns
//   S         the address of a bf16 tensor of any strides, one value
//   q         a 64-bit integer      n   a 32-bit integer      r   an fp32 number
// names: a name for each tensor, in order, for the errors.  A tensor of another type, or
// not contiguous, or not on a GPU raises TypeError; of another shape or on another
// GPU than `device`, or a number out of range, ValueError.
#include <Python.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <torch/csrc/autograd/python_variable.h>

#include <climits>
#include <cstring>
#include <string>

namespace {

constexpr size_t kMaxBytes = 256;

const char* dtype_name(at::ScalarType t) {
    switch (t) {
        case at::kBFloat16: return "torch.bfloat16";
        case at::kFloat: return "torch.float32";
        case at::kInt: return "torch.int32";
        default: return "torch.uint8";
    }
}

// Memory of one call: the work that the call has queued on `stream` is done with it before what the
// stream is given later.
struct CallMemory {
    void* ptr = nullptr;
    ~CallMemory() {
        try {
            if (ptr) c10::cuda::CUDACachingAllocator::raw_delete(ptr);
        } catch (...) {  // after a CUDA error, which the call itself or the next one reports
        }
    }

    // False with a Python error set: torch.OutOfMemoryError, or RuntimeError for any other failure.
    bool allocate(size_t bytes, void* stream) {
        bool out_of_memory = false;
        std::string what;
        try {
            ptr = c10::cuda::CUDACachingAllocator::raw_alloc_with_stream(bytes, (cudaStream_t)stream);
            return true;
        } catch (const c10::OutOfMemoryError& e) {
            out_of_memory = true;
            what = e.what_without_backtrace();
        } catch (const std::exception& e) {
            what = e.what();
        }
        PyObject* torch = out_of_memory ? PyImport_ImportModule("torch") : nullptr;
        PyObject* error = torch ? PyObject_GetAttrString(torch, "OutOfMemoryError") : nullptr;
        if (!PyErr_Occurred()) PyErr_SetString(error ? error : PyExc_RuntimeError, what.c_str());
        Py_XDECREF(error);
        Py_XDECREF(torch);
        return false;
    }
};

// The address of `obj`, checked; false with a Python error set.
bool tensor_address(PyObject* obj, PyObject* shape, at::ScalarType type, bool contiguous, long long device, PyObject* name,
                    uint64_t* out) {
    const at::Tensor* t = THPVariable_Check(obj) ? &THPVariable_Unpack(obj) : nullptr;
    if (!t || t->scalar_type() != type || !t->is_cuda() || (contiguous && !t->is_contiguous())) {
        PyErr_Format(PyExc_TypeError, "%U must be a %sCUDA %s tensor", name, contiguous ? "contiguous " : "", dtype_name(type));
        return false;
    }
    if (shape && shape != Py_None) {
        const auto sizes = t->sizes();
        bool same = PyTuple_Check(shape) && (size_t)PyTuple_GET_SIZE(shape) == sizes.size();
        for (size_t i = 0; same && i < sizes.size(); ++i) {
            const long long n = PyLong_AsLongLong(PyTuple_GET_ITEM(shape, i));
            if (n == -1 && PyErr_Occurred()) return false;
            same = n == sizes[i];
        }
        if (!same) {
            PyObject* got = PyObject_GetAttrString(obj, "shape");
            PyObject* list = got ? PySequence_Tuple(got) : nullptr;
            if (list) PyErr_Format(PyExc_ValueError, "%U must be %R, got %R", name, shape, list);
            Py_XDECREF(list);
            Py_XDECREF(got);
            return false;
        }
    }
    if (t->get_device() != device) {
        PyErr_Format(PyExc_ValueError, "%U must be on cuda:%lld", name, device);
        return false;
    }
    *out = reinterpret_cast<uint64_t>(t->const_data_ptr());
    return true;
}

bool integer(PyObject* obj, long long lo, long long hi, long long* out) {
    PyObject* n = PyNumber_Index(obj);
    if (!n) return false;
    int over = 0;
    *out = PyLong_AsLongLongAndOverflow(n, &over);
    Py_DECREF(n);
    if (PyErr_Occurred()) return false;
    if (over || *out < lo || *out > hi) {
        PyErr_Format(PyExc_ValueError, "%R is out of range", obj);
        return false;
    }
    return true;
}

PyObject* call_checked(PyObject* const* args, Py_ssize_t nargs) {
    if (nargs < 4 || !PyBytes_Check(args[1]) || !PyTuple_Check(args[2])) {
        PyErr_SetString(PyExc_TypeError, "call(function, layout, names, device, *values)");
        return nullptr;
    }
    void* fn = PyLong_AsVoidPtr(args[0]);
    const long long device = PyLong_AsLongLong(args[3]);
    if (PyErr_Occurred()) return nullptr;
    alignas(8) unsigned char block[kMaxBytes];
    size_t at = 0;
    Py_ssize_t next = 4, tensor = 0;
    CallMemory own;
    for (const char* c = PyBytes_AS_STRING(args[1]); *c; ++c) {
        const bool has_shape = std::strchr("BFIUbfiu", *c) != nullptr, strided = *c == 'S';
        if (next + (has_shape ? 2 : 1) > nargs || at + 8 > kMaxBytes) {
            PyErr_SetString(PyExc_TypeError, "too few values, or a layout that is too long");
            return nullptr;
        }
        if (has_shape || strided) {
            PyObject* obj = args[next++];
            PyObject* shape = has_shape ? args[next++] : nullptr;
            if (tensor >= PyTuple_GET_SIZE(args[2])) {
                PyErr_SetString(PyExc_TypeError, "too few names");
                return nullptr;
            }
            PyObject* name = PyTuple_GET_ITEM(args[2], tensor++);
            uint64_t p = 0;
            if (*c == 'u' && PyLong_CheckExact(obj)) {
                const long long n = PyLong_AsLongLong(obj);
                void* stream = n < 0 ? nullptr : PyLong_AsVoidPtr(shape);
                if (PyErr_Occurred()) return nullptr;
                if (n < 0 || own.ptr) {
                    PyErr_SetString(PyExc_ValueError, "one number of bytes, not negative, expected");
                    return nullptr;
                }
                if (!own.allocate((size_t)n, stream)) return nullptr;
                p = reinterpret_cast<uint64_t>(own.ptr);
            } else if (obj != Py_None || strided || (*c >= 'A' && *c <= 'Z')) {
                const char k = *c | 0x20;
                const at::ScalarType type = k == 'f' ? at::kFloat : k == 'i' ? at::kInt : k == 'u' ? at::kByte : at::kBFloat16;
                if (!tensor_address(obj, shape, type, !strided, device, name, &p)) return nullptr;
            }
            std::memcpy(block + at, &p, 8);
            at += 8;
        } else if (*c == 'q') {
            long long n;
            if (!integer(args[next++], LLONG_MIN, LLONG_MAX, &n)) return nullptr;
            std::memcpy(block + at, &n, 8);
            at += 8;
        } else if (*c == 'n') {
            long long n;
            if (!integer(args[next++], INT_MIN, INT_MAX, &n)) return nullptr;
            const int v = (int)n;
            std::memcpy(block + at, &v, 4);
            at += 4;
        } else if (*c == 'r') {
            const double d = PyFloat_AsDouble(args[next++]);
            if (d == -1.0 && PyErr_Occurred()) return nullptr;
            const float v = (float)d;
            std::memcpy(block + at, &v, 4);
            at += 4;
        } else {
            PyErr_Format(PyExc_TypeError, "unknown layout character %c", *c);
            return nullptr;
        }
    }
    if (next != nargs) {
        PyErr_SetString(PyExc_TypeError, "too many values");
        return nullptr;
    }
    int rc;
    Py_BEGIN_ALLOW_THREADS
    rc = reinterpret_cast<int (*)(const void*)>(fn)(block);
    Py_END_ALLOW_THREADS
    return PyLong_FromLong(rc);
}

PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t nargs) {
    try {
        return call_checked(args, nargs);
    } catch (const std::exception& e) {  // a tensor without storage, for example
        PyErr_SetString(PyExc_TypeError, e.what());
        return nullptr;
    }
}

PyMethodDef methods[] = {{"call", (PyCFunction)(void (*)(void))call, METH_FASTCALL, nullptr}, {nullptr, nullptr, 0, nullptr}};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_tensor_args", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__tensor_args(void) { return PyModule_Create(&module); }
