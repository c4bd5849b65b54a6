// Reads what the library needs of a Python list of torch tensors: addresses,
// sizes, types.  A model has hundreds of tensors and an optimizer's call several
// lists of them; the same attributes read from Python take 0.2 us a tensor and list, here 0.01.
//
// Called through ctypes.PyDLL, which holds the interpreter's lock.
#include <torch/csrc/autograd/python_variable.h>

#include <cstdint>

namespace {

enum Problem { kNone = 0, kNoTensor = 1, kDevice = 2, kType = 3, kStrided = 4, kConjugate = 5, kNoList = 6 };

// Codes of include/fno.h, and 4 for bytes.
int type_code(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return 0;
        case at::kBFloat16: return 1;
        case at::kHalf: return 2;
        case at::kComplexFloat: return 3;
        case at::kByte: return 4;
        default: return -1;
    }
}

}  // namespace

// tensors: a list.  Every entry must be a contiguous tensor on one GPU, of a type in
// `types` (bit k: code k); None where `optional` (address and size 0, type -1).
// Writes an address, a number of elements and a type for each, and the device's
// index (-1 for no tensors).  Returns a Problem, its entry's index in *where.
extern "C" int fno_read_tensors(PyObject* tensors, int types, int optional, int64_t* address, int64_t* numel,
                                int32_t* type, int32_t* device, int64_t* where) {
    *device = -1;
    *where = 0;
    if (!PyList_Check(tensors)) return kNoList;
    const Py_ssize_t n = PyList_GET_SIZE(tensors);
    try {
        for (Py_ssize_t i = 0; i < n; ++i) {
            *where = i;
            PyObject* o = PyList_GET_ITEM(tensors, i);
            if (o == Py_None && optional) {
                address[i] = numel[i] = 0;
                type[i] = -1;
                continue;
            }
            if (!THPVariable_Check(o)) return kNoTensor;
            const at::Tensor& t = THPVariable_Unpack(o);
            if (!t.is_cuda()) return kDevice;
            const int on = (int)t.get_device();
            if (*device < 0) *device = on;
            if (on != *device) return kDevice;
            const int code = t.layout() == at::kStrided ? type_code(t.scalar_type()) : -1;
            if (code < 0 || !(types >> code & 1)) return kType;
            if (!t.is_contiguous()) return kStrided;
            if (t.is_conj() || t.is_neg()) return kConjugate;
            address[i] = reinterpret_cast<int64_t>(t.data_ptr());
            numel[i] = t.numel();
            type[i] = code;
        }
    } catch (...) {                 // a tensor without memory
        return kNoTensor;
    }
    return kNone;
}

// Moments of an optimizer against their parameters: float32 of the parameter's
// values (two a complex one), or the bytes of 8-bit ones.  Writes 32 or 8 bits for
// each; returns -1, or the index of the first whose size is another.
extern "C" int64_t fno_read_moments(int64_t count, const int64_t* numel, const int32_t* type, const int64_t* held,
                                    const int32_t* held_type, int32_t* bits) {
    for (int64_t i = 0; i < count; ++i) {
        const int64_t n = numel[i] * (type[i] == 3 ? 2 : 1), blocks = (n + 127) / 128;
        const bool bytes = held_type[i] == 4;
        const int64_t want = bytes ? (129 * blocks + 15) / 16 * 16 : n;
        if ((held_type[i] == 3 ? 2 : 1) * held[i] != want) return i;
        bits[i] = bytes ? 8 : 32;
    }
    return -1;
}
