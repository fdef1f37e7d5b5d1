// Python binding of the readout-tuning calls: checks the tensors, allocates outputs and
// workspace from PyTorch's caching allocator and calls the C ABI on the current stream.
// A C extension rather than ctypes because these calls are small: at 64 replicas the
// kernels take 3-10 us, argument marshalling through ctypes 6-14 us, this 1-3 us.
// Each function returns its tensors, or the status of a refused call as an int.
#include <Python.h>

#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/core/GradMode.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <initializer_list>

#include "../../include/schnet.h"

namespace {

using at::ScalarType;
using at::Tensor;

[[noreturn]] void refuse(const std::string& what) { throw c10::ValueError({__func__, __FILE__, __LINE__}, what); }

// These calls record nothing for autograd: an argument whose gradient would get lost is refused.
const Tensor& tensor(PyObject* o, const char* name)
{
    if (!THPVariable_Check(o)) throw torch::TypeError(std::string(name) + " must be a tensor");
    const Tensor& t = THPVariable_Unpack(o);
    if (t.requires_grad() && c10::GradMode::is_enabled())
        refuse(std::string(name) + " requires grad, and this call forms no autograd graph: detach it, or call under "
                                   "torch.no_grad()");
    return t;
}

// t: a contiguous tensor of that shape on device dev
void check(const char* name, const Tensor& t, int dev, ScalarType dtype, std::initializer_list<int64_t> shape)
{
    if (t.is_cuda() && t.get_device() == dev && t.scalar_type() == dtype && t.is_contiguous() &&
        t.sizes() == at::IntArrayRef(shape.begin(), shape.size()))
        return;
    std::string want;
    for (int64_t s : shape) want += (want.empty() ? "" : ", ") + std::to_string(s);
    refuse(std::string(name) + " must be a contiguous tensor of " + c10::toString(dtype) + " and shape (" + want +
           ") on device " + std::to_string(dev));
}

// the type of stored codes or scales: their own, or plain bytes; any other 8-bit type means other values
ScalarType stored_type(const char* name, const Tensor& t, ScalarType own)
{
    const ScalarType type = t.scalar_type();
    if (type != own && type != ScalarType::Byte)
        refuse(std::string(name) + " must be " + c10::toString(own) + " or Byte, not " + c10::toString(type));
    return type;
}

Tensor make(int dev, ScalarType dtype, std::initializer_list<int64_t> shape)
{
    return at::detail::empty_cuda(at::IntArrayRef(shape.begin(), shape.size()), dtype, c10::Device(c10::kCUDA, dev),
                                  c10::nullopt);
}

template <class T = void>
T* ptr(const Tensor& t)
{
    return static_cast<T*>(t.data_ptr());
}

void* stream_of(int dev) { return c10::cuda::getCurrentCUDAStream(dev).stream(); }

PyObject* results(schnet_status st, std::initializer_list<Tensor> ts)
{
    if (st != SCHNET_OK) return PyLong_FromLong(st);
    PyObject* out = PyTuple_New(ts.size());
    if (!out) return nullptr;
    Py_ssize_t k = 0;
    for (const Tensor& t : ts) PyTuple_SET_ITEM(out, k++, THPVariable_Wrap(t));
    return out;
}

bool arity(Py_ssize_t have, Py_ssize_t want)
{
    if (have == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, have);
    return false;
}

int64_t width(int64_t F) { return (F + 15) / 16 * 16; }

PyObject* store_features(PyObject*, PyObject* const* args, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!arity(n_args, 1)) return nullptr;
    const Tensor& x = tensor(args[0], "x");
    const ScalarType t = x.scalar_type();
    const int dtype = t == ScalarType::Float ? SCHNET_FLOAT32 : t == ScalarType::Half ? SCHNET_FLOAT16 : SCHNET_BFLOAT16;
    if (!x.is_cuda() || x.dim() != 2 || (t != ScalarType::Float && t != ScalarType::Half && t != ScalarType::BFloat16))
        refuse("store_features: x must be a 2-d float32, float16 or bfloat16 CUDA tensor");
    const int64_t n = x.size(0), F = x.size(1), stride = x.stride(0);
    if (n > 0 && (x.stride(1) != 1 || (n > 1 && stride < F)))
        refuse("store_features: columns must be adjacent and rows must not overlap");
    if (F > 128 || F < 2 || (F & 1)) return PyLong_FromLong(SCHNET_ERR_UNSUPPORTED);
    const int dev = x.get_device();
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor codes = make(dev, ScalarType::Float8_e4m3fn, {n, width(F)});
    const Tensor scales = make(dev, ScalarType::Float8_e8m0fnu, {n});
    const schnet_status st = schnet_store_features(x.data_ptr(), dtype, n, (int32_t)F, std::max(stride, F),
                                                   ptr<uint8_t>(codes), ptr<uint8_t>(scales), stream_of(dev));
    return results(st, {codes, scales});
    END_HANDLE_TH_ERRORS
}

// the tensors both readout calls take: codes, scales, replica_offsets, R1, c1, R2, c2
struct ReadoutCall {
    const Tensor &codes, &scales, &off, &R1, &c1, &R2, &c2;
    int dev = -1;
    int64_t n = 0, F = 0, H = 0, R = 0;
    explicit ReadoutCall(PyObject* const* a)
        : codes(tensor(a[0], "codes")), scales(tensor(a[1], "scales")), off(tensor(a[2], "replica_offsets")),
          R1(tensor(a[3], "R1")), c1(tensor(a[4], "c1")), R2(tensor(a[5], "R2")), c2(tensor(a[6], "c2"))
    {
        const ScalarType code_type = stored_type("codes", codes, ScalarType::Float8_e4m3fn);
        const ScalarType scale_type = stored_type("scales", scales, ScalarType::Float8_e8m0fnu);
        if (!codes.is_cuda() || codes.dim() != 2 || R1.dim() != 2 || off.dim() != 1 || c2.numel() != 1)
            refuse("codes [n, width], R1 [F, F / 2], c2 [1] and replica_offsets [R + 1] must be CUDA tensors");
        dev = codes.get_device();
        n = codes.size(0);
        F = R1.size(0);
        H = R1.size(1);
        R = off.size(0) - 1;
        if (F != 2 * H || R < 1 || n >= INT32_MAX || R >= INT32_MAX)
            refuse("R1 must be [F, F / 2]; replica_offsets [R + 1] with R >= 1; fewer than 2^31 atoms and replicas");
        check("codes", codes, dev, code_type, {n, width(F)});
        check("scales", scales, dev, scale_type, {n});
        check("replica_offsets", off, dev, ScalarType::Int, {R + 1});
        check("R1", R1, dev, ScalarType::Float, {F, H});
        check("c1", c1, dev, ScalarType::Float, {H});
        check("R2", R2, dev, ScalarType::Float, {H});
        if (!c2.is_cuda() || c2.get_device() != dev || c2.scalar_type() != ScalarType::Float)
            refuse("c2 must be one float32 on the device of codes");
    }
};

PyObject* readout_energy(PyObject*, PyObject* const* args, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!arity(n_args, 7)) return nullptr;
    const ReadoutCall c(args);
    size_t size = 0;
    schnet_status st = schnet_readout_workspace_bytes((int32_t)c.n, (int32_t)c.F, &size);
    if (st != SCHNET_OK) return PyLong_FromLong(st);
    const c10::cuda::CUDAGuard guard(c.dev);
    const Tensor energy = make(c.dev, ScalarType::Float, {c.R}), eps = make(c.dev, ScalarType::Float, {c.n});
    const Tensor ws = make(c.dev, ScalarType::Byte, {(int64_t)size});
    st = schnet_readout_energy(ptr<uint8_t>(c.codes), ptr<uint8_t>(c.scales), (int32_t)c.n, (int32_t)c.F, (int32_t)c.R,
                               ptr<int32_t>(c.off), ptr<float>(c.R1), ptr<float>(c.c1), ptr<float>(c.R2),
                               ptr<float>(c.c2), ptr<float>(energy), ptr<float>(eps), ptr(ws), size, stream_of(c.dev));
    return results(st, {energy, eps});
    END_HANDLE_TH_ERRORS
}

PyObject* readout_gradients(PyObject*, PyObject* const* args, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!arity(n_args, 8)) return nullptr;
    const Tensor& g = tensor(args[7], "grad_energy");
    const ReadoutCall c(args);
    check("grad_energy", g, c.dev, ScalarType::Float, {c.R});
    size_t size = 0;
    schnet_status st = schnet_readout_workspace_bytes((int32_t)c.n, (int32_t)c.F, &size);
    if (st != SCHNET_OK) return PyLong_FromLong(st);
    const c10::cuda::CUDAGuard guard(c.dev);
    const Tensor d1 = make(c.dev, ScalarType::Float, {c.F, c.H}), d2 = make(c.dev, ScalarType::Float, {c.H});
    const Tensor d3 = make(c.dev, ScalarType::Float, {c.H}), d4 = make(c.dev, ScalarType::Float, {1});
    const Tensor ws = make(c.dev, ScalarType::Byte, {(int64_t)size});
    st = schnet_readout_gradients(ptr<uint8_t>(c.codes), ptr<uint8_t>(c.scales), (int32_t)c.n, (int32_t)c.F,
                                  (int32_t)c.R, ptr<int32_t>(c.off), ptr<float>(c.R1), ptr<float>(c.c1),
                                  ptr<float>(c.R2), ptr<float>(c.c2), ptr<float>(g), ptr<float>(d1), ptr<float>(d2),
                                  ptr<float>(d3), ptr<float>(d4), ptr(ws), size, stream_of(c.dev));
    return results(st, {d1, d2, d3, d4});
    END_HANDLE_TH_ERRORS
}

// energy, pairs, reference or None, flags or None, kT, smoothing
PyObject* preference_loss(PyObject*, PyObject* const* args, Py_ssize_t n_args)
{
    HANDLE_TH_ERRORS
    if (!arity(n_args, 6)) return nullptr;
    const Tensor &energy = tensor(args[0], "energy"), &pairs = tensor(args[1], "pairs");
    const Tensor* ref = args[2] == Py_None ? nullptr : &tensor(args[2], "reference");
    const Tensor* bits = args[3] == Py_None ? nullptr : &tensor(args[3], "flags");
    if (bits && bits->scalar_type() != ScalarType::Int && bits->scalar_type() != ScalarType::UInt32)
        refuse("flags must be one 32-bit integer on the energies' device");
    const ScalarType t = energy.scalar_type();
    if (!energy.is_cuda() || energy.dim() != 1 || energy.size(0) < 1 || !energy.is_contiguous() ||
        (t != ScalarType::Float && t != ScalarType::Double))
        refuse("energy must be a contiguous float32 or float64 CUDA tensor [R]");
    if (pairs.dim() != 2) refuse("pairs must be [P, 2]");
    const int dev = energy.get_device();
    const int64_t R = energy.size(0), P = pairs.size(0);
    if (R >= INT32_MAX || P >= INT32_MAX) refuse("fewer than 2^31 replicas and pairs");
    check("pairs", pairs, dev, ScalarType::Int, {P, 2});
    const void* reference = nullptr;
    if (ref) {
        check("reference", *ref, dev, t, {R});
        reference = ref->data_ptr();
    }
    uint32_t* flags = nullptr;
    if (bits) {
        if (!bits->is_cuda() || bits->get_device() != dev || bits->numel() != 1)
            refuse("flags must be one 32-bit integer on the energies' device");
        flags = ptr<uint32_t>(*bits);
    }
    const double kT = PyFloat_AsDouble(args[4]), smoothing = PyFloat_AsDouble(args[5]);
    if (PyErr_Occurred()) return nullptr;
    size_t size = 0;
    schnet_status st = schnet_preference_workspace_bytes((int32_t)R, P, &size);
    if (st != SCHNET_OK) return PyLong_FromLong(st);
    const c10::cuda::CUDAGuard guard(dev);
    const Tensor loss = make(dev, ScalarType::Double, {}), margins = make(dev, ScalarType::Float, {P});
    const Tensor grad = make(dev, ScalarType::Float, {R}), ws = make(dev, ScalarType::Byte, {(int64_t)size});
    st = schnet_preference_loss(energy.data_ptr(), reference, t == ScalarType::Float ? SCHNET_FLOAT32 : SCHNET_FLOAT64,
                                (int32_t)R, ptr<int32_t>(pairs), P, kT, smoothing, ptr<double>(loss),
                                ptr<float>(margins), ptr<float>(grad), flags, ptr(ws), size, stream_of(dev));
    return results(st, {loss, margins, grad});
    END_HANDLE_TH_ERRORS
}

template <class F>
PyCFunction fast(F* f)
{
    return reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(f));
}

PyMethodDef methods[] = {
    {"store_features", fast(store_features), METH_FASTCALL, nullptr},
    {"readout_energy", fast(readout_energy), METH_FASTCALL, nullptr},
    {"readout_gradients", fast(readout_gradients), METH_FASTCALL, nullptr},
    {"preference_loss", fast(preference_loss), METH_FASTCALL, nullptr},
    {nullptr, nullptr, 0, nullptr},
};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_binding", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__binding() { return PyModule_Create(&module); }
