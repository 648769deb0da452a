// The NVFP4 and expert-routing calls on PyTorch tensors: checks of types,
// shapes and places, new outputs, the current stream, and one call of the C ABI
// (include/ts_nvfp4_moe.h).
//
// A decoded token's operator runs for 2 to 6 us on the GPU, and the same
// marshalling through ctypes took 6 to 18 us of the calling thread on the
// node's CPU; here it takes 2 to 5, of which letting go of the interpreter and
// taking it back is 0.06 to 0.2.  The documented functions are those of
// _nvfp4_moe.py, which pass their arguments on by position.
#define PY_SSIZE_T_CLEAN
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/cuda/EmptyTensor.h>
#include <ATen/ops/empty.h>
#include <c10/cuda/CUDAFunctions.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/autograd/python_variable.h>

#include "ts_nvfp4_moe.h"

namespace {

// Thrown with a Python error set.
struct Raised {};

[[noreturn]] void raise(PyObject *type, const char *format, ...)
{
    va_list ap;
    va_start(ap, format);
    PyErr_FormatV(type, format, ap);
    va_end(ap);
    throw Raised{};
}

// The interpreter is left to other threads: a launch may wait for room in its queue,
// an allocation for the device.
class Unlocked {
public:
    Unlocked() : state_(PyEval_SaveThread()) {}
    ~Unlocked() { PyEval_RestoreThread(state_); }
    Unlocked(const Unlocked &) = delete;
    Unlocked &operator=(const Unlocked &) = delete;

private:
    PyThreadState *state_;
};

// A shape to compare with or to say.
struct Dims {
    int64_t d[3];
    int n;
    at::IntArrayRef ref() const { return {d, (size_t)n}; }
};
Dims dims(int64_t a) { return {{a}, 1}; }
Dims dims(int64_t a, int64_t b) { return {{a, b}, 2}; }
Dims dims(int64_t a, int64_t b, int64_t c) { return {{a, b, c}, 3}; }

constexpr at::ScalarType kU8 = at::kByte, kI32 = at::kInt, kF32 = at::kFloat, kBF16 = at::kBFloat16;

const char *type_name(at::ScalarType t)
{
    switch (t) {
    case kU8: return "torch.uint8";
    case kI32: return "torch.int32";
    case kF32: return "torch.float32";
    case kBF16: return "torch.bfloat16";
    default: return at::toString(t);
    }
}

// One call: its arguments, the device they are on, and what it allocates.
class Call {
public:
    Call(PyObject *const *args, Py_ssize_t n, Py_ssize_t want) : args_(args), n_(n)
    {
        if (n != want)
            raise(PyExc_TypeError, "%zd arguments, %zd are wanted", n, want);
        PyObject *stream = args[n - 1];
        if (stream != Py_None) {  // a torch.cuda.Stream or a raw handle
            PyObject *raw = PyObject_HasAttrString(stream, "cuda_stream") ? PyObject_GetAttrString(stream, "cuda_stream")
                                                                          : PyNumber_Index(stream);
            if (raw == nullptr)
                throw Raised{};
            stream_ = static_cast<cudaStream_t>(PyLong_AsVoidPtr(raw));
            Py_DECREF(raw);
            if (PyErr_Occurred())
                throw Raised{};
            given_ = true;
        }
    }

    bool none(int i) const { return args_[i] == Py_None; }

    int64_t integer(int i) const
    {
        PyObject *v = PyNumber_Index(args_[i]);
        if (v == nullptr)
            throw Raised{};
        const long long x = PyLong_AsLongLong(v);
        Py_DECREF(v);
        if (x == -1 && PyErr_Occurred())
            throw Raised{};
        return x;
    }

    // A scale-factor layout.  Refused here: the shapes of outputs follow it, and
    // a wider integer must not become another layout on its way to the library.
    int layout(int i) const
    {
        const int64_t v = integer(i);
        if (v == TS_SF_SWIZZLED_128x4 || v == TS_SF_SWIZZLED_8x4 || v == TS_SF_LINEAR)
            return (int)v;
        const std::string detail = "sf_layout " + std::to_string(v) + " is not a QuantizationSFLayout code";
        PyObject *module = PyImport_ImportModule("reduce_residual_rmsnorm_gb300._binding");
        PyObject *type = module == nullptr ? nullptr : PyObject_GetAttrString(module, "TsError");
        PyObject *error = type == nullptr ? nullptr
                                          : PyObject_CallFunction(type, "iss", TS_ERR_BAD_PATTERN,
                                                                  ts_status_string(TS_ERR_BAD_PATTERN), detail.c_str());
        if (error != nullptr)
            PyErr_SetObject(type, error);
        Py_XDECREF(error);
        Py_XDECREF(type);
        Py_XDECREF(module);
        throw Raised{};
    }

    // A tensor that the kernels can address, of a type.
    const at::Tensor &tensor(int i, const char *name, at::ScalarType type)
    {
        if (!THPVariable_Check(args_[i]))
            raise(PyExc_TypeError, "%s must be a CUDA tensor or a pinned host tensor", name);
        const at::Tensor &t = THPVariable_Unpack(args_[i]);
        if (t.is_cuda()) {
            const int d = t.get_device();
            if (device_ >= 0 && d != device_)
                raise(PyExc_ValueError, "tensors on different devices: cuda:%d, cuda:%d", device_, d);
            device_ = d;
        } else if (!t.device().is_cpu() || !t.is_pinned()) {
            raise(PyExc_TypeError, "%s must be a CUDA tensor or a pinned host tensor", name);
        }
        if (t.scalar_type() != type)
            raise(PyExc_TypeError, "%s must be %s, got %s", name, type_name(type), type_name(t.scalar_type()));
        return t;
    }

    static void shape(const at::Tensor &t, const char *name, const Dims &want)
    {
        if (t.sizes() != want.ref()) {
            std::string w, g;
            for (int64_t v : want.ref())
                w += std::to_string(v) + ", ";
            for (int64_t v : t.sizes())
                g += std::to_string(v) + ", ";
            raise(PyExc_ValueError, "%s must have shape (%s), got (%s)", name, w.c_str(), g.c_str());
        }
    }

    const at::Tensor &flat(int i, const char *name, at::ScalarType type)
    {
        const at::Tensor &t = tensor(i, name, type);
        if (!t.is_contiguous())
            raise(PyExc_ValueError, "%s must be contiguous", name);
        return t;
    }

    const at::Tensor &flat(int i, const char *name, at::ScalarType type, const Dims &want)
    {
        const at::Tensor &t = flat(i, name, type);
        shape(t, name, want);
        return t;
    }

    // In device memory: the tensor copy engine reads it.
    const at::Tensor &on_gpu(int i, const char *name, at::ScalarType type)
    {
        const at::Tensor &t = flat(i, name, type);
        if (!t.is_cuda())
            raise(PyExc_TypeError, "%s must be a CUDA tensor", name);
        return t;
    }

    // A bf16 matrix with unit column stride; its row stride.
    const at::Tensor &matrix(int i, const char *name, int64_t *ld)
    {
        const at::Tensor &t = tensor(i, name, kBF16);
        if (t.dim() != 2 || (t.size(1) > 1 && t.stride(1) != 1))
            raise(PyExc_ValueError, "%s must be 2-D with unit column stride", name);
        *ld = t.stride(0);
        if (t.size(0) <= 1)  // a single row has no stride that matters; torch may report any
            *ld = (t.size(1) + 7) / 8 * 8;
        return t;
    }

    // The output of a product, which the tensor copy engine writes.
    at::Tensor product_output(int i, int64_t rows, int64_t cols, const at::Tensor &like, int64_t *ld)
    {
        const at::Tensor t = matrix_output(i, "out", rows, cols, like, ld);
        if (!t.is_cuda())
            raise(PyExc_TypeError, "out must be a CUDA tensor");
        return t;
    }

    const float *one(int i, const char *name)
    {
        const at::Tensor &t = tensor(i, name, kF32);
        if (t.numel() != 1)
            raise(PyExc_ValueError, "%s must hold one value", name);
        return static_cast<const float *>(t.data_ptr());
    }

    const int32_t *optional_i32(int i, const char *name, const Dims &want)
    {
        return none(i) ? nullptr : static_cast<const int32_t *>(flat(i, name, kI32, want).data_ptr());
    }

    // A new contiguous tensor where `like` lives, from the memory of the stream
    // that writes it: another stream's free memory may still be in use there.
    at::Tensor fresh(const Dims &d, at::ScalarType type, const at::Tensor &like) const
    {
        const Unlocked unlocked;
        if (like.is_cuda()) {
            if (!given_)
                return at::detail::empty_cuda(d.ref(), type, like.device(), std::nullopt);
            const c10::DeviceIndex device = like.device().index();
            const c10::cuda::CUDAStreamGuard guard(stream_ == nullptr
                                                       ? c10::cuda::getDefaultCUDAStream(device)
                                                       : c10::cuda::getStreamFromExternal(stream_, device));
            return at::detail::empty_cuda(d.ref(), type, like.device(), std::nullopt);
        }
        return at::empty(d.ref(), at::TensorOptions().dtype(type).pinned_memory(true));
    }

    // A contiguous tensor on part of another's storage.
    static at::Tensor part_of(const at::Tensor &all, int64_t offset, const Dims &d)
    {
        at::Tensor t = at::detail::make_tensor<c10::TensorImpl>(c10::Storage(all.storage()), all.key_set(), all.dtype());
        t.unsafeGetTensorImpl()->set_storage_offset(offset);
        t.unsafeGetTensorImpl()->set_sizes_contiguous(d.ref());
        return t;
    }

    // NVFP4 codes and scale factors, given or new; small new ones share an allocation,
    // which takes 0.7 us of the thread.
    std::pair<at::Tensor, at::Tensor> nvfp4_outputs(int i, const Dims &q, const Dims &s, const at::Tensor &like)
    {
        const int64_t at = (c10::multiply_integers(q.ref()) + 255) / 256 * 256, all = at + c10::multiply_integers(s.ref());
        if (!none(i) || !none(i + 1) || all > 65536)
            return {output(i, "quant_out", kU8, q, like), output(i + 1, "scale_out", kU8, s, like)};
        const at::Tensor both = fresh(dims(all), kU8, like);
        return {part_of(both, 0, q), part_of(both, at, s)};
    }

    // The output that is given, checked, or a new one.
    at::Tensor output(int i, const char *name, at::ScalarType type, const Dims &want, const at::Tensor &like)
    {
        return none(i) ? fresh(want, type, like) : flat(i, name, type, want);
    }

    at::Tensor matrix_output(int i, const char *name, int64_t rows, int64_t cols, const at::Tensor &like, int64_t *ld)
    {
        if (none(i)) {
            *ld = cols;
            return fresh(dims(rows, cols), kBF16, like);
        }
        const at::Tensor &t = matrix(i, name, ld);
        shape(t, name, dims(rows, cols));
        return t;
    }

    // Run `call(flags, stream)` with the tensors' device current; the last two
    // arguments are launch_with_pdl and stream.
    template <typename F>
    void run(F &&call)
    {
        const int pdl = PyObject_IsTrue(args_[n_ - 2]);
        if (pdl < 0)
            throw Raised{};
        const int now = c10::cuda::current_device();
        const int device = device_ < 0 ? now : device_;
        void *stream = given_ ? stream_ : c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)device).stream();
        const uint32_t flags = pdl ? TS_FLAG_PDL : 0u;
        int status;
        {
            const Unlocked unlocked;
            if (device == now) {
                status = call(flags, stream);
            } else {
                const c10::cuda::CUDAGuard guard((c10::DeviceIndex)device);
                status = call(flags, stream);
            }
        }
        if (status != TS_OK)
            failed(status);
    }

    [[noreturn]] static void failed(int status)
    {
        PyObject *module = PyImport_ImportModule("reduce_residual_rmsnorm_gb300._binding");
        PyObject *none = module == nullptr ? nullptr : PyObject_CallMethod(module, "_check", "i", status);
        Py_XDECREF(none);
        Py_XDECREF(module);
        if (!PyErr_Occurred())
            PyErr_Format(PyExc_RuntimeError, "status %d", status);
        throw Raised{};
    }

private:
    PyObject *const *args_;
    Py_ssize_t n_;
    int device_ = -1;
    cudaStream_t stream_ = nullptr;
    bool given_ = false;
};

Dims sf_dims(int64_t T, int64_t K, int layout)
{
    if (layout == TS_SF_LINEAR)
        return dims(T, K / 16);
    const int64_t tile = layout == TS_SF_SWIZZLED_128x4 ? 128 : 8;
    return dims((T + tile - 1) / tile * tile, (K / 16 + 3) / 4 * 4);
}

template <typename T = void>
T *ptr(const at::Tensor &t)
{
    return static_cast<T *>(t.data_ptr());
}

// x, scale_factor, row_src, quant_out, scale_out, sf_layout, pdl, stream
PyObject *quantize(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 8);
    const int layout = c.layout(5);
    int64_t ldx;
    const at::Tensor &x = c.matrix(0, "x", &ldx);
    const int64_t T = x.size(0), K = x.size(1);
    const float *g = c.one(1, "scale_factor");
    const int32_t *src = c.optional_i32(2, "row_src", dims(T));
    const auto [q, s] = c.nvfp4_outputs(3, dims(T, K / 2), sf_dims(T, K, layout), x);
    void *const qp = ptr(q), *const sp = ptr(s);
    c.run([&](uint32_t flags, void *stream) {
        return ts_nvfp4_quantize(ptr(x), T, K, ldx, g, src, qp, sp, layout, flags, stream);
    });
    return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(s));
}

// quant, scale, scale_factor, sf_layout, row_src, out, pdl, stream
PyObject *dequantize(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 8);
    const int layout = c.layout(3);
    const at::Tensor &q = c.flat(0, "quant", kU8);
    if (q.dim() != 2)
        raise(PyExc_ValueError, "quant must be [T, K/2]");
    const int64_t T = q.size(0), K = 2 * q.size(1);
    const at::Tensor &s = c.flat(1, "scale", kU8, sf_dims(T, K, layout));
    const float *g = c.one(2, "scale_factor");
    const int32_t *src = c.optional_i32(4, "row_src", dims(T));
    int64_t ldo;
    const at::Tensor out = c.matrix_output(5, "out", T, K, q, &ldo);
    c.run([&](uint32_t flags, void *stream) {
        return ts_nvfp4_dequantize(ptr(q), ptr(s), layout, T, K, g, src, ptr(out), ldo, flags, stream);
    });
    return THPVariable_Wrap(out);
}

// a, a_scale, b, b_scale, alpha, out, pdl, stream
PyObject *gemm(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 8);
    const at::Tensor &a = c.on_gpu(0, "a", kU8), &b = c.on_gpu(2, "b", kU8);
    if (a.dim() != 2 || b.dim() != 2 || a.size(1) != b.size(1))
        raise(PyExc_ValueError, "a must be [M, K/2] and b [N, K/2]");
    const int64_t M = a.size(0), N = b.size(0), K = 2 * a.size(1);
    const at::Tensor &as = c.on_gpu(1, "a_scale", kU8), &bs = c.on_gpu(3, "b_scale", kU8);
    Call::shape(as, "a_scale", sf_dims(M, K, TS_SF_SWIZZLED_128x4));
    Call::shape(bs, "b_scale", sf_dims(N, K, TS_SF_SWIZZLED_128x4));
    const float *alpha = c.one(4, "alpha");
    int64_t ldo;
    const at::Tensor out = c.product_output(5, M, N, a, &ldo);
    c.run([&](uint32_t flags, void *stream) {
        return ts_nvfp4_gemm(ptr(a), ptr(as), ptr(b), ptr(bs), alpha, M, N, K, ptr(out), ldo, flags, stream);
    });
    return THPVariable_Wrap(out);
}

// expert_ids, num_experts, row_align, row_of, row_src, expert_start, expert_count, pdl, stream; the four None for new ones
PyObject *sort(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 9);
    const at::Tensor &ids = c.flat(0, "expert_ids", kI32);
    if (ids.dim() != 2)
        raise(PyExc_ValueError, "expert_ids must be [T, k]");
    const int64_t T = ids.size(0), k = ids.size(1), E = c.integer(1), align = c.integer(2);
    const bool fresh = c.none(3);
    int64_t rows = 0;
    if (fresh) {
        rows = ts_moe_rows(T, k, E, align);
        if (rows < 0)
            raise(PyExc_ValueError, "ts_moe_rows: T=%lld, k=%lld, num_experts=%lld, row_align=%lld out of range", (long long)T,
                  (long long)k, (long long)E, (long long)align);
    }
    if (E < 0 || E > (1 << 20))
        raise(PyExc_ValueError, "num_experts out of range");
    at::Tensor of, src, start, count;
    if (fresh) {  // parts of one allocation, each on a 256-byte boundary
        const Dims d[4] = {dims(T, k), dims(rows), dims(E + 1), dims(E)};
        int64_t at[5] = {0};
        for (int i = 0; i < 4; ++i)
            at[i + 1] = at[i] + (c10::multiply_integers(d[i].ref()) + 63) / 64 * 64;
        const at::Tensor all = c.fresh(dims(at[4]), kI32, ids);
        at::Tensor *const part[4] = {&of, &src, &start, &count};
        for (int i = 0; i < 4; ++i)
            *part[i] = Call::part_of(all, at[i], d[i]);
    } else {
        of = c.flat(3, "rows.row_of", kI32, dims(T, k));
        src = c.flat(4, "rows.row_src", kI32);
        start = c.flat(5, "rows.expert_start", kI32, dims(E + 1));
        count = c.flat(6, "rows.expert_count", kI32, dims(E));
    }
    c.run([&](uint32_t flags, void *stream) {
        return ts_moe_sort(ptr<int32_t>(ids), T, k, E, align, src.numel(), ptr<int32_t>(of), ptr<int32_t>(src),
                           ptr<int32_t>(start), ptr<int32_t>(count), flags, stream);
    });
    return Py_BuildValue("(NNNN)", THPVariable_Wrap(of), THPVariable_Wrap(src), THPVariable_Wrap(start),
                         THPVariable_Wrap(count));
}

const at::Tensor &row_of(Call &c, int i)
{
    const at::Tensor &of = c.flat(i, "rows.row_of", kI32);
    if (of.dim() != 2)
        raise(PyExc_ValueError, "rows.row_of must be [T, k]");
    return of;
}

// x, row_of, rows, scale_factor, out, quant_out, scale_out, sf_layout, pdl, stream
PyObject *dispatch(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 10);
    const bool fp4 = !c.none(3);
    const int layout = fp4 ? c.layout(7) : TS_SF_LINEAR;  // (the bf16 form has none)
    int64_t ldx;
    const at::Tensor &x = c.matrix(0, "x", &ldx);
    const int64_t T = x.size(0), H = x.size(1), rows = c.integer(2);
    const at::Tensor &of = row_of(c, 1);
    if (of.size(0) != T)
        raise(PyExc_ValueError, "rows.row_of must be [T, k]");
    if (!fp4) {
        if (!c.none(5) || !c.none(6))
            raise(PyExc_ValueError, "quant_out and scale_out need scale_factor");
        const at::Tensor out = c.output(4, "out", kBF16, dims(rows, H), x);
        c.run([&](uint32_t flags, void *stream) {
            return ts_moe_dispatch(ptr(x), T, H, ldx, ptr<int32_t>(of), of.size(1), rows, ptr(out), nullptr, nullptr, nullptr,
                                   layout, flags, stream);
        });
        return THPVariable_Wrap(out);
    }
    if (!c.none(4))
        raise(PyExc_ValueError, "out and scale_factor exclude each other");
    const float *g = c.one(3, "scale_factor");
    const auto [q, s] = c.nvfp4_outputs(5, dims(rows, H / 2), sf_dims(rows, H, layout), x);
    void *const qp = ptr(q), *const sp = ptr(s);
    c.run([&](uint32_t flags, void *stream) {
        return ts_moe_dispatch(ptr(x), T, H, ldx, ptr<int32_t>(of), of.size(1), rows, nullptr, g, qp, sp, layout, flags,
                               stream);
    });
    return Py_BuildValue("(NN)", THPVariable_Wrap(q), THPVariable_Wrap(s));
}

// a, a_scale, b, b_scale, alpha, expert_start, expert_count, entries, out, pdl, stream
PyObject *grouped_gemm(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 11);
    const at::Tensor &a = c.on_gpu(0, "a", kU8), &b = c.on_gpu(2, "b", kU8);
    if (a.dim() != 2 || b.dim() != 3 || a.size(1) != b.size(2))
        raise(PyExc_ValueError, "a must be [rows, K/2] and b [E, N, K/2]");
    const int64_t rows = a.size(0), K = 2 * a.size(1), E = b.size(0), N = b.size(1);
    const at::Tensor &as = c.on_gpu(1, "a_scale", kU8), &bs = c.on_gpu(3, "b_scale", kU8);
    const Dims sf = sf_dims(N, K, TS_SF_SWIZZLED_128x4);
    Call::shape(as, "a_scale", sf_dims(rows, K, TS_SF_SWIZZLED_128x4));
    Call::shape(bs, "b_scale", dims(E, sf.d[0], sf.d[1]));
    const at::Tensor &alpha = c.flat(4, "alpha", kF32, dims(E));
    const at::Tensor &start = c.flat(5, "rows.expert_start", kI32, dims(E + 1));
    const at::Tensor &count = c.flat(6, "rows.expert_count", kI32, dims(E));
    const int64_t entries = c.integer(7);
    int64_t ldo;
    const at::Tensor out = c.product_output(8, rows, N, a, &ldo);
    c.run([&](uint32_t flags, void *stream) {
        return ts_nvfp4_grouped_gemm(ptr(a), ptr(as), ptr(b), ptr(bs), ptr<float>(alpha), ptr<int32_t>(start),
                                     ptr<int32_t>(count), E, rows, entries, N, K, ptr(out), ldo, flags, stream);
    });
    return THPVariable_Wrap(out);
}

// y, row_of, weights, out, pdl, stream
PyObject *combine(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 6);
    int64_t ldy, ldo;
    const at::Tensor &y = c.matrix(0, "y", &ldy);
    const at::Tensor &of = row_of(c, 1);
    const int64_t rows = y.size(0), H = y.size(1), T = of.size(0), k = of.size(1);
    const float *w = c.none(2) ? nullptr : ptr<float>(c.flat(2, "weights", kF32, dims(T, k)));
    const at::Tensor out = c.matrix_output(3, "out", T, H, y, &ldo);
    c.run([&](uint32_t flags, void *stream) {
        return ts_moe_combine(ptr(y), rows, H, ldy, ptr<int32_t>(of), w, T, k, ptr(out), ldo, flags, stream);
    });
    return THPVariable_Wrap(out);
}

// dout, y, row_of, weights, dy, dweights, pdl, stream
PyObject *combine_grad(PyObject *const *args, Py_ssize_t n)
{
    Call c(args, n, 8);
    int64_t ldd, ldy, lddy;
    const at::Tensor &d = c.matrix(0, "dout", &ldd), &y = c.matrix(1, "y", &ldy);
    const at::Tensor &of = row_of(c, 2);
    const int64_t rows = y.size(0), H = y.size(1), T = of.size(0), k = of.size(1);
    Call::shape(d, "dout", dims(T, H));
    const at::Tensor &w = c.flat(3, "weights", kF32, dims(T, k));
    const at::Tensor dy = c.matrix_output(4, "dy", rows, H, y, &lddy);
    const at::Tensor dw = c.output(5, "dweights", kF32, dims(T, k), y);
    c.run([&](uint32_t flags, void *stream) {
        return ts_moe_combine_grad(ptr(d), ldd, ptr(y), ldy, rows, H, ptr<int32_t>(of), ptr<float>(w), T, k, ptr(dy), lddy,
                                   ptr<float>(dw), flags, stream);
    });
    return Py_BuildValue("(NN)", THPVariable_Wrap(dy), THPVariable_Wrap(dw));
}

// No C++ exception leaves a call.
template <PyObject *(*F)(PyObject *const *, Py_ssize_t)>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n)
{
    try {
        return F(args, n);
    } catch (const Raised &) {
    } catch (const c10::OutOfMemoryError &e) {
        PyObject *torch = PyImport_ImportModule("torch");
        PyObject *type = torch == nullptr ? nullptr : PyObject_GetAttrString(torch, "OutOfMemoryError");
        if (type != nullptr)
            PyErr_SetString(type, e.what_without_backtrace());
        Py_XDECREF(type);
        Py_XDECREF(torch);
    } catch (const c10::Error &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what_without_backtrace());
    } catch (const std::exception &e) {
        PyErr_SetString(PyExc_RuntimeError, e.what());
    }
    return nullptr;
}

#define TS_METHOD(name) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(entry<name>)), METH_FASTCALL, nullptr}
PyMethodDef methods[] = {TS_METHOD(quantize), TS_METHOD(dequantize),   TS_METHOD(gemm),    TS_METHOD(sort),
                         TS_METHOD(dispatch), TS_METHOD(grouped_gemm), TS_METHOD(combine), TS_METHOD(combine_grad),
                         {nullptr, nullptr, 0, nullptr}};
PyModuleDef module_def = {PyModuleDef_HEAD_INIT, "_python_calls", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__python_calls(void) { return PyModule_Create(&module_def); }
