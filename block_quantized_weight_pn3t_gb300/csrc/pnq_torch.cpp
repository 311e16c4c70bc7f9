// pnq_torch.cpp -- the torch wrappers of the 4-bit operands and the expert layer (module _native): checks of the tensors,
// allocation of the results, and one call of the C ABI. No arithmetic happens here, and no autograd: results require no
// gradient whatever the inputs do; expert_gather and expert_combine have their gradients as calls of their own.
//
// These calls run several times per layer of a decode step, each a few microseconds of GPU work. Through ctypes and
// Python an encode cost the host some 8 us, of which the launch is two; here the checks read the tensors' fields
// directly.
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDACachingAllocator.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>

#include <cstdint>
#include <optional>
#include <string>

#include "pnq.h"

namespace {

PyObject* g_error = nullptr;  // PnqError of the package

// ---- errors ---------------------------------------------------------------------------------------

// Raised inside, turned into PnqError(what) or PnqError(what, status) at the entry.
struct Refusal {
    std::string what;
    int status;  // 0: none
};

[[noreturn]] void refuse(const std::string& what, int status = 0) { throw Refusal{what, status}; }

void check(int rc, const char* call) {
    if (rc != PNQ_OK) throw Refusal{call, rc};
}

void raise(const Refusal& r) {
    PyObject* e = r.status ? PyObject_CallFunction(g_error, "si", r.what.c_str(), r.status)
                           : PyObject_CallFunction(g_error, "s", r.what.c_str());
    if (e) PyErr_SetObject(g_error, e);
    Py_XDECREF(e);
}

struct PythonError {};  // a Python exception is set already

// Runs body() as the body of a Python entry: refusals, Python's own errors and torch's become Python exceptions.
template <class F>
PyObject* entry(F&& body) {
    HANDLE_TH_ERRORS
    try {
        return body();
    } catch (const Refusal& r) {
        raise(r);
    } catch (const PythonError&) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// ---- arguments --------------------------------------------------------------------------------------

// Positional and keyword arguments of a call, by the names' places; missing ones are null.
template <size_t N>
struct Args {
    PyObject* v[N] = {};
    Args(const char* call, const char* const (&names)[N], size_t required, PyObject* const* args, Py_ssize_t nargs,
         PyObject* kwnames) {
        if (static_cast<size_t>(nargs) > N) fail(call, "too many arguments");
        for (Py_ssize_t i = 0; i < nargs; ++i) v[i] = args[i];
        const Py_ssize_t nk = kwnames ? PyTuple_GET_SIZE(kwnames) : 0;
        for (Py_ssize_t k = 0; k < nk; ++k) {
            PyObject* key = PyTuple_GET_ITEM(kwnames, k);
            size_t at = 0;
            while (at < N && PyUnicode_CompareWithASCIIString(key, names[at]) != 0) ++at;
            if (at == N || v[at]) fail(call, "an unexpected or repeated keyword");
            v[at] = args[nargs + k];
        }
        for (size_t i = 0; i < N; ++i) {
            if (v[i] == Py_None) v[i] = nullptr;
            if (i < required && !v[i]) fail(call, names[i]);
        }
    }
    static void fail(const char* call, const char* what) {
        PyErr_Format(PyExc_TypeError, "%s(): bad arguments (%s)", call, what);
        throw PythonError{};
    }
    PyObject* operator[](size_t i) const { return v[i]; }
};

int64_t to_int(PyObject* o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw PythonError{};
    return v;
}

int to_type(PyObject* o) {
    if (PyLong_Check(o)) {
        const int64_t v = to_int(o);
        if (v == PNQ_NVFP4 || v == PNQ_MXFP4) return static_cast<int>(v);
    }
    refuse("this type is not a 4-bit microscaled format", PNQ_ERR_TYPE);
}

double to_double(PyObject* o) {
    const double v = PyFloat_AsDouble(o);
    if (v == -1.0 && PyErr_Occurred()) throw PythonError{};
    return v;
}

std::string shape_text(at::IntArrayRef s) {
    std::string t = "(";
    for (size_t i = 0; i < s.size(); ++i) t += (i ? ", " : "") + std::to_string(s[i]);
    return t + ")";
}

const at::Tensor& tensor(PyObject* o, const char* what) {
    if (!o || !THPVariable_Check(o)) refuse(std::string(what) + " must be a torch.Tensor");
    return THPVariable_Unpack(o);
}

int float_type(at::ScalarType t, const char* what) {
    if (t == at::kFloat) return PNQ_F32;
    if (t == at::kBFloat16) return PNQ_BF16;
    refuse(std::string(what) + " has dtype " + at::toString(t) + "; expected float32 or bfloat16");
}

at::ScalarType dtype_of(PyObject* o, at::ScalarType otherwise) {
    if (!o) return otherwise;
    if (!THPDtype_Check(o)) refuse("dtype must be a torch.dtype");
    return reinterpret_cast<THPDtype*>(o)->scalar_type;
}

// t is a contiguous CUDA tensor of `dtype` that holds at least `numel` elements.
void require(const at::Tensor& t, const char* what, at::ScalarType dtype, int64_t numel) {
    if (t.scalar_type() != dtype)
        refuse(std::string(what) + " has dtype " + at::toString(t.scalar_type()) + "; expected " + at::toString(dtype));
    if (!t.is_contiguous()) refuse(std::string(what) + " must be contiguous");
    if (t.numel() < numel)
        refuse(std::string(what) + " holds " + std::to_string(t.numel()) + " elements; the call needs " + std::to_string(numel));
    if (!t.is_cuda()) refuse(std::string(what) + " must be a CUDA tensor");
}

void require_device(const at::Tensor& t, const char* what, int device) {
    if (t.get_device() != device)
        refuse(std::string(what) + " is on cuda:" + std::to_string(t.get_device()) + "; the other tensors are on cuda:" +
               std::to_string(device));
}

// t is a contiguous [rows][cols] tensor of `dtype` on CUDA device `device`.
void require_matrix(const at::Tensor& t, const char* what, at::ScalarType dtype, int64_t rows, int64_t cols, int device) {
    if (t.dim() != 2 || t.size(0) != rows || t.size(1) != cols)
        refuse(std::string(what) + " has shape " + shape_text(t.sizes()) + "; expected (" + std::to_string(rows) + ", " +
               std::to_string(cols) + ")");
    require(t, what, dtype, 0);
    require_device(t, what, device);
}

// The device and stream of a call: the tensors' device, and the given stream or that device's current one. On a stream
// other than the current one, results are allocated there, and the tensors named by record() are kept from
// reuse until the work on it is done (they belong to another stream's pool).
class Place {
public:
    Place(PyObject* stream, int device) : guard_(static_cast<c10::DeviceIndex>(device)) {
        const auto current = c10::cuda::getCurrentCUDAStream(static_cast<c10::DeviceIndex>(device));
        stream_ = current.stream();
        if (!stream) return;
        PyObject* h = PyObject_GetAttrString(stream, "cuda_stream");
        if (!h) throw PythonError{};
        void* p = PyLong_AsVoidPtr(h);
        Py_DECREF(h);
        if (!p && PyErr_Occurred()) throw PythonError{};
        if (p == stream_) return;
        stream_ = static_cast<cudaStream_t>(p);
        const auto other = c10::cuda::getStreamFromExternal(stream_, static_cast<c10::DeviceIndex>(device));
        other_.emplace(other);
    }
    cudaStream_t stream() const { return stream_; }
    template <class... Tensors>
    void record(const Tensors&... t) const {
        if (other_) (record_one(t), ...);
    }

private:
    void record_one(const at::Tensor& t) const {
        if (t.defined()) c10::cuda::CUDACachingAllocator::recordStream(t.storage().data_ptr(), other_->current_stream());
    }
    c10::cuda::CUDAGuard guard_;
    cudaStream_t stream_;
    std::optional<c10::cuda::CUDAStreamGuard> other_;
};

// A new CUDA tensor (from torch's caching allocator, without the dispatcher on the way).
at::Tensor new_tensor(at::IntArrayRef sizes, at::ScalarType dtype, int device) {
    return at::Tensor(at::detail::empty_cuda(sizes, dtype, c10::Device(c10::kCUDA, static_cast<c10::DeviceIndex>(device)),
                                             std::nullopt));
}

at::Tensor new_matrix(int64_t rows, int64_t cols, at::ScalarType dtype, int device) {
    return new_tensor({rows, cols}, dtype, device);
}

// A contiguous view of `count` elements of a buffer (a buffer of integers: nothing differentiates through it). Made
// directly: the first narrow() of a new tensor took 5 us, a view made here 0.3.
at::Tensor view_of(const at::Tensor& buffer, int64_t first, at::IntArrayRef sizes) {
    auto impl = c10::make_intrusive<c10::TensorImpl>(c10::TensorImpl::VIEW, c10::Storage(buffer.storage()), buffer.key_set(),
                                                     buffer.dtype());
    impl->set_storage_offset(buffer.storage_offset() + first);
    impl->set_sizes_contiguous(sizes);
    return at::Tensor(std::move(impl));
}

PyObject* wrap(at::Tensor t) { return THPVariable_Wrap(std::move(t)); }

// ---- ExpertPlan ---------------------------------------------------------------------------------------

struct PlanObject {
    PyObject_HEAD
    int64_t rows;  // tokens * slots
    int device;
    pnq_expert_plan desc;
    at::Tensor buffer;
};

extern PyTypeObject PlanType;

// Lays the arrays of a plan out in its buffer.
void lay_out(PlanObject* p, int64_t tokens, int64_t slots, int64_t experts, at::Tensor buffer) {
    int32_t* at = buffer.data_ptr<int32_t>();
    p->rows = tokens * slots;
    p->device = buffer.get_device();
    p->desc.offsets = at;
    p->desc.block_start = at + experts + 1;
    p->desc.order = p->desc.block_start + experts + 1;
    p->desc.position = p->desc.order + p->rows;
    p->desc.scale_row = p->desc.position + p->rows;
    p->desc.tokens = tokens;
    p->desc.slots = static_cast<int32_t>(slots);
    p->desc.experts = static_cast<int32_t>(experts);
    p->buffer = std::move(buffer);
}

void check_plan_shape(int64_t tokens, int64_t slots, int64_t experts) {
    if (slots < 1 || slots > 64 || experts < 1 || experts > 1024 || tokens < 0 || tokens > (int64_t(1) << 30) / slots)
        refuse(std::to_string(tokens) + " tokens, " + std::to_string(slots) + " slots, " + std::to_string(experts) +
                   " experts; 1..64 slots, 1..1024 experts and at most 2^30 choices are wanted",
               PNQ_ERR_SHAPE);
}

int64_t plan_size(int64_t tokens, int64_t slots, int64_t experts) { return 2 * (experts + 1) + 3 * tokens * slots; }

PlanObject* new_plan(int64_t tokens, int64_t slots, int64_t experts, int device) {
    at::Tensor buffer = new_tensor({plan_size(tokens, slots, experts)}, at::kInt, device);
    PlanObject* p = reinterpret_cast<PlanObject*>(PlanType.tp_alloc(&PlanType, 0));
    if (!p) throw PythonError{};
    new (&p->buffer) at::Tensor();
    lay_out(p, tokens, slots, experts, std::move(buffer));
    return p;
}

PyObject* plan_vectorcall(PyObject*, PyObject* const* args, size_t nargsf, PyObject* kwnames) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"tokens", "slots", "experts", "buffer", "device"};
        const Args<5> a("ExpertPlan", names, 3, args, PyVectorcall_NARGS(nargsf), kwnames);
        const int64_t tokens = to_int(a[0]), slots = to_int(a[1]), experts = to_int(a[2]);
        check_plan_shape(tokens, slots, experts);
        if (!a[3]) {
            int device = c10::cuda::current_device();
            if (a[4]) {
                PyObject* index = PyObject_GetAttrString(a[4], "index");
                if (!index) throw PythonError{};
                const bool none = index == Py_None;
                if (!none) device = static_cast<int>(PyLong_AsLong(index));
                Py_DECREF(index);
                if (PyErr_Occurred()) throw PythonError{};
            }
            return reinterpret_cast<PyObject*>(new_plan(tokens, slots, experts, device));
        }
        const at::Tensor& t = tensor(a[3], "plan buffer");
        require(t, "plan buffer", at::kInt, plan_size(tokens, slots, experts));
        PlanObject* p = reinterpret_cast<PlanObject*>(PlanType.tp_alloc(&PlanType, 0));
        if (!p) throw PythonError{};
        new (&p->buffer) at::Tensor();
        lay_out(p, tokens, slots, experts, t);
        return reinterpret_cast<PyObject*>(p);
    });
}

void plan_dealloc(PyObject* self) {
    reinterpret_cast<PlanObject*>(self)->buffer.~Tensor();
    Py_TYPE(self)->tp_free(self);
}

PlanObject* to_plan(PyObject* o) {
    if (!o || Py_TYPE(o) != &PlanType) refuse("plan must be an ExpertPlan");
    return reinterpret_cast<PlanObject*>(o);
}

template <int WHICH>
PyObject* plan_part(PyObject* self, void*) {
    return entry([&]() -> PyObject* {
        const PlanObject* p = reinterpret_cast<PlanObject*>(self);
        const int64_t e = p->desc.experts + 1, n = p->rows;
        const int64_t first[] = {0, e, 2 * e, 2 * e + n, 2 * e + 2 * n}, count[] = {e, e, n, n, n};
        return wrap(view_of(p->buffer, first[WHICH], {count[WHICH]}));
    });
}

PyObject* plan_buffer(PyObject* self, void*) {
    return entry([&]() -> PyObject* { return wrap(reinterpret_cast<PlanObject*>(self)->buffer); });
}
PyObject* plan_tokens(PyObject* self, void*) { return PyLong_FromLongLong(reinterpret_cast<PlanObject*>(self)->desc.tokens); }
PyObject* plan_slots(PyObject* self, void*) { return PyLong_FromLong(reinterpret_cast<PlanObject*>(self)->desc.slots); }
PyObject* plan_experts(PyObject* self, void*) { return PyLong_FromLong(reinterpret_cast<PlanObject*>(self)->desc.experts); }
PyObject* plan_rows(PyObject* self, void*) { return PyLong_FromLongLong(reinterpret_cast<PlanObject*>(self)->rows); }

PyGetSetDef plan_getset[] = {
    {"tokens", plan_tokens, nullptr, "tokens of the layer", nullptr},
    {"slots", plan_slots, nullptr, "choices per token", nullptr},
    {"experts", plan_experts, nullptr, "experts of the layer", nullptr},
    {"rows", plan_rows, nullptr, "sorted rows there is room for: tokens * slots", nullptr},
    {"buffer", plan_buffer, nullptr, "the int32 buffer", nullptr},
    {"offsets", plan_part<0>, nullptr, "[experts + 1] first sorted row of each expert", nullptr},
    {"block_start", plan_part<1>, nullptr, "[experts + 1] first 128-row scale block of each expert", nullptr},
    {"order", plan_part<2>, nullptr, "[rows] slot number of each sorted row, -1 past the rows in use", nullptr},
    {"position", plan_part<3>, nullptr, "[rows] sorted row of each slot, -1 for a dropped one", nullptr},
    {"scale_row", plan_part<4>, nullptr, "[rows] row of each sorted row in the tiled scales", nullptr},
    {nullptr, nullptr, nullptr, nullptr, nullptr}};

PyTypeObject PlanType = {PyVarObject_HEAD_INIT(nullptr, 0)};

// ---- Fp4Matrix -----------------------------------------------------------------------------------------

struct MatrixObject {
    PyObject_HEAD
    int type, device;
    int64_t rows, K, matrices;
    double scale;          // global multiplier, where `scales_of` is not defined
    uint8_t *codes_at, *scales_at;
    int64_t pitch, scale_bytes;
    PyObject* plan;        // the PlanObject whose rows it holds, or null
    at::Tensor codes, scales;  // apart, or codes undefined and `scales` the one buffer of both
    at::Tensor per_matrix;     // fp32 [matrices] global multipliers, or undefined
};

extern PyTypeObject MatrixType;

void layout_of(int type, int64_t rows, int64_t K, int64_t matrices, int64_t plan_experts, int64_t* pitch, int64_t* bytes) {
    uint64_t p = 0, n = 0;
    check(pnq_fp4_layout(type, rows, K, matrices, plan_experts, &p, &n), "pnq_fp4_layout");
    *pitch = static_cast<int64_t>(p);
    *bytes = static_cast<int64_t>(n);
}

MatrixObject* alloc_matrix(int type, int64_t rows, int64_t K, int64_t matrices, PyObject* plan) {
    int64_t pitch = 0, bytes = 0;
    layout_of(type, rows, K, matrices, plan ? reinterpret_cast<PlanObject*>(plan)->desc.experts : 0, &pitch, &bytes);
    MatrixObject* m = reinterpret_cast<MatrixObject*>(MatrixType.tp_alloc(&MatrixType, 0));
    if (!m) throw PythonError{};
    new (&m->codes) at::Tensor();
    new (&m->scales) at::Tensor();
    new (&m->per_matrix) at::Tensor();
    m->type = type;
    m->rows = rows;
    m->K = K;
    m->matrices = matrices;
    m->scale = 1.0;
    m->pitch = pitch;
    m->scale_bytes = bytes;
    Py_XINCREF(plan);
    m->plan = plan;
    return m;
}

struct Owned {  // a new reference, dropped unless released
    PyObject* o;
    ~Owned() { Py_XDECREF(o); }
    PyObject* release() {
        PyObject* r = o;
        o = nullptr;
        return r;
    }
};

// Codes and scales of m in one allocation.
void allocate(MatrixObject* m, int device) {
    const int64_t codes = m->matrices * m->rows * m->pitch;  // rows of whole 16 bytes: the scales stay aligned
    m->scales = new_tensor({codes + m->scale_bytes}, at::kByte, device);
    m->device = device;
    m->codes_at = m->scales.data_ptr<uint8_t>();
    m->scales_at = m->codes_at + codes;
}

void set_scale(MatrixObject* m, PyObject* v) {
    if (v && THPVariable_Check(v)) {
        const at::Tensor& t = THPVariable_Unpack(v);
        if (t.dim() != 1 || t.size(0) != m->matrices)
            refuse("global_scale has shape " + shape_text(t.sizes()) + "; expected (" + std::to_string(m->matrices) + ",)");
        require(t, "global_scale", at::kFloat, m->matrices);
        require_device(t, "global_scale", m->device);
        m->per_matrix = t;
        return;
    }
    m->scale = v ? to_double(v) : 1.0;
    m->per_matrix = at::Tensor();
}

PyObject* matrix_vectorcall(PyObject*, PyObject* const* args, size_t nargsf, PyObject* kwnames) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"type_", "rows", "K", "codes", "scales", "global_scale", "matrices", "plan"};
        const Args<8> a("Fp4Matrix", names, 5, args, PyVectorcall_NARGS(nargsf), kwnames);
        const PlanObject* plan = a[7] ? to_plan(a[7]) : nullptr;
        const at::Tensor &codes = tensor(a[3], "codes"), &scales = tensor(a[4], "scales");
        Owned o{reinterpret_cast<PyObject*>(
            alloc_matrix(to_type(a[0]), to_int(a[1]), to_int(a[2]), a[6] ? to_int(a[6]) : 1, a[7]))};
        MatrixObject* m = reinterpret_cast<MatrixObject*>(o.o);
        // the product by experts reads as many rows as the plan has
        if (plan && m->rows != plan->rows)
            refuse("an operand of " + std::to_string(m->rows) + " rows; the plan has " + std::to_string(plan->rows) + " sorted rows");
        require(codes, "codes", at::kByte, m->matrices * m->rows * m->pitch);
        require(scales, "scales", at::kByte, m->scale_bytes);
        m->device = codes.get_device();
        require_device(scales, "scales", m->device);
        if (plan && plan->device != m->device)
            refuse("codes are on cuda:" + std::to_string(m->device) + ", the plan on cuda:" + std::to_string(plan->device));
        m->codes = codes;
        m->scales = scales;
        m->codes_at = codes.data_ptr<uint8_t>();
        m->scales_at = scales.data_ptr<uint8_t>();
        set_scale(m, a[5]);
        return o.release();
    });
}

void matrix_dealloc(PyObject* self) {
    MatrixObject* m = reinterpret_cast<MatrixObject*>(self);
    m->codes.~Tensor();
    m->scales.~Tensor();
    m->per_matrix.~Tensor();
    Py_XDECREF(m->plan);
    Py_TYPE(self)->tp_free(self);
}

MatrixObject* to_matrix(PyObject* o, const char* what) {
    if (!o || Py_TYPE(o) != &MatrixType) refuse(std::string(what) + " must be an Fp4Matrix");
    return reinterpret_cast<MatrixObject*>(o);
}

PyObject* matrix_codes(PyObject* self, void*) {
    return entry([&]() -> PyObject* {
        MatrixObject* m = reinterpret_cast<MatrixObject*>(self);
        if (m->codes.defined()) return wrap(m->codes);
        const int64_t n = m->matrices * m->rows;
        return wrap(view_of(m->scales, 0, {n, m->pitch}));
    });
}
PyObject* matrix_scales(PyObject* self, void*) {
    return entry([&]() -> PyObject* {
        MatrixObject* m = reinterpret_cast<MatrixObject*>(self);
        if (m->codes.defined()) return wrap(m->scales);
        return wrap(view_of(m->scales, m->matrices * m->rows * m->pitch, {m->scale_bytes}));
    });
}
PyObject* matrix_get_scale(PyObject* self, void*) {
    return entry([&]() -> PyObject* {
        MatrixObject* m = reinterpret_cast<MatrixObject*>(self);
        return m->per_matrix.defined() ? wrap(m->per_matrix) : PyFloat_FromDouble(m->scale);
    });
}
int matrix_set_scale(PyObject* self, PyObject* v, void*) {
    Owned r{entry([&]() -> PyObject* {
        if (!v) refuse("global_scale cannot be deleted");
        set_scale(reinterpret_cast<MatrixObject*>(self), v);
        Py_RETURN_NONE;
    })};
    return r.o ? 0 : -1;
}
PyObject* matrix_plan(PyObject* self, void*) {
    PyObject* p = reinterpret_cast<MatrixObject*>(self)->plan;
    return Py_NewRef(p ? p : Py_None);
}
PyObject* matrix_type(PyObject* self, void*) { return PyLong_FromLong(reinterpret_cast<MatrixObject*>(self)->type); }
PyObject* matrix_rows(PyObject* self, void*) { return PyLong_FromLongLong(reinterpret_cast<MatrixObject*>(self)->rows); }
PyObject* matrix_K(PyObject* self, void*) { return PyLong_FromLongLong(reinterpret_cast<MatrixObject*>(self)->K); }
PyObject* matrix_matrices(PyObject* self, void*) {
    return PyLong_FromLongLong(reinterpret_cast<MatrixObject*>(self)->matrices);
}

PyGetSetDef matrix_getset[] = {
    {"type", matrix_type, nullptr, "NVFP4 or MXFP4", nullptr},
    {"rows", matrix_rows, nullptr, "rows of one matrix", nullptr},
    {"K", matrix_K, nullptr, "elements of a row", nullptr},
    {"matrices", matrix_matrices, nullptr, "matrices it holds", nullptr},
    {"global_scale", matrix_get_scale, matrix_set_scale, "a float, or a CUDA fp32 tensor [matrices]", nullptr},
    {"plan", matrix_plan, nullptr, "the ExpertPlan whose sorted rows it holds, or None", nullptr},
    {"codes", matrix_codes, nullptr, "uint8 [matrices * rows][pitch]", nullptr},
    {"scales", matrix_scales, nullptr, "uint8, the tiled scale words", nullptr},
    {nullptr, nullptr, nullptr, nullptr, nullptr}};

PyTypeObject MatrixType = {PyVarObject_HEAD_INIT(nullptr, 0)};

// ---- operands ----------------------------------------------------------------------------------------------

#define PNQ_ENTRY(name) PyObject* name(PyObject*, PyObject* const* args, Py_ssize_t nargs, PyObject* kwnames)

PNQ_ENTRY(fp4_layout) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"type_", "rows", "K", "matrices", "plan_experts"};
        const Args<5> a("fp4_layout", names, 3, args, nargs, kwnames);
        int64_t pitch = 0, bytes = 0;
        layout_of(to_type(a[0]), to_int(a[1]), to_int(a[2]), a[3] ? to_int(a[3]) : 1, a[4] ? to_int(a[4]) : 0, &pitch, &bytes);
        return Py_BuildValue("LL", static_cast<long long>(pitch), static_cast<long long>(bytes));
    });
}

PNQ_ENTRY(fp4_quantize) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"type_", "x", "global_scale", "plan", "out", "stream", "sorted"};
        const Args<7> a("fp4_quantize", names, 2, args, nargs, kwnames);
        const int type = to_type(a[0]), G = type == PNQ_MXFP4 ? 32 : 16;
        const at::Tensor& x = tensor(a[1], "x");
        if (x.dim() != 2 && x.dim() != 3) refuse("x must be a torch.Tensor [rows][K] or [matrices][rows][K]");
        const int xt = float_type(x.scalar_type(), "x");
        if (!x.is_cuda()) refuse("x must be a CUDA tensor");
        const int device = x.get_device();
        const int64_t matrices = x.dim() == 3 ? x.size(0) : 1, rows = x.size(-2), K = x.size(-1);
        if (x.dim() == 3 && !x.is_contiguous()) refuse("x [matrices][rows][K] must be contiguous");
        if (x.stride(-1) != 1 && K > 1 && rows * matrices) refuse("the elements of a row of x must be consecutive");
        const int64_t ldx = x.dim() == 3 || rows <= 1 ? K : x.stride(0);
        if (ldx < K) refuse("rows of x are " + std::to_string(ldx) + " elements apart; at least K = " + std::to_string(K) + " is wanted");
        if (K == 0 || K % G)
            refuse("K = " + std::to_string(K) + " is not a positive multiple of " + std::to_string(G), PNQ_ERR_SHAPE);
        PlanObject* plan = a[3] ? to_plan(a[3]) : nullptr;
        const int sorted = a[6] ? PyObject_IsTrue(a[6]) : 0;
        if (sorted < 0) throw PythonError{};
        if (sorted && !plan) refuse("sorted rows are a plan's: plan is missing", PNQ_ERR_FLAGS);
        if (plan) {
            if (matrices != 1 || rows != (sorted ? plan->rows : plan->desc.tokens))
                refuse("x has shape " + shape_text(x.sizes()) + "; the plan has " + std::to_string(plan->desc.tokens) + " tokens and " +
                       std::to_string(plan->rows) + " rows");
            require_device(x, "x", plan->device);
        }
        const double g = a[2] ? to_double(a[2]) : 1.0;
        const int64_t out_rows = plan ? plan->rows : rows;
        const Place place(a[5], device);
        Owned o{nullptr};
        if (a[4]) {
            MatrixObject* m = to_matrix(a[4], "out");
            const int64_t have = m->plan ? reinterpret_cast<PlanObject*>(m->plan)->desc.experts : 0;
            if (m->type != type || m->rows != out_rows || m->K != K || m->matrices != matrices || m->device != device ||
                have != (plan ? plan->desc.experts : 0))
                refuse("out is an operand of another type, shape or device");
            o.o = Py_NewRef(a[4]);
        } else {
            o.o = reinterpret_cast<PyObject*>(alloc_matrix(type, out_rows, K, matrices, a[3]));
            allocate(reinterpret_cast<MatrixObject*>(o.o), device);
        }
        MatrixObject* m = reinterpret_cast<MatrixObject*>(o.o);
        place.record(x, m->scales, m->codes);
        if (plan) place.record(plan->buffer);
        check(pnq_fp4_quantize(type, xt, x.data_ptr(), ldx, rows, K, matrices, static_cast<float>(g), plan ? &plan->desc : nullptr,
                               sorted ? PNQ_FP4_SORTED : 0u, m->codes_at, m->scales_at, place.stream()),
              "pnq_fp4_quantize");
        // only now: a refused call leaves `out` as it was
        m->scale = g;
        m->per_matrix = at::Tensor();
        if (plan && m->plan != a[3]) {
            Py_INCREF(a[3]);
            Py_XSETREF(m->plan, a[3]);
        }
        return o.release();
    });
}

// The result: `out` checked, or a new [rows][cols] tensor of dtype.
at::Tensor result(PyObject* out, int64_t rows, int64_t cols, at::ScalarType dtype, int device, int* type) {
    if (!out) {
        *type = float_type(dtype, "the result");
        return new_matrix(rows, cols, dtype, device);
    }
    const at::Tensor& t = tensor(out, "out");
    *type = float_type(t.scalar_type(), "out");
    require_matrix(t, "out", t.scalar_type(), rows, cols, device);
    return t;
}

// `out` as it was given, or the new tensor.
PyObject* returned(PyObject* out, at::Tensor& t) { return out ? Py_NewRef(out) : wrap(std::move(t)); }

PNQ_ENTRY(fp4_dequantize) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"m", "dtype", "out", "stream"};
        const Args<4> a("fp4_dequantize", names, 1, args, nargs, kwnames);
        MatrixObject* m = to_matrix(a[0], "m");
        if (m->per_matrix.defined()) refuse("an operand with a global scale per matrix is read back matrix by matrix");
        const Place place(a[3], m->device);
        int type = 0;
        at::Tensor t = result(a[2], m->matrices * m->rows, m->K, dtype_of(a[1], at::kFloat), m->device, &type);
        place.record(m->codes, m->scales, t);
        if (m->plan) place.record(reinterpret_cast<PlanObject*>(m->plan)->buffer);
        check(pnq_fp4_dequantize(m->type, m->codes_at, m->scales_at, m->rows, m->K, m->matrices, static_cast<float>(m->scale),
                                 m->plan ? &reinterpret_cast<PlanObject*>(m->plan)->desc : nullptr, type, t.data_ptr(),
                                 place.stream()),
              "pnq_fp4_dequantize");
        return returned(a[2], t);
    });
}

PNQ_ENTRY(fp4_pack) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"type_", "codes", "scales", "rows", "K", "global_scale", "matrices", "stream"};
        const Args<8> a("fp4_pack", names, 5, args, nargs, kwnames);
        const int type = to_type(a[0]);
        const at::Tensor &codes = tensor(a[1], "codes"), &scales = tensor(a[2], "scales");
        const int64_t rows = to_int(a[3]), K = to_int(a[4]), matrices = a[6] ? to_int(a[6]) : 1;
        Owned o{reinterpret_cast<PyObject*>(alloc_matrix(type, rows, K, matrices, nullptr))};
        MatrixObject* m = reinterpret_cast<MatrixObject*>(o.o);
        const int64_t n = matrices * rows;
        require(codes, "codes", at::kByte, n * (K / 2));
        require(scales, "scales", at::kByte, n * (K / (type == PNQ_MXFP4 ? 32 : 16)));
        m->device = codes.get_device();
        require_device(scales, "scales", m->device);
        set_scale(m, a[5]);
        const Place place(a[7], m->device);
        const bool keep = K % 32 == 0 && reinterpret_cast<uintptr_t>(codes.data_ptr()) % 16 == 0;
        m->codes = keep ? codes : new_tensor({n, m->pitch}, at::kByte, m->device);
        m->scales = new_tensor({m->scale_bytes}, at::kByte, m->device);
        m->codes_at = m->codes.data_ptr<uint8_t>();
        m->scales_at = m->scales.data_ptr<uint8_t>();
        place.record(codes, scales);
        check(pnq_fp4_pack(type, codes.data_ptr<uint8_t>(), scales.data_ptr<uint8_t>(), rows, K, matrices, m->codes_at, m->scales_at,
                           place.stream()),
              "pnq_fp4_pack");
        return o.release();
    });
}

// x and w can be multiplied.
void check_operands(const MatrixObject* x, const MatrixObject* w) {
    if (x->type != w->type || x->K != w->K)
        refuse("operands differ: type " + std::to_string(x->type) + ", K = " + std::to_string(x->K) + " and type " +
               std::to_string(w->type) + ", K = " + std::to_string(w->K));
    if (x->matrices != 1 || x->per_matrix.defined()) refuse("the activations are one matrix with one global scale");
    if (x->device != w->device)
        refuse("operands are on cuda:" + std::to_string(x->device) + " and cuda:" + std::to_string(w->device));
}

unsigned to_flags(PyObject* o) {
    const int64_t v = o ? to_int(o) : 0;
    if (v < 0 || v > UINT32_MAX) refuse("flags = " + std::to_string(v) + " are not known", PNQ_ERR_FLAGS);
    return static_cast<unsigned>(v);
}

PNQ_ENTRY(fp4_gemm) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"x", "w", "dtype", "out", "flags", "stream"};
        const Args<6> a("fp4_gemm", names, 2, args, nargs, kwnames);
        const MatrixObject *x = to_matrix(a[0], "x"), *w = to_matrix(a[1], "w");
        check_operands(x, w);
        if (w->matrices != 1 || w->per_matrix.defined() || x->plan || w->plan)
            refuse("fp4_gemm takes one matrix each; expert layers go through fp4_gemm_experts");
        const Place place(a[5], x->device);
        int type = 0;
        at::Tensor t = result(a[3], x->rows, w->rows, dtype_of(a[2], at::kFloat), x->device, &type);
        place.record(x->codes, x->scales, w->codes, w->scales, t);
        check(pnq_fp4_gemm(x->type, x->codes_at, x->scales_at, x->rows, w->codes_at, w->scales_at, w->rows, x->K,
                           static_cast<float>(x->scale * w->scale), type, t.data_ptr(), to_flags(a[4]), place.stream()),
              "pnq_fp4_gemm");
        return returned(a[3], t);
    });
}

PNQ_ENTRY(fp4_gemm_experts) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"x", "w", "plan", "dtype", "out", "flags", "stream"};
        const Args<7> a("fp4_gemm_experts", names, 3, args, nargs, kwnames);
        const MatrixObject *x = to_matrix(a[0], "x"), *w = to_matrix(a[1], "w");
        PlanObject* plan = to_plan(a[2]);
        check_operands(x, w);
        // the same plan, or another view of its memory: a plan of the same sizes sorts other rows (another layer's, say)
        const PlanObject* made = reinterpret_cast<PlanObject*>(x->plan);
        if (!made || (made != plan && (made->desc.tokens != plan->desc.tokens || made->desc.slots != plan->desc.slots ||
                                       made->desc.experts != plan->desc.experts || made->desc.offsets != plan->desc.offsets)))
            refuse("x is not an operand of this plan's sorted rows");
        if (w->matrices != plan->desc.experts || w->plan)
            refuse("w has " + std::to_string(w->matrices) + " matrices; one for each of the plan's experts is wanted");
        if (plan->device != x->device)
            refuse("the operands are on cuda:" + std::to_string(x->device) + ", the plan on cuda:" + std::to_string(plan->device));
        const Place place(a[6], x->device);
        int type = 0;
        at::Tensor t = result(a[4], plan->rows, w->rows, dtype_of(a[3], at::kFloat), x->device, &type);
        const bool per = w->per_matrix.defined();
        place.record(x->codes, x->scales, w->codes, w->scales, w->per_matrix, plan->buffer, t);
        check(pnq_fp4_gemm_experts(x->type, x->codes_at, x->scales_at, &plan->desc, w->codes_at, w->scales_at, w->rows, x->K,
                                   static_cast<float>(per ? x->scale : x->scale * w->scale),
                                   per ? w->per_matrix.data_ptr<float>() : nullptr, type, t.data_ptr(), to_flags(a[5]),
                                   place.stream()),
              "pnq_fp4_gemm_experts");
        return returned(a[4], t);
    });
}

// ---- tokens to their experts and back -----------------------------------------------------------------------

PNQ_ENTRY(expert_sort) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"ids", "experts", "plan", "stream"};
        const Args<4> a("expert_sort", names, 2, args, nargs, kwnames);
        const at::Tensor& ids = tensor(a[0], "ids");
        if (ids.dim() != 2) refuse("ids must be a torch.Tensor [tokens][slots]");
        require(ids, "ids", at::kInt, 0);
        const int64_t tokens = ids.size(0), slots = ids.size(1), experts = to_int(a[1]);
        check_plan_shape(tokens, slots, experts);
        const int device = ids.get_device();
        const Place place(a[3], device);
        Owned o{nullptr};
        if (a[2]) {
            const PlanObject* p = to_plan(a[2]);
            if (p->desc.tokens != tokens || p->desc.slots != slots || p->desc.experts != experts || p->device != device)
                refuse("the plan is of another shape or device");
            o.o = Py_NewRef(a[2]);
        } else {
            o.o = reinterpret_cast<PyObject*>(new_plan(tokens, slots, experts, device));
        }
        place.record(ids, reinterpret_cast<PlanObject*>(o.o)->buffer);
        check(pnq_expert_sort(ids.data_ptr<int32_t>(), &reinterpret_cast<PlanObject*>(o.o)->desc, place.stream()),
              "pnq_expert_sort");
        return o.release();
    });
}

// A contiguous CUDA [rows][D] tensor on the plan's device: its element type.
int rows_of(const at::Tensor& t, const char* what, int64_t rows, const PlanObject* plan) {
    if (t.dim() != 2) refuse(std::string(what) + " must be a torch.Tensor [rows][D]");
    const int type = float_type(t.scalar_type(), what);
    require_matrix(t, what, t.scalar_type(), rows, t.size(1), plan->device);
    return type;
}

at::Tensor rows_out(PyObject* out, const at::Tensor& like, int64_t rows, const PlanObject* plan) {
    if (!out) return new_matrix(rows, like.size(1), like.scalar_type(), plan->device);
    const at::Tensor& t = tensor(out, "out");
    require_matrix(t, "out", like.scalar_type(), rows, like.size(1), plan->device);
    return t;
}

const at::Tensor& weights_of(PyObject* o, const PlanObject* plan, const char* what) {
    const at::Tensor& t = tensor(o, what);
    require_matrix(t, what, at::kFloat, plan->desc.tokens, plan->desc.slots, plan->device);
    return t;
}

PNQ_ENTRY(expert_gather) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"x", "plan", "out", "stream"};
        const Args<4> a("expert_gather", names, 2, args, nargs, kwnames);
        PlanObject* plan = to_plan(a[1]);
        const at::Tensor& x = tensor(a[0], "x");
        const int type = rows_of(x, "x", plan->desc.tokens, plan);
        const Place place(a[3], plan->device);
        at::Tensor t = rows_out(a[2], x, plan->rows, plan);
        place.record(x, plan->buffer, t);
        check(pnq_expert_gather(type, x.data_ptr(), x.size(1), &plan->desc, t.data_ptr(), place.stream()),
              "pnq_expert_gather");
        return returned(a[2], t);
    });
}

PNQ_ENTRY(expert_gather_backward) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"dxs", "plan", "out", "stream"};
        const Args<4> a("expert_gather_backward", names, 2, args, nargs, kwnames);
        PlanObject* plan = to_plan(a[1]);
        const at::Tensor& dxs = tensor(a[0], "dxs");
        const int type = rows_of(dxs, "dxs", plan->rows, plan);
        const Place place(a[3], plan->device);
        at::Tensor t = rows_out(a[2], dxs, plan->desc.tokens, plan);
        place.record(dxs, plan->buffer, t);
        check(pnq_expert_gather_backward(type, dxs.data_ptr(), dxs.size(1), &plan->desc, t.data_ptr(), place.stream()),
              "pnq_expert_gather_backward");
        return returned(a[2], t);
    });
}

PNQ_ENTRY(expert_combine) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"ys", "plan", "weights", "out", "stream"};
        const Args<5> a("expert_combine", names, 3, args, nargs, kwnames);
        PlanObject* plan = to_plan(a[1]);
        const at::Tensor& ys = tensor(a[0], "ys");
        const int type = rows_of(ys, "ys", plan->rows, plan);
        const at::Tensor& w = weights_of(a[2], plan, "weights");
        const Place place(a[4], plan->device);
        at::Tensor t = rows_out(a[3], ys, plan->desc.tokens, plan);
        place.record(ys, w, plan->buffer, t);
        check(pnq_expert_combine(type, ys.data_ptr(), ys.size(1), &plan->desc, w.data_ptr<float>(), t.data_ptr(),
                                 place.stream()),
              "pnq_expert_combine");
        return returned(a[3], t);
    });
}

PNQ_ENTRY(expert_combine_backward) {
    return entry([&]() -> PyObject* {
        static const char* const names[] = {"dy", "ys", "plan", "weights", "out", "dweights", "stream"};
        const Args<7> a("expert_combine_backward", names, 4, args, nargs, kwnames);
        PlanObject* plan = to_plan(a[2]);
        const at::Tensor &dy = tensor(a[0], "dy"), &ys = tensor(a[1], "ys");
        const int type = rows_of(ys, "ys", plan->rows, plan);
        require_matrix(dy, "dy", ys.scalar_type(), plan->desc.tokens, ys.size(1), plan->device);
        const at::Tensor& w = weights_of(a[3], plan, "weights");
        const Place place(a[6], plan->device);
        at::Tensor t = rows_out(a[4], ys, plan->rows, plan);
        at::Tensor dw = a[5] ? weights_of(a[5], plan, "dweights")
                             : new_matrix(plan->desc.tokens, plan->desc.slots, at::kFloat, plan->device);
        place.record(dy, ys, w, plan->buffer, t, dw);
        check(pnq_expert_combine_backward(type, dy.data_ptr(), ys.data_ptr(), ys.size(1), &plan->desc, w.data_ptr<float>(),
                                          t.data_ptr(), dw.data_ptr<float>(), place.stream()),
              "pnq_expert_combine_backward");
        Owned first{returned(a[4], t)}, second{returned(a[5], dw)};
        return PyTuple_Pack(2, first.o, second.o);
    });
}

// ---- the module -------------------------------------------------------------------------------------------------

#define PNQ_METHOD(name, doc) {#name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(name)), METH_FASTCALL | METH_KEYWORDS, doc}

PyMethodDef methods[] = {
    PNQ_METHOD(fp4_layout, "fp4_layout(type_, rows, K, matrices=1, plan_experts=0)\n--\n\n"
                           "(pitch of a row of codes, bytes of the tiled scales) of an operand."),
    PNQ_METHOD(fp4_quantize, "fp4_quantize(type_, x, global_scale=1.0, plan=None, out=None, stream=None, sorted=False)\n--\n\n"
                             "Encode x (CUDA bf16 or fp32, [rows][K], or [matrices][rows][K] contiguous; 2-D rows may be strided)\n"
                             "for the global multiplier (a number on the host: one computed on the device has to be read back). With a plan, x holds the plan's tokens (sorted: its sorted rows)\n"
                             "and the operand its sorted rows. out: an operand of the same shape to write into. Returns the Fp4Matrix."),
    PNQ_METHOD(fp4_dequantize, "fp4_dequantize(m, dtype=torch.float32, out=None, stream=None)\n--\n\n"
                               "The values an operand stands for, fp32 or bf16 [matrices * rows][K] (of a plan's operand: its\n"
                               "sorted rows, zeros past the rows in use). Its global_scale must be one float."),
    PNQ_METHOD(fp4_pack, "fp4_pack(type_, codes, scales, rows, K, global_scale=1.0, matrices=1, stream=None)\n--\n\n"
                         "Row-major weights (codes uint8 [matrices * rows][K / 2], scale words uint8 [matrices * rows][K / group])\n"
                         "as an operand, once, when they are loaded. Where K is a multiple of 32 and the codes are 16-byte\n"
                         "aligned they are kept as they are, not copied."),
    PNQ_METHOD(fp4_gemm, "fp4_gemm(x, w, dtype=torch.float32, out=None, flags=0, stream=None)\n--\n\n"
                         "Y[m][n] = sum_k X[m][k] W[n][k] of two operands of one type; fp32 or bf16 [M][N]. There is no\n"
                         "gradient of it: operands are codes."),
    PNQ_METHOD(fp4_gemm_experts, "fp4_gemm_experts(x, w, plan, dtype=torch.float32, out=None, flags=0, stream=None)\n--\n\n"
                                 "Every sorted row of x (made with `plan`) times its expert's matrix of w (matrices = the plan's\n"
                                 "experts): fp32 or bf16 [tokens * slots][N], zeros past the rows in use. No gradient, as fp4_gemm."),
    PNQ_METHOD(expert_sort, "expert_sort(ids, experts, plan=None, stream=None)\n--\n\n"
                            "The plan of ids (CUDA int32 [tokens][slots]: the expert of each choice; one outside 0 .. experts - 1\n"
                            "is dropped): stable, so equal experts keep the order of their slots."),
    PNQ_METHOD(expert_gather, "expert_gather(x, plan, out=None, stream=None)\n--\n\n"
                              "Sorted rows of x (fp32 or bf16 [tokens][D]): [tokens * slots][D], zeros past the rows in use. Outside\n"
                              "autograd: the result requires no gradient; expert_gather_backward gives x's."),
    PNQ_METHOD(expert_gather_backward, "expert_gather_backward(dxs, plan, out=None, stream=None)\n--\n\n"
                                       "Gradient of expert_gather: dx [tokens][D], each token's rows summed in fp32 in slot order."),
    PNQ_METHOD(expert_combine, "expert_combine(ys, plan, weights, out=None, stream=None)\n--\n\n"
                               "y[t] = sum over t's slots of weights[t][j] * its row of ys ([tokens * slots][D]; weights fp32\n"
                               "[tokens][slots]). Outside autograd: the result requires no gradient; expert_combine_backward gives\n"
                               "those of ys and weights."),
    PNQ_METHOD(expert_combine_backward, "expert_combine_backward(dy, ys, plan, weights, out=None, dweights=None, stream=None)\n--\n\n"
                                        "Gradients of expert_combine: (dys [tokens * slots][D], dweights fp32 [tokens][slots])."),
    {nullptr, nullptr, 0, nullptr}};

PyModuleDef module = {PyModuleDef_HEAD_INIT, "_native", "Torch wrappers of the 4-bit operands and the expert layer.", -1, methods};

// type(args) goes through vectorcall; tp_new is what a type needs for it.
PyObject* no_new(PyTypeObject* type, PyObject* args, PyObject* kwargs) {
    (void)type, (void)args, (void)kwargs;
    PyErr_SetString(PyExc_TypeError, "call the type itself");
    return nullptr;
}

void make_type(PyTypeObject* t, const char* name, const char* doc, Py_ssize_t size, destructor dealloc, PyGetSetDef* getset,
               vectorcallfunc call) {
    t->tp_name = name;
    t->tp_doc = doc;
    t->tp_basicsize = size;
    t->tp_flags = Py_TPFLAGS_DEFAULT;
    t->tp_dealloc = dealloc;
    t->tp_getset = getset;
    t->tp_new = no_new;
    t->tp_vectorcall = call;
}

}  // namespace

PyMODINIT_FUNC PyInit__native() {
    make_type(&PlanType, "block_quantized_weight_pn3t_gb300._native.ExpertPlan",
              "ExpertPlan(tokens, slots, experts, buffer=None, device=None)\n--\n\n"
              "How the (token, slot) choices of an expert layer are sorted by expert: one int32 CUDA buffer that holds, one\n"
              "after the other, offsets [experts + 1], block_start [experts + 1], order [n], position [n] and scale_row [n]\n"
              "(n = tokens * slots; meanings in include/pnq.h, pnq_expert_plan).",
              sizeof(PlanObject), plan_dealloc, plan_getset, plan_vectorcall);
    make_type(&MatrixType, "block_quantized_weight_pn3t_gb300._native.Fp4Matrix",
              "Fp4Matrix(type_, rows, K, codes, scales, global_scale=1.0, matrices=1, plan=None)\n--\n\n"
              "A 4-bit microscaled operand: `matrices` matrices of `rows` x `K`. codes: uint8 [matrices * rows][pitch];\n"
              "scales: uint8, the tiled scale words; global_scale: a float, or for expert weights a CUDA fp32 tensor\n"
              "[matrices]. plan: the ExpertPlan whose sorted rows it holds (None otherwise).",
              sizeof(MatrixObject), matrix_dealloc, matrix_getset, matrix_vectorcall);
    if (PyType_Ready(&PlanType) < 0 || PyType_Ready(&MatrixType) < 0) return nullptr;
    PyObject* binding = PyImport_ImportModule("block_quantized_weight_pn3t_gb300._binding");
    if (!binding) return nullptr;
    g_error = PyObject_GetAttrString(binding, "PnqError");
    Py_DECREF(binding);
    if (!g_error) return nullptr;
    PyObject* m = PyModule_Create(&module);
    if (!m) return nullptr;
    if (PyModule_AddObjectRef(m, "ExpertPlan", reinterpret_cast<PyObject*>(&PlanType)) < 0 ||
        PyModule_AddObjectRef(m, "Fp4Matrix", reinterpret_cast<PyObject*>(&MatrixType)) < 0) {
        Py_DECREF(m);
        return nullptr;
    }
    return m;
}
