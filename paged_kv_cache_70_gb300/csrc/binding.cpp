// binding.cpp -- the Python side of the calls that a serving loop makes for every layer
// of every step (paged_kv_write_rope, paged_kv_write_q8, paged_kv_read_q8,
// paged_decode_q8), compiled: argument checks, outputs, the current stream, and the call
// into libpagedkv.so, whose entry points _binding.py hands over.  A small call takes the
// GPU 4 us; marshalled in Python it took the host 17 to 20.  Like the rest of the
// binding it computes nothing.
#include <ATen/cuda/EmptyTensor.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <cmath>
#include <string>

#include "../../include/pagedkv.h"

namespace {

// ---- what _binding.py hands over
decltype(&paged_kv_write_rope) g_write_rope;
decltype(&paged_kv_write_q8) g_write_q8;
decltype(&paged_kv_read_q8) g_read_q8;
decltype(&paged_decode_q8) g_decode_q8;
decltype(&paged_decode_q8_workspace_size) g_decode_q8_size;
PyObject* g_check;  // raises for a status

struct ArgumentError {
    PyObject* type;
    std::string what;
};
[[noreturn]] void value_error(const std::string& s) { throw ArgumentError{PyExc_ValueError, s}; }
[[noreturn]] void type_error(const std::string& s) { throw ArgumentError{PyExc_TypeError, s}; }

constexpr int64_t kInt32 = 0x7fffffff;

const at::Tensor& tensor(PyObject* o, const char* name) {
    if (!THPVariable_Check(o)) type_error(std::string(name) + " must be a tensor");
    return THPVariable_Unpack(o);
}

int device_of(const at::Tensor& t, const char* name) {
    if (!t.is_cuda()) value_error(std::string(name) + " must be a CUDA tensor");
    return t.get_device();
}

void check_device(const at::Tensor& t, const char* name, int index) {
    if (device_of(t, name) != index)
        value_error(std::string(name) + " must be on the device of the other tensors");
}

void check_type(const at::Tensor& t, const char* name, at::ScalarType dtype) {
    if (t.scalar_type() != dtype)
        type_error(std::string(name) + " must be " + c10::toString(dtype) + ", got " +
                   c10::toString(t.scalar_type()));
}

// the address of a contiguous tensor of `dtype` on device `index`
void* address(const at::Tensor& t, const char* name, int index, at::ScalarType dtype) {
    check_device(t, name, index);
    if (!t.is_contiguous()) value_error(std::string(name) + " must be contiguous");
    check_type(t, name, dtype);
    return t.data_ptr();
}
int32_t* int32s(const at::Tensor& t, const char* name, int index) {
    return static_cast<int32_t*>(address(t, name, index, at::kInt));
}
int32_t* int32s_or_null(PyObject* o, const char* name, int index, int64_t n) {
    if (o == Py_None) return nullptr;
    const at::Tensor& t = tensor(o, name);
    if (t.numel() != n) value_error(std::string(name) + " must have one entry per token row");
    return int32s(t, name, index);
}

// (straight from the allocator: the dispatcher's way there takes as long again)
at::Tensor new_tensor(at::IntArrayRef sizes, at::ScalarType dtype, int index) {
    return at::Tensor(at::detail::empty_cuda(
        sizes, dtype, c10::Device(c10::kCUDA, (c10::DeviceIndex)index), std::nullopt));
}

int32_t dtype_code(at::ScalarType t) {
    if (t == at::kFloat) return PKV_F32;
    if (t == at::kBFloat16) return PKV_BF16;
    type_error(std::string("unsupported dtype ") + c10::toString(t) + " (float32 or bfloat16)");
}

// rows [N, H, d] whose heads are contiguous: their address and token stride in elements
void* row_address(const at::Tensor& t, const char* name, int index, at::ScalarType dtype,
                  int64_t* stride) {
    check_device(t, name, index);
    check_type(t, name, dtype);
    const int64_t n = t.size(0), h = t.size(1), d = t.size(2);
    if (t.numel() && ((d > 1 && t.stride(2) != 1) || (h > 1 && t.stride(1) != d)))
        value_error(std::string(name) + ": the heads of a token must be contiguous");
    *stride = n > 1 ? t.stride(0) : h * d;
    return t.data_ptr();
}

// pkv_geom of an 8-bit pool
pkv_geom q8_geom(const at::Tensor& pool) {
    if (pool.scalar_type() != at::kFloat8_e4m3fn || pool.dim() != 4 ||
        (pool.size(3) != 64 && pool.size(3) != 128))
        value_error("an 8-bit pool is float8_e4m3fn [num_blocks, Hkv, block_size, head_dim]");
    if (pool.size(1) > kInt32 || pool.size(2) > kInt32)
        value_error("num_kv_heads and block_size are 32-bit");
    return pkv_geom{(int32_t)pool.size(1), (int32_t)pool.size(1), (int32_t)pool.size(3),
                    (int32_t)pool.size(2), pool.size(0), PKV_Q8};
}
struct Pools {
    void *k, *v;
    float *k_scale, *v_scale;  // of 8-bit pools
};
Pools q8_pools(const at::Tensor& k, const at::Tensor& v, const at::Tensor& ks,
                 const at::Tensor& vs, int index) {
    const bool same = v.sizes() == k.sizes() && ks.dim() == 2 && vs.sizes() == ks.sizes() &&
                      ks.size(0) == k.size(0) && ks.size(1) == k.size(1);
    if (!same) value_error("the pools have one shape and the scales are [num_blocks, Hkv]");
    return Pools{address(k, "k_cache", index, at::kFloat8_e4m3fn),
                   address(v, "v_cache", index, at::kFloat8_e4m3fn),
                   static_cast<float*>(address(ks, "k_scale", index, at::kFloat)),
                   static_cast<float*>(address(vs, "v_scale", index, at::kFloat))};
}

// Other Python threads run while one of these lives: around allocations and launches, which
// wait where the launch queue is full or memory has to be freed, perhaps for a host function
// of the stream that needs Python.  (No Python object is touched meanwhile; the caller holds
// the arguments.)
class OthersRun {
public:
    OthersRun() : state_(PyEval_SaveThread()) {}
    ~OthersRun() { PyEval_RestoreThread(state_); }
    OthersRun(const OthersRun&) = delete;
    OthersRun& operator=(const OthersRun&) = delete;

private:
    PyThreadState* state_;
};

// raises (returns false) for a status
bool ok(const char* func, int status) {
    if (status == PKV_OK) return true;
    PyObject* r = PyObject_CallFunction(g_check, "si", func, status);
    Py_XDECREF(r);
    if (r) PyErr_SetString(PyExc_RuntimeError, func);
    return false;
}

PyObject* same(PyObject* o) {
    Py_INCREF(o);
    return o;
}

bool has_args(Py_ssize_t n, Py_ssize_t want) {
    if (n == want) return true;
    PyErr_Format(PyExc_TypeError, "expected %zd arguments, got %zd", want, n);
    return false;
}

// k, v, cos_sin, block_table, token_seq, token_pos, k_cache, v_cache, k_scale, v_scale, q,
// q_out, rope_pos, interleaved, slot_mapping_out -> q_out; scales given: 8-bit pools
PyObject* write_impl(PyObject* const* a) {
    const at::Tensor &k = tensor(a[0], "k"), &v = tensor(a[1], "v");
    const at::Tensor &table = tensor(a[3], "block_table"), &seq = tensor(a[4], "token_seq"),
                     &pos = tensor(a[5], "token_pos");
    const at::Tensor &kc = tensor(a[6], "k_cache"), &vc = tensor(a[7], "v_cache");
    const bool q8 = a[8] != Py_None;
    const int index = device_of(k, "k");
    pkv_geom g;
    if (q8) {
        g = q8_geom(kc);
    } else {
        if (kc.dim() != 4 || vc.sizes() != kc.sizes() || kc.size(1) > kInt32 ||
            kc.size(2) > kInt32 || kc.size(3) > kInt32)
            value_error("shape mismatch between the pools");
        g = pkv_geom{(int32_t)kc.size(2), (int32_t)kc.size(2), (int32_t)kc.size(3),
                     (int32_t)kc.size(1), kc.size(0), dtype_code(kc.scalar_type())};
    }
    if (k.dim() != 3 || v.sizes() != k.sizes() || k.size(1) != g.num_kv_heads ||
        k.size(2) != g.head_dim)
        value_error("shape mismatch between k/v rows and the pools");
    const int64_t n = k.size(0);
    if (seq.numel() != n || pos.numel() != n)
        value_error("token_seq and token_pos must have one entry per token row");
    if (table.dim() != 2 || table.size(0) > kInt32 || table.size(1) > kInt32)
        value_error("block_table must be [sequences, blocks], both 32-bit");
    const at::ScalarType dtype = k.scalar_type();
    const int32_t code = dtype_code(dtype);
    int64_t k_stride, v_stride;
    const void* kp = row_address(k, "k", index, dtype, &k_stride);
    const void* vp = row_address(v, "v", index, dtype, &v_stride);
    const int32_t* tp = int32s(table, "block_table", index);
    const int32_t* sp = int32s(seq, "token_seq", index);
    const int32_t* pp = int32s(pos, "token_pos", index);
    int32_t* slots = int32s_or_null(a[14], "slot_mapping_out", index, n);
    pkv_rope rope{};
    PyObject* result = Py_None;
    at::Tensor made;
    const at::Tensor* q_like = nullptr;  // q, where q_out is to be made
    if (a[2] == Py_None) {
        if (!q8) value_error("cos_sin is needed (paged_kv_write_positions writes without it)");
        if (a[10] != Py_None || a[11] != Py_None || a[12] != Py_None)
            value_error("q, q_out and rope_pos go with cos_sin");
    } else {
        const at::Tensor& cs = tensor(a[2], "cos_sin");
        if (cs.dim() != 2 || cs.size(0) > kInt32 || cs.size(1) > kInt32)
            value_error("cos_sin must be [positions, rotary_dim]");
        rope.cos_sin = static_cast<const float*>(address(cs, "cos_sin", index, at::kFloat));
        rope.num_positions = (int32_t)cs.size(0);
        rope.rotary_dim = (int32_t)cs.size(1);
        rope.interleaved = PyObject_IsTrue(a[13]);
        if (rope.interleaved < 0) return nullptr;
        rope.positions = int32s_or_null(a[12], "rope_pos", index, n);
        if (a[10] == Py_None) {
            if (a[11] != Py_None) value_error("q_out goes with q");
        } else {
            const at::Tensor& q = tensor(a[10], "q");
            if (q.dim() != 3 || q.size(0) != n || q.size(2) != g.head_dim || q.size(1) > kInt32)
                value_error("q must be [N, Hq, d]");
            g.num_heads = (int32_t)q.size(1);
            rope.q = row_address(q, "q", index, dtype, &rope.q_stride);
            if (a[11] == Py_None) {
                q_like = &q;
            } else {
                const at::Tensor& out = tensor(a[11], "q_out");
                if (out.sizes() != q.sizes()) value_error("q_out must have q's shape");
                rope.q_out = row_address(out, "q_out", index, dtype, &rope.q_out_stride);
                result = a[11];
            }
        }
    }
    const pkv_rope* r = a[2] == Py_None ? nullptr : &rope;
    Pools p;
    if (q8)
        p = q8_pools(kc, vc, tensor(a[8], "k_scale"), tensor(a[9], "v_scale"), index);
    else
        p = Pools{address(kc, "k_cache", index, kc.scalar_type()),
                    address(vc, "v_cache", index, kc.scalar_type()), nullptr, nullptr};
    const int32_t rows = (int32_t)table.size(0), width = (int32_t)table.size(1);
    int status;
    {
        const OthersRun others;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
        cudaStream_t stream = c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index);
        if (q_like) {
            made = new_tensor(q_like->sizes(), dtype, index);
            rope.q_out = row_address(made, "q_out", index, dtype, &rope.q_out_stride);
        }
        status = q8 ? g_write_q8(kp, k_stride, vp, v_stride, code, r, tp, width, rows, sp, pp, n,
                                 p.k, p.v, p.k_scale, p.v_scale, &g, stream)
                    : g_write_rope(kp, k_stride, vp, v_stride, code, r, tp, width, rows, sp, pp, n,
                                   slots, p.k, p.v, &g, stream);
    }
    if (!ok(q8 ? "paged_kv_write_q8" : "paged_kv_write_rope", status)) return nullptr;
    return made.defined() ? THPVariable_Wrap(std::move(made)) : same(result);
}

// k_cache, v_cache, k_scale, v_scale, slot_mapping, dtype, k_out, v_out -> (k_out, v_out)
PyObject* read_q8_impl(PyObject* const* a) {
    const at::Tensor &kc = tensor(a[0], "k_cache"), &vc = tensor(a[1], "v_cache");
    const at::Tensor& slots = tensor(a[4], "slot_mapping");
    const int index = device_of(kc, "k_cache");
    const pkv_geom g = q8_geom(kc);
    const Pools p = q8_pools(kc, vc, tensor(a[2], "k_scale"), tensor(a[3], "v_scale"), index);
    const int64_t n = slots.numel();
    const int64_t shape[3] = {n, g.num_kv_heads, g.head_dim};
    at::ScalarType dtype;
    at::Tensor out[2];
    if (a[6] != Py_None) {
        out[0] = tensor(a[6], "k_out");
        dtype = out[0].scalar_type();
    } else {
        if (!THPDtype_Check(a[5])) type_error("dtype must be a torch.dtype");
        dtype = reinterpret_cast<THPDtype*>(a[5])->scalar_type;
    }
    const int32_t code = dtype_code(dtype);
    if (a[7] != Py_None) out[1] = tensor(a[7], "v_out");
    for (const at::Tensor& t : out)
        if (t.defined() && t.sizes() != at::IntArrayRef(shape, 3))
            value_error("k_out / v_out must be [N, Hkv, d]");
    const int32_t* sp = int32s(slots, "slot_mapping", index);
    int status;
    {
        const OthersRun others;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
        for (at::Tensor& t : out)
            if (!t.defined()) t = new_tensor(at::IntArrayRef(shape, 3), dtype, index);
        void* kp = address(out[0], "k_out", index, dtype);
        void* vp = address(out[1], "v_out", index, dtype);
        status = g_read_q8(p.k, p.v, p.k_scale, p.v_scale, sp, n, kp, vp, code, &g,
                           c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index));
    }
    if (!ok("paged_kv_read_q8", status)) return nullptr;
    PyObject* pair = PyTuple_New(2);
    if (!pair) return nullptr;
    for (int i = 0; i < 2; ++i)
        PyTuple_SET_ITEM(pair, i,
                         a[6 + i] != Py_None ? same(a[6 + i]) : THPVariable_Wrap(std::move(out[i])));
    return pair;
}

// q, k_cache, v_cache, k_scale, v_scale, block_table, cache_seqlens, scale, out, workspace
// -> out
PyObject* decode_q8_impl(PyObject* const* a) {
    const at::Tensor &q = tensor(a[0], "q"), &kc = tensor(a[1], "k_cache"),
                     &vc = tensor(a[2], "v_cache");
    const at::Tensor &table = tensor(a[5], "block_table"), &lens = tensor(a[6], "cache_seqlens");
    const int index = device_of(q, "q");
    pkv_geom g = q8_geom(kc);
    if (q.dim() != 3 || q.size(2) != g.head_dim || table.dim() != 2 ||
        table.size(0) < q.size(0) || lens.numel() < q.size(0))
        value_error("shape mismatch");
    if (q.size(0) > kInt32 || q.size(1) > kInt32 || table.size(1) > kInt32)
        value_error("q and a table's row hold 2^31 - 1 entries at most");
    const at::ScalarType dtype = q.scalar_type();
    const int32_t code = dtype_code(dtype), batch = (int32_t)q.size(0);
    g.num_heads = (int32_t)q.size(1);
    double scale = 1.0 / std::sqrt((double)g.head_dim);
    if (a[7] != Py_None) {
        scale = PyFloat_AsDouble(a[7]);
        if (scale == -1.0 && PyErr_Occurred()) return nullptr;
    }
    const Pools p = q8_pools(kc, vc, tensor(a[3], "k_scale"), tensor(a[4], "v_scale"), index);
    const void* qp = address(q, "q", index, dtype);
    const int32_t* tp = int32s(table, "block_table", index);
    const int32_t* lp = int32s(lens, "cache_seqlens", index);
    at::Tensor out, workspace;
    if (a[8] != Py_None) {
        out = tensor(a[8], "out");
        if (out.sizes() != q.sizes()) value_error("out must have q's shape");
    }
    if (a[9] != Py_None) {
        workspace = tensor(a[9], "workspace");
        address(workspace, "workspace", index, workspace.scalar_type());
    }
    int status;
    {
        const OthersRun others;
        const c10::cuda::CUDAGuard guard((c10::DeviceIndex)index);
        if (!out.defined()) out = new_tensor(q.sizes(), dtype, index);
        void* op = address(out, "out", index, dtype);
        if (!workspace.defined())
            workspace = new_tensor({(int64_t)g_decode_q8_size(batch, code, &g)}, at::kByte, index);
        status = g_decode_q8(qp, code, p.k, p.v, p.k_scale, p.v_scale, tp, (int32_t)table.size(1),
                             lp, batch, (float)scale, op, workspace.data_ptr(),
                             (size_t)workspace.numel() * workspace.element_size(), &g,
                             c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)index));
    }
    if (!ok("paged_decode_q8", status)) return nullptr;
    return a[8] != Py_None ? same(a[8]) : THPVariable_Wrap(std::move(out));
}

template <PyObject* (*F)(PyObject* const*), int N>
PyObject* call(PyObject*, PyObject* const* args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (!has_args(n, N)) return nullptr;
    try {
        return F(args);
    } catch (const ArgumentError& e) {
        PyErr_SetString(e.type, e.what.c_str());
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

// check, then the addresses of the five entry points
PyObject* bind(PyObject*, PyObject* const* args, Py_ssize_t n) {
    if (!has_args(n, 6)) return nullptr;
    void* p[5];
    for (int i = 0; i < 5; ++i) {
        p[i] = PyLong_AsVoidPtr(args[1 + i]);
        if (!p[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an entry point is missing");
            return nullptr;
        }
    }
    Py_XDECREF(g_check);
    g_check = same(args[0]);
    g_write_rope = reinterpret_cast<decltype(g_write_rope)>(p[0]);
    g_write_q8 = reinterpret_cast<decltype(g_write_q8)>(p[1]);
    g_read_q8 = reinterpret_cast<decltype(g_read_q8)>(p[2]);
    g_decode_q8 = reinterpret_cast<decltype(g_decode_q8)>(p[3]);
    g_decode_q8_size = reinterpret_cast<decltype(g_decode_q8_size)>(p[4]);
    Py_RETURN_NONE;
}

#define PKV_METHOD(name, f) \
    {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void*>(f)), METH_FASTCALL, nullptr}
PyMethodDef g_methods[] = {PKV_METHOD("bind", bind),
                           PKV_METHOD("write", (&call<write_impl, 15>)),
                           PKV_METHOD("read_q8", (&call<read_q8_impl, 8>)),
                           PKV_METHOD("decode_q8", (&call<decode_q8_impl, 10>)),
                           {nullptr, nullptr, 0, nullptr}};
PyModuleDef g_module = {PyModuleDef_HEAD_INIT, "_pagedkv", nullptr, -1, g_methods,
                        nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__pagedkv() { return PyModule_Create(&g_module); }
