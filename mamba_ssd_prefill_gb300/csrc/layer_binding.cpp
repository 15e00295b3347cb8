// Python binding of the operators around the SSD: shape and type checks, outputs, workspace, stream, and the call of
// the C entry. The functions are those of layer.py, which documents them; here their arguments come by position.
//
// A call of a small operator is the time of its marshalling (a single-token step runs 2.4 us on the GPU): as Python the
// checks and the two outputs of a scan took 19 us on the host, here a whole call takes 5.4. The C entries are those of the
// library that the package loaded (bind() takes their addresses), so that another build of it may be chosen there.
#include <Python.h>

#include <ATen/core/Tensor.h>
#include <ATen/ops/empty.h>
#include <ATen/ops/maximum.h>
#include <ATen/ops/zeros.h>
#include <c10/cuda/CUDAGuard.h>
#include <c10/cuda/CUDAStream.h>
#include <torch/csrc/Dtype.h>
#include <torch/csrc/Exceptions.h>
#include <torch/csrc/autograd/python_variable.h>

#include <map>
#include <optional>
#include <sstream>
#include <stdexcept>
#include <string>
#include <utility>
#include <vector>

#include "../../include/ssd.h"

namespace {

using at::Tensor;

// A refusal of the arguments (ValueError), a status of the library (SsdError), an exception that Python already has.
struct Refusal {
    std::string text;
};
struct Status {
    int status;
    const char *what;
};
struct Raised {};

decltype(&::ssd_selective_scan_workspace_size) f_scan_size;
decltype(&::ssd_selective_scan) f_scan;
decltype(&::ssd_conv) f_conv;
decltype(&::ssd_group_norm) f_norm;
decltype(&::ssd_fp8_quantize) f_quantize;
decltype(&::ssd_fp8_matmul) f_matmul;
PyObject *ssd_error, *workspace_class;

const Tensor &tensor(PyObject *o, const char *name) {
    if (!THPVariable_Check(o)) throw Refusal{std::string(name) + ": expected a tensor"};
    return THPVariable_Unpack(o);
}
const Tensor *optional(PyObject *o, const char *name) { return o == Py_None ? nullptr : &tensor(o, name); }
bool truth(PyObject *o) {
    const int v = PyObject_IsTrue(o);
    if (v < 0) throw Raised{};
    return v;
}
int64_t whole(PyObject *o) {
    const long long v = PyLong_AsLongLong(o);
    if (v == -1 && PyErr_Occurred()) throw Raised{};
    return v;
}
at::ScalarType dtype(PyObject *o, const char *name) {
    if (!THPDtype_Check(o)) throw Refusal{std::string(name) + ": expected a torch.dtype"};
    return reinterpret_cast<THPDtype *>(o)->scalar_type;
}

const char *type_name(at::ScalarType t) {
    switch (t) {
        case at::kFloat: return "torch.float32";
        case at::kBFloat16: return "torch.bfloat16";
        case at::kHalf: return "torch.float16";
        case at::kFloat8_e4m3fn: return "torch.float8_e4m3fn";
        case at::kInt: return "torch.int32";
        default: return c10::toString(t);
    }
}
int io_code(at::ScalarType t, const char *name) {
    if (t == at::kFloat) return SSD_F32;
    if (t == at::kBFloat16) return SSD_BF16;
    if (t == at::kHalf) return SSD_F16;
    throw Refusal{std::string(name) + ": unsupported dtype " + type_name(t)};
}

void show(std::ostringstream &s, at::IntArrayRef v) {
    s << '(';
    for (size_t i = 0; i < v.size(); ++i) s << (i ? ", " : "") << v[i];
    s << ')';
}
[[noreturn]] void refuse(const char *name, const Tensor &t, at::IntArrayRef shape, at::ScalarType type, int dev,
                         const char *how) {
    std::ostringstream s;
    s << name << ": expected " << type_name(type) << ' ';
    show(s, shape);
    s << " on cuda:" << dev << ", " << how << ", got " << type_name(t.scalar_type()) << ' ';
    show(s, t.sizes());
    s << " with strides ";
    show(s, t.strides());
    s << " on " << t.device().str();
    throw Refusal{s.str()};
}
bool is(const Tensor &t, at::IntArrayRef shape, at::ScalarType type, int dev) {
    return t.sizes() == shape && t.scalar_type() == type && t.is_cuda() && t.get_device() == dev;
}
// shape, type, device, and rows (the last dimension) contiguous
void rows(const char *name, const Tensor &t, at::IntArrayRef shape, at::ScalarType type, int dev) {
    if (!is(t, shape, type, dev) || (shape.size() && shape.back() > 1 && t.strides().back() != 1))
        refuse(name, t, shape, type, dev, "the last dimension contiguous");
}
void flat(const char *name, const Tensor *t, at::IntArrayRef shape, at::ScalarType type, int dev) {
    if (t && (!is(*t, shape, type, dev) || !t->is_contiguous())) refuse(name, *t, shape, type, dev, "contiguous");
}
// [..., K] as evenly spaced rows: their stride. Dimensions of size 1 hold one index, so their strides say nothing.
int64_t row_stride(const char *name, const Tensor &t, at::IntArrayRef shape, at::ScalarType type, int dev) {
    rows(name, t, shape, type, dev);
    if (shape.size() == 1 || t.is_contiguous()) return shape.back();
    const auto st = t.strides();
    int64_t row = shape.back(), next = 0;  // next: what the dimension before must step by
    bool any = false;
    for (int64_t i = (int64_t)shape.size() - 2; i >= 0; --i) {
        if (shape[i] == 1) continue;
        if (!any) row = st[i];
        else if (st[i] != next) refuse(name, t, shape, type, dev, "evenly spaced rows");
        any = true;
        next = st[i] * shape[i];
    }
    return row;
}
int device(const char *what, const Tensor &t) {
    if (!t.is_cuda()) throw Refusal{std::string(what) + " runs on CUDA tensors only (there is no CPU path)"};
    return t.get_device();
}
void *ptr(const Tensor *t) { return t ? t->data_ptr() : nullptr; }

void cuda_ok(cudaError_t e, const char *what) {
    if (e != cudaSuccess) {
        (void)cudaGetLastError();
        throw std::runtime_error(std::string(what) + ": " + cudaGetErrorString(e));
    }
}

// Calls beside a capture that the capture's mode would forbid on this thread (allocations, waits for other streams).
struct Relaxed {
    cudaStreamCaptureMode mode = cudaStreamCaptureModeRelaxed;
    Relaxed() { cuda_ok(cudaThreadExchangeStreamCaptureMode(&mode), "a workspace"); }
    ~Relaxed() { (void)cudaThreadExchangeStreamCaptureMode(&mode); }
};
bool is_capturing(const c10::cuda::CUDAStream &stream) {
    cudaStreamCaptureStatus capture = cudaStreamCaptureStatusNone;
    cuda_ok(cudaStreamIsCapturing(stream.stream(), &capture), "a workspace");
    return capture != cudaStreamCaptureStatusNone;
}

// A stream of PyTorch's that no graph is being captured on.
c10::cuda::CUDAStream stream_apart(int dev) {
    for (int i = 0; i < 64; ++i) {
        const auto side = c10::cuda::getStreamFromPool(false, (c10::DeviceIndex)dev);
        if (!is_capturing(side)) return side;
    }
    throw std::runtime_error("a workspace: every stream is being captured");
}
// Zeroes a tensor now, whatever is being captured. Called with its device current.
void zero_now(const Tensor &t, const c10::cuda::CUDAStream &side) {
    cuda_ok(cudaMemsetAsync(t.data_ptr(), 0, t.nbytes(), side.stream()), "a workspace");
    cuda_ok(cudaStreamSynchronize(side.stream()), "a workspace");
}

std::map<int, Tensor> &device_headers() {
    static auto *all = new std::map<int, Tensor>();
    return *all;
}
// The status header (256 bytes) of all calls on a device that are given no workspace: kernels only ever set its status,
// so any calls may share it, and a call inside a capture finds it zeroed and at an address that stays, whatever becomes
// of the graph. Called with the device current.
const Tensor &device_status(int dev) {
    Tensor &t = device_headers()[dev];
    if (!t.defined()) {
        const Relaxed relaxed;
        const auto side = stream_apart(dev);  // no memory of a graph's
        const c10::cuda::CUDAStreamGuard on(side);
        const Tensor header =
            at::empty({256}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, (c10::DeviceIndex)dev));
        zero_now(header, side);
        t = header;
    }
    return t;
}
Tensor status_word(const Tensor &header) { return header.narrow(0, 12, 4).view(at::kInt); }

// Workspaces of calls that need more than the header: one per device and stream, grown, kept for the process's life.
std::map<std::pair<int, cudaStream_t>, Tensor> &stream_workspaces() {
    static auto *kept = new std::map<std::pair<int, cudaStream_t>, Tensor>();
    return *kept;
}

// Device, stream and workspace of one call.
struct Call {
    int dev;
    c10::cuda::CUDAGuard guard;
    std::optional<c10::cuda::CUDAStreamGuard> on;  // another stream than the current one: outputs belong to it
    c10::cuda::CUDAStream stream;
    Tensor ws;
    bool of_capture = false;  // ws is scratch of the graph that is being captured

    Call(int dev_, PyObject *stream_, PyObject *workspace, size_t bytes)
        : dev(dev_), guard((c10::DeviceIndex)dev_), stream(c10::cuda::getCurrentCUDAStream((c10::DeviceIndex)dev_)) {
        if (stream_ != Py_None) {
            auto get = [&](const char *name) {
                PyObject *v = PyObject_GetAttrString(stream_, name);
                if (!v) throw Raised{};
                const int64_t n = PyLong_AsLongLong(v);
                Py_DECREF(v);
                if (n == -1 && PyErr_Occurred()) throw Raised{};
                return n;
            };
            const auto s = c10::cuda::CUDAStream::unpack3(get("stream_id"), (c10::DeviceIndex)get("device_index"),
                                                          (c10::DeviceType)get("device_type"));
            if (s.device_index() != dev) throw Refusal{"stream: expected one of the tensors' device"};
            if (s != stream) {
                on.emplace(s);
                stream = s;
            }
        }
        if (workspace == Py_None) {
            own(bytes);
            return;
        }
        const int is_workspace = PyObject_IsInstance(workspace, workspace_class);
        if (is_workspace < 0) throw Raised{};
        if (is_workspace) {
            static PyObject *get_layer = PyUnicode_InternFromString("get_layer");
            PyObject *n = PyLong_FromSize_t(bytes);
            if (!n || !get_layer) throw Raised{};
            PyObject *args[3] = {workspace, n, is_capturing(stream) ? Py_True : Py_False};
            PyObject *t = PyObject_VectorcallMethod(get_layer, args, 3, nullptr);
            Py_DECREF(n);
            if (!t) throw Raised{};
            if (THPVariable_Check(t)) ws = THPVariable_Unpack(t);
            Py_DECREF(t);
        } else {
            ws = tensor(workspace, "workspace");
        }
        if (!ws.defined() || !ws.is_cuda() || ws.get_device() != dev || !ws.is_contiguous())
            throw Refusal{"workspace: expected a Workspace, or a contiguous tensor on the tensors' device"};
    }
    // The workspace of a call that is given none. A graph that is being captured gets scratch of its own, from its own
    // memory: the stream's workspace may be replaced by a larger one while the graph lives, and graphs captured on one
    // stream may be replayed on several. A captured call of the scan so takes two small nodes more (the header zeroed,
    // its status passed on); those that need only the header take none.
    void own(size_t bytes) {
        const Tensor &status = device_status(dev);
        if (bytes <= (size_t)status.numel()) {
            ws = status;
            return;
        }
        if (is_capturing(stream)) {
            of_capture = true;
            ws = make({(int64_t)bytes}, at::kByte);
            ws.narrow(0, 0, status.numel()).zero_();
            return;
        }
        Tensor &t = stream_workspaces()[{dev, stream.stream()}];
        if (!t.defined() || (size_t)t.nbytes() < bytes) {
            Tensor larger = at::zeros({(int64_t)bytes}, at::TensorOptions().dtype(at::kByte).device(at::kCUDA, dev));
            if (t.defined()) {  // what the smaller one has reported and nobody has read
                Tensor word = status_word(larger);
                word.copy_(status_word(t));
            }
            t = larger;
        }
        ws = t;
    }
    // After the launch: the status of a graph's own scratch goes to the header that outlives it.
    void pass_status_on() const {
        if (!of_capture) return;
        Tensor to = status_word(device_status(dev));
        at::maximum_out(to, to, status_word(ws));
    }
    size_t ws_bytes() const { return (size_t)ws.nbytes(); }
    Tensor make(at::IntArrayRef shape, at::ScalarType type) const {
        return at::empty(shape, at::TensorOptions().dtype(type).device(at::kCUDA, (c10::DeviceIndex)dev));
    }
    // Memory of other streams is not reused before the work on this one is done with it.
    void keep(std::initializer_list<const Tensor *> used) const {
        if (on)
            for (const Tensor *t : used)
                if (t && t->defined()) t->record_stream(stream);
    }
};

void check(int status, const char *what) {
    if (status) throw Status{status, what};
}

PyObject *pair(const Tensor &a, const Tensor &b, bool with_b) {
    PyObject *t = PyTuple_New(2);
    if (!t) throw Raised{};
    PyTuple_SET_ITEM(t, 0, THPVariable_Wrap(a));
    if (with_b) {
        PyTuple_SET_ITEM(t, 1, THPVariable_Wrap(b));
    } else {
        Py_INCREF(Py_None);
        PyTuple_SET_ITEM(t, 1, Py_None);
    }
    return t;
}

// x [batch, seqlen, channels] (packed: [1, T, channels]) -> its device and the number of sequences
int sequences(const char *what, const Tensor &x, const Tensor *cu, int64_t &nseq) {
    if (x.dim() != 3) throw Refusal{"x: expected [batch, seqlen, channels] (packed: [1, T, channels])"};
    const int dev = device(what, x);
    nseq = x.size(0);
    if (cu) {
        if (x.size(0) != 1) throw Refusal{"x: expected [1, T, channels] with cu_seqlens (sequences packed along T)"};
        if (cu->scalar_type() != at::kInt || !cu->is_cuda() || cu->get_device() != dev || cu->dim() != 1 ||
            cu->numel() < 1 || !cu->is_contiguous())
            throw Refusal{"cu_seqlens: expected a contiguous int32 [nseq + 1] tensor on the device of x"};
        nseq = cu->numel() - 1;
        if (nseq == 0 && x.size(1) > 0) throw Refusal{"cu_seqlens: offsets of no sequences, but x has tokens"};
    }
    return dev;
}

// x, dt_raw, dt_bias, A, B, C, D, z, init_states, cu_seqlens, state_dtype, softplus, y, final_states,
// return_final_states, workspace, stream
PyObject *selective_scan(PyObject *const *a) {
    const char *what = "ssd_selective_scan";
    const Tensor &x = tensor(a[0], "x"), &dt = tensor(a[1], "dt_raw"), &A = tensor(a[3], "A"), &B = tensor(a[4], "B"),
                 &C = tensor(a[5], "C");
    const Tensor *bias = optional(a[2], "dt_bias"), *D = optional(a[6], "D"), *z = optional(a[7], "z"),
                 *init = optional(a[8], "init_states"), *cu = optional(a[9], "cu_seqlens"), *yt = optional(a[12], "y"),
                 *ft = optional(a[13], "final_states");
    int64_t nseq;
    const int dev = sequences(what, x, cu, nseq);
    const int64_t b = x.size(0), L = x.size(1), Dc = x.size(2);
    const auto io = x.scalar_type();
    const int code = io_code(io, "x");
    if (B.dim() != 4) throw Refusal{"B: expected [batch, seqlen, ngroups, dstate]"};
    const int64_t G = B.size(2), N = B.size(3);
    const auto state = a[10] != Py_None ? dtype(a[10], "state_dtype") : init ? init->scalar_type() : at::kFloat;
    if (state != at::kFloat && state != at::kHalf)
        throw Refusal{std::string("state_dtype: expected fp32 or fp16, got ") + type_name(state)};
    if (Dc < 1 || N < 1 || G < 1 || Dc % G) {
        std::ostringstream s;
        s << "channels " << Dc << " must be a positive multiple of the " << G << " groups, with at least one state";
        throw Refusal{s.str()};
    }
    const int64_t shape[3] = {b, L, Dc}, bshape[4] = {b, L, G, N}, sshape[3] = {nseq, Dc, N};
    rows("x", x, shape, io, dev);
    rows("dt_raw", dt, shape, io, dev);
    rows("B", B, bshape, io, dev);
    rows("C", C, bshape, io, dev);
    if (G > 1 && (B.stride(2) != N || C.stride(2) != N))
        throw Refusal{"B, C: a token's [ngroups, dstate] must be contiguous"};
    flat("A", &A, {Dc, N}, at::kFloat, dev);
    flat("dt_bias", bias, {Dc}, at::kFloat, dev);
    flat("D", D, {Dc}, at::kFloat, dev);
    if (z) rows("z", *z, shape, io, dev);
    if (yt) rows("y", *yt, shape, io, dev);
    flat("init_states", init, sshape, state, dev);
    flat("final_states", ft, sshape, state, dev);
    ssd_scan_problem_t p{nseq, L, Dc, N, G, code, state == at::kFloat ? SSD_F32 : SSD_F16, cu != nullptr, truth(a[11])};
    c10::cuda::CUDAGuard guard((c10::DeviceIndex)dev);
    size_t bytes = 0;
    check(f_scan_size(&p, &bytes), what);
    Call call(dev, a[16], a[15], bytes);
    const Tensor y = yt ? *yt : call.make(shape, io);
    const bool with_final = ft || truth(a[14]);
    const Tensor fin = ft ? *ft : with_final ? call.make(sshape, state) : Tensor();
    ssd_scan_tensors_t t{};
    t.x = x.data_ptr();
    t.dt_raw = dt.data_ptr();
    t.z = ptr(z);
    t.B = B.data_ptr();
    t.C = C.data_ptr();
    t.y = y.data_ptr();
    t.A = static_cast<const float *>(A.data_ptr());
    t.dt_bias = static_cast<const float *>(ptr(bias));
    t.D = static_cast<const float *>(ptr(D));
    t.init_states = ptr(init);
    t.final_states = with_final ? fin.data_ptr() : nullptr;
    t.cu_seqlens = static_cast<const int32_t *>(ptr(cu));
    t.x_seq = x.stride(0), t.x_tok = x.stride(1);
    t.dt_seq = dt.stride(0), t.dt_tok = dt.stride(1);
    if (z) t.z_seq = z->stride(0), t.z_tok = z->stride(1);
    t.b_seq = B.stride(0), t.b_tok = B.stride(1);
    t.c_seq = C.stride(0), t.c_tok = C.stride(1);
    t.y_seq = y.stride(0), t.y_tok = y.stride(1);
    check(f_scan(&p, &t, call.ws.data_ptr(), call.ws_bytes(), call.stream.stream()), what);
    call.pass_status_on();
    call.keep({&x, &dt, bias, &A, &B, &C, D, z, init, cu, &y, &fin, &call.ws});
    return pair(y, fin, with_final);
}

int activation(PyObject *o) {
    if (PyUnicode_Check(o)) {
        if (PyUnicode_CompareWithASCIIString(o, "silu") == 0) return SSD_ACT_SILU;
        if (PyUnicode_CompareWithASCIIString(o, "none") == 0) return SSD_ACT_NONE;
    }
    throw Refusal{"activation: expected 'none' or 'silu'"};
}

// x, conv_weight, conv_bias, conv_state, cu_seqlens, activation, out, conv_state_out, return_conv_state, workspace,
// stream
PyObject *conv(PyObject *const *a) {
    const char *what = "ssd_conv";
    const Tensor &x = tensor(a[0], "x"), &w = tensor(a[1], "conv_weight");
    const Tensor *bias = optional(a[2], "conv_bias"), *state = optional(a[3], "conv_state"),
                 *cu = optional(a[4], "cu_seqlens"), *ot = optional(a[6], "out"), *st = optional(a[7], "conv_state_out");
    int64_t nseq;
    const int dev = sequences(what, x, cu, nseq);
    const int64_t b = x.size(0), L = x.size(1), Dc = x.size(2);
    const auto io = x.scalar_type();
    const int code = io_code(io, "x"), act = activation(a[5]);
    if (w.dim() != 2 || w.size(1) < 1 || w.size(1) > 8)
        throw Refusal{"conv_weight: expected [channels, k] with k from 1 to 8"};
    const int64_t k = w.size(1), shape[3] = {b, L, Dc}, sshape[3] = {nseq, Dc, k - 1};
    rows("x", x, shape, io, dev);
    flat("conv_weight", &w, {Dc, k}, at::kFloat, dev);
    flat("conv_bias", bias, {Dc}, at::kFloat, dev);
    flat("conv_state", state, sshape, io, dev);
    flat("conv_state_out", st, sshape, io, dev);
    if (ot) rows("out", *ot, shape, io, dev);
    Call call(dev, a[10], a[9], 256);
    const Tensor out = ot ? *ot : call.make(shape, io);
    const bool with_state = st || truth(a[8]);
    const Tensor left = st ? *st : with_state ? call.make(sshape, io) : Tensor();
    ssd_conv_problem_t p{nseq, L, Dc, (int32_t)k, act, code, cu != nullptr};
    ssd_conv_tensors_t t{};
    t.x = x.data_ptr();
    t.out = out.data_ptr();
    t.weight = static_cast<const float *>(w.data_ptr());
    t.bias = static_cast<const float *>(ptr(bias));
    t.conv_state = ptr(state);
    t.conv_state_out = with_state ? left.data_ptr() : nullptr;
    t.cu_seqlens = static_cast<const int32_t *>(ptr(cu));
    t.x_seq = x.stride(0), t.x_tok = x.stride(1);
    t.out_seq = out.stride(0), t.out_tok = out.stride(1);
    check(f_conv(&p, &t, call.ws.data_ptr(), call.stream.stream()), what);
    call.keep({&x, &w, bias, state, cu, &out, &left, &call.ws});
    return pair(out, left, with_state);
}

std::vector<int64_t> with_last(at::IntArrayRef shape, int64_t last) {
    std::vector<int64_t> v(shape.begin(), shape.end());
    v.back() = last;
    return v;
}

// x, weight, bias, z, ngroups, eps, center, activation, gate_first, quantize, y, workspace, stream
PyObject *group_norm(PyObject *const *a) {
    const char *what = "ssd_group_norm";
    const Tensor &x = tensor(a[0], "x");
    const Tensor *w = optional(a[1], "weight"), *bias = optional(a[2], "bias"), *z = optional(a[3], "z"),
                 *yt = optional(a[10], "y");
    const int dev = device(what, x);
    const auto io = x.scalar_type();
    const int code = io_code(io, "x"), act = activation(a[7]);
    const int64_t groups = whole(a[4]);
    const double eps = PyFloat_AsDouble(a[5]);
    if (eps == -1.0 && PyErr_Occurred()) throw Raised{};
    const bool center = truth(a[6]), gate_first = truth(a[8]), quantize = truth(a[9]);
    const auto shape = x.sizes();
    if (x.dim() < 1 || shape.back() < 1 || groups < 1 || shape.back() % groups) {
        std::ostringstream s;
        s << "x: the channels of ";
        show(s, shape);
        s << " must be a positive multiple of the " << groups << " groups";
        throw Refusal{s.str()};
    }
    if (gate_first && !z) throw Refusal{"gate_first needs a gate z"};
    const int64_t Dc = shape.back();
    const auto out = quantize ? at::kFloat8_e4m3fn : io;
    ssd_norm_tensors_t t{};
    t.x_row = row_stride("x", x, shape, io, dev);
    if (z) t.z_row = row_stride("z", *z, shape, io, dev);
    t.y_row = yt ? row_stride("y", *yt, shape, out, dev) : Dc;
    flat("weight", w, {Dc}, at::kFloat, dev);
    flat("bias", bias, {Dc}, at::kFloat, dev);
    Call call(dev, a[12], a[11], 256);
    const Tensor y = yt ? *yt : call.make(shape, out);
    const Tensor scales = quantize ? call.make(with_last(shape, (Dc + 127) / 128), at::kFloat) : Tensor();
    t.x = x.data_ptr();
    t.z = ptr(z);
    t.y = y.data_ptr();
    t.scales = quantize ? static_cast<float *>(scales.data_ptr()) : nullptr;
    t.weight = static_cast<const float *>(ptr(w));
    t.bias = static_cast<const float *>(ptr(bias));
    ssd_norm_problem_t p{x.numel() / Dc, Dc, groups, code, act, center, gate_first, (float)eps, 0};
    check(f_norm(&p, &t, call.ws.data_ptr(), call.stream.stream()), what);
    call.keep({&x, z, w, bias, &y, &scales, &call.ws});
    return quantize ? pair(y, scales, true) : THPVariable_Wrap(y);
}

// x, block_rows, workspace, stream
PyObject *fp8_quantize(PyObject *const *a) {
    const char *what = "ssd_fp8_quantize";
    const Tensor &x = tensor(a[0], "x");
    const int dev = device(what, x);
    const auto io = x.scalar_type();
    const int code = io_code(io, "x");
    const int64_t block_rows = whole(a[1]);
    if (block_rows != 1 && block_rows != 128) throw Refusal{"block_rows: expected 1 or 128"};
    if (x.dim() < 1 || (block_rows == 128 && x.dim() != 2))
        throw Refusal{"x: expected [..., K], or a matrix [N, K] with block_rows=128"};
    const auto shape = x.sizes();
    const int64_t K = shape.back(), kb = (K + 127) / 128;
    int64_t n = 1;  // rows, also of rows without elements
    for (int64_t i = 0; i + 1 < x.dim(); ++i) n *= shape[i];
    const int64_t row = row_stride("x", x, shape, io, dev);
    Call call(dev, a[3], a[2], 256);
    const Tensor q = call.make(shape, at::kFloat8_e4m3fn);
    const Tensor scales = block_rows == 1 ? call.make(with_last(shape, kb), at::kFloat)
                                          : call.make({(n + 127) / 128, kb}, at::kFloat);
    check(f_quantize(n, K, (int32_t)block_rows, code, x.data_ptr(), row, q.data_ptr(),
                     static_cast<float *>(scales.data_ptr()), call.ws.data_ptr(), call.stream.stream()),
          what);
    call.keep({&x, &q, &scales, &call.ws});
    return pair(q, scales, true);
}

// a, a_scales, b, b_scales, bias, out_dtype, out, workspace, stream
PyObject *fp8_matmul(PyObject *const *v) {
    const char *what = "ssd_fp8_matmul";
    const Tensor &a = tensor(v[0], "a"), &sa = tensor(v[1], "a_scales"), &b = tensor(v[2], "b"),
                 &sb = tensor(v[3], "b_scales");
    const Tensor *bias = optional(v[4], "bias"), *ot = optional(v[6], "out");
    const int dev = device(what, a);
    if (a.dim() < 1 || b.dim() != 2 || a.sizes().back() != b.size(1)) {
        std::ostringstream s;
        s << "expected a [..., K] and b [N, K], got ";
        show(s, a.sizes());
        s << " and ";
        show(s, b.sizes());
        throw Refusal{s.str()};
    }
    const auto type = dtype(v[5], "out_dtype");
    const int code = io_code(type, "out_dtype");
    const int64_t N = b.size(0), K = b.size(1), kb = (K + 127) / 128;
    flat("a", &a, a.sizes(), at::kFloat8_e4m3fn, dev);
    flat("b", &b, b.sizes(), at::kFloat8_e4m3fn, dev);
    flat("a_scales", &sa, with_last(a.sizes(), kb), at::kFloat, dev);
    flat("b_scales", &sb, {(N + 127) / 128, kb}, at::kFloat, dev);
    flat("bias", bias, {N}, at::kFloat, dev);
    int64_t M = 1;
    for (int64_t i = 0; i + 1 < a.dim(); ++i) M *= a.size(i);
    const auto shape = with_last(a.sizes(), N);
    const int64_t row = ot ? row_stride("out", *ot, shape, type, dev) : N;
    Call call(dev, v[8], v[7], 256);
    const Tensor out = ot ? *ot : call.make(shape, type);
    ssd_matmul_problem_t p{M, N, K, code, 0};
    check(f_matmul(&p, a.data_ptr(), static_cast<const float *>(sa.data_ptr()), b.data_ptr(),
                   static_cast<const float *>(sb.data_ptr()), static_cast<const float *>(ptr(bias)), out.data_ptr(), row,
                   call.ws.data_ptr(), call.ws_bytes(), call.stream.stream()),
          what);
    call.keep({&a, &sa, &b, &sb, bias, &out, &call.ws});
    return THPVariable_Wrap(out);
}

// The five entries, with every C++ exception turned into a Python one.
template <PyObject *(*F)(PyObject *const *), int ARGS>
PyObject *entry(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != ARGS) {
        PyErr_Format(PyExc_TypeError, "expected %d arguments, got %zd", ARGS, n);
        return nullptr;
    }
    if (!f_scan) {
        PyErr_SetString(PyExc_RuntimeError, "bind() has not been called");
        return nullptr;
    }
    try {
        return F(args);
    } catch (const Refusal &r) {
        PyErr_SetString(PyExc_ValueError, r.text.c_str());
    } catch (const Status &s) {
        PyObject *e = PyObject_CallFunction(ssd_error, "is", s.status, s.what);
        if (e) {
            PyErr_SetObject(reinterpret_cast<PyObject *>(Py_TYPE(e)), e);
            Py_DECREF(e);
        }
    } catch (const Raised &) {
    }
    return nullptr;
    END_HANDLE_TH_ERRORS
}

// zero_now(tensor), for the Workspace class
PyObject *zero(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 1 || !THPVariable_Check(args[0])) {
        PyErr_SetString(PyExc_TypeError, "expected a tensor");
        return nullptr;
    }
    const Tensor &t = THPVariable_Unpack(args[0]);
    const c10::cuda::CUDAGuard guard(t.device());
    const Relaxed relaxed;
    zero_now(t, stream_apart(t.get_device()));
    Py_RETURN_NONE;
    END_HANDLE_TH_ERRORS
}

// bind(addresses of the six C entries in the order above, SsdError, Workspace)
PyObject *bind(PyObject *, PyObject *const *args, Py_ssize_t n) {
    if (n != 8) {
        PyErr_Format(PyExc_TypeError, "expected 8 arguments, got %zd", n);
        return nullptr;
    }
    void *at[6];
    for (int i = 0; i < 6; ++i) {
        at[i] = PyLong_AsVoidPtr(args[i]);
        if (!at[i]) {
            if (!PyErr_Occurred()) PyErr_SetString(PyExc_ValueError, "an address is 0");
            return nullptr;
        }
    }
    f_scan_size = reinterpret_cast<decltype(f_scan_size)>(at[0]);
    f_scan = reinterpret_cast<decltype(f_scan)>(at[1]);
    f_conv = reinterpret_cast<decltype(f_conv)>(at[2]);
    f_norm = reinterpret_cast<decltype(f_norm)>(at[3]);
    f_quantize = reinterpret_cast<decltype(f_quantize)>(at[4]);
    f_matmul = reinterpret_cast<decltype(f_matmul)>(at[5]);
    Py_XINCREF(args[6]);
    Py_XINCREF(args[7]);
    ssd_error = args[6];
    workspace_class = args[7];
    Py_RETURN_NONE;
}

// reported(device index, stream): the buffers whose headers hold the status of calls without a workspace on that stream
PyObject *reported(PyObject *, PyObject *const *args, Py_ssize_t n) {
    HANDLE_TH_ERRORS
    if (n != 2) {
        PyErr_Format(PyExc_TypeError, "expected 2 arguments, got %zd", n);
        return nullptr;
    }
    try {
        const int dev = (int)whole(args[0]);
        void *stream = PyLong_AsVoidPtr(args[1]);
        if (PyErr_Occurred()) return nullptr;
        std::vector<Tensor> found;
        const auto h = device_headers().find(dev);
        if (h != device_headers().end() && h->second.defined()) found.push_back(h->second);
        const auto w = stream_workspaces().find({dev, static_cast<cudaStream_t>(stream)});
        if (w != stream_workspaces().end() && w->second.defined()) found.push_back(w->second);
        PyObject *list = PyList_New((Py_ssize_t)found.size());
        if (!list) return nullptr;
        for (size_t i = 0; i < found.size(); ++i) PyList_SET_ITEM(list, (Py_ssize_t)i, THPVariable_Wrap(found[i]));
        return list;
    } catch (const Raised &) {
        return nullptr;
    }
    END_HANDLE_TH_ERRORS
}

template <PyObject *(*F)(PyObject *, PyObject *const *, Py_ssize_t)> PyMethodDef method(const char *name) {
    return {name, reinterpret_cast<PyCFunction>(reinterpret_cast<void (*)()>(F)), METH_FASTCALL, nullptr};
}
PyMethodDef methods[] = {
    method<bind>("bind"),
    method<zero>("zero_now"),
    method<reported>("reported"),
    method<entry<selective_scan, 17>>("selective_scan"),
    method<entry<conv, 11>>("conv"),
    method<entry<group_norm, 13>>("group_norm"),
    method<entry<fp8_quantize, 4>>("fp8_quantize"),
    method<entry<fp8_matmul, 9>>("fp8_matmul"),
    {nullptr, nullptr, 0, nullptr},
};
PyModuleDef module = {PyModuleDef_HEAD_INIT, "_layer", nullptr, -1, methods, nullptr, nullptr, nullptr, nullptr};

}  // namespace

PyMODINIT_FUNC PyInit__layer() { return PyModule_Create(&module); }
