// mx_ops.cu -- the extern "C" entry points of the norm, activation, 8-bit
// checkpoint, gradient norm and optimizer calls declared in include/mx.h:
// argument validation on the host and the launches.
#include "mx_act8.cuh"
#include "mx_internal.cuh"
#include "mx_norm.cuh"

#include <cmath>
#include <initializer_list>

using namespace mx;

namespace {

constexpr int64_t kMaxCols = int64_t(1) << 30;
constexpr int64_t kMaxFlat = int64_t(1) << 34;  // values of one of many tensors: 32-bit units of eight
constexpr int64_t kMaxTensors = int64_t(1) << 24;
constexpr int64_t kMaxElems = int64_t(1) << 60;  // rows x stride: byte offsets fit 64 bits

bool valid_dtype(int t) { return t == MX_OUT_F32 || t == MX_OUT_BF16; }
int dtype_bytes(int t) { return t == MX_OUT_BF16 ? 2 : 4; }
bool aligned(const void* p, int bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }
bool empty(int64_t rows, int64_t cols) { return rows == 0 || cols == 0; }

int check_shape(int64_t rows, int64_t cols)
{
    if (rows < 0 || cols < 0 || cols > kMaxCols)
        return MX_ERR_INVALID_ARG;
    return rows <= kMaxElems / (act8_groups(cols) * kAct8Group + 1) ? MX_OK : MX_ERR_INVALID_ARG;
}

// A matrix of a checked shape.
int check_matrix(const void* p, int64_t rows, int64_t cols, int64_t ld, int dtype)
{
    if (!valid_dtype(dtype) || ld < cols || (ld > 0 && rows > kMaxElems / ld))
        return MX_ERR_INVALID_ARG;
    if (!p && !empty(rows, cols))
        return MX_ERR_INVALID_ARG;
    return aligned(p, dtype_bytes(dtype)) ? MX_OK : MX_ERR_ALIGNMENT;
}

int check_act8(const mx_act8* a, int64_t rows, int64_t cols)
{
    if (a->rows != rows || a->cols != cols || (!empty(rows, cols) && (!a->codes || !a->sf)))
        return MX_ERR_INVALID_ARG;
    return aligned(a->codes, 16) ? MX_OK : MX_ERR_ALIGNMENT;
}

Act8View view(const mx_act8* a)
{
    Act8View v;
    if (a) {
        v.codes = a->codes;
        v.sf = a->sf;
    }
    return v;
}

// The first error of several checks.
struct Checks {
    int rc = MX_OK;
    Checks& operator()(int r)
    {
        if (rc == MX_OK)
            rc = r;
        return *this;
    }
    Checks& require(bool ok) { return (*this)(ok ? MX_OK : MX_ERR_INVALID_ARG); }
    Checks& words(const void* p) { return (*this)(aligned(p, 4) ? MX_OK : MX_ERR_ALIGNMENT); }
};

// A call's vectors: none that it writes overlaps another that it writes or reads.
// The kernels read weights and statistics while, or after, other CTAs write these.
struct Vector {
    const void* p;
    int64_t bytes;
    bool overlaps(const Vector& v) const
    {
        const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(v.p);
        return p && v.p && a < b + v.bytes && b < a + bytes;
    }
};
int check_apart(std::initializer_list<Vector> written, std::initializer_list<Vector> read)
{
    for (const Vector* w = written.begin(); w != written.end(); ++w) {
        for (const Vector* v = w + 1; v != written.end(); ++v)
            if (w->overlaps(*v))
                return MX_ERR_INVALID_ARG;
        for (const Vector& v : read)
            if (w->overlaps(v))
                return MX_ERR_INVALID_ARG;
    }
    return MX_OK;
}

int zero(void* p, size_t bytes, cudaStream_t s)
{
    return !p || bytes == 0 || cudaMemsetAsync(p, 0, bytes, s) == cudaSuccess ? MX_OK : MX_ERR_CUDA;
}

thread_local int g_norm_fail_at = -1;  // test hook: the norm kernels' forced wait failure

}  // namespace

extern "C" {

void mx_debug_set_norm_fail_at(int64_t row) { g_norm_fail_at = row < 0 || row > INT32_MAX ? -1 : static_cast<int>(row); }

size_t mx_act8_codes_bytes(int64_t rows, int64_t cols)
{
    return check_shape(rows, cols) == MX_OK ? static_cast<size_t>(rows * act8_groups(cols) * kAct8Group) : 0;
}

size_t mx_act8_sf_bytes(int64_t rows, int64_t cols)
{
    return check_shape(rows, cols) == MX_OK ? static_cast<size_t>(rows * act8_groups(cols)) : 0;
}

int mx_act8_save(const void* x, int64_t ldx, int x_dtype, const mx_act8* out, void* stream)
{
    if (!out)
        return MX_ERR_INVALID_ARG;
    Checks ok;
    ok(check_shape(out->rows, out->cols));
    if (ok.rc == MX_OK)
        ok(check_matrix(x, out->rows, out->cols, ldx, x_dtype))(check_act8(out, out->rows, out->cols));
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    if (empty(out->rows, out->cols))
        return MX_OK;
    return launch_act8_save(x, ldx, x_dtype, out->rows, out->cols, view(out), d, static_cast<cudaStream_t>(stream));
}

int mx_act8_restore(const mx_act8* a, void* out, int64_t ldo, int out_dtype, void* stream)
{
    if (!a)
        return MX_ERR_INVALID_ARG;
    Checks ok;
    ok(check_shape(a->rows, a->cols));
    if (ok.rc == MX_OK)
        ok(check_matrix(out, a->rows, a->cols, ldo, out_dtype))(check_act8(a, a->rows, a->cols));
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    if (empty(a->rows, a->cols))
        return MX_OK;
    return launch_act8_restore(view(a), a->rows, a->cols, out, ldo, out_dtype, d, static_cast<cudaStream_t>(stream));
}

int mx_norm_fwd(const void* x, int64_t ldx, const void* residual, int64_t ldr, int x_dtype, int64_t rows,
                int64_t cols, int kind, const void* weight, const void* bias, int w_dtype, float eps, void* sum_out,
                int64_t lds, void* y, int64_t ldy, int y_dtype, float* mean, float* rstd, const mx_act8* save,
                float* amax_out, void* stream)
{
    Checks ok;
    ok(check_shape(rows, cols));
    ok.require(kind == MX_NORM_LAYER || kind == MX_NORM_RMS);
    ok.require(valid_dtype(w_dtype) && eps >= 0.0f);  // a NaN eps is refused too
    if (ok.rc == MX_OK) {
        ok(check_matrix(x, rows, cols, ldx, x_dtype))(check_matrix(y, rows, cols, ldy, y_dtype));
        if (residual)
            ok(check_matrix(residual, rows, cols, ldr, x_dtype))(check_matrix(sum_out, rows, cols, lds, x_dtype));
        else
            ok.require(!sum_out || empty(rows, cols));
        if (save)
            ok(check_act8(save, rows, cols));
        const bool w_ok = aligned(weight, dtype_bytes(w_dtype)) && aligned(bias, dtype_bytes(w_dtype));
        ok(w_ok ? MX_OK : MX_ERR_ALIGNMENT).words(mean).words(rstd).words(amax_out);
    }
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    const int64_t param = cols * dtype_bytes(w_dtype), stat = rows * static_cast<int64_t>(sizeof(float));
    if (ok(check_apart({{kind == MX_NORM_LAYER ? mean : nullptr, stat}, {rstd, stat}, {amax_out, sizeof(float)}},
                       {{weight, param}, {bias, param}})).rc != MX_OK)
        return ok.rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty(rows, cols))
        return zero(amax_out, sizeof(float), s);
    NormFwdArgs a = {};
    a.x = x;
    a.residual = residual;
    a.ldx = ldx;
    a.ldr = ldr;
    a.rows = rows;
    a.cols = cols;
    a.weight = weight;
    a.bias = bias;
    a.sum_out = sum_out;
    a.y = y;
    a.lds = lds;
    a.ldy = ldy;
    a.mean = mean;
    a.rstd = rstd;
    a.save = view(save);
    a.amax = reinterpret_cast<unsigned*>(amax_out);
    a.eps = eps;
    a.x_dtype = x_dtype;
    a.y_dtype = y_dtype;
    a.w_dtype = w_dtype;
    a.kind = kind;
    a.status = d.status;
    a.wait_ns = g_norm_fail_at < 0 ? kWaitLimitNs : 2000000;  // the hook's wait runs out in 2 ms
    a.fail_at = g_norm_fail_at;
    return launch_norm_fwd(a, d, s);
}

size_t mx_norm_bwd_workspace_bytes(int64_t rows, int64_t cols)
{
    if (check_shape(rows, cols) != MX_OK || empty(rows, cols))
        return 0;
    return static_cast<size_t>(norm_bwd_parts(rows, cols) * part_stride(cols)) * 2 * sizeof(float);
}

int mx_norm_bwd(const void* dy, int64_t ldy, int dy_dtype, const void* x, int64_t ldx, const mx_act8* x8,
                const float* mean, const float* rstd, const void* weight, int w_dtype, int64_t rows, int64_t cols,
                int kind, const void* dres, int64_t ldres, void* dx, int64_t lddx, int dx_dtype, float* dw, float* db,
                float* amax_out, void* workspace, size_t ws_bytes, void* stream)
{
    Checks ok;
    ok(check_shape(rows, cols));
    ok.require(kind == MX_NORM_LAYER || kind == MX_NORM_RMS);
    ok.require(valid_dtype(w_dtype) && (!x || !x8));
    if (ok.rc == MX_OK) {
        const bool none = empty(rows, cols);
        ok(check_matrix(dy, rows, cols, ldy, dy_dtype))(check_matrix(dx, rows, cols, lddx, dx_dtype));
        if (x8)
            ok(check_act8(x8, rows, cols));
        else
            ok(check_matrix(x, rows, cols, ldx, dx_dtype));
        if (dres)
            ok(check_matrix(dres, rows, cols, ldres, dx_dtype));
        ok.require(none || (rstd && (mean || kind == MX_NORM_RMS)));
        ok(aligned(weight, dtype_bytes(w_dtype)) ? MX_OK : MX_ERR_ALIGNMENT);
        ok.words(mean).words(rstd).words(dw).words(db).words(amax_out);
        if ((dw || db) && !none) {
            const size_t need = mx_norm_bwd_workspace_bytes(rows, cols);
            ok(need == 0 || (workspace && ws_bytes >= need) ? MX_OK : MX_ERR_WORKSPACE);
            ok(aligned(workspace, 16) ? MX_OK : MX_ERR_ALIGNMENT);
        }
    }
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    const int64_t stat = rows * static_cast<int64_t>(sizeof(float)), grad = cols * static_cast<int64_t>(sizeof(float));
    if (ok(check_apart({{dw, grad}, {db, grad}, {amax_out, sizeof(float)}},
                       {{weight, cols * dtype_bytes(w_dtype)}, {kind == MX_NORM_LAYER ? mean : nullptr, stat}, {rstd, stat}}))
            .rc != MX_OK)
        return ok.rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty(rows, cols))
        return ok(zero(amax_out, sizeof(float), s))(zero(dw, cols * sizeof(float), s))(zero(db, cols * sizeof(float), s)).rc;
    NormBwdArgs a = {};
    a.dy = dy;
    a.x = x;
    a.x8 = view(x8);
    a.ldy = ldy;
    a.ldx = ldx;
    a.rows = rows;
    a.cols = cols;
    a.mean = mean;
    a.rstd = rstd;
    a.weight = weight;
    a.dres = dres;
    a.dx = dx;
    a.ldres = ldres;
    a.lddx = lddx;
    a.dw = dw;
    a.db = db;
    a.parts = static_cast<float*>(workspace);
    a.amax = reinterpret_cast<unsigned*>(amax_out);
    a.dy_dtype = dy_dtype;
    a.dx_dtype = dx_dtype;
    a.w_dtype = w_dtype;
    a.kind = kind;
    a.status = d.status;
    a.wait_ns = g_norm_fail_at < 0 ? kWaitLimitNs : 2000000;  // the hook's wait runs out in 2 ms
    a.fail_at = g_norm_fail_at;
    return launch_norm_bwd(a, d, s);
}

int mx_act_fwd(const void* gate, int64_t ldg, const void* up, int64_t ldu, int64_t rows, int64_t cols, int act,
               int dtype, void* h, int64_t ldh, const mx_act8* gate8, const mx_act8* up8, float* amax_out,
               void* stream)
{
    Checks ok;
    ok(check_shape(rows, cols));
    ok.require(act >= MX_ACT_SILU && act <= MX_ACT_GELU_TANH);
    if (ok.rc == MX_OK) {
        ok(check_matrix(gate, rows, cols, ldg, dtype))(check_matrix(h, rows, cols, ldh, dtype));
        if (up)
            ok(check_matrix(up, rows, cols, ldu, dtype));
        if (gate8)
            ok(check_act8(gate8, rows, cols));
        if (up8)
            ok.require(up || empty(rows, cols))(check_act8(up8, rows, cols));
        ok.words(amax_out);
    }
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty(rows, cols))
        return zero(amax_out, sizeof(float), s);
    ActArgs a = {};
    a.gate = gate;
    a.up = up;
    a.h = h;
    a.ldg = ldg;
    a.ldu = ldu;
    a.ldh = ldh;
    a.rows = rows;
    a.cols = cols;
    a.gate8 = view(gate8);
    a.up8 = view(up8);
    a.amax = reinterpret_cast<unsigned*>(amax_out);
    a.act = act;
    a.dtype = dtype;
    a.gated = up != nullptr;
    return launch_act_fwd(a, d, s);
}

int mx_act_bwd(const void* dh, int64_t ldh, const void* gate, int64_t ldg, const void* up, int64_t ldu,
               const mx_act8* gate8, const mx_act8* up8, int64_t rows, int64_t cols, int act, int dtype, void* dgate,
               int64_t lddg, void* dup, int64_t lddu, float* amax_out, void* stream)
{
    Checks ok;
    ok(check_shape(rows, cols));
    ok.require(act >= MX_ACT_SILU && act <= MX_ACT_GELU_TANH);
    // gate and up are both kept or both checkpoints, and dup goes with up
    ok.require(gate8 ? !gate && !up : !up8);
    if (ok.rc == MX_OK) {
        ok(check_matrix(dh, rows, cols, ldh, dtype))(check_matrix(dgate, rows, cols, lddg, dtype));
        if (gate8)
            ok(check_act8(gate8, rows, cols));
        else
            ok(check_matrix(gate, rows, cols, ldg, dtype));
        if (up)
            ok(check_matrix(up, rows, cols, ldu, dtype));
        if (up8)
            ok(check_act8(up8, rows, cols));
        if (up || up8)
            ok(check_matrix(dup, rows, cols, lddu, dtype));
        else
            ok.require(!dup || empty(rows, cols));
        ok.words(amax_out);
    }
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (empty(rows, cols))
        return zero(amax_out, sizeof(float), s);
    ActArgs a = {};
    a.gate = gate;
    a.up = up;
    a.h = const_cast<void*>(dh);  // read only in the backward kernels
    a.dgate = dgate;
    a.dup = dup;
    a.ldg = ldg;
    a.ldu = ldu;
    a.ldh = ldh;
    a.lddg = lddg;
    a.lddu = lddu;
    a.rows = rows;
    a.cols = cols;
    a.gate8 = view(gate8);
    a.up8 = view(up8);
    a.amax = reinterpret_cast<unsigned*>(amax_out);
    a.act = act;
    a.dtype = dtype;
    a.gated = up || up8;
    return launch_act_bwd(a, d, s);
}

size_t mx_grad_norm_workspace_bytes(int64_t count)
{
    return count < 0 || count > kMaxTensors ? 0 : static_cast<size_t>(grad_norm_parts(count)) * sizeof(double);
}

int mx_grad_norm(const mx_grad* grads, int64_t count, double max_norm, float* out, void* workspace, size_t ws_bytes,
                 void* stream)
{
    Checks ok;
    ok.require(count >= 0 && count <= kMaxTensors && (grads || count == 0) && out && max_norm > 0.0);
    ok.words(out);
    for (int64_t i = 0; ok.rc == MX_OK && i < count; ++i) {
        const mx_grad& g = grads[i];
        ok.require(g.n >= 0 && g.n <= kMaxFlat && valid_dtype(g.dtype) && (g.data || g.n == 0));
        if (ok.rc == MX_OK)
            ok(aligned(g.data, dtype_bytes(g.dtype)) ? MX_OK : MX_ERR_ALIGNMENT);
    }
    if (ok.rc == MX_OK) {
        ok(workspace && ws_bytes >= mx_grad_norm_workspace_bytes(count) ? MX_OK : MX_ERR_WORKSPACE);
        ok(aligned(workspace, 8) ? MX_OK : MX_ERR_ALIGNMENT);
    }
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    return launch_grad_norm(grads, count, max_norm, out, static_cast<double*>(workspace), d,
                            static_cast<cudaStream_t>(stream));
}

int mx_adamw_step(const mx_adamw_tensor* tensors, int64_t count, const mx_adamw_opts* opts, const float* grad_scale,
                  float* amax_out, void* stream)
{
    Checks ok;
    ok.require(count >= 0 && count <= kMaxTensors && (tensors || count == 0) && opts);
    if (ok.rc != MX_OK)
        return ok.rc;
    const mx_adamw_opts& o = *opts;
    ok.require(std::isfinite(o.lr) && o.beta1 >= 0.0 && o.beta1 < 1.0 && o.beta2 >= 0.0 && o.beta2 < 1.0);
    ok.require(o.eps >= 0.0 && std::isfinite(o.eps) && (o.t >= 1 || o.t_at));
    ok.require(o.rounding == MX_ROUND_RNE || o.rounding == MX_ROUND_SR);
    ok.words(o.lr_at)(aligned(o.t_at, 8) ? MX_OK : MX_ERR_ALIGNMENT).words(grad_scale).words(amax_out);
    for (int64_t i = 0; ok.rc == MX_OK && i < count; ++i) {
        const mx_adamw_tensor& t = tensors[i];
        ok.require(t.n >= 0 && t.n <= kMaxFlat && valid_dtype(t.p_dtype) && valid_dtype(t.g_dtype));
        ok.require((t.bits == 8 || t.bits == 32) && std::isfinite(t.weight_decay));
        if (ok.rc != MX_OK)
            break;
        ok(t.copy && t.p_dtype != MX_OUT_F32 ? MX_ERR_UNSUPPORTED : MX_OK);
        ok.require(t.n == 0 || (t.param && t.m && t.v && (t.bits == 32 || (t.m_sf && t.v_sf))));
        const int state = t.bits == 8 ? 16 : 4;
        ok(aligned(t.param, dtype_bytes(t.p_dtype)) && aligned(t.grad, dtype_bytes(t.g_dtype)) && aligned(t.m, state) &&
                   aligned(t.v, state) && aligned(t.copy, 2)
               ? MX_OK
               : MX_ERR_ALIGNMENT);
    }
    Device d;
    if (ok.rc != MX_OK || ok(current_device(&d)).rc != MX_OK)
        return ok.rc;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (ok(zero(amax_out, static_cast<size_t>(count) * sizeof(float), s)).rc != MX_OK)
        return ok.rc;
    return launch_adamw(tensors, count, o, grad_scale, amax_out, d, s);
}

}  // extern "C"
