// train_api.cu -- the C ABI of the training operators (see include/credit.h):
// argument checks, workspace layout and dispatch.
#include <cuda_runtime.h>

#include <cmath>
#include <cstdint>

#include "credit.h"
#include "common.cuh"
#include "internal.h"
#include "planner.h"

using namespace credit;

namespace {

struct Span {  // a buffer of a call
    const void* p;
    uint64_t bytes;
};

bool overlap(const Span& a, const Span& b) {
    const uintptr_t x = (uintptr_t)a.p, y = (uintptr_t)b.p;
    return a.p && b.p && a.bytes && b.bytes && x < y + b.bytes && y < x + a.bytes;
}

// Every output is disjoint from every other buffer, except that a matrix
// output may be exactly a matrix input (in place: an element is read before
// the same thread writes it).  The first `mats` inputs and the first two
// outputs (one for credit_dropout) are the call's matrices.
bool buffers_ok(const Span* in, int nin, int mats, const Span* out, int nout) {
    for (int i = 0; i < nout; ++i) {
        for (int j = 0; j < nin; ++j) {
            const bool same = i < 2 && j < mats && in[j].p == out[i].p;
            if (!same && overlap(out[i], in[j])) return false;
        }
        for (int j = 0; j < i; ++j)
            if (overlap(out[i], out[j])) return false;
    }
    return true;
}

bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool dtype_ok(credit_dtype_t d) { return d == CREDIT_F32 || d == CREDIT_BF16; }
size_t esize(credit_dtype_t d) { return d == CREDIT_F32 ? 4 : 2; }

credit_status_t matrix_ok(int64_t rows, int64_t cols, credit_dtype_t dtype, uint64_t* bytes) {
    if (rows < 0 || cols < 1) return CREDIT_ERR_INVALID_ARG;
    if (!dtype_ok(dtype)) return CREDIT_ERR_UNSUPPORTED;
    const int64_t es = (int64_t)esize(dtype);
    if (rows > 0 && (rows > INT64_MAX / cols || rows * cols > INT64_MAX / es))
        return CREDIT_ERR_INVALID_ARG;
    if (cols > ((int64_t)1 << 30)) return CREDIT_ERR_INVALID_ARG;  // counted in 32 bits
    *bytes = (uint64_t)(rows * cols * es);
    return CREDIT_OK;
}

// A call's dropout: null or p = 0 is none.  The mask's counter holds the row
// in 32 bits.
credit_status_t drop_args(const credit_dropout_t* d, int64_t rows, DropArgs* a) {
    *a = DropArgs{};
    a->scale = 1.f;
    if (!d) return CREDIT_OK;
    if (!(d->p >= 0.0 && d->p < 1.0)) return CREDIT_ERR_INVALID_ARG;
    if (!aligned(d->device_offset, 8)) return CREDIT_ERR_INVALID_ARG;
    if (d->p == 0.0) return CREDIT_OK;
    if (rows > ((int64_t)1 << 32)) return CREDIT_ERR_INVALID_ARG;
    a->on = 1;
    a->threshold = (uint32_t)(uint64_t)std::floor(d->p * 4294967296.0);
    // the key of a round is the last one's plus two constants
    for (uint32_t i = 0; i < 10; ++i) {
        a->key[2 * i] = (uint32_t)d->seed + i * 0x9E3779B9u;
        a->key[2 * i + 1] = (uint32_t)(d->seed >> 32) + i * 0xBB67AE85u;
    }
    a->offset = d->offset;
    a->device_offset = d->device_offset;
    a->scale = (float)(1.0 / (1.0 - d->p));
    return CREDIT_OK;
}

credit_status_t device(int* dev, const DevInfo** info) {
    if (cudaGetDevice(dev) != cudaSuccess) { cudaGetLastError(); return CREDIT_ERR_CUDA; }
    *info = device_info(*dev);
    return *info ? CREDIT_OK : CREDIT_ERR_CUDA;
}

credit_status_t from_cuda(cudaError_t e) { return e == cudaSuccess ? CREDIT_OK : CREDIT_ERR_CUDA; }

// Workspace bytes of a backward call with this layout: the row sums, then the
// groups' sums.
uint64_t bwd_bytes(const TrainLayout& l) {
    return (uint64_t)(l.partials + 15) / 16 * 16 + (uint64_t)l.room_groups * 2 * (uint64_t)l.pitch * 4;
}

}  // namespace

extern "C" {

credit_status_t credit_norm_workspace(credit_op_t op, int backward, int64_t rows, int64_t cols,
                                      credit_dtype_t dtype, int device, size_t* bytes) {
    uint64_t mb;
    if (!bytes) return CREDIT_ERR_INVALID_ARG;
    if (op != CREDIT_LAYERNORM && op != CREDIT_RMSNORM) return CREDIT_ERR_UNSUPPORTED;
    const credit_status_t st = matrix_ok(rows, cols, dtype, &mb);
    if (st != CREDIT_OK) return st;
    const DevInfo* d = device_info(device);
    if (!d) return CREDIT_ERR_CUDA;
    *bytes = backward ? (size_t)bwd_bytes(norm_bwd_layout((int)dtype, rows, cols, d->sms, d->l2_bytes))
                      : (size_t)norm_fwd_partials((int)dtype, rows, cols, d->sms);
    return CREDIT_OK;
}

credit_status_t credit_dropout(const void* x, const void* residual, void* y, int64_t rows,
                               int64_t cols, credit_dtype_t dtype, const credit_dropout_t* drop,
                               void* stream) {
    uint64_t mb;
    credit_status_t st = matrix_ok(rows, cols, dtype, &mb);
    if (st != CREDIT_OK) return st;
    DropoutArgs a{};
    st = drop_args(drop, rows, &a.drop);
    if (st != CREDIT_OK) return st;
    if (rows == 0) return CREDIT_OK;
    if (!x || !y) return CREDIT_ERR_INVALID_ARG;
    const size_t es = esize(dtype);
    if (!aligned(x, es) || !aligned(y, es) || !aligned(residual, es)) return CREDIT_ERR_INVALID_ARG;
    const Span in[] = {{x, mb}, {residual, mb}, {a.drop.device_offset, 8}}, out[] = {{y, mb}};
    if (!buffers_ok(in, 3, 2, out, 1)) return CREDIT_ERR_INVALID_ARG;
    int dev;
    const DevInfo* d;
    st = device(&dev, &d);
    if (st != CREDIT_OK) return st;
    a.x = x;
    a.residual = residual;
    a.y = y;
    a.rows = rows;
    a.cols = cols;
    const bool vec = aligned(x, 16) && aligned(y, 16) && aligned(residual, 16) &&
                     (uint64_t)cols * es % 16 == 0;
    return from_cuda(launch_dropout((int)dtype, vec, a, d->sms, (cudaStream_t)stream));
}

credit_status_t credit_norm_forward(credit_op_t op, const void* x, const void* residual,
                                    const credit_dropout_t* drop, void* y, void* h, float* mean,
                                    float* rstd, int64_t rows, int64_t cols, credit_dtype_t dtype,
                                    const void* gamma, const void* beta,
                                    credit_dtype_t param_dtype, float eps, void* workspace,
                                    size_t workspace_bytes, void* stream) {
    if (op != CREDIT_LAYERNORM && op != CREDIT_RMSNORM) return CREDIT_ERR_UNSUPPORTED;
    uint64_t mb;
    credit_status_t st = matrix_ok(rows, cols, dtype, &mb);
    if (st != CREDIT_OK) return st;
    if ((gamma || beta) && !dtype_ok(param_dtype)) return CREDIT_ERR_UNSUPPORTED;
    if (!(eps >= 0.f)) return CREDIT_ERR_INVALID_ARG;
    if (op == CREDIT_RMSNORM && (beta || mean)) return CREDIT_ERR_INVALID_ARG;
    NormFwdArgs a{};
    st = drop_args(drop, rows, &a.drop);
    if (st != CREDIT_OK) return st;
    if (rows == 0) return CREDIT_OK;
    if (!x || !y) return CREDIT_ERR_INVALID_ARG;
    const size_t es = esize(dtype), ps = (gamma || beta) ? esize(param_dtype) : 1;
    if (!aligned(x, es) || !aligned(y, es) || !aligned(residual, es) || !aligned(h, es) ||
        !aligned(gamma, ps) || !aligned(beta, ps) || !aligned(mean, 4) || !aligned(rstd, 4))
        return CREDIT_ERR_INVALID_ARG;
    const uint64_t pb = (uint64_t)cols * ps, rb = (uint64_t)rows * 4;
    const Span in[] = {{x, mb}, {residual, mb}, {a.drop.device_offset, 8}, {gamma, pb}, {beta, pb}};
    const Span out[] = {{y, mb}, {h, mb}, {mean, rb}, {rstd, rb},
                        {workspace, workspace ? workspace_bytes : 0}};
    if (!buffers_ok(in, 5, 2, out, 5)) return CREDIT_ERR_INVALID_ARG;
    int dev;
    const DevInfo* d;
    st = device(&dev, &d);
    if (st != CREDIT_OK) return st;
    const uint64_t need = (uint64_t)norm_fwd_partials((int)dtype, rows, cols, d->sms);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return CREDIT_ERR_INVALID_ARG;
    a.x = x; a.residual = residual; a.y = y;
    // a copy of x that is x itself is not written
    a.h = h == x && !residual && !a.drop.on ? nullptr : h;
    a.mean = mean; a.rstd = rstd; a.gamma = gamma; a.beta = beta;
    a.rows = rows; a.cols = (int32_t)cols; a.inv_cols = 1.f / (float)cols; a.eps = eps;
    a.half = (gamma || beta) && param_dtype == CREDIT_BF16;
    a.ws = static_cast<float*>(workspace);
    a.nch = train_chunks((int)dtype, cols);
    a.l2_bytes = d->l2_bytes;
    const bool vec = aligned(x, 16) && aligned(y, 16) && aligned(residual, 16) && aligned(h, 16) &&
                     aligned(gamma, 16) && aligned(beta, 16) && (uint64_t)cols * es % 16 == 0;
    const TrainKey k{(int)op, (int)dtype, vec};
    return from_cuda(launch_norm_fwd(k, a, d->sms, (cudaStream_t)stream));
}

credit_status_t credit_norm_backward(credit_op_t op, const void* dy, const void* dh, const void* h,
                                     const float* mean, const float* rstd, const void* gamma,
                                     credit_dtype_t param_dtype, const credit_dropout_t* drop,
                                     void* dx, void* dresidual, void* dgamma, void* dbeta,
                                     int64_t rows, int64_t cols, credit_dtype_t dtype,
                                     void* workspace, size_t workspace_bytes, void* stream) {
    if (op != CREDIT_LAYERNORM && op != CREDIT_RMSNORM) return CREDIT_ERR_UNSUPPORTED;
    uint64_t mb;
    credit_status_t st = matrix_ok(rows, cols, dtype, &mb);
    if (st != CREDIT_OK) return st;
    const bool params = gamma || dgamma || dbeta;
    if (params && !dtype_ok(param_dtype)) return CREDIT_ERR_UNSUPPORTED;
    if (op == CREDIT_RMSNORM && (dbeta || mean)) return CREDIT_ERR_INVALID_ARG;
    NormBwdArgs a{};
    st = drop_args(drop, rows, &a.drop);
    if (st != CREDIT_OK) return st;
    if (rows == 0 && !dgamma && !dbeta) return CREDIT_OK;
    if (rows > 0 && (!dy || !h || !rstd || !dx || (op == CREDIT_LAYERNORM && !mean)))
        return CREDIT_ERR_INVALID_ARG;
    const size_t es = esize(dtype), ps = params ? esize(param_dtype) : 1;
    if (!aligned(dy, es) || !aligned(dh, es) || !aligned(h, es) || !aligned(dx, es) ||
        !aligned(dresidual, es) || !aligned(mean, 4) || !aligned(rstd, 4) || !aligned(gamma, ps) ||
        !aligned(dgamma, ps) || !aligned(dbeta, ps))
        return CREDIT_ERR_INVALID_ARG;
    const uint64_t pb = (uint64_t)cols * ps, rb = (uint64_t)rows * 4;
    const Span in[] = {{dy, mb}, {dh, mb}, {h, mb}, {mean, rb}, {rstd, rb}, {gamma, pb},
                       {a.drop.device_offset, 8}};
    const Span out[] = {{dx, mb}, {dresidual, mb}, {dgamma, pb}, {dbeta, pb},
                        {workspace, workspace ? workspace_bytes : 0}};
    if (!buffers_ok(in, 7, 3, out, 5)) return CREDIT_ERR_INVALID_ARG;
    int dev;
    const DevInfo* d;
    st = device(&dev, &d);
    if (st != CREDIT_OK) return st;
    const TrainLayout l = norm_bwd_layout((int)dtype, rows, cols, d->sms, d->l2_bytes);
    const uint64_t need = bwd_bytes(l);
    if (need && (!workspace || workspace_bytes < need || !aligned(workspace, 16)))
        return CREDIT_ERR_INVALID_ARG;
    a.dy = dy; a.dh = dh; a.h = h; a.mean = mean; a.rstd = rstd; a.gamma = gamma;
    a.dx = dx; a.dres = dresidual; a.dgamma = dgamma; a.dbeta = dbeta;
    a.rows = rows; a.cols = (int32_t)cols; a.inv_cols = 1.f / (float)cols;
    a.half = params && param_dtype == CREDIT_BF16;
    a.ws = static_cast<float*>(workspace);
    a.pws = reinterpret_cast<float*>(static_cast<char*>(workspace) + (l.partials + 15) / 16 * 16);
    a.pitch = l.pitch;
    a.nch = l.nch;
    a.groups = l.groups;
    a.batch = l.batch;
    const bool vec = aligned(dy, 16) && aligned(dh, 16) && aligned(h, 16) && aligned(dx, 16) &&
                     aligned(dresidual, 16) && aligned(gamma, 16) && (uint64_t)cols * es % 16 == 0;
    const TrainKey k{(int)op, (int)dtype, vec};
    return from_cuda(launch_norm_bwd(k, a, d->sms, (cudaStream_t)stream));
}

}  // extern "C"
