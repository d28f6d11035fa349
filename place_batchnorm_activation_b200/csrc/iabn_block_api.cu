// iabn_block_api.cu -- the extern "C" entry points declared in iabn_block.h:
// argument checks and launch.
#include <cuda_runtime.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>

#include <initializer_list>
#include <mutex>

#include "iabn_block.h"
#include "iabn_block_internal.h"
#include "iabn_device.cuh"

using namespace iabn;

namespace {

iabn_status from_cuda(cudaError_t e) {
    if (e == cudaSuccess) return IABN_OK;
    cudaGetLastError();   // clear a launch error so later calls are not blamed
    if (getenv("IABN_DEBUG")) fprintf(stderr, "iabn: CUDA error %d: %s\n", (int)e,
                                      cudaGetErrorString(e));
    return IABN_ERR_CUDA;
}

// SM count of the current device, queried once per device.
cudaError_t current_sms(int& sms) {
    static std::mutex mu;
    static int cache[64] = {0};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    std::lock_guard<std::mutex> lock(mu);
    int* slot = dev >= 0 && dev < 64 ? &cache[dev] : nullptr;
    if (slot && *slot) {
        sms = *slot;
        return cudaSuccess;
    }
    e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    if (e == cudaSuccess && slot) *slot = sms;
    return e;
}

int elem_size(int32_t dtype) { return dtype == IABN_F32 ? 4 : 2; }
bool good_dtype(int32_t t) { return t == IABN_F32 || t == IABN_BF16 || t == IABN_F16; }
bool good_format(int32_t f) { return f == IABN_Q8_E4M3 || f == IABN_Q8_INT8; }
bool good_norm(int32_t k) { return k == IABN_NORM_NONE || k == IABN_NORM_RMS || k == IABN_NORM_LAYER; }

// rows x cols of a tensor, within what 64-bit byte offsets hold.
iabn_status check_size(int64_t rows, int64_t cols, int64_t ld) {
    if (rows < 0 || cols < 1 || ld < cols) return IABN_ERR_INVALID_ARG;
    if (cols > ((int64_t)1 << 30) || rows > ((int64_t)1 << 40)) return IABN_ERR_UNSUPPORTED;
    if ((__int128)rows * ld > ((__int128)1 << 58)) return IABN_ERR_UNSUPPORTED;
    return IABN_OK;
}

// A tensor's memory: `rows` runs of `width` bytes, `stride` bytes apart.
struct Region {
    uintptr_t at;
    int64_t rows, width, stride;
};

Region region(const void* p, int64_t rows, int64_t cols, int64_t ld, int esize) {
    return {(uintptr_t)p, rows, cols * esize, ld * esize};
}

bool same(const Region& a, const Region& b) {
    return a.at == b.at && a.rows == b.rows && a.width == b.width &&
           (a.stride == b.stride || a.rows <= 1);
}

// False if the two share a byte (or, for unequal strides, if their ranges meet).
bool disjoint(const Region& a, const Region& b) {
    if (!a.at || !b.at || a.rows == 0 || b.rows == 0) return true;
    const uintptr_t ea = a.at + (uintptr_t)((a.rows - 1) * a.stride + a.width);
    const uintptr_t eb = b.at + (uintptr_t)((b.rows - 1) * b.stride + b.width);
    if (ea <= b.at || eb <= a.at) return true;
    if (a.stride != b.stride) return false;
    // equal strides: compare where the runs lie within a stride
    const uintptr_t L = (uintptr_t)a.stride;
    const uintptr_t d = b.at >= a.at ? (b.at - a.at) % L : (L - (a.at - b.at) % L) % L;
    return d >= (uintptr_t)a.width && d + (uintptr_t)b.width <= L;
}

Region floats(const void* p, int64_t rows, int64_t cols) { return region(p, rows, cols, cols, 4); }

// A call's tensors.  Outputs are disjoint from each other and from the inputs,
// but for an output in the storage type, which may be an input in it.
struct Overlaps {
    struct Tensor {
        Region at;
        bool storage;
    } in[16], out[16];
    int ni = 0, no = 0;
    void input(const Region& r) { add(in, ni, r, true); }
    void output(const Region& r) { add(out, no, r, true); }
    void other_input(const Region& r) { add(in, ni, r, false); }     // codes, scales, parameters, statistics
    void other_output(const Region& r) { add(out, no, r, false); }   // these, gradients of parameters, workspace
    bool ok() const {
        for (int i = 0; i < no; ++i) {
            for (int j = 0; j < i; ++j)
                if (!disjoint(out[i].at, out[j].at)) return false;
            for (int j = 0; j < ni; ++j)
                if (!disjoint(out[i].at, in[j].at) &&
                    !(out[i].storage && in[j].storage && same(out[i].at, in[j].at)))
                    return false;
        }
        return true;
    }

private:
    static void add(Tensor* list, int& n, const Region& r, bool storage) {
        if (r.at && r.rows > 0) list[n++] = {r, storage};
    }
};

bool misaligned(int size, std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if ((uintptr_t)p % (uintptr_t)size) return true;
    return false;
}

iabn_status check_block_desc(const iabn_block_desc* d) {
    if (!d) return IABN_ERR_INVALID_ARG;
    if (!good_dtype(d->dtype) || !good_norm(d->post) || !good_norm(d->pre)) return IABN_ERR_INVALID_ARG;
    if (d->rows_per_gate < 0) return IABN_ERR_INVALID_ARG;
    if (!isfinite(d->residual_scale) || !(d->eps_post >= 0.f) || !isfinite(d->eps_post) ||
        !(d->eps_pre >= 0.f) || !isfinite(d->eps_pre))
        return IABN_ERR_INVALID_ARG;
    const iabn_status st = check_size(d->rows, d->cols, d->cols);
    if (st != IABN_OK) return st;
    if (d->cols > IABN_BLOCK_MAX_COLS || d->rows > 0x7fffffff) return IABN_ERR_UNSUPPORTED;
    return IABN_OK;
}

int64_t gate_rows(const iabn_block_desc* d) {
    if (d->rows_per_gate == 0) return 1;
    return d->rows / d->rows_per_gate + (d->rows % d->rows_per_gate != 0);
}

Region whole(const iabn_block_desc* d, const void* p) {
    return region(p, d->rows, d->cols, d->cols, elem_size(d->dtype));
}
Region bytes(const iabn_block_desc* d, const void* p) {
    return region(p, d->rows, d->cols, d->cols, 1);
}

iabn_status block_fwd_call(const iabn_block_desc* d, const void* u, const void* h, void* h_out,
                           void* n, const float* gamma_post, const float* beta_post,
                           const float* gate, const float* gamma_pre, const float* beta_pre,
                           float* mean_post, float* rstd_post, float* mean_pre, float* rstd_pre,
                           void* q_post, float* scale_post, void* q_pre, float* scale_pre,
                           void* stream) {
    iabn_status st = check_block_desc(d);
    if (st != IABN_OK) return st;
    if (d->post == IABN_NORM_NONE && (gamma_post || beta_post || rstd_post)) return IABN_ERR_INVALID_ARG;
    if (d->pre == IABN_NORM_NONE && (gamma_pre || beta_pre || rstd_pre || q_pre || scale_pre))
        return IABN_ERR_INVALID_ARG;
    if ((mean_post && d->post != IABN_NORM_LAYER) || (mean_pre && d->pre != IABN_NORM_LAYER))
        return IABN_ERR_INVALID_ARG;
    if (!q_post != !scale_post || !q_pre != !scale_pre) return IABN_ERR_INVALID_ARG;
    if (d->rows == 0) return IABN_OK;
    if (!h || (!h_out && !n) || !n != (d->pre == IABN_NORM_NONE)) return IABN_ERR_INVALID_ARG;
    if (!u && (d->post != IABN_NORM_NONE || gate || d->residual_scale != 1.f || h_out || q_post))
        return IABN_ERR_INVALID_ARG;
    if (misaligned(elem_size(d->dtype), {u, h, h_out, n}) ||
        misaligned(4, {gamma_post, beta_post, gate, gamma_pre, beta_pre, mean_post, rstd_post,
                       mean_pre, rstd_pre, scale_post, scale_pre}))
        return IABN_ERR_MISALIGNED;
    Overlaps o;
    o.input(whole(d, u));
    o.input(whole(d, h));
    o.output(whole(d, h_out));
    o.output(whole(d, n));
    o.other_output(bytes(d, q_post));
    o.other_output(bytes(d, q_pre));
    for (const float* p : {scale_post, scale_pre}) o.other_output(floats(p, d->rows, q_groups(d->cols)));
    for (const float* p : {mean_post, rstd_post, mean_pre, rstd_pre}) o.other_output(floats(p, d->rows, 1));
    for (const float* p : {gamma_post, beta_post, gamma_pre, beta_pre}) o.other_input(floats(p, 1, d->cols));
    o.other_input(floats(gate, gate_rows(d), d->cols));
    if (!o.ok()) return IABN_ERR_INVALID_ARG;
    int sms = 0;
    const cudaError_t e = current_sms(sms);
    if (e != cudaSuccess) return from_cuda(e);
    BlockFwd a{};
    a.u = u;
    a.h = h;
    a.h_out = h_out;
    a.n = n;
    a.gamma_post = gamma_post;
    a.beta_post = beta_post;
    a.gate = gate;
    a.gamma_pre = gamma_pre;
    a.beta_pre = beta_pre;
    a.mean_post = mean_post;
    a.rstd_post = rstd_post;
    a.mean_pre = mean_pre;
    a.rstd_pre = rstd_pre;
    a.q_post = static_cast<uint8_t*>(q_post);
    a.q_pre = static_cast<uint8_t*>(q_pre);
    a.scale_post = scale_post;
    a.scale_pre = scale_pre;
    a.rows = d->rows;
    a.rows_per_gate = d->rows_per_gate;
    a.cols = (int)d->cols;
    a.groups = (int)q_groups(d->cols);
    a.post = d->post;
    a.pre = d->pre;
    a.format = d->format;
    a.alpha = d->residual_scale;
    a.eps_post = d->eps_post;
    a.eps_pre = d->eps_pre;
    return from_cuda(block_forward(a, d->dtype, static_cast<cudaStream_t>(stream), sms));
}

size_t block_ws_bytes(const iabn_block_desc* d) {
    const int64_t workers = block_bwd_workers(d->rows, d->cols);
    const int64_t rows = 2 * block_bwd_slots(workers, gate_rows(d)) + 2 * workers;
    return ((size_t)rows * (size_t)((d->cols + 3) / 4 * 4) * sizeof(float) + 255) / 256 * 256;
}

iabn_status block_bwd_call(const iabn_block_desc* d, bool codes, const void* su,
                           const float* scale_post, const void* sh, const float* scale_pre,
                           const void* dh_out, const void* dn, void* dh, void* du,
                           const float* gamma_post, const float* beta_post, const float* gate,
                           const float* gamma_pre, const float* mean_post,
                           const float* rstd_post, const float* mean_pre, const float* rstd_pre,
                           float* dgamma_post, float* dbeta_post, float* dgate,
                           float* dgamma_pre, float* dbeta_pre, void* workspace,
                           size_t ws_bytes, void* stream) {
    iabn_status st = check_block_desc(d);
    if (st != IABN_OK) return st;
    if (codes && !good_format(d->format)) return IABN_ERR_INVALID_ARG;
    const bool post = d->post != IABN_NORM_NONE, pre = d->pre != IABN_NORM_NONE;
    if (!post && (gamma_post || beta_post || dgamma_post || dbeta_post)) return IABN_ERR_INVALID_ARG;
    if (!pre && (gamma_pre || dgamma_pre || dbeta_pre)) return IABN_ERR_INVALID_ARG;
    if (dgate && !gate) return IABN_ERR_INVALID_ARG;
    const bool need_u = post || dgate;
    if (d->rows > 0) {
        if (!dh || (!dh_out && !dn) || !dn != !pre) return IABN_ERR_INVALID_ARG;
        if (need_u && (!su || (codes && !scale_post))) return IABN_ERR_INVALID_ARG;
        if (pre && (!sh || (codes && !scale_pre))) return IABN_ERR_INVALID_ARG;
        if ((post && !rstd_post) || (pre && !rstd_pre)) return IABN_ERR_INVALID_ARG;
        if (!codes && ((d->post == IABN_NORM_LAYER && !mean_post) ||
                       (d->pre == IABN_NORM_LAYER && !mean_pre)))
            return IABN_ERR_INVALID_ARG;
    }
    if (!need_u) su = nullptr;
    if (!pre) sh = nullptr;
    if (misaligned(elem_size(d->dtype), {dh_out, dn, dh, du}) ||
        (!codes && misaligned(elem_size(d->dtype), {su, sh})) ||
        misaligned(4, {scale_post, scale_pre, gamma_post, beta_post, gate, gamma_pre, mean_post,
                       rstd_post, mean_pre, rstd_pre, dgamma_post, dbeta_post, dgate, dgamma_pre,
                       dbeta_pre}))
        return IABN_ERR_MISALIGNED;
    Overlaps o;
    o.input(whole(d, dh_out));
    o.input(whole(d, dn));
    if (codes) {
        o.other_input(bytes(d, su));
        o.other_input(bytes(d, sh));
        if (su) o.other_input(floats(scale_post, d->rows, q_groups(d->cols)));
        if (sh) o.other_input(floats(scale_pre, d->rows, q_groups(d->cols)));
    } else {
        o.input(whole(d, su));
        o.input(whole(d, sh));
    }
    for (const float* p : {gamma_post, beta_post, gamma_pre}) o.other_input(floats(p, 1, d->cols));
    o.other_input(floats(gate, gate_rows(d), d->cols));
    for (const float* p : {mean_post, rstd_post, mean_pre, rstd_pre}) o.other_input(floats(p, d->rows, 1));
    o.output(whole(d, dh));
    o.output(whole(d, du));
    for (const float* p : {dgamma_post, dbeta_post, dgamma_pre, dbeta_pre}) o.other_output(floats(p, 1, d->cols));
    o.other_output(floats(dgate, gate_rows(d), d->cols));
    const size_t need = block_ws_bytes(d);
    o.other_output(region(workspace, 1, (int64_t)need, (int64_t)need, 1));
    if (!o.ok()) return IABN_ERR_INVALID_ARG;
    if (!workspace || ws_bytes < need || misaligned(16, {workspace}))
        return IABN_ERR_WORKSPACE;
    int sms = 0;
    const cudaError_t e = current_sms(sms);
    if (e != cudaSuccess) return from_cuda(e);
    BlockBwd a{};
    a.su = su;
    a.sh = sh;
    a.scale_post = scale_post;
    a.scale_pre = scale_pre;
    a.dh_out = dh_out;
    a.dn = dn;
    a.dh = dh;
    a.du = du;
    a.gamma_post = gamma_post;
    a.beta_post = beta_post;
    a.gate = gate;
    a.gamma_pre = gamma_pre;
    a.mean_post = d->post == IABN_NORM_LAYER ? mean_post : nullptr;
    a.rstd_post = post ? rstd_post : nullptr;
    a.mean_pre = d->pre == IABN_NORM_LAYER ? mean_pre : nullptr;
    a.rstd_pre = pre ? rstd_pre : nullptr;
    a.dgamma_post = dgamma_post;
    a.dbeta_post = dbeta_post;
    a.dgate = dgate;
    a.dgamma_pre = dgamma_pre;
    a.dbeta_pre = dbeta_pre;
    a.work = static_cast<float*>(workspace);
    a.rows = d->rows;
    a.rows_per_gate = gate ? d->rows_per_gate : 0;
    a.gates = gate ? gate_rows(d) : 1;
    a.workers = block_bwd_workers(d->rows, d->cols);
    a.cols = (int)d->cols;
    a.groups = (int)q_groups(d->cols);
    a.post = d->post;
    a.pre = d->pre;
    a.format = d->format;
    a.alpha = d->residual_scale;
    return from_cuda(block_backward(a, d->dtype, codes, static_cast<cudaStream_t>(stream), sms));
}

iabn_status check_gated_desc(const iabn_gated_desc* d, bool codes, bool back, bool reads_ab) {
    if (!d) return IABN_ERR_INVALID_ARG;
    if (!good_dtype(d->dtype) || (codes && !good_format(d->format))) return IABN_ERR_INVALID_ARG;
    if (d->act != IABN_GLU_SILU && d->act != IABN_GLU_GELU && d->act != IABN_GLU_GELU_TANH)
        return IABN_ERR_INVALID_ARG;
    iabn_status st = check_size(d->rows, d->cols, reads_ab ? d->ld : d->cols);
    if (st == IABN_OK && back) st = check_size(d->rows, d->cols, d->ld_grad);
    return st;
}

iabn_status gated_fwd_call(const iabn_gated_desc* d, const void* a, const void* b, void* z,
                           bool codes, void* qa, float* sa, void* qb, float* sb, void* stream) {
    const iabn_status st = check_gated_desc(d, codes, false, true);
    if (st != IABN_OK) return st;
    if (d->rows == 0) return IABN_OK;
    if (!a || !b || !z || (codes && (!qa || !sa || !qb || !sb))) return IABN_ERR_INVALID_ARG;
    const int es = elem_size(d->dtype);
    if (misaligned(es, {a, b, z}) || misaligned(4, {sa, sb})) return IABN_ERR_MISALIGNED;
    Overlaps o;
    o.input(region(a, d->rows, d->cols, d->ld, es));
    o.input(region(b, d->rows, d->cols, d->ld, es));
    o.output(region(z, d->rows, d->cols, d->cols, es));
    for (const void* q : {qa, qb}) o.other_output(region(q, d->rows, d->cols, d->cols, 1));
    for (const float* p : {sa, sb}) o.other_output(floats(p, d->rows, q_groups(d->cols)));
    if (!o.ok()) return IABN_ERR_INVALID_ARG;
    int sms = 0;
    const cudaError_t e = current_sms(sms);
    if (e != cudaSuccess) return from_cuda(e);
    Gated g{};
    g.a = a;
    g.b = b;
    g.z = z;
    g.qa_out = static_cast<uint8_t*>(qa);
    g.qb_out = static_cast<uint8_t*>(qb);
    g.sa_out = sa;
    g.sb_out = sb;
    g.rows = d->rows;
    g.cols = d->cols;
    g.ld = d->ld;
    g.act = d->act;
    g.format = d->format;
    return from_cuda(gated_forward(g, d->dtype, static_cast<cudaStream_t>(stream), sms));
}

iabn_status gated_bwd_call(const iabn_gated_desc* d, bool codes, const void* a, const float* sa,
                           const void* b, const float* sb, const void* dz, void* da, void* db,
                           void* z, void* stream) {
    const iabn_status st = check_gated_desc(d, codes, true, !codes);
    if (st != IABN_OK) return st;
    if (d->rows == 0) return IABN_OK;
    if (!a || !b || !dz || !da || !db || (codes && (!sa || !sb))) return IABN_ERR_INVALID_ARG;
    const int es = elem_size(d->dtype);
    if (misaligned(es, {dz, da, db, z}) || (!codes && misaligned(es, {a, b})) ||
        misaligned(4, {sa, sb}))
        return IABN_ERR_MISALIGNED;
    Overlaps o;
    o.input(region(dz, d->rows, d->cols, d->cols, es));
    if (codes) {
        for (const void* q : {a, b}) o.other_input(region(q, d->rows, d->cols, d->cols, 1));
        for (const float* p : {sa, sb}) o.other_input(floats(p, d->rows, q_groups(d->cols)));
    } else {
        o.input(region(a, d->rows, d->cols, d->ld, es));
        o.input(region(b, d->rows, d->cols, d->ld, es));
    }
    o.output(region(da, d->rows, d->cols, d->ld_grad, es));
    o.output(region(db, d->rows, d->cols, d->ld_grad, es));
    o.output(region(z, d->rows, d->cols, d->cols, es));
    if (!o.ok()) return IABN_ERR_INVALID_ARG;
    int sms = 0;
    const cudaError_t e = current_sms(sms);
    if (e != cudaSuccess) return from_cuda(e);
    Gated g{};
    if (codes) {
        g.qa = static_cast<const uint8_t*>(a);
        g.qb = static_cast<const uint8_t*>(b);
        g.sa = sa;
        g.sb = sb;
    } else {
        g.a = a;
        g.b = b;
        g.ld = d->ld;
    }
    g.dz = dz;
    g.da = da;
    g.db = db;
    g.z = z;
    g.rows = d->rows;
    g.cols = d->cols;
    g.ld_grad = d->ld_grad;
    g.act = d->act;
    g.format = d->format;
    return from_cuda(gated_backward(g, d->dtype, codes, static_cast<cudaStream_t>(stream), sms));
}

iabn_status check8_call(bool load, int64_t rows, int64_t cols, int64_t ld, int32_t dtype,
                        int32_t format, const void* x, void* y, const void* q, const float* scale,
                        const float* gamma, const float* beta, void* stream) {
    if (!good_dtype(dtype) || !good_format(format)) return IABN_ERR_INVALID_ARG;
    const iabn_status st = check_size(rows, cols, ld);
    if (st != IABN_OK) return st;
    if (rows == 0) return IABN_OK;
    const void* t = load ? y : x;
    if (!t || !q || !scale) return IABN_ERR_INVALID_ARG;
    const int es = elem_size(dtype);
    if (misaligned(es, {t}) || misaligned(4, {scale, gamma, beta})) return IABN_ERR_MISALIGNED;
    Overlaps o;
    if (load) {
        o.output(region(y, rows, cols, ld, es));
        o.other_input(region(q, rows, cols, cols, 1));
        o.other_input(floats(scale, rows, q_groups(cols)));
        for (const float* p : {gamma, beta}) o.other_input(floats(p, 1, cols));
    } else {
        o.input(region(x, rows, cols, ld, es));
        o.other_output(region(q, rows, cols, cols, 1));
        o.other_output(floats(scale, rows, q_groups(cols)));
    }
    if (!o.ok()) return IABN_ERR_INVALID_ARG;
    int sms = 0;
    const cudaError_t e = current_sms(sms);
    if (e != cudaSuccess) return from_cuda(e);
    Check8 a{};
    a.x = x;
    a.y = y;
    a.q = const_cast<uint8_t*>(static_cast<const uint8_t*>(q));
    a.scale = const_cast<float*>(scale);
    a.gamma = gamma;
    a.beta = beta;
    a.rows = rows;
    a.cols = cols;
    a.ld = ld;
    a.format = format;
    const cudaStream_t s = static_cast<cudaStream_t>(stream);
    return from_cuda(load ? check8_load(a, dtype, s, sms) : check8_store(a, dtype, s, sms));
}

}  // namespace

extern "C" iabn_status iabn_checkpoint8_store(int64_t rows, int64_t cols, int64_t ldx,
                                              int32_t dtype, int32_t format, const void* x,
                                              void* q, float* scale, void* stream) {
    return check8_call(false, rows, cols, ldx, dtype, format, x, nullptr, q, scale, nullptr,
                       nullptr, stream);
}

extern "C" iabn_status iabn_checkpoint8_load(int64_t rows, int64_t cols, int64_t ldy,
                                             int32_t dtype, int32_t format, const void* q,
                                             const float* scale, const float* gamma,
                                             const float* beta, void* y, void* stream) {
    return check8_call(true, rows, cols, ldy, dtype, format, nullptr, y, q, scale, gamma, beta,
                       stream);
}

extern "C" iabn_status iabn_block_norm_forward(
    const iabn_block_desc* d, const void* u, const void* h, void* h_out, void* n,
    const float* gamma_post, const float* beta_post, const float* gate, const float* gamma_pre,
    const float* beta_pre, float* mean_post, float* rstd_post, float* mean_pre, float* rstd_pre,
    void* stream) {
    return block_fwd_call(d, u, h, h_out, n, gamma_post, beta_post, gate, gamma_pre, beta_pre,
                          mean_post, rstd_post, mean_pre, rstd_pre, nullptr, nullptr, nullptr,
                          nullptr, stream);
}

extern "C" iabn_status iabn_block_norm_forward_checkpoint8(
    const iabn_block_desc* d, const void* u, const void* h, void* h_out, void* n,
    const float* gamma_post, const float* beta_post, const float* gate, const float* gamma_pre,
    const float* beta_pre, float* rstd_post, float* rstd_pre, void* q_post, float* scale_post,
    void* q_pre, float* scale_pre, void* stream) {
    if (d && !good_format(d->format)) return IABN_ERR_INVALID_ARG;
    return block_fwd_call(d, u, h, h_out, n, gamma_post, beta_post, gate, gamma_pre, beta_pre,
                          nullptr, rstd_post, nullptr, rstd_pre, q_post, scale_post, q_pre,
                          scale_pre, stream);
}

extern "C" size_t iabn_block_norm_workspace_size(const iabn_block_desc* d) {
    if (!d || d->rows_per_gate < 0 || check_size(d->rows, d->cols, d->cols) != IABN_OK ||
        d->cols > IABN_BLOCK_MAX_COLS || d->rows > 0x7fffffff)
        return 0;
    return block_ws_bytes(d);
}

extern "C" iabn_status iabn_block_norm_backward(
    const iabn_block_desc* d, const void* u, const void* h_out, const void* dh_out,
    const void* dn, void* dh, void* du, const float* gamma_post, const float* beta_post,
    const float* gate, const float* gamma_pre, const float* mean_post, const float* rstd_post,
    const float* mean_pre, const float* rstd_pre, float* dgamma_post, float* dbeta_post,
    float* dgate, float* dgamma_pre, float* dbeta_pre, void* workspace, size_t ws_bytes,
    void* stream) {
    return block_bwd_call(d, false, u, nullptr, h_out, nullptr, dh_out, dn, dh, du, gamma_post,
                          beta_post, gate, gamma_pre, mean_post, rstd_post, mean_pre, rstd_pre,
                          dgamma_post, dbeta_post, dgate, dgamma_pre, dbeta_pre, workspace,
                          ws_bytes, stream);
}

extern "C" iabn_status iabn_block_norm_backward_checkpoint8(
    const iabn_block_desc* d, const void* q_post, const float* scale_post, const void* q_pre,
    const float* scale_pre, const void* dh_out, const void* dn, void* dh, void* du,
    const float* gamma_post, const float* beta_post, const float* gate, const float* gamma_pre,
    const float* rstd_post, const float* rstd_pre, float* dgamma_post, float* dbeta_post,
    float* dgate, float* dgamma_pre, float* dbeta_pre, void* workspace, size_t ws_bytes,
    void* stream) {
    return block_bwd_call(d, true, q_post, scale_post, q_pre, scale_pre, dh_out, dn, dh, du,
                          gamma_post, beta_post, gate, gamma_pre, nullptr, rstd_post, nullptr,
                          rstd_pre, dgamma_post, dbeta_post, dgate, dgamma_pre, dbeta_pre,
                          workspace, ws_bytes, stream);
}

extern "C" iabn_status iabn_gated_forward(const iabn_gated_desc* d, const void* a, const void* b,
                                          void* z, void* stream) {
    return gated_fwd_call(d, a, b, z, false, nullptr, nullptr, nullptr, nullptr, stream);
}

extern "C" iabn_status iabn_gated_forward_checkpoint8(const iabn_gated_desc* d, const void* a,
                                                      const void* b, void* z, void* qa,
                                                      float* scale_a, void* qb, float* scale_b,
                                                      void* stream) {
    return gated_fwd_call(d, a, b, z, true, qa, scale_a, qb, scale_b, stream);
}

extern "C" iabn_status iabn_gated_backward(const iabn_gated_desc* d, const void* a, const void* b,
                                           const void* dz, void* da, void* db, void* z_out,
                                           void* stream) {
    return gated_bwd_call(d, false, a, nullptr, b, nullptr, dz, da, db, z_out, stream);
}

extern "C" iabn_status iabn_gated_backward_checkpoint8(const iabn_gated_desc* d, const void* qa,
                                                       const float* scale_a, const void* qb,
                                                       const float* scale_b, const void* dz,
                                                       void* da, void* db, void* z_out,
                                                       void* stream) {
    return gated_bwd_call(d, true, qa, scale_a, qb, scale_b, dz, da, db, z_out, stream);
}
