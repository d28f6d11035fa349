// iabn_gated.cu -- the gated activation z = phi(a) b and its backward, with
// or without 8-bit checkpoints of a and b.
//
// Each phi is written as a w(a), w the logistic function of a (SILU), of
// 2 sqrt(2/pi) (a + 0.044715 a^3) (GELU_TANH: (1 + tanh y)/2 = 1/(1 + e^-2y),
// which does not cancel for large negative y), or the normal distribution
// function (GELU), so phi' = w + a w'.
// Elementwise; a warp takes 256 columns of a row at a time (two checkpoint
// groups).  Bound: HBM bandwidth: 3 s bytes an element forward (2 more with
// checkpoints), 3 s + 2 backward from codes, s more for z.
#include "iabn_rows.cuh"

namespace iabn {

void count_launches(int n);

namespace {

template <int DT>
__device__ __forceinline__ float exp_of(float x) {
    return DT == kF32 ? expf(x) : __expf(x);
}
template <int DT>
__device__ __forceinline__ float inverse(float x) {   // of 1 + e^y: in [1, inf]
    return DT == kF32 ? 1.f / x : __fdividef(1.f, x);
}

// w(a), and a w'(a) where SLOPE.
template <int ACT, int DT, bool SLOPE>
__device__ __forceinline__ void weight(float a, float& w, float& aw) {
    if (ACT == kSilu) {
        w = inverse<DT>(1.f + exp_of<DT>(-a));
        if (SLOPE) aw = a * w * (1.f - w);
    } else if (ACT == kGelu) {
        w = 0.5f * erfcf(a * -0.70710678118654752f);
        if (SLOPE) aw = a * 0.39894228040143268f * exp_of<DT>(-0.5f * a * a);
    } else {
        // beyond +-32 w is 0 or 1 in fp32: the clamp keeps a^3 finite
        const float c = fminf(fmaxf(a, -32.f), 32.f);
        const float q = 0.044715f * c * c;
        w = inverse<DT>(1.f + exp_of<DT>(-1.5957691216057308f * c * (1.f + q)));
        if (SLOPE) aw = c * w * (1.f - w) * 1.5957691216057308f * fmaf(3.f, q, 1.f);
        if (a != a) w = a;
    }
}

// Rows and segments of a warp's walk over [rows, cols] in steps of all warps.
struct Walk {
    int64_t row;
    int seg;
    int64_t drow;
    int dseg, segs;
    __device__ __forceinline__ Walk(int64_t cols) {
        segs = (int)((cols + kSeg - 1) / kSeg);
        const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
        const int64_t at = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
        row = at / segs;
        seg = (int)(at - row * segs);
        drow = warps / segs;
        dseg = (int)(warps - drow * segs);
    }
    __device__ __forceinline__ void next() {
        row += drow;
        seg += dseg;
        if (seg >= segs) {
            seg -= segs;
            ++row;
        }
    }
};

template <int DT, bool VEC, int ACT>
__global__ void __launch_bounds__(256) gated_fwd(const Gated p) {
    using T = typename Storage<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for (Walk k(p.cols); k.row < p.rows; k.next()) {
        const int64_t c0 = (int64_t)k.seg * kSeg;
        const int left = (int)min(p.cols - c0, (int64_t)kSeg);
        Raw<DT, VEC> ra, rb;
        ra.load(static_cast<const T*>(p.a) + k.row * p.ld + c0, lane, left);
        rb.load(static_cast<const T*>(p.b) + k.row * p.ld + c0, lane, left);
        float a[kEl], b[kEl], z[kEl];
        ra.get(a);
        rb.get(b);
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
            float w, aw;
            weight<ACT, DT, false>(a[j], w, aw);
            z[j] = a[j] * w * b[j];
        }
        store8<DT, VEC>(static_cast<T*>(p.z) + k.row * p.cols + c0, lane, left, z);
        if (p.qa_out) {
            const int64_t at = k.row * p.cols + c0;
            quantise8<VEC>(p.format, a, p.qa_out + at, p.sa_out + k.row * groups, c0, lane, left);
            quantise8<VEC>(p.format, b, p.qb_out + at, p.sb_out + k.row * groups, c0, lane, left);
        }
    }
}

template <int DT, bool VEC, int ACT, bool CODES>
__global__ void __launch_bounds__(256) gated_bwd(const Gated p) {
    using T = typename Storage<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for (Walk k(p.cols); k.row < p.rows; k.next()) {
        const int64_t c0 = (int64_t)k.seg * kSeg;
        const int left = (int)min(p.cols - c0, (int64_t)kSeg);
        const int64_t at = k.row * p.cols + c0;
        float a[kEl], b[kEl], dz[kEl];
        Raw<DT, VEC> rz;
        rz.load(static_cast<const T*>(p.dz) + at, lane, left);
        if (CODES) {
            Codes<VEC> qa, qb;
            float sa[2], sb[2];
            qa.load(p.qa + at, lane, left);
            qb.load(p.qb + at, lane, left);
            load_scales<VEC>(p.sa + k.row * groups, c0, lane, left, sa);
            load_scales<VEC>(p.sb + k.row * groups, c0, lane, left, sb);
            qa.get(p.format, sa, a);
            qb.get(p.format, sb, b);
        } else {
            Raw<DT, VEC> ra, rb;
            ra.load(static_cast<const T*>(p.a) + k.row * p.ld + c0, lane, left);
            rb.load(static_cast<const T*>(p.b) + k.row * p.ld + c0, lane, left);
            ra.get(a);
            rb.get(b);
        }
        rz.get(dz);
        float da[kEl], db[kEl], z[kEl];
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
            float w, aw;
            weight<ACT, DT, true>(a[j], w, aw);
            const float phi = a[j] * w;
            da[j] = dz[j] * b[j] * (w + aw);
            db[j] = dz[j] * phi;
            z[j] = phi * b[j];
        }
        store8<DT, VEC>(static_cast<T*>(p.da) + k.row * p.ld_grad + c0, lane, left, da);
        store8<DT, VEC>(static_cast<T*>(p.db) + k.row * p.ld_grad + c0, lane, left, db);
        if (p.z) store8<DT, VEC>(static_cast<T*>(p.z) + at, lane, left, z);
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(256) store_kernel(const Check8 p) {
    using T = typename Storage<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for (Walk k(p.cols); k.row < p.rows; k.next()) {
        const int64_t c0 = (int64_t)k.seg * kSeg;
        const int left = (int)min(p.cols - c0, (int64_t)kSeg);
        Raw<DT, VEC> r;
        r.load(static_cast<const T*>(p.x) + k.row * p.ld + c0, lane, left);
        float x[kEl];
        r.get(x);
        quantise8<VEC>(p.format, x, p.q + k.row * p.cols + c0, p.scale + k.row * groups, c0, lane, left);
    }
}

template <int DT, bool VEC>
__global__ void __launch_bounds__(256) load_kernel(const Check8 p) {
    using T = typename Storage<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for (Walk k(p.cols); k.row < p.rows; k.next()) {
        const int64_t c0 = (int64_t)k.seg * kSeg;
        const int left = (int)min(p.cols - c0, (int64_t)kSeg);
        Codes<VEC> q;
        float s[2], x[kEl], ga[kEl], be[kEl];
        q.load(p.q + k.row * p.cols + c0, lane, left);
        load_scales<VEC>(p.scale + k.row * groups, c0, lane, left, s);
        q.get(p.format, s, x);
        load_param<VEC>(p.gamma, c0, lane, left, 1.f, ga);
        load_param<VEC>(p.beta, c0, lane, left, 0.f, be);
#pragma unroll
        for (int j = 0; j < kEl; ++j) x[j] = fmaf(ga[j], x[j], be[j]);
        store8<DT, VEC>(static_cast<T*>(p.y) + k.row * p.ld + c0, lane, left, x);
    }
}

// Blocks of 8 warps: as many as there are segments, at most eight waves.
unsigned blocks(int64_t rows, int64_t cols, int sms) {
    const int64_t segs = (cols + kSeg - 1) / kSeg;
    const int64_t most = (int64_t)sms * 64;
    if (rows >= most * 8 / segs + 1) return (unsigned)most;
    const int64_t need = (rows * segs + 7) / 8;
    return (unsigned)(need < most ? need : most);
}

template <int DT, bool VEC, int ACT>
void run_gated(const Gated& a, bool back, bool codes, unsigned n, cudaStream_t s) {
    if (!back) gated_fwd<DT, VEC, ACT><<<n, 256, 0, s>>>(a);
    else if (codes) gated_bwd<DT, VEC, ACT, true><<<n, 256, 0, s>>>(a);
    else gated_bwd<DT, VEC, ACT, false><<<n, 256, 0, s>>>(a);
}

template <int DT, bool VEC>
void by_act(const Gated& a, bool back, bool codes, unsigned n, cudaStream_t s) {
    if (a.act == kSilu) run_gated<DT, VEC, kSilu>(a, back, codes, n, s);
    else if (a.act == kGelu) run_gated<DT, VEC, kGelu>(a, back, codes, n, s);
    else run_gated<DT, VEC, kGeluTanh>(a, back, codes, n, s);
}

template <int DT>
void by_vec(const Gated& a, bool vec, bool back, bool codes, unsigned n, cudaStream_t s) {
    if (vec) by_act<DT, true>(a, back, codes, n, s);
    else by_act<DT, false>(a, back, codes, n, s);
}

cudaError_t run(const Gated& a, int dtype, bool back, bool codes, cudaStream_t s, int sms) {
    if (a.rows == 0) return cudaSuccess;
    const bool strides = (codes || a.ld % kEl == 0) && (!back || a.ld_grad % kEl == 0);
    const bool vec = a.cols % kEl == 0 && strides && on16(a.a) && on16(a.b) && on16(a.qa) &&
                     on16(a.qb) && on16(a.qa_out) && on16(a.qb_out) && on16(a.dz) && on16(a.z) &&
                     on16(a.da) && on16(a.db);
    const unsigned n = blocks(a.rows, a.cols, sms);
    if (dtype == kF32) by_vec<kF32>(a, vec, back, codes, n, s);
    else if (dtype == kBF16) by_vec<kBF16>(a, vec, back, codes, n, s);
    else by_vec<kF16>(a, vec, back, codes, n, s);
    count_launches(1);
    return cudaGetLastError();
}

template <int DT>
void run_check8(const Check8& a, bool load, bool vec, unsigned n, cudaStream_t s) {
    if (load) {
        if (vec) load_kernel<DT, true><<<n, 256, 0, s>>>(a);
        else load_kernel<DT, false><<<n, 256, 0, s>>>(a);
    } else {
        if (vec) store_kernel<DT, true><<<n, 256, 0, s>>>(a);
        else store_kernel<DT, false><<<n, 256, 0, s>>>(a);
    }
}

cudaError_t check8(const Check8& a, int dtype, bool load, cudaStream_t s, int sms) {
    if (a.rows == 0) return cudaSuccess;
    const bool vec = a.cols % kEl == 0 && a.ld % kEl == 0 && on16(a.x) && on16(a.y) && on16(a.q);
    const unsigned n = blocks(a.rows, a.cols, sms);
    if (dtype == kF32) run_check8<kF32>(a, load, vec, n, s);
    else if (dtype == kBF16) run_check8<kBF16>(a, load, vec, n, s);
    else run_check8<kF16>(a, load, vec, n, s);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t gated_forward(const Gated& a, int dtype, cudaStream_t s, int sms) {
    return run(a, dtype, false, false, s, sms);
}
cudaError_t gated_backward(const Gated& a, int dtype, bool codes, cudaStream_t s, int sms) {
    return run(a, dtype, true, codes, s, sms);
}
cudaError_t check8_store(const Check8& a, int dtype, cudaStream_t s, int sms) {
    return check8(a, dtype, false, s, sms);
}
cudaError_t check8_load(const Check8& a, int dtype, cudaStream_t s, int sms) {
    return check8(a, dtype, true, s, sms);
}

}  // namespace iabn
