// iabn_block_fwd.cu -- the block norm's forward: a block's output u through
// its post-norm, gate and residual add, then the next block's pre-norm, in
// one read of u and h and one write of h' and n (and the 8-bit checkpoints).
//
//   uhat = post(u);  h' = alpha h + gate (gamma_post uhat + beta_post);
//   xhat = pre(h');  n = gamma_pre xhat + beta_pre.
//
// A row is held in registers between its two reductions, eight columns a lane
// and segment; LAYER's variance is the mean square about the mean already
// known (two reductions), so it does not cancel for rows far from zero.
// Bound: HBM bandwidth, 4 s bytes an element (s the storage size), 2 more
// with checkpoints.
#include "iabn_rows.cuh"

namespace iabn {

void count_launches(int n);

namespace {

// Statistics of one row held as V segments; v becomes the normalised row.
template <bool VEC, int V>
__device__ __forceinline__ void norm_row(float (&v)[V][kEl], int kind, int cols, float eps,
                                         RowWarps& rw, float& mean, float& rstd) {
    const float inv_n = 1.f / (float)cols;
    mean = 0.f;
    if (kind == kNormLayer) {
        float s = 0.f;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < kEl; ++j) s += v[k][j];
        mean = rw.sum(s) * inv_n;
    }
    float q = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int left = cols - (k * rw.n + rw.w) * kSeg;
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
            if (kind == kNormLayer) v[k][j] = seg_col<VEC>(rw.lane, j) < left ? v[k][j] - mean : 0.f;
            q = fmaf(v[k][j], v[k][j], q);
        }
    }
    rstd = __frcp_rn(__fsqrt_rn(fmaf(rw.sum(q), inv_n, eps)));
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < kEl; ++j) v[k][j] *= rstd;
}

template <int DT, bool VEC, int V, int MAXT>
__global__ void __launch_bounds__(MAXT) block_fwd(const BlockFwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    __shared__ float2 red[64];
    const int warp = threadIdx.x >> 5;
    const int y = warp / row_warps;
    RowWarps rw;
    rw.n = row_warps;
    rw.w = warp - y * row_warps;
    rw.lane = threadIdx.x & 31;
    rw.bar = 1 + y;
    rw.red = red + y * 2 * row_warps;
    rw.half = 0;
    const int lanes_y = (blockDim.x >> 5) / row_warps;
    const T* U = static_cast<const T*>(p.u);
    const T* H = static_cast<const T*>(p.h);
    for (int64_t row = (int64_t)blockIdx.x * lanes_y + y; row < p.rows;
         row += (int64_t)gridDim.x * lanes_y) {
        const int64_t at = row * p.cols;
        float x[V][kEl], h[V][kEl];
        {
            Raw<DT, VEC> ru[V], rh[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c0 = (k * rw.n + rw.w) * kSeg, left = p.cols - c0;
                if (U) ru[k].load(U + at + c0, rw.lane, left);
                rh[k].load(H + at + c0, rw.lane, left);
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                if (U) ru[k].get(x[k]);
                rh[k].get(h[k]);
            }
        }
        float mean, rstd;
        if (U) {
            if (p.post != kNormNone) {
                norm_row<VEC, V>(x, p.post, p.cols, p.eps_post, rw, mean, rstd);
                if (rw.w == 0 && rw.lane == 0) {
                    if (p.mean_post) p.mean_post[row] = mean;
                    if (p.rstd_post) p.rstd_post[row] = rstd;
                }
            }
            const float* gate = p.gate;
            if (gate && p.rows_per_gate > 0) gate += row / p.rows_per_gate * p.cols;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c0 = (k * rw.n + rw.w) * kSeg, left = p.cols - c0;
                if (p.q_post && left > 0) {
                    uint32_t m[2];
                    group_amax<VEC>(x[k], m);
                    quantise8<VEC>(p.format, x[k], m, p.q_post + at + c0,
                                   p.scale_post + row * p.groups + c0 / kQGroup, rw.lane, left);
                }
                float g[kEl], ga[kEl], be[kEl];
                load_param<VEC>(gate, c0, rw.lane, left, 1.f, g);
                load_param<VEC>(p.gamma_post, c0, rw.lane, left, 1.f, ga);
                load_param<VEC>(p.beta_post, c0, rw.lane, left, 0.f, be);
#pragma unroll
                for (int j = 0; j < kEl; ++j)
                    h[k][j] = fmaf(p.alpha, h[k][j], g[j] * fmaf(ga[j], x[k][j], be[j]));
                // (past the row's end h stays 0 only if beta is 0 there: it is)
                if (p.h_out) store8<DT, VEC>(static_cast<T*>(p.h_out) + at + c0, rw.lane, left, h[k]);
            }
        }
        if (p.pre != kNormNone) {
            norm_row<VEC, V>(h, p.pre, p.cols, p.eps_pre, rw, mean, rstd);
            if (rw.w == 0 && rw.lane == 0) {
                if (p.mean_pre) p.mean_pre[row] = mean;
                if (p.rstd_pre) p.rstd_pre[row] = rstd;
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c0 = (k * rw.n + rw.w) * kSeg, left = p.cols - c0;
                if (p.q_pre && left > 0) {
                    uint32_t m[2];
                    group_amax<VEC>(h[k], m);
                    quantise8<VEC>(p.format, h[k], m, p.q_pre + at + c0,
                                   p.scale_pre + row * p.groups + c0 / kQGroup, rw.lane, left);
                }
                float ga[kEl], be[kEl], o[kEl];
                load_param<VEC>(p.gamma_pre, c0, rw.lane, left, 1.f, ga);
                load_param<VEC>(p.beta_pre, c0, rw.lane, left, 0.f, be);
#pragma unroll
                for (int j = 0; j < kEl; ++j) o[j] = fmaf(ga[j], h[k][j], be[j]);
                store8<DT, VEC>(static_cast<T*>(p.n) + at + c0, rw.lane, left, o);
            }
        }
    }
}

template <int DT, bool VEC, int V, int MAXT>
cudaError_t launch(const BlockFwd& a, int row_warps, int rows_cta, cudaStream_t s, int sms) {
    const int threads = 32 * row_warps * rows_cta;
    const int64_t need = (a.rows + rows_cta - 1) / rows_cta;
    const int64_t most = (int64_t)sms * 32;
    block_fwd<DT, VEC, V, MAXT><<<(unsigned)(need < most ? need : most), threads, 0, s>>>(a, row_warps);
    count_launches(1);
    return cudaGetLastError();
}

template <int DT, bool VEC>
cudaError_t by_width(const BlockFwd& a, cudaStream_t s, int sms) {
    const int segs = (a.cols + kSeg - 1) / kSeg;
    if (segs <= 16) {
        const int n = segs;
        return launch<DT, VEC, 1, 512>(a, n, n >= 8 ? 1 : 8 / n, s, sms);
    }
    if (segs <= 32) return launch<DT, VEC, 2, 512>(a, (segs + 1) / 2, 1, s, sms);
    return launch<DT, VEC, 4, 1024>(a, (segs + 3) / 4, 1, s, sms);
}

}  // namespace

cudaError_t block_forward(const BlockFwd& a, int dtype, cudaStream_t s, int sms) {
    if (a.rows == 0) return cudaSuccess;
    const bool vec = a.cols % kEl == 0 && on16(a.u) && on16(a.h) && on16(a.h_out) && on16(a.n) &&
                     on16(a.q_post) && on16(a.q_pre);
    switch (dtype) {
        case kF32: return vec ? by_width<kF32, true>(a, s, sms) : by_width<kF32, false>(a, s, sms);
        case kBF16: return vec ? by_width<kBF16, true>(a, s, sms) : by_width<kBF16, false>(a, s, sms);
        default: return vec ? by_width<kF16, true>(a, s, sms) : by_width<kF16, false>(a, s, sms);
    }
}

}  // namespace iabn
