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
// FULL: the norm may be LAYER.
template <bool VEC, bool FULL, int V, class RW>
__device__ __forceinline__ void norm_row(Lane8 (&v)[V], int kind, int c0, int cols, float eps, RW& rw,
                                         float& mean, float& rstd) {
    const float inv_n = 1.f / (float)cols;
    mean = 0.f;
    if (FULL && kind == kNormLayer) {
        float2 s = both(0.f);
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) s = add2(s, v[k][j]);
        mean = rw.sum(s) * inv_n;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < kEl; ++j)
                el(v[k], j) = c0 + k * kSeg + seg_col<VEC>(rw.lane, j) < cols ? el(v[k], j) - mean : 0.f;
    }
    float2 q = both(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) q = fma2(v[k][j], v[k][j], q);
    rstd = rsqrtf(fmaf(rw.sum(q), inv_n, eps));
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) v[k][j] = mul2(v[k][j], both(rstd));
}

// A row's gate row.
__device__ __forceinline__ const float* gate_of(const BlockFwd& p, int64_t row) {
    if (!p.gate || p.rows_per_gate == 0) return p.gate;
    return p.gate + row / p.rows_per_gate * p.cols;
}

// gate*gamma_post (which = 0) or gamma_pre (1) of segment k, from the parameters.
template <bool VEC, int V>
struct Params {
    const BlockFwd& p;
    const float* gate;
    int c0, lane;
    __device__ __forceinline__ void get(int which, int k, Lane8& f) const {
        const int c = c0 + k * kSeg, left = p.cols - c;
        load_param<VEC>(which == 0 ? p.gamma_post : p.gamma_pre, c, lane, left, 1.f, f);
        if (which == 0 && gate) {
            Lane8 g;
            load_param<VEC>(gate, c, lane, left, 1.f, g);
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) f[j] = mul2(f[j], g[j]);
        }
    }
};

// The same kept in the thread's own part of shared memory, 16 bytes at a time,
// while it stays the same from row to row.  (Registers would hold it too, but
// these 16 V cost a third of the warps.)
template <int V>
struct Coef {
    static constexpr int kQuads = 2 * V * 2;   // a thread's
    float4* mine;   // [which][segment][half] x blockDim
    __device__ __forceinline__ void get(int which, int k, Lane8& f) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = mine[((which * V + k) * 2 + i) * blockDim.x];
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    }
    __device__ __forceinline__ void set(int which, const Params<true, V>& from) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Lane8 f;
            from.get(which, k, f);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                mine[((which * V + k) * 2 + i) * blockDim.x] =
                    make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
        }
    }
};

// One row, held as V segments: x holds u (if has_u), h the residual stream.
// c: what goes by column (the shifts are read here).  FULL: there may be LAYER
// norms and shifts.
template <int DT, bool VEC, bool FULL, int V, int FMT, class C, class RW>
__device__ __forceinline__ void block_row(const BlockFwd& p, int64_t row, bool has_u,
                                          int c0, const C& c, Lane8 (&x)[V], Lane8 (&h)[V],
                                          RW& rw) {
    using T = typename Storage<DT>::T;
    const int64_t at = row * p.cols;
    float mean, rstd;
    if (has_u) {
        if (p.post != kNormNone) {
            norm_row<VEC, FULL, V>(x, p.post, c0, p.cols, p.eps_post, rw, mean, rstd);
            if (rw.w == 0 && rw.lane == 0) {
                if (FULL && p.mean_post) p.mean_post[row] = mean;
                if (p.rstd_post) p.rstd_post[row] = rstd;
            }
        }
        if constexpr (FMT != kNoCodes)
            if (p.q_post)
                quantise_row<FMT, VEC, V>(x, p.q_post + at, p.scale_post + row * p.groups, c0,
                                          p.cols, rw.lane);
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col = c0 + k * kSeg, left = p.cols - col;
            Lane8 ga;
            c.get(0, k, ga);
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) x[k][j] = mul2(x[k][j], ga[j]);
            if (FULL && p.beta_post) {
                Lane8 g, be;
                load_param<VEC>(gate_of(p, row), col, rw.lane, left, 1.f, g);
                load_param<VEC>(p.beta_post, col, rw.lane, left, 0.f, be);
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) x[k][j] = fma2(g[j], be[j], x[k][j]);
            }
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) h[k][j] = fma2(both(p.alpha), h[k][j], x[k][j]);
            if (p.h_out)
                store8<DT, VEC>(static_cast<T*>(p.h_out) + at + col, rw.lane, left, h[k]);
        }
    }
    if (p.pre == kNormNone) return;
    norm_row<VEC, FULL, V>(h, p.pre, c0, p.cols, p.eps_pre, rw, mean, rstd);
    if (rw.w == 0 && rw.lane == 0) {
        if (FULL && p.mean_pre) p.mean_pre[row] = mean;
        if (p.rstd_pre) p.rstd_pre[row] = rstd;
    }
    if constexpr (FMT != kNoCodes)
        if (p.q_pre)
            quantise_row<FMT, VEC, V>(h, p.q_pre + at, p.scale_pre + row * p.groups, c0, p.cols,
                                      rw.lane);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int col = c0 + k * kSeg, left = p.cols - col;
        Lane8 ga;
        c.get(1, k, ga);
        if (FULL && p.beta_pre) {
            Lane8 be;
            load_param<VEC>(p.beta_pre, col, rw.lane, left, 0.f, be);
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) h[k][j] = fma2(ga[j], h[k][j], be[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) h[k][j] = mul2(ga[j], h[k][j]);
        }
        store8<DT, VEC>(static_cast<T*>(p.n) + at + col, rw.lane, left, h[k]);
    }
}

// Any width and alignment: each row is loaded as its turn comes.
template <int DT, bool VEC, int V, int FMT>
__global__ void __launch_bounds__(V == 4 ? 1024 : 512, 1) block_fwd_any(const BlockFwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    __shared__ __align__(16) float red[8 * kRowFloats];
    RowWarps<V == 4 ? 32 : 16> rw(row_warps, red);
    const int rows_cta = (blockDim.x >> 5) / row_warps;
    const T* U = static_cast<const T*>(p.u);
    const T* H = static_cast<const T*>(p.h);
    const int c0 = rw.w * V * kSeg;
    for (int64_t row = (int64_t)blockIdx.x * rows_cta + rw.bar - 1; row < p.rows;
         row += (int64_t)gridDim.x * rows_cta) {
        const int64_t at = row * p.cols;
        Lane8 x[V], h[V];
        Raw<DT, VEC> ru[V], rh[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (U) ru[k].load(U + at + c0 + k * kSeg, rw.lane, p.cols - c0 - k * kSeg);
            rh[k].load(H + at + c0 + k * kSeg, rw.lane, p.cols - c0 - k * kSeg);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if (U) ru[k].get(x[k]);
            rh[k].get(h[k]);
        }
        const Params<VEC, V> c{p, gate_of(p, row), c0, rw.lane};
        block_row<DT, VEC, true, V, FMT>(p, row, U != nullptr, c0, c, x, h, rw);
    }
}

// VEC widths up to 8192: a thread copies its share of the rows to come into a
// ring of its own, kStages - 1 rows ahead.
constexpr int kStages = 2;
constexpr int kFwdV = 2;          // segments a warp
constexpr int kFwdThreads = 256;  // a block's least threads (several rows, if need be)


template <int DT, int V>
size_t shared_bytes(int threads) {
    return ((size_t)kStages * 2 * V * Raw<DT, true>::kQuads + Coef<V>::kQuads) * 16 * threads;
}

template <int DT, int V, int FMT, bool FULL, int MAXT>
__global__ void __launch_bounds__(MAXT, MAXT == 256 ? 3 : 1) block_fwd(const BlockFwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    constexpr int Q = Raw<DT, true>::kQuads;
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float red[8 * kRowFloats];
    RowWarps<MAXT / 32> rw(row_warps, red);
    Coef<V> c{reinterpret_cast<float4*>(shared) + threadIdx.x};
    uint4* ring = shared + Coef<V>::kQuads * blockDim.x + threadIdx.x;   // the thread's own
    const int rows_cta = (blockDim.x >> 5) / row_warps;
    const bool has_u = p.u != nullptr;
    const int c0 = rw.w * V * kSeg;
    // a block takes consecutive rows, so that gate rows change seldom
    const int64_t end = (blockIdx.x + 1) * p.rows / gridDim.x;
    int64_t row = blockIdx.x * p.rows / gridDim.x + rw.bar - 1;
    auto slot = [&](int stage, int tensor, int k, int i) {
        return ring + (((stage * 2 + tensor) * V + k) * Q + i) * blockDim.x;
    };
    auto fetch = [&](int64_t r, int stage) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int col = c0 + k * kSeg + rw.lane * kEl;
            const bool on = r < end && col < p.cols;
            const int64_t at = r * p.cols + col;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                copy_async<16>(slot(stage, 0, k, i), static_cast<const T*>(p.u) + at + i * 4, on && has_u);
                copy_async<16>(slot(stage, 1, k, i), static_cast<const T*>(p.h) + at + i * 4, on);
            }
        }
        copies_end();
    };
    // (what no copy writes, past the row's end and u where there is none, reads as zero)
    for (int i = 0; i < kStages * 2 * V * Q; ++i) ring[i * blockDim.x] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(row + i * rows_cta, i);
    c.set(1, Params<true, V>{p, nullptr, c0, rw.lane});
    int64_t gate_end = -1;   // row at which another gate row begins
    int stage = 0;
    for (; row < end; row += rows_cta) {
        fetch(row + (kStages - 1) * rows_cta, stage == 0 ? kStages - 1 : stage - 1);
        if (row >= gate_end && has_u) {
            c.set(0, Params<true, V>{p, gate_of(p, row), c0, rw.lane});
            gate_end = p.gate && p.rows_per_gate > 0 ? (row / p.rows_per_gate + 1) * p.rows_per_gate : end;
        }
        copies_wait<kStages - 1>();
        Lane8 x[V], h[V];
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Raw<DT, true> ru, rh;
#pragma unroll
            for (int i = 0; i < Q; ++i) {
                ru.v[i] = *slot(stage, 0, k, i);
                rh.v[i] = *slot(stage, 1, k, i);
            }
            ru.get(x[k]);
            rh.get(h[k]);
        }
        block_row<DT, true, FULL, V, FMT>(p, row, has_u, c0, c, x, h, rw);
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
}

template <int DT, bool VEC, int V, int FMT>
cudaError_t launch_any(const BlockFwd& a, int row_warps, int rows_cta, cudaStream_t s, int sms) {
    const int64_t need = (a.rows + rows_cta - 1) / rows_cta, most = (int64_t)sms * 32;
    block_fwd_any<DT, VEC, V, FMT>
        <<<(unsigned)(need < most ? need : most), 32 * row_warps * rows_cta, 0, s>>>(a, row_warps);
    count_launches(1);
    return cudaGetLastError();
}

template <int DT, int FMT, bool FULL>
cudaError_t launch(const BlockFwd& a, int segs, cudaStream_t s, int sms) {
    const int row_warps = (segs + kFwdV - 1) / kFwdV;
    const int rows_cta = row_warps * 32 >= kFwdThreads ? 1 : kFwdThreads / 32 / row_warps;
    const int threads = 32 * row_warps * rows_cta;
    const size_t smem = shared_bytes<DT, kFwdV>(threads);
    auto kernel = threads <= 256 ? block_fwd<DT, kFwdV, FMT, FULL, 256> : block_fwd<DT, kFwdV, FMT, FULL, 512>;
    cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    int blocks = 0;
    if (e == cudaSuccess) e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, smem);
    if (e != cudaSuccess) return e;
    const int64_t need = (a.rows + rows_cta - 1) / rows_cta, most = (int64_t)sms * blocks;
    kernel<<<(unsigned)(need < most ? need : most), threads, smem, s>>>(a, row_warps);
    count_launches(1);
    return cudaGetLastError();
}

template <int DT, int FMT>
cudaError_t by_width(const BlockFwd& a, bool vec, cudaStream_t s, int sms) {
    const int segs = (a.cols + kSeg - 1) / kSeg;
    if (vec && segs <= 32) {
        const bool full = a.post == kNormLayer || a.pre == kNormLayer || a.beta_post || a.beta_pre;
        return full ? launch<DT, FMT, true>(a, segs, s, sms) : launch<DT, FMT, false>(a, segs, s, sms);
    }
    if (vec) return launch_any<DT, true, 4, FMT>(a, (segs + 3) / 4, 1, s, sms);
    if (segs <= 16) return launch_any<DT, false, 1, FMT>(a, segs, segs >= 8 ? 1 : 8 / segs, s, sms);
    if (segs <= 32) return launch_any<DT, false, 2, FMT>(a, (segs + 1) / 2, 1, s, sms);
    return launch_any<DT, false, 4, FMT>(a, (segs + 3) / 4, 1, s, sms);
}

template <int DT>
cudaError_t by_format(const BlockFwd& a, bool vec, cudaStream_t s, int sms) {
    if (!a.q_post && !a.q_pre) return by_width<DT, kNoCodes>(a, vec, s, sms);
    return a.format == kE4M3 ? by_width<DT, kE4M3>(a, vec, s, sms)
                             : by_width<DT, kInt8>(a, vec, s, sms);
}

}  // namespace

cudaError_t block_forward(const BlockFwd& a, int dtype, cudaStream_t s, int sms) {
    if (a.rows == 0) return cudaSuccess;
    const bool vec = a.cols % kEl == 0 && on16(a.u) && on16(a.h) && on16(a.h_out) && on16(a.n) &&
                     on16(a.q_post) && on16(a.q_pre);
    switch (dtype) {
        case kF32: return by_format<kF32>(a, vec, s, sms);
        case kBF16: return by_format<kBF16>(a, vec, s, sms);
        default: return by_format<kF16>(a, vec, s, sms);
    }
}

}  // namespace iabn
