// iabn_block_fwd.cu -- the block norm's forward: a block's output u through
// its post-norm, gate and residual add, then the next block's pre-norm, in
// one read of u and h and one write of h' and n (and the 8-bit checkpoints).
//
//   uhat = post(u);  h' = alpha h + gate (gamma_post uhat + beta_post);
//   xhat = pre(h');  n = gamma_pre xhat + beta_pre.
//
// A row is held in registers between its two reductions (one for each norm),
// eight columns a lane and segment; the rows to come are on their way into
// shared memory meanwhile.  What a lane does by itself is what bounds it before
// HBM does, so values are worked on two at a time and a division serves four
// checkpoint groups.
// Floor: 4 s bytes an element (s the storage size), 2 more with checkpoints.
// Measured (GPU time, B200): 16384 x 4096 bf16, RMS norms, e4m3 checkpoints
// 121 us (5.6 TB/s, floor 105 at the 6.43 TB/s of a copy), nothing kept 93 us
// (floor 83.5); layer norms 149 us, with shifts 163 us; 8192 x 8192 130 us;
// 16384 x 5120 199 us (floor 131: five warps an SM); 8192 x 4096 fp32, nothing
// kept, 129 us (floor 83.5); 3001 x 1021 fp16 layer norms 16 us (floor 3.8); 8 x
// 4096 without checkpoints 3.6 us, the launch's own time and two reductions.
#include "iabn_rows.cuh"

namespace iabn {

void count_launches(int n);

namespace {

// Statistics of one row held as V segments; v becomes the normalised row.
// FULL: the norm may be LAYER.  Its variance is the mean square about a mean
// that is already known, so it does not cancel for rows far from zero: about
// the warp's own mean first, and between the warps' means once they have been
// exchanged with those sums (one barrier for both).
template <bool VEC, bool FULL, int V, class RW>
__device__ __forceinline__ void norm_row(Lane8 (&v)[V], int kind, int c0, int cols, float eps, RW& rw,
                                         float& mean, float& rstd) {
    const float inv_n = 1.f / (float)cols;
    if (FULL && kind == kNormLayer) {
        const int left = cols - c0;   // the warp's columns, if below V kSeg
        float2 s = both(0.f), q = both(0.f);
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) s = add2(s, v[k][j]);
        const float own = left > 0 ? rw.warp_total(s) / (float)min(left, V * kSeg) : 0.f;
        auto mask = [&]() {   // past the row's end v stays zero
            if (left < V * kSeg)
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (int j = 0; j < kEl; ++j)
                        if (k * kSeg + seg_col<VEC>(rw.lane, j) >= left) el(v[k], j) = 0.f;
        };
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) v[k][j] = add2(v[k][j], both(-own));
        mask();
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) q = fma2(v[k][j], v[k][j], q);
        float square = rw.warp_total(q);
        mean = own;
        rw.template merge<V * kSeg>(mean, square, cols, inv_n);
        rstd = rsqrtf(fmaf(square, inv_n, eps));
        const float shift = (own - mean) * rstd;
#pragma unroll
        for (int k = 0; k < V; ++k)
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) v[k][j] = fma2(v[k][j], both(rstd), both(shift));
        mask();
        return;
    }
    mean = 0.f;
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

// What goes by column and stays the same from row to row.
enum : int { kScalePost = 0, kScalePre = 1, kShiftPost = 2, kShiftPre = 3 };

// Those of segment k, from the parameters: gate*gamma_post, gamma_pre,
// gate*beta_post, beta_pre.
template <bool VEC, int V>
struct Params {
    const BlockFwd& p;
    const float* gate;
    int c0, lane;
    __device__ __forceinline__ void get(int which, int k, Lane8& f) const {
        const int c = c0 + k * kSeg, left = p.cols - c;
        const float* from = which == kScalePost   ? p.gamma_post
                            : which == kScalePre  ? p.gamma_pre
                            : which == kShiftPost ? p.beta_post
                                                  : p.beta_pre;
        load_param<VEC>(from, c, lane, left, which < kShiftPost ? 1.f : 0.f, f);
        if ((which == kScalePost || which == kShiftPost) && gate) {
            Lane8 g;
            load_param<VEC>(gate, c, lane, left, 1.f, g);
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) f[j] = mul2(f[j], g[j]);
        }
    }
};

// The same kept in the thread's own part of shared memory, 16 bytes at a time.
// (In registers they would cost a third of the warps; read for every row, they
// miss the L1 that is left and double the traffic to L2: 16384 x 4096 layer
// norms with shifts 188 us.)  FULL: with the shifts.
template <bool VEC, int V, bool FULL>
struct Coef {
    static constexpr int kQuads = (FULL ? 4 : 2) * V * 2;   // a thread's
    float4* mine;   // [which][segment][half] x blockDim
    __device__ __forceinline__ void get(int which, int k, Lane8& f) const {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = mine[((which * V + k) * 2 + i) * blockDim.x];
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    }
    __device__ __forceinline__ void set(int which, const Params<VEC, V>& from) {
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
// c: what goes by column.  FULL: there may be LAYER norms and shifts.
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
            c.get(kScalePost, k, ga);
            if (FULL && p.beta_post) {
                Lane8 be;
                c.get(kShiftPost, k, be);
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) x[k][j] = fma2(x[k][j], ga[j], be[j]);
            } else {
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) x[k][j] = mul2(x[k][j], ga[j]);
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
        c.get(kScalePre, k, ga);
        if (FULL && p.beta_pre) {
            Lane8 be;
            c.get(kShiftPre, k, be);
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) h[k][j] = fma2(ga[j], h[k][j], be[j]);
        } else {
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) h[k][j] = mul2(ga[j], h[k][j]);
        }
        store8<DT, VEC>(static_cast<T*>(p.n) + at + col, rw.lane, left, h[k]);
    }
}

// Tensors off 16-byte boundaries: each row is loaded as its turn comes.
constexpr int kAnyV = 2;   // segments a warp

template <int DT, int V, int FMT, bool CLUSTER>
__global__ void __launch_bounds__(256) block_fwd_any(const BlockFwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    __shared__ __align__(16) float red[kRedFloats];
    RowWarps<CLUSTER> rw(row_warps, red);
    const T* U = static_cast<const T*>(p.u);
    const T* H = static_cast<const T*>(p.h);
    const int c0 = rw.w * V * kSeg;
    const int64_t step = (int64_t)(gridDim.x / (CLUSTER ? cluster_size() : 1)) * rw.rows;
    for (int64_t row = (int64_t)rw.block * rw.rows + rw.y; row < p.rows; row += step) {
        const int64_t at = row * p.cols;
        Lane8 x[V], h[V];
        Raw<DT, false> ru[V], rh[V];
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
        const Params<false, V> c{p, gate_of(p, row), c0, rw.lane};
        block_row<DT, false, true, V, FMT>(p, row, U != nullptr, c0, c, x, h, rw);
    }
    rw.end();
}

// A thread (not VEC: a warp) copies its share of the rows to come into a ring
// of its own, kStages - 1 rows ahead.
constexpr int kStages = 2;
constexpr int kFwdWarps = 8;      // of a row in one block
constexpr int kFwdThreads = 256;  // a block's least threads (several rows, if need be)

// Blocks of 256 threads an SM.
template <int V, bool FULL>
constexpr int kFwdBlocks = V == 4 ? 1 : FULL ? 2 : 3;

// Bytes of a warp's ring.
template <int DT, bool VEC, int V>
constexpr int kFwdRing = kStages * 2 * V * (VEC ? Raw<DT, true>::kQuads * 512
                                                : kSegBytes<(int)sizeof(typename Storage<DT>::T)>);

template <int DT, bool VEC, int V, bool FULL>
size_t shared_bytes(int threads) {
    return (size_t)Coef<VEC, V, FULL>::kQuads * 16 * threads + (size_t)kFwdRing<DT, VEC, V> * (threads / 32);
}

template <int DT, bool VEC, int V, int FMT, bool FULL, bool CLUSTER>
__global__ void __launch_bounds__(256, kFwdBlocks<V, FULL>) block_fwd(const BlockFwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    constexpr int Q = Raw<DT, true>::kQuads, ES = sizeof(T);
    extern __shared__ uint4 shared[];
    __shared__ __align__(16) float red[kRedFloats];
    RowWarps<CLUSTER> rw(row_warps, red);
    Coef<VEC, V, FULL> c{reinterpret_cast<float4*>(shared) + threadIdx.x};
    uint4* rings = shared + Coef<VEC, V, FULL>::kQuads * blockDim.x;
    const bool has_u = p.u != nullptr;
    const int c0 = rw.w * V * kSeg;
    // a block takes consecutive rows, so that gate rows change seldom
    const int64_t blocks = gridDim.x / (CLUSTER ? cluster_size() : 1);
    const int64_t end = (rw.block + 1) * p.rows / blocks;
    int64_t row = rw.block * p.rows / blocks + rw.y;
    auto slot = [&](int stage, int tensor, int k, int i) {   // VEC: the thread's
        return rings + (((stage * 2 + tensor) * V + k) * Q + i) * blockDim.x + threadIdx.x;
    };
    auto segment = [&](int stage, int tensor, int k) {       // else the warp's
        return reinterpret_cast<char*>(rings) + (size_t)(threadIdx.x >> 5) * kFwdRing<DT, VEC, V> +
               ((stage * 2 + tensor) * V + k) * kSegBytes<ES>;
    };
    auto fetch = [&](int64_t r, int stage) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (VEC) {
                const int col = c0 + k * kSeg + rw.lane * kEl;
                const bool on = r < end && col < p.cols;
                const int64_t at = r * p.cols + col;
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    copy_async<16>(slot(stage, 0, k, i), static_cast<const T*>(p.u) + at + i * 4, on && has_u);
                    copy_async<16>(slot(stage, 1, k, i), static_cast<const T*>(p.h) + at + i * 4, on);
                }
            } else {
                const int left = r < end ? p.cols - c0 - k * kSeg : 0;
                const int64_t at = r * p.cols + c0 + k * kSeg, total = p.rows * p.cols;
                copy_segment<ES>(segment(stage, 0, k), p.u, at, has_u ? left : 0, total, rw.lane);
                copy_segment<ES>(segment(stage, 1, k), p.h, at, left, total, rw.lane);
            }
        }
        copies_end();
    };
    // (what no copy writes, past the row's end and u where there is none, reads as zero)
    if (VEC)
        for (int i = 0; i < kStages * 2 * V * Q; ++i) rings[i * blockDim.x + threadIdx.x] = make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) fetch(row + i * rw.rows, i);
    c.set(kScalePre, Params<VEC, V>{p, nullptr, c0, rw.lane});
    if (FULL && p.beta_pre) c.set(kShiftPre, Params<VEC, V>{p, nullptr, c0, rw.lane});
    int64_t gate_end = -1;   // row at which another gate row begins
    int stage = 0;
    for (; row < end; row += rw.rows) {
        fetch(row + (kStages - 1) * rw.rows, stage == 0 ? kStages - 1 : stage - 1);
        if (row >= gate_end && has_u) {
            const Params<VEC, V> from{p, gate_of(p, row), c0, rw.lane};
            c.set(kScalePost, from);
            if (FULL && p.beta_post) c.set(kShiftPost, from);
            gate_end = p.gate && p.rows_per_gate > 0 ? (row / p.rows_per_gate + 1) * p.rows_per_gate : end;
        }
        copies_wait<kStages - 1>();
        Lane8 x[V], h[V];
        if (!VEC) __syncwarp();
#pragma unroll
        for (int k = 0; k < V; ++k) {
            if constexpr (VEC) {
                Raw<DT, true> ru, rh;
#pragma unroll
                for (int i = 0; i < Q; ++i) {
                    ru.v[i] = *slot(stage, 0, k, i);
                    rh.v[i] = *slot(stage, 1, k, i);
                }
                ru.get(x[k]);
                rh.get(h[k]);
            } else {
                const int left = p.cols - c0 - k * kSeg;
                const int64_t at = row * p.cols + c0 + k * kSeg;
                read_segment<DT>(segment(stage, 0, k), at, has_u ? left : 0, rw.lane, x[k]);
                read_segment<DT>(segment(stage, 1, k), at, left, rw.lane, h[k]);
            }
        }
        if (!VEC) __syncwarp();   // read by all lanes before the next copies into it
        block_row<DT, VEC, FULL, V, FMT>(p, row, has_u, c0, c, x, h, rw);
        stage = stage == kStages - 1 ? 0 : stage + 1;
    }
    copies_wait<0>();
    rw.end();
}

template <int DT, int FMT, bool CLUSTER>
cudaError_t launch_any(const BlockFwd& a, const RowShape& s, cudaStream_t stream, int sms) {
    const int64_t need = (a.rows + s.rows - 1) / s.rows, most = (int64_t)sms * 32 / s.cluster;
    return launch_rows<block_fwd_any<DT, kAnyV, FMT, CLUSTER>>(s, need < most ? need : most, 0, stream, a);
}

template <int DT, bool VEC, int V, int FMT, bool FULL, bool CLUSTER>
cudaError_t launch(const BlockFwd& a, const RowShape& s, cudaStream_t stream, int sms) {
    const size_t smem = shared_bytes<DT, VEC, V, FULL>(s.threads());
    const int blocks = blocks_an_sm(kFwdBlocks<V, FULL>, s.threads(), smem);
    const int64_t need = (a.rows + s.rows - 1) / s.rows, most = (int64_t)sms * blocks / s.cluster;
    return launch_rows<block_fwd<DT, VEC, V, FMT, FULL, CLUSTER>>(s, need < most ? need : most, smem, stream, a);
}

// SHARED: the width may take a cluster.
template <int DT, bool VEC, int V, int FMT, bool FULL, bool SHARED>
cudaError_t by_shape(const BlockFwd& a, cudaStream_t stream, int sms) {
    const RowShape s = RowShape::of<V>(a.cols, kFwdThreads, kFwdWarps);
    if constexpr (SHARED)
        if (s.cluster > 1) return launch<DT, VEC, V, FMT, FULL, true>(a, s, stream, sms);
    return launch<DT, VEC, V, FMT, FULL, false>(a, s, stream, sms);
}

// vec: 16-byte accesses.
// Segments a warp, by measurement: two up to 4096 columns (16384 x 4096 bf16,
// e4m3, compared on one box: 119 us, with four 125), four above, which keep a
// row of up to 8192 in one block (8192 x 8192: 129 us, 165 with two and a cluster
// of two blocks).  In fp32 four segments and the shifts exceed a block's shared
// memory: two.  So have odd widths, which therefore take clusters above 4096.
template <int DT, int FMT, bool FULL>
cudaError_t by_width(const BlockFwd& a, bool vec, cudaStream_t stream, int sms) {
    constexpr int kWide = DT == kF32 && FULL ? 2 : 4;
    if (vec && a.cols <= 4096) return by_shape<DT, true, 2, FMT, FULL, false>(a, stream, sms);
    if (vec) return by_shape<DT, true, kWide, FMT, FULL, true>(a, stream, sms);
    return by_shape<DT, false, 2, FMT, FULL, true>(a, stream, sms);
}

// ring: tensors on 16-byte boundaries.
template <int DT, int FMT>
cudaError_t by_norms(const BlockFwd& a, bool vec, bool ring, cudaStream_t stream, int sms) {
    count_launches(1);
    if (!ring) {
        const RowShape s = RowShape::of<kAnyV>(a.cols, 256, kFwdWarps);
        return s.cluster > 1 ? launch_any<DT, FMT, true>(a, s, stream, sms)
                             : launch_any<DT, FMT, false>(a, s, stream, sms);
    }
    const bool full = a.post == kNormLayer || a.pre == kNormLayer || a.beta_post || a.beta_pre;
    return full ? by_width<DT, FMT, true>(a, vec, stream, sms) : by_width<DT, FMT, false>(a, vec, stream, sms);
}

template <int DT>
cudaError_t by_format(const BlockFwd& a, bool vec, bool ring, cudaStream_t s, int sms) {
    if (!a.q_post && !a.q_pre) return by_norms<DT, kNoCodes>(a, vec, ring, s, sms);
    return a.format == kE4M3 ? by_norms<DT, kE4M3>(a, vec, ring, s, sms)
                             : by_norms<DT, kInt8>(a, vec, ring, s, sms);
}

}  // namespace

cudaError_t block_forward(const BlockFwd& a, int dtype, cudaStream_t s, int sms) {
    if (a.rows == 0) return cudaSuccess;
    const bool ring = on16(a.u) && on16(a.h);
    const bool vec = a.cols % kEl == 0 && ring && on16(a.h_out) && on16(a.n) && on16(a.q_post) && on16(a.q_pre);
    switch (dtype) {
        case kF32: return by_format<kF32>(a, vec, ring, s, sms);
        case kBF16: return by_format<kBF16>(a, vec, ring, s, sms);
        default: return by_format<kF16>(a, vec, ring, s, sms);
    }
}

}  // namespace iabn
