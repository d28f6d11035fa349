// iabn_block_bwd.cu -- the block norm's backward, from the kept u and h' or
// from the 8-bit codes of uhat and xhat.
//
// For a row, with g = dn gamma_pre:
//   t  = dh' + rho_h (g - [mean g] - xhat mean(g xhat)),   dh = alpha t,
//   e  = t gate gamma_post,
//   du = rho_u (e - [mean e] - uhat mean(e uhat)).
// For a column, over rows: C = sum dn xhat, E = sum dn (dgamma_pre, dbeta_pre)
// and, for every gate row, A = sum t uhat, B = sum t, from which
//   dgate = gamma_post A + beta_post B,
//   dgamma_post = sum gate A,  dbeta_post = sum gate B.
//
// Two launches.  The row pass: worker w (a CTA) takes a contiguous range of
// rows, holds A, B, C, E of its columns in registers, writes A and B where a
// gate row's tokens end and all at its end.  The column pass adds the workers'
// partial sums in their order, so the sums are the same bits every time.
// Bound: HBM bandwidth, 4 s + 2 bytes an element from codes, 6 s kept.
#include "iabn_rows.cuh"

namespace iabn {

void count_launches(int n);

namespace {

constexpr int kBwdCtas = 296;   // workers of the row pass at most

struct Span {
    int64_t lo, hi;
};
__host__ __device__ inline Span worker_rows(int64_t w, int64_t rows, int64_t workers) {
    return {w * rows / workers, (w + 1) * rows / workers};
}

template <int DT, bool VEC, int V, bool CODES, int MAXT>
__global__ void __launch_bounds__(MAXT) block_bwd_rows(const BlockBwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    extern __shared__ float4 shared[];   // sums of a row, then (several rows a CTA) of columns
    const int warp = threadIdx.x >> 5;
    const int lanes_y = (blockDim.x >> 5) / row_warps;
    RowWarps<32> rw(row_warps, reinterpret_cast<float*>(shared));
    const int y = rw.bar - 1;
    float* columns = reinterpret_cast<float*>(shared) + lanes_y * kRowFloats;
    const float inv_n = 1.f / (float)p.cols;
    const int64_t D = p.cols;
    const int64_t slots = block_bwd_slots(p.workers, p.gates);
    Lane8 A[V], B[V], C[V], E[V];
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) A[k][j] = B[k][j] = C[k][j] = E[k][j] = both(0.f);

    // Adds the CTA's row lanes and writes a partial-sum row.
    auto flush = [&](Lane8 (&s)[V], float* out) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c0 = (k * rw.n + rw.w) * kSeg, left = p.cols - c0;
            if (lanes_y > 1) {
                __syncthreads();
                float* mine = columns + warp * kSeg;
#pragma unroll
                for (int j = 0; j < kEl; ++j) mine[rw.lane + 32 * j] = el(s[k], j);
                __syncthreads();
                if (y == 0)
                    for (int o = 1; o < lanes_y; ++o) {
                        const float* other = columns + (o * rw.n + rw.w) * kSeg;
#pragma unroll
                        for (int j = 0; j < kEl; ++j) el(s[k], j) += other[rw.lane + 32 * j];
                    }
            }
            if (y == 0) {
#pragma unroll
                for (int j = 0; j < kEl; ++j) {
                    const int c = seg_col<VEC>(rw.lane, j);
                    if (c < left) out[c0 + c] = el(s[k], j);
                }
            }
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) s[k][j] = both(0.f);
        }
    };

    // The normalised segment k of a row: from codes, or from the kept tensor.
    auto hat = [&](const void* src, const float* scales, const float* means, const float* rstds,
                   int64_t row, int k, Lane8& f) {
        const int c0 = (k * rw.n + rw.w) * kSeg, left = p.cols - c0;
        if (CODES) {
            Codes<VEC> c;
            float sc[2] = {0.f, 0.f};
            c.load(static_cast<const uint8_t*>(src) + row * D + c0, rw.lane, left);
            load_scales<VEC>(scales + row * p.groups + c0 / kQGroup, rw.lane, left, sc);
            if (p.format == kE4M3) c.template get<kE4M3>(sc, f);
            else c.template get<kInt8>(sc, f);
        } else {
            Raw<DT, VEC> r;
            r.load(static_cast<const T*>(src) + row * D + c0, rw.lane, left);
            r.get(f);
            const float mean = means ? __ldg(means + row) : 0.f;
            const float rstd = rstds ? __ldg(rstds + row) : 1.f;
#pragma unroll
            for (int j = 0; j < kEl; ++j)
                el(f, j) = seg_col<VEC>(rw.lane, j) < left ? (el(f, j) - mean) * rstd : 0.f;
        }
    };

    const Span mine = worker_rows(blockIdx.x, p.rows, p.workers);
    for (int64_t lo = mine.lo; lo < mine.hi;) {
        const int64_t gr = p.rows_per_gate > 0 ? lo / p.rows_per_gate : 0;
        const int64_t end = p.rows_per_gate > 0 ? (gr + 1) * p.rows_per_gate : mine.hi;
        const int64_t hi = end < mine.hi ? end : mine.hi;
        const float* gate = p.gate ? p.gate + gr * D : nullptr;
        for (int64_t row = lo + y; row < hi; row += lanes_y) {
            Lane8 t[V];
            if (p.dh_out) {
                Raw<DT, VEC> r[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int c0 = (k * rw.n + rw.w) * kSeg;
                    r[k].load(static_cast<const T*>(p.dh_out) + row * D + c0, rw.lane, p.cols - c0);
                }
#pragma unroll
                for (int k = 0; k < V; ++k) r[k].get(t[k]);
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (int j = 0; j < kEl / 2; ++j) t[k][j] = both(0.f);
            }
            if (p.pre != kNormNone) {
                Lane8 g[V], x[V];
                float2 s = both(0.f), sx = both(0.f);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int c0 = (k * rw.n + rw.w) * kSeg, left = p.cols - c0;
                    Raw<DT, VEC> r;
                    r.load(static_cast<const T*>(p.dn) + row * D + c0, rw.lane, left);
                    hat(p.sh, p.scale_pre, p.mean_pre, p.rstd_pre, row, k, x[k]);
                    r.get(g[k]);
                    Lane8 ga;
                    load_param<VEC>(p.gamma_pre, c0, rw.lane, left, 1.f, ga);
#pragma unroll
                    for (int j = 0; j < kEl / 2; ++j) {
                        C[k][j] = fma2(g[k][j], x[k][j], C[k][j]);
                        E[k][j] = add2(E[k][j], g[k][j]);
                        g[k][j] = mul2(g[k][j], ga[j]);
                        s = add2(s, g[k][j]);
                        sx = fma2(g[k][j], x[k][j], sx);
                    }
                }
                const float2 m = rw.sum(s, sx);
                const float level = p.pre == kNormLayer ? m.x * inv_n : 0.f, slope = m.y * inv_n;
                const float rstd = __ldg(p.rstd_pre + row);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const int left = p.cols - (k * rw.n + rw.w) * kSeg;
#pragma unroll
                    for (int j = 0; j < kEl; ++j) {
                        const float d = fmaf(-slope, el(x[k], j), el(g[k], j) - level);
                        if (seg_col<VEC>(rw.lane, j) < left) el(t[k], j) = fmaf(rstd, d, el(t[k], j));
                    }
                }
            }
            Lane8 x[V];
            float2 s = both(0.f), sx = both(0.f);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c0 = (k * rw.n + rw.w) * kSeg, left = p.cols - c0;
                if (p.su) {
                    hat(p.su, p.scale_post, p.mean_post, p.rstd_post, row, k, x[k]);
                } else {
#pragma unroll
                    for (int j = 0; j < kEl / 2; ++j) x[k][j] = both(0.f);
                }
                // (all inputs of this column have been read: dh may be any of them)
                Lane8 o;
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) o[j] = mul2(both(p.alpha), t[k][j]);
                store8<DT, VEC>(static_cast<T*>(p.dh) + row * D + c0, rw.lane, left, o);
                Lane8 ga, gt;
                load_param<VEC>(p.gamma_post, c0, rw.lane, left, 1.f, ga);
                load_param<VEC>(gate, c0, rw.lane, left, 1.f, gt);
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) {
                    A[k][j] = fma2(t[k][j], x[k][j], A[k][j]);
                    B[k][j] = add2(B[k][j], t[k][j]);
                    t[k][j] = mul2(t[k][j], mul2(gt[j], ga[j]));
                    s = add2(s, t[k][j]);
                    sx = fma2(t[k][j], x[k][j], sx);
                }
            }
            if (!p.du) continue;
            if (p.post != kNormNone) {
                const float2 m = rw.sum(s, sx);
                const float level = p.post == kNormLayer ? m.x * inv_n : 0.f, slope = m.y * inv_n;
                const float rstd = __ldg(p.rstd_post + row);
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (int j = 0; j < kEl; ++j)
                        el(t[k], j) = rstd * fmaf(-slope, el(x[k], j), el(t[k], j) - level);
            }
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int c0 = (k * rw.n + rw.w) * kSeg;
                store8<DT, VEC>(static_cast<T*>(p.du) + row * D + c0, rw.lane, p.cols - c0, t[k]);
            }
        }
        const int64_t slot = blockIdx.x + gr;
        flush(A, p.work + slot * D);
        flush(B, p.work + (slots + slot) * D);
        lo = hi;
    }
    flush(C, p.work + (2 * slots + blockIdx.x) * D);
    flush(E, p.work + (2 * slots + p.workers + blockIdx.x) * D);
}

// The column pass: a block takes 32 columns, its 32 warps share the partial
// sums of them.  blockIdx.y 0: dgamma_pre, dbeta_pre; 1: dgamma_post,
// dbeta_post; from 2: the gate rows.
constexpr int kColWarps = 32;

__device__ __forceinline__ float add_warps(float v, float (&sh)[kColWarps][33]) {
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    __syncthreads();
    sh[w][l] = v;
    __syncthreads();
    const float t = sh[l][w];   // column w of the block, partial l
    return warp_sum(t);         // valid for column w
}

__global__ void __launch_bounds__(1024) block_bwd_columns(const BlockBwd p) {
    __shared__ float sh[kColWarps][33];
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    const int64_t D = p.cols;
    const int64_t c = (int64_t)blockIdx.x * 32 + l;       // column this thread reads
    const int64_t co = (int64_t)blockIdx.x * 32 + w;      // column this warp writes
    const bool in = c < D, out = co < D && l == 0;
    const int64_t slots = block_bwd_slots(p.workers, p.gates);
    const float* A = p.work;
    const float* B = p.work + slots * D;
    const float* C = p.work + 2 * slots * D;
    const float* E = p.work + (2 * slots + p.workers) * D;
    const int64_t P = p.rows > 0 ? p.workers : 0;
    if (blockIdx.y == 0) {
        float a = 0.f, b = 0.f;
        for (int64_t i = w; i < P && in; i += kColWarps) {
            a += C[i * D + c];
            b += E[i * D + c];
        }
        a = add_warps(a, sh);
        b = add_warps(b, sh);
        if (out && p.dgamma_pre) p.dgamma_pre[co] = a;
        if (out && p.dbeta_pre) p.dbeta_pre[co] = b;
    } else if (blockIdx.y == 1) {
        float a = 0.f, b = 0.f;
        for (int64_t i = w; i < P && in; i += kColWarps) {
            const Span r = worker_rows(i, p.rows, p.workers);
            const int64_t g0 = p.rows_per_gate > 0 ? r.lo / p.rows_per_gate : 0;
            const int64_t g1 = p.rows_per_gate > 0 ? (r.hi - 1) / p.rows_per_gate : 0;
            for (int64_t g = g0; g <= g1; ++g) {
                const float gt = p.gate ? p.gate[g * D + c] : 1.f;
                a = fmaf(gt, A[(i + g) * D + c], a);
                b = fmaf(gt, B[(i + g) * D + c], b);
            }
        }
        a = add_warps(a, sh);
        b = add_warps(b, sh);
        if (out && p.dgamma_post) p.dgamma_post[co] = a;
        if (out && p.dbeta_post) p.dbeta_post[co] = b;
    } else {
        for (int64_t g = blockIdx.y - 2; g < p.gates; g += gridDim.y - 2) {
            float a = 0.f, b = 0.f;
            if (P > 0) {
                const int64_t lo = p.rows_per_gate > 0 ? g * p.rows_per_gate : 0;
                int64_t hi = p.rows_per_gate > 0 ? lo + p.rows_per_gate : p.rows;
                if (hi > p.rows) hi = p.rows;
                // workers whose ranges meet [lo, hi)
                int64_t w0 = lo * P / p.rows, w1 = (hi - 1) * P / p.rows;
                while (w0 > 0 && worker_rows(w0 - 1, p.rows, P).hi > lo) --w0;
                while (worker_rows(w0, p.rows, P).hi <= lo) ++w0;
                while (worker_rows(w1, p.rows, P).hi < hi) ++w1;
                while (worker_rows(w1, p.rows, P).lo >= hi) --w1;
                for (int64_t i = w0 + w; i <= w1 && in; i += kColWarps) {
                    a += A[(i + g) * D + c];
                    b += B[(i + g) * D + c];
                }
            }
            a = add_warps(a, sh);
            b = add_warps(b, sh);
            if (out) {
                const float ga = p.gamma_post ? p.gamma_post[co] : 1.f;
                const float be = p.beta_post ? p.beta_post[co] : 0.f;
                p.dgate[g * D + co] = fmaf(ga, a, be * b);
            }
        }
    }
}

template <int DT, bool VEC, bool CODES, int V, int MAXT>
cudaError_t launch(const BlockBwd& a, int row_warps, int rows_cta, cudaStream_t s) {
    const int threads = 32 * row_warps * rows_cta;
    const size_t smem = (rows_cta * kRowFloats + (rows_cta > 1 ? threads / 32 * kSeg : 0)) * sizeof(float);
    block_bwd_rows<DT, VEC, V, CODES, MAXT><<<(unsigned)a.workers, threads, smem, s>>>(a, row_warps);
    count_launches(1);
    return cudaGetLastError();
}

template <int DT, bool VEC, bool CODES>
cudaError_t by_width(const BlockBwd& a, cudaStream_t s) {
    const int segs = (a.cols + kSeg - 1) / kSeg;
    if (segs <= 16)
        return launch<DT, VEC, CODES, 1, 512>(a, segs, segs >= 8 ? 1 : 8 / segs, s);
    if (segs <= 32) return launch<DT, VEC, CODES, 2, 512>(a, (segs + 1) / 2, 1, s);
    return launch<DT, VEC, CODES, 4, 1024>(a, (segs + 3) / 4, 1, s);
}

template <int DT>
cudaError_t by_kind(const BlockBwd& a, bool vec, bool codes, cudaStream_t s) {
    if (codes) return vec ? by_width<DT, true, true>(a, s) : by_width<DT, false, true>(a, s);
    return vec ? by_width<DT, true, false>(a, s) : by_width<DT, false, false>(a, s);
}

}  // namespace

int64_t block_bwd_workers(int64_t rows, int64_t) {
    return rows < 1 ? 1 : rows < kBwdCtas ? rows : kBwdCtas;
}

cudaError_t block_backward(const BlockBwd& a, int dtype, bool codes, cudaStream_t s, int) {
    if (a.rows > 0) {
        const bool vec = a.cols % kEl == 0 && on16(a.su) && on16(a.sh) && on16(a.dh_out) &&
                         on16(a.dn) && on16(a.dh) && on16(a.du);
        const cudaError_t e = dtype == kF32    ? by_kind<kF32>(a, vec, codes, s)
                              : dtype == kBF16 ? by_kind<kBF16>(a, vec, codes, s)
                                               : by_kind<kF16>(a, vec, codes, s);
        if (e != cudaSuccess) return e;
    }
    const bool pre = a.dgamma_pre || a.dbeta_pre, post = a.dgamma_post || a.dbeta_post;
    if (!pre && !post && !a.dgate) return cudaSuccess;
    const int64_t gates = a.dgate ? (a.gates < 4096 ? a.gates : 4096) : 0;
    const dim3 grid((unsigned)((a.cols + 31) / 32), (unsigned)(2 + gates));
    block_bwd_columns<<<grid, 1024, 0, s>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace iabn
