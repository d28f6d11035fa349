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
// Two launches.  The row pass: worker w (a block, or a cluster of them) takes
// consecutive rows, holds A, B, C, E of its columns in registers (B and E only
// where something asks for them or a mean), writes A and B where a gate row's
// tokens end and all at its end.  The column pass adds the workers' partial
// sums in their order, so the sums are the same bits every time.
// Floor: 4 s + 2 bytes an element from codes, 6 s kept.  The sums take the
// registers of half the warps that an SM could hold, so what bounds it is the
// latency between a row's reductions, then the instructions.
// Measured (GPU time, B200): 16384 x 4096 bf16 RMS norms from e4m3 129 us (5.2
// TB/s, floor 105), kept 139 us (floor 125); layer norms with or without shifts
// 161 us; 16384 x 5120 RMS 209 us (floor 131: five warps an SM); 8192 x 4096 fp32
// kept 218 us (floor 125); 2048 x 8192 layer norms 76 us (floor 26); 3001 x 1021
// kept fp32 33 us (floor 11.5).  The row pass by itself is 122 us of the first,
// 61 and 24 us of the last two; the rest is the column pass and its launch.
#include "iabn_rows.cuh"

namespace iabn {

void count_launches(int n);

namespace {

constexpr int kBwdWarps = 8;      // of a row in one block
constexpr int kBwdThreads = 128;  // a block's least threads (several rows, if need be)

// Worker w's rows: rows / workers of them, one more for the first rows %
// workers.  (32 bits: there are fewer than 2^31 rows.)
struct Split {
    int each, more;
    __device__ __forceinline__ Split(const BlockBwd& p)
        : each((int)p.rows / (int)p.workers), more((int)p.rows % (int)p.workers) {}
    __device__ __forceinline__ int first(int w) const { return w * each + min(w, more); }
    __device__ __forceinline__ int worker(int row) const {   // that holds the row
        const int big = more * (each + 1);
        return row < big ? row / (each + 1) : more + (row - big) / each;
    }
};

// Columns as workspace rows hold them: whole 16-byte vectors.
__host__ __device__ inline int64_t work_cols(int64_t cols) { return (cols + 3) / 4 * 4; }

// Adds the rows of a block and writes one partial-sum row; s starts again from
// zero.  The whole block calls it.
template <bool VEC, int V, class RW>
__device__ __forceinline__ void flush(Lane8 (&s)[V], float* out, int cols, const RW& rw,
                                      float* columns) {
    const int y = rw.y, rows = rw.rows;
#pragma unroll
    for (int k = 0; k < V; ++k) {
        const int c0 = (rw.w * V + k) * kSeg, left = cols - c0;
        if (rows > 1) {
            __syncthreads();
            float* mine = columns + (y * rw.n + rw.w) * kSeg;
#pragma unroll
            for (int j = 0; j < kEl; ++j) mine[rw.lane + 32 * j] = el(s[k], j);
            __syncthreads();
            if (y == 0)
                for (int o = 1; o < rows; ++o) {
                    const float* other = columns + (o * rw.n + rw.w) * kSeg;
#pragma unroll
                    for (int j = 0; j < kEl; ++j) el(s[k], j) += other[rw.lane + 32 * j];
                }
        }
        if (y == 0) {
            if (VEC) {
                if (rw.lane * kEl < left) {
                    float4* q = reinterpret_cast<float4*>(out + c0 + rw.lane * kEl);
                    q[0] = make_float4(s[k][0].x, s[k][0].y, s[k][1].x, s[k][1].y);
                    q[1] = make_float4(s[k][2].x, s[k][2].y, s[k][3].x, s[k][3].y);
                }
            } else {
#pragma unroll
                for (int j = 0; j < kEl; ++j)
                    if (rw.lane + 32 * j < left) out[c0 + rw.lane + 32 * j] = el(s[k], j);
            }
        }
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) s[k][j] = both(0.f);
    }
}

// A worker's rows in steps of the block's row count, none of which crosses
// from one gate row's tokens into the next's.
struct Steps {
    int at, hi, end, per, gate, rows;
    __device__ __forceinline__ Steps(const BlockBwd& p, int worker, int rows_cta) {
        const Split s(p);
        at = s.first(worker);
        end = s.first(worker + 1);
        per = (int)min(p.rows_per_gate, p.rows);   // (one gate row covers them all)
        rows = rows_cta;
        open();
    }
    __device__ __forceinline__ void open() {   // the gate row that `at` is in
        gate = per > 0 ? at / per : 0;
        hi = per > 0 && end - at > per - (at - gate * per) ? (gate + 1) * per : end;
    }
    __device__ __forceinline__ bool done() const { return at >= end; }
    // the block's y-th row of this step, and whether there is one
    __device__ __forceinline__ bool has(int y) const { return hi - at > y; }
    __device__ __forceinline__ int row(int y) const { return (int)((unsigned)at + y); }
    __device__ __forceinline__ bool last() const { return hi - at <= rows; }   // of this gate row
    __device__ __forceinline__ void next() {
        if (last()) {
            at = hi;
            open();
        } else {
            at += rows;
        }
    }
};

template <int V>
__device__ __forceinline__ void zero(Lane8 (&s)[V]) {
#pragma unroll
    for (int k = 0; k < V; ++k)
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) s[k][j] = both(0.f);
}

// Columns of a segment past the row's end are kept at zero where a LAYER
// norm's mean would have moved them.
template <bool VEC>
__device__ __forceinline__ void mask8(Lane8& f, int lane, int left) {
    if (left >= kSeg) return;   // (the same for the whole warp)
#pragma unroll
    for (int j = 0; j < kEl; ++j)
        if (seg_col<VEC>(lane, j) >= left) el(f, j) = 0.f;
}

// The kept tensor's values as normalised ones.
__device__ __forceinline__ void kept_hat(Lane8& f, float mean, float rstd) {
#pragma unroll
    for (int j = 0; j < kEl / 2; ++j) f[j] = mul2(add2(f[j], both(-mean)), both(rstd));
}

// A row between its loads and its stores, shared by the kernels below.
// First half: from g = dn and x = xhat, C += g x, E += g, g *= gamma_pre, and
// the row's sums (level, slope) of g and g x.
template <bool FULL, int V, class RW, class G>
__device__ __forceinline__ float2 pre_half(Lane8 (&g)[V], const Lane8 (&x)[V], Lane8 (&C)[V],
                                           Lane8 (&E)[V], RW& rw, const G& gamma) {
    float2 s = both(0.f), sx = both(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        Lane8 ga;
        gamma(k, ga);
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) {
            C[k][j] = fma2(g[k][j], x[k][j], C[k][j]);
            if (FULL) E[k][j] = add2(E[k][j], g[k][j]);
            g[k][j] = mul2(g[k][j], ga[j]);
            if (FULL) s = add2(s, g[k][j]);
            sx = fma2(g[k][j], x[k][j], sx);
        }
    }
    if (FULL) return rw.sum(s, sx);
    return make_float2(0.f, rw.sum(sx));
}

// g becomes rstd (g - level - x slope).
template <bool VEC, bool FULL, int V, class RW>
__device__ __forceinline__ void back_through(Lane8 (&g)[V], const Lane8 (&x)[V], float level,
                                             float slope, float rstd, int cols, const RW& rw) {
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) {
            const float2 d = FULL ? add2(g[k][j], both(-level)) : g[k][j];
            g[k][j] = mul2(fma2(x[k][j], both(-slope), d), both(rstd));
        }
        if (FULL) mask8<VEC>(g[k], rw.lane, cols - (rw.w * V + k) * kSeg);
    }
}

// Second half: from t and x = uhat, A += t x, B += t, t *= gate gamma_post,
// and the row's sums of t and t x.
template <bool FULL, int V, class RW, class G>
__device__ __forceinline__ float2 post_half(Lane8 (&t)[V], const Lane8 (&x)[V], Lane8 (&A)[V],
                                            Lane8 (&B)[V], RW& rw, bool sums, const G& weight) {
    float2 s = both(0.f), sx = both(0.f);
#pragma unroll
    for (int k = 0; k < V; ++k) {
        Lane8 ga;
        weight(k, ga);
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) {
            A[k][j] = fma2(t[k][j], x[k][j], A[k][j]);
            if (FULL) B[k][j] = add2(B[k][j], t[k][j]);
            t[k][j] = mul2(t[k][j], ga[j]);
            if (FULL) s = add2(s, t[k][j]);
            sx = fma2(t[k][j], x[k][j], sx);
        }
    }
    if (!sums) return make_float2(0.f, 0.f);
    if (FULL) return rw.sum(s, sx);
    return make_float2(0.f, rw.sum(sx));
}

// gate gamma_post of a segment (either may be null: 1).
template <bool VEC>
__device__ __forceinline__ void load_weight(const float* gamma, const float* gate, int c0, int lane,
                                            int left, Lane8& f) {
    load_param<VEC>(gamma, c0, lane, left, 1.f, f);
    if (!gate) return;
    Lane8 g;
    load_param<VEC>(gate, c0, lane, left, 1.f, g);
#pragma unroll
    for (int j = 0; j < kEl / 2; ++j) f[j] = mul2(f[j], g[j]);
}

// The sums of a finished gate row, and of a finished worker.
template <bool VEC, bool FULL, int V, class RW>
__device__ __forceinline__ void flush_gate(const BlockBwd& p, int64_t gate, Lane8 (&A)[V],
                                           Lane8 (&B)[V], const RW& rw, float* columns) {
    const int64_t W = work_cols(p.cols), slots = block_bwd_slots(p.workers, p.gates);
    const int64_t slot = rw.block + gate;
    flush<VEC, V>(A, p.work + slot * W, p.cols, rw, columns);
    if (FULL) flush<VEC, V>(B, p.work + (slots + slot) * W, p.cols, rw, columns);
}
template <bool VEC, bool FULL, int V, class RW>
__device__ __forceinline__ void flush_worker(const BlockBwd& p, Lane8 (&C)[V], Lane8 (&E)[V],
                                             const RW& rw, float* columns) {
    const int64_t W = work_cols(p.cols), slots = block_bwd_slots(p.workers, p.gates);
    flush<VEC, V>(C, p.work + (2 * slots + rw.block) * W, p.cols, rw, columns);
    if (FULL)
        flush<VEC, V>(E, p.work + (2 * slots + p.workers + rw.block) * W, p.cols, rw, columns);
}

// Tensors off 16-byte boundaries: each row is loaded as its turn comes.
constexpr int kAnyV = 2;   // segments a warp

template <int DT, int V, int FMT, bool CLUSTER>
__global__ void __launch_bounds__(256, 2) block_bwd_any(const BlockBwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    constexpr bool VEC = false;
    extern __shared__ float4 shared[];   // several rows a block: their sums of columns
    __shared__ __align__(16) float red[kRedFloats];
    RowWarps<CLUSTER> rw(row_warps, red);
    float* columns = reinterpret_cast<float*>(shared);
    const float inv_n = 1.f / (float)p.cols;
    const int64_t D = p.cols;
    const int c0 = rw.w * V * kSeg;
    Lane8 A[V], B[V], C[V], E[V];
    zero(A);
    zero(B);
    zero(C);
    zero(E);
    // The normalised segment k of a row: from codes, or from the kept tensor.
    auto hat = [&](const void* src, const float* scales, const float* means, const float* rstds,
                   int64_t row, int k, Lane8& f) {
        const int c = c0 + k * kSeg, left = p.cols - c;
        if constexpr (FMT != kNoCodes) {
            Codes<VEC> q;
            float sc[2] = {0.f, 0.f};
            q.load(static_cast<const uint8_t*>(src) + row * D + c, rw.lane, left);
            load_scales<VEC>(scales + row * p.groups + c / kQGroup, rw.lane, left, sc);
            q.template get<FMT>(sc, f);
        } else {
            Raw<DT, VEC> r;
            r.load(static_cast<const T*>(src) + row * D + c, rw.lane, left);
            r.get(f);
            kept_hat(f, means ? __ldg(means + row) : 0.f, rstds ? __ldg(rstds + row) : 1.f);
            mask8<VEC>(f, rw.lane, left);
        }
    };
    for (Steps st(p, rw.block, rw.rows); !st.done(); st.next()) {
        const int64_t row = st.row(rw.y);
        if (st.has(rw.y)) {
            Lane8 t[V], x[V];
            zero(t);
            if (p.dh_out) {
                Raw<DT, VEC> r[V];
#pragma unroll
                for (int k = 0; k < V; ++k)
                    r[k].load(static_cast<const T*>(p.dh_out) + row * D + c0 + k * kSeg, rw.lane,
                              p.cols - c0 - k * kSeg);
#pragma unroll
                for (int k = 0; k < V; ++k) r[k].get(t[k]);
            }
            if (p.pre != kNormNone) {
                Lane8 g[V];
                Raw<DT, VEC> r[V];
#pragma unroll
                for (int k = 0; k < V; ++k)
                    r[k].load(static_cast<const T*>(p.dn) + row * D + c0 + k * kSeg, rw.lane,
                              p.cols - c0 - k * kSeg);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    hat(p.sh, p.scale_pre, p.mean_pre, p.rstd_pre, row, k, x[k]);
                    r[k].get(g[k]);
                }
                const float2 m = pre_half<true, V>(g, x, C, E, rw, [&](int k, Lane8& f) {
                    load_param<VEC>(p.gamma_pre, c0 + k * kSeg, rw.lane, p.cols - c0 - k * kSeg, 1.f, f);
                });
                back_through<VEC, true, V>(g, x, p.pre == kNormLayer ? m.x * inv_n : 0.f, m.y * inv_n,
                                           __ldg(p.rstd_pre + row), p.cols, rw);
#pragma unroll
                for (int k = 0; k < V; ++k)
#pragma unroll
                    for (int j = 0; j < kEl / 2; ++j) t[k][j] = add2(t[k][j], g[k][j]);
            }
            zero(x);
            if (p.su)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    hat(p.su, p.scale_post, p.mean_post, p.rstd_post, row, k, x[k]);
            // (all inputs of these columns have been read: dh may be any of them)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                Lane8 o;
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) o[j] = mul2(both(p.alpha), t[k][j]);
                store8<DT, VEC>(static_cast<T*>(p.dh) + row * D + c0 + k * kSeg, rw.lane,
                                p.cols - c0 - k * kSeg, o);
            }
            const float* gate = p.gate ? p.gate + st.gate * D : nullptr;
            const float2 m = post_half<true, V>(t, x, A, B, rw, p.post != kNormNone, [&](int k, Lane8& f) {
                load_weight<VEC>(p.gamma_post, gate, c0 + k * kSeg, rw.lane, p.cols - c0 - k * kSeg, f);
            });
            if (p.post != kNormNone)
                back_through<VEC, true, V>(t, x, p.post == kNormLayer ? m.x * inv_n : 0.f, m.y * inv_n,
                                           __ldg(p.rstd_post + row), p.cols, rw);
            if (p.du)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    store8<DT, VEC>(static_cast<T*>(p.du) + row * D + c0 + k * kSeg, rw.lane,
                                    p.cols - c0 - k * kSeg, t[k]);
        }
        if (st.last()) flush_gate<VEC, true, V>(p, st.gate, A, B, rw, columns);
    }
    flush_worker<VEC, true, V>(p, C, E, rw, columns);
    rw.end();
}

// A thread (not VEC: a warp) copies its share of the rows to come into a ring of
// its own, two rows ahead, dn and xhat in one group of copies, dh' and uhat in
// the next: each half of a slot is filled again as soon as it has been read.
// Shared memory: of a thread, in 16-byte quads, gate*gamma_post and gamma_pre;
// then two slots of two halves, a gradient (dn | dh') and what was kept (xhat |
// uhat), in quads of a thread or in bytes of a warp.
template <int DT, bool VEC, int V, int FMT>
struct BwdShared {
    static constexpr int Q = Raw<DT, true>::kQuads, ES = sizeof(typename Storage<DT>::T);
    static constexpr int kCoef = 2 * V * 2;
    static constexpr int kKept = V * Q;   // first quad of what was kept
    static constexpr int kHalf = FMT == kNoCodes ? 2 * V * Q : V * Q + (V + 1) / 2;
    static constexpr int kKeptBytes = FMT == kNoCodes ? kSegBytes<ES> : kSegBytes<1>;
    static constexpr int kHalfBytes = V * (kSegBytes<ES> + kKeptBytes);
    // of a warp
    static constexpr int kBytes = kCoef * 512 + 4 * (VEC ? kHalf * 512 : kHalfBytes);
};

// A row's scalars on one side (pre or post), read into registers a row ahead.
// (As 4-byte asynchronous copies they cost more than the registers: 167 us in
// place of 140 for 16384 x 4096 bf16 from e4m3.)
template <bool VEC, int V>
struct Scalars {
    float rstd, mean, scale[VEC ? V : 2 * V];
};

template <int DT, bool VEC, int V, int FMT, bool FULL, bool CLUSTER>
__global__ void __launch_bounds__(256, V == 4 || (FULL && V == 2) ? 1 : 2) block_bwd(const BlockBwd p, int row_warps) {
    using T = typename Storage<DT>::T;
    using S = BwdShared<DT, VEC, V, FMT>;
    constexpr int Q = S::Q, ES = S::ES;
    constexpr bool CODES = FMT != kNoCodes;
    extern __shared__ float4 shared[];
    __shared__ __align__(16) float red[kRedFloats];
    RowWarps<CLUSTER> rw(row_warps, red);
    const int y = rw.y;
    float4* mine = shared + threadIdx.x;   // quad i of the thread: mine[i * blockDim.x]
    const float inv_n = 1.f / (float)p.cols;
    const int c0 = rw.w * V * kSeg;
    const int col = c0 + rw.lane * kEl;
    const int group = (c0 >> 7) + (rw.lane >> 4);   // of the lane's first segment
    const bool has_pre = p.pre != kNormNone;
    // several rows a block: their sums of columns, behind all else
    float* columns = reinterpret_cast<float*>(reinterpret_cast<char*>(shared) + (blockDim.x >> 5) * S::kBytes);

    auto quad = [&](int slot, int half, int i) {
        return mine + (S::kCoef + (slot * 2 + half) * S::kHalf + i) * blockDim.x;
    };
    // not VEC: the warp's gradients and kept values of segment k
    auto segment = [&](int slot, int half, int k) {
        return reinterpret_cast<char*>(shared + S::kCoef * blockDim.x) +
               ((threadIdx.x >> 5) * 4 + slot * 2 + half) * S::kHalfBytes + k * kSegBytes<ES>;
    };
    auto kept = [&](int slot, int half, int k) {
        return segment(slot, half, V) + k * S::kKeptBytes;
    };
    // segment k's 8 codes
    auto code = [&](int slot, int half, int k) {
        return reinterpret_cast<uint2*>(quad(slot, half, S::kKept + k / 2)) + (k & 1);
    };
    auto fetch = [&](int slot, int half, int row, bool on) {
        const T* a = static_cast<const T*>(half == 0 ? p.dn : p.dh_out);
        const void* b = half == 0 ? p.sh : p.su;
        if constexpr (!VEC) {
            const int64_t total = p.rows * p.cols;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const int left = on ? p.cols - c0 - k * kSeg : 0;
                const int64_t first = (int64_t)row * p.cols + c0 + k * kSeg;
                copy_segment<ES>(segment(slot, half, k), a, first, a ? left : 0, total, rw.lane);
                copy_segment<CODES ? 1 : ES>(kept(slot, half, k), b, first, b ? left : 0, total, rw.lane);
            }
            copies_end();
            return;
        }
        const int64_t at = (int64_t)row * p.cols + col;
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const bool in = on && col + k * kSeg < p.cols;
#pragma unroll
            for (int i = 0; i < Q; ++i)
                copy_async<16>(quad(slot, half, k * Q + i), a + at + k * kSeg + i * 4, in && a);
            if constexpr (CODES) {
                copy_async<8>(code(slot, half, k), static_cast<const uint8_t*>(b) + at + k * kSeg, in && b);
            } else {
#pragma unroll
                for (int i = 0; i < Q; ++i)
                    copy_async<16>(quad(slot, half, S::kKept + k * Q + i),
                                   static_cast<const T*>(b) + at + k * kSeg + i * 4, in && b);
            }
        }
        copies_end();
    };
    // what no copy writes (past the row's end, a tensor that is not there) reads as zero
    if (VEC)
        for (int i = 0; i < S::kCoef + 4 * S::kHalf; ++i) mine[i * blockDim.x] = make_float4(0.f, 0.f, 0.f, 0.f);

    auto scalars = [&](Scalars<VEC, V>& r, bool pre, int row, bool on) {
        const float* rstd = pre ? p.rstd_pre : p.rstd_post;
        r.rstd = on && rstd ? __ldg(rstd + row) : 1.f;
        if constexpr (CODES) {
            const float* scale = pre ? p.scale_pre : p.scale_post;
            const bool in = on && (pre ? p.sh : p.su);
            const float* s = scale + (int64_t)row * p.groups;
            if constexpr (VEC) {
#pragma unroll
                for (int k = 0; k < V; ++k)
                    r.scale[k] = in && col + k * kSeg < p.cols ? __ldg(s + group + 2 * k) : 0.f;
            } else {
                const int g = c0 / kQGroup;
#pragma unroll
                for (int k = 0; k < 2 * V; ++k) r.scale[k] = in && g + k < p.groups ? __ldg(s + g + k) : 0.f;
            }
        } else if constexpr (FULL) {
            const float* mean = pre ? p.mean_pre : p.mean_post;
            r.mean = on && mean ? __ldg(mean + row) : 0.f;
        }
    };
    // the normalised values and the gradients of segment k of the row in a slot
    auto hat = [&](int slot, int half, int k, int row, const Scalars<VEC, V>& r, Lane8& f) {
        const int left = p.cols - c0 - k * kSeg;
        if constexpr (CODES) {
            if constexpr (VEC) {
                Codes<true> c;
                c.v = *code(slot, half, k);
                const float two[2] = {r.scale[k], r.scale[k]};
                c.template get<FMT>(two, f);
            } else {
                const Codes<false> c = read_codes(kept(slot, half, k), (int64_t)row * p.cols + c0 + k * kSeg, rw.lane);
                const float two[2] = {r.scale[2 * k], r.scale[2 * k + 1]};
                c.template get<FMT>(two, f);
                mask8<false>(f, rw.lane, (half == 0 ? p.sh : p.su) ? left : 0);
            }
        } else {
            if constexpr (VEC) {
                Raw<DT, true> q;
#pragma unroll
                for (int i = 0; i < Q; ++i) q.v[i] = *reinterpret_cast<uint4*>(quad(slot, half, S::kKept + k * Q + i));
                q.get(f);
            } else {
                read_segment<DT>(kept(slot, half, k), (int64_t)row * p.cols + c0 + k * kSeg,
                                 (half == 0 ? p.sh : p.su) ? left : 0, rw.lane, f);
            }
            kept_hat(f, FULL ? r.mean : 0.f, r.rstd);
            if (FULL) mask8<VEC>(f, rw.lane, left);
        }
    };
    auto grad = [&](int slot, int half, int k, int row, Lane8& f) {
        if constexpr (VEC) {
            Raw<DT, true> q;
#pragma unroll
            for (int i = 0; i < Q; ++i) q.v[i] = *reinterpret_cast<uint4*>(quad(slot, half, k * Q + i));
            q.get(f);
        } else {
            read_segment<DT>(segment(slot, half, k), (int64_t)row * p.cols + c0 + k * kSeg,
                             (half == 0 ? p.dn : p.dh_out) ? p.cols - c0 - k * kSeg : 0, rw.lane, f);
        }
    };
    // not VEC: a warp's copies are there for all of its lanes, or read by all
    auto lanes_meet = [&]() {
        if (!VEC) __syncwarp();
    };
    auto coef = [&](int which, int k, Lane8& f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = mine[((which * V + k) * 2 + i) * blockDim.x];
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    };
    auto set_coef = [&](int which, const float* gamma, const float* gate) {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Lane8 f;
            load_weight<VEC>(gamma, gate, c0 + k * kSeg, rw.lane, p.cols - c0 - k * kSeg, f);
#pragma unroll
            for (int i = 0; i < 2; ++i)
                mine[((which * V + k) * 2 + i) * blockDim.x] =
                    make_float4(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x, f[2 * i + 1].y);
        }
    };

    Steps st(p, rw.block, rw.rows), ahead(p, rw.block, rw.rows);
    auto fetch_next = [&](int slot, int half) { fetch(slot, half, ahead.row(y), !ahead.done() && ahead.has(y)); };
    fetch_next(0, 0);
    fetch_next(0, 1);
    Scalars<VEC, V> pre, post;
    scalars(pre, true, st.row(y), st.has(y));
    scalars(post, false, st.row(y), st.has(y));
    ahead.next();
    fetch_next(1, 0);
    fetch_next(1, 1);
    set_coef(1, p.gamma_pre, nullptr);
    set_coef(0, p.gamma_post, p.gate ? p.gate + st.gate * p.cols : nullptr);
    Lane8 A[V], B[V], C[V], E[V];
    zero(A);
    zero(C);
    if (FULL) {
        zero(B);
        zero(E);
    }
    for (int slot = 0; !st.done(); slot ^= 1) {
        const int row = st.row(y);
        const bool here = st.has(y);
        const int next = ahead.row(y);
        const bool next_on = !ahead.done() && ahead.has(y);
        ahead.next();
        copies_wait<3>();
        lanes_meet();
        Lane8 g[V], x[V];   // g: dn, then t
        if (has_pre) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                grad(slot, 0, k, row, g[k]);
                hat(slot, 0, k, row, pre, x[k]);
            }
            const float rstd = pre.rstd;
            scalars(pre, true, next, next_on);
            lanes_meet();
            fetch_next(slot, 0);
            if (here) {
                const float2 m = pre_half<FULL, V>(g, x, C, E, rw, [&](int k, Lane8& f) { coef(1, k, f); });
                back_through<VEC, FULL, V>(g, x, FULL && p.pre == kNormLayer ? m.x * inv_n : 0.f, m.y * inv_n,
                                            rstd, p.cols, rw);
            }
        } else {
            zero(g);
            fetch_next(slot, 0);
        }
        copies_wait<3>();
        lanes_meet();
#pragma unroll
        for (int k = 0; k < V; ++k) {
            Lane8 d;
            grad(slot, 1, k, row, d);
#pragma unroll
            for (int j = 0; j < kEl / 2; ++j) g[k][j] = add2(g[k][j], d[j]);
            hat(slot, 1, k, row, post, x[k]);
        }
        const float rstd = post.rstd;
        scalars(post, false, next, next_on);
        lanes_meet();
        fetch_next(slot, 1);
        if (here) {
            const int64_t at = (int64_t)row * p.cols + c0;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                Lane8 o;
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) o[j] = mul2(both(p.alpha), g[k][j]);
                store8<DT, VEC>(static_cast<T*>(p.dh) + at + k * kSeg, rw.lane, p.cols - c0 - k * kSeg, o);
            }
            const float2 m = post_half<FULL, V>(g, x, A, B, rw, p.post != kNormNone,
                                                [&](int k, Lane8& f) { coef(0, k, f); });
            if (p.post != kNormNone)
                back_through<VEC, FULL, V>(g, x, FULL && p.post == kNormLayer ? m.x * inv_n : 0.f,
                                            m.y * inv_n, rstd, p.cols, rw);
            if (p.du)
#pragma unroll
                for (int k = 0; k < V; ++k)
                    store8<DT, VEC>(static_cast<T*>(p.du) + at + k * kSeg, rw.lane, p.cols - c0 - k * kSeg, g[k]);
        }
        const bool last = st.last();
        if (last)
            flush_gate<VEC, FULL, V>(p, st.gate, A, B, rw,
                                      columns);
        st.next();
        if (last && p.gate && p.rows_per_gate > 0 && !st.done())
            set_coef(0, p.gamma_post, p.gate + st.gate * p.cols);
    }
    copies_wait<0>();
    flush_worker<VEC, FULL, V>(p, C, E, rw, columns);
    rw.end();
}

// The column pass: a block takes 64 columns, two a thread of a warp, its 32
// warps share the partial sums of them.  blockIdx.y 0: dgamma_pre, dbeta_pre;
// 1: dgamma_post, dbeta_post and, of a single gate row, dgate; from 2: the
// gate rows, of several.
constexpr int kColWarps = 32;
constexpr int kColCols = 64;

// The block's totals of a and b, of column `threadIdx.x` (threads below 64).
__device__ __forceinline__ float2 add_warps(float2 a, float2 b, float2 (&sh)[2][kColWarps][32]) {
    __syncthreads();
    sh[0][threadIdx.x >> 5][threadIdx.x & 31] = a;
    sh[1][threadIdx.x >> 5][threadIdx.x & 31] = b;
    __syncthreads();
    float2 t = both(0.f);
    if (threadIdx.x < kColCols)
#pragma unroll
        for (int w = 0; w < kColWarps; ++w) {
            t.x += reinterpret_cast<const float*>(sh[0][w])[threadIdx.x];
            t.y += reinterpret_cast<const float*>(sh[1][w])[threadIdx.x];
        }
    return t;
}

__global__ void __launch_bounds__(32 * kColWarps) block_bwd_columns(const BlockBwd p) {
    __shared__ float2 sh[2][kColWarps][32];
    const int w = threadIdx.x >> 5, l = threadIdx.x & 31;
    const int64_t W = work_cols(p.cols);
    const int c = blockIdx.x * kColCols + 2 * l;          // columns this thread reads
    const int co = blockIdx.x * kColCols + threadIdx.x;   // column it writes
    const bool in = c < W, out = co < p.cols && threadIdx.x < kColCols;
    const int64_t slots = block_bwd_slots(p.workers, p.gates);
    const float* A = p.work + c;
    const float* B = A + slots * W;
    const float* C = B + slots * W;
    const float* E = C + p.workers * W;
    const int P = p.rows > 0 ? (int)p.workers : 0;
    float2 a = both(0.f), b = both(0.f);
    auto row = [&](const float* base, int64_t i) { return __ldcs(reinterpret_cast<const float2*>(base + i * W)); };
    // the sum of partial rows [lo, hi), every kColWarps-th of them a warp's
    auto add_rows = [&](const float* base, int lo, int hi) {
        float2 t = both(0.f);
        if (in)
#pragma unroll 8
            for (int i = lo + w; i < hi; i += kColWarps) t = add2(t, row(base, i));
        return t;
    };
    const bool one_gate = p.gates == 1;
    if (blockIdx.y == 0) {
        if (p.dgamma_pre) a = add_rows(C, 0, P);
        if (p.dbeta_pre) b = add_rows(E, 0, P);
        const float2 t = add_warps(a, b, sh);
        if (out && p.dgamma_pre) p.dgamma_pre[co] = t.x;
        if (out && p.dbeta_pre) p.dbeta_pre[co] = t.y;
    } else if (blockIdx.y == 1 && one_gate) {
        a = add_rows(A, 0, P);
        if (p.dbeta_post || (p.dgate && p.beta_post)) b = add_rows(B, 0, P);
        const float2 t = add_warps(a, b, sh);
        if (out) {
            const float gate = p.gate ? p.gate[co] : 1.f;
            if (p.dgamma_post) p.dgamma_post[co] = gate * t.x;
            if (p.dbeta_post) p.dbeta_post[co] = gate * t.y;
            if (p.dgate)
                p.dgate[co] = fmaf(p.gamma_post ? p.gamma_post[co] : 1.f, t.x,
                                   p.beta_post ? p.beta_post[co] * t.y : 0.f);
        }
    } else if (blockIdx.y == 1) {
        if (in && P > 0 && (p.dgamma_post || p.dbeta_post)) {
            const Split s(p);
            const int per = (int)p.rows_per_gate;
            for (int i = w; i < P; i += kColWarps) {
                const int g1 = (s.first(i + 1) - 1) / per;
                for (int g = s.first(i) / per; g <= g1; ++g) {
                    const float* q = p.gate + (int64_t)g * p.cols + c;   // (several gate rows: there is a gate)
                    const float2 gt = make_float2(c < p.cols ? __ldg(q) : 0.f, c + 1 < p.cols ? __ldg(q + 1) : 0.f);
                    if (p.dgamma_post) a = fma2(gt, row(A, i + g), a);
                    if (p.dbeta_post) b = fma2(gt, row(B, i + g), b);
                }
            }
        }
        const float2 t = add_warps(a, b, sh);
        if (out && p.dgamma_post) p.dgamma_post[co] = t.x;
        if (out && p.dbeta_post) p.dbeta_post[co] = t.y;
    } else {
        const int per = (int)p.rows_per_gate;
        const Split s(p);
        for (int64_t g = blockIdx.y - 2; g < p.gates; g += gridDim.y - 2) {
            const int64_t lo = g * per, hi = min(lo + per, p.rows);
            // partial rows of the workers that hold rows lo .. hi - 1
            const int w0 = s.worker((int)lo), w1 = s.worker((int)(hi - 1)) + 1;
            a = add_rows(A + g * W, w0, w1);
            if (p.beta_post) b = add_rows(B + g * W, w0, w1);
            const float2 t = add_warps(a, b, sh);
            if (out)
                p.dgate[g * p.cols + co] = fmaf(p.gamma_post ? p.gamma_post[co] : 1.f, t.x,
                                                p.beta_post ? p.beta_post[co] * t.y : 0.f);
        }
    }
}

// Shared memory for the sums of columns of a block's rows.
size_t columns_bytes(const RowShape& s) {
    return s.rows > 1 ? s.rows * s.warps * kSeg * sizeof(float) : 0;
}

template <int DT, int FMT, bool CLUSTER>
cudaError_t launch_any(const BlockBwd& a, const RowShape& s, cudaStream_t stream) {
    return launch_rows<block_bwd_any<DT, kAnyV, FMT, CLUSTER>>(s, a.workers, columns_bytes(s), stream, a);
}

template <int DT, bool VEC, int V, int FMT, bool FULL, bool CLUSTER>
cudaError_t launch(const BlockBwd& a, const RowShape& s, cudaStream_t stream) {
    const size_t smem = (size_t)BwdShared<DT, VEC, V, FMT>::kBytes * (s.threads() / 32) + columns_bytes(s);
    return launch_rows<block_bwd<DT, VEC, V, FMT, FULL, CLUSTER>>(s, a.workers, smem, stream, a);
}

// SHARED: the width may take a cluster.
template <int DT, bool VEC, int V, int FMT, bool FULL, bool SHARED>
cudaError_t by_shape(const BlockBwd& a, cudaStream_t stream) {
    const RowShape s = RowShape::of<V>(a.cols, V == 4 ? kBwdThreads : 2 * kBwdThreads, kBwdWarps);
    if constexpr (SHARED)
        if (s.cluster > 1) return launch<DT, VEC, V, FMT, FULL, true>(a, s, stream);
    return launch<DT, VEC, V, FMT, FULL, false>(a, s, stream);
}

// Segments a warp, by measurement (bf16 from e4m3): with all four sums of
// columns (FULL) two segments leave 54 registers spilled at two blocks an SM,
// four keep everything in registers (16384 x 4096: 261 and 162 us; x 2048: 144
// and 92); with two sums both fit, and two segments are as fast up to 4096
// columns (16384 x 4096: 130 and 132 us; x 1024: 41 and 44), while above four
// keep a row in one block (8192 x 8192: 196 us with a cluster of two, 143).
// One segment a warp makes a row's way through its warps shorter, which counts
// where a worker has few rows: 3001 x 1021 kept fp32 53 us with two, 32 with
// one; 300 x 2048 16.7 and 12.6; and up to 1024 columns with all four sums
// always (16384 x 1024: 59 and 52).
// In fp32 four take too much shared memory for more than one small block an SM:
// two (3001 x 4096 kept: 131 and 111 us), and clusters above 4096 columns.
template <int DT, bool VEC, int FMT, bool FULL>
cudaError_t by_width(const BlockBwd& a, cudaStream_t stream) {
    if (a.cols <= 2048 && ((FULL && a.cols <= 1024) || a.rows < 16 * a.workers))
        return by_shape<DT, VEC, 1, FMT, FULL, false>(a, stream);
    if constexpr (DT == kF32) {
        return by_shape<DT, VEC, 2, FMT, FULL, true>(a, stream);
    } else {
        if constexpr (!FULL)
            if (a.cols <= 4096) return by_shape<DT, VEC, 2, FMT, FULL, false>(a, stream);
        return by_shape<DT, VEC, 4, FMT, FULL, true>(a, stream);
    }
}

// vec: 16-byte accesses; ring: tensors on 16-byte boundaries.
template <int DT, int FMT>
cudaError_t by_alignment(const BlockBwd& a, bool vec, bool ring, cudaStream_t stream) {
    count_launches(1);
    const bool full = a.post == kNormLayer || a.pre == kNormLayer || a.dbeta_post || a.dbeta_pre ||
                      (a.dgate && a.beta_post);
    if (vec) return full ? by_width<DT, true, FMT, true>(a, stream) : by_width<DT, true, FMT, false>(a, stream);
    if (ring) return full ? by_width<DT, false, FMT, true>(a, stream) : by_width<DT, false, FMT, false>(a, stream);
    const RowShape s = RowShape::of<kAnyV>(a.cols, 256, kBwdWarps);
    return s.cluster > 1 ? launch_any<DT, FMT, true>(a, s, stream) : launch_any<DT, FMT, false>(a, s, stream);
}

template <int DT>
cudaError_t by_format(const BlockBwd& a, bool vec, bool ring, bool codes, cudaStream_t s) {
    if (!codes) return by_alignment<DT, kNoCodes>(a, vec, ring, s);
    return a.format == kE4M3 ? by_alignment<DT, kE4M3>(a, vec, ring, s) : by_alignment<DT, kInt8>(a, vec, ring, s);
}

}  // namespace

// For the 16-bit types one wave of the row pass's blocks on 148 SMs: two an SM
// up to 4096 columns, one above, where clusters of them share rows of more than
// 8192.  fp32 takes the same number of workers, since the workspace's size does
// not know the type; with its two segments a warp above 2048 columns a block of
// six warps or more has an SM to itself and rows of more than 4096 columns take
// clusters, so its 296 blocks are two waves (3001 x 4096 kept layer norms 101 us,
// floor 46).
int64_t block_bwd_workers(int64_t rows, int64_t cols) {
    const int64_t most = cols <= 4096 ? 296 : 148 / RowShape::of<4>((int)cols, kBwdThreads, kBwdWarps).cluster;
    return rows < 1 ? 1 : rows < most ? rows : most;
}

cudaError_t block_backward(const BlockBwd& a, int dtype, bool codes, cudaStream_t s, int) {
    if (a.rows > 0) {
        const bool ring = on16(a.su) && on16(a.sh) && on16(a.dh_out) && on16(a.dn);
        const bool vec = a.cols % kEl == 0 && ring && on16(a.dh) && on16(a.du);
        const cudaError_t e = dtype == kF32    ? by_format<kF32>(a, vec, ring, codes, s)
                              : dtype == kBF16 ? by_format<kBF16>(a, vec, ring, codes, s)
                                               : by_format<kF16>(a, vec, ring, codes, s);
        if (e != cudaSuccess) return e;
    }
    const bool pre = a.dgamma_pre || a.dbeta_pre, post = a.dgamma_post || a.dbeta_post;
    if (!pre && !post && !a.dgate) return cudaSuccess;
    const int64_t gates = a.dgate && a.gates > 1 ? (a.gates < 4096 ? a.gates : 4096) : 0;
    const dim3 grid((unsigned)((a.cols + kColCols - 1) / kColCols), (unsigned)(2 + gates));
    block_bwd_columns<<<grid, 32 * kColWarps, 0, s>>>(a);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace iabn
