// iabn_gated.cu -- the gated activation z = phi(a) b and its backward, with
// or without 8-bit checkpoints of a and b.
//
// Each phi is written as a w(a), w the logistic function of a (SILU), of
// 2 sqrt(2/pi) (a + 0.044715 a^3) (GELU_TANH: (1 + tanh y)/2 = 1/(1 + e^-2y),
// which does not cancel for large negative y), or the normal distribution
// function (GELU), so phi' = w + a w'.
// Elementwise; a warp takes 256 columns (two checkpoint groups) of many rows.
// Floor: 3 s bytes an element forward (2 more with checkpoints), 3 s + 2
// backward from codes, s more for z.
// Measured (GPU time, B200): 8192 x 14336 bf16 SiLU with int8 checkpoints,
// forward 163 us (5.8 TB/s, floor 147), backward with z 204 us (floor 184); GELU
// by erfc 280 and 321 us; storing 16384 x 5120 bf16 as e4m3 44 us (floor 39.5),
// loading 16384 x 4096 with a scale 36 us (floor 31.6); 777 x 2731 fp16 GELU
// backward from e4m3 11 us (floor 2.7), SiLU 6.2 us, and in 2736 columns, eight
// at a time, 7.9 and 4.6 us: erfc and elements one by one.
#include "iabn_rows.cuh"

namespace iabn {

void count_launches(int n);

namespace {

// 2^x and 1/x for the 16-bit types: one special-function instruction each
// (relative error about 2^-22 and 2^-23), results below 2^-126 flushed to 0.
// e^x is 2^(x log2 e), whose rounded argument adds about |x| 2^-24 to that.
__device__ __forceinline__ float fast_exp2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float fast_inverse(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
template <int DT>
__device__ __forceinline__ float2 exp_of(float2 x) {
    if (DT == kF32) return make_float2(expf(x.x), expf(x.y));
    x = mul2(x, both(1.4426950408889634f));
    return make_float2(fast_exp2(x.x), fast_exp2(x.y));
}
template <int DT>
__device__ __forceinline__ float inverse(float x) {   // of 1 + e^y: in [1, inf]
    return DT == kF32 ? 1.f / x : fast_inverse(x);
}

// w(a), and a w'(a) where SLOPE, of two values.
template <int ACT, int DT, bool SLOPE>
__device__ __forceinline__ void weight2(float2 a, float2& w, float2& aw) {
    if constexpr (ACT == kSilu || ACT == kGeluTanh) {
        float2 y = mul2(a, both(-1.f)), c = a, q;   // w = 1/(1 + e^y)
        if constexpr (ACT == kGeluTanh) {
            // beyond +-32 w is 0 or 1 in fp32: the clamp keeps a^3 finite
            c = make_float2(fminf(fmaxf(a.x, -32.f), 32.f), fminf(fmaxf(a.y, -32.f), 32.f));
            q = mul2(mul2(c, c), both(0.044715f));
            y = mul2(mul2(c, both(-1.5957691216057308f)), add2(q, both(1.f)));
        }
        const float2 d = add2(exp_of<DT>(y), both(1.f));
        w = make_float2(inverse<DT>(d.x), inverse<DT>(d.y));
        if (SLOPE) {
            aw = mul2(mul2(c, w), fma2(w, both(-1.f), both(1.f)));
            if constexpr (ACT == kGeluTanh)
                aw = mul2(mul2(aw, both(1.5957691216057308f)), fma2(q, both(3.f), both(1.f)));
        }
        if constexpr (ACT == kGeluTanh) {   // the clamp loses NaN
            if (a.x != a.x) w.x = a.x;
            if (a.y != a.y) w.y = a.y;
        }
    } else {
        w = make_float2(0.5f * erfcf(a.x * -0.70710678118654752f),
                        0.5f * erfcf(a.y * -0.70710678118654752f));
        if (SLOPE)
            aw = mul2(mul2(a, both(0.39894228040143268f)),
                      exp_of<DT>(mul2(mul2(a, a), both(-0.5f))));
    }
}

// A warp's share of [rows, cols]: one segment of columns (so that what goes by
// column is read once) of every `lanes`-th row, from `row` on; consecutive
// warps hold consecutive segments of a row.  Where there are more segments
// than warps, a warp takes several in turn.
struct Strip {
    int segs, lanes;
};

template <class F>
__device__ __forceinline__ void for_strips(const Strip& t, int64_t cols, F body) {
    const int64_t all = (int64_t)t.segs * t.lanes;
    const int64_t warps = (int64_t)gridDim.x * (blockDim.x >> 5);
    for (int64_t w = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5); w < all; w += warps) {
        const int64_t row = w / t.segs;
        const int64_t c0 = (w - row * t.segs) * kSeg;
        body(row, c0, (int)min(cols - c0, (int64_t)kSeg));
    }
}

// An offset that walks down a strip of a tensor with row stride ld: [i] is i
// rows of the strip ahead.  Tensors of one stride share it.
struct Down {
    int64_t at, step;
    __device__ __forceinline__ Down(int64_t row, int64_t ld, int64_t col, int lanes)
        : at(row * ld + col), step(ld * lanes) {}
    __device__ __forceinline__ int64_t operator[](int i) const { return at + i * step; }
    __device__ __forceinline__ void advance(int n) { at += n * step; }
};

// Rows of a strip that are loaded before any is worked on, and blocks an SM:
// with fewer bytes in flight HBM waits, with more the registers run out (8192 x
// 14336 bf16, int8 checkpoints, forward: 2 rows and 4 blocks 182 us; 1 and 4
// 193, 1 and 6 195, 2 and 3 189, 4 and 2 194, 4 and 3 186; all before later
// steps made each faster).  Elements one by one take eight times the load
// instructions, so one row ahead is enough (777 x 2731, compared on one box: 10.4
// us, 13.1 with two).
constexpr int kVecAhead = 2;
constexpr int kBlocks = 4;

template <int DT, bool VEC, int ACT, int FMT>
__global__ void __launch_bounds__(256, kBlocks) gated_fwd(const Gated p, const Strip t) {
    constexpr int kAhead = VEC ? kVecAhead : 1;
    using T = typename Storage<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for_strips(t, p.cols, [&](int64_t row0, int64_t c0, int left) {
        Down in(row0, p.ld, c0, t.lanes), out(row0, p.cols, c0, t.lanes);
        Down grp(row0, groups, c0 / kQGroup, t.lanes);
        const T *pa = static_cast<const T*>(p.a), *pb = static_cast<const T*>(p.b);
        T* pz = static_cast<T*>(p.z);
        for (int64_t rows = p.rows - row0; rows > 0; rows -= kAhead * t.lanes) {
            Raw<DT, VEC> ra[kAhead], rb[kAhead];
            bool on[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                on[i] = rows > i * t.lanes;
                ra[i].load(pa + in[i], lane, on[i] ? left : 0);
                rb[i].load(pb + in[i], lane, on[i] ? left : 0);
            }
            float by[2 * kAhead];
            if constexpr (FMT != kNoCodes && VEC) {
                const uint32_t m[4] = {raw_amax(ra[0]), raw_amax(rb[0]), raw_amax(ra[1]), raw_amax(rb[1])};
                const float scale = group_scales<FMT, DT, 4>(m, lane, by);
                const int i = group_carried<4>(lane);   // row i/2, a or b
                if (group_writer<4>(lane) && (lane & 16) * kEl < left && rows > (i >> 1) * t.lanes)
                    (i & 1 ? p.sb_out : p.sa_out)[grp[i >> 1] + (lane >> 4)] = scale;
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (!on[i]) break;
                Lane8 a, b, z;
                ra[i].get(a);
                rb[i].get(b);
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) {
                    float2 w, aw;
                    weight2<ACT, DT, false>(a[j], w, aw);
                    z[j] = mul2(mul2(a[j], w), b[j]);
                }
                store8<DT, VEC>(pz + out[i], lane, left, z);
                if constexpr (FMT != kNoCodes && VEC) {
                    encode8<FMT>(a, by[2 * i], p.qa_out + out[i], lane, left);
                    encode8<FMT>(b, by[2 * i + 1], p.qb_out + out[i], lane, left);
                } else if constexpr (FMT != kNoCodes) {
                    quantise_any<FMT>(a, p.qa_out + out[i], p.sa_out + grp[i], lane, left);
                    quantise_any<FMT>(b, p.qb_out + out[i], p.sb_out + grp[i], lane, left);
                }
            }
            in.advance(kAhead);
            out.advance(kAhead);
            grp.advance(kAhead);
        }
    });
}

template <int DT, bool VEC, int ACT, int FMT>
__global__ void __launch_bounds__(256, kBlocks) gated_bwd(const Gated p, const Strip t) {
    constexpr int kAhead = VEC ? kVecAhead : 1;
    using T = typename Storage<DT>::T;
    constexpr bool CODES = FMT != kNoCodes;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for_strips(t, p.cols, [&](int64_t row0, int64_t c0, int left) {
        Down in(row0, p.ld, c0, t.lanes), out(row0, p.cols, c0, t.lanes);
        Down grad(row0, p.ld_grad, c0, t.lanes), grp(row0, groups, c0 / kQGroup, t.lanes);
        const T *pa = static_cast<const T*>(p.a), *pb = static_cast<const T*>(p.b);
        const T* pdz = static_cast<const T*>(p.dz);
        T *pda = static_cast<T*>(p.da), *pdb = static_cast<T*>(p.db), *pz = static_cast<T*>(p.z);
        for (int64_t rows = p.rows - row0; rows > 0; rows -= kAhead * t.lanes) {
            Raw<DT, VEC> rz[kAhead], ra[CODES ? 1 : kAhead], rb[CODES ? 1 : kAhead];
            Codes<VEC> ca[CODES ? kAhead : 1], cb[CODES ? kAhead : 1];
            float fa[CODES ? kAhead : 1][2], fb[CODES ? kAhead : 1][2];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const int here = rows > i * t.lanes ? left : 0;
                rz[i].load(pdz + out[i], lane, here);
                if constexpr (CODES) {
                    ca[i].load(p.qa + out[i], lane, here);
                    cb[i].load(p.qb + out[i], lane, here);
                    load_scales<VEC>(p.sa + grp[i], lane, here, fa[i]);
                    load_scales<VEC>(p.sb + grp[i], lane, here, fb[i]);
                } else {
                    ra[i].load(pa + in[i], lane, here);
                    rb[i].load(pb + in[i], lane, here);
                }
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                if (rows <= i * t.lanes) break;
                Lane8 a, b, dz, z;
                if constexpr (CODES) {
                    ca[i].template get<FMT>(fa[i], a);
                    cb[i].template get<FMT>(fb[i], b);
                } else {
                    ra[i].get(a);
                    rb[i].get(b);
                }
                rz[i].get(dz);
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) {
                    float2 w, aw;
                    weight2<ACT, DT, true>(a[j], w, aw);
                    const float2 phi = mul2(a[j], w);
                    z[j] = mul2(phi, b[j]);
                    a[j] = mul2(mul2(dz[j], b[j]), add2(w, aw));
                    b[j] = mul2(dz[j], phi);
                }
                store8<DT, VEC>(pda + grad[i], lane, left, a);
                store8<DT, VEC>(pdb + grad[i], lane, left, b);
                if (p.z) store8<DT, VEC>(pz + out[i], lane, left, z);
            }
            out.advance(kAhead);
            grad.advance(kAhead);
            if constexpr (CODES) grp.advance(kAhead);
            else in.advance(kAhead);
        }
    });
}

constexpr int kCheckAhead = 4;

template <int DT, bool VEC, int FMT>
__global__ void __launch_bounds__(256, kBlocks) store_kernel(const Check8 p, const Strip t) {
    using T = typename Storage<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for_strips(t, p.cols, [&](int64_t row0, int64_t c0, int left) {
        Down in(row0, p.ld, c0, t.lanes), out(row0, p.cols, c0, t.lanes);
        Down grp(row0, groups, c0 / kQGroup, t.lanes);
        const T* px = static_cast<const T*>(p.x);
        for (int64_t rows = p.rows - row0; rows > 0; rows -= kCheckAhead * t.lanes) {
            Raw<DT, VEC> raw[kCheckAhead];
            bool on[kCheckAhead];
#pragma unroll
            for (int i = 0; i < kCheckAhead; ++i) {
                on[i] = rows > i * t.lanes;
                raw[i].load(px + in[i], lane, on[i] ? left : 0);
            }
            float by[kCheckAhead];
            if constexpr (VEC) {
                const uint32_t m[4] = {raw_amax(raw[0]), raw_amax(raw[1]), raw_amax(raw[2]), raw_amax(raw[3])};
                const float scale = group_scales<FMT, DT, 4>(m, lane, by);
                const int i = group_carried<4>(lane);
                if (group_writer<4>(lane) && (lane & 16) * kEl < left && rows > i * t.lanes)
                    p.scale[grp[i] + (lane >> 4)] = scale;
            }
#pragma unroll
            for (int i = 0; i < kCheckAhead; ++i) {
                if (!on[i]) break;
                Lane8 x;
                raw[i].get(x);
                if constexpr (VEC) {
                    encode8<FMT>(x, by[i], p.q + out[i], lane, left);
                } else {
                    quantise_any<FMT>(x, p.q + out[i], p.scale + grp[i], lane, left);
                }
            }
            in.advance(kCheckAhead);
            out.advance(kCheckAhead);
            grp.advance(kCheckAhead);
        }
    });
}

template <int DT, bool VEC, int FMT>
__global__ void __launch_bounds__(256, kBlocks) load_kernel(const Check8 p, const Strip t) {
    using T = typename Storage<DT>::T;
    const int lane = threadIdx.x & 31;
    const int64_t groups = (p.cols + kQGroup - 1) / kQGroup;
    for_strips(t, p.cols, [&](int64_t row0, int64_t c0, int left) {
        Lane8 ga, be;
        load_param<VEC>(p.gamma, c0, lane, left, 1.f, ga);
        load_param<VEC>(p.beta, c0, lane, left, 0.f, be);
        Down in(row0, p.cols, c0, t.lanes), out(row0, p.ld, c0, t.lanes);
        Down grp(row0, groups, c0 / kQGroup, t.lanes);
        T* py = static_cast<T*>(p.y);
        for (int64_t rows = p.rows - row0; rows > 0; rows -= kCheckAhead * t.lanes) {
            Codes<VEC> c[kCheckAhead];
            float f[kCheckAhead][2];
#pragma unroll
            for (int i = 0; i < kCheckAhead; ++i) {
                const int here = rows > i * t.lanes ? left : 0;
                c[i].load(p.q + in[i], lane, here);
                load_scales<VEC>(p.scale + grp[i], lane, here, f[i]);
            }
#pragma unroll
            for (int i = 0; i < kCheckAhead; ++i) {
                if (rows <= i * t.lanes) break;
                Lane8 x;
                c[i].template get<FMT>(f[i], x);
#pragma unroll
                for (int j = 0; j < kEl / 2; ++j) x[j] = fma2(ga[j], x[j], be[j]);
                store8<DT, VEC>(py + out[i], lane, left, x);
            }
            in.advance(kCheckAhead);
            out.advance(kCheckAhead);
            grp.advance(kCheckAhead);
        }
    });
}

// Strips for one wave of `warps` warps an SM, and the blocks of 8 warps.
unsigned strips(int64_t rows, int64_t cols, int sms, int warps, Strip& t) {
    t.segs = (int)((cols + kSeg - 1) / kSeg);
    const int64_t all = (int64_t)sms * warps;
    int64_t lanes = all / t.segs;
    if (lanes > rows) lanes = rows;
    t.lanes = (int)(lanes < 1 ? 1 : lanes);
    const int64_t n = ((int64_t)t.segs * t.lanes + 7) / 8;
    return (unsigned)(n < all / 8 ? n : all / 8);
}

// The launch of one operator for a storage type, alignment and format.
struct Launch {
    Strip t;
    unsigned n;
    cudaStream_t s;
};

template <int DT, bool VEC, int ACT, int FMT>
void run_gated(const Gated& a, bool back, const Launch& l) {
    if (back) gated_bwd<DT, VEC, ACT, FMT><<<l.n, 256, 0, l.s>>>(a, l.t);
    else gated_fwd<DT, VEC, ACT, FMT><<<l.n, 256, 0, l.s>>>(a, l.t);
}

template <int DT, bool VEC, int ACT>
void by_format(const Gated& a, int format, bool back, const Launch& l) {
    if (format == kNoCodes) run_gated<DT, VEC, ACT, kNoCodes>(a, back, l);
    else if (format == kE4M3) run_gated<DT, VEC, ACT, kE4M3>(a, back, l);
    else run_gated<DT, VEC, ACT, kInt8>(a, back, l);
}

template <int DT, bool VEC>
void by_act(const Gated& a, int format, bool back, const Launch& l) {
    if (a.act == kSilu) by_format<DT, VEC, kSilu>(a, format, back, l);
    else if (a.act == kGelu) by_format<DT, VEC, kGelu>(a, format, back, l);
    else by_format<DT, VEC, kGeluTanh>(a, format, back, l);
}

template <int DT>
void by_vec(const Gated& a, bool vec, int format, bool back, const Launch& l) {
    if (vec) by_act<DT, true>(a, format, back, l);
    else by_act<DT, false>(a, format, back, l);
}

cudaError_t run(const Gated& a, int dtype, bool back, bool codes, cudaStream_t s, int sms) {
    if (a.rows == 0) return cudaSuccess;
    const bool strides = (!a.a || a.ld % kEl == 0) && (!back || a.ld_grad % kEl == 0);
    const bool vec = a.cols % kEl == 0 && strides && on16(a.a) && on16(a.b) && on16(a.qa) &&
                     on16(a.qb) && on16(a.qa_out) && on16(a.qb_out) && on16(a.dz) && on16(a.z) &&
                     on16(a.da) && on16(a.db);
    Launch l;
    l.n = strips(a.rows, a.cols, sms, 8 * kBlocks, l.t);
    l.s = s;
    const int format = codes ? a.format : kNoCodes;
    if (dtype == kF32) by_vec<kF32>(a, vec, format, back, l);
    else if (dtype == kBF16) by_vec<kBF16>(a, vec, format, back, l);
    else by_vec<kF16>(a, vec, format, back, l);
    count_launches(1);
    return cudaGetLastError();
}

template <int DT, bool VEC, int FMT>
void run_check8(const Check8& a, bool load, const Launch& l) {
    if (load) load_kernel<DT, VEC, FMT><<<l.n, 256, 0, l.s>>>(a, l.t);
    else store_kernel<DT, VEC, FMT><<<l.n, 256, 0, l.s>>>(a, l.t);
}

template <int DT>
void by_format(const Check8& a, bool vec, bool load, const Launch& l) {
    if (a.format == kE4M3) {
        if (vec) run_check8<DT, true, kE4M3>(a, load, l);
        else run_check8<DT, false, kE4M3>(a, load, l);
    } else {
        if (vec) run_check8<DT, true, kInt8>(a, load, l);
        else run_check8<DT, false, kInt8>(a, load, l);
    }
}

cudaError_t check8(const Check8& a, int dtype, bool load, cudaStream_t s, int sms) {
    if (a.rows == 0) return cudaSuccess;
    const bool vec = a.cols % kEl == 0 && a.ld % kEl == 0 && on16(a.x) && on16(a.y) && on16(a.q);
    Launch l;
    l.n = strips(a.rows, a.cols, sms, 8 * kBlocks, l.t);
    l.s = s;
    if (dtype == kF32) by_format<kF32>(a, vec, load, l);
    else if (dtype == kBF16) by_format<kBF16>(a, vec, load, l);
    else by_format<kF16>(a, vec, load, l);
    count_launches(1);
    return cudaGetLastError();
}

}  // namespace

cudaError_t gated_forward(const Gated& a, int dtype, cudaStream_t s, int sms) {
    return run(a, dtype, false, a.qa_out != nullptr, s, sms);
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
