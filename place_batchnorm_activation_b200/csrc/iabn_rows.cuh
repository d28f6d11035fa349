// iabn_rows.cuh -- device-side building blocks of the row operators
// (iabn_block.h): how a warp's lanes share a row, loads and stores of the
// storage types and of 8-bit codes, the 8-bit quantiser, sums over a row and
// a thread's asynchronous ring.
//
// A warp takes a segment of 256 columns of a row, eight a lane.  Two maps:
//   VEC   lane l holds columns 8l .. 8l+7: one 16-byte access (two for fp32)
//         and one 8-byte access of codes a lane.  Needs widths that are
//         multiples of 8 and 16-byte aligned rows.
//   else  lane l holds columns l, l+32, .., l+224: any width and alignment, a
//         warp's accesses still being consecutive elements.
// Either way a segment holds two checkpoint groups of 128 columns: lanes 0-15
// and 16-31 under VEC, elements 0-3 and 4-7 of every lane otherwise.
//
// A lane's eight values are four float2, worked on two at a time (the f32x2
// instructions): these kernels are bound by the instructions they issue as
// soon as they are near the HBM rate.
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "iabn_block_internal.h"
#include "iabn_device.cuh"

namespace iabn {

constexpr int kSeg = 256;   // columns of a warp's segment
constexpr int kEl = 8;      // of them, a lane's
using Lane8 = float2[kEl / 2];

template <bool VEC>
__device__ __forceinline__ int seg_col(int lane, int j) {
    return VEC ? lane * kEl + j : lane + 32 * j;
}

// ------------------------------------------------------ two values at a time

__device__ __forceinline__ unsigned long long bits2(float2 v) {
    unsigned long long r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(v.x), "f"(v.y));
    return r;
}
__device__ __forceinline__ float2 float2_of(unsigned long long b) {
    float2 v;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(v.x), "=f"(v.y) : "l"(b));
    return v;
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
    unsigned long long r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
    unsigned long long r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)));
    return float2_of(r);
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
    unsigned long long r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;"
        : "=l"(r) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
    return float2_of(r);
}
__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }

// Element j of a lane's eight.
__device__ __forceinline__ float& el(Lane8& f, int j) { return j & 1 ? f[j / 2].y : f[j / 2].x; }
__device__ __forceinline__ float el(const Lane8& f, int j) { return j & 1 ? f[j / 2].y : f[j / 2].x; }

// ----------------------------------------------------------- loads and stores

template <int DT> struct Pair { using T = __nv_bfloat162; };
template <> struct Pair<kF16> { using T = __half2; };

template <int DT>
__device__ __forceinline__ float2 unpack2(uint32_t w) {
    if (DT == kBF16) return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
    return __half22float2(*reinterpret_cast<const __half2*>(&w));
}
template <int DT>
__device__ __forceinline__ uint32_t pack2(float2 v) {
    if (DT == kBF16) {
        const __nv_bfloat162 t = __floats2bfloat162_rn(v.x, v.y);
        return *reinterpret_cast<const uint32_t*>(&t);
    }
    const __half2 t = __floats2half2_rn(v.x, v.y);
    return *reinterpret_cast<const uint32_t*>(&t);
}

// A lane's eight elements as they were loaded (a batch of loads is in flight
// before any is converted).
template <int DT, bool VEC>
struct Raw {
    using T = typename Storage<DT>::T;
    static constexpr int kQuads = DT == kF32 ? 2 : 1;   // 16-byte accesses under VEC
    union {
        uint4 v[kQuads];
        T e[kEl];
    };
    __device__ __forceinline__ Raw() {}
    // `p`: the segment's first element; `left`: columns of the row from there
    // (elements past it read as zero).
    __device__ __forceinline__ void load(const T* p, int lane, int left) {
        if (VEC) {
            const bool in = lane * kEl < left;
            const uint4* q = reinterpret_cast<const uint4*>(p + lane * kEl);
#pragma unroll
            for (int i = 0; i < kQuads; ++i) v[i] = in ? ldg_cs(q + i) : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < kEl; ++j) {
                const int c = lane + 32 * j;
                e[j] = c < left ? p[c] : T(0.f);
            }
        }
    }
    __device__ __forceinline__ void get(Lane8& f) const {
        if constexpr (DT == kF32 && VEC) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                f[2 * i] = make_float2(__uint_as_float(v[i].x), __uint_as_float(v[i].y));
                f[2 * i + 1] = make_float2(__uint_as_float(v[i].z), __uint_as_float(v[i].w));
            }
        } else if constexpr (!VEC) {
#pragma unroll
            for (int j = 0; j < kEl; ++j) el(f, j) = Storage<DT>::load(&e[j]);
        } else {
            f[0] = unpack2<DT>(v[0].x);
            f[1] = unpack2<DT>(v[0].y);
            f[2] = unpack2<DT>(v[0].z);
            f[3] = unpack2<DT>(v[0].w);
        }
    }
};

// Streaming stores where `on`, likewise without a branch.
__device__ __forceinline__ void store16_if(void* p, uint4 v, bool on) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %5, 0;\n\t"
                 "@p st.global.cs.v4.b32 [%0], {%1, %2, %3, %4}; }" ::"l"(p), "r"(v.x), "r"(v.y),
                 "r"(v.z), "r"(v.w), "r"((int)on)
                 : "memory");
}
__device__ __forceinline__ void store8_if(void* p, uint2 v, bool on) {
    asm volatile("{ .reg .pred p; setp.ne.b32 p, %3, 0;\n\t"
                 "@p st.global.cs.v2.b32 [%0], {%1, %2}; }" ::"l"(p), "r"(v.x), "r"(v.y),
                 "r"((int)on)
                 : "memory");
}

template <int DT, bool VEC>
__device__ __forceinline__ void store8(typename Storage<DT>::T* p, int lane, int left,
                                       const Lane8& f) {
    using T = typename Storage<DT>::T;
    if constexpr (VEC) {
        const bool on = lane * kEl < left;
        uint4* q = reinterpret_cast<uint4*>(p + lane * kEl);
        if constexpr (DT == kF32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                store16_if(q + i,
                           make_uint4(__float_as_uint(f[2 * i].x), __float_as_uint(f[2 * i].y),
                                      __float_as_uint(f[2 * i + 1].x), __float_as_uint(f[2 * i + 1].y)),
                           on);
        } else {
            store16_if(q, make_uint4(pack2<DT>(f[0]), pack2<DT>(f[1]), pack2<DT>(f[2]), pack2<DT>(f[3])), on);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
            const int c = lane + 32 * j;
            if (c < left) Storage<DT>::store(reinterpret_cast<T*>(p) + c, el(f, j));
        }
    }
}

// Eight float32 parameters by column (gamma, beta, gate), `def` where p is
// null or past the row's end.
template <bool VEC>
__device__ __forceinline__ void load_param(const float* p, int64_t col0, int lane, int left,
                                           float def, Lane8& f) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) f[j] = both(def);
        return;
    }
    if (VEC && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const bool in = lane * kEl < left;
        const float4* q = reinterpret_cast<const float4*>(p + col0 + lane * kEl);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = in ? __ldg(q + i) : make_float4(def, def, def, def);
            f[2 * i] = make_float2(v.x, v.y);
            f[2 * i + 1] = make_float2(v.z, v.w);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
            const int c = seg_col<VEC>(lane, j);
            el(f, j) = c < left ? __ldg(p + col0 + c) : def;
        }
    }
}

// ------------------------------------------------------------- 8-bit values

template <int FMT> struct Q8;
template <> struct Q8<kE4M3> {
    static constexpr float kMax = 448.f;
    static __device__ __forceinline__ float2 times(float2 v, float by) { return mul2(v, both(by)); }
    static __device__ __forceinline__ uint32_t encode4(float2 a, float2 b) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(a, __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(b, __NV_SATFINITE, __NV_E4M3);
        return __byte_perm(lo, hi, 0x5410);
    }
    static __device__ __forceinline__ void decode4(uint32_t w, float2* f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2_raw r =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
            f[i] = __half22float2(__half2(r));
        }
    }
};
template <> struct Q8<kInt8> {
    static constexpr float kMax = 127.f;
    // One value at a time: mul2 and the addition below would be made one fused
    // operation, which rounds once where the format says twice.
    static __device__ __forceinline__ float2 times(float2 v, float by) {
        return make_float2(__fmul_rn(v.x, by), __fmul_rn(v.y, by));
    }
    // |v| <= 127: adding 1.5 * 2^23 leaves round-to-nearest-even(v) in the low
    // byte (two's complement).
    static __device__ __forceinline__ uint32_t encode4(float2 a, float2 b) {
        a = add2(a, both(12582912.f));
        b = add2(b, both(12582912.f));
        const uint32_t lo = __byte_perm(__float_as_uint(a.x), __float_as_uint(a.y), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(b.x), __float_as_uint(b.y), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
    // The byte, its sign bit flipped, below 2^23: (2^23 + byte + 128) - (2^23 + 128).
    static __device__ __forceinline__ void decode4(uint32_t w, float2* f) {
        w ^= 0x80808080u;
        const float2 base = both(-8388736.f);
        f[0] = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7440)),
                                __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7441))), base);
        f[1] = add2(make_float2(__uint_as_float(__byte_perm(w, 0x4b000000u, 0x7442)),
                                __uint_as_float(__byte_perm(w, 0x4b000000u, 0x7443))), base);
    }
};

// A lane's eight codes.
template <bool VEC>
struct Codes {
    uint2 v;
    __device__ __forceinline__ void load(const uint8_t* p, int lane, int left) {
        if (VEC) {
            v = lane * kEl < left ? __ldcs(reinterpret_cast<const uint2*>(p + lane * kEl))
                                  : make_uint2(0, 0);
        } else {
            uint32_t w[2] = {0, 0};
#pragma unroll
            for (int j = 0; j < kEl; ++j) {
                const int c = lane + 32 * j;
                if (c < left) w[j / 4] |= (uint32_t)p[c] << (8 * (j % 4));
            }
            v = make_uint2(w[0], w[1]);
        }
    }
    __device__ __forceinline__ void store(uint8_t* p, int lane, int left) const {
        if (VEC) {
            store8_if(p + lane * kEl, v, lane * kEl < left);
        } else {
            const uint32_t w[2] = {v.x, v.y};
#pragma unroll
            for (int j = 0; j < kEl; ++j) {
                const int c = lane + 32 * j;
                if (c < left) p[c] = (uint8_t)(w[j / 4] >> (8 * (j % 4)));
            }
        }
    }
    // scale[0], scale[1]: those of elements 0-3 and 4-7.
    template <int FMT>
    __device__ __forceinline__ void get(const float (&scale)[2], Lane8& f) const {
        Q8<FMT>::decode4(v.x, f);
        Q8<FMT>::decode4(v.y, f + 2);
#pragma unroll
        for (int j = 0; j < kEl / 2; ++j) f[j] = mul2(f[j], both(scale[j / 2]));
    }
};

// A lane's two scales of the segment whose first one is at `s`.
template <bool VEC>
__device__ __forceinline__ void load_scales(const float* s, int lane, int left,
                                            float (&scale)[2]) {
    if (VEC) {
        scale[0] = scale[1] = lane * kEl < left ? __ldg(s + (lane >> 4)) : 0.f;
    } else {
        scale[0] = left > 0 ? __ldg(s) : 0.f;
        scale[1] = left > kQGroup ? __ldg(s + 1) : 0.f;
    }
}

// Scale and multiplier of a group from the bits of its largest magnitude
// (as unsigned integers magnitudes keep their order; infinities and NaN come
// out above every finite value).
template <int FMT>
__device__ __forceinline__ void group_scale(uint32_t bits, float& scale, float& by) {
    const float amax = __uint_as_float(bits);
    scale = amax * (1.f / Q8<FMT>::kMax);
    by = __fdiv_rn(Q8<FMT>::kMax, amax);
    if (amax < 7.7037197775489434e-34f) scale = by = 0.f;   // 2^-110
    if (bits >= 0x7f800000u) {
        scale = __uint_as_float(0x7fffffffu);
        by = 0.f;
    }
}

// max(|a|, |b|, |c|), NaN if one is.
__device__ __forceinline__ float amax3(float a, float b, float c) {
    float y;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
    return y;
}

// A lane's own largest magnitude of eight floats, as bits.
__device__ __forceinline__ uint32_t own_amax(const Lane8& f) {
    return __float_as_uint(amax3(amax3(f[0].x, f[0].y, f[1].x), amax3(f[1].y, f[2].x, f[2].y),
                                 amax3(f[3].x, f[3].y, 0.f)));
}

// The same (VEC) from elements as they were loaded: as fp32 bits for fp32, as
// the 16 bits of the storage type otherwise.
template <int DT>
__device__ __forceinline__ uint32_t raw_amax(const Raw<DT, true>& r) {
    if constexpr (DT == kF32) {
        Lane8 f;
        r.get(f);
        return own_amax(f);
    } else {
        constexpr uint32_t k = 0x7fff7fffu;
        const uint32_t a = __vmaxu2(__vimax3_u16x2(r.v[0].x & k, r.v[0].y & k, r.v[0].z & k),
                                    r.v[0].w & k);
        return max(a & 0xffffu, a >> 16);
    }
}
template <int DT>
__device__ __forceinline__ uint32_t amax_bits(uint32_t m) {   // of raw_amax: as fp32 bits
    if (DT == kF32) return m;
    if (DT == kBF16) return m << 16;
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}

// N = 2 or 4 groups at once (VEC): m[i] is the lane's own largest magnitude
// in group i of its half-warp.  The sixteen lanes halve the number of groups
// that each carries while they reduce, so that four reductions cost five
// exchanges in place of sixteen, and the N divisions are one.  Returns every
// group's multiplier and the scale of the group that this lane carries,
// group_carried<N>.
template <int FMT, int DT, int N>
__device__ __forceinline__ float group_scales(const uint32_t (&m)[N], int lane, float (&by)[N]) {
    const bool hi = lane & 8, odd = lane & 4;
    uint32_t a;
    if constexpr (N == 4) {
        a = hi ? m[2] : m[0];
        uint32_t b = hi ? m[3] : m[1];
        a = max(a, __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[2], 8));
        b = max(b, __shfl_xor_sync(0xffffffffu, hi ? m[1] : m[3], 8));
        const uint32_t give = odd ? a : b;
        a = max(odd ? b : a, __shfl_xor_sync(0xffffffffu, give, 4));
    } else {
        a = max(hi ? m[1] : m[0], __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[1], 8));
        a = max(a, __shfl_xor_sync(0xffffffffu, a, 4));
    }
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    float scale, mine;
    group_scale<FMT>(amax_bits<DT>(a), scale, mine);
#pragma unroll
    for (int i = 0; i < N; ++i)
        by[i] = __shfl_sync(0xffffffffu, mine, (lane & 16) | i * (16 / N));
    return scale;
}
// Which of the N groups a lane carries, and whether it is the one to write it.
template <int N>
__device__ __forceinline__ int group_carried(int lane) {
    return N == 4 ? (lane >> 2) & 3 : (lane >> 3) & 1;
}
template <int N>
__device__ __forceinline__ bool group_writer(int lane) {
    return (lane & (16 / N - 1)) == 0;
}

// A lane's eight codes with their group's multiplier.
template <int FMT>
__device__ __forceinline__ void encode8(const Lane8& f, float by, uint8_t* q, int lane, int left) {
    Codes<true> c;
    c.v = make_uint2(Q8<FMT>::encode4(Q8<FMT>::times(f[0], by), Q8<FMT>::times(f[1], by)),
                     Q8<FMT>::encode4(Q8<FMT>::times(f[2], by), Q8<FMT>::times(f[3], by)));
    c.store(q, lane, left);
}

// Quantises a segment element by element (not VEC) and writes its codes (at q)
// and scales (at s, the segment's first).  All lanes of the warp call it, with
// zeros past the row's end.
template <int FMT>
__device__ __forceinline__ void quantise_any(const Lane8& f, uint8_t* q, float* s, int lane,
                                             int left) {
    float scale[2], by[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const float a = amax3(amax3(f[2 * i].x, f[2 * i].y, f[2 * i + 1].x), f[2 * i + 1].y, 0.f);
        group_scale<FMT>(__reduce_max_sync(0xffffffffu, __float_as_uint(a)), scale[i], by[i]);
    }
    if (lane == 0) {
        s[0] = scale[0];
        if (left > kQGroup) s[1] = scale[1];
    }
    Codes<false> c;
    c.v = make_uint2(Q8<FMT>::encode4(Q8<FMT>::times(f[0], by[0]), Q8<FMT>::times(f[1], by[0])),
                     Q8<FMT>::encode4(Q8<FMT>::times(f[2], by[1]), Q8<FMT>::times(f[3], by[1])));
    c.store(q, lane, left);
}

// Quantises a warp's V adjacent segments of a row, the first starting at
// column c0, into the row's codes q and scales s.
template <int FMT, bool VEC, int V>
__device__ __forceinline__ void quantise_row(const Lane8 (&f)[V], uint8_t* q, float* s, int c0,
                                             int cols, int lane) {
    if constexpr (VEC) {
        uint32_t m[V];
        float by[V];
#pragma unroll
        for (int k = 0; k < V; ++k) m[k] = own_amax(f[k]);
        const float scale = group_scales<FMT, kF32, V>(m, lane, by);
        const int g = c0 / kQGroup + 2 * group_carried<V>(lane) + (lane >> 4);
        if (group_writer<V>(lane) && g * kQGroup < cols) s[g] = scale;
#pragma unroll
        for (int k = 0; k < V; ++k) encode8<FMT>(f[k], by[k], q + c0 + k * kSeg, lane, cols - c0 - k * kSeg);
    } else {
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const int c = c0 + k * kSeg;
            if (cols > c) quantise_any<FMT>(f[k], q + c, s + c / kQGroup, lane, cols - c);
        }
    }
}

// ---------------------------------------------------------- sums over a row

// The warps of one row: `n` of them, this one being `w`.  Up to eight are in
// one block, which then may hold several rows (this warp's is the block's y-th
// of `rows`) with a named barrier each; where a row needs more, a cluster of
// blocks shares it (CLUSTER), every warp's partial sums go to all of its
// blocks' shared memory, and the cluster's barrier takes the named one's
// place.  A sum's partials alternate between the two halves of `red`, so one
// barrier a sum is enough: a half is written again only after the next sum's
// barrier, which every warp passes after reading it.  The order of the
// additions is fixed.
constexpr int kRowWarps = 8;                       // of one block
constexpr int kMaxCluster = 8;
constexpr int kRedFloats = 2 * 2 * kRowWarps * kMaxCluster;   // `red` of a block

__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t cluster_size() {
    uint32_t r;
    asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\t"
                 "barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// *p (in this block's shared memory) of block `rank` = v.
__device__ __forceinline__ void store_in_block(float* p, uint32_t rank, float v) {
    asm volatile("{ .reg .b32 a; mapa.shared::cluster.u32 a, %0, %1;\n\t"
                 "st.shared::cluster.f32 [a], %2; }" ::"r"((uint32_t)__cvta_generic_to_shared(p)),
                 "r"(rank), "f"(v)
                 : "memory");
}

template <bool CLUSTER>
struct RowWarps {
    int n, w, lane, y, rows, block;   // block: which of the grid's blocks or clusters
    float* red;
    int half;
    // warps: those of a row in one block.  `all`: kRedFloats floats.
    __device__ __forceinline__ RowWarps(int warps, float* all) {
        const int warp = threadIdx.x >> 5;
        lane = threadIdx.x & 31;
        rows = (blockDim.x >> 5) / warps;
        y = warp / warps;
        w = warp - y * warps;
        n = warps;
        block = blockIdx.x;
        half = 0;
        if (CLUSTER) {
            w += cluster_rank() * warps;
            n *= cluster_size();
            block /= cluster_size();
        }
        red = all + y * (4 * kRowWarps);
        for (int i = threadIdx.x; i < kRedFloats; i += blockDim.x) all[i] = 0.f;
        if (CLUSTER) cluster_barrier();
        else __syncthreads();
    }
    // The last thing that a block does: the others may still write to it.
    __device__ __forceinline__ void end() const {
        if (CLUSTER) cluster_barrier();
    }
    static constexpr int kMost = CLUSTER ? kRowWarps * kMaxCluster : kRowWarps;
    // Puts every warp's v[i] at the returned r[i * kMost + warp].
    template <int N>
    __device__ __forceinline__ const float* exchange(const float (&v)[N]) {
        float* r = red + half * (2 * kMost);
        half ^= 1;
        if (CLUSTER) {
            if (lane < cluster_size())
#pragma unroll
                for (int i = 0; i < N; ++i) store_in_block(r + i * kMost + w, lane, v[i]);
            cluster_barrier();
        } else {
            if (lane == 0)
#pragma unroll
                for (int i = 0; i < N; ++i) r[i * kMost + w] = v[i];
            asm volatile("bar.sync %0, %1;" ::"r"(1 + y), "r"(n * 32) : "memory");
        }
        return r;
    }
    template <int N>
    __device__ __forceinline__ void sum(float (&v)[N]) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
#pragma unroll
            for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        if (!CLUSTER && n == 1) return;
        const float* r = exchange(v);
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float4* q = reinterpret_cast<const float4*>(r + i * kMost);
            float4 t = q[0];
            auto add = [&](const float4& a) {
                t.x += a.x;
                t.y += a.y;
                t.z += a.z;
                t.w += a.w;
            };
            if (CLUSTER)
                for (int k = 1; k * 4 < n; ++k) add(q[k]);
            else
#pragma unroll
                for (int k = 1; k * 4 < kMost; ++k) add(q[k]);
            v[i] = (t.x + t.y) + (t.z + t.w);
        }
    }
    __device__ __forceinline__ float warp_total(float2 a) const {
        float v = a.x + a.y;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        return v;
    }
    // From every warp's mean and sum of squares about it, of its EACH columns
    // (fewer at the row's end): the row's.
    template <int EACH>
    __device__ __forceinline__ void merge(float& mean, float& square, int cols, float inv_n) {
        if (!CLUSTER && n == 1) return;
        const float v[2] = {mean, square};
        const float* r = exchange(v);
        // a lane takes a warp of the row (of a cluster, two), eight lanes all
        // of a block's eight
        constexpr int kLanes = CLUSTER ? 32 : kRowWarps, kEach = CLUSTER ? kMost / 32 : 1;
        auto total = [&](float t) {
#pragma unroll
            for (int o = kLanes / 2; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            return t;
        };
        float m[kEach], count[kEach], t = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            const int k = lane % kLanes + i * kLanes;
            count[i] = (float)max(0, min(EACH, cols - k * EACH));
            m[i] = r[k];
            t = fmaf(count[i], m[i], t);
        }
        mean = total(t) * inv_n;
        t = 0.f;
#pragma unroll
        for (int i = 0; i < kEach; ++i) {
            // (a warp without columns adds nothing, even where mean^2 overflows)
            const float d = count[i] > 0.f ? m[i] - mean : 0.f;
            t += fmaf(d * d, count[i], r[kMost + lane % kLanes + i * kLanes]);
        }
        square = total(t);
    }
    __device__ __forceinline__ float sum(float2 a) {
        float v[1] = {a.x + a.y};
        sum(v);
        return v[0];
    }
    __device__ __forceinline__ float2 sum(float2 a, float2 b) {
        float v[2] = {a.x + a.y, b.x + b.y};
        sum(v);
        return make_float2(v[0], v[1]);
    }
};

// ------------------------------------------- a thread's own asynchronous ring
// Rows ahead of the one being worked on are copied into shared memory by the
// very thread that will read them (cp.async), so that a ring needs neither
// barriers nor flags between threads: a thread waits for its own copies only.

// (where `on`; the predicate in the instruction keeps branches out of the loops)
template <int BYTES>
__device__ __forceinline__ void copy_async(void* dst, const void* src, bool on) {
    const uint32_t d = (uint32_t)__cvta_generic_to_shared(dst);
    if constexpr (BYTES == 16)
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %2, 0;\n\t"
                     "@p cp.async.cg.shared.global [%0], [%1], 16; }" ::"r"(d), "l"(src), "r"((int)on)
                     : "memory");
    else
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %2, 0;\n\t"
                     "@p cp.async.ca.shared.global [%0], [%1], %3; }" ::"r"(d), "l"(src),
                     "r"((int)on), "n"(BYTES)
                     : "memory");
}
__device__ __forceinline__ void copies_end() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most N of the groups that copies_end() closed are still on the way.
template <int N>
__device__ __forceinline__ void copies_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// --------------------------------------------------- a warp's own ring (not VEC)
// Rows of any width begin on any element, which no asynchronous copy can read.
// So a warp copies the whole 16-byte words that a segment touches, and its
// lanes pick their elements from shared memory.  The tensor itself has to
// begin on a 16-byte boundary, and the last word is cut at its end, so nothing
// outside of it is read.  (What a word holds of the neighbouring rows is not
// looked at.)  The warp synchronises between its lanes' copies and reads.

template <int ES>
constexpr int kSegBytes = kSeg * ES + 16;

// at: the segment's first element; left: columns from there; total: the
// tensor's elements.
template <int ES>
__device__ __forceinline__ void copy_segment(char* dst, const void* base, int64_t at, int left,
                                             int64_t total, int lane) {
    const int64_t from = at * ES & ~(int64_t)15;
    const int words = (int)((at * ES & 15) + min(left, kSeg) * ES + 15) >> 4;
    const int64_t end = total * ES - from;   // bytes of the tensor from the first word on
#pragma unroll
    for (int i = 0; i < (kSegBytes<ES> + 511) / 512; ++i) {
        const int w = lane + 32 * i;
        const int bytes = (int)min((int64_t)16, end - w * 16);
        const bool on = left > 0 && w < words;
        asm volatile("{ .reg .pred p; setp.ne.b32 p, %3, 0;\n\t"
                     "@p cp.async.cg.shared.global [%0], [%1], 16, %2; }" ::"r"(
                         (uint32_t)__cvta_generic_to_shared(dst + w * 16)),
                     "l"(static_cast<const char*>(base) + from + w * 16), "r"(bytes), "r"((int)on)
                     : "memory");
    }
}

// The lane's eight elements (zero past the row's end).
template <int DT>
__device__ __forceinline__ void read_segment(const char* src, int64_t at, int left, int lane, Lane8& f) {
    using T = typename Storage<DT>::T;
    const T* p = reinterpret_cast<const T*>(src + (at * (int64_t)sizeof(T) & 15)) + lane;
#pragma unroll
    for (int j = 0; j < kEl; ++j) el(f, j) = lane + 32 * j < left ? Storage<DT>::load(p + 32 * j) : 0.f;
}
__device__ __forceinline__ Codes<false> read_codes(const char* src, int64_t at, int lane) {
    const uint8_t* p = reinterpret_cast<const uint8_t*>(src + (at & 15)) + lane;
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i)
        w[i] = __byte_perm(__byte_perm(p[128 * i], p[128 * i + 32], 0x0040),
                           __byte_perm(p[128 * i + 64], p[128 * i + 96], 0x0040), 0x5410);
    Codes<false> c;
    c.v = make_uint2(w[0], w[1]);
    return c;
}

// Host: how a row of `cols` columns is shared, V segments a warp: blocks of a
// cluster, warps a block, and rows a block (of at least `threads` threads).
struct RowShape {
    int cluster, warps, rows;
    template <int V>
    static RowShape of(int cols, int threads, int most_warps) {
        const int all = (cols + V * kSeg - 1) / (V * kSeg);
        RowShape s;
        s.cluster = 1;
        while (s.cluster * most_warps < all) s.cluster *= 2;
        s.warps = (all + s.cluster - 1) / s.cluster;
        s.rows = s.cluster > 1 || s.warps * 32 >= threads ? 1 : threads / 32 / s.warps;
        return s;
    }
    int threads() const { return 32 * warps * rows; }
};

constexpr size_t kFreeShared = 46 * 1024;    // a block's dynamic shared memory without asking
constexpr size_t kSharedAnSm = 227 * 1024;   // an SM's shared memory for blocks

// Blocks an SM that a kernel with __launch_bounds__(256, `least`) may count on
// (whole blocks of what its registers are bounded for: one of five to seven
// warps counts as one of eight).
inline int blocks_an_sm(int least, int threads, size_t smem) {
    const int by_registers = least * 256 / threads;
    const int by_shared = (int)(kSharedAnSm / (smem + kRedFloats * sizeof(float) + 1024));
    const int n = by_registers < by_shared ? by_registers : by_shared;
    return n < 1 ? 1 : n;
}

// Launches `blocks` clusters of s.cluster blocks.  A kernel serves many widths
// with as many amounts of shared memory, from several host threads: its limit
// is raised once on each device, to all that a block may have, and never
// lowered (a call that set its own amount could fail another thread's launch).
template <auto KERNEL, class Args>
inline cudaError_t launch_rows(const RowShape& s, int64_t blocks, size_t smem, cudaStream_t stream,
                               const Args& args) {
    if (smem > kFreeShared) {
        static std::atomic<uint64_t> raised{0};   // a bit a device
        int dev = 0, most = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const uint64_t bit = dev < 64 ? 1ull << dev : 0;
        if (!(raised.load(std::memory_order_acquire) & bit)) {
            e = cudaDeviceGetAttribute(&most, cudaDevAttrMaxSharedMemoryPerBlockOptin, dev);
            if (e != cudaSuccess) return e;
            e = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                     most - (int)(kRedFloats * sizeof(float)));
            if (e != cudaSuccess) return e;
            raised.fetch_or(bit, std::memory_order_release);
        }
    }
    cudaLaunchConfig_t c = {};
    c.gridDim = dim3((unsigned)(blocks * s.cluster));
    c.blockDim = dim3((unsigned)s.threads());
    c.dynamicSmemBytes = smem;
    c.stream = stream;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)s.cluster;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    c.attrs = at;
    c.numAttrs = s.cluster > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&c, KERNEL, args, s.warps);
}

// Host: whether a pointer is on a 16-byte boundary (null is).
inline bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace iabn
