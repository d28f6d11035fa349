// iabn_rows.cuh -- device-side building blocks of the row operators
// (iabn_block.h): how a warp's lanes share a row, loads and stores of the
// storage types and of 8-bit codes, the 8-bit quantiser and sums over a row.
//
// A warp takes a segment of 256 columns of a row, eight a lane.  Two maps:
//   VEC   lane l holds columns 8l .. 8l+7: one 16-byte access (two for fp32)
//         and one 8-byte access of codes a lane.  Needs widths that are
//         multiples of 8 and 16-byte aligned rows.
//   else  lane l holds columns l, l+32, .., l+224: any width and alignment, a
//         warp's accesses still being consecutive elements.
// Either way a segment holds two checkpoint groups of 128 columns: lanes 0-15
// and 16-31 under VEC, elements 0-3 and 4-7 of every lane otherwise.
#pragma once

#include <cuda_fp8.h>

#include "iabn_block_internal.h"
#include "iabn_device.cuh"

namespace iabn {

constexpr int kSeg = 256;   // columns of a warp's segment
constexpr int kEl = 8;      // of them, a lane's

template <bool VEC>
__device__ __forceinline__ int seg_col(int lane, int j) {
    return VEC ? lane * kEl + j : lane + 32 * j;
}

__device__ __forceinline__ float2 unpack2(__nv_bfloat162 v) { return __bfloat1622float2(v); }
__device__ __forceinline__ float2 unpack2(__half2 v) { return __half22float2(v); }

template <class T2>
__device__ __forceinline__ T2 pack2(float a, float b);
template <>
__device__ __forceinline__ __nv_bfloat162 pack2<__nv_bfloat162>(float a, float b) {
    return __floats2bfloat162_rn(a, b);
}
template <>
__device__ __forceinline__ __half2 pack2<__half2>(float a, float b) {
    return __floats2half2_rn(a, b);
}
template <int DT> struct Pair { using T = __nv_bfloat162; };
template <> struct Pair<kF16> { using T = __half2; };

// A lane's eight elements as they were loaded (a batch of loads is in flight
// before any is converted).
template <int DT, bool VEC>
struct Raw {
    using T = typename Storage<DT>::T;
    union {
        uint4 v[DT == kF32 ? 2 : 1];
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
            for (int i = 0; i < (DT == kF32 ? 2 : 1); ++i)
                v[i] = in ? ldg_cs(q + i) : make_uint4(0, 0, 0, 0);
        } else {
#pragma unroll
            for (int j = 0; j < kEl; ++j) {
                const int c = lane + 32 * j;
                e[j] = c < left ? p[c] : T(0.f);
            }
        }
    }
    __device__ __forceinline__ void get(float (&f)[kEl]) const {
        if constexpr (DT == kF32 || !VEC) {
#pragma unroll
            for (int j = 0; j < kEl; ++j) f[j] = Storage<DT>::load(&e[j]);
        } else {
            const uint32_t w[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 t = unpack2(*reinterpret_cast<const typename Pair<DT>::T*>(&w[j]));
                f[2 * j] = t.x;
                f[2 * j + 1] = t.y;
            }
        }
    }
};

template <int DT, bool VEC>
__device__ __forceinline__ void store8(typename Storage<DT>::T* p, int lane, int left,
                                       const float (&f)[kEl]) {
    using T = typename Storage<DT>::T;
    if constexpr (VEC) {
        if (lane * kEl >= left) return;
        uint4* q = reinterpret_cast<uint4*>(p + lane * kEl);
        if constexpr (DT == kF32) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
                __stcs(q + i, make_uint4(__float_as_uint(f[4 * i]), __float_as_uint(f[4 * i + 1]),
                                         __float_as_uint(f[4 * i + 2]),
                                         __float_as_uint(f[4 * i + 3])));
        } else {
            using P = typename Pair<DT>::T;
            uint32_t w[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const P t = pack2<P>(f[2 * j], f[2 * j + 1]);
                w[j] = *reinterpret_cast<const uint32_t*>(&t);
            }
            __stcs(q, make_uint4(w[0], w[1], w[2], w[3]));
        }
    } else {
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
            const int c = lane + 32 * j;
            if (c < left) Storage<DT>::store(reinterpret_cast<T*>(p) + c, f[j]);
        }
    }
}

// Eight float32 parameters by column (gamma, beta, gate), `def` where p is
// null or past the row's end.  Read again for every row: they stay in cache.
template <bool VEC>
__device__ __forceinline__ void load_param(const float* p, int64_t col0, int lane, int left,
                                           float def, float (&f)[kEl]) {
    if (!p) {
#pragma unroll
        for (int j = 0; j < kEl; ++j) f[j] = def;
        return;
    }
    if (VEC && (reinterpret_cast<uintptr_t>(p) & 15) == 0) {
        const bool in = lane * kEl < left;
        const float4* q = reinterpret_cast<const float4*>(p + col0 + lane * kEl);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float4 v = in ? __ldg(q + i) : make_float4(def, def, def, def);
            f[4 * i] = v.x;
            f[4 * i + 1] = v.y;
            f[4 * i + 2] = v.z;
            f[4 * i + 3] = v.w;
        }
    } else {
#pragma unroll
        for (int j = 0; j < kEl; ++j) {
            const int c = seg_col<VEC>(lane, j);
            f[j] = c < left ? __ldg(p + col0 + c) : def;
        }
    }
}

// ------------------------------------------------------------- 8-bit values

template <int FMT> struct Q8;
template <> struct Q8<kE4M3> {
    static constexpr float kMax = 448.f;
    static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | hi << 16;
    }
    static __device__ __forceinline__ void decode4(uint32_t w, float* f) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const __half2_raw r =
                __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w >> (16 * i)), __NV_E4M3);
            const float2 t = __half22float2(__half2(r));
            f[2 * i] = t.x;
            f[2 * i + 1] = t.y;
        }
    }
};
template <> struct Q8<kInt8> {
    static constexpr float kMax = 127.f;
    // |v| <= 127: adding 1.5 * 2^23 leaves round-to-nearest-even(v) in the low
    // byte (two's complement).
    static __device__ __forceinline__ uint32_t round1(float v) {
        return __float_as_uint(__fadd_rn(v, 12582912.f));
    }
    static __device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d) {
        const uint32_t lo = __byte_perm(round1(a), round1(b), 0x0040);
        const uint32_t hi = __byte_perm(round1(c), round1(d), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
    static __device__ __forceinline__ void decode4(uint32_t w, float* f) {
#pragma unroll
        for (int i = 0; i < 4; ++i) f[i] = (float)(int8_t)(w >> (8 * i));
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
            if (lane * kEl < left) __stcs(reinterpret_cast<uint2*>(p + lane * kEl), v);
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
    __device__ __forceinline__ void get(const float (&scale)[2], float (&f)[kEl]) const {
        Q8<FMT>::decode4(v.x, f);
        Q8<FMT>::decode4(v.y, f + 4);
#pragma unroll
        for (int j = 0; j < kEl; ++j) f[j] *= scale[j / 4];
    }
    __device__ __forceinline__ void get(int fmt, const float (&scale)[2], float (&f)[kEl]) const {
        if (fmt == kE4M3) get<kE4M3>(scale, f);
        else get<kInt8>(scale, f);
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

// The largest magnitude, as bits, of the groups that a lane's elements are in:
// m[0] under VEC (the lane's group), else m[0] and m[1] (of elements 0-3 and
// 4-7).  All lanes of the warp call it.
template <bool VEC>
__device__ __forceinline__ void group_amax(const float (&f)[kEl], uint32_t (&m)[2]) {
    m[0] = m[1] = 0;
#pragma unroll
    for (int j = 0; j < kEl; ++j)
        m[j / 4] = max(m[j / 4], __float_as_uint(f[j]) & 0x7fffffffu);
    if (VEC) {
        m[0] = max(m[0], m[1]);
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) m[0] = max(m[0], __shfl_xor_sync(0xffffffffu, m[0], o));
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) m[i] = __reduce_max_sync(0xffffffffu, m[i]);
    }
}

// A lane's own largest magnitude (VEC), as fp32 bits for fp32 and as the 16
// bits of the storage type otherwise, from elements as they were loaded.
template <int DT>
__device__ __forceinline__ uint32_t raw_amax(const Raw<DT, true>& r) {
    if constexpr (DT == kF32) {
        uint32_t a = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = r.v[i];
            a = max(max(a, max(v.x & 0x7fffffffu, v.y & 0x7fffffffu)),
                    max(v.z & 0x7fffffffu, v.w & 0x7fffffffu));
        }
        return a;
    } else {
        constexpr uint32_t k = 0x7fff7fffu;
        const uint32_t a = __vmaxu2(__vmaxu2(r.v[0].x & k, r.v[0].y & k),
                                    __vmaxu2(r.v[0].z & k, r.v[0].w & k));
        return max(a & 0xffffu, a >> 16);
    }
}
template <int DT>
__device__ __forceinline__ uint32_t amax_bits(uint32_t m) {   // of raw_amax: as fp32 bits
    if (DT == kF32) return m;
    if (DT == kBF16) return m << 16;
    return __float_as_uint(__half2float(__ushort_as_half((unsigned short)m)));
}

// Four groups at once (VEC): m[i] is the lane's own largest magnitude in group
// i of its half-warp.  The sixteen lanes halve the number of groups that each
// carries while they reduce, so that four reductions cost five exchanges, and
// the four divisions one.  Writes the scales (at s[i], of the segment, where
// on[i]) and returns every group's multiplier.
template <int FMT, int DT>
__device__ __forceinline__ void four_scales(const uint32_t (&m)[4], float* const (&s)[4],
                                            const bool (&on)[4], int lane, int left,
                                            float (&by)[4]) {
    const bool hi = lane & 8, odd = lane & 4;
    uint32_t a = hi ? m[2] : m[0], b = hi ? m[3] : m[1];
    a = max(a, __shfl_xor_sync(0xffffffffu, hi ? m[0] : m[2], 8));
    b = max(b, __shfl_xor_sync(0xffffffffu, hi ? m[1] : m[3], 8));
    const uint32_t give = odd ? a : b;
    a = max(odd ? b : a, __shfl_xor_sync(0xffffffffu, give, 4));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 2));
    a = max(a, __shfl_xor_sync(0xffffffffu, a, 1));
    float scale, mine;
    group_scale<FMT>(amax_bits<DT>(a), scale, mine);
    float* p = hi ? (odd ? s[3] : s[2]) : (odd ? s[1] : s[0]);
    const bool w = hi ? (odd ? on[3] : on[2]) : (odd ? on[1] : on[0]);
    if ((lane & 3) == 0 && w && (lane & 16) * kEl < left) p[lane >> 4] = scale;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        by[i] = __shfl_sync(0xffffffffu, mine, (lane & 16) | i << 2);
}

// A lane's eight codes with their group's multiplier.
template <int FMT>
__device__ __forceinline__ void encode8(const float (&f)[kEl], float by, uint8_t* q, int lane,
                                        int left) {
    float t[kEl];
#pragma unroll
    for (int j = 0; j < kEl; ++j) t[j] = __fmul_rn(f[j], by);
    Codes<true> c;
    c.v = make_uint2(Q8<FMT>::encode4(t[0], t[1], t[2], t[3]),
                     Q8<FMT>::encode4(t[4], t[5], t[6], t[7]));
    c.store(q, lane, left);
}

// Quantises a segment with its group_amax and writes its codes (at `q`) and
// scales (at `s`, the segment's first).  Past the row's end f is zero.
template <int FMT, bool VEC>
__device__ __forceinline__ void quantise8(const float (&f)[kEl], const uint32_t (&m)[2],
                                          uint8_t* q, float* s, int lane, int left) {
    float scale[2], by[2];
    group_scale<FMT>(m[0], scale[0], by[0]);
    if (VEC) {
        by[1] = by[0];
        if ((lane & 15) == 0 && lane * kEl < left) s[lane >> 4] = scale[0];
    } else {
        group_scale<FMT>(m[1], scale[1], by[1]);
        if (lane == 0) {
            s[0] = scale[0];
            if (left > kQGroup) s[1] = scale[1];
        }
    }
    float t[kEl];
#pragma unroll
    for (int j = 0; j < kEl; ++j) t[j] = __fmul_rn(f[j], by[j / 4]);
    Codes<VEC> c;
    c.v = make_uint2(Q8<FMT>::encode4(t[0], t[1], t[2], t[3]),
                     Q8<FMT>::encode4(t[4], t[5], t[6], t[7]));
    c.store(q, lane, left);
}

template <bool VEC>
__device__ __forceinline__ void quantise8(int fmt, const float (&f)[kEl], const uint32_t (&m)[2],
                                          uint8_t* q, float* s, int lane, int left) {
    if (fmt == kE4M3) quantise8<kE4M3, VEC>(f, m, q, s, lane, left);
    else quantise8<kInt8, VEC>(f, m, q, s, lane, left);
}

// ---------------------------------------------------------- sums over a row

// The warps of one row: `n` of them, this one being `w`; `bar` their named
// barrier, `red` 2 x n float2 of shared memory.  A sum's partials alternate
// between the two halves of `red`, so one barrier a sum is enough: a half is
// written again only after the next sum's barrier, which every warp passes
// after reading it.
struct RowWarps {
    int n, w, lane, bar;
    float2* red;
    int half;
    __device__ __forceinline__ float2 sum(float a, float b) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a += __shfl_xor_sync(0xffffffffu, a, o);
            b += __shfl_xor_sync(0xffffffffu, b, o);
        }
        if (n == 1) return make_float2(a, b);
        float2* r = red + half * n;
        half ^= 1;
        if (lane == 0) r[w] = make_float2(a, b);
        asm volatile("bar.sync %0, %1;" ::"r"(bar), "r"(n * 32) : "memory");
        float2 t = lane < n ? r[lane] : make_float2(0.f, 0.f);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            t.x += __shfl_xor_sync(0xffffffffu, t.x, o);
            t.y += __shfl_xor_sync(0xffffffffu, t.y, o);
        }
        return t;
    }
    __device__ __forceinline__ float sum(float a) { return sum(a, 0.f).x; }
};

// Host: whether a pointer is on a 16-byte boundary (null is).
inline bool on16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

}  // namespace iabn
