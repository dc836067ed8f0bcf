// gd_norm.h -- what the norms with an 8-bit output share: loads and stores of groups of
// elements, the row's sums, and the decision of codes and scales.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <type_traits>

#include "gd_quant.h"
#include "gd_types.h"

namespace gd {

// h = x + residual of P groups of four elements side by side, as stored; both terms are
// read before h is written, so h may overwrite either.
template <int P, typename T>
__device__ __forceinline__ void load_groups(const T *x, const T *res, int64_t e4, f32x4 *h) {
    typedef T Vec __attribute__((ext_vector_type(4 * P)));
    typedef float Wide __attribute__((ext_vector_type(4 * P)));
    Wide v = __builtin_convertvector(*reinterpret_cast<const Vec *>(x + 4 * e4), Wide);
    if (res) {
        v += __builtin_convertvector(*reinterpret_cast<const Vec *>(res + 4 * e4), Wide);
        v = __builtin_convertvector(__builtin_convertvector(v, Vec), Wide);
    }
#pragma unroll
    for (int i = 0; i < 4 * P; i++) h[i / 4][i % 4] = v[i];
}

template <int P, typename T>
__device__ __forceinline__ void store_groups(T *x, int64_t e4, const f32x4 *h) {
    typedef T Vec __attribute__((ext_vector_type(4 * P)));
    Vec v;
#pragma unroll
    for (int i = 0; i < 4 * P; i++) v[i] = static_cast<T>(h[i / 4][i % 4]);
    *reinterpret_cast<Vec *>(x + 4 * e4) = v;
}

__device__ __forceinline__ double square4(f32x4 h) {
    double s = 0.0;
#pragma unroll
    for (int j = 0; j < 4; j++) s = __builtin_fma(static_cast<double>(h[j]), static_cast<double>(h[j]), s);
    return s;
}

// Codes and scales are decided in f32 where that gives what the f64 rule gives, and
// as the rule is written in the rest. With P = f32(h w), A = max|P| (which is
// f32(max|h w|)) and I = f32(127 / A), the value t = P I is off the rule's by four
// roundings, 127 * 4 * 2^-24 = 3.1e-5 at most, so that the code is the rule's unless t
// lies within kTieGuard = 6.4e-5 of a half; the f32 scale A r is off by three, so that
// its f16 rounding is the rule's unless its 13 dropped bits lie within 4 steps of a
// half. Where any lane of a wave is in doubt (in about one wave of thirty, of f32
// values) the wave decides again in f64.
struct Products {
    f32x4 h, w;
    float p[4];
    __device__ __forceinline__ Products(f32x4 h_, f32x4 w_) : h(h_), w(w_) {
#pragma unroll
        for (int j = 0; j < 4; j++) p[j] = h[j] * w[j];
    }
    __device__ __forceinline__ float absmax() const { return absmax4(float4{p[0], p[1], p[2], p[3]}); }
    __device__ __forceinline__ double exact(int j) const { return static_cast<double>(h[j]) * static_cast<double>(w[j]); }
    __device__ __forceinline__ double exact_absmax() const {
        return fmax(fmax(fabs(exact(0)), fabs(exact(1))), fmax(fabs(exact(2)), fabs(exact(3))));
    }
    // Byte j: the code of element j, inv = 127 / absmax; doubt: whether one is.
    __device__ __forceinline__ uint32_t codes(float inv, bool &doubt) const {
        uint32_t packed = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const float t = p[j] * inv;
            packed |= (static_cast<uint32_t>(static_cast<int32_t>(floorf(t + 0.5f))) & 0xffu) << (8 * j);
            doubt |= !(fabsf(__builtin_amdgcn_fractf(t) - 0.5f) >= kTieGuard);
        }
        return packed;
    }
    __device__ __forceinline__ uint32_t exact_codes(double inv) const {
        uint32_t packed = 0;
#pragma unroll
        for (int j = 0; j < 4; j++) packed |= (static_cast<uint32_t>(round_code(exact(j) * inv)) & 0xffu) << (8 * j);
        return packed;
    }
};

// An f32 A whose reciprocal and products stay in f32's normal range: others are
// decided in f64.
__device__ __forceinline__ bool in_range(float a) { return a >= 1e-30f && a <= 1e30f; }

// f16 rounding of t, an f32 value up to 4 f32 steps off: whether it is in doubt.
__device__ __forceinline__ bool f16_doubt(float t) {
    const uint32_t dropped = __builtin_bit_cast(uint32_t, t) & 0x1fffu;
    return !(t >= 6.2e-5f && t <= 65000.0f) || (dropped >= 0x1000u - 4 && dropped <= 0x1000u + 4);   // normal in f16
}

__device__ __forceinline__ double max4d(double v) {   // max over the four lanes of a block
#pragma unroll
    for (int o = 2; o >= 1; o >>= 1) v = fmax(v, __shfl_xor(v, o));
    return v;
}

// 1 / sqrt(x), x > 0 finite, to f64's last bits: the hardware's estimate (some 24
// bits) and two Newton steps.
__device__ __forceinline__ double rsqrt_f64(double x) {
    double y = __builtin_amdgcn_rsq(x);
#pragma unroll
    for (int i = 0; i < 2; i++) y = y * __builtin_fma(-0.5 * x * y, y, 1.5);
    return y;
}

// v by an operation over a wave, in all its lanes, without LDS: with the lanes 32, 16, 8, 4, 2
// and 1 away in turn (8 and 4 by rotations of 16 lanes, which meet the same value there).
template <typename F>
__device__ __forceinline__ double over_wave(double v, F f) {
    typedef uint32_t Words __attribute__((ext_vector_type(2)));
    const auto joined = [](uint32_t lo, uint32_t hi) { return __builtin_bit_cast(double, Words{lo, hi}); };
    Words w = __builtin_bit_cast(Words, v);
    auto lo = __builtin_amdgcn_permlane32_swap(w[0], w[0], false, false), hi = __builtin_amdgcn_permlane32_swap(w[1], w[1], false, false);
    v = f(joined(lo[0], hi[0]), joined(lo[1], hi[1]));
    w = __builtin_bit_cast(Words, v);
    lo = __builtin_amdgcn_permlane16_swap(w[0], w[0], false, false);
    hi = __builtin_amdgcn_permlane16_swap(w[1], w[1], false, false);
    v = f(joined(lo[0], hi[0]), joined(lo[1], hi[1]));
    const auto with = [&](auto ctrl) {
        const Words u = __builtin_bit_cast(Words, v);
        constexpr int kCtrl = decltype(ctrl)::value;
        v = f(v, joined(static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u[0]), kCtrl, 0xF, 0xF, false)),
                        static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(u[1]), kCtrl, 0xF, 0xF, false))));
    };
    with(std::integral_constant<int, 0x128>{});   // row_ror:8
    with(std::integral_constant<int, 0x124>{});   // row_ror:4
    with(std::integral_constant<int, 0x4E>{});    // quad_perm [2,3,0,1]
    with(std::integral_constant<int, 0xB1>{});    // quad_perm [1,0,3,2]
    return v;
}

// Sum (and max) over a row's waves; every thread gets them.
template <int kWaves, bool kMax>
__device__ __forceinline__ void group_sum_max(double &sum, double &mx, double (*red)[2]) {
    sum = over_wave(sum, [](double a, double b) { return a + b; });
    if (kMax) mx = over_wave(mx, [](double a, double b) { return fmax(a, b); });
    if (kWaves == 1) return;
    if (threadIdx.x % 64 == 0) {
        red[threadIdx.x / 64][0] = sum;
        if (kMax) red[threadIdx.x / 64][1] = mx;
    }
    __syncthreads();
    sum = red[0][0];
    if (kMax) mx = red[0][1];
#pragma unroll
    for (int w = 1; w < kWaves; w++) {
        sum += red[w][0];
        if (kMax) mx = fmax(mx, red[w][1]);
    }
}

// Eight neighbouring products of each of four lanes (p0, p1: threadIdx.x % 4 in order) as a
// block's codes in bit planes: one word of each plane, at `o` and each `groups` words on.
// amax is the row's largest product, row_top its f32 rounding, row_inv 127 over that.
__device__ __forceinline__ void put_planes(const Products &p0, const Products &p1, const ByteTranspose &tr, double amax,
                                           float row_top, float row_inv, uint32_t *o, int64_t groups) {
    bool doubt = !in_range(row_top);
    uint32_t lo = p0.codes(row_inv, doubt), hi = p1.codes(row_inv, doubt);
    if (__any(doubt)) {
        const double factor = factor_of(amax);
        lo = p0.exact_codes(factor);
        hi = p1.exact_codes(factor);
    }
    lo = bits_to_nibbles(lo);
    hi = bits_to_nibbles(hi);
    // A byte of each plane: the even planes', the odd planes'.
    o += 2 * (threadIdx.x % 4) * groups;
    o[0] = tr((lo & 0x0F0F0F0Fu) | ((hi & 0x0F0F0F0Fu) << 4));
    o[groups] = tr(((lo >> 4) & 0x0F0F0F0Fu) | (hi & 0xF0F0F0F0u));
}

// Likewise as a q8_0 block (34 bytes = 17 halves) at o; rstd127 the row's factor over 127,
// r32 its f32 rounding.
__device__ __forceinline__ void put_block(const Products &p0, const Products &p1, double rstd127, float r32, uint16_t *o) {
    const int k4 = threadIdx.x % 4;
    const float a = max4(fmaxf(p0.absmax(), p1.absmax()));
    float d32 = a * r32;
    bool doubt = !in_range(a) || f16_doubt(d32);
    const float inv = a > 0.0f ? recip127(a) : 0.0f;
    uint32_t lo = p0.codes(inv, doubt), hi = p1.codes(inv, doubt);
    if (__any(doubt)) {
        const double exact = max4d(fmax(p0.exact_absmax(), p1.exact_absmax())), factor = factor_of(exact);
        lo = p0.exact_codes(factor);
        hi = p1.exact_codes(factor);
        d32 = exact > 0.0 ? static_cast<float>(exact * rstd127) : 0.0f;
    }
    typedef uint32_t Words __attribute__((ext_vector_type(2), aligned(2)));
    *reinterpret_cast<Words *>(o + 1 + 4 * k4) = Words{lo, hi};
    if (k4 == 0) o[0] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(d32));
}

}  // namespace gd
