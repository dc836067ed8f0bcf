// gd_quant.h -- device side of the activation quantization rule (absmax to
// int8, stated in include/gemm_decode.h under "Activation quantization"),
// as the norms with an 8-bit output and the 8-bit cache apply it: the factor
// is 127 * (1 / absmax), as torch evaluates `127 / tensor`, so that rows quantized by
// such code are reproduced bit for bit. (quantize.hip, for plain f32 activations, has it
// as 127 / absmax; the two lead to different codes only at exact halves. It has its own
// text: the HBM traffic the benchmark reports for it is tied to that file's bytes.)
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>

namespace gd {

__device__ __forceinline__ int32_t round_code(double v) {
    const double f = floor(v);
    double q = f + ((v - f) >= 0.5 ? 1.0 : 0.0);
    q = q > 127.0 ? 127.0 : q;
    q = q < -127.0 ? -127.0 : q;
    return static_cast<int32_t>(q);
}

__device__ __forceinline__ float absmax4(const float4 &v) {
    return fmaxf(fmaxf(fabsf(v.x), fabsf(v.y)), fmaxf(fabsf(v.z), fabsf(v.w)));
}

// What the rule multiplies by: 127 * (1 / absmax), each step rounded in f64
// (0 for a group of zeros).
__device__ __forceinline__ double factor_of(double absmax) { return absmax > 0.0 ? 127.0 * (1.0 / absmax) : 0.0; }

// ------------------------------------------------------ f32 decisions
// Codes are decided in f32 first: with inv32 = f32(127/absmax) and v32 = x *
// inv32 (two roundings), |v32 - v| <= 127 * 2^-23 ~ 1.5e-5 for the f64
// product v the rule rounds, so Math.round(v32) = Math.round(v) unless v32
// lies within kTieGuard of a half-integer; only those elements are decided
// again in f64 exactly as the rule states.
constexpr float kTieGuard = 6.4e-5f;   // 4x the f32 error bound above

// f32(127 / a) and f32(a / 127) for a finite f32 a > 0, correctly rounded
// f32 divisions. They equal the rule's f64 factor (two roundings) and quotient
// (one) rounded to f32: an f32 midpoint is never within 2^-49 (relative) of
// either exact quotient, beyond what f64 rounds off, so rounding again cannot
// differ.
__device__ __forceinline__ float recip127(float a) { return 127.0f / a; }
__device__ __forceinline__ float scale_of(float a) { return a / 127.0f; }

// Four codes, byte j of the result the code of element j. A code is
// floor(v32 + 0.5) for v32 = x * inv32: outside kTieGuard of a half-integer
// that is Math.round of the f64 product (v32 + 0.5 rounds by at most 2^-17
// for |v32| < 128, and |v32| <= 127 + 2^-16 keeps it in [-127, 127] without
// a clamp). A lane with any of its codes near a tie, or whose reciprocal
// overflowed f32 (f64_only), decides its four codes again in f64 exactly as
// the rule states.
__device__ __forceinline__ uint32_t codes4(const float4 &v, float inv32, float absmax, bool f64_only) {
    const float e[4] = {v.x, v.y, v.z, v.w};
    int32_t q[4];
    bool exact = f64_only;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float t = e[j] * inv32;
        q[j] = static_cast<int32_t>(floorf(t + 0.5f));
        exact |= fabsf(__builtin_amdgcn_fractf(t) - 0.5f) < kTieGuard;
    }
    if (exact) {   // rare
        const double inv = factor_of(static_cast<double>(absmax));
#pragma unroll
        for (int j = 0; j < 4; j++) q[j] = round_code(static_cast<double>(e[j]) * inv);
    }
    uint32_t packed = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) packed |= (static_cast<uint32_t>(q[j]) & 0xffu) << (8 * j);
    return packed;
}

// Max over the eight lanes that hold one 32-element block (three DPP steps).
__device__ __forceinline__ float max8(float v) {   // max over the 8 lanes of a half-row
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false)));
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false)));
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x141, 0xF, 0xF, false)));
    return v;
}

// The same over four lanes.
__device__ __forceinline__ float max4(float v) {
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0xB1, 0xF, 0xF, false)));
    return fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x4E, 0xF, 0xF, false)));
}

// ------------------------------------------------------ bit planes
__device__ __forceinline__ uint32_t bits_to_nibbles(uint32_t x) {   // bit 8j + b -> bit 4b + j
    uint32_t t;
    t = (x ^ (x >> 12)) & 0x0000F0F0u;
    x ^= t ^ (t << 12);
    t = (x ^ (x >> 6)) & 0x00CC00CCu;
    x ^= t ^ (t << 6);
    t = (x ^ (x >> 3)) & 0x0A0A0A0Au;
    x ^= t ^ (t << 3);
    t = (x ^ (x >> 1)) & 0x22222222u;
    x ^= t ^ (t << 1);
    return x;
}

__device__ __forceinline__ uint32_t nibbles_to_bits(uint32_t x) {   // bit 4b + j -> bit 8j + b: the steps back
    uint32_t t;
    t = (x ^ (x >> 1)) & 0x22222222u;
    x ^= t ^ (t << 1);
    t = (x ^ (x >> 3)) & 0x0A0A0A0Au;
    x ^= t ^ (t << 3);
    t = (x ^ (x >> 6)) & 0x00CC00CCu;
    x ^= t ^ (t << 6);
    t = (x ^ (x >> 12)) & 0x0000F0F0u;
    return x ^ t ^ (t << 12);
}

// One exchange step of the 8 x 8 nibble transpose: keep the nibbles whose
// slot bit t equals this lane's bit t, take the partner's others, moved by
// 2^t slots (a rotate by sh bits, sh per lane).
__device__ __forceinline__ uint32_t nibble_step(uint32_t x, uint32_t partner, uint32_t sh, uint32_t keep) {
    const uint32_t rot = __builtin_amdgcn_alignbit(partner, partner, sh);
    return (x & keep) | (rot & ~keep);
}

// The 8 x 8 nibble transpose among eight lanes (lane k8 of its group): three
// exchange steps with the lanes k8 ^ 1, k8 ^ 2 and k8 ^ 4, after which lane
// k8 holds slot k8's nibble of every lane.
struct NibbleTranspose {
    uint32_t sh[3], keep[3];   // the steps' per-lane rotates and keep masks
    __device__ __forceinline__ explicit NibbleTranspose(int k8) {
        constexpr uint32_t kLow[3] = {0x0F0F0F0Fu, 0x00FF00FFu, 0x0000FFFFu};   // slot bit t = 0
#pragma unroll
        for (int t = 0; t < 3; t++) {
            const bool hi = (k8 >> t) & 1;
            sh[t] = hi ? (4u << t) : 32u - (4u << t);
            keep[t] = hi ? ~kLow[t] : kLow[t];
        }
    }
    __device__ __forceinline__ uint32_t operator()(uint32_t w) const {
        int p = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), 0xB1, 0xF, 0xF, false);   // lane k ^ 1
        w = nibble_step(w, static_cast<uint32_t>(p), sh[0], keep[0]);
        p = __builtin_amdgcn_update_dpp(0, static_cast<int>(w), 0x4E, 0xF, 0xF, false);       // lane k ^ 2
        w = nibble_step(w, static_cast<uint32_t>(p), sh[1], keep[1]);
        p = __builtin_amdgcn_ds_swizzle(static_cast<int>(w), 0x101F);   // lane k ^ 4: xor mask 4, 32-lane groups
        return nibble_step(w, static_cast<uint32_t>(p), sh[2], keep[2]);
    }
};

// The 4 x 4 byte transpose among four lanes, its own inverse: lane k holds byte k of
// every lane. With a byte of each even plane in one word and of each odd one in another,
// lane k comes to hold the words of the planes 2 k and 2 k + 1.
struct ByteTranspose {
    uint32_t one, two;   // what the exchanges with the lanes k ^ 1 and k ^ 2 keep
    __device__ __forceinline__ explicit ByteTranspose(int k)
        : one(k % 2 ? 0x03070105u : 0x06020400u), two(k / 2 ? 0x03020706u : 0x05040100u) {}
    __device__ __forceinline__ uint32_t operator()(uint32_t x) const {
        uint32_t p = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0xB1, 0xF, 0xF, false));
        x = __builtin_amdgcn_perm(p, x, one);
        p = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x4E, 0xF, 0xF, false));
        return __builtin_amdgcn_perm(p, x, two);
    }
};

}  // namespace gd
