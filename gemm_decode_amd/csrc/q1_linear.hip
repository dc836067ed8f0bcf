// q1_linear.hip -- Q1_0 . q8_0 products with an epilogue: bias, activation, residual or the
// product with a second weight's sums, and the output in the stream's type or as q8_0 blocks.
#include "gd_internal.h"
#include "gd_quant.h"
#include "gd_types.h"

namespace {

using namespace gd;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// One weight: its Q1 planes and the bias of its rows.
struct Weight {
    const u32x2 *bits;
    const uint16_t *scales;
    const float *bias;
};

// What a product makes of its sums.
struct Epilogue {
    const void *residual;
    void *y;
    uint16_t *y_q8;
    int64_t rows, n;
    int32_t act;
};

__device__ __forceinline__ float f16_value(uint16_t h) { return static_cast<float>(__builtin_bit_cast(_Float16, h)); }

// exp(x): the product with log2(e) in two parts, so that the error stays at a few steps for
// every x (one part alone loses |x| 2^-24 of the result).
__device__ __forceinline__ float exp_f32(float x) {
    const float hi = x * 1.442695041f;
    const float lo = fmaf(x, 1.442695041f, -hi) + x * 1.925963033e-8f;
    const float e = __builtin_amdgcn_exp2f(hi);
    return hi > -126.0f && hi < 128.0f ? fmaf(e, lo * 0.693147181f, e) : e;   // past the range: 0 or infinity, no NaN
}

__device__ __forceinline__ float activate(float t, int32_t act) {
    switch (act) {
        case GD_ACT_RELU: return t <= 0.0f ? 0.0f : t;   // a NaN stays
        case GD_ACT_RELU2: return t <= 0.0f ? 0.0f : t * t;
        case GD_ACT_GELU: return 0.5f * t * erfcf(-0.70710678f * t);
        case GD_ACT_GELU_TANH: return t / (1.0f + exp_f32(-1.59576912f * fmaf(0.044715f * t * t, t, t)));
        case GD_ACT_SILU: return t / (1.0f + exp_f32(-t));
        default: return t;
    }
}

// Max over the 32 lanes of a half wave.
__device__ __forceinline__ float max32(float v) {
    v = max8(v);
    v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, false)));
    return fmaxf(v, __shfl_xor(v, 16));
}

// The 8-bit code of v among 32 values whose largest magnitude is a, by the rule of
// q8_0_quantize: in f32 where that gives what the f64 rule gives.
__device__ __forceinline__ uint32_t code_of(float v, float a) {
    if (!(a > 0.0f)) return 0;
    const float inv = recip127(a), t = v * inv;
    int32_t q = static_cast<int32_t>(floorf(t + 0.5f));
    if (!(inv <= 3.40282347e38f) || fabsf(__builtin_amdgcn_fractf(t) - 0.5f) < kTieGuard)
        q = round_code(static_cast<double>(v) * (127.0 / static_cast<double>(a)));
    return static_cast<uint32_t>(q) & 0xffu;
}

// One value of column c and row r; where q8_0 blocks are written, the 32 lanes of a half
// wave hold the 32 rows of one block (r % 32 = lane % 32) and all of them call this.
template <typename T>
__device__ __forceinline__ void finish(const Epilogue &e, float v, int64_t c, int64_t r, bool live) {
    const int64_t at = c * e.rows + r;
    if (e.residual && live) v += static_cast<float>(static_cast<const T *>(e.residual)[at]);
    if (e.y && live) static_cast<T *>(e.y)[at] = static_cast<T>(v);
    if (e.y_q8) {
        const float a = max32(live ? fabsf(v) : 0.0f);
        const uint32_t q = code_of(v, a);
        if (live) {
            uint16_t *o = e.y_q8 + at / 32 * 17;   // 34 bytes = 17 halves
            reinterpret_cast<uint8_t *>(o + 1)[r % 32] = static_cast<uint8_t>(q);
            if (r % 32 == 0) o[0] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(a > 0.0f ? scale_of(a) : 0.0f));
        }
    }
}

// The sum of one row and one column.
__device__ float sum_of(const Weight &w, const uint16_t *a, int64_t r, int64_t K) {
    const int64_t nb = K / 128, nb8 = (nb + 7) / 8;
    float acc = 0.0f;
    for (int64_t i = 0; i < nb; i++) {
        const u32x2 lo = w.bits[((r / 64 * nb + i) * 2 + 0) * 64 + r % 64], hi = w.bits[((r / 64 * nb + i) * 2 + 1) * 64 + r % 64];
        float t = 0.0f;
        for (int k = 0; k < 4; k++) {
            const uint16_t *b = a + (4 * i + k) * 17;
            const int8_t *q = reinterpret_cast<const int8_t *>(b + 1);
            int s = 0;
            for (int j = 0; j < 32; j++) {
                const uint32_t word = j < 16 ? lo[k / 2] : hi[k / 2];
                const int bit = (8 * (j / 4 % 4) + 2 + 4 * (k % 2) + j % 4) % 32;
                s += word >> bit & 1 ? q[j] : -q[j];
            }
            const float d = f16_value(b[0]);
            t = fmaf(fabsf(d) <= 65504.0f ? d : __builtin_nanf(""), static_cast<float>(s), t);
        }
        acc = fmaf(f16_value(w.scales[(r / 64 * nb8 + i / 8) * 512 + r % 64 * 8 + i % 8]), t, acc);
    }
    return acc;
}

// Plain: a thread per row and column.
template <typename T, bool kGated>
__global__ __launch_bounds__(256) void q1_linear_plain_kernel(Weight g, Weight u, const uint16_t *a_q8, Epilogue e, int64_t K) {
    const int64_t r = static_cast<int64_t>(blockIdx.x) * 32 + threadIdx.x % 32;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 8 + threadIdx.x / 32;
    const bool live = r < e.rows && c < e.n;
    float v = 0.0f;
    if (live) {
        const uint16_t *a = a_q8 + c * (K / 32) * 17;
        v = sum_of(g, a, r, K);
        if (g.bias) v += g.bias[r];
        v = activate(v, e.act);
        if (kGated) {
            float up = sum_of(u, a, r, K);
            if (u.bias) up += u.bias[r];
            v *= up;
        }
    }
    finish<T>(e, v, c, r, live);
}

constexpr int64_t kMaxK = INT64_C(1) << 20, kMaxColumns = INT64_C(1) << 20;
constexpr int64_t kFewColumns = 4;   // so many columns take no workspace

int check_sizes(const char *name, int64_t K, int64_t n_act) {
    GD_REQUIRE(K >= 1 && n_act >= 1, GD_EINVAL, "%s: K (%lld) and n_act (%lld) must be >= 1", name, (long long)K,
               (long long)n_act);
    GD_REQUIRE(K % 128 == 0, GD_ESHAPE, "%s: K (%lld) must be a multiple of 128", name, (long long)K);
    GD_REQUIRE(K <= kMaxK && n_act <= kMaxColumns, GD_ERANGE, "%s: K or n_act too large", name);
    return GD_OK;
}

// The activations as the matrix cores read them: 100 bytes for 32 elements.
int64_t workspace_need(int64_t K, int64_t n_act) {
    return n_act <= kFewColumns ? 0 : (n_act + 31) / 32 * 100 * K;   // below 2^42
}

int check(const char *name, const Weight *w, int count, const void *a_q8, const Epilogue &e, int64_t K, int32_t dtype,
          const void *workspace, size_t workspace_bytes) {
    for (int i = 0; i < count; i++) GD_REQUIRE(w[i].bits && w[i].scales, GD_EINVAL, "%s: null pointer", name);
    GD_REQUIRE(a_q8 && (e.y || e.y_q8), GD_EINVAL, "%s: null pointer", name);
    GD_REQUIRE(e.rows >= 1, GD_EINVAL, "%s: rows (%lld) must be >= 1", name, (long long)e.rows);
    GD_REQUIRE(dtype_ok(dtype), GD_EINVAL, "%s: unknown dtype %d", name, dtype);
    GD_REQUIRE(e.act >= GD_ACT_NONE && e.act <= GD_ACT_SILU, GD_EINVAL, "%s: unknown activation %d", name, e.act);
    int st = check_sizes(name, K, e.n);
    if (st) return st;
    GD_REQUIRE(!e.y_q8 || e.rows % 32 == 0, GD_ESHAPE, "%s: rows (%lld) must be a multiple of 32 for q8_0 blocks", name,
               (long long)e.rows);
    GD_REQUIRE(e.rows <= (INT64_C(1) << 31) - 64, GD_ERANGE, "%s: rows too large", name);
    const int64_t size = dtype_size(dtype);
    for (int i = 0; i < count; i++)
        GD_REQUIRE(aligned(w[i].bits, 16) && aligned(w[i].scales, 16) && aligned(w[i].bias, 4), GD_EALIGN,
                   "%s: planes must be 16-byte aligned, a bias 4", name);
    GD_REQUIRE(aligned(a_q8, 2) && aligned(e.y_q8, 2) && aligned(e.residual, size) && aligned(e.y, size) &&
                   aligned(workspace, 16),
               GD_EALIGN, "%s: a_q8 and y_q8 must be 2-byte aligned, residual and y to their element, workspace 16", name);
    const int64_t need = workspace_need(K, e.n), bytes = e.n * e.rows * size;   // below 2^53
    GD_REQUIRE(need == 0 || workspace, GD_EINVAL, "%s: null workspace", name);
    GD_REQUIRE(static_cast<uint64_t>(need) <= workspace_bytes || need == 0, GD_ERANGE, "%s: workspace of %zu bytes, %lld are needed",
               name, workspace_bytes, (long long)need);
    GD_REQUIRE(e.y == e.residual || !overlaps(e.residual, bytes, bytes, 1, e.y, bytes), GD_EINVAL,
               "%s: y may be residual itself, but not overlap it otherwise", name);
    const int64_t a_bytes = e.n * (K / 32) * 34, q_bytes = e.n * (e.rows / 32) * 34;
    GD_REQUIRE(!overlaps(a_q8, a_bytes, a_bytes, 1, e.y, bytes) &&
                   (!e.y_q8 || !overlaps(a_q8, a_bytes, a_bytes, 1, e.y_q8, q_bytes)) &&
                   (!e.y_q8 || !overlaps(e.residual, bytes, bytes, 1, e.y_q8, q_bytes)) &&
                   (!e.y_q8 || !overlaps(e.y, bytes, bytes, 1, e.y_q8, q_bytes)),
               GD_EINVAL, "%s: y and y_q8 must not overlap a_q8, residual or each other", name);
    return GD_OK;
}

template <bool kGated>
void run(const Weight &g, const Weight &u, const void *a_q8, const Epilogue &e, int64_t K, int32_t dtype, hipStream_t hs) {
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const dim3 grid(static_cast<uint32_t>((e.rows + 31) / 32), static_cast<uint32_t>((e.n + 7) / 8));
        hipLaunchKernelGGL((q1_linear_plain_kernel<T, kGated>), grid, dim3(256), 0, hs, g, u,
                           static_cast<const uint16_t *>(a_q8), e, K);
    });
}

}  // namespace

extern "C" int q1_q8_linear_workspace_bytes(int64_t K, int64_t n_act, size_t *bytes) {
    GD_REQUIRE(bytes, GD_EINVAL, "q1_q8_linear_workspace_bytes: null pointer");
    const int st = check_sizes("q1_q8_linear_workspace_bytes", K, n_act);
    if (st) return st;
    *bytes = static_cast<size_t>(workspace_need(K, n_act));
    clear_error();
    return GD_OK;
}

extern "C" int q1_q8_linear(const void *bits_plane, const void *scale_plane, const void *a_q8, const float *bias,
                            int32_t act, const void *residual, void *y, void *y_q8, int64_t rows, int64_t K,
                            int64_t n_act, int32_t dtype, void *workspace, size_t workspace_bytes, void *stream) {
    const Weight w = {static_cast<const u32x2 *>(bits_plane), static_cast<const uint16_t *>(scale_plane), bias};
    const Epilogue e = {residual, y, static_cast<uint16_t *>(y_q8), rows, n_act, act};
    const int st = check("q1_q8_linear", &w, 1, a_q8, e, K, dtype, workspace, workspace_bytes);
    if (st) return st;
    run<false>(w, w, a_q8, e, K, dtype, as_stream(stream));
    return check_launch("q1_q8_linear");
}

extern "C" int q1_q8_gated(const void *gate_bits, const void *gate_scales, const void *up_bits, const void *up_scales,
                           const void *a_q8, const float *gate_bias, const float *up_bias, int32_t act, void *y,
                           void *y_q8, int64_t rows, int64_t K, int64_t n_act, int32_t dtype, void *workspace,
                           size_t workspace_bytes, void *stream) {
    const Weight w[2] = {{static_cast<const u32x2 *>(gate_bits), static_cast<const uint16_t *>(gate_scales), gate_bias},
                         {static_cast<const u32x2 *>(up_bits), static_cast<const uint16_t *>(up_scales), up_bias}};
    const Epilogue e = {nullptr, y, static_cast<uint16_t *>(y_q8), rows, n_act, act};
    const int st = check("q1_q8_gated", w, 2, a_q8, e, K, dtype, workspace, workspace_bytes);
    if (st) return st;
    run<true>(w[0], w[1], a_q8, e, K, dtype, as_stream(stream));
    return check_launch("q1_q8_gated");
}
