// norm_sandwich.hip -- the norms behind and before a block in one pass over a row: the
// block's output x is normed (rstd(x) * post_weight), gated and scaled, added to the scaled
// residual, rounded to the stream's type (h), and h normed into an 8-bit output.
//   u = x rstd(x) post_weight,  h = residual_scale residual + block_scale gate u,
//   out = quantized h rstd(h) weight
// 4099 rows of 4096 bf16 with gates to q8_0 take 38 us: 118 MB, 24 us as a copy; the vector units
// are busy for four fifths of the time (56 instructions an element, a third of them f64 or to and
// from it) and each row's two sums stand between its reads and its writes.
//
// h is worked out in f64 from values that f64 holds exactly, so that its rounding, and with
// it the codes, do not depend on the order of the sums (up to f64's own rounding); codes and
// scales are decided as in the norm without the first half.
#include <type_traits>

#include "gd_internal.h"
#include "gd_norm.h"

namespace {

using namespace gd;

template <typename T>
struct Sandwich {
    const T *x;
    const float *post_weight;
    const T *gate;
    const int32_t *gate_index;
    const T *residual;
    const float *weight;
    T *h_out;
    void *out;
    float *x_scale;
    int64_t n, K, n_gates;
    double residual_scale, block_scale;
    double per;   // 1 / K
    float eps;
};

// Four elements of h: factor is the block's scale and, with a norm behind it, its rstd.
template <typename T>
__device__ __forceinline__ f32x4 join4(const Sandwich<T> &s, f32x4 x, f32x4 res, f32x4 post, f32x4 gate, double factor) {
    f32x4 h;
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const double u = static_cast<double>(x[j]) * factor * static_cast<double>(post[j]);
        h[j] = static_cast<float>(static_cast<T>(static_cast<float>(__builtin_fma(u, static_cast<double>(gate[j]), s.residual_scale * static_cast<double>(res[j])))));
    }
    return h;
}

// W waves per row, and a workgroup per row (W = 1: four rows). As in the norm without the
// first half, thread t holds pairs of float4s t, t + 64 W, ... of the row, R float4s in
// registers; what is past them is read again: twice for h, and then back from h_out where
// that is written (it may overwrite an input), each thread its own.
template <typename T, int R, int W, bool kTernary>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rmsnorm_sandwich_kernel(const Sandwich<T> s) {
    constexpr int kT = 64 * W;
    __shared__ double red[2][W][2];
    const int tid = threadIdx.x % kT;
    const int64_t row = W == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64 : blockIdx.x;
    if (row >= s.n) return;   // W = 1: a whole wave, and no barriers
    const int nq = static_cast<int>(s.K / 4);
    const T *x = s.x + row * s.K, *res = s.residual + row * s.K;
    T *h_out = s.h_out ? s.h_out + row * s.K : nullptr;
    double factor = s.block_scale;
    const T *gate = s.gate;
    bool dropped = false;   // nothing of the block is taken, whatever it holds
    if (gate) {
        int64_t g = s.gate_index ? s.gate_index[row] : s.n_gates == 1 ? 0 : row;
        dropped = g < 0 || g >= s.n_gates;
        gate = dropped ? nullptr : gate + g * s.K;
        if (dropped) factor = 0.0;
    }
    const float *post_weight = dropped ? nullptr : s.post_weight;   // (a whole workgroup's, or a wave's without barriers)
    const auto group_of = [&](int i) { return i * kT + 2 * tid; };
    const f32x4 ones = {1.0f, 1.0f, 1.0f, 1.0f};
    const auto load_side = [&](int64_t at, f32x4 *post, f32x4 *gates) {
        post[0] = post[1] = gates[0] = gates[1] = ones;
        if (post_weight) load_groups<2, float>(post_weight, nullptr, at, post);
        if (gate) load_groups<2, T>(gate, nullptr, at, gates);
    };
    f32x4 h[R], r[R], w[R], post[R], gates[R];
    double ss = 0.0, amax = 0.0;
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const int e4 = group_of(i);
        const int at = e4 < nq ? e4 : nq - 2;   // clamped: issued, not used
        load_groups<2, T>(x, nullptr, at, h + i);
        load_groups<2, T>(res, nullptr, at, r + i);
        load_side(at, post + i, gates + i);
        load_groups<2, float>(s.weight, nullptr, at, w + i);
    }
    if (post_weight) {
#pragma unroll
        for (int i = 0; i < R; i++)
            if (group_of(i - i % 2) < nq) ss += square4(h[i]);
        for (int e4 = R * kT + 2 * tid; e4 < nq; e4 += 2 * kT) {
            f32x4 v[2];
            load_groups<2, T>(x, nullptr, e4, v);
            ss += square4(v[0]) + square4(v[1]);
        }
        group_sum_max<W, false>(ss, amax, red[0]);
        const double mean = __builtin_fma(ss, s.per, static_cast<double>(s.eps));
        factor *= mean == 0.0 ? 0.0 : rsqrt_f64(mean);   // a row of zeros without eps
        ss = 0.0;
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const int e4 = group_of(i);
        if (e4 >= nq) continue;
        if (dropped) h[i] = h[i + 1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = i; j < i + 2; j++) {
            h[j] = join4(s, h[j], r[j], post[j], gates[j], factor);
            ss += square4(h[j]);
            if (kTernary) top = fmaxf(top, Products(h[j], w[j]).absmax());
        }
        if (h_out) store_groups<2>(h_out, e4, h + i);
    }
    if constexpr (kTernary) {   // the largest product in f64: among those whose f32 rounding is the largest
#pragma unroll
        for (int i = 0; i < R; i++) {
            const Products pr(h[i], w[i]);
            if (group_of(i - i % 2) < nq && (pr.absmax() == top || !in_range(top))) amax = fmax(amax, pr.exact_absmax());
        }
    }
    const auto join_at = [&](int64_t e4, f32x4 *v) {
        f32x4 rr[2], pp[2], gg[2];
        load_groups<2, T>(x, nullptr, e4, v);
        load_groups<2, T>(res, nullptr, e4, rr);
        load_side(e4, pp, gg);
        if (dropped) v[0] = v[1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int j = 0; j < 2; j++) v[j] = join4(s, v[j], rr[j], pp[j], gg[j], factor);
    };
    for (int e4 = R * kT + 2 * tid; e4 < nq; e4 += 2 * kT) {
        f32x4 v[2];
        join_at(e4, v);
        if (h_out) store_groups<2>(h_out, e4, v);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            ss += square4(v[j]);
            if (kTernary) amax = fmax(amax, Products(v[j], load4(s.weight + 4 * (e4 + j))).exact_absmax());
        }
    }
    group_sum_max<W, kTernary>(ss, amax, red[1]);
    const double rstd127 = rsqrt_f64(__builtin_fma(ss, s.per, static_cast<double>(s.eps))) * (1.0 / 127.0);
    const float r32 = static_cast<float>(rstd127);
    const float row_top = static_cast<float>(amax), row_inv = row_top > 0.0f ? recip127(row_top) : 0.0f;
    if (kTernary && tid == 0) s.x_scale[row] = amax > 0.0 ? static_cast<float>(amax * rstd127) : 0.0f;
    const int64_t groups = s.K / 32;
    const ByteTranspose tr(threadIdx.x % 4);
    const auto put = [&](f32x4 h0, f32x4 h1, f32x4 w0, f32x4 w1, int64_t e4) {
        if constexpr (kTernary)
            put_planes(Products(h0, w0), Products(h1, w1), tr, amax, row_top, row_inv,
                       static_cast<uint32_t *>(s.out) + row * 8 * groups + e4 / 8, groups);
        else
            put_block(Products(h0, w0), Products(h1, w1), rstd127, r32,
                      static_cast<uint16_t *>(s.out) + (row * groups + e4 / 8) * 17);
    };
#pragma unroll
    for (int i = 0; i < R; i += 2)
        if (group_of(i) < nq) put(h[i], h[i + 1], w[i], w[i + 1], group_of(i));
    for (int e4 = R * kT + 2 * tid; e4 < nq; e4 += 2 * kT) {   // past the registers, read once more
        f32x4 v[2], ww[2];
        if (h_out)
            load_groups<2, T>(h_out, nullptr, e4, v);
        else
            join_at(e4, v);
        load_groups<2, float>(s.weight, nullptr, e4, ww);
        put(v[0], v[1], ww[0], ww[1], e4);
    }
}

struct Args {
    const void *x;
    const float *post_weight;
    const void *gate;
    int64_t n_gates;
    const int32_t *gate_index;
    const void *residual;
    float residual_scale, block_scale;
    const float *weight;
    void *h_out, *out;
    float *x_scale;
    int64_t n, K;
    float eps;
    int32_t dtype;
};

bool finite(float v) { return v >= -3.40282347e38f && v <= 3.40282347e38f; }

int check(const char *name, const Args &a) {
    GD_REQUIRE(a.x && a.residual && a.weight && a.out, GD_EINVAL, "%s: null pointer", name);
    GD_REQUIRE(a.n >= 1 && a.K >= 1, GD_EINVAL, "%s: n (%lld) and K (%lld) must be >= 1", name, (long long)a.n,
               (long long)a.K);
    GD_REQUIRE(dtype_ok(a.dtype), GD_EINVAL, "%s: unknown dtype %d", name, a.dtype);
    GD_REQUIRE(a.eps >= 0.0f && finite(a.eps), GD_EINVAL, "%s: eps must be finite and >= 0", name);
    GD_REQUIRE(finite(a.residual_scale) && finite(a.block_scale), GD_EINVAL,
               "%s: residual_scale and block_scale must be finite", name);
    GD_REQUIRE(a.gate || !a.gate_index, GD_EINVAL, "%s: gate_index needs gate", name);
    GD_REQUIRE(a.K % 32 == 0, GD_ESHAPE, "%s: K (%lld) must be a multiple of 32", name, (long long)a.K);
    GD_REQUIRE(a.n < (INT64_C(1) << 23) && a.K <= (INT64_C(1) << 30), GD_ERANGE, "%s: n or K too large", name);
    if (a.gate) {
        GD_REQUIRE(a.n_gates >= 1, GD_EINVAL, "%s: n_gates (%lld) must be >= 1", name, (long long)a.n_gates);
        GD_REQUIRE(a.n_gates < (INT64_C(1) << 23), GD_ERANGE, "%s: n_gates too large", name);
        GD_REQUIRE(a.gate_index || a.n_gates == 1 || a.n_gates == a.n, GD_EINVAL,
                   "%s: without gate_index n_gates must be 1 or n", name);
    }
    GD_REQUIRE(aligned(a.x, 16) && aligned(a.post_weight, 16) && aligned(a.gate, 16) && aligned(a.residual, 16) &&
                   aligned(a.weight, 16) && aligned(a.h_out, 16) && aligned(a.gate_index, 4),
               GD_EALIGN, "%s: x, post_weight, gate, residual, weight and h_out must be 16-byte aligned, gate_index 4",
               name);
    return GD_OK;
}

// After the other checks: h_out is x or residual, or apart from them, and from the gates; the
// 8-bit output (out_bytes) and its scales are apart from all of them.
int check_in_place(const char *name, const Args &a, int64_t out_bytes) {
    const int64_t size = dtype_size(a.dtype), bytes = a.n * a.K * size;   // below 2^55
    GD_REQUIRE((a.h_out == a.x || !overlaps(a.x, bytes, bytes, 1, a.h_out, bytes)) &&
                   (a.h_out == a.residual || !overlaps(a.residual, bytes, bytes, 1, a.h_out, bytes)),
               GD_EINVAL, "%s: h_out may be x or residual itself, but not overlap them otherwise", name);
    const int64_t gates = a.gate ? a.n_gates * a.K * size : 0;
    GD_REQUIRE(!a.gate || !a.h_out || !overlaps(a.gate, gates, gates, 1, a.h_out, bytes), GD_EINVAL,
               "%s: h_out must not overlap gate", name);
    const void *outs[2] = {a.out, a.x_scale};
    const int64_t sizes[2] = {out_bytes, a.n * 4};
    for (int i = 0; i < 2; i++)
        GD_REQUIRE(!outs[i] || (!overlaps(a.x, bytes, bytes, 1, outs[i], sizes[i]) && !overlaps(a.residual, bytes, bytes, 1, outs[i], sizes[i]) &&
                                (!a.gate || !overlaps(a.gate, gates, gates, 1, outs[i], sizes[i])) &&
                                (!a.h_out || !overlaps(a.h_out, bytes, bytes, 1, outs[i], sizes[i]))),
                   GD_EINVAL, "%s: the 8-bit output and its scales must not overlap x, residual, gate or h_out", name);
    GD_REQUIRE(!a.x_scale || !overlaps(a.out, out_bytes, out_bytes, 1, a.x_scale, sizes[1]), GD_EINVAL,
               "%s: planes and x_scale must not overlap", name);
    return GD_OK;
}

template <bool kTernary>
void launch(const Args &a, hipStream_t hs) {
    dispatch_dtype(a.dtype, [&](auto t) {
        using T = decltype(t);
        const Sandwich<T> s = {static_cast<const T *>(a.x), a.post_weight, static_cast<const T *>(a.gate), a.gate_index,
                               static_cast<const T *>(a.residual), a.weight, static_cast<T *>(a.h_out), a.out, a.x_scale,
                               a.n, a.K, a.n_gates, a.residual_scale, a.block_scale, 1.0 / static_cast<double>(a.K),
                               a.eps};
        const auto go = [&](auto r, auto w) {
            constexpr int W = decltype(w)::value;
            const dim3 grid(static_cast<uint32_t>(W == 1 ? (a.n + 3) / 4 : a.n));
            hipLaunchKernelGGL((rmsnorm_sandwich_kernel<T, decltype(r)::value, W, kTernary>), grid,
                               dim3(W == 1 ? 256 : 64 * W), 0, hs, s);
        };
        // As the norm without the first half: a wave per row where many rows are short; eight waves
        // a row for few rows, whose latency counts (one row of 4096 f32 5.3 us with its reader,
        // with four waves 5.7); of many rows four, half the sums over waves (4099 rows of 4096 bf16
        // 51.9 us with their reader, with eight waves 53.8, with two 57).
        const bool many = a.n >= 1024;
        if (a.K <= 512 && many)
            go(std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{});
        else if (a.K <= 1024 && many)
            go(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
        else if (a.K <= 4096 && many)
            go(std::integral_constant<int, 4>{}, std::integral_constant<int, 4>{});
        else if (a.K <= 4096)
            go(std::integral_constant<int, 2>{}, std::integral_constant<int, 8>{});
        else
            go(std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{});
    });
}

}  // namespace

extern "C" int rmsnorm_sandwich_q8_0(const void *x, const float *post_weight, const void *gate, int64_t n_gates,
                                     const int32_t *gate_index, const void *residual, float residual_scale,
                                     float block_scale, const float *weight, void *h_out, void *a_q8, int64_t n,
                                     int64_t K, float eps, int32_t dtype, void *stream) {
    const char *name = "rmsnorm_sandwich_q8_0";
    const Args a = {x, post_weight, gate, n_gates, gate_index, residual, residual_scale, block_scale,
                    weight, h_out, a_q8, nullptr, n, K, eps, dtype};
    int st = check(name, a);
    if (st) return st;
    GD_REQUIRE(aligned(a_q8, 2), GD_EALIGN, "%s: a_q8 must be 2-byte aligned", name);
    st = check_in_place(name, a, n * (K / 32) * 34);
    if (st) return st;
    launch<false>(a, as_stream(stream));
    return check_launch(name);
}

extern "C" int rmsnorm_sandwich_ternary_act(const void *x, const float *post_weight, const void *gate, int64_t n_gates,
                                            const int32_t *gate_index, const void *residual, float residual_scale,
                                            float block_scale, const float *weight, void *h_out, uint32_t *planes,
                                            float *x_scale, int64_t n, int64_t K, float eps, int32_t dtype,
                                            void *stream) {
    const char *name = "rmsnorm_sandwich_ternary_act";
    const Args a = {x, post_weight, gate, n_gates, gate_index, residual, residual_scale, block_scale,
                    weight, h_out, planes, x_scale, n, K, eps, dtype};
    int st = check(name, a);
    if (st) return st;
    GD_REQUIRE(x_scale, GD_EINVAL, "%s: null pointer", name);
    GD_REQUIRE(aligned(planes, 4) && aligned(x_scale, 4), GD_EALIGN, "%s: planes and x_scale must be 4-byte aligned", name);
    st = check_in_place(name, a, n * K);
    if (st) return st;
    launch<true>(a, as_stream(stream));
    return check_launch(name);
}
