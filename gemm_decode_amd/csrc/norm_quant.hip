// norm_quant.hip -- root-mean-square norm with the residual's addition and an
// 8-bit output: the step between the residual stream and a product, in the
// activation formats of the products (q8_0 blocks for q1_q8_gemv, per-token
// int8 bit planes for ternary_gemv), and the readers of those formats.
//
// With h = x + residual (rounded to the stream's type), p = h * w and
// rstd = 1 / sqrt(mean h^2 + eps), the norm is y = rstd * p. The quantization rule
// rounds y times 127 over max|y|: rstd divides out, so the codes depend on p alone
// and only the scale, max|p| * rstd / 127, needs the row's sum. p is a product of two
// f32 values, exact in f64, and the sum of squares is taken in f64, so codes and
// scales do not depend on the order of the sum (up to f64's own rounding, 2^-29 of an
// f32 step).
#include <type_traits>

#include "gd_internal.h"
#include "gd_norm.h"

namespace {

using namespace gd;

constexpr int kThreads = 256;
constexpr int64_t kMaxThreads = (INT64_C(1) << 32) - 1;   // of one launch

// W waves per row, and a workgroup per row (W = 1: four rows). Thread t of a row holds
// pairs of float4s t, t + 64 W, ... of it, R float4s of them in registers (rows of up to
// 256 W R elements are read once); what is past them is read again in the second pass,
// from h_out if that is written (it may overwrite an input), each thread reading back its
// own. A pair is one load of a 16-bit type, and four lanes make a block of 32 (one float4
// a thread and eight lanes: 4099 rows of 4096 in bf16 3.9 us more to q8_0 and 3.0 to
// planes). 4099 rows of 4096 in bf16: 27.8 us to q8_0, 4.3 TB/s, and 32.8 to planes with the
// inputs in memory, 24.9 and 30.7 with them in the last cache; bound by memory with the
// row's sum between its reads and its writes. One row: 3.2 us, bound by the chain load,
// sum, barrier, codes, store.
template <typename T, int R, int W, bool kTernary>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void rmsnorm_quant_kernel(const T *x, const T *res, const float *__restrict__ weight,
                                                               T *h_out, void *__restrict__ out,
                                                               float *__restrict__ x_scale, int64_t n, int64_t K,
                                                               float eps) {
    constexpr int kT = 64 * W;
    __shared__ double red[W][2];
    const int tid = threadIdx.x % kT;
    const int64_t row = W == 1 ? static_cast<int64_t>(blockIdx.x) * 4 + threadIdx.x / 64 : blockIdx.x;
    if (row >= n) return;   // W = 1: a whole wave, and no barriers
    const int nq = static_cast<int>(K / 4);
    x += row * K;
    if (res) res += row * K;
    if (h_out) h_out += row * K;
    // Groups of four elements, in pairs of neighbours: pair i / 2 of the thread, i even.
    const auto group_of = [&](int i) { return i * kT + 2 * tid; };
    f32x4 h[R], w[R];
    double ss = 0.0, amax = 0.0;
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const int e4 = group_of(i);
        const int at = e4 < nq ? e4 : nq - 2;   // clamped: issued, not used
        load_groups<2>(x, res, at, h + i);
        load_groups<2, float>(weight, nullptr, at, w + i);
    }
    float top = 0.0f;
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const int e4 = group_of(i);
        if (e4 < nq) {
            if (h_out) store_groups<2>(h_out, e4, h + i);
#pragma unroll
            for (int j = 0; j < 2; j++) {
                ss += square4(h[i + j]);
                if (kTernary) top = fmaxf(top, Products(h[i + j], w[i + j]).absmax());
            }
        }
    }
    if constexpr (kTernary) {   // the largest product in f64: among those whose f32 rounding is the largest
#pragma unroll
        for (int i = 0; i < R; i++) {
            const Products pr(h[i], w[i]);
            if (group_of(i - i % 2) < nq && (pr.absmax() == top || !in_range(top))) amax = fmax(amax, pr.exact_absmax());
        }
    }
    for (int e4 = R * kT + 2 * tid; e4 < nq; e4 += 2 * kT) {
        f32x4 v[2];
        load_groups<2>(x, res, e4, v);
        if (h_out) store_groups<2>(h_out, e4, v);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            ss += square4(v[j]);
            if (kTernary) amax = fmax(amax, Products(v[j], load4(weight + 4 * (e4 + j))).exact_absmax());
        }
    }
    group_sum_max<W, kTernary>(ss, amax, red);
    const double rstd127 = rsqrt_f64(ss / static_cast<double>(K) + static_cast<double>(eps)) * (1.0 / 127.0);
    const float r32 = static_cast<float>(rstd127);
    const float row_top = static_cast<float>(amax), row_inv = row_top > 0.0f ? recip127(row_top) : 0.0f;
    if (kTernary && tid == 0) x_scale[row] = amax > 0.0 ? static_cast<float>(amax * rstd127) : 0.0f;
    const int64_t groups = K / 32;
    const ByteTranspose tr(threadIdx.x % 4);
    const auto planes = [&](const Products &p0, const Products &p1, int e4) {
        put_planes(p0, p1, tr, amax, row_top, row_inv, static_cast<uint32_t *>(out) + row * 8 * groups + e4 / 8, groups);
    };
    const auto block = [&](const Products &p0, const Products &p1, int e4) {
        put_block(p0, p1, rstd127, r32, static_cast<uint16_t *>(out) + (row * groups + e4 / 8) * 17);
    };
#pragma unroll
    for (int i = 0; i < R; i += 2) {
        const int e4 = group_of(i);
        if (e4 >= nq) continue;
        if constexpr (kTernary)
            planes(Products(h[i], w[i]), Products(h[i + 1], w[i + 1]), e4);
        else
            block(Products(h[i], w[i]), Products(h[i + 1], w[i + 1]), e4);
    }
    for (int e4 = R * kT + 2 * tid; e4 < nq; e4 += 2 * kT) {   // past the registers, read once more
        if (h_out)
            load_groups<2, T>(h_out, nullptr, e4, h);
        else
            load_groups<2>(x, res, e4, h);
        load_groups<2, float>(weight, nullptr, e4, w);
        if constexpr (kTernary)
            planes(Products(h[0], w[0]), Products(h[1], w[1]), e4);
        else
            block(Products(h[0], w[0]), Products(h[1], w[1]), e4);
    }
}

// ------------------------------------------------------------- readers
// code * scale, one f32 product, rounded to T: of the four codes in a word, or eight in
// two. A thread has 16 bytes to write: eight elements of a 16-bit type (four: 4096 rows of
// 4096 in bf16 10.3 us from q8_0 and 12.5 from planes, where these take 8.5 and 10.0),
// four of f32 (eight, as two stores: 2048 rows of 6912 13.5 and 14.9, where these take
// 11.8 and 13.5). Bound by memory: 16.8 M values from q8_0 to f32 in 13.6 us, 6.2 TB/s.
template <typename T>
constexpr int kWords = 4 / sizeof(T);   // of codes, a thread
template <typename T>
__device__ __forceinline__ void store_codes(T *y, int64_t unit, const uint32_t *codes, float d) {
    f32x4 v[kWords<T>];
#pragma unroll
    for (int j = 0; j < 4 * kWords<T>; j++)
        v[j / 4][j % 4] = static_cast<float>(static_cast<int8_t>(codes[j / 4] >> (8 * (j % 4)))) * d;
    store_groups<kWords<T>>(y, kWords<T> * unit, v);
}

template <typename T>
__global__ __launch_bounds__(kThreads) void q8_0_dequantize_kernel(const uint16_t *__restrict__ a, T *__restrict__ y,
                                                                   int64_t units) {
    constexpr int kPer = 8 / kWords<T>;   // threads of a block
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (gid >= units) return;
    const uint16_t *b = a + (gid / kPer) * 17;
    typedef uint32_t Word __attribute__((aligned(2)));
    uint32_t codes[kWords<T>];
#pragma unroll
    for (int i = 0; i < kWords<T>; i++)
        codes[i] = reinterpret_cast<const Word *>(b + 1)[kWords<T> * (gid % kPer) + i];
    store_codes(y, gid, codes, static_cast<float>(__builtin_bit_cast(_Float16, b[0])));
}

// Eight elements: lane k of a block's four loads the words of the planes 2 k and 2 k + 1,
// and the norm's transpose, taken back, gives it its codes. Four: lane k of eight loads
// plane k's word, and nibbles are transposed.
template <typename T>
__global__ __launch_bounds__(kThreads) void ternary_dequantize_kernel(const uint32_t *__restrict__ planes,
                                                                      const float *__restrict__ x_scale,
                                                                      T *__restrict__ y, int64_t K, int64_t units) {
    constexpr int kPer = 8 / kWords<T>;
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (gid >= units) return;   // whole blocks
    const uint32_t q = static_cast<uint32_t>(K / (4 * kWords<T>));
    const uint32_t row = static_cast<uint32_t>(gid) / q, at = static_cast<uint32_t>(gid) % q;
    const int64_t W = K / 32;
    const int k = static_cast<int>(at % kPer);
    const uint32_t *p = planes + (static_cast<int64_t>(row) * 8 + kWords<T> * k) * W + at / kPer;
    uint32_t codes[kWords<T>];
    if constexpr (kWords<T> == 1) {
        codes[0] = nibbles_to_bits(NibbleTranspose(k)(p[0]));
    } else {
        const ByteTranspose tr(k);
        const uint32_t even = tr(p[0]), odd = tr(p[W]);   // a byte of each even plane, of each odd one
        codes[0] = nibbles_to_bits((even & 0x0F0F0F0Fu) | ((odd & 0x0F0F0F0Fu) << 4));
        codes[1] = nibbles_to_bits(((even >> 4) & 0x0F0F0F0Fu) | (odd & 0xF0F0F0F0u));
    }
    store_codes(y, gid, codes, x_scale[row]);
}

int check_norm(const char *name, const void *x, const void *residual, const float *weight, const void *h_out, int64_t n,
               int64_t K, float eps, int32_t dtype) {
    GD_REQUIRE(x && weight, GD_EINVAL, "%s: null pointer", name);
    GD_REQUIRE(n >= 1 && K >= 1, GD_EINVAL, "%s: n (%lld) and K (%lld) must be >= 1", name, (long long)n, (long long)K);
    GD_REQUIRE(dtype_ok(dtype), GD_EINVAL, "%s: unknown dtype %d", name, dtype);
    GD_REQUIRE(eps >= 0.0f && eps <= 3.40282347e38f, GD_EINVAL, "%s: eps must be finite and >= 0", name);
    GD_REQUIRE(K % 32 == 0, GD_ESHAPE, "%s: K (%lld) must be a multiple of 32", name, (long long)K);
    GD_REQUIRE(n <= kMaxThreads / 512 && K <= (INT64_C(1) << 30), GD_ERANGE, "%s: n or K too large", name);
    GD_REQUIRE(aligned(x, 16) && aligned(residual, 16) && aligned(weight, 16) && aligned(h_out, 16), GD_EALIGN,
               "%s: x, residual, weight and h_out must be 16-byte aligned", name);
    return GD_OK;
}

// After the other checks: h_out is x or residual, or apart from them.
int check_in_place(const char *name, const void *x, const void *residual, const void *h_out, int64_t n, int64_t K,
                   int32_t dtype) {
    const int64_t bytes = n * K * dtype_size(dtype);   // below 2^55
    GD_REQUIRE((h_out == x || !overlaps(x, bytes, bytes, 1, h_out, bytes)) &&
                   (h_out == residual || !overlaps(residual, bytes, bytes, 1, h_out, bytes)),
               GD_EINVAL, "%s: h_out may be x or residual itself, but not overlap them otherwise", name);
    return GD_OK;
}

template <bool kTernary>
void launch_norm(const void *x, const void *residual, const float *weight, void *h_out, void *out, float *x_scale,
                 int64_t n, int64_t K, float eps, int32_t dtype, hipStream_t hs) {
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const T *xt = static_cast<const T *>(x), *rt = static_cast<const T *>(residual);
        T *ht = static_cast<T *>(h_out);
        const auto launch = [&](auto r, auto w) {
            constexpr int W = decltype(w)::value;
            const dim3 grid(static_cast<uint32_t>(W == 1 ? (n + 3) / 4 : n));
            hipLaunchKernelGGL((rmsnorm_quant_kernel<T, decltype(r)::value, W, kTernary>), grid,
                               dim3(W == 1 ? 256 : 64 * W), 0, hs, xt, rt, weight, ht, out, x_scale, n, K, eps);
        };
        // Many short rows: a wave each (16384 rows of 512 in bf16: 13.8 us, 41.8 with eight waves a row, most of
        // them idle; 1024 rows of 1024 4.7 and 5.6, 512 of them 4.5 and 4.2, one 3.2 and 2.8). Else eight waves a
        // row (one f32 row of 4096: 3.4 us, 3.9 with four waves; 4099 rows in bf16 26.4 and 27.3; sixteen for rows
        // past 4096: 1024 rows of 14336 in bf16 27.1 where eight take 25.8, one in f32 5.9 and 6.5). Each pair of
        // figures is of one run, inputs of two or three states in turn; single figures differ by 5 % from card to card.
        const bool many = n >= 1024;
        if (K <= 512 && many)
            launch(std::integral_constant<int, 2>{}, std::integral_constant<int, 1>{});
        else if (K <= 1024 && many)
            launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 1>{});
        else if (K <= 4096)
            launch(std::integral_constant<int, 2>{}, std::integral_constant<int, 8>{});
        else
            launch(std::integral_constant<int, 4>{}, std::integral_constant<int, 8>{});
    });
}

int check_reader(const char *name, const void *in, const void *y, int64_t n, int64_t K, int32_t dtype, int64_t *quads) {
    GD_REQUIRE(in && y, GD_EINVAL, "%s: null pointer", name);
    GD_REQUIRE(n >= 1 && K >= 1, GD_EINVAL, "%s: n (%lld) and K (%lld) must be >= 1", name, (long long)n, (long long)K);
    GD_REQUIRE(dtype_ok(dtype), GD_EINVAL, "%s: unknown dtype %d", name, dtype);
    GD_REQUIRE(K % 32 == 0, GD_ESHAPE, "%s: K (%lld) must be a multiple of 32", name, (long long)K);
    GD_REQUIRE(mul_ok(n, K / 4, quads) && *quads <= kMaxThreads - kThreads, GD_ERANGE, "%s: n * K too large", name);
    GD_REQUIRE(aligned(y, 16), GD_EALIGN, "%s: y must be 16-byte aligned", name);
    return GD_OK;
}

}  // namespace

extern "C" int rmsnorm_q8_0(const void *x, const void *residual, const float *weight, void *h_out, void *a_q8, int64_t n,
                            int64_t K, float eps, int32_t dtype, void *stream) {
    int st = check_norm("rmsnorm_q8_0", x, residual, weight, h_out, n, K, eps, dtype);
    if (st) return st;
    GD_REQUIRE(a_q8, GD_EINVAL, "rmsnorm_q8_0: null pointer");
    GD_REQUIRE(aligned(a_q8, 2), GD_EALIGN, "rmsnorm_q8_0: a_q8 must be 2-byte aligned");
    st = check_in_place("rmsnorm_q8_0", x, residual, h_out, n, K, dtype);
    if (st) return st;
    launch_norm<false>(x, residual, weight, h_out, a_q8, nullptr, n, K, eps, dtype, as_stream(stream));
    return check_launch("rmsnorm_q8_0");
}

extern "C" int rmsnorm_ternary_act(const void *x, const void *residual, const float *weight, void *h_out,
                                   uint32_t *planes, float *x_scale, int64_t n, int64_t K, float eps, int32_t dtype,
                                   void *stream) {
    int st = check_norm("rmsnorm_ternary_act", x, residual, weight, h_out, n, K, eps, dtype);
    if (st) return st;
    GD_REQUIRE(planes && x_scale, GD_EINVAL, "rmsnorm_ternary_act: null pointer");
    GD_REQUIRE(aligned(planes, 4) && aligned(x_scale, 4), GD_EALIGN,
               "rmsnorm_ternary_act: planes and x_scale must be 4-byte aligned");
    st = check_in_place("rmsnorm_ternary_act", x, residual, h_out, n, K, dtype);
    if (st) return st;
    launch_norm<true>(x, residual, weight, h_out, planes, x_scale, n, K, eps, dtype, as_stream(stream));
    return check_launch("rmsnorm_ternary_act");
}

extern "C" int q8_0_dequantize(const void *a_q8, void *y, int64_t n, int64_t K, int32_t dtype, void *stream) {
    int64_t quads;
    int st = check_reader("q8_0_dequantize", a_q8, y, n, K, dtype, &quads);
    if (st) return st;
    GD_REQUIRE(aligned(a_q8, 2), GD_EALIGN, "q8_0_dequantize: a_q8 must be 2-byte aligned");
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t units = quads / kWords<T>;
        const dim3 grid(static_cast<uint32_t>((units + kThreads - 1) / kThreads));
        hipLaunchKernelGGL((q8_0_dequantize_kernel<T>), grid, dim3(kThreads), 0, as_stream(stream),
                           static_cast<const uint16_t *>(a_q8), static_cast<T *>(y), units);
    });
    return check_launch("q8_0_dequantize");
}

extern "C" int ternary_dequantize_act(const uint32_t *planes, const float *x_scale, void *y, int64_t n, int64_t K,
                                      int32_t dtype, void *stream) {
    int64_t quads;
    int st = check_reader("ternary_dequantize_act", planes, y, n, K, dtype, &quads);
    if (st) return st;
    GD_REQUIRE(x_scale, GD_EINVAL, "ternary_dequantize_act: null pointer");
    GD_REQUIRE(aligned(planes, 4) && aligned(x_scale, 4), GD_EALIGN,
               "ternary_dequantize_act: planes and x_scale must be 4-byte aligned");
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        const int64_t units = quads / kWords<T>;
        const dim3 grid(static_cast<uint32_t>((units + kThreads - 1) / kThreads));
        hipLaunchKernelGGL((ternary_dequantize_kernel<T>), grid, dim3(kThreads), 0, as_stream(stream), planes, x_scale,
                           static_cast<T *>(y), K, units);
    });
    return check_launch("ternary_dequantize_act");
}
