// kv_q8.hip -- the 8-bit cache of keys and values: rotary positions with the
// quantizing write, the read back, and the table of rotary angles.
//
// Cache planes (one pool of pages, keys and values alike): codes int8
// [n_pages][n_kv_heads][page_size][head_dim] and scales f16
// [n_pages][n_kv_heads][page_size][head_dim / 32]; position p of page g of
// head h stands for codes * scale, 32 dims to a scale. Rows are kept whole and
// in the order of the dims: a token's write and a position's read are runs of
// head_dim bytes, and a tile of 16 positions of one head is contiguous.
#include <cmath>

#include "gd_internal.h"
#include "gd_quant.h"
#include "gd_types.h"

namespace {

using namespace gd;

constexpr int kThreads = 256;
constexpr int64_t kMaxThreads = (INT64_C(1) << 32) - 1;   // of one launch
constexpr int kMaxRot = 256;

// ------------------------------------------------------- rotary table
struct RopeFreqs {
    double f[kMaxRot / 2];
    double attention;
};

// (cos, sin) of position * freq, in f64 (the angles of far positions lose
// their low bits in f32), rounded once.
__global__ __launch_bounds__(kThreads) void rope_table_kernel(f32x2 *__restrict__ table, RopeFreqs fr, int32_t half,
                                                              int64_t n) {
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    if (gid >= n) return;
    double s, c;
    sincos(static_cast<double>(gid / half) * fr.f[gid % half], &s, &c);
    table[gid] = f32x2{static_cast<float>(c * fr.attention), static_cast<float>(s * fr.attention)};
}

// --------------------------------------------------------------- store
struct StoreArgs {
    const void *q, *k, *v;
    void *q_out;
    const f32x2 *rope;
    const int32_t *positions;
    const int64_t *slots;
    int64_t q_stride, k_stride, v_stride, n_pos, n_tok;
    int32_t n_heads, rot, interleaved;
    gd_kv_q8 c;
};

// Four dims d0 .. d0 + 3 of a head row, turned by the row's angles: the f64
// sum of products that are exact in f64, rounded to f32.
template <typename T>
__device__ __forceinline__ f32x4 rotated(const T *row, int d0, const f32x2 *cs, int rot, bool interleaved) {
    const f32x4 x = load4(row + d0);
    if (d0 >= rot) return x;
    f32x4 y;
    if (interleaved) {   // pairs (2i, 2i + 1), both here
        const f32x4 t = *reinterpret_cast<const f32x4 *>(cs + d0 / 2);
#pragma unroll
        for (int i = 0; i < 2; i++) {
            const double a = x[2 * i], b = x[2 * i + 1], c = t[2 * i], s = t[2 * i + 1];
            y[2 * i] = static_cast<float>(a * c - b * s);
            y[2 * i + 1] = static_cast<float>(b * c + a * s);
        }
    } else {   // pairs (i, i + rot / 2): the partners are another lane's
        const int half = rot / 2;
        const bool first = d0 < half;
        const int i0 = first ? d0 : d0 - half;
        const f32x4 o = load4(row + (first ? d0 + half : d0 - half));
        const f32x4 t0 = *reinterpret_cast<const f32x4 *>(cs + i0);
        const f32x4 t1 = *reinterpret_cast<const f32x4 *>(cs + i0 + 2);
#pragma unroll
        for (int j = 0; j < 4; j++) {
            const double a = x[j], b = o[j];
            const double c = j < 2 ? t0[2 * j] : t1[2 * j - 4], s = j < 2 ? t0[2 * j + 1] : t1[2 * j - 3];
            y[j] = static_cast<float>(a * c + (first ? -(b * s) : b * s));
        }
    }
    return y;
}

// Four dims per thread, head_dim / 4 threads per head row (a row never leaves
// its wave, so q_out may be q itself: a wave reads its rows before it writes
// them). Rows of a token in the order q heads, k heads, v heads.
template <typename T>
__global__ __launch_bounds__(kThreads) void kv_q8_store_kernel(StoreArgs a) {
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int D = static_cast<int>(a.c.head_dim), lanes = D / 4;
    const int Hkv = static_cast<int>(a.c.n_kv_heads);
    const int rows = a.n_heads + 2 * Hkv;
    const int64_t r = gid / lanes;
    const int64_t tok = r / rows;
    if (tok >= a.n_tok) return;
    int h = static_cast<int>(r % rows);
    const int d0 = static_cast<int>(gid % lanes) * 4;
    const int64_t slot = a.slots[tok];
    const bool live = slot >= 0 && slot < a.c.n_pages * a.c.page_size;
    const f32x2 *cs = nullptr;
    if (a.rope) {
        const int64_t pos = a.positions[tok];
        if (pos < 0 || pos >= a.n_pos) return;   // no angles for it: the token is left out
        cs = a.rope + pos * (a.rot / 2);
    }
    const int rot = a.rope ? a.rot : 0;
    if (h < a.n_heads) {
        const f32x4 y = rotated(static_cast<const T *>(a.q) + tok * a.q_stride + h * D, d0, cs, rot, a.interleaved);
        store4(static_cast<T *>(a.q_out) + (tok * a.n_heads + h) * D + d0, y);
        return;
    }
    if (!live) return;
    h -= a.n_heads;
    const bool is_v = h >= Hkv;
    if (is_v) h -= Hkv;
    const f32x4 y = is_v ? load4(static_cast<const T *>(a.v) + tok * a.v_stride + h * D + d0)
                         : rotated(static_cast<const T *>(a.k) + tok * a.k_stride + h * D, d0, cs, rot, a.interleaved);
    const float4 y4 = {y[0], y[1], y[2], y[3]};
    const float m = max8(absmax4(y4));
    uint32_t packed = 0;
    _Float16 d = 0;
    if (m > 0.0f) {
        const float inv32 = recip127(m);
        packed = codes4(y4, inv32, m, !(inv32 <= 3.40282347e38f));   // f64 only if the reciprocal overflowed
        d = static_cast<_Float16>(scale_of(m));
    }
    const int64_t page = slot / a.c.page_size, off = slot % a.c.page_size;
    const int64_t row = (page * Hkv + h) * a.c.page_size + off;
    *reinterpret_cast<uint32_t *>((is_v ? a.c.v_codes : a.c.k_codes) + row * D + d0) = packed;
    if (d0 % 32 == 0)
        (is_v ? a.c.v_scales : a.c.k_scales)[row * (D / 32) + d0 / 32] = __builtin_bit_cast(uint16_t, d);
}

// ---------------------------------------------------------------- load
template <typename T>
__global__ __launch_bounds__(kThreads) void kv_q8_load_kernel(gd_kv_q8 c, const int64_t *__restrict__ slots,
                                                              T *__restrict__ k_out, T *__restrict__ v_out,
                                                              int64_t n_tok) {
    const int64_t gid = static_cast<int64_t>(blockIdx.x) * kThreads + threadIdx.x;
    const int D = static_cast<int>(c.head_dim), lanes = D / 4;
    const int Hkv = static_cast<int>(c.n_kv_heads);
    const int64_t r = gid / lanes;
    const int64_t tok = r / (2 * Hkv);
    if (tok >= n_tok) return;
    int h = static_cast<int>(r % (2 * Hkv));
    const bool is_v = h >= Hkv;
    if (is_v) h -= Hkv;
    const int d0 = static_cast<int>(gid % lanes) * 4;
    T *out = is_v ? v_out : k_out;
    if (!out) return;
    const int64_t slot = slots[tok];
    f32x4 y = {0.0f, 0.0f, 0.0f, 0.0f};
    if (slot >= 0 && slot < c.n_pages * c.page_size) {
        const int64_t row = ((slot / c.page_size) * Hkv + h) * c.page_size + slot % c.page_size;
        const uint32_t w = *reinterpret_cast<const uint32_t *>((is_v ? c.v_codes : c.k_codes) + row * D + d0);
        const float d = static_cast<float>(
            __builtin_bit_cast(_Float16, (is_v ? c.v_scales : c.k_scales)[row * (D / 32) + d0 / 32]));
#pragma unroll
        for (int j = 0; j < 4; j++) y[j] = static_cast<float>(static_cast<int8_t>(w >> (8 * j))) * d;
    }
    store4(out + (tok * Hkv + h) * D + d0, y);
}

// The row stride of an input of `heads` head rows per token.
bool stride_ok(int64_t stride, int64_t heads, int64_t D, int32_t dtype) {
    return stride >= heads * D && (stride * dtype_size(dtype)) % 16 == 0 && stride <= (INT64_C(1) << 40);
}

}  // namespace

namespace gd {

int check_kv_q8(const gd_kv_q8 *c, const char *name) {
    GD_REQUIRE(c, GD_EINVAL, "%s: null cache", name);
    GD_REQUIRE(c->k_codes && c->k_scales && c->v_codes && c->v_scales, GD_EINVAL, "%s: null cache plane", name);
    GD_REQUIRE(c->n_pages >= 1 && c->page_size >= 1 && c->n_kv_heads >= 1, GD_EINVAL,
               "%s: cache n_pages (%lld), page_size (%lld) and n_kv_heads (%lld) must be >= 1", name,
               (long long)c->n_pages, (long long)c->page_size, (long long)c->n_kv_heads);
    GD_REQUIRE(c->head_dim == 64 || c->head_dim == 128 || c->head_dim == 256, GD_ESHAPE,
               "%s: cache head_dim (%lld) must be 64, 128 or 256", name, (long long)c->head_dim);
    GD_REQUIRE(c->page_size % 16 == 0, GD_ESHAPE, "%s: cache page_size (%lld) must be a multiple of 16", name,
               (long long)c->page_size);
    int64_t t;
    GD_REQUIRE(c->n_pages <= INT64_C(2147483647) && c->n_kv_heads <= 4096 && c->page_size <= (INT64_C(1) << 30) &&
                   mul_ok(c->n_pages, c->page_size, &t) && mul_ok(t, c->n_kv_heads * c->head_dim, &t) &&
                   t <= (INT64_C(1) << 50),
               GD_ERANGE, "%s: cache too large", name);
    GD_REQUIRE(aligned(c->k_codes, 16) && aligned(c->k_scales, 16) && aligned(c->v_codes, 16) &&
                   aligned(c->v_scales, 16),
               GD_EALIGN, "%s: cache planes must be 16-byte aligned", name);
    return GD_OK;
}

}  // namespace gd

extern "C" int rope_table(float *table, int64_t n_pos, int64_t rot_dim, double base, const gd_rope_scaling *scaling,
                          void *stream) {
    GD_REQUIRE(table, GD_EINVAL, "rope_table: null pointer");
    GD_REQUIRE(n_pos >= 1 && rot_dim >= 1, GD_EINVAL, "rope_table: n_pos (%lld) and rot_dim (%lld) must be >= 1",
               (long long)n_pos, (long long)rot_dim);
    GD_REQUIRE(base > 1.0 && base <= 1e300, GD_EINVAL, "rope_table: base must be finite and above 1");
    GD_REQUIRE(rot_dim % 8 == 0, GD_ESHAPE, "rope_table: rot_dim (%lld) must be a multiple of 8", (long long)rot_dim);
    GD_REQUIRE(rot_dim <= kMaxRot && n_pos <= (INT64_C(1) << 31) - 1 &&
                   n_pos * (rot_dim / 2) <= kMaxThreads - kThreads,
               GD_ERANGE, "rope_table: n_pos or rot_dim (at most %d) too large", kMaxRot);
    GD_REQUIRE(aligned(table, 16), GD_EALIGN, "rope_table: table must be 16-byte aligned");
    const int kind = scaling ? scaling->kind : GD_ROPE_NONE;
    GD_REQUIRE(kind >= GD_ROPE_NONE && kind <= GD_ROPE_LLAMA3, GD_EINVAL, "rope_table: unknown scaling kind %d", kind);
    if (kind != GD_ROPE_NONE)
        GD_REQUIRE(scaling->factor >= 1.0 && scaling->factor <= 1e9, GD_EINVAL,
                   "rope_table: scaling factor must be in [1, 1e9]");
    if (kind == GD_ROPE_YARN || kind == GD_ROPE_LLAMA3) {
        GD_REQUIRE(scaling->original_len >= 1.0 && scaling->original_len <= 1e18, GD_EINVAL,
                   "rope_table: scaling original_len must be >= 1");
        GD_REQUIRE(scaling->low > 0.0 && scaling->high > scaling->low && scaling->high <= 1e18, GD_EINVAL,
                   "rope_table: scaling needs 0 < low < high");
        GD_REQUIRE(scaling->attention >= 0.0 && scaling->attention <= 1e9, GD_EINVAL,
                   "rope_table: scaling attention must be finite and >= 0");
    }
    const double two_pi = 6.283185307179586476925;
    const double rot = static_cast<double>(rot_dim);
    const int half = static_cast<int>(rot_dim / 2);
    RopeFreqs fr;
    fr.attention = 1.0;
    if (kind == GD_ROPE_NTK) base *= std::pow(scaling->factor, rot / (rot - 2.0));
    double ramp_lo = 0.0, ramp_hi = 1.0;
    if (kind == GD_ROPE_YARN) {   // the pairs that turn `high` and `low` times over the original length
        const auto pair_of = [&](double turns) {
            return rot * std::log(scaling->original_len / (turns * two_pi)) / (2.0 * std::log(base));
        };
        ramp_lo = std::fmax(std::floor(pair_of(scaling->high)), 0.0);
        ramp_hi = std::fmin(std::ceil(pair_of(scaling->low)), rot - 1.0);
        if (ramp_hi <= ramp_lo) ramp_hi = ramp_lo + 0.001;
        fr.attention = scaling->attention > 0.0 ? scaling->attention : 0.1 * std::log(scaling->factor) + 1.0;
    }
    for (int i = 0; i < half; i++) {
        double f = std::pow(base, -2.0 * i / rot);
        if (kind == GD_ROPE_LINEAR) {
            f /= scaling->factor;
        } else if (kind == GD_ROPE_YARN) {
            const double t = std::fmin(std::fmax((i - ramp_lo) / (ramp_hi - ramp_lo), 0.0), 1.0);
            f = f / scaling->factor * t + f * (1.0 - t);
        } else if (kind == GD_ROPE_LLAMA3) {
            const double turns = scaling->original_len * f / two_pi;   // over the original length
            const double t = std::fmin(std::fmax((turns - scaling->low) / (scaling->high - scaling->low), 0.0), 1.0);
            f = f / scaling->factor * (1.0 - t) + f * t;
        }
        fr.f[i] = f;
    }
    for (int i = half; i < kMaxRot / 2; i++) fr.f[i] = 0.0;
    const int64_t n = n_pos * half;
    hipLaunchKernelGGL(rope_table_kernel, dim3(static_cast<uint32_t>((n + kThreads - 1) / kThreads)), dim3(kThreads), 0,
                       as_stream(stream), reinterpret_cast<f32x2 *>(table), fr, half, n);
    return check_launch("rope_table");
}

extern "C" int kv_q8_store(const gd_kv_q8 *cache, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                           const void *v, int64_t v_stride, void *q_out, const float *rope, int64_t n_pos,
                           int64_t rot_dim, int32_t interleaved, const int32_t *positions, const int64_t *slots,
                           int64_t n_tok, int64_t n_heads, int32_t dtype, void *stream) {
    int st = check_kv_q8(cache, "kv_q8_store");
    if (st) return st;
    const int64_t D = cache->head_dim, Hkv = cache->n_kv_heads;
    GD_REQUIRE(k && v && slots, GD_EINVAL, "kv_q8_store: null pointer");
    GD_REQUIRE(n_tok >= 1 && n_heads >= 0, GD_EINVAL, "kv_q8_store: n_tok (%lld) must be >= 1, n_heads (%lld) >= 0",
               (long long)n_tok, (long long)n_heads);
    GD_REQUIRE(dtype_ok(dtype), GD_EINVAL, "kv_q8_store: unknown dtype %d", dtype);
    GD_REQUIRE(n_heads == 0 || (q && q_out), GD_EINVAL, "kv_q8_store: null q or q_out with n_heads %lld",
               (long long)n_heads);
    GD_REQUIRE((rope == nullptr) == (positions == nullptr), GD_EINVAL,
               "kv_q8_store: rope and positions are given together or not at all");
    if (rope) {
        GD_REQUIRE(n_pos >= 1 && rot_dim >= 1, GD_EINVAL, "kv_q8_store: n_pos (%lld) and rot_dim (%lld) must be >= 1",
                   (long long)n_pos, (long long)rot_dim);
        GD_REQUIRE(rot_dim % 8 == 0 && rot_dim <= D, GD_ESHAPE,
                   "kv_q8_store: rot_dim (%lld) must be a multiple of 8 and at most head_dim (%lld)",
                   (long long)rot_dim, (long long)D);
        GD_REQUIRE(n_pos <= (INT64_C(1) << 31), GD_ERANGE, "kv_q8_store: n_pos (%lld) too large", (long long)n_pos);
        GD_REQUIRE(aligned(rope, 16) && aligned(positions, 4), GD_EALIGN,
                   "kv_q8_store: rope must be 16-byte aligned, positions 4-byte");
    }
    GD_REQUIRE((n_heads == 0 || stride_ok(q_stride, n_heads, D, dtype)) && stride_ok(k_stride, Hkv, D, dtype) &&
                   stride_ok(v_stride, Hkv, D, dtype),
               GD_ESHAPE, "kv_q8_store: a row stride must cover the token's heads and be a multiple of 16 bytes");
    int64_t threads;
    GD_REQUIRE(n_heads <= 65536 && mul_ok(n_tok, (n_heads + 2 * Hkv) * (D / 4), &threads) &&
                   threads <= kMaxThreads - kThreads,
               GD_ERANGE, "kv_q8_store: n_tok * heads too large");
    GD_REQUIRE(aligned(k, 16) && aligned(v, 16) && (n_heads == 0 || (aligned(q, 16) && aligned(q_out, 16))) &&
                   aligned(slots, 8),
               GD_EALIGN, "kv_q8_store: q, k, v and q_out must be 16-byte aligned, slots 8-byte");
    StoreArgs a;
    a.q = q, a.k = k, a.v = v, a.q_out = q_out;
    a.rope = reinterpret_cast<const f32x2 *>(rope);
    a.positions = positions, a.slots = slots;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.n_pos = n_pos, a.n_tok = n_tok;
    a.n_heads = static_cast<int32_t>(n_heads), a.rot = static_cast<int32_t>(rot_dim), a.interleaved = interleaved != 0;
    a.c = *cache;
    const dim3 grid(static_cast<uint32_t>((threads + kThreads - 1) / kThreads));
    dispatch_dtype(dtype, [&](auto t) {
        hipLaunchKernelGGL((kv_q8_store_kernel<decltype(t)>), grid, dim3(kThreads), 0, as_stream(stream), a);
    });
    return check_launch("kv_q8_store");
}

extern "C" int kv_q8_load(const gd_kv_q8 *cache, const int64_t *slots, void *k_out, void *v_out, int64_t n_tok,
                          int32_t dtype, void *stream) {
    int st = check_kv_q8(cache, "kv_q8_load");
    if (st) return st;
    GD_REQUIRE(slots && (k_out || v_out), GD_EINVAL, "kv_q8_load: null pointer");
    GD_REQUIRE(n_tok >= 1, GD_EINVAL, "kv_q8_load: n_tok (%lld) must be >= 1", (long long)n_tok);
    GD_REQUIRE(dtype_ok(dtype), GD_EINVAL, "kv_q8_load: unknown dtype %d", dtype);
    int64_t threads;
    GD_REQUIRE(mul_ok(n_tok, 2 * cache->n_kv_heads * (cache->head_dim / 4), &threads) &&
                   threads <= kMaxThreads - kThreads,
               GD_ERANGE, "kv_q8_load: n_tok (%lld) too large", (long long)n_tok);
    GD_REQUIRE(aligned(slots, 8) && aligned(k_out, 16) && aligned(v_out, 16), GD_EALIGN,
               "kv_q8_load: outputs must be 16-byte aligned, slots 8-byte");
    const dim3 grid(static_cast<uint32_t>((threads + kThreads - 1) / kThreads));
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        hipLaunchKernelGGL((kv_q8_load_kernel<T>), grid, dim3(kThreads), 0, as_stream(stream), *cache, slots,
                           static_cast<T *>(k_out), static_cast<T *>(v_out), n_tok);
    });
    return check_launch("kv_q8_load");
}
