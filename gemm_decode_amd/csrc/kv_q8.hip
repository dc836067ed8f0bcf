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
#include <type_traits>

#include "gd_internal.h"
#include "gd_quant.h"
#include "gd_types.h"

namespace {

using namespace gd;

constexpr int kThreads = 256;
constexpr int64_t kMaxThreads = (INT64_C(1) << 32) - 1;   // of one launch
constexpr int kMaxRot = 256;
constexpr int64_t kMaxStride = INT64_C(1) << 36;   // elements between tokens
// From here on a workgroup per token (store) or four tokens (load) fills the card: 8191
// tokens stored and read back in 57 us, 86 with a workgroup per 16 rows of a token, and
// 65521 read in 138 us, 160 one by one; fewer tokens are spread as far as they go (one
// token stored and read back in 5.5 us, a microsecond more by one workgroup).
constexpr int64_t kManyTokens = 1024;

// ------------------------------------------------------- rotary table
struct RopeFreqs {
    double f[kMaxRot / 2];
    double attention;
};

// (cos, sin) of position * freq, in f64 (the angles of far positions lose
// their low bits in f32), rounded once. Run once per model. 131072 positions of 64 pairs:
// 31 us (a copy writes as much in 14), of which the vector instructions, 119 a wave and
// most of them f64's sincos at 4 cycles each, take 25.
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
    int64_t q_stride, k_stride, v_stride, n_pos;
    int32_t n_heads, rot, interleaved, page_shift;
    gd_kv_q8 c;
};

// Where a slot lies. A division of 64-bit numbers is some hundred scalar
// instructions, as many as the rest of a workgroup's start: pages of a power of two
// (shift >= 0), the usual ones, do without.
struct Slot {
    int64_t page, off;
    __device__ __forceinline__ Slot(int64_t slot, int64_t page_size, int shift) {
        page = shift >= 0 ? slot >> shift : slot / page_size;
        off = slot - page * page_size;
    }
};

int page_shift_of(int64_t page_size) {
    return (page_size & (page_size - 1)) == 0 ? __builtin_ctzll(static_cast<uint64_t>(page_size)) : -1;
}

// E consecutive elements, in one load of 4 E or 2 E bytes; and as f32.
template <typename T, int E>
struct Elements {
    typedef T type __attribute__((ext_vector_type(E)));
};

template <int E, typename T>
__device__ __forceinline__ void widen(typename Elements<T, E>::type v, f32x4 (&x)[E / 4]) {
#pragma unroll
    for (int i = 0; i < E; i++) x[i / 4][i % 4] = static_cast<float>(v[i]);
}

// Written past the caches: what is written here is read by a later launch (a long
// read back 145 -> 138 us).
template <int E, typename T>
__device__ __forceinline__ void store_n(T *p, const f32x4 (&x)[E / 4]) {
    typedef T Vec __attribute__((ext_vector_type(E)));
    Vec v;
#pragma unroll
    for (int i = 0; i < E; i++) v[i] = static_cast<T>(x[i / 4][i % 4]);
    __builtin_nontemporal_store(v, reinterpret_cast<Vec *>(p));
}

// a c - b s. Queries: the second product rounded to f32, the first one fused with the sum, so
// off by half an f32 step of the larger product before the last rounding (f32 queries 3.1e-8
// off on the average, 2.6e-8 as the keys are turned; nothing decides by their last bit, and a
// 16-bit result's own rounding is 2^13 times larger). As the keys are turned, 8191 tokens of
// bf16 take 46 us instead of 44 and 4096 of f16 at head dim 64 14.4 instead of 13.7.
// Keys (kExact): rounded to f32 from about twice its bits, since a code next to a half
// must not change sides: the two products' errors (exact, by fma) and their sum's
// (exact, by the usual six operations) are added up before the last rounding. In f64,
// where both products are exact, the same took a third of a long store's time.
template <bool kExact>
__device__ __forceinline__ float turn1(float a, float b, float c, float s) {
    const float q = b * s;
    if constexpr (!kExact) return __builtin_fmaf(a, c, -q);
    const float p = a * c;
    const float low = __builtin_fmaf(a, c, -p) - __builtin_fmaf(b, s, -q);
    const float h = p - q, t = h - p;
    const float err = (p - (h - t)) - (q + t);
    return h + (err + low);
}

// E dims of a head row turned by the token's angles: x are these dims, o their
// partners (half layout), c and s the angles of x's pairs (E of them, or E/2).
template <bool kExact, int E>
__device__ __forceinline__ void turn(f32x4 (&x)[E / 4], const f32x4 (&o)[E / 4], const float (&c)[E], const float (&s)[E],
                                     bool first, bool interleaved) {
    if (interleaved) {   // pairs (2i, 2i + 1), both in x
#pragma unroll
        for (int i = 0; i < E / 2; i++) {
            const float a = x[i / 2][2 * (i % 2)], b = x[i / 2][2 * (i % 2) + 1];
            x[i / 2][2 * (i % 2)] = turn1<kExact>(a, b, c[i], s[i]);
            x[i / 2][2 * (i % 2) + 1] = turn1<kExact>(b, a, c[i], -s[i]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < E; j++)
            x[j / 4][j % 4] = turn1<kExact>(x[j / 4][j % 4], o[j / 4][j % 4], c[j], first ? s[j] : -s[j]);
    }
}

// A workgroup serves one token (or its rows blockIdx.y, blockIdx.y + gridDim.y, ...
// of kRows at a time): D/E threads per head row, E dims each, so that a thread has the
// same dims in every row it takes and its angles are loaded once. Rows in the order q
// heads, k heads, v heads; a batch of them is loaded while the one before it is turned and
// quantized, the first while the token's slot, position and angles are looked up. A row
// never leaves its wave and the batches differ in their rows, so q_out may be q itself.
// 8191 tokens of 32 / 8 heads of 128 in bf16: 42 us, 4.4 TB/s (35 with the inputs still in
// the last cache), near memory's rate with the quantizer's arithmetic beside it (36 with
// loads behind the look-up and between the batches, 37 with batches of two rows, 53 at 80
// registers; of f32, four elements a thread, 2000 tokens 17.4 us with one row, 16.7 with
// two); one token: 2.7 us, bound by its chain of loads.
template <typename T, int D, int E>
__global__ __launch_bounds__(kThreads) void kv_q8_store_kernel(StoreArgs a) {
    constexpr int kLanes = D / E, kRows = kThreads / kLanes, kBatch = E == 4 ? 2 : 1;
    const int64_t tok = blockIdx.x;
    const int Hkv = static_cast<int>(a.c.n_kv_heads), Hq = a.n_heads;
    const int d0 = static_cast<int>(threadIdx.x % kLanes) * E;
    const bool turned = a.rope && d0 < a.rot;
    const int half = a.rot / 2;
    const bool first = d0 < half;
    const int partner = turned && !a.interleaved ? (first ? half : -half) : 0;   // where a dim's partner lies
    const T *q = static_cast<const T *>(a.q) + tok * a.q_stride + d0;
    const T *k = static_cast<const T *>(a.k) + tok * a.k_stride + d0;
    const T *v = static_cast<const T *>(a.v) + tok * a.v_stride + d0;
    typedef typename Elements<T, E>::type Vec;
    Vec x_in[kBatch] = {}, o_in[kBatch] = {};
    const int step = kRows * static_cast<int>(gridDim.y);
    const auto load = [&](int r0) {
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int r = r0 + i * step;
            if (r >= Hq + 2 * Hkv) break;
            const T *p = r < Hq ? q + r * D : r < Hq + Hkv ? k + (r - Hq) * D : v + (r - Hq - Hkv) * D;
            x_in[i] = *reinterpret_cast<const Vec *>(p);
            if (partner != 0 && r < Hq + Hkv) o_in[i] = *reinterpret_cast<const Vec *>(p + partner);
        }
    };
    int r0 = kRows * static_cast<int>(blockIdx.y) + static_cast<int>(threadIdx.x) / kLanes;
    load(r0);   // on its way while the slot, the position and its angles are looked up
    __builtin_amdgcn_sched_barrier(0);
    const int64_t slot = a.slots[tok];
    const bool live = slot >= 0 && slot < a.c.n_pages * a.c.page_size;
    float c[E] = {}, s[E] = {};
    if (a.rope) {
        const int64_t pos = a.positions[tok];
        if (pos < 0 || pos >= a.n_pos) return;   // no angles for it: the token is left out
        if (turned) {
            const f32x4 *t = reinterpret_cast<const f32x4 *>(
                a.rope + pos * half + (a.interleaved ? d0 / 2 : first ? d0 : d0 - half));
#pragma unroll
            for (int i = 0; i < E; i += 2) {
                if (i >= E / 2 && a.interleaved) break;
                const f32x4 v = t[i / 2];
                c[i] = v[0], s[i] = v[1], c[i + 1] = v[2], s[i + 1] = v[3];
            }
        }
    }
    T *qo = static_cast<T *>(a.q_out) + tok * Hq * D + d0;
    const Slot at(live ? slot : 0, a.c.page_size, a.page_shift);
    const int rows = Hq + (live ? 2 * Hkv : 0);
    for (int next; r0 < rows; r0 = next) {
        f32x4 x[kBatch][E / 4], o[kBatch][E / 4];
#pragma unroll
        for (int i = 0; i < kBatch; i++) widen<E, T>(x_in[i], x[i]), widen<E, T>(o_in[i], o[i]);
        next = r0 + kBatch * step;
        load(next);
#pragma unroll
        for (int i = 0; i < kBatch; i++) {
            const int r = r0 + i * step;
            if (r >= rows) break;
            if (r < Hq) {
                if (turned) turn<false, E>(x[i], o[i], c, s, first, a.interleaved);
                store_n<E>(qo + r * D, x[i]);
                continue;
            }
            const bool is_v = r >= Hq + Hkv;
            const int h = is_v ? r - Hq - Hkv : r - Hq;
            if (turned && !is_v) turn<true, E>(x[i], o[i], c, s, first, a.interleaved);
            float m = 0.0f;   // the largest of the 32 dims that the lane's are among: 32 / E lanes
#pragma unroll
            for (int w = 0; w < E / 4; w++) m = fmaxf(m, absmax4(float4{x[i][w][0], x[i][w][1], x[i][w][2], x[i][w][3]}));
            m = E == 4 ? max8(m) : max4(m);
            uint32_t packed[E / 4] = {};
            _Float16 d = 0;
            if (m > 0.0f) {
                const float inv32 = recip127(m);
                const bool f64_only = !(inv32 <= 3.40282347e38f);   // the reciprocal overflowed
#pragma unroll
                for (int w = 0; w < E / 4; w++)
                    packed[w] = codes4(float4{x[i][w][0], x[i][w][1], x[i][w][2], x[i][w][3]}, inv32, m, f64_only);
                d = static_cast<_Float16>(scale_of(m));
            }
            const int64_t row = (at.page * Hkv + h) * a.c.page_size + at.off;
            uint32_t *codes = reinterpret_cast<uint32_t *>((is_v ? a.c.v_codes : a.c.k_codes) + row * D + d0);
            if constexpr (E == 4)
                codes[0] = packed[0];
            else
                *reinterpret_cast<uint2 *>(codes) = uint2{packed[0], packed[E / 4 - 1]};
            if (d0 % 32 == 0)
                (is_v ? a.c.v_scales : a.c.k_scales)[row * (D / 32) + d0 / 32] = __builtin_bit_cast(uint16_t, d);
        }
    }
}

// ---------------------------------------------------------------- load
// A workgroup serves kTok tokens, D/E threads per head row, E = 16 / sizeof(T) dims
// each (16-byte stores, and the outputs are most of the traffic): the keys' rows
// first, then the values'; the loads of its tokens are all issued before any is used.
// 65521 tokens of 8 heads of 128 to f32: 138 us, 4.9 TB/s, what a copy reaches.
template <typename T, int D, int kTok>
__global__ __launch_bounds__(kThreads) void kv_q8_load_kernel(gd_kv_q8 c, const int64_t *__restrict__ slots,
                                                              T *__restrict__ k_out, T *__restrict__ v_out,
                                                              int64_t n_tok, int page_shift) {
    constexpr int E = 16 / sizeof(T), kLanes = D / E, kRows = kThreads / kLanes;
    typedef int8_t Codes __attribute__((ext_vector_type(E)));
    const int64_t tok0 = static_cast<int64_t>(blockIdx.x) * kTok;
    const int Hkv = static_cast<int>(c.n_kv_heads);
    const int d0 = static_cast<int>(threadIdx.x % kLanes) * E;
    int64_t at[kTok];   // row of KV head 0; -1: none
#pragma unroll
    for (int i = 0; i < kTok; i++) {
        const int64_t slot = tok0 + i < n_tok ? slots[tok0 + i] : -1;
        const bool live = slot >= 0 && slot < c.n_pages * c.page_size;
        const Slot s(live ? slot : 0, c.page_size, page_shift);
        at[i] = live ? s.page * Hkv * c.page_size + s.off : -1;
    }
    for (int r = threadIdx.x / kLanes; r < 2 * Hkv; r += kRows) {
        const bool is_v = r >= Hkv;
        const int h = is_v ? r - Hkv : r;
        T *out = is_v ? v_out : k_out;
        if (!out) continue;
        const int8_t *codes = is_v ? c.v_codes : c.k_codes;
        const uint16_t *scales = is_v ? c.v_scales : c.k_scales;
        Codes w[kTok];
        uint16_t d[kTok];
#pragma unroll
        for (int i = 0; i < kTok; i++) {
            const int64_t row = (at[i] < 0 ? 0 : at[i]) + h * c.page_size;   // row 0 of none: loaded, not used
            w[i] = *reinterpret_cast<const Codes *>(codes + row * D + d0);
            d[i] = scales[row * (D / 32) + d0 / 32];
        }
#pragma unroll
        for (int i = 0; i < kTok; i++) {
            if (tok0 + i >= n_tok) break;
            const float f = static_cast<float>(__builtin_bit_cast(_Float16, d[i]));
            f32x4 y[E / 4];
#pragma unroll
            for (int j = 0; j < E; j++) y[j / 4][j % 4] = at[i] < 0 ? 0.0f : static_cast<float>(w[i][j]) * f;
            store_n<E>(out + ((tok0 + i) * Hkv + h) * D + d0, y);
        }
    }
}

// Calls fn with the head dim as a constant.
template <typename F>
void dispatch_dim(int64_t head_dim, F fn) {
    if (head_dim == 64)
        fn(std::integral_constant<int, 64>{});
    else if (head_dim == 128)
        fn(std::integral_constant<int, 128>{});
    else
        fn(std::integral_constant<int, 256>{});
}

// The row stride of an input of `heads` head rows per token.
bool stride_ok(int64_t stride, int64_t heads, int64_t D, int32_t dtype) {
    return stride >= heads * D && stride % (16 / dtype_size(dtype)) == 0;
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
    GD_REQUIRE(n_heads <= 65536 && n_tok <= kMaxThreads / kThreads, GD_ERANGE,
               "kv_q8_store: n_tok (%lld) or n_heads (%lld) too large", (long long)n_tok, (long long)n_heads);
    GD_REQUIRE(q_stride <= kMaxStride && k_stride <= kMaxStride && v_stride <= kMaxStride, GD_ERANGE,
               "kv_q8_store: a row stride is too large");
    GD_REQUIRE((n_heads == 0 || stride_ok(q_stride, n_heads, D, dtype)) && stride_ok(k_stride, Hkv, D, dtype) &&
                   stride_ok(v_stride, Hkv, D, dtype),
               GD_ESHAPE, "kv_q8_store: a row stride must cover the token's heads and be a multiple of 16 bytes");
    GD_REQUIRE(n_heads == 0 || q_out != q || n_tok == 1 || q_stride == n_heads * D, GD_EINVAL,
               "kv_q8_store: q_out may be q only if q_stride is n_heads * head_dim");
    GD_REQUIRE(aligned(k, 16) && aligned(v, 16) && (n_heads == 0 || (aligned(q, 16) && aligned(q_out, 16))) &&
                   aligned(slots, 8),
               GD_EALIGN, "kv_q8_store: q, k, v and q_out must be 16-byte aligned, slots 8-byte");
    if (n_heads > 0) {
        const int64_t size = dtype_size(dtype), out_bytes = n_tok * n_heads * D * size;
        GD_REQUIRE(q_out == q || !overlaps(q, q_stride * size, n_heads * D * size, n_tok, q_out, out_bytes), GD_EINVAL,
                   "kv_q8_store: q_out may be q itself, but not overlap it otherwise");
        GD_REQUIRE(!overlaps(k, k_stride * size, Hkv * D * size, n_tok, q_out, out_bytes) &&
                       !overlaps(v, v_stride * size, Hkv * D * size, n_tok, q_out, out_bytes),
                   GD_EINVAL, "kv_q8_store: q_out must not overlap k or v");
    }
    StoreArgs a;
    a.q = q, a.k = k, a.v = v, a.q_out = q_out;
    a.rope = reinterpret_cast<const f32x2 *>(rope);
    a.positions = positions, a.slots = slots;
    a.q_stride = q_stride, a.k_stride = k_stride, a.v_stride = v_stride, a.n_pos = n_pos;
    a.n_heads = static_cast<int32_t>(n_heads), a.rot = static_cast<int32_t>(rot_dim), a.interleaved = interleaved != 0;
    a.page_shift = page_shift_of(cache->page_size);
    a.c = *cache;
    // 16-byte loads, unless a pair's halves would not start on one (16-bit types, rot_dim not a multiple of 16).
    const bool wide = dtype != GD_F32 && (!rope || rot_dim % 16 == 0);
    const int64_t at_once = kThreads / (D / (wide ? 8 : 4));
    // few tokens: their rows over as many workgroups as they fill
    const int64_t chunks = n_tok >= kManyTokens ? 1 : (n_heads + 2 * Hkv + at_once - 1) / at_once;
    const dim3 grid(static_cast<uint32_t>(n_tok), static_cast<uint32_t>(chunks));
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        dispatch_dim(D, [&](auto dim) {
            constexpr int kD = decltype(dim)::value;
            if constexpr (sizeof(T) == 2) {
                if (wide) {
                    hipLaunchKernelGGL((kv_q8_store_kernel<T, kD, 8>), grid, dim3(kThreads), 0, as_stream(stream), a);
                    return;
                }
            }
            hipLaunchKernelGGL((kv_q8_store_kernel<T, kD, 4>), grid, dim3(kThreads), 0, as_stream(stream), a);
        });
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
    GD_REQUIRE(n_tok <= kMaxThreads / kThreads, GD_ERANGE, "kv_q8_load: n_tok (%lld) too large", (long long)n_tok);
    GD_REQUIRE(aligned(slots, 8) && aligned(k_out, 16) && aligned(v_out, 16), GD_EALIGN,
               "kv_q8_load: outputs must be 16-byte aligned, slots 8-byte");
    const bool many = n_tok >= kManyTokens;
    const int shift = page_shift_of(cache->page_size);
    const dim3 grid(static_cast<uint32_t>(many ? (n_tok + 3) / 4 : n_tok));
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        T *ko = static_cast<T *>(k_out), *vo = static_cast<T *>(v_out);
        dispatch_dim(cache->head_dim, [&](auto dim) {
            constexpr int kD = decltype(dim)::value;
            if (many)
                hipLaunchKernelGGL((kv_q8_load_kernel<T, kD, 4>), grid, dim3(kThreads), 0, as_stream(stream), *cache,
                                   slots, ko, vo, n_tok, shift);
            else
                hipLaunchKernelGGL((kv_q8_load_kernel<T, kD, 1>), grid, dim3(kThreads), 0, as_stream(stream), *cache,
                                   slots, ko, vo, n_tok, shift);
        });
    });
    return check_launch("kv_q8_load");
}
