// q1_linear.hip -- Q1_0 . q8_0 products with an epilogue: bias, activation, residual or the
// product with a second weight's sums, and the output in the stream's type or as q8_0 blocks.
//
//   v[c][r] = sum over blocks of 128 of d0 sum over sub-blocks of 32 of d1 sum (+-1) q
//
// on the matrix cores, every product exact. One launch up to four columns (a token) and, with a
// second one that joins slices of K, up to 16 (q1_few_kernel); for more the activations are laid
// out once as operands (q1_digits_kernel), and a batch's weights are taken by waves that share
// K (q1_split_kernel), a prompt's by waves side by side with all they read in LDS
// (q1_wide_kernel). All end in the same epilogue, of sums in f32.
#include <type_traits>

#include "gd_internal.h"
#include "gd_quant.h"
#include "gd_types.h"

namespace {

using namespace gd;

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));

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
    int32_t act, dtype;   // GD_ACT_, GD_F32 .. of residual and y
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

// Four codes, byte j that of v[j], among 32 values whose largest magnitude is a, by the rule
// of q8_0_quantize: in f32 where that gives what the f64 rule gives.
__device__ __forceinline__ uint32_t codes_of(f32x4 v, float a) {
    if (!(a > 0.0f)) return 0;
    const float inv = recip127(a);
    bool doubt = !(inv <= 3.40282347e38f);
    int32_t q[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
        const float t = v[j] * inv;
        q[j] = static_cast<int32_t>(floorf(t + 0.5f));
        doubt |= fabsf(__builtin_amdgcn_fractf(t) - 0.5f) < kTieGuard;
    }
    if (doubt) {   // rare
        const double factor = 127.0 / static_cast<double>(a);
#pragma unroll
        for (int j = 0; j < 4; j++) q[j] = round_code(static_cast<double>(v[j]) * factor);
    }
    uint32_t packed = 0;
#pragma unroll
    for (int j = 0; j < 4; j++) packed |= (static_cast<uint32_t>(q[j]) & 0xffu) << (8 * j);
    return packed;
}

// Four elements at p (aligned to one), `count` of them there.
template <typename T>
__device__ __forceinline__ f32x4 load_some(const T *p, int count) {
    typedef T Vec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    if (count >= 4) return __builtin_convertvector(*reinterpret_cast<const Vec *>(p), f32x4);
    f32x4 v = {};
#pragma unroll
    for (int j = 0; j < 3; j++)
        if (j < count) v[j] = static_cast<float>(p[j]);
    return v;
}
template <typename T>
__device__ __forceinline__ void store_some(T *p, f32x4 v, int count) {
    typedef T Vec __attribute__((ext_vector_type(4), aligned(sizeof(T))));
    if (count >= 4) {
        *reinterpret_cast<Vec *>(p) = __builtin_convertvector(v, Vec);
        return;
    }
#pragma unroll
    for (int j = 0; j < 3; j++)
        if (j < count) p[j] = static_cast<T>(v[j]);
}

// What becomes of the sums v (and u, the second weight's) of rows r .. r + 3, r % 4 = 0, and
// column c. Where q8_0 blocks are written, eight neighbouring lanes hold the 32 rows of one
// (r / 4 % 8 = lane % 8) and all of them call this.
template <int S>
__device__ __forceinline__ void finish(const Weight &w0, const Weight &w1, const Epilogue &e, f32x4 v, f32x4 u, int64_t c, int64_t r) {
    const int64_t rest = c < e.n ? e.rows - r : 0;
    const int count = rest >= 4 ? 4 : rest > 0 ? static_cast<int>(rest) : 0;
    if (w0.bias) v += load_some(w0.bias + r, count);
    if (S == 2 && w1.bias) u += load_some(w1.bias + r, count);
#pragma unroll
    for (int j = 0; j < 4; j++) v[j] = activate(v[j], e.act);
    if (S == 2) v *= u;
    const int64_t at = c * e.rows + r;
    const auto outer = [&](auto one) {
        using T = decltype(one);
        if (e.residual) v += load_some(static_cast<const T *>(e.residual) + at, count);
        if (e.y) store_some(static_cast<T *>(e.y) + at, v, count);
    };
    if (e.dtype == GD_F32)
        outer(float{});
    else if (e.dtype == GD_F16)
        outer(_Float16{});
    else
        outer(__bf16{});
    if (e.y_q8) {
        const float a = max8(absmax4(float4{v[0], v[1], v[2], v[3]}));
        const uint32_t q = codes_of(v, a);
        if (count) {
            uint16_t *o = e.y_q8 + at / 32 * 17;   // 34 bytes = 17 halves
            const int k8 = static_cast<int>(r / 4 % 8);
            typedef uint32_t Word __attribute__((aligned(2)));
            *reinterpret_cast<Word *>(o + 1 + 2 * k8) = q;
            if (k8 == 0) o[0] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(a > 0.0f ? scale_of(a) : 0.0f));
        }
    }
}

// One value: the outer operands of row r and column c, asked for before the sums are there,
struct Outer {
    float bias[2], residual;
};
template <int S>
__device__ __forceinline__ Outer load_outer(const Weight &w0, const Weight &w1, const Epilogue &e, int64_t c, int64_t r, bool live) {
    Outer o = {{0.0f, 0.0f}, 0.0f};
    if (live) {
        if (w0.bias) o.bias[0] = w0.bias[r];
        if (S == 2 && w1.bias) o.bias[1] = w1.bias[r];
        if (e.residual) {
            const int64_t at = c * e.rows + r;
            o.residual = e.dtype == GD_F32 ? static_cast<const float *>(e.residual)[at]
                                           : e.dtype == GD_F16 ? static_cast<float>(static_cast<const _Float16 *>(e.residual)[at])
                                                               : static_cast<float>(static_cast<const __bf16 *>(e.residual)[at]);
        }
    }
    return o;
}
// and what becomes of it. Where q8_0 blocks are written, 32 lanes hold the rows of one
// (r % 32 = lane % 32) and all of them call this.
template <int S>
__device__ __forceinline__ void finish_one(const Epilogue &e, const Outer &o, float v, float u, int64_t c, int64_t r, bool live) {
    v = activate(v + o.bias[0], e.act);
    if (S == 2) v *= u + o.bias[1];
    v += o.residual;
    const int64_t at = c * e.rows + r;
    if (e.y && live) {
        if (e.dtype == GD_F32)
            static_cast<float *>(e.y)[at] = v;
        else if (e.dtype == GD_F16)
            static_cast<_Float16 *>(e.y)[at] = static_cast<_Float16>(v);
        else
            static_cast<__bf16 *>(e.y)[at] = static_cast<__bf16>(v);
    }
    if (e.y_q8) {
        float a = max8(fabsf(v));
        a = fmaxf(a, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, a), 0x140, 0xF, 0xF, false)));
        a = fmaxf(a, __shfl_xor(a, 16));
        const uint32_t q = codes_of(f32x4{v, 0.0f, 0.0f, 0.0f}, a);
        if (live) {
            uint16_t *b = e.y_q8 + at / 32 * 17;   // 34 bytes = 17 halves
            reinterpret_cast<uint8_t *>(b + 1)[r % 32] = static_cast<uint8_t>(q);
            if (r % 32 == 0) b[0] = __builtin_bit_cast(uint16_t, static_cast<_Float16>(a > 0.0f ? scale_of(a) : 0.0f));
        }
    }
}

// ------------------------------------------------------------- operands
// The matrix instructions take 6-bit floats (e2m3) for the activations and 4-bit ones
// (e2m1) for the weights, 32 of a lane with a power of two for all of them. A weight is its
// sign, +1 or -1. An activation d1 q, d1 = m 2^e an f16 value with |m| < 2^11, is the whole
// number m q, |m q| < 2^18, times 2^e: four digits to the base 32, each in [-16, 16], which
// e2m3 holds exactly (as that many eighths, and the code of n eighths is n for n <= 16).
// So four instructions multiply exactly, and their sums round in f32 alone; d0 is
// multiplied to the sum over a weight block's 128 elements.
//
// The 32 elements of a sub-block stand in the order that the plane words give up with the
// fewest steps: place 8 j + 2 jj + h holds element 16 h + 4 jj + j.
constexpr uint32_t kBias = 0x84210u;   // 16 in each digit: keeps m q + bias positive
constexpr int kFp6 = 2, kFp4 = 4;      // operand formats
constexpr int kOne = 0x7f7f7f7f;       // scales of 1

// Byte p: the e2m3 code of digit p of q m.
__device__ __forceinline__ uint32_t digit_codes(int32_t q, int32_t m) {
    const uint32_t u = static_cast<uint32_t>(__mul24(q, m)) + kBias;   // digits + 16, five bits each
    uint32_t t = (u & 0x3ffu) | (u << 6 & ~0x3ffu);
    t = ((t & 0x001f001fu) | (t << 3 & ~0x001f001fu)) & 0x1f1f1f1fu;   // a byte each
    const uint32_t minus = ~t & 0x10101010u, one = minus >> 4;         // digits below 0
    return ((((t & 0x0f0f0f0fu) ^ (minus - one)) + one) | minus << 1);   // 16 - d there, d elsewhere; the sign bit
}

// Bits 6 k: byte k of x, six bits of it.
__device__ __forceinline__ uint32_t pack6(uint32_t x) {
    const uint32_t t = (x & 0x003f003fu) | (x >> 2 & ~0x003f003fu);
    return (t & 0xfffu) | (t >> 4 & 0xfff000u);
}

// Places 8 j .. 8 j + 7 of a sub-block's digits p: r[0][p] and r[1][p] hold four each, 24
// bits. d: the sub-block's codes as eight words.
__device__ __forceinline__ void digits8(const uint32_t *d, int j, int32_t m, uint32_t r[2][4]) {
#pragma unroll
    for (int a = 0; a < 2; a++) {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; i++) {
            const uint32_t word = d[2 * a + (i >> 1) + 4 * (i & 1)];
            w[i] = digit_codes(static_cast<int32_t>(word << (24 - 8 * j)) >> 24, m);
        }
        const uint32_t lo0 = __builtin_amdgcn_perm(w[1], w[0], 0x05010400u), lo1 = __builtin_amdgcn_perm(w[3], w[2], 0x05010400u);
        const uint32_t hi0 = __builtin_amdgcn_perm(w[1], w[0], 0x07030602u), hi1 = __builtin_amdgcn_perm(w[3], w[2], 0x07030602u);
        r[a][0] = pack6(__builtin_amdgcn_perm(lo1, lo0, 0x05040100u));
        r[a][1] = pack6(__builtin_amdgcn_perm(lo1, lo0, 0x07060302u));
        r[a][2] = pack6(__builtin_amdgcn_perm(hi1, hi0, 0x05040100u));
        r[a][3] = pack6(__builtin_amdgcn_perm(hi1, hi0, 0x07060302u));
    }
}

// m of an f16 scale d1 = m 2^(E - 25), and the powers of two of its four digits (biased, a
// byte each; NaN for an infinity or a NaN).
struct Scale {
    int32_t m;
    uint32_t powers;
    __device__ __forceinline__ explicit Scale(uint32_t h) {
        const uint32_t e = h >> 10 & 31u;
        m = static_cast<int32_t>((h & 0x3ffu) | (e ? 0x400u : 0u));
        if (h & 0x8000u) m = -m;
        powers = e == 31u ? 0xffffffffu : 0x0f0a0500u + (105u + (e ? e : 1u)) * 0x01010101u;
    }
};

// A q8_0 block's codes as words, and its scale (34 bytes, 2-byte aligned).
__device__ __forceinline__ uint32_t load_block(const uint16_t *b, uint32_t d[8]) {
    typedef uint32_t Words __attribute__((ext_vector_type(4), aligned(2)));
    const Words lo = *reinterpret_cast<const Words *>(b + 1), hi = *reinterpret_cast<const Words *>(b + 9);
#pragma unroll
    for (int i = 0; i < 4; i++) {
        d[i] = lo[i];
        d[4 + i] = hi[i];
    }
    return b[0];
}

// The 32 signs of a lane's sub-block as e2m1 codes, from its words of the two halves (which
// hold those of the neighbouring sub-block as well: odd says which of the two).
struct Signs {
    uint32_t lo, hi;   // rotations
    __device__ __forceinline__ explicit Signs(int odd) : lo(2 + 4 * odd), hi((30 + 4 * odd) & 31) {}
    __device__ __forceinline__ i32x8 operator()(uint32_t half0, uint32_t half1) const {
        const uint32_t a = __builtin_amdgcn_alignbit(half0, half0, lo), b = __builtin_amdgcn_alignbit(half1, half1, hi);
        const uint32_t y = (a & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);   // nibble 2 jj + h: the signs of j = 0..3
        i32x8 v = {};
#pragma unroll
        for (int j = 0; j < 4; j++) v[j] = static_cast<int>((~(y << (3 - j)) & 0x88888888u) | 0x22222222u);
        return v;
    }
};

__device__ __forceinline__ i32x8 frag(u32x4 lo, u32x2 hi) {
    return i32x8{static_cast<int>(lo[0]), static_cast<int>(lo[1]), static_cast<int>(lo[2]), static_cast<int>(lo[3]),
                 static_cast<int>(hi[0]), static_cast<int>(hi[1]), 0, 0};
}

// ------------------------------------------------- up to four columns
// For few columns the digits are those of the codes alone, q = 16 h + l with l in [0, 16) and h
// in [-8, 8), which takes a quarter of the work (5.6 vector instructions a code instead of 22),
// and d1 is multiplied to the sums. A 16 x 16 x 128 instruction takes a block of 16 weight rows;
// its other 16 rows are, for each of the four sub-blocks, l and h of two columns, or one of the
// two of four columns, zero outside that sub-block. So a lane's four results are the whole sums
// of one sub-block and one weight row, and acc += (d0 d1) (l + h) rounds once (d0 d1 has 22 bits).
//
// A workgroup of eight waves holds the digits of kBlocks blocks in LDS and takes 16-row tiles
// of the weights, kw waves sharing a tile by its K in quads of blocks. A wave's loads of its
// TILES tiles and Q quads all go out before the digits are worked out: the call is as long
// as a few memory latencies, and this hides the digits behind one. Beyond four columns K is cut
// into slices for workgroups of their own, and another launch joins their sums.
//
// What it takes, replayed from a graph (1.8 us of it the launch): one column 4.2 us at 4096 x
// 4096, 6.7 at 4096 x 14336 and, gated, 8.7 at 14336 x 4096 (16.5 MB of weights, 1.9 TB/s);
// four 6.2, 11.3 and 10.8; eight at 4096 x 4096 7.0; 13 at 4096 x 14336 15.4. The weights' bytes
// alone would take 0.3 to 2.4 us: it is the chain of launch, loads, digits, barrier, products
// and sums over waves that counts.
constexpr int kFew = 512;
template <int C>
constexpr int kBlocks = C < 4 ? 128 : 256 / C;   // digits of 49 KiB (a column 25)

struct FewShape {
    int64_t nb;   // blocks of a row
    int kw, kw_log;   // waves along K: 1, 2, 4 or 8
    int slices, share;   // of K, and the blocks of one
    int64_t row_tiles;   // tiles of 32 rows
    float *parts;        // sums of the slices, [slices][S][n][32 row_tiles]
};

// Half of a sub-block, its places 16 part .. 16 part + 15, as the three words each of l and h.
__device__ __forceinline__ void code_digits(const uint32_t d[8], int part, uint32_t l[3], uint32_t h[3]) {
    const uint32_t sel = part ? 0x07030602u : 0x05010400u;
    uint32_t rl[4], rh[4];
#pragma unroll
    for (int a = 0; a < 2; a++) {
        const uint32_t x = __builtin_amdgcn_perm(d[4 + 2 * a], d[2 * a], sel), y = __builtin_amdgcn_perm(d[5 + 2 * a], d[2 * a + 1], sel);
#pragma unroll
        for (int j = 0; j < 2; j++) {
            const uint32_t w = __builtin_amdgcn_perm(y, x, j ? 0x07060302u : 0x05040100u);   // four codes
            const uint32_t n = w >> 4 & 0x0f0f0f0fu, minus = n & 0x08080808u, one = minus >> 3;
            rl[2 * j + a] = pack6(w & 0x0f0f0f0fu);
            rh[2 * j + a] = pack6(((n ^ ((minus << 1) - one)) + one) | minus << 2);   // magnitude and sign
        }
    }
    const auto words = [](const uint32_t r[4], uint32_t w[3]) {
        w[0] = r[0] | r[1] << 24;
        w[1] = r[1] >> 8 | r[2] << 16;
        w[2] = r[2] >> 16 | r[3] << 8;
    };
    words(rl, l);
    words(rh, h);
}

// Sums of a's two halves in the lower half of a wave and of b's in the upper one, and likewise
// of neighbouring 16-lane rows: a's in even rows, b's in odd ones.
__device__ __forceinline__ float halves(float a, float b) {
    const auto p = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    return __builtin_bit_cast(float, static_cast<uint32_t>(p[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(p[1]));
}
__device__ __forceinline__ float rows16(float a, float b) {
    const auto p = __builtin_amdgcn_permlane16_swap(__builtin_bit_cast(uint32_t, a), __builtin_bit_cast(uint32_t, b), false, false);
    return __builtin_bit_cast(float, static_cast<uint32_t>(p[0])) + __builtin_bit_cast(float, static_cast<uint32_t>(p[1]));
}

// Sum over the four 16-lane rows of a wave, in all of them.
__device__ __forceinline__ float sum_rows(float v) {
    v = halves(v, v);
    return rows16(v, v);
}

template <int C, int S, int TILES, int Q>
__global__ __launch_bounds__(kFew, 2) void q1_few_kernel(Weight w0, Weight w1, const uint16_t *__restrict__ a_q8, Epilogue e,
                                                         FewShape f) {
    constexpr int N = TILES * S;   // a wave's tiles of both weights
    constexpr int kRow = 6;        // words of a row of digits
    constexpr int kShare = C < 4 ? 2 : 1;                                         // threads to a sub-block
    constexpr int kPer = kBlocks<C> * 4 * kShare, kItems = C * kPer / kFew;        // threads' items in a chunk's column, a thread's
    constexpr int kColumn = kBlocks<C> * 4 * 2 * kRow + 32, kZeros = C * kColumn;   // words of a column's digits, of all
    constexpr int M = (C + 3) / 4, kWords = kZeros + 8, kSums = 8 * N * 64 * M;
    constexpr bool kShared = C > 4;   // the sums where the digits were
    __shared__ __attribute__((aligned(16))) uint32_t digits[kShared && kSums > kWords ? kSums : kWords];   // and a row of zeros
    __shared__ __attribute__((aligned(16))) float d1[kBlocks<C> * 4 * C];
    __shared__ __attribute__((aligned(16))) float own[kShared ? 4 : kSums];
    float *red = kShared ? reinterpret_cast<float *>(digits) : own;
    const int tid = threadIdx.x, lane = tid % 64, wave = __builtin_amdgcn_readfirstlane(tid / 64);
    const int g = lane / 16, n16 = lane % 16, n = static_cast<int>(e.n), nb = static_cast<int>(f.nb), nb8 = (nb + 7) / 8;
    const int kpart = wave & (f.kw - 1), ipart = wave >> f.kw_log, groups_log = 3 - f.kw_log;
    const int tw = TILES << groups_log;   // the workgroup's tiles
    const uint32_t group = C > 4 ? blockIdx.x / static_cast<uint32_t>(f.slices) : blockIdx.x;
    const int slice = C > 4 ? static_cast<int>(blockIdx.x - group * static_cast<uint32_t>(f.slices)) : 0;
    const int first = C > 4 ? slice * f.share : 0, stop = C > 4 && first + f.share < nb ? first + f.share : nb;
    const int64_t tile0 = static_cast<int64_t>(group) * tw;
    // Where a column's digits start: so that the 16 rows that an instruction reads, four columns of
    // four neighbouring sub-blocks (12 words apart), lie in banks of their own.
    const auto column_at = [](int c) { return c * kColumn + (c & 1) * 2 + (c & 2) * 8; };
    float acc[N][C];
#pragma unroll
    for (int i = 0; i < N; i++)
#pragma unroll
        for (int c = 0; c < C; c++) acc[i][c] = 0.0f;
    Outer outer;
    for (int b0 = first; b0 < stop; b0 += kBlocks<C>) {
        const int blocks = stop - b0 < kBlocks<C> ? stop - b0 : kBlocks<C>;
        // The codes first (without a branch around the loads: behind one, the compiler waits for
        // all that is on its way),
        uint32_t d[kItems][8], scale[kItems];
        const auto column_of = [&](int k) { return kPer < kFew ? tid / kPer + k * (kFew / kPer) : k * kFew / kPer; };
        const auto item_of = [&](int k) { return kPer < kFew ? tid % kPer : tid + k * kFew % kPer; };
#pragma unroll
        for (int k = 0; k < kItems; k++) {
            const int c = column_of(k), i = item_of(k) < blocks * 4 * kShare ? item_of(k) : blocks * 4 * kShare - 1;
            scale[k] = load_block(a_q8 + (static_cast<int64_t>(c < n ? c : 0) * nb + b0) * 68 + i / kShare * 17, d[k]);
        }
        if (C <= 4 && b0 == 0) {   // then what the thread's sum meets,
            const int i = tid < n * 16 * tw ? tid : 0, c = i / (16 * tw);
            const int64_t r = tile0 * 16 + (i - c * 16 * tw);
            outer = load_outer<S>(w0, w1, e, c, r, r < e.rows);
        }
        __builtin_amdgcn_sched_barrier(0);
        // then the weights.
        u32x2 word[Q][N][2], d0[Q][N];
        const int last = static_cast<int>((e.rows + 15) / 16 - 1);
#pragma unroll
        for (int i = 0; i < N; i++) {
            const Weight &w = i / TILES ? w1 : w0;
            int tile = static_cast<int>(tile0) + ((i % TILES) << groups_log) + ipart;
            tile = tile <= last ? tile : last;
            const uint8_t *bits = reinterpret_cast<const uint8_t *>(w.bits) + (static_cast<int64_t>(tile / 4) * nb * 1024 + tile % 4 * 128);
            const uint8_t *scales = reinterpret_cast<const uint8_t *>(w.scales) + (static_cast<int64_t>(tile / 4) * nb8 * 1024 + tile % 4 * 256);
#pragma unroll
            for (int q = 0; q < Q; q++) {
                int i0 = 4 * (kpart + q * f.kw);
                i0 = b0 + (i0 < blocks ? i0 : 0);   // past the end: loaded, not used
#pragma unroll
                for (int k = 0; k < 2; k++) {   // block i0 + 2 k + g / 2, half g % 2
                    const int b = i0 + 2 * k + (g >> 1);
                    const uint32_t at = static_cast<uint32_t>(b < nb ? b : nb - 1) * 1024u + static_cast<uint32_t>((g & 1) * 512 + n16 * 8);
                    word[q][i][k] = __builtin_nontemporal_load(reinterpret_cast<const u32x2 *>(bits + at));
                }
                d0[q][i] = *reinterpret_cast<const u32x2 *>(scales + (i0 / 8 * 1024 + i0 % 8 * 2) + static_cast<uint32_t>(n16 * 16));
            }
        }
        __builtin_amdgcn_sched_barrier(0);
        if (b0 != first) __syncthreads();
        if (tid < 8) digits[kZeros + tid] = 0;
#pragma unroll
        for (int k = 0; k < kItems; k++) {
            const int c = column_of(k), i = item_of(k);
            const float v = f16_value(static_cast<uint16_t>(scale[k]));
#pragma unroll
            for (int part = 0; part < 2; part += kShare) {
                const int mine = kShare == 2 ? i & 1 : part;
                uint32_t l[3], h[3];
                code_digits(d[k], mine, l, h);
                if (i < blocks * 4 * kShare && c < n) {
                    uint32_t *o = digits + column_at(c) + i / kShare * 2 * kRow + mine * 3;
#pragma unroll
                    for (int j = 0; j < 3; j++) {
                        o[j] = l[j];
                        o[kRow + j] = h[j];
                    }
                    if (mine == 0) d1[i / kShare * C + c] = fabsf(v) <= 65504.0f ? v : __builtin_nanf("");
                }
            }
        }
        __syncthreads();
        const Signs signs(g & 1);
        const auto frag_at = [&](int at) {
            const u32x2 *dig = reinterpret_cast<const u32x2 *>(digits + at);
            const u32x2 f0 = dig[0], f1 = dig[1], f2 = dig[2];
            return frag(u32x4{f0[0], f0[1], f1[0], f1[1]}, f2);
        };
        const auto multiply = [&](i32x8 a, i32x8 w, f32x4 t, int power) {
            return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, w, t, kFp6, kFp4, 0, power, 0, kOne);
        };
        // The lane's row of an instruction, where n16 / 4 is its sub-block: up to two columns,
        // digit n16 % 2 of column n16 / 2 % 2; more, both digits in turn of column 4 m + n16 % 4.
        constexpr int kL = 130, kH = 134;   // 2^3 and 2^7: e2m3 codes are eighths
        int row[M];
#pragma unroll
        for (int m = 0; m < M; m++) {
            const int c = C > 2 ? 4 * m + n16 % 4 : n16 / 2 % 2;
            row[m] = n16 / 4 == g && c < n ? column_at(c) + (g * 2 + (C > 2 ? 0 : n16 % 2)) * kRow : -1;
        }
#pragma unroll
        for (int q = 0; q < Q; q++) {
            const int i0 = 4 * (kpart + q * f.kw);
            uint32_t x[2][N];   // words 0 and 1 of both halves of a block to the lanes of their sub-blocks
#pragma unroll
            for (int k = 0; k < 4; k++) {
                if (i0 + k >= blocks) break;
                if (k % 2 == 0) {
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        const auto two = __builtin_amdgcn_permlane32_swap(word[q][i][k / 2][0], word[q][i][k / 2][1], false, false);
                        x[0][i] = two[0];
                        x[1][i] = two[1];
                    }
                }
                const auto at = [&](int m) { return row[m] >= 0 ? row[m] + (i0 + k) * (4 * 2 * kRow) : kZeros; };
                const float *s1 = d1 + ((i0 + k) * 4 + g) * C;
                const auto sign_of = [&](int i) {
                    const auto h = __builtin_amdgcn_permlane16_swap(x[k % 2][i], x[k % 2][i], false, false);
                    return signs(h[0], h[1]);
                };
                const auto scale_of = [&](int i) { return f16_value(static_cast<uint16_t>(d0[q][i][k / 2] >> (16 * (k & 1)))); };
                const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
                if constexpr (C <= 2) {
                    const i32x8 a = frag_at(at(0));
                    float s[C];
#pragma unroll
                    for (int c = 0; c < C; c++) s[c] = s1[c];
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        const f32x4 t = multiply(a, sign_of(i), zero, n16 % 2 ? kH : kL);
                        const float d0f = scale_of(i);
#pragma unroll
                        for (int c = 0; c < C; c++) acc[i][c] = fmaf(d0f * s[c], t[2 * c] + t[2 * c + 1], acc[i][c]);
                    }
                } else {
                    i32x8 w[N];
                    float d0f[N];
#pragma unroll
                    for (int i = 0; i < N; i++) {
                        w[i] = sign_of(i);
                        d0f[i] = scale_of(i);
                    }
#pragma unroll
                    for (int m = 0; m < M; m++) {
                        const i32x8 l = frag_at(at(m)), h = frag_at(row[m] >= 0 ? at(m) + kRow : kZeros);
                        const f32x4 s = *reinterpret_cast<const f32x4 *>(s1 + 4 * m);
                        f32x4 t[N];
#pragma unroll
                        for (int i = 0; i < N; i++) t[i] = multiply(h, w[i], zero, kH);
#pragma unroll
                        for (int i = 0; i < N; i++) t[i] = multiply(l, w[i], t[i], kL);
#pragma unroll
                        for (int i = 0; i < N; i++)
#pragma unroll
                            for (int c = 0; c < 4; c++) acc[i][4 * m + c] = fmaf(d0f[i] * s[c], t[i][c], acc[i][4 * m + c]);
                    }
                }
            }
        }
    }
    if (kShared) __syncthreads();
#pragma unroll
    for (int i = 0; i < N; i++) {
        float *to = red + ((kpart * S + i / TILES) * tw + ((i % TILES) << groups_log) + ipart) * 64 * M + lane;
#pragma unroll
        for (int m = 0; m < M; m++) {   // of the lane's column, 4 m + g
            if constexpr (C == 1)
                to[0] = sum_rows(acc[i][0]);
            else if constexpr (C == 2)
                to[0] = rows16(halves(acc[i][0], acc[i][0]), halves(acc[i][1], acc[i][1]));
            else
                to[64 * m] = rows16(halves(acc[i][4 * m], acc[i][4 * m + 2]), halves(acc[i][4 * m + 1], acc[i][4 * m + 3]));
        }
    }
    __syncthreads();
    for (int i = tid; i < n * 16 * tw; i += kFew) {   // 32 lanes together hold 32 rows where blocks are written (tw even)
        const int c = i / (16 * tw), rr = i - c * 16 * tw;
        const int64_t r = tile0 * 16 + rr;
        const bool live = r < e.rows;
        if (C > 4 || i >= kFew) outer = load_outer<S>(w0, w1, e, c, r, live && (C <= 4 || f.slices == 1));
        float v[2] = {0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 8; k++)
            if (k < f.kw)
#pragma unroll
                for (int s = 0; s < S; s++) v[s] += red[((k * S + s) * tw + rr / 16) * 64 * M + c * 16 + rr % 16];
        if (C <= 4 || f.slices == 1) {
            finish_one<S>(e, outer, v[0], v[1], c, r, live);
        } else if (r < 32 * f.row_tiles) {
#pragma unroll
            for (int s = 0; s < S; s++) f.parts[((static_cast<int64_t>(slice) * S + s) * n + c) * 32 * f.row_tiles + r] = v[s];
        }
    }
}

// ------------------------------------------------------- more columns
// The activations as operands of 32 x 32 x 64 instructions: for each 32 columns and 64
// elements (a step) a fragment of 1536 bytes per digit (16 bytes of each lane, then 8), and
// behind all of them a word of each lane with the digits' powers of two.
constexpr int64_t kStepBytes = 4 * 1536;

// A thread takes a sub-block of a column, or half of one (kHalf: below 1024 blocks, where the
// way through the arithmetic is what takes time: 5 columns of 4096 10.5 us in all instead of
// 11.1; 2039 of 14336 262 instead of 271 with whole ones). 2039 columns of 14336 take 30 us,
// 31 MB read and 97 written.
template <bool kHalf>
__global__ __launch_bounds__(256) void q1_digits_kernel(const uint16_t *__restrict__ a_q8, uint8_t *__restrict__ out, int64_t n,
                                                        int64_t steps) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64, half = kHalf ? wave % 2 : 0;
    const int64_t step = kHalf ? static_cast<int64_t>(blockIdx.x) * 2 + wave / 2 : static_cast<int64_t>(blockIdx.x) * 4 + wave;
    const int64_t tile = blockIdx.y, c = tile * 32 + lane % 32;
    if (step >= steps) return;
    uint32_t d[8] = {}, h = 0;
    if (c < n) h = load_block(a_q8 + ((c * steps + step) * 2 + lane / 32) * 17, d);
    const Scale s(h);
    uint8_t *o = out + (tile * steps + step) * kStepBytes;
    uint32_t w[2][4][3];   // three words for each half and digit
#pragma unroll
    for (int k = 0; k < (kHalf ? 1 : 2); k++) {
        uint32_t r[4][4];   // by places 4 i .. 4 i + 3 of the half
        const int j = kHalf ? 2 * half : 2 * k;
        digits8(d, j, s.m, r);
        digits8(d, j + 1, s.m, r + 2);
#pragma unroll
        for (int p = 0; p < 4; p++) {
            w[k][p][0] = r[0][p] | r[1][p] << 24;
            w[k][p][1] = r[1][p] >> 8 | r[2][p] << 16;
            w[k][p][2] = r[2][p] >> 16 | r[3][p] << 8;
        }
    }
#pragma unroll
    for (int p = 0; p < 4; p++, o += 1536) {
        uint32_t *lo = reinterpret_cast<uint32_t *>(o) + lane * 4, *hi = reinterpret_cast<uint32_t *>(o + 1024) + lane * 2;
        if (!kHalf) {
            *reinterpret_cast<u32x4 *>(lo) = u32x4{w[0][p][0], w[0][p][1], w[0][p][2], w[1][p][0]};
            *reinterpret_cast<u32x2 *>(hi) = u32x2{w[1][p][1], w[1][p][2]};
        } else if (half == 0) {
            *reinterpret_cast<u32x2 *>(lo) = u32x2{w[0][p][0], w[0][p][1]};
            lo[2] = w[0][p][2];
        } else {
            lo[3] = w[0][p][0];
            *reinterpret_cast<u32x2 *>(hi) = u32x2{w[0][p][1], w[0][p][2]};
        }
    }
    if (half == 0) reinterpret_cast<uint32_t *>(out + gridDim.y * steps * kStepBytes)[(tile * steps + step) * 64 + lane] = s.powers;
}

struct ManyShape {
    int64_t nb, col_tiles, row_tiles;   // blocks of a row, tiles of 32 columns, of 32 rows
    int64_t row_groups;                 // of a workgroup's tiles
    int64_t slices, share;              // of K, and the blocks of one
    float *parts;                       // sums of the slices, [slices][S][n][32 row_tiles]
};

// t += the products of one digit. (The builtin takes the digit's byte as an immediate.)
template <int P>
__device__ __forceinline__ f32x16 mma(i32x8 a, i32x8 b, f32x16 t, uint32_t powers) {
    return __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, t, kFp6, kFp4, P, static_cast<int>(powers), 0, kOne);
}

// One step of NT tiles: t[i] += a w[i], the four digits one after the other.
template <int NT>
__device__ __forceinline__ void step(f32x16 (&t)[NT], const i32x8 (&a)[4], const i32x8 (&w)[NT], uint32_t powers) {
    const auto digit = [&](auto p) {
#pragma unroll
        for (int i = 0; i < NT; i++) t[i] = mma<decltype(p)::value>(a[decltype(p)::value], w[i], t[i], powers);
    };
    digit(std::integral_constant<int, 0>{});
    digit(std::integral_constant<int, 1>{});
    digit(std::integral_constant<int, 2>{});
    digit(std::integral_constant<int, 3>{});
}

// acc += d0 t, d0 of the lane's weight row.
template <int NT>
__device__ __forceinline__ void fold(f32x16 (&acc)[NT], const f32x16 (&t)[NT], const uint16_t (&d0)[NT]) {
#pragma unroll
    for (int i = 0; i < NT; i++) {
        const float d = f16_value(d0[i]);
#pragma unroll
        for (int k = 0; k < 16; k++) acc[i][k] = fmaf(d, t[i][k], acc[i][k]);
    }
}

// A tile's sums to LDS, a column's rows kPitch apart: value k of a lane is column 8 (k / 4) +
// 4 g + k % 4 of its tile and row n32 of the other. From there a lane takes four rows of a
// column at a time: column lane / 8 of each eight, rows 4 (lane % 8) on.
constexpr int kPitch = 36, kTile = 32 * kPitch;
__device__ __forceinline__ void put_tile(const f32x16 &v, float *to, int g, int n32) {
#pragma unroll
    for (int k = 0; k < 16; k++) to[(8 * (k / 4) + 4 * g + k % 4) * kPitch + n32] = v[k];
}

// Workgroups with consecutive numbers go to the eight dies in turn: each die takes a run of
// row groups with all their slices and columns, so that a weight is read by one die.
__device__ __forceinline__ bool place(const ManyShape &f, int64_t &col, int64_t &row_group, int64_t &slice) {
    const int64_t total = f.col_tiles * f.row_groups * f.slices, id = blockIdx.x, per = (total + 7) / 8, at = id % 8 * per + id / 8;
    col = at % f.col_tiles;
    slice = at / f.col_tiles % f.slices;
    row_group = at / f.col_tiles / f.slices;
    return id / 8 < per && at < total;
}

// Sums of four rows: finished, or a slice's share kept for the joining launch.
template <int S>
__device__ __forceinline__ void emit(const Weight &w0, const Weight &w1, const Epilogue &e, const ManyShape &f, int64_t slice, f32x4 v,
                                     f32x4 u, int64_t c, int64_t r) {
    if (f.slices == 1) {
        finish<S>(w0, w1, e, v, u, c, r);
    } else if (c < e.n && r < 32 * f.row_tiles) {
        float *to = f.parts + (slice * S * e.n + c) * 32 * f.row_tiles + r;
        *reinterpret_cast<f32x4 *>(to) = v;
        if (S == 2) *reinterpret_cast<f32x4 *>(to + e.n * 32 * f.row_tiles) = u;
    }
}

// One value a thread; all that it needs is asked for at once: the call is a memory latency long.
template <int S>
__global__ __launch_bounds__(256) void q1_join_kernel(Weight w0, Weight w1, Epilogue e, int slices, int64_t row_tiles,
                                                      const float *__restrict__ parts) {
    const int64_t padded = 32 * row_tiles, i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;   // 32 lanes to 32 rows
    if (i >= e.n * padded) return;
    const int64_t c = i / padded, r = i % padded, next = S * e.n * padded;
    const bool live = r < e.rows;
    const Outer outer = load_outer<S>(w0, w1, e, c, r, live);
    const float *from = parts + i;
    float v[2] = {0.0f, 0.0f};
    constexpr int kAtOnce = 8;
    for (int s = 0; s < slices; s += kAtOnce) {
        float p[kAtOnce][S];
#pragma unroll
        for (int k = 0; k < kAtOnce; k++)
#pragma unroll
            for (int j = 0; j < S; j++) p[k][j] = from[(s + k < slices ? s + k : s) * next + j * e.n * padded];
#pragma unroll
        for (int k = 0; k < kAtOnce; k++)
#pragma unroll
            for (int j = 0; j < S; j++) v[j] += s + k < slices ? p[k][j] : 0.0f;
    }
    finish_one<S>(e, outer, v[0], v[1], c, r, live);
}

// Loads of 16 (or 4) bytes a lane from base + `at` (per lane) to LDS, lane after lane from `to`
// on: N of them, 1 KiB apart on both sides. The compiler does not see these loads: who reads
// what they bring waits for them first.
template <int N>
__device__ __forceinline__ void lds_load16(const void *base, uint32_t at, uint32_t to) {
    static_assert(N == 1 || N == 3, "as written");
    if constexpr (N == 1)
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(at), "s"(base) : "memory", "m0");
    else
        asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2\n\tglobal_load_lds_dwordx4 %1, %2 offset:1024\n\t"
                     "global_load_lds_dwordx4 %1, %2 offset:2048" ::"s"(to), "v"(at), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void lds_load4(const void *base, uint32_t at, uint32_t to) {
    asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, %2" ::"s"(to), "v"(at), "s"(base) : "memory", "m0");
}

// Prompts: four waves side by side along the rows (each NT = TN S tiles of 32, TN of each of the
// S weights) share a tile of 32 columns and take what a block of 128 needs from LDS, loaded
// kBuffers blocks before it is used. A wave has the digits of a step in registers, reads the
// next step's, and goes through its tiles, four instructions on the same sums each. Two
// workgroups on a CU, so that one wave of a SIMD works while the other one waits for its own.
//
// 2039 columns at 4096 x 14336 take 220 to 230 us (1.05 PFLOP/s of products, 4.2 of the digits'),
// gated 509 at 14336 x 4096 129. The instructions alone, on such operands, would take 163: fed
// without a pause on random digits the cores' clock falls (21.5 ns an instruction; 16.4 on
// constant ones), and here they are busy for 61 % of the cycles at 1.7 GHz. Without the loads
// and the barrier the same products took 207.
template <int TN, int S>
__global__ __launch_bounds__(256, 2) void q1_wide_kernel(Weight w0, Weight w1, const uint8_t *__restrict__ digits, Epilogue e,
                                                         ManyShape f) {
    constexpr int NT = TN * S, kWaves = 4, kBuffers = 3;
    static_assert(NT == 4, "the waves' shares of the loads");
    // A buffer: the column tile's digits, the waves' signs and scales, the powers of two (twice).
    constexpr int kSigns = 2 * kStepBytes, kScales = kSigns + kWaves * NT * 512, kPowers = kScales + kWaves * NT * 128,
                  kBuffer = kPowers + kWaves * 256;
    constexpr int kIssued = 3 + 2 + 2 + 1;   // loads of a wave and block
    constexpr int kSums = kWaves * S * kTile * 4;
    __shared__ __attribute__((aligned(16))) uint8_t lds[kBuffers * kBuffer > kSums ? kBuffers * kBuffer : kSums];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 32, n32 = lane % 32;
    const int64_t nb = f.nb, nb8 = (nb + 7) / 8, steps = 2 * nb;
    int64_t col, row0, slice;
    if (!place(f, col, row0, slice)) return;
    row0 = (row0 * kWaves + wave) * TN;
    const int from = static_cast<int>(slice * f.share);   // the slice's first block
    // Where a block lies for the wave: three of the 12 KiB of digits (two steps are together), the
    // powers of one step, the signs and scales of its tiles, two at a time. Signs 16 bytes a
    // lane, the rows 2 (lane % 16) and one more of half lane / 16 % 2; scales those of a block
    // and its neighbour.
    const uint8_t *chunk = digits + col * steps * kStepBytes + wave * static_cast<int>(2 * kStepBytes / kWaves);
    const uint8_t *power = digits + (f.col_tiles * steps * kStepBytes + (col * steps + wave % 2) * 256);
    const uint8_t *sign[2], *scale[2];
    uint32_t sign_at[2], scale_at[2];
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const Weight &w = 2 * i >= TN ? w1 : w0;
        const int64_t last = f.row_tiles - 1, ra = row0 + 2 * i % TN < last ? row0 + 2 * i % TN : last, rb = ra < last ? ra + 1 : last;
        sign[i] = reinterpret_cast<const uint8_t *>(w.bits + ra / 2 * nb * 128 + ra % 2 * 32);
        scale[i] = reinterpret_cast<const uint8_t *>(w.scales + ra / 2 * nb8 * 512 + ra % 2 * 256);
        sign_at[i] = g * static_cast<uint32_t>((rb / 2 - ra / 2) * nb * 1024 + (rb % 2 - ra % 2) * 256) + lane / 16 % 2 * 512 + lane % 16 * 16;
        scale_at[i] = g * static_cast<uint32_t>((rb / 2 - ra / 2) * nb8 * 1024 + (rb % 2 - ra % 2) * 512) + n32 * 16;
    }
    const uint32_t lane16 = lane * 16, lane4 = lane * 4;
    const uint32_t base = __builtin_amdgcn_readfirstlane(
        static_cast<uint32_t>(reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) uint8_t *)lds)));
    const int blocks = static_cast<int>(nb - from < f.share ? nb - from : f.share);
    // The kIssued loads of block i, two of them in each part but the first; past the end the last
    // block's again, into a buffer not read.
    const auto stage = [&](int i, uint32_t to, int part) {
        const uint32_t b = from + (i < blocks ? i : blocks - 1);
        if (part == 0) {
            lds_load16<3>(chunk + b * static_cast<uint32_t>(2 * kStepBytes), lane16, to + wave * static_cast<int>(2 * kStepBytes / kWaves));
        } else if (part == 1) {
            lds_load4(power + b * 512u, lane4, to + kPowers + wave * 256);
        } else {
            lds_load16<1>(sign[part - 2] + b * 1024u, sign_at[part - 2], to + kSigns + wave * 2048 + (part - 2) * 1024);
            lds_load4(scale[part - 2] + (b / 8 * 1024u + b % 8 / 2 * 4), scale_at[part - 2], to + kScales + wave * 512 + (part - 2) * 256);
        }
    };
    const auto arrive = [&](auto behind) {   // all but the loads of so many newer blocks, in every wave
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(behind)::value * kIssued) : "memory");
    };
    // What a wave has of a step in registers: digits, their powers, the words of both halves.
    struct Step {
        i32x8 a[4];
        uint32_t powers, half0[NT], half1[NT];
    };
    const auto read = [&](uint32_t at, int s) {   // at: the buffer's place
        const uint8_t *in = lds + at;
        const uint8_t *lo = in + lane * 16, *hi = in + (1024 + lane * 8), *sg = in + (kSigns + wave * 2048 + n32 * 8),
                      *po = in + (kPowers + lane * 4);
        Step k;
#pragma unroll
        for (int p = 0; p < 4; p++) {
            const int at = s * static_cast<int>(kStepBytes) + 1536 * p;
            // (volatile: not two of them in one instruction, whose results would have to be moved)
            const u32x2 h = *(const volatile __attribute__((address_space(3))) u32x2 *)(hi + at);
            k.a[p] = frag(*reinterpret_cast<const u32x4 *>(lo + at), h);
        }
        k.powers = *reinterpret_cast<const uint32_t *>(po + s * 256);
#pragma unroll
        for (int i = 0; i < NT; i++) {
            k.half0[i] = *reinterpret_cast<const uint32_t *>(sg + i * 512 + s * 4);
            k.half1[i] = *reinterpret_cast<const uint32_t *>(sg + i * 512 + s * 4 + 256);
        }
        return k;
    };
    const Signs signs(g);
    f32x16 acc[NT], t[NT];
    float d0[NT], before[NT];   // scales of this block and of the one before it
#pragma unroll
    for (int i = 0; i < NT; i++) {
        acc[i] = t[i] = f32x16{};
        before[i] = 0.0f;
    }
    // acc += d0 t, values k .. k + 7 of a tile
    const auto fold8 = [&](int i, int k, float d) {
#pragma unroll
        for (int j = k; j < k + 8; j++) acc[i][j] = fmaf(d, t[i][j], acc[i][j]);
    };
    // Four instructions of tile i with `vector` others spread between them: a matrix instruction
    // hides up to five or six of those, whichever wave they are of, but not a run of them.
    const auto multiply = [&](const Step &k, int i, const i32x8 &x) {
        t[i] = mma<0>(k.a[0], x, t[i], k.powers);
        t[i] = mma<1>(k.a[1], x, t[i], k.powers);
        t[i] = mma<2>(k.a[2], x, t[i], k.powers);
        t[i] = mma<3>(k.a[3], x, t[i], k.powers);
    };
    const auto spread = [](auto vector) {
#pragma unroll
        for (int i = 0; i < 4; i++) {
            __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
            __builtin_amdgcn_sched_group_barrier(0x002, decltype(vector)::value, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
    };
    using Few = std::integral_constant<int, 4>;
    using More = std::integral_constant<int, 7>;
#pragma unroll
    for (int k = 0; k < kBuffers; k++)
#pragma unroll
        for (int part = 0; part < 4; part++) stage(k, base + k * kBuffer, part);
    arrive(std::integral_constant<int, kBuffers - 1>{});
    Step first = read(0, 0);
    i32x8 x = signs(first.half0[0], first.half1[0]);
    uint32_t at = 0;
    for (int b = 0; b < blocks; b++) {
        const Step second = read(at, 1);
        const uint8_t *sc = lds + at + (kScales + wave * 512 + n32 * 4 + ((from + b) & 1) * 2);
#pragma unroll
        for (int i = 0; i < NT; i++) d0[i] = f16_value(*reinterpret_cast<const uint16_t *>(sc + i * 128));
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < NT; i++) {   // the first step, with what is left of the block before it
            if (i < 2) {
                fold8(2 + i, 0, before[2 + i]);
                fold8(2 + i, 8, before[2 + i]);
            }
            const i32x8 next = i + 1 < NT ? signs(first.half0[(i + 1) % NT], first.half1[(i + 1) % NT]) : signs(second.half0[0], second.half1[0]);
            t[i] = f32x16{};
            multiply(first, i, x);
            x = next;
            if (i < 2)
                spread(More{});
            else
                spread(Few{});
        }
        arrive(std::integral_constant<int, kBuffers - 2>{});   // the next block; and nobody reads this one any more
        const uint32_t to = base + at;
        at = at == (kBuffers - 1) * kBuffer ? 0 : at + kBuffer;
        first = read(at, 0);
#pragma unroll
        for (int i = 0; i < NT; i++) {
            stage(b + kBuffers, to, i);
            if (i >= 2) {
                fold8(i - 2, 0, d0[i - 2]);
                fold8(i - 2, 8, d0[i - 2]);
            }
            const i32x8 next = i + 1 < NT ? signs(second.half0[(i + 1) % NT], second.half1[(i + 1) % NT]) : signs(first.half0[0], first.half1[0]);
            multiply(second, i, x);
            x = next;
            if (i >= 2)
                spread(More{});
            else
                spread(Few{});
        }
#pragma unroll
        for (int i = 0; i < NT; i++) before[i] = d0[i];
    }
#pragma unroll
    for (int i = 2; i < NT; i++) {
        fold8(i, 0, before[i]);
        fold8(i, 8, before[i]);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float *own = reinterpret_cast<float *>(lds) + wave * S * kTile;   // a wave's own: its LDS accesses stay in order
    const int mine = lane / 8 * kPitch + lane % 8 * 4;
#pragma unroll
    for (int i = 0; i < TN; i++) {
#pragma unroll
        for (int s = 0; s < S; s++) put_tile(acc[s * TN + i], own + s * kTile, g, n32);
        __builtin_amdgcn_wave_barrier();
#pragma unroll 1
        for (int q = 0; q < 4; q++)
            emit<S>(w0, w1, e, f, slice, *reinterpret_cast<const f32x4 *>(own + mine + q * 8 * kPitch),
                    *reinterpret_cast<const f32x4 *>(own + (S - 1) * kTile + mine + q * 8 * kPitch), col * 32 + 8 * q + lane / 8,
                    (row0 + i) * 32 + lane % 8 * 4);
        __builtin_amdgcn_wave_barrier();
    }
}

// Batches: KS waves share the sums of 32 columns and NT = TN S tiles of 32 weight rows by K,
// each loading its digits to registers a block ahead, and add them up in LDS. 37 columns gated at
// 6912 x 2560 take 13.5 to 14.2 us, 64 at 4096 x 4096 15.1 to 15.6: two or three launches, each a few latencies
// long, and what the digits take from L2 (12.5 KB for a wave's block; 54 MB in all for the former).
template <int TN, int S, int KS>
__global__ __launch_bounds__(64 * KS, 2) void q1_split_kernel(Weight w0, Weight w1, const uint8_t *__restrict__ digits, Epilogue e,
                                                              ManyShape f) {
    constexpr int NT = TN * S;
    __shared__ __attribute__((aligned(16))) float sums[KS * NT * kTile];
    const int lane = threadIdx.x % 64, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / 64);
    const int g = lane / 32, n32 = lane % 32;
    const int64_t nb = f.nb, nb8 = (nb + 7) / 8, steps = 2 * nb;
    int64_t col, row0, slice;
    if (!place(f, col, row0, slice)) return;
    row0 *= TN;
    const int64_t stop = (slice + 1) * f.share < nb ? (slice + 1) * f.share : nb, share = (f.share + KS - 1) / KS;
    int64_t b = slice * f.share + wave * share;
    const int64_t end = b + share < stop ? b + share : stop;
    const uint8_t *frags = digits + col * steps * kStepBytes + lane * 16;
    const uint32_t *powers = reinterpret_cast<const uint32_t *>(digits + f.col_tiles * steps * kStepBytes) + col * steps * 64 + lane;
    const u32x2 *bits[NT];
    const uint16_t *scales[NT];
#pragma unroll
    for (int i = 0; i < NT; i++) {
        const Weight &w = i / TN ? w1 : w0;
        int64_t rt = row0 + i % TN;
        rt = rt < f.row_tiles ? rt : f.row_tiles - 1;
        const int64_t in64 = rt % 2 * 32 + n32;
        bits[i] = w.bits + rt / 2 * nb * 128 + g * 64 + in64;
        scales[i] = w.scales + rt / 2 * nb8 * 512 + in64 * 8;
    }
    const Signs signs(g);
    f32x16 acc[NT];
#pragma unroll
    for (int i = 0; i < NT; i++) acc[i] = f32x16{};
    struct Loads {
        u32x2 bits[NT];
        uint16_t scales[NT];
        uint32_t powers[2];
        u32x4 lo[2][4];
        u32x2 hi[2][4];
    };
    const auto load = [&](int64_t i) {
        Loads l;
#pragma unroll
        for (int k = 0; k < NT; k++) {
            l.bits[k] = bits[k][i * 128];
            l.scales[k] = scales[k][i / 8 * 512 + i % 8];
        }
#pragma unroll
        for (int s = 0; s < 2; s++) {
            l.powers[s] = powers[(2 * i + s) * 64];
#pragma unroll
            for (int p = 0; p < 4; p++) {
                const uint8_t *src = frags + (2 * i + s) * kStepBytes + 1536 * p;
                l.lo[s][p] = *reinterpret_cast<const u32x4 *>(src);
                l.hi[s][p] = *reinterpret_cast<const u32x2 *>(src + 1024 - lane * 8);
            }
        }
        return l;
    };
    if (b < end) {
        Loads l = load(b);
        for (; b < end; b++) {
            const Loads ahead = load(b + 1 < end ? b + 1 : b);
            f32x16 t[NT];
#pragma unroll
            for (int i = 0; i < NT; i++) t[i] = f32x16{};
#pragma unroll
            for (int s = 0; s < 2; s++) {
                i32x8 a[4], x[NT];
#pragma unroll
                for (int p = 0; p < 4; p++) a[p] = frag(l.lo[s][p], l.hi[s][p]);
#pragma unroll
                for (int i = 0; i < NT; i++) {
                    const auto h = __builtin_amdgcn_permlane32_swap(l.bits[i][s], l.bits[i][s], false, false);
                    x[i] = signs(h[0], h[1]);
                }
                step(t, a, x, l.powers[s]);
            }
            fold(acc, t, l.scales);
            l = ahead;
        }
    }
#pragma unroll
    for (int i = 0; i < NT; i++) put_tile(acc[i], sums + (wave * NT + i) * kTile, g, n32);
    __syncthreads();
    const int from = lane / 8 * kPitch + lane % 8 * 4;
    for (int j = wave; j < TN * 4; j += KS) {   // eight columns of a tile at a time
        const int q = j % 4, i = j / 4;
        f32x4 v[2] = {};
#pragma unroll
        for (int k = 0; k < KS; k++)
#pragma unroll
            for (int s = 0; s < S; s++) v[s] += *reinterpret_cast<const f32x4 *>(sums + (k * NT + s * TN + i) * kTile + from + q * 8 * kPitch);
        emit<S>(w0, w1, e, f, slice, v[0], v[1], col * 32 + 8 * q + lane / 8, (row0 + i) * 32 + lane % 8 * 4);
    }
}

constexpr int64_t kMaxK = INT64_C(1) << 20, kMaxColumns = INT64_C(1) << 20;
// so that a launch's threads stay below 2^32
constexpr int64_t kMaxRows = INT64_C(1) << 26, kMaxOutputs = INT64_C(1) << 36;
constexpr int64_t kFewColumns = 4;   // so many columns take no workspace

int check_sizes(const char *name, int64_t K, int64_t n_act) {
    GD_REQUIRE(K >= 1 && n_act >= 1, GD_EINVAL, "%s: K (%lld) and n_act (%lld) must be >= 1", name, (long long)K,
               (long long)n_act);
    GD_REQUIRE(K % 128 == 0, GD_ESHAPE, "%s: K (%lld) must be a multiple of 128", name, (long long)K);
    GD_REQUIRE(K <= kMaxK && n_act <= kMaxColumns, GD_ERANGE, "%s: K or n_act too large", name);
    return GD_OK;
}

// The activations as the matrix cores read them, 100 bytes for 32 elements, and the sums of
// slices of K.
int64_t digits_bytes(int64_t K, int64_t n_act) { return (n_act + 31) / 32 * 100 * K; }   // below 2^42
int64_t parts_bytes(int64_t n_act) { return n_act < 32 ? n_act << 19 : INT64_C(1) << 24; }
int64_t workspace_need(int64_t K, int64_t n_act) {
    return n_act <= kFewColumns ? 0 : digits_bytes(K, n_act) + parts_bytes(n_act);
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
    GD_REQUIRE(e.rows <= kMaxRows && e.rows * e.n <= kMaxOutputs, GD_ERANGE, "%s: rows or n_act too large", name);
    const int64_t size = dtype_size(dtype);
    for (int i = 0; i < count; i++)
        GD_REQUIRE(aligned(w[i].bits, 16) && aligned(w[i].scales, 16) && aligned(w[i].bias, 4), GD_EALIGN,
                   "%s: planes must be 16-byte aligned, a bias 4", name);
    GD_REQUIRE(aligned(a_q8, 2) && aligned(e.y_q8, 2) && aligned(e.residual, size) && aligned(e.y, size) &&
                   aligned(workspace, 16),
               GD_EALIGN, "%s: a_q8 and y_q8 must be 2-byte aligned, residual and y to their element, workspace 16", name);
    const int64_t need = workspace_need(K, e.n), bytes = e.n * e.rows * size;   // below 2^39
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

// With so many blocks for its workgroups to go through the wide kernel is the faster one (both
// on one card): 64 columns at 4096 x 4096 (512) 20.1 us against 15.1, 509 (4096) 40.8 against 34.4,
// 1000 (8192) 56 against 65, gated, 37 at 14336 x 4096 (3584) 33.3 against 26.2, 200 at 14336 x 4096
// (12544) 69 against 76, 2039 at 4096 x 14336 (57344) 254 against 420.
constexpr int64_t kWideFrom = 8000;
// Up to so many workgroups of four tiles a wave the kernel without an operand pass is the faster
// one: of 8 columns 14336 x 4096 9.6 us against 15.6, 49152 x 4096 (768 workgroups) 25.8 against
// 28.4, gated (1536) 43.2 against 40.1; of 13 (a workgroup a CU, and twice the matrix
// instructions a column) 28672 x 4096 (224) 20.3 against 25.4, 49152 x 4096 (384) 37.7 against 29.9.
constexpr int64_t kCus = 256, kSomeGroups8 = 1024, kSomeGroups16 = kCus;

template <int S>
void join(const Weight &w0, const Weight &w1, const Epilogue &e, int64_t slices, int64_t row_tiles, const float *parts, hipStream_t hs) {
    hipLaunchKernelGGL((q1_join_kernel<S>), dim3(static_cast<uint32_t>((e.n * row_tiles * 32 + 255) / 256)), dim3(256), 0, hs, w0, w1, e,
                       static_cast<int>(slices), row_tiles, parts);
}

// As many waves along K as a chunk has quads of blocks; the number of these.
template <int C>
int64_t waves_along_k(FewShape &f) {
    const int64_t quads = ((f.nb < kBlocks<C> ? f.nb : kBlocks<C>) + 3) / 4;
    while (f.kw < 8 && f.kw < quads) {
        f.kw *= 2;
        f.kw_log++;
    }
    return quads;
}

template <int C, int S>
void run_few(const Weight &w0, const Weight &w1, const uint16_t *a_q8, const Epilogue &e, int64_t K, hipStream_t hs) {
    FewShape f = {K / 128, 1, 0, 1, static_cast<int>(K / 128), 0, nullptr};
    const int64_t quads = waves_along_k<C>(f), tiles = (e.rows + 15) / 16;
    const auto go = [&](auto tiles_, auto q) {
        constexpr int TILES = decltype(tiles_)::value, Q = decltype(q)::value;
        const int64_t per = TILES * (8 / f.kw);
        hipLaunchKernelGGL((q1_few_kernel<C, S, TILES, Q>), dim3(static_cast<uint32_t>((tiles + per - 1) / per)), dim3(kFew), 0, hs, w0, w1,
                           a_q8, e, f);
    };
    using One = std::integral_constant<int, 1>;
    using Two = std::integral_constant<int, 2>;
    using Four = std::integral_constant<int, 4>;
    // More tiles a wave once they come to 224 workgroups: 4096 x 4096, one column: one tile 4.2 us,
    // two 4.7, four 5.7; 14336 x 4096: 7.3, 6.2, 6.1; 32768 x 4096: 13.4, 9.6, 8.4. (Blocks of 32
    // rows need two tiles in a workgroup.)
    const int64_t full = tiles * f.kw / 8;   // workgroups with a tile a wave
    if (quads <= f.kw) {
        if (full >= 4 * 224)
            go(Four{}, One{});
        else if (full >= 2 * 224 || (e.y_q8 && f.kw == 8))
            go(Two{}, One{});
        else
            go(One{}, One{});
    } else if (quads <= 2 * f.kw) {
        if (full >= 2 * 224 || e.y_q8)
            go(Two{}, Two{});
        else
            go(One{}, Two{});
    } else if constexpr (C <= 2) {
        if (e.y_q8)
            go(Two{}, Four{});
        else
            go(One{}, Four{});
    }
}

// Up to 16 columns; false where the launches below for more of them are the faster ones.
template <int C, int S>
bool run_some(const Weight &w0, const Weight &w1, const uint16_t *a_q8, const Epilogue &e, int64_t K, uint8_t *workspace,
              hipStream_t hs) {
    FewShape f = {K / 128, 1, 0, 1, static_cast<int>(K / 128), (e.rows + 31) / 32, reinterpret_cast<float *>(workspace)};
    const int64_t chunks = (f.nb + kBlocks<C> - 1) / kBlocks<C>, tiles = (e.rows + 15) / 16;
    waves_along_k<C>(f);
    const auto groups_of = [&](int64_t t) { return (tiles + t * (8 / f.kw) - 1) / (t * (8 / f.kw)); };   // of t tiles a wave
    if (groups_of(4 / S) > (C == 8 ? kSomeGroups8 : kSomeGroups16)) return false;
    const auto go = [&](auto tiles_) {
        constexpr int TILES = decltype(tiles_)::value;
        const int64_t groups = groups_of(TILES), room = parts_bytes(e.n) / (S * e.n * f.row_tiles * 128);
        int64_t z = kCus / groups;
        z = z < chunks ? z : chunks;
        z = z < room ? z : room;
        if (z < 1) z = 1;
        f.share = static_cast<int>((chunks + z - 1) / z * kBlocks<C>);
        f.slices = static_cast<int>((f.nb + f.share - 1) / f.share);
        hipLaunchKernelGGL((q1_few_kernel<C, S, TILES, 1>), dim3(static_cast<uint32_t>(groups * f.slices)), dim3(kFew), 0, hs, w0, w1, a_q8, e,
                           f);
    };
    // As few tiles a wave as let all chunks of K side by side in workgroups of their own (4096 x
    // 4096, 8 columns: one tile 7.1 us, two 7.6, four 9.2; 6144 x 4096: 9.4, 7.9, 9.3; 11000 x 4096:
    // 13.3, 11.1, 9.6; 4096 x 14336, 13 columns: 23.2, 16.8, 15.5).
    if (groups_of(1) * chunks <= kCus && !(e.y_q8 && f.kw == 8))   // (blocks of 32 rows need two tiles in a workgroup)
        go(std::integral_constant<int, 1>{});
    else if (S == 2 || groups_of(2) * chunks <= kCus)
        go(std::integral_constant<int, 2>{});
    else
        go(std::integral_constant<int, 4 / S>{});
    if (f.slices > 1) join<S>(w0, w1, e, f.slices, f.row_tiles, f.parts, hs);
    return true;
}

template <int S>
void run_many(const Weight &w0, const Weight &w1, const uint16_t *a_q8, const Epilogue &e, int64_t K, uint8_t *workspace,
              hipStream_t hs) {
    ManyShape f = {K / 128, (e.n + 31) / 32, (e.rows + 31) / 32, 0, 1, K / 128, reinterpret_cast<float *>(workspace + digits_bytes(K, e.n))};
    const auto cut = [](int64_t steps, int64_t by) { return static_cast<uint32_t>((steps + by - 1) / by); };
    if (f.col_tiles * f.nb < 1024)
        hipLaunchKernelGGL((q1_digits_kernel<true>), dim3(cut(2 * f.nb, 2), static_cast<uint32_t>(f.col_tiles)), dim3(256), 0, hs, a_q8,
                           workspace, e.n, 2 * f.nb);
    else
        hipLaunchKernelGGL((q1_digits_kernel<false>), dim3(cut(2 * f.nb, 4), static_cast<uint32_t>(f.col_tiles)), dim3(256), 0, hs, a_q8,
                           workspace, e.n, 2 * f.nb);
    const auto groups = [&](int64_t tiles) {   // of so many tiles of rows
        f.row_groups = (f.row_tiles + tiles - 1) / tiles;
        return f.col_tiles * f.row_groups;
    };
    // Slices of K, of eight blocks at least, until there are `want` workgroups or no room for their
    // sums: 13 columns at 4096 x 14336 on the split kernel 17 us, unsliced 28; on the wide one
    // 256 columns there 49 and 114.
    const auto slice = [&](int64_t have, int64_t want) {
        const int64_t room = parts_bytes(e.n) / (S * e.n * f.row_tiles * 128);
        int64_t z = want / have;
        z = z < f.nb / 8 ? z : f.nb / 8;
        z = z < room ? z : room;
        if (z < 1) z = 1;
        f.share = (f.nb + z - 1) / z;
        f.slices = (f.nb + f.share - 1) / f.share;
        return dim3(static_cast<uint32_t>((have * f.slices + 7) / 8 * 8));
    };
    constexpr int TN = 4 / S;
    const int64_t wide = groups(4 * TN);
    if (wide * f.nb >= kWideFrom) {
        const dim3 grid = slice(wide, 512 + wide - 1);
        hipLaunchKernelGGL((q1_wide_kernel<TN, S>), grid, dim3(256), 0, hs, w0, w1, workspace, e, f);
    } else {
        const auto go = [&](auto tiles, auto ks, int64_t want) {
            constexpr int T = decltype(tiles)::value, KS = decltype(ks)::value;
            const dim3 grid = slice(groups(T / S), want);
            hipLaunchKernelGGL((q1_split_kernel<T / S, S, KS>), grid, dim3(64 * KS), 0, hs, w0, w1, workspace, e, f);
        };
        using Two = std::integral_constant<int, 2>;
        using Four = std::integral_constant<int, 4>;
        using Eight = std::integral_constant<int, 8>;
        // Four tiles read the digits, which the waves load for themselves, half as often as two, if
        // they fill the device, alone or by slices: 64 columns at 4096 x 14336 23.2 us and 29.1, gated
        // 37 at 6912 x 2560 14.2 and 17.8, 20 at 14336 x 4096 17.7 and 24.6. Where two tiles fill it
        // without slices and K is short they save the joining launch: 128 at 4096 x 4096 18.0 and 19.7,
        // 100 at 4096 x 14336, of 112 blocks, 38.8 and 32.2; and where neither does: 64 at 1024 x 1024
        // 9.2 and 10.4. Four waves along K instead of eight once there is a workgroup for each CU:
        // gated 100 at 6912 x 2560 (432) 20.4 and 23.6, 37 (216) 17.9 and 14.2.
        const int64_t two = groups(2 / S), four = groups(4 / S), most = f.nb / 8 < 1 ? 1 : f.nb / 8;
        if (four > kCus)
            go(Four{}, Four{}, 1);
        else if (two > kCus || ((two <= kCus / 2 || f.nb >= 64) && four * most >= kCus * 3 / 4))
            go(Four{}, Eight{}, kCus);
        else
            go(Two{}, Eight{}, kCus);
    }
    if (f.slices > 1) join<S>(w0, w1, e, f.slices, f.row_tiles, f.parts, hs);
}

template <int S>
void run(const Weight &w0, const Weight &w1, const void *a_q8, const Epilogue &e, int64_t K, void *workspace, hipStream_t hs) {
    const uint16_t *a = static_cast<const uint16_t *>(a_q8);
    uint8_t *space = static_cast<uint8_t *>(workspace);
    if (e.n == 1)
        run_few<1, S>(w0, w1, a, e, K, hs);
    else if (e.n == 2)
        run_few<2, S>(w0, w1, a, e, K, hs);
    else if (e.n <= kFewColumns)
        run_few<4, S>(w0, w1, a, e, K, hs);
    else if (!(e.n <= 8 && run_some<8, S>(w0, w1, a, e, K, space, hs)) && !(e.n > 8 && e.n <= 16 && run_some<16, S>(w0, w1, a, e, K, space, hs)))
        run_many<S>(w0, w1, a, e, K, space, hs);
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
    const Epilogue e = {residual, y, static_cast<uint16_t *>(y_q8), rows, n_act, act, dtype};
    const int st = check("q1_q8_linear", &w, 1, a_q8, e, K, dtype, workspace, workspace_bytes);
    if (st) return st;
    run<1>(w, w, a_q8, e, K, workspace, as_stream(stream));
    return check_launch("q1_q8_linear");
}

extern "C" int q1_q8_gated(const void *gate_bits, const void *gate_scales, const void *up_bits, const void *up_scales,
                           const void *a_q8, const float *gate_bias, const float *up_bias, int32_t act, void *y,
                           void *y_q8, int64_t rows, int64_t K, int64_t n_act, int32_t dtype, void *workspace,
                           size_t workspace_bytes, void *stream) {
    const Weight w[2] = {{static_cast<const u32x2 *>(gate_bits), static_cast<const uint16_t *>(gate_scales), gate_bias},
                         {static_cast<const u32x2 *>(up_bits), static_cast<const uint16_t *>(up_scales), up_bias}};
    const Epilogue e = {nullptr, y, static_cast<uint16_t *>(y_q8), rows, n_act, act, dtype};
    const int st = check("q1_q8_gated", w, 2, a_q8, e, K, dtype, workspace, workspace_bytes);
    if (st) return st;
    run<2>(w[0], w[1], a_q8, e, K, workspace, as_stream(stream));
    return check_launch("q1_q8_gated");
}
