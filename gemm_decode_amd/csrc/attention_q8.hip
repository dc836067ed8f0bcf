// attention_q8.hip -- attention of the last tokens of several sequences (one
// decode token, a chain or a tree of drafted ones) over the 8-bit cache.
//
// Mathematics. One pass over the keys with a running maximum m, sum l and
// weighted sum o per query row, both rescaled when m grows; several passes
// over parts of the keys are joined by bringing them to the largest m.
//
// Shape of the work. The rows that read one KV head (its n_heads / n_kv_heads
// query heads of every query token) are taken together, 16 to a matrix-core
// tile, so that each key and value is read once for all of them. A workgroup
// of four waves serves one KV head, one part of the keys of one sequence and
// RT tiles of rows; its waves take 32 keys each in turn and never wait for one
// another until the end, where they are joined through LDS. A second launch
// joins the parts of a sequence, if it has more than one.
//
// Loads. Every load of codes is 16 bytes a lane, past the caches, and a wave's load is
// 1 KB of consecutive memory (K) or whole rows (V): reading alone, loads of 8 bytes a
// lane, four to a line, ran at 4.2 TB/s, these at 6.3. The K codes are turned into
// operand order through the wave's own part of LDS; V is exchanged between lanes.
//
// Products. Scores are taken transposed, S^T = K Q^T: lane (n, g) = (lane % 16,
// lane / 16) holds 16 dims of key n, half of them is swapped with lane (n, g ^ 2), and
// then one matrix instruction contracts exactly one 32-dim group; its result,
// multiplied by the group's scale, is added up in f32. The result has lane (n, g) hold
// keys 4g .. 4g+3 of query row n, which is how the second product, O^T = V^T P^T, takes
// its weights: they never leave their lane. For V^T the lane has to hold D/16 dims of
// the same four keys; a row of D bytes is D/16 lanes' loads, so up to four lanes load
// one key each and exchange parts. The dims of a lane lie in one scale group, so a value
// is its code times one scale per key. The scales come as one number a lane and tile,
// and are handed round by DPP.
//
// What bounds it. 32 sequences of 16k to 32k keys (32 / 8 heads, head dim 128, bf16,
// 1.75 GB of cache): 285 us with the 5 of the joining launch, 6.1 TB/s, 89 % of what a
// streaming read reaches; bound by memory. Few keys (4096 of one sequence, f32: 6.6 us, and
// 3.8 for the joining launch) are bound by the chain of dependent loads before the first
// product, many rows (64 tokens of four sequences, 210 TFLOP/s) by vector instructions,
// some 590 for 32 keys and 32 rows.
//
// Waits. Loads complete in order and a wait counts those behind the one it is for, so a
// wait is only as exact as that count is the same on every path: loads stand outside
// conditions, the last step is compiled apart, queries go out before keys, keys before
// values, and page numbers come by scalar loads. Without that each step waited for all
// of the next one's keys (32 sequences 286 us, f32 of 8k to 16k keys 205 where it is
// 172, 64 tokens of four 94).
//
// Precision. Codes are whole numbers below 2^8, exact in f16. f32 inputs: q (as
// a power of two times its row) and the weights are split into two f16 parts, 22
// bits; code * scale has at most 19 bits and is split exactly; the product of the
// two low parts, below 2^-22 of the result, is dropped. f16 and bf16 inputs: q is
// exact in f16 at its row's power of two, a weight and code * scale are rounded to
// f16, half a step being 2^-12 to 2^-11 of them, which is below a bf16 result's
// rounding and near a f16 result's. Sums, maxima and the softmax are f32. The
// scales of the values are brought near f16's upper end by a power of two per
// wave, which follows the largest scale seen.
#include <cmath>
#include <type_traits>

#include "gd_internal.h"
#include "gd_quant.h"
#include "gd_types.h"

namespace {

using namespace gd;

typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kStep = 32;                  // keys per wave and step
constexpr int kGroupKeys = kStep * kWaves; // keys per workgroup and step
constexpr float kNone = -3.0e38f;          // the maximum of no scores: below any, and finite
constexpr float kLog2e = 1.44269504088896340736f;
constexpr float kWeightBits = 14.0f;       // weights are held times 2^14, so that small ones keep their f16 bits

struct AttnArgs {
    gd_kv_q8 c;
    const void *q;
    void *out;
    const int32_t *page_table, *kv_lens, *q_start;
    const uint64_t *tree;
    int64_t max_pages, n_q, n_heads, max_q, max_kv_len;
    int64_t chunk;         // keys per part, a multiple of kGroupKeys
    int32_t splits;        // parts of the longest sequence
    int32_t row_block0, row_blocks;   // the launch's first block of 16 RT rows, and how many
    uint32_t page_magic;   // tile / (page_size / 16) = tile * page_magic >> page_shift
    int32_t page_shift, page_tiles;   // page_size / 16
    float factor, softcap;   // factor 2^factor_exp: from q . k to a score over the cap, or times log2 e without a cap
    int32_t factor_exp;
    float *part_o, *part_ml;
};

// What the kernels read of one sequence, clamped to what the host checked.
struct Seq {
    int64_t row0;   // first query row
    int rows;       // query tokens, at most max_q
    int64_t len;    // keys, the drafted ones included
    int64_t ctx;    // keys before the drafted ones
    __device__ __forceinline__ Seq(const AttnArgs &a, int64_t b) {
        int64_t lo = b * a.max_q, hi = lo + a.max_q;
        if (a.q_start) {
            lo = a.q_start[b];
            hi = a.q_start[b + 1];
        }
        lo = lo < 0 ? 0 : lo > a.n_q ? a.n_q : lo;
        hi = hi < lo ? lo : hi > a.n_q ? a.n_q : hi;
        row0 = lo;
        rows = static_cast<int>(hi - lo < a.max_q ? hi - lo : a.max_q);
        len = a.kv_lens[b];
        len = len < 0 ? 0 : len > a.max_kv_len ? a.max_kv_len : len;
        ctx = len - rows > 0 ? len - rows : 0;
    }
};

// r / G for r < 64 G: the f32 quotient is off by less than 2^-16, half a step of it
// is 2^-13 or more.
__device__ __forceinline__ int over_group(int r, int G) {
    return static_cast<int>((static_cast<float>(r) + 0.5f) * __builtin_amdgcn_rcpf(static_cast<float>(G)));
}

// 32 positions of one KV head, as two tiles of 16: where their codes begin (the
// scales at a sixteenth of that), and whether they are there (a page outside the
// pool is read as page 0 and masked; a tile past the end is the last one again,
// masked by its positions).
struct Place {
    int64_t at[2];
    bool ok[2];
};

// *p, the same for the whole wave and not written by the launch, as a scalar load: a
// vector load would be waited for with every load before it.
__device__ __forceinline__ int32_t uniform(const int32_t *p) {
    return *(const __attribute__((address_space(4))) int32_t *)reinterpret_cast<uintptr_t>(p);
}

// Page `i` of sequence b, 0 and false if there is none.
__device__ __forceinline__ int32_t page_of(const AttnArgs &a, int64_t b, int i, bool &ok) {
    const int32_t page = a.page_table ? uniform(a.page_table + (b * a.max_pages + i)) : static_cast<int32_t>(b);
    ok = static_cast<uint32_t>(page) < static_cast<uint32_t>(a.c.n_pages);
    return ok ? page : 0;
}

// Tile `tile` (16 positions) of sequence b and the one behind it. `of_page`:
// bytes of codes between pages; `of_head`: where the KV head's lie in a page.
template <int D>
__device__ __forceinline__ Place place_of(const AttnArgs &a, int64_t b, int64_t of_page, int64_t of_head, int tile, int last) {
    const int per = a.page_tiles;
    Place p;
    const int i = static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(tile)) * a.page_magic) >> a.page_shift);
    const int in = tile - i * per;
    p.at[0] = page_of(a, b, i, p.ok[0]) * of_page + of_head + static_cast<int64_t>(in) * (16 * D);
    if (tile == last) {
        p.at[1] = p.at[0], p.ok[1] = p.ok[0];
    } else if (in + 1 < per) {
        p.at[1] = p.at[0] + 16 * D, p.ok[1] = p.ok[0];
    } else {
        p.at[1] = page_of(a, b, i + 1, p.ok[1]) * of_page + of_head;
    }
    return p;
}

// v of this lane and of the lane 16 (32) further round, in some order.
template <int kLanes>
__device__ __forceinline__ f32x2 with_other(float v) {
    const uint32_t x = __builtin_bit_cast(uint32_t, v);
    u32x2 r;
    if constexpr (kLanes == 16)
        r = __builtin_amdgcn_permlane16_swap(x, x, false, false);
    else
        r = __builtin_amdgcn_permlane32_swap(x, x, false, false);
    return __builtin_bit_cast(f32x2, r);   // whole: a bit cast of r[1] alone is compiled as one of r[0]
}

__device__ __forceinline__ float max_across(float v) {   // over the four lanes that share lane % 16
    f32x2 r = with_other<16>(v);
    r = with_other<32>(fmaxf(r[0], r[1]));
    return fmaxf(r[0], r[1]);
}

__device__ __forceinline__ float sum_across(float v) {
    f32x2 r = with_other<16>(v);
    r = with_other<32>(r[0] + r[1]);
    return r[0] + r[1];
}

__device__ __forceinline__ f16x2 as_h2(uint32_t v) { return __builtin_bit_cast(f16x2, v); }

__device__ __forceinline__ f32x4 mfma(f16x8 a, f16x8 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
}

union Frag {   // one matrix operand of a lane: eight f16 along the contraction
    f16x8 v;
    f16x2 h[4];
};

// Eight codes (bytes, code + 128) as f16: 0x6400 | (code + 128) is 1024 + 128 + code.
__device__ __forceinline__ f16x8 codes_f16(u32x2 biased) {
    Frag f;
    const f16x2 bias = {static_cast<_Float16>(-1152.0f), static_cast<_Float16>(-1152.0f)};
#pragma unroll
    for (int i = 0; i < 2; i++) {
        const uint32_t u = biased[i];
        f.h[2 * i] = as_h2(__builtin_amdgcn_perm(0x64646464u, u, 0x04010400u)) + bias;
        f.h[2 * i + 1] = as_h2(__builtin_amdgcn_perm(0x64646464u, u, 0x04030402u)) + bias;
    }
    return f.v;
}

// tanh to about 2^-21 of itself: its series below kSeries (the first term left out,
// x^12 / 277, is 2^-26 there), 1 - 2 / (e^2|x| + 1) above.
constexpr float kSeries = 0.35f;

__device__ __forceinline__ float tanh_series(float x) {
    const float y = x * x;
    float r = __builtin_fmaf(y, -1382.0f / 155925.0f, 62.0f / 2835.0f);
    r = __builtin_fmaf(y, r, -17.0f / 315.0f);
    r = __builtin_fmaf(y, r, 2.0f / 15.0f);
    r = __builtin_fmaf(y, r, -1.0f / 3.0f);
    return __builtin_fmaf(x * y, r, x);
}

__device__ __forceinline__ float tanh_any(float x) {
    const float e = __builtin_amdgcn_exp2f(fabsf(x) * (2.0f * kLog2e));
    const float t = __builtin_copysignf(1.0f - 2.0f * __builtin_amdgcn_rcpf(e + 1.0f), x);
    return fabsf(x) < kSeries ? tanh_series(x) : t;
}

// 2^k as f16, -14 <= k <= 15.
__device__ __forceinline__ _Float16 pow2_f16(int k) { return __builtin_bit_cast(_Float16, static_cast<uint16_t>((k + 15) << 10)); }

// Dims of the lane's V operand: VB of them from v_dim on, for operand row m.
template <int D>
__device__ __forceinline__ int v_dim(int m) {
    return D == 64 ? 16 * (m % 4) + 4 * (m / 4) : D == 128 ? 16 * (m % 8) + 8 * (m / 8) : 16 * m;
}

// The keys and values of one step of a wave, as loaded, for each of its two tiles
// of 16 keys: the K codes as they lie in memory, 16 bytes a lane; 16 dims of one of
// the keys 4g .. 4g+3, of which several lanes with one g load all; and scales.
template <int D>
struct Step {
    u32x4 k[2][D / 64], v[2][D / 64];
    uint32_t ks[2], vs[2];
};

__device__ __forceinline__ u32x4 load16(const int8_t *p) {
    return __builtin_nontemporal_load(reinterpret_cast<const u32x4 *>(p));
}

template <int D>
__device__ __forceinline__ void load_keys(const AttnArgs &a, const Place &t, int lane, Step<D> &s) {
    const int n = lane % 16, g = lane / 16;
#pragma unroll
    for (int u = 0; u < 2; u++) {
        const int8_t *p = a.c.k_codes + t.at[u];
        const uint16_t *d = a.c.k_scales + t.at[u] / 32;
#pragma unroll
        for (int i = 0; i < D / 64; i++) s.k[u][i] = load16(p + (1024 * i + 16 * lane));
        // scale number n (two of them for D = 256) of the D/8 of keys 4g .. 4g+3, key-major
        if constexpr (D == 256)
            s.ks[u] = reinterpret_cast<const uint32_t *>(d)[lane];
        else
            s.ks[u] = d[D == 128 ? lane : 8 * g + n % 8];
    }
}

template <int D>
__device__ __forceinline__ void load_values(const AttnArgs &a, const Place &t, int lane, Step<D> &s) {
    const int n = lane % 16, g = lane / 16;
#pragma unroll
    for (int u = 0; u < 2; u++) {
        const int8_t *p = a.c.v_codes + t.at[u];
        const uint32_t *d = reinterpret_cast<const uint32_t *>(a.c.v_scales + t.at[u] / 32);
#pragma unroll
        for (int i = 0; i < D / 64; i++) {
            const int key = D == 64 ? n / 4 : D == 128 ? 2 * (n / 8) + i : i;
            const int piece = D == 64 ? n % 4 : D == 128 ? n % 8 : n;
            s.v[u][i] = load16(p + ((4 * g + key) * D + 16 * piece));
        }
        // the pair of scales with the lane's group in it, of key 4g + n % 4 (a quad of lanes has all four)
        s.vs[u] = d[(4 * g + n % 4) * (D / 64) + v_dim<D>(n) / 64];
    }
}

// The two tiles' K codes turned through the wave's own part of LDS from the order of
// memory (lane after lane, D/16 lanes to a key) to 16 dims of key n per lane, from
// 64 i + 16 g on. The 16-byte pieces of a key are stored in an order that differs
// between the eight keys that one cycle reads, so that they lie in distinct banks.
template <int D>
__device__ __forceinline__ int piece_at(int key, int piece) {
    return key * (D / 16) + (piece ^ (D == 64 ? key / 2 % 4 : key % 8));
}

template <int D>
__device__ __forceinline__ void turn_keys(u32x4 (&k)[2][D / 64], u32x4 (*lds)[D], int lane) {
    constexpr int P = D / 16;   // pieces of a key
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < D / 64; i++) lds[u][piece_at<D>(64 / P * i + lane / P, lane % P)] = k[u][i];
#pragma unroll
    for (int u = 0; u < 2; u++)
#pragma unroll
        for (int i = 0; i < D / 64; i++) k[u][i] = lds[u][piece_at<D>(lane % 16, 4 * i + lane / 16)];
}

// The lane's K operand of every group: the groups 2i and 2i + 1 lie in lanes g < 2
// and g >= 2; the upper lanes' first halves change places with the lower lanes'
// second halves. Codes come out as code + 128.
template <int D>
__device__ __forceinline__ void spread_keys(const u32x4 (&k)[D / 64], u32x2 (&out)[D / 32]) {
#pragma unroll
    for (int i = 0; i < D / 64; i++)
#pragma unroll
        for (int w = 0; w < 2; w++) {
            const u32x2 r = __builtin_amdgcn_permlane32_swap(k[i][w] ^ 0x80808080u, k[i][w + 2] ^ 0x80808080u, false, false);
            out[2 * i][w] = r[0];
            out[2 * i + 1][w] = r[1];
        }
}

// lo and hi of the lanes change places between lane n and the lane kBy further
// in its row of 16: the lanes of the banks kLow keep lo and take the other's lo
// as hi, the others keep hi and take the other's hi as lo.
template <int kBy, int kLow>
__device__ __forceinline__ void exchange(uint32_t &lo, uint32_t &hi) {
    const int l = static_cast<int>(lo), h = static_cast<int>(hi);
    lo = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(l, h, 0x120 + kBy, 0xF, 0xF & ~kLow, false));
    hi = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(h, l, 0x120 + 16 - kBy, 0xF, kLow, false));
}

// out[i][w]: dims v_dim + 4w .. of key 4g + i.
template <int D>
__device__ __forceinline__ void spread_values(const u32x4 (&v)[D / 64], uint32_t (&out)[4][D / 64]) {
    if constexpr (D == 64) {   // lane n: key n / 4, to be dims 4 (n / 4) .. of every key
        uint32_t x[4] = {v[0][0], v[0][1], v[0][2], v[0][3]};
        exchange<8, 0x3>(x[0], x[2]);
        exchange<8, 0x3>(x[1], x[3]);
        exchange<4, 0x5>(x[0], x[1]);
        exchange<4, 0x5>(x[2], x[3]);
#pragma unroll
        for (int i = 0; i < 4; i++) out[i][0] = x[i];
    } else if constexpr (D == 128) {   // lanes n < 8: keys 0 and 1, n >= 8: 2 and 3; to be dims 8 (n / 8) .. of every key
#pragma unroll
        for (int i = 0; i < 2; i++)
#pragma unroll
            for (int w = 0; w < 2; w++) {
                uint32_t lo = v[i][w], hi = v[i][w + 2];
                exchange<8, 0x3>(lo, hi);
                out[i][w] = lo;
                out[2 + i][w] = hi;
            }
    } else {
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int w = 0; w < 4; w++) out[i][w] = v[i][w];
    }
}

// x of lane kLane of each row of 16 lanes.
template <int kLane>
__device__ __forceinline__ float row_lane(float x) {
    return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, x), 0x150 + kLane, 0xF, 0xF, true));
}

template <int kLane>
__device__ __forceinline__ uint32_t quad_lane(uint32_t x) {   // of each quad
    return static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), kLane * 0x55, 0xF, 0xF, true));
}

// The bits of all lanes of a row of 16.
__device__ __forceinline__ uint32_t or_in_row(uint32_t x) {
    x |= static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x121, 0xF, 0xF, true));
    x |= static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x122, 0xF, 0xF, true));
    x |= static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x124, 0xF, 0xF, true));
    return x | static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(x), 0x128, 0xF, 0xF, true));
}

// The largest v of kPer lanes, 8 or 16, side by side in a row of 16.
template <int kPer>
__device__ __forceinline__ float max_of_row(float v) {
    v = max8(v);
    if constexpr (kPer == 16)
        v = fmaxf(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), 0x140, 0xF, 0xF, true)));
    return v;
}

// The scale of key 4g + kKey and group kC from a lane's share of them (f32; the
// second word holds the odd ones for D = 256).
template <int D, int kKey, int kC>
__device__ __forceinline__ float key_scale(const float (&x)[2]) {
    constexpr int at = kKey * (D / 32) + kC;
    return D == 256 ? row_lane<(at / 2) % 16>(x[at % 2]) : row_lane<at % 16>(x[0]);
}

// s[i] += d[i] * the scale of key 4g + i and group kC.
template <int D, int kC>
__device__ __forceinline__ void add_scaled(float (&s)[4], f32x4 d, const float (&x)[2]) {
    if constexpr (kC == 0) {
        s[0] = d[0] * key_scale<D, 0, 0>(x);
        s[1] = d[1] * key_scale<D, 1, 0>(x);
        s[2] = d[2] * key_scale<D, 2, 0>(x);
        s[3] = d[3] * key_scale<D, 3, 0>(x);
    } else {
        s[0] = __builtin_fmaf(key_scale<D, 0, kC>(x), d[0], s[0]);
        s[1] = __builtin_fmaf(key_scale<D, 1, kC>(x), d[1], s[1]);
        s[2] = __builtin_fmaf(key_scale<D, 2, kC>(x), d[2], s[2]);
        s[3] = __builtin_fmaf(key_scale<D, 3, kC>(x), d[3], s[3]);
    }
}

// NS = 2: operands in two f16 parts (f32 inputs), NS = 1: in one. A workgroup
// serves RT tiles of 16 query rows. Waves a SIMD: one tile at head dims 64 and 128 is
// held to three, which f32 at 128 reaches with 166 registers and is on the edge of (left
// alone, it takes 181 or 165 with the text around it: 32 sequences of 8k to 16k keys 180
// us with two waves, 172 with three; 4 rows of 16 sequences 56 and 59).
template <typename T, int D, int NS, int RT>
__global__ __launch_bounds__(kThreads, D <= 128 && RT == 1 ? 3 : D <= 128 || NS == 1 ? 2 : 1) void attn_q8_kernel(AttnArgs a) {
    constexpr int C = D / 32, VB = D / 16, R = 16 * RT;
    typedef f32x4 Joined[R][D / 4 + 1];   // a wave's sums, padded: 16 lanes write one column
    __shared__ union {
        Joined o[kWaves];
        struct {
            u32x4 k[kWaves][2][D];       // the K codes of a wave's two tiles
            u32x4 q[NS][R][D / 8 + 1];   // query rows as f16, padded: 16 lanes read one column
        } in;
    } lds;
    __shared__ float lds_scale[R];
    __shared__ float lds_m[kWaves][R], lds_l[kWaves][R];
    const int Hkv = static_cast<int>(a.c.n_kv_heads);
    // A sequence's blocks of rows side by side: they read the same keys (64 drafted tokens
    // of four sequences 86.5 us with blocks slowest, 84.5 so).
    const int kvh = blockIdx.x, split = blockIdx.y;
    const uint32_t blocks = static_cast<uint32_t>(a.row_blocks);
    const int64_t b = blockIdx.z / blocks;
    const int r0 = (a.row_block0 + static_cast<int>(blockIdx.z % blocks)) * R;
    const Seq sq(a, b);
    const int G = static_cast<int>(a.n_heads) / Hkv;
    const int rows = sq.rows * G;   // of this KV head
    // A sequence has ceil(len / chunk) parts, and at least one, which also serves the
    // rows of an empty sequence.
    if (r0 >= rows || (split > 0 && split * a.chunk >= sq.len)) return;
    const bool only = sq.len <= a.chunk;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / 64);
    const int lane = threadIdx.x % 64, n = lane % 16, g = lane / 16;
    const int len = static_cast<int>(sq.len), ctx = static_cast<int>(sq.ctx);
    const int j0 = static_cast<int>(split * a.chunk);
    const int j1 = j0 + static_cast<int>(a.chunk) < len ? j0 + static_cast<int>(a.chunk) : len;

    // The query rows, prepared by all waves together: kPerRow threads to a row, E dims
    // each. A row past the last repeats the first; what comes of it is not written.
    constexpr int kPerRow = kThreads / R, E = D / kPerRow;
    const int row = static_cast<int>(threadIdx.x) / kPerRow, d0 = static_cast<int>(threadIdx.x) % kPerRow * E;
    typename Vec4<T>::type raw[E / 4];   // as loaded: a conversion here would wait for them
    {
        const int r = r0 + row < rows ? r0 + row : r0;
        const int t = over_group(r, G), h = kvh * G + r - t * G;
        const T *p = static_cast<const T *>(a.q) + ((sq.row0 + t) * a.n_heads + h) * D + d0;
#pragma unroll
        for (int i = 0; i < E / 4; i++) raw[i] = *reinterpret_cast<const typename Vec4<T>::type *>(p + 4 * i);
    }
    uint64_t word[RT];      // the drafted keys that the lane's rows see
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int r = r0 + 16 * rt + n < rows ? r0 + 16 * rt + n : r0;
        const int t = over_group(r, G);
        word[rt] = a.tree ? a.tree[sq.row0 + t] : (t >= 63 ? ~0ull : (1ull << (t + 1)) - 1);
    }
    __builtin_amdgcn_sched_barrier(0);

    Step<D> st;
    int j = j0 + kStep * wave;
    const int last = (j1 > 0 ? j1 - 1 : 0) / 16;
    const int64_t of_page = a.c.page_size * Hkv * D, of_head = a.c.page_size * kvh * D;
    // Keys are loaded before values everywhere, and the scheduler is kept from mixing
    // the two: loads complete in order, and a wait for the keys must not include the
    // values behind them. A wave without keys loads the last tile and does not use it:
    // with as many loads on every path, the wait for the queries is for them alone.
    Place next = place_of<D>(a, b, of_page, of_head, j / 16 < last ? j / 16 : last, last);
    load_keys<D>(a, next, lane, st);
    __builtin_amdgcn_sched_barrier(0);
    load_values<D>(a, next, lane, st);
    __builtin_amdgcn_sched_barrier(0);

    // A query row times a power of two that brings its largest value into [2^13, 2^14).
    {
        f32x4 qx[E / 4];
        float mx = 0.0f;
#pragma unroll
        for (int i = 0; i < E / 4; i++) {
            qx[i] = __builtin_convertvector(raw[i], f32x4);
#pragma unroll
            for (int x = 0; x < 4; x++) mx = fmaxf(mx, fabsf(qx[i][x]));
        }
        mx = max_of_row<kPerRow>(mx);
        const int e = mx > 0.0f && mx <= 3.40282347e38f ? 14 - __builtin_amdgcn_frexp_expf(mx) : 0;
        // Finite, so that a product of 0 stays a score of 0 (a larger factor would take any other past the cap).
        if (d0 == 0) lds_scale[row] = ldexpf(a.factor, a.factor_exp - e < 127 ? a.factor_exp - e : 127);
        f16x2 hi[E / 2], lo[E / 2];
#pragma unroll
        for (int i = 0; i < E; i += 2) {
            const float v0 = ldexpf(qx[i / 4][i % 4], e), v1 = ldexpf(qx[i / 4][i % 4 + 1], e);
            hi[i / 2] = f16x2{static_cast<_Float16>(v0), static_cast<_Float16>(v1)};
            if constexpr (NS == 2)
                lo[i / 2] = f16x2{static_cast<_Float16>(v0 - static_cast<float>(hi[i / 2][0])),
                                  static_cast<_Float16>(v1 - static_cast<float>(hi[i / 2][1]))};
        }
        f16x2 *to = reinterpret_cast<f16x2 *>(lds.in.q[0][row]) + d0 / 2;
#pragma unroll
        for (int i = 0; i < E / 2; i++) to[i] = hi[i];
        if constexpr (NS == 2) {
            to = reinterpret_cast<f16x2 *>(lds.in.q[NS - 1][row]) + d0 / 2;
#pragma unroll
            for (int i = 0; i < E / 2; i++) to[i] = lo[i];
        }
    }
    __syncthreads();
    Frag q[RT][C][NS];
    float scale2[RT];       // from a contraction to a score (times log2 e without a cap)
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        scale2[rt] = lds_scale[16 * rt + n];
#pragma unroll
        for (int c = 0; c < C; c++)
#pragma unroll
            for (int i = 0; i < NS; i++)
                q[rt][c][i].v = __builtin_bit_cast(f16x8, lds.in.q[i][16 * rt + n][4 * c + 2 * (g % 2) + g / 2]);
    }

    f32x4 o[RT][VB];   // o[rt][t][i]: dim v_dim(4g + i) + t of row n
    float m[RT], l[RT];
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        m[rt] = kNone;
        l[rt] = 0.0f;
#pragma unroll
        for (int t = 0; t < VB; t++) o[rt][t] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // Powers of two on the V scales: 2^vk in all, so that the largest seen lies
    // below 2^15 (below 2^15 without a change: vlim of the raw scale).
    int vk = 15;
    _Float16 vmul = pow2_f16(15);
    _Float16 vlim = static_cast<_Float16>(0.0f);   // the largest scale that vk was made for

    // One step; kMore: there is another, whose loads it issues. The last one is a copy of
    // its own, since a wait for loads counts those behind them, which have to be there on
    // every path.
    const auto step = [&](auto more) {
        constexpr bool kMore = decltype(more)::value;
        const bool ok[2] = {next.ok[0], next.ok[1]};
        const bool plain = j + kStep <= (ctx < j1 ? ctx : j1) && ok[0] && ok[1];   // every row sees every key
        if constexpr (kMore) next = place_of<D>(a, b, of_page, of_head, (j + kGroupKeys) / 16, last);
        float s[RT][2][4];
        turn_keys<D>(st.k, lds.in.k[wave], lane);
#pragma unroll
        for (int u = 0; u < 2; u++) {
            u32x2 kw[C];
            spread_keys<D>(st.k[u], kw);
            const f16x2 ks = as_h2(st.ks[u]);
            const float x[2] = {static_cast<float>(ks[0]), static_cast<float>(ks[1])};
            const auto group = [&](auto cc) {
                constexpr int c = decltype(cc)::value;
                const f16x8 kf = codes_f16(kw[c]);
#pragma unroll
                for (int rt = 0; rt < RT; rt++) {
                    f32x4 d = mfma(kf, q[rt][c][0].v, f32x4{0.0f, 0.0f, 0.0f, 0.0f});
                    if constexpr (NS == 2) d = mfma(kf, q[rt][c][NS - 1].v, d);
                    add_scaled<D, c>(s[rt][u], d, x);
                }
            };
            group(std::integral_constant<int, 0>{});
            group(std::integral_constant<int, 1>{});
            if constexpr (C > 2) {
                group(std::integral_constant<int, 2>{});
                group(std::integral_constant<int, 3>{});
            }
            if constexpr (C > 4) {
                group(std::integral_constant<int, 4>{});
                group(std::integral_constant<int, 5>{});
                group(std::integral_constant<int, 6>{});
                group(std::integral_constant<int, 7>{});
            }
            // One tile's operands at a time in registers: its scores are made here, not
            // where they are used next.
#pragma unroll
            for (int rt = 0; rt < RT; rt++)
                asm volatile("" : "+v"(s[rt][u][0]), "+v"(s[rt][u][1]), "+v"(s[rt][u][2]), "+v"(s[rt][u][3]));
            __builtin_amdgcn_sched_barrier(0);
        }
        if constexpr (kMore) load_keys<D>(a, next, lane, st);
        __builtin_amdgcn_sched_barrier(0);
        // Weights, each lane its 8 keys of row n.
        Frag p[RT][NS];
        uint32_t seen = 0;   // bit x: a row of this lane sees key x of its eight (set where not all do)
#pragma unroll
        for (int rt = 0; rt < RT; rt++) {
#pragma unroll
            for (int x = 0; x < 8; x++) s[rt][x / 4][x % 4] *= scale2[rt];
            if (a.softcap > 0.0f) {
                float far = 0.0f;
#pragma unroll
                for (int x = 0; x < 8; x++) far = fmaxf(far, fabsf(s[rt][x / 4][x % 4]));
                if (__any(far >= kSeries)) {
#pragma unroll
                    for (int x = 0; x < 8; x++) s[rt][x / 4][x % 4] = tanh_any(s[rt][x / 4][x % 4]) * (a.softcap * kLog2e);
                } else {   // scores well below the cap, the usual ones: no exponential for them
#pragma unroll
                    for (int x = 0; x < 8; x++) s[rt][x / 4][x % 4] = tanh_series(s[rt][x / 4][x % 4]) * (a.softcap * kLog2e);
                }
            }
            if (!plain) {
#pragma unroll
                for (int x = 0; x < 8; x++) {
                    const int jj = j + 16 * (x / 4) + 4 * g + x % 4;
                    const bool sees = ok[x / 4] && jj < j1 && (jj < ctx || ((word[rt] >> ((jj - ctx) & 63)) & 1));
                    s[rt][x / 4][x % 4] = sees ? s[rt][x / 4][x % 4] : -__builtin_inff();
                    seen |= sees ? 1u << x : 0u;
                }
            }
            float mx = m[rt];
#pragma unroll
            for (int x = 0; x < 8; x++) mx = fmaxf(mx, s[rt][x / 4][x % 4]);
            if (__any(mx > m[rt])) {   // no row's maximum grows in most steps of a long sequence
                const float mn = max_across(mx);
                const float corr = __builtin_amdgcn_exp2f(m[rt] - mn);
                m[rt] = mn;
                l[rt] *= corr;
#pragma unroll
                for (int t = 0; t < VB; t++) o[rt][t] *= corr;
            }
            const float off = m[rt] - kWeightBits;
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int i = 0; i < 4; i += 2) {
                    const float p0 = __builtin_amdgcn_exp2f(s[rt][u][i] - off), p1 = __builtin_amdgcn_exp2f(s[rt][u][i + 1] - off);
                    l[rt] += p0 + p1;
                    const f16x2 hi = {static_cast<_Float16>(p0), static_cast<_Float16>(p1)};
                    p[rt][0].h[2 * u + i / 2] = hi;
                    if constexpr (NS == 2)
                        p[rt][NS - 1].h[2 * u + i / 2] = f16x2{static_cast<_Float16>(p0 - static_cast<float>(hi[0])),
                                                               static_cast<_Float16>(p1 - static_cast<float>(hi[1]))};
                }
        }
        // The V scales of the lane's 8 keys at its dims' group, in pairs.
        uint32_t pr[2][2];
        {
            const uint32_t sel = (v_dim<D>(n) / 32) % 2 ? 0x07060302u : 0x05040100u;
#pragma unroll
            for (int u = 0; u < 2; u++) {
                pr[u][0] = __builtin_amdgcn_perm(quad_lane<1>(st.vs[u]), quad_lane<0>(st.vs[u]), sel);
                pr[u][1] = __builtin_amdgcn_perm(quad_lane<3>(st.vs[u]), quad_lane<2>(st.vs[u]), sel);
            }
        }
        // The row of a key that none of the 16 RT rows sees need not have been stored: its
        // scales may be anything, and weights of 0 would hide neither an infinity nor, since
        // the largest scale sets the others' power of two, a scale far above the others.
        if (!plain) {
            seen = or_in_row(seen);
#pragma unroll
            for (int x = 0; x < 8; x += 2)
                pr[x / 4][x / 2 % 2] &= ((seen >> x & 1) ? 0x0000ffffu : 0u) | ((seen >> (x + 1) & 1) ? 0xffff0000u : 0u);
        }
        f16x2 vs[2][2];
#pragma unroll
        for (int x = 0; x < 4; x++) vs[x / 2][x % 2] = as_h2(pr[x / 2][x % 2]);
        f16x2 top = __builtin_elementwise_max(__builtin_elementwise_max(vs[0][0], vs[0][1]),
                                              __builtin_elementwise_max(vs[1][0], vs[1][1]));
        _Float16 lane_top = top[0] > top[1] ? top[0] : top[1];
        if (__any(lane_top > vlim)) {   // a scale above those that vk was made for (rare after the first steps)
            float w = static_cast<float>(lane_top);
#pragma unroll
            for (int x = 32; x >= 1; x >>= 1) w = fmaxf(w, __shfl_xor(w, x));
            int k = 15 - __builtin_amdgcn_frexp_expf(w);   // w 2^k in [2^14, 2^15)
            k = k < vk ? k : vk;
            vlim = static_cast<_Float16>(k < 15 ? ldexpf(1.0f, 15 - k) : 1.0f);   // exact, at most 2^16 (infinity)
            if (k != vk) {
                const float f = ldexpf(1.0f, k - vk);
#pragma unroll
                for (int rt = 0; rt < RT; rt++)
#pragma unroll
                    for (int t = 0; t < VB; t++) o[rt][t] *= f;
                vk = k;
                vmul = pow2_f16(k);
            }
        }
#pragma unroll
        for (int u = 0; u < 2; u++)
#pragma unroll
            for (int i = 0; i < 2; i++) vs[u][i] *= f16x2{vmul, vmul};
        uint32_t vx[2][4][VB / 4];
#pragma unroll
        for (int u = 0; u < 2; u++) {
            u32x4 biased[D / 64];
#pragma unroll
            for (int i = 0; i < D / 64; i++) biased[i] = st.v[u][i] ^ 0x80808080u;
            spread_values<D>(biased, vx[u]);
        }
#pragma unroll
        for (int t = 0; t < VB; t++) {
            // byte t of two keys as (code + 128) 2^-24 (f16's smallest steps), times 2^14, less 2^-3: code 2^-10
            const uint32_t sel = 0x0c000c00u | static_cast<uint32_t>((4 + t % 4) << 16) | static_cast<uint32_t>(t % 4);
            const f16x2 up = {pow2_f16(14), pow2_f16(14)}, off = {static_cast<_Float16>(-0.125f), static_cast<_Float16>(-0.125f)};
            Frag vh, vl;
#pragma unroll
            for (int u = 0; u < 2; u++)
#pragma unroll
                for (int i = 0; i < 2; i++) {
                    const f16x2 x = as_h2(__builtin_amdgcn_perm(vx[u][2 * i + 1][t / 4], vx[u][2 * i][t / 4], sel));
                    const f16x2 c = __builtin_elementwise_fma(x, up, off);
                    vh.h[2 * u + i] = c * vs[u][i];
                    if constexpr (NS == 2) vl.h[2 * u + i] = __builtin_elementwise_fma(c, vs[u][i], -vh.h[2 * u + i]);
                }
#pragma unroll
            for (int rt = 0; rt < RT; rt++) {
                o[rt][t] = mfma(vh.v, p[rt][0].v, o[rt][t]);
                if constexpr (NS == 2) {
                    o[rt][t] = mfma(vl.v, p[rt][0].v, o[rt][t]);
                    o[rt][t] = mfma(vh.v, p[rt][NS - 1].v, o[rt][t]);
                }
            }
        }
        // Behind the products, in registers that they have left (before them: f32 of 8k to
        // 16k keys 182 us where this takes 172; 8 tokens of 16 sequences 62 and 62.5).
        __builtin_amdgcn_sched_barrier(0);
        if constexpr (kMore) load_values<D>(a, next, lane, st);
        __builtin_amdgcn_sched_barrier(0);
    };
    for (; j + kGroupKeys < j1; j += kGroupKeys) step(std::true_type{});
    if (j < j1) step(std::false_type{});

    // Join the four waves.
    __syncthreads();   // the K codes are no longer needed by any
#pragma unroll
    for (int rt = 0; rt < RT; rt++) {
        const int r = 16 * rt + n;
        const float sum = sum_across(l[rt]);
        if (g == 0) {
            lds_m[wave][r] = m[rt];
            lds_l[wave][r] = sum;
        }
        const float f = ldexpf(1.0f, 10 - vk);   // codes were held times 2^-10
#pragma unroll
        for (int i = 0; i < 4; i++)
#pragma unroll
            for (int t = 0; t < VB; t += 4)
                lds.o[wave][r][(v_dim<D>(4 * g + i) + t) / 4] =
                    f32x4{o[rt][t][i], o[rt][t + 1][i], o[rt][t + 2][i], o[rt][t + 3][i]} * f;
    }
    __syncthreads();
    const int r = row;
    if (r0 + r >= rows) return;
    float mx = lds_m[0][r];
#pragma unroll
    for (int w = 1; w < kWaves; w++) mx = fmaxf(mx, lds_m[w][r]);
    float sum = 0.0f, f[kWaves];
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        f[w] = __builtin_amdgcn_exp2f(lds_m[w][r] - mx);
        sum += lds_l[w][r] * f[w];
    }
    const int t = over_group(r0 + r, G), h = kvh * G + (r0 + r) - t * G;
    const int64_t at = (sq.row0 + t) * a.n_heads + h;
    const float inv = only ? (sum > 0.0f ? 1.0f / sum : 0.0f) : 1.0f;
    float *part = a.part_o + (at * a.splits + split) * D;
    for (int d4 = threadIdx.x % kPerRow; d4 < D / 4; d4 += kPerRow) {
        f32x4 x = lds.o[0][r][d4] * f[0];
#pragma unroll
        for (int w = 1; w < kWaves; w++) x += lds.o[w][r][d4] * f[w];
        if (only)
            store4(static_cast<T *>(a.out) + at * D + 4 * d4, x * inv);
        else
            *reinterpret_cast<f32x4 *>(part + 4 * d4) = x;
    }
    if (!only && threadIdx.x % kPerRow == 0)
        *reinterpret_cast<f32x2 *>(a.part_ml + (at * a.splits + split) * 2) = f32x2{mx, sum};
}

// Joins the parts of one query row and head. A step takes 64 parts: lane i of every
// wave holds part i's maximum and sum, wave w adds up the parts w, w + 4, ..., D/64
// dims to a lane, all of them loaded before any is used. 5.2 us for 1024 rows of 16
// parts (8.5 MB), of which a launch is about 2: bound by its two loads in a chain.
template <typename T, int D>
__global__ __launch_bounds__(kThreads) void attn_q8_merge_kernel(AttnArgs a) {
    constexpr int E = D / 64, kPer = 64 / kWaves;
    __shared__ float lds_o[kWaves][D];
    const Seq sq(a, blockIdx.z);
    if (static_cast<int>(blockIdx.y) >= sq.rows || sq.len <= a.chunk) return;   // a single part is written by itself
    const int parts = static_cast<int>(static_cast<uint32_t>(sq.len - 1) / static_cast<uint32_t>(a.chunk)) + 1;
    const int64_t at = (sq.row0 + blockIdx.y) * a.n_heads + blockIdx.x;
    const float *po = a.part_o + at * a.splits * D, *pml = a.part_ml + at * a.splits * 2;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / 64), lane = threadIdx.x % 64;
    float m = kNone, l = 0.0f, o[E];
#pragma unroll
    for (int i = 0; i < E; i++) o[i] = 0.0f;
    for (int p0 = 0; p0 < parts; p0 += 64) {
        const int mine = p0 + lane < parts ? p0 + lane : parts - 1;   // clamped: weighed 0 below
        const f32x2 ml = *reinterpret_cast<const f32x2 *>(pml + 2 * mine);
        float x[kPer][E];
#pragma unroll
        for (int k = 0; k < kPer; k++) {
            if (p0 + kWaves * k >= parts) break;
            const int part = p0 + kWaves * k + wave < parts ? p0 + kWaves * k + wave : parts - 1;
#pragma unroll
            for (int i = 0; i < E; i++) x[k][i] = po[static_cast<int64_t>(part) * D + lane * E + i];
        }
        const float pm = p0 + lane < parts ? ml[0] : kNone;
        float mn = fmaxf(m, pm);
#pragma unroll
        for (int s = 32; s >= 1; s >>= 1) mn = fmaxf(mn, __shfl_xor(mn, s));
        const float before = __builtin_amdgcn_exp2f(m - mn);
        const float w = p0 + lane < parts ? __builtin_amdgcn_exp2f(pm - mn) : 0.0f;
        l = l * before + w * ml[1];   // per lane
        m = mn;
#pragma unroll
        for (int i = 0; i < E; i++) o[i] *= before;
#pragma unroll
        for (int k = 0; k < kPer; k++) {
            if (p0 + kWaves * k >= parts) break;
            const float f = __builtin_bit_cast(
                float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, w), kWaves * k + wave));
#pragma unroll
            for (int i = 0; i < E; i++) o[i] = __builtin_fmaf(x[k][i], f, o[i]);
        }
    }
#pragma unroll
    for (int s = 32; s >= 1; s >>= 1) l += __shfl_xor(l, s);   // every wave has all parts' sums
#pragma unroll
    for (int i = 0; i < E; i++) lds_o[wave][lane * E + i] = o[i];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += kThreads) {
        const float x = (lds_o[0][d] + lds_o[1][d]) + (lds_o[2][d] + lds_o[3][d]);
        static_cast<T *>(a.out)[at * D + d] = static_cast<T>(l > 0.0f ? x / l : 0.0f);
    }
}

// Parts per sequence. While there is not a workgroup for every CU at one part each
// (kCus), parts are made for kFill workgroups, however short they get; a call with more
// rows than a block for kFillBlocks, since the later blocks are empty in sequences of fewer
// rows. (Parts are rounded up: 80 groups become 560.) Beyond that, parts of no fewer than
// kMinSteps steps a wave, up to kFine workgroups in all: many of them even out the end of
// the launch and sequences of different lengths, but each prepares its queries and joins
// its waves anew.
// kFill and kFillBlocks are what measured best on these shapes, not what a CU holds: of
// one tile of rows that is four workgroups at head dim 64, three at 128, and two (f32: one)
// at 256; of two tiles three and two. Measured (bf16, head dim 128, 32 / 8 heads), planned
// for 384, 512 and 768: 8 sequences of 2k to 4k keys 20.4, 16.6 and 17.9 us, one of 32k 21.0,
// 18.0 and 20.9, trees of up to 13 over 2.5k to 5k keys (two blocks) 26.9, 29.6 and 24.6.
// Where they lose: two blocks that are both full are slower planned for 768 than for 512
// (13 rows of each of three sequences of 5k keys 30.7 and 25.3 us, of five 43 and 42, 16 rows
// of eight of 4k 52 and 44, 33 rows of two of 8k 57 and 54, 64 rows of one 45 and 39), and f32
// at head dim 256 planned for 512 than for 256 (8 sequences of 2k to 4k keys 24.3 and 20.4 us,
// one of 32k 27.9 and 21.9).
// kMinSteps: 128 sequences of 1k keys 50 us with parts of 4 steps, 41 with 8; 48 of 512 keys
// (one and a half for each CU) 13.4 us whole, 16.3 in two parts. kFine: 32 sequences of 16k
// to 32k keys 281 with 4096 workgroups or 6144, and 6 % more with 2048.
constexpr int kCus = 256, kFill = 512, kFillBlocks = 768, kFine = 4096, kMinSteps = 8;

// How the work is cut: rows per workgroup, and keys per part.
struct Plan {
    int row_tiles;       // RT
    int64_t row_blocks, chunk, splits;
};

Plan plan_of(int64_t n_seqs, int64_t n_heads, int64_t n_kv_heads, int64_t head_dim, int64_t max_q, int64_t max_kv_len) {
    Plan p;
    const int64_t rows = max_q * (n_heads / n_kv_heads);
    // Two tiles of 16 rows share a step's conversions (64 drafted tokens of four sequences over 8k keys 87 us, 112 with
    // one, 24.5 against 34 for five trees of up to 13, though 8 tokens of one over 4k 12.7 against 12.1); for head dim
    // 256 their sums do not fit the registers.
    p.row_tiles = rows > 16 && head_dim <= 128 ? 2 : 1;
    p.row_blocks = (rows + 16 * p.row_tiles - 1) / (16 * p.row_tiles);
    const int64_t groups = n_seqs * n_kv_heads * p.row_blocks;   // at one part each
    const int64_t steps = (max_kv_len + kGroupKeys - 1) / kGroupKeys;
    const int64_t most = p.row_blocks > 1 ? kFillBlocks : kFill;
    const int64_t fill = groups < kCus ? (most + groups - 1) / groups : 1, fine = (kFine + groups - 1) / groups;
    int64_t parts = fine < steps / kMinSteps ? fine : steps / kMinSteps;
    parts = parts > fill ? parts : fill;
    parts = parts < steps ? parts : steps;
    p.chunk = (steps + parts - 1) / parts * kGroupKeys;
    p.splits = (max_kv_len + p.chunk - 1) / p.chunk;
    return p;
}

// Rows of partial sums that the workspace has to hold: an upper bound on n_q * n_heads *
// splits of this call and of every call that is no larger in n_seqs, n_q, max_q and
// max_kv_len (the same heads), and itself no smaller for a larger call, so that a
// workspace made for the largest call serves the others. The plan's own product is not:
// a call of more sequences or more keys may be cut into fewer parts. Two bounds, the
// smaller one taken: every row in as many parts as the smallest batch is cut into, and as
// many workgroups as any plan makes, each with the rows of its block. With g workgroups at
// one part each, ceil(c / g) parts are at most c + g - 1 workgroups, for g < kCus where a
// plan fills the CUs and for g < kFine where it cuts finer.
int64_t part_rows(int64_t n_seqs, int64_t n_q, int64_t n_heads, int64_t n_kv_heads, int64_t head_dim, int64_t max_q,
                  int64_t max_kv_len) {
    const int64_t rows = max_q * (n_heads / n_kv_heads), tall = head_dim <= 128 ? 32 : 16;   // of a KV head, of a block
    const int64_t row_blocks = rows <= 16 ? 1 : (rows + tall - 1) / tall;
    const int64_t groups = n_seqs * n_kv_heads * row_blocks;
    const int64_t steps = (max_kv_len + kGroupKeys - 1) / kGroupKeys, fine = steps / kMinSteps;
    const int64_t most = row_blocks > 1 ? kFillBlocks : kFill;
    const int64_t fill1 = n_kv_heads < kCus ? (most + n_kv_heads - 1) / n_kv_heads : 1;   // one sequence, one block
    const int64_t fine1 = (kFine + n_kv_heads - 1) / n_kv_heads;
    int64_t parts = fine < fine1 ? fine : fine1;
    parts = parts > fill1 ? parts : fill1;
    parts = parts < steps ? parts : steps;
    if (parts <= 1) return 0;
    int64_t workgroups = most + (groups < kCus - 1 ? groups : kCus - 1) - 1;
    if (fine > 1) {
        const int64_t cut = kFine + (groups < kFine - 1 ? groups : kFine - 1) - 1;
        const int64_t n = groups * fine < cut ? groups * fine : cut;
        workgroups = workgroups > n ? workgroups : n;
    }
    workgroups = workgroups < groups * steps ? workgroups : groups * steps;
    const int64_t by_parts = n_q * n_heads * parts, by_blocks = (rows < tall ? rows : tall) * workgroups;
    return by_parts < by_blocks ? by_parts : by_blocks;
}

int check_sizes(const char *name, int64_t n_seqs, int64_t n_q, int64_t n_heads, int64_t n_kv_heads, int64_t head_dim,
                int64_t max_q, int64_t max_kv_len) {
    GD_REQUIRE(n_seqs >= 1 && n_q >= 1 && n_heads >= 1 && n_kv_heads >= 1 && max_q >= 1 && max_kv_len >= 1, GD_EINVAL,
               "%s: n_seqs (%lld), n_q (%lld), n_heads (%lld), n_kv_heads (%lld), max_q (%lld) and max_kv_len (%lld) "
               "must be >= 1", name, (long long)n_seqs, (long long)n_q, (long long)n_heads, (long long)n_kv_heads,
               (long long)max_q, (long long)max_kv_len);
    GD_REQUIRE(head_dim == 64 || head_dim == 128 || head_dim == 256, GD_ESHAPE,
               "%s: head_dim (%lld) must be 64, 128 or 256", name, (long long)head_dim);
    GD_REQUIRE(n_heads % n_kv_heads == 0, GD_ESHAPE, "%s: n_heads (%lld) not a multiple of n_kv_heads (%lld)", name,
               (long long)n_heads, (long long)n_kv_heads);
    GD_REQUIRE(max_q <= 64 && n_heads <= 4096 && n_seqs <= 65535 && n_q <= n_seqs * max_q &&
                   max_kv_len <= (INT64_C(1) << 30),
               GD_ERANGE, "%s: max_q (%lld) above 64, n_q (%lld) above n_seqs * max_q, or a size too large", name,
               (long long)max_q, (long long)n_q);
    return GD_OK;
}

}  // namespace

extern "C" int attn_decode_q8_workspace_bytes(int64_t n_seqs, int64_t n_q, int64_t n_heads, int64_t n_kv_heads,
                                              int64_t head_dim, int64_t max_q, int64_t max_kv_len, size_t *bytes) {
    GD_REQUIRE(bytes, GD_EINVAL, "attn_decode_q8_workspace_bytes: null output pointer");
    int st = check_sizes("attn_decode_q8_workspace_bytes", n_seqs, n_q, n_heads, n_kv_heads, head_dim, max_q, max_kv_len);
    if (st) return st;
    // a sum of head_dim values, a maximum and a denominator per row, head and part
    const int64_t rows = part_rows(n_seqs, n_q, n_heads, n_kv_heads, head_dim, max_q, max_kv_len);
    *bytes = rows > 0 ? static_cast<size_t>(rows * (head_dim + 2) * 4) : 16;
    clear_error();
    return GD_OK;
}

extern "C" int attn_decode_q8(const gd_kv_q8 *cache, const void *q, void *out, const int32_t *page_table,
                              int64_t max_pages, const int32_t *kv_lens, const int32_t *q_start,
                              const uint64_t *tree_mask, int64_t n_seqs, int64_t n_q, int64_t n_heads, int64_t max_q,
                              int64_t max_kv_len, float scale, float softcap, int32_t dtype, void *workspace,
                              size_t workspace_bytes, void *stream) {
    int st = check_kv_q8(cache, "attn_decode_q8");
    if (st) return st;
    GD_REQUIRE(q && out && kv_lens, GD_EINVAL, "attn_decode_q8: null pointer");
    GD_REQUIRE(dtype_ok(dtype), GD_EINVAL, "attn_decode_q8: unknown dtype %d", dtype);
    st = check_sizes("attn_decode_q8", n_seqs, n_q, n_heads, cache->n_kv_heads, cache->head_dim, max_q, max_kv_len);
    if (st) return st;
    GD_REQUIRE(q_start || n_q == n_seqs * max_q, GD_EINVAL,
               "attn_decode_q8: without q_start every sequence has max_q (%lld) rows: n_q (%lld) must be n_seqs * max_q",
               (long long)max_q, (long long)n_q);
    GD_REQUIRE(scale - scale == 0.0f, GD_EINVAL, "attn_decode_q8: scale must be finite");
    GD_REQUIRE(softcap >= 0.0f && softcap <= 1e30f, GD_EINVAL,
               "attn_decode_q8: softcap must be in [0, 1e30] (0: none)");
    GD_REQUIRE(page_table ? max_pages >= 1 : cache->n_pages >= n_seqs, GD_EINVAL,
               "attn_decode_q8: max_pages must be >= 1 with a page table, the cache must have a page per sequence without");
    int64_t cap;
    GD_REQUIRE(max_pages <= INT64_C(2147483647) && mul_ok(page_table ? max_pages : 1, cache->page_size, &cap), GD_ERANGE,
               "attn_decode_q8: max_pages too large");
    GD_REQUIRE(max_kv_len <= cap, GD_EINVAL, "attn_decode_q8: max_kv_len (%lld) above the %lld positions of a sequence's pages",
               (long long)max_kv_len, (long long)cap);
    GD_REQUIRE(aligned(q, 16) && aligned(out, 16) && aligned(page_table, 4) && aligned(kv_lens, 4) &&
                   aligned(q_start, 4) && aligned(tree_mask, 8),
               GD_EALIGN, "attn_decode_q8: q and out must be 16-byte aligned, tree_mask 8-byte, the other arrays 4-byte");
    size_t need;
    st = attn_decode_q8_workspace_bytes(n_seqs, n_q, n_heads, cache->n_kv_heads, cache->head_dim, max_q, max_kv_len, &need);
    if (st) return st;
    GD_REQUIRE(workspace, GD_EINVAL, "attn_decode_q8: null workspace");
    GD_REQUIRE(aligned(workspace, 16), GD_EALIGN, "attn_decode_q8: workspace must be 16-byte aligned");
    GD_REQUIRE(workspace_bytes >= need, GD_ERANGE, "attn_decode_q8: workspace of %zu bytes, %zu needed",
               workspace_bytes, need);
    const int64_t row_bytes = n_q * n_heads * cache->head_dim * dtype_size(dtype);
    GD_REQUIRE(!overlaps(q, row_bytes, row_bytes, 1, out, row_bytes), GD_EINVAL,
               "attn_decode_q8: out must not overlap q");
    const Plan p = plan_of(n_seqs, n_heads, cache->n_kv_heads, cache->head_dim, max_q, max_kv_len);
    AttnArgs a;
    a.c = *cache;
    a.q = q, a.out = out, a.page_table = page_table, a.kv_lens = kv_lens, a.q_start = q_start, a.tree = tree_mask;
    a.max_pages = max_pages, a.n_q = n_q, a.n_heads = n_heads, a.max_q = max_q;
    a.max_kv_len = max_kv_len, a.softcap = softcap;
    // apart from its power of two: scale / softcap can pass f32's range where, times the queries', it does not
    int factor_exp;
    a.factor = static_cast<float>(std::frexp(
        softcap > 0.0f ? static_cast<double>(scale) / softcap : static_cast<double>(scale) * kLog2e, &factor_exp));
    a.factor_exp = factor_exp;
    a.chunk = p.chunk, a.splits = static_cast<int32_t>(p.splits);
    // 16-key tiles (fewer than 2^27) to pages by a multiplication: with 2^(L-1) < per <= 2^L and
    // magic = ceil(2^(31+L) / per), tile * (magic * per - 2^(31+L)) < 2^(27+L), so the quotient is exact.
    const uint64_t per = static_cast<uint64_t>(cache->page_size / 16);
    int shift = 31;
    while ((UINT64_C(1) << (shift - 31)) < per) shift++;
    a.page_magic = static_cast<uint32_t>(((UINT64_C(1) << shift) + per - 1) / per);
    a.page_shift = shift;
    a.page_tiles = static_cast<int32_t>(per);
    a.part_o = static_cast<float *>(workspace);
    a.part_ml = a.part_o + n_q * n_heads * p.splits * cache->head_dim;
    const dim3 merge_grid(static_cast<uint32_t>(n_heads), static_cast<uint32_t>(max_q), static_cast<uint32_t>(n_seqs));
    hipStream_t hs = as_stream(stream);
    dispatch_dtype(dtype, [&](auto t) {
        using T = decltype(t);
        constexpr int NS = sizeof(T) == 4 ? 2 : 1;
        const auto launch = [&](auto dim) {
            constexpr int D = decltype(dim)::value;
            const int64_t most = 65535 / n_seqs;   // blocks of rows that one grid holds: all of them, but for huge batches
            for (int64_t rb = 0; rb < p.row_blocks; rb += most) {
                const int64_t blocks = p.row_blocks - rb < most ? p.row_blocks - rb : most;
                const dim3 grid(static_cast<uint32_t>(cache->n_kv_heads), static_cast<uint32_t>(p.splits),
                                static_cast<uint32_t>(n_seqs * blocks));
                a.row_block0 = static_cast<int32_t>(rb), a.row_blocks = static_cast<int32_t>(blocks);
                if (p.row_tiles == 2) {
                    if constexpr (D <= 128)
                        hipLaunchKernelGGL((attn_q8_kernel<T, D, NS, 2>), grid, dim3(kThreads), 0, hs, a);
                } else {
                    hipLaunchKernelGGL((attn_q8_kernel<T, D, NS, 1>), grid, dim3(kThreads), 0, hs, a);
                }
            }
            if (p.splits > 1)
                hipLaunchKernelGGL((attn_q8_merge_kernel<T, D>), merge_grid, dim3(kThreads), 0, hs, a);
        };
        if (cache->head_dim == 64)
            launch(std::integral_constant<int, 64>{});
        else if (cache->head_dim == 128)
            launch(std::integral_constant<int, 128>{});
        else
            launch(std::integral_constant<int, 256>{});
    });
    return check_launch("attn_decode_q8");
}
