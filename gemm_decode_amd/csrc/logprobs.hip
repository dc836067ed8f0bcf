// logprobs.hip -- log probabilities of given tokens, entropy and the k largest logits of
// each row of logits, in one pass over them.
//
// With m the largest logit, d_j = z_j - z_m <= 0 (z the scaled, possibly capped logit) and
// S the sum of exp(d_j) over all tokens but m, log sum exp(z) = z_m + log1p(S): so
//   lp_j = d_j - log1p(S),   entropy = log1p(S) - (sum exp(d_j) d_j) / (1 + S),
// and a token that the model is sure of keeps its small log probability's digits. A wave
// keeps S and D = sum exp(d) d against the largest logit it has met; when a larger one comes,
// the one before joins S and both are rescaled. Exponents are to the base 2.
//
// The k largest: a wave keeps those of its own logits in LDS, and the smallest that can still
// be among the row's (the k-th largest of any wave). Of most vectors no lane's largest logit
// reaches that, so that the selection costs a comparison.
#include <algorithm>
#include <type_traits>

#include "gd_internal.h"
#include "gd_norm.h"
#include "gd_types.h"

namespace {

using namespace gd;

constexpr int kThreads = 256, kWaves = kThreads / 64;
constexpr int kMaxK = 64;
constexpr int kRoom = 512;           // candidates of a wave
constexpr int kMinPart = 2048;       // tokens of a part of a row at least
constexpr int kFill = 512;           // parts of all rows that fill the device
constexpr float kInf = __builtin_inff();
constexpr float kLog2e = 1.44269504f;
constexpr double kLn2 = 0.693147180559945309;
constexpr float kNear = 24.0f;       // a step this far below the largest logit (to the base 2) has one of its own
typedef unsigned long long u64;

struct Task {
    const void *logits;
    const int64_t *tokens;
    float *logprobs, *entropy;
    int64_t *top_ids;
    float *top_logprobs;
    int64_t stride, n_given, k, V;
    float c, more, small;   // see Cap
    int64_t parts, part;   // of a row; tokens of one
    uint8_t *workspace;    // a Part and k keys for each part
};

// What is known of a part of a row: its largest logit (raw), S and D against it, whether it
// holds a NaN or an infinity.
struct Part {
    double S, D;
    float top;
    uint32_t bad;
    uint64_t unused;
};

// An unsigned key that orders as the logits do (0 and -0 alike), and with the token's place
// behind it one number for each token: the larger the earlier in the answer's order.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}
__device__ __forceinline__ u64 order_of(float x, uint32_t place) { return static_cast<u64>(key_of(x)) << 32 | ~place; }

// tanh(u) up to kSmall: u (1 + s q(s)), s = u^2, within 6.4e-9 (a least largest error, fitted). Without
// the last term it is 1.3e-7, and three times the entropies' error under a softcap of 30.
constexpr float kSmall = 0.7f;
constexpr float kTanh[5] = {-0.33333102f, 0.13327664f, -0.05347994f, 0.01991601f, -0.005000424f};

// What exponents are taken of: the logit, or over the cap tanh(x / cap); -infinity stays. Where x
// is small next to the cap the digits are those of x, not of the cap.
template <bool kOn>
struct Cap {
    float over, c;   // 1 / softcap; what comes out is multiplied by c
    float rest;      // what c lacks by its rounding, without a cap
    float small;     // up to which Exponent may be used, with one
    __device__ __forceinline__ explicit Cap(const Task &t) : over(kOn ? t.more : 1.0f), c(t.c), rest(kOn ? 0.0f : t.more), small(t.small) {}
    __device__ __forceinline__ float operator()(float x) const {
        if (!kOn) return x;
        const float u = x * over, s = u * u, q = fmaf(fmaf(fmaf(fmaf(kTanh[4], s, kTanh[3]), s, kTanh[2]), s, kTanh[1]), s, kTanh[0]);
        const float t = fmaf(-2.0f, __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(u * (2.0f * kLog2e))), 1.0f);
        return x == -kInf ? x : s <= kSmall * kSmall ? fmaf(u * s, q, u) : t;
    }
};

// (cap(x) - ref) c for many x: plainly, or with a cap, where |x / softcap| <= kSmall, as x times a
// polynomial in x^2, a[] its coefficients behind c / softcap.
template <bool kCap>
struct Exponent {
    float ref, c, off, a[5];
    __device__ __forceinline__ Exponent(const Cap<kCap> &cap, float ref_) : ref(ref_), c(cap.c) {
        if (!kCap) return;
        c = cap.c * cap.over;
        float p = c;
#pragma unroll
        for (int k = 0; k < 5; k++) {
            p *= cap.over * cap.over;
            a[k] = kTanh[k] * p;
        }
        off = -ref * cap.c;
    }
    __device__ __forceinline__ float operator()(float x) const {
        if (!kCap) return (x - ref) * c;
        const float s = x * x, q = fmaf(fmaf(fmaf(fmaf(a[4], s, a[3]), s, a[2]), s, a[1]), s, a[0]);
        return fmaf(x, fmaf(s, q, c), off);
    }
};

__device__ __forceinline__ float max_nan(float a, float b) { return __builtin_elementwise_maximum(a, b); }   // a NaN stays

// Over the lanes of a wave, in all of them: four steps within rows of 16, then the rows.
template <typename F>
__device__ __forceinline__ float over_wave(float v, F join) {
    const auto dpp = [&](auto control) {
        v = join(v, __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), decltype(control)::value, 0xF, 0xF, false)));
    };
    dpp(std::integral_constant<int, 0xB1>{});    // lane ^ 1
    dpp(std::integral_constant<int, 0x4E>{});    // lane ^ 2
    dpp(std::integral_constant<int, 0x141>{});   // the other four of eight
    dpp(std::integral_constant<int, 0x140>{});   // the other eight of 16
    const uint32_t u = __builtin_bit_cast(uint32_t, v);
    const auto p = __builtin_amdgcn_permlane16_swap(u, u, false, false);
    const uint32_t w = __builtin_bit_cast(uint32_t, join(__builtin_bit_cast(float, static_cast<uint32_t>(p[0])),
                                                         __builtin_bit_cast(float, static_cast<uint32_t>(p[1]))));
    const auto q = __builtin_amdgcn_permlane32_swap(w, w, false, false);
    return join(__builtin_bit_cast(float, static_cast<uint32_t>(q[0])), __builtin_bit_cast(float, static_cast<uint32_t>(q[1])));
}
__device__ __forceinline__ float wave_max(float v) {
    return over_wave(v, [](float a, float b) { return fmaxf(a, b); });
}

// A wave's candidates: the `count` first of room[], at most kRoom.
struct Best {
    u64 *room, *shared;   // shared: the largest of the waves' k-th largest (0: none has k)
    int count, k;
    u64 least;            // only larger ones are taken
    float least_logit;    // and its logit

    __device__ __forceinline__ void raise(u64 to) {
        least = to > least ? to : least;
        least_logit = least ? logit_of(static_cast<uint32_t>(least >> 32)) : -kInf;
    }
    // The largest number that at least `k_` of R 64 numbers, the lanes', reach (0: there are not so
    // many above 0), its bits below `lowest` 0; `reach`: how many do.
    template <int R, typename U>
    __device__ __forceinline__ static U reached(const U (&v)[R], int k_, int &reach, int lowest = 0) {
        U at = 0;
        reach = 64 * R;
#pragma unroll 1
        for (int b = 8 * sizeof(U) - 1; b >= lowest; b--) {
            const U next = at | U{1} << b;
            int n = 0;
#pragma unroll
            for (int r = 0; r < R; r++) n += __popcll(__ballot(v[r] >= next));
            if (n >= k_) {
                at = next;
                reach = n;
            }
        }
        return at;
    }
    // The k-th largest of R 64 orders (no two alike but 0: none).
    template <int R>
    __device__ __forceinline__ u64 kth(const u64 (&v)[R]) const {
        uint32_t key[R];
#pragma unroll
        for (int r = 0; r < R; r++) key[r] = static_cast<uint32_t>(v[r] >> 32);
        int reach;
        const uint32_t at = reached<R>(key, k, reach);
        if (at == 0 || reach == k) return static_cast<u64>(at) << 32;   // all of this logit are among them
        int above = 0;
        uint32_t low[R];
#pragma unroll
        for (int r = 0; r < R; r++) {
            above += __popcll(__ballot(key[r] > at));
            low[r] = key[r] == at ? static_cast<uint32_t>(v[r]) : 0;
        }
        return static_cast<u64>(at) << 32 | reached<R>(low, k - above, reach);
    }
    template <int R>
    __device__ __forceinline__ void keep() {   // the k largest only
        const int lane = threadIdx.x % 64;
        u64 v[R];
#pragma unroll
        for (int r = 0; r < R; r++) v[r] = r * 64 + lane < count ? room[r * 64 + lane] : 0;
        const u64 at = kth<R>(v);
        int n = 0;
#pragma unroll
        for (int r = 0; r < R; r++) {
            const u64 stay = __ballot(v[r] >= at && v[r] > 0);
            if (v[r] >= at && v[r] > 0) room[n + __popcll(stay & ((u64{1} << lane) - 1))] = v[r];
            n += __popcll(stay);
        }
        count = n;
        if (n >= k) {
            raise(at);
            if (lane == 0 && at > *shared) atomicMax(shared, at);
        }
    }
    __device__ __forceinline__ void shrink() {
        if (count <= k) return;
        if (count <= 64)
            keep<1>();
        else if (count <= 128)
            keep<2>();
        else
            keep<kRoom / 64>();
    }
    __device__ __forceinline__ void add(float x, uint32_t place, bool live) {
        const u64 o = order_of(x, place), lane_bit = u64{1} << (threadIdx.x % 64);
        const u64 in = __ballot(live && o > least);
        if (!in) return;
        if (in & lane_bit) room[count + __popcll(in & (lane_bit - 1))] = o;
        count += __popcll(in);
        if (count > kRoom - 64) shrink();
    }
};

// d where it is an exponent that counts: up to 0 (tanh's roundings, times a large cap, may pass it)
// and down to where the exponential is 0.
__device__ __forceinline__ float exponent(float d) { return __builtin_amdgcn_fmed3f(d, -1000.0f, 0.0f); }
__device__ __forceinline__ double exponent(double d) { return fmin(fmax(d, -1000.0), 0.0); }

// The exponential of (a - b) c for an a up to b, to f32's last bits however far they are apart
// (an exponent rounded to f32 is off by up to |exponent| 2^-25).
template <bool kCap>
__device__ __forceinline__ double apart(const Cap<kCap> &cap, float a, float b, double &d) {
    d = exponent((static_cast<double>(a) - b) * (kCap ? cap.c : static_cast<double>(cap.c) + cap.rest));
    const float hi = static_cast<float>(d), e = __builtin_amdgcn_exp2f(hi);
    return kCap ? e : e * (1.0 + kLn2 * (d - hi));
}

// What a wave has met so far: the largest logit (-infinity before there is one), capped in
// ref, and the lanes' shares of S and D against it. A step's terms are summed in f32, the steps in
// f64: terms that are all alike all round the same way, which a chain of f32 sums over a row of
// 2^18 tokens would bring to 2^-16 of S.
struct Met {
    float top, ref;
    double S, D;
    float low, near;   // without a cap: logits from here on need no care, or no largest one of their own (see absorb)
    bool bad;
};

// `N` logits of each lane join (and may be changed), x[i] the token place[i / PER] + i % PER;
// PER: of one vector.
template <int N, int PER, bool kEntropy, bool kCap>
__device__ __forceinline__ void absorb(Met &w, Best &best, const Cap<kCap> &cap, float (&x)[N],
                                       const uint32_t (&place)[(N + PER - 1) / PER]) {
    constexpr int G = (N + PER - 1) / PER;
    float most[G], mine = -kInf, least = kInf;
#pragma unroll
    for (int g = 0; g < G; g++) {
        most[g] = x[g * PER];
#pragma unroll
        for (int i = g * PER + 1; i < g * PER + PER && i < N; i++) most[g] = max_nan(most[g], x[i]);
        mine = max_nan(mine, most[g]);
    }
#pragma unroll
    for (int i = 0; i < N; i++) least = fminf(least, x[i]);
    w.bad |= !(mine < kInf);
    if (best.k && __any(mine >= best.least_logit)) {
        best.raise(*best.shared);
        // None yet: k lanes' largest are k candidates. (To half of the bits: a step is some 50 cycles,
        // one row of 49152 10.5 us instead of 11.1; to 12 of them there are too many, 11.7.)
        if (best.least == 0 && N >= 8) {
            const uint32_t v[1] = {mine > -kInf ? key_of(mine) : 0};
            int reach;
            const u64 to = static_cast<u64>(Best::reached<1>(v, best.k, reach, 16)) << 32;   // below all tokens of this logit
            best.raise(to);
            if (threadIdx.x % 64 == 0 && to > *best.shared) atomicMax(best.shared, to);
        }
#pragma unroll
        for (int g = 0; g < G; g++)
            if (__any(most[g] >= best.least_logit)) {
                uint32_t in = 0;
#pragma unroll
                for (int i = 0; i < PER && g * PER + i < N; i++) in |= x[g * PER + i] >= best.least_logit ? 1u << i : 0u;
                while (__any(in != 0)) {   // a lane's one after the other
                    const int j = in ? __builtin_ctz(in) : 0;
                    float v = x[g * PER];
#pragma unroll
                    for (int i = 1; i < PER && g * PER + i < N; i++) v = i == j ? x[g * PER + i] : v;
                    best.add(v, place[g] + j, in != 0 && v > -kInf);
                    in &= in - 1;
                }
            }
        if (best.count >= 2 * best.k) best.shrink();
    }
    const auto is_easy = [&]() { return kCap ? least >= -cap.small && mine <= cap.small : least >= w.low; };
    bool chosen = false;   // the lane that holds the step's new largest logit
    float out = -kInf;     // what stands in its place
    if (__any(mine > w.top)) {   // a larger one: what was the largest joins the others, in lane 0
        const float top = wave_max(mine), ref = cap(top);
        if (w.top > -kInf) {
            double d;
            const double f = apart(cap, w.ref, ref, d);
            const double own = threadIdx.x % 64 == 0 ? 1.0 : 0.0;
            if (kEntropy) w.D = f * (w.D + d * (w.S + own));
            w.S = f * (w.S + own);
        }
        w.top = top;
        w.ref = ref;
        if (!kCap) w.near = ref - kNear / cap.c;
        if (!kCap) w.low = fmaxf(ref - fminf(1000.0f / cap.c, 3e38f), -3e38f);   // (differences stay in range)
        // The new one stays out of S: the first of them in the first lane that has one.
        // What stands in its place counts for nothing; where the short way below is taken, which
        // has no -infinity, what it counts for is taken off S first.
        if (__all(is_easy())) out = kCap ? -cap.small : w.low;
        chosen = static_cast<int>(threadIdx.x % 64) == __ffsll(__ballot(mine == top)) - 1;
        bool here = chosen;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const bool is = here && x[i] == top;
            x[i] = is ? out : x[i];
            here = here && !is;
        }
        if (!kCap) {   // the largest of the others
            mine = -kInf;
#pragma unroll
            for (int i = 0; i < N; i++) mine = max_nan(mine, x[i]);
        }
    }
    // A step whose logits all lie far below the largest one, as next to a token that the model is sure
    // of, is summed against its own largest one: an f32 exponent d against the other is off by up to
    // |d| 2^-22.4, and so is its exponential.
    float ref = w.top > -kInf ? w.ref : 0.0f;
    float down = 0.0f, factor = 1.0f;
    if (!kCap && !__any(mine >= w.near)) {
        const float most_here = wave_max(mine);
        if (most_here > -kInf) {
            double d;
            factor = static_cast<float>(apart(cap, most_here, ref, d));
            down = static_cast<float>(d);
            ref = most_here;
        }
    }
    float S = 0.0f, D = 0.0f;
    if (__all(is_easy())) {   // no 0 times infinity in D, and a short tanh
        const Exponent<kCap> of(cap, ref);
        if (chosen) {   // (what stands there counts for nothing)
            const float d = of(out), e = __builtin_amdgcn_exp2f(d);
            S = -e;
            if (kEntropy) D = -e * d;
        }
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float d = of(x[i]), e = __builtin_amdgcn_exp2f(d);
            S += e;
            if (kEntropy) D = fmaf(e, d, D);
        }
    } else {
        // (half of the difference: that of two logits may leave f32's range)
        const float half = 0.5f * ref, c = 2.0f * cap.c;
#pragma unroll
        for (int i = 0; i < N; i++) {
            const float d = exponent(fmaf(0.5f, cap(x[i]), -half) * c), e = __builtin_amdgcn_exp2f(d);
            S += e;
            if (kEntropy) D = fmaf(e, d, D);
        }
    }
    if (kEntropy) w.D += factor * fmaf(down, S, D);
    w.S += factor * S;
}

// What a part adds to the sums against `top`, a logit as large as its own: its share of S and D
// with its own largest logit, which it holds out of them; nothing if it has none.
template <bool kCap>
__device__ __forceinline__ void against(const Cap<kCap> &cap, float top, const Part &p, double &S, double &D) {
    double d;
    const double e = apart(cap, cap(p.top), cap(top), d), f = p.top > -kInf ? e : 0.0;
    S = f * (p.S + 1.0);
    D = f * (p.D + d * (p.S + 1.0));
}

// Both parts' sums against the larger logit.
template <bool kCap>
__device__ __forceinline__ void join(Part &a, const Part &b, const Cap<kCap> &cap) {
    const Part &hi = a.top >= b.top ? a : b, &lo = a.top >= b.top ? b : a;
    double S, D;
    against(cap, hi.top, lo, S, D);
    a = Part{hi.S + S, hi.D + D, hi.top, a.bad | b.bad, 0};
}

__device__ __forceinline__ double wave_sum(double v) {
    return gd::over_wave(v, [](double a, double b) { return a + b; });
}

// The threads' parts as one, in all of them: the largest logit first, then each part's share
// against it, the first that has it being left as it is (joined two and two in five steps, one
// row of 49152 took 0.8 us longer). waves[]: room of the workgroup's.
template <bool kCap>
__device__ __forceinline__ Part join_all(const Cap<kCap> &cap, const Part &mine, Part *waves) {
    const int lane = threadIdx.x % 64, wave = threadIdx.x / 64;
    const float most = wave_max(mine.top);
    if (lane == 0) waves[wave].top = most;
    __syncthreads();
    float top = waves[0].top;
    int holder = 0;
#pragma unroll
    for (int w = 1; w < kWaves; w++)
        if (waves[w].top > top) {
            top = waves[w].top;
            holder = w;
        }
    double S, D;
    against(cap, top, mine, S, D);
    if (wave == holder && lane == __ffsll(__ballot(mine.top == top)) - 1) {
        S = mine.S;
        D = mine.D;
    }
    S = wave_sum(S);
    D = wave_sum(D);
    const bool bad = __any(mine.bad);
    if (lane == 0) {
        waves[wave].S = S;
        waves[wave].D = D;
        waves[wave].bad = bad ? 1u : 0u;
    }
    __syncthreads();
    Part all = {0.0, 0.0, top, 0, 0};
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        all.S += waves[w].S;
        all.D += waves[w].D;
        all.bad |= waves[w].bad;
    }
    return all;
}

// The k largest of `count` orders in LDS, by their ranks, to out[]; behind them there is room for
// kRanked more, which are written, so that a step takes kRanked and no rest is left (eight at a
// time and the rest one by one, 8 rows of 128256 with 20 alternatives 15.4 us, now 14.5). Called
// by the workgroup.
constexpr int kRanked = 32;
__device__ __forceinline__ void sort_best(u64 *in, int count, int k, u64 *out) {
    if (static_cast<int>(threadIdx.x) < kRanked) in[count + threadIdx.x] = 0;
    for (int i = threadIdx.x; i < k; i += kThreads) out[i] = 0;
    __syncthreads();
    for (int i = threadIdx.x; i < count; i += kThreads) {
        const u64 v = in[i];
        int rank = 0;
        for (int j = 0; j < count; j += kRanked)
#pragma unroll
            for (int r = 0; r < kRanked; r++) rank += in[j + r] > v ? 1 : 0;
        if (rank < k) out[rank] = v;
    }
    __syncthreads();
}

// The first given token of a thread: asked for before it is needed.
struct Given {
    int64_t id;
    float x;
};
template <typename T>
__device__ __forceinline__ Given given(const Task &t, int64_t row, int64_t i) {
    Given g = {-1, 0.0f};
    if (i < t.n_given) {
        g.id = t.tokens[row * t.n_given + i];
        if (g.id >= 0 && g.id < t.V) g.x = static_cast<float>((static_cast<const T *>(t.logits) + row * t.stride)[g.id]);
    }
    return g;
}

// What a row answers, once `all` is known of it and best[] is sorted.
template <typename T, bool kCap>
__device__ __forceinline__ void answer(const Task &t, const Cap<kCap> &cap, int64_t row, const Part &all, const u64 *best, Given g) {
    const bool bad = all.bad || all.top == kInf, none = !(all.top > -kInf);
    const float lse = log1pf(static_cast<float>(all.S)), y = cap(all.top);
    const auto lp_of = [&](float x) {
        if (bad) return __builtin_nanf("");
        if (none || x == -kInf) return -kInf;
        return static_cast<float>(fmin((static_cast<double>(cap(x)) - y) * cap.c, 0.0) * kLn2 - lse);
    };
    if (t.entropy && threadIdx.x == 0)
        t.entropy[row] = bad ? __builtin_nanf("") : none ? 0.0f : lse - static_cast<float>(kLn2 * all.D) / (1.0f + static_cast<float>(all.S));
    for (int64_t i = threadIdx.x; i < t.n_given; i += kThreads) {
        t.logprobs[row * t.n_given + i] = g.id >= 0 && g.id < t.V ? lp_of(g.x) : 0.0f;
        g = given<T>(t, row, i + kThreads);
    }
    for (int i = threadIdx.x; i < t.k; i += kThreads) {
        const u64 o = best[i];
        t.top_ids[row * t.k + i] = o && !bad ? static_cast<int64_t>(~static_cast<uint32_t>(o)) : -1;
        t.top_logprobs[row * t.k + i] = bad ? __builtin_nanf("") : o ? lp_of(logit_of(static_cast<uint32_t>(o >> 32))) : -kInf;
    }
}

// A part of a row: whole 16-byte vectors, U of them a thread at a time with the next ones on
// their way, and the tokens before and behind them one by one.
//
// 2039 rows of 100003 bf16 (408 MB) take 116 us with a softcap and 95 without: some 22 and 18
// vector instructions a logit (an exponential counts for four), 59 us for the bytes alone. Four waves
// a SIMD (launch bounds) instead of two saved 8 % of it. Few rows are a chain of latencies, of which
// the selection is the longer half: one row of 49152 5.8 us and with 8 alternatives 10.4, both
// launches together; 61 of 50021 f16 8.1 and with 20 alternatives 17.4. There each wave goes once
// through some 2000 instructions, and waits for about half of the time, for memory, barriers and
// the instructions themselves.
template <typename T, int U, bool kEntropy, bool kCap>
__global__ __launch_bounds__(kThreads, 4) void logprobs_part_kernel(Task t) {
    constexpr int PER = 16 / sizeof(T);
    typedef T Vec __attribute__((ext_vector_type(PER)));
    __shared__ u64 room[kWaves][kRoom];
    __shared__ u64 sorted[kMaxK], shared;
    __shared__ Part parts[kWaves];
    __shared__ int counts[kWaves];
    const int tid = threadIdx.x, wave = tid / 64, lane = tid % 64;
    const int64_t row = blockIdx.y, first = blockIdx.x * t.part;
    const int64_t length = first + t.part < t.V ? t.part : t.V - first;   // at least 1
    const T *x = static_cast<const T *>(t.logits) + row * t.stride + first;
    int head = static_cast<int>((16 - reinterpret_cast<uintptr_t>(x) % 16) % 16 / sizeof(T));
    head = head < length ? head : static_cast<int>(length);
    const uint32_t vectors = static_cast<uint32_t>((length - head) / PER);
    const int tail = static_cast<int>(length - head - static_cast<int64_t>(vectors) * PER);
    const Vec *body = reinterpret_cast<const Vec *>(x + head);
    const Cap<kCap> cap(t);
    Met met = {-kInf, 0.0f, 0.0, 0.0, kInf, kInf, false};
    Best best = {room[wave], &shared, 0, static_cast<int>(t.k), 0, -kInf};
    if (tid == 0) shared = 0;
    __syncthreads();
    Vec next[U];
    const auto load = [&](uint32_t v) {
#pragma unroll
        for (int u = 0; u < U; u++) {
            const uint32_t at = v + u * kThreads + tid;
            next[u] = body[at < vectors ? at : vectors - 1];   // clamped: loaded, not used
        }
    };
    Given asked = {-1, 0.0f};
    if (vectors) load(0);
    if (t.parts == 1) asked = given<T>(t, row, tid);
    for (uint32_t v = 0; v < vectors; v += U * kThreads) {
        if (v + U * kThreads > vectors) {
#pragma unroll
            for (int u = 0; u < U; u++)
                if (v + u * kThreads + tid >= vectors) next[u] = Vec(static_cast<T>(-kInf));
        }
        float e[U * PER];
        uint32_t place[U];
#pragma unroll
        for (int u = 0; u < U; u++) {
            place[u] = static_cast<uint32_t>(first) + head + (v + u * kThreads + tid) * PER;
#pragma unroll
            for (int i = 0; i < PER; i++) e[u * PER + i] = static_cast<float>(next[u][i]);
        }
        if (v + U * kThreads < vectors) load(v + U * kThreads);
        absorb<U * PER, PER, kEntropy, kCap>(met, best, cap, e, place);
    }
    {   // the ends: fewer than PER tokens each, of wave 0
        const int at = lane < head ? lane : lane < head + tail ? static_cast<int>(length) - tail + lane - head : -1;
        float e[1] = {wave == 0 && at >= 0 ? static_cast<float>(x[at]) : -kInf};
        const uint32_t place[1] = {static_cast<uint32_t>(first) + (at >= 0 ? at : 0)};
        if (head + tail > 0 && wave == 0) absorb<1, 1, kEntropy, kCap>(met, best, cap, e, place);
    }
    if (best.count > kMaxK) best.shrink();
    {
        const double S = wave_sum(met.S), D = wave_sum(met.D);
        const bool bad = __any(met.bad);
        if (lane == 0) {
            parts[wave] = Part{S, D, met.top, bad ? 1u : 0u, 0};
            counts[wave] = best.count;
        }
    }
    __syncthreads();
    int total = 0;
    if (t.k) {   // the waves' candidates side by side, those that can still be among the k
        const u64 least = shared;
        static_assert(kWaves * kMaxK == kThreads, "a candidate a thread");
        const int c = counts[wave];
        u64 mine = lane < c ? room[wave][lane] : 0;
        if (mine < least) mine = 0;
        const u64 in = __ballot(mine > 0);
        __syncthreads();
        if (lane == 0) counts[wave] = __popcll(in);
        __syncthreads();
        int at = __popcll(in & ((u64{1} << lane) - 1));
        for (int w = 0; w < kWaves; w++) {
            if (w < wave) at += counts[w];
            total += counts[w];
        }
        u64 *list = room[0];
        if (mine) list[at] = mine;
        __syncthreads();
        sort_best(list, total, static_cast<int>(t.k), sorted);
    }
    Part all = {0.0, 0.0, parts[0].top, 0, 0};
    int holder = 0;
#pragma unroll
    for (int w = 1; w < kWaves; w++)
        if (parts[w].top > all.top) {
            all.top = parts[w].top;
            holder = w;
        }
#pragma unroll
    for (int w = 0; w < kWaves; w++) {
        double S, D;
        against(cap, all.top, parts[w], S, D);
        all.S += w == holder ? parts[w].S : S;
        all.D += w == holder ? parts[w].D : D;
        all.bad |= parts[w].bad;
    }
    if (t.parts == 1) {
        answer<T, kCap>(t, cap, row, all, sorted, asked);
        return;
    }
    uint8_t *out = t.workspace + (row * t.parts + blockIdx.x) * (sizeof(Part) + 8 * t.k);
    if (tid == 0) *reinterpret_cast<Part *>(out) = all;
    if (tid < t.k) reinterpret_cast<u64 *>(out + sizeof(Part))[tid] = sorted[tid];
}

// The parts of a row joined, by one workgroup: 4 us, with alternatives 5 to 9 (the rows' parts
// times k candidates are ranked in LDS).
constexpr int kMost = 2048;   // candidates of a row at a time
template <typename T, bool kCap>
__global__ __launch_bounds__(kThreads) void logprobs_join_kernel(Task t) {
    __shared__ u64 stage[kMost], list[kMost + kRanked], sorted[kMaxK];
    __shared__ Part waves[kWaves];
    __shared__ int count;
    const int64_t row = blockIdx.x, size = sizeof(Part) + 8 * t.k;
    const uint8_t *in = t.workspace + row * t.parts * size;
    const Cap<kCap> cap(t);
    const int k = static_cast<int>(t.k), tid = threadIdx.x;
    const Given asked = given<T>(t, row, tid);
    const auto entry = [&](int64_t p, int i) { return reinterpret_cast<const u64 *>(in + p * size + sizeof(Part))[i]; };
    Part all = {0.0, 0.0, -kInf, 0, 0};
    for (int64_t p = tid; p < t.parts; p += kThreads) join(all, *reinterpret_cast<const Part *>(in + p * size), cap);
    all = join_all(cap, all, waves);
    if (k) {   // as many parts' candidates at a time as there is room for, behind the k best so far
        const int64_t fit = (kMost - kMaxK) / k;
        for (int64_t p0 = 0; p0 < t.parts; p0 += fit) {
            const int fits = static_cast<int>(t.parts - p0 < fit ? t.parts - p0 : fit), kept = p0 ? k : 0;
            for (int i = tid; i < fits * k; i += kThreads) stage[i] = entry(p0 + i / k, i % k);
            for (int i = tid; i < kept; i += kThreads) list[i] = sorted[i];
            if (tid == 0) count = kept;
            __syncthreads();
            // The k-th largest of the parts' first ones is reached by k: what lies below is not of the k.
            const int heads = (k + fits - 1) / fits;   // of each part
            u64 *first = list + kMaxK;
            for (int i = tid; i < fits * heads; i += kThreads) first[i] = stage[i / heads * k + i % heads];
            __syncthreads();
            sort_best(first, fits * heads, k, sorted);
            const u64 least = sorted[k - 1];
            __syncthreads();
            for (int i = tid; i < fits * k; i += kThreads) {
                const u64 o = stage[i];
                if (o && o >= least) list[atomicAdd(&count, 1)] = o;   // in any order: no two are alike
            }
            __syncthreads();
            sort_best(list, count, k, sorted);
        }
    }
    __syncthreads();
    answer<T, kCap>(t, cap, row, all, sorted, asked);
}

// Rows are cut into up to kFill parts in all, two workgroups a CU, of kMinPart tokens at least.
// (A few parts more, and some CUs have three: 61 rows of 50021 f16 without alternatives 8.1 us,
// with 549 parts 9.6; 400 rows of 100003 f32 uncut 30.6, cut in two 37.3. Half as many parts: 16
// rows of 50021 with 20 alternatives 13.7 us -> 16.0, 32 of 128256 15.4 -> 18.8.)
int64_t parts_of(int64_t n, int64_t V) {
    const int64_t want = n < kFill ? kFill / n : 1, most = (V + kMinPart - 1) / kMinPart;
    return want < most ? want : most;
}

int check_sizes(const char *name, int64_t n, int64_t V, int64_t k) {
    GD_REQUIRE(n >= 1 && V >= 1 && k >= 0, GD_EINVAL, "%s: n (%lld) and V (%lld) must be >= 1, k (%lld) >= 0", name,
               (long long)n, (long long)V, (long long)k);
    GD_REQUIRE(n < (INT64_C(1) << 23) && V <= (INT64_C(1) << 30) && k <= 64, GD_ERANGE, "%s: n, V or k too large", name);
    return GD_OK;
}

}  // namespace

extern "C" int token_logprobs_workspace_bytes(int64_t n, int64_t V, int64_t k, size_t *bytes) {
    GD_REQUIRE(bytes, GD_EINVAL, "token_logprobs_workspace_bytes: null pointer");
    const int st = check_sizes("token_logprobs_workspace_bytes", n, V, k);
    if (st) return st;
    // Every smaller call's parts: at most kFill in all, and as many as fit into V.
    const int64_t most = (V + kMinPart - 1) / kMinPart;
    const int64_t parts = most == 1 ? 0 : n * most < kFill ? n * most : kFill;
    *bytes = static_cast<size_t>(parts * (static_cast<int64_t>(sizeof(Part)) + 8 * k));
    clear_error();
    return GD_OK;
}

extern "C" int token_logprobs(const void *logits, int64_t stride, const int64_t *tokens, int64_t n_given, float *logprobs,
                              float *entropy, int64_t *top_ids, float *top_logprobs, int64_t k, int64_t n, int64_t V,
                              float scale, float softcap, int32_t dtype, void *workspace, size_t workspace_bytes,
                              void *stream) {
    const char *name = "token_logprobs";
    GD_REQUIRE(logits, GD_EINVAL, "%s: null pointer", name);
    const int st = check_sizes(name, n, V, k);
    if (st) return st;
    GD_REQUIRE(n_given >= 0 && stride >= V, GD_EINVAL, "%s: n_given (%lld) must be >= 0, stride (%lld) >= V", name,
               (long long)n_given, (long long)stride);
    GD_REQUIRE(n_given == 0 || (tokens && logprobs), GD_EINVAL, "%s: null tokens or logprobs", name);
    GD_REQUIRE(k == 0 || (top_ids && top_logprobs), GD_EINVAL, "%s: null top_ids or top_logprobs", name);
    GD_REQUIRE(n_given || k || entropy, GD_EINVAL, "%s: nothing is asked for", name);
    GD_REQUIRE(dtype_ok(dtype), GD_EINVAL, "%s: unknown dtype %d", name, dtype);
    // (Where scale * softcap stays in f32's range.)
    GD_REQUIRE(scale > 0.0f && scale <= 1e30f, GD_EINVAL, "%s: scale must be > 0 and at most 1e30", name);
    GD_REQUIRE(softcap == 0.0f || (softcap >= 1e-4f && softcap <= 1e30f && static_cast<double>(scale) * softcap <= 1e30f), GD_EINVAL,
               "%s: softcap must be 0 or in [1e-4, 1e30], times scale at most 1e30", name);
    GD_REQUIRE(n_given <= 65536 && n * n_given < (INT64_C(1) << 31) && stride <= (INT64_C(1) << 40), GD_ERANGE,
               "%s: n_given or stride too large", name);
    GD_REQUIRE(aligned(logits, dtype_size(dtype)) && aligned(tokens, 8) && aligned(logprobs, 4) && aligned(entropy, 4) &&
                   aligned(top_ids, 8) && aligned(top_logprobs, 4) && aligned(workspace, 16),
               GD_EALIGN, "%s: a pointer is not aligned to its element (the workspace: 16)", name);
    const float over = softcap > 0.0f ? 1.0f / softcap : 1.0f, c = (softcap > 0.0f ? scale * softcap : scale) * kLog2e;
    const float more = softcap > 0.0f ? over : static_cast<float>(scale / kLn2 - c);
    // Where the polynomial's coefficients and x^10 stay in range (none otherwise: the careful way), and both
    // terms of an exponent below 2e4, so that their roundings are small.
    const bool easy = softcap >= 0x1p-10f && softcap <= 0x1p10f && scale >= 0x1p-16f && scale <= 0x1p16f;
    const float small = easy ? std::min(kSmall / over, 1e4f / (c * over)) : -1.0f;
    Task t = {logits, tokens, logprobs, entropy, top_ids, top_logprobs, stride, n_given, k, V, c, more, small,
              parts_of(n, V), 0, static_cast<uint8_t *>(workspace)};
    if (t.parts > 1) {
        t.part = (V + t.parts - 1) / t.parts;
        t.part = (t.part + kMinPart - 1) / kMinPart * kMinPart;
        t.parts = (V + t.part - 1) / t.part;
    } else {
        t.part = V;
    }
    if (t.parts > 1) {
        const uint64_t need = static_cast<uint64_t>(n * t.parts) * (sizeof(Part) + 8 * static_cast<uint64_t>(k));
        GD_REQUIRE(workspace, GD_EINVAL, "%s: null workspace", name);
        GD_REQUIRE(workspace_bytes >= need, GD_ERANGE, "%s: workspace of %zu bytes, %llu are needed", name, workspace_bytes,
                   (unsigned long long)need);
    }
    const int64_t size = dtype_size(dtype);
    const struct {
        const void *at;
        int64_t bytes;
    } outs[4] = {{logprobs, n * n_given * 4}, {entropy, n * 4}, {top_ids, n * k * 8}, {top_logprobs, n * k * 4}};
    for (int i = 0; i < 4; i++) {
        if (!outs[i].at || !outs[i].bytes) continue;
        GD_REQUIRE(!overlaps(logits, stride * size, V * size, n, outs[i].at, outs[i].bytes) &&
                       (!n_given || !overlaps(tokens, n * n_given * 8, n * n_given * 8, 1, outs[i].at, outs[i].bytes)),
                   GD_EINVAL, "%s: an output must not overlap logits or tokens", name);
        for (int j = 0; j < i; j++)
            GD_REQUIRE(!outs[j].at || !outs[j].bytes || !overlaps(outs[j].at, outs[j].bytes, outs[j].bytes, 1, outs[i].at, outs[i].bytes),
                       GD_EINVAL, "%s: outputs must not overlap each other", name);
    }
    const hipStream_t hs = as_stream(stream);
    dispatch_dtype(dtype, [&](auto one) {
        using T = decltype(one);
        const auto go = [&](auto u, auto ent, auto capped) {
            // The grid's second axis is limited to 65535 rows.
            for (int64_t from = 0; from < n; from += 65535) {
                Task s = t;
                const int64_t rows = n - from < 65535 ? n - from : 65535;
                s.logits = static_cast<const T *>(logits) + from * stride;
                if (tokens) s.tokens += from * n_given;
                if (logprobs) s.logprobs += from * n_given;
                if (entropy) s.entropy += from;
                if (top_ids) s.top_ids += from * k;
                if (top_logprobs) s.top_logprobs += from * k;
                hipLaunchKernelGGL((logprobs_part_kernel<T, decltype(u)::value, decltype(ent)::value, decltype(capped)::value>),
                                   dim3(static_cast<uint32_t>(t.parts), static_cast<uint32_t>(rows)), dim3(kThreads), 0, hs, s);
            }
        };
        constexpr int PER = 16 / sizeof(T);
        const auto with = [&](auto ent, auto capped) {
            if (t.part > kMinPart)   // a part of kMinPart is one vector of 16-bit logits, two of f32, a thread
                go(std::integral_constant<int, 4>{}, ent, capped);
            else
                go(std::integral_constant<int, 8 / PER>{}, ent, capped);
            if (t.parts > 1)
                hipLaunchKernelGGL((logprobs_join_kernel<T, decltype(capped)::value>), dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0, hs, t);
        };
        const std::true_type yes;
        const std::false_type no;
        if (softcap > 0.0f)
            entropy ? with(yes, yes) : with(no, yes);
        else
            entropy ? with(yes, no) : with(no, no);
    });
    return check_launch(name);
}
