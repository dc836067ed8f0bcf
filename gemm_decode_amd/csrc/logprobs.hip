// logprobs.hip -- log probabilities of given tokens, entropy and the k largest logits of
// each row of logits.
//
// With m the largest logit, d_j = z_j - z_m <= 0 (z the scaled, possibly capped logit) and
// S the sum of exp(d_j) over all tokens but m, log sum exp(z) = z_m + log1p(S): so
//   lp_j = d_j - log1p(S),   entropy = log1p(S) - (sum exp(d_j) d_j) / (1 + S),
// and a token that the model is sure of keeps its small log probability's digits.
#include "gd_internal.h"
#include "gd_types.h"

namespace {

using namespace gd;

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

struct Task {
    const void *logits;
    const int64_t *tokens;
    float *logprobs, *entropy;
    int64_t *top_ids;
    float *top_logprobs;
    int64_t stride, n_given, k, n, V;
    float scale, softcap;
};

// An unsigned key that orders as the logits do (0 and -0 alike), larger logits first.
__device__ __forceinline__ uint32_t key_of(float x) {
    const uint32_t b = __builtin_bit_cast(uint32_t, x + 0.0f);
    return b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float logit_of(uint32_t key) {
    return __builtin_bit_cast(float, key & 0x80000000u ? key & 0x7fffffffu : ~key);
}

// z_j - z_m for the largest logit m; -infinity for a banned token.
__device__ __forceinline__ float below(const Task &t, float x, float m) {
    if (t.softcap > 0.0f) {
        if (x == -kInf) return x;
        return t.scale * t.softcap * (tanhf(x / t.softcap) - tanhf(m / t.softcap));
    }
    return t.scale * (x - m);
}

template <typename V, typename F>
__device__ V over_workgroup(V v, F join, V *red) {
    for (int o = 32; o >= 1; o >>= 1) v = join(v, __shfl_xor(v, o));
    __syncthreads();
    if (threadIdx.x % 64 == 0) red[threadIdx.x / 64] = v;
    __syncthreads();
    v = red[0];
    for (int w = 1; w < kThreads / 64; w++) v = join(v, red[w]);
    return v;
}

// Plain: a workgroup per row, a pass for the maximum, one for the sums and one per alternative.
template <typename T>
__global__ __launch_bounds__(kThreads) void logprobs_plain_kernel(Task t) {
    __shared__ double sums[kThreads / 64];
    __shared__ unsigned long long keys[kThreads / 64];
    const int64_t row = blockIdx.x;
    const T *x = static_cast<const T *>(t.logits) + row * t.stride;
    const auto largest = [](unsigned long long a, unsigned long long b) { return a > b ? a : b; };
    const auto plus = [](double a, double b) { return a + b; };
    // (key, place from behind): one number per token, the larger the earlier in the order
    const auto ordered = [&](int64_t j) {
        return static_cast<unsigned long long>(key_of(static_cast<float>(x[j]))) << 32 | (0xffffffffull - j);
    };
    unsigned long long best = 0;
    double odd = 0.0;
    for (int64_t j = threadIdx.x; j < t.V; j += kThreads) {
        const float v = static_cast<float>(x[j]);
        if (!(v < kInf)) odd = 1.0;   // NaN or infinity
        best = largest(best, ordered(j));
    }
    odd = over_workgroup(odd, plus, sums);
    best = over_workgroup(best, largest, keys);
    const float m = logit_of(static_cast<uint32_t>(best >> 32));
    const int64_t at = 0xffffffffll - static_cast<int64_t>(best & 0xffffffffu);
    const bool bad = odd > 0.0, none = !bad && m == -kInf;
    double S = 0.0, D = 0.0;
    if (!bad && !none)
        for (int64_t j = threadIdx.x; j < t.V; j += kThreads) {
            const float d = below(t, static_cast<float>(x[j]), m);
            if (j != at && d > -200.0f) {
                const double e = exp(static_cast<double>(d));
                S += e;
                D += e * d;
            }
        }
    S = over_workgroup(S, plus, sums);
    D = over_workgroup(D, plus, sums);
    const double lse = log1p(S);
    const auto lp_of = [&](float v) {
        return bad ? __builtin_nanf("") : none ? -kInf : static_cast<float>(static_cast<double>(below(t, v, m)) - lse);
    };
    if (threadIdx.x == 0 && t.entropy)
        t.entropy[row] = bad ? __builtin_nanf("") : none ? 0.0f : static_cast<float>(lse - D / (1.0 + S));
    for (int64_t i = threadIdx.x; i < t.n_given; i += kThreads) {
        const int64_t id = t.tokens[row * t.n_given + i];
        t.logprobs[row * t.n_given + i] = id >= 0 && id < t.V ? lp_of(static_cast<float>(x[id])) : 0.0f;
    }
    unsigned long long before = ~0ull;
    for (int64_t i = 0; i < t.k; i++) {
        unsigned long long next = 0;
        for (int64_t j = threadIdx.x; j < t.V; j += kThreads) {
            const unsigned long long o = ordered(j);
            if (o < before) next = largest(next, o);
        }
        before = next = over_workgroup(next, largest, keys);
        if (threadIdx.x == 0) {
            const float v = next ? logit_of(static_cast<uint32_t>(next >> 32)) : -kInf;
            t.top_ids[row * t.k + i] = !bad && v > -kInf ? 0xffffffffll - static_cast<int64_t>(next & 0xffffffffu) : -1;
            t.top_logprobs[row * t.k + i] = bad ? __builtin_nanf("") : v > -kInf ? lp_of(v) : -kInf;
        }
    }
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
    *bytes = 0;
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
    GD_REQUIRE(scale > 0.0f && scale <= 3.40282347e38f, GD_EINVAL, "%s: scale must be finite and > 0", name);
    GD_REQUIRE(softcap >= 0.0f && softcap <= 1e30f, GD_EINVAL, "%s: softcap must be in [0, 1e30]", name);
    GD_REQUIRE(n_given <= 65536 && n * n_given < (INT64_C(1) << 31) && stride <= (INT64_C(1) << 40), GD_ERANGE,
               "%s: n_given or stride too large", name);
    GD_REQUIRE(aligned(logits, dtype_size(dtype)) && aligned(tokens, 8) && aligned(logprobs, 4) && aligned(entropy, 4) &&
                   aligned(top_ids, 8) && aligned(top_logprobs, 4) && aligned(workspace, 16),
               GD_EALIGN, "%s: a pointer is not aligned to its element (the workspace: 16)", name);
    (void)workspace_bytes;
    const Task t = {logits, tokens, logprobs, entropy, top_ids, top_logprobs, stride, n_given, k, n, V, scale, softcap};
    dispatch_dtype(dtype, [&](auto e) {
        hipLaunchKernelGGL((logprobs_plain_kernel<decltype(e)>), dim3(static_cast<uint32_t>(n)), dim3(kThreads), 0,
                           as_stream(stream), t);
    });
    return check_launch(name);
}
