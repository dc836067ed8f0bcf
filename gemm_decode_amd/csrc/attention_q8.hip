// attention_q8.hip -- attention of the last tokens of several sequences (one
// decode token, a chain or a tree of drafted ones) over the 8-bit cache.
#include "gd_internal.h"
#include "gd_types.h"

namespace {

using namespace gd;

struct AttnArgs {
    gd_kv_q8 c;
    const void *q;
    void *out;
    const int32_t *page_table, *kv_lens, *q_start;
    const uint64_t *tree;
    int64_t max_pages, n_seqs, n_q, n_heads, max_q, max_kv_len;
    float scale, softcap;
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

// The page that holds position j of sequence b, or -1 if its entry is none.
__device__ __forceinline__ int64_t page_of(const AttnArgs &a, int64_t b, int64_t j) {
    const int64_t i = j / a.c.page_size;
    const int64_t p = a.page_table ? a.page_table[b * a.max_pages + i] : b;
    return p >= 0 && p < a.c.n_pages ? p : -1;
}

__device__ __forceinline__ float capped(float s, float cap) { return cap > 0.0f ? cap * tanhf(s / cap) : s; }

// One wave per query row and head, one key at a time.
template <typename T>
__global__ __launch_bounds__(64) void attn_q8_kernel(AttnArgs a) {
    const int64_t b = blockIdx.z;
    const int t = blockIdx.y;
    const int h = blockIdx.x, lane = threadIdx.x;
    const Seq sq(a, b);
    if (t >= sq.rows) return;
    const int D = static_cast<int>(a.c.head_dim), Hkv = static_cast<int>(a.c.n_kv_heads);
    const int kvh = h / static_cast<int>(a.n_heads / Hkv), n = D / 64;
    const int64_t row = sq.row0 + t;
    const T *q = static_cast<const T *>(a.q) + (row * a.n_heads + h) * D;
    const uint64_t word = a.tree ? a.tree[row] : (t >= 63 ? ~0ull : (1ull << (t + 1)) - 1);
    float qv[4], acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int i = 0; i < n; i++) qv[i] = static_cast<float>(q[lane + 64 * i]);
    float m = -__builtin_inff(), l = 0.0f;
    for (int64_t j = 0; j < sq.len; j++) {
        if (j >= sq.ctx && !((word >> (j - sq.ctx)) & 1)) continue;
        const int64_t page = page_of(a, b, j);
        if (page < 0) continue;
        const int64_t r = (page * Hkv + kvh) * a.c.page_size + j % a.c.page_size;
        float s = 0.0f;
        for (int i = 0; i < n; i++) {
            const int d = lane + 64 * i;
            s += qv[i] * static_cast<float>(a.c.k_codes[r * D + d]) *
                 static_cast<float>(__builtin_bit_cast(_Float16, a.c.k_scales[r * (D / 32) + d / 32]));
        }
        for (int o = 32; o >= 1; o >>= 1) s += __shfl_xor(s, o);
        s = capped(s * a.scale, a.softcap);
        const float mn = fmaxf(m, s), corr = m == -__builtin_inff() ? 0.0f : expf(m - mn), p = expf(s - mn);
        l = l * corr + p;
        for (int i = 0; i < n; i++) {
            const int d = lane + 64 * i;
            const float v = static_cast<float>(a.c.v_codes[r * D + d]) *
                            static_cast<float>(__builtin_bit_cast(_Float16, a.c.v_scales[r * (D / 32) + d / 32]));
            acc[i] = acc[i] * corr + p * v;
        }
        m = mn;
    }
    T *o = static_cast<T *>(a.out) + (row * a.n_heads + h) * D;
    for (int i = 0; i < n; i++) o[lane + 64 * i] = static_cast<T>(l > 0.0f ? acc[i] / l : 0.0f);
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
                   max_kv_len <= INT64_C(2147483647),
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
    *bytes = 16;
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
    GD_REQUIRE(softcap >= 0.0f && softcap <= 3.40282347e38f, GD_EINVAL,
               "attn_decode_q8: softcap must be finite and >= 0 (0: none)");
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
    AttnArgs a;
    a.c = *cache;
    a.q = q, a.out = out, a.page_table = page_table, a.kv_lens = kv_lens, a.q_start = q_start, a.tree = tree_mask;
    a.max_pages = max_pages, a.n_seqs = n_seqs, a.n_q = n_q, a.n_heads = n_heads, a.max_q = max_q;
    a.max_kv_len = max_kv_len, a.scale = scale, a.softcap = softcap;
    const dim3 grid(static_cast<uint32_t>(n_heads), static_cast<uint32_t>(max_q), static_cast<uint32_t>(n_seqs));
    dispatch_dtype(dtype, [&](auto t) {
        hipLaunchKernelGGL((attn_q8_kernel<decltype(t)>), grid, dim3(64), 0, as_stream(stream), a);
    });
    return check_launch("attn_decode_q8");
}
