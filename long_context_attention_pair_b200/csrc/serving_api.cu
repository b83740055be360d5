// C ABI of the calls around a paged KV cache (declared in include/atflash.h):
// rotary positions, appending, tree attention, compaction and page copies.
// Argument checks and launches only.
#include <math.h>
#include <string.h>

#include "serving.h"

using namespace atf;

namespace {

bool aligned(const void *p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

// Frequencies (at most pi) to turn counts of at most 2^63, in long double so that
// the quotient adds no error to the table's own.
const RopeTurns &turns_of(int dims, const double *theta) {
    static thread_local struct {
        double theta[kMaxPairs];
        RopeTurns rt;
    } last;  // (zero pairs at first)
    RopeTurns &rt = last.rt;
    if (rt.pairs == dims / 2 && memcmp(theta, last.theta, sizeof(double) * (dims / 2)) == 0) return rt;
    memcpy(last.theta, theta, sizeof(double) * (dims / 2));
    rt.pairs = dims / 2;
    for (int r = 0; r < rt.pairs; ++r)
        rt.turn[r] = (uint64_t)rintl((long double)theta[r] / 6.283185307179586476925286766559L * 18446744073709551616.0L);
    return rt;
}

// A caller's strides (host, {batch, token, head} in elements), or those of a
// contiguous [B][T][heads][D] tensor.
Strides strides_of(const int64_t *s, int64_t T, int heads, int D) {
    if (s) return Strides{s[0], s[1], s[2]};
    return Strides{T * heads * D, (int64_t)heads * D, (int64_t)D};
}

bool multiple_of(const Strides &s, int v) { return s.batch % v == 0 && s.token % v == 0 && s.head % v == 0; }

// The pool's shape, as every paged call checks it.
int check_pool(int Hkv, int D, int num_pages, int page_size, int kv_layout) {
    if (Hkv < 1 || num_pages < 1 || page_size < 64 || page_size % 64 != 0) return ATFLASH_ERR_INVALID_ARG;
    if (kv_layout != ATFLASH_KV_NHD && kv_layout != ATFLASH_KV_PACKED) return ATFLASH_ERR_INVALID_ARG;
    if (D != 64 && D != 128) return ATFLASH_ERR_UNSUPPORTED;
    if ((int64_t)num_pages * Hkv * (D / 16) > INT32_MAX) return ATFLASH_ERR_INVALID_ARG;
    return ATFLASH_OK;
}

// A table of B rows over at most 2^31 - 1 slots.
int check_table(int B, int max_pages, int page_size) {
    if (B < 1 || max_pages < 1 || (int64_t)max_pages * page_size > INT32_MAX) return ATFLASH_ERR_INVALID_ARG;
    return ATFLASH_OK;
}

// The frequency table of a base, and turn counts of a table: a serving loop asks for the
// same ones at every call, so each thread keeps the last (compared by value).
struct BaseTheta {
    const double *theta = nullptr;
    int rc;
    BaseTheta(int D, double base) {
        static thread_local struct {
            int D = 0;
            double base = 0, theta[kMaxPairs];
        } last;
        if (last.D != D || last.base != base) {
            last.D = 0;
            if ((rc = theta_from_base(D, base, last.theta)) != ATFLASH_OK) return;
            last.D = D, last.base = base;
        }
        rc = ATFLASH_OK;
        theta = last.theta;
    }
};

// Whether [a, a + na) and [b, b + nb) overlap.
bool overlap(const void *a, int64_t na, const void *b, int64_t nb) {
    const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
    return x < y + nb && y < x + na;
}

int done(cudaError_t e) { return e == cudaSuccess ? ATFLASH_OK : ATFLASH_ERR_CUDA; }

}  // namespace

extern "C" {

int atflash_rope_apply_theta(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides,
                             void *q_out, const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides,
                             const int32_t *positions, int B, int64_t T, int Hq, int Hkv, int D, int rotary_dim,
                             const double *theta, double scale, int interleaved, int inverse, int dtype,
                             cudaStream_t stream) {
    if (!q || !q_out || !positions || (k == nullptr) != (k_out == nullptr)) return ATFLASH_ERR_INVALID_ARG;
    if (B < 1 || T < 1 || Hq < 1 || (k && Hkv < 1) || (int64_t)B * T > INT32_MAX) return ATFLASH_ERR_INVALID_ARG;
    if (Hq > 32767 || (k && Hkv > 32767)) return ATFLASH_ERR_INVALID_ARG;
    if (D < 2 || D > 2 * kMaxPairs || (D & 1) || rotary_dim < 2 || rotary_dim > D || (rotary_dim & 1))
        return ATFLASH_ERR_INVALID_ARG;
    if (!theta_valid(rotary_dim, theta) || !isfinite(scale)) return ATFLASH_ERR_INVALID_ARG;
    if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1)) return ATFLASH_ERR_INVALID_ARG;
    if (dtype != ATFLASH_F32 && dtype != ATFLASH_BF16) return ATFLASH_ERR_UNSUPPORTED;
    if (!aligned(q, 16) || !aligned(q_out, 16) || !aligned(k, 16) || !aligned(k_out, 16)) return ATFLASH_ERR_ALIGNMENT;
    RopeTensor tq{q, q_out, strides_of(q_strides, T, Hq, D), strides_of(q_out_strides, T, Hq, D), Hq};
    RopeTensor tk{k, k_out, strides_of(k_strides, T, Hkv, D), strides_of(k_out_strides, T, Hkv, D), k ? Hkv : 0};
    return done(launch_rope_apply(tq, tk, positions, B, T, D, turns_of(rotary_dim, theta), (float)scale, interleaved,
                                  inverse, dtype == ATFLASH_F32, stream));
}

int atflash_rope_apply(const void *q, const int64_t *q_strides, const void *k, const int64_t *k_strides, void *q_out,
                       const int64_t *q_out_strides, void *k_out, const int64_t *k_out_strides,
                       const int32_t *positions, int B, int64_t T, int Hq, int Hkv, int D, int rotary_dim,
                       double rope_base, double scale, int interleaved, int inverse, int dtype, cudaStream_t stream) {
    BaseTheta bt(rotary_dim, rope_base);
    if (bt.rc != ATFLASH_OK) return bt.rc;
    return atflash_rope_apply_theta(q, q_strides, k, k_strides, q_out, q_out_strides, k_out, k_out_strides, positions,
                                    B, T, Hq, Hkv, D, rotary_dim, bt.theta, scale, interleaved, inverse, dtype, stream);
}

int atflash_cache_append_theta(const void *k, const int64_t *k_strides, const void *v, const int64_t *v_strides,
                               void *kpages, void *vpages, const int32_t *block_table, const int32_t *seqlens,
                               const int32_t *positions, const int32_t *counts, int B, int T, int Hkv, int max_pages,
                               int num_pages, int page_size, int D, const double *theta, int kcache_rotated,
                               int kv_layout, cudaStream_t stream) {
    if (!k || !v || !kpages || !vpages || !block_table || !seqlens) return ATFLASH_ERR_INVALID_ARG;
    int rc = check_pool(Hkv, D, num_pages, page_size, kv_layout);
    if (rc != ATFLASH_OK) return rc;
    if ((rc = check_table(B, max_pages, page_size)) != ATFLASH_OK) return rc;
    if (T < 1 || (int64_t)B * T > INT32_MAX || !theta_valid(D, theta)) return ATFLASH_ERR_INVALID_ARG;
    if (kcache_rotated != 0 && kcache_rotated != 1) return ATFLASH_ERR_INVALID_ARG;
    if (kv_layout == ATFLASH_KV_PACKED && !kcache_rotated) return ATFLASH_ERR_INVALID_ARG;
    AppendArgs a{};
    a.k = k, a.v = v;
    a.ks = strides_of(k_strides, T, Hkv, D), a.vs = strides_of(v_strides, T, Hkv, D);
    if (!aligned(k, 16) || !aligned(v, 16) || !aligned(kpages, 16) || !aligned(vpages, 16) || !multiple_of(a.ks, 8) ||
        !multiple_of(a.vs, 8))
        return ATFLASH_ERR_ALIGNMENT;
    a.kpages = kpages, a.vpages = vpages;
    a.pk = PagedKV{block_table, max_pages, page_size, num_pages};
    a.seqlens = seqlens, a.positions = positions, a.counts = counts;
    a.B = B, a.T = T, a.Hkv = Hkv, a.D = D;
    a.packed = kv_layout == ATFLASH_KV_PACKED, a.rotate = kcache_rotated;
    if (!(a.status = device_status_word())) return ATFLASH_ERR_CUDA;
    return done(launch_cache_append(a, turns_of(D, theta), stream));
}

int atflash_cache_append(const void *k, const int64_t *k_strides, const void *v, const int64_t *v_strides, void *kpages,
                         void *vpages, const int32_t *block_table, const int32_t *seqlens, const int32_t *positions,
                         const int32_t *counts, int B, int T, int Hkv, int max_pages, int num_pages, int page_size,
                         int D, double rope_base, int kcache_rotated, int kv_layout, cudaStream_t stream) {
    BaseTheta bt(D, rope_base);
    if (bt.rc != ATFLASH_OK) return bt.rc;
    return atflash_cache_append_theta(k, k_strides, v, v_strides, kpages, vpages, block_table, seqlens, positions,
                                      counts, B, T, Hkv, max_pages, num_pages, page_size, D, bt.theta, kcache_rotated,
                                      kv_layout, stream);
}

int atflash_cache_compact(void *kpages, void *vpages, const int32_t *block_table, const int32_t *seqlens,
                          const int32_t *path, const int32_t *accepted, int32_t *new_seqlens, int B, int M, int Hkv,
                          int max_pages, int num_pages, int page_size, int D, int kv_layout, cudaStream_t stream) {
    if (!kpages || !vpages || !block_table || !seqlens || !path || !accepted) return ATFLASH_ERR_INVALID_ARG;
    int rc = check_pool(Hkv, D, num_pages, page_size, kv_layout);
    if (rc != ATFLASH_OK) return rc;
    if ((rc = check_table(B, max_pages, page_size)) != ATFLASH_OK) return rc;
    if (M < 1 || (int64_t)B * Hkv * (D / 16) > INT32_MAX) return ATFLASH_ERR_INVALID_ARG;
    if (M > kCompactMaxPath) return ATFLASH_ERR_UNSUPPORTED;
    // Other blocks still read the inputs when the first one writes its new length.
    const int64_t n = 4 * (int64_t)B;
    if (new_seqlens && (overlap(new_seqlens, n, seqlens, n) || overlap(new_seqlens, n, accepted, n) ||
                        overlap(new_seqlens, n, path, n * M) || overlap(new_seqlens, n, block_table, n * max_pages)))
        return ATFLASH_ERR_INVALID_ARG;
    if (!aligned(kpages, 16) || !aligned(vpages, 16)) return ATFLASH_ERR_ALIGNMENT;
    CompactArgs a{};
    a.kpages = kpages, a.vpages = vpages;
    a.pk = PagedKV{block_table, max_pages, page_size, num_pages};
    a.seqlens = seqlens, a.path = path, a.accepted = accepted, a.new_seqlens = new_seqlens;
    a.B = B, a.M = M, a.Hkv = Hkv, a.D = D, a.packed = kv_layout == ATFLASH_KV_PACKED;
    if (!(a.status = device_status_word())) return ATFLASH_ERR_CUDA;
    return done(launch_cache_compact(a, stream));
}

int atflash_cache_copy_pages(void *kpages, void *vpages, const int32_t *src, const int32_t *dst, const int32_t *tokens,
                             int n, int Hkv, int num_pages, int page_size, int D, int kv_layout, cudaStream_t stream) {
    if (!kpages || !vpages || !src || !dst || n < 1) return ATFLASH_ERR_INVALID_ARG;
    int rc = check_pool(Hkv, D, num_pages, page_size, kv_layout);
    if (rc != ATFLASH_OK) return rc;
    // Indices of 16-byte units, a round of loads past the last included, fit 32 bits.
    if ((int64_t)page_size * Hkv * D / 8 > INT32_MAX / 2) return ATFLASH_ERR_INVALID_ARG;
    if (!aligned(kpages, 16) || !aligned(vpages, 16)) return ATFLASH_ERR_ALIGNMENT;
    CopyPagesArgs a{kpages, vpages, src, dst, tokens, n, Hkv, D, num_pages, page_size, kv_layout == ATFLASH_KV_PACKED,
                    device_status_word()};
    if (!a.status) return ATFLASH_ERR_CUDA;
    return done(launch_cache_copy_pages(a, stream));
}

static int check_tree_shape(int B, int T, int Hq, int Hkv) {
    if (B < 1 || T < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return ATFLASH_ERR_INVALID_ARG;
    if ((int64_t)B * T > INT32_MAX / Hq) return ATFLASH_ERR_INVALID_ARG;
    return ATFLASH_OK;
}

size_t atflash_tree_decode_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
    if (check_tree_shape(B, T, Hq, Hkv) != ATFLASH_OK || (D != 64 && D != 128)) return 0;
    return tree_workspace_bytes(B, T, Hq, Hkv, D);
}

int atflash_tree_decode_paged_theta(const void *q, const int64_t *q_strides, const void *kpages, const void *vpages,
                                    const int32_t *block_table, const int32_t *seqlens, const uint8_t *tree_mask,
                                    const int32_t *positions, const int32_t *counts, void *out, float *lse, int B,
                                    int T, int Hq, int Hkv, int max_pages, int num_pages, int page_size, int D,
                                    const double *theta, double k_window, int kv_layout, int out_dtype, void *workspace,
                                    size_t workspace_bytes, cudaStream_t stream) {
    if (!q || !kpages || !vpages || !block_table || !seqlens || !out) return ATFLASH_ERR_INVALID_ARG;
    int rc = check_tree_shape(B, T, Hq, Hkv);
    if (rc != ATFLASH_OK) return rc;
    if ((rc = check_pool(Hkv, D, num_pages, page_size, kv_layout)) != ATFLASH_OK) return rc;
    if ((rc = check_table(B, max_pages, page_size)) != ATFLASH_OK) return rc;
    if (!theta_valid(D, theta) || isnan(k_window) || k_window < 0.0) return ATFLASH_ERR_INVALID_ARG;
    if (out_dtype != ATFLASH_F32 && out_dtype != ATFLASH_BF16) return ATFLASH_ERR_UNSUPPORTED;
    const Strides qs = strides_of(q_strides, T, Hq, D);
    if (!aligned(q, 16) || !aligned(kpages, 16) || !aligned(vpages, 16) || !aligned(out, 16) || !multiple_of(qs, 8))
        return ATFLASH_ERR_ALIGNMENT;
    const size_t need = tree_workspace_bytes(B, T, Hq, Hkv, D);
    if (!workspace || workspace_bytes < need) return ATFLASH_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return ATFLASH_ERR_ALIGNMENT;
    // Distances between positions reach 2^31 - 1 whatever the cache's length, so
    // the windows are clamped there.
    int64_t w[kMaxPairs];
    if ((rc = window_table_theta(D, theta, k_window, (int64_t)INT32_MAX + 1, w)) != ATFLASH_OK) return rc;
    WindowParams wp;
    memset(&wp, 0, sizeof(wp));
    wp.H = D / 2;
    for (int r = 0; r < D / 2; ++r) wp.w[r] = (int32_t)w[r], wp.theta[r] = theta[r];
    TreeArgs a{};
    a.q = q, a.qs = qs;
    a.kpages = kpages, a.vpages = vpages;
    a.pk = PagedKV{block_table, max_pages, page_size, num_pages};
    a.seqlens = seqlens, a.positions = positions, a.counts = counts, a.mask = tree_mask;
    a.out = out, a.lse = lse, a.out_f32 = out_dtype == ATFLASH_F32, a.packed = kv_layout == ATFLASH_KV_PACKED;
    a.B = B, a.T = T, a.Hq = Hq, a.Hkv = Hkv, a.D = D;
    a.workspace = static_cast<float *>(workspace);
    a.limit_ns = wait_limit_ns();
    if (!(a.status = device_status_word())) return ATFLASH_ERR_CUDA;
    return done(launch_tree_decode(a, wp, turns_of(D, theta), stream));
}

int atflash_tree_decode_paged(const void *q, const int64_t *q_strides, const void *kpages, const void *vpages,
                              const int32_t *block_table, const int32_t *seqlens, const uint8_t *tree_mask,
                              const int32_t *positions, const int32_t *counts, void *out, float *lse, int B, int T,
                              int Hq, int Hkv, int max_pages, int num_pages, int page_size, int D, double rope_base,
                              double k_window, int kv_layout, int out_dtype, void *workspace, size_t workspace_bytes,
                              cudaStream_t stream) {
    BaseTheta bt(D, rope_base);
    if (bt.rc != ATFLASH_OK) return bt.rc;
    return atflash_tree_decode_paged_theta(q, q_strides, kpages, vpages, block_table, seqlens, tree_mask, positions,
                                           counts, out, lse, B, T, Hq, Hkv, max_pages, num_pages, page_size, D,
                                           bt.theta, k_window, kv_layout, out_dtype, workspace, workspace_bytes,
                                           stream);
}

}  // extern "C"
