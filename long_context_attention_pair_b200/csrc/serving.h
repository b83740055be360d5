// Interfaces between the C ABI of the paged serving calls (serving_api.cu) and
// their kernels.
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"

namespace atf {

// theta_r / (2*pi) of each rotated pair, in units of 2^-64 turns.  A position
// times such a count wraps modulo 2^64, that is modulo whole turns, so the angle
// of any 32-bit position is reduced exactly in integer arithmetic; the count
// itself carries fp64's precision of theta_r (theta_r <= pi: at most 2^63).
struct RopeTurns {
    int pairs;
    uint64_t turn[kMaxPairs];
};

// Element strides of a [batch][token][head][dim] tensor whose dims are contiguous.
struct Strides {
    int64_t batch, token, head;
};

#ifdef __CUDACC__
// (cos, sin) of position * theta_r.
__device__ __forceinline__ float2 turn_cos_sin(int32_t pos, uint64_t turn) {
    const int64_t t = (int64_t)((uint64_t)(int64_t)pos * turn);  // in [-1/2, 1/2) turns
    float s, c;
    sincospif((float)t * 1.0842021724855044e-19f, &s, &c);       // 2^-63: half-turns in [-1, 1)
    return make_float2(c, s);
}

// The same by the hardware's sin and cos (2^-21.2 on [-pi, pi]) of the angle in radians
// (three roundings, 3 * 2^-23): a rotated element x c - z s is within 2^-20 (|x| + |z|),
// products included.  For results rounded to bf16, half a step of which is 2^-8 of the
// result: the bound is larger only where the two products cancel to 2^-12 of their sizes.
__device__ __forceinline__ float2 turn_cos_sin_fast(int32_t pos, uint64_t turn) {
    float s, c;
    __sincosf((float)(int64_t)((uint64_t)(int64_t)pos * turn) * 3.4061215800865545e-19f, &s, &c);  // 2 pi / 2^64
    return make_float2(c, s);
}

// 16 bytes copied to shared memory asynchronously; groups of copies are waited for in order.
__device__ __forceinline__ void copy_async(void *smem, const void *global) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"((uint32_t)__cvta_generic_to_shared(smem)), "l"(global) : "memory");
}
__device__ __forceinline__ void copy_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the latest N groups have landed
__device__ __forceinline__ void copy_async_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Pool page of a cache slot; -1, recorded in the device status word, for a slot
// outside the sequence's table row or a page id outside the pool.
__device__ __forceinline__ int page_of(const PagedKV &pk, int b, int64_t slot, int *status) {
    // (A slot that the row has room for fits 31 bits: no 64-bit division.)
    const bool inside = slot >= 0 && slot < (int64_t)pk.max_pages * pk.page_size;
    const uint32_t i = inside ? (uint32_t)slot / (uint32_t)pk.page_size : 0u;
    int page = inside ? pk.block_table[(size_t)b * pk.max_pages + i] : -1;
    if (page < 0 || page >= pk.num_pages) {
        atomicCAS(status, 0, ATFLASH_DEVICE_BAD_PAGE);
        page = -1;
    }
    return page;
}
#endif

// One rotated tensor: heads == 0 when absent.
struct RopeTensor {
    const void *x;
    void *y;
    Strides xs, ys;
    int heads;
};
cudaError_t launch_rope_apply(const RopeTensor &q, const RopeTensor &k, const int32_t *positions, int B, int64_t T,
                              int D, const RopeTurns &rt, float scale, int interleaved, int inverse, int f32,
                              cudaStream_t s);

struct AppendArgs {
    const void *k, *v;
    Strides ks, vs;
    void *kpages, *vpages;
    PagedKV pk;
    const int32_t *seqlens, *positions, *counts;
    int B, T, Hkv, D, packed, rotate;
    int *status;
};
cudaError_t launch_cache_append(const AppendArgs &a, const RopeTurns &rt, cudaStream_t s);

struct CompactArgs {
    void *kpages, *vpages;
    PagedKV pk;
    const int32_t *seqlens, *path, *accepted;
    int32_t *new_seqlens;
    int B, M, Hkv, D, packed;
    int *status;
};
constexpr int kCompactMaxPath = 1024;
cudaError_t launch_cache_compact(const CompactArgs &a, cudaStream_t s);

struct CopyPagesArgs {
    void *kpages, *vpages;
    const int32_t *src, *dst, *tokens;
    int n, Hkv, D, num_pages, page_size, packed;
    int *status;
};
cudaError_t launch_cache_copy_pages(const CopyPagesArgs &a, cudaStream_t s);

struct TreeArgs {
    const void *q;
    Strides qs;
    const void *kpages, *vpages;
    PagedKV pk;
    const int32_t *seqlens, *positions, *counts;
    const uint8_t *mask;
    void *out;
    float *lse;
    int out_f32, packed;
    int B, T, Hq, Hkv, D;
    float *workspace;
    int *status;
    uint64_t limit_ns;
};
size_t tree_workspace_bytes(int B, int T, int Hq, int Hkv, int D);
cudaError_t launch_tree_decode(const TreeArgs &a, const WindowParams &wp, const RopeTurns &rt, cudaStream_t s);

}  // namespace atf
