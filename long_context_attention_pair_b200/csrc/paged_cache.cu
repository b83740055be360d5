// Writing and moving tokens of a paged KV cache (bf16): appending new tokens,
// compacting the accepted nodes of a drafted tree, copying pages.
//
// Pools: V [num_pages][page_size][Hkv][D]; K the same (NHD) or packed
// [num_pages][Hkv][D/16][page_size][16], whose 32-byte chunk c of a token holds
// the rotated pairs 8c..8c+7 as (x~_r, x~_{r+D/2}) interleaved.  All three
// kernels move data in 16-byte accesses and are bound by HBM (or, for the few
// tokens of a drafted step, by the chain of dependent loads: length, table, row).
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "serving.h"

namespace atf {
namespace {

// Where 16 elements (32 bytes) `c` of a token lie: of K in either layout, or of V.
__device__ __forceinline__ size_t natural_off(int page, int at, int h, int c, int P, int Hkv, int D) {
    return ((((size_t)page * P + at) * Hkv + h) * D) + 16 * c;
}
__device__ __forceinline__ size_t packed_off(int page, int at, int h, int c, int P, int Hkv, int D) {
    return ((((size_t)page * Hkv + h) * (D / 16) + c) * P + at) * 16;
}

// Thread = (token, c): pairs 8c..8c+7 of K and dims 16c..16c+15 of V, for every
// KV head.  The cos and sin of the 8 pairs are taken once per token.
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns rt) {
    const int C = a.D / 16, H = a.D / 2;
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t bt = id / C;
    if (bt >= (int64_t)a.B * a.T) return;
    const int c = (int)(id - bt * C), b = (int)(bt / a.T), i = (int)(bt - (int64_t)b * a.T);
    if (a.counts && i >= a.counts[b]) return;
    const int64_t slot = (int64_t)a.seqlens[b] + i;
    const int page = page_of(a.pk, b, slot, a.status);
    if (page < 0) return;
    const int P = a.pk.page_size, at = (int)(slot % P);
    const int32_t pos = a.positions ? a.positions[bt] : (int32_t)slot;
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = a.rotate ? turn_cos_sin(pos, rt.turn[8 * c + j]) : make_float2(1.f, 0.f);
    for (int h = 0; h < a.Hkv; ++h) {
        const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + b * a.ks.batch + i * a.ks.token + h * a.ks.head;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + b * a.vs.batch + i * a.vs.token + h * a.vs.head;
        const uint4 lo = *reinterpret_cast<const uint4 *>(k + 8 * c), hi = *reinterpret_cast<const uint4 *>(k + H + 8 * c);
        const uint4 v0 = *reinterpret_cast<const uint4 *>(v + 16 * c), v1 = *reinterpret_cast<const uint4 *>(v + 16 * c + 8);
        const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, z[4] = {hi.x, hi.y, hi.z, hi.w};
        float f[8], g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xa = (j & 1) ? bf16hi(x[j >> 1]) : bf16lo(x[j >> 1]);
            const float xb = (j & 1) ? bf16hi(z[j >> 1]) : bf16lo(z[j >> 1]);
            f[j] = xa * cs[j].x - xb * cs[j].y;
            g[j] = xb * cs[j].x + xa * cs[j].y;
        }
        __nv_bfloat16 *kp = static_cast<__nv_bfloat16 *>(a.kpages), *vp = static_cast<__nv_bfloat16 *>(a.vpages);
        if (a.packed) {
            uint4 *dst = reinterpret_cast<uint4 *>(kp + packed_off(page, at, h, c, P, a.Hkv, a.D));
            dst[0] = make_uint4(pack_bf16x2(f[0], g[0]), pack_bf16x2(f[1], g[1]), pack_bf16x2(f[2], g[2]), pack_bf16x2(f[3], g[3]));
            dst[1] = make_uint4(pack_bf16x2(f[4], g[4]), pack_bf16x2(f[5], g[5]), pack_bf16x2(f[6], g[6]), pack_bf16x2(f[7], g[7]));
        } else {
            __nv_bfloat16 *dst = kp + natural_off(page, at, h, 0, P, a.Hkv, a.D);
            *reinterpret_cast<uint4 *>(dst + 8 * c) =
                make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
            *reinterpret_cast<uint4 *>(dst + H + 8 * c) =
                make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7]));
        }
        uint4 *dv = reinterpret_cast<uint4 *>(vp + natural_off(page, at, h, c, P, a.Hkv, a.D));
        dv[0] = v0;
        dv[1] = v1;
    }
}

// Block = (sequence, KV head, c): chunk c of K and of V of every accepted token.
// All of them are read into shared memory before the first is written, so a slot
// may be read and written in any order (and an index may come twice).
__global__ void __launch_bounds__(128) cache_compact_kernel(const CompactArgs a) {
    extern __shared__ uint4 stage[];  // [token][K 0, K 1, V 0, V 1]
    const int C = a.D / 16;
    const int c = blockIdx.x % C, h = blockIdx.x / C % a.Hkv, b = blockIdx.x / C / a.Hkv;
    const int64_t L = a.seqlens[b];
    const int n = max(0, min(a.accepted[b], a.M)), P = a.pk.page_size;
    uint4 *kp = static_cast<uint4 *>(a.kpages), *vp = static_cast<uint4 *>(a.vpages);
    for (int e = threadIdx.x; e < 4 * n; e += blockDim.x) {
        const int node = a.path[(size_t)b * a.M + (e >> 2)];
        const int64_t slot = L + node;
        const int page = node >= 0 ? page_of(a.pk, b, slot, a.status) : page_of(a.pk, b, -1, a.status);
        if (page < 0) continue;
        const int at = (int)(slot % P), part = e & 1;
        const size_t nat = natural_off(page, at, h, c, P, a.Hkv, a.D) / 8;
        if (e & 2) stage[e] = vp[nat + part];
        else stage[e] = kp[(a.packed ? packed_off(page, at, h, c, P, a.Hkv, a.D) / 8 : nat) + part];
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 4 * n; e += blockDim.x) {
        const int node = a.path[(size_t)b * a.M + (e >> 2)];
        const int64_t slot = L + (e >> 2);
        // A token whose source does not exist is not moved (reported above).
        if (node < 0 || page_of(a.pk, b, L + node, a.status) < 0) continue;
        const int page = page_of(a.pk, b, slot, a.status);
        if (page < 0) continue;
        const int at = (int)(slot % P), part = e & 1;
        const size_t nat = natural_off(page, at, h, c, P, a.Hkv, a.D) / 8;
        if (e & 2) vp[nat + part] = stage[e];
        else kp[(a.packed ? packed_off(page, at, h, c, P, a.Hkv, a.D) / 8 : nat) + part] = stage[e];
    }
    if (a.new_seqlens && c == 0 && h == 0 && threadIdx.x == 0) a.new_seqlens[b] = (int32_t)(L + n);
}

// Block = (page pair, K or V).  The filled part of a page is one run of bytes
// (V, NHD K) or one run per (head, chunk) (packed K).
__global__ void __launch_bounds__(256) cache_copy_pages_kernel(const CopyPagesArgs a) {
    const int pair = blockIdx.x, src = a.src[pair], dst = a.dst[pair];
    if (src < 0 || src >= a.num_pages || dst < 0 || dst >= a.num_pages) {
        if (threadIdx.x == 0) atomicCAS(a.status, 0, ATFLASH_DEVICE_BAD_PAGE);
        return;
    }
    const int n = a.tokens ? max(0, min(a.tokens[pair], a.page_size)) : a.page_size;
    const size_t page16 = (size_t)a.page_size * a.Hkv * a.D / 8;  // 16-byte units of a page
    const bool v = blockIdx.y != 0;
    uint4 *pool = static_cast<uint4 *>(v ? a.vpages : a.kpages);
    const uint4 *from = pool + (size_t)src * page16;
    uint4 *to = pool + (size_t)dst * page16;
    if (v || !a.packed || n == a.page_size) {
        const size_t run = (size_t)n * a.Hkv * a.D / 8;
        for (size_t e = threadIdx.x; e < run; e += blockDim.x) to[e] = from[e];
    } else {
        const int chunks = a.Hkv * a.D / 16;
        for (int e = threadIdx.x; e < chunks * 2 * n; e += blockDim.x) {
            const size_t o = (size_t)(e / (2 * n)) * 2 * a.page_size + e % (2 * n);
            to[o] = from[o];
        }
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs &a, const RopeTurns &rt, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.B * a.T * (a.D / 16) + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    cache_append_kernel<<<(unsigned)blocks, 256, 0, s>>>(a, rt);
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs &a, cudaStream_t s) {
    const size_t smem = (size_t)a.M * 64;
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(cache_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kCompactMaxPath * 64);
        if (e != cudaSuccess) return e;
    }
    cache_compact_kernel<<<(unsigned)(a.B * a.Hkv * (a.D / 16)), 128, smem, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_cache_copy_pages(const CopyPagesArgs &a, cudaStream_t s) {
    cache_copy_pages_kernel<<<dim3((unsigned)a.n, 2), 256, 0, s>>>(a);
    return cudaGetLastError();
}

}  // namespace atf
