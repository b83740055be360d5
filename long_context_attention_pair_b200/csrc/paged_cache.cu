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

// Two 16-byte halves of 32 bytes: one store where the pool allows it, so that no sector is
// written in two requests.
__device__ __forceinline__ void store32(void *p, uint4 x, uint4 y, bool whole) {
    if (whole) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x.x), "r"(x.y), "r"(x.z), "r"(x.w), "r"(y.x),
                     "r"(y.y), "r"(y.z), "r"(y.w)
                     : "memory");
    } else {
        static_cast<uint4 *>(p)[0] = x;
        static_cast<uint4 *>(p)[1] = y;
    }
}

// Thread = (token, c): pairs 8c..8c+7 of K and dims 8c.. and D/2 + 8c.. of V, for every KV
// head.  The cos and sin of the 8 pairs are taken once per token; a warp covers 32 / C
// consecutive tokens, so its reads and its writes are whole runs.  Each thread copies
// its first kStages heads asynchronously into shared memory of its own before it looks
// up the page and the angles, and stays that far ahead.
constexpr int kStages = 2;
__global__ void __launch_bounds__(256) cache_append_kernel(const AppendArgs a, const __grid_constant__ RopeTurns rt) {
    extern __shared__ uint4 ring[];  // [stage][K low half, K high half, V 0, V 1][thread]
    const int C = a.D / 16, H = a.D / 2;
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int bt = (int)(id >> (a.D == 128 ? 3 : 2));
    const bool exists = bt < a.B * a.T;
    const int c = (int)(id & (C - 1)), b = exists ? bt / a.T : 0, i = exists ? bt - b * a.T : 0;
    const bool live = exists && (!a.counts || i < a.counts[b]);
    const __nv_bfloat16 *k = static_cast<const __nv_bfloat16 *>(a.k) + b * a.ks.batch + i * a.ks.token;
    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.v) + b * a.vs.batch + i * a.vs.token;
    auto fetch = [&](int h) {
        if (live && h < a.Hkv) {
            uint4 *to = ring + h % kStages * 1024 + threadIdx.x;
            const __nv_bfloat16 *kh = k + h * a.ks.head, *vh = v + h * a.vs.head;
            copy_async(to, kh + 8 * c);
            copy_async(to + 256, kh + H + 8 * c);
            copy_async(to + 512, vh + 8 * c);
            copy_async(to + 768, vh + H + 8 * c);
        }
        copy_async_commit();
    };
#pragma unroll
    for (int h = 0; h < kStages; ++h) fetch(h);
    // (A parameter indexed by lane costs a pass for each distinct index: once per block here.)
    __shared__ uint64_t turn_of[64];
    if ((int)threadIdx.x < H) turn_of[threadIdx.x] = rt.turn[threadIdx.x];
    __syncthreads();
    if (!live) return;
    const int64_t L = a.seqlens[b], slot = L < 0 ? -1 : L + i;  // of a negative length no slot exists
    const int page = page_of(a.pk, b, slot, a.status);
    if (page < 0) {
        copy_async_wait<0>();  // nothing of this thread's is in flight when it leaves
        return;
    }
    const int P = a.pk.page_size, at = (int)((uint32_t)slot % (uint32_t)P);
    const int32_t pos = a.positions ? a.positions[bt] : (int32_t)slot;
    __nv_bfloat16 *kp = static_cast<__nv_bfloat16 *>(a.kpages), *vp = static_cast<__nv_bfloat16 *>(a.vpages);
    const bool whole = (reinterpret_cast<uintptr_t>(kp) & 31u) == 0;
    float2 cs[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) cs[j] = turn_cos_sin_fast(pos, turn_of[8 * c + j]);
    for (int h = 0; h < a.Hkv; ++h) {
        copy_async_wait<kStages - 1>();
        const uint4 *from = ring + h % kStages * 1024 + threadIdx.x;
        const uint4 lo = from[0], hi = from[256], v0 = from[512], v1 = from[768];
        fetch(h + kStages);
        const uint32_t x[4] = {lo.x, lo.y, lo.z, lo.w}, z[4] = {hi.x, hi.y, hi.z, hi.w};
        float f[8], g[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float xa = (j & 1) ? bf16hi(x[j >> 1]) : bf16lo(x[j >> 1]);
            const float xb = (j & 1) ? bf16hi(z[j >> 1]) : bf16lo(z[j >> 1]);
            f[j] = xa * cs[j].x - xb * cs[j].y;
            g[j] = xb * cs[j].x + xa * cs[j].y;
        }
        if (a.packed) {
            store32(kp + packed_off(page, at, h, c, P, a.Hkv, a.D),
                    make_uint4(pack_bf16x2(f[0], g[0]), pack_bf16x2(f[1], g[1]), pack_bf16x2(f[2], g[2]), pack_bf16x2(f[3], g[3])),
                    make_uint4(pack_bf16x2(f[4], g[4]), pack_bf16x2(f[5], g[5]), pack_bf16x2(f[6], g[6]), pack_bf16x2(f[7], g[7])), whole);
        } else {
            __nv_bfloat16 *dst = kp + natural_off(page, at, h, 0, P, a.Hkv, a.D);
            // Un-rotated keys are copied: a turn by nothing would still mix in 0 * infinity.
            *reinterpret_cast<uint4 *>(dst + 8 * c) =
                a.rotate ? make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7])) : lo;
            *reinterpret_cast<uint4 *>(dst + H + 8 * c) =
                a.rotate ? make_uint4(pack_bf16x2(g[0], g[1]), pack_bf16x2(g[2], g[3]), pack_bf16x2(g[4], g[5]), pack_bf16x2(g[6], g[7])) : hi;
        }
        __nv_bfloat16 *dv = vp + natural_off(page, at, h, 0, P, a.Hkv, a.D);
        *reinterpret_cast<uint4 *>(dv + 8 * c) = v0;
        *reinterpret_cast<uint4 *>(dv + H + 8 * c) = v1;
    }
}

// Block = (sequence, KV head, group of `per` chunks): those chunks of K and of V of every
// accepted token.  All of them are read into shared memory before the first is written,
// so a slot may be read and written in any order (and an index may come twice).  Where
// each token comes from and goes to is looked up once per block.
__global__ void __launch_bounds__(128) cache_compact_kernel(const CompactArgs a, int per) {
    extern __shared__ uint4 stage[];  // [token][chunk][K 0, K 1, V 0, V 1], then the places
    int2 *from = reinterpret_cast<int2 *>(stage + (size_t)a.M * per * 4), *to = from + a.M;  // (page, place in it)
    const int C = a.D / 16, groups = C / per;
    const int c0 = blockIdx.x % groups * per, h = blockIdx.x / groups % a.Hkv, b = blockIdx.x / groups / a.Hkv;
    const int64_t L = a.seqlens[b];
    const int n = max(0, min(a.accepted[b], a.M)), P = a.pk.page_size;
    uint4 *kp = static_cast<uint4 *>(a.kpages), *vp = static_cast<uint4 *>(a.vpages);
    for (int p = threadIdx.x; p < n; p += blockDim.x) {
        const int node = a.path[(size_t)b * a.M + p];
        const int64_t src = node >= 0 && L >= 0 ? L + node : -1;
        int2 f = make_int2(page_of(a.pk, b, src, a.status), 0), t = make_int2(page_of(a.pk, b, L + p, a.status), 0);
        if (f.x < 0 || t.x < 0) f.x = -1;  // a token whose source (or target) does not exist is not moved
        else f.y = (int)((uint32_t)src % (uint32_t)P), t.y = (int)((uint32_t)(L + p) % (uint32_t)P);
        from[p] = f;
        to[p] = t;
    }
    __syncthreads();
    auto place = [&](int2 at, int c, int part) -> uint4 * {  // part: K 0, K 1, V 0, V 1 of chunk c
        const size_t nat = natural_off(at.x, at.y, h, c, P, a.Hkv, a.D) / 8;
        if (part & 2) return vp + nat + (part & 1);
        return kp + (a.packed ? packed_off(at.x, at.y, h, c, P, a.Hkv, a.D) / 8 : nat) + (part & 1);
    };
    for (int e = threadIdx.x; e < 4 * per * n; e += blockDim.x) {
        const int p = e / (4 * per), x = e - p * 4 * per;
        if (from[p].x >= 0) stage[e] = *place(from[p], c0 + x / 4, x & 3);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 4 * per * n; e += blockDim.x) {
        const int p = e / (4 * per), x = e - p * 4 * per;
        if (from[p].x >= 0) *place(to[p], c0 + x / 4, x & 3) = stage[e];
    }
    if (a.new_seqlens && c0 == 0 && h == 0 && threadIdx.x == 0) a.new_seqlens[b] = (int32_t)(L + n);
}

// Block = (page pair, K or V, part of the page).  The filled part of a page is one run of
// bytes (V, NHD K) or one run per (head, chunk) (packed K).  Four 16-byte loads in flight
// per thread.
constexpr int kCopy = 4;
__global__ void __launch_bounds__(256) cache_copy_pages_kernel(const CopyPagesArgs a, int parts) {
    const int pair = blockIdx.x / parts, part = blockIdx.x - pair * parts, src = a.src[pair], dst = a.dst[pair];
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
    const bool runs = !v && a.packed && n < a.page_size;  // one run of 2 n units every 2 page_size
    const uint32_t total = (uint32_t)n * (uint32_t)(a.Hkv * a.D / 8), run = 2u * n;
    const uint32_t step = blockDim.x * parts;
    for (uint32_t e0 = part * blockDim.x + threadIdx.x; e0 < total; e0 += kCopy * step) {
        uint4 x[kCopy];
        uint32_t o[kCopy];
#pragma unroll
        for (int i = 0; i < kCopy; ++i) {
            const uint32_t e = e0 + i * step;
            if (e < total) {
                o[i] = runs ? e / run * 2u * a.page_size + e % run : e;
                x[i] = from[o[i]];
            }
        }
#pragma unroll
        for (int i = 0; i < kCopy; ++i)
            if (e0 + i * step < total) to[o[i]] = x[i];
    }
}

}  // namespace

cudaError_t launch_cache_append(const AppendArgs &a, const RopeTurns &rt, cudaStream_t s) {
    const int64_t blocks = ((int64_t)a.B * a.T * (a.D / 16) + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    constexpr int smem = kStages * 4 * 256 * 16;
    static_assert(smem + 64 * 8 <= 48 * 1024, "the ring and the turn counts need no opt-in");
    cache_append_kernel<<<(unsigned)blocks, 256, smem, s>>>(a, rt);
    return cudaGetLastError();
}

cudaError_t launch_cache_compact(const CompactArgs &a, cudaStream_t s) {
    // As many chunks per block as leave two blocks for each SM and stay within 32 KB; one for the
    // longest paths (64 bytes a token, and 16 for its places).
    const int C = a.D / 16;
    int per = C;
    while (per > 1 && ((int64_t)a.B * a.Hkv * (C / per) < 2 * 148 || (int64_t)a.M * (64 * per + 16) > 32 * 1024)) per /= 2;
    const size_t smem = (size_t)a.M * (64 * per + 16);
    if (smem > 48 * 1024) {
        cudaError_t e = cudaFuncSetAttribute(cache_compact_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             kCompactMaxPath * 80);
        if (e != cudaSuccess) return e;
    }
    cache_compact_kernel<<<(unsigned)(a.B * a.Hkv * (C / per)), 128, smem, s>>>(a, per);
    return cudaGetLastError();
}

cudaError_t launch_cache_copy_pages(const CopyPagesArgs &a, cudaStream_t s) {
    // 16 KB per block (one round of its threads' loads): many small blocks keep every SM's loads in flight.
    const int64_t page16 = (int64_t)a.page_size * a.Hkv * a.D / 8;
    int64_t parts = (page16 + 256 * kCopy - 1) / (256 * kCopy);
    while (parts * a.n > INT32_MAX) parts = (parts + 1) / 2;
    cache_copy_pages_kernel<<<dim3((unsigned)(parts * a.n), 2), 256, 0, s>>>(a, (int)parts);
    return cudaGetLastError();
}

}  // namespace atf
