// Windowed attention of a tree of drafted tokens over a paged KV cache.
//
// Query node i of sequence b (position p_i) attends the cached slots m < L
// (position m) and the nodes j it sees (slot L + j, position p_j), with
//   s(i, m) = D^-1/2 * sum over pairs r with p_i - p_m <= w_r of (q~ . k~)_r,
// a softmax over what it sees and the weighted sum of values.  K is rotated
// already (NHD or packed pages); the query is rotated here.
//
// One block per (sequence, node, query head): each warp takes every eighth key,
// a lane holds D/64 pairs of the query and D/32 dims of the output, in fp32.
#include <cuda_bf16.h>
#include <math.h>

#include "ptx.cuh"
#include "serving.h"

namespace atf {
namespace {

constexpr int kWarps = 8;

template <int D>
__global__ void __launch_bounds__(32 * kWarps) tree_decode_kernel(const TreeArgs a,
                                                                  const __grid_constant__ WindowParams wp,
                                                                  const __grid_constant__ RopeTurns rt) {
    constexpr int H = D / 2, PL = D / 64;
    __shared__ float sm[kWarps], sl[kWarps], so[kWarps][D];
    const int hq = blockIdx.x % a.Hq, i = blockIdx.x / a.Hq % a.T, b = blockIdx.x / a.Hq / a.T;
    const int nodes = a.counts ? min(a.counts[b], a.T) : a.T;
    if (i >= nodes) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int h = hq / (a.Hq / a.Hkv);
    const int64_t L = a.seqlens[b];
    const int64_t bt = (int64_t)b * a.T;
    const int64_t pos = a.positions ? a.positions[bt + i] : L + i;
    const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + b * a.qs.batch + i * a.qs.token + hq * a.qs.head;
    float qa[PL], qb[PL];
    int w[PL];
#pragma unroll
    for (int u = 0; u < PL; ++u) {
        const int r = 32 * u + lane;
        const float2 cs = turn_cos_sin((int32_t)pos, rt.turn[r]);
        const float x = __bfloat162float(q[r]), z = __bfloat162float(q[r + H]);
        qa[u] = x * cs.x - z * cs.y;
        qb[u] = z * cs.x + x * cs.y;
        w[u] = wp.w[r];
    }
    const float scale = 1.4426950408889634f * rsqrtf((float)D);
    float m = -INFINITY, l = 0.f, o[D / 32];
#pragma unroll
    for (int u = 0; u < D / 32; ++u) o[u] = 0.f;
    const int P = a.pk.page_size;
    const __nv_bfloat16 *kp = static_cast<const __nv_bfloat16 *>(a.kpages), *vp = static_cast<const __nv_bfloat16 *>(a.vpages);
    for (int64_t slot = warp; slot < L + nodes; slot += kWarps) {
        const int64_t j = slot - L;
        if (j >= 0) {
            const bool sees = a.mask ? a.mask[(bt + i) * a.T + j] != 0 : j <= i;
            if (!sees) continue;
        }
        const int64_t kpos = j < 0 ? slot : (a.positions ? a.positions[bt + j] : slot);
        const int page = page_of(a.pk, b, slot, a.status);
        if (page < 0) continue;
        const int at = (int)(slot % P);
        const __nv_bfloat16 *v = vp + (((size_t)page * P + at) * a.Hkv + h) * D;
        float s = 0.f;
#pragma unroll
        for (int u = 0; u < PL; ++u) {
            const int r = 32 * u + lane;
            float ka, kb;
            if (a.packed) {
                const __nv_bfloat16 *kc = kp + ((((size_t)page * a.Hkv + h) * (D / 16) + (r >> 3)) * P + at) * 16;
                ka = __bfloat162float(kc[2 * (r & 7)]);
                kb = __bfloat162float(kc[2 * (r & 7) + 1]);
            } else {
                const __nv_bfloat16 *kc = kp + (((size_t)page * P + at) * a.Hkv + h) * D;
                ka = __bfloat162float(kc[r]);
                kb = __bfloat162float(kc[r + H]);
            }
            s += pos - kpos <= w[u] ? qa[u] * ka + qb[u] * kb : 0.f;
        }
#pragma unroll
        for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= scale;
        const float mn = fmaxf(m, s), mr = mn == -INFINITY ? 0.f : mn;
        const float al = fast_exp2(m - mr), p = fast_exp2(s - mr);
        l = l * al + p;
#pragma unroll
        for (int u = 0; u < D / 32; ++u) o[u] = o[u] * al + p * __bfloat162float(v[32 * u + lane]);
        m = mn;
    }
    if (lane == 0) sm[warp] = m, sl[warp] = l;
#pragma unroll
    for (int u = 0; u < D / 32; ++u) so[warp][32 * u + lane] = o[u];
    __syncthreads();
    const int d = threadIdx.x;
    if (d >= D) return;
    float M = -INFINITY, sum = 0.f, acc = 0.f;
    for (int x = 0; x < kWarps; ++x) M = fmaxf(M, sm[x]);
    for (int x = 0; x < kWarps; ++x) {
        if (sl[x] == 0.f) continue;
        const float f = fast_exp2(sm[x] - M);
        sum += sl[x] * f;
        acc += so[x][d] * f;
    }
    const float res = sum == 0.f ? 0.f : acc / sum;
    const size_t off = ((size_t)(bt + i) * a.Hq + hq) * D + d;
    if (a.out_f32) static_cast<float *>(a.out)[off] = res;
    else static_cast<__nv_bfloat16 *>(a.out)[off] = __float2bfloat16_rn(res);
    if (a.lse && d == 0)
        a.lse[((size_t)b * a.Hq + hq) * a.T + i] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
}

}  // namespace

size_t tree_workspace_bytes(int, int, int, int, int) { return 256; }

cudaError_t launch_tree_decode(const TreeArgs &a, const WindowParams &wp, const RopeTurns &rt, cudaStream_t s) {
    const unsigned grid = (unsigned)(a.B * a.T * a.Hq);
    if (a.D == 128) tree_decode_kernel<128><<<grid, 32 * kWarps, 0, s>>>(a, wp, rt);
    else tree_decode_kernel<64><<<grid, 32 * kWarps, 0, s>>>(a, wp, rt);
    return cudaGetLastError();
}

}  // namespace atf
