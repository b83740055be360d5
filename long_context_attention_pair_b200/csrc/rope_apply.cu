// Rotary positions of queries and keys at given positions.
//
// Pair r of a head (dims (r, r + R/2), or (2r, 2r + 1) when interleaved, R the
// rotated dims) becomes (x c - z s, z c + x s) with (c, s) = scale * (cos, sin)
// of position * theta_r; the other dims are copied.  The inverse (angles
// negated) is the gradient of the forward rotation.
//
// A thread owns V pairs of one token, takes their cos and sin once and applies
// them to every head of its block's head range, so the trigonometry is shared by
// all heads; consecutive threads own consecutive pairs, so a warp reads and
// writes whole 128-byte runs.  The work is bound by HBM: each element is read
// once and written once.
#include <cuda_bf16.h>

#include "ptx.cuh"
#include "serving.h"

namespace atf {
namespace {

template <typename T>
__device__ __forceinline__ float to_f(T x) { return (float)x; }
template <typename T>
__device__ __forceinline__ T from_f(float x);
template <>
__device__ __forceinline__ float from_f<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f<__nv_bfloat16>(float x) { return __float2bfloat16_rn(x); }

// V elements as one aligned access (V * sizeof(E) is 16, or one element).
template <typename E, int V>
struct alignas(V * sizeof(E)) Vec {
    E e[V];
};

template <typename E, int V>
__global__ void __launch_bounds__(256) rope_apply_kernel(RopeTensor q, RopeTensor k,
                                                         const int32_t *__restrict__ positions, int64_t BT, int64_t T,
                                                         int D, int units, int interleaved, float scale, float sgn,
                                                         int heads_per_block, const __grid_constant__ RopeTurns rt) {
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    const int64_t bt = id / units;
    if (bt >= BT) return;
    const int u = (int)(id - bt * units);
    const int64_t b = bt / T, t = bt - b * T;
    const int R = rt.pairs, RU = R / V;  // rotated units come first
    const bool rot = u < RU;
    // The unit's two runs of V elements.
    const int d0 = rot ? (interleaved ? 2 * V * u : V * u) : 2 * R + 2 * V * (u - RU);
    const int d1 = rot && !interleaved ? d0 + R : d0 + V;
    float c[V], s[V];
    if (rot) {
        const int32_t pos = positions[bt];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const float2 cs = turn_cos_sin(pos, rt.turn[V * u + i]);
            c[i] = cs.x * scale;
            s[i] = cs.y * scale * sgn;
        }
    }
    const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, q.heads + k.heads);
    for (int h = h0; h < h1; ++h) {
        const RopeTensor &x = h < q.heads ? q : k;
        const int hh = h < q.heads ? h : h - q.heads;
        const E *src = static_cast<const E *>(x.x) + b * x.xs.batch + t * x.xs.token + hh * x.xs.head;
        E *dst = static_cast<E *>(x.y) + b * x.ys.batch + t * x.ys.token + hh * x.ys.head;
        Vec<E, V> a = *reinterpret_cast<const Vec<E, V> *>(src + d0);
        Vec<E, V> z = *reinterpret_cast<const Vec<E, V> *>(src + d1);
        if (rot) {
            if (interleaved) {
                // Elements 2i, 2i + 1 of the 2V contiguous ones are pair i.
                E p[2 * V];
#pragma unroll
                for (int i = 0; i < V; ++i) p[i] = a.e[i], p[V + i] = z.e[i];
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float f = to_f(p[2 * i]), g = to_f(p[2 * i + 1]);
                    p[2 * i] = from_f<E>(f * c[i] - g * s[i]);
                    p[2 * i + 1] = from_f<E>(g * c[i] + f * s[i]);
                }
#pragma unroll
                for (int i = 0; i < V; ++i) a.e[i] = p[i], z.e[i] = p[V + i];
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float f = to_f(a.e[i]), g = to_f(z.e[i]);
                    a.e[i] = from_f<E>(f * c[i] - g * s[i]);
                    z.e[i] = from_f<E>(g * c[i] + f * s[i]);
                }
            }
        }
        *reinterpret_cast<Vec<E, V> *>(dst + d0) = a;
        *reinterpret_cast<Vec<E, V> *>(dst + d1) = z;
    }
}

bool multiple_of(const Strides &s, int v) { return s.batch % v == 0 && s.token % v == 0 && s.head % v == 0; }

template <typename E, int V>
cudaError_t launch(const RopeTensor &q, const RopeTensor &k, const int32_t *positions, int B, int64_t T, int D,
                   const RopeTurns &rt, float scale, int interleaved, int inverse, cudaStream_t s) {
    // D - 2 * pairs elements are copied; with V = 1 a copied unit is 2 elements (both counts are even).
    const int units = rt.pairs / V + (D - 2 * rt.pairs) / (2 * V);
    const int64_t BT = B * T, blocks = (BT * units + 255) / 256;
    if (blocks > INT32_MAX) return cudaErrorInvalidValue;
    const int heads = q.heads + k.heads;
    rope_apply_kernel<E, V><<<dim3((unsigned)blocks, (unsigned)heads), 256, 0, s>>>(
        q, k, positions, BT, T, D, units, interleaved, scale, inverse ? -1.f : 1.f, 1, rt);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope_apply(const RopeTensor &q, const RopeTensor &k, const int32_t *positions, int B, int64_t T,
                              int D, const RopeTurns &rt, float scale, int interleaved, int inverse, int f32,
                              cudaStream_t s) {
    // 16-byte accesses where every run of a unit starts on a 16-byte boundary:
    // whole vectors of pairs, whole units of copied dims, and strides that keep
    // rows aligned (the tensors themselves are).  Single elements otherwise.
    const int v = f32 ? 4 : 8;
    const bool wide = rt.pairs % v == 0 && (D - 2 * rt.pairs) % (2 * v) == 0 && multiple_of(q.xs, v) &&
                      multiple_of(q.ys, v) && (k.heads == 0 || (multiple_of(k.xs, v) && multiple_of(k.ys, v)));
    if (f32)
        return wide ? launch<float, 4>(q, k, positions, B, T, D, rt, scale, interleaved, inverse, s)
                    : launch<float, 1>(q, k, positions, B, T, D, rt, scale, interleaved, inverse, s);
    return wide ? launch<__nv_bfloat16, 8>(q, k, positions, B, T, D, rt, scale, interleaved, inverse, s)
                : launch<__nv_bfloat16, 1>(q, k, positions, B, T, D, rt, scale, interleaved, inverse, s);
}

}  // namespace atf
