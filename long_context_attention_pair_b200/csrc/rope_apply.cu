// Rotary positions of queries and keys at given positions.
//
// Pair r of a head (dims (r, r + R/2), or (2r, 2r + 1) when interleaved, R the
// rotated dims) becomes (x c - z s, z c + x s) with (c, s) = scale * (cos, sin)
// of position * theta_r; the other dims are copied.  The inverse (angles
// negated) is the gradient of the forward rotation.
//
// A thread owns V pairs of one token, takes their cos and sin once and applies
// them to the heads of its block's range; consecutive threads own consecutive
// pairs, so a warp reads and writes whole 128-byte runs.  The work is bound by
// HBM (each element is read once and written once), that is by the bytes in
// flight: each thread copies its next kStages heads asynchronously into shared
// memory that no other thread touches, which takes neither registers nor barriers
// (the same loads into registers, two heads ahead, reached 0.73 of the copy rate
// on a prompt of 32768 tokens, 28 + 4 heads of 128 bf16).
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

constexpr int kStages = 4;  // heads whose loads a thread has in flight

template <typename E, int V>
__global__ void __launch_bounds__(256) rope_apply_kernel(RopeTensor q, RopeTensor k, const int32_t *__restrict__ positions, int BT,
                                                         int T, int D, int units, int interleaved, float scale, float sgn,
                                                         int heads_per_block, const __grid_constant__ RopeTurns rt) {
    // (A parameter indexed by lane costs a pass for each distinct index: once per block here.)
    __shared__ uint64_t turn_of[kMaxPairs];
    for (int r = threadIdx.x; r < rt.pairs; r += blockDim.x) turn_of[r] = rt.turn[r];
    __syncthreads();
    const int64_t id = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
    if (id >= (int64_t)BT * units) return;
    const int bt = (int)(id >> 31 ? id / units : (uint32_t)id / (uint32_t)units);
    const int u = (int)(id - (int64_t)bt * units);
    const int b = bt / T, t = bt - b * T;
    const int R = rt.pairs, RU = R / V;  // rotated units come first
    const bool rot = u < RU;
    // The unit's two runs of V elements: of the rotated dims the u-th of either half (which are
    // partners, or with interleaved pairs hold V/2 pairs each), of the others likewise.  A single
    // interleaved pair is its two neighbours.
    const bool one = V == 1 && interleaved && rot;
    const int rest = D - 2 * R;
    const int d0 = one ? 2 * u : rot ? V * u : 2 * R + V * (u - RU);
    const int d1 = one ? d0 + 1 : d0 + (rot ? R : rest / 2);
    float c[V], s[V];
    auto trig = [&]() {
        if (!rot) return;
        const int32_t pos = positions[bt];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int r = V > 1 && interleaved ? (i < V / 2 ? d0 / 2 + i : d1 / 2 + i - V / 2) : V * u + i;
            const float2 cs = sizeof(E) == 2 ? turn_cos_sin_fast(pos, turn_of[r]) : turn_cos_sin(pos, turn_of[r]);
            c[i] = cs.x * scale;
            s[i] = cs.y * scale * sgn;
        }
    };
    auto turn = [&](Vec<E, V> &a, Vec<E, V> &z) {
        if (!rot) return;
        if (V > 1 && interleaved) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                E *e = (i < V / 2 ? a.e : z.e) + 2 * (i % (V > 1 ? V / 2 : 1));
                const float f = to_f(e[0]), g = to_f(e[1]);
                e[0] = from_f<E>(f * c[i] - g * s[i]);
                e[1] = from_f<E>(g * c[i] + f * s[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const float f = to_f(a.e[i]), g = to_f(z.e[i]);
                a.e[i] = from_f<E>(f * c[i] - g * s[i]);
                z.e[i] = from_f<E>(g * c[i] + f * s[i]);
            }
        }
    };
    const int h0 = blockIdx.y * heads_per_block, h1 = min(h0 + heads_per_block, q.heads + k.heads);
    auto source = [&](int h) {
        const RopeTensor &x = h < q.heads ? q : k;
        return static_cast<const E *>(x.x) + b * x.xs.batch + t * x.xs.token + (h < q.heads ? h : h - q.heads) * x.xs.head;
    };
    auto target = [&](int h) {
        const RopeTensor &x = h < q.heads ? q : k;
        return static_cast<E *>(x.y) + b * x.ys.batch + t * x.ys.token + (h < q.heads ? h : h - q.heads) * x.ys.head;
    };
    if constexpr (V == 1) {
        trig();
        for (int h = h0; h < h1; ++h) {
            const E *src = source(h);
            E *dst = target(h);
            Vec<E, V> a{src[d0]}, z{src[d1]};
            turn(a, z);
            dst[d0] = a.e[0];
            dst[d1] = z.e[0];
        }
    } else {
        extern __shared__ uint4 ring[];  // [stage][run][thread]
        auto fetch = [&](int h) {
            if (h < h1) {
                uint4 *to = ring + (h - h0) % kStages * 512 + threadIdx.x;
                const E *src = source(h);
                copy_async(to, src + d0);
                copy_async(to + 256, src + d1);
            }
            copy_async_commit();
        };
#pragma unroll
        for (int i = 0; i < kStages; ++i) fetch(h0 + i);
        trig();
        for (int h = h0; h < h1; ++h) {
            copy_async_wait<kStages - 1>();
            const uint4 *at = ring + (h - h0) % kStages * 512 + threadIdx.x;
            Vec<E, V> a = *reinterpret_cast<const Vec<E, V> *>(at), z = *reinterpret_cast<const Vec<E, V> *>(at + 256);
            turn(a, z);
            E *dst = target(h);
            *reinterpret_cast<Vec<E, V> *>(dst + d0) = a;
            *reinterpret_cast<Vec<E, V> *>(dst + d1) = z;
            fetch(h + kStages);
        }
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
    // The heads of a token share its trigonometry; they are split between blocks as far as it
    // takes to have sixteen blocks for each SM, four to a block at least.
    const int heads = q.heads + k.heads;
    int per = (int)((heads * blocks + 16 * 148 - 1) / (16 * 148));
    per = per < 4 ? 4 : per;
    if (per > heads) per = heads;
    const size_t smem = V == 1 ? 0 : kStages * 2 * 256 * 16;
    rope_apply_kernel<E, V><<<dim3((unsigned)blocks, (unsigned)((heads + per - 1) / per)), 256, smem, s>>>(
        q, k, positions, (int)BT, (int)T, D, units, interleaved, scale, inverse ? -1.f : 1.f, per, rt);
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
