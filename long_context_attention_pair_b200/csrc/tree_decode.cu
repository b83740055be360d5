// Windowed attention of a tree of drafted tokens over a paged KV cache, on the
// sm_100a tensor cores (tcgen05 + TMEM + TMA).
//
// Query node i of sequence b (position p_i) attends the cached slots m < L
// (position m) and the nodes j it sees (slot L + j, position p_j), with
//   s(i, m) = D^-1/2 * sum over pairs r with p_i - p_m <= w_r of (q~ . k~)_r,
// a softmax over what it sees and the weighted sum of values.
//
// Rows and keys.  The T nodes of a sequence times the G query heads of a KV head
// are the rows of one problem, node-major, cut into row tiles of 128 (the M of
// one tcgen05.mma); keys come in tiles of 128 slots.  A CTA holds one row tile's
// queries and walks key tiles: all rows share each K and V byte read.
//
// Work split.  A unit is one key tile of one (sequence, KV head, group of R row
// tiles); R CTAs, one for each row tile of the group, walk the same units at the
// same time (the second reads of a tile hit L2).  The units of the whole batch,
// counted on the device from seqlens and counts, are cut into equal runs, one for
// each of the 148 / R CTA groups, so a ragged batch loads the SMs evenly and no
// length is known on the host.  A run that covers an item whole writes its output;
// otherwise it leaves (max, sum, unscaled output) in the workspace, at most twice
// per CTA (its first and its last item), and tree_merge_kernel joins them.
//
// Windows.  Inside one tile the distances span [d_min, d_max]: pairs r < r_lo are
// pruned for every cell and their packed chunks not loaded, pairs r >= r_full are
// kept for every cell and go through the MMA, and the boundary pairs between are
// added per cell where the cell keeps them (the MMA sees zeros in their place, so
// a pruned element takes no part whatever it holds).
//
// Precision.  q~ is kept as two bf16 parts (hi + lo, 2^-16 of its value), so
// scores carry fp32-grade error; P is rounded to bf16 (the MMA's operand type,
// V's own), which moves an output by at most 2^-8 of sum p |v|; sums, maxima and
// O are fp32.
//
// 12 warps: 0-7 softmax (warp 4 hc + q4: TMEM lane quarter q4, columns 64 hc..;
// the two warps of a row exchange maxima per tile), 8 TMA producer, 9 QK issuer,
// 10 fix-up (zeroes boundary pairs in K, stages them, clears V behind the last
// node), 11 PV issuer.  S and P are double-buffered in TMEM, so the next tile's QK
// runs under this tile's softmax.  Every mbarrier wait is bounded; on expiry the
// CTA records ATFLASH_ERR_TIMEOUT, lets its copies and MMAs finish and exits.
#include <cuda_bf16.h>
#include <math.h>

#include "ptx.cuh"
#include "serving.h"

namespace atf {
namespace tree {

constexpr int kBM = 128, kBN = 128;
constexpr int kSoft = 8;
constexpr int kProducer = 8, kQk = 9, kFix = 10, kPv = 11;
constexpr int kThreads = 32 * 12;
// Registers: 168 per thread at launch; the last warpgroup drops to 96 and the two
// softmax warpgroups rise to 200, within the launch's total (checked here and,
// against the compiled kernel, at launch).
constexpr int kLaunchRegs = 168, kSoftRegs = 200, kOtherRegs = 96;
static_assert(256 * kSoftRegs + 128 * kOtherRegs <= kThreads * kLaunchRegs, "register split exceeds the launch");
constexpr int kSMs = 148;
constexpr int kMaxGroup = 8;     // row tiles that walk the same key tiles together
constexpr int kStaged = 16;      // boundary pairs staged per tile (at least one natural K-step)
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int D>
struct Cfg {
    static constexpr int H = D / 2;
    static constexpr int C = D / 16;                 // K-steps
    static constexpr int ST = D == 128 ? 2 : 4;      // K and V stages: 128 KB in flight or in use
    static constexpr int TileBytes = kBM * D * 2;    // Q hi, Q lo, a K stage, a V stage
    static constexpr int OffQ = 0;
    static constexpr int OffK = OffQ + 2 * TileBytes;
    static constexpr int OffV = OffK + ST * TileBytes;
    static constexpr int OffStage = OffV + ST * TileBytes;       // [ST][kStaged][128] words (k_r, k_{r+H})
    static constexpr int StageBytes = kStaged * kBN * 4;
    static constexpr int OffKpos = OffStage + ST * StageBytes;   // [ST][128] key positions
    static constexpr int OffCtl = OffKpos + ST * kBN * 4;
    static constexpr int CtlBytes = 5120;
    static constexpr int Request = OffCtl + CtlBytes + 1024;
    static_assert(Request <= 232448, "shared memory of one CTA");
    static constexpr uint32_t TmemS = 0, TmemO = 256, TmemP = 384, TmemCols = 512;
};

struct Ctl {
    uint64_t q_ready;
    uint64_t k_full[4], k_ready[4], k_empty[4], v_full[4], v_ready[4], v_empty[4];
    uint64_t s_full[2], s_read[2], p_full[2], o_done[2];
    uint64_t drain;
    uint64_t xbar[4], lbar[4];       // per lane quarter: both column halves have posted
    uint32_t tmem_base;
    int abort_flag;
    int first_b;
    int64_t first_off, run;          // this group's first unit inside sequence first_b, and its number of units
    int64_t total;
    int band[4][2];                  // (r_lo, r_full) of the tile in each stage
    int nf_seg[8];                   // segment (mod 8) whose tree holds a non-finite value
    int w[64];
    float xval[4][2][2][32];         // (quarter, tile parity, column half, lane)
    float lval[4][2][32];
};
static_assert(sizeof(Ctl) <= 5120, "control block outgrew its space");

// What the scheduler needs to know of a sequence.
struct Seq {
    int64_t L;
    int nodes;    // 0: nothing to do
    int tiles;    // key tiles
    int groups;   // row groups
};

struct Shape {
    int B, T, G, Hkv, R;  // R: row tiles per group
    int groups;           // CTA groups of the grid
};

__device__ __forceinline__ Seq seq_of(const TreeArgs &a, const Shape &sh, int b) {
    Seq s;
    s.L = a.seqlens[b];
    s.nodes = a.counts ? max(0, min(a.counts[b], a.T)) : a.T;
    // Slots that the table row has no room for: reported by tree_merge_kernel.
    if (s.L < 0 || s.L + s.nodes > (int64_t)a.pk.max_pages * a.pk.page_size) s.nodes = 0;
    s.tiles = s.nodes ? (int)((s.L + s.nodes + kBN - 1) / kBN) : 0;
    s.groups = (int)(((int64_t)s.nodes * sh.G + kBM * sh.R - 1) / (kBM * sh.R));
    return s;
}
__device__ __forceinline__ int64_t units_of(const Seq &s, int Hkv) { return (int64_t)Hkv * s.groups * s.tiles; }

// Units before sequence `b` (all of them for b = B), by a whole warp.
__device__ __forceinline__ int64_t units_before(const TreeArgs &a, const Shape &sh, int b) {
    int64_t sum = 0;
    for (int x = threadIdx.x & 31; x < b; x += 32) sum += units_of(seq_of(a, sh, x), sh.Hkv);
#pragma unroll
    for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    return sum;
}
// CTA groups with work, and the first unit of group g.
__device__ __forceinline__ int active_groups(int64_t total, int groups) { return total < groups ? (int)total : groups; }
__device__ __forceinline__ int64_t first_unit(int64_t total, int active, int g) { return (int64_t)g * total / active; }

// One run of key tiles of one item, as every warp of a CTA walks them.
struct Segment {
    int b, h;         // sequence, KV head
    int64_t L;
    int nodes;
    int row0, rows;   // this CTA's rows of the problem (rows <= 0: none)
    int tile0, ntile, tiles;
};
struct Walk {
    int b;
    int64_t off, left;
    Seq s;
    __device__ __forceinline__ void init(const TreeArgs &a, const Shape &sh, const Ctl *ctl) {
        b = ctl->first_b;
        off = ctl->first_off;
        left = ctl->run;
        if (left > 0) s = seq_of(a, sh, b);
    }
    __device__ __forceinline__ bool next(const TreeArgs &a, const Shape &sh, int member, Segment &g) {
        while (left > 0) {
            if (off >= units_of(s, sh.Hkv)) {
                off = 0;
                s = seq_of(a, sh, ++b);
                continue;
            }
            const int item = (int)(off / s.tiles);
            g.b = b;
            g.h = item / s.groups;
            g.L = s.L;
            g.nodes = s.nodes;
            g.row0 = (item % s.groups * sh.R + member) * kBM;
            g.rows = min(kBM, s.nodes * sh.G - g.row0);
            g.tiles = s.tiles;
            g.tile0 = (int)(off - (int64_t)item * s.tiles);
            g.ntile = (int)min((int64_t)(s.tiles - g.tile0), left);
            off += g.ntile;
            left -= g.ntile;
            if (g.rows > 0) return true;
        }
        return false;
    }
};

// Offset of 32-bit word `word` of row `row` in a K-step of 128 rows x 32 bytes
// (SWIZZLE_32B), and of element d in 128-byte rows of 64 dims (SWIZZLE_128B, one
// 16 KB block per 64 dims).
__device__ __forceinline__ uint32_t sw32_off(int row, int word) {
    return (uint32_t)row * 32u + (((uint32_t)word * 4u) ^ (((uint32_t)row & 4u) << 2));
}
__device__ __forceinline__ uint32_t sw128_off(int row, int d) {
    return (uint32_t)(d >> 6) * 16384u + (uint32_t)row * 128u + ((((uint32_t)(d & 63) >> 3) ^ ((uint32_t)row & 7u)) << 4) +
           ((uint32_t)d & 7u) * 2u;
}
// Pair r of a row of a Q or K tile as one word (x_r, x_{r+H}).
template <int D, bool kPacked>
__device__ __forceinline__ uint32_t load_pair(const uint8_t *tile, int row, int r) {
    if constexpr (kPacked) {
        return *reinterpret_cast<const uint32_t *>(tile + (r >> 3) * 4096 + sw32_off(row, r & 7));
    } else {
        const uint32_t lo = *reinterpret_cast<const uint16_t *>(tile + sw128_off(row, r));
        return lo | (uint32_t) * reinterpret_cast<const uint16_t *>(tile + sw128_off(row, r + D / 2)) << 16;
    }
}
template <int D, bool kPacked>
__device__ __forceinline__ void store_pair(uint8_t *tile, int row, int r, uint32_t x) {
    if constexpr (kPacked) {
        *reinterpret_cast<uint32_t *>(tile + (r >> 3) * 4096 + sw32_off(row, r & 7)) = x;
    } else {
        *reinterpret_cast<uint16_t *>(tile + sw128_off(row, r)) = (uint16_t)x;
        *reinterpret_cast<uint16_t *>(tile + sw128_off(row, r + D / 2)) = (uint16_t)(x >> 16);
    }
}

__device__ __forceinline__ int first_kept(const int *w, int H, int64_t d) {
    int lo = 0, hi = H;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if ((int64_t)w[mid] >= d) hi = mid; else lo = mid + 1;
    }
    return lo;
}

__device__ __forceinline__ bool wait_drain(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit_ns) return false;
    return true;
}

// Position of node i.
__device__ __forceinline__ int64_t node_pos(const TreeArgs &a, const Segment &g, int i) {
    return a.positions ? (int64_t)a.positions[(size_t)g.b * a.T + i] : g.L + i;
}
// Whether node i sees node j (both below g.nodes).
__device__ __forceinline__ bool node_sees(const TreeArgs &a, const Segment &g, int i, int j) {
    return a.mask ? a.mask[((size_t)g.b * a.T + i) * a.T + j] != 0 : j <= i;
}

template <int D, bool kPacked>
__global__ void __launch_bounds__(kThreads, 1)
    tree_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ TreeArgs a, const __grid_constant__ Shape sh,
                       const __grid_constant__ WindowParams wp, const __grid_constant__ RopeTurns rt, int box_keys) {
    using F = Cfg<D>;
    constexpr int H = F::H, C = F::C, ST = F::ST;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + F::OffQ, *sK = smem + F::OffK, *sV = smem + F::OffV;
    uint32_t *sStage = reinterpret_cast<uint32_t *>(smem + F::OffStage);
    int *sKpos = reinterpret_cast<int *>(smem + F::OffKpos);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + F::OffCtl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int member = blockIdx.x % sh.R, group = blockIdx.x / sh.R;

    if (warp == kQk) {
        tmem_alloc(&ctl->tmem_base, F::TmemCols);
        tmem_relinquish();
    } else if (warp == kPv) {
        if (lane == 0) {
            mbar_init(&ctl->q_ready, kSoft);
            for (int s = 0; s < ST; ++s) {
                mbar_init(&ctl->k_full[s], 1);
                mbar_init(&ctl->k_ready[s], 1);
                mbar_init(&ctl->k_empty[s], 1 + kSoft);
                mbar_init(&ctl->v_full[s], 1);
                mbar_init(&ctl->v_ready[s], 1);
                mbar_init(&ctl->v_empty[s], 1);
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(&ctl->s_full[s], 1);
                mbar_init(&ctl->s_read[s], kSoft);
                mbar_init(&ctl->p_full[s], kSoft);
                mbar_init(&ctl->o_done[s], 1);
            }
            mbar_init(&ctl->drain, 2);
            for (int q = 0; q < 4; ++q) {
                mbar_init(&ctl->xbar[q], 2);
                mbar_init(&ctl->lbar[q], 2);
            }
            ctl->abort_flag = 0;
            for (int s = 0; s < 8; ++s) ctl->nf_seg[s] = -1;
            fence_mbar_init();
        }
    } else if (warp == kProducer) {
        // This group's run of units: the total, then the sequence that holds the first.
        const int64_t total = units_before(a, sh, sh.B);
        const int active = active_groups(total, sh.groups);
        const int64_t u0 = group < active ? first_unit(total, active, group) : 0;
        const int64_t u1 = group < active ? first_unit(total, active, group + 1) : 0;
        int64_t base = 0;
        int found = 0;
        int64_t off = 0;
        for (int b0 = 0; b0 < sh.B && u1 > u0; b0 += 32) {
            const int b = b0 + lane;
            const int64_t n = b < sh.B ? units_of(seq_of(a, sh, b), sh.Hkv) : 0;
            int64_t incl = n;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const bool here = u0 >= base + incl - n && u0 < base + incl;
            const uint32_t m = __ballot_sync(0xffffffffu, here);
            if (m) {
                const int src = __ffs(m) - 1;
                found = b0 + src;
                off = u0 - __shfl_sync(0xffffffffu, base + incl - n, src);
                break;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        if (lane == 0) {
            ctl->first_b = found;
            ctl->first_off = off;
            ctl->run = u1 - u0;
            ctl->total = total;
            prefetch_tmap(&tm_k);
            prefetch_tmap(&tm_v);
        }
    } else if (warp == kFix) {
        for (int r = lane; r < H; r += 32) ctl->w[r] = wp.w[r];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_allow_dependents();
    const uint32_t tmem = ctl->tmem_base;
    const int *w = ctl->w;
    WaitCtl wc{&ctl->abort_flag, a.status, a.limit_ns, 40};
    Walk walk;
    walk.init(a, sh, ctl);
    Segment g;
    int it = 0, seg = 0;  // tiles and segments this CTA has walked
    bool ok = true;

    if (warp >= kSoft) setmaxnreg_dec<kOtherRegs>();
    if (warp == kProducer) {
        // ------------------------------------------------------------ producer
        int last[ST];
#pragma unroll
        for (int s = 0; s < ST; ++s) last[s] = -1;
        int lastv = -1;
        for (; ok && walk.next(a, sh, member, g); ++seg) {
            // Positions of this row tile's nodes, and the nearest position of any node as a key.
            const int i0 = g.row0 / sh.G, i1 = (g.row0 + g.rows - 1) / sh.G;
            int64_t pmin, pmax, kmin;
            if (a.positions) {
                int lo = INT32_MAX, hi = INT32_MIN, kl = INT32_MAX;
                for (int i = lane; i < g.nodes; i += 32) {
                    const int p = a.positions[(size_t)g.b * a.T + i];
                    kl = min(kl, p);
                    if (i >= i0 && i <= i1) lo = min(lo, p), hi = max(hi, p);
                }
                pmin = __reduce_min_sync(0xffffffffu, lo);
                pmax = __reduce_max_sync(0xffffffffu, hi);
                kmin = __reduce_min_sync(0xffffffffu, kl);
            } else {
                pmin = g.L + i0, pmax = g.L + i1, kmin = g.L;
            }
            const int64_t end = g.L + g.nodes;
            int r_lo = H, r_full = H;
            int page = -1;  // page of half-tile (tile0 & ~15) * 2 + lane
            for (int j = g.tile0; ok && j < g.tile0 + g.ntile; ++j, ++it) {
                const int st = it % ST;
                const int64_t m0 = (int64_t)j * kBN;
                if (j == g.tile0 || (j & 15) == 0) {
                    const int64_t slot = ((int64_t)(j & ~15) * 2 + lane) * 64;
                    page = slot < end ? page_of(a.pk, g.b, slot, a.status) : -1;
                }
                const int pg0 = __shfl_sync(0xffffffffu, page, (j & 15) * 2);
                const int pg1 = __shfl_sync(0xffffffffu, page, (j & 15) * 2 + 1);
                // The tile's band.  Over prefix tiles both distances shrink, so the bounds only
                // move down; a tile with nodes may hold any small distance.
                if (m0 + kBN <= g.L) {
                    const int64_t dmin = pmin - (m0 + kBN - 1), dmax = pmax - m0;
                    if (j == g.tile0) {
                        r_lo = first_kept(w, H, dmin);
                        r_full = first_kept(w, H, dmax);
                    }
                    while (r_lo > 0 && (int64_t)w[r_lo - 1] >= dmin) --r_lo;
                    while (r_full > 0 && (int64_t)w[r_full - 1] >= dmax) --r_full;
                } else {
                    r_lo = 0;
                    r_full = first_kept(w, H, pmax - (m0 < g.L && m0 < kmin ? m0 : kmin));
                }
                wc.site = 41;
                if (!(ok = mbar_wait_warp(&ctl->k_empty[st], ((it / ST) & 1) ^ 1, wc))) break;
                const int halves = box_keys == kBN || m0 + 64 < end ? 2 : 1;
                const int ca = r_lo >> 3;
                if (lane == 0) {
                    ctl->band[st][0] = r_lo;
                    ctl->band[st][1] = r_full;
                    const uint32_t bytes = kPacked ? (uint32_t)(C - ca) * 2048u * halves : (uint32_t)(D / 64) * 8192u * halves;
                    mbar_expect_tx(&ctl->k_full[st], bytes);
                }
                __syncwarp();
                last[st] = it;
                const int at = (int)(m0 % a.pk.page_size);
                const int hf = lane & 1, u = lane >> 1;  // lane = (K-step or dim group, half)
                const int pg = hf ? pg1 : pg0;
                const int hat = box_keys == kBN ? at : (int)((m0 + 64 * hf) % a.pk.page_size);
                const bool issue = hf < (box_keys == kBN ? 1 : halves);
                uint8_t *kst = sK + st * F::TileBytes, *vst = sV + st * F::TileBytes;
                if constexpr (kPacked) {
                    if (issue && u >= ca && u < C)
                        tma_load_3d(kst + u * 4096 + hf * 2048, &tm_k, &ctl->k_full[st], 0, hat, (pg * sh.Hkv + g.h) * C + u);
                } else {
                    if (issue && u < D / 64)
                        tma_load_4d(kst + u * 16384 + hf * 8192, &tm_k, &ctl->k_full[st], 64 * u, g.h, hat, pg);
                }
                wc.site = 42;
                if (!(ok = mbar_wait_warp(&ctl->v_empty[st], ((it / ST) & 1) ^ 1, wc))) break;
                if (lane == 0) mbar_expect_tx(&ctl->v_full[st], (uint32_t)(D / 64) * 8192u * halves);
                __syncwarp();
                lastv = it;
                if (issue && u < D / 64)
                    tma_load_4d(vst + u * 16384 + hf * 8192, &tm_v, &ctl->v_full[st], 64 * u, g.h, hat, pg);
            }
        }
        if (!ok) {
            // Let every copy land before the CTA exits.
            const uint64_t drain_ns = atflash_drain_limit_ns(a.limit_ns);
            for (int s = 0; s < ST; ++s)
                if (last[s] >= 0) {
                    wait_drain(&ctl->k_full[s], (last[s] / ST) & 1, drain_ns);
                    const int v = last[s] <= lastv ? last[s] : last[s] - ST;
                    if (v >= 0) wait_drain(&ctl->v_full[s], (v / ST) & 1, drain_ns);
                }
        }
    } else if (warp == kFix) {
        // ------------------------------------- boundary pairs of K, tail of V
        for (; ok && walk.next(a, sh, member, g); ++seg) {
            const int64_t end = g.L + g.nodes;
            for (int j = g.tile0; ok && j < g.tile0 + g.ntile; ++j, ++it) {
                const int st = it % ST;
                const int64_t m0 = (int64_t)j * kBN;
                wc.site = 43;
                if (!(ok = mbar_wait_warp(&ctl->k_full[st], (it / ST) & 1, wc))) break;
                const int r_lo = ctl->band[st][0], r_full = ctl->band[st][1];
                uint8_t *kst = sK + st * F::TileBytes;
                if (r_lo < r_full) {
                    int *kp = sKpos + st * kBN;
                    for (int e = lane; e < kBN; e += 32) {
                        const int64_t slot = m0 + e;
                        kp[e] = slot < g.L || slot >= end ? (int)slot : (int)node_pos(a, g, (int)(slot - g.L));
                    }
                    const int rs = max(r_lo, r_full - kStaged), nb = r_full - rs;
                    uint32_t *sw = sStage + st * (kStaged * kBN);
                    for (int e = lane; e < nb * kBN; e += 32)
                        sw[e] = load_pair<D, kPacked>(kst, e & (kBN - 1), rs + (e >> 7));
                    __syncwarp();
                }
                // Pairs of the first K-step of the MMA that are not kept by every cell.
                constexpr int kPer = kPacked ? 8 : 16;
                const int z0 = r_full / kPer * kPer;
                if (r_full > z0 && r_full <= H) {
                    const int nz = r_full - z0;
                    for (int e = lane; e < nz * kBN; e += 32) store_pair<D, kPacked>(kst, e & (kBN - 1), z0 + (e >> 7), 0u);
                    fence_proxy_async_smem();
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->k_ready[st]);
                if (m0 + kBN > g.L) {
                    // V behind the last node may hold anything (0 * NaN must not reach O), and so
                    // may a node that some rows do not see: its non-finite values are taken out
                    // here and put back for the rows that see them at the end of the segment.
                    wc.site = 44;
                    if (!(ok = mbar_wait_warp(&ctl->v_full[st], (it / ST) & 1, wc))) break;
                    uint8_t *vst = sV + st * F::TileBytes;
                    constexpr int kUnits = D / 8;  // 16-byte units of a row
                    bool bad = false;
                    const int first = (int)max(g.L - m0, (int64_t)0);
                    for (int e = first * kUnits + lane; e < kBN * kUnits; e += 32) {
                        const int row = e / kUnits, d = e % kUnits * 8;
                        uint4 *p = reinterpret_cast<uint4 *>(vst + sw128_off(row, d));
                        if (m0 + row >= end) {
                            *p = make_uint4(0, 0, 0, 0);
                            continue;
                        }
                        uint4 x = *p;
                        uint32_t *xs = reinterpret_cast<uint32_t *>(&x);
                        bool odd = false;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            if ((xs[i] & 0x7F80u) == 0x7F80u) xs[i] &= 0xFFFF0000u, odd = true;
                            if ((xs[i] & 0x7F800000u) == 0x7F800000u) xs[i] &= 0x0000FFFFu, odd = true;
                        }
                        if (odd) *p = x;
                        bad |= odd;
                    }
                    if (__any_sync(0xffffffffu, bad) && lane == 0) ctl->nf_seg[seg & 7] = seg;
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->v_ready[st]);
                }
            }
        }
    } else if (warp == kQk) {
        // ------------------------------------------------------- QK issuer
        const uint32_t idesc = idesc_bf16_f32(kBM, kBN, false, false);
        const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK);
        constexpr int kPer = kPacked ? 8 : 16, kSteps = H / kPer;
        for (; ok && walk.next(a, sh, member, g); ++seg) {
            wc.site = 45;
            if (!(ok = mbar_wait_warp(&ctl->q_ready, seg & 1, wc))) break;
            for (int j = 0; ok && j < g.ntile; ++j, ++it) {
                const int st = it % ST, buf = it & 1;
                wc.site = 46;
                if (!(ok = mbar_wait_warp(&ctl->k_ready[st], (it / ST) & 1, wc))) break;
                const int c0 = ctl->band[st][1] / kPer;
                wc.site = 47;
                if (it >= 2 && !(ok = mbar_wait_warp(&ctl->s_read[buf], ((it >> 1) - 1) & 1, wc))) break;
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t k0 = sKa + st * F::TileBytes, d = tmem + F::TmemS + buf * kBN;
                    uint32_t acc = 0;
                    for (int c = c0; c < kSteps; ++c) {
#pragma unroll
                        for (int part = 0; part < (kPacked ? 1 : 2); ++part) {
                            // Packed: one K-step is 8 whole pairs.  Natural: 16 dims of the low half,
                            // then their partners in the high half.
                            const int dim = 16 * c + part * H;
                            const uint32_t o = kPacked ? c * 4096u : (uint32_t)(dim >> 6) * 16384u + (uint32_t)(dim & 63) * 2u;
                            const uint64_t db = kPacked ? smem_desc(k0 + o, 16, 256, kSwizzle32B) : smem_desc(k0 + o, 16, 1024, kSwizzle128B);
#pragma unroll
                            for (int lo = 0; lo < 2; ++lo) {
                                const uint32_t q0 = sQa + lo * F::TileBytes + o;
                                const uint64_t da = kPacked ? smem_desc(q0, 16, 256, kSwizzle32B) : smem_desc(q0, 16, 1024, kSwizzle128B);
                                umma_bf16_ss(d, da, db, idesc, acc);
                                acc = 1;
                            }
                        }
                    }
                    umma_commit(&ctl->s_full[buf]);
                    umma_commit(&ctl->k_empty[st]);
                }
                __syncwarp();
            }
        }
    } else if (warp == kPv) {
        // ------------------------------------------------------- PV issuer
        const uint32_t idesc = idesc_bf16_f32(kBM, D, false, true);
        const uint32_t sVa = smem_u32(sV);
        uint32_t tails = 0;  // phase bit of v_ready per stage
        for (; ok && walk.next(a, sh, member, g); ++seg) {
            for (int j = g.tile0; ok && j < g.tile0 + g.ntile; ++j, ++it) {
                const int st = it % ST, buf = it & 1;
                wc.site = 48;
                if (!(ok = mbar_wait_warp(&ctl->v_full[st], (it / ST) & 1, wc))) break;
                if ((int64_t)(j + 1) * kBN > g.L) {
                    wc.site = 49;
                    if (!(ok = mbar_wait_warp(&ctl->v_ready[st], (tails >> st) & 1, wc))) break;
                    tails ^= 1u << st;
                }
                wc.site = 50;
                if (!(ok = mbar_wait_warp(&ctl->p_full[buf], (it >> 1) & 1, wc))) break;
                if (lane == 0) {
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kBN / 16; ++kk) {
                        const uint64_t db = smem_desc(sVa + st * F::TileBytes + kk * 2048, 16384, 1024, kSwizzle128B);
                        umma_bf16_ts(tmem + F::TmemO, tmem + F::TmemP + buf * 64 + kk * 8, db, idesc, (j > g.tile0 || kk > 0) ? 1u : 0u);
                    }
                    umma_commit(&ctl->o_done[buf]);
                    umma_commit(&ctl->v_empty[st]);
                }
                __syncwarp();
            }
        }
    } else {
        // ------------------------------------------------------------- softmax
        setmaxnreg_inc<kSoftRegs>();
        const int q4 = warp & 3, hc = warp >> 2;
        const int c0 = 64 * hc;
        constexpr int kO = D / 2;  // O columns of this warp
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint32_t tS = tmem + F::TmemS + lane_off + c0, tP = tmem + F::TmemP + lane_off + c0 / 2;
        const uint32_t tO = tmem + F::TmemO + lane_off + hc * kO;
        const float scale_log2 = 1.4426950408889634f * rsqrtf((float)D);
        int nx = 0, nl = 0;  // exchanges with the row's other warp
        for (; ok && walk.next(a, sh, member, g); ++seg) {
            const bool live = q4 * 32 < g.rows;  // some row of this quarter exists
            const int row = q4 * 32 + lane;
            const bool valid = row < g.rows;
            const int tok = valid ? (g.row0 + row) / sh.G : 0, head = valid ? (g.row0 + row) % sh.G : 0;
            const int64_t pos = valid ? node_pos(a, g, tok) : 0;
            const int64_t end = g.L + g.nodes;
            if (live) {
                // Rotate this quarter's queries into the MMA's layout (this warp: half of the
                // pairs of each row) as hi + lo bf16.  The previous segment's MMAs have read
                // their Q (its last S was waited for), the row's other warp too (it has posted
                // its sum).
                constexpr int kLP = H / 2, kRows = 32 / kLP;  // lanes per row, rows at a time
                const int pr = hc * kLP + lane % kLP;
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + g.b * a.qs.batch;
                int last_tok = -1;
                float2 cs = make_float2(1.f, 0.f);
#pragma unroll 1
                for (int r8 = 0; r8 < 32; r8 += 8 * kRows) {
                    __nv_bfloat16 xa[8], xb[8];
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int rr = q4 * 32 + r8 + u * kRows + lane / kLP;
                        xa[u] = xb[u] = __float2bfloat16_rn(0.f);
                        if (rr < g.rows) {
                            const int t = (g.row0 + rr) / sh.G, hh = g.h * sh.G + (g.row0 + rr) % sh.G;
                            const __nv_bfloat16 *src = q + t * a.qs.token + hh * a.qs.head;
                            xa[u] = src[pr];
                            xb[u] = src[pr + H];
                        }
                    }
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int rr = q4 * 32 + r8 + u * kRows + lane / kLP;
                        const int t = min(g.row0 + rr, g.row0 + g.rows - 1) / sh.G;
                        if (t != last_tok) {
                            cs = turn_cos_sin((int32_t)node_pos(a, g, t), rt.turn[pr]);
                            last_tok = t;
                        }
                        const float fa = __bfloat162float(xa[u]), fb = __bfloat162float(xb[u]);
                        const float x = fa * cs.x - fb * cs.y, y = fb * cs.x + fa * cs.y;
                        const uint32_t hi = pack_bf16x2(x, y);
                        const uint32_t lo = pack_bf16x2(x - bf16lo(hi), y - bf16hi(hi));
                        store_pair<D, kPacked>(sQ, rr, pr, hi);
                        store_pair<D, kPacked>(sQ + F::TileBytes, rr, pr, lo);
                    }
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->q_ready);
            wc.site = 51;
            if (!(ok = mbar_wait_warp(&ctl->q_ready, seg & 1, wc))) break;  // the other warp's half, for the boundary pairs

            float m_used = -INFINITY, lrun = 0.f;
            for (int j = g.tile0; ok && j < g.tile0 + g.ntile; ++j, ++it) {
                const int st = it % ST, buf = it & 1;
                const int64_t m0 = (int64_t)j * kBN;
                const bool tail = m0 + kBN > g.L;
                uint32_t see0 = 0xffffffffu, see1 = 0xffffffffu;  // this row's columns c0.., c0 + 32..
                if (tail && live) {
                    // Columns 32 c.. of every node of this quarter's rows, by ballot.
                    const int64_t s0 = m0 + c0 + lane, s1 = s0 + 32;
                    const int ta = (g.row0 + q4 * 32) / sh.G, tb = (g.row0 + min(q4 * 32 + 31, g.rows - 1)) / sh.G;
                    see0 = see1 = 0;
                    for (int t = ta; t <= tb; ++t) {
                        const bool v0 = s0 < end && (s0 < g.L || node_sees(a, g, t, (int)(s0 - g.L)));
                        const bool v1 = s1 < end && (s1 < g.L || node_sees(a, g, t, (int)(s1 - g.L)));
                        const uint32_t b0 = __ballot_sync(0xffffffffu, v0), b1 = __ballot_sync(0xffffffffu, v1);
                        if (t == tok) see0 = b0, see1 = b1;
                    }
                }
                wc.site = 52;
                if (!(ok = mbar_wait_warp(&ctl->k_ready[st], (it / ST) & 1, wc))) break;
                const int r_lo = ctl->band[st][0], r_full = ctl->band[st][1];
                wc.site = 53;
                if (!(ok = mbar_wait_warp(&ctl->s_full[buf], (it >> 1) & 1, wc))) break;
                tc_fence_after();
                float s[64];
                if (live) {
                    if (r_full < H) {
                        uint32_t ra[64];
                        tmem_ld_32x32b_x64(tS + buf * kBN, ra);
                        tmem_ld_wait(ra);
#pragma unroll
                        for (int i = 0; i < 64; ++i) s[i] = __uint_as_float(ra[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 64; ++i) s[i] = 0.f;
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->s_read[buf]);
                if (live && r_lo < r_full) {
                    const uint8_t *kst = sK + st * F::TileBytes;
                    const int4 *kp = reinterpret_cast<const int4 *>(sKpos + st * kBN + c0);
                    const int rs = max(r_lo, r_full - kStaged);
                    for (int r = r_lo; r < r_full; ++r) {
                        // Keys at positions >= lim keep the pair.
                        const int64_t l64 = pos - (int64_t)w[r];
                        const int lim = !valid || l64 > INT32_MAX ? INT32_MAX : (l64 < INT32_MIN ? INT32_MIN : (int)l64);
                        const uint32_t qh = load_pair<D, kPacked>(sQ, row, r), ql = load_pair<D, kPacked>(sQ + F::TileBytes, row, r);
                        const float qa = bf16lo(qh) + bf16lo(ql), qb = bf16hi(qh) + bf16hi(ql);
                        auto add4 = [&](int i, uint4 k) {
                            const int4 p = kp[i];
                            s[4 * i] += p.x >= lim ? fmaf(qa, bf16lo(k.x), qb * bf16hi(k.x)) : 0.f;
                            s[4 * i + 1] += p.y >= lim ? fmaf(qa, bf16lo(k.y), qb * bf16hi(k.y)) : 0.f;
                            s[4 * i + 2] += p.z >= lim ? fmaf(qa, bf16lo(k.z), qb * bf16hi(k.z)) : 0.f;
                            s[4 * i + 3] += p.w >= lim ? fmaf(qa, bf16lo(k.w), qb * bf16hi(k.w)) : 0.f;
                        };
                        if (r >= rs) {
                            const uint4 *kw = reinterpret_cast<const uint4 *>(sStage + st * (kStaged * kBN) + (r - rs) * kBN + c0);
#pragma unroll
                            for (int i = 0; i < 16; ++i) add4(i, kw[i]);
                        } else {
                            // More boundary pairs than staged: those below are whole in the K tile.
#pragma unroll
                            for (int i = 0; i < 16; ++i) {
                                uint4 k;
                                k.x = load_pair<D, kPacked>(kst, c0 + 4 * i, r);
                                k.y = load_pair<D, kPacked>(kst, c0 + 4 * i + 1, r);
                                k.z = load_pair<D, kPacked>(kst, c0 + 4 * i + 2, r);
                                k.w = load_pair<D, kPacked>(kst, c0 + 4 * i + 3, r);
                                add4(i, k);
                            }
                        }
                    }
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&ctl->k_empty[st]);
                float alpha = 1.f;
                bool need = false;
                uint32_t pk[32];
                float psum = 0.f;
                if (live) {
                    if (tail) {
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            if (!((see0 >> i) & 1u)) s[i] = -INFINITY;
                            if (!((see1 >> i) & 1u)) s[32 + i] = -INFINITY;
                        }
                    }
                    float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY, mx3 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < 64; i += 8) {
                        mx0 = max3(mx0, s[i], s[i + 1]);
                        mx1 = max3(mx1, s[i + 2], s[i + 3]);
                        mx2 = max3(mx2, s[i + 4], s[i + 5]);
                        mx3 = max3(mx3, s[i + 6], s[i + 7]);
                    }
                    float mx = fmaxf(fmaxf(mx0, mx1), fmaxf(mx2, mx3));
                    // The row's maximum over both column halves (a slot of this parity is rewritten
                    // only after the partner has passed the next exchange).
                    float *slot = ctl->xval[q4][nx & 1][0];
                    slot[hc * 32 + lane] = mx;
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->xbar[q4]);
                    wc.site = 54;
                    if (!(ok = mbar_wait_warp(&ctl->xbar[q4], nx & 1, wc))) break;
                    mx = fmaxf(mx, slot[(hc ^ 1) * 32 + lane]);
                    ++nx;
                    // The running max is kept unless it grew by more than 2^8: O / l uses the same
                    // one, so the result does not depend on it.
                    const float tile_max = mx * scale_log2;
                    need = tile_max > m_used + kRescaleThreshold;
                    const float m_new = need ? tile_max : m_used;
                    alpha = need ? fast_exp2(m_used - m_new) : 1.f;
                    m_used = m_new;
                    const float mr = m_used == -INFINITY ? 0.f : m_used;  // nothing seen so far
                    const float2 mneg = make_float2(-mr, -mr), sc2 = make_float2(scale_log2, scale_log2);
                    float2 l0 = make_float2(0.f, 0.f), l1 = make_float2(0.f, 0.f);
#pragma unroll
                    for (int i = 0; i < 32; i += 2) {
                        float2 xa = fma2(make_float2(s[2 * i], s[2 * i + 1]), sc2, mneg);
                        float2 xb = fma2(make_float2(s[2 * i + 2], s[2 * i + 3]), sc2, mneg);
                        xa.x = fast_exp2(xa.x);
                        xa.y = fast_exp2(xa.y);
                        xb.x = fast_exp2(xb.x);
                        xb.y = fast_exp2(xb.y);
                        l0 = add2(l0, xa);
                        l1 = add2(l1, xb);
                        pk[i] = pack_bf16x2(xa.x, xa.y);
                        pk[i + 1] = pack_bf16x2(xb.x, xb.y);
                    }
                    const float2 ls = add2(l0, l1);
                    psum = ls.x + ls.y;
                }
                // P of this parity is free once PV(it - 2) is done (every warp waits, also one
                // without rows: its arrivals must not run ahead of the others').
                if (it >= 2) {
                    wc.site = 55;
                    if (!(ok = mbar_wait_warp(&ctl->o_done[buf], ((it >> 1) - 1) & 1, wc))) break;
                    tc_fence_after();
                }
                if (live) {
                    if (j > g.tile0 && __any_sync(0xffffffffu, need)) {
                        // O may be rescaled once PV(it - 1) is done.
                        wc.site = 56;
                        if (!(ok = mbar_wait_warp(&ctl->o_done[buf ^ 1], ((it - 1) >> 1) & 1, wc))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int cc = 0; cc < kO / 32; ++cc) {
                            uint32_t r[32];
                            tmem_ld_32x32b_x32(tO + cc * 32, r);
                            tmem_ld_wait(r);
#pragma unroll
                            for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                            tmem_st_32x32b_x32(tO + cc * 32, r);
                        }
                    }
                    tmem_st_32x32b_x32(tP + buf * 64, pk);
                    tmem_st_wait();
                    lrun = lrun * alpha + psum;
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[buf]);
            }
            if (!ok) break;
            if (!live) continue;
            // The row's sum over both column halves, then O.
            ctl->lval[q4][hc][lane] = lrun;
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->lbar[q4]);
            wc.site = 57;
            if (!(ok = mbar_wait_warp(&ctl->lbar[q4], nl & 1, wc))) break;
            ++nl;
            lrun += ctl->lval[q4][hc ^ 1][lane];
            wc.site = 58;
            if (!(ok = mbar_wait_warp(&ctl->o_done[(it - 1) & 1], ((it - 1) >> 1) & 1, wc))) break;
            tc_fence_after();
            const bool whole = g.ntile == g.tiles;
            const bool odd = ctl->nf_seg[seg & 7] == seg;
            const float inv = whole ? (lrun == 0.f ? 0.f : 1.f / lrun) : 1.f;
            float *part = a.workspace + ((size_t)blockIdx.x * 2 + (g.tile0 > 0 ? 0 : 1)) * kBM * (D + 2);
            const size_t orow = ((size_t)g.b * a.T + tok) * a.Hq + g.h * sh.G + head;
#pragma unroll 1
            for (int cc = 0; cc < kO / 32; ++cc) {
                uint32_t r[32];
                __syncwarp();
                tmem_ld_32x32b_x32(tO + cc * 32, r);
                tmem_ld_wait(r);
                const int d0 = hc * kO + cc * 32;
                if (odd && valid) {
                    // Non-finite values of the nodes this row sees in this run of tiles.
                    const int64_t lo = max(g.L, (int64_t)g.tile0 * kBN), hi = min(end, (int64_t)(g.tile0 + g.ntile) * kBN);
                    for (int64_t slot = lo; slot < hi; ++slot) {
                        if (!node_sees(a, g, tok, (int)(slot - g.L))) continue;
                        const int page = page_of(a.pk, g.b, slot, a.status);
                        if (page < 0) continue;
                        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.vpages) +
                                                 (((size_t)page * a.pk.page_size + slot % a.pk.page_size) * sh.Hkv + g.h) * D + d0;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x = __bfloat162float(v[i]);
                            if (!isfinite(x)) r[i] = __float_as_uint(__uint_as_float(r[i]) + x);
                        }
                    }
                }
                if (!valid) continue;
                if (!whole) {
                    float4 *dst = reinterpret_cast<float4 *>(part + 2 * kBM + (size_t)row * D + d0);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[i] = make_float4(__uint_as_float(r[4 * i]), __uint_as_float(r[4 * i + 1]), __uint_as_float(r[4 * i + 2]),
                                             __uint_as_float(r[4 * i + 3]));
                } else if (a.out_f32) {
                    float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + orow * D + d0);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        dst[i] = make_float4(__uint_as_float(r[4 * i]) * inv, __uint_as_float(r[4 * i + 1]) * inv,
                                             __uint_as_float(r[4 * i + 2]) * inv, __uint_as_float(r[4 * i + 3]) * inv);
                } else {
                    uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D + d0);
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        uint32_t x[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            x[e] = pack_bf16x2(__uint_as_float(r[8 * i + 2 * e]) * inv, __uint_as_float(r[8 * i + 2 * e + 1]) * inv);
                        dst[i] = make_uint4(x[0], x[1], x[2], x[3]);
                    }
                }
            }
            if (valid && hc == 0) {
                if (!whole) {
                    part[row] = m_used;
                    part[kBM + row] = lrun;
                } else if (a.lse) {
                    a.lse[((size_t)g.b * a.Hq + g.h * sh.G + head) * a.T + tok] =
                        lrun == 0.f ? -INFINITY : (m_used + log2f(lrun)) * 0.69314718055994531f;
                }
            }
        }
    }

    // Teardown: every tensor-core operation must be complete before TMEM is freed.
    __syncthreads();
    if (warp == kPv && lane == 0) umma_commit(&ctl->drain);
    if (warp == kQk) {
        if (lane == 0) {
            umma_commit(&ctl->drain);
            wait_drain(&ctl->drain, 0, atflash_drain_limit_ns(a.limit_ns));
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tmem, F::TmemCols);
    }
}

// Joins the partial states of the rows whose item was cut between CTA groups; a
// warp takes one row.  Rows of whole items were written by the kernel above.
template <int D>
__global__ void __launch_bounds__(256) tree_merge_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ Shape sh) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31;
    const int64_t id = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
    const bool exists = id < (int64_t)a.B * a.T * a.Hq;
    const int hq = (int)(id % a.Hq), i = (int)(id / a.Hq % a.T), b = exists ? (int)(id / a.Hq / a.T) : 0;
    const Seq s = seq_of(a, sh, b);
    const int64_t before = units_before(a, sh, b), total = units_before(a, sh, sh.B);
    if (exists && i == 0 && hq == 0 && lane == 0) {
        const int64_t L = a.seqlens[b];
        const int n = a.counts ? max(0, min(a.counts[b], a.T)) : a.T;
        if (L < 0 || L + n > (int64_t)a.pk.max_pages * a.pk.page_size) atomicCAS(a.status, 0, ATFLASH_DEVICE_BAD_PAGE);
    }
    pdl_wait();  // by every warp, so that this grid never ends before the one it depends on
    if (!exists || i >= s.nodes) return;
    const int h = hq / sh.G, r = i * sh.G + hq % sh.G, rt = r / kBM;
    const int64_t first = before + ((int64_t)h * s.groups + rt / sh.R) * s.tiles;
    const int active = active_groups(total, sh.groups);
    // Group of unit x: the largest g with floor(g * total / active) <= x.
    const int g0 = (int)(((first + 1) * active - 1) / total), g1 = (int)(((first + s.tiles) * active - 1) / total);
    if (g0 == g1) return;
    const int row = r % kBM;
    auto state = [&](int g) {
        // The item is the last of group g0's run and the first of the later ones'.
        return a.workspace + (((size_t)g * sh.R + rt % sh.R) * 2 + (g == g0 ? 1 : 0)) * kBM * (D + 2);
    };
    float M = -INFINITY;
    for (int g = g0 + lane; g <= g1; g += 32) M = fmaxf(M, state(g)[row]);
#pragma unroll
    for (int o = 16; o; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float mr = M == -INFINITY ? 0.f : M;
    float sum = 0.f, acc[V];
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] = 0.f;
#pragma unroll 4
    for (int g = g0; g <= g1; ++g) {
        const float *p = state(g);
        const float l = p[kBM + row], f = fast_exp2(p[row] - mr);
        sum += l * f;
        const float *o = p + 2 * kBM + (size_t)row * D + lane * V;
#pragma unroll
        for (int v = 0; v < V; ++v) acc[v] += o[v] * f;
    }
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const size_t off = (size_t)id * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (a.out_f32) static_cast<float *>(a.out)[off + v] = acc[v] * inv;
        else static_cast<__nv_bfloat16 *>(a.out)[off + v] = __float2bfloat16_rn(acc[v] * inv);
    }
    if (a.lse && lane == 0)
        a.lse[((size_t)b * a.Hq + hq) * a.T + i] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
}

Shape shape_of(int B, int T, int Hq, int Hkv) {
    Shape sh{B, T, Hq / Hkv, Hkv, 1, kSMs};
    const int64_t rt = ((int64_t)T * sh.G + kBM - 1) / kBM, groups = (rt + kMaxGroup - 1) / kMaxGroup;
    sh.R = (int)((rt + groups - 1) / groups);
    sh.groups = kSMs / sh.R;
    return sh;
}

cudaError_t make_map(CUtensorMap *map, const void *base, int rank, const cuuint64_t *dims, const cuuint64_t *strides,
                     const cuuint32_t *box, CUtensorMapSwizzle swz) {
    EncodeTiledFn enc = encode_tiled_fn();
    if (!enc) return cudaErrorNotSupported;
    cuuint32_t estr[5] = {1, 1, 1, 1, 1};
    const CUresult r = enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, (cuuint32_t)rank, const_cast<void *>(base), dims, strides, box, estr,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, swz, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int D, bool kPacked>
cudaError_t launch(const TreeArgs &a, const WindowParams &wp, const RopeTurns &rt, cudaStream_t s) {
    const Shape sh = shape_of(a.B, a.T, a.Hq, a.Hkv);
    // One box covers a tile where pages hold whole tiles, half a tile otherwise.
    const int box_keys = a.pk.page_size % kBN == 0 ? kBN : 64;
    const cuuint64_t P = (cuuint64_t)a.pk.page_size, NP = (cuuint64_t)a.pk.num_pages, Hk = (cuuint64_t)a.Hkv;
    CUtensorMap tk, tv;
    cudaError_t e;
    cuuint64_t dv[4] = {D, Hk, P, NP}, sv[3] = {D * 2, Hk * D * 2, P * Hk * D * 2};
    cuuint32_t bv[4] = {64, 1, (cuuint32_t)box_keys, 1};
    if ((e = make_map(&tv, a.vpages, 4, dv, sv, bv, CU_TENSOR_MAP_SWIZZLE_128B)) != cudaSuccess) return e;
    if (kPacked) {
        cuuint64_t dk[3] = {16, P, NP * Hk * (D / 16)}, sk[2] = {32, P * 32};
        cuuint32_t bk[3] = {16, (cuuint32_t)box_keys, 1};
        e = make_map(&tk, a.kpages, 3, dk, sk, bk, CU_TENSOR_MAP_SWIZZLE_32B);
    } else {
        e = make_map(&tk, a.kpages, 4, dv, sv, bv, CU_TENSOR_MAP_SWIZZLE_128B);
    }
    if (e != cudaSuccess) return e;
    if ((e = cudaFuncSetAttribute(tree_decode_kernel<D, kPacked>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::Request)) !=
        cudaSuccess)
        return e;
    // The in-kernel register split assumes this launch count: refuse to run otherwise.
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, tree_decode_kernel<D, kPacked>)) != cudaSuccess) return e;
    if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
    tree_decode_kernel<D, kPacked><<<sh.groups * sh.R, kThreads, Cfg<D>::Request, s>>>(tk, tv, a, sh, wp, rt, box_keys);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    const int64_t rows = (int64_t)a.B * a.T * a.Hq;
    return launch_dependent(tree_merge_kernel<D>, dim3((unsigned)((rows + 7) / 8)), dim3(256), 0, s, a, sh);
}

}  // namespace tree

// Two partial states of one row tile per CTA, whatever the lengths.
size_t tree_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
    const tree::Shape sh = tree::shape_of(B, T, Hq, Hkv);
    return (size_t)sh.groups * sh.R * 2 * tree::kBM * (D + 2) * sizeof(float);
}

cudaError_t launch_tree_decode(const TreeArgs &a, const WindowParams &wp, const RopeTurns &rt, cudaStream_t s) {
    if (a.D == 128) return a.packed ? tree::launch<128, true>(a, wp, rt, s) : tree::launch<128, false>(a, wp, rt, s);
    return a.packed ? tree::launch<64, true>(a, wp, rt, s) : tree::launch<64, false>(a, wp, rt, s);
}

}  // namespace atf
