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
// each of the 148 / R CTA groups, so sequences of unequal lengths load the groups
// evenly and no length is known on the host.  (Unequal node counts do not where R > 1:
// R comes from T, and CTAs whose row tiles a smaller tree lacks skip its items.)  A run
// that covers an item whole writes its output; otherwise it leaves (max, sum, unscaled
// output) in the workspace, at most twice per CTA (its first and its last item), and
// tree_merge_kernel joins them.
//
// Softmax.  Two sets of four warps take alternate key tiles; a row's two warps hand
// its running max on from tile to tile and add into one O, so a set has two tile
// times for its part of the chain S -> P -> PV.  NC is the number of a tile's columns
// that one warp takes: with at most 32 (64) rows the queries are repeated in all four
// (both halves) of the MMA's 128 rows and each copy takes a quarter (half) of the
// columns, P being zero in the others, which shortens the chain where few rows leave
// the lanes empty.  The copies' states are joined at the end of a run of tiles.
//
// Windows.  Inside one tile the distances span [d_min, d_max]: pairs r < r_lo are
// pruned for every cell and their packed chunks not loaded, pairs r >= r_full are
// kept for every cell.  Of a boundary pair in between, the keys that every row keeps
// stay in the MMA's operand, the others are zeroed there, and those that some rows
// keep (as many as the nodes' positions differ by; none for a single token) are added
// per cell.  A pruned element thus takes no part whatever it holds.
//
// Precision.  q~ is kept as two bf16 parts (hi + lo, 2^-16 of its value), so
// scores carry fp32-grade error; sums, maxima and O are fp32.  So is P (two parts, two
// MMAs for each 16 keys) for fp32 outputs and for row tiles with rows that may see 128
// keys or fewer, where a rounding of P does not average out.  Otherwise P is rounded to
// bf16 once, which moves an output by at most 2^-8 of sum p |v|, as much as its own
// rounding to bf16 may.  On 8 ragged sequences of up to 8192 keys the rms error of bf16
// outputs is 0.0023 of theirs (0.0017 with two parts, their own rounding), of fp32 ones
// 4e-6.  Two parts everywhere took 63.6 us against 60.5 there, 116 against 108 on 4
// sequences of 64K keys and 430 against 368 on 2 of 128K with trees of 64 nodes.
//
// Warps: the softmax warps, then one each for loading K, issuing QK, the fix-up of K
// (boundary pairs staged, they and pruned pairs zeroed), issuing PV, loading V and
// scheduling (it publishes the runs of tiles through a ring), and two for the tails (mask
// bits of tiles with nodes, V behind the last node cleared).  Every mbarrier wait is
// bounded; on expiry the CTA records ATFLASH_ERR_TIMEOUT, lets its copies and MMAs finish
// and exits.
//
// What bounds it.  A steady key tile takes 2 200 to 2 600 clocks: two K stages (D = 128)
// whose cycle is copy issue 900, arrival 1 300 to 1 900, fix-up 400, QK 1 200 to 1 600 and
// release 300.  Within it the tensor pipe has 1 190 clocks of work on 2 sequences of 128K
// keys with trees of 64 nodes and k = 16 (5.3 of 8 K-steps of QK, each for both parts of
// q~, and PV: 320 GFLOP issued, padded rows included, where the kept pairs and one part of
// q~ need 194) and the exponentials 1 024; its counters read 44 % (tensor) and 56 % (tc) of
// the elapsed clocks.  A CTA's first P comes about 20 000 clocks after its start, through
// code that is fetched cold, and a change of item costs as much again: that bounds small
// calls and ragged batches, and there short loops beat unrolled ones (the MMA issue loops:
// 68 -> 61 us on 8 ragged sequences of up to 8192 keys with trees of 16).  Device time back
// to back in bursts at 1965 MHz: 1 sequence of 1021 keys 22.4 us; the 8 ragged ones 60.9;
// 4 sequences of 64K keys, one token each, no window 106, 0.77 of the copy rate; the 2 of
// 128K keys 342, 566 TFLOP/s of the 194 GFLOP.
#include <cuda_bf16.h>
#include <math.h>

#include <atomic>
#include <type_traits>

#include "ptx.cuh"
#include "serving.h"

namespace atf {
namespace tree {

constexpr int kBM = 128, kBN = 128;
constexpr int kSoft = 8;
constexpr int kProducer = 8, kQk = 9, kFix = 10, kPv = 11, kVProducer = 12, kSched = 13, kTail = 14;
constexpr int kThreads = 32 * 16;
// Registers: 128 per thread at launch; the last two warpgroups drop to 72 and the two
// softmax warpgroups rise to 184, within the launch's total (checked here and,
// against the compiled kernel, at launch).
constexpr int kLaunchRegs = 128, kSoftRegs = 184, kOtherRegs = 72;
static_assert(256 * kSoftRegs + 256 * kOtherRegs <= kThreads * kLaunchRegs, "register split exceeds the launch");
constexpr int kSMs = 148;
constexpr int kMaxGroup = 8;     // row tiles that walk the same key tiles together
// Key tiles that an item's own cost counts for.  us for 3, 6, 8, 10, 12: 8 ragged sequences of
// up to 8192 keys (48 rows) 61.7, 60.8, 62.4, 64.2, 64.2; 32 of up to 4000 111, 98.9, 101, 102,
// 104; 6 of up to 16K with 448 rows 134, 125, 124, 123, 124; 6 of up to 30K with 14 rows 63.9,
// 64.3, 64.9, 64.3, 65.5.
constexpr int kItemCost = 6;
constexpr int kBufs = 3;         // S / P buffers
constexpr int kRing = 4;         // runs of tiles published ahead
constexpr int kMergeThreads = 256;
constexpr int kShort = 128;      // a row that sees so few keys is one of a sequence with as few committed tokens
constexpr float kRescaleThreshold = 8.0f;  // log2 units

template <int D, bool kPacked>
struct Cfg {
    static constexpr int H = D / 2;
    static constexpr int C = D / 16;                 // K-steps
    static constexpr int ST = D == 128 ? 2 : 4;      // K and V stages: 128 KB in flight or in use (even: a stage serves one set)
    static constexpr int TileBytes = kBM * D * 2;    // Q hi, Q lo, a K stage, a V stage
    static constexpr int OffQ = 0;                   // also the fp32 exchange of repeated rows: 128 x D x 4
    static constexpr int OffK = OffQ + 2 * TileBytes;
    static constexpr int OffV = OffK + ST * TileBytes;
    // Boundary pairs staged per tile (at least those of one K-step), and buffers of them.  A
    // packed tile's K stage is released when its QK is done, so its staged pairs need a ring
    // that is rewritten only after its softmax: K of tile it + Cells is loaded after QK(it + 3),
    // which waits for PV(it).  In natural order the softmax holds the K stage instead.
    static constexpr int Staged = kPacked ? 8 : 16, Cells = kPacked ? ST + 3 : ST;
    static constexpr int OffStage = OffV + ST * TileBytes;       // [Cells][Staged][128] words (k_r, k_{r+H})
    static constexpr int OffKpos = OffStage + Cells * Staged * kBN * 4;  // [Cells][128] key positions
    static constexpr int OffMask = OffKpos + Cells * kBN * 4;    // [2][128] rows of 128 mask bits, one per node
    static constexpr int OffCtl = OffMask + 2 * kBM * 16;
    static constexpr int CtlBytes = 6144;
    static constexpr int Request = OffCtl + CtlBytes + 1024;
    static_assert(Request <= 232448, "shared memory of one CTA");
    // TMEM: S of a tile in one of three buffers at 0, 128 and 256, its P over the columns of S that
    // have been read (64 columns of bf16 pairs; in two parts, for each 16 keys 8 columns of high and 8
    // of low parts in the place of their scores), O at 384.
    static constexpr uint32_t TmemO = 384, TmemCols = 512;
};

// One run of key tiles of one item.
struct Segment {
    int b, h;         // sequence, KV head
    int L, nodes;
    int row0, rows;   // this CTA's rows of the problem; rows == 0: no more runs
    int tile0, ntile, tiles;
    int pmin, pmax;   // positions of the row tile's nodes
    int kmin;         // smallest position of a node (as a key)
    int fine;         // P in two bf16 parts
};

struct Ctl {
    uint64_t seg_full[kRing], seg_empty[kRing];
    uint64_t q_ready;
    uint64_t k_full[4], k_ready[4], k_empty[4], v_full[4], v_tail[4], v_ready[4], v_empty[4];
    uint64_t s_full[kBufs], p_full[kBufs], o_done[kBufs];  // per S / P buffer
    uint64_t m_full[2], m_empty[2];
    uint64_t max_bar[2][4];          // per set and lane quarter: the running max after its tile is posted
    uint64_t drain, soft_bar;
    uint32_t tmem_base;
    int abort_flag;
    Segment seg[kRing];
    int4 band[8];                    // of tile it in entry it % 8: (r_lo, rs, r_full, flags), see make_band.  (A tile's
                                     // entry is rewritten only after its PV, hence after every reader.)
    uint32_t chunks[7];              // 32-key chunks of the tile in which cells are added
    uint32_t zone[7][16];            // of staged pair rs + i: first key and end of the keys added per cell
    int nf_seg[8];                   // run (mod 8) whose tree holds a non-finite value
    int w[64];
    uint64_t turn[64];
    float2 stat[2][kBM];             // (max, sum) of each set and MMA row
    float run_max[2][kBM];           // running max after each set's latest tile
};
static_assert(sizeof(Ctl) <= 6144, "control block outgrew its space");

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
    s.groups = (int)(((uint32_t)s.nodes * (uint32_t)sh.G + (uint32_t)(kBM * sh.R) - 1u) / (uint32_t)(kBM * sh.R));  // B*T*Hq < 2^31
    return s;
}
// Units of one item, and of a sequence: its tiles and kItemCost for what a run costs beside
// them (queries in, state out, the boundary pairs near the queries), counted at its end.
__device__ __forceinline__ int item_units(const Seq &s) { return s.tiles ? s.tiles + kItemCost : 0; }
__device__ __forceinline__ int64_t units_of(const Seq &s, int Hkv) { return (int64_t)Hkv * s.groups * item_units(s); }

// CTA groups with work, and the first unit of group g.
__device__ __forceinline__ int active_groups(int64_t total, int groups) { return total < groups ? (int)total : groups; }
__device__ __forceinline__ int64_t first_unit(int64_t total, int active, int g) {
    const int64_t x = (int64_t)g * total;
    return x >> 31 ? x / active : (uint32_t)x / (uint32_t)active;  // the 64-bit division is a long subroutine
}

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
// Pairs r .. r + 3 (r a multiple of 4) of a row.
template <int D, bool kPacked>
__device__ __forceinline__ void store_quad(uint8_t *tile, int row, int r, const uint32_t (&x)[4]) {
    if constexpr (kPacked) {
        *reinterpret_cast<uint4 *>(tile + (r >> 3) * 4096 + sw32_off(row, r & 7)) = make_uint4(x[0], x[1], x[2], x[3]);
    } else {
        *reinterpret_cast<uint2 *>(tile + sw128_off(row, r)) = make_uint2(__byte_perm(x[0], x[1], 0x5410), __byte_perm(x[2], x[3], 0x5410));
        *reinterpret_cast<uint2 *>(tile + sw128_off(row, r + D / 2)) = make_uint2(__byte_perm(x[0], x[1], 0x7632), __byte_perm(x[2], x[3], 0x7632));
    }
}
// The first n words of 32 bytes that lie in two 16-byte units.
__device__ __forceinline__ void zero_words(uint8_t *u0, uint8_t *u1, int n) {
    uint8_t *u = n < 4 ? u0 : u1;
    if (n >= 4) *reinterpret_cast<uint4 *>(u0) = make_uint4(0, 0, 0, 0);
    if (n & 2) *reinterpret_cast<uint2 *>(u) = make_uint2(0, 0);
    if (n & 1) *reinterpret_cast<uint32_t *>(u + (n & 2) * 4) = 0;
}
// Pairs of one MMA K-step (packed) or of a K-step and its partner (natural).
template <bool kPacked>
constexpr int kPairsPerStep = kPacked ? 8 : 16;
// How a tile's pairs are treated: r < r_lo pruned for every cell; [r_lo, rs) added per
// cell for every key, straight from the K tile (only when more pairs are boundary
// than can be staged); [rs, r_full) staged, the MMA keeping the keys that every row
// keeps; r >= r_full kept for every cell.  The MMA starts at the K-step of rs.
// Flags: boundary pairs exist (the fix-up warp has work); some cells are added; the
// softmax warps hold the K stage.
//
// With a boundary pair rs < r_full <= H: either all of them are staged and rs = r_lo, or
// r_full - kStaged is rounded up to a K-step and kStaged is one.  In a tile with nodes r_lo
// is 0, so rs < H there too: the MMA leaves no S unwritten that cells are added to or
// hidden in.
enum : int { kBandFix = 1, kBandCells = 2, kBandHold = 4 };
template <int D, bool kPacked>
__device__ __forceinline__ int4 make_band(int r_lo, int r_full, bool spread) {
    constexpr int kPer = kPairsPerStep<kPacked>, kStaged = Cfg<D, kPacked>::Staged;
    static_assert(kStaged >= kPer, "a K-step's pairs fit the staging");
    const int rs = r_full - r_lo > kStaged ? (r_full - kStaged + kPer - 1) / kPer * kPer : r_lo;
    int flags = r_lo < r_full ? kBandFix : 0;
    if (r_lo < rs || (spread && r_lo < r_full)) flags |= kBandCells | (!kPacked || r_lo < rs ? kBandHold : 0);
    return make_int4(r_lo, rs, r_full, flags);
}

// r*(d) = the smallest r with w_r >= d (H when none), by a warp whose lanes hold the
// windows of pairs lane and lane + 32 (INT32_MAX past H): the windows do not decrease.
__device__ __forceinline__ int first_kept(int w0, int w1, int64_t d) {
    return __popc(__ballot_sync(0xffffffffu, w0 < d)) + __popc(__ballot_sync(0xffffffffu, w1 < d));
}

// Bounded wait of a whole warp.  Short, for the instruction cache's sake; the (slow)
// global timer is first read after a whole suspended attempt.
__device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, const WaitCtl &wc, uint32_t site) {
    bool ok = mbar_try_wait(bar, parity);
    if (!ok) {
        uint64_t t0 = 0, now = 0;
        while (!(ok = mbar_try_wait_sleep(bar, parity, 20000u)) && !*wc.abort_flag && now - t0 <= wc.limit_ns) {
            now = globaltimer_ns();
            if (t0 == 0) t0 = now;
        }
        if (!ok) {
            *wc.abort_flag = 1;
            atomicCAS(wc.status, 0, ATFLASH_DEVICE_TIMEOUT_BASE + (int)site);
        }
    }
    return __all_sync(0xffffffffu, ok);
}
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile("{\n\t.reg .b64 st;\n\tmbarrier.arrive.shared::cta.b64 st, [%0], %1;\n\t}" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ bool wait_drain(uint64_t *bar, uint32_t parity, uint64_t limit_ns) {
    const uint64_t t0 = globaltimer_ns();
    while (!mbar_try_wait(bar, parity))
        if (globaltimer_ns() - t0 > limit_ns) return false;
    return true;
}

// The runs of tiles, in order, as every warp but the scheduler sees them.
struct Runs {
    Ctl *ctl;
    int n = 0;  // runs taken
    __device__ __forceinline__ explicit Runs(Ctl *c) : ctl(c) {}
    __device__ __forceinline__ const Segment &now() const { return ctl->seg[(n - 1) % kRing]; }
    __device__ __forceinline__ bool next(WaitCtl &wc, bool &ok) {
        ok = wait(&ctl->seg_full[n % kRing], (n / kRing) & 1, wc, 59);
        if (!ok) return false;
        ++n;
        return now().rows > 0;
    }
    __device__ __forceinline__ void done(int lane) {  // every lane has read what it needs of the run
        __syncwarp();
        if (lane == 0) mbar_arrive(&ctl->seg_empty[(n - 1) % kRing]);
    }
};

__device__ __forceinline__ int node_pos(const TreeArgs &a, int b, int L, int i) {
    return a.positions ? a.positions[(size_t)b * a.T + i] : L + i;
}
// Whether node i sees node j (both below the sequence's count).
__device__ __forceinline__ bool node_sees(const TreeArgs &a, int b, int i, int j) {
    return a.mask ? a.mask[((size_t)b * a.T + i) * a.T + j] != 0 : j <= i;
}

__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t *r) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(
            taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
        "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

// Non-finite values of the nodes that row `tok` sees among the slots of tiles
// [tile0, tile0 + ntile), added to its output dims d0 .. d0 + N - 1 (the fix-up of the
// values that the tail warps took out of the MMA's operand).
template <int N>
__device__ __noinline__ void add_nonfinite(const TreeArgs &a, const Segment &g, int D, int tok, int d0, float *o) {
    const int64_t end = (int64_t)g.L + g.nodes;
    const int64_t lo = max((int64_t)g.L, (int64_t)g.tile0 * kBN), hi = min(end, (int64_t)(g.tile0 + g.ntile) * kBN);
    for (int64_t slot = lo; slot < hi; ++slot) {
        if (!node_sees(a, g.b, tok, (int)(slot - g.L))) continue;
        const int page = page_of(a.pk, g.b, slot, a.status);
        if (page < 0) continue;
        const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(a.vpages) +
                                 (((size_t)page * a.pk.page_size + slot % a.pk.page_size) * a.Hkv + g.h) * D + d0;
        for (int i = 0; i < N; ++i) {
            const float x = __bfloat162float(v[i]);
            if (!isfinite(x)) o[i] += x;
        }
    }
}

template <int D, bool kPacked, int NC>
__global__ void __launch_bounds__(kThreads, 1)
    tree_decode_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ TreeArgs a, const __grid_constant__ Shape sh,
                       const __grid_constant__ WindowParams wp, const __grid_constant__ RopeTurns rt, int box_keys) {
    using F = Cfg<D, kPacked>;
    constexpr int kStaged = F::Staged;
    constexpr int H = F::H, C = F::C, ST = F::ST;
    constexpr int kRep = kBN / NC, kRows = kBM / kRep;  // copies of the rows, rows of a copy
    constexpr int kPer = kPairsPerStep<kPacked>;
    constexpr int CW = 32;                             // columns in registers at a time
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem + F::OffQ, *sK = smem + F::OffK, *sV = smem + F::OffV;
    uint32_t *sStage = reinterpret_cast<uint32_t *>(smem + F::OffStage);
    int *sKpos = reinterpret_cast<int *>(smem + F::OffKpos);
    uint4 *sMask = reinterpret_cast<uint4 *>(smem + F::OffMask);
    Ctl *ctl = reinterpret_cast<Ctl *>(smem + F::OffCtl);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == kQk) {
        tmem_alloc(&ctl->tmem_base, F::TmemCols);
        tmem_relinquish();
    } else if (warp == kPv) {
        if (lane == 0) {
            for (int s = 0; s < kRing; ++s) {
                mbar_init(&ctl->seg_full[s], 1);
                mbar_init(&ctl->seg_empty[s], kThreads / 32 - 1);
            }
            mbar_init(&ctl->q_ready, kSoft);
            for (int s = 0; s < ST; ++s) {
                mbar_init(&ctl->k_full[s], 1);
                mbar_init(&ctl->k_ready[s], 1);
                mbar_init(&ctl->k_empty[s], 1 + 4);  // QK, the set's softmax warps
                mbar_init(&ctl->v_full[s], 1);
                mbar_init(&ctl->v_tail[s], 1);
                mbar_init(&ctl->v_ready[s], 2);
                mbar_init(&ctl->v_empty[s], 1);
            }
            for (int s = 0; s < kBufs; ++s) {
                mbar_init(&ctl->s_full[s], 2);  // the MMAs, and the issuing warp (for what it has seen of the stage)
                mbar_init(&ctl->p_full[s], 4);
                mbar_init(&ctl->o_done[s], 1);
            }
            for (int s = 0; s < 2; ++s) {
                mbar_init(&ctl->m_full[s], 2);
                mbar_init(&ctl->m_empty[s], 4);
                for (int q = 0; q < 4; ++q) mbar_init(&ctl->max_bar[s][q], 1);
            }
            mbar_init(&ctl->drain, 2);
            mbar_init(&ctl->soft_bar, kSoft);
            ctl->abort_flag = 0;
            for (int s = 0; s < 8; ++s) ctl->nf_seg[s] = -1;
            fence_mbar_init();
        }
    } else if (warp == kProducer) {
        if (lane == 0) prefetch_tmap(&tm_k);
    } else if (warp == kVProducer) {
        if (lane == 0) prefetch_tmap(&tm_v);
    } else if (warp == kFix) {
        for (int r = lane; r < H; r += 32) ctl->w[r] = wp.w[r];
    } else if (warp == kTail) {
        // (Read by lane from shared memory later: a parameter indexed by lane costs a pass per lane.)
        for (int r = lane; r < H; r += 32) ctl->turn[r] = rt.turn[r];
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_allow_dependents();
    const uint32_t tmem = ctl->tmem_base;
    const int *w = ctl->w;
    WaitCtl wc{&ctl->abort_flag, a.status, a.limit_ns, 40};
    Runs runs(ctl);
    int it = 0;  // tiles this CTA has walked
    bool ok = true;

    if (warp >= kSoft) setmaxnreg_dec<kOtherRegs>();
    if (warp == kSched) {
        // ------------------------------------------------------------ scheduler
        // This group's run of units: the total, then the sequence that holds the first.
        const int member = blockIdx.x % sh.R, group = blockIdx.x / sh.R;
        Seq ls{};  // this lane's sequence of the first 32
        int64_t ln = 0, total = 0;
        for (int b0 = 0; b0 < sh.B; b0 += 32) {
            const Seq x = b0 + lane < sh.B ? seq_of(a, sh, b0 + lane) : Seq{};
            const int64_t n = units_of(x, sh.Hkv);
            if (b0 == 0) ls = x, ln = n;
            total += n;
        }
#pragma unroll
        for (int o = 16; o; o >>= 1) total += __shfl_xor_sync(0xffffffffu, total, o);
        const int active = active_groups(total, sh.groups);
        const int64_t u0 = group < active ? first_unit(total, active, group) : 0;
        int64_t left = (group < active ? first_unit(total, active, group + 1) : 0) - u0, off = 0, base = 0;
        int b = 0;
        Seq s{};
        for (int b0 = 0; b0 < sh.B && left > 0; b0 += 32) {
            if (b0 > 0) {
                ls = b0 + lane < sh.B ? seq_of(a, sh, b0 + lane) : Seq{};
                ln = units_of(ls, sh.Hkv);
            }
            int64_t incl = ln;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += y;
            }
            const uint32_t m = __ballot_sync(0xffffffffu, u0 >= base + incl - ln && u0 < base + incl);
            if (m) {
                const int src = __ffs(m) - 1;
                b = b0 + src;
                off = u0 - __shfl_sync(0xffffffffu, base + incl - ln, src);
                s.L = __shfl_sync(0xffffffffu, ls.L, src);
                s.nodes = __shfl_sync(0xffffffffu, ls.nodes, src);
                s.tiles = __shfl_sync(0xffffffffu, ls.tiles, src);
                s.groups = __shfl_sync(0xffffffffu, ls.groups, src);
                break;
            }
            base += __shfl_sync(0xffffffffu, incl, 31);
        }
        for (int n = 0; ok; ++n) {
            Segment g{};
            while (left > 0) {
                if (off >= units_of(s, sh.Hkv)) {
                    off = 0;
                    s = seq_of(a, sh, ++b);
                    continue;
                }
                const int per = item_units(s);
                const int item = (int)(off >> 31 ? off / per : (uint32_t)off / (uint32_t)per);
                const int v0 = (int)(off - (int64_t)item * per), nv = (int)min((int64_t)(per - v0), left);
                off += nv;
                left -= nv;
                g.b = b;
                g.h = item / s.groups;
                g.L = (int)s.L;
                g.nodes = s.nodes;
                g.row0 = (item % s.groups * sh.R + member) * kBM;
                g.rows = min(kBM, s.nodes * sh.G - g.row0);
                g.tiles = s.tiles;
                // A row sees its committed tokens, and in a chain the nodes up to its own.
                g.fine = a.out_f32 || (a.mask ? s.L : s.L + g.row0 / sh.G + 1) <= kShort;
                g.tile0 = min(v0, s.tiles);
                g.ntile = min(v0 + nv, s.tiles) - g.tile0;
                if (g.ntile == 0) g.rows = 0;  // nothing but the item's cost
                if (g.rows > 0) break;
                g.rows = 0;  // this CTA's row tile does not exist in this item
            }
            if (g.rows > 0) {
                const int i0 = g.row0 / sh.G, i1 = (g.row0 + g.rows - 1) / sh.G;
                if (a.positions) {
                    int lo = INT32_MAX, hi = INT32_MIN, kl = INT32_MAX;
                    for (int i = lane; i < g.nodes; i += 32) {
                        const int p = a.positions[(size_t)b * a.T + i];
                        kl = min(kl, p);
                        if (i >= i0 && i <= i1) lo = min(lo, p), hi = max(hi, p);
                    }
                    g.pmin = __reduce_min_sync(0xffffffffu, lo);
                    g.pmax = __reduce_max_sync(0xffffffffu, hi);
                    g.kmin = __reduce_min_sync(0xffffffffu, kl);
                } else {
                    g.pmin = g.L + i0, g.pmax = g.L + i1, g.kmin = g.L;
                }
            }
            if (!(ok = wait(&ctl->seg_empty[n % kRing], ((n / kRing) & 1) ^ 1, wc, 60))) break;
            if (lane == 0) {
                ctl->seg[n % kRing] = g;
                mbar_arrive(&ctl->seg_full[n % kRing]);
            }
            __syncwarp();
            if (g.rows == 0) break;
        }
    } else if (warp == kProducer || warp == kVProducer) {
        // ------------------------------------------- producers of K and of V
        const bool v = warp == kVProducer;
        uint64_t *full = v ? ctl->v_full : ctl->k_full, *empty = v ? ctl->v_empty : ctl->k_empty;
        const int u = lane >> 1, hf = lane & 1;  // lane = (K-step or dim group, half of the tile)
        const uint32_t P = (uint32_t)a.pk.page_size;
        const int w0 = w[lane], w1 = H > 32 ? w[lane + 32] : INT32_MAX;
        while (ok && runs.next(wc, ok)) {
            const Segment g = runs.now();
            runs.done(lane);
            const int64_t end = (int64_t)g.L + g.nodes;
            int r_lo = H, r_full = H;
            int page = -1;  // page of half-tile 2 * (j & ~15) + lane
            for (int j = g.tile0; ok && j < g.tile0 + g.ntile; ++j, ++it) {
                const int st = it % ST;
                const int64_t m0 = (int64_t)j * kBN;
                if (j == g.tile0 || (j & 15) == 0) {
                    const int64_t slot = ((int64_t)(j & ~15) * 2 + lane) * 64;
                    page = slot + 64 > (int64_t)g.tile0 * kBN && slot < end ? page_of(a.pk, g.b, slot, a.status) : -1;
                }
                const int pg = __shfl_sync(0xffffffffu, page, (j & 15) * 2 + (box_keys == kBN ? 0 : hf));
                const int halves = box_keys == kBN || m0 + 64 < end ? 2 : 1;
                const bool issue = hf < (box_keys == kBN ? 1 : halves);
                const int at = (int)(((uint32_t)m0 + 64u * hf) % P);
                if (!v) {
                    // The tile's band; a tile with nodes may hold any small distance.
                    const bool prefix = m0 + kBN <= g.L;
                    r_lo = prefix ? first_kept(w0, w1, g.pmin - (m0 + kBN - 1)) : 0;
                    r_full = first_kept(w0, w1, g.pmax - (prefix || (m0 < g.L && m0 < g.kmin) ? m0 : (int64_t)g.kmin));
                }
                const int ca = v || !kPacked ? 0 : r_lo >> 3;
                const uint32_t bytes = (v || !kPacked ? (uint32_t)(D / 64) * 8192u : (uint32_t)(C - ca) * 2048u) * halves;
                uint8_t *dst = (v ? sV : sK) + st * F::TileBytes + (kPacked && !v ? u * 4096 + hf * 2048 : u * 16384 + hf * 8192);
                const bool mine = issue && (kPacked && !v ? u >= ca && u < C : u < D / 64);
                const int z = (pg * sh.Hkv + g.h) * C + u;
                // (Entry it % 8 is free: the wait for tile it - 1 has shown the PV of it - 8.)
                if (!v && lane == 0) ctl->band[it % 8] = make_band<D, kPacked>(r_lo, r_full, g.pmin != g.pmax);
                if (!(ok = wait(&empty[st], ((it / ST) & 1) ^ 1, wc, v ? 42 : 41))) break;
                if (lane == 0) {
                    if (v && m0 + kBN > g.L) mbar_arrive(&ctl->v_tail[st]);  // a tile with nodes is on its way
                    mbar_expect_tx(&full[st], bytes);
                }
                __syncwarp();
                if (mine) {
                    if (kPacked && !v) tma_load_3d(dst, &tm_k, &full[st], 0, at, z);
                    else tma_load_4d(dst, v ? &tm_v : &tm_k, &full[st], 64 * u, g.h, at, pg);
                }
            }
        }
        // Let every copy land before the CTA exits: the tiles before `it` are issued.  Also after the
        // last run: another warp's wait may run out before anyone has waited for this warp's last tiles.
        for (int x = it > ST ? it - ST : 0; x < it; ++x)
            wait_drain(&full[x % ST], (x / ST) & 1, atflash_drain_limit_ns(a.limit_ns));
    } else if (warp == kFix) {
        // ------------------------------------------------ boundary pairs of K
        while (ok && runs.next(wc, ok)) {
            const Segment g = runs.now();
            runs.done(lane);
            const int64_t end = (int64_t)g.L + g.nodes;
            for (int j = g.tile0; ok && j < g.tile0 + g.ntile; ++j, ++it) {
                const int st = it % ST, cb = it % F::Cells;
                const int64_t m0 = (int64_t)j * kBN;
                if (!(ok = wait(&ctl->k_full[st], (it / ST) & 1, wc, 43))) break;
                const int4 bd = ctl->band[it % 8];
                uint8_t *kst = sK + st * F::TileBytes;
                // Pairs below rs that share its K-step are pruned for every cell: zeroed whole.
                const int z = bd.y % kPer;
                if (z) {
                    const int c = bd.y / kPer;
#pragma unroll 1
                    for (int e = 0; e < kBN; e += 32) {
                        if constexpr (kPacked) zero_words(kst + c * 4096 + sw32_off(lane + e, 0), kst + c * 4096 + sw32_off(lane + e, 4), z);
                        else {
                            for (int half = 0; half < 2; ++half) {
                                const int d = 16 * c + half * H;
                                uint8_t *u0 = kst + sw128_off(lane + e, d), *u1 = kst + sw128_off(lane + e, d + 8);
                                zero_words(u0, u1, z / 2);
                                if (z & 1) *reinterpret_cast<uint16_t *>((z < 8 ? u0 : u1) + (z & 6) * 2) = 0;
                            }
                        }
                    }
                }
                if (!(bd.w & kBandFix)) {
                    if (z) fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&ctl->k_ready[st]);
                    continue;
                }
                constexpr int kK = kBN / 32;  // this lane's keys: lane, lane + 32, ..
                const bool prefix = m0 + kBN <= g.L;
                int kp[kK];
#pragma unroll
                for (int e = 0; e < kK; ++e) {
                    const int64_t slot = m0 + lane + 32 * e;
                    kp[e] = slot < g.L || slot >= end ? (int)slot : node_pos(a, g.b, g.L, (int)(slot - g.L));
                    if (bd.w & kBandCells) sKpos[cb * kBN + lane + 32 * e] = kp[e];
                }
                uint32_t chunks = prefix ? 0u : 0xfu;  // 32-key chunks in which some cell is added
                // Addresses of this lane's first key; its others are 32 rows further each.
                const uint8_t *row0 = kst + (kPacked ? lane * 32 : lane * 128);
                const uint32_t swz = kPacked ? (lane & 4) << 2 : (lane & 7) << 4;
                for (int r = bd.y; r < bd.z; ++r) {
                    // Keys at positions >= all are kept by every row, below none by no row.
                    const int64_t all = (int64_t)g.pmax - w[r], none = (int64_t)g.pmin - w[r];
                    uint32_t *stage = sStage + (cb * kStaged + r - bd.y) * kBN + lane;
                    uint8_t *x0, *x1 = nullptr;
                    if (kPacked) {
                        x0 = const_cast<uint8_t *>(row0) + (r >> 3) * 4096 + (((r & 7) * 4) ^ swz);
                    } else {
                        x0 = const_cast<uint8_t *>(row0) + (r >> 6) * 16384 + ((((r & 63) >> 3) << 4) ^ swz) + (r & 7) * 2;
                        x1 = const_cast<uint8_t *>(row0) + ((r + H) >> 6) * 16384 + (((((r + H) & 63) >> 3) << 4) ^ swz) + (r & 7) * 2;
                    }
#pragma unroll
                    for (int e = 0; e < kK; ++e) {
                        if (kp[e] >= all) continue;
                        if (kPacked) {
                            uint32_t *x = reinterpret_cast<uint32_t *>(x0 + e * 1024);
                            if (kp[e] >= none) stage[32 * e] = *x;
                            *x = 0;
                        } else {
                            uint16_t *lo = reinterpret_cast<uint16_t *>(x0 + e * 4096), *hi = reinterpret_cast<uint16_t *>(x1 + e * 4096);
                            if (kp[e] >= none) stage[32 * e] = *lo | (uint32_t)*hi << 16;
                            *lo = 0;
                            *hi = 0;
                        }
                    }
                    if (none < all) {
                        // Staged keys lie in [z0, z1) of a prefix tile, anywhere in one with nodes.
                        const int z0 = prefix ? (int)min(max(none - m0, (int64_t)0), (int64_t)kBN) : 0;
                        const int z1 = prefix ? (int)min(max(all - m0, (int64_t)0), (int64_t)kBN) : kBN;
                        if (lane == 0) ctl->zone[cb][r - bd.y] = (uint32_t)z0 | (uint32_t)z1 << 16;
                        if (z0 < z1) chunks |= (2u << (z1 - 1) / 32) - (1u << z0 / 32);
                    }
                }
                if (lane == 0) ctl->chunks[cb] = bd.x < bd.y ? 0xfu : chunks;
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->k_ready[st]);
            }
        }
    } else if (warp >= kTail) {
        // ---------------- tiles with nodes: mask bits, V behind the last node
        const int t2 = warp - kTail;
        uint32_t used = 0, tails = 0;  // phase bits of each set's mask buffer, of v_tail per stage
        while (ok && runs.next(wc, ok)) {
            const Segment g = runs.now();
            runs.done(lane);
            const int seg = runs.n - 1;
            const int64_t end = (int64_t)g.L + g.nodes;
            const int i0 = g.row0 / sh.G, i1 = (g.row0 + g.rows - 1) / sh.G;
            for (int j = g.tile0; ok && j < g.tile0 + g.ntile; ++j, ++it) {
                const int st = it % ST, set = it & 1;
                const int64_t m0 = (int64_t)j * kBN;
                if (m0 + kBN <= g.L) continue;
                // One mask buffer per set.
                if (!(ok = wait(&ctl->m_empty[set], ((used >> set) & 1) ^ 1, wc, 44))) break;
                used ^= 1u << set;
                for (int i = i0 + t2; i <= i1; i += 4) {
                    uint32_t x[8];
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const int i2 = i + 2 * (e >> 2);
                        const int64_t slot = m0 + 32 * (e & 3) + lane;
                        const bool sees = i2 <= i1 && slot < end && (slot < g.L || node_sees(a, g.b, i2, (int)(slot - g.L)));
                        x[e] = __ballot_sync(0xffffffffu, sees);
                    }
                    if (lane == 0) {
                        sMask[set * kBM + i - i0] = make_uint4(x[0], x[1], x[2], x[3]);
                        if (i + 2 <= i1) sMask[set * kBM + i + 2 - i0] = make_uint4(x[4], x[5], x[6], x[7]);
                    }
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->m_full[set]);
                // V behind the last node may hold anything (0 * NaN must not reach O), and so may
                // a node that some rows do not see: its non-finite values are taken out here and
                // put back, for the rows that see them, at the end of the run.
                // These warps skip the tiles before, so they may look at v_full only once its phase can
                // be this tile's: the V producer says when.
                if (!(ok = wait(&ctl->v_tail[st], (tails >> st) & 1, wc, 66))) break;
                tails ^= 1u << st;
                if (!(ok = wait(&ctl->v_full[st], (it / ST) & 1, wc, 45))) break;
                uint8_t *vst = sV + st * F::TileBytes;
                constexpr int kUnits = D / 8;  // 16-byte units of a row
                bool bad = false;
                const int first = (int)max(g.L - m0, (int64_t)0);
                for (int e = first * kUnits + t2 * 32 + lane; e < kBN * kUnits; e += 64) {
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
    } else if (warp == kQk) {
        // ------------------------------------------------------- QK issuer
        const uint32_t idesc = idesc_bf16_f32(kBM, kBN, false, false);
        const uint32_t sQa = smem_u32(sQ), sKa = smem_u32(sK);
        while (ok && runs.next(wc, ok)) {
            const int ntile = runs.now().ntile;
            runs.done(lane);
            if (!(ok = wait(&ctl->q_ready, (runs.n - 1) & 1, wc, 46))) break;
            for (int j = 0; ok && j < ntile; ++j, ++it) {
                const int st = it % ST, buf = it % kBufs;
                if (!(ok = wait(&ctl->k_ready[st], (it / ST) & 1, wc, 48))) break;
                const int4 bd = ctl->band[it % 8];
                if (it >= kBufs && !(ok = wait(&ctl->o_done[buf], (it / kBufs - 1) & 1, wc, 49))) break;
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t k0 = sKa + st * F::TileBytes, d = tmem + buf * kBN;
                    uint32_t acc = 0;
#pragma unroll 1  // (a short loop: see the head of this file)
                    for (int c = bd.y / kPer; c < H / kPer; ++c) {
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
                    mbar_arrive(&ctl->s_full[buf]);
                    // Where the softmax warps do not read the stage, their arrivals are made here.
                    if (!(bd.w & kBandHold)) mbar_arrive_n(&ctl->k_empty[st], 4);
                }
                __syncwarp();
            }
        }
    } else if (warp == kPv) {
        // ------------------------------------------------------- PV issuer
        const uint32_t idesc = idesc_bf16_f32(kBM, D, false, true);
        const uint32_t sVa = smem_u32(sV);
        uint32_t tails = 0;  // phase bit of v_ready per stage
        while (ok && runs.next(wc, ok)) {
            const int L = runs.now().L, tile0 = runs.now().tile0, ntile = runs.now().ntile, fine = runs.now().fine;
            runs.done(lane);
            for (int j = tile0; ok && j < tile0 + ntile; ++j, ++it) {
                const int st = it % ST, buf = it % kBufs;
                if (!(ok = wait(&ctl->v_full[st], (it / ST) & 1, wc, 50))) break;
                if ((int64_t)(j + 1) * kBN > L) {
                    if (!(ok = wait(&ctl->v_ready[st], (tails >> st) & 1, wc, 51))) break;
                    tails ^= 1u << st;
                }
                if (!(ok = wait(&ctl->p_full[buf], (it / kBufs) & 1, wc, 52))) break;
                if (lane == 0) {
                    tc_fence_after();
                    const uint32_t o = tmem + F::TmemO, p = tmem + buf * kBN;
                    if (fine) {
#pragma unroll 1
                        for (int kk = 0; kk < kBN / 16; ++kk) {
                            const uint64_t db = smem_desc(sVa + st * F::TileBytes + kk * 2048, 16384, 1024, kSwizzle128B);
                            umma_bf16_ts(o, p + kk * 16, db, idesc, (j > tile0 || kk > 0) ? 1u : 0u);
                            umma_bf16_ts(o, p + kk * 16 + 8, db, idesc, 1u);
                        }
                    } else {
#pragma unroll 1
                        for (int kk = 0; kk < kBN / 16; ++kk) {
                            const uint64_t db = smem_desc(sVa + st * F::TileBytes + kk * 2048, 16384, 1024, kSwizzle128B);
                            umma_bf16_ts(o, p + kk * 8, db, idesc, (j > tile0 || kk > 0) ? 1u : 0u);
                        }
                    }
                    umma_commit(&ctl->o_done[buf]);
                    umma_commit(&ctl->v_empty[st]);
                }
                __syncwarp();
            }
        }
    } else if (warp < kSoft) {
        // ------------------------------------------------------------- softmax
        setmaxnreg_inc<kSoftRegs>();
        const int set = warp >> 2, q4 = warp & 3;
        const int copy = q4 * 32 / kRows;                // which copy of the rows, hence which columns
        const int c0 = copy * NC;
        const int row = (q4 * 32) % kRows + lane;        // row of the tile
        const uint32_t lane_off = (uint32_t)(q4 * 32) << 16;
        const uint32_t tO = tmem + F::TmemO + lane_off;
        const float scale_log2 = 1.4426950408889634f * rsqrtf((float)D);
        int syncs = 0, tails = 0;
        // All softmax warps (bounded, unlike a named barrier).
        auto soft_sync = [&]() -> bool {
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->soft_bar);
            return wait(&ctl->soft_bar, syncs++ & 1, wc, 53);
        };
        while (ok && runs.next(wc, ok)) {
            const Segment &g = runs.now();
            const int rows = g.rows, row0 = g.row0, b = g.b, L = g.L, tile0 = g.tile0, ntile = g.ntile, fine = g.fine;
            const bool live = (q4 * 32) % kRows < rows;  // some row of this warp exists
            const bool valid = row < rows;
            const int tok = (row0 + (valid ? row : 0)) / sh.G;
            {
                // Rotate the queries into the MMA's layout as hi + lo bf16, four pairs of a row per
                // thread.  A run's first instructions come from L2 a line at a time, so this is a short
                // loop rather than an unrolled one.
                constexpr int kQuads = H / 4, kStep = 32 * kSoft / kQuads;  // threads per row, rows at a time
                const int pr = threadIdx.x % kQuads * 4;
                const __nv_bfloat16 *q = static_cast<const __nv_bfloat16 *>(a.q) + b * a.qs.batch + (int64_t)g.h * sh.G * a.qs.head + pr;
                const ulonglong2 tu01 = *reinterpret_cast<const ulonglong2 *>(&ctl->turn[pr]);
                const ulonglong2 tu23 = *reinterpret_cast<const ulonglong2 *>(&ctl->turn[pr + 2]);
                const uint64_t turn[4] = {tu01.x, tu01.y, tu23.x, tu23.y};
                uint2 xa, xb;
                int ps = 0;
                auto fetch = [&](int r) {
                    if (r >= rows) return;
                    const int t = (row0 + r) / sh.G, hh = (row0 + r) - t * sh.G;
                    const __nv_bfloat16 *src = q + t * a.qs.token + hh * a.qs.head;
                    xa = *reinterpret_cast<const uint2 *>(src);
                    xb = *reinterpret_cast<const uint2 *>(src + H);
                    ps = node_pos(a, b, L, t);
                };
                int r = threadIdx.x / kQuads;
                fetch(r);
#pragma unroll 1
                for (; r < rows; r += kStep) {
                    const uint2 ya = xa, yb = xb;
                    const int pos = ps;
                    fetch(r + kStep);  // under this row's arithmetic
                    uint32_t hi[4], lo[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t wa = i < 2 ? ya.x : ya.y, wb = i < 2 ? yb.x : yb.y;
                        const float fa = i & 1 ? bf16hi(wa) : bf16lo(wa), fb = i & 1 ? bf16hi(wb) : bf16lo(wb);
                        // (Within 2^-20 (|fa| + |fb|), far below the 2^-16 of hi + lo.)
                        const float2 cs = turn_cos_sin_fast(pos, turn[i]);
                        const float x = fa * cs.x - fb * cs.y, y = fb * cs.x + fa * cs.y;
                        hi[i] = pack_bf16x2(x, y);
                        lo[i] = pack_bf16x2(x - bf16lo(hi[i]), y - bf16hi(hi[i]));
                    }
#pragma unroll
                    for (int cp = 0; cp < kRep; ++cp) {
                        store_quad<D, kPacked>(sQ, cp * kRows + r, pr, hi);
                        store_quad<D, kPacked>(sQ + F::TileBytes, cp * kRows + r, pr, lo);
                    }
                }
                fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&ctl->q_ready);
            const int pos = valid ? node_pos(a, b, L, tok) : 0;
            if (!(ok = wait(&ctl->q_ready, (runs.n - 1) & 1, wc, 54))) break;  // the other warps' pairs, for the boundary

            float m_used = -INFINITY, lrun = 0.f;  // this set's sum, scaled by its latest running max
            const int pmax = g.pmax;
            const int j0 = tile0 + ((it ^ set) & 1);  // this set's tiles
            for (int j = j0; j < tile0 + ntile; j += 2) {
                const int x = it + (j - tile0), st = x % ST, buf = x % kBufs, cb = x % F::Cells;
                const uint32_t tS = tmem + buf * kBN + lane_off;  // S, and P over it
                const bool tail = (int64_t)(j + 1) * kBN > L;
                if (!(ok = wait(&ctl->s_full[buf], (x / kBufs) & 1, wc, 56))) break;
                tc_fence_after();
                const int4 bd = ctl->band[x % 8];
                const bool cells = bd.w & kBandCells;
                const bool dense = bd.y < H;  // S holds something (always where cells are added or hidden: see make_band)
                if (tail) {
                    if (!(ok = wait(&ctl->m_full[set], tails & 1, wc, 58))) break;
                    ++tails;
                }
                if (cells || tail) {
                    // Cells added or hidden, in S itself, 32 columns at a time.
                    const uint32_t chunks = (cells ? ctl->chunks[cb] : 0u) | (tail ? 0xfu : 0u);
#pragma unroll 1
                    for (int cc = c0; live && cc < c0 + NC; cc += 32) {
                        if (!((chunks >> (cc / 32)) & 1u)) continue;
                        uint32_t ra[32];
                        float s[32];
                        __syncwarp();
                        tmem_ld_32x32b_x32(tS + cc, ra);
                        tmem_ld_wait(ra);
#pragma unroll
                        for (int i = 0; i < 32; ++i) s[i] = __uint_as_float(ra[i]);
                        if (cells) {
                            const int4 *kp = reinterpret_cast<const int4 *>(sKpos + cb * kBN + cc);
#pragma unroll 1
                            for (int r = bd.x; r < bd.z; ++r) {
                                if (r >= bd.y && !tail) {
                                    const uint32_t z = ctl->zone[cb][r - bd.y];
                                    if ((int)(z >> 16) <= cc || (int)(z & 0xffff) >= cc + 32) continue;
                                }
                                const uint32_t qh = load_pair<D, kPacked>(sQ, copy * kRows + row, r);
                                const uint32_t ql = load_pair<D, kPacked>(sQ + F::TileBytes, copy * kRows + row, r);
                                const float qa = bf16lo(qh) + bf16lo(ql), qb = bf16hi(qh) + bf16hi(ql);
                                // This row keeps keys at positions >= lim; of a staged pair the MMA has
                                // those at lim + span and beyond (differences modulo 2^32 are exact here,
                                // and taken in unsigned arithmetic: they pass 31 bits).
                                const int lim = pos - w[r];
                                if (r >= bd.y) {
                                    const uint32_t span = (uint32_t)(pmax - pos), low = (uint32_t)lim;
                                    const uint4 *kw = reinterpret_cast<const uint4 *>(sStage + (cb * kStaged + r - bd.y) * kBN + cc);
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        const uint4 k = kw[i];
                                        const int4 p = kp[i];
                                        s[4 * i] += (uint32_t)p.x - low < span ? fmaf(qa, bf16lo(k.x), qb * bf16hi(k.x)) : 0.f;
                                        s[4 * i + 1] += (uint32_t)p.y - low < span ? fmaf(qa, bf16lo(k.y), qb * bf16hi(k.y)) : 0.f;
                                        s[4 * i + 2] += (uint32_t)p.z - low < span ? fmaf(qa, bf16lo(k.z), qb * bf16hi(k.z)) : 0.f;
                                        s[4 * i + 3] += (uint32_t)p.w - low < span ? fmaf(qa, bf16lo(k.w), qb * bf16hi(k.w)) : 0.f;
                                    }
                                } else {
                                    const uint8_t *kst = sK + st * F::TileBytes;
#pragma unroll
                                    for (int i = 0; i < 32; ++i) {
                                        const uint32_t k = load_pair<D, kPacked>(kst, cc + i, r);
                                        s[i] += sKpos[cb * kBN + cc + i] >= lim ? fmaf(qa, bf16lo(k), qb * bf16hi(k)) : 0.f;
                                    }
                                }
                            }
                        }
                        if (tail) {
                            const uint32_t see = reinterpret_cast<const uint32_t *>(sMask + set * kBM + (tok - row0 / sh.G))[cc / 32];
#pragma unroll
                            for (int i = 0; i < 32; ++i)
                                if (!((see >> i) & 1u)) s[i] = -INFINITY;
                        }
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 32; ++i) ra[i] = __float_as_uint(s[i]);
                        tmem_st_32x32b_x32(tS + cc, ra);
                    }
                    tmem_st_wait();
                    __syncwarp();
                    if ((bd.w & kBandHold) && lane == 0) mbar_arrive(&ctl->k_empty[st]);
                    if (tail && lane == 0) mbar_arrive(&ctl->m_empty[set]);
                }
                // The row's maximum, then the exponentials, CW columns at a time.  More columns are read
                // twice, by loops: their unrolled code would not stay in the instruction cache (on 2
                // sequences of 128K keys with trees of 64 nodes: 128 columns unrolled 498 us, 64 at a time 439, 32 384;
                // later 16 took 354 and 32 343).
                float s[CW], row_max = -INFINITY;
                auto load = [&](int c) {
                    if (dense) {
                        uint32_t ra[CW];
                        tmem_ld_32x32b_x32(tS + c, ra);
                        tmem_ld_wait(ra);
#pragma unroll
                        for (int i = 0; i < CW; ++i) s[i] = __uint_as_float(ra[i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < CW; ++i) s[i] = 0.f;
                    }
                };
#pragma unroll 1
                for (int c = c0; c < c0 + NC; c += CW) {
                    load(c);
                    float mx0 = -INFINITY, mx1 = -INFINITY, mx2 = -INFINITY;
#pragma unroll
                    for (int i = 0; i < CW; i += 8) {
                        row_max = max3(row_max, s[i], s[i + 1]);
                        mx0 = max3(mx0, s[i + 2], s[i + 3]);
                        mx1 = max3(mx1, s[i + 4], s[i + 5]);
                        mx2 = max3(mx2, s[i + 6], s[i + 7]);
                    }
                    row_max = fmaxf(fmaxf(row_max, mx0), fmaxf(mx1, mx2));
                }
                const float tile_max = row_max * scale_log2;
                // The running max after the previous tile, from the row's warp of the other set.  It is
                // kept unless it grew by more than 2^8: O / l uses the same one, so the result does not
                // depend on it.
                float m_prev = -INFINITY;
                if (j > tile0) {
                    if (!(ok = wait(&ctl->max_bar[set ^ 1][q4], ((x - 1) >> 1) & 1, wc, 63))) break;
                    m_prev = ctl->run_max[set ^ 1][q4 * 32 + lane];
                }
                const bool need = tile_max > m_prev + kRescaleThreshold;
                const float m_new = need ? tile_max : m_prev;
                ctl->run_max[set][q4 * 32 + lane] = m_new;
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->max_bar[set][q4]);
                if (m_new != m_used) lrun *= fast_exp2(m_used - m_new);
                m_used = m_new;
                const float mr = m_new == -INFINITY ? 0.f : m_new;  // nothing seen so far
                const float2 mneg = make_float2(-mr, -mr), sc2 = make_float2(scale_log2, scale_log2);
                float2 l0 = make_float2(0.f, 0.f), l1 = make_float2(0.f, 0.f);
                const auto weigh = [&](auto parts) {
                    constexpr bool kFine = decltype(parts)::value;
#pragma unroll 1
                    for (int c = c0; c < c0 + NC; c += CW) {
                        if (NC > CW) load(c);
                        uint32_t pk[kFine ? CW : CW / 2];  // two parts: of each 16 keys 8 high words, then 8 low ones
#pragma unroll
                        for (int i = 0; i < CW / 2; i += 2) {
                            float2 xa = fma2(make_float2(s[2 * i], s[2 * i + 1]), sc2, mneg);
                            float2 xb = fma2(make_float2(s[2 * i + 2], s[2 * i + 3]), sc2, mneg);
                            xa.x = fast_exp2(xa.x);
                            xa.y = fast_exp2(xa.y);
                            xb.x = fast_exp2(xb.x);
                            xb.y = fast_exp2(xb.y);
                            l0 = add2(l0, xa);
                            l1 = add2(l1, xb);
                            uint32_t *p = pk + (kFine ? i / 8 * 16 + i % 8 : i);
                            p[0] = pack_bf16x2(xa.x, xa.y);
                            p[1] = pack_bf16x2(xb.x, xb.y);
                            if constexpr (kFine) {
                                const float2 minus = make_float2(-1.f, -1.f);
                                xa = fma2(make_float2(bf16lo(p[0]), bf16hi(p[0])), minus, xa);
                                xb = fma2(make_float2(bf16lo(p[1]), bf16hi(p[1])), minus, xb);
                                p[8] = pack_bf16x2(xa.x, xa.y);
                                p[9] = pack_bf16x2(xb.x, xb.y);
                            }
                        }
                        if constexpr (kFine) tmem_st_32x32b_x32(tS + c, pk);
                        else tmem_st_x16(tS + c / 2, pk);
                    }
                    if (kRep > 1) {
                        // P is zero in the other copies' columns.
                        constexpr int kW = kFine ? 32 : 16;  // columns of 32 keys
                        uint32_t zero[kW];
#pragma unroll
                        for (int i = 0; i < kW; ++i) zero[i] = 0;
#pragma unroll 1
                        for (int c = 0; c < kBN / 32; ++c) {
                            if (c / (NC / 32) == copy) continue;
                            if constexpr (kFine) tmem_st_32x32b_x32(tS + c * kW, zero);
                            else tmem_st_x16(tS + c * kW, zero);
                        }
                    }
                };
                if (live) {
                    if (fine) weigh(std::true_type{});
                    else weigh(std::false_type{});
                    const float2 ls = add2(l0, l1);
                    lrun += ls.x + ls.y;
                }
                if (j > tile0 && __any_sync(0xffffffffu, need)) {
                    // O may be rescaled once the previous tile's PV is done.
                    if (!(ok = wait(&ctl->o_done[(x - 1) % kBufs], ((x - 1) / kBufs) & 1, wc, 64))) break;
                    tc_fence_after();
                    const float alpha = need ? fast_exp2(m_prev - m_new) : 1.f;
#pragma unroll 1
                    for (int cc = 0; cc < D; cc += 32) {
                        uint32_t r[32];
                        tmem_ld_32x32b_x32(tO + cc, r);
                        tmem_ld_wait(r);
#pragma unroll
                        for (int i = 0; i < 32; ++i) r[i] = __float_as_uint(__uint_as_float(r[i]) * alpha);
                        tmem_st_32x32b_x32(tO + cc, r);
                    }
                }
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ctl->p_full[buf]);
            }
            if (!ok) break;
            it += ntile;
            // ---- end of the run: the sets' sums and the copies' states of each row joined
            const int lastx = it - 1 - ((it - 1 - set) & 1);  // this set's last tile
            if (j0 < tile0 + ntile && !(ok = wait(&ctl->o_done[lastx % kBufs], (lastx / kBufs) & 1, wc, 62))) break;
            ctl->stat[set][q4 * 32 + lane] = make_float2(m_used, lrun);
            if (!(ok = soft_sync())) break;  // both sets' sums, and O
            tc_fence_after();
            // O of a copy is scaled by the running max after the run's last tile; a set's sum by that
            // after its own.
            const int lset = (it - 1) & 1;
            float M = -INFINITY, sum = 0.f, f = 1.f;
#pragma unroll
            for (int cp = 0; cp < kRep; ++cp) M = fmaxf(M, ctl->stat[lset][cp * kRows + row].x);
            const float Mr = M == -INFINITY ? 0.f : M;
#pragma unroll
            for (int cp = 0; cp < kRep; ++cp) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    const float2 y = ctl->stat[i][cp * kRows + row];
                    sum += y.y == 0.f ? 0.f : y.y * fast_exp2(y.x - Mr);
                }
                if (cp == copy) f = fast_exp2(ctl->stat[lset][cp * kRows + row].x - Mr);
            }
            const bool whole = g.ntile == g.tiles;
            const bool odd = ctl->nf_seg[(runs.n - 1) & 7] == runs.n - 1;
            const float inv = whole ? (sum == 0.f ? 0.f : 1.f / sum) : 1.f;
            float *part = a.workspace + ((size_t)blockIdx.x * 2 + (tile0 > 0 ? 0 : 1)) * kBM * (D + 2);
            const size_t obase = (size_t)b * a.T;
            if (valid && set == 0 && copy == 0) {
                if (!whole) {
                    part[row] = M;
                    part[kBM + row] = sum;
                } else if (a.lse) {
                    const int hq = g.h * sh.G + (row0 + row) % sh.G;
                    a.lse[((size_t)b * a.Hq + hq) * a.T + tok] = sum == 0.f ? -INFINITY : (M + log2f(sum)) * 0.69314718055994531f;
                }
            }
            // This warp takes half of the dims (by its set) of its lanes' O.
            constexpr int kO = D / 2;
            float *sX = reinterpret_cast<float *>(sQ);  // exchange of repeated rows: every QK of the run is done
#pragma unroll 1
            for (int cc = 0; cc < kO; cc += 32) {
                const int d0 = set * kO + cc;
                uint32_t ra[32];
                __syncwarp();
                tmem_ld_32x32b_x32(tO + d0, ra);
                tmem_ld_wait(ra);
                float o[32];
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = kRep > 1 ? __uint_as_float(ra[i]) * f : __uint_as_float(ra[i]);
                if (odd && valid && copy == 0) {
                    float t[32];  // (in local memory, only here)
#pragma unroll
                    for (int i = 0; i < 32; ++i) t[i] = o[i];
                    add_nonfinite<32>(a, g, D, tok, d0, t);
#pragma unroll
                    for (int i = 0; i < 32; ++i) o[i] = t[i];
                }
                if (kRep > 1) {
                    // Rows of float4 units, the unit index swizzled by the row against bank conflicts.
#pragma unroll
                    for (int i = 0; i < 32 / 4; ++i) {
                        const int unit = (d0 / 4 + i) ^ (lane & 7);
                        *reinterpret_cast<float4 *>(sX + (q4 * 32 + lane) * D + unit * 4) = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    }
                } else if (valid) {
                    if (!whole) {
                        float4 *dst = reinterpret_cast<float4 *>(part + 2 * kBM + (size_t)row * D + d0);
#pragma unroll
                        for (int i = 0; i < 32 / 4; ++i) dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
                    } else {
                        const size_t orow = (obase + tok) * a.Hq + g.h * sh.G + (row0 + row) % sh.G;
                        if (a.out_f32) {
                            float4 *dst = reinterpret_cast<float4 *>(static_cast<float *>(a.out) + orow * D + d0);
#pragma unroll
                            for (int i = 0; i < 32 / 4; ++i)
                                dst[i] = make_float4(o[4 * i] * inv, o[4 * i + 1] * inv, o[4 * i + 2] * inv, o[4 * i + 3] * inv);
                        } else {
                            uint4 *dst = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(a.out) + orow * D + d0);
#pragma unroll
                            for (int i = 0; i < 32 / 8; ++i)
                                dst[i] = make_uint4(pack_bf16x2(o[8 * i] * inv, o[8 * i + 1] * inv), pack_bf16x2(o[8 * i + 2] * inv, o[8 * i + 3] * inv),
                                                    pack_bf16x2(o[8 * i + 4] * inv, o[8 * i + 5] * inv), pack_bf16x2(o[8 * i + 6] * inv, o[8 * i + 7] * inv));
                        }
                    }
                }
            }
            if (kRep > 1) {
                if (set == 0 && copy == 0) ctl->run_max[0][row] = inv;  // for the threads that write the row
                if (!(ok = soft_sync())) break;
                // Copies summed, a float4 unit at a time, neighbouring threads on neighbouring units.
                for (int e = threadIdx.x; e < rows * (D / 4); e += 32 * kSoft) {
                    const int r = e / (D / 4), u = e % (D / 4);
                    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                    for (int cp = 0; cp < kRep; ++cp) {
                        const float4 x = *reinterpret_cast<const float4 *>(sX + (cp * kRows + r) * D + (u ^ (r & 7)) * 4);
                        o.x += x.x, o.y += x.y, o.z += x.z, o.w += x.w;
                    }
                    if (!whole) {
                        *reinterpret_cast<float4 *>(part + 2 * kBM + (size_t)r * D + 4 * u) = o;
                        continue;
                    }
                    const float iv = ctl->run_max[0][r];
                    const size_t off = ((obase + (row0 + r) / sh.G) * a.Hq + g.h * sh.G + (row0 + r) % sh.G) * D + 4 * u;
                    if (a.out_f32) *reinterpret_cast<float4 *>(static_cast<float *>(a.out) + off) = make_float4(o.x * iv, o.y * iv, o.z * iv, o.w * iv);
                    else
                        *reinterpret_cast<uint2 *>(static_cast<__nv_bfloat16 *>(a.out) + off) =
                            make_uint2(pack_bf16x2(o.x * iv, o.y * iv), pack_bf16x2(o.z * iv, o.w * iv));
                }
            }
            // The next run's queries and sums go where this one's were; O is overwritten by its
            // first PV, which waits for these warps' P.
            tc_fence_before();
            runs.done(lane);
            if (!(ok = soft_sync())) break;
        }
    }

    // Teardown: every tensor-core operation must be complete before TMEM is freed.  (A softmax warp
    // that gave up between its stores to TMEM and their wait has them in flight here.)
    if (warp < kSoft) tmem_st_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
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

// Joins the partial states of the items that were cut between CTA groups.  A block takes eight
// rows of one row tile at one cut (the first unit of a group): at most 147 cuts, however
// many rows the batch has.  The first cut of an item does the work for all of its cuts, in
// the order of the groups; a warp takes one row.  Rows of whole items were written by the
// kernel above.  (A warp for every row of the batch, each adding up the units before it:
// 3.9 ms a call on 2048 sequences of 8 nodes and 32 heads, 1.1 now.  Two and four rows to a
// warp, in turn: 26 and 30 us where one takes 23, on one sequence of 1021 tokens.)
template <int D>
__global__ void __launch_bounds__(kMergeThreads) tree_merge_kernel(const __grid_constant__ TreeArgs a, const __grid_constant__ Shape sh,
                                                                   int row_blocks) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int member = blockIdx.x / row_blocks % sh.R, g0 = blockIdx.x / row_blocks / sh.R;
    const int row = blockIdx.x % row_blocks * (kMergeThreads / 32) + warp;
    // Sequences that have no room for their nodes: reported here, a thread each.
    for (int b = blockIdx.x * kMergeThreads + threadIdx.x; b < sh.B; b += gridDim.x * kMergeThreads) {
        const int64_t L = a.seqlens[b];
        const int n = a.counts ? max(0, min(a.counts[b], a.T)) : a.T;
        if (L < 0 || L + n > (int64_t)a.pk.max_pages * a.pk.page_size) atomicCAS(a.status, 0, ATFLASH_DEVICE_BAD_PAGE);
    }
    // Units of this thread's sequences, before them, and of the batch.
    __shared__ int64_t warp_units[kMergeThreads / 32], at_units;
    __shared__ int at_b;
    const int each = (sh.B - 1) / kMergeThreads + 1, b0 = min((int)threadIdx.x * each, sh.B), b1 = min(b0 + each, sh.B);
    int64_t own = 0;
    for (int b = b0; b < b1; ++b) own += units_of(seq_of(a, sh, b), sh.Hkv);
    int64_t before = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, before, o);
        if (lane >= o) before += y;
    }
    if (lane == 31) warp_units[warp] = before;
    __syncthreads();
    before -= own;
    int64_t total = 0;
    for (int x = 0; x < kMergeThreads / 32; ++x) {
        if (x < warp) before += warp_units[x];
        total += warp_units[x];
    }
    // The sequence that holds the cut's unit.
    const int active = active_groups(total, sh.groups);
    const int64_t cut = g0 + 1 < active ? first_unit(total, active, g0 + 1) : -1;
    if (cut >= before && cut < before + own) {
        int b = b0;
        for (int64_t n; cut >= before + (n = units_of(seq_of(a, sh, b), sh.Hkv)); ++b) before += n;
        at_units = before;
        at_b = b;
    }
    __syncthreads();
    // Blocks without work end at once and make room; the first one waits in any case, so that this
    // grid never ends before the one it depends on.
    if (blockIdx.x == 0) pdl_wait();
    if (cut < 0) return;
    const int b = at_b;
    const Seq s = seq_of(a, sh, b);
    const int64_t off = cut - at_units;
    const int per = item_units(s);
    const int item = (int)(off >> 31 ? off / per : (uint32_t)off / (uint32_t)per);
    const int64_t first = at_units + (int64_t)item * per;
    // No cut between two items, nor in an item's cost; and the item's first cut only.
    if (cut == first || cut - first >= s.tiles || first_unit(total, active, g0) > first) return;
    const int row0 = (item % s.groups * sh.R + member) * kBM;
    if (row >= s.nodes * sh.G - row0) return;
    // Group of the last tile's unit x: the largest g with floor(g * total / active) <= x.
    const int64_t y = (first + s.tiles) * active - 1;
    const int g1 = (int)((y | total) >> 31 ? y / total : (uint32_t)y / (uint32_t)total);
    auto state = [&](int g) {
        // The item is the last of group g0's run and the first of the later ones'.
        return a.workspace + (((size_t)g * sh.R + member) * 2 + (g == g0 ? 1 : 0)) * kBM * (D + 2);
    };
    pdl_wait();
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
    const int i = (row0 + row) / sh.G, hq = item / s.groups * sh.G + (row0 + row) % sh.G;
    const size_t to = (((size_t)b * a.T + i) * a.Hq + hq) * D + lane * V;
#pragma unroll
    for (int v = 0; v < V; ++v) {
        if (a.out_f32) static_cast<float *>(a.out)[to + v] = acc[v] * inv;
        else static_cast<__nv_bfloat16 *>(a.out)[to + v] = __float2bfloat16_rn(acc[v] * inv);
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

template <int D, bool kPacked, int NC>
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
    // Once per device: the shared memory, and that the in-kernel register split finds the
    // launch count it assumes.
    static std::atomic<uint64_t> configured{0};
    int dev = 0;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
    if (!(configured.load(std::memory_order_relaxed) & bit)) {
        const auto kernel = tree_decode_kernel<D, kPacked, NC>;
        if ((e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D, kPacked>::Request)) != cudaSuccess) return e;
        cudaFuncAttributes fa;
        if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
        if (fa.numRegs != kLaunchRegs) return cudaErrorInvalidConfiguration;
        configured.fetch_or(bit, std::memory_order_relaxed);
    }
    tree_decode_kernel<D, kPacked, NC><<<sh.groups * sh.R, kThreads, Cfg<D, kPacked>::Request, s>>>(tk, tv, a, sh, wp, rt, box_keys);
    if ((e = cudaGetLastError()) != cudaSuccess) return e;
    // As many cuts as CTA groups that can have work (units of the longest sequences that the table
    // has room for), less one; of a single row tile, the rows that exist.
    const int64_t rows = (int64_t)a.T * sh.G, row_groups = (rows + kBM * sh.R - 1) / (kBM * sh.R);
    const int64_t tiles = ((int64_t)a.pk.max_pages * a.pk.page_size + kBN - 1) / kBN;
    const int64_t units = a.B * row_groups * a.Hkv * (tiles + kItemCost);
    const int cuts = (int)(units < sh.groups ? units : sh.groups) - 1;
    const int row_blocks = (int)((rows < kBM ? rows : kBM) + kMergeThreads / 32 - 1) / (kMergeThreads / 32);
    return launch_dependent(tree_merge_kernel<D>, dim3((unsigned)(cuts * sh.R * row_blocks)), dim3(kMergeThreads), 0, s, a, sh, row_blocks);
}

}  // namespace tree

// Two partial states of one row tile per CTA, whatever the lengths.
size_t tree_workspace_bytes(int B, int T, int Hq, int Hkv, int D) {
    const tree::Shape sh = tree::shape_of(B, T, Hq, Hkv);
    return (size_t)sh.groups * sh.R * 2 * tree::kBM * (D + 2) * sizeof(float);
}

cudaError_t launch_tree_decode(const TreeArgs &a, const WindowParams &wp, const RopeTurns &rt, cudaStream_t s) {
    // Columns per softmax warp: as many copies of the rows as the 128 MMA rows hold.
    const int64_t rows = (int64_t)a.T * (a.Hq / a.Hkv);
#define ATF_TREE(DD, PK)                                                 \
    (rows <= 32 ? tree::launch<DD, PK, 32>(a, wp, rt, s)                 \
                : rows <= 64 ? tree::launch<DD, PK, 64>(a, wp, rt, s) : tree::launch<DD, PK, 128>(a, wp, rt, s))
    if (a.D == 128) return a.packed ? ATF_TREE(128, true) : ATF_TREE(128, false);
    return a.packed ? ATF_TREE(64, true) : ATF_TREE(64, false);
#undef ATF_TREE
}

}  // namespace atf
