// Gradients of cross attention on the 5th-generation tensor cores.
//
//   P = exp(scale Q K^T - lse),  dP = dO V^T,  delta = rowsum(dO * O),  dS = P * (dP - delta),
//   dQ = scale dS K,   dK = scale dS^T Q,   dV = P^T dO.
//
// dQ sums over the keys, dK and dV over the queries.  One pass that forms all three has to add its
// parts of dQ across CTAs, with atomics whose order changes the result or through memory; here they
// are two launches of one kernel instead, which computes S and dP twice (7 products, not 5) and
// whose every output has one owner:
//   dQ launch : a unit holds a query tile's Q and dO and streams the key tiles' K and V;
//   dKV launch: a unit holds a key tile's K and V and streams the query tiles' Q and dO, of all
//               heads that share the key head.  The query tiles are cut into `splits` ranges so that
//               a prompt's few key tiles fill the SMs; the ranges' fp32 parts go through the
//               workspace and are added in order by a last kernel.
// With R0, R1 the tiles that a unit holds and T0, T1 those that it streams, both are
//   S = R0 T0^T,  dP = R1 T1^T,  acc0 += dS T0,  and for dKV also  acc1 += P T1,
// rows being queries (dQ) or keys (dKV): lse and delta belong to the rows or to the columns.
//
// A CTA walks a contiguous range of units, cut by cost.  Roles (20 warps):
//   warps 0-15: thread = row and 32 of the 128 columns.  S is turned into P, which takes its place as packed
//               bf16, the A operand of dV += P^T dO; then dP into dS in its place.  A step's chain is
//               dS(i) -> acc0 -> dP(i+1) -> dS(i+1); dV, the next S and its exponentials fit beside it.
//   warps 16, 18: T0 tiles (3 slots), T1 tiles (dKV 2, dQ 1); 19: R tiles; 17: MMA.
// Both T tiles of a step are read to its end, and a slot that is filled only then comes too late for
// the next step's S: with two slots of each, a dKV step waited about 1500 cycles for its load.  Seven
// tiles fit; the third T0 slot takes the place of an output tile in dKV (its read-out goes through R0
// and R1, once for many steps), and of the second T1 slot in dQ (V is only needed for dP).
// What orders the reads of a slot before its next copy: -lse lies in the T0 slot, which is released behind DSFULL, after
// every read of it.  The T1 slot is released earlier, by the product behind SREAD, and its -delta is read later, when dS
// is formed: it has a barrier of its own (DFREE), at which the MMA warp arrives once DSFULL of the step is through.  The
// load of dO goes ahead of it, the 512 bytes of -delta wait for it.  T1FULL completes with both copies, so that it cannot
// go round again before every compute thread is past it.
// A first kernel leaves -lse (log2 units) and -delta of every query tile's 128 rows side by side in the
// workspace, so that dKV copies them with the tiles.  O is at hand in bf16 only, and its rounding reaches every dS
// of the row through delta; the fewer keys, the less of it averages out (three keys, two queries: 0.005 of dQ, where
// the roundings of P, dS and dQ come to 0.0024).  With one key tile (128 keys or fewer) the dQ launch has the
// whole row: it takes delta = rowsum(P * dP) instead and puts it in the workspace for dKV.
// P and dS are rounded to bf16 (by 2^-8 of themselves at most) for the products that they are operands of, as Q, K and dO
// are bf16 and the tensor cores take both operands in one type; the gradients are off by 0.0025 in the 2-norm against 64
// bits, 0.0017 of which is their own rounding.  Scores, dP, delta, lse and all sums are fp32.
// The launches are chained: a kernel's CTAs set up, and load what no launch writes, on SMs that the launch before has
// left (480p: 67.6 us in a stream and 57.2 in a graph without, 57.8 and 54.9 with).  dKV may be there as long as dQ
// runs, so that its roles wait for dQ's end before their first bounded wait for one another: the limit is for what a
// block waits of itself, not for the launch before.
// Measured in a graph: 4680 queries x 12 heads x 512 states 54.8 us (672 TFLOP/s of the five products; of the launches
// alone under a profiler, with cold caches: statistics 8.8 us, dQ 24.4 with the tensor pipe busy 46 % of the cycles, dKV
// 28.3 with 54 %, fold 8.4), 40 heads 176 us (698).  A step's chain bounds both: S, exponentials, dP, dS and the last
// product follow one another, and dKV reads both operands of S and dP from shared memory, whose bandwidth those
// products take whole.  Slower: the last range of a key tile adding the parts itself instead of a launch (480p 57.6 -> 61.8 us).
// Tensor memory: acc0 | acc1 | S | dP, 128 columns each.  dQ has no acc1: its columns hold Q and dO, which the
// compute warps put there as the A operands of S and dP, so that their shared memory takes the next
// unit's tiles while this unit runs (loading them between units cost 2000 of a unit's 12600 cycles).
#include <algorithm>

#include "chained.cuh"
#include "cross_tma.cuh"
#include "internal.h"
#include "per_device.h"
#include "softmax_tile.cuh"

namespace sdv2 {
namespace {

constexpr int HD = 128, BM = 128;
constexpr int T0ST = 3;
constexpr uint32_t TILE = 128 * HD * 2;
constexpr uint32_t HALF = TILE / 2;
constexpr int COMPUTE = 512;                   // threads of the compute warps
constexpr int T0_WARP = 16, MMA_WARP = 17, T1_WARP = 18, R_WARP = 19;
constexpr int NTHREADS = 20 * 32;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t ACC0 = 0, ACC1 = 128, SCOL = 256, XCOL = 384;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSms = 152;
constexpr int kMaxSplits = 8;

enum Bar { RFULL, REMPTY, T0FULL, T0EMPTY = T0FULL + T0ST, T1FULL = T0EMPTY + T0ST, T1EMPTY = T1FULL + 2, DFREE = T1EMPTY + 2,
           SFULL = DFREE + 2, SREAD, DPFULL, DSFULL, ACCFULL, RREADY, MMADONE, NBARS };

constexpr uint32_t SMEM_TILES = 7 * TILE;                      // R0 R1, T0 slots, T1 slots, dQ: an output tile
constexpr uint32_t SMEM_STATS = (T0ST + 2) * BM * 4;           // dKV: -lse per T0 slot, -delta per T1 slot
constexpr uint32_t SMEM_USED = SMEM_TILES + SMEM_STATS + 256;
constexpr uint32_t SMEM_BYTES = 232448;                        // 256 bytes to spare: the base has to be 1024-byte aligned
static_assert(SMEM_USED <= SMEM_BYTES && NBARS * 8 + 8 <= 256, "shared memory layout");

template <int CAP>
struct Params {
    CUtensorMap qmap, domap, dqmap;            // query tiles: 4D, boxes of 64 dims x pack x tokens
    CUtensorMap kmap[CAP], vmap[CAP];          // per stream: valid rows
    CUtensorMap dkmap, dvmap;                  // (D, Hk, Nk, B): boxes of 64 dims x 1 x 128 rows
    int32_t n[CAP];
    float* stats;                              // [query tile][-lse (log2 units), -delta][128]
    uint16_t *dk, *dv;                         // [B][Nk][Hk][D]
    float* part;                               // dKV: [split][unit][2][D/4][128][4]
    uint32_t* err;
    uint64_t timeout_ns;
    int64_t drop_tile;                         // this streamed tile is not copied (-1: none), for tests of the waits
    int32_t B, H, Hk, Nq, Nk;
    int32_t pack, tokens, group;               // heads and tokens of a query tile, query heads of a key head
    int32_t qtiles, packs;                     // query tiles of a (stream, pack), packs of a stream
    int32_t ktiles;                            // key tiles of Nk
    int32_t splits;                            // dKV: ranges of query tiles
    int32_t start[kSms + 1];                   // first unit of every CTA
    int64_t units;                             // dKV: units of one split
    float scale, scale_log2;
};

// A unit: dQ: (stream, pack of heads, query tile); dKV: (stream, key head, key tile, split).
struct Unit {
    int b, head, tile;                         // head: first query head (dQ) or key head (dKV)
    int split, index;
    int steps;                                 // streamed tiles
    int s0;                                    // dKV: first of them, counted over the group's packs
};

template <bool DKV, int CAP>
struct Walk {
    int cur, end;
    __device__ explicit Walk(const Params<CAP>& p) : cur(p.start[blockIdx.x]), end(p.start[blockIdx.x + 1]) {}
    __device__ bool next(const Params<CAP>& p, Unit& u)
    {
        if (cur >= end) return false;
        uint32_t x = static_cast<uint32_t>(cur++);
        u.index = static_cast<int>(x);
        if constexpr (DKV) {
            const uint32_t a = x / static_cast<uint32_t>(p.splits);
            u.split = static_cast<int>(x - a * p.splits);
            u.index = static_cast<int>(a);
            const uint32_t bh = a / static_cast<uint32_t>(p.ktiles);
            u.tile = static_cast<int>(a - bh * p.ktiles);
            const uint32_t b = bh / static_cast<uint32_t>(p.Hk);
            u.b = static_cast<int>(b);
            u.head = static_cast<int>(bh - b * p.Hk);
            const int all = p.qtiles * (p.group / p.pack);
            u.s0 = static_cast<int>(static_cast<int64_t>(all) * u.split / p.splits);
            u.steps = u.tile * BM < p.n[u.b] ? static_cast<int>(static_cast<int64_t>(all) * (u.split + 1) / p.splits) - u.s0 : 0;
        } else {
            const uint32_t bp = x / static_cast<uint32_t>(p.qtiles);
            u.tile = static_cast<int>(x - bp * p.qtiles);
            const uint32_t b = bp / static_cast<uint32_t>(p.packs);
            u.b = static_cast<int>(b);
            u.head = static_cast<int>(bp - b * p.packs) * p.pack;
            u.steps = p.n[u.b] > 1 ? (p.n[u.b] + BM - 1) / BM : 0;       // one key: the softmax is constant
            u.split = 0;
            u.s0 = 0;
        }
        return true;
    }
};

__device__ __forceinline__ void give_up(volatile int* abort_flag, uint32_t* err)
{
    *abort_flag = 1;
    atomicOr(err, kErrTimeout);
}

__device__ __forceinline__ void compute_barrier() { asm volatile("bar.sync 1, 512;" ::: "memory"); }

template <bool DKV, int CAP>
__global__ void __launch_bounds__(NTHREADS, 1) cross_backward_kernel(const __grid_constant__ Params<CAP> p)
{
    if constexpr (!DKV) launch_dependents();   // from dKV for the fold it is slower (480p: 57.2 us in a graph, 54.9 without)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if (static_cast<uint32_t>(smem - smem_raw) + SMEM_USED > SMEM_BYTES) {   // uniform: the base is the same for all
        if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
        return;
    }
    constexpr int T1ST = DKV ? 2 : 1;
    const uint32_t sR = smem_u32(smem), sT0 = sR + 2 * TILE, sT1 = sT0 + T0ST * TILE;
    const uint32_t sO = DKV ? sR : sR + 6 * TILE;                          // read-out: R0 and R1, or the seventh tile
    const uint32_t sL = sR + SMEM_TILES, sD = sL + T0ST * BM * 4;          // dKV: statistics of the T slots
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SMEM_TILES + SMEM_STATS);
    const uint32_t bar0 = smem_u32(bars);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint64_t tmo = p.timeout_ns;
    const int used_rows = p.pack * p.tokens;

    // The load warps only need the barriers: they start while the rest of the block is still setting up.
    if (warp >= T0_WARP) {
        if (threadIdx.x == T0_WARP * 32) {
            for (int i = 0; i < NBARS; ++i)
                mbar_init(bar(i), i == SREAD || i == DSFULL || i == RREADY || (i == REMPTY && !DKV) ? COMPUTE : 1);
            *abort_flag = 0;
            fence_mbar_init();
        }
        asm volatile("bar.sync 2, 128;" ::: "memory");
    } else {
        // Rows of a query tile that no load writes (the pack does not divide 128) are zero: as streamed tiles
        // they are summed over, with probability 0.  Only the tiles that queries go to: key tiles are loaded
        // whole, by warps that do not wait for this.
        constexpr int kFirst = DKV ? 2 : 0, kTiles = DKV ? T0ST + 2 : 2;
        for (int i = threadIdx.x; i < (BM - used_rows) * 16 * kTiles; i += COMPUTE) {
            const int part = i & 15, r = i >> 4, tile = r / (BM - used_rows), row = used_rows + r - tile * (BM - used_rows);
            *reinterpret_cast<uint4*>(smem + (kFirst + tile) * TILE + (part >> 3) * HALF + row * 128 + (part & 7) * 16) = make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
    }
    uint32_t tmem = 0;
    if (warp <= MMA_WARP && warp != T0_WARP) {
        if (warp == MMA_WARP) {
            tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
            tmem_relinquish();
        }
        tc_fence_before();
        asm volatile("bar.sync 3, 544;" ::: "memory");           // compute warps and the MMA warp
        tc_fence_after();
        tmem = *tmem_slot;
    }
    Walk<DKV, CAP> walk(p);
    Unit u;
    bool ok = true;

    // One 128-row operand tile: a query tile (Q or dO) or a key tile (K or V).
    auto load_queries = [&](const CUtensorMap* map, uint32_t dst, int b_full, int h0, int tok, int b) {
        for (int hf = 0; hf < 2; ++hf) tma_load_4d(dst + hf * HALF, map, bar(b_full), hf * 64, h0, tok, b);
    };
    auto load_keys = [&](const CUtensorMap* map, uint32_t dst, int b_full, int hk, int row) {
        for (int hf = 0; hf < 2; ++hf) tma_load_3d(dst + hf * HALF, map, bar(b_full), hf * 64, hk, row);
    };
    const uint32_t query_bytes = static_cast<uint32_t>(used_rows) * HD * 2;

    if (warp == R_WARP) {
        if (lane == 0) {
            uint32_t units = 0;
            while (ok && walk.next(p, u)) {
                if (u.steps == 0) continue;
                if (!mbar_wait_bounded(bar(REMPTY), (units & 1u) ^ 1u, tmo, abort_flag)) { ok = false; break; }
                if constexpr (DKV) {
                    mbar_arrive_expect_tx(bar(RFULL), 2 * TILE);
                    load_keys(&p.kmap[u.b], sR, RFULL, u.head, u.tile * BM);
                    load_keys(&p.vmap[u.b], sR + TILE, RFULL, u.head, u.tile * BM);
                } else {
                    mbar_arrive_expect_tx(bar(RFULL), 2 * query_bytes);
                    load_queries(&p.qmap, sR, RFULL, u.head, u.tile * p.tokens, u.b);
                    load_queries(&p.domap, sR + TILE, RFULL, u.head, u.tile * p.tokens, u.b);
                }
                ++units;
                if (DKV && units == 1) wait_for_launch_before();
            }
            if (!ok) give_up(abort_flag, p.err);
            volatile int never = 0;            // every copy lands before the CTA may exit
            if (units) mbar_wait_bounded(bar(RFULL), (units - 1) & 1u, tmo, &never);
        }
        __syncwarp();
    } else if (warp == T0_WARP || warp == T1_WARP) {
        if (lane == 0) {
            const bool t0 = warp == T0_WARP;
            const int nst = t0 ? T0ST : T1ST;
            const int full = t0 ? T0FULL : T1FULL, empty = t0 ? T0EMPTY : T1EMPTY;
            const uint32_t ring = t0 ? sT0 : sT1, stat_ring = t0 ? sL : sD;
            if constexpr (DKV) {
                wait_for_launch_before();      // the statistics, and the deltas that dQ put there
                asm volatile("fence.proxy.async.global;" ::: "memory");
            }
            int slot = 0;
            uint32_t phase = 0, pending = 0;
            while (ok && walk.next(p, u)) {
                int tile = 0, h0 = 0;          // dKV: query tile and first head of its pack
                const float* stat = nullptr;
                if constexpr (DKV) {
                    const int pk = u.s0 / p.qtiles;
                    tile = u.s0 - pk * p.qtiles;
                    h0 = u.head * p.group + pk * p.pack;
                    const int64_t q = (static_cast<int64_t>(u.b) * p.packs + u.head * (p.group / p.pack) + pk) * p.qtiles + tile;
                    stat = p.stats + q * 2 * BM + (t0 ? 0 : BM);
                }
                const int hk = DKV ? 0 : u.head / p.group;
                for (int i = 0; i < u.steps; ++i) {
                    if (!mbar_wait_bounded(bar(empty + slot), phase ^ 1u, tmo, abort_flag)) { ok = false; break; }
                    const uint32_t dst = ring + slot * TILE;
                    if ((DKV ? tile : i) != p.drop_tile) {
                        if constexpr (DKV) {
                            mbar_arrive_expect_tx(bar(full + slot), query_bytes + BM * 4);
                            load_queries(t0 ? &p.qmap : &p.domap, dst, full + slot, h0, tile * p.tokens, u.b);
                            // copied even when the wait runs out, so that the phase that dO has begun completes
                            if (!t0 && !mbar_wait_bounded(bar(DFREE + slot), phase ^ 1u, tmo, abort_flag)) ok = false;
                            bulk_load(stat_ring + slot * BM * 4, stat, BM * 4, bar(full + slot));
                        } else {
                            mbar_arrive_expect_tx(bar(full + slot), TILE);
                            load_keys(t0 ? &p.kmap[u.b] : &p.vmap[u.b], dst, full + slot, hk, i * BM);
                        }
                        pending = (pending & ~(17u << slot)) | (1u << slot) | (phase << (slot + 4));
                        if (!ok) break;
                    }
                    if constexpr (DKV) {
                        stat += 2 * BM;        // the packs of a key head follow one another
                        if (++tile == p.qtiles) {
                            tile = 0;
                            h0 += p.pack;
                        }
                    }
                    if (++slot == nst) {
                        slot = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (!ok) give_up(abort_flag, p.err);
            volatile int never = 0;            // every copy lands before the CTA may exit
            for (int i = 0; i < nst; ++i)
                if (pending >> i & 1u) mbar_wait_bounded(bar(full + i), pending >> (i + 4) & 1u, tmo, &never);
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        constexpr uint32_t idKK = idesc_bf16_f32(BM, BM, false);        // both operands K-major
        constexpr uint32_t idKM = idesc_bf16_f32(BM, HD, true);         // B is summed over its rows
        // shared-memory descriptors from their low word (address, leading stride); the high word is constant
        constexpr uint64_t kDescHigh = (uint64_t(1024 >> 4) << 32) | (uint64_t(1) << 46) | (uint64_t(2) << 61);
        auto desc = [&](uint32_t addr, uint32_t lbo) { return kDescHigh | ((addr >> 4) & 0x3FFFu) | ((lbo >> 4) << 16); };
        auto wait = [&](int i, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity, tmo, abort_flag));
            return ok;
        };
        auto product_tm = [&](uint32_t d, uint32_t a, uint32_t b) {      // D = A B^T, A in tensor memory
#pragma unroll
            for (int k = 0; k < HD / 16; ++k)
                mma_ts_warp(tmem + d, tmem + a + k * 8, desc(b + (k >> 2) * HALF + (k & 3) * 32, 16), idKK, k > 0 ? 1u : 0u);
        };
        auto product = [&](uint32_t d, uint32_t a, uint32_t b) {         // D = A B^T
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                const uint32_t o = (k >> 2) * HALF + (k & 3) * 32;
                mma_ss_warp(tmem + d, desc(a + o, 16), desc(b + o, 16), idKK, k > 0 ? 1u : 0u);
            }
        };
        // D += A B with A = 128 columns packed to bf16, each quarter of them at the start of its 32
        auto accumulate = [&](uint32_t d, uint32_t a, uint32_t b, bool add) {
#pragma unroll
            for (int k = 0; k < BM / 16; ++k)
                mma_ts_warp(tmem + d, tmem + a + (k >> 1) * 32 + (k & 1) * 8, desc(b + k * 2048u, HALF), idKM,
                            (add || k > 0) ? 1u : 0u);
        };
        uint32_t count = 0, units = 0;         // steps, units begun
        // T slots and phases of the next S, the next dP and the step being finished
        int s_slot = 0, p_slot = 0, a_slot0 = 0, a_slot1 = 0;
        uint32_t s_ph = 0, p_ph = 0;
        auto begin_s = [&]() {
            if (!wait(T0FULL + s_slot, s_ph)) return;
            tc_fence_after();
            if constexpr (DKV) product(SCOL, sR, sT0 + s_slot * TILE);
            else product_tm(SCOL, ACC1, sT0 + s_slot * TILE);
            mma_commit_warp(bar(SFULL));
            if (++s_slot == T0ST) {
                s_slot = 0;
                s_ph ^= 1u;
            }
        };
        auto begin_dp = [&]() {
            if (!wait(T1FULL + p_slot, p_ph)) return;
            tc_fence_after();
            if constexpr (DKV) product(XCOL, sR + TILE, sT1 + p_slot * TILE);
            else product_tm(XCOL, ACC1 + 64, sT1 + p_slot * TILE);
            mma_commit_warp(bar(DPFULL));
            if (!DKV) mma_commit_warp(bar(T1EMPTY + p_slot));            // V has done its part
            if (++p_slot == T1ST) {
                p_slot = 0;
                p_ph ^= 1u;
            }
        };
        if constexpr (DKV) wait_for_launch_before();
        while (ok && walk.next(p, u)) {
            if (u.steps == 0) continue;
            // the unit before has read its last S and written its last dS, so both score tiles are free
            if (!wait(DKV ? RFULL : RREADY, units & 1u)) break;
            ++units;
            tc_fence_after();
            begin_s();
            if (!ok) break;
            begin_dp();
            for (int i = 0; ok && i < u.steps; ++i, ++count) {
                const bool more = i + 1 < u.steps;
                if (DKV || more) {
                    if (!wait(SREAD, count & 1u)) break;
                    tc_fence_after();
                }
                if constexpr (DKV) {
                    accumulate(ACC1, SCOL, sT1 + a_slot1 * TILE, i > 0);         // dV += P^T dO
                    mma_commit_warp(bar(T1EMPTY + a_slot1));
                }
                if (more) {
                    begin_s();
                    if (!ok) break;
                }
                if (!wait(DSFULL, count & 1u)) break;
                tc_fence_after();
                accumulate(ACC0, XCOL, sT0 + a_slot0 * TILE, i > 0);             // dQ += dS K, dK += dS^T Q
                mma_commit_warp(bar(T0EMPTY + a_slot0));
                if (++a_slot0 == T0ST) a_slot0 = 0;
                if constexpr (DKV) {
                    mbar_arrive_warp(bar(DFREE + a_slot1));                      // every thread has read the step's -delta
                    if (++a_slot1 == T1ST) a_slot1 = 0;
                }
                if (!more) mma_commit_warp(bar(ACCFULL));
                else begin_dp();
            }
        }
        if (!ok && lane == 0) give_up(abort_flag, p.err);
        mma_commit_warp(bar(MMADONE));         // every MMA completes before tensor memory is freed
        if (lane == 0) {
            volatile int never = 0;
            mbar_wait_bounded(bar(MMADONE), 0, tmo, &never);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- P and dS, thread = (row, 32 columns)
        const int quarter = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t tL = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const bool leader = threadIdx.x == 0;
        uint32_t count = 0, units = 0;
        float row_lse = 0.f, row_delta = 0.f;  // dQ: of the thread's row, negated, and of the unit that comes next
        auto fetch_unit = [&](const Unit& v) {
            if constexpr (!DKV) {
                if (v.steps == 0) return;
                row_lse = p.stats[static_cast<int64_t>(v.index) * 2 * BM + row];
                row_delta = p.stats[static_cast<int64_t>(v.index) * 2 * BM + BM + row];
            }
        };
        int slot0 = 0, slot1 = 0;              // dKV: T slots of the step
        uint32_t phase0 = 0, phase1 = 0;
        uint32_t resident = 0;                 // dQ: units whose Q and dO went to tensor memory
        // Every lane takes part in the vote over a wait's outcome, which leaves `ok` the same in all of a warp: tensor-memory
        // loads are warp-collective, and a lane that went past a vote alone would leave the others there.
        auto all = [&](bool here) { return __all_sync(0xffffffffu, here); };
        auto arrived = [&](int i, uint32_t parity) { return mbar_wait_bounded(bar(i), parity, tmo, abort_flag); };
        auto put_resident = [&](const Unit& v) {
            if constexpr (!DKV) {
                if (v.steps == 0) return;
                ok = all(ok && arrived(RFULL, resident & 1u));
                ++resident;
                tc_fence_after();
#pragma unroll
                for (int which = 0; which < 2; ++which) {
                    const uint8_t* src = smem + which * TILE + (quarter >> 1) * HALF + row * 128;
                    uint32_t w[16];
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint4 x = *reinterpret_cast<const uint4*>(src + ((((quarter & 1) * 4 + e) ^ (row & 7)) << 4));
                        w[4 * e] = x.x;
                        w[4 * e + 1] = x.y;
                        w[4 * e + 2] = x.z;
                        w[4 * e + 3] = x.w;
                    }
                    tmem_st_x16(tL + ACC1 + which * 64 + quarter * 16, w);
                }
                mbar_arrive(bar(REMPTY));
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(RREADY));
            }
        };
        bool has = walk.next(p, u);
        if constexpr (!DKV) wait_for_launch_before();              // the statistics
        bool waited = false;                                       // dKV: rows behind a stream's last need not wait
        if (has) {
            fetch_unit(u);
            put_resident(u);
        }
        while (has) {
            Unit nx;                           // decoded here, not between the last step and the read-out
            const bool more_units = walk.next(p, nx);
            const bool constant = DKV && p.n[u.b] == 1;           // a softmax over one key has no gradient
            if (DKV && u.steps > 0 && !waited) {
                wait_for_launch_before();
                waited = true;
            }
            const uint64_t lse2 = f32x2_pack(row_lse, row_lse);
            uint64_t delta2 = f32x2_pack(row_delta, row_delta);
            // a thread whose wait ran out still runs through all steps, to meet the others at every barrier
#pragma unroll 1
            for (int i = 0; i < u.steps; ++i, ++count) {
                const float* cl = reinterpret_cast<const float*>(smem + SMEM_TILES) + slot0 * BM + quarter * 32;
                const float* cd = reinterpret_cast<const float*>(smem + SMEM_TILES) + (T0ST + slot1) * BM + quarter * 32;
                ok = all(ok && (!DKV || arrived(T0FULL + slot0, phase0)) && arrived(SFULL, count & 1u));
                tc_fence_after();
                const uint64_t sl2x2 = f32x2_pack(p.scale_log2, p.scale_log2);
                uint64_t pr[16];                                   // P, two columns each
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[16], w[8];
                    tmem_ld_x16_sync(tL + SCOL + quarter * 32 + c * 16, x);
                    ulonglong2 st[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[e] = DKV ? reinterpret_cast<const ulonglong2*>(cl)[c * 4 + e] : ulonglong2{lse2, lse2};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint64_t m2 = e & 1 ? st[e >> 1].y : st[e >> 1].x;
                        float a, b;
                        f32x2_unpack(ffma2(f32x2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sl2x2, m2), a, b);
                        a = ex2_approx(a);
                        b = ex2_approx(b);
                        pr[c * 8 + e] = f32x2_pack(a, b);
                        w[e] = bf16_pair(a, b);
                    }
                    // the first 16 columns have been read, the second are not written over
                    if constexpr (DKV) tmem_st_x8(tL + SCOL + quarter * 32 + c * 8, w);
                }
                if constexpr (DKV) tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(SREAD));
                if constexpr (!DKV) {
                    // Columns behind the stream's last key have a score of 0, whose exponential is no number where
                    // the row's lse is below -88; their keys are zero, but the product would not be.
                    const int keys = p.n[u.b] - i * BM - quarter * 32;
                    if (keys < 32)
#pragma unroll
                        for (int e = 0; e < 16; ++e)
                            pr[e] = 2 * e >= keys ? 0 : 2 * e + 1 >= keys ? pr[e] & 0xFFFFFFFFu : pr[e];
                }
                ok = all(ok && (!DKV || arrived(T1FULL + slot1, phase1)) && arrived(DPFULL, count & 1u));
                if (!ok) give_up(abort_flag, p.err);
                tc_fence_after();
                if constexpr (!DKV)
                    if (u.steps == 1) {                            // delta = rowsum(P * dP), see the head of the file
                        uint64_t sum2 = 0;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t x[16];
                            tmem_ld_x16_sync(tL + XCOL + quarter * 32 + c * 16, x);
#pragma unroll
                            for (int e = 0; e < 8; ++e)
                                sum2 = ffma2(f32x2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), pr[c * 8 + e], sum2);
                        }
                        float a, b;
                        f32x2_unpack(sum2, a, b);
                        float* part = reinterpret_cast<float*>(smem + SMEM_TILES);     // [quarter][row]
                        part[quarter * BM + row] = a + b;
                        compute_barrier();                         // the next write lies behind the read-out's barriers
                        const float d = -((part[row] + part[BM + row]) + (part[2 * BM + row] + part[3 * BM + row]));
                        delta2 = f32x2_pack(d, d);
                        if (quarter == 0) p.stats[static_cast<int64_t>(u.index) * 2 * BM + BM + row] = d;
                    }
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t x[16], w[8];
                    tmem_ld_x16_sync(tL + XCOL + quarter * 32 + c * 16, x);
                    ulonglong2 st[4];
#pragma unroll
                    for (int e = 0; e < 4; ++e) st[e] = DKV ? reinterpret_cast<const ulonglong2*>(cd)[c * 4 + e] : ulonglong2{delta2, delta2};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint64_t m2 = e & 1 ? st[e >> 1].y : st[e >> 1].x;
                        float a, b;
                        f32x2_unpack(fmul2(fadd2(f32x2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), m2), pr[c * 8 + e]), a, b);
                        w[e] = constant ? 0u : bf16_pair(a, b);
                    }
                    tmem_st_x8(tL + XCOL + quarter * 32 + c * 8, w);
                }
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(DSFULL));
                if constexpr (DKV) {
                    if (++slot0 == T0ST) {
                        slot0 = 0;
                        phase0 ^= 1u;
                    }
                    if (++slot1 == T1ST) {
                        slot1 = 0;
                        phase1 ^= 1u;
                    }
                }
            }
            // the next unit's statistics and tiles are on their way while the accumulators are read out
            has = more_units;
            if (has) {
                put_resident(nx);              // dP of the last step is there, so the unit is done with its own
                fetch_unit(nx);
            }
            // ------------------------------------------------------------ read out the accumulators
            if (DKV && u.steps == 0 && p.splits == 1) {            // rows behind the stream's last are zero
                // not through R0 and R1, which may hold the next unit; a half-warp a row (a thread a row: 3 us a unit)
                const int64_t first = (static_cast<int64_t>(u.b) * p.Nk + u.tile * BM) * p.Hk + u.head;
                const int rows = min(BM, p.Nk - u.tile * BM);
                for (int i = threadIdx.x; i < rows * 16; i += COMPUTE) {
                    const int64_t at = (first + static_cast<int64_t>(i >> 4) * p.Hk) * HD + (i & 15) * 8;
                    *reinterpret_cast<uint4*>(p.dk + at) = make_uint4(0, 0, 0, 0);
                    *reinterpret_cast<uint4*>(p.dv + at) = make_uint4(0, 0, 0, 0);
                }
                u = nx;
                continue;
            }
            if (u.steps > 0) {
                ok = all(ok && arrived(ACCFULL, units & 1u));
                ++units;
                tc_fence_after();
            }
            if (!ok) give_up(abort_flag, p.err);                   // and on, past every barrier, with whatever is there
            const bool zero = u.steps == 0 || (DKV && u.tile * BM + row >= p.n[u.b]);
#pragma unroll 1
            for (int acc = 0; acc < (DKV ? 2 : 1); ++acc) {
                uint32_t o[32];
                tmem_ld_x32_sync(tL + acc * 128 + quarter * 32, o);
                if (DKV && p.splits > 1) {
                    float4* part = reinterpret_cast<float4*>(p.part) +
                                   ((u.split * p.units + u.index) * 2 + acc) * (HD / 4) * BM + quarter * 8 * BM + row;
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        part[v * BM] = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                                            : make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                          __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                    continue;
                }
                const float f = acc == 0 ? p.scale : 1.0f;
                uint32_t w[16];
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    w[e] = zero ? 0u : bf16_pair(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
                if (!DKV) {
                    if (leader) tma_store_wait_read();             // the output tile is free
                    compute_barrier();
                }
                uint8_t* dst = smem + (sO - sR) + acc * TILE + (quarter >> 1) * HALF + row * 128;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    *reinterpret_cast<uint4*>(dst + ((((quarter & 1) * 4 + v) ^ (row & 7)) << 4)) =
                        make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
                fence_proxy_async();
                compute_barrier();
                if (leader)
                    for (int hf = 0; hf < 2; ++hf) {
                        if constexpr (DKV)
                            tma_store_4d(acc == 0 ? &p.dkmap : &p.dvmap, sO + acc * TILE + hf * HALF, hf * 64, u.head, u.tile * BM, u.b);
                        else
                            tma_store_4d(&p.dqmap, sO + hf * HALF, hf * 64, u.head, u.tile * p.tokens, u.b);
                    }
            }
            if (DKV && u.steps > 0 && leader) {                    // R0 and R1 are free for the next unit's tiles
                tma_store_wait_read();
                mbar_arrive(bar(REMPTY));
            }
            tc_fence_before();
            u = nx;
        }
        if (leader) tma_store_wait();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// Adds the splits of a key tile's dK or dV in order.  grid: (units, 2, 4): a block adds 32 dims of 128 rows, turned
// around in shared memory because the parts lie [dims / 4][row].
__global__ void __launch_bounds__(256) cross_fold_kernel(const float4* part, int splits, int64_t units, int ktiles, int Hk,
                                                         int Nk, float scale, uint16_t* dk, uint16_t* dv)
{
    wait_for_launch_before();
    __shared__ __align__(16) uint16_t tile[BM][32 + 8];
    const int64_t unit = blockIdx.x;
    const int which = blockIdx.y;
    const int64_t step = units * 2 * (BM * (HD / 4));
    const float4* src = part + (unit * 2 + which) * (BM * (HD / 4)) + blockIdx.z * 8 * BM + threadIdx.x;
    float4 s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = src[i * 256];
#pragma unroll 1
    for (int k = 1; k < splits; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 x = src[k * step + i * 256];
            s[i].x += x.x;
            s[i].y += x.y;
            s[i].z += x.z;
            s[i].w += x.w;
        }
    const float f = which == 0 ? scale : 1.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint2*>(&tile[threadIdx.x & 127][(2 * i + (threadIdx.x >> 7)) * 4]) =
            make_uint2(bf16_pair(s[i].x * f, s[i].y * f), bf16_pair(s[i].z * f, s[i].w * f));
    __syncthreads();
    const int64_t bh = unit / ktiles;
    const int kt = static_cast<int>(unit - bh * ktiles);
    const int64_t b = bh / Hk;
    const int hk = static_cast<int>(bh - b * Hk);
    uint16_t* out = which == 0 ? dk : dv;
#pragma unroll
    for (int i = threadIdx.x; i < BM * 4; i += 256) {
        const int r = i >> 2, v = i & 3;
        const int64_t j = static_cast<int64_t>(kt) * BM + r;
        if (j < Nk)
            *reinterpret_cast<uint4*>(out + ((b * Nk + j) * Hk + hk) * HD + blockIdx.z * 32 + v * 8) =
                *reinterpret_cast<const uint4*>(&tile[r][v * 8]);
    }
}

// -lse (log2 units) and -delta = -rowsum(dO * O) of a query tile's rows; rows that are none get lse = infinity, so
// that their probabilities are 0.  grid: (query tiles, 4): a half-warp per row, two rows each.
__global__ void __launch_bounds__(256) cross_stats_kernel(const uint16_t* out, const uint16_t* dout, const float* lse,
                                                          float* stats, int H, int Nq, int pack, int tokens, int qtiles, int packs)
{
    wait_for_launch_before();
    launch_dependents();                       // behind the wait: dQ reads what was there before the call without one
    const int half = threadIdx.x >> 4, sub = threadIdx.x & 15;
    const uint32_t bp = blockIdx.x / static_cast<uint32_t>(qtiles);
    const int tile = static_cast<int>(blockIdx.x - bp * qtiles);
    const int b = static_cast<int>(bp / static_cast<uint32_t>(packs));
    const int h0 = static_cast<int>(bp - b * packs) * pack;
    uint4 x[2], y[2];
    float l[2];
    bool live[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int r = blockIdx.y * 32 + half + 16 * i;
        const int rt = pack == 1 ? r : r / pack;
        const int64_t tok = static_cast<int64_t>(tile) * tokens + rt;
        live[i] = rt < tokens && tok < Nq;
        x[i] = y[i] = make_uint4(0, 0, 0, 0);
        l[i] = INFINITY;
        if (live[i]) {
            const int h = h0 + (r - rt * pack);
            const int64_t o = ((static_cast<int64_t>(b) * Nq + tok) * H + h) * HD + sub * 8;
            x[i] = *reinterpret_cast<const uint4*>(out + o);
            y[i] = *reinterpret_cast<const uint4*>(dout + o);
            l[i] = lse[(static_cast<int64_t>(b) * H + h) * Nq + tok];
        }
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint32_t xs[4] = {x[i].x, x[i].y, x[i].z, x[i].w}, ys[4] = {y[i].x, y[i].y, y[i].z, y[i].w};
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            sum = fmaf(__uint_as_float(xs[k] << 16), __uint_as_float(ys[k] << 16), sum);
            sum = fmaf(__uint_as_float(xs[k] & 0xFFFF0000u), __uint_as_float(ys[k] & 0xFFFF0000u), sum);
        }
#pragma unroll
        for (int o = 8; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        if (sub == 0) {
            float* dst = stats + static_cast<int64_t>(blockIdx.x) * 2 * BM + blockIdx.y * 32 + half + 16 * i;
            dst[0] = -l[i] * kLog2e;
            dst[BM] = live[i] ? -sum : 0.f;
        }
    }
}

struct Shape {
    int pack, tokens, qtiles, packs, group, ktiles, splits;
    int64_t kunits;                            // (stream, key head, key tile)
};

// Streamed tiles of a key tile's unit.
int64_t steps_of(const Shape& s) { return static_cast<int64_t>(s.qtiles) * (s.group / s.pack); }

// Ranges of query tiles for `units` key tiles: the smallest estimated time, a unit costing its steps and four more
// for its start, end and parts.
int best_splits(int64_t units, int64_t steps, int most)
{
    int splits = 1;
    int64_t best = INT64_MAX;
    for (int k = 1; k <= most && k <= steps; ++k) {
        const int64_t t = ((units * k + kSms - 1) / kSms) * ((steps + k - 1) / k + 4);
        if (t < best) {
            best = t;
            splits = k;
        }
    }
    return splits;
}

// The splits are those for full streams; they size the workspace.
Shape shape_of(int B, int H, int Hk, int64_t Nq, int64_t Nk)
{
    Shape s;
    s.group = H / Hk;
    s.pack = cross_pack(s.group);
    s.tokens = BM / s.pack;
    s.qtiles = static_cast<int>((Nq + s.tokens - 1) / s.tokens);
    s.packs = H / s.pack;
    s.ktiles = static_cast<int>((Nk + BM - 1) / BM);
    s.kunits = static_cast<int64_t>(B) * Hk * s.ktiles;
    s.splits = best_splits(s.kunits, steps_of(s), kMaxSplits);
    return s;
}

// Ranges of `units` units of equal cost; cost(i) of the i-th of `groups` runs of units.
template <typename F>
void cut(int32_t* start, int ctas, int64_t runs, int64_t units_per_run, F&& cost)
{
    int64_t total = 0;
    for (int64_t r = 0; r < runs; ++r) total += cost(r) * units_per_run;
    int64_t r = 0, before = 0;
    for (int i = 0; i <= ctas; ++i) {
        const int64_t x = total * i / ctas;
        while (r + 1 < runs && x > before + cost(r) * units_per_run) before += cost(r++) * units_per_run;
        start[i] = static_cast<int32_t>(std::min(runs * units_per_run, r * units_per_run + (x - before + cost(r) - 1) / cost(r)));
    }
}

template <typename K>
cudaError_t prepare_kernel(K kernel, PerDevice& prepared)
{
    int dev = 0;
    cudaGetDevice(&dev);
    return prepared.run(dev, [&]() {
        return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES));
    });
}

template <int CAP>
cudaError_t launch(const CrossBackward& f, cudaStream_t s)
{
    const CrossProblem& c = f.c;
    Shape sh = shape_of(c.B, c.H, c.Hk, c.Nq, c.Nk);
    // key tiles behind a stream's last row have no work: no more ranges than the others need
    int64_t live = 0;
    for (int b = 0; b < c.B; ++b) live += static_cast<int64_t>(c.Hk) * ((c.n[b] + BM - 1) / BM);
    sh.splits = best_splits(std::max<int64_t>(live, 1), steps_of(sh), sh.splits);
    static thread_local Params<CAP> p;
    p = Params<CAP>{};
    const CrossStrides dense = {int64_t(c.H) * HD, HD, int64_t(c.H) * HD * c.Nq};
    if (!encode_query_map(&p.qmap, c.q, c.H, c.Nq, c.B, c.qs, sh.pack, sh.tokens) ||
        !encode_query_map(&p.domap, f.dout, c.H, c.Nq, c.B, dense, sh.pack, sh.tokens) ||
        !encode_query_map(&p.dqmap, f.dq, c.H, c.Nq, c.B, dense, sh.pack, sh.tokens))
        return cudaErrorInvalidValue;
    for (int b = 0; b < c.B; ++b) {
        p.n[b] = c.n[b];
        if (c.n[b] > 0 && (!encode_key_map(&p.kmap[b], c.k + b * c.kvs.batch, c.Hk, c.n[b], c.kvs) ||
                           !encode_key_map(&p.vmap[b], c.v + b * c.kvs.batch, c.Hk, c.n[b], c.kvs)))
            return cudaErrorInvalidValue;
    }
    if (c.Nk > 0) {
        const CrossStrides kd = {int64_t(c.Hk) * HD, HD, int64_t(c.Hk) * HD * c.Nk};
        if (!encode_query_map(&p.dkmap, f.dk, c.Hk, c.Nk, c.B, kd, 1, BM) || !encode_query_map(&p.dvmap, f.dv, c.Hk, c.Nk, c.B, kd, 1, BM))
            return cudaErrorInvalidValue;
    }
    p.stats = f.stats;
    p.part = f.part;
    p.dk = f.dk;
    p.dv = f.dv;
    p.err = c.err;
    p.timeout_ns = c.timeout_ns;
    p.drop_tile = debug_drop_tile();
    p.B = c.B;
    p.H = c.H;
    p.Hk = c.Hk;
    p.Nq = c.Nq;
    p.Nk = c.Nk;
    p.pack = sh.pack;
    p.tokens = sh.tokens;
    p.group = sh.group;
    p.qtiles = sh.qtiles;
    p.packs = sh.packs;
    p.ktiles = sh.ktiles;
    p.splits = sh.splits;
    p.scale = c.scale;
    p.scale_log2 = c.scale * kLog2e;
    const int64_t qunits = static_cast<int64_t>(c.B) * sh.packs * sh.qtiles;
    if (qunits > INT32_MAX || sh.kunits * sh.splits > INT32_MAX) return cudaErrorInvalidConfiguration;

    cudaError_t e = launch_chained(cross_stats_kernel, dim3(static_cast<unsigned>(qunits), 4), dim3(256), 0, s, f.out, f.dout, f.lse,
                                   f.stats, c.H, c.Nq, sh.pack, sh.tokens, sh.qtiles, sh.packs);
    if (e != cudaSuccess) return e;
    static PerDevice dq_set, dkv_set;
    auto dq_kernel = cross_backward_kernel<false, CAP>;
    auto dkv_kernel = cross_backward_kernel<true, CAP>;
    if ((e = prepare_kernel(dq_kernel, dq_set)) != cudaSuccess || (e = prepare_kernel(dkv_kernel, dkv_set)) != cudaSuccess) return e;

    int ctas = static_cast<int>(std::min<int64_t>(qunits, kSms));
    cut(p.start, ctas, c.B, static_cast<int64_t>(sh.packs) * sh.qtiles, [&](int64_t b) { return c.n[b] > 1 ? (c.n[b] + BM - 1) / BM + int64_t(1) : 1; });
    e = launch_chained(dq_kernel, dim3(static_cast<unsigned>(ctas)), dim3(NTHREADS), SMEM_BYTES, s, p);
    if (e != cudaSuccess || c.Nk == 0) return e;
    // dKV: a run is a key tile's splits
    const int64_t all_steps = static_cast<int64_t>(sh.qtiles) * (sh.group / sh.pack);
    ctas = static_cast<int>(std::min<int64_t>(sh.kunits * sh.splits, kSms));
    cut(p.start, ctas, sh.kunits, sh.splits, [&](int64_t r) {
        const int64_t b = r / (static_cast<int64_t>(c.Hk) * sh.ktiles);
        return (r % sh.ktiles) * BM < c.n[b] ? (all_steps + sh.splits - 1) / sh.splits + 4 : int64_t(1);
    });
    p.units = sh.kunits;
    e = launch_chained(dkv_kernel, dim3(static_cast<unsigned>(ctas)), dim3(NTHREADS), SMEM_BYTES, s, p);
    if (e == cudaSuccess && sh.splits > 1)
        e = launch_chained(cross_fold_kernel, dim3(static_cast<unsigned>(sh.kunits), 2, 4), dim3(256), 0, s,
                           reinterpret_cast<const float4*>(f.part), sh.splits, sh.kunits, sh.ktiles, c.Hk, c.Nk, c.scale, f.dk, f.dv);
    return e;
}

}  // namespace

size_t cross_backward_stats_bytes(int B, int H, int Hk, int64_t Nq)
{
    const Shape s = shape_of(B, H, Hk, Nq, 0);
    return static_cast<size_t>(B) * s.packs * s.qtiles * 2 * BM * sizeof(float);
}

size_t cross_backward_part_bytes(int B, int H, int Hk, int64_t Nq, int64_t Nk)
{
    if (Nk == 0) return 0;
    const Shape s = shape_of(B, H, Hk, Nq, Nk);
    return s.splits > 1 ? static_cast<size_t>(s.splits) * s.kunits * 2 * BM * HD * sizeof(float) : 0;
}

cudaError_t launch_cross_backward(const CrossBackward& f, cudaStream_t s)
{
    return f.c.B <= 4 ? launch<4>(f, s) : launch<kCrossStreams>(f, s);
}

}  // namespace sdv2
