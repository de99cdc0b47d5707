// Cross attention on the 5th-generation tensor cores (tcgen05 + tensor memory).
//
//   out[b, i, h, :] = sum_{j < n_b} softmax_j(scale * q[b, i, h] . k[b, j, h']) v[b, j, h']
//
// The chunk attention's key range is long; a prompt's is a few 128-key tiles, so what decides here
// is not the key loop but how items follow one another and how evenly they fill the SMs.
//
// Rows.  A query tile holds 128 rows of one key head: `pack` of the heads that share it times
// 128 / pack tokens (rows are token-major), so that a few queries of many heads fill one tile and
// read the keys once.
//
// Schedule.  One CTA per SM walks a contiguous range of the query tiles in (stream, head, tile)
// order; the ranges are cut by cost (key tiles + 1 per query tile).  Two tiles of one head are a
// pair: two lanes of the CTA, each with its scores and its accumulator in tensor memory, use every
// key tile that is loaded.  A tile left over is a single: the lanes take the two halves of its
// keys and both accumulators, in the same rows of tensor memory, are joined when they are read
// out.  A single costs half a pair, so a range of three tiles takes one and a half times two, not
// twice.  With fewer tiles than SMs, a cluster of CTAs shares one tile's keys and joins through
// the cluster's shared memory.
//
// Roles in a CTA (12 warps):
//   warps 0-3, 4-7: softmax of lane 0, 1; thread = query row.  Then the row's epilogue.
//   warp 8: K tiles (2 slots); 10: V tiles (2 slots); 11: Q tiles (1 slot per lane).
//   warp 9: issues S_t = Q_t K^T and O_t += P_t V.
// Nothing is drained between items: a lane's next Q is loaded when its last S is done, its next S
// is issued behind its last PV, and the tensor cores run the other lane meanwhile.
//
// Measured (calls captured in a graph, inputs from more buffers than L2 holds): 4680 queries x 12 heads x 512 states
// 20.6 us (716 TFLOP/s), 10800 x 12 x 769 56.9 us (897), a key range of 8192 1440 TFLOP/s.  With one pair per SM a
// call takes 6.5 us (launch, first loads, one step's latency, last read-out) and 8.5 us for a pair over 512 keys, 1.65 us
// per 128 keys once the loop runs (the two products alone: 1.08).  In the loop the softmax's instructions bound it:
// 128 exponentials, maxima, sums and conversions a thread and step, eight warps.  Slower: four softmax warpgroups (22.0 us
// for the first case, 20.7 with two at the time), P stored in halves with the product begun early (8192 keys: 180 us, 163).
//
// Every wait is bounded; on expiry the kernel records the timeout in the workspace's error word,
// lets all roles finish what they have in flight and returns.
#include <algorithm>

#include "chained.cuh"
#include "cross_tma.cuh"
#include "internal.h"
#include "per_device.h"
#include "ptx_pair.cuh"
#include "softmax_tile.cuh"
#include "tensor_map.h"

namespace sdv2 {
namespace {

constexpr int BM = 128, BN = 128, HD = 128;
constexpr int KST = 2, VST = 2;
constexpr uint32_t TILE = 128 * HD * 2;
constexpr uint32_t HALF = TILE / 2;           // 64 dims of 128 rows
constexpr int K_WARP = 8, MMA_WARP = 9, V_WARP = 10, Q_WARP = 11;
constexpr int NTHREADS = 12 * 32;
constexpr uint32_t TMEM_COLS = 512;           // S_0 | S_1 | O_0 | O_1
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr int kMaxCluster = 16;
constexpr int kMaxCtas = 160;

enum Bar { QFULL = 0, QEMPTY = 2, KFULL = 4, KEMPTY = KFULL + KST, VFULL = KEMPTY + KST, VEMPTY = VFULL + VST,
           SFULL = VEMPTY + VST, PFULL = SFULL + 2, OFULL = PFULL + 2,
           MMADONE = OFULL + 2, NBARS = MMADONE + 1 };

constexpr uint32_t SMEM_TILES = (2 + KST + VST + 1) * TILE;   // Q, K, V, and half an output tile per lane
constexpr uint32_t SMEM_STATS = 2 * BM * 8;   // (max, sum) of every row and lane
constexpr uint32_t SMEM_USED = SMEM_TILES + SMEM_STATS + 256;
constexpr uint32_t SMEM_BYTES = 232448;       // all of it: 768 bytes are left to align the tiles with
static_assert(SMEM_USED + 768 <= SMEM_BYTES && NBARS * 8 + 8 <= 256, "shared memory layout");

template <int CAP>
struct Params {
    CUtensorMap qmap, omap;
    CUtensorMap kmap[CAP], vmap[CAP];
    int32_t n[CAP];
    uint16_t* out;
    float* lse;
    uint32_t* err;
    uint64_t timeout_ns;
    int64_t drop_tile;
    int32_t B, H, Hk, Nq;
    int32_t pack, tokens;                     // heads and tokens of a tile
    int32_t packs;                            // packs of heads of a stream
    int32_t group;                            // query heads of a key head
    int32_t tiles;                            // query tiles of one (stream, pack of heads)
    int32_t splits;                           // CTAs of a cluster that share a tile's keys
    int32_t start[kMaxCtas + 1];              // first query tile of every CTA (not of clusters)
    float scale_log2;
};

// What the two lanes of a CTA do next: two query tiles of one head, or the two halves of one tile's keys.
struct Item {
    int b, h0, tile;                          // stream, first head of the pack, first query tile
    bool pair;
    int keys, k0;                             // key tiles of the item, the first one
    __device__ int steps(int t) const { return pair ? keys : (t == 0 ? (keys + 1) / 2 : keys / 2); }
    __device__ int first(int t) const { return pair || t == 0 ? k0 : k0 + (keys + 1) / 2; }
};

// Key tiles of stream b.
template <int CAP>
__device__ __forceinline__ int key_tiles(const Params<CAP>& p, int b) { return (p.n[b] + BN - 1) / BN; }

// The CTA's items.  The start is decoded once; from then on the walk only counts, because a division
// by a launch parameter in every role and item cost more than the key tiles of a short prompt.
struct Walk {
    int b, h0, tile, left;                    // next query tile, tiles left
    template <int CAP>
    __device__ explicit Walk(const Params<CAP>& p)
    {
        uint32_t cur;
        if (p.splits > 1) {
            cur = blockIdx.x / static_cast<uint32_t>(p.splits);
            left = 1;
        } else {
            cur = static_cast<uint32_t>(p.start[blockIdx.x]);
            left = p.start[blockIdx.x + 1] - static_cast<int>(cur);
        }
        const uint32_t group = cur / static_cast<uint32_t>(p.tiles);
        tile = static_cast<int>(cur - group * p.tiles);
        const uint32_t bb = group / static_cast<uint32_t>(p.packs);
        b = static_cast<int>(bb);
        h0 = static_cast<int>(group - bb * p.packs) * p.pack;
    }
    template <int CAP>
    __device__ void peek(const Params<CAP>& p, Item& it) const
    {
        it.b = b;
        it.h0 = h0;
        it.tile = tile;
        it.keys = key_tiles(p, b);
        it.k0 = 0;
        it.pair = left > 1 && tile + 1 < p.tiles;
        if (p.splits > 1) {
            const uint32_t r = cluster_ctarank(), all = it.keys, n = p.splits;
            it.k0 = static_cast<int>(all * r / n);
            it.keys = static_cast<int>(all * (r + 1) / n) - it.k0;
        }
    }
    template <int CAP>
    __device__ bool next(const Params<CAP>& p, Item& it)
    {
        if (left <= 0) return false;
        peek(p, it);
        const int k = it.pair ? 2 : 1;
        left -= k;
        tile += k;
        if (tile == p.tiles) {
            tile = 0;
            h0 += p.pack;
            if (h0 == p.H) {
                h0 = 0;
                ++b;
            }
        }
        return true;
    }
};

__device__ __forceinline__ void give_up(volatile int* abort_flag, uint32_t* err)
{
    *abort_flag = 1;
    atomicOr(err, kErrTimeout);
}

// Barrier of lane t's softmax warpgroup.
__device__ __forceinline__ void lane_barrier(int t) { asm volatile("bar.sync %0, 128;" ::"r"(2 + t) : "memory"); }

// Barrier of both.
__device__ __forceinline__ void softmax_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float2 ld_cluster_f32x2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// Weight of a part of a row: 2^(m - M), 0 for a part without keys.
__device__ __forceinline__ float weight_of(float2 ml, float M) { return ml.y == 0.f ? 0.f : ex2_approx(ml.x - M); }

template <int CAP>
__global__ void __launch_bounds__(NTHREADS, 1) cross_attention_kernel(const __grid_constant__ Params<CAP> p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if (static_cast<uint32_t>(smem - smem_raw) + SMEM_USED > SMEM_BYTES) {   // uniform: the base is the same for all
        if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
        return;
    }
    const uint32_t sQ = smem_u32(smem), sK = sQ + 2 * TILE, sV = sK + KST * TILE, sO = sV + VST * TILE;
    float2* stats = reinterpret_cast<float2*>(smem + SMEM_TILES);               // [2][128]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SMEM_TILES + SMEM_STATS);
    const uint32_t bar0 = smem_u32(bars);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint64_t tmo = p.timeout_ns;
    const int splits = p.splits;

    // The load warps only need the barriers: they start while the rest of the block is still setting up.
    const int used_rows = p.pack * p.tokens;
    if (warp >= K_WARP) {
        if (threadIdx.x == K_WARP * 32) {
            for (int i = 0; i < NBARS; ++i) mbar_init(bar(i), i >= PFULL && i < PFULL + 2 ? 128 : 1);
            *abort_flag = 0;
            fence_mbar_init();
        }
        asm volatile("bar.sync 4, 128;" ::: "memory");
    } else {
        // rows of a Q tile that no load writes (the pack does not divide 128): zero, so that they stay finite
        for (int i = threadIdx.x; i < (BM - used_rows) * 32; i += K_WARP * 32) {
            const int part = i & 31, row = used_rows + (i >> 5);               // 2 tiles x 2 halves x 8 vectors
            *reinterpret_cast<uint4*>(smem + (part >> 4) * TILE + ((part >> 3) & 1) * HALF + row * 128 + (part & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        fence_proxy_async();
    }
    uint32_t tmem = 0;
    if (warp <= MMA_WARP && warp != K_WARP) {
        if (warp == MMA_WARP) {
            tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
            tmem_relinquish();
        }
        tc_fence_before();
        asm volatile("bar.sync 5, 288;" ::: "memory");         // softmax warps and the MMA warp
        tc_fence_after();
        tmem = *tmem_slot;
    }
    wait_for_launch_before();
    Walk walk(p);
    Item it;
    bool ok = true;

    if (warp == K_WARP || warp == V_WARP) {
        // ---------------------------------------------------------------- K and V tiles
        if (lane == 0) {
            const bool is_k = warp == K_WARP;
            const int nst = is_k ? KST : VST;
            const int full = is_k ? KFULL : VFULL, empty = is_k ? KEMPTY : VEMPTY;
            const uint32_t ring = is_k ? sK : sV;
            int slot = 0;
            uint32_t phase = 0, pending = 0;
            while (ok && walk.next(p, it)) {
                const CUtensorMap* map = is_k ? &p.kmap[it.b] : &p.vmap[it.b];
                const int hk = p.group == 1 ? it.h0 : it.h0 / p.group;
                for (int i = 0; i < it.keys; ++i) {
                    // a single's lanes alternate
                    const int j = it.pair ? it.k0 + i : it.first(i & 1) + (i >> 1);
                    if (!mbar_wait_bounded(bar(empty + slot), phase ^ 1u, tmo, abort_flag)) { ok = false; break; }
                    if (j != p.drop_tile) {
                        mbar_arrive_expect_tx(bar(full + slot), TILE);
                        for (int hf = 0; hf < 2; ++hf)
                            tma_load_3d(ring + slot * TILE + hf * HALF, map, bar(full + slot), hf * 64, hk, j * BN);
                        pending = (pending & ~(17u << slot)) | (1u << slot) | (phase << (slot + 4));
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
    } else if (warp == Q_WARP) {
        // ---------------------------------------------------------------- Q tiles
        if (lane == 0) {
            uint32_t loads[2] = {0, 0};
            const uint32_t bytes = static_cast<uint32_t>(used_rows) * HD * 2;
            while (ok && walk.next(p, it)) {
                for (int t = 0; t < 2; ++t) {
                    if (it.steps(t) == 0) continue;
                    if (!mbar_wait_bounded(bar(QEMPTY + t), (loads[t] & 1u) ^ 1u, tmo, abort_flag)) { ok = false; break; }
                    const int tok = (it.pair ? it.tile + t : it.tile) * p.tokens;
                    mbar_arrive_expect_tx(bar(QFULL + t), bytes);
                    for (int hf = 0; hf < 2; ++hf)
                        tma_load_4d(sQ + t * TILE + hf * HALF, &p.qmap, bar(QFULL + t), hf * 64, it.h0, tok, it.b);
                    ++loads[t];
                }
                Walk ahead = walk;        // the next item's queries reach L2 while this one runs
                Item nx;
                if (ok && ahead.next(p, nx) && nx.keys > 0)
                    for (int t = 0; t < (nx.pair ? 2 : 1); ++t)
                        for (int hf = 0; hf < 2; ++hf)
                            tma_prefetch_4d(&p.qmap, hf * 64, nx.h0, (nx.tile + t) * p.tokens, nx.b);
            }
            if (!ok) give_up(abort_flag, p.err);
            volatile int never = 0;
            for (int t = 0; t < 2; ++t)
                if (loads[t]) mbar_wait_bounded(bar(QFULL + t), (loads[t] - 1) & 1u, tmo, &never);
        }
        __syncwarp();
    } else if (warp == MMA_WARP) {
        // ---------------------------------------------------------------- MMA issue (converged warp)
        constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false), idO = idesc_bf16_f32(BM, HD, true);
        const uint64_t dQ = sdesc_sw128(sQ, 16, 1024), dK = sdesc_sw128(sK, 16, 1024), dV = sdesc_sw128(sV, HALF, 1024);
        constexpr uint64_t kTileStep = TILE >> 4;
        auto wait = [&](int i, uint32_t parity) {
            ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity, tmo, abort_flag));
            return ok;
        };
        int kslot = 0, vslot = 0;             // slots of the tile that the next S, PV uses
        uint32_t kph = 0, vph = 0;
        bool knew = true, vnew = true;        // a wait costs 100 cycles even when the tile is there: once a slot
        uint32_t qn[2] = {0, 0}, pn[2] = {0, 0};
        // S_t of the lane's next step; `release`: no other lane uses the key tile after it
        auto issue_s = [&](int t, bool first, bool last, bool release) {
            if (first && !wait(QFULL + t, qn[t] & 1u)) return;
            if (knew && !wait(KFULL + kslot, kph)) return;
            knew = false;
            tc_fence_after();
            const uint64_t a0 = dQ + static_cast<uint64_t>(t) * kTileStep, b0 = dK + static_cast<uint64_t>(kslot) * kTileStep;
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                const uint64_t o = static_cast<uint64_t>(((k >> 2) * HALF + (k & 3) * 32) >> 4);
                mma_ss_warp(tmem + t * 128, a0 + o, b0 + o, idS, k > 0 ? 1u : 0u);
            }
            mma_commit_warp(bar(SFULL + t));
            if (last) {
                mma_commit_warp(bar(QEMPTY + t));
                ++qn[t];
            }
            if (release) {
                mma_commit_warp(bar(KEMPTY + kslot));
                knew = true;
                if (++kslot == KST) {
                    kslot = 0;
                    kph ^= 1u;
                }
            }
        };
        bool has = walk.next(p, it);
        bool begun[2] = {false, false};       // the item's first S is already under way
        while (ok && has) {
            Item nx;
            const bool more = walk.next(p, nx);
            const int n0 = it.steps(0), n1 = it.steps(1);
            for (int t = 0; ok && t < 2; ++t)
                if (it.steps(t) > 0 && !begun[t]) issue_s(t, true, it.steps(t) == 1, !it.pair || t == 1);
            begun[0] = begun[1] = false;
            for (int j = 0; ok && j < n0; ++j) {
                for (int t = 0; ok && t < 2; ++t) {
                    const int nt = t ? n1 : n0;
                    if (j >= nt) continue;
                    if (vnew && !wait(VFULL + vslot, vph)) break;
                    vnew = false;
                    if (!wait(PFULL + t, pn[t] & 1u)) break;
                    ++pn[t];
                    tc_fence_after();
                    const uint64_t b0 = dV + static_cast<uint64_t>(vslot) * kTileStep;
#pragma unroll
                    for (int k = 0; k < BN / 16; ++k)
                        mma_ts_warp(tmem + 256 + t * 128, tmem + t * 128 + static_cast<uint32_t>(k) * 8u,
                                    b0 + static_cast<uint64_t>(k) * (2048u >> 4), idO, (j > 0 || k > 0) ? 1u : 0u);
                    if (j + 1 == nt) mma_commit_warp(bar(OFULL + t));
                    if (!it.pair || t == 1) {
                        mma_commit_warp(bar(VEMPTY + vslot));
                        vnew = true;
                        if (++vslot == VST) {
                            vslot = 0;
                            vph ^= 1u;
                        }
                    }
                    if (j + 1 < nt) {
                        issue_s(t, false, j + 2 == nt, !it.pair || t == 1);
                    } else if (more && nx.steps(t) > 0 && (t == 0 || begun[0])) {
                        issue_s(t, true, nx.steps(t) == 1, !nx.pair || t == 1);
                        begun[t] = true;
                    }
                }
            }
            it = nx;
            has = more;
        }
        if (!ok && lane == 0) give_up(abort_flag, p.err);
        mma_commit_warp(bar(MMADONE));        // every MMA completes before tensor memory is freed
        if (lane == 0) {
            volatile int never = 0;
            mbar_wait_bounded(bar(MMADONE), 0, tmo, &never);
        }
        __syncwarp();
    } else {
        // ---------------------------------------------------------------- softmax, thread = row
        // Beside the 128 scores a thread has few registers left: what the read-out needs of the item and
        // of the thread's place is worked out again there, and the barriers' phases are bits of one word.
        const int t = warp >> 2;
        uint32_t phases = 0;                   // 1: SFULL of the lane; 2, 4: OFULL of lanes 0, 1
        // a warp whose wait ran out still meets the others at every barrier of the items that are left
        while (walk.left > 0) {
            float m = -INFINITY, l = 0.f;
            {
                walk.peek(p, it);
                int left = p.n[it.b] - it.first(t) * BN;       // valid keys from the lane's next tile on
                int steps = it.steps(t);
                const uint32_t tS = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + t * 128;
                for (bool first = true; ok && steps > 0; --steps, left -= BN, first = false) {
                    ok = __all_sync(0xffffffffu, mbar_wait_bounded(bar(SFULL + t), phases & 1u, tmo, abort_flag));
                    if (!ok) break;
                    phases ^= 1u;
                    tc_fence_after();
                    softmax_step(tS, tS + 256, p.scale_log2, left, first, m, l);
                    tmem_wait_st();
                    tc_fence_before();
                    mbar_arrive(bar(PFULL + t));
                }
            }
            asm volatile("" : "+r"(walk.b), "+r"(walk.h0), "+r"(walk.tile), "+r"(walk.left));
            walk.next(p, it);
            const int n = p.n[it.b];
            int tid;
            asm volatile("mov.u32 %0, %%tid.x;" : "=r"(tid));
            const int row = tid & 127;
            const bool leader = row == 0;
            const int row_tok = p.pack == 1 ? row : row / p.pack;
            const uint32_t tO = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + 256;
            // Half a tile's output (64 dims) goes through shared memory: rows are written by their threads in
            // the swizzled layout (8 rows hit 8 different bank groups), and one TMA store writes whole sectors.
            // Writing rows of 256 bytes straight from their threads took 4500 cycles a tile pair.
            const uint32_t stage = sO + static_cast<uint32_t>(t) * HALF;
            auto stage_begin = [&]() {
                if (leader) tma_store_wait_read();
                lane_barrier(t);
            };
            auto stage_put = [&](int c, const uint32_t (&w)[16]) {     // 32 dims
                uint8_t* dst = smem + (stage - sQ) + row * 128;
#pragma unroll
                for (int v = 0; v < 4; ++v)
                    *reinterpret_cast<uint4*>(dst + (((c * 4 + v) ^ (row & 7)) << 4)) =
                        make_uint4(w[4 * v], w[4 * v + 1], w[4 * v + 2], w[4 * v + 3]);
            };
            auto stage_end = [&](int hf, int tok0) {
                fence_proxy_async();
                lane_barrier(t);
                if (leader) tma_store_4d(&p.omap, stage, hf * 64, it.h0, tok0, it.b);
            };
            // both accumulators of a single are read by both warpgroups
            for (int u = 0; u < 2; ++u) {
                if (it.steps(u) == 0) continue;
                if (ok && (u == t || !it.pair) && !mbar_wait_bounded(bar(OFULL + u), (phases >> (1 + u)) & 1u, tmo, abort_flag)) ok = false;
                phases ^= 2u << u;
            }
            // warp-uniform from here on: tensor-memory loads are warp-collective
            ok = __all_sync(0xffffffffu, ok);
            const int tok0 = (it.pair ? it.tile + t : it.tile) * p.tokens;
            const bool whole = it.pair || (n == 0 && t == 0);   // this warpgroup writes out a whole tile
            if (!ok) {
                give_up(abort_flag, p.err);
                if (whole) {
                    for (int i = 0; i < 4; ++i) lane_barrier(t);
                } else if (n > 0) {
                    softmax_barrier();
                    if (splits == 1) {
                        lane_barrier(t);
                        lane_barrier(t);
                    }
                    softmax_barrier();
                }
                continue;
            }
            tc_fence_after();
            const int64_t tok = static_cast<int64_t>(tok0) + row_tok;
            const bool live = row < used_rows && tok < p.Nq;
            const int64_t stat = (static_cast<int64_t>(it.b) * p.H + it.h0 + row - row_tok * p.pack) * p.Nq + tok;
            if (whole) {
                if (splits > 1 && cluster_ctarank() != 0) {   // a tile without keys: the cluster's first CTA writes it
                    for (int i = 0; i < 4; ++i) lane_barrier(t);
                    continue;
                }
                const float inv = 1.0f / l;
#pragma unroll 1
                for (int hf = 0; hf < 2; ++hf) {
                    // 64 dims are converted before the staging space is waited for
                    uint32_t out[2][16];
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t o[32];
                        tmem_ld_x32_sync(tO + t * 128 + hf * 64 + c * 32, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            out[c][i] = n > 0 ? bf16_pair(__uint_as_float(o[2 * i]) * inv, __uint_as_float(o[2 * i + 1]) * inv) : 0u;
                    }
                    stage_begin();
                    stage_put(0, out[0]);
                    stage_put(1, out[1]);
                    stage_end(hf, tok0);
                }
                if (p.lse && live) p.lse[stat] = n > 0 ? (m + __log2f(l)) * kLn2 : -INFINITY;
                continue;
            }
            if (n == 0) continue;
            // single: warpgroup t reads out dims [64t, 64t + 64) of both accumulators
            stats[t * BM + row] = make_float2(m, l);
            softmax_barrier();
            const float2 a = stats[row], b = stats[BM + row];
            const float M = a.y == 0.f ? b.x : (b.y == 0.f ? a.x : fmaxf(a.x, b.x));
            const float wa = weight_of(a, M), wb = weight_of(b, M);
            const float L = a.y * wa + b.y * wb;
            const bool two = it.steps(1) > 0, one = it.steps(0) > 0;   // a cluster's CTA may have no keys
            const float inv = splits > 1 ? 1.0f : 1.0f / L;
            if (splits == 1) stage_begin();
#pragma unroll 1
            for (int c = 2 * t; c < 2 * t + 2; ++c) {
                // a part without keys has whatever its columns held before, and counts as 0
                uint32_t o[32];
                float f[32];
                tmem_ld_x32_sync(tO + c * 32, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = one ? __uint_as_float(o[i]) * wa : 0.f;
                tmem_ld_x32_sync(tO + 128 + c * 32, o);
#pragma unroll
                for (int i = 0; i < 32; ++i) f[i] = (two ? fmaf(__uint_as_float(o[i]), wb, f[i]) : f[i]) * inv;
                if (splits > 1) {            // [dims / 4][row] so that a warp writes 512 contiguous bytes
                    float4* part = reinterpret_cast<float4*>(smem);
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        part[(c * 8 + v) * BM + row] = make_float4(f[4 * v], f[4 * v + 1], f[4 * v + 2], f[4 * v + 3]);
                } else {
                    uint32_t out[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) out[i] = bf16_pair(f[2 * i], f[2 * i + 1]);
                    stage_put(c & 1, out);
                }
            }
            if (splits == 1) stage_end(t, tok0);
            tc_fence_before();
            softmax_barrier();                 // both accumulators and the statistics have been read
            if (splits > 1) {
                if (t == 0) stats[row] = make_float2(M, L);
            } else if (t == 0 && live && p.lse) {
                p.lse[stat] = (M + __log2f(L)) * kLn2;
            }
        }
        if ((threadIdx.x & 127) == 0) tma_store_wait();
        __syncwarp();
    }
    if (splits > 1) {
        // join the parts of the cluster's CTAs: a thread keeps its row, the CTAs share the dims
        cluster_sync_all();
        Walk again(p);
        again.next(p, it);
        const int row = threadIdx.x & 127;
        const int64_t tok = static_cast<int64_t>(it.tile) * p.tokens + (p.pack == 1 ? row : row / p.pack);
        if (p.n[it.b] > 0 && row < used_rows && tok < p.Nq) {
            float2 ml[kMaxCluster];
            float M = -INFINITY, L = 0.f;
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c)
                if (c < splits) {
                    ml[c] = ld_cluster_f32x2(map_to_rank(smem_u32(&stats[row]), c));
                    if (ml[c].y != 0.f) M = fmaxf(M, ml[c].x);
                }
#pragma unroll
            for (int c = 0; c < kMaxCluster; ++c)
                if (c < splits) {
                    const float w = weight_of(ml[c], M);
                    L = fmaf(ml[c].y, w, L);
                    ml[c].x = w;
                }
            const float inv = 1.0f / L;
            const int rank = static_cast<int>(cluster_ctarank());
            const int h = it.h0 + (p.pack == 1 ? 0 : row % p.pack);
            uint16_t* dst = p.out + ((static_cast<int64_t>(it.b) * p.Nq + tok) * p.H + h) * HD;
#pragma unroll 2
            for (int d4 = rank * (NTHREADS / 128) + (threadIdx.x >> 7); d4 < HD / 4; d4 += splits * (NTHREADS / 128)) {
                float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
                for (int c = 0; c < kMaxCluster; ++c)
                    if (c < splits) {
                        const float4 o = ld_cluster_f32x4(map_to_rank(sQ + static_cast<uint32_t>(d4 * BM + row) * 16u, c));
                        const float w = ml[c].x;
                        acc.x = fmaf(o.x, w, acc.x);
                        acc.y = fmaf(o.y, w, acc.y);
                        acc.z = fmaf(o.z, w, acc.z);
                        acc.w = fmaf(o.w, w, acc.w);
                    }
                *reinterpret_cast<uint2*>(dst + d4 * 4) =
                    make_uint2(bf16_pair(acc.x * inv, acc.y * inv), bf16_pair(acc.z * inv, acc.w * inv));
            }
            if (rank == 0 && threadIdx.x < 128 && p.lse)
                p.lse[(static_cast<int64_t>(it.b) * p.H + h) * p.Nq + tok] = (M + __log2f(L)) * kLn2;
        }
        cluster_sync_all();                    // no CTA leaves while others read its memory
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

// How many clusters of each size a device holds at once (a cluster lies within one of the GPU's processing
// clusters, whose sizes differ: 152 SMs take 36 clusters of 4, but 23 of 6 and 7 of 16).
struct Placement {
    int clusters[kMaxCluster + 1] = {};
    template <typename K>
    cudaError_t ask(K kernel)
    {
        cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES));
        if (e == cudaSuccess) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
        for (int n = 2; e == cudaSuccess && n <= kMaxCluster; ++n) {
            cudaLaunchConfig_t cfg{};
            cfg.gridDim = dim3(static_cast<unsigned>(n));
            cfg.blockDim = dim3(NTHREADS);
            cfg.dynamicSmemBytes = SMEM_BYTES;
            cudaLaunchAttribute attr{};
            attr.id = cudaLaunchAttributeClusterDimension;
            attr.val.clusterDim.x = static_cast<unsigned>(n);
            attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
            cfg.attrs = &attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&clusters[n], kernel, &cfg);
            if (e == cudaErrorInvalidClusterSize) {            // a size that the device does not take
                cudaGetLastError();
                clusters[n] = 0;
                e = cudaSuccess;
            }
        }
        return e;
    }
};

template <int CAP>
cudaError_t launch(const CrossForward& f, int sms, cudaStream_t s)
{
    Params<CAP> p{};
    const CrossProblem& c = f.c;
    p.pack = cross_pack(c.H / c.Hk);
    p.tokens = BM / p.pack;
    p.tiles = (c.Nq + p.tokens - 1) / p.tokens;
    p.packs = c.H / p.pack;
    p.group = c.H / c.Hk;
    const CrossStrides dense = {int64_t(c.H) * HD, HD, int64_t(c.H) * HD * c.Nq};
    if (!encode_query_map(&p.qmap, c.q, c.H, c.Nq, c.B, c.qs, p.pack, p.tokens) ||
        !encode_query_map(&p.omap, f.out, c.H, c.Nq, c.B, dense, p.pack, p.tokens))
        return cudaErrorInvalidValue;
    int least = 1 << 30;                       // key tiles of the shortest stream that has any
    for (int b = 0; b < c.B; ++b) {
        p.n[b] = c.n[b];
        if (c.n[b] == 0) continue;
        least = std::min(least, (c.n[b] + BN - 1) / BN);
        if (!encode_key_map(&p.kmap[b], c.k + b * c.kvs.batch, c.Hk, c.n[b], c.kvs) ||
            !encode_key_map(&p.vmap[b], c.v + b * c.kvs.batch, c.Hk, c.n[b], c.kvs))
            return cudaErrorInvalidValue;
    }
    p.out = f.out;
    p.lse = f.lse;
    p.err = c.err;
    p.timeout_ns = c.timeout_ns;
    p.drop_tile = debug_drop_tile();
    p.B = c.B;
    p.H = c.H;
    p.Hk = c.Hk;
    p.Nq = c.Nq;
    p.scale_log2 = c.scale * kLog2e;
    const int64_t tiles = static_cast<int64_t>(p.tiles) * (c.H / p.pack) * c.B;
    if (tiles > INT32_MAX / kMaxCluster) return cudaErrorInvalidConfiguration;
    auto kernel = cross_attention_kernel<CAP>;
    static PerDevice asked;
    static Placement placements[64];
    int dev = 0;
    cudaGetDevice(&dev);
    Placement& fit = placements[dev & 63];
    const cudaError_t e = asked.run(dev, [&]() { return fit.ask(kernel); });
    if (e != cudaSuccess) return e;
    // A cluster shares a tile's keys, as wide as all tiles' clusters fit at once and every CTA has a key tile.
    int splits = 1;
    for (int c = 2; least != 1 << 30 && c <= std::min(least, kMaxCluster); ++c)
        if (tiles <= fit.clusters[c]) splits = c;
    p.splits = splits;
    const int ctas = static_cast<int>(std::min<int64_t>(tiles, std::min(sms, kMaxCtas)));
    if (splits == 1) {
        // ranges of equal cost; a query tile costs its key tiles, and one for its start and end
        const int64_t per_stream = static_cast<int64_t>(p.tiles) * p.packs;
        int64_t total = 0;
        for (int b = 0; b < c.B; ++b) total += ((c.n[b] + BN - 1) / BN + 1) * per_stream;
        int b = 0;
        int64_t before = 0;                    // cost of the streams before b
        for (int i = 0; i <= ctas; ++i) {
            const int64_t x = total * i / ctas;
            int64_t w = (c.n[b] + BN - 1) / BN + 1;
            while (x > before + w * per_stream && b + 1 < c.B) {
                before += w * per_stream;
                ++b;
                w = (c.n[b] + BN - 1) / BN + 1;
            }
            p.start[i] = static_cast<int32_t>(b * per_stream + (x - before + w - 1) / w);
        }
    }

    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(splits > 1 ? tiles * splits : ctas));
    cfg.blockDim = dim3(NTHREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cudaLaunchAttribute attrs[2] = {chained_attribute(), {}};
    attrs[1].id = cudaLaunchAttributeClusterDimension;
    attrs[1].val.clusterDim.x = static_cast<unsigned>(splits);
    attrs[1].val.clusterDim.y = attrs[1].val.clusterDim.z = 1;
    cfg.attrs = attrs;
    cfg.numAttrs = splits > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

bool encode_query_map(CUtensorMap* map, const void* base, int heads, int64_t tokens, int batch, const CrossStrides& st,
                      int heads_box, int tokens_box)
{
    const cuuint64_t dims[4] = {HD, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(tokens), static_cast<cuuint64_t>(batch)};
    const cuuint64_t strides[3] = {static_cast<cuuint64_t>(st.hd) * 2, static_cast<cuuint64_t>(st.tok) * 2,
                                   static_cast<cuuint64_t>(st.batch) * 2};
    const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(heads_box), static_cast<cuuint32_t>(tokens_box), 1};
    return encode_tensor_map(map, base, 4, dims, strides, box);
}

bool encode_key_map(CUtensorMap* map, const void* base, int heads, int64_t rows, const CrossStrides& st)
{
    const cuuint64_t dims[3] = {HD, static_cast<cuuint64_t>(heads), static_cast<cuuint64_t>(rows)};
    const cuuint64_t strides[2] = {static_cast<cuuint64_t>(st.hd) * 2, static_cast<cuuint64_t>(st.tok) * 2};
    const cuuint32_t box[3] = {64, 1, BN};
    return encode_tensor_map(map, base, 3, dims, strides, box);
}

int cross_pack(int group)
{
    for (int d = std::min(group, BM); d > 1; --d)
        if (group % d == 0) return d;
    return 1;
}

cudaError_t launch_cross_attention(const CrossForward& f, cudaStream_t s)
{
    int dev = 0, sms = 0;
    cudaGetDevice(&dev);
    cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    return f.c.B <= 4 ? launch<4>(f, sms, s) : launch<kCrossStreams>(f, sms, s);
}

}  // namespace sdv2
