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
// A CTA walks a contiguous range of units, cut by cost.  Roles (12 warps):
//   warps 0-7 : thread = row and half of the 128 columns.  S is read out and turned into P as soon as
//               it is there, which frees it for the next step's S while dP is still computed; P and dS
//               then take dP's place as packed bf16, the A operands of the accumulating products.
//   warp 8: T tiles (2 stages); 10: R tiles (loaded while the unit before is read out); 9: MMA.
// Tensor memory: acc0 | acc1 | S | dP, 128 columns each.
#include <algorithm>
#include <atomic>

#include "cross_tma.cuh"
#include "internal.h"
#include "softmax_tile.cuh"

namespace sdv2 {
namespace {

constexpr int HD = 128, BM = 128;
constexpr int TST = 2;
constexpr uint32_t TILE = 128 * HD * 2;
constexpr uint32_t HALF = TILE / 2;
constexpr int T_WARP = 8, MMA_WARP = 9, R_WARP = 10;
constexpr int NTHREADS = 12 * 32;
constexpr uint32_t TMEM_COLS = 512;
constexpr uint32_t ACC0 = 0, ACC1 = 128, SCOL = 256, XCOL = 384;
constexpr float kLog2e = 1.4426950408889634f;
constexpr int kSms = 152;
constexpr int kMaxSplits = 8;

enum Bar { RFULL, REMPTY, TFULL, TEMPTY = TFULL + TST, SFULL = TEMPTY + TST, SREAD, DPFULL, DSFULL, ACCFULL, MMADONE, NBARS };

constexpr uint32_t SMEM_TILES = (2 + 2 * TST + 1) * TILE;      // R0 R1, (T0 T1) per stage, an output tile
constexpr uint32_t SMEM_STATS = 2 * 2 * BM * 4;                // dKV: lse and delta of a query tile, two steps
constexpr uint32_t SMEM_USED = SMEM_TILES + SMEM_STATS + 256;
constexpr uint32_t SMEM_BYTES = 232448;
static_assert(SMEM_USED + 768 <= SMEM_BYTES && NBARS * 8 + 8 <= 256, "shared memory layout");

template <int CAP>
struct Params {
    CUtensorMap qmap, domap, dqmap;            // query tiles: 4D, boxes of 64 dims x pack x tokens
    CUtensorMap kmap[CAP], vmap[CAP];          // per stream: valid rows
    CUtensorMap dkmap, dvmap;                  // (D, Hk, Nk, B): boxes of 64 dims x 1 x 128 rows
    int32_t n[CAP];
    const float* lse;                          // [B][H][Nq]
    const float* delta;
    float* part;                               // dKV: [split][unit][2][D/4][128][4]
    uint32_t* err;
    uint64_t timeout_ns;
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

__device__ __forceinline__ void compute_barrier() { asm volatile("bar.sync 1, 256;" ::: "memory"); }

template <bool DKV, int CAP>
__global__ void __launch_bounds__(NTHREADS, 1) cross_backward_kernel(const __grid_constant__ Params<CAP> p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if (static_cast<uint32_t>(smem - smem_raw) + SMEM_USED > SMEM_BYTES) {   // uniform: the base is the same for all
        if (threadIdx.x == 0) atomicOr(p.err, kErrTimeout);
        return;
    }
    const uint32_t sR = smem_u32(smem), sT = sR + 2 * TILE, sO = sT + 2 * TST * TILE;
    float* colstat = reinterpret_cast<float*>(smem + SMEM_TILES);           // [2][2][128]
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + SMEM_TILES + SMEM_STATS);
    const uint32_t bar0 = smem_u32(bars);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };

    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const uint64_t tmo = p.timeout_ns;
    const int used_rows = p.pack * p.tokens;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NBARS; ++i) mbar_init(bar(i), i == SREAD || i == DSFULL ? 256 : 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    // Rows of a query tile that no load writes (the pack does not divide 128) are zero: as streamed tiles
    // they are summed over, with probability 0.
    for (int i = threadIdx.x; i < (BM - used_rows) * 16 * (2 + 2 * TST); i += NTHREADS) {
        const int part = i & 15, r = i >> 4, tile = r / (BM - used_rows), row = used_rows + r - tile * (BM - used_rows);
        *reinterpret_cast<uint4*>(smem + tile * TILE + (part >> 3) * HALF + row * 128 + (part & 7) * 16) = make_uint4(0, 0, 0, 0);
    }
    fence_proxy_async();
    if (warp == MMA_WARP) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
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
            }
            if (!ok) give_up(abort_flag, p.err);
            volatile int never = 0;            // every copy lands before the CTA may exit
            if (units) mbar_wait_bounded(bar(RFULL), (units - 1) & 1u, tmo, &never);
        }
        __syncwarp();
    } else if (warp == T_WARP) {
        if (lane == 0) {
            uint32_t count = 0;
            while (ok && walk.next(p, u)) {
                int tile = 0, h0 = 0;          // dKV: query tile and first head of its pack
                if constexpr (DKV) {
                    const int pk = u.s0 / p.qtiles;
                    tile = u.s0 - pk * p.qtiles;
                    h0 = u.head * p.group + pk * p.pack;
                }
                const int hk = DKV ? 0 : u.head / p.group;
                for (int i = 0; i < u.steps; ++i, ++count) {
                    const int st = count & (TST - 1);
                    if (!mbar_wait_bounded(bar(TEMPTY + st), ((count / TST) & 1u) ^ 1u, tmo, abort_flag)) { ok = false; break; }
                    const uint32_t dst = sT + st * 2 * TILE;
                    if constexpr (DKV) {
                        mbar_arrive_expect_tx(bar(TFULL + st), 2 * query_bytes);
                        load_queries(&p.qmap, dst, TFULL + st, h0, tile * p.tokens, u.b);
                        load_queries(&p.domap, dst + TILE, TFULL + st, h0, tile * p.tokens, u.b);
                        if (++tile == p.qtiles) {
                            tile = 0;
                            h0 += p.pack;
                        }
                    } else {
                        mbar_arrive_expect_tx(bar(TFULL + st), 2 * TILE);
                        load_keys(&p.kmap[u.b], dst, TFULL + st, hk, i * BM);
                        load_keys(&p.vmap[u.b], dst + TILE, TFULL + st, hk, i * BM);
                    }
                }
            }
            if (!ok) give_up(abort_flag, p.err);
            volatile int never = 0;
            for (uint32_t k = 1; k <= TST && k <= count; ++k)
                mbar_wait_bounded(bar(TFULL + ((count - k) & (TST - 1))), ((count - k) / TST) & 1u, tmo, &never);
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
        auto product = [&](uint32_t d, uint32_t a, uint32_t b) {         // D = A B^T
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
                const uint32_t o = (k >> 2) * HALF + (k & 3) * 32;
                mma_ss_warp(tmem + d, desc(a + o, 16), desc(b + o, 16), idKK, k > 0 ? 1u : 0u);
            }
        };
        // D += A B with A = 128 packed columns written by the two column halves: their parts `a_off` into each half
        auto accumulate = [&](uint32_t d, uint32_t a_off, uint32_t b, bool add) {
#pragma unroll
            for (int k = 0; k < BM / 16; ++k)
                mma_ts_warp(tmem + d, tmem + XCOL + (k >> 2) * 64 + a_off + (k & 3) * 8, desc(b + k * 2048u, HALF), idKM,
                            (add || k > 0) ? 1u : 0u);
        };
        uint32_t count = 0, units = 0;         // steps, units begun
        auto stage = [&](uint32_t c) { return sT + (c & (TST - 1)) * 2 * TILE; };
        auto begin_s = [&](uint32_t c) {       // S of step c
            if (!wait(TFULL + (c & (TST - 1)), (c / TST) & 1u)) return;
            tc_fence_after();
            product(SCOL, sR, stage(c));
            mma_commit_warp(bar(SFULL));
        };
        auto begin_dp = [&](uint32_t c, bool last) {
            product(XCOL, sR + TILE, stage(c) + TILE);
            mma_commit_warp(bar(DPFULL));
            if (last) mma_commit_warp(bar(REMPTY));
        };
        while (ok && walk.next(p, u)) {
            if (u.steps == 0) continue;
            // the unit before has read its last S and written its last dS, so both score tiles are free
            if (!wait(RFULL, units & 1u)) break;
            ++units;
            begin_s(count);
            if (!ok) break;
            begin_dp(count, u.steps == 1);
            for (int i = 0; ok && i < u.steps; ++i, ++count) {
                const bool more = i + 1 < u.steps;
                if (more) {
                    if (!wait(SREAD, count & 1u)) break;
                    begin_s(count + 1);
                    if (!ok) break;
                }
                if (!wait(DSFULL, count & 1u)) break;
                tc_fence_after();
                if constexpr (DKV) accumulate(ACC1, 0, stage(count) + TILE, i > 0);      // dV += P^T dO
                accumulate(ACC0, 32, stage(count), i > 0);                               // dQ += dS K, dK += dS^T Q
                mma_commit_warp(bar(TEMPTY + (count & (TST - 1))));
                if (!more) mma_commit_warp(bar(ACCFULL));
                else begin_dp(count + 1, i + 2 == u.steps);
            }
        }
        if (!ok && lane == 0) give_up(abort_flag, p.err);
        mma_commit_warp(bar(MMADONE));         // every MMA completes before tensor memory is freed
        if (lane == 0) {
            volatile int never = 0;
            mbar_wait_bounded(bar(MMADONE), 0, tmo, &never);
        }
        __syncwarp();
    } else if (warp < 8) {
        // ---------------------------------------------------------------- P and dS, thread = (row, column half)
        const int half = warp >> 2;
        const int row = (warp & 3) * 32 + lane;
        const uint32_t tL = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        const bool leader = threadIdx.x == 0;
        uint32_t count = 0, units = 0;
        // lse (log2 units, so that padding rows have probability 0) and delta of row `r` of a query tile
        auto stat_index = [&](int b, int h0, int tok0, int r) {
            const int rt = p.pack == 1 ? r : r / p.pack;
            const int64_t tok = static_cast<int64_t>(tok0) + rt;
            return r < used_rows && tok < p.Nq ? (static_cast<int64_t>(b) * p.H + h0 + (r - rt * p.pack)) * p.Nq + tok : int64_t(-1);
        };
        while (walk.next(p, u)) {
            float lse2 = 0.f, delta = 0.f;     // dQ: of the thread's row
            int tile = 0, h0 = 0;              // dKV: query tile whose statistics come next
            float next_stat = 0.f;             // dKV: this thread's entry of the next step's statistics
            auto fetch = [&]() {
                const int64_t i = stat_index(u.b, h0, tile * p.tokens, threadIdx.x & 127);
                if (half == 0) next_stat = i >= 0 ? p.lse[i] * kLog2e : INFINITY;
                else next_stat = i >= 0 ? p.delta[i] : 0.f;
                if (++tile == p.qtiles) {
                    tile = 0;
                    h0 += p.pack;
                }
            };
            if (u.steps > 0) {
                if constexpr (DKV) {
                    const int pk = u.s0 / p.qtiles;
                    tile = u.s0 - pk * p.qtiles;
                    h0 = u.head * p.group + pk * p.pack;
                    fetch();
                } else {
                    const int64_t i = stat_index(u.b, u.head, u.tile * p.tokens, row);
                    lse2 = i >= 0 ? p.lse[i] * kLog2e : INFINITY;
                    delta = i >= 0 ? p.delta[i] : 0.f;
                }
            }
            const bool constant = DKV && p.n[u.b] == 1;           // a softmax over one key has no gradient
            // a thread whose wait ran out still runs through all steps, to meet the others at every barrier
            for (int i = 0; i < u.steps; ++i, ++count) {
                const float* cl = colstat + (count & 1u) * 2 * BM + half * 64;
                if constexpr (DKV) {
                    colstat[(count & 1u) * 2 * BM + half * BM + (threadIdx.x & 127)] = next_stat;
                    if (i + 1 < u.steps) fetch();
                    compute_barrier();
                }
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(SFULL), count & 1u, tmo, abort_flag));
                tc_fence_after();
                float pr[64];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t s[32];
                    tmem_ld_x32_sync(tL + SCOL + half * 64 + c * 32, s);
#pragma unroll
                    for (int e = 0; e < 32; ++e)
                        pr[c * 32 + e] = ex2_approx(fmaf(__uint_as_float(s[e]), p.scale_log2, DKV ? -cl[c * 32 + e] : -lse2));
                }
                tc_fence_before();
                mbar_arrive(bar(SREAD));
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(DPFULL), count & 1u, tmo, abort_flag));
                if (!ok) give_up(abort_flag, p.err);
                tc_fence_after();
                uint32_t ds[2][16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t d[32];
                    tmem_ld_x32_sync(tL + XCOL + half * 64 + c * 32, d);
#pragma unroll
                    for (int e = 0; e < 16; ++e) {
                        float a = __uint_as_float(d[2 * e]) - (DKV ? cl[BM + c * 32 + 2 * e] : delta);
                        float b = __uint_as_float(d[2 * e + 1]) - (DKV ? cl[BM + c * 32 + 2 * e + 1] : delta);
                        a *= pr[c * 32 + 2 * e];
                        b *= pr[c * 32 + 2 * e + 1];
                        if (DKV && constant) a = b = 0.f;
                        ds[c][e] = bf16_pair(a, b);
                    }
                }
                if constexpr (DKV) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) {
                        uint32_t w[16];
#pragma unroll
                        for (int e = 0; e < 16; ++e) w[e] = bf16_pair(pr[c * 32 + 2 * e], pr[c * 32 + 2 * e + 1]);
                        tmem_st_x16(tL + XCOL + half * 64 + c * 16, w);
                    }
                }
                tmem_st_x16(tL + XCOL + half * 64 + 32, ds[0]);
                tmem_st_x16(tL + XCOL + half * 64 + 48, ds[1]);
                tmem_wait_st();
                tc_fence_before();
                mbar_arrive(bar(DSFULL));
            }
            // ------------------------------------------------------------ read out the accumulators
            if (u.steps > 0) {
                ok = ok && __all_sync(0xffffffffu, mbar_wait_bounded(bar(ACCFULL), units & 1u, tmo, abort_flag));
                ++units;
                tc_fence_after();
            }
            if (!ok) give_up(abort_flag, p.err);                   // and on, past every barrier, with whatever is there
            const bool zero = u.steps == 0 || (DKV && u.tile * BM + row >= p.n[u.b]);
            if (DKV && p.splits > 1) {
                float4* part = reinterpret_cast<float4*>(p.part) +
                               (u.split * p.units + u.index) * 2 * (HD / 4) * BM + row;
#pragma unroll 1
                for (int c = 0; c < 4; ++c) {                      // acc0 and acc1, this thread's 64 dims of each
                    uint32_t o[32];
                    tmem_ld_x32_sync(tL + (c >> 1) * 128 + half * 64 + (c & 1) * 32, o);
                    float4* dst = part + ((c >> 1) * (HD / 4) + half * 16 + (c & 1) * 8) * BM;
#pragma unroll
                    for (int v = 0; v < 8; ++v)
                        dst[v * BM] = zero ? make_float4(0.f, 0.f, 0.f, 0.f)
                                           : make_float4(__uint_as_float(o[4 * v]), __uint_as_float(o[4 * v + 1]),
                                                         __uint_as_float(o[4 * v + 2]), __uint_as_float(o[4 * v + 3]));
                }
                tc_fence_before();
                continue;
            }
#pragma unroll 1
            for (int acc = 0; acc < (DKV ? 2 : 1); ++acc) {
                const float f = acc == 0 ? p.scale : 1.0f;
                uint32_t w[2][16];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    uint32_t o[32];
                    tmem_ld_x32_sync(tL + acc * 128 + half * 64 + c * 32, o);
#pragma unroll
                    for (int e = 0; e < 16; ++e)
                        w[c][e] = zero ? 0u : bf16_pair(__uint_as_float(o[2 * e]) * f, __uint_as_float(o[2 * e + 1]) * f);
                }
                if (leader) tma_store_wait_read();                 // the staging tile is free
                compute_barrier();
                uint8_t* dst = smem + (sO - sR) + half * HALF + row * 128;
#pragma unroll
                for (int v = 0; v < 8; ++v)
                    *reinterpret_cast<uint4*>(dst + ((v ^ (row & 7)) << 4)) =
                        make_uint4(w[v >> 2][4 * (v & 3)], w[v >> 2][4 * (v & 3) + 1], w[v >> 2][4 * (v & 3) + 2],
                                   w[v >> 2][4 * (v & 3) + 3]);
                fence_proxy_async();
                compute_barrier();
                if (leader)
                    for (int hf = 0; hf < 2; ++hf) {
                        if constexpr (DKV)
                            tma_store_4d(acc == 0 ? &p.dkmap : &p.dvmap, sO + hf * HALF, hf * 64, u.head, u.tile * BM, u.b);
                        else
                            tma_store_4d(&p.dqmap, sO + hf * HALF, hf * 64, u.head, u.tile * p.tokens, u.b);
                    }
            }
            tc_fence_before();
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

// Adds the splits of a key tile's dK or dV in order.  grid: (units, 2); the tile is turned around in shared
// memory, because its parts lie [dims / 4][row].
__global__ void __launch_bounds__(256) cross_fold_kernel(const float4* __restrict__ part, int splits, int64_t units, int ktiles,
                                                         int Hk, int Nk, float scale, uint16_t* __restrict__ dk,
                                                         uint16_t* __restrict__ dv)
{
    __shared__ __align__(16) uint16_t tile[BM][HD + 8];
    const int64_t unit = blockIdx.x;
    const int which = blockIdx.y;
    for (int i = threadIdx.x; i < BM * (HD / 4); i += 256) {
        float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int k = 0; k < splits; ++k) {
            const float4 x = part[((k * units + unit) * 2 + which) * (BM * (HD / 4)) + i];
            s.x += x.x;
            s.y += x.y;
            s.z += x.z;
            s.w += x.w;
        }
        const float f = which == 0 ? scale : 1.0f;
        *reinterpret_cast<uint2*>(&tile[i & 127][(i >> 7) * 4]) = make_uint2(bf16_pair(s.x * f, s.y * f), bf16_pair(s.z * f, s.w * f));
    }
    __syncthreads();
    const int64_t bh = unit / ktiles;
    const int kt = static_cast<int>(unit - bh * ktiles);
    const int64_t b = bh / Hk;
    const int hk = static_cast<int>(bh - b * Hk);
    uint16_t* out = which == 0 ? dk : dv;
    for (int i = threadIdx.x; i < BM * 16; i += 256) {
        const int r = i >> 4, v = i & 15;
        const int64_t j = static_cast<int64_t>(kt) * BM + r;
        if (j < Nk)
            *reinterpret_cast<uint4*>(out + ((b * Nk + j) * Hk + hk) * HD + v * 8) = *reinterpret_cast<const uint4*>(&tile[r][v * 8]);
    }
}

struct Shape {
    int pack, tokens, qtiles, packs, group, ktiles, splits;
    int64_t kunits;                            // (stream, key head, key tile)
};

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
    // ranges of query tiles: the smallest estimated time, a unit costing its steps and four for its start, end and parts
    const int64_t steps = static_cast<int64_t>(s.qtiles) * (s.group / s.pack);
    s.splits = 1;
    int64_t best = INT64_MAX;
    for (int k = 1; k <= kMaxSplits && k <= steps; ++k) {
        const int64_t t = ((s.kunits * k + kSms - 1) / kSms) * ((steps + k - 1) / k + 4);
        if (t < best) {
            best = t;
            s.splits = k;
        }
    }
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
cudaError_t prepare_kernel(K kernel, std::atomic<uint64_t>& done)
{
    int dev = 0;
    cudaGetDevice(&dev);
    if (done.load() >> (dev & 63) & 1u) return cudaSuccess;
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES));
    if (e == cudaSuccess) done.fetch_or(uint64_t(1) << (dev & 63));
    return e;
}

template <int CAP>
cudaError_t launch(const CrossBackward& f, cudaStream_t s)
{
    const CrossProblem& c = f.c;
    const Shape sh = shape_of(c.B, c.H, c.Hk, c.Nq, c.Nk);
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
    p.lse = f.lse;
    p.delta = f.delta;
    p.part = f.part;
    p.err = c.err;
    p.timeout_ns = c.timeout_ns;
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

    cudaError_t e = launch_cross_delta(f, s);
    if (e != cudaSuccess) return e;
    static std::atomic<uint64_t> dq_set{0}, dkv_set{0};
    auto dq_kernel = cross_backward_kernel<false, CAP>;
    auto dkv_kernel = cross_backward_kernel<true, CAP>;
    if ((e = prepare_kernel(dq_kernel, dq_set)) != cudaSuccess || (e = prepare_kernel(dkv_kernel, dkv_set)) != cudaSuccess) return e;

    int ctas = static_cast<int>(std::min<int64_t>(qunits, kSms));
    cut(p.start, ctas, c.B, static_cast<int64_t>(sh.packs) * sh.qtiles, [&](int64_t b) { return c.n[b] > 1 ? (c.n[b] + BM - 1) / BM + int64_t(1) : 1; });
    dq_kernel<<<dim3(static_cast<unsigned>(ctas)), NTHREADS, SMEM_BYTES, s>>>(p);
    if (c.Nk == 0) return cudaGetLastError();
    // dKV: a run is a key tile's splits
    const int64_t all_steps = static_cast<int64_t>(sh.qtiles) * (sh.group / sh.pack);
    ctas = static_cast<int>(std::min<int64_t>(sh.kunits * sh.splits, kSms));
    cut(p.start, ctas, sh.kunits, sh.splits, [&](int64_t r) {
        const int64_t b = r / (static_cast<int64_t>(c.Hk) * sh.ktiles);
        return (r % sh.ktiles) * BM < c.n[b] ? (all_steps + sh.splits - 1) / sh.splits + 4 : int64_t(1);
    });
    p.units = sh.kunits;
    dkv_kernel<<<dim3(static_cast<unsigned>(ctas)), NTHREADS, SMEM_BYTES, s>>>(p);
    if (sh.splits > 1)
        cross_fold_kernel<<<dim3(static_cast<unsigned>(sh.kunits), 2), 256, 0, s>>>(reinterpret_cast<const float4*>(f.part), sh.splits,
                                                                                    sh.kunits, sh.ktiles, c.Hk, c.Nk, c.scale,
                                                                                    f.dk, f.dv);
    return cudaGetLastError();
}

}  // namespace

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
