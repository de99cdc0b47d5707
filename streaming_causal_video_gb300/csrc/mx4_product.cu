// Products of microscaled 4-bit matrices on the tensor cores: out[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]).
//
// Clusters of two CTAs on the two SMs of a TPC share each MMA (tcgen05.mma.cta_group::2.kind::mxf4, M = 256, N = 256, 64
// columns a step): a pair tile is 256 rows of a by 256 (or 192 or 128) rows of b; each CTA holds half of the rows of either and gets
// the sums of its 128 rows of a in its own tensor memory.  A ring stage is 256 columns: 128 bytes of codes of a row, so that the tiles in
// shared memory, their swizzle and their descriptors are those of 64 bf16 columns; with the scales 35 KB a CTA.  The scales lie
// in global memory as the tensor memory takes them and go there by tcgen05.cp, in front of the MMAs that use them: those of a
// CTA's own 128 rows of a, and those of all 256 rows of b, which both CTAs read.
//   warp 0: TMA producer (both CTAs load into their own shared memory and count the bytes on the leader's stage barrier, which
//   the leader arms for both); warp 1: in the leader, scale copies and MMAs, whose commits arrive on the barriers of both CTAs;
//   warps 2-17: epilogue, four per quarter of the tensor memory's lanes, thread = row of a, while the next tile's MMAs run; 64
//   bytes of a row at a time go through swizzled shared memory to a TMA store, or to coalesced stores where rows of out are not
//   whole 16 bytes.
// What bounds a deep product is the ring: a stage's memory comes round again after 1.4 us, its MMAs and the way of its next copies, so
// that five stages of 256 x 256 give one in 288 ns (four 340, six 280), where the MMAs take 262 (512 cycles) and shared memory, which
// they read while copies write it, little less.  4680 x 5120 of depth 20480 takes 127 us in bursts of 5 ms at 2070 MHz (7.7 PFLOP/s; the
// MMAs alone 105) and 142 back to back, where the power limit holds the SMs at 1620 to 1680 MHz; of depth 5120 39 us.  Shallow ones have the start and the end of tiles as well: 4680 x
// 6144 of depth 1536 takes 21.3 us to bf16, 23.4 with GELU and 27.1 to fp32; 4680 x 1536 of depth 1536 8.6.
// Where tiles are fewer than pairs, the depth is cut into two or four parts, one for each pair of a larger cluster.  Their sums are
// exchanged through shared memory when the ring is free, and each pair adds up and writes its share of the columns, in the order of
// the parts, so that results do not depend on which part ends first.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "cross_tma.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "mx4_maps.h"
#include "per_device.h"
#include "project.h"
#include "ptx.cuh"
#include "ptx_mx4.cuh"
#include "ptx_pair.cuh"
#include "tensor_map.h"

namespace sdv2 {
namespace {

constexpr int TM = 256, CM = TM / 2;           // rows of a in a pair tile and in each CTA
constexpr int STEP_TILES = 2;                  // scale tiles (128 columns) of a stage
constexpr int EPI_WARPS = 16;
constexpr int THREADS = 32 * (2 + EPI_WARPS);

// What depends on the rows of b in a pair tile.
template <int TN>
struct Tile {
    static constexpr int CN = TN / 2;                                  // rows of b in each CTA
    static constexpr int STAGES = TN == 256 ? 5 : TN == 192 ? 6 : 7;
    static constexpr int B_FULL = 0, B_EMPTY = STAGES, B_ACC_FULL = 2 * STAGES, B_ACC_EMPTY = 2 * STAGES + 2, B_SHARED = 2 * STAGES + 4,
                         B_DONE = 2 * STAGES + 5, NBARS = 2 * STAGES + 6;
    static constexpr uint32_t A_BYTES = CM * 128, B_BYTES = CN * 128;
    static constexpr int B_ROW_TILES = TN == 128 ? 1 : 2;              // scale tiles that these lie in
    static constexpr uint32_t AS_BYTES = STEP_TILES * 512, BS_BYTES = B_ROW_TILES * STEP_TILES * 512;
    static constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + AS_BYTES + BS_BYTES;
    static constexpr uint32_t STAGE_PITCH = (STAGE_BYTES + 1023) / 1024 * 1024;
    static constexpr uint32_t OUT_BYTES = 32 * 64;                     // a warp's staging of its rows
    static constexpr uint32_t OUT_OFF = STAGES * STAGE_PITCH;
    static constexpr uint32_t BIAS_OFF = OUT_OFF + EPI_WARPS * OUT_BYTES;
    static constexpr uint32_t BAR_OFF = BIAS_OFF + EPI_WARPS * 64 * 4;
    static constexpr uint32_t SMEM_BYTES = BAR_OFF + 256 + 1024;
    // Tensor memory: the sums of two tiles, and behind them the scales of a and of b of a step.  Two tiles of 256 columns do
    // not fit beside the scales: the second begins with the first's last 32.  The epilogue takes the shared columns of a tile
    // first, and the next tile begins when they are free, about 1300 cycles behind the last one's end; tiles of 192 columns
    // follow at once.
    static constexpr bool SHARES = TN == 256;
    // Columns that a warp of the epilogue takes: of 192 columns, one of the four groups has none in each tile, by turns.
    static constexpr int GROUP_COLS = TN == 128 ? 32 : 64;
    static constexpr uint32_t COL_SECOND = SHARES ? TN - 32 : TN;
    static constexpr uint32_t COL_AS = COL_SECOND + TN, COL_BS = COL_AS + 4 * STEP_TILES;
    static_assert(TN == 256 || TN == 192 || TN == 128, "rows of b from a multiple of 64 on, in two scale tiles, or a scale tile's");
    static_assert(COL_AS + 12 * STEP_TILES <= 512, "tensor memory");
    static_assert(A_BYTES % 1024 == 0 && B_BYTES % 1024 == 0 && OUT_OFF % 1024 == 0, "128-byte swizzle");
    static_assert(NBARS * 8 + 16 <= 256 && SMEM_BYTES <= 232448, "shared memory");
};
constexpr uint32_t TMEM_COLS = 512;

struct ProductParams {
    CUtensorMap a, as, b, bs, out;
    const float* bias;
    void* direct;                              // out, where rows are not whole 16 bytes, else null
    int64_t out_stride;
    uint32_t* err;
    uint64_t timeout_ns;
    int64_t drop;
    int32_t M, N, steps, splits, units;
    int32_t m_fastest, inner;                  // whether the tiles of a vary fastest, and how many there are
    int32_t step_i, step_j;                    // the grid's pairs in whole rows of them and the rest
    int32_t gelu;
};

// A pair's tiles and parts of the depth, one after the other.
struct Unit {
    int u, i, j;                               // place in the grid's inner and outer direction
    int m0, n0, split, first, last;            // the tile's first rows, the part of the depth and its steps
    __device__ __forceinline__ Unit(const ProductParams& p, int u_, int tn) : u(u_) { find(p, tn); }
    // The unit `pairs` places on: without divisions where the depth is whole, as these are in the way of the next MMAs.
    __device__ __forceinline__ void next(const ProductParams& p, int pairs, int tn)
    {
        u += pairs;
        if (p.splits == 1) {
            i += p.step_i;
            j += p.step_j;
            if (i >= p.inner) {
                i -= p.inner;
                ++j;
            }
            place(p, tn);
        } else {
            find(p, tn);
        }
    }

private:
    __device__ __forceinline__ void find(const ProductParams& p, int tn)
    {
        const int t = u / p.splits;
        split = u - t * p.splits;
        first = p.steps / p.splits * split + min(split, p.steps % p.splits);
        last = first + p.steps / p.splits + (split < p.steps % p.splits);
        j = t / p.inner;
        i = t - j * p.inner;
        place(p, tn);
    }
    __device__ __forceinline__ void place(const ProductParams& p, int tn)
    {
        m0 = (p.m_fastest ? i : j) * TM;
        n0 = (p.m_fastest ? j : i) * tn;
    }
};

__device__ __forceinline__ uint32_t pack2(float lo, float hi)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t pack2(uint64_t v)
{
    float lo, hi;
    f32x2_unpack(v, lo, hi);
    return pack2(lo, hi);
}

// Rows of out that TMA cannot write: a warp stores the 64 staged bytes of its rows number by number, a row (bf16) or two (fp32) at
// a time, with eight of them under way.
template <bool F32>
__device__ __forceinline__ void store_rows(const ProductParams& p, const uint8_t* stage, int row0, int n)
{
    constexpr int COLS = F32 ? 16 : 32, ROWS = 32 / COLS, PER = F32 ? 4 : 8;
    const int lane = threadIdx.x & 31, j = lane % COLS, first = lane / COLS;
    if (n + j >= p.N) return;
    const int rows = min(32, p.M - row0);
    const int64_t at = (row0 + first) * p.out_stride + n + j;
#pragma unroll 8
    for (int i = 0; i < 32 / ROWS; ++i) {
        const int r = first + i * ROWS;
        if (r >= rows) break;
        const uint8_t* from = stage + r * 64 + (((j / PER) ^ ((r >> 1) & 3)) << 4);
        const int64_t o = at + i * ROWS * p.out_stride;
        if constexpr (F32) static_cast<float*>(p.direct)[o] = reinterpret_cast<const float*>(from)[j % PER];
        else static_cast<uint16_t*>(p.direct)[o] = reinterpret_cast<const uint16_t*>(from)[j % PER];
    }
}

// A warp's way to out: PIECE columns of its 32 rows at a time, 64 bytes of a row, thread = row.
template <bool F32>
struct Epilogue {
    static constexpr int PIECE = F32 ? 16 : 32;
    const ProductParams& p;
    uint8_t* stage;                            // 2 KB, swizzled as TMA takes 64-byte rows
    float* bias;                               // of 64 columns

    __device__ __forceinline__ Epilogue(const ProductParams& p_, uint8_t* stage_, uint8_t* bias_)
        : p(p_), stage(stage_), bias(reinterpret_cast<float*>(bias_))
    {
    }

    // Brings the bias of columns n to n + 64, while their sums are still being formed.
    __device__ __forceinline__ void begin(int n)
    {
        if (!p.bias) return;
        const int lane = threadIdx.x & 31;
        __syncwarp();
        bias[lane] = n + lane < p.N ? p.bias[n + lane] : 0.0f;
        bias[32 + lane] = n + 32 + lane < p.N ? p.bias[n + 32 + lane] : 0.0f;
        __syncwarp();
    }

    // Columns n to n + PIECE of rows row0 to row0 + 32, of which there is one at least; column n is the c-th from begin's.
    __device__ __forceinline__ void write(const uint32_t (&y)[PIECE], int row0, int n, int c)
    {
        const int lane = threadIdx.x & 31;
        uint64_t v[PIECE / 2];
#pragma unroll
        for (int j = 0; j < PIECE / 2; ++j) v[j] = f32x2_pack(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]));
        if (p.bias) {
#pragma unroll
            for (int j = 0; j < PIECE / 4; ++j) {
                const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(bias + c + 4 * j);
                v[2 * j] = fadd2(v[2 * j], b4.x);
                v[2 * j + 1] = fadd2(v[2 * j + 1], b4.y);
            }
        }
        if (p.gelu) {
#pragma unroll
            for (int j = 0; j < PIECE / 2; ++j) v[j] = gelu2(v[j]);
        }
        if (lane == 0) tma_store_wait_read();
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            uint4 w;
            if constexpr (F32)
                w = make_uint4(static_cast<uint32_t>(v[2 * j]), static_cast<uint32_t>(v[2 * j] >> 32), static_cast<uint32_t>(v[2 * j + 1]),
                               static_cast<uint32_t>(v[2 * j + 1] >> 32));
            else
                w = make_uint4(pack2(v[4 * j]), pack2(v[4 * j + 1]), pack2(v[4 * j + 2]), pack2(v[4 * j + 3]));
            *reinterpret_cast<uint4*>(stage + lane * 64 + ((j ^ ((lane >> 1) & 3)) << 4)) = w;
        }
        if (!p.direct) {
            fence_proxy_async();
            __syncwarp();
            if (lane == 0) tma_store_3d(&p.out, smem_u32(stage), n, row0, 0);
        } else {
            __syncwarp();
            store_rows<F32>(p, stage, row0, n);
            __syncwarp();
        }
    }

    // The staged bytes have been read.  (The stores themselves end before the kernel does.)
    __device__ __forceinline__ void finish()
    {
        if ((threadIdx.x & 31) == 0) tma_store_wait_read();
        __syncwarp();
    }
};

// SPLIT: a cluster is p.splits pairs, which take the parts of the depth of one tile.
template <int TN, bool F32, bool SPLIT>
__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ ProductParams p)
{
    using T = Tile<TN>;
    constexpr uint32_t A_BYTES = T::A_BYTES, B_BYTES = T::B_BYTES, AS_BYTES = T::AS_BYTES, STAGE_BYTES = T::STAGE_BYTES;
    constexpr uint32_t COL_AS = T::COL_AS, COL_BS = T::COL_BS;
    constexpr int STAGES = T::STAGES, B_FULL = T::B_FULL, B_EMPTY = T::B_EMPTY, B_ACC_FULL = T::B_ACC_FULL,
                  B_ACC_EMPTY = T::B_ACC_EMPTY, B_SHARED = T::B_SHARED, B_DONE = T::B_DONE;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + T::BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + T::NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* peer_abort = abort_flag + 1;          // a CTA of the cluster gave up
    volatile int* peer_steps = abort_flag + 2;
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const int in_cluster = static_cast<int>(cluster_ctarank());
    const int rank = in_cluster & 1;                                 // 0: the pair's leader, which issues the MMAs
    const uint32_t leader = SPLIT ? static_cast<uint32_t>(in_cluster & ~1) : 0u;
    const uint16_t both = static_cast<uint16_t>(3u << leader);       // the pair's CTAs
    const int units = p.units;
    const int pair = SPLIT ? static_cast<int>(cluster_id_x()) * p.splits + (in_cluster >> 1) : static_cast<int>(cluster_id_x());
    const int pairs = SPLIT ? units : static_cast<int>(cluster_count_x());
    const uint64_t tmo = p.timeout_ns;

    if (threadIdx.x == 32) {
        tma_prefetch_desc(&p.a);
        tma_prefetch_desc(&p.b);
        tma_prefetch_desc(&p.as);
        tma_prefetch_desc(&p.bs);
    }
    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * STAGES; ++i) mbar_init(bar(i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_ACC_FULL + i), 1);
            mbar_init(bar(B_ACC_EMPTY + i), 2 * EPI_WARPS);
        }
        mbar_init(bar(B_SHARED), EPI_WARPS / 2);   // a quarter of the warps of each CTA
        mbar_init(bar(B_DONE), 1);
        *abort_flag = 0;
        *peer_abort = 0;
        *peer_steps = 0;
        fence_mbar_init();
    }
    if (warp == 1) {
        tmem_alloc_pair(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();          // both CTAs' barriers are initialised before either signals the other's
    tc_fence_after();
    constexpr uint32_t tmem = 0;                                     // of all 512 columns the first (what the allocation returns)
    wait_for_launch_before();
    launch_dependents();

    auto give_up = [&]() {
        *abort_flag = 1;
        atomicOr(p.err, kErrTimeout);
    };
    int issued = 0;              // the producer's steps
    if (warp == 0) {
        const uint32_t full_leader = map_to_rank(bar(B_FULL), leader);
        int st = 0;                                                  // the ring's stage and its phase
        uint32_t phase = 1;
        bool ok = true;
        for (Unit t(p, pair, TN); ok && t.u < units; t.next(p, pairs, TN)) {
            const int m0 = t.m0 + rank * CM, n0 = t.n0 + rank * T::CN;
            for (int k = t.first; k < t.last; ++k) {
                if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(B_EMPTY + st), phase, tmo, abort_flag))) {
                    if (lane == 0) give_up();
                    ok = false;
                    break;
                }
                const uint32_t sa = s0 + st * T::STAGE_PITCH;
                if (k != p.drop)
                    mx4_load_pair_warp(rank == 0, bar(B_FULL + st), 2 * STAGE_BYTES, full_leader + 8u * static_cast<uint32_t>(st), &p.a, &p.b, &p.as, &p.bs,
                                       sa, sa + A_BYTES, sa + A_BYTES + B_BYTES, sa + A_BYTES + B_BYTES + AS_BYTES, k * 128, m0, n0, k * STEP_TILES,
                                       m0 / 128, t.n0 / 128);
                else if (rank == 0 && lane == 0)
                    mbar_arrive_expect_tx(bar(B_FULL + st), 2 * STAGE_BYTES);
                ++issued;
                if (++st == STAGES) {
                    st = 0;
                    phase ^= 1u;
                }
            }
        }
        if (rank == 1 && lane == 0) st_cluster(map_to_rank(smem_u32(const_cast<int*>(peer_steps)), leader), issued);
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint64_t dA = sdesc_sw128(s0, 16, 1024);
            const uint64_t dB = sdesc_sw128(s0 + A_BYTES, 16, 1024);
            const uint64_t dAS = sdesc_scales(s0 + A_BYTES + B_BYTES);
            const uint64_t dBS = sdesc_scales(s0 + A_BYTES + B_BYTES + AS_BYTES);
            auto wait = [&](int i, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_bounded(bar(i), parity, tmo, abort_flag));
            };
            bool ok = true;
            int li = 0, st = 0;                                      // tiles so far; the ring's stage, its phase and its offset
            uint32_t phase = 0;
            uint64_t at = 0;
            for (Unit t(p, pair, TN); ok && t.u < units; t.next(p, pairs, TN), ++li) {
                const int buf = li & 1;
                // the tile before last has been read, and of the last one the columns that both use
                ok = wait(B_ACC_EMPTY + buf, (static_cast<uint32_t>(li >> 1) & 1u) ^ 1u) &&
                     (!T::SHARES || li == 0 || wait(B_SHARED, static_cast<uint32_t>(li - 1) & 1u));
                if (!ok) break;
                tc_fence_after();
                const uint32_t acc = tmem + (buf ? T::COL_SECOND : 0u);
                const uint32_t b_scales = tmem + COL_BS + static_cast<uint32_t>(t.n0 / 32 % 4);    // of the tile's first row
                for (int k = t.first; k < t.last; ++k) {
                    if (!wait(B_FULL + st, phase)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    mx4_stage_pair_warp<T::B_ROW_TILES>(acc, dA + at, dB + at, dAS + at, dBS + at, tmem + COL_AS, tmem + COL_BS, b_scales, idesc_mx4(TM, TN, 0),
                                        idesc_mx4(TM, TN, 1), k > t.first ? 1u : 0u);
                    mma_commit_pair_warp(bar(B_EMPTY + st), both);
                    at += T::STAGE_PITCH >> 4;
                    if (++st == STAGES) {
                        st = 0;
                        at = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) break;
                mma_commit_pair_warp(bar(B_ACC_FULL + buf), both);
            }
            if (!ok && lane == 0) give_up();
            mma_commit_pair_warp(bar(B_DONE), both);            // tensor memory is freed only behind the last MMA
        }
        if (lane == 0) {
            volatile int no_abort = 0;
            mbar_wait_cluster_bounded(bar(B_DONE), 0, tmo, &no_abort);
        }
        __syncwarp();
    } else {
        // Four warps per quarter.
        const int group = (warp - 2) >> 2, quarter = warp & 3;
        constexpr int PIECE = Epilogue<F32>::PIECE, GROUP = T::GROUP_COLS, PIECES = GROUP / PIECE;
        Epilogue<F32> out(p, smem + T::OUT_OFF + (warp - 2) * T::OUT_BYTES, smem + T::BIAS_OFF + (warp - 2) * 256);
        const uint32_t empty_leader = map_to_rank(bar(B_ACC_EMPTY), leader), shared_leader = map_to_rank(bar(B_SHARED), leader);
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        int li = 0;
        for (Unit t(p, pair, TN); t.u < units; t.next(p, pairs, TN), ++li) {
            const int buf = li & 1;
            const int place = TN == 192 ? (group + li) & 3 : group;
            const int row0 = t.m0 + rank * CM + quarter * 32, n0 = t.n0 + place * GROUP;
            const bool mine = (TN != 192 || place < 3) && row0 < p.M && n0 < p.N;
            if (!SPLIT && mine) out.begin(n0);
            const bool ok = mbar_wait_bounded(bar(B_ACC_FULL + buf), static_cast<uint32_t>(li >> 1) & 1u, tmo, abort_flag) && !*abort_flag;
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up();
                break;
            }
            tc_fence_after();
            if constexpr (SPLIT) continue;                           // the sums of the parts are added below
            // the arrivals order no memory but the loads of tensor memory before them
            auto arrive = [&](uint32_t at) {
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_cluster_relaxed(at);
            };
            // the first buffer's last columns and the second's first are the ones that both use
            const bool shared = T::SHARES && place == (buf ? 0 : 3);
            if (!mine) {
                if (shared) arrive(shared_leader);
                arrive(empty_leader + 8u * static_cast<uint32_t>(buf));
                continue;
            }
            const uint32_t trow = lanes + (buf ? T::COL_SECOND : 0u) + static_cast<uint32_t>(place * GROUP);
            const int flip = T::SHARES && buf == 0 ? PIECES - 1 : 0;
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                const int c = (i ^ flip) * PIECE;
                uint32_t y[PIECE];
                tmem_ld_cols(trow + c, y);
                if (shared && (i + 1) * PIECE == 32) arrive(shared_leader);
                if (i == PIECES - 1) arrive(empty_leader + 8u * static_cast<uint32_t>(buf));
                out.write(y, row0, n0 + c, c);
            }
        }
        if constexpr (!SPLIT) out.finish();
    }
    if constexpr (SPLIT) {
        // The parts' sums change hands through shared memory: pair s of the cluster adds up, in the order of the parts, and writes
        // the s-th of equal ranges of the tile's columns.  The ring is free when every pair's MMAs are done.
        tc_fence_before();
        __syncthreads();
        cluster_sync_all();
        tc_fence_after();
        const int parts = p.splits, own = in_cluster >> 1, width = TN / parts;
        const int quarter = warp & 3, group = (warp - 2) >> 2;
        const uint32_t lanes = tmem + (static_cast<uint32_t>(quarter * 32) << 16);
        const uint32_t my_row = static_cast<uint32_t>(quarter * 32 + lane) * 16;
        const bool sound = !*abort_flag;
        if (warp >= 2 && sound) {
            const Unit t(p, pair, TN);
            constexpr int GROUP = TN / 4;
            const int owner = group * GROUP / width;
            if (owner != own && t.m0 + rank * CM + quarter * 32 < p.M && t.n0 + group * GROUP < p.N) {
                // [part][four columns][row][column]: a warp stores 512 bytes together
                const uint32_t to = map_to_rank(s0, static_cast<uint32_t>(2 * owner + rank)) +
                                    static_cast<uint32_t>((own < owner ? own : own - 1) * width + group * GROUP % width) * (CM * 4) + my_row;
#pragma unroll
                for (int c = 0; c < GROUP; c += 32) {
                    uint32_t y[32];
                    tmem_ld_x32_sync(lanes + group * GROUP + c, y);
#pragma unroll
                    for (int j = 0; j < 32; j += 4) st_cluster_v4(to + static_cast<uint32_t>(c + j) * (CM * 4), y[j], y[j + 1], y[j + 2], y[j + 3]);
                }
            }
        }
        cluster_sync_all();
        if (warp >= 2 && sound) {
            constexpr int PIECE = Epilogue<F32>::PIECE;
            Epilogue<F32> out(p, smem + T::OUT_OFF + (warp - 2) * T::OUT_BYTES, smem + T::BIAS_OFF + (warp - 2) * 256);
            const Unit t(p, pair, TN);
            const int row0 = t.m0 + rank * CM + quarter * 32;
            for (int c = group * PIECE; c < width; c += 4 * PIECE) {
                const int n = t.n0 + own * width + c;
                if (row0 >= p.M || n >= p.N) continue;
                uint32_t mine[PIECE];
                tmem_ld_cols(lanes + own * width + c, mine);
                uint32_t y[PIECE] = {};
                for (int part = 0; part < parts; ++part) {
                    const uint8_t* from = smem + ((part < own ? part : part - 1) * width + c) * (CM * 4) + my_row;
#pragma unroll
                    for (int j = 0; j < PIECE; j += 4) {
                        uint4 v = make_uint4(mine[j], mine[j + 1], mine[j + 2], mine[j + 3]);
                        if (part != own) v = *reinterpret_cast<const uint4*>(from + j * (CM * 4));
                        y[j] = __float_as_uint(__uint_as_float(y[j]) + __uint_as_float(v.x));
                        y[j + 1] = __float_as_uint(__uint_as_float(y[j + 1]) + __uint_as_float(v.y));
                        y[j + 2] = __float_as_uint(__uint_as_float(y[j + 2]) + __uint_as_float(v.z));
                        y[j + 3] = __float_as_uint(__uint_as_float(y[j + 3]) + __uint_as_float(v.w));
                    }
                }
                out.begin(n);
                out.write(y, row0, n, 0);
            }
            out.finish();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x == 0 && *abort_flag)
        for (int c = 0; c < (SPLIT ? 2 * p.splits : 2); ++c) st_cluster(map_to_rank(smem_u32(const_cast<int*>(peer_abort)), static_cast<uint32_t>(c)), 1);
    cluster_sync_all();          // no CTA leaves while the other may still signal or read it
    if (*peer_abort) {
        // The ring's copies land before the pair may go.  A step that only one of the two CTAs issued is squared up: armed for the
        // peer's copies alone, or told that the peer's do not come.
        if (threadIdx.x == 0 && rank == 0) {
            const int mine = issued, peer = *peer_steps;
            for (int g = mine; g < peer; ++g) mbar_arrive_expect_tx(bar(B_FULL + g % STAGES), STAGE_BYTES);
            for (int g = peer; g < mine; ++g) mbar_complete_tx(bar(B_FULL + g % STAGES), STAGE_BYTES);
            const int end = max(mine, peer);
            volatile int no_abort = 0;
            for (int g = max(0, end - STAGES); g < end; ++g)
                mbar_wait_cluster_bounded(bar(B_FULL + g % STAGES), static_cast<uint32_t>(g / STAGES) & 1u, tmo, &no_abort);
        }
        __syncthreads();
        cluster_sync_all();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

constexpr int kPairs = 76;                     // a pair for each TPC's two SMs

// Results: boxes of 64 bytes x 32 rows.
bool out_map(CUtensorMap* map, const void* base, bool f32, int64_t M, int64_t N, int64_t stride)
{
    const cuuint64_t pitch = static_cast<cuuint64_t>(stride) * (f32 ? 4 : 2);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M), 1};
    const cuuint64_t strides[2] = {pitch, pitch * static_cast<cuuint64_t>(M)};
    const cuuint32_t box[3] = {f32 ? 16u : 32u, 32, 1};
    return encode_tensor_map_of(f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_64B,
                                map, base, 3, dims, strides, box);
}

template <int TN, bool F32, bool SPLIT>
cudaError_t launch(ProductParams& p, cudaStream_t s)
{
    constexpr uint32_t SMEM_BYTES = Tile<TN>::SMEM_BYTES;
    auto kernel = product_kernel<TN, F32, SPLIT>;
    cudaLaunchAttribute attr[2] = {chained_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = SPLIT ? 2 * p.splits : 2;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(2);
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = SMEM_BYTES;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    static PerDevice once;
    static int resident[64];                   // pairs that a device holds at once; written before `once` reports success
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    e = once.run(dev, [&]() -> cudaError_t {
        cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES));
        if (err == cudaSuccess && !SPLIT) err = cudaOccupancyMaxActiveClusters(&resident[dev & 63], kernel, &cfg);
        return err != cudaSuccess ? err : SPLIT || resident[dev & 63] > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
    });
    if (e != cudaSuccess) return e;
    const int pairs = SPLIT ? p.units : std::min(p.units, resident[dev & 63]);
    p.step_j = pairs / p.inner;
    p.step_i = pairs % p.inner;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * pairs));
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

bool mx4_codes_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int tiles, int box_rows)
{
    const cuuint64_t pitch = static_cast<cuuint64_t>(tiles) * kMx4TileBytes;
    const cuuint64_t dims[3] = {pitch, static_cast<cuuint64_t>(rows), 1}, strides[2] = {pitch, pitch * static_cast<cuuint64_t>(rows)};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_rows), 1};
    return encode_tensor_map_of(CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, map, base, 3, dims, strides, box);
}

bool mx4_scales_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int tiles, int box_tiles, int box_row_tiles)
{
    const cuuint64_t n = static_cast<cuuint64_t>((rows + kMx4Tile - 1) / kMx4Tile);
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(tiles), n}, strides[2] = {512, static_cast<cuuint64_t>(tiles) * 512};
    const cuuint32_t box[3] = {128, static_cast<cuuint32_t>(box_tiles), static_cast<cuuint32_t>(box_row_tiles)};
    return encode_tensor_map_of(CU_TENSOR_MAP_DATA_TYPE_UINT32, CU_TENSOR_MAP_SWIZZLE_NONE, map, base, 3, dims, strides, box);
}

// Rows of b in a tile, and parts of the depth, by an estimate of the time in nanoseconds: what a step and a tile were measured to
// take.  Tiles of fewer rows read more for the same work, but have less to wait for and fill the pairs evenly at other sizes; us with
// 256, 192 and 128 rows: 4680 x 5120 of depth 5120 39.1, 42.1 and 52.5, 4680 x 1536 of depth 1536 9.1, 8.5 and 9.6, 1536 x 1536 of depth
// 4680 11.6, 10.3 and 9.7.  Where even tiles of 128 rows are few, two or four pairs may share the depth of each (the GPU holds 36
// clusters of four CTAs and 15 of eight at once), if that saves more than the exchange of their sums from SM to SM, at 25 bytes a
// nanosecond, and what comes with it cost; us in one part, two and four: 512 x 512 of depth 8192 10.6, 9.6 and 9.0, of depth 4096 6.9, 7.5
// and 7.7; 512 x 1536 of depth 12288 14.1 and 12.0, of depth 4096 7.5 and 8.6; 1000 x 1000 of depth 8192 11.0 and 10.7.
Mx4Plan mx4_product_plan(int64_t M, int64_t N, int tiles)
{
    const int64_t mtiles = (M + TM - 1) / TM;
    const int steps = (tiles + STEP_TILES - 1) / STEP_TILES;
    Mx4Plan best{256, 1, 1};
    double least = 0;
    auto offer = [&](int tn, int parts, int64_t rounds, double time) {
        if (least == 0 || time < least) {
            least = time;
            best = {tn, parts, static_cast<int>(rounds)};
        }
    };
    constexpr struct {
        int tn;
        double step, tile;
    } kinds[] = {{256, 290, 1380}, {192, 225, 1000}, {128, 200, 750}};
    for (const auto& kind : kinds) {
        const int64_t rounds = (mtiles * ((N + kind.tn - 1) / kind.tn) + kPairs - 1) / kPairs;
        offer(kind.tn, 1, rounds, static_cast<double>(rounds) * (kind.step * steps + kind.tile));
    }
    const int64_t units = mtiles * ((N + 127) / 128);
    const double exchange = static_cast<double>(std::min<int64_t>(M, CM) * 128 * 4) / 25;     // of all sums
    if (units <= 36 && steps >= 2) offer(128, 2, 1, 200.0 * ((steps + 1) / 2) + 750 + 1500 + exchange / 2);
    if (units <= 15 && steps >= 4) offer(128, 4, 1, 200.0 * ((steps + 3) / 4) + 750 + 2200 + exchange * 3 / 4);
    return best;
}

cudaError_t launch_mx4_product(const Mx4Product& q, cudaStream_t s)
{
    ProductParams p{};
    p.M = static_cast<int32_t>(q.M);
    p.N = static_cast<int32_t>(q.N);
    const Mx4Plan plan = mx4_product_plan(q.M, q.N, q.tiles);
    const int32_t mtiles = static_cast<int32_t>((q.M + TM - 1) / TM), ntiles = static_cast<int32_t>((q.N + plan.width - 1) / plan.width);
    p.steps = (q.tiles + STEP_TILES - 1) / STEP_TILES;
    p.splits = plan.parts;
    p.bias = q.bias;
    p.gelu = q.gelu;
    p.err = q.err;
    p.timeout_ns = q.timeout_ns;
    p.drop = q.drop;
    p.out_stride = q.out_stride;
    // the operand with the fewer bytes is read again for every tile of the other
    p.m_fastest = q.N > q.M;
    p.inner = p.m_fastest ? mtiles : ntiles;
    p.units = mtiles * ntiles * p.splits;
    if (!mx4_codes_map(&p.a, q.a, q.M, q.tiles, CM) || !mx4_codes_map(&p.b, q.b, q.N, q.tiles, plan.width / 2) ||
        !mx4_scales_map(&p.as, q.as, q.M, q.tiles, STEP_TILES, 1) || !mx4_scales_map(&p.bs, q.bs, q.N, q.tiles, STEP_TILES, plan.width == 128 ? 1 : 2))
        return cudaErrorInvalidValue;
    const int64_t size = q.out_f32 ? 4 : 2, pitch = q.out_stride * size;
    // (a store's last 16 bytes of a row are written whole)
    if ((pitch | q.N * size) % 16 != 0 || pitch > (int64_t(1) << 39) / q.M) p.direct = q.out;
    else if (!out_map(&p.out, q.out, q.out_f32, q.M, q.N, q.out_stride)) return cudaErrorInvalidValue;
    if (p.splits > 1) return q.out_f32 ? launch<128, true, true>(p, s) : launch<128, false, true>(p, s);
    if (plan.width == 128) return q.out_f32 ? launch<128, true, false>(p, s) : launch<128, false, false>(p, s);
    if (plan.width == 256) return q.out_f32 ? launch<256, true, false>(p, s) : launch<256, false, false>(p, s);
    return q.out_f32 ? launch<192, true, false>(p, s) : launch<192, false, false>(p, s);
}

}  // namespace sdv2
