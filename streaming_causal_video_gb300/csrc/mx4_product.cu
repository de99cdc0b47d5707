// Products of microscaled 4-bit matrices on the tensor cores: out[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]).
//
// Clusters of two CTAs on the two SMs of a TPC share each MMA (tcgen05.mma.cta_group::2.kind::mxf4, M = 256, N = 256, 64
// columns a step): a pair tile is 256 rows of a by 256 rows of b; each CTA holds 128 rows of either and gets the sums of its
// 128 rows of a in its own tensor memory.  A ring stage is 256 columns: 128 bytes of codes of a row, so that the tiles in
// shared memory, their swizzle and their descriptors are those of 64 bf16 columns; with the scales 35 KB a CTA.  The scales lie
// in global memory as the tensor memory takes them and go there by tcgen05.cp, in front of the MMAs that use them: those of a
// CTA's own 128 rows of a, and those of all 256 rows of b, which both CTAs read.
//   warp 0: TMA producer (both CTAs load into their own shared memory and count the bytes on the leader's stage barrier, which
//   the leader arms for both); warp 1: in the leader, scale copies and MMAs, whose commits arrive on the barriers of both CTAs;
//   warps 2-9: epilogue, two per quarter of the tensor memory's lanes, thread = row of a, while the next tile's MMAs run; 128 bytes of a row at a time go
//   through swizzled shared memory to a TMA store, or to coalesced stores where rows of out are not whole 16 bytes.
// Where tiles are fewer than pairs, the depth is cut into parts; their sums go to the workspace in fp32 and a second kernel adds
// them in order, so that results do not depend on which part ends first.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "cross_tma.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "per_device.h"
#include "project.h"
#include "ptx.cuh"
#include "ptx_mx4.cuh"
#include "ptx_pair.cuh"
#include "tensor_map.h"

namespace sdv2 {
namespace {

constexpr int TM = 256, TN = 256;              // rows of a and of b in a pair tile
constexpr int CM = TM / 2, CN = TN / 2;        // and in each CTA
constexpr int STEP_TILES = 2;                  // scale tiles (128 columns) of a stage
constexpr int STAGES = 5;
constexpr uint32_t A_BYTES = CM * 128, B_BYTES = CN * 128;
constexpr uint32_t AS_BYTES = STEP_TILES * 512, BS_BYTES = 2 * STEP_TILES * 512;
constexpr uint32_t STAGE_BYTES = A_BYTES + B_BYTES + AS_BYTES + BS_BYTES;
constexpr int EPI_WARPS = 8;
constexpr int THREADS = 32 * (2 + EPI_WARPS);
constexpr uint32_t OUT_BYTES = 32 * 128;       // a warp's staging of its rows
// Tensor memory: the sums of two tiles, the second's 256 columns beginning with the first's last 32, and behind them the scales of
// a and of b.  The epilogue takes the shared columns of a tile first, and the next tile begins when they are free.
constexpr uint32_t COL_SECOND = TN - 32, COL_AS = COL_SECOND + TN, COL_BS = COL_AS + 4 * STEP_TILES, TMEM_COLS = 512;
static_assert(COL_BS + 8 * STEP_TILES <= TMEM_COLS, "tensor memory");
constexpr int B_FULL = 0, B_EMPTY = STAGES, B_ACC_FULL = 2 * STAGES, B_ACC_EMPTY = 2 * STAGES + 2, B_SHARED = 2 * STAGES + 4,
              B_DONE = 2 * STAGES + 5, NBARS = 2 * STAGES + 6;
constexpr uint32_t OUT_OFF = STAGES * STAGE_BYTES;
constexpr uint32_t BIAS_OFF = OUT_OFF + EPI_WARPS * OUT_BYTES;
constexpr uint32_t BAR_OFF = BIAS_OFF + EPI_WARPS * (TN / 2) * 4;
constexpr uint32_t SMEM_BYTES = BAR_OFF + 256 + 1024;
constexpr uint16_t kBothCtas = 3;
static_assert(STAGE_BYTES % 1024 == 0 && A_BYTES % 1024 == 0 && OUT_OFF % 1024 == 0, "128-byte swizzle");
static_assert(NBARS * 8 + 16 <= 256 && SMEM_BYTES <= 232448, "shared memory");

struct ProductParams {
    CUtensorMap a, as, b, bs, out;             // out: the result, or partial sums
    const float* bias;
    void* direct;                              // out, where rows are not whole 16 bytes, else null
    int64_t out_stride;
    uint32_t* err;
    uint64_t timeout_ns;
    int64_t drop;
    int32_t M, N, mtiles, ntiles, steps, splits;
    int32_t m_fastest, gelu;
};

struct Unit {
    int m0, n0, split, first, last;            // tile's first rows, part of the depth and its steps
    __device__ __forceinline__ Unit(const ProductParams& p, int u)
    {
        const int t = u / p.splits;
        split = u - t * p.splits;
        first = static_cast<int>(static_cast<int64_t>(p.steps) * split / p.splits);
        last = static_cast<int>(static_cast<int64_t>(p.steps) * (split + 1) / p.splits);
        const int j = t / (p.m_fastest ? p.mtiles : p.ntiles);
        const int i = t - j * (p.m_fastest ? p.mtiles : p.ntiles);
        m0 = (p.m_fastest ? i : j) * TM;
        n0 = (p.m_fastest ? j : i) * TN;
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

// Rows of out that TMA cannot write: a warp stores a row's 128 staged bytes number by number.
template <bool F32>
__device__ __noinline__ void store_rows(const ProductParams& p, const uint8_t* stage, int row0, int n)
{
    const int lane = threadIdx.x & 31, rows = min(32, p.M - row0);
    constexpr int PER = F32 ? 4 : 8;
    for (int r = 0; r < rows; ++r)
        for (int j = lane; j < 8 * PER; j += 32) {
            if (n + j >= p.N) continue;
            const uint8_t* at = stage + r * 128 + (((j / PER) ^ (r & 7)) << 4);
            const int64_t o = (row0 + r) * p.out_stride + n + j;
            if constexpr (F32) static_cast<float*>(p.direct)[o] = reinterpret_cast<const float*>(at)[j % PER];
            else static_cast<uint16_t*>(p.direct)[o] = reinterpret_cast<const uint16_t*>(at)[j % PER];
        }
}

template <bool F32>
__global__ void __launch_bounds__(THREADS, 1) product_kernel(const __grid_constant__ ProductParams p)
{
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile int* peer_steps = abort_flag + 1;
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const int rank = static_cast<int>(cluster_ctarank());            // 0: the leader, which issues the MMAs
    const int pair = static_cast<int>(cluster_id_x()), pairs = static_cast<int>(cluster_count_x());
    const int units = p.mtiles * p.ntiles * p.splits;
    const uint64_t tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < 2 * STAGES; ++i) mbar_init(bar(i), 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(bar(B_ACC_FULL + i), 1);
            mbar_init(bar(B_ACC_EMPTY + i), 2 * EPI_WARPS);
        }
        mbar_init(bar(B_SHARED), EPI_WARPS);       // half of the warps of each CTA
        mbar_init(bar(B_DONE), 1);
        *abort_flag = 0;
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
    const uint32_t tmem = *tmem_slot;
    wait_for_launch_before();

    auto give_up = [&]() {
        *abort_flag = 1;
        atomicOr(p.err, kErrTimeout);
    };
    int issued = 0;              // the producer's steps
    if (warp == 0) {
        if (lane == 0) {
            tma_prefetch_desc(&p.a);
            tma_prefetch_desc(&p.b);
            const uint32_t full_leader = map_to_rank(bar(B_FULL), 0);
            bool ok = true;
            for (int u = pair; ok && u < units; u += pairs) {
                const Unit t(p, u);
                const int m0 = t.m0 + rank * CM, n0 = t.n0 + rank * CN;
                for (int k = t.first; k < t.last; ++k) {
                    const int st = issued % STAGES;
                    if (!mbar_wait_cluster_bounded(bar(B_EMPTY + st), (static_cast<uint32_t>(issued / STAGES) & 1u) ^ 1u, tmo, abort_flag)) {
                        give_up();
                        ok = false;
                        break;
                    }
                    const uint32_t sa = s0 + st * STAGE_BYTES, fb = full_leader + 8u * static_cast<uint32_t>(st);
                    if (rank == 0) mbar_arrive_expect_tx(bar(B_FULL + st), 2 * STAGE_BYTES);
                    ++issued;
                    if (k == p.drop) continue;
                    tma_load_3d_pair(sa, &p.a, fb, k * 128, m0, 0);
                    tma_load_3d_pair(sa + A_BYTES, &p.b, fb, k * 128, n0, 0);
                    tma_load_3d_pair(sa + A_BYTES + B_BYTES, &p.as, fb, 0, k * STEP_TILES, m0 / 128);
                    tma_load_3d_pair(sa + A_BYTES + B_BYTES + AS_BYTES, &p.bs, fb, 0, k * STEP_TILES, t.n0 / 128);
                }
            }
            if (rank == 1) st_cluster(map_to_rank(smem_u32(const_cast<int*>(peer_steps)), 0), issued);
        }
        __syncwarp();
    } else if (warp == 1) {
        if (rank == 0) {
            const uint64_t dA = sdesc_sw128(s0, 16, 1024);
            const uint64_t dB = sdesc_sw128(s0 + A_BYTES, 16, 1024);
            const uint64_t dAS = sdesc_scales(s0 + A_BYTES + B_BYTES);
            const uint64_t dBS = sdesc_scales(s0 + A_BYTES + B_BYTES + AS_BYTES);
            auto wait = [&](int i, uint32_t parity) -> bool {
                return __all_sync(0xffffffffu, mbar_wait_cluster_bounded(bar(i), parity, tmo, abort_flag));
            };
            bool ok = true;
            int g = 0, li = 0;
            for (int u = pair; ok && u < units; u += pairs, ++li) {
                const Unit t(p, u);
                const int buf = li & 1;
                // the tile before last has been read, and of the last one the columns that both use
                if (!wait(B_ACC_EMPTY + buf, (static_cast<uint32_t>(li >> 1) & 1u) ^ 1u) ||
                    (li > 0 && !wait(B_SHARED, static_cast<uint32_t>(li - 1) & 1u))) {
                    ok = false;
                    break;
                }
                tc_fence_after();
                const uint32_t acc = tmem + (buf ? COL_SECOND : 0u);
                for (int k = t.first; k < t.last; ++k, ++g) {
                    const int st = g % STAGES;
                    if (!wait(B_FULL + st, static_cast<uint32_t>(g / STAGES) & 1u)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after();
                    const uint64_t at = static_cast<uint64_t>(st) * (STAGE_BYTES >> 4);
#pragma unroll
                    for (int c = 0; c < STEP_TILES; ++c) {
                        scales_to_tmem_pair_warp(tmem + COL_AS + 4 * c, dAS + at + c * 32);
                        scales_to_tmem_pair_warp(tmem + COL_BS + 8 * c, dBS + at + c * 32);
                        scales_to_tmem_pair_warp(tmem + COL_BS + 8 * c + 4, dBS + at + (STEP_TILES + c) * 32);
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        mma_mx4_pair_warp(acc, dA + at + 2 * i, dB + at + 2 * i, (i & 1) ? idesc_mx4(TM, TN, 1) : idesc_mx4(TM, TN, 0),
                                          tmem + COL_AS + 4 * (i >> 1), tmem + COL_BS + 8 * (i >> 1), (k > t.first || i > 0) ? 1u : 0u);
                    mma_commit_pair_warp(bar(B_EMPTY + st), kBothCtas);
                }
                if (!ok) break;
                mma_commit_pair_warp(bar(B_ACC_FULL + buf), kBothCtas);
            }
            if (!ok && lane == 0) give_up();
            mma_commit_pair_warp(bar(B_DONE), kBothCtas);            // tensor memory is freed only behind the last MMA
        }
        if (lane == 0) {
            volatile int no_abort = 0;
            mbar_wait_cluster_bounded(bar(B_DONE), 0, tmo, &no_abort);
        }
        __syncwarp();
    } else {
        const int part = (warp - 2) >> 2, quarter = warp & 3;
        const int col0 = part * (TN / 2);
        constexpr int PIECE = 32, PIECES = TN / 2 / PIECE;           // columns that a thread has at once
        constexpr int TOGETHER = F32 ? 1 : 2;                        // pieces that make 128 bytes
        uint8_t* stage = smem + OUT_OFF + (warp - 2) * OUT_BYTES;
        float* bias = reinterpret_cast<float*>(smem + BIAS_OFF) + (warp - 2) * (TN / 2);
        const uint32_t empty_leader = map_to_rank(bar(B_ACC_EMPTY), 0), shared_leader = map_to_rank(bar(B_SHARED), 0);
        const bool whole = p.splits == 1;                            // else partial sums
        int li = 0;
        for (int u = pair; u < units; u += pairs, ++li) {
            const Unit t(p, u);
            const int buf = li & 1;
            const int row0 = t.m0 + rank * CM + quarter * 32;
#pragma unroll
            for (int j = 0; j < TN / 2 / 32; ++j) {
                const int n = t.n0 + col0 + j * 32 + lane;
                bias[j * 32 + lane] = whole && p.bias && n < p.N ? p.bias[n] : 0.0f;
            }
            __syncwarp();
            const bool ok = mbar_wait_cluster_bounded(bar(B_ACC_FULL + buf), static_cast<uint32_t>(li >> 1) & 1u, tmo, abort_flag) && !*abort_flag;
            if (!__all_sync(0xffffffffu, ok)) {
                if (lane == 0) give_up();
                break;
            }
            tc_fence_after();
            const uint32_t trow = tmem + (static_cast<uint32_t>(quarter * 32) << 16) + static_cast<uint32_t>(col0) + (buf ? COL_SECOND : 0u);
            // the first buffer backwards: its last columns are the ones that the second shares
            const int flip = buf ? 0 : PIECES - 1;
            uint32_t raw[2][PIECE];
            tmem_ld_x32_start(trow + (0 ^ flip) * PIECE, raw[0]);
#pragma unroll
            for (int i = 0; i < PIECES; ++i) {
                uint32_t(&y)[PIECE] = raw[i & 1];
                tmem_ld_x32_finish(y);
                if (i == 0 && part != buf) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(shared_leader);
                }
                if (i + 1 < PIECES) {
                    tmem_ld_x32_start(trow + ((i + 1) ^ flip) * PIECE, raw[(i + 1) & 1]);
                } else {                                             // all sums have been read; the arrival orders no memory
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_cluster_relaxed(empty_leader + 8u * static_cast<uint32_t>(buf));
                }
                const int c = (i ^ flip) * PIECE;
                uint64_t v[PIECE / 2];
#pragma unroll
                for (int j = 0; j < PIECE; j += 4) {
                    const ulonglong2 b4 = *reinterpret_cast<const ulonglong2*>(bias + c + j);
                    v[j / 2] = fadd2(f32x2_pack(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), b4.x);
                    v[j / 2 + 1] = fadd2(f32x2_pack(__uint_as_float(y[j + 2]), __uint_as_float(y[j + 3])), b4.y);
                }
                if (whole && p.gelu) {
#pragma unroll
                    for (int j = 0; j < PIECE / 2; ++j) v[j] = gelu2(v[j]);
                }
                if (i % TOGETHER == 0) {
                    if (lane == 0) tma_store_wait_read();
                    __syncwarp();
                }
                // 16-byte vectors of a row of 128 bytes, swizzled as TMA takes them
#pragma unroll
                for (int j = 0; j < 8 / TOGETHER; ++j) {
                    uint4 w;
                    if constexpr (F32) {
                        w = make_uint4(static_cast<uint32_t>(v[2 * j]), static_cast<uint32_t>(v[2 * j] >> 32),
                                       static_cast<uint32_t>(v[2 * j + 1]), static_cast<uint32_t>(v[2 * j + 1] >> 32));
                    } else {
                        w = make_uint4(pack2(v[4 * j]), pack2(v[4 * j + 1]), pack2(v[4 * j + 2]), pack2(v[4 * j + 3]));
                    }
                    const int at = F32 ? j : j + 4 * ((i ^ flip) & 1);
                    *reinterpret_cast<uint4*>(stage + lane * 128 + ((at ^ (lane & 7)) << 4)) = w;
                }
                if (i % TOGETHER != TOGETHER - 1) continue;
                const int n = t.n0 + col0 + (F32 ? c : c & ~63);
                if (!p.direct) {
                    fence_proxy_async();
                    __syncwarp();
                    if (lane == 0 && row0 < p.M && n < p.N) tma_store_3d(&p.out, smem_u32(stage), n, row0, t.split);
                } else {
                    __syncwarp();
                    store_rows<F32>(p, stage, row0, n);
                    __syncwarp();
                }
            }
        }
        if (lane == 0) tma_store_wait();
        __syncwarp();
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync_all();          // no CTA leaves while the other may still signal or read it
    if (threadIdx.x == 0 && rank == 0 && *abort_flag) {
        // The ring's copies land before the pair may go.  A step that only one of the two CTAs issued is squared up: armed for the
        // peer's copies alone, or told that the peer's do not come.
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
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc_pair(tmem, TMEM_COLS);
    }
}

// Adds the parts of the depth in order, then bias, activation and the rounding of out.
template <bool F32>
__global__ void __launch_bounds__(256) join_kernel(const float* part, const float* bias, void* out, int64_t M, int N, int64_t stride,
                                                   int64_t part_stride, int splits, int gelu_too, int vectors)
{
    wait_for_launch_before();
    const int64_t quads = part_stride / 4;
    const int64_t i = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
    if (i >= M * quads) return;
    const int64_t m = i / quads;
    const int n = static_cast<int>(i - m * quads) * 4;
    const float4* src = reinterpret_cast<const float4*>(part + m * part_stride + n);
    const int64_t step = M * quads;
    float y[4] = {};
#pragma unroll 4
    for (int s = 0; s < splits; ++s) {
        const float4 v = src[s * step];
        y[0] += v.x, y[1] += v.y, y[2] += v.z, y[3] += v.w;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= N) continue;
        if (bias) y[j] += bias[n + j];
        if (gelu_too) y[j] = gelu(y[j]);
    }
    const int64_t o = m * stride + n;
    if (vectors && n + 4 <= N) {
        if constexpr (F32) *reinterpret_cast<float4*>(static_cast<float*>(out) + o) = make_float4(y[0], y[1], y[2], y[3]);
        else *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + o) = make_uint2(pack2(y[0], y[1]), pack2(y[2], y[3]));
        return;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        if (n + j >= N) continue;
        if constexpr (F32) static_cast<float*>(out)[o + j] = y[j];
        else static_cast<__nv_bfloat16*>(out)[o + j] = __float2bfloat16_rn(y[j]);
    }
}

constexpr int kPairs = 76;                     // a pair for each TPC's two SMs

// Codes: boxes of 128 bytes x 128 rows.
bool codes_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int tiles)
{
    const cuuint64_t pitch = static_cast<cuuint64_t>(tiles) * kMx4TileBytes;
    const cuuint64_t dims[3] = {pitch, static_cast<cuuint64_t>(rows), 1}, strides[2] = {pitch, pitch * static_cast<cuuint64_t>(rows)};
    const cuuint32_t box[3] = {128, 128, 1};
    return encode_tensor_map_of(CU_TENSOR_MAP_DATA_TYPE_UINT8, CU_TENSOR_MAP_SWIZZLE_128B, map, base, 3, dims, strides, box);
}

// Scales: boxes of a tile's 128 words x two tiles x `row_tiles`; tiles past the matrix's arrive as zeros.
bool scales_map(CUtensorMap* map, const uint8_t* base, int64_t rows, int tiles, int row_tiles)
{
    const cuuint64_t n = static_cast<cuuint64_t>((rows + kMx4Tile - 1) / kMx4Tile);
    const cuuint64_t dims[3] = {128, static_cast<cuuint64_t>(tiles), n}, strides[2] = {512, static_cast<cuuint64_t>(tiles) * 512};
    const cuuint32_t box[3] = {128, STEP_TILES, static_cast<cuuint32_t>(row_tiles)};
    return encode_tensor_map_of(CU_TENSOR_MAP_DATA_TYPE_UINT32, CU_TENSOR_MAP_SWIZZLE_NONE, map, base, 3, dims, strides, box);
}

// Results or partial sums: boxes of 128 bytes x 32 rows.
bool out_map(CUtensorMap* map, const void* base, bool f32, int64_t M, int64_t N, int64_t stride, int splits)
{
    const cuuint64_t pitch = static_cast<cuuint64_t>(stride) * (f32 ? 4 : 2);
    const cuuint64_t dims[3] = {static_cast<cuuint64_t>(N), static_cast<cuuint64_t>(M), static_cast<cuuint64_t>(splits)};
    const cuuint64_t strides[2] = {pitch, pitch * static_cast<cuuint64_t>(M)};
    const cuuint32_t box[3] = {f32 ? 32u : 64u, 32, 1};
    return encode_tensor_map_of(f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, CU_TENSOR_MAP_SWIZZLE_128B,
                                map, base, 3, dims, strides, box);
}

template <bool F32>
cudaError_t launch(const ProductParams& p, cudaStream_t s)
{
    cudaLaunchAttribute attr[2] = {chained_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = 2;
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
        cudaError_t err = cudaFuncSetAttribute(product_kernel<F32>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(SMEM_BYTES));
        if (err == cudaSuccess) err = cudaOccupancyMaxActiveClusters(&resident[dev & 63], product_kernel<F32>, &cfg);
        return err != cudaSuccess ? err : resident[dev & 63] > 0 ? cudaSuccess : cudaErrorInvalidConfiguration;
    });
    if (e != cudaSuccess) return e;
    const int64_t units = static_cast<int64_t>(p.mtiles) * p.ntiles * p.splits;
    cfg.gridDim = dim3(static_cast<unsigned>(2 * std::min<int64_t>(units, resident[dev & 63])));
    return cudaLaunchKernelEx(&cfg, product_kernel<F32>, p);
}

}  // namespace

int mx4_splits(int64_t M, int64_t N, int tiles)
{
    const int64_t units = ((M + TM - 1) / TM) * ((N + TN - 1) / TN);
    const int steps = (tiles + STEP_TILES - 1) / STEP_TILES;
    const int s = static_cast<int>(std::min<int64_t>(kPairs / std::min<int64_t>(units, kPairs), std::max(1, steps / 2)));
    return steps - steps / s >= 12 ? s : 1;
}

cudaError_t launch_mx4_product(const Mx4Product& q, cudaStream_t s)
{
    ProductParams p{};
    p.M = static_cast<int32_t>(q.M);
    p.N = static_cast<int32_t>(q.N);
    p.mtiles = static_cast<int32_t>((q.M + TM - 1) / TM);
    p.ntiles = static_cast<int32_t>((q.N + TN - 1) / TN);
    p.steps = (q.tiles + STEP_TILES - 1) / STEP_TILES;
    p.splits = mx4_splits(q.M, q.N, q.tiles);
    p.bias = q.bias;
    p.gelu = q.gelu;
    p.err = q.err;
    p.timeout_ns = q.timeout_ns;
    p.drop = q.drop;
    p.out_stride = q.out_stride;
    // the operand with the fewer bytes is read again for every tile of the other
    p.m_fastest = q.N > q.M;
    const bool parts = p.splits > 1;
    const bool f32 = parts || q.out_f32;
    if (!codes_map(&p.a, q.a, q.M, q.tiles) || !codes_map(&p.b, q.b, q.N, q.tiles) || !scales_map(&p.as, q.as, q.M, q.tiles, 1) ||
        !scales_map(&p.bs, q.bs, q.N, q.tiles, 2))
        return cudaErrorInvalidValue;
    const int64_t stride = parts ? mx4_part_stride(q.N) : q.out_stride;
    const int64_t pitch = stride * (f32 ? 4 : 2);
    const int64_t width = parts ? stride : q.N;
    // (a store's last 16 bytes of a row are written whole)
    const bool boxes = (pitch | width * (f32 ? 4 : 2)) % 16 == 0 && pitch <= (int64_t(1) << 39) / q.M;
    if (!boxes) p.direct = q.out;
    else if (!out_map(&p.out, parts ? q.part : q.out, f32, q.M, width, stride, p.splits)) return cudaErrorInvalidValue;
    cudaError_t e = f32 ? launch<true>(p, s) : launch<false>(p, s);
    if (e != cudaSuccess || !parts) return e;
    const int64_t blocks = (q.M * (stride / 4) + 255) / 256;
    const int vectors = q.out_stride % 4 == 0;
    return launch_chained(q.out_f32 ? join_kernel<true> : join_kernel<false>, static_cast<unsigned>(blocks), 256, 0, s,
                          static_cast<const float*>(q.part), q.bias, q.out, q.M, static_cast<int>(q.N), q.out_stride, stride, p.splits, q.gelu,
                          vectors);
}

}  // namespace sdv2
