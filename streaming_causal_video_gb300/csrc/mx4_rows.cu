// Products of a few rows with a 4-bit matrix: out[m][n] = act(sum_k a[m][k] b[n][k] + bias[n]) for at most 64 rows of a.
//
// Every byte of b is read once and takes part in few operations, so that reading b bounds this, and at small sizes the latency of
// a launch.  The operands change places: 128 rows of b are the rows of a tcgen05 MMA (kind::mxf4, M = 128), and the rows of a its
// 16, 32 or 64 columns, so that an MMA takes a fraction of the time that its rows of b take to come.  (Decoding b on the CUDA cores
// for mma.sync was bound by that: 3 rows at 5120 x 20480 took 30 us.)  A CTA has four stages of 256 columns, 16 KB of b each, and two
// CTAs fit an SM: 3 rows at 5120 x 20480 take 12.3 us (4.5 TB/s), at 9216 x 1536 4.3.  Where rows of b are few, up to eight CTAs of a
// cluster share the depth; their sums change hands through shared memory, and each adds up, in the order of the parts, and writes
// its share of the rows of a.
//   warps 0-3: epilogue, thread = row of b: its sums lie in its lane of tensor memory, and a warp's stores of a row of out are
//   neighbours; warp 4: TMA producer; warp 5: scale copies and MMAs.
#include <cuda_bf16.h>

#include <algorithm>

#include "chained.cuh"
#include "internal.h"
#include "mx4.cuh"
#include "mx4_maps.h"
#include "per_device.h"
#include "project.h"
#include "ptx.cuh"
#include "ptx_mx4.cuh"
#include "ptx_pair.cuh"

namespace sdv2 {
namespace {

constexpr int ROWS = 128;                      // of b, of a CTA
constexpr int STEP_TILES = 2;                  // scale tiles (128 columns) of a stage
constexpr int STAGES = 4;
constexpr int B_FULL = 0, B_EMPTY = STAGES, B_DONE = 2 * STAGES, NBARS = 2 * STAGES + 1;
constexpr uint32_t COL_BS = 64, COL_AS = COL_BS + 4 * STEP_TILES, TMEM_COLS = 128;    // of tensor memory, behind the sums
constexpr int THREADS = 6 * 32;
constexpr uint32_t B_BYTES = ROWS * 128, SCALE_BYTES = STEP_TILES * 512;
constexpr int kMaxParts = 8;

// What depends on the columns of the MMA, as many rows of a.
template <int COLS>
struct Stage {
    static constexpr uint32_t A_BYTES = COLS * 128;
    static constexpr uint32_t BYTES = B_BYTES + A_BYTES + 2 * SCALE_BYTES;
    static constexpr uint32_t BAR_OFF = STAGES * BYTES;
    static constexpr uint32_t SMEM_BYTES = BAR_OFF + 128 + 1024;
    static_assert(BYTES % 1024 == 0 && NBARS * 8 + 8 <= 128, "128-byte swizzle; barriers");
    static_assert(ROWS * COLS * 4 <= STAGES * BYTES && 2 * (SMEM_BYTES + 1024) <= 228 * 1024, "sums of the other parts; two CTAs an SM");
};

struct RowsParams {
    CUtensorMap a, as, b, bs;
    const float* bias;
    void* out;
    int64_t out_stride;
    uint32_t* err;
    uint64_t timeout_ns;
    int64_t drop;
    int32_t M, N, steps, parts, out_f32, gelu;
};

template <int COLS>
__global__ void __launch_bounds__(THREADS, 1) rows_kernel(const __grid_constant__ RowsParams p)
{
    using S = Stage<COLS>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s0 = smem_u32(smem);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + S::BAR_OFF);
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + NBARS);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    const uint32_t bar0 = smem_u32(bars);
    auto bar = [&](int i) { return bar0 + 8u * static_cast<uint32_t>(i); };
    const int warp = __shfl_sync(0xffffffffu, static_cast<int>(threadIdx.x) >> 5, 0);
    const int lane = threadIdx.x & 31;
    const int part = static_cast<int>(cluster_ctarank());
    const int n0 = static_cast<int>(cluster_id_x()) * ROWS;
    const int steps = p.steps / p.parts + (part < p.steps % p.parts);
    const int first = p.steps / p.parts * part + min(part, p.steps % p.parts);
    const uint64_t tmo = p.timeout_ns;

    if (threadIdx.x == 0) {
        for (int i = 0; i < NBARS; ++i) mbar_init(bar(i), 1);
        *abort_flag = 0;
        fence_mbar_init();
    }
    if (threadIdx.x == 128) {
        tma_prefetch_desc(&p.b);
        tma_prefetch_desc(&p.bs);
        tma_prefetch_desc(&p.a);
        tma_prefetch_desc(&p.as);
    }
    if (warp == 5) {
        tmem_alloc(smem_u32(tmem_slot), TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    wait_for_launch_before();
    launch_dependents();

    const int row = warp * 32 + lane, n = n0 + row;              // of b, of warps 0-3
    const float bias = warp < 4 && p.bias && n < p.N ? p.bias[n] : 0.0f;
    auto give_up = [&]() {
        *abort_flag = 1;
        atomicOr(p.err, kErrTimeout);
    };
    if (warp == 4) {
        int issued = 0, st = 0;                                  // steps; the ring's stage and its phase
        uint32_t phase = 1;
        for (; issued < steps; ++issued) {
            const int k = first + issued;
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(B_EMPTY + st), phase, tmo, abort_flag))) {
                if (lane == 0) give_up();
                break;
            }
            const uint32_t sb = s0 + st * S::BYTES;
            if (k != p.drop)
                mx4_load_warp(bar(B_FULL + st), S::BYTES, &p.b, &p.a, &p.bs, &p.as, sb, sb + B_BYTES, sb + B_BYTES + S::A_BYTES,
                              sb + B_BYTES + S::A_BYTES + SCALE_BYTES, k * 128, n0, 0, k * STEP_TILES, n0 / 128, 0);
            else if (lane == 0)
                mbar_arrive_expect_tx(bar(B_FULL + st), S::BYTES);
            if (++st == STAGES) {
                st = 0;
                phase ^= 1u;
            }
        }
        if (lane == 0) {
            // the last copies land before their memory is used again or left
            volatile int no_abort = 0;
            for (int g = max(0, issued - STAGES); g < issued; ++g)
                mbar_wait_bounded(bar(B_FULL + g % STAGES), static_cast<uint32_t>(g / STAGES) & 1u, tmo, &no_abort);
        }
        __syncwarp();
    } else if (warp == 5) {
        const uint64_t dB = sdesc_sw128(s0, 16, 1024), dA = sdesc_sw128(s0 + B_BYTES, 16, 1024);
        const uint64_t dBS = sdesc_scales(s0 + B_BYTES + S::A_BYTES), dAS = sdesc_scales(s0 + B_BYTES + S::A_BYTES + SCALE_BYTES);
        int st = 0;
        uint32_t phase = 0;
        uint64_t at = 0;
        for (int i = 0; i < steps; ++i) {
            if (!__all_sync(0xffffffffu, mbar_wait_bounded(bar(B_FULL + st), phase, tmo, abort_flag))) {
                if (lane == 0) give_up();
                break;
            }
            tc_fence_after();
            mx4_stage_warp(tmem, dB + at, dA + at, dBS + at, dAS + at, tmem + COL_BS, tmem + COL_AS, idesc_mx4(ROWS, COLS, 0), idesc_mx4(ROWS, COLS, 1),
                           i > 0 ? 1u : 0u);
            mma_commit_warp(bar(B_EMPTY + st));
            at += S::BYTES >> 4;
            if (++st == STAGES) {
                st = 0;
                at = 0;
                phase ^= 1u;
            }
        }
        mma_commit_warp(bar(B_DONE));
        if (lane == 0) {
            volatile int no_abort = 0;
            mbar_wait_bounded(bar(B_DONE), 0, tmo, &no_abort);
        }
        __syncwarp();
    } else {
        const bool ok = mbar_wait_bounded(bar(B_DONE), 0, tmo, abort_flag);
        if (!__all_sync(0xffffffffu, ok) && lane == 0) give_up();
    }
    __syncthreads();
    const bool sound = !*abort_flag;
    // `count` rows of out from m on, of which y has room for all
    auto write = [&](int m, int count, auto& y) {
        constexpr int ROOM = sizeof(y) / sizeof(float);
#pragma unroll
        for (int j = 0; j < ROOM; ++j) y[j] += bias;
        if (p.gelu) {
#pragma unroll
            for (int j = 0; j < ROOM; ++j) y[j] = gelu(y[j]);
        }
        if (n >= p.N) return;
        const int64_t at = m * p.out_stride + n;
        if (p.out_f32) {
            float* const o = static_cast<float*>(p.out) + at;
#pragma unroll
            for (int j = 0; j < ROOM; ++j)
                if (j < count) o[j * p.out_stride] = y[j];
        } else {
            __nv_bfloat16* const o = static_cast<__nv_bfloat16*>(p.out) + at;
#pragma unroll
            for (int j = 0; j < ROOM; ++j)
                if (j < count) o[j * p.out_stride] = __float2bfloat16_rn(y[j]);
        }
    };
    const uint32_t lanes = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    tc_fence_after();
    if (p.parts == 1) {
        if (warp < 4 && sound) {
#pragma unroll 1
            for (int m0 = 0; m0 < p.M; m0 += 16) {
                uint32_t sums[16];
                tmem_ld_x16_sync(lanes + m0, sums);
                float y[16];
#pragma unroll
                for (int j = 0; j < 16; ++j) y[j] = __uint_as_float(sums[j]);
                write(m0, p.M - m0, y);
            }
        }
    } else {
        // [part][row of a][row of b] of the CTA that adds up this row of a
        const int shift = 31 - __clz(COLS / p.parts), share = 1 << shift;
        cluster_sync_all();                                      // every ring is free
        if (warp < 4 && sound) {
            const uint32_t slot = s0 + static_cast<uint32_t>((part * share * ROWS + row) * 4);
#pragma unroll 1
            for (int m0 = 0; m0 < p.M; m0 += 16) {
                uint32_t y[16];
                tmem_ld_x16_sync(lanes + m0, y);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const int m = m0 + j;
                    if (m < p.M)
                        st_cluster(map_to_rank(slot + static_cast<uint32_t>((m & (share - 1)) * (ROWS * 4)), static_cast<uint32_t>(m >> shift)),
                                   static_cast<int32_t>(y[j]));
                }
            }
        }
        cluster_sync_all();
        if (warp < 4 && sound) {
            const int m0 = part * share, rows = min(share, p.M - m0);
            constexpr int TOGETHER = 4;
#pragma unroll 1
            for (int j0 = 0; j0 < rows; j0 += TOGETHER) {
                const float* sums = reinterpret_cast<const float*>(smem) + j0 * ROWS + row;
                const int count = min(rows - j0, TOGETHER);
                float y[TOGETHER];
#pragma unroll
                for (int j = 0; j < TOGETHER; ++j) y[j] = j < count ? sums[j * ROWS] : 0.0f;
                for (int from = 1; from < p.parts; ++from) {
                    sums += share * ROWS;
#pragma unroll
                    for (int j = 0; j < TOGETHER; ++j)
                        if (j < count) y[j] += sums[j * ROWS];
                }
                write(m0 + j0, count, y);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 5) {
        tc_fence_after();
        tmem_dealloc(tmem, TMEM_COLS);
    }
}

template <int COLS>
cudaError_t launch(const Mx4Product& q, int parts, cudaStream_t s)
{
    RowsParams p{};
    if (!mx4_codes_map(&p.a, q.a, q.M, q.tiles, COLS) || !mx4_codes_map(&p.b, q.b, q.N, q.tiles, ROWS) ||
        !mx4_scales_map(&p.as, q.as, q.M, q.tiles, STEP_TILES, 1) || !mx4_scales_map(&p.bs, q.bs, q.N, q.tiles, STEP_TILES, 1))
        return cudaErrorInvalidValue;
    p.bias = q.bias;
    p.out = q.out;
    p.out_stride = q.out_stride;
    p.err = q.err;
    p.timeout_ns = q.timeout_ns;
    p.drop = q.drop;
    p.M = static_cast<int32_t>(q.M);
    p.N = static_cast<int32_t>(q.N);
    p.steps = (q.tiles + STEP_TILES - 1) / STEP_TILES;
    p.out_f32 = q.out_f32;
    p.gelu = q.gelu;
    const int64_t clusters = (q.N + ROWS - 1) / ROWS;
    p.parts = parts;
    constexpr int kBytes = static_cast<int>(Stage<COLS>::SMEM_BYTES);
    static PerDevice once;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e == cudaSuccess) e = once.run(dev, [] { return cudaFuncSetAttribute(rows_kernel<COLS>, cudaFuncAttributeMaxDynamicSharedMemorySize, kBytes); });
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[2] = {chained_attribute(), {}};
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.parts);
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(static_cast<unsigned>(clusters * p.parts));
    cfg.blockDim = dim3(THREADS);
    cfg.dynamicSmemBytes = kBytes;
    cfg.stream = s;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, rows_kernel<COLS>, p);
}

}  // namespace

// Parts of the depth for as many CTAs as the GPU holds (two an SM), of two steps at least, where that saves more steps than the
// exchange costs: 3 rows at 5120 x 20480 take 23.4 us in one part and 12.3 in four, at 512 x 4096 (16 steps) 4.2 in one, 3.9 in
// two, 3.4 in four and 3.2 in eight, at 1536 x 1536 (six) 2.9 in one and 3.3 in two.
Mx4Plan mx4_rows_plan(int64_t M, int64_t N, int tiles)
{
    const int64_t clusters = (N + ROWS - 1) / ROWS;
    const int steps = (tiles + STEP_TILES - 1) / STEP_TILES;
    int parts = 1;
    while (parts < kMaxParts && clusters * parts * 2 <= 304 && steps >= std::max(12, 4 * parts)) parts *= 2;
    return {M <= 16 ? 16 : M <= 32 ? 32 : 64, parts, 1};
}

cudaError_t launch_mx4_rows(const Mx4Product& p, cudaStream_t s)
{
    const Mx4Plan plan = mx4_rows_plan(p.M, p.N, p.tiles);
    return plan.width == 16 ? launch<16>(p, plan.parts, s) : plan.width == 32 ? launch<32>(p, plan.parts, s) : launch<64>(p, plan.parts, s);
}

}  // namespace sdv2
