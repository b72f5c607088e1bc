// Product of few rows with a weight matrix, with bias, activation and
// residual: Y[T, N] = act(X·W + bias) + R for up to 128 rows (single tokens,
// small batches, short prompts).
//
// With few rows the time is that of reading W once from memory, so the work is
// cut to keep every SM loading: the output's transpose is computed, 128 columns
// of W per tile as the tensor cores' 128 rows (W [K][N] is read MN-major, as it
// lies) and TN ≥ T rows of X as their N, and the tile's K range is split over a
// cluster of S CTAs. Each CTA streams its part of W through a shared-memory
// ring. Every CTA of the cluster owns 128/S of the tile's columns: the others
// store their fp32 partial sums of them straight into its shared memory, and
// after one cluster barrier it adds them in ascending k. So nothing goes through
// global memory, no counters are needed, and the result does not depend on
// timing. (Sums read from the other CTAs after the barrier took 5 µs more.)
//
// Measured on B200: 1 row, 4096 → 16384, GeLU 24.3 µs and 24 rows, 16384 → 4096
// with a residual 26.4 µs, for 134 MB of W, 20.5 µs at the measured copy rate;
// one 128-row tile per CTA without the split took 51 and 61 µs. What is left is
// the start (barriers, tensor memory, the first loads) and the sums' exchange.
//
// 192 threads: warp 0 TMA producer, warp 1 MMA issuer, warps 2..5 epilogue
// (each the 32 tensor-memory lanes, i.e. columns of W, of its sub-partition).
// Waits are bounded as in gemm_tc.cuh.
#pragma once

#include "gemm_tc.cuh"

namespace tpmlp {

constexpr int kFewThreads = 192;
constexpr int kFewCols = 128;  // columns of W per tile

template <int TN>
struct FewCfg {
    static constexpr int W_BYTES = kFewCols * kBK * 2;
    static constexpr int X_BYTES = TN * kBK * 2;
    static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
    // partial sums of this CTA's columns: [rank][row][column], 128/S columns
    static constexpr int PART_BYTES = TN * kFewCols * 4;
    // Two CTAs per SM (at most 113 KB each), so that one's prologue and sums
    // run beside the other's loads; a tile of 128 rows leaves room for one.
    static constexpr int CTAS = TN <= 64 ? 2 : 1;
    static constexpr int STAGES = ((CTAS == 2 ? 114000 : 228000) - PART_BYTES) / STAGE_BYTES;
    static constexpr int TMEM_COLS = TN < 32 ? 32 : TN;
    static constexpr int BAR_BYTES = 8 * (2 * STAGES + 1) + 16;
    static constexpr int SMEM_BYTES = 1024 + PART_BYTES + STAGES * STAGE_BYTES + BAR_BYTES;
};

struct FewArgs {
    int T, N, k_blocks;
    int act;  // 0 GeLU, 1 its tanh form, 2 none
    const __nv_bfloat16* bias;   // N, or null
    const __nv_bfloat16* resid;  // T × N, or null; may be Y
    __nv_bfloat16* H;            // T × N, or null
    __nv_bfloat16* Y;
    uint64_t wait_limit_ns;
};

// Output (t, n) from its sum.
__device__ __forceinline__ void few_store(const FewArgs& g, int t, int n, float v, float bias) {
    const int64_t off = static_cast<int64_t>(t) * g.N + n;
    v += bias;
    if (g.H != nullptr) g.H[off] = __float2bfloat16_rn(v);
    float unused;
    if (g.act == 0) gelu_fast_x2(v, v, v, unused);
    else if (g.act == 1) gelu_tanh_fast_x2(v, v, v, unused);
    if (g.resid != nullptr) v += __bfloat162float(g.resid[off]);
    g.Y[off] = __float2bfloat16_rn(v);
}

// Grid: tiles of W's columns × S, in clusters of S (a power of two).
template <int TN>
__global__ void __launch_bounds__(kFewThreads, FewCfg<TN>::CTAS)
    gemm_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX,
                    const FewArgs g, int S) {
    using C = FewCfg<TN>;
    constexpr int STAGES = C::STAGES;
    constexpr uint32_t IDESC = idesc_bf16_f32(kFewCols, TN, true, false);

    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                               ~static_cast<uintptr_t>(1023));
    uint8_t* sW = smem;
    uint8_t* sX = smem + STAGES * C::W_BYTES;
    float* parts = reinterpret_cast<float*>(smem + STAGES * C::STAGE_BYTES);
    uint64_t* bars = reinterpret_cast<uint64_t*>(smem + STAGES * C::STAGE_BYTES + C::PART_BYTES);
    uint64_t* full = bars;
    uint64_t* empty = bars + STAGES;
    uint64_t* done = bars + 2 * STAGES;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(done + 1);
    volatile int* abort = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const int rank = S > 1 ? static_cast<int>(cluster_ctarank()) : 0;
    const int n0 = static_cast<int>(blockIdx.x) / S * kFewCols;
    const int kb0 = static_cast<int>(static_cast<int64_t>(rank) * g.k_blocks / S);
    const int kb1 = static_cast<int>(static_cast<int64_t>(rank + 1) * g.k_blocks / S);

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(smem_u32(&full[s]), 1);
            mbar_init(smem_u32(&empty[s]), 1);
        }
        mbar_init(smem_u32(done), 1);
        *abort = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmW);
        tma_prefetch_desc(&tmX);
    }
    if (warp == 1) {
        tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (S > 1) cluster_arrive();  // this CTA has started (waited for before the sums are pushed)
    grid_dep_wait();
    grid_dep_launch();
    const uint64_t limit = g.wait_limit_ns;

    bool ok = true;
    if (warp == 0) {
        if (lane == 0) {
            int issued = 0;
            for (int kb = kb0; kb < kb1; ++kb, ++issued) {
                const int s = issued % STAGES;
                if (!mbar_wait_bounded(smem_u32(&empty[s]), (static_cast<uint32_t>(issued / STAGES) & 1u) ^ 1u,
                                       abort, limit)) {
                    raise_timeout(abort);
                    break;
                }
                const uint32_t fb = smem_u32(&full[s]);
                mbar_arrive_expect_tx(fb, C::STAGE_BYTES);
                const uint32_t w_dst = smem_u32(sW + s * C::W_BYTES);
                tma_load_2d(w_dst, &tmW, fb, n0, kb * kBK);
                tma_load_2d(w_dst + 8192, &tmW, fb, n0 + 64, kb * kBK);
                tma_load_2d(smem_u32(sX + s * C::X_BYTES), &tmX, fb, kb * kBK, 0);
            }
            // every slot's last release has arrived before this CTA may exit
            for (int i = issued > STAGES ? issued - STAGES : 0; i < issued && !*abort; ++i)
                if (!mbar_wait_bounded(smem_u32(&empty[i % STAGES]), static_cast<uint32_t>(i / STAGES) & 1u, abort,
                                       limit))
                    raise_timeout(abort);
            if (*abort) {
                // wind down: the copies in flight, the last min(issued, STAGES) slots
                for (int i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i) {
                    volatile int never = 0;
                    mbar_wait_bounded(smem_u32(&full[i % STAGES]), static_cast<uint32_t>(i / STAGES) & 1u, &never,
                                      limit);
                }
            }
        }
        __syncwarp();
        if (S > 1) cluster_wait();
    } else if (warp == 1) {
        if (lane == 0) {
            for (int kb = kb0; kb < kb1; ++kb) {
                const int i = kb - kb0, s = i % STAGES;
                if (!mbar_wait_bounded(smem_u32(&full[s]), static_cast<uint32_t>(i / STAGES) & 1u, abort, limit)) {
                    raise_timeout(abort);
                    break;
                }
                tc_fence_after();
                const uint32_t w = smem_u32(sW + s * C::W_BYTES), x = smem_u32(sX + s * C::X_BYTES);
#pragma unroll
                for (int k = 0; k < kBK / 16; ++k)
                    umma_bf16(tmem, smem_desc_sw128(w + k * 2048, 8192, 1024), smem_desc_sw128(x + k * 32, 16, 1024),
                              IDESC, (i > 0 || k > 0) ? 1u : 0u);
                umma_commit(smem_u32(&empty[s]));
            }
            // also on the way out after a timeout: every MMA issued has ended
            umma_commit(smem_u32(done));
            volatile int never = 0;
            mbar_wait_bounded(smem_u32(done), 0, &never, limit);
        }
        __syncwarp();
        if (S > 1) cluster_wait();
    } else {
        const int quad = warp & 3;
        const int c = quad * 32 + lane;  // column of W within the tile
        const int rows = g.T;
        if (g.resid != nullptr && (lane & 15) == 0 && n0 + c < g.N) {
            // the residual's first touch of memory runs beside the product
            for (int t = rank; t < rows; t += S)
                prefetch_l2(g.resid + static_cast<int64_t>(t) * g.N + n0 + c);
        }
        // every lane waits and the warp goes on only together (.sync.aligned loads)
        ok = mbar_wait_bounded(smem_u32(done), 0, abort, limit);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) raise_timeout(abort);
        if (S > 1) cluster_wait();  // the other CTAs have started
        if (ok) {
            tc_fence_after();
            const int n = n0 + c;
            const uint32_t src = tmem + (static_cast<uint32_t>(quad * 32) << 16);
            float bias = 0.0f;
            if (S == 1 && g.bias != nullptr && n < g.N) bias = __bfloat162float(g.bias[n]);
            // the owner of column c, and where this rank's sums of it go
            const int cols = kFewCols / S;
            const uint32_t dst = S > 1 ? mapa_shared(smem_u32(parts + rank * TN * cols + c % cols), c / cols) : 0u;
#pragma unroll 1
            for (int j = 0; j < rows; j += 16) {
                uint32_t v[16];
                tmem_ld_32x32b_x16(src + j, v);
                tmem_wait_ld();
                if (S == 1) {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (j + i < rows && n < g.N) few_store(g, j + i, n, __uint_as_float(v[i]), bias);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        if (j + i < rows) st_shared_cluster_u32(dst + 4 * (j + i) * cols, v[i]);
                }
            }
        }
    }
    tc_fence_before();
    if (S > 1) {
        cluster_sync();  // every rank's sums of this rank's columns have arrived
        if (warp >= 2 && ok) {
            const int cols = kFewCols / S;  // S rows at a time, one column a thread
            const int e = static_cast<int>(threadIdx.x) - 64;
            const int n = n0 + rank * cols + e % cols;
            if (n < g.N) {
                const float bias = g.bias != nullptr ? __bfloat162float(g.bias[n]) : 0.0f;
                const float* p = parts + e % cols;
#pragma unroll 4
                for (int t = e / cols; t < g.T; t += S) {
                    float v = p[t * cols];
#pragma unroll
                    for (int q = 1; q < 8; ++q)
                        if (q < S) v += p[(q * TN + t) * cols];
                    few_store(g, t, n, v, bias);
                }
            }
        }
    } else {
        __syncthreads();
    }
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::TMEM_COLS);
    }
}

}  // namespace tpmlp
