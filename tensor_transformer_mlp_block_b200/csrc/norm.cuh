// Layer norm, forward and backward (include/tpmlp.h states the formulas).
//
// One pass over the data: a row's elements stay in registers (forward) or in
// shared memory (backward) between the sums and the output, so everything is
// read and written once. The variance is summed around the mean, and x̂ is
// (x − mean)·rstd in two fp32 steps everywhere, so an offset of the row costs
// only what rounding its mean to fp32 costs. (One fma, x·rstd − mean·rstd, is off
// by the product's rounding, up to 2^-24·|mean|·rstd in a whole row: at a mean of
// 100 deviations dgamma is 2.1e-6 off, and 2.5e-8 in two steps, which cost 0-2% of
// the backward's time.) Rows whose start and length are multiples of 16
// bytes move 16 bytes per access, any others one element. Rows too wide for that
// go through the looped kernels at the end, which read X again.
//
// Measured on B200 (copy rate 6.56 TB/s), 8192 × 4096: forward 26.7 µs in bf16
// (5.0 TB/s) and 43 µs in fp32 (6.2 TB/s); backward with the residual's gradient
// 51 µs in bf16 (5.2 TB/s) and 84 µs in fp32 (6.4 TB/s). fp32 is bound by memory;
// in bf16 the same instructions move half the bytes, and issue slots (65% of the
// cycles forward, 55% backward) and the sums' latency bound it: packed fp32x2
// arithmetic brought the forward from 41 to 29 µs, rows by bulk copies the
// backward from 116 to 56, keeping its intermediate values from 56 to 51.
#pragma once

#include "aux_kernels.cuh"
#include "simt.cuh"

namespace tpmlp {

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int w = 16; w >= 1; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w);
    return v;
}

// Sum over the block's threads (a warp if blockDim.x is 32), the same in every
// thread and run: a fixed tree inside each warp, then over the warps. `red`:
// 32 floats of shared memory, free for reuse after the next __syncthreads.
__device__ __forceinline__ float row_sum(float v, float* red) {
    v = warp_sum(v);
    if (blockDim.x == 32) return v;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (lane == 0) red[warp] = v;
    __syncthreads();
    return warp_sum(lane < static_cast<int>(blockDim.x >> 5) ? red[lane] : 0.0f);
}

// The 16 bytes of a vector as packed pairs of fp32.
template <typename T>
__device__ __forceinline__ void vec_pairs(const uint4& v, uint64_t* p) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            p[i] = f2_pack(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
        p[0] = f2_pack(__uint_as_float(w[0]), __uint_as_float(w[1]));
        p[1] = f2_pack(__uint_as_float(w[2]), __uint_as_float(w[3]));
    }
}
template <typename T>
__device__ __forceinline__ uint4 pairs_vec(const uint64_t* p) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            f2_unpack(p[i], a, b);
            w[i] = pack_bf16x2(a, b);
        }
    } else {
        float a, b;
        f2_unpack(p[0], a, b);
        w[0] = __float_as_uint(a);
        w[1] = __float_as_uint(b);
        f2_unpack(p[1], a, b);
        w[2] = __float_as_uint(a);
        w[3] = __float_as_uint(b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}

// Forward. Block (threads per row, rows): with 32 threads per row the rows of a
// block are independent warps; else one row per block. Thread t holds the vectors
// t, t + threads, ... of the row, as packed pairs of fp32.
template <typename T, int NV>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const T* __restrict__ X, const T* __restrict__ gamma,
                                                       const T* __restrict__ beta, T* __restrict__ Y,
                                                       float* __restrict__ mean, float* __restrict__ rstd,
                                                       int64_t R, int h, float inv_h, float eps) {
    constexpr int VE = 16 / sizeof(T), PV = VE / 2;
    __shared__ float red[2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (r >= R) return;  // a whole warp of a 32-thread row; never with one row per block
    const int nvec = h / VE;
    const uint4* x = reinterpret_cast<const uint4*>(X + r * h);
    uint4 raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        raw[i] = v < nvec ? x[v] : make_uint4(0, 0, 0, 0);
    }
    uint64_t f[NV][PV];
    uint64_t s = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        vec_pairs<T>(raw[i], f[i]);
#pragma unroll
        for (int e = 0; e < PV; ++e) s = f2_add(s, f[i][e]);
    }
    float a, b;
    f2_unpack(s, a, b);
    const float mu = row_sum(a + b, red[0]) * inv_h;
    const uint64_t less = f2_splat(-mu);
    uint64_t q = 0ull;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (static_cast<int>(threadIdx.x + i * blockDim.x) >= nvec) continue;
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            f[i][e] = f2_add(f[i][e], less);
            q = f2_fma(f[i][e], f[i][e], q);
        }
    }
    f2_unpack(q, a, b);
    const float rs = rsqrtf(row_sum(a + b, red[1]) * inv_h + eps);
    if (threadIdx.x == 0 && mean != nullptr) {
        mean[r] = mu;
        rstd[r] = rs;
    }
    const uint64_t rs2 = f2_splat(rs);
    uint4* y = reinterpret_cast<uint4*>(Y + r * h);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v >= nvec) continue;
        uint64_t g[PV], c[PV];
        if (gamma != nullptr) vec_pairs<T>(reinterpret_cast<const uint4*>(gamma)[v], g);
        if (beta != nullptr) vec_pairs<T>(reinterpret_cast<const uint4*>(beta)[v], c);
#pragma unroll
        for (int e = 0; e < PV; ++e) {
            uint64_t o = f2_mul(f[i][e], rs2);
            if (gamma != nullptr && beta != nullptr) o = f2_fma(o, g[e], c[e]);
            else if (gamma != nullptr) o = f2_mul(o, g[e]);
            else if (beta != nullptr) o = f2_add(o, c[e]);
            f[i][e] = o;
        }
        y[v] = pairs_vec<T>(f[i]);
    }
}

// The same for rows that are not whole vectors: element t, t + threads, ...
template <typename T, int NV>
__global__ void __launch_bounds__(1024) norm_fwd_scalar_kernel(const T* __restrict__ X,
                                                              const T* __restrict__ gamma,
                                                              const T* __restrict__ beta, T* __restrict__ Y,
                                                              float* __restrict__ mean,
                                                              float* __restrict__ rstd, int64_t R, int h,
                                                              float inv_h, float eps) {
    __shared__ float red[2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (r >= R) return;
    const int nt = static_cast<int>(blockDim.x);
    float f[NV], s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * nt;
        f[i] = c < h ? to_f32<T>(X[r * h + c]) : 0.0f;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) s += f[i];
    const float mu = row_sum(s, red[0]) * inv_h;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        f[i] -= mu;
        if (static_cast<int>(threadIdx.x) + i * nt < h) q += f[i] * f[i];
    }
    const float rs = rsqrtf(row_sum(q, red[1]) * inv_h + eps);
    if (threadIdx.x == 0 && mean != nullptr) {
        mean[r] = mu;
        rstd[r] = rs;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c >= h) continue;
        float o = f[i] * rs;
        if (gamma != nullptr) o *= to_f32<T>(gamma[c]);
        if (beta != nullptr) o += to_f32<T>(beta[c]);
        Y[r * h + c] = from_f32<T>(o);
    }
}

// Backward of rows that are not whole 16-byte vectors. Blocks walk the rows r =
// block, block + grid, ...; a thread owns the same NV columns in every row and
// keeps their dgamma and dbeta sums in registers, so the weight gradients cost
// no second pass over the data: each block writes one row of partial sums,
// which colsum_final2_kernel adds in block order.
template <typename T, int NV>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const T* dY, const T* __restrict__ X,
                                                       const T* __restrict__ gamma,
                                                       const float* __restrict__ mean,
                                                       const float* __restrict__ rstd, const T* dR, T* dX,
                                                       float* __restrict__ part_g, float* __restrict__ part_b,
                                                       int64_t R, int h) {
    __shared__ float red[2][2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nt = static_cast<int>(blockDim.x);
    const float inv_h = 1.0f / static_cast<float>(h);
    const bool in = lane < nt >> 5;
    float ag[NV], ab[NV];
    T rg[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * nt;
        ag[i] = ab[i] = 0.0f;
        rg[i] = gamma != nullptr && c < h ? gamma[c] : from_f32<T>(1.0f);
    }
    int turn = 0;
    for (int64_t r = blockIdx.x; r < R; r += gridDim.x) {
        const float mu = mean[r], rs = rstd[r];
        const int64_t off = r * h;
        T rx[NV], ry[NV], rd[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * nt;
            rx[i] = ry[i] = rd[i] = from_f32<T>(0.0f);
            if (c < h) {
                rx[i] = X[off + c];
                ry[i] = dY[off + c];
                if (dR != nullptr) rd[i] = dR[off + c];
            }
        }
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (static_cast<int>(threadIdx.x) + i * nt >= h) continue;
            const float y = to_f32<T>(ry[i]), xh = (to_f32<T>(rx[i]) - mu) * rs;
            const float gy = y * to_f32<T>(rg[i]);
            c1 += gy;
            c2 += gy * xh;
            ag[i] += y * xh;
            ab[i] += y;
        }
        c1 = warp_sum(c1);
        c2 = warp_sum(c2);
        // two sets of slots in turn: one barrier per row
        if (lane == 0) {
            red[turn][0][warp] = c1;
            red[turn][1][warp] = c2;
        }
        __syncthreads();
        c1 = warp_sum(in ? red[turn][0][lane] : 0.0f) * inv_h;
        c2 = warp_sum(in ? red[turn][1][lane] : 0.0f) * inv_h;
        turn ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = threadIdx.x + i * nt;
            if (c >= h) continue;
            const float xh = (to_f32<T>(rx[i]) - mu) * rs;
            const float gy = to_f32<T>(ry[i]) * to_f32<T>(rg[i]);
            dX[off + c] = from_f32<T>(rs * (gy - c1 - xh * c2) + to_f32<T>(rd[i]));
        }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int c = threadIdx.x + i * nt;
        if (c < h) {
            part_g[static_cast<int64_t>(blockIdx.x) * h + c] = ag[i];
            part_b[static_cast<int64_t>(blockIdx.x) * h + c] = ab[i];
        }
    }
}

// Backward of rows that are whole 16-byte vectors. As norm_bwd_kernel, but the
// rows arrive through a shared-memory ring of bulk copies, so the bytes in
// flight do not depend on the registers a thread can spare: a row's X, dY and
// dR are one stage, read for the sums and again for dX. A group of threads (a
// warp, or the block) owns a ring and walks the rows group, group + groups, ...;
// a row's stage is refilled after the next row's sums, whose barrier tells that
// every thread is through with it (with one stage, after a barrier of its own).
// In a warp's ring a vote stands for that barrier. A vote orders no memory, so it
// serves only because what a lane reads of a stage is used before: x and dY in the
// sums that the warp has exchanged, dR in the dX it has stored. No read can still
// be under way when lane 0 issues the refill.
// KEEP: x̂ and dY ⊙ gamma stay in registers between the two uses, up to 16
// elements per thread (a warp's ring needs it: see above). ONE: one stage, gamma read
// from global memory (rows so wide that no more fits). Waits are bounded.
struct NormRing {
    int stages;  // rows a group's ring holds (1..8)
    uint64_t wait_limit_ns;
};

template <typename T, int NV, bool WARP, int MAX_THREADS, int PER_SM, bool KEEP, bool ONE = false>
__global__ void __launch_bounds__(MAX_THREADS, PER_SM) norm_bwd_ring_kernel(const T* dY, const T* __restrict__ X,
                                                            const T* __restrict__ gamma,
                                                            const float* __restrict__ mean,
                                                            const float* __restrict__ rstd, const T* dR, T* dX,
                                                            float* __restrict__ part_g,
                                                            float* __restrict__ part_b, int64_t R, int h,
                                                            NormRing ring) {
    static_assert(KEEP || !WARP, "a warp's refill relies on x and dY being used up by the vote");
    constexpr int VE = 16 / sizeof(T), PV = VE / 2;
    extern __shared__ __align__(128) uint8_t sm[];
    __shared__ float red[2][2][32];
    __shared__ __align__(8) uint64_t bars[4 * 8];
    __shared__ int abort_flag;
    const int nvec = h / VE;
    const uint32_t row_bytes = static_cast<uint32_t>(h) * sizeof(T);
    const uint32_t stage_bytes = row_bytes * (dR != nullptr ? 3 : 2);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int groups = WARP ? static_cast<int>(blockDim.y) : 1;
    const int gi = WARP ? static_cast<int>(threadIdx.y) : 0;
    const int S = ONE ? 1 : ring.stages;
    uint64_t* full = bars + gi * 8;
    uint8_t* base = sm + static_cast<size_t>(gi) * S * stage_bytes;
    volatile int* abort = &abort_flag;
    if (threadIdx.x == 0) {
        for (int s = 0; s < S; ++s) mbar_init(smem_u32(&full[s]), 1);
        if (gi == 0) *abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    grid_dep_wait();
    grid_dep_launch();

    const int64_t step = static_cast<int64_t>(gridDim.x) * groups;
    const int64_t first = static_cast<int64_t>(blockIdx.x) * groups + gi;
    auto issue = [&](int64_t row, int s) {  // one thread: a row into stage s
        const int64_t off = row * h;
        const uint32_t bar = smem_u32(&full[s]), dst = smem_u32(base + s * stage_bytes);
        mbar_arrive_expect_tx(bar, stage_bytes);
        bulk_load(dst, X + off, row_bytes, bar);
        bulk_load(dst + row_bytes, dY + off, row_bytes, bar);
        if (dR != nullptr) bulk_load(dst + 2 * row_bytes, dR + off, row_bytes, bar);
    };
    if (threadIdx.x == 0)
        for (int s = 0; s < S && first + s * step < R; ++s) issue(first + s * step, s);

    const float inv_h = 1.0f / static_cast<float>(h);
    const uint4* gg = reinterpret_cast<const uint4*>(gamma);
    uint4* sg = reinterpret_cast<uint4*>(sm + static_cast<size_t>(groups) * S * stage_bytes);
    if (!ONE && gamma != nullptr) {
        const int n = blockDim.x * blockDim.y;
        for (int v = threadIdx.y * blockDim.x + threadIdx.x; v < nvec; v += n) sg[v] = gg[v];
        __syncthreads();
    }
    uint64_t ag[NV][PV], ab[NV][PV];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < PV; ++e) ag[i][e] = ab[i][e] = 0ull;
    float mu_next = first < R ? mean[first] : 0.0f, rs_next = first < R ? rstd[first] : 0.0f;
    bool failed = false;
    int at = 0, turn = 0;  // the row's stage, and its phase
    uint32_t phase = 0;
    int64_t r = first;
    for (; r < R; r += step) {
        const float mu = mu_next, rs = rs_next;
        if (r + step < R) {
            mu_next = mean[r + step];
            rs_next = rstd[r + step];
        }
        const uint8_t* stage = base + at * stage_bytes;
        const uint4* sx = reinterpret_cast<const uint4*>(stage);
        const uint4* sy = reinterpret_cast<const uint4*>(stage + row_bytes);
        const uint4* sr = reinterpret_cast<const uint4*>(stage + 2 * row_bytes);
        const bool got = mbar_wait_bounded(smem_u32(&full[at]), phase, abort, ring.wait_limit_ns);
        const uint64_t rs2 = f2_splat(rs), less = f2_splat(-mu);
        uint64_t s1 = 0ull, s2 = 0ull;
        uint64_t kx[KEEP ? NV : 1][PV], ky[KEEP ? NV : 1][PV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= nvec) continue;
            uint64_t x[PV], y[PV], g[PV];
            vec_pairs<T>(sx[v], x);
            vec_pairs<T>(sy[v], y);
            if (gamma != nullptr) vec_pairs<T>(ONE ? gg[v] : sg[v], g);
#pragma unroll
            for (int e = 0; e < PV; ++e) {
                const uint64_t xh = f2_mul(f2_add(x[e], less), rs2);
                const uint64_t gy = gamma != nullptr ? f2_mul(y[e], g[e]) : y[e];
                s1 = f2_add(s1, gy);
                s2 = f2_fma(gy, xh, s2);
                ag[i][e] = f2_fma(y[e], xh, ag[i][e]);
                ab[i][e] = f2_add(ab[i][e], y[e]);
                if constexpr (KEEP) {
                    kx[i][e] = xh;
                    ky[i][e] = gy;
                }
            }
        }
        float c1, c2, hi;
        f2_unpack(s1, c1, hi);
        c1 = warp_sum(c1 + hi);
        f2_unpack(s2, c2, hi);
        c2 = warp_sum(c2 + hi);
        if constexpr (WARP) {
            failed = !__all_sync(0xffffffffu, got);
        } else {
            if (lane == 0) {
                red[turn][0][warp] = c1;
                red[turn][1][warp] = c2;
            }
            failed = __syncthreads_or(!got) != 0;
            const bool in = lane < static_cast<int>(blockDim.x >> 5);
            c1 = warp_sum(in ? red[turn][0][lane] : 0.0f);
            c2 = warp_sum(in ? red[turn][1][lane] : 0.0f);
            turn ^= 1;
        }
        if (failed) break;
        // every thread is through with the previous row's stage: S - 1 rows on
        if (!ONE && threadIdx.x == 0 && r > first && r + (S - 1) * step < R)
            issue(r + (S - 1) * step, at == 0 ? S - 1 : at - 1);
        const uint64_t k1 = f2_splat(-rs * (c1 * inv_h)), k2 = f2_splat(-rs * (c2 * inv_h));
        T* out = dX + r * h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= nvec) continue;
            uint64_t x[PV], y[PV], g[PV], d[PV];
            if constexpr (!KEEP) {
                vec_pairs<T>(sx[v], x);
                vec_pairs<T>(sy[v], y);
                if (gamma != nullptr) vec_pairs<T>(ONE ? gg[v] : sg[v], g);
            }
            if (dR != nullptr) vec_pairs<T>(sr[v], d);
#pragma unroll
            for (int e = 0; e < PV; ++e) {
                uint64_t xh, gy;
                if constexpr (KEEP) {
                    xh = kx[KEEP ? i : 0][e];
                    gy = ky[KEEP ? i : 0][e];
                } else {
                    xh = f2_mul(f2_add(x[e], less), rs2);
                    gy = gamma != nullptr ? f2_mul(y[e], g[e]) : y[e];
                }
                uint64_t o = f2_fma(xh, k2, f2_fma(gy, rs2, k1));
                if (dR != nullptr) o = f2_add(o, d[e]);
                x[e] = o;
            }
            *reinterpret_cast<uint4*>(out + v * VE) = pairs_vec<T>(x);
        }
        if constexpr (ONE) {
            __syncthreads();
            if (threadIdx.x == 0 && r + step < R) issue(r + step, 0);
        }
        if (++at == S) {
            at = 0;
            phase ^= 1u;
        }
    }
    if (failed) {
        if (lane == 0) raise_timeout(abort);
        if (threadIdx.x == 0) {
            // wind down: the copies still in flight, from this row's on (the
            // previous row's stage has not been filled again)
            for (int q = 0; q < (r == first || ONE ? S : S - 1) && r + q * step < R; ++q) {
                volatile int never = 0;
                mbar_wait_bounded(smem_u32(&full[at]), phase, &never, ring.wait_limit_ns);
                if (++at == S) {
                    at = 0;
                    phase ^= 1u;
                }
            }
        }
    }
    if constexpr (!WARP) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= nvec) continue;
            float4* pg = reinterpret_cast<float4*>(part_g + static_cast<int64_t>(blockIdx.x) * h + v * VE);
            float4* pb = reinterpret_cast<float4*>(part_b + static_cast<int64_t>(blockIdx.x) * h + v * VE);
#pragma unroll
            for (int e = 0; e < PV; e += 2) {
                float4 a;
                f2_unpack(ag[i][e], a.x, a.y);
                f2_unpack(ag[i][e + 1], a.z, a.w);
                pg[e / 2] = a;
                f2_unpack(ab[i][e], a.x, a.y);
                f2_unpack(ab[i][e + 1], a.z, a.w);
                pb[e / 2] = a;
            }
        }
    } else {
        // the block's warps in order, through the ring's memory: dgamma's sums,
        // then dbeta's (the host leaves room for groups × h floats)
        float* fold = reinterpret_cast<float*>(sm);
        for (int which = 0; which < 2; ++which) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int v = threadIdx.x + i * blockDim.x;
                if (v >= nvec) continue;
                float2* f = reinterpret_cast<float2*>(fold + gi * h + v * VE);
#pragma unroll
                for (int e = 0; e < PV; ++e) {
                    float a, b;
                    f2_unpack(which == 0 ? ag[i][e] : ab[i][e], a, b);
                    f[e] = make_float2(a, b);
                }
            }
            __syncthreads();
            float* out = (which == 0 ? part_g : part_b) + static_cast<int64_t>(blockIdx.x) * h;
            for (int c = gi * 32 + lane; c < h; c += 32 * groups) {
                float s = fold[c];
                for (int y = 1; y < groups; ++y) s += fold[y * h + c];
                out[c] = s;
            }
        }
    }
}

// Rows too wide for registers: one block of 1024 threads per row, X read three
// times (from L2 after the first), one element per access.
template <typename T>
__global__ void __launch_bounds__(1024) norm_fwd_wide_kernel(const T* __restrict__ X,
                                                            const T* __restrict__ gamma,
                                                            const T* __restrict__ beta, T* __restrict__ Y,
                                                            float* __restrict__ mean,
                                                            float* __restrict__ rstd, int64_t h, float eps) {
    __shared__ float red[2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = blockIdx.x;
    const T* x = X + r * h;
    float s = 0.0f;
    for (int64_t c = threadIdx.x; c < h; c += blockDim.x) s += to_f32<T>(x[c]);
    const float mu = row_sum(s, red[0]) / static_cast<float>(h);
    float q = 0.0f;
    for (int64_t c = threadIdx.x; c < h; c += blockDim.x) {
        const float d = to_f32<T>(x[c]) - mu;
        q += d * d;
    }
    const float rs = rsqrtf(row_sum(q, red[1]) / static_cast<float>(h) + eps);
    if (threadIdx.x == 0 && mean != nullptr) {
        mean[r] = mu;
        rstd[r] = rs;
    }
    for (int64_t c = threadIdx.x; c < h; c += blockDim.x) {
        float o = (to_f32<T>(x[c]) - mu) * rs;
        if (gamma != nullptr) o *= to_f32<T>(gamma[c]);
        if (beta != nullptr) o += to_f32<T>(beta[c]);
        Y[r * h + c] = from_f32<T>(o);
    }
}

// Backward of the wide rows. The weight gradients' partial sums come first
// (norm_bwd_wide_cols_kernel), because dX may be written over dY.
template <typename T>
__global__ void __launch_bounds__(1024) norm_bwd_wide_kernel(const T* dY, const T* __restrict__ X,
                                                            const T* __restrict__ gamma,
                                                            const float* __restrict__ mean,
                                                            const float* __restrict__ rstd, const T* dR,
                                                            T* dX, int64_t h) {
    __shared__ float red[2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = blockIdx.x, off = r * h;
    const float mu = mean[r], rs = rstd[r];
    float c1 = 0.0f, c2 = 0.0f;
    for (int64_t c = threadIdx.x; c < h; c += blockDim.x) {
        float gy = to_f32<T>(dY[off + c]);
        if (gamma != nullptr) gy *= to_f32<T>(gamma[c]);
        c1 += gy;
        c2 += gy * ((to_f32<T>(X[off + c]) - mu) * rs);
    }
    c1 = row_sum(c1, red[0]) / static_cast<float>(h);
    c2 = row_sum(c2, red[1]) / static_cast<float>(h);
    for (int64_t c = threadIdx.x; c < h; c += blockDim.x) {
        float gy = to_f32<T>(dY[off + c]);
        if (gamma != nullptr) gy *= to_f32<T>(gamma[c]);
        float o = rs * (gy - c1 - (to_f32<T>(X[off + c]) - mu) * rs * c2);
        if (dR != nullptr) o += to_f32<T>(dR[off + c]);
        dX[off + c] = from_f32<T>(o);
    }
}

// One thread per column (grid y) and chunk of rows (grid x): partial dgamma and dbeta.
template <typename T>
__global__ void __launch_bounds__(256) norm_bwd_wide_cols_kernel(const T* __restrict__ dY,
                                                                const T* __restrict__ X,
                                                                const float* __restrict__ mean,
                                                                const float* __restrict__ rstd,
                                                                float* __restrict__ part_g,
                                                                float* __restrict__ part_b, int64_t R,
                                                                int64_t h, int64_t rows_per_chunk) {
    grid_dep_wait();
    grid_dep_launch();
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x;
    if (c >= h) return;
    const int64_t r1 = min(R, (static_cast<int64_t>(blockIdx.x) + 1) * rows_per_chunk);
    float g = 0.0f, b = 0.0f;
    for (int64_t r = static_cast<int64_t>(blockIdx.x) * rows_per_chunk; r < r1; ++r) {
        const float y = to_f32<T>(dY[r * h + c]);
        g += y * ((to_f32<T>(X[r * h + c]) - mean[r]) * rstd[r]);
        b += y;
    }
    part_g[static_cast<int64_t>(blockIdx.x) * h + c] = g;
    part_b[static_cast<int64_t>(blockIdx.x) * h + c] = b;
}

}  // namespace tpmlp
