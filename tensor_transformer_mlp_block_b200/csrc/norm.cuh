// Layer norm, forward and backward (include/tpmlp.h states the formulas).
//
// One pass over the data: a row's elements stay in registers between the sums
// and the output (up to 32 elements in each of 512 or 1024 threads), so X is read once and Y written once; both directions are bound by
// memory bandwidth. The variance is summed around the mean from the registers,
// so an offset of the row costs no precision. Rows whose start and length are
// multiples of 16 bytes move 16 bytes per access, any others one element.
// Wider rows go through the looped kernels at the end, which read X again.
#pragma once

#include "aux_kernels.cuh"
#include "simt.cuh"

namespace tpmlp {

// VE elements of a row as they lie in memory: 16 bytes, or one element.
template <typename T, int VE>
struct RawVec {
    uint4 v;
    __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
    __device__ __forceinline__ void clear() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ void get(float* f) const {
        if constexpr (sizeof(T) == 2) {
            unpack_bf16x8(v, f);
        } else {
            f[0] = __uint_as_float(v.x);
            f[1] = __uint_as_float(v.y);
            f[2] = __uint_as_float(v.z);
            f[3] = __uint_as_float(v.w);
        }
    }
    __device__ __forceinline__ static void store(T* p, const float* f) {
        uint4 o;
        if constexpr (sizeof(T) == 2) {
            o.x = pack_bf16x2(f[0], f[1]);
            o.y = pack_bf16x2(f[2], f[3]);
            o.z = pack_bf16x2(f[4], f[5]);
            o.w = pack_bf16x2(f[6], f[7]);
        } else {
            o = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]),
                           __float_as_uint(f[3]));
        }
        *reinterpret_cast<uint4*>(p) = o;
    }
};
template <typename T>
struct RawVec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T* p) { v = *p; }
    __device__ __forceinline__ void clear() { v = from_f32<T>(0.0f); }
    __device__ __forceinline__ void get(float* f) const { f[0] = to_f32<T>(v); }
    __device__ __forceinline__ static void store(T* p, const float* f) { *p = from_f32<T>(f[0]); }
};

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

// Block (threads per row, rows): with 32 threads per row the rows of a block
// are independent warps; else one row per block. Thread t holds the vectors
// t, t + threads, ... of the row.
template <typename T, int VE, int NV>
__global__ void __launch_bounds__(1024) norm_fwd_kernel(const T* __restrict__ X, const T* __restrict__ gamma,
                                                       const T* __restrict__ beta, T* __restrict__ Y,
                                                       float* __restrict__ mean, float* __restrict__ rstd,
                                                       int64_t R, int h, float eps) {
    __shared__ float red[2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    if (r >= R) return;  // a whole warp of a 32-thread row; never with one row per block
    const int nvec = h / VE;
    const T* x = X + r * h;
    RawVec<T, VE> raw[NV];
    float f[NV][VE];
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        raw[i].clear();
        if (v < nvec) raw[i].load(x + v * VE);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        raw[i].get(f[i]);
#pragma unroll
        for (int e = 0; e < VE; ++e) s += f[i][e];
    }
    const float inv_h = 1.0f / static_cast<float>(h);
    const float mu = row_sum(s, red[0]) * inv_h;
    float q = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (static_cast<int>(threadIdx.x + i * blockDim.x) < nvec) {
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float c = f[i][e] - mu;
                q += c * c;
            }
        }
    }
    const float rs = 1.0f / sqrtf(row_sum(q, red[1]) * inv_h + eps);
    if (threadIdx.x == 0 && mean != nullptr) {
        mean[r] = mu;
        rstd[r] = rs;
    }
    T* y = Y + r * h;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        if (v < nvec) {
            float o[VE];
            RawVec<T, VE> g, b;
            float gf[VE], bf[VE];
            if (gamma != nullptr) {
                g.load(gamma + v * VE);
                g.get(gf);
            }
            if (beta != nullptr) {
                b.load(beta + v * VE);
                b.get(bf);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                o[e] = (f[i][e] - mu) * rs;
                if (gamma != nullptr) o[e] *= gf[e];
                if (beta != nullptr) o[e] += bf[e];
            }
            RawVec<T, VE>::store(y + v * VE, o);
        }
    }
}

// Backward. Blocks walk the rows r = block, block + grid, ...; a thread owns
// the same columns in every row and keeps their dgamma and dbeta sums in
// registers, so the weight gradients cost no second pass over the data: each
// block writes one row of partial sums, which colsum_final2_kernel adds in
// block order. The next row's loads are issued before the current row's sums.
template <typename T, int VE, int NV>
__global__ void __launch_bounds__(512) norm_bwd_kernel(const T* dY, const T* __restrict__ X,
                                                       const T* __restrict__ gamma,
                                                       const float* __restrict__ mean,
                                                       const float* __restrict__ rstd, const T* dR, T* dX,
                                                       float* __restrict__ part_g, float* __restrict__ part_b,
                                                       int64_t R, int h) {
    extern __shared__ float fold[];  // rows of a block > 1: its groups' sums
    __shared__ float red[2][2][32];
    grid_dep_wait();
    grid_dep_launch();
    const int nvec = h / VE;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t step = static_cast<int64_t>(gridDim.x) * blockDim.y;
    const float inv_h = 1.0f / static_cast<float>(h);
    RawVec<T, VE> rg[NV];
    float ag[NV][VE], ab[NV][VE];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        const int v = threadIdx.x + i * blockDim.x;
        rg[i].clear();
        if (gamma != nullptr && v < nvec) rg[i].load(gamma + v * VE);
#pragma unroll
        for (int e = 0; e < VE; ++e) ag[i][e] = ab[i][e] = 0.0f;
    }
    int64_t r = static_cast<int64_t>(blockIdx.x) * blockDim.y + threadIdx.y;
    int turn = 0;
    for (; r < R; r += step) {
        RawVec<T, VE> rx[NV], ry[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            rx[i].clear();
            ry[i].clear();
            if (v < nvec) {
                rx[i].load(X + r * h + v * VE);
                ry[i].load(dY + r * h + v * VE);
            }
        }
        const float mu = mean[r], rs = rstd[r];
        float c1 = 0.0f, c2 = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (static_cast<int>(threadIdx.x + i * blockDim.x) >= nvec) continue;
            float x[VE], y[VE], g[VE];
            rx[i].get(x);
            ry[i].get(y);
            rg[i].get(g);
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float xh = (x[e] - mu) * rs;
                const float gy = gamma != nullptr ? y[e] * g[e] : y[e];
                c1 += gy;
                c2 += gy * xh;
                ag[i][e] += y[e] * xh;
                ab[i][e] += y[e];
            }
        }
        c1 = warp_sum(c1);
        c2 = warp_sum(c2);
        if (blockDim.x > 32) {
            // two sets of slots in turn: one barrier per row
            if (lane == 0) {
                red[turn][0][warp] = c1;
                red[turn][1][warp] = c2;
            }
            __syncthreads();
            const bool in = lane < static_cast<int>(blockDim.x >> 5);
            c1 = warp_sum(in ? red[turn][0][lane] : 0.0f);
            c2 = warp_sum(in ? red[turn][1][lane] : 0.0f);
            turn ^= 1;
        }
        c1 *= inv_h;
        c2 *= inv_h;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v >= nvec) continue;
            float x[VE], y[VE], g[VE], o[VE];
            rx[i].get(x);
            ry[i].get(y);
            rg[i].get(g);
            float d[VE];
            if (dR != nullptr) {
                RawVec<T, VE> q;
                q.load(dR + r * h + v * VE);
                q.get(d);
            }
#pragma unroll
            for (int e = 0; e < VE; ++e) {
                const float xh = (x[e] - mu) * rs;
                const float gy = gamma != nullptr ? y[e] * g[e] : y[e];
                o[e] = rs * (gy - c1 - xh * c2);
                if (dR != nullptr) o[e] += d[e];
            }
            RawVec<T, VE>::store(dX + r * h + v * VE, o);
        }
    }
    if (blockDim.y == 1) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v < nvec) {
#pragma unroll
                for (int e = 0; e < VE; ++e) {
                    part_g[static_cast<int64_t>(blockIdx.x) * h + v * VE + e] = ag[i][e];
                    part_b[static_cast<int64_t>(blockIdx.x) * h + v * VE + e] = ab[i][e];
                }
            }
        }
        return;
    }
    // the block's rows in ascending order, dgamma's sums and then dbeta's
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = threadIdx.x + i * blockDim.x;
            if (v < nvec) {
#pragma unroll
                for (int e = 0; e < VE; ++e)
                    fold[threadIdx.y * h + v * VE + e] = which == 0 ? ag[i][e] : ab[i][e];
            }
        }
        __syncthreads();
        float* out = (which == 0 ? part_g : part_b) + static_cast<int64_t>(blockIdx.x) * h;
        for (int c = threadIdx.y * 32 + threadIdx.x; c < h; c += 32 * blockDim.y) {
            float s = fold[c];
            for (int y = 1; y < static_cast<int>(blockDim.y); ++y) s += fold[y * h + c];
            out[c] = s;
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
    const float rs = 1.0f / sqrtf(row_sum(q, red[1]) / static_cast<float>(h) + eps);
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
