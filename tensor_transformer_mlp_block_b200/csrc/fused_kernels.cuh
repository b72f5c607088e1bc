// Element-wise kernels of the linear layer's backward and of the 8-bit
// checkpoint, and the plain path's tiled product.
#pragma once

#include "aux_kernels.cuh"
#include "simt.cuh"

namespace tpmlp {

// Activation and derivative of eight values: bf16 results take the forms of
// the tensor-core epilogues, fp32 results CUDA's erff / tanhf.
template <typename T, bool TANH>
__device__ __forceinline__ void act_grad8(const float* x, float* d) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        if constexpr (sizeof(T) == 2) {
            if constexpr (TANH) gelu_tanh_grad_fast_x2(x[i], x[i + 1], d[i], d[i + 1]);
            else gelu_grad_fast_x2(x[i], x[i + 1], d[i], d[i + 1]);
        } else {
            d[i] = TANH ? gelu_tanh_grad_f32(x[i]) : gelu_grad_f32(x[i]);
            d[i + 1] = TANH ? gelu_tanh_grad_f32(x[i + 1]) : gelu_grad_f32(x[i + 1]);
        }
    }
}

// Eight consecutive elements from column c of a row of n; VEC: n % 8 == 0 and
// 16-byte aligned rows. Elements at n and beyond read as zero.
template <typename T, bool VEC>
__device__ __forceinline__ void load8(const T* p, int64_t c, int64_t n, float* f) {
    if constexpr (VEC) {
        if (c >= n) {
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] = 0.0f;
        } else if constexpr (sizeof(T) == 2) {
            unpack_bf16x8(*reinterpret_cast<const uint4*>(p + c), f);
        } else {
            const float4 a = *reinterpret_cast<const float4*>(p + c);
            const float4 b = *reinterpret_cast<const float4*>(p + c + 4);
            f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
            f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = c + i < n ? to_f32<T>(p[c + i]) : 0.0f;
    }
}

template <typename T, bool VEC>
__device__ __forceinline__ void store8(T* p, int64_t c, int64_t n, const float* f) {
    if constexpr (VEC) {
        if (c >= n) return;
        if constexpr (sizeof(T) == 2) {
            *reinterpret_cast<uint4*>(p + c) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                                          pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
        } else {
            *reinterpret_cast<float4*>(p + c) = make_float4(f[0], f[1], f[2], f[3]);
            *reinterpret_cast<float4*>(p + c + 4) = make_float4(f[4], f[5], f[6], f[7]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (c + i < n) p[c + i] = from_f32<T>(f[i]);
    }
}

// dH = dY ⊙ act′(H) and the partial column sums of dH before it is rounded:
// one pass over dY and H. Grid (row chunks, ⌈C/256⌉), block (32, 8) as
// colsum_partial_block: lane x holds columns [by·256 + 8x, +8), phase y the rows chunk_begin + y, +8, ...; the 8
// phases are added in order.
template <typename T, bool TANH, bool VEC>
__global__ void __launch_bounds__(256) act_grad_kernel(const T* __restrict__ dY, const T* __restrict__ H,
                                                       T* __restrict__ dH, int64_t R, int64_t C,
                                                       int64_t rows_per_chunk, float* __restrict__ partial) {
    __shared__ float red[8][256];
    grid_dep_wait();
    grid_dep_launch();
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x * 8;
    const int64_t r0 = static_cast<int64_t>(blockIdx.x) * rows_per_chunk;
    const int64_t r1 = min(R, r0 + rows_per_chunk);
    float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
    // the loads of kU rows are issued before any of them is used
    constexpr int kU = sizeof(T) == 2 && VEC ? 4 : 1;
    int64_t r = r0 + threadIdx.y;
    if constexpr (kU > 1) {
        for (; c0 < C && r + 8 * (kU - 1) < r1; r += 8 * kU) {
            uint4 ry[kU], rx[kU];
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                ry[u] = *reinterpret_cast<const uint4*>(dY + (r + 8 * u) * C + c0);
                rx[u] = *reinterpret_cast<const uint4*>(H + (r + 8 * u) * C + c0);
            }
#pragma unroll
            for (int u = 0; u < kU; ++u) {
                float y[8], x[8], d[8];
                unpack_bf16x8(ry[u], y);
                unpack_bf16x8(rx[u], x);
                act_grad8<T, TANH>(x, d);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    y[i] *= d[i];
                    acc[i] += y[i];
                }
                store8<T, VEC>(dH + (r + 8 * u) * C, c0, C, y);
            }
        }
    }
    for (; r < r1; r += 8) {
        float y[8], x[8], d[8];
        load8<T, VEC>(dY + r * C, c0, C, y);
        load8<T, VEC>(H + r * C, c0, C, x);
        act_grad8<T, TANH>(x, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            y[i] *= d[i];
            acc[i] += y[i];
        }
        store8<T, VEC>(dH + r * C, c0, C, y);
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) red[threadIdx.y][threadIdx.x * 8 + i] = acc[i];
    __syncthreads();
    const int t = threadIdx.y * 32 + threadIdx.x;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + t;
    if (c < C) {
        float s = red[0][t];
        for (int y = 1; y < 8; ++y) s += red[y][t];
        partial[static_cast<int64_t>(blockIdx.x) * C + c] = s;
    }
}

// ------------------------------------------------------- 8-bit checkpoint
// Tiles of 32 rows × 256 columns (8 blocks of 32), row tiles on grid x, 8 warps: a lane holds 8
// columns, so 4 lanes share a block and exchange its maximum in two steps. The
// tile's 256 scale bytes are gathered in shared memory and written 32 to a row
// of S (one row of the tile each would touch a 32-byte sector per byte).

// H to C and S.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) ckpt8_encode_kernel(const T* __restrict__ H, uint8_t* __restrict__ C,
                                                           uint8_t* __restrict__ S, int64_t R, int64_t F) {
    __shared__ uint8_t sS[8][32];
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ldc = (F + kC8Block - 1) / kC8Block * kC8Block;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 32;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + lane * 8;
    float h[4][8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = row0 + warp + 8 * k;
        if (r < R) {
            load8<T, VEC>(H + r * F, c, F, h[k]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) h[k][i] = 0.0f;
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = row0 + warp + 8 * k;
        float top = 0.0f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_nan(top, fabsf(h[k][i]));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, 2));
        const uint32_t sb = c8_scale_byte(top);
        const float inv = c8_inverse(sb);
        uint2 w = make_uint2(c8_pack4(h[k][0], h[k][1], h[k][2], h[k][3], inv),
                             c8_pack4(h[k][4], h[k][5], h[k][6], h[k][7], inv));
        if (sb == kC8NaN) w = make_uint2(0u, 0u);
        if ((lane & 3) == 0) sS[lane >> 2][warp + 8 * k] = static_cast<uint8_t>(sb);
        if (r < R && c < ldc) *reinterpret_cast<uint2*>(C + r * ldc + c) = w;
    }
    __syncthreads();
    const int64_t block = static_cast<int64_t>(blockIdx.y) * 8 + warp;
    if (block * kC8Block < F && row0 + lane < R) S[block * R + row0 + lane] = sS[warp][lane];
}

// The values C and S stand for.
template <typename T, bool VEC>
__global__ void __launch_bounds__(256) ckpt8_decode_kernel(const uint8_t* __restrict__ C,
                                                           const uint8_t* __restrict__ S, T* __restrict__ H,
                                                           int64_t R, int64_t F) {
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ldc = (F + kC8Block - 1) / kC8Block * kC8Block;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 32;
    const int64_t c = static_cast<int64_t>(blockIdx.y) * 256 + lane * 8;
    if (c >= F) return;
    uint2 w[4];
    uint32_t sb[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = row0 + warp + 8 * k;
        w[k] = make_uint2(0u, 0u);
        sb[k] = 0u;
        if (r < R) {
            w[k] = *reinterpret_cast<const uint2*>(C + r * ldc + c);
            sb[k] = S[c / kC8Block * R + r];
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = row0 + warp + 8 * k;
        if (r >= R) continue;
        const float s = c8_scale(sb[k]);
        float x[8];
        c8_unpack4(w[k].x, s, x);
        c8_unpack4(w[k].y, s, x + 4);
        store8<T, VEC>(H + r * F, c, F, x);
    }
}

// --------------------------------------------------- plain path, tiled product
// The CUDA-core product of simt.cuh with register tiles: BT × BT outputs per
// block of 256 threads, TM × TM each (TM = BT/16), 16-deep k tiles in shared
// memory, the next tile's global loads in flight during the current one's
// arithmetic. Each output is an fp32 accumulator updated with fmaf over k in
// ascending order; with S > 1 (BT = 64) a cluster of S blocks takes consecutive
// parts of K, and each block adds the parts of its 64/S rows in ascending k
// (few output tiles and a long K: weight gradients of narrow layers, single
// tokens). A launch may hold a second product of the same kind, whose tiles
// follow the first's.
struct TiledProduct {
    SimtArgs a;
    const void* resid;  // kResid: M × N of the operands' type, row stride ld_out; may be null
    uint8_t* c8;        // kC8Out, kC8In: the 8-bit checkpoint (ckpt8.cuh)
    uint8_t* c8_scale;
    int64_t c8_ld;
    int mb, nb;         // tiles
};

// Output (m, n) of a product from its sum.
template <typename TI, typename TO, int EPI>
__device__ __forceinline__ void tiled_store(const TiledProduct& p, int64_t m, int64_t n, float v) {
    const SimtArgs& g = p.a;
    const int64_t off = m * g.ld_out + n;
    if constexpr (EpiTraits<EPI>::kBias && !EpiTraits<EPI>::kC8Out) {
        if (g.bias != nullptr) v += ld_f32<TI>(static_cast<const TI*>(g.bias) + n);
    }
    float res = 0.0f;
    if constexpr (EpiTraits<EPI>::kResid) {
        if (p.resid != nullptr) res = ld_f32<TI>(static_cast<const TI*>(p.resid) + off);
    }
    if constexpr (EpiTraits<EPI>::kC8In) {
        const float h = static_cast<float>(static_cast<int8_t>(p.c8[m * p.c8_ld + n])) *
                        c8_scale(p.c8_scale[n / kC8Block * g.M + m]);
        static_cast<TO*>(g.out0)[off] =
            from_f32<TO>(v * (EpiTraits<EPI>::kTanh ? gelu_tanh_grad_f32(h) : gelu_grad_f32(h)));
        static_cast<TO*>(g.out1)[off] = from_f32<TO>(EpiTraits<EPI>::kTanh ? gelu_tanh_f32(h) : gelu_f32(h));
    } else if constexpr (EpiTraits<EPI>::kAct) {
        static_cast<TO*>(g.out0)[off] = from_f32<TO>(v);
        static_cast<TO*>(g.out1)[off] =
            from_f32<TO>((EpiTraits<EPI>::kTanh ? gelu_tanh_f32(v) : gelu_f32(v)) + res);
    } else {
        if constexpr (EpiTraits<EPI>::kActOnly) v = EpiTraits<EPI>::kTanh ? gelu_tanh_f32(v) : gelu_f32(v);
        static_cast<TO*>(g.out0)[off] = from_f32<TO>(v + res);
    }
}

template <typename TI, typename TO, int EPI, int BT>
__global__ void __launch_bounds__(256) simt_tiled_kernel(const TiledProduct p0, const TiledProduct p1, int S) {
    constexpr int TM = BT / 16, BK = 16, LD = BT + 4;
    __shared__ float sA[2][BK][LD];
    __shared__ float sB[2][BK][LD];
    __shared__ float parts[BT == 64 ? 64 * 64 : 1];  // [rank][row of this block's][column]
    const int tiles0 = p0.mb * p0.nb;
    const bool second = static_cast<int>(blockIdx.x) >= tiles0;
    const TiledProduct& p = second ? p1 : p0;
    const SimtArgs& g = p.a;
    const int tile = static_cast<int>(blockIdx.x) - (second ? tiles0 : 0);
    const int t = threadIdx.x;
    const int tx = t & 15, ty = t >> 4;
    const int64_t m0 = static_cast<int64_t>(tile % p.mb) * BT, n0 = static_cast<int64_t>(tile / p.mb) * BT;
    const int rank = static_cast<int>(blockIdx.z);
    const int steps = (g.K + BK - 1) / BK;
    const int kbeg = static_cast<int>(static_cast<int64_t>(rank) * steps / S) * BK;
    const int kend = min(g.K, static_cast<int>(static_cast<int64_t>(rank + 1) * steps / S) * BK);
    const TI* A = static_cast<const TI*>(g.A);
    const TI* B = static_cast<const TI*>(g.B);
    // consecutive threads along the operand's unit stride
    const bool a_k = g.sak == 1, b_k = g.sbk == 1;
    float ra[TM], rb[TM];
    auto fetch = [&](int k0) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int e = t + 256 * i;
            const int am = a_k ? e / BK : e % BT, ak = a_k ? e % BK : e / BT;
            const int bn = b_k ? e / BK : e % BT, bk = b_k ? e % BK : e / BT;
            ra[i] = (m0 + am < g.M && k0 + ak < kend) ? ld_f32<TI>(A + (m0 + am) * g.sam + (k0 + ak) * g.sak) : 0.0f;
            rb[i] = (n0 + bn < g.N && k0 + bk < kend) ? ld_f32<TI>(B + (k0 + bk) * g.sbk + (n0 + bn) * g.sbn) : 0.0f;
        }
    };
    auto stash = [&](int buf) {
#pragma unroll
        for (int i = 0; i < TM; ++i) {
            const int e = t + 256 * i;
            const int am = a_k ? e / BK : e % BT, ak = a_k ? e % BK : e / BT;
            const int bn = b_k ? e / BK : e % BT, bk = b_k ? e % BK : e / BT;
            sA[buf][ak][am] = ra[i];
            sB[buf][bk][bn] = rb[i];
        }
    };
    float acc[TM][TM];
#pragma unroll
    for (int i = 0; i < TM; ++i)
#pragma unroll
        for (int j = 0; j < TM; ++j) acc[i][j] = 0.0f;
    fetch(kbeg);
    stash(0);
    __syncthreads();
    int buf = 0;
    for (int k0 = kbeg; k0 < kend; k0 += BK) {
        if (k0 + BK < kend) fetch(k0 + BK);
        // terms beyond the range are fmaf(0, 0, acc), which leaves acc as it is
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            float a[TM], b[TM];
#pragma unroll
            for (int i = 0; i < TM; i += 4) {
                *reinterpret_cast<float4*>(a + i) = *reinterpret_cast<const float4*>(&sA[buf][k][16 * i + 4 * ty]);
                *reinterpret_cast<float4*>(b + i) = *reinterpret_cast<const float4*>(&sB[buf][k][16 * i + 4 * tx]);
            }
#pragma unroll
            for (int i = 0; i < TM; ++i)
#pragma unroll
                for (int j = 0; j < TM; ++j) acc[i][j] = fmaf(a[i], b[j], acc[i][j]);
        }
        if (k0 + BK < kend) {
            stash(buf ^ 1);
            __syncthreads();
            buf ^= 1;
        }
    }
    if constexpr (BT == 64) {
        if (S > 1) {
            const int own = 64 / S;  // rows per block; S divides 64
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int row = 4 * ty + i;
                const uint32_t dst = mapa_shared(smem_u32(parts + (rank * own + row % own) * 64 + 4 * tx), row / own);
#pragma unroll
                for (int j = 0; j < 4; ++j) st_shared_cluster_u32(dst + 4 * j, __float_as_uint(acc[i][j]));
            }
            cluster_sync();  // every block's sums of this block's rows have arrived
            for (int e = t; e < own * 64; e += 256) {
                const int row = e / 64, col = e % 64;
                float v = parts[row * 64 + col];
                for (int q = 1; q < S; ++q) v += parts[(q * own + row) * 64 + col];
                const int64_t m = m0 + rank * own + row, n = n0 + col;
                if (m < g.M && n < g.N) tiled_store<TI, TO, EPI>(p, m, n, v);
            }
            return;
        }
    }
#pragma unroll
    for (int i = 0; i < TM; ++i) {
        const int64_t m = m0 + 16 * (i & ~3) + 4 * ty + (i & 3);
        if constexpr (EpiTraits<EPI>::kC8Out) {
            // 32 columns of a row are 8 neighbouring threads' groups of four
#pragma unroll
            for (int j = 0; j < TM; j += 4) {
                const int64_t n = n0 + 16 * j + 4 * tx;
                float top = 0.0f;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    if (g.bias != nullptr && n + c < g.N)
                        acc[i][j + c] += ld_f32<TI>(static_cast<const TI*>(g.bias) + n + c);
                    top = max_nan(top, fabsf(acc[i][j + c]));
                }
                for (int w = 1; w < 8; w <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, w));
                const uint32_t sb = c8_scale_byte(top);
                const uint32_t word = sb == kC8NaN ? 0u : c8_pack4(acc[i][j], acc[i][j + 1], acc[i][j + 2],
                                                                   acc[i][j + 3], c8_inverse(sb));
                if (m < g.M && n < p.c8_ld) *reinterpret_cast<uint32_t*>(p.c8 + m * p.c8_ld + n) = word;
                if (m < g.M && n < g.N && (tx & 7) == 0)
                    p.c8_scale[n / kC8Block * g.M + m] = static_cast<uint8_t>(sb);
            }
        }
        if (m >= g.M) continue;
#pragma unroll
        for (int j = 0; j < TM; ++j) {
            const int64_t n = n0 + 16 * (j & ~3) + 4 * tx + (j & 3);
            if (n < g.N) tiled_store<TI, TO, EPI>(p, m, n, acc[i][j]);
        }
    }
}

}  // namespace tpmlp
