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
// colsum_partial_block: lane x holds columns [by·256 + 8x, +8), phase y the rows
// chunk_begin + y, +8, ...; the 8 phases are added in order. dH is rounded to
// dY's type because both products take it as a tensor-core operand, bf16 by bf16:
// bf16 gradients are then 2.35e-3 off (2-norm), where rounding them alone is
// 1.66e-3; keeping dH whole would take it in two parts and twice the products.
// 6144 × 4096 bf16 on B200: 32 µs (4.7 TB/s; 23 µs at the copy rate), bound by the derivative's
// arithmetic beside the loads.
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
// Tiles of 32 rows × 256 columns (8 blocks of 32), row tiles on grid x, 8 warps:
// a lane holds 8 columns, so 4 lanes share a block and exchange its maximum in
// two steps. The tile's 256 scale bytes are gathered in shared memory and written
// 32 to a row of S (one row of the tile each would touch a 32-byte sector per
// byte). Encoding 8192 × 16384 takes 96 µs in bf16 (4.2 TB/s: half of the issue
// slots busy, the rest waiting for a lane's four loads) and 101 µs in fp32
// (6.7 TB/s, the copy rate).

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

// The values C and S stand for. W columns per access and lane: 16 bytes of H where
// its rows allow them, else 1, so that a warp's stores fill whole sectors. 8192 ×
// 16384: bf16 68 µs (6.0 TB/s), fp32 111 µs (6.1 TB/s; with 32 bytes a lane 130);
// 4096 × 4099, single elements: 44 µs in both types, bound by the number of
// accesses (8 neighbouring single stores a lane: 51 and 69).
template <typename T, int W>
__global__ void __launch_bounds__(256) ckpt8_decode_kernel(const uint8_t* __restrict__ C,
                                                           const uint8_t* __restrict__ S, T* __restrict__ H,
                                                           int64_t R, int64_t F) {
    grid_dep_wait();
    grid_dep_launch();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t ldc = (F + kC8Block - 1) / kC8Block * kC8Block;
    const int64_t row0 = static_cast<int64_t>(blockIdx.x) * 32;
    const int64_t c0 = static_cast<int64_t>(blockIdx.y) * 256 + lane * W;
    constexpr int G = 8 / W;  // accesses per row
    using Code = std::conditional_t<W == 8, uint2, std::conditional_t<W == 4, uint32_t, uint8_t>>;
    Code w[4][G];
    uint8_t sb[4][G];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = row0 + warp + 8 * k;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int64_t c = c0 + i * 32 * W;
            w[k][i] = Code{};
            sb[k][i] = 0;
            if (r < R && c < F) {
                w[k][i] = *reinterpret_cast<const Code*>(C + r * ldc + c);
                sb[k][i] = S[c / kC8Block * R + r];
            }
        }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const int64_t r = row0 + warp + 8 * k;
#pragma unroll
        for (int i = 0; i < G; ++i) {
            const int64_t c = c0 + i * 32 * W;
            if (r >= R || c >= F) continue;
            const float s = c8_scale(sb[k][i]);
            if constexpr (W == 8) {
                float x[8];
                c8_unpack4(w[k][i].x, s, x);
                c8_unpack4(w[k][i].y, s, x + 4);
                store8<T, true>(H + r * F, c, F, x);
            } else if constexpr (W == 4) {
                static_assert(sizeof(T) == 4, "16 bytes per access");
                float x[4];
                c8_unpack4(w[k][i], s, x);
                *reinterpret_cast<float4*>(H + r * F + c) = make_float4(x[0], x[1], x[2], x[3]);
            } else {
                H[r * F + c] = from_f32<T>(static_cast<float>(static_cast<int8_t>(w[k][i])) * s);
            }
        }
    }
}

// --------------------------------------------------- plain path, tiled product
// The CUDA-core product of simt.cuh with register tiles: BT × BT outputs per
// block (64 or 128), 8 × BT/16 a thread as packed pairs of fp32 (two rows), and
// 16-deep k tiles in shared memory. fp32 operands come through a ring of
// asynchronous copies, 16 bytes where rows allow it, or, 16 bytes along k, through
// registers; bf16 operands are converted on the way, one tile ahead in registers.
// Each output is an fp32 accumulator updated with fma over k in ascending order.
// SPLIT (BT = 64): a cluster of S blocks takes consecutive parts of K, and each
// block adds the parts of its 64/S rows in ascending k (few output tiles and a
// long K: weight gradients of narrow layers, short batches). A launch may hold a
// second product of the same kind, whose tiles follow the first's. Bound by the
// CUDA cores' arithmetic; 2048 × 1024, K = 1024 fp32 114 µs (37 TFLOP/s), the
// backward's products 243 µs (with copies through registers 169 and 345).
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

// One operand's part of a k tile: element (x, k), x the tile's row (or column),
// at p[x·sx + k·sk]; one of the strides is 1. It lies in shared memory as [k][LD]
// whichever it is, so that a thread's eight rows are pairs of registers as they
// come from there (with [x][k] the packing costs more than the copies save:
// 2048 × 1024, K = 1024 fp32 170-200 µs against 127-147). vec: x is the unit
// stride and 16-byte copies of 4 elements are aligned.
template <typename TI, int BT>
struct TiledOperand {
    static constexpr int BK = 16, LD = BT + 4, NT = BT == 128 ? 256 : 128;
    static constexpr int PER = BT * BK / NT;
    const TI* p;  // at the tile's first row
    int64_t sx, sk;
    int left;  // rows of the tile inside the matrix
    bool k_unit, vec, kvec;

    // fp32, k the unit stride, 16-byte loads of 4 elements aligned: through
    // registers, transposed on the way into s
    __device__ __forceinline__ void fetch4(float4 (&r)[PER / 4], int k0, int kend, int t) const {
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            const int e = t + NT * i, x = e / (BK / 4), k = k0 + e % (BK / 4) * 4;
            r[i] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            const float* q = reinterpret_cast<const float*>(p) + x * sx + k;
            if (x < left && k + 3 < kend) {
                r[i] = *reinterpret_cast<const float4*>(q);
            } else if (x < left) {
                if (k < kend) r[i].x = q[0];
                if (k + 1 < kend) r[i].y = q[1];
                if (k + 2 < kend) r[i].z = q[2];
            }
        }
    }
    __device__ __forceinline__ void stash4(float (*s)[LD], const float4 (&r)[PER / 4], int t) const {
#pragma unroll
        for (int i = 0; i < PER / 4; ++i) {
            const int e = t + NT * i, x = e / (BK / 4), k = e % (BK / 4) * 4;
            s[k][x] = r[i].x;
            s[k + 1][x] = r[i].y;
            s[k + 2][x] = r[i].z;
            s[k + 3][x] = r[i].w;
        }
    }

    // element e of the tile: consecutive threads along the unit stride
    __device__ __forceinline__ void place(int e, int& x, int& k) const {
        x = k_unit ? e / BK : e % BT;
        k = k_unit ? e % BK : e / BT;
    }
    // fp32: asynchronous copies of k tile k0 (up to kend) into s[k][x]
    __device__ __forceinline__ void copy(float (*s)[LD], int k0, int kend, int t) const {
        if (vec) {
#pragma unroll
            for (int i = 0; i < PER / 4; ++i) {
                const int e = t + NT * i, x = e % (BT / 4) * 4, k = e / (BT / 4);
                const int in = k0 + k < kend ? min(max(left - x, 0), 4) : 0;
                cp_async16(smem_u32(&s[k][x]), in > 0 ? p + (k0 + k) * sk + x : p, 4 * in);
            }
        } else {
#pragma unroll
            for (int i = 0; i < PER; ++i) {
                int x, k;
                place(t + NT * i, x, k);
                const bool in = x < left && k0 + k < kend;
                cp_async4(smem_u32(&s[k][x]), in ? p + x * sx + (k0 + k) * sk : p, in ? 4 : 0);
            }
        }
    }
    __device__ __forceinline__ void fetch(TI (&r)[PER], int k0, int kend, int t) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            int x, k;
            place(t + NT * i, x, k);
            r[i] = x < left && k0 + k < kend ? p[x * sx + (k0 + k) * sk] : from_f32<TI>(0.0f);
        }
    }
    __device__ __forceinline__ void stash(float (*s)[LD], const TI (&r)[PER], int t) const {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            int x, k;
            place(t + NT * i, x, k);
            s[k][x] = to_f32<TI>(r[i]);
        }
    }
};

template <typename TI, int BT>
__device__ __forceinline__ TiledOperand<TI, BT> tiled_operand(const void* base, int64_t sx, int64_t sk, int64_t x0,
                                                              int extent) {
    TiledOperand<TI, BT> o;
    o.p = static_cast<const TI*>(base) + x0 * sx;
    o.sx = sx;
    o.sk = sk;
    o.left = static_cast<int>(min(static_cast<int64_t>(BT), extent - x0));
    o.k_unit = sk == 1;
    const bool aligned = sizeof(TI) == 4 && (reinterpret_cast<uintptr_t>(base) & 15u) == 0;
    o.vec = sx == 1 && sk % 4 == 0 && aligned;
    o.kvec = sk == 1 && sx % 4 == 0 && sx > 1 && aligned;  // (a k tile starts at a multiple of 16)
    return o;
}

template <typename TI, typename TO, int EPI, int BT, bool SPLIT>
__global__ void __launch_bounds__(BT == 128 ? 256 : 128, BT == 128 ? 2 : 4)
    simt_tiled_kernel(const TiledProduct p0, const TiledProduct p1, int S) {
    static_assert(BT == 64 || (BT == 128 && !SPLIT), "tiles of 64 (K may be split) or 128");
    constexpr int BK = 16, LD = BT + 4, NT = BT == 128 ? 256 : 128, TN = BT / 16;
    // fp32: tiles in flight and in use; bf16: the tile in use and the next one
    constexpr int STAGES = sizeof(TI) == 4 && BT == 64 ? 4 : 2;
    __shared__ __align__(16) float sA[STAGES][BK][LD];
    __shared__ __align__(16) float sB[STAGES][BK][LD];
    const int tiles0 = p0.mb * p0.nb;
    const bool second = static_cast<int>(blockIdx.x) >= tiles0;
    const TiledProduct& p = second ? p1 : p0;
    const SimtArgs& g = p.a;
    const int tile = static_cast<int>(blockIdx.x) - (second ? tiles0 : 0);
    const int t = threadIdx.x;
    const int tx = t % 16, ty = t / 16;  // rows 4·ty.. and BT/2 + 4·ty..; columns 4·tx.. (and 64 + 4·tx..)
    auto column = [&](int j) { return 16 * (j & ~3) + 4 * tx + (j & 3); };
    const int64_t m0 = static_cast<int64_t>(tile % p.mb) * BT, n0 = static_cast<int64_t>(tile / p.mb) * BT;
    const int rank = SPLIT ? static_cast<int>(blockIdx.z) : 0;
    const int steps = (g.K + BK - 1) / BK;
    const int kbeg = SPLIT ? static_cast<int>(static_cast<int64_t>(rank) * steps / S) * BK : 0;
    const int kend = SPLIT ? min(g.K, static_cast<int>(static_cast<int64_t>(rank + 1) * steps / S) * BK) : g.K;
    const auto A = tiled_operand<TI, BT>(g.A, g.sam, g.sak, m0, g.M);
    const auto B = tiled_operand<TI, BT>(g.B, g.sbn, g.sbk, n0, g.N);
    uint64_t acc[4][TN];  // pairs of rows (2i, 2i + 1) of the thread's eight
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int j = 0; j < TN; ++j) acc[i][j] = 0ull;
    // terms beyond the range are fma(0, 0, acc), which leaves acc as it is
    auto multiply = [&](int s) {
#pragma unroll
        for (int k = 0; k < BK; ++k) {
            const float4 a0 = *reinterpret_cast<const float4*>(&sA[s][k][4 * ty]);
            const float4 a1 = *reinterpret_cast<const float4*>(&sA[s][k][BT / 2 + 4 * ty]);
            const uint64_t a[4] = {f2_pack(a0.x, a0.y), f2_pack(a0.z, a0.w), f2_pack(a1.x, a1.y), f2_pack(a1.z, a1.w)};
            float b[TN];
#pragma unroll
            for (int j = 0; j < TN; j += 4)
                *reinterpret_cast<float4*>(b + j) = *reinterpret_cast<const float4*>(&sB[s][k][16 * j + 4 * tx]);
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                const uint64_t bb = f2_splat(b[j]);
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[i][j] = f2_fma(a[i], bb, acc[i][j]);
            }
        }
    };
    const int n_steps = kend > kbeg ? (kend - kbeg + BK - 1) / BK : 0;
    if constexpr (SPLIT && sizeof(TI) != 4) cluster_arrive();
    if constexpr (sizeof(TI) == 4) {
        float4 ra[TiledOperand<TI, BT>::PER / 4], rb[TiledOperand<TI, BT>::PER / 4];
#pragma unroll
        for (int s = 0; s < STAGES - 1; ++s) {
            if (s < n_steps) {
                if (A.kvec) A.fetch4(ra, kbeg + s * BK, kend, t);
                else A.copy(sA[s], kbeg + s * BK, kend, t);
                if (B.kvec) B.fetch4(rb, kbeg + s * BK, kend, t);
                else B.copy(sB[s], kbeg + s * BK, kend, t);
                if (A.kvec) A.stash4(sA[s], ra, t);
                if (B.kvec) B.stash4(sB[s], rb, t);
            }
            cp_async_commit();
        }
        for (int q = 0; q < n_steps; ++q) {
            cp_async_wait<STAGES - 2>();  // tile q has arrived (this thread's part)
            __syncthreads();              // everyone's; and tile q - 1 is no longer read
            const int f = q + STAGES - 1;
            if (f < n_steps) {
                if (A.kvec) A.fetch4(ra, kbeg + f * BK, kend, t);
                else A.copy(sA[f % STAGES], kbeg + f * BK, kend, t);
                if (B.kvec) B.fetch4(rb, kbeg + f * BK, kend, t);
                else B.copy(sB[f % STAGES], kbeg + f * BK, kend, t);
            }
            cp_async_commit();
            multiply(q % STAGES);
            // the stage is free: tile q - 1 was its last, before this round's barrier
            if (f < n_steps) {
                if (A.kvec) A.stash4(sA[f % STAGES], ra, t);
                if (B.kvec) B.stash4(sB[f % STAGES], rb, t);
            }
        }
        cp_async_wait<0>();
    } else {
        TI ra[TiledOperand<TI, BT>::PER], rb[TiledOperand<TI, BT>::PER];
        if (n_steps > 0) {
            A.fetch(ra, kbeg, kend, t);
            B.fetch(rb, kbeg, kend, t);
        }
        for (int q = 0; q < n_steps; ++q) {
            A.stash(sA[q & 1], ra, t);
            B.stash(sB[q & 1], rb, t);
            __syncthreads();  // tile q is there; tile q - 1 (the other buffer) may still be read
            if (q + 1 < n_steps) {
                A.fetch(ra, kbeg + (q + 1) * BK, kend, t);
                B.fetch(rb, kbeg + (q + 1) * BK, kend, t);
            }
            multiply(q & 1);
        }
    }
    if constexpr (SPLIT) {
        static_assert(TN == 4, "64-wide tiles");
        // the sums of rank q's part: [q][row of this block's][column], in the
        // ring's memory once every block of the cluster is through with its own
        float* parts = &sA[0][0][0];
        static_assert(sizeof(sA) >= 64 * 64 * 4 || sizeof(TI) != 4, "parts fit the A ring");
        __shared__ __align__(16) float own_parts[sizeof(TI) == 4 ? 1 : 64 * 64];
        if constexpr (sizeof(TI) != 4) {
            parts = own_parts;
            cluster_wait();  // the other blocks have started
        } else {
            cluster_sync();
        }
        const int own = 64 / S;  // rows per block; S divides 64
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo[4], hi[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) f2_unpack(acc[i][j], lo[j], hi[j]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = (i & 2) * 16 + 4 * ty + 2 * (i & 1) + r;
                const float* v = r == 0 ? lo : hi;
                st_shared_cluster_v4(mapa_shared(smem_u32(parts + (rank * own + row % own) * 64 + 4 * tx), row / own),
                                     v[0], v[1], v[2], v[3]);
            }
        }
        cluster_sync();  // every block's sums of this block's rows have arrived
        for (int e = t; e < own * 64; e += NT) {
            const int row = e / 64, col = e % 64;
            float v = parts[row * 64 + col];
            for (int q = 1; q < S; ++q) v += parts[(q * own + row) * 64 + col];
            const int64_t m = m0 + rank * own + row, n = n0 + col;
            if (m < g.M && n < g.N) tiled_store<TI, TO, EPI>(p, m, n, v);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int64_t m = m0 + (i & 4) * (BT / 8) + 4 * ty + (i & 3);
            float v[TN];
#pragma unroll
            for (int j = 0; j < TN; ++j) {
                float lo, hi;
                f2_unpack(acc[i / 2][j], lo, hi);
                v[j] = (i & 1) ? hi : lo;
            }
#pragma unroll
            for (int j = 0; j < TN; j += 4) {
                const int64_t n = n0 + column(j);
                if constexpr (EpiTraits<EPI>::kC8Out) {
                    // 32 columns of a row are 8 neighbouring threads' groups of four
                    float* x = v + j;
                    float top = 0.0f;
#pragma unroll
                    for (int c = 0; c < 4; ++c) {
                        if (g.bias != nullptr && n + c < g.N) x[c] += ld_f32<TI>(static_cast<const TI*>(g.bias) + n + c);
                        top = max_nan(top, fabsf(x[c]));
                    }
                    for (int w = 1; w < 8; w <<= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, w));
                    const uint32_t sb = c8_scale_byte(top);
                    const uint32_t word = sb == kC8NaN ? 0u : c8_pack4(x[0], x[1], x[2], x[3], c8_inverse(sb));
                    if (m < g.M && n < p.c8_ld) *reinterpret_cast<uint32_t*>(p.c8 + m * p.c8_ld + n) = word;
                    if (m < g.M && n < g.N && (tx & 7) == 0)
                        p.c8_scale[n / kC8Block * g.M + m] = static_cast<uint8_t>(sb);
                }
                if (m >= g.M) continue;
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    const int64_t nc = n0 + column(j + c);
                    if (nc < g.N) tiled_store<TI, TO, EPI>(p, m, nc, v[j + c]);
                }
            }
        }
    }
}

}  // namespace tpmlp
