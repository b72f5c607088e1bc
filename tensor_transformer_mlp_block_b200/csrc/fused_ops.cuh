// Host side of the layer norm, of the linear layer with bias, activation and
// residual, and of the block with its pre-activation in 8 bits: argument
// checks, planning, launches. Part of tpmlp.cu's translation unit (included
// there), whose helpers it uses.

namespace tpmlp {
namespace {

using bf16 = __nv_bfloat16;

constexpr int64_t kMaxGridY = 65535;

tpmlp_status check_device() {
    const DeviceInfo* d = device_info();
    if (d == nullptr) return TPMLP_ERR_CUDA;
    return d->cc_major == 10 ? TPMLP_OK : TPMLP_ERR_UNSUPPORTED;
}

bool known_dtype(tpmlp_dtype dt) { return dt == TPMLP_BF16 || dt == TPMLP_FP32; }
bool known_act(tpmlp_activation a) { return a == TPMLP_GELU_ERF || a == TPMLP_GELU_TANH; }
bool known_grad(tpmlp_dtype g, tpmlp_dtype dt) { return g == TPMLP_FP32 || (g == TPMLP_BF16 && dt == TPMLP_BF16); }
// Sizes that the kernels' 32-bit row and column indices hold, tiles' last rows included.
bool fits32(int64_t x) { return x < (int64_t(1) << 31) - 1024; }

// A matrix of a call, as bytes.
struct Span {
    const void* p;
    int64_t bytes;
};

// Whether some output shares memory with an input or with another output
// (null pointers share none). Products read their operands while other tiles of
// the output are written, so such a call has no defined result.
bool overlapping(std::initializer_list<Span> outs, std::initializer_list<Span> ins) {
    auto meet = [](const Span& a, const Span& b) {
        const uintptr_t x = reinterpret_cast<uintptr_t>(a.p), y = reinterpret_cast<uintptr_t>(b.p);
        return a.p != nullptr && b.p != nullptr && x < y + static_cast<uintptr_t>(b.bytes) &&
               y < x + static_cast<uintptr_t>(a.bytes);
    };
    for (const Span* o = outs.begin(); o != outs.end(); ++o) {
        for (const Span& i : ins)
            if (meet(*o, i)) return true;
        for (const Span* q = o + 1; q != outs.end(); ++q)
            if (meet(*o, *q)) return true;
    }
    return false;
}

int64_t size_of(tpmlp_dtype dt) { return dt == TPMLP_BF16 ? 2 : 4; }

// ------------------------------------------------------------- plain products

// One product, or two of the same kind in one launch (q may be null). Tiles
// of 128 × 128 where there are four per SM, else 64 × 64, of which an SM holds
// four; with fewer than eight per SM, K is split over a cluster of up to 8 blocks
// (at least four 16-deep steps each). Measured on B200, fp32, µs with 64 × 64
// unsplit and split 2 / 4 / 8 ways: 2048 × 1024, K = 1024 123 and 109 / 119 / 127
// (123 with 128 × 128); 1024 × 1024, K = 2048 135 and 124 / 122 / 119 (238); 512³
// 29 and 18.5 / 14.5 / 14.4 (64).
template <typename TI, typename TO, int EPI>
tpmlp_status gemm_plain(int kind, TiledProduct p, cudaStream_t st, const TiledProduct* q = nullptr) {
    double flops = 0.0, bytes = 0.0;
    int64_t tiles128 = 0, tiles64 = 0, k = p.a.K;
    for (const TiledProduct* x : {static_cast<const TiledProduct*>(&p), q}) {
        if (x == nullptr) continue;
        const double M = x->a.M, N = x->a.N, K = x->a.K;
        flops += 2.0 * M * N * K;
        bytes += sizeof(TI) * (M * K + K * N) + sizeof(TO) * M * N;
        tiles128 += ((int64_t(x->a.M) + 127) / 128) * ((int64_t(x->a.N) + 127) / 128);
        tiles64 += ((int64_t(x->a.M) + 63) / 64) * ((int64_t(x->a.N) + 63) / 64);
    }
    const int sms = plan_num_sms();
    const int bt = tiles128 >= 4 * sms ? 128 : 64;
    int S = 1;
    if (bt == 64 && !EpiTraits<EPI>::kC8Out)
        while (S < 8 && tiles64 * S * 2 <= 8 * sms && k >= 128 * S) S *= 2;
    TiledProduct none{};
    TiledProduct p1 = q != nullptr ? *q : none;
    for (TiledProduct* x : {&p, &p1}) {
        x->mb = (x->a.M + bt - 1) / bt;
        x->nb = (x->a.N + bt - 1) / bt;
    }
    return timed(kind, flops, bytes, st, [&] {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(static_cast<unsigned>(bt == 128 ? tiles128 : tiles64), 1, static_cast<unsigned>(S));
        cfg.blockDim = dim3(bt == 128 ? 256 : 128);
        cfg.stream = st;
        cudaLaunchAttribute attr;
        attr.id = cudaLaunchAttributeClusterDimension;
        attr.val.clusterDim.x = 1;
        attr.val.clusterDim.y = 1;
        attr.val.clusterDim.z = static_cast<unsigned>(S);
        cfg.attrs = &attr;
        cfg.numAttrs = S > 1 ? 1 : 0;
        cudaError_t e;
        if (bt == 128) {
            e = cudaLaunchKernelEx(&cfg, simt_tiled_kernel<TI, TO, EPI, 128, false>, p, p1, S);
        } else if (S == 1) {
            e = cudaLaunchKernelEx(&cfg, simt_tiled_kernel<TI, TO, EPI, 64, false>, p, p1, S);
        } else if constexpr (!EpiTraits<EPI>::kC8Out) {
            e = cudaLaunchKernelEx(&cfg, simt_tiled_kernel<TI, TO, EPI, 64, true>, p, p1, S);
        }
        g_launches.fetch_add(1, std::memory_order_relaxed);
        if (e != cudaSuccess) cudaGetLastError();
        return e == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
    });
}

// Tiles of a plain product fit the grid (checked before a call's first launch).
bool plain_grid_ok(int64_t M, int64_t N) { return ((M + 63) / 64) * ((N + 63) / 64) < (int64_t(1) << 31); }

// Column tiles of the element-wise kernels (grid y) fit the grid.
bool columns_ok(int64_t n) { return (n + 255) / 256 <= kMaxGridY; }

// Aop(m, k), Bop(k, n) of one product by strides.
TiledProduct plain_args(int64_t M, int64_t N, int64_t K, const void* A, int64_t sam, int64_t sak, const void* B,
                        int64_t sbk, int64_t sbn, void* out) {
    TiledProduct p{};
    SimtArgs& a = p.a;
    a.M = static_cast<int>(M);
    a.N = static_cast<int>(N);
    a.K = static_cast<int>(K);
    a.A = A;
    a.sam = sam;
    a.sak = sak;
    a.B = B;
    a.sbk = sbk;
    a.sbn = sbn;
    a.out0 = out;
    a.ld_out = N;
    return p;
}

// ------------------------------------------------------------------ layer norm

// Shape of a norm kernel's blocks: `elems` elements per thread, `threads` per
// row, `rows` rows per block. threads = 0: the row does not fit the registers
// (looped kernels).
struct NormShape {
    int elems, threads, rows;
};

constexpr int kNormRows = 4;  // rows per block with one warp per row

// Forward. With few rows (no more than two per SM) latency counts: as many
// threads per row as there are. Else 64 bytes or more per thread keep enough
// of memory in flight. Measured on B200, µs at 8 / 16 / 32 elements: 1 row of
// 4096 bf16 2.6 / 3.1 / 3.6; 8192 rows 51 / 41 / 32 (fp32 50 / 46 / 44). Rows up
// to 1024 go to a warp each (1024 columns: 15.4 against 20-23 µs at 16384
// rows). Single elements do best with 8 per thread (4099 columns: 72 / 82 / 114).
NormShape norm_shape(int64_t T, int64_t h, bool vec) {
    auto fit = [&](int e, int most) {
        const int64_t t = ((h + e - 1) / e + 31) / 32 * 32;
        return t <= most ? static_cast<int>(t) : 0;
    };
    const bool few = T <= 2 * static_cast<int64_t>(plan_num_sms());
    if (vec && !few && h <= 1024) {
        for (int e : {8, 16, 32})
            if (h <= 32 * e) return {e, 32, kNormRows};
    }
    if (vec && !few && fit(32, 1024) > 0) return {32, fit(32, 1024), 1};
    for (int e : {8, 16, 32}) {
        const int t = fit(e, 1024);
        if (t > 0) return {e, t, t == 32 ? kNormRows : 1};
    }
    return {0, 0, 1};
}

// Shape of the backward kernel of rows that are not whole vectors
// (norm_bwd_kernel): 8 columns per thread up to 4096, else 16 (up to 128
// registers a thread). threads = 0: wider rows (looped kernels).
NormShape norm_scalar_shape(int64_t h) {
    const int e = h <= 8 * 512 ? 8 : 16;
    const int64_t t = ((h + e - 1) / e + 31) / 32 * 32;
    return NormShape{e, t <= 512 ? static_cast<int>(t) : 0, 1};
}

// Its blocks (each leaves one partial row of dgamma and dbeta).
int64_t norm_bwd_blocks(int64_t T, const NormShape& s) {
    if (s.threads == 0) return std::max<int64_t>(1, std::min<int64_t>((T + 127) / 128, 1024));
    return std::max<int64_t>(1, std::min<int64_t>(T, int64_t(plan_num_sms()) * std::min(16, std::max(1, 768 / s.threads))));
}

// Shape of the ring kernel (norm_bwd_ring_kernel) for rows of whole 16-byte
// vectors: `elems` elements per thread, `threads` per row, `rows` groups per
// block, `per_sm` blocks per SM, a ring of `stages` rows per group. threads =
// 0: not even one row of X, dY and dR fits a block's shared memory, or the row
// has more than 512 × 32 elements.
// The table is measured (B200, µs at 128 Mi elements or less, bf16): a warp per
// row up to 512 columns (512: 32 against 43 with blocks); 16 columns per thread
// from there (1024: 35 against 38 with 8 per thread and 79 with a warp per row
// and 32; 4096: 51.5 against 60 and 74), as many blocks as 64 K registers hold.
struct NormRingShape {
    int elems, threads, rows, per_sm, stages;
    bool gamma_shared;
};

// Dynamic shared memory of one block with `per_sm` resident: of 228 KB per SM
// a block costs 1 KB, may have 227 KB, and the kernel's static part needs 2 KB.
int64_t norm_ring_room(int per_sm) { return std::min(227, 228 / per_sm - 1) * int64_t(1024) - 2048; }

NormRingShape norm_ring_shape(int64_t h, int esize) {
    const NormRingShape none{0, 0, 1, 1, 0, false};
    NormRingShape s = none;
    const int64_t stage = 3 * h * esize, gamma = h * esize;
    if (h <= 512) {  // a warp per row
        s.elems = h <= 256 ? 8 : 16;
        s.threads = 32;
        s.rows = kNormRows;
        s.per_sm = 4;
    } else {
        s.elems = h <= 16 * 768 && (esize == 2 || 2 * stage + gamma <= norm_ring_room(1)) ? 16 : 32;
        const int64_t t = ((h + s.elems - 1) / s.elems + 31) / 32 * 32;
        if (t > (s.elems == 16 ? 768 : 512)) return none;
        s.threads = static_cast<int>(t);
        s.per_sm = t <= 64 ? 8 : t <= 128 ? 4 : t <= 256 ? 2 : 1;
    }
    auto fit = [&] { return (norm_ring_room(s.per_sm) - gamma) / (stage * s.rows); };
    while (s.per_sm > 1 && fit() < 3) --s.per_sm;
    s.gamma_shared = fit() >= 2;
    s.stages = static_cast<int>(s.gamma_shared ? std::min<int64_t>(fit(), 4) : 1);
    if (!s.gamma_shared && (stage > norm_ring_room(1) || s.elems != 32)) return none;
    return s;
}

int64_t norm_ring_blocks(int64_t T, const NormRingShape& s) {
    return std::max<int64_t>(1, std::min<int64_t>((T + s.rows - 1) / s.rows, int64_t(plan_num_sms()) * s.per_sm));
}

size_t norm_workspace(int64_t T, int64_t h, tpmlp_dtype dt) {
    const int esize = dt == TPMLP_BF16 ? 2 : 4;
    int64_t blocks = norm_bwd_blocks(T, norm_scalar_shape(h));
    if (h % (16 / esize) == 0) {
        const NormRingShape ring = norm_ring_shape(h, esize);
        if (ring.threads > 0) blocks = std::max(blocks, norm_ring_blocks(T, ring));
    }
    return 2 * round256(static_cast<size_t>(blocks) * h * sizeof(float));
}

// Lets `kern` use any dynamic shared memory that norm_ring_shape asks for
// (once per device).
template <auto KERNEL>
tpmlp_status allow_ring_smem() {
    static std::atomic<bool> set[kMaxDevices] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TPMLP_ERR_CUDA;
    if (!set[dev].load()) {
        if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 static_cast<int>(norm_ring_room(1))) != cudaSuccess)
            return TPMLP_ERR_CUDA;
        set[dev].store(true);
    }
    return TPMLP_OK;
}

template <typename T, int NV, bool WARP, int MAX_THREADS, int PER_SM, bool KEEP, bool ONE = false>
tpmlp_status norm_ring_launch(const NormRingShape& s, const T* dY, const T* X, const T* gamma, const float* mean,
                              const float* rstd, const T* dR, T* dX, float* pg, float* pb, int64_t blocks, int64_t R,
                              int64_t h, cudaStream_t st) {
    TPMLP_TRY((allow_ring_smem<norm_bwd_ring_kernel<T, NV, WARP, MAX_THREADS, PER_SM, KEEP, ONE>>()));
    // the rings, and gamma behind them
    const size_t smem = (static_cast<size_t>(s.rows) * s.stages * (dR != nullptr ? 3 : 2) + (s.gamma_shared ? 1 : 0)) *
                        h * sizeof(T);
    return launch_dep(norm_bwd_ring_kernel<T, NV, WARP, MAX_THREADS, PER_SM, KEEP, ONE>,
                      dim3(static_cast<unsigned>(blocks)), dim3(s.threads, s.rows), smem, st, dY, X, gamma, mean,
                      rstd, dR, dX, pg, pb, R, static_cast<int>(h),
                      NormRing{s.stages, g_wait_limit_ns.load()});
}

template <typename T>
tpmlp_status norm_ring(const NormRingShape& s, const T* dY, const T* X, const T* gamma, const float* mean,
                       const float* rstd, const T* dR, T* dX, float* pg, float* pb, int64_t blocks, int64_t R,
                       int64_t h, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(T);
#define TPMLP_RING(NV, ...) \
    norm_ring_launch<T, NV, __VA_ARGS__>(s, dY, X, gamma, mean, rstd, dR, dX, pg, pb, blocks, R, h, st)
    if (s.threads == 32)
        return s.elems == 8 ? TPMLP_RING(8 / kVec, true, 32 * kNormRows, 4, true)
                            : TPMLP_RING(16 / kVec, true, 32 * kNormRows, 4, true);
    if (s.elems == 16) {
        // registers a thread: 128 up to 512 threads per SM, 80 at 768
        if (s.threads <= 256) return TPMLP_RING(16 / kVec, false, 256, 2, true);
        return s.threads <= 512 ? TPMLP_RING(16 / kVec, false, 512, 1, true)
                                : TPMLP_RING(16 / kVec, false, 768, 1, false);
    }
    return s.gamma_shared ? TPMLP_RING(32 / kVec, false, 512, 1, false)
                          : TPMLP_RING(32 / kVec, false, 512, 1, false, true);
#undef TPMLP_RING
}

template <typename T>
tpmlp_status norm_fwd_impl(const void* X_, const void* gamma_, const void* beta_, void* Y_, float* mean,
                           float* rstd, int64_t R, int64_t h, float eps, cudaStream_t st) {
    constexpr int kVec = 16 / sizeof(T);
    const bool vec = h % kVec == 0 && aligned16(X_) && aligned16(Y_) && aligned16(gamma_) && aligned16(beta_);
    const NormShape s = norm_shape(R, h, vec);
    const T *X = static_cast<const T*>(X_), *gamma = static_cast<const T*>(gamma_),
            *beta = static_cast<const T*>(beta_);
    T* Y = static_cast<T*>(Y_);
    return timed(K_N_FWD, 0.0, sizeof(T) * (2.0 * R * h + 2.0 * h) + 8.0 * R, st, [&] {
        if (s.threads == 0)
            return launch_dep(norm_fwd_wide_kernel<T>, dim3(static_cast<unsigned>(R)), dim3(1024), 0, st, X, gamma,
                              beta, Y, mean, rstd, h, eps);
        const dim3 grid(static_cast<unsigned>((R + s.rows - 1) / s.rows)), block(s.threads, s.rows);
        auto kern = vec ? (s.elems == 8    ? norm_fwd_kernel<T, 8 / kVec>
                           : s.elems == 16 ? norm_fwd_kernel<T, 16 / kVec>
                                           : norm_fwd_kernel<T, 32 / kVec>)
                        : (s.elems == 8    ? norm_fwd_scalar_kernel<T, 8>
                           : s.elems == 16 ? norm_fwd_scalar_kernel<T, 16>
                                           : norm_fwd_scalar_kernel<T, 32>);
        return launch_dep(kern, grid, block, 0, st, X, gamma, beta, Y, mean, rstd, R, static_cast<int>(h),
                          1.0f / static_cast<float>(h), eps);
    });
}

template <typename T>
tpmlp_status norm_bwd_impl(const void* dY, const void* X, const void* gamma, const float* mean,
                           const float* rstd, const void* dR, void* dX, float* dgamma, float* dbeta, int64_t R,
                           int64_t h, void* workspace, cudaStream_t st) {
    const bool vec = h % (16 / sizeof(T)) == 0 && aligned16(dY) && aligned16(X) && aligned16(gamma) &&
                     aligned16(dR) && aligned16(dX);
    const NormShape s = norm_scalar_shape(h);
    const NormRingShape ring = vec ? norm_ring_shape(h, sizeof(T)) : NormRingShape{0, 0, 1, 1, 0, false};
    const int64_t blocks = ring.threads > 0 ? norm_ring_blocks(R, ring) : norm_bwd_blocks(R, s);
    float* pg = static_cast<float*>(workspace);
    float* pb = reinterpret_cast<float*>(static_cast<char*>(workspace) +
                                         round256(static_cast<size_t>(blocks) * h * sizeof(float)));
    const T* y = static_cast<const T*>(dY);
    const T* x = static_cast<const T*>(X);
    const T* g = static_cast<const T*>(gamma);
    const T* d = static_cast<const T*>(dR);
    T* dx = static_cast<T*>(dX);
    const double bytes = sizeof(T) * ((dR ? 4.0 : 3.0) * R * h + h) + 8.0 * R + 8.0 * blocks * h;
    TPMLP_TRY(timed(K_N_BWD, 0.0, bytes, st, [&]() -> tpmlp_status {
        if (ring.threads > 0) return norm_ring<T>(ring, y, x, g, mean, rstd, d, dx, pg, pb, blocks, R, h, st);
        if (s.threads == 0) {
            const dim3 cols(static_cast<unsigned>(blocks), static_cast<unsigned>((h + 255) / 256));
            TPMLP_TRY(launch_dep(norm_bwd_wide_cols_kernel<T>, cols, dim3(256), 0, st, y, x, mean, rstd, pg, pb,
                                 R, h, (R + blocks - 1) / blocks));
            return launch_dep(norm_bwd_wide_kernel<T>, dim3(static_cast<unsigned>(R)), dim3(1024), 0, st, y, x,
                              g, mean, rstd, d, dx, h);
        }
        const dim3 grid(static_cast<unsigned>(blocks)), block(s.threads);
        if (s.elems == 8)
            return launch_dep(norm_bwd_kernel<T, 8>, grid, block, 0, st, y, x, g, mean, rstd, d, dx, pg, pb, R,
                              static_cast<int>(h));
        return launch_dep(norm_bwd_kernel<T, 16>, grid, block, 0, st, y, x, g, mean, rstd, d, dx, pg, pb, R,
                          static_cast<int>(h));
    }));
    return colsum_finish2(K_N_DGB, pg, blocks, h, dgamma, pb, blocks, h, dbeta, st);
}

// -------------------------------------------- linear layer, fused epilogue

// CTAs of a cluster that share a tile's K range (gemm_few.cuh): the power of
// two up to 8 that fills the resident CTAs without a second wave and leaves
// each at least two k-blocks. A CTA alone on its SM streams 44 to 51 GB/s (the
// S = 1 times below), however much its ring holds, so what counts is that all
// SMs load. Measured on B200 (µs, S = 1 / 2 / 4 / 8): 24 rows, 16384 → 4096 (32 tiles) 82 / 45 / 27 / 24; 1
// row, 4096 → 16384 (128 tiles) 24.0 / 23.9 / 27 / 34; 16 rows, 4096 → 1024
// (8 tiles) 23 / 14 / 8.5 / 5.9. Clusters of 3, 5, 6 or 7 leave SMs idle and
// gain nothing (1 row, 12288 → 12288: S = 2 52, S = 3 66).
int few_split(int64_t tiles, int64_t k_blocks, int ctas_per_sm) {
    int s = 1;
    while (s < 8 && tiles * s * 2 <= ctas_per_sm * plan_num_sms() && k_blocks >= 4 * s) s *= 2;
    return s;
}

template <int TN>
tpmlp_status gemm_few_launch(const void* X, const void* W, int T, int N, int K, FewArgs g, cudaStream_t st) {
    using Cfg = FewCfg<TN>;
    CUtensorMap tmW, tmX;
    if (!make_map(&tmW, W, K, N, kBK) || !make_map(&tmX, X, T, K, TN)) return TPMLP_ERR_CUDA;
    g.T = T;
    g.N = N;
    g.k_blocks = (K + kBK - 1) / kBK;
    g.wait_limit_ns = g_wait_limit_ns.load();
    auto kern = gemm_few_kernel<TN>;
    {
        std::lock_guard<std::mutex> lock(g_dev_mutex);
        static bool set[kMaxDevices] = {};  // guarded by the lock
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return TPMLP_ERR_CUDA;
        if (!set[dev]) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg::SMEM_BYTES) !=
                cudaSuccess)
                return TPMLP_ERR_CUDA;
            set[dev] = true;
        }
    }
    const int tiles = (N + kFewCols - 1) / kFewCols;
    const int S = few_split(tiles, g.k_blocks, Cfg::CTAS);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(static_cast<unsigned>(tiles * S));
    cfg.blockDim = dim3(kFewThreads);
    cfg.dynamicSmemBytes = Cfg::SMEM_BYTES;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = static_cast<unsigned>(S);
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = g_overlap.load(std::memory_order_relaxed) ? 2 : 1;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, tmW, tmX, g, S);
    g_launches.fetch_add(1, std::memory_order_relaxed);
    if (e != cudaSuccess) cudaGetLastError();
    return e == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

// Rows up to which the few-row kernel serves the forward: one tile of 128.
// Measured at 128 rows against the one-CTA kernel under its best schedule: 4096
// → 4096 15.4 against 31.5 µs, 16384 → 4096 33 against 62, 4096 → 16384 34.5
// against 35.3. A second tile would read W again.
constexpr int64_t kFewMaxRows = 128;

static_assert(kFewMaxRows >= kBM, "gemm_tc_pick relies on it");

tpmlp_status linear_few(int kind, const void* X, const void* W, const void* bias, const void* R, void* H, void* Y,
                        int T, int N, int K, tpmlp_activation act, cudaStream_t st) {
    FewArgs g{};
    g.act = static_cast<int>(act);
    g.bias = static_cast<const bf16*>(bias);
    g.resid = static_cast<const bf16*>(R);
    g.H = static_cast<bf16*>(H);
    g.Y = static_cast<bf16*>(Y);
    const double bytes = 2.0 * (double(T) * K + double(K) * N + (1.0 + (R != nullptr) + (H != nullptr)) * T * N);
    return timed(kind, 2.0 * T * N * K, bytes, st, [&] {
        if (T <= 16) return gemm_few_launch<16>(X, W, T, N, K, g, st);
        if (T <= 32) return gemm_few_launch<32>(X, W, T, N, K, g, st);
        if (T <= 64) return gemm_few_launch<64>(X, W, T, N, K, g, st);
        return gemm_few_launch<128>(X, W, T, N, K, g, st);
    });
}

// The forward's product with EPI (kResid) on the tensor cores.
template <int EPI>
tpmlp_status linear_ex_tc(const void* X, const void* W, int T, int N, int K, const SchedReq& req, const GemmArgs& g,
                          cudaStream_t st) {
    return gemm_tc<256, false, true, EPI>(K_L_FWD, X, W, T, N, K, req, g, st);
}

template <typename T>
tpmlp_status linear_ex_plain(tpmlp_activation act, bool keep, const TiledProduct& p, cudaStream_t st) {
    if (act == TPMLP_ACT_NONE) return gemm_plain<T, T, EPI_ADD>(K_L_FWD, p, st);
    if (act == TPMLP_GELU_ERF)
        return keep ? gemm_plain<T, T, EPI_GELU_ADD>(K_L_FWD, p, st) : gemm_plain<T, T, EPI_ACT_ADD>(K_L_FWD, p, st);
    return keep ? gemm_plain<T, T, EPI_GELU_ADD_TANH>(K_L_FWD, p, st)
                : gemm_plain<T, T, EPI_ACT_ADD_TANH>(K_L_FWD, p, st);
}

tpmlp_status linear_fwd_ex_impl(const void* X, const void* W, const void* bias, const void* R, void* H, void* Y,
                                int64_t T, int64_t K, int64_t N, int p, int split, tpmlp_dtype dt,
                                tpmlp_activation act, void* workspace, size_t workspace_bytes,
                                cudaStream_t st) {
    LinPlan pl;
    TPMLP_TRY(lin_checks(T, K, N, p, split, dt, &pl, workspace, workspace_bytes, false));
    if (act != TPMLP_ACT_NONE && !known_act(act)) return TPMLP_ERR_INVALID;
    if (act == TPMLP_ACT_NONE && H != nullptr) return TPMLP_ERR_INVALID;
    if (T == 0) return TPMLP_OK;
    if (!X || !W || !Y) return TPMLP_ERR_INVALID;
    if (!fits32(T) || !fits32(K) || !fits32(N)) return TPMLP_ERR_UNSUPPORTED;
    const int64_t es = size_of(dt);
    if (overlapping({{Y, T * N * es}, {H, T * N * es}},
                    {{X, T * K * es}, {W, K * N * es}, {bias, N * es}, {R == Y ? nullptr : R, T * N * es}}))
        return TPMLP_ERR_INVALID;
    // the relaying activation epilogues run whole tiles (kSplittable)
    const SchedReq req = (act != TPMLP_ACT_NONE && K >= kRelayMinKAct) ? SchedReq{} : pl.fwd;
    const bool splits = pl.tc && T > kFewMaxRows && req.kind != SCHED_TILES;
    if (splits && (workspace == nullptr || workspace_bytes < pl.total)) return TPMLP_ERR_WORKSPACE;
    const int iT = static_cast<int>(T), iK = static_cast<int>(K), iN = static_cast<int>(N);
    if (pl.tc) {
        for (const void* q : {X, W, bias, R, static_cast<const void*>(H), static_cast<const void*>(Y)})
            if (q && !aligned16(q)) return TPMLP_ERR_ALIGN;
        if (T <= kFewMaxRows) return linear_few(K_L_FWD, X, W, bias, R, H, Y, iT, iN, iK, act, st);
        GemmArgs g{};
        if (splits) set_split_space(g, workspace, pl.off_part, pl.off_ctr);
        if (splits) TPMLP_TRY(reset_counters(workspace, pl.off_ctr, pl.ctr_bytes, st));
        g.out0 = H != nullptr ? H : Y;
        g.out1 = Y;
        g.ld_out = N;
        g.bias = static_cast<const bf16*>(bias);
        g.resid = static_cast<const bf16*>(R);
        if (act == TPMLP_ACT_NONE)
            return R ? linear_ex_tc<EPI_ADD>(X, W, iT, iN, iK, req, g, st)
                     : linear_ex_tc<EPI_BIAS>(X, W, iT, iN, iK, req, g, st);
        if (act == TPMLP_GELU_ERF) {
            if (!H) return linear_ex_tc<EPI_ACT_ADD>(X, W, iT, iN, iK, req, g, st);
            return R ? linear_ex_tc<EPI_GELU_ADD>(X, W, iT, iN, iK, req, g, st)
                     : linear_ex_tc<EPI_GELU>(X, W, iT, iN, iK, req, g, st);
        }
        if (!H) return linear_ex_tc<EPI_ACT_ADD_TANH>(X, W, iT, iN, iK, req, g, st);
        return R ? linear_ex_tc<EPI_GELU_ADD_TANH>(X, W, iT, iN, iK, req, g, st)
                 : linear_ex_tc<EPI_GELU_TANH>(X, W, iT, iN, iK, req, g, st);
    }
    if (!plain_grid_ok(T, N)) return TPMLP_ERR_UNSUPPORTED;
    TiledProduct q = plain_args(T, N, K, X, K, 1, W, N, 1, H != nullptr ? H : Y);
    q.a.out1 = Y;
    q.a.bias = bias;
    q.resid = R;
    if (dt == TPMLP_FP32) return linear_ex_plain<float>(act, H != nullptr, q, st);
    return linear_ex_plain<bf16>(act, H != nullptr, q, st);
}

// Rows per block of act_grad_kernel: all 32 in flight at once, and blocks small
// enough that a last, partly filled wave of them costs little (with 128 rows,
// 6144 × 4096 is 1.04 waves of 740 blocks: 44 µs, against 32).
constexpr int64_t kActGradRows = 32;

int64_t act_grad_chunks(int64_t T) { return T > 0 ? (T + kActGradRows - 1) / kActGradRows : 1; }

// Workspace of the linear layer's calls: its plan's, with room for the partial
// column sums of the activation's pass.
size_t lin_ex_total(const LinPlan& pl, int64_t T, int64_t N) {
    return pl.off_cs + round256(static_cast<size_t>(act_grad_chunks(T)) * N * sizeof(float));
}

template <typename T, bool TANH>
tpmlp_status act_grad_launch(const void* dY, const void* H, void* dH, int64_t R, int64_t C, int64_t chunks,
                             float* partial, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>(chunks), static_cast<unsigned>((C + 255) / 256));
    const T *y = static_cast<const T*>(dY), *x = static_cast<const T*>(H);
    if (C % 8 == 0 && aligned16(dY) && aligned16(H) && aligned16(dH))
        return launch_dep(act_grad_kernel<T, TANH, true>, grid, dim3(32, 8), 0, st, y, x, static_cast<T*>(dH), R,
                          C, kActGradRows, partial);
    return launch_dep(act_grad_kernel<T, TANH, false>, grid, dim3(32, 8), 0, st, y, x, static_cast<T*>(dH), R, C,
                      kActGradRows, partial);
}

// TG: type of dW and dbias. T: type of the rest.
template <typename T, typename TG>
tpmlp_status linear_bwd_ex_run(const LinPlan& pl, const void* dY, const void* X, const void* W, const void* H,
                               void* dX, void* dW, void* dbias, void* dH, int64_t R, int64_t K, int64_t N,
                               tpmlp_activation act, void* workspace, cudaStream_t st) {
    float* cs = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_cs);
    TG* db = static_cast<TG*>(dbias);
    const void* g = dY;
    if (act == TPMLP_ACT_NONE) {
        TPMLP_TRY(colsum(K_L_DB, static_cast<const T*>(dY), R, N, pl.chunks, cs, db, st));
    } else {
        g = dH;
        const int64_t chunks = act_grad_chunks(R);
        TPMLP_TRY(timed(K_L_DH, 0.0, 3.0 * sizeof(T) * double(R) * N, st, [&] {
            return act == TPMLP_GELU_TANH ? act_grad_launch<T, true>(dY, H, dH, R, N, chunks, cs, st)
                                          : act_grad_launch<T, false>(dY, H, dH, R, N, chunks, cs, st);
        }));
        TPMLP_TRY(timed(K_L_DB, 0.0, 4.0 * (double(chunks) + 1) * N, st, [&] {
            return launch_dep(colsum_final_kernel<TG>, dim3(static_cast<unsigned>((N + 31) / 32)), dim3(32, 8), 0,
                              st, static_cast<const float*>(cs), static_cast<int>(chunks), N, db);
        }));
    }
    if constexpr (sizeof(T) == 2) {
        if (pl.tc) {
            const int iT = static_cast<int>(R), iK = static_cast<int>(K), iN = static_cast<int>(N);
            GemmArgs gw{};
            set_split_space(gw, workspace, pl.off_part, pl.off_ctr);
            if (pl.bwd_split)
                TPMLP_TRY(zero_counters_before(gw, pl.dw, workspace, pl.off_ctr, pl.ctr_bytes, st));
            gw.out0 = dW;
            gw.ld_out = N;
            TPMLP_TRY((gemm_tc<256, true, true, sizeof(TG) == 2 ? EPI_BIAS : EPI_F32>(K_L_DW, X, g, iK, iN, iT, pl.dw,
                                                                                     gw, st)));
            GemmArgs gx{};
            set_split_space(gx, workspace, pl.off_part, pl.off_ctr);
            gx.out0 = dX;
            gx.ld_out = K;
            return gemm_tc<256, false, false, EPI_BIAS>(K_L_DX, g, W, iT, iK, iN, pl.dx, gx, st);
        }
    }
    TPMLP_TRY((gemm_plain<T, TG, EPI_F32>(K_L_DW, plain_args(K, N, R, X, 1, K, g, N, 1, dW), st)));
    return gemm_plain<T, T, EPI_F32>(K_L_DX, plain_args(R, K, N, g, N, 1, W, 1, N, dX), st);
}

// ------------------------------------------------------------ 8-bit checkpoint

int64_t c8_blocks(int64_t F) { return (F + kC8Block - 1) / kC8Block; }

template <typename T>
tpmlp_status ckpt8_encode_launch(const void* H, void* C, void* S, int64_t R, int64_t F, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((R + 31) / 32), static_cast<unsigned>((F + 255) / 256));
    auto kern = F % 8 == 0 && aligned16(H) ? ckpt8_encode_kernel<T, true> : ckpt8_encode_kernel<T, false>;
    return launch_dep(kern, grid, dim3(256), 0, st, static_cast<const T*>(H), static_cast<uint8_t*>(C),
                      static_cast<uint8_t*>(S), R, F);
}

template <typename T>
tpmlp_status ckpt8_decode_launch(const void* C, const void* S, void* H, int64_t R, int64_t F, cudaStream_t st) {
    const dim3 grid(static_cast<unsigned>((R + 31) / 32), static_cast<unsigned>((F + 255) / 256));
    constexpr int W = 16 / static_cast<int>(sizeof(T));
    auto kern = F % W == 0 && aligned16(H) ? ckpt8_decode_kernel<T, W> : ckpt8_decode_kernel<T, 1>;
    return launch_dep(kern, grid, dim3(256), 0, st, static_cast<const uint8_t*>(C),
                      static_cast<const uint8_t*>(S), static_cast<T*>(H), R, F);
}

tpmlp_status c8_checks(int64_t T, int64_t h, int64_t F, int p, tpmlp_dtype dt, tpmlp_activation act, Plan* pl,
                       void* ws, size_t ws_bytes, bool need_ws) {
    if (!known_act(act)) return TPMLP_ERR_INVALID;
    TPMLP_TRY(common_checks(T, h, F, p, dt, pl, ws, ws_bytes, need_ws));
    if (!fits32(T) || !fits32(h) || !fits32(F)) return TPMLP_ERR_UNSUPPORTED;
    if (!plain_grid_ok(T, F) || !plain_grid_ok(T, h) || !plain_grid_ok(h, F) || pl->chunks > kMaxGridY)
        return TPMLP_ERR_UNSUPPORTED;
    return TPMLP_OK;
}

template <int EPI>
tpmlp_status c8_fwd_tc(const Plan& pl, const void* X, const void* A, const void* a, const void* B, const void* b,
                       const void* R, void* C, void* S, void* Y, void* Z, int64_t T, int64_t h, int64_t F,
                       void* workspace, cudaStream_t st) {
    const int iT = static_cast<int>(T), ih = static_cast<int>(h), iF = static_cast<int>(F);
    // (a workspace is there only if some product splits or runs dynamically)
    GemmArgs g1{};
    if (workspace != nullptr) {
        set_split_space(g1, workspace, pl.off_part, pl.off_ctr);
        g1.dyn_counter = dyn_space(workspace, pl.off_dyn);
    }
    if (pl.fwd_dyn)
        TPMLP_TRY(reset_counters(workspace, pl.off_ctr, pl.ctr_bytes, st));
    else if (pl.fwd_split)
        TPMLP_TRY(zero_counters_before(g1, pl.f1, workspace, pl.off_ctr, pl.ctr_bytes, st));
    g1.out0 = Y;
    g1.ld_out = F;
    g1.bias = static_cast<const bf16*>(a);
    g1.c8 = static_cast<uint8_t*>(C);
    g1.c8_scale = static_cast<uint8_t*>(S);
    g1.c8_ld = c8_blocks(F) * kC8Block;
    TPMLP_TRY((gemm_tc<256, false, true, EPI>(K_F1, X, A, iT, iF, ih, pl.f1, g1, st)));
    if (T <= kFewMaxRows) return linear_few(K_F2, Y, B, b, R, nullptr, Z, iT, ih, iF, TPMLP_ACT_NONE, st);
    GemmArgs g2{};
    if (workspace != nullptr) {
        set_split_space(g2, workspace, pl.off_part, pl.off_ctr);
        g2.dyn_counter = dyn_space(workspace, pl.off_dyn);
    }
    g2.out0 = Z;
    g2.ld_out = h;
    g2.bias = static_cast<const bf16*>(b);
    g2.resid = static_cast<const bf16*>(R);
    if (R) return gemm_tc<256, false, true, EPI_ADD>(K_F2, Y, B, iT, ih, iF, pl.f2, g2, st);
    return gemm_tc<256, false, true, EPI_BIAS>(K_F2, Y, B, iT, ih, iF, pl.f2, g2, st);
}

void set_c8(TiledProduct& p, const void* C, const void* S, int64_t F) {
    p.c8 = static_cast<uint8_t*>(const_cast<void*>(C));
    p.c8_scale = static_cast<uint8_t*>(const_cast<void*>(S));
    p.c8_ld = c8_blocks(F) * kC8Block;
}

template <typename T>
tpmlp_status c8_fwd_plain(const void* X, const void* A, const void* a, const void* B, const void* b, const void* R,
                          void* C, void* S, void* Y, void* Z, int64_t rows, int64_t h, int64_t F,
                          tpmlp_activation act, cudaStream_t st) {
    TiledProduct p1 = plain_args(rows, F, h, X, h, 1, A, F, 1, Y);
    p1.a.bias = a;
    set_c8(p1, C, S, F);
    TPMLP_TRY((act == TPMLP_GELU_TANH ? gemm_plain<T, T, EPI_GELU_C8_TANH>(K_F1, p1, st)
                                      : gemm_plain<T, T, EPI_GELU_C8>(K_F1, p1, st)));
    TiledProduct p2 = plain_args(rows, h, F, Y, F, 1, B, h, 1, Z);
    p2.a.bias = b;
    p2.resid = R;
    return gemm_plain<T, T, EPI_ADD>(K_F2, p2, st);
}

template <int EPI, typename TG>
tpmlp_status c8_bwd_tc(const Plan& pl, const void* dZ, const void* X, const void* A, const void* B, const void* C,
                       const void* S, void* dX, TG* dA, TG* da, TG* dB, TG* db, void* dH, void* Y, int64_t T,
                       int64_t h, int64_t F, void* workspace, cudaStream_t st) {
    constexpr int kGrad = sizeof(TG) == 2 ? EPI_BIAS : EPI_F32;
    const int iT = static_cast<int>(T), ih = static_cast<int>(h), iF = static_cast<int>(F);
    const bf16* dZb = static_cast<const bf16*>(dZ);
    float* cs_h = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_cs_h);
    float* cs_f = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_cs_f);
    int* dyn = dyn_space(workspace, pl.off_dyn);
    if (pl.bwd_dyn) TPMLP_TRY(reset_counters(workspace, pl.off_ctr, pl.ctr_bytes, st));
    // column sums as in bwd_impl: da's partials from the relaying epilogue for
    // long K, else both sums after the product
    const bool fused_da = h >= kRelayMinKAct;
    if (fused_da) TPMLP_TRY(colsum_first(K_B1_DB, dZb, T, h, pl.chunks, cs_h, st));
    GemmArgs g2{};
    set_split_space(g2, workspace, pl.off_part, pl.off_ctr);
    g2.dyn_counter = dyn;
    if (pl.bwd_split && !pl.bwd_dyn)
        TPMLP_TRY(zero_counters_before(g2, pl.b2, workspace, pl.off_ctr, pl.ctr_bytes, st));
    g2.out0 = dH;
    g2.out1 = Y;
    g2.ld_out = F;
    g2.c8 = static_cast<uint8_t*>(const_cast<void*>(C));
    g2.c8_scale = static_cast<uint8_t*>(const_cast<void*>(S));
    g2.c8_ld = c8_blocks(F) * kC8Block;
    g2.colsum_out = fused_da ? cs_f : nullptr;
    TPMLP_TRY((gemm_tc<256, false, false, EPI>(K_B2, dZ, B, iT, iF, ih, pl.b2, g2, st)));
    if (fused_da)
        TPMLP_TRY(colsum_finish2(K_B12, cs_h, pl.chunks, h, db, cs_f, da_partial_rows(T), F, da, st));
    else
        TPMLP_TRY(colsum2(K_B12, dZb, h, cs_h, db, static_cast<const bf16*>(dH), F, cs_f, da, T, pl.chunks, st));
    if (pl.group34) {
        TPMLP_TRY((gemm_tc_grouped<256, true, true, kGrad>(K_B34, Y, dZ, iF, ih, dB, X, dH, ih, iF, dA, iT, st)));
    } else {
        GemmArgs g3{};
        set_split_space(g3, workspace, pl.off_part, pl.off_ctr);
        g3.out0 = dB;
        g3.ld_out = h;
        TPMLP_TRY((gemm_tc<256, true, true, kGrad>(K_B3, Y, dZ, iF, ih, iT, pl.b3, g3, st)));
        GemmArgs g4{};
        set_split_space(g4, workspace, pl.off_part, pl.off_ctr);
        g4.out0 = dA;
        g4.ld_out = F;
        TPMLP_TRY((gemm_tc<256, true, true, kGrad>(K_B4, X, dH, ih, iF, iT, pl.b4, g4, st)));
    }
    GemmArgs g5{};
    set_split_space(g5, workspace, pl.off_part, pl.off_ctr);
    g5.dyn_counter = dyn;
    g5.out0 = dX;
    g5.ld_out = h;
    return gemm_tc<256, false, false, EPI_BIAS>(K_B5, dH, A, iT, ih, iF, pl.b5, g5, st);
}

template <typename T, typename TG>
tpmlp_status c8_bwd_plain(const Plan& pl, const void* dZ, const void* X, const void* A, const void* B, const void* C,
                          const void* S, void* dX, TG* dA, TG* da, TG* dB, TG* db, void* dH, void* Y, int64_t rows,
                          int64_t h, int64_t F, tpmlp_activation act, void* workspace, cudaStream_t st) {
    float* cs_h = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_cs_h);
    float* cs_f = reinterpret_cast<float*>(static_cast<char*>(workspace) + pl.off_cs_f);
    TiledProduct p2 = plain_args(rows, F, h, dZ, h, 1, B, 1, h, dH);
    p2.a.out1 = Y;
    set_c8(p2, C, S, F);
    TPMLP_TRY((act == TPMLP_GELU_TANH ? gemm_plain<T, T, EPI_DGELU_C8_TANH>(K_B2, p2, st)
                                      : gemm_plain<T, T, EPI_DGELU_C8>(K_B2, p2, st)));
    TPMLP_TRY(colsum2(K_B12, static_cast<const T*>(dZ), h, cs_h, db, static_cast<const T*>(dH), F, cs_f, da, rows,
                      pl.chunks, st));
    const TiledProduct p4 = plain_args(h, F, rows, X, 1, h, dH, F, 1, dA);
    TPMLP_TRY((gemm_plain<T, TG, EPI_F32>(K_B34, plain_args(F, h, rows, Y, 1, F, dZ, h, 1, dB), st, &p4)));
    return gemm_plain<T, T, EPI_F32>(K_B5, plain_args(rows, h, F, dH, F, 1, A, 1, F, dX), st);
}

template <typename TG>
tpmlp_status c8_bwd_typed(const Plan& pl, const void* dZ, const void* X, const void* A, const void* B, const void* C,
                          const void* S, void* dX, void* dA, void* da, void* dB, void* db, void* dH, void* Y,
                          int64_t T, int64_t h, int64_t F, tpmlp_dtype dt, tpmlp_activation act,
                          void* workspace, cudaStream_t st) {
    TG *gA = static_cast<TG*>(dA), *ga = static_cast<TG*>(da), *gB = static_cast<TG*>(dB),
       *gb = static_cast<TG*>(db);
    if (pl.tc) {
        if (act == TPMLP_GELU_TANH)
            return c8_bwd_tc<EPI_DGELU_C8_TANH, TG>(pl, dZ, X, A, B, C, S, dX, gA, ga, gB, gb, dH, Y, T, h, F,
                                                    workspace, st);
        return c8_bwd_tc<EPI_DGELU_C8, TG>(pl, dZ, X, A, B, C, S, dX, gA, ga, gB, gb, dH, Y, T, h, F, workspace,
                                           st);
    }
    if constexpr (sizeof(TG) == 4) {
        if (dt == TPMLP_FP32)
            return c8_bwd_plain<float, TG>(pl, dZ, X, A, B, C, S, dX, gA, ga, gB, gb, dH, Y, T, h, F, act,
                                           workspace, st);
    }
    return c8_bwd_plain<bf16, TG>(pl, dZ, X, A, B, C, S, dX, gA, ga, gB, gb, dH, Y, T, h, F, act, workspace,
                                  st);
}

// n elements of type dt set to zero (an all-zero pattern in either type).
tpmlp_status zero_any(void* p, int64_t n, tpmlp_dtype dt, cudaStream_t st) {
    if (dt == TPMLP_FP32) return zero_f32(static_cast<float*>(p), n, st);
    return cudaMemsetAsync(p, 0, static_cast<size_t>(n) * 2, st) == cudaSuccess ? TPMLP_OK : TPMLP_ERR_CUDA;
}

}  // namespace
}  // namespace tpmlp

extern "C" {

size_t tpmlp_layernorm_workspace_size(int64_t T, int64_t h, tpmlp_dtype dt) {
    if (T < 0 || h < 1 || !fits32(T) || !fits32(h) || !known_dtype(dt)) return 0;
    return norm_workspace(T, h, dt);
}

tpmlp_status tp_layernorm_fwd(const void* X, const void* gamma, const void* beta, void* Y, float* mean, float* rstd,
                              int64_t T, int64_t h, float eps, tpmlp_dtype dt, void* stream) {
    cudaGetLastError();
    // eps >= 0 and finite; a NaN fails both comparisons
    if (T < 0 || h < 1 || !known_dtype(dt) || !(eps >= 0.0f && eps <= 3.0e38f)) return TPMLP_ERR_INVALID;
    if ((mean == nullptr) != (rstd == nullptr)) return TPMLP_ERR_INVALID;
    if (T > 0 && (!X || !Y)) return TPMLP_ERR_INVALID;
    if (!fits32(T) || !fits32(h)) return TPMLP_ERR_UNSUPPORTED;
    const int64_t es = size_of(dt);
    if (overlapping({{Y, T * h * es}, {mean, T * 4}, {rstd, T * 4}},
                    {{X, T * h * es}, {gamma, h * es}, {beta, h * es}}))
        return TPMLP_ERR_INVALID;
    TPMLP_TRY(check_device());
    if (T == 0) return TPMLP_OK;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (dt == TPMLP_BF16) return norm_fwd_impl<bf16>(X, gamma, beta, Y, mean, rstd, T, h, eps, st);
    return norm_fwd_impl<float>(X, gamma, beta, Y, mean, rstd, T, h, eps, st);
}

tpmlp_status tp_layernorm_bwd(const void* dY, const void* X, const void* gamma, const float* mean,
                              const float* rstd, const void* dR, void* dX, float* dgamma, float* dbeta, int64_t T,
                              int64_t h, tpmlp_dtype dt, void* workspace, size_t workspace_bytes, void* stream) {
    cudaGetLastError();
    if (T < 0 || h < 1 || !known_dtype(dt) || !dgamma || !dbeta) return TPMLP_ERR_INVALID;
    if (T > 0 && (!dY || !X || !mean || !rstd || !dX)) return TPMLP_ERR_INVALID;
    if (!fits32(T) || !fits32(h) || (h + 255) / 256 > kMaxGridY) return TPMLP_ERR_UNSUPPORTED;
    TPMLP_TRY(check_device());
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        TPMLP_TRY(zero_f32(dgamma, h, st));
        return zero_f32(dbeta, h, st);
    }
    if (workspace == nullptr || workspace_bytes < norm_workspace(T, h, dt)) return TPMLP_ERR_WORKSPACE;
    if (!aligned16(workspace)) return TPMLP_ERR_ALIGN;
    const int64_t es = size_of(dt);
    if (overlapping({{dX, T * h * es}, {dgamma, h * 4}, {dbeta, h * 4}},
                    {{dX == dY ? nullptr : dY, T * h * es}, {X, T * h * es}, {gamma, h * es}, {mean, T * 4},
                     {rstd, T * 4}, {dX == dR ? nullptr : dR, T * h * es}}))
        return TPMLP_ERR_INVALID;
    if (dt == TPMLP_BF16)
        return norm_bwd_impl<bf16>(dY, X, gamma, mean, rstd, dR, dX, dgamma, dbeta, T, h, workspace, st);
    return norm_bwd_impl<float>(dY, X, gamma, mean, rstd, dR, dX, dgamma, dbeta, T, h, workspace, st);
}

size_t tpmlp_linear_ex_workspace_size(int64_t T, int64_t K, int64_t N, int p, tpmlp_split split, tpmlp_dtype dt) {
    LinPlan pl;
    if (!make_lin_plan(T, K, N, p, static_cast<int>(split), dt, &pl)) return 0;
    return lin_ex_total(pl, T, N);
}

tpmlp_status tp_linear_fwd_ex(const void* X, const void* W, const void* bias, const void* R, void* H, void* Y,
                              int64_t T, int64_t K, int64_t N, int p, tpmlp_split split, tpmlp_dtype dt,
                              tpmlp_activation act, void* workspace, size_t workspace_bytes, void* stream) {
    cudaGetLastError();
    return linear_fwd_ex_impl(X, W, bias, R, H, Y, T, K, N, p, static_cast<int>(split), dt, act, workspace,
                              workspace_bytes, static_cast<cudaStream_t>(stream));
}

tpmlp_status tp_linear_bwd_ex(const void* dY, const void* X, const void* W, const void* H, void* dX, void* dW,
                              void* dbias, void* dH, int64_t T, int64_t K, int64_t N, int p, tpmlp_split split,
                              tpmlp_dtype dt, tpmlp_dtype grad_dt, tpmlp_activation act, void* workspace,
                              size_t workspace_bytes, void* stream) {
    cudaGetLastError();
    LinPlan pl;
    TPMLP_TRY(lin_checks(T, K, N, p, static_cast<int>(split), dt, &pl, workspace, workspace_bytes));
    if (workspace_bytes < lin_ex_total(pl, T, N)) return TPMLP_ERR_WORKSPACE;
    if (!known_grad(grad_dt, dt) || (act != TPMLP_ACT_NONE && !known_act(act))) return TPMLP_ERR_INVALID;
    if (!dW || !dbias) return TPMLP_ERR_INVALID;
    if (act == TPMLP_ACT_NONE && (H || dH)) return TPMLP_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        TPMLP_TRY(zero_any(dW, K * N, grad_dt, st));
        return zero_any(dbias, N, grad_dt, st);
    }
    if (!dY || !X || !W || !dX || (act != TPMLP_ACT_NONE && (!H || !dH))) return TPMLP_ERR_INVALID;
    if (pl.tc) {
        for (const void* q : {dY, X, W, H, static_cast<const void*>(dX), static_cast<const void*>(dW),
                              static_cast<const void*>(dbias), static_cast<const void*>(dH)})
            if (q && !aligned16(q)) return TPMLP_ERR_ALIGN;
    }
    if (!fits32(T) || !fits32(K) || !fits32(N) || !columns_ok(N) || !plain_grid_ok(K, N) ||
        !plain_grid_ok(T, K) || pl.chunks > kMaxGridY)
        return TPMLP_ERR_UNSUPPORTED;
    const int64_t es = size_of(dt), eg = size_of(grad_dt);
    if (overlapping({{dX, T * K * es}, {dW, K * N * eg}, {dbias, N * eg}, {dH, T * N * es}},
                    {{dY, T * N * es}, {X, T * K * es}, {W, K * N * es}, {H, T * N * es}}))
        return TPMLP_ERR_INVALID;
    if (dt == TPMLP_FP32)
        return linear_bwd_ex_run<float, float>(pl, dY, X, W, H, dX, dW, dbias, dH, T, K, N, act, workspace, st);
    if (grad_dt == TPMLP_BF16)
        return linear_bwd_ex_run<bf16, bf16>(pl, dY, X, W, H, dX, dW, dbias, dH, T, K, N, act, workspace, st);
    return linear_bwd_ex_run<bf16, float>(pl, dY, X, W, H, dX, dW, dbias, dH, T, K, N, act, workspace, st);
}

size_t tpmlp_ckpt8_workspace_size(int64_t T, int64_t h, int64_t F, int p, tpmlp_dtype dt) {
    return tpmlp_workspace_size(T, h, F, p, dt);
}

tpmlp_status tp_mlp_fwd_ckpt8(const void* X, const void* A, const void* a, const void* B, const void* b,
                              const void* R, void* C, void* S, void* Y, void* Z, int64_t T, int64_t h, int64_t F,
                              int p, tpmlp_dtype dt, tpmlp_activation act, void* workspace, size_t workspace_bytes,
                              void* stream) {
    cudaGetLastError();
    Plan pl;
    TPMLP_TRY(c8_checks(T, h, F, p, dt, act, &pl, workspace, workspace_bytes, false));
    if (T == 0) return TPMLP_OK;
    if (!X || !A || !B || !C || !S || !Y || !Z) return TPMLP_ERR_INVALID;
    // up to kFewMaxRows rows the second product is the few-row kernel's, which splits no tiles
    if (pl.tc && T <= kFewMaxRows) {
        pl.f2 = SchedReq{};
        pl.fwd_split = pl.f1.kind != SCHED_TILES;
    }
    if ((pl.fwd_split || pl.fwd_dyn) && (workspace == nullptr || workspace_bytes < pl.total))
        return TPMLP_ERR_WORKSPACE;
    if (!pl.fwd_split && !pl.fwd_dyn) workspace = nullptr;
    if (!aligned16(C)) return TPMLP_ERR_ALIGN;
    const int64_t es = size_of(dt), blocks = c8_blocks(F);
    if (overlapping({{C, T * blocks * kC8Block}, {S, T * blocks}, {Y, T * F * es}, {Z, T * h * es}},
                    {{X, T * h * es}, {A, h * F * es}, {a, F * es}, {B, F * h * es}, {b, h * es},
                     {R == Z ? nullptr : R, T * h * es}}))
        return TPMLP_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (pl.tc) {
        for (const void* q : {X, A, a, B, b, R, static_cast<const void*>(Y), static_cast<const void*>(Z)})
            if (q && !aligned16(q)) return TPMLP_ERR_ALIGN;
        if (act == TPMLP_GELU_TANH)
            return c8_fwd_tc<EPI_GELU_C8_TANH>(pl, X, A, a, B, b, R, C, S, Y, Z, T, h, F, workspace, st);
        return c8_fwd_tc<EPI_GELU_C8>(pl, X, A, a, B, b, R, C, S, Y, Z, T, h, F, workspace, st);
    }
    if (dt == TPMLP_FP32) return c8_fwd_plain<float>(X, A, a, B, b, R, C, S, Y, Z, T, h, F, act, st);
    return c8_fwd_plain<bf16>(X, A, a, B, b, R, C, S, Y, Z, T, h, F, act, st);
}

tpmlp_status tp_mlp_bwd_ckpt8(const void* dZ, const void* X, const void* A, const void* B, const void* C,
                              const void* S, void* dX, void* dA, void* da, void* dB, void* db, void* dH, void* Y,
                              int64_t T, int64_t h, int64_t F, int p, tpmlp_dtype dt, tpmlp_dtype grad_dt,
                              tpmlp_activation act, void* workspace, size_t workspace_bytes, void* stream) {
    cudaGetLastError();
    Plan pl;
    TPMLP_TRY(c8_checks(T, h, F, p, dt, act, &pl, workspace, workspace_bytes, true));
    if (!known_grad(grad_dt, dt) || !dA || !da || !dB || !db) return TPMLP_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    if (T == 0) {
        TPMLP_TRY(zero_any(dA, h * F, grad_dt, st));
        TPMLP_TRY(zero_any(da, F, grad_dt, st));
        TPMLP_TRY(zero_any(dB, F * h, grad_dt, st));
        return zero_any(db, h, grad_dt, st);
    }
    if (!dZ || !X || !A || !B || !C || !S || !dX || !dH || !Y) return TPMLP_ERR_INVALID;
    if (!aligned16(C)) return TPMLP_ERR_ALIGN;
    const int64_t es = size_of(dt), eg = size_of(grad_dt), blocks = c8_blocks(F);
    if (overlapping({{dX, T * h * es}, {dA, h * F * eg}, {da, F * eg}, {dB, F * h * eg}, {db, h * eg},
                     {dH, T * F * es}, {Y, T * F * es}},
                    {{dZ, T * h * es}, {X, T * h * es}, {A, h * F * es}, {B, F * h * es},
                     {C, T * blocks * kC8Block}, {S, T * blocks}}))
        return TPMLP_ERR_INVALID;
    if (pl.tc) {
        for (const void* q : {dZ, X, A, B, static_cast<const void*>(dX), static_cast<const void*>(dA),
                              static_cast<const void*>(da), static_cast<const void*>(dB),
                              static_cast<const void*>(db), static_cast<const void*>(dH),
                              static_cast<const void*>(Y)})
            if (!aligned16(q)) return TPMLP_ERR_ALIGN;
    }
    if (grad_dt == TPMLP_BF16)
        return c8_bwd_typed<bf16>(pl, dZ, X, A, B, C, S, dX, dA, da, dB, db, dH, Y, T, h, F, dt, act,
                                  workspace, st);
    return c8_bwd_typed<float>(pl, dZ, X, A, B, C, S, dX, dA, da, dB, db, dH, Y, T, h, F, dt, act, workspace,
                               st);
}

tpmlp_status tpmlp_ckpt8_encode(const void* H, void* C, void* S, int64_t T, int64_t F, tpmlp_dtype dt,
                                void* stream) {
    cudaGetLastError();
    if (T < 0 || F < 1 || !known_dtype(dt) || (T > 0 && (!H || !C || !S))) return TPMLP_ERR_INVALID;
    if (!fits32(T) || !fits32(F) || !columns_ok(F)) return TPMLP_ERR_UNSUPPORTED;
    TPMLP_TRY(check_device());
    if (T == 0) return TPMLP_OK;
    if (!aligned16(C)) return TPMLP_ERR_ALIGN;
    const int64_t es = size_of(dt), blocks = c8_blocks(F);
    if (overlapping({{C, T * blocks * kC8Block}, {S, T * blocks}}, {{H, T * F * es}})) return TPMLP_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return timed(K_C8, 0.0, (es + 33.0 / 32.0) * T * F, st, [&] {
        return dt == TPMLP_BF16 ? ckpt8_encode_launch<bf16>(H, C, S, T, F, st)
                                : ckpt8_encode_launch<float>(H, C, S, T, F, st);
    });
}

tpmlp_status tpmlp_ckpt8_decode(const void* C, const void* S, void* H, int64_t T, int64_t F, tpmlp_dtype dt,
                                void* stream) {
    cudaGetLastError();
    if (T < 0 || F < 1 || !known_dtype(dt) || (T > 0 && (!H || !C || !S))) return TPMLP_ERR_INVALID;
    if (!fits32(T) || !fits32(F) || !columns_ok(F)) return TPMLP_ERR_UNSUPPORTED;
    TPMLP_TRY(check_device());
    if (T == 0) return TPMLP_OK;
    if (!aligned16(C)) return TPMLP_ERR_ALIGN;
    const int64_t es = size_of(dt), blocks = c8_blocks(F);
    if (overlapping({{H, T * F * es}}, {{C, T * blocks * kC8Block}, {S, T * blocks}})) return TPMLP_ERR_INVALID;
    cudaStream_t st = static_cast<cudaStream_t>(stream);
    return timed(K_C8, 0.0, (es + 33.0 / 32.0) * T * F, st, [&] {
        return dt == TPMLP_BF16 ? ckpt8_decode_launch<bf16>(C, S, H, T, F, st)
                                : ckpt8_decode_launch<float>(C, S, H, T, F, st);
    });
}

}  // extern "C"
