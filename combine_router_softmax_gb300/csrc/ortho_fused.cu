// ortho_fused.cu -- small matrices through all Newton-Schulz steps in one kernel.
//
// As three products a step, launched one after the other, a matrix of 128 rows takes 6 us a product whatever its
// work: launch, first copies, last stores. Up to 128 rows (of the wide form) X stays in shared memory instead, the
// same halves and roundings as in ortho_gemm.cuh: a cluster of up to eight CTAs takes a matrix, each CTA 256 of its
// columns, and only the sums of A's parts pass between them. One copy of hi serves as both operands of A = X X^T
// (128 bytes of a row's columns, swizzled) and, read the other way, as the second of B X. A and then B lie in
// one place; lo is read and written by the thread that owns it alone.
//
// What bounds it is the chain of a step: three waits for a few MMAs, three epilogues, as many fences and barriers.
#include "ortho_values.cuh"

namespace ep {

namespace {

constexpr int kFusedThreads = 512;
constexpr int kFusedRows = 128, kFusedCols = 256;  // of a CTA
constexpr int kFusedCtas = 8;                      // of a cluster, at most
constexpr int kBlock = kFusedRows * 128;           // bytes of 64 columns
constexpr int kHalves = kFusedCols / 64 * kBlock;  // of hi, of lo
constexpr int kSquare = kFusedRows / 64 * kBlock;  // of A, B
constexpr int kPart = kFusedRows * kFusedRows * 4;
constexpr int kFusedSteps = 64;

struct FusedParams {
    const void *m;
    ep_bf16 *out;
    int32_t N, K, steps, ctas;  // ctas: of a cluster
    float eps;
    int32_t *error;
    float k[kFusedSteps][3];
};

// 16 bytes of a row: the 8 columns from `col` on (of the CTA's).
__device__ __forceinline__ int unit_at(int row, int col) { return col / 64 * kBlock + row * 128 + ((col % 64 / 8) ^ (row & 7)) * 16; }
// Four floats of A's part.
__device__ __forceinline__ int part_at(int row, int col) { return row * 512 + ((col / 4) ^ (row & 7)) * 16; }

__device__ __forceinline__ void get_32(const unsigned char *p, int row, int col, uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = *reinterpret_cast<const uint4 *>(p + unit_at(row, col + 8 * i));
        v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
}
__device__ __forceinline__ void put_32(unsigned char *p, int row, int col, const uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(p + unit_at(row, col + 8 * i)) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ float ld_cluster_f32x4(uint32_t addr, float4 &v) {
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v.x;
}
__device__ __forceinline__ double ld_cluster_f64(uint32_t addr) {
    double v;
    asm volatile("ld.shared::cluster.f64 %0, [%1];" : "=d"(v) : "r"(addr) : "memory");
    return v;
}

// 32 values of A, or B, that this thread has as floats x[] (times kA or kB), from column `col` on, to `to` as halves, the
// diagonal's as zero; returns whether it was among them.
__device__ __forceinline__ bool put_square(unsigned char *to, int row, int col, uint64_t (&x)[16], float &diagonal) {
    const bool mine = row / 32 == col / 32;
    if (mine) {
#pragma unroll
        for (int k = 0; k < 32; ++k)
            if (k == row % 32) {
                diagonal = k % 2 ? high(x[k / 2]) : low(x[k / 2]);
                x[k / 2] = k % 2 ? pair(low(x[k / 2]), 0.0f) : pair(0.0f, high(x[k / 2]));
            }
    }
    uint32_t o[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) o[k] = half_pair(low(x[k]), high(x[k]));
    put_32(to, row, col, o);
    return mine;
}

template <typename V>
__global__ void __launch_bounds__(kFusedThreads, 1) ortho_fused_kernel(const __grid_constant__ FusedParams p) {
    extern __shared__ unsigned char smem_raw[];
    __shared__ uint64_t done;
    __shared__ uint32_t tmem_addr;
    __shared__ volatile int failed;
    __shared__ __align__(16) float d[kFusedRows], dB[kFusedRows];  // A's diagonal; a + B's
    __shared__ float warp_sums[kFusedThreads / 32];
    __shared__ double squares;
    __shared__ int out_of_range;
    __shared__ OrthoScale scale_shared;

    unsigned char *hi = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    unsigned char *lo = hi + kHalves, *square = lo + kHalves, *part = square + kSquare;
    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int ctas = p.ctas;
    const uint32_t rank = ctas > 1 ? cluster_cta_rank() : 0;
    const bool tall = p.N > p.K;
    const int m = tall ? p.K : p.N, n = tall ? p.N : p.K;
    const int c0 = (int)rank * kFusedCols, cols = min(kFusedCols, n - c0);  // this CTA's columns of X
    const int64_t matrix = blockIdx.x / ctas;
    const V *src = static_cast<const V *>(p.m) + matrix * p.N * p.K;

    if (tid == 0) {
        mbar_init(&done, 1);
        failed = 0;
        fence_mbar_init();
    }
    if (warp == 0) tmem_alloc<1>(&tmem_addr, 512);
    grid_dependency_wait();
    grid_launch_dependents();

    // ---- the norm. This thread's values of the CTA's part, X[i][c0 + j], i < m, j < cols, neighbours in memory to neighbours
    const int along = tall ? m : cols, across = tall ? cols : m;  // in memory a line of `along` values, `across` of them
    const int64_t line = tall ? m : p.K, first = tall ? (int64_t)c0 * m : c0;
    const auto sum_squares = [&](float by, bool &any) {
        float s = 0.0f;
        for (int l = warp; l < across; l += kFusedThreads / 32)
            for (int i = lane; i < along; i += 32) {
                const float v = Io<V>::load(src + first + l * line + i);
                any |= v != 0.0f;
                s = fmaf(v * by, v * by, s);
            }
#pragma unroll
        for (int k = 16; k > 0; k /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
        __syncthreads();
        if (lane == 0) warp_sums[warp] = s;
        __syncthreads();
        s = 0.0f;
        for (int i = 0; i < kFusedThreads / 32; ++i) s += warp_sums[i];
        return s;
    };
    bool any = false;
    float sum = sum_squares(1.0f, any);
    any = __syncthreads_or(any);
    double back = 1.0;
    if (any && !(sum >= 0x1p-90f && sum <= 0x1p126f)) {  // the squares leave fp32's range: again, times a power of two
        const bool small = sum < 0x1p-90f;
        sum = sum_squares(small ? 0x1p90f : 0x1p-90f, any);
        back = small ? 0x1p-180 : 0x1p180;
    }
    if (tid == 0) squares = sum * back;
    if (ctas > 1)
        cluster_sync();
    else
        __syncthreads();
    if (tid == 0) {
        double all = 0;
        for (int r = 0; r < ctas; ++r) all += ctas > 1 ? ld_cluster_f64(cluster_smem_u32(&squares, r)) : squares;
        scale_shared = ortho_scale(all, p.eps);
    }
    __syncthreads();
    const OrthoScale scale = scale_shared;

    // ---- X as halves: zeros behind the last row and column
    for (int i = tid; i < 2 * kHalves / 16; i += kFusedThreads) reinterpret_cast<uint4 *>(hi)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    for (int l = warp; l < across; l += kFusedThreads / 32)
        for (int i = lane; i < along; i += 32) {
            uint32_t h, r;
            split_pair(scale(Io<V>::load(src + first + l * line + i)), 0.0f, h, r);
            const int row = tall ? i : l, col = tall ? l : i;
            const int at = unit_at(row, col) + col % 8 * 2;
            *reinterpret_cast<uint16_t *>(hi + at) = (uint16_t)h;
            *reinterpret_cast<uint16_t *>(lo + at) = (uint16_t)r;
        }

    const int quarter = warp % 4, group = warp / 4;  // the TMEM lanes that this warp may read, its columns
    const int row = quarter * 32 + lane;
    uint32_t phase = 0;
    // What all have written becomes operands: MMAs issued by one thread, waited for by all.
    const auto multiply = [&](auto issue) {
        asm volatile("fence.proxy.async;" ::: "memory");
        tmem_fence_before();
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tmem_fence_after();
            if (!failed) issue();
            mma_commit<1>(&done);
        }
        __syncwarp();
        mbar_wait_warp(&done, phase, &failed);
        phase ^= 1;
        tmem_fence_after();
    };
    const auto block_desc = [&](const unsigned char *base, int k) { return smem_desc(smem_u32(base) + k / 4 * kBlock + k % 4 * 32, 16); };
    constexpr uint32_t kColA = 0, kColB = 128, kColX = 256;  // the products' accumulators
    const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
    __syncthreads();
    const uint32_t tmem = tmem_addr;
    const int k_cols = (cols + 15) / 16, k_rows = (m + 15) / 16;

    for (int step = 0; step < p.steps; ++step) {
        const float a = p.k[step][0], b = p.k[step][1], c = p.k[step][2];
        uint32_t v[32];
        // ---- A = X X^T
        multiply([&] {
            for (int k = 0; k < k_cols; ++k) {
                const uint64_t x = block_desc(hi, k);
                mma_bf16<1>(tmem + kColA, x, x, mma_idesc_f16(128, 128, false), k > 0);
            }
        });
        const uint64_t by = pair(kA / (kX * kX), kA / (kX * kX));
        float diagonal = 0.0f;
        if (ctas == 1) {
            uint64_t x[16];
            tmem_load_32(tmem + kColA + lanes + group * 32, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) x[k] = mul2(pair_of(v[2 * k], v[2 * k + 1]), by);
            if (put_square(square, row, group * 32, x, diagonal)) d[row] = diagonal * (1.0f / kA);
        } else {
            // every CTA adds some rows of all parts up, in the same order, and hands them to all
            tmem_load_32(tmem + kColA + lanes + group * 32, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4 *>(part + part_at(row, group * 32 + 4 * k)) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
            cluster_sync();
            const int rows = (kFusedRows + ctas - 1) / ctas, r0 = (int)rank * rows;
            for (int i = tid; i < rows * (kFusedRows / 8); i += kFusedThreads) {
                const int r = r0 + i / (kFusedRows / 8), col = i % (kFusedRows / 8) * 8;
                if (r >= kFusedRows) break;
                uint64_t x[4] = {0, 0, 0, 0};
                for (int q = 0; q < ctas; ++q) {
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        float4 f;
                        ld_cluster_f32x4(cluster_smem_u32(part + part_at(r, col + 4 * h), q), f);
                        x[2 * h] = add2(x[2 * h], pair(f.x, f.y));
                        x[2 * h + 1] = add2(x[2 * h + 1], pair(f.z, f.w));
                    }
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) x[k] = mul2(x[k], by);
                const bool mine = r >= col && r < col + 8;
                float e = 0.0f;
#pragma unroll
                for (int k = 0; k < 8; ++k)
                    if (mine && k == r - col) {
                        e = k % 2 ? high(x[k / 2]) : low(x[k / 2]);
                        x[k / 2] = k % 2 ? pair(low(x[k / 2]), 0.0f) : pair(0.0f, high(x[k / 2]));
                    }
                uint32_t o[4];
#pragma unroll
                for (int k = 0; k < 4; ++k) o[k] = half_pair(low(x[k]), high(x[k]));
                for (int q = 0; q < ctas; ++q) {
                    asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(cluster_smem_u32(square + unit_at(r, col), q)),
                                 "r"(o[0]), "r"(o[1]), "r"(o[2]), "r"(o[3])
                                 : "memory");
                    if (mine)
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_smem_u32(&d[r], q)), "f"(e * (1.0f / kA)) : "memory");
                }
            }
            asm volatile("fence.proxy.async;" ::: "memory");
            cluster_sync();
        }
        // ---- B = b A + c A A
        multiply([&] {
            for (int k = 0; k < k_rows; ++k) {
                const uint64_t x = block_desc(square, k);
                mma_bf16<1>(tmem + kColB, x, x, mma_idesc_f16(128, 128, false), k > 0);
            }
        });
        {
            const float di = d[row];
            uint32_t o[16];
            uint64_t x[16];
            get_32(square, row, group * 32, o);
            tmem_load_32(tmem + kColB + lanes + group * 32, v);
            tmem_wait_ld(v);
            const float by_a = kB / kA, base = by_a * fmaf(c, di, b);
            const uint64_t base2 = pair(base, base), cc2 = pair(by_a * c, by_a * c), acc2 = pair(c * (kB / (kA * kA)), c * (kB / (kA * kA)));
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint64_t d2 = *reinterpret_cast<const uint64_t *>(&d[group * 32 + 2 * k]);
                x[k] = fma2(halves(o[k]), fma2(cc2, d2, base2), mul2(pair_of(v[2 * k], v[2 * k + 1]), acc2));
            }
            if (put_square(square, row, group * 32, x, diagonal)) dB[row] = fmaf(diagonal, 1.0f / kB, a + fmaf(c * di, di, b * di));
        }
        // ---- X = a X + B X
        multiply([&] {
            for (int k = 0; k < k_rows; ++k)
                mma_bf16<1>(tmem + kColX, block_desc(square, k), smem_desc(smem_u32(hi) + k * 2048, kBlock),
                            mma_idesc_f16(128, 256, true), k > 0);
        });
        const float di = dB[row];
        const uint64_t d2 = pair(di, di), by_lo = pair(1.0f / kLo, 1.0f / kLo), by_b = pair(1.0f / kB, 1.0f / kB);
        const bool last = step + 1 == p.steps;
        for (int col = group * 64; col < group * 64 + 64; col += 32) {
            uint32_t h[16], l[16];
            get_32(hi, row, col, h);
            get_32(lo, row, col, l);
            tmem_load_32(tmem + kColX + lanes + col, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint64_t x = fma2(d2, fma2(halves(l[k]), by_lo, halves(h[k])), mul2(pair_of(v[2 * k], v[2 * k + 1]), by_b));
                if (last) {
                    const uint64_t y = mul2(x, pair(1.0f / kX, 1.0f / kX));
                    h[k] = bf16_pair(low(y), high(y));
                } else {
                    h[k] = half_pair(low(x), high(x));
                    const uint64_t r = mul2(fma2(halves(h[k]), pair(-1.0f, -1.0f), x), pair(kLo, kLo));
                    l[k] = half_pair(low(r), high(r));
                }
            }
            put_32(hi, row, col, h);
            if (!last) put_32(lo, row, col, l);
        }
    }

    // ---- the result, rounded already, from hi's place
    tmem_fence_before();
    __syncthreads();
    ep_bf16 *out = p.out + matrix * p.N * p.K;
    if (!failed) {
        if (!tall && p.K % 8 == 0) {
            for (int i = tid; i < m * (cols / 8); i += kFusedThreads) {
                const int r = i / (cols / 8), col = i % (cols / 8) * 8;
                st_v4(reinterpret_cast<uint4 *>(out + (int64_t)r * p.K + c0 + col), *reinterpret_cast<const uint4 *>(hi + unit_at(r, col)));
            }
        } else {
            for (int l = warp; l < across; l += kFusedThreads / 32)
                for (int i = lane; i < along; i += 32) {
                    const int r = tall ? i : l, col = tall ? l : i;
                    out[first + l * line + i] = *reinterpret_cast<const uint16_t *>(hi + unit_at(r, col) + col % 8 * 2);
                }
        }
    }
    if (failed) {  // MMAs under way read shared memory and write TMEM
        if (tid == 0) {
            int gave_up = 0;
            mbar_wait_limited(&done, phase ^ 1, &gave_up);
            atomicOr(p.error, kErrOrthoWait);
        }
        __syncthreads();
    }
    if (ctas > 1) cluster_sync();  // no CTA may end while another one reads its memory
    if (warp == 0) tmem_free<1>(tmem, 512);
}

template <typename V>
cudaError_t run_fused(const FusedParams &p, int batch, cudaStream_t s) {
    const size_t smem = 1024 + 2 * (size_t)kHalves + kSquare + (p.ctas > 1 ? kPart : 0);
    static SharedMemoryLimit limit;
    const cudaError_t e = limit.allow(ortho_fused_kernel<V>, smem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)batch * (unsigned)p.ctas);
    cfg.blockDim = dim3(kFusedThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)p.ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = p.ctas == 1 ? 1 : 2;
    return cudaLaunchKernelEx(&cfg, ortho_fused_kernel<V>, p);
}

}  // namespace

bool ortho_fits_fused(const ep_ortho_config &c) {
    const int m = c.N < c.K ? c.N : c.K, n = c.N < c.K ? c.K : c.N;
    return m <= kFusedRows && n <= kFusedCtas * kFusedCols;
}

cudaError_t launch_ortho_fused(const ep_ortho_config &c, const float *k, const void *m, ep_bf16 *out, cudaStream_t s) {
    FusedParams p = {};
    const int n = c.N < c.K ? c.K : c.N;
    p.m = m;
    p.out = out;
    p.N = c.N;
    p.K = c.K;
    p.steps = c.steps;
    p.ctas = (n + kFusedCols - 1) / kFusedCols;
    p.eps = c.eps;
    for (int i = 0; i < c.steps; ++i)
        for (int j = 0; j < 3; ++j) p.k[i][j] = k[3 * i + j];
    const cudaError_t e = expert_error_word(&p.error);
    if (e != cudaSuccess) return e;
    return c.dtype == EP_F32    ? run_fused<float>(p, c.B, s)
           : c.dtype == EP_BF16 ? run_fused<__nv_bfloat16>(p, c.B, s)
                                : run_fused<__half>(p, c.B, s);
}

}  // namespace ep
