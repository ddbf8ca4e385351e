// ortho_fused.cu -- small matrices through all Newton-Schulz steps in one kernel.
//
// As three products a step, launched one after the other, a matrix of 128 rows takes 6 us a product whatever its
// work: launch, first copies, last stores. Up to 128 rows (of the wide form) X stays on the chip instead: a cluster of
// up to sixteen CTAs takes a matrix, each CTA 256 of its columns, and only the sums of A's parts pass between them.
// X itself is fp32, in registers (a thread has 64 columns of a row); its halves, rounded as
// in ortho_gemm.cuh, lie in shared memory and serve as both operands of A = X X^T (128 bytes of a row's columns,
// swizzled) and, read the other way, as the second of B X. A and then B lie in one place. What the halves leave out becomes
// halves of its own in the steps that take X whole (OrthoForm), where A's parts lie otherwise.
//
// What bounds it is the chain of a step: three waits for a few MMAs, three epilogues, as many fences and barriers.
// 64 matrices of 128 x 256 take 30 us for five steps (84 by products of their own, in a graph), 1024 of them 212 (1119), one
// of 128 x 4096 by sixteen CTAs 59 (76), 32 of those 294 (431). A step that takes X whole is 2 to 3 us of that (eight steps of the
// 64, four of them such, 62 us; 54 without).
#include "ortho_values.cuh"

namespace ep {

namespace {

constexpr int kFusedThreads = 512;
constexpr int kFusedRows = 128, kFusedCols = 256;  // of a CTA
constexpr int kFusedCtas = 16;                     // of a cluster, at most
constexpr int kBlock = kFusedRows * 128;           // bytes of 64 columns
constexpr int kHalves = kFusedCols / 64 * kBlock;  // of X's halves
constexpr int kSquare = kFusedRows / 64 * kBlock;  // of A, B
constexpr int kPart = kFusedRows * kFusedRows * 4;
static_assert(kPart == kHalves, "X's lower halves and A's parts take turns");
constexpr int kStaging = kFusedRows * kFusedCols * 4;  // the matrix as it comes in, before there is anything else
constexpr int kFusedSteps = 64;
// Up to so many rows a step that takes X whole does so in A as well: an element of A is one of few then, and its
// rounding is not lost among others' (16 x 24 of full rank, five steps: 0.09% off and 0.06; 8 x 8 0.14 and 0.12).
constexpr int kFewRows = 16;

struct FusedParams {
    const void *m;
    ep_bf16 *out;
    int32_t N, K, steps, ctas;  // ctas: of a cluster
    float eps;
    int32_t *error;
    float k[kFusedSteps][3];
    OrthoForm form[kFusedSteps];
};

// 16 bytes of a row: the 8 columns from `col` on (of the CTA's).
__device__ __forceinline__ int unit_at(int row, int col) { return col / 64 * kBlock + row * 128 + ((col % 64 / 8) ^ (row & 7)) * 16; }
// Four floats of A's part, one of the matrix as it comes in.
__device__ __forceinline__ int part_at(int row, int col) { return row * 512 + ((col / 4) ^ (row & 7)) * 16; }
__device__ __forceinline__ int staging_at(int row, int col) { return row * 1024 + ((col / 4) ^ (row & 7)) * 16 + col % 4 * 4; }

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
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr));
    return v;
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
    __shared__ OrthoScale scale_shared;

    unsigned char *hi = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    unsigned char *square = hi + kHalves, *part = square + kSquare, *staging = hi;
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

    // ---- X: this thread's row, columns [64 group, + 64) of the CTA's; zeros behind the last row and column
    const int quarter = warp % 4, group = warp / 4;  // the TMEM lanes that this warp may read, its columns
    const int row = quarter * 32 + lane;
    uint64_t x_own[32];
    if (tall) {  // a column is a line in memory: neighbours read neighbours
        const V *line = src + (int64_t)(c0 + group * 64) * m + row;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const int col = group * 64 + 2 * k;
            const bool in = row < m;
            x_own[k] = pair(in && col < cols ? Io<V>::load(line + 2 * k * (int64_t)m) : 0.0f,
                            in && col + 1 < cols ? Io<V>::load(line + (2 * k + 1) * (int64_t)m) : 0.0f);
        }
    } else {  // a row is one: read line by line and handed over
        if (p.K % 8 == 0 && reinterpret_cast<uintptr_t>(src) % 16 == 0) {
            constexpr int kVec = Io<V>::kVec, kPieces = 8 / kVec;  // 16 bytes hold kVec values
            uint4 q[8][kPieces];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (tid + i * kFusedThreads) / 32, col = (tid + i * kFusedThreads) % 32 * 8;
#pragma unroll
                for (int h = 0; h < kPieces; ++h)
                    q[i][h] = r < m && col < cols ? *reinterpret_cast<const uint4 *>(src + (int64_t)r * p.K + c0 + col + h * kVec)
                                                  : make_uint4(0, 0, 0, 0);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const int r = (tid + i * kFusedThreads) / 32, col = (tid + i * kFusedThreads) % 32 * 8;
                float f[8];
#pragma unroll
                for (int h = 0; h < kPieces; ++h) {
                    float u[kVec];
                    Io<V>::unpack(q[i][h], u);
#pragma unroll
                    for (int j = 0; j < kVec; ++j) f[h * kVec + j] = u[j];
                }
#pragma unroll
                for (int h = 0; h < 2; ++h)
                    *reinterpret_cast<float4 *>(staging + staging_at(r, col + 4 * h)) = make_float4(f[4 * h], f[4 * h + 1], f[4 * h + 2], f[4 * h + 3]);
            }
        } else {
            for (int r = warp; r < kFusedRows; r += 2 * kFusedThreads / 32) {  // 16 values asked for together
                float f[2][8];
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < 8; ++u) {
                        const int at = r + h * kFusedThreads / 32, col = lane + 32 * u;
                        f[h][u] = at < m && col < cols ? Io<V>::load(src + (int64_t)at * p.K + c0 + col) : 0.0f;
                    }
#pragma unroll
                for (int h = 0; h < 2; ++h)
#pragma unroll
                    for (int u = 0; u < 8; ++u)
                        *reinterpret_cast<float *>(staging + staging_at(r + h * kFusedThreads / 32, lane + 32 * u)) = f[h][u];
            }
        }
        __syncthreads();
#pragma unroll
        for (int u = 0; u < 16; ++u) {
            const float4 f = *reinterpret_cast<const float4 *>(staging + staging_at(row, group * 64 + 4 * u));
            x_own[2 * u] = pair(f.x, f.y), x_own[2 * u + 1] = pair(f.z, f.w);
        }
    }
    // ---- the norm
    const auto sum_squares = [&](float by) {
        uint64_t s2 = 0;
        const uint64_t by2 = pair(by, by);
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const uint64_t v = mul2(x_own[k], by2);
            s2 = fma2(v, v, s2);
        }
        float s = total(s2);
#pragma unroll
        for (int k = 16; k > 0; k /= 2) s += __shfl_xor_sync(0xFFFFFFFFu, s, k);
        __syncthreads();
        if (lane == 0) warp_sums[warp] = s;
        __syncthreads();
        s = 0.0f;
#pragma unroll
        for (int i = 0; i < kFusedThreads / 32; ++i) s += warp_sums[i];
        return s;
    };
    float sum = sum_squares(1.0f);
    double back = 1.0;
    if (!(sum >= 0x1p-90f && sum <= 0x1p126f)) {  // all zeros, or the squares leave fp32's range: times a power of two
        const bool small = sum < 0x1p-90f;
        sum = sum_squares(small ? 0x1p90f : 0x1p-90f);
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
    const OrthoScale scale = scale_shared;  // and all have read what they stage

    // ---- X, times kX from here on, and its halves
    const auto put_halves = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = half_pair(low(x_own[16 * h + k]), high(x_own[16 * h + k]));
            put_32(hi, row, group * 64 + 32 * h, o);
        }
    };
#pragma unroll
    for (int k = 0; k < 32; ++k)
        x_own[k] = mul2(mul2(mul2(x_own[k], pair(scale.p1, scale.p1)), pair(scale.p2, scale.p2)), pair(scale.f * kX, scale.f * kX));
    put_halves();
    // what they leave out
    const auto put_rest = [&] {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                const uint64_t x = x_own[16 * h + k], r = fma2(halves(half_pair(low(x), high(x))), pair(-1.0f, -1.0f), x);
                o[k] = half_pair(low(r), high(r));
            }
            put_32(part, row, group * 64 + 32 * h, o);
        }
    };

    uint32_t phase = 0;
    // What all have written becomes operands: MMAs issued by one thread, waited for by all.
    const auto multiply = [&](auto issue) {
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tmem_fence_before();
        __syncthreads();
        if (warp == 0 && elect_one()) {
            tmem_fence_after();
            if (!failed) issue();
            mma_commit<1>(&done);
        }
        __syncwarp();
        if (lane == 0) mbar_poll_limited(&done, phase, &failed);
        __syncwarp();
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
        const OrthoForm form = p.form[step];
        uint32_t v[32];
        // ---- A = X X^T
        const bool whole = form == OrthoForm::kWhole, whole_a = whole && m <= kFewRows;
        if (whole_a) put_rest();
        multiply([&] {
            for (int k = 0; k < k_cols; ++k) {
                const uint64_t x = block_desc(hi, k);
                mma_bf16<1>(tmem + kColA, x, x, mma_idesc_f16(128, 128, false), k > 0);
                if (whole_a) {
                    const uint64_t r = block_desc(part, k);  // of one shape: only such products are added in order
                    mma_bf16<1>(tmem + kColA, x, r, mma_idesc_f16(128, 128, false), true);
                    mma_bf16<1>(tmem + kColA, r, x, mma_idesc_f16(128, 128, false), true);
                }
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
            for (int i = tid; i < rows * (kFusedRows / 4); i += kFusedThreads) {
                const int r = r0 + i / (kFusedRows / 4), col = i % (kFusedRows / 4) * 4;
                if (r >= kFusedRows) break;
                float x[4] = {0, 0, 0, 0};
#pragma unroll
                for (int q0 = 0; q0 < kFusedCtas; q0 += 8) {
                    if (q0 >= ctas) break;
                    float4 f[8];  // asked for together
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        f[q] = q0 + q < ctas ? ld_cluster_f32x4(cluster_smem_u32(part + part_at(r, col), q0 + q)) : make_float4(0, 0, 0, 0);
#pragma unroll
                    for (int q = 0; q < 8; ++q) x[0] += f[q].x, x[1] += f[q].y, x[2] += f[q].z, x[3] += f[q].w;
                }
                const bool mine = r >= col && r < col + 4;
                float e = 0.0f;
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    x[k] *= kA / (kX * kX);
                    if (mine && k == r - col) e = x[k], x[k] = 0.0f;
                }
                const uint32_t o[2] = {half_pair(x[0], x[1]), half_pair(x[2], x[3])};
                for (int q = 0; q < ctas; ++q) {
                    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(cluster_smem_u32(square + unit_at(r, col) + col % 8 * 2, q)),
                                 "r"(o[0]), "r"(o[1])
                                 : "memory");
                    if (mine)
                        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_smem_u32(&d[r], q)), "f"(e * (1.0f / kA)) : "memory");
                }
            }
            asm volatile("fence.proxy.async.shared::cluster;" ::: "memory");
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
        if (whole && !(whole_a && ctas == 1)) put_rest();  // A's parts have taken its place
        multiply([&] {
            for (int k = 0; k < k_rows; ++k)
                mma_bf16<1>(tmem + kColX, block_desc(square, k), smem_desc(smem_u32(hi) + k * 2048, kBlock),
                            mma_idesc_f16(128, 256, true), k > 0);
            if (whole)
                for (int k = 0; k < k_rows; ++k)
                    mma_bf16<1>(tmem + kColX, block_desc(square, k), smem_desc(smem_u32(part) + k * 2048, kBlock),
                                mma_idesc_f16(128, 256, true), true);
        });
        const float di = dB[row];
        const uint64_t d2 = pair(di, di), by_b = pair(1.0f / kB, 1.0f / kB);
        const bool upper = form == OrthoForm::kUpper;
        const uint64_t a2 = pair(a, a);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            tmem_load_32(tmem + kColX + lanes + group * 64 + 32 * h, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 16; ++k) {
                uint64_t x = x_own[16 * h + k], sum = mul2(pair_of(v[2 * k], v[2 * k + 1]), by_b);
                if (upper) {  // the diagonal times the upper half alone, a times both
                    const uint64_t hi2 = halves(half_pair(low(x), high(x)));
                    sum = fma2(a2, fma2(hi2, pair(-1.0f, -1.0f), x), sum);
                    x = hi2;
                }
                x_own[16 * h + k] = fma2(d2, x, sum);
            }
        }
        if (step + 1 < p.steps) put_halves();
    }
    // ---- the result: by columns as X came in, by rows through the halves' place
    ep_bf16 *out = p.out + matrix * p.N * p.K;
    const auto result = [&](int k) {
        const uint64_t y = mul2(x_own[k], pair(1.0f / kX, 1.0f / kX));
        return bf16_pair(low(y), high(y));
    };
    if (tall) {
        ep_bf16 *line = out + (int64_t)(c0 + group * 64) * m + row;
#pragma unroll
        for (int k = 0; k < 32; ++k) {
            const uint32_t o = result(k);
            const int col = group * 64 + 2 * k;
            if (row < m && !failed) {
                if (col < cols) line[2 * k * (int64_t)m] = (ep_bf16)o;
                if (col + 1 < cols) line[(2 * k + 1) * (int64_t)m] = (ep_bf16)(o >> 16);
            }
        }
    } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t o[16];
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = result(16 * h + k);
            put_32(hi, row, group * 64 + 32 * h, o);
        }
        __syncthreads();
        if (p.K % 8 == 0) {
            for (int i = tid; i < m * 32; i += kFusedThreads) {
                const int r = i / 32, col = i % 32 * 8;
                if (col < cols && !failed)
                    st_v4(reinterpret_cast<uint4 *>(out + (int64_t)r * p.K + c0 + col), *reinterpret_cast<const uint4 *>(hi + unit_at(r, col)));
            }
        } else {
            for (int r = warp; r < m; r += kFusedThreads / 32)
                for (int col = lane; col < cols; col += 32)
                    if (!failed) out[(int64_t)r * p.K + c0 + col] = *reinterpret_cast<const uint16_t *>(hi + unit_at(r, col) + col % 8 * 2);
        }
    }
    tmem_fence_before();
    __syncthreads();
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

constexpr int kAnyDeviceCtas = 8;  // clusters up to here run on every device

// *ran: false, and nothing launched, where the device has no place for a cluster of so many CTAs (a partition of a GPU
// with few SMs, for instance).
template <typename V>
cudaError_t run_fused(const FusedParams &p, int batch, bool *ran, cudaStream_t s) {
    constexpr size_t work = (size_t)kHalves + kSquare + kPart, smem = 1024 + (work > kStaging ? work : kStaging);
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
    *ran = true;
    if (p.ctas > kAnyDeviceCtas) {
        static std::atomic<int> places[kMaxDevices_][kFusedCtas + 1];  // clusters at a time, and one; 0: no answer yet
        int dev = 0;
        const cudaError_t e = current_device(&dev);
        if (e != cudaSuccess) return e;
        int n = places[dev][p.ctas].load(std::memory_order_acquire);
        if (n == 0) {
            if (cudaFuncSetAttribute(ortho_fused_kernel<V>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) == cudaSuccess &&
                cudaOccupancyMaxActiveClusters(&n, ortho_fused_kernel<V>, &cfg) == cudaSuccess) {
                places[dev][p.ctas].store(++n, std::memory_order_release);
            } else {
                cudaGetLastError();
                n = 0;
            }
        }
        if (n <= 1) {
            *ran = false;
            return cudaSuccess;
        }
    }
    return cudaLaunchKernelEx(&cfg, ortho_fused_kernel<V>, p);
}

}  // namespace

bool ortho_fits_fused(const ep_ortho_config &c) {
    const int m = c.N < c.K ? c.N : c.K, n = c.N < c.K ? c.K : c.N;
    return m <= kFusedRows && n <= kFusedCtas * kFusedCols;
}

bool ortho_fits_any_device(const ep_ortho_config &c) {
    return ortho_fits_fused(c) && (c.N < c.K ? c.K : c.N) <= kAnyDeviceCtas * kFusedCols;
}

cudaError_t launch_ortho_fused(const ep_ortho_config &c, const float *k, const void *m, ep_bf16 *out, bool *ran, cudaStream_t s) {
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
    ortho_steps(k, c.steps, c.N < c.K ? c.N : c.K, p.form);
    const cudaError_t e = expert_error_word(&p.error);
    if (e != cudaSuccess) return e;
    return c.dtype == EP_F32    ? run_fused<float>(p, c.B, ran, s)
           : c.dtype == EP_BF16 ? run_fused<__nv_bfloat16>(p, c.B, ran, s)
                                : run_fused<__half>(p, c.B, ran, s);
}

}  // namespace ep
