// ortho_gemm.cuh -- the three products of a Newton-Schulz step on the tensor cores, for a batch of matrices.
//
// X is [m, n], m <= n (a taller matrix is held transposed). A step is
//   Gram    A = X X^T                     symmetric: tiles on and below the diagonal, mirrored on storing
//   Poly    B = b A + c A A               likewise
//   Apply   X <- a X + B X
// Operands have to fit 16 bits, and the step magnifies small singular values by `a` (3.44) each time: with
// bf16 operands the result is 1% off for a matrix of independent values and up to 9% for one whose singular
// values fall quickly. fp16 rounds eight times finer, its range is no limit (every value here has a known
// bound, and a power of two that goes with it, kX, kA, kB), and three things keep its roundings out of the
// result, 0.05% off before it is rounded itself:
//   - X is two halves, hi + lo / 2^10. hi is the operand; a X is formed of both in fp32.
//   - the diagonals of A and B, which are most of them once the singular values are alike, are fp32
//     vectors; the halves hold the rest, with zeros there.
//   - what of B lo is left out is then the rest's part alone.
// Sums are fp32, in TMEM.
//
// One persistent CTA per SM (CG = 2: a pair, a tile of 256 x 256): two producer warps feed a ring of stages by
// TMA, warp 1 issues the MMAs into one of two accumulators, eight warps turn the other into results. Every
// wait has a time limit (kErrOrthoWait).
#pragma once

#include "expert_gemm.cuh"

namespace ep {

enum class OrthoOp { kGram, kPoly, kApply };

// What is stored is the value times these: |X| < 4, |A| < 16 and |B| < 31 (ortho_fits) stay below 65504.
constexpr float kX = 8192.0f, kA = 1024.0f, kB = 2048.0f, kLo = 1024.0f;

struct OrthoParams {
    CUtensorMap a, b;
    int32_t batch;
    int32_t m, n;    // of X
    int32_t mp, np;  // row lengths of A and B, and of X: m and n filled up to 8, with zeros
    const uint16_t *o;      // Poly: A without its diagonal [batch, m, mp]
    const float *d;         // Poly: A's diagonal; Apply: a + B's [batch, mp]
    const uint16_t *hi, *lo;  // Apply: X [batch, m, np]
    uint16_t *out;          // Gram, Poly: without the diagonal; Apply: hi
    float *d_out;           // Gram, Poly
    uint16_t *lo_out;       // Apply; may be lo
    ep_bf16 *result;        // Apply: not null in the last step: [batch, m, n], or [batch, n, m] if `transposed`
    int32_t transposed;
    float ca, cb, cc;
    int32_t *error;
};

template <OrthoOp OP, int CG, int NB>
struct OrthoShape {
    static constexpr bool kSymmetric = OP != OrthoOp::kApply;
    static constexpr bool kBMn = OP == OrthoOp::kApply;  // B is X, whose rows are contracted
    static constexpr int kBM = kGemmBM * CG;
    static constexpr int kBRows = NB / CG;
    static constexpr int kABytes = kGemmBM * 128;
    static constexpr int kStageBytes = kABytes + kBRows * 128;
    static constexpr int kStages = 196608 / kStageBytes;
    static_assert(kStages % kProducers == 0, "a stage has one producer");
    static_assert(!kSymmetric || kBM % NB == 0, "tiles beside the diagonal blocks");
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + kEpilogueWarps * kSlabBytes;
};

struct OrthoTile {
    int matrix, m0, n0;
    bool mirror;  // to be stored transposed as well
};

// The tiles of one CTA (pair). Symmetric: block rows of kBM, in each the tiles up to the end of the diagonal block.
template <OrthoOp OP, int CG, int NB>
struct OrthoWalk {
    using Sh = OrthoShape<OP, CG, NB>;
    int64_t tile, step, total;
    int mt, nt, per;
    __host__ __device__ static int tiles(int m, int n) {
        const int mt = (m + Sh::kBM - 1) / Sh::kBM;
        return Sh::kSymmetric ? mt * (mt + 1) / 2 * (Sh::kBM / NB) : mt * ((n + NB - 1) / NB);
    }
    __device__ explicit OrthoWalk(const OrthoParams &p)
        : tile(blockIdx.x / CG), step(gridDim.x / CG), mt((p.m + Sh::kBM - 1) / Sh::kBM), nt((p.n + NB - 1) / NB),
          per(tiles(p.m, p.n)) {
        total = (int64_t)per * p.batch;
    }
    __device__ bool next(OrthoTile &t) {
        if (tile >= total) return false;
        t.matrix = (int)(tile / per);
        const int r = (int)(tile % per);
        if constexpr (Sh::kSymmetric) {
            constexpr int kSub = Sh::kBM / NB;  // tiles of a diagonal block
            const int block = r / kSub;
            int i = (int)((sqrtf(8.0f * (float)block + 1.0f) - 1.0f) * 0.5f);
            while (i * (i + 1) / 2 > block) --i;
            while ((i + 1) * (i + 2) / 2 <= block) ++i;
            t.m0 = i * Sh::kBM;
            t.n0 = (block - i * (i + 1) / 2) * Sh::kBM + r % kSub * NB;
            t.mirror = t.n0 < t.m0;
        } else {
            t.m0 = r % mt * Sh::kBM;  // down the columns: a few column tiles of X, all of B
            t.n0 = r / mt * NB;
            t.mirror = false;
        }
        tile += step;
        return true;
    }
};

constexpr uint32_t mma_idesc_f16(int m, int n, bool b_mn_major) {
    return 1u << 4 | (b_mn_major ? 1u : 0u) << 16 | (uint32_t)(n >> 3) << 17 | (uint32_t)(m >> 4) << 24;
}

// The slab with rows and columns exchanged: this thread's row of 32 values becomes column `lane`.
__device__ __forceinline__ void slab_put_transposed(unsigned char *slab, int lane, const uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        *reinterpret_cast<uint16_t *>(slab + slab_at(i, lane / 8) + lane % 8 * 2) = (uint16_t)(v[i / 2] >> (i % 2 * 16));
}
// slab_store for rows of any length, value by value: columns [n, n + 32) of N.
__device__ __forceinline__ void slab_store_any(const unsigned char *slab, int lane, ep_bf16 *base, int N, int n, int rows) {
    __syncwarp();
    if (n + lane < N)
        for (int r = 0; r < rows; ++r)
            base[(size_t)r * N + n + lane] = *reinterpret_cast<const uint16_t *>(slab + slab_at(r, lane / 8) + lane % 8 * 2);
    __syncwarp();
}

template <OrthoOp OP, int CG, int NB>
__global__ void __launch_bounds__(kGemmThreads, 1) ortho_gemm_kernel(const __grid_constant__ OrthoParams p) {
    using Sh = OrthoShape<OP, CG, NB>;
    constexpr int kStages = Sh::kStages;
    extern __shared__ unsigned char smem_raw[];
    // CG = 2: both CTAs' copies report to the first CTA's `full`
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_addr;
    __shared__ volatile int failed;

    unsigned char *stages = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    unsigned char *slabs = stages + kStages * Sh::kStageBytes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0;
    const int kb = ((OP == OrthoOp::kGram ? p.n : p.m) + kGemmBK - 1) / kGemmBK;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], kEpilogueWarps * CG);
        mbar_init(&drained, 1);
        failed = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.a);
        tma_prefetch_map(&p.b);
    }
    if (warp == 1) tmem_alloc<CG>(&tmem_addr, 2 * NB);
    tmem_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_addr;
    grid_dependency_wait();
    grid_launch_dependents();

    OrthoWalk<OP, CG, NB> walk(p);
    OrthoTile t;
    bool produces = false;
    uint32_t it = 0;  // the next fill of this producer

    if (warp == 0 || warp > 1 + kEpilogueWarps) {
        // ---- producers: one lane each, which take the stages in turn
        if (elect_one()) {
            const uint32_t mine = warp == 0 ? 0 : warp - 1 - kEpilogueWarps;
            produces = true;
            it = mine;
            uint32_t s = mine, phase = 0;
            int b = mine;
            bool ok = true, ready = false;
            while (ok && walk.next(t)) {
#pragma unroll 2
                for (; b < kb; b += kProducers, it += kProducers) {
                    if (it >= kStages && !ready && !mbar_poll_limited(&empty[s], phase ^ 1, &failed)) {
                        ok = false;
                        break;
                    }
                    const bool wraps = s + kProducers >= kStages;
                    const uint32_t next = s + kProducers - (wraps ? kStages : 0), next_phase = wraps ? phase ^ 1 : phase;
                    ready = it + kProducers >= kStages && mbar_test(&empty[next], next_phase ^ 1);
                    if (rank == 0) mbar_arrive_expect_tx(&full[s], Sh::kStageBytes * CG);
                    const uint32_t bar = CG == 2 ? cluster_smem_u32(&full[s], 0) : smem_u32(&full[s]);
                    unsigned char *sa = stages + s * Sh::kStageBytes, *sb = sa + Sh::kABytes;
                    const int k = b * kGemmBK;
                    tma_load_3d<CG>(sa, &p.a, k, t.m0 + (int)rank * kGemmBM, t.matrix, bar);
                    if constexpr (Sh::kBMn) {
#pragma unroll
                        for (int i = 0; i < Sh::kBRows / 64; ++i)
                            tma_load_3d<CG>(sb + i * 8192, &p.b, t.n0 + (int)rank * Sh::kBRows + 64 * i, k, t.matrix, bar);
                    } else {
                        tma_load_3d<CG>(sb, &p.b, k, t.n0 + (int)rank * Sh::kBRows, t.matrix, bar);
                    }
                    s = next;
                    phase = next_phase;
                }
                b -= kb;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer (CG = 2: of the pair's first CTA), one lane
        if (rank == 0 && elect_one()) {
            constexpr uint32_t idesc = mma_idesc_f16(Sh::kBM, NB, Sh::kBMn);
            const uint64_t da_first = smem_desc(smem_u32(stages), 16);
            const uint64_t db_first = smem_desc(smem_u32(stages) + Sh::kABytes, Sh::kBMn ? 8192 : 16);
            uint32_t s = 0, phase = 0, acc_it = 0;
            bool ok = true, ready = false;
            while (ok && walk.next(t)) {
                const uint32_t slot = acc_it & 1, d = tmem + slot * NB;
                if (acc_it >= 2) ok = mbar_poll_limited<CG == 2>(&acc_empty[slot], (acc_it / 2 - 1) & 1, &failed);
                tmem_fence_after();
#pragma unroll 4
                for (int b = 0; ok && b < kb; ++b) {
                    ok = ready || mbar_poll_limited(&full[s], phase, &failed);
                    const uint32_t at = s;
                    if (++s == kStages) s = 0, phase ^= 1;
                    ready = mbar_test(&full[s], phase);
                    if (!ok) break;
                    const uint64_t da = da_first + at * (Sh::kStageBytes / 16), db = db_first + at * (Sh::kStageBytes / 16);
#pragma unroll
                    for (int k = 0; k < kGemmBK / 16; ++k)
                        mma_bf16<CG>(d, da + k * 2, db + k * (Sh::kBMn ? 128 : 2), idesc, b + k > 0);
                    mma_commit<CG>(&empty[at]);
                    if (b == kb - 1) mma_commit<CG>(&acc_full[slot]);
                }
                ++acc_it;
            }
        }
        __syncwarp();
    } else {
        // ---- epilogue: warp w reads lanes [32 (w mod 4), + 32) of the accumulators, one row a thread, and
        // two warps take the same rows' columns in turns of 32
        const int quarter = warp % 4, turn = (warp - 2) / 4;
        unsigned char *slab = slabs + (warp - 2) * kSlabBytes;
        uint32_t acc_it = 0;
        while (walk.next(t)) {
            const uint32_t slot = acc_it & 1;
            const int first = t.m0 + (int)rank * kGemmBM + quarter * 32;  // the warp's first row
            const int i = first + lane;
            const int rows = min(p.m - first, 32);
            const int width = Sh::kSymmetric ? p.mp : p.np;
            const int c_end = min(NB, width - t.n0);
            const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + slot * NB;
            const size_t row = (size_t)t.matrix * p.m + first;  // of [batch, m]
            const size_t diag = (size_t)t.matrix * p.mp;
            float di = 0.0f;
            if (OP != OrthoOp::kGram && i < p.m) di = p.d[diag + i];
            // what goes with the accumulator is asked for a turn ahead, the first before that is there
            uint4 q0[4], q1[4];
            const auto ask = [&](int c) {
                if (OP == OrthoOp::kGram || rows <= 0 || c >= c_end) return;
                if constexpr (OP == OrthoOp::kPoly) {
                    slab_load(q0, lane, p.o + row * p.mp, p.mp, t.n0 + c, rows);
                } else {
                    slab_load(q0, lane, p.hi + row * p.np, p.np, t.n0 + c, rows);
                    slab_load(q1, lane, p.lo + row * p.np, p.np, t.n0 + c, rows);
                }
            };
            int c = turn * kCols;
            ask(c);
            bool ok = true;
            if (lane == 0) ok = mbar_wait_limited(&acc_full[slot], (acc_it / 2) & 1, &failed);
            if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
            ++acc_it;
            tmem_fence_after();
            for (; rows > 0 && c < c_end; c += 2 * kCols) {
                const int n = t.n0 + c;
                uint32_t v[32], o[16];
                if constexpr (OP == OrthoOp::kApply) {
                    uint32_t hi[16], lo[16];
                    slab_fill(slab, lane, q0);
                    slab_get(slab, lane, hi);
                    __syncwarp();
                    slab_fill(slab, lane, q1);
                    slab_get(slab, lane, lo);
                    __syncwarp();
                    ask(c + 2 * kCols);
                    tmem_load_32(src + c, v);
                    tmem_wait_ld(v);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        const float2 h = saved_values<false>(hi[k]), l = saved_values<false>(lo[k]);
                        const float x0 = fmaf(di, fmaf(l.x, 1.0f / kLo, h.x), __uint_as_float(v[2 * k]) * (1.0f / kB));
                        const float x1 = fmaf(di, fmaf(l.y, 1.0f / kLo, h.y), __uint_as_float(v[2 * k + 1]) * (1.0f / kB));
                        if (p.result) {
                            o[k] = bf16_pair(x0 * (1.0f / kX), x1 * (1.0f / kX));
                        } else {
                            o[k] = half_pair(x0, x1);
                            const float2 r = saved_values<false>(o[k]);
                            lo[k] = half_pair((x0 - r.x) * kLo, (x1 - r.y) * kLo);
                        }
                    }
                    if (!p.result) {
                        slab_put(slab, lane, o);
                        slab_store(slab, lane, p.out + row * p.np, p.np, n, rows);
                        slab_put(slab, lane, lo);
                        slab_store(slab, lane, p.lo_out + row * p.np, p.np, n, rows);
                    } else if (p.transposed) {
                        slab_put_transposed(slab, lane, o);
                        ep_bf16 *base = p.result + ((size_t)t.matrix * p.n + n) * p.m;
                        const int high = min(32, p.n - n);
                        if (p.m % 8 == 0)
                            slab_store(slab, lane, base, p.m, first, high);
                        else
                            slab_store_any(slab, lane, base, p.m, first, high);
                    } else {
                        slab_put(slab, lane, o);
                        if (p.n % 8 == 0)
                            slab_store(slab, lane, p.result + row * p.n, p.n, n, rows);
                        else
                            slab_store_any(slab, lane, p.result + row * p.n, p.n, n, rows);
                    }
                } else {
                    float x[32];
                    if constexpr (OP == OrthoOp::kPoly) {
                        uint32_t a[16];
                        slab_fill(slab, lane, q0);
                        slab_get(slab, lane, a);
                        __syncwarp();
                        ask(c + 2 * kCols);
                        const float dj = n + lane < p.m ? p.d[diag + n + lane] : 0.0f;  // lane j: of column j
                        tmem_load_32(src + c, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int k = 0; k < 32; ++k) {
                            const float2 a2 = saved_values<false>(a[k / 2]);
                            const float f = fmaf(p.cc, di + __shfl_sync(0xFFFFFFFFu, dj, k), p.cb);
                            x[k] = fmaf(kB / kA * (k % 2 ? a2.y : a2.x), f, p.cc * (kB / (kA * kA)) * __uint_as_float(v[k]));
                        }
                    } else {
                        tmem_load_32(src + c, v);
                        tmem_wait_ld(v);
#pragma unroll
                        for (int k = 0; k < 32; ++k) x[k] = __uint_as_float(v[k]) * (kA / (kX * kX));
                    }
                    // columns behind the last are zeros, the diagonal is apart
#pragma unroll
                    for (int k = 0; k < 32; ++k) {
                        if (n + k == i && i < p.m)
                            p.d_out[diag + i] = OP == OrthoOp::kGram ? x[k] * (1.0f / kA)
                                                                     : fmaf(x[k], 1.0f / kB, p.ca + fmaf(p.cc * di, di, p.cb * di));
                        if (n + k == i || n + k >= p.m || i >= p.m) x[k] = 0.0f;
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = half_pair(x[2 * k], x[2 * k + 1]);
                    slab_put(slab, lane, o);
                    slab_store(slab, lane, p.out + row * p.mp, p.mp, n, rows);
                    if (t.mirror) {
                        slab_put_transposed(slab, lane, o);
                        slab_store(slab, lane, p.out + ((size_t)t.matrix * p.m + n) * p.mp, p.mp, first, min(32, p.m - n));
                    }
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2)
                    mbar_arrive_cluster(cluster_smem_u32(&acc_empty[slot], 0));
                else
                    mbar_arrive(&acc_empty[slot]);
            }
        }
    }

    __syncthreads();
    if constexpr (CG == 2) {
        // a CTA that gave up tells the other one, whose memory its copies and MMAs may use
        if (threadIdx.x == 0 && failed) st_cluster(cluster_smem_u32(const_cast<int *>(&failed), rank ^ 1), 1);
        cluster_sync();
    }
    // after a failure: what is under way is waited for before the CTA ends
    if (failed) {
        if (produces) {
            if (rank == 0) {
                wait_for_fills(full, it, warp == 0 ? 0 : warp - 1 - kEpilogueWarps, kProducers, kStages);
            } else {  // copies for which the first CTA's barrier was not armed any more
                for (int i = 0; i < 100; ++i) __nanosleep(10000);
            }
        } else if (warp == 1 && rank == 0) {
            if (elect_one()) mma_commit<CG>(&drained);
            __syncwarp();
            int gave_up = 0;
            mbar_wait_limited(&drained, 0, &gave_up);
        }
        __syncthreads();
        if constexpr (CG == 2) cluster_sync();
        if (threadIdx.x == 0) atomicOr(p.error, kErrOrthoWait);
    }
    if (warp == 1) tmem_free<CG>(tmem, 2 * NB);
}

}  // namespace ep
