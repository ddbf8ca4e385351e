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
// result, 0.05 to 0.1% off before it is rounded itself:
//   - X is two halves, hi + lo. hi is the operand; a X is formed of both in fp32.
//   - the diagonals of A and B, which are most of them once the singular values are alike, are fp32
//     vectors; the halves hold the rest, with zeros there.
//   - what B X takes of lo goes by the step (OrthoForm).
// Sums are fp32, in TMEM.
//
// One persistent CTA per SM (CG = 2: a pair, a tile of 256 x 256): two producer warps feed a ring of stages by
// TMA, warp 1 issues the MMAs into one of two accumulators, eight warps turn the other into results. Every
// wait has a time limit (kErrOrthoWait).
//
// 16 matrices of 2048 x 4096: Gram 186 us, Poly 101, Apply 370 (the last one 335), the tensor pipe 73 to 88 % busy; the
// clock falls to 1.6 GHz, as power bounds them (a quarter fewer cycles for a tile left the time as it was). No step of five
// takes X whole there; three of eight do (7.0 ms instead of 6.2). One matrix of
// 256 x 7168 takes 98 to 101 us for five steps, 17 kernels one after another: launch, first copies, last stores of each.
#pragma once

#include "expert_gemm.cuh"
#include "pairs.cuh"

namespace ep {

enum class OrthoOp { kGram, kPoly, kApply };

// What B X takes of X's lower half. With D the diagonal of B, which is at hand in fp32:
//   kDiagonal  a X + D X + (B - D) hi. What is missing, (B - D) lo, is little where the singular values are alike, as B
//              is nearly its diagonal then. But it is noise in all directions, those included that X has none in, and
//              there every later step multiplies it by its `a`: a matrix of half its rank is 5% off after eight steps.
//   kUpper     a X + B hi. What is missing, B lo, is more, but has the directions of B's columns, which are X's: it turns
//              them a little, and none grows. As cheap.
//   kWhole     a X + B X, by a second pass over lo.
// Which one is ortho_steps' rule: the diagonal's in the last steps, behind which nothing grows, before that the upper
// half where B is small beside a for singular values that are all alike, else X whole. Off by (as the kernels round, before the
// last rounding, default coefficients): 256 x 384 of rank 128, five steps 0.17% (kDiagonal alone), 0.11% (kUpper alone),
// 0.10% (the rule); eight steps 5.6, 0.18, 0.14; of full rank 0.067, 0.127, 0.067.
enum class OrthoForm : uint8_t { kDiagonal, kUpper, kWhole };

// What is stored is the value times these: |X| < 4, |A| < 16 and |B| < 31 (ortho_steps) stay below 65504. lo, a 4096th of
// X at most, has X's factor, so that both are terms of one sum: what fp16's range takes from it is below 2^-38 of X's bound.
constexpr float kX = 8192.0f, kA = 1024.0f, kB = 2048.0f;

struct OrthoParams {
    CUtensorMap a, b, b_lo;  // operands; Apply that takes X whole: b_lo is its lower half
    CUtensorMap in[2];       // Poly: A without its diagonal; Apply: hi and lo of X. Boxes of 32 x 32 of the tile
    CUtensorMap out[2];      // Gram, Poly: A, B without its diagonal; Apply: hi and lo, or the result
    int32_t batch;
    int32_t m, n;    // of X
    int32_t mp, np;  // row lengths of A and B, and of X: m and n filled up to 8, with zeros
    const float *d;  // Poly: A's diagonal; Apply: a + B's [batch, mp], and 32 more values behind them
    float *d_out;    // Gram, Poly
    ep_bf16 *result; // Apply: not null in the last step: [batch, m, n], or [batch, n, m] if `transposed`
    int32_t transposed;
    float ca, cb, cc;
    OrthoForm form;       // Apply
    int32_t split;        // SPLIT: CTAs of a tile (2, 4 or 8)
    uint16_t *split_out;  // A without its diagonal
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
    // An epilogue warp's buffers, each two slabs: Apply hi and lo; Poly and Gram a tile and its mirror image. A pair has
    // one, and six stages in its ring: its main loops are as long as an epilogue that waits for what it has asked
    // for, and with four stages they take longer (Gram 185 -> 195 us). Single CTAs, which have the shorter tiles, have
    // three where something is fetched: the one that is worked on, the next one's and the last one's.
    static constexpr int kBuffers = OP == OrthoOp::kGram || CG == 2 ? 1 : 3;
    static constexpr int kBufferBytes = 2 * kSlabBytes;
    static constexpr int kInBytes = OP == OrthoOp::kGram ? 0 : OP == OrthoOp::kPoly ? kSlabBytes : 2 * kSlabBytes;
    static constexpr int kStages = (kBuffers == 1 ? 196608 : 131072) / kStageBytes / kProducers * kProducers;
    static_assert(!kSymmetric || kBM % NB == 0, "tiles beside the diagonal blocks");
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStageBytes + (size_t)kEpilogueWarps * kBuffers * kBufferBytes;
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
    __device__ OrthoWalk(const OrthoParams &p, int ctas)  // ctas: of a tile
        : tile(blockIdx.x / ctas), step(gridDim.x / ctas), mt((p.m + Sh::kBM - 1) / Sh::kBM), nt((p.n + NB - 1) / NB),
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

// An epilogue warp's tile of 32 x 32 halves lies in shared memory as TMA writes and reads a box of 64 bytes' width
// swizzled over 64 bytes, which is slab_at: 2 KB, one row to a lane. It comes and goes by TMA: with loads and stores of
// the warp's own, through registers, an epilogue took longer than the main loop of 2048 (Poly of 16 x 2048 rows 113 us, 101
// now; wavefronts of loads and stores 62 % of what is possible, now 14).
__device__ __forceinline__ void tma_store_3d(const CUtensorMap *map, const void *src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(map), "r"(smem_u32(src)),
                 "r"(x), "r"(y), "r"(z)
                 : "memory");
}
// What the warp has written to its slabs, or read from them, comes before the copies that one lane issues next, out of
// them or into them.
__device__ __forceinline__ void slabs_to_copies() {
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
}
// Rows and columns exchanged: this thread's row of 32 values becomes column `lane`.
__device__ __forceinline__ void slab_put_transposed(unsigned char *slab, int lane, const uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 32; ++i)
        *reinterpret_cast<uint16_t *>(slab + slab_at(i, lane / 8) + lane % 8 * 2) = (uint16_t)(v[i / 2] >> (i % 2 * 16));
}
// To rows of any length, value by value: columns [n, n + 32) of N. The slab is the next copies' from here on.
__device__ __forceinline__ void slab_store_any(const unsigned char *slab, int lane, ep_bf16 *base, int N, int n, int rows) {
    __syncwarp();
    if (n + lane < N)
        for (int r = 0; r < rows; ++r)
            base[(size_t)r * N + n + lane] = *reinterpret_cast<const uint16_t *>(slab + slab_at(r, lane / 8) + lane % 8 * 2);
    slabs_to_copies();
}
// Two halves as floats, and two registers as a pair.
__device__ __forceinline__ uint64_t halves(uint32_t v) {
    const float2 f = saved_values<false>(v);
    return pair(f.x, f.y);
}
__device__ __forceinline__ uint64_t pair_of(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }

// The 32 x 32 pieces of the tiles that an epilogue warp turns into results, in order.
template <OrthoOp OP, int CG, int NB>
struct OrthoPieces {
    using Sh = OrthoShape<OP, CG, NB>;
    OrthoWalk<OP, CG, NB> walk;
    OrthoTile t;
    int row, turn, width, m;  // the warp's first row of a tile; its turn of the columns
    int c = 0, c_end = 0;     // column of the tile; not c < c_end: no tile yet, or done with it
    __device__ OrthoPieces(const OrthoParams &p, int row_, int turn_)
        : walk(p, CG), row(row_), turn(turn_), width(Sh::kSymmetric ? p.mp : p.np), m(p.m) {}
    __device__ bool next_tile() {
        if (!walk.next(t)) return false;
        c = turn * kCols;
        c_end = t.m0 + row < m ? min(NB, width - t.n0) : 0;
        return true;
    }
    __device__ bool next() {
        c += 2 * kCols;
        while (c >= c_end)
            if (!next_tile()) return false;
        return true;
    }
};

// The CTAs of a cluster have added up a part of the contraction each (SPLIT), and left it in shared memory, a row of NB
// floats after the other. Each adds some rows of all parts up, in the same order, and stores them as the epilogue
// does. By `threads` threads.
template <int NB>
__device__ __forceinline__ int split_at(int row, int col) { return row * (NB * 4) + ((col / 4) ^ (row & 7)) * 16; }
template <int NB>
__device__ __forceinline__ void join_split(const OrthoParams &p, const OrthoTile &t, unsigned char *part, uint16_t *out, int rank, int ctas,
                                           int thread, int threads) {
    const int rows = kGemmBM / ctas;
    for (int i = thread; i < rows * (NB / 4); i += threads) {
        const int r = rank * rows + i / (NB / 4), c = i % (NB / 4) * 4;
        float4 f[8];  // asked for together
#pragma unroll
        for (int q = 0; q < 8; ++q) {
            f[q] = make_float4(0, 0, 0, 0);
            if (q < ctas)
                asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                             : "=f"(f[q].x), "=f"(f[q].y), "=f"(f[q].z), "=f"(f[q].w)
                             : "r"(cluster_smem_u32(part + split_at<NB>(r, c), q)));
        }
        float x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int q = 0; q < 8; ++q) x[0] += f[q].x, x[1] += f[q].y, x[2] += f[q].z, x[3] += f[q].w;
        const int row = t.m0 + r, n = t.n0 + c;
        if (row >= p.mp || n >= p.mp) continue;  // behind the last row: zeros, for the mirror image's last columns
        const size_t first = (size_t)t.matrix * p.m;
        alignas(8) __half h[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            float v = x[k] * (kA / (kX * kX));
            if (n + k == row && row < p.m) p.d_out[(size_t)t.matrix * p.mp + row] = v * (1.0f / kA), v = 0.0f;  // the diagonal is kept apart
            h[k] = __float2half_rn(v);
        }
        if (row < p.m) *reinterpret_cast<uint2 *>(out + (first + row) * p.mp + n) = *reinterpret_cast<const uint2 *>(h);
        if (t.mirror)
#pragma unroll
            for (int k = 0; k < 4; ++k) out[(first + n + k) * p.mp + row] = *reinterpret_cast<const uint16_t *>(&h[k]);
    }
}

// SPLIT (Gram, CG = 1): a cluster takes a tile, each CTA a part of its contraction; one tile for each cluster.
template <OrthoOp OP, int CG, int NB, bool SPLIT>
__global__ void __launch_bounds__(kGemmThreads, 1) ortho_gemm_kernel(const __grid_constant__ OrthoParams p) {
    using Sh = OrthoShape<OP, CG, NB>;
    constexpr int kStages = Sh::kStages;
    static_assert(!SPLIT || (OP == OrthoOp::kGram && CG == 1), "the epilogue of a split product");
    extern __shared__ unsigned char smem_raw[];
    // CG = 2: both CTAs' copies report to the first CTA's `full`
    __shared__ uint64_t full[kStages], empty[kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint64_t in_full[kEpilogueWarps][Sh::kBuffers];
    __shared__ uint32_t tmem_addr;
    __shared__ volatile int failed;

    unsigned char *stages = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    unsigned char *buffers = stages + kStages * Sh::kStageBytes;
    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0;
    const int kb_once = ((OP == OrthoOp::kGram ? p.n : p.m) + kGemmBK - 1) / kGemmBK;
    const int kb_all = OP == OrthoOp::kApply && p.form == OrthoForm::kWhole ? 2 * kb_once : kb_once;
    // this CTA's stages of the contraction
    const int part_of = SPLIT ? p.split : 1, part = SPLIT ? (int)cluster_cta_rank() : 0;
    const int kb_first = kb_all * part / part_of, kb = kb_all * (part + 1) / part_of - kb_first;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], kEpilogueWarps * CG);
        for (int i = 0; i < kEpilogueWarps * Sh::kBuffers; ++i) mbar_init(&in_full[0][i], 1);
        mbar_init(&drained, 1);
        failed = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.a);
        tma_prefetch_map(&p.b);
        if (Sh::kInBytes > 0) tma_prefetch_map(&p.in[0]);
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

    OrthoWalk<OP, CG, NB> walk(p, SPLIT ? p.split : CG);
    OrthoTile t;
    bool produces = false;
    uint32_t it = 0;     // the next fill of this producer
    uint32_t asked = 0;  // pieces that this epilogue warp has asked for

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
                    const bool lower = OP == OrthoOp::kApply && b >= kb_once;
                    const int k = (kb_first + b - (lower ? kb_once : 0)) * kGemmBK;
                    tma_load_3d<CG>(sa, &p.a, k, t.m0 + (int)rank * kGemmBM, t.matrix, bar);
                    if constexpr (Sh::kBMn) {
                        const CUtensorMap *x = lower ? &p.b_lo : &p.b;
#pragma unroll
                        for (int i = 0; i < Sh::kBRows / 64; ++i)
                            tma_load_3d<CG>(sb + i * 8192, x, t.n0 + (int)rank * Sh::kBRows + 64 * i, k, t.matrix, bar);
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
    } else if constexpr (SPLIT) {
        // ---- the accumulator as it is, into the stages' place: they have been read when it is complete
        const int quarter = warp % 4, turn = (warp - 2) / 4, row = quarter * 32 + lane;
        bool ok = true;
        if (lane == 0) ok = mbar_wait_limited(&acc_full[0], 0, &failed);
        __syncwarp();
        tmem_fence_after();
        for (int c = turn * kCols; c < NB; c += 2 * kCols) {
            uint32_t v[32];
            tmem_load_32(tmem + ((uint32_t)(quarter * 32) << 16) + c, v);
            tmem_wait_ld(v);
#pragma unroll
            for (int k = 0; k < 8; ++k)
                *reinterpret_cast<uint4 *>(stages + split_at<NB>(row, c + 4 * k)) = make_uint4(v[4 * k], v[4 * k + 1], v[4 * k + 2], v[4 * k + 3]);
        }
    } else {
        // ---- epilogue: warp w reads lanes [32 (w mod 4), + 32) of the accumulators, one row a thread, and
        // two warps take the same rows' columns in turns of 32
        constexpr bool kFetches = Sh::kInBytes > 0;
        const int quarter = warp % 4, turn = (warp - 2) / 4;
        const int row = (int)rank * kGemmBM + quarter * 32;  // of the tile
        unsigned char *mine = buffers + (warp - 2) * Sh::kBuffers * Sh::kBufferBytes;
        uint64_t *arrived = in_full[warp - 2];
        OrthoPieces<OP, CG, NB> ahead(p, row, turn);  // what has been asked for
        // The next piece into the buffer after the last one's. What was sent out from there has to have been read:
        // with three buffers only the last piece's copies may still be under way.
        const auto ask = [&]() {
            if (!kFetches || !ahead.next()) return;
            if (lane == 0) {
                unsigned char *to = mine + asked % Sh::kBuffers * Sh::kBufferBytes;
                uint64_t *bar = &arrived[asked % Sh::kBuffers];
                bulk_wait_read<(Sh::kBuffers > 1)>();
                mbar_arrive_expect_tx(bar, Sh::kInBytes);
                const int x = ahead.t.n0 + ahead.c, y = ahead.t.m0 + row;
                tma_load_3d<1>(to, &p.in[0], x, y, ahead.t.matrix, smem_u32(bar));
                if (OP == OrthoOp::kApply) tma_load_3d<1>(to + kSlabBytes, &p.in[1], x, y, ahead.t.matrix, smem_u32(bar));
            }
            ++asked;
        };
        ask();
        uint32_t acc_it = 0, piece = 0;
        OrthoPieces<OP, CG, NB> at(p, row, turn);
        bool ok = true;
        while (ok && at.next_tile()) {
            const OrthoTile &t = at.t;
            const uint32_t slot = acc_it & 1;
            const int first = t.m0 + row, i = first + lane;  // the warp's first row, and this thread's
            const uint32_t src = tmem + ((uint32_t)(quarter * 32) << 16) + slot * NB;
            const size_t diag = (size_t)t.matrix * p.mp;
            float di = 0.0f;
            if (OP != OrthoOp::kGram && i < p.m) di = p.d[diag + i];
            if (lane == 0) ok = mbar_wait_limited(&acc_full[slot], (acc_it / 2) & 1, &failed);
            ok = __shfl_sync(0xFFFFFFFFu, ok, 0);
            if (!ok) break;
            ++acc_it;
            tmem_fence_after();
            for (; at.c < at.c_end; at.c += 2 * kCols, ++piece) {
                const int c = at.c, n = t.n0 + c;
                unsigned char *slab = mine + piece % Sh::kBuffers * Sh::kBufferBytes, *second = slab + kSlabBytes;
                uint32_t v[32], o[16];
                float4 dj[8];  // Poly: A's diagonal at the piece's columns
                if constexpr (OP == OrthoOp::kPoly) {
#pragma unroll
                    for (int k = 0; k < 8; ++k) dj[k] = *reinterpret_cast<const float4 *>(p.d + diag + n + 4 * k);
                }
                if (Sh::kBuffers > 1) ask();
                if (kFetches) {
                    ok = mbar_wait_warp(&arrived[piece % Sh::kBuffers], piece / Sh::kBuffers & 1, &failed);
                    if (!ok) break;
                }
                if constexpr (OP == OrthoOp::kApply) {
                    uint32_t hi[16], lo[16];
                    slab_get(slab, lane, hi);
                    slab_get(second, lane, lo);
                    tmem_load_32(src + c, v);
                    tmem_wait_ld(v);
                    const float dl = p.form == OrthoForm::kUpper ? p.ca : di;
                    const uint64_t d2 = pair(di, di), dl2 = pair(dl, dl), by_b = pair(1.0f / kB, 1.0f / kB);
#pragma unroll
                    for (int k = 0; k < 16; ++k) {
                        // a + B's diagonal times hi + lo (kUpper: a times lo), and the product
                        const uint64_t x = fma2(d2, halves(hi[k]), fma2(dl2, halves(lo[k]), mul2(pair_of(v[2 * k], v[2 * k + 1]), by_b)));
                        if (p.result) {
                            const uint64_t y = mul2(x, pair(1.0f / kX, 1.0f / kX));
                            o[k] = bf16_pair(low(y), high(y));
                        } else {
                            o[k] = half_pair(low(x), high(x));
                            const uint64_t r = fma2(halves(o[k]), pair(-1.0f, -1.0f), x);
                            lo[k] = half_pair(low(r), high(r));
                        }
                    }
                    if (!p.result) {
                        slab_put(slab, lane, o);
                        slab_put(second, lane, lo);
                        slabs_to_copies();
                        if (lane == 0) {
                            tma_store_3d(&p.out[0], slab, n, first, t.matrix);
                            tma_store_3d(&p.out[1], second, n, first, t.matrix);
                        }
                    } else if (p.transposed) {
                        __syncwarp();  // other lanes' rows are written over
                        slab_put_transposed(slab, lane, o);
                        if (p.m % 8 == 0) {
                            slabs_to_copies();
                            if (lane == 0) tma_store_3d(&p.out[0], slab, first, n, t.matrix);
                        } else {
                            slab_store_any(slab, lane, p.result + ((size_t)t.matrix * p.n + n) * p.m, p.m, first, min(32, p.n - n));
                        }
                    } else {
                        slab_put(slab, lane, o);
                        if (p.n % 8 == 0) {
                            slabs_to_copies();
                            if (lane == 0) tma_store_3d(&p.out[0], slab, n, first, t.matrix);
                        } else {
                            slab_store_any(slab, lane, p.result + ((size_t)t.matrix * p.m + first) * p.n, p.n, n, min(32, p.m - first));
                        }
                    }
                } else {
                    uint64_t x[16];
                    if constexpr (OP == OrthoOp::kPoly) {
                        uint32_t a[16];
                        slab_get(slab, lane, a);
                        tmem_load_32(src + c, v);
                        tmem_wait_ld(v);
                        // kB (A (b + c (di + dj)) + c acc), A and acc as they are stored
                        const float by_a = kB / kA, base = by_a * fmaf(p.cc, di, p.cb);
                        const uint64_t base2 = pair(base, base), cc2 = pair(by_a * p.cc, by_a * p.cc);
                        const uint64_t acc2 = pair(p.cc * (kB / (kA * kA)), p.cc * (kB / (kA * kA)));
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const uint64_t d2 = k % 2 ? pair(dj[k / 2].z, dj[k / 2].w) : pair(dj[k / 2].x, dj[k / 2].y);
                            x[k] = fma2(halves(a[k]), fma2(cc2, d2, base2), mul2(pair_of(v[2 * k], v[2 * k + 1]), acc2));
                        }
                    } else {
                        tmem_load_32(src + c, v);
                        tmem_wait_ld(v);
                        const uint64_t by = pair(kA / (kX * kX), kA / (kX * kX));
#pragma unroll
                        for (int k = 0; k < 16; ++k) x[k] = mul2(pair_of(v[2 * k], v[2 * k + 1]), by);
                    }
                    if (n == first) {  // the diagonal is kept apart, by selections: 32 branches of one lane each took 1.5 us
                        float e = 0.0f;
#pragma unroll
                        for (int k = 0; k < 16; ++k) {
                            const bool even = lane == 2 * k, odd = lane == 2 * k + 1;
                            e = even ? low(x[k]) : odd ? high(x[k]) : e;
                            x[k] = pair(even ? 0.0f : low(x[k]), odd ? 0.0f : high(x[k]));
                        }
                        if (i < p.m)
                            p.d_out[diag + i] = OP == OrthoOp::kGram ? e * (1.0f / kA) : fmaf(e, 1.0f / kB, p.ca + fmaf(p.cc * di, di, p.cb * di));
                    }
                    if (n + 32 > p.m) {  // zeros behind the last column
#pragma unroll
                        for (int k = 0; k < 16; ++k)
                            x[k] = pair(n + 2 * k < p.m ? low(x[k]) : 0.0f, n + 2 * k + 1 < p.m ? high(x[k]) : 0.0f);
                    }
#pragma unroll
                    for (int k = 0; k < 16; ++k) o[k] = half_pair(low(x[k]), high(x[k]));
                    if (!kFetches) {  // the buffer's last content has to be out
                        if (lane == 0) bulk_wait_read<0>();
                        __syncwarp();
                    }
                    slab_put(slab, lane, o);
                    if (t.mirror) slab_put_transposed(second, lane, o);
                    slabs_to_copies();
                    if (lane == 0) {
                        tma_store_3d(&p.out[0], slab, n, first, t.matrix);
                        if (t.mirror) tma_store_3d(&p.out[0], second, first, n, t.matrix);
                    }
                }
                if (lane == 0) bulk_commit();
                if (Sh::kBuffers == 1) ask();
            }
            if (!ok) break;
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) {
                if constexpr (CG == 2)
                    mbar_arrive_cluster(cluster_smem_u32(&acc_empty[slot], 0));
                else
                    mbar_arrive(&acc_empty[slot]);
            }
        }
        if (lane == 0) bulk_wait<0>();
        __syncwarp();
    }

    __syncthreads();
    if constexpr (SPLIT) {
        cluster_sync();
        walk.next(t);  // the cluster's tile
        join_split<NB>(p, t, stages, p.split_out, part, part_of, threadIdx.x, kGemmThreads);
        cluster_sync();  // no CTA may end while another one reads its memory
    }
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
        } else if (warp > 1 && warp < 2 + kEpilogueWarps) {
            if (lane == 0) wait_for_fills(in_full[warp - 2], asked, 0, 1, Sh::kBuffers);
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
