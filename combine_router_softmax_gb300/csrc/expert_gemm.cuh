// expert_gemm.cuh -- the experts' matrix products on the tensor cores, grouped by expert.
//
// The rows of the send buffer lie grouped by expert: expert e owns rows
// [expert_offset[e], expert_offset[e + 1]), known on the device only. Five products share
// one kernel (S rows, the weights of expert e in brackets, s the owner's rows):
//   GateUp   g = x Wg[e]^T, u = x Wu[e]^T, and h = silu(g) u from the accumulators
//   Down     y = h Wd[e]^T
//   DGateUp  dh = dy Wd[e], and from the accumulators du = dh silu(g),
//            dg = dh u s (1 + g (1 - s)), s = sigmoid(g)
//   DRows    dx = dg Wg[e] + du Wu[e]: one accumulation over 2 I
//   DWeight  dWd[e] = dy^T h, dWg[e] = dg^T x, dWu[e] = du^T x over the expert's rows
// Operands are bf16, sums fp32 (in TMEM), results are rounded to bf16 once. h, dg and du are
// rounded to bf16 where they become operands of the next product. g and u are no operands: they are
// kept for the backward pass in fp16, which rounds eight times finer in the same 16 bits (the weights'
// gradients are 0.0024 off in norm with it, 0.0031 with bf16) from 6e-5 on, or in bf16, whose range is fp32's.
// What is finite and lies beyond the type's largest value is kept as that (65504: silu and its derivative
// are at their limits there); as infinity it would make NaN of a gradient of 0 (s = 0 times g).
//
// One persistent CTA per SM (CG = 2: one CTA pair per two SMs, a tile of 256 rows, each CTA
// holding half of either operand): two producer warps feed a ring of shared-memory stages by TMA, in
// turn, warp 1 issues the MMAs into one of two accumulators, warps 2 to 9 turn the other one into
// results. Every wait has a time limit (kErrExpertWait).
//
// What bounds it. With many rows the tensor pipe: 16 experts x 1024 rows, 4096 to 2048 and back,
// forward 466 us = 1771 TFLOP/s, DGateUp 1572, DRows 1844, DWeight 1728 (64 KB written for
// every 16 stages) of a library product's 2040 in the same burst; experts of uneven size lose what their
// last tiles do not fill. As single CTAs the forward is 10% slower: 128 x 256 tiles
// move 48 KB into shared memory and read 48 KB out for 512 cycles of MMA, 192 bytes a cycle
// where there are 128; a pair's 256 x 256 halves what each SM moves. With few rows an expert the
// weights' stream: 512 rows over 64 experts of 7168 / 2048 in 809 us = 7.0 TB/s. Between the two, what
// a stage costs the threads that serve it: one producer took 520 cycles a stage whatever its copies, as
// many as the MMAs of a pair's stage (two: 16384 rows, 4096 to 2048, all gradients 1670 -> 1607 us), the
// issuer takes 330 (470 without its loop unrolled).
#pragma once

#include <cuda_fp16.h>

#include "tcgen05.cuh"

namespace ep {

enum class ExpertOp { kGateUp, kDown, kDGateUp, kDRows, kDWeight };

constexpr int kEpilogueWarps = 8;
constexpr int kProducers = 2;
constexpr int kGemmThreads = 32 * (1 + kEpilogueWarps + kProducers);
constexpr int kGemmBK = 64;   // contraction per stage: 128 bytes of bf16, one swizzled row
constexpr int kGemmBM = 128;  // rows of a CTA's tile: the TMEM lanes
constexpr int kSlabBytes = 32 * 64;

struct GemmParams {
    CUtensorMap a[3];    // K-major: box 64 k x 128 rows; MN-major: box 64 m x 64 k
    CUtensorMap a64[2], a16[2];  // K-major: boxes of 64 and 16 rows, for tiles with few rows
    CUtensorMap b[3];
    const int32_t *expert_offset;
    int32_t E, S;
    int32_t K;         // contraction of the row products (of each half, DRows)
    int32_t M[3];      // DWeight: output rows of each problem
    int32_t N[3];      // output columns of each problem (row products: N[0])
    int32_t problems;  // DWeight: how many of the three are wanted
    ep_bf16 *out[3];   // GateUp: h; DGateUp: dg, du; DWeight: the gradients [E, M, N]
    uint16_t *g, *u;   // GateUp: written when not null; DGateUp: read
    int32_t saved_bf16;  // their type: 0 fp16, 1 bf16
    int32_t *error;
};

template <ExpertOp OP, int CG, int NB>
struct GemmShape {
    static constexpr bool kDW = OP == ExpertOp::kDWeight;
    static constexpr bool kAMn = kDW;
    static constexpr bool kBMn = OP == ExpertOp::kDGateUp || OP == ExpertOp::kDRows || kDW;
    static constexpr int kOutN = OP == ExpertOp::kGateUp ? NB / 2 : NB;  // output columns of a tile
    static constexpr int kGate = kOutN < 64 ? kOutN : 64;  // GateUp: B is so many rows of Wg, as many of Wu, and so on
    static constexpr int kBRows = NB / CG;                 // B rows a CTA holds
    static constexpr int kABytes = kGemmBM * 128;
    static constexpr int kBBytes = kBRows * 128;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = 196608 / kStageBytes;
    static_assert(kStages % kProducers == 0 && kStages < 32, "a stage has one producer, and a bit");
    static constexpr int kTmemCols = 2 * NB;
    static constexpr size_t smem_bytes(int E) { return 1024 + (size_t)kStages * kStageBytes + kEpilogueWarps * kSlabBytes + (size_t)(E + 1) * 8 + (size_t)E * 8; }
};

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t half_pair(float lo, float hi) {
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}
// exp(-x) overflows to infinity for x below -88: the quotient is then 0, the limit.
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.0f, 1.0f + __expf(-x)); }
// 32 sums as they are kept for the backward pass. Beyond the type's largest value, which hardly ever occurs,
// a finite one is kept as that; infinities and NaN stay.
__device__ __forceinline__ void saved_pairs(const uint32_t (&v)[32], uint32_t (&o)[16], bool bf16) {
    const float top = bf16 ? 3.38953139e38f : 65504.0f;
    float most = 0.0f;
#pragma unroll
    for (int i = 0; i < 32; ++i) most = fmaxf(most, fabsf(__uint_as_float(v[i])));
    if (most > top) {
        const auto within = [&](uint32_t bits) {
            const float x = __uint_as_float(bits);
            return fabsf(x) < INFINITY ? fminf(fmaxf(x, -top), top) : x;
        };
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float lo = within(v[2 * i]), hi = within(v[2 * i + 1]);
            o[i] = bf16 ? bf16_pair(lo, hi) : half_pair(lo, hi);
        }
    } else if (bf16) {
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = bf16_pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) o[i] = half_pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
    }
}
template <bool BF16>
__device__ __forceinline__ float2 saved_values(uint32_t v) {
    if constexpr (BF16)
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    else
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
}
// d_g and d_u of a row's 32 columns from d_h; u's place takes d_u.
template <bool BF16>
__device__ __forceinline__ void gate_gradients(const uint32_t (&dh)[32], const uint32_t (&g)[16], uint32_t (&u)[16],
                                               uint32_t (&d_g)[16]) {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        float dg[2], du[2];
        const float2 g2 = saved_values<BF16>(g[i]), u2 = saved_values<BF16>(u[i]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float d = __uint_as_float(dh[2 * i + k]);
            const float gg = k ? g2.y : g2.x, uu = k ? u2.y : u2.x;
            const float s = sigmoid(gg);
            // s first: it may be 0 where dh g or dh u overflows
            du[k] = d * (gg * s);
            dg[k] = d * (uu * (s * (1.0f + gg * (1.0f - s))));
        }
        d_g[i] = bf16_pair(dg[0], dg[1]);
        u[i] = bf16_pair(du[0], du[1]);
    }
}

// An epilogue warp's results lie one row to a thread, 32 columns at a time; they pass through a slab
// of shared memory (32 rows of 64 bytes, 16-byte words swizzled by the row) so that global memory
// is written, and read, 64 bytes of a row at a time: 4 threads to a row. Stores straight from the
// registers touch 32 rows at once, 16 bytes of each, and took longer than the main loop of a short
// contraction.
constexpr int kCols = 32;
__device__ __forceinline__ int slab_at(int row, int word) { return row * 64 + ((word ^ (row / 2 % 4)) * 16); }

// 32 values of this thread's row into the slab.
__device__ __forceinline__ void slab_put(unsigned char *slab, int lane, const uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
        *reinterpret_cast<uint4 *>(slab + slab_at(lane, i)) = make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}
__device__ __forceinline__ void slab_get(const unsigned char *slab, int lane, uint32_t (&v)[16]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint4 q = *reinterpret_cast<const uint4 *>(slab + slab_at(lane, i));
        v[4 * i] = q.x, v[4 * i + 1] = q.y, v[4 * i + 2] = q.z, v[4 * i + 3] = q.w;
    }
}
// The slab's first `rows` rows to columns [n, n + 32) of N, N % 8 == 0, of the rows from `base` on.
__device__ __forceinline__ void slab_store(const unsigned char *slab, int lane, ep_bf16 *base, int N, int n, int rows) {
    __syncwarp();
    const int c = lane % 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * j + lane / 4;
        if (r < rows && n + 8 * c < N)
            st_v4(reinterpret_cast<uint4 *>(base + (size_t)r * N + n + 8 * c),
                  *reinterpret_cast<const uint4 *>(slab + slab_at(r, c)));
    }
    __syncwarp();
}
// The other way round, as loads that are put into the slab once they are there (slab_fill).
__device__ __forceinline__ void slab_load(uint4 (&q)[4], int lane, const uint16_t *base, int N, int n, int rows) {
    const int c = lane % 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int r = 8 * j + lane / 4;
        q[j] = r < rows && n + 8 * c < N ? *reinterpret_cast<const uint4 *>(base + (size_t)r * N + n + 8 * c)
                                         : make_uint4(0, 0, 0, 0);
    }
}
__device__ __forceinline__ void slab_fill(unsigned char *slab, int lane, const uint4 (&q)[4]) {
#pragma unroll
    for (int j = 0; j < 4; ++j) *reinterpret_cast<uint4 *>(slab + slab_at(8 * j + lane / 4, lane % 4)) = q[j];
    __syncwarp();
}

// One tile of the kernel's list, the same for every warp.
struct Tile {
    int e, problem;
    int m0;     // first row (row products), first output row (DWeight)
    int valid;  // rows of the expert from m0 on / output rows from m0 on
    int n0;     // first output column
    int row0, rows;  // DWeight: the expert's rows
};

// Walks the tiles of one CTA (pair): first, first + step, ... The tables are in shared memory.
template <ExpertOp OP, int CG, int NB>
struct Walk {
    using Sh = GemmShape<OP, CG, NB>;
    static constexpr int kBM = kGemmBM * CG;
    const GemmParams &p;
    const int *lo, *count;  // first row and rows of an expert
    const int64_t *prefix;  // m-tiles before it
    int64_t tile, step;
    int e = 0;

    __device__ Walk(const GemmParams &p_, const int *lo_, const int *count_, const int64_t *prefix_)
        : p(p_), lo(lo_), count(count_), prefix(prefix_), tile(blockIdx.x / CG), step(gridDim.x / CG) {}

    // Tile `rest` of mt x nt: down the `band` tiles of a band, then along the columns. With bands of 2048
    // rows the tiles at work at a time form a block about as high as wide, which reads the fewest
    // different rows of A and B: one expert of 8192 rows, 8192 to 8192 and back, forward 1878 -> 1743 us,
    // the weights' gradients 2172 -> 1978. Where the whole contraction fits L2 it gains nothing, and for
    // the weights' gradients costs: 8 experts of 1024 rows 2267 -> 2377 us, so there only with more than
    // 2048 rows.
    static constexpr int kBand = 2048 / kBM;
    __device__ static void place(int64_t rest, int64_t mt, int nt, int64_t band, int &m, int &n) {
        const int64_t first = rest / (band * nt) * band;
        const int high = (int)min(band, mt - first);
        const int r = (int)(rest - first * nt);
        m = (int)first + r % high;
        n = r / high;
    }

    __device__ bool next(Tile &t) {
        if constexpr (Sh::kDW) {
            int64_t per_e = 0;
            for (int i = 0; i < p.problems; ++i)
                per_e += (int64_t)((p.M[i] + kBM - 1) / kBM) * ((p.N[i] + NB - 1) / NB);
            t.e = (int)(tile / per_e);
            if (t.e >= p.E) return false;
            int64_t rest = tile % per_e;
            int i = 0;
            for (; i < p.problems - 1; ++i) {
                const int64_t n = (int64_t)((p.M[i] + kBM - 1) / kBM) * ((p.N[i] + NB - 1) / NB);
                if (rest < n) break;
                rest -= n;
            }
            const int mt = (p.M[i] + kBM - 1) / kBM;
            t.problem = i;
            int m, n;
            place(rest, mt, (p.N[i] + NB - 1) / NB, count[t.e] > 2048 ? kBand : mt, m, n);
            t.m0 = m * kBM;
            t.n0 = n * NB;
            t.valid = p.M[i] - t.m0;
            t.row0 = lo[t.e];
            t.rows = count[t.e];
        } else {
            const int nt = (p.N[0] + Sh::kOutN - 1) / Sh::kOutN;
            if (tile >= prefix[p.E] * nt) return false;
            while (tile >= prefix[e + 1] * nt) ++e;
            const int64_t rest = tile - prefix[e] * nt;
            const int64_t mt = prefix[e + 1] - prefix[e];
            int m, n;
            place(rest, mt, nt, kBand, m, n);
            t.e = e;
            t.problem = 0;
            t.m0 = lo[e] + m * kBM;
            t.valid = count[e] - m * kBM;
            t.n0 = n * Sh::kOutN;
        }
        tile += step;
        return true;
    }
    // stages that the tile's contraction takes
    __device__ int blocks(const Tile &t) const {
        if constexpr (Sh::kDW) return (t.rows + kGemmBK - 1) / kGemmBK;
        const int kb = (p.K + kGemmBK - 1) / kGemmBK;
        return OP == ExpertOp::kDRows ? 2 * kb : kb;
    }
};

// Rows of A that are fetched for a CTA with `valid` rows left, of `most`: one box of 128 or 64, or one or
// two of 16. A copy costs its thread about 60 cycles whatever its size, so more than 32 rows are one box
// (prefill with uneven experts 892 -> 868 us). The MMA computes all rows; what lies in the others reaches
// only result rows that are not stored.
__device__ __forceinline__ int a_rows_fetched(int valid, int most) {
    valid = min(valid, most);
    return valid <= 0 ? 0 : valid > 64 ? 128 : valid > 32 ? 64 : (valid + 15) / 16 * 16;
}

// A CTA pair's last tile of an expert, when 128 rows or fewer are left: half the MMA (M = 128), 64 rows
// a CTA. Its accumulator lies in half the columns: lanes 0 to 63 hold the rows' first half of the N
// columns, lanes 64 to 127 the second.
template <ExpertOp OP, int CG>
__device__ __forceinline__ bool half_tile(const Tile &t) {
    return CG == 2 && OP != ExpertOp::kDWeight && t.valid <= kGemmBM;
}

// DWeight: a stage whose rows go past the expert's end also holds rows of the next one, which
// count for nothing: zeroed, in both operands, up to a whole step of 16. `left` rows are the
// expert's. Returns the steps the stage takes. By one warp.
template <typename Sh>
__device__ __forceinline__ int zero_rows_past_end(unsigned char *stage, int left, int lane) {
    if (left >= kGemmBK) return kGemmBK / 16;
    const int steps = (left + 15) / 16;
    const int zero = (steps * 16 - left) * 8;  // 16-byte words of a 64-wide column block
    for (int i = lane; i < (kGemmBM + Sh::kBRows) / 64 * zero; i += 32)
        reinterpret_cast<uint4 *>(stage + i / zero * 8192 + left * 128)[i % zero] = make_uint4(0, 0, 0, 0);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    return steps;
}

template <ExpertOp OP, int CG, int NB>
__global__ void __launch_bounds__(kGemmThreads, 1) expert_gemm_kernel(const __grid_constant__ GemmParams p) {
    using Sh = GemmShape<OP, CG, NB>;
    constexpr int kStages = Sh::kStages;
    extern __shared__ unsigned char smem_raw[];
    // CG = 2: both CTAs' copies report to the first CTA's `full`. Only the last stage of a DWeight
    // tile, when it goes past the expert's end, differs: the second CTA's copies report to its own
    // `full`, it zeroes those rows and arrives on the first one's `other`. Both barriers of a stage
    // count such uses alone, so their parities are kept as bits, one a stage.
    constexpr bool kRelay = Sh::kDW && CG == 2;
    __shared__ uint64_t full[kStages], empty[kStages], other[kStages], acc_full[2], acc_empty[2], drained;
    __shared__ uint32_t tmem_addr;
    __shared__ volatile int failed;

    unsigned char *stages = smem_raw + (1024 - (smem_u32(smem_raw) & 1023)) % 1024;
    unsigned char *slabs = stages + kStages * Sh::kStageBytes;
    int64_t *prefix = reinterpret_cast<int64_t *>(slabs + kEpilogueWarps * kSlabBytes);
    int *lo = reinterpret_cast<int *>(prefix + p.E + 1), *count = lo + p.E;

    const int warp = threadIdx.x / 32, lane = threadIdx.x % 32;
    const uint32_t rank = CG == 2 ? cluster_cta_rank() : 0;

    if (warp == 0 && lane == 0) {
        for (int i = 0; i < kStages; ++i) mbar_init(&full[i], 1), mbar_init(&empty[i], 1), mbar_init(&other[i], 1);
        for (int i = 0; i < 2; ++i) mbar_init(&acc_full[i], 1), mbar_init(&acc_empty[i], kEpilogueWarps * CG);
        mbar_init(&drained, 1);
        failed = 0;
        fence_mbar_init();
        tma_prefetch_map(&p.a[0]);
        tma_prefetch_map(&p.b[0]);
    }
    if (warp == 1) tmem_alloc<CG>(&tmem_addr, Sh::kTmemCols);
    grid_dependency_wait();
    grid_launch_dependents();
    // bounds come from device memory: kept inside the row buffer whatever they hold
    for (int e = threadIdx.x; e < p.E; e += kGemmThreads) {
        const int first = min(max(p.expert_offset[e], 0), p.S);
        lo[e] = first;
        count[e] = min(max(p.expert_offset[e + 1], first), p.S) - first;
    }
    __syncthreads();
    if (!Sh::kDW && warp == 2) {
        int64_t sum = 0;
        for (int base = 0; base < p.E; base += 32) {
            const int e = base + lane;
            int64_t v = e < p.E ? (count[e] + (int64_t)kGemmBM * CG - 1) / (kGemmBM * CG) : 0;
            for (int d = 1; d < 32; d *= 2) {
                const int64_t o = __shfl_up_sync(0xFFFFFFFFu, v, d);
                if (lane >= d) v += o;
            }
            if (e < p.E) prefix[e + 1] = sum + v;
            sum += __shfl_sync(0xFFFFFFFFu, v, 31);
        }
        if (lane == 0) prefix[0] = 0;
    }
    tmem_fence_before();
    if constexpr (CG == 2)
        cluster_sync();
    else
        __syncthreads();
    tmem_fence_after();
    const uint32_t tmem = tmem_addr;

    Walk<OP, CG, NB> walk(p, lo, count, prefix);
    Tile t;
    // what a producer has under way (it: the next fill of its thread; kRelay's uses of the second CTA's `full`)
    bool produces = false;
    uint32_t it = 0, relayed = 0, ever = 0;

    if (warp == 0 || warp > 1 + kEpilogueWarps) {
        // ---- producers: one lane each, which take the stages in turn
        if (elect_one()) {
            const uint32_t mine = warp == 0 ? 0 : warp - 1 - kEpilogueWarps;
            produces = true;
            it = mine;
            uint32_t s = mine, phase = 0;  // it % kStages, it / kStages % 2: kept by counting, a stage is few instructions
            int b = mine;                  // of the tile
            bool ok = true, ready = false;
            while (ok && walk.next(t)) {
                const int kb = walk.blocks(t);
                const int most = half_tile<OP, CG>(t) ? kGemmBM / 2 : kGemmBM;  // rows of a CTA
                const int fetched = Sh::kDW ? 0 : a_rows_fetched(t.valid - (int)rank * most, most);
                uint32_t bytes = Sh::kBBytes * CG;
                if constexpr (Sh::kDW)
                    bytes += Sh::kABytes * CG;
                else
                    for (int r = 0; r < CG; ++r) bytes += a_rows_fetched(t.valid - r * most, most) * 128;
#pragma unroll 2
                for (; b < kb; b += kProducers, it += kProducers) {
                    if (it >= kStages && !ready && !mbar_poll_limited(&empty[s], phase ^ 1, &failed)) {
                        ok = false;
                        break;
                    }
                    const bool wraps = s + kProducers >= kStages;
                    const uint32_t next = s + kProducers - (wraps ? kStages : 0), next_phase = wraps ? phase ^ 1 : phase;
                    ready = it + kProducers >= kStages && mbar_test(&empty[next], next_phase ^ 1);
                    const bool relay = kRelay && t.rows - b * kGemmBK < kGemmBK;
                    if (rank == 0 || relay) mbar_arrive_expect_tx(&full[s], relay ? bytes / 2 : bytes);
                    if (relay) relayed ^= 1u << s, ever |= 1u << s;
                    const uint32_t bar = CG == 2 && !relay ? cluster_smem_u32(&full[s], 0) : smem_u32(&full[s]);
                    unsigned char *sa = stages + s * Sh::kStageBytes, *sb = sa + Sh::kABytes;
                    if constexpr (Sh::kDW) {
                        const int k = t.row0 + b * kGemmBK;
#pragma unroll
                        for (int i = 0; i < kGemmBM / 64; ++i)
                            tma_load_2d<CG>(sa + i * 8192, &p.a[t.problem], t.m0 + (int)rank * kGemmBM + 64 * i, k, bar);
#pragma unroll
                        for (int i = 0; i < Sh::kBRows / 64; ++i)
                            tma_load_2d<CG>(sb + i * 8192, &p.b[t.problem], t.n0 + (int)rank * Sh::kBRows + 64 * i, k, bar);
                    } else {
                        const int half = OP == ExpertOp::kDRows && b >= kb / 2 ? 1 : 0;
                        const int k = (half ? b - kb / 2 : b) * kGemmBK;
                        const int row = t.m0 + (int)rank * most;
                        if (fetched == 128)
                            tma_load_2d<CG>(sa, &p.a[half], k, row, bar);
                        else if (fetched == 64)
                            tma_load_2d<CG>(sa, &p.a64[half], k, row, bar);
                        else
                            for (int i = 0; i < fetched; i += 16)
                                tma_load_2d<CG>(sa + i * 128, &p.a16[half], k, row + i, bar);
                        if constexpr (OP == ExpertOp::kGateUp) {
#pragma unroll
                            for (int i = 0; i < Sh::kBRows / Sh::kGate; ++i)
                                tma_load_3d<CG>(sb + i * Sh::kGate * 128, &p.b[i % 2], k,
                                                t.n0 + (int)rank * (Sh::kBRows / 2) + i / 2 * Sh::kGate, t.e, bar);
                        } else if constexpr (!Sh::kBMn) {
                            tma_load_3d<CG>(sb, &p.b[0], k, t.n0 + (int)rank * Sh::kBRows, t.e, bar);
                        } else {
#pragma unroll
                            for (int i = 0; i < Sh::kBRows / 64; ++i)
                                tma_load_3d<CG>(sb + i * 8192, &p.b[half], t.n0 + (int)rank * Sh::kBRows + 64 * i, k,
                                                t.e, bar);
                        }
                    }
                    s = next;
                    phase = next_phase;
                }
                b -= kb;
            }
        }
        __syncwarp();
    } else if (warp == 1) {
        // ---- MMA issuer (CG = 2: of the pair's first CTA)
        if (rank == 0) {
            constexpr uint32_t idesc_whole = mma_idesc(kGemmBM * CG, NB, Sh::kAMn, Sh::kBMn);
            constexpr uint32_t idesc_half = mma_idesc(kGemmBM, NB, Sh::kAMn, Sh::kBMn);
            const uint64_t da_first = smem_desc(smem_u32(stages), Sh::kAMn ? 8192 : 16);
            const uint64_t db_first = smem_desc(smem_u32(stages) + Sh::kABytes, Sh::kBMn ? 8192 : 16);
            uint32_t s = 0, phase = 0, acc_it = 0;
            bool ok = true, ready = false;
            while (ok && walk.next(t)) {
                const int kb = walk.blocks(t);
                if (kb == 0) continue;
                const uint32_t slot = acc_it & 1;
                const uint32_t d = tmem + slot * NB;
                const uint32_t idesc = half_tile<OP, CG>(t) ? idesc_half : idesc_whole;
                // the stage's MMAs; one thread
                const auto issue = [&](uint32_t s, int steps, int b) {
                    const uint64_t da = da_first + s * (Sh::kStageBytes / 16), db = db_first + s * (Sh::kStageBytes / 16);
                    for (int k = 0; k < steps; ++k)
                        mma_bf16<CG>(d, da + k * (Sh::kAMn ? 128 : 2), db + k * (Sh::kBMn ? 128 : 2), idesc, b + k > 0);
                    mma_commit<CG>(&empty[s]);
                    if (b == kb - 1) mma_commit<CG>(&acc_full[slot]);
                };
                const int whole = Sh::kDW ? t.rows / kGemmBK : kb;  // stages without a row past the expert's end
                bool issued = false;
                if (elect_one()) {
                    if (acc_it >= 2) ok = mbar_poll_limited<CG == 2>(&acc_empty[slot], (acc_it / 2 - 1) & 1, &failed);
                    tmem_fence_after();
                    uint32_t at = s, parity = phase;
#pragma unroll 4
                    for (int b = 0; ok && b < whole; ++b) {
                        ok = ready || mbar_poll_limited(&full[at], parity, &failed);
                        const uint32_t next = at + 1 == kStages ? 0 : at + 1;
                        if (next == 0) parity ^= 1;
                        ready = mbar_test(&full[next], parity);
                        if (ok) issue(at, kGemmBK / 16, b);
                        at = next;
                    }
                    issued = ok;
                }
                // that thread's waits count for all: lanes that each read `failed` could part here, and the
                // next elect.sync would wait for the missing ones without a limit
                ok = __any_sync(0xFFFFFFFFu, issued);
                phase ^= (s + whole) / kStages % 2;
                s = (s + whole) % kStages;
                if constexpr (Sh::kDW)
                    if (whole < kb) {
                        ready = false;
                        // every lane waits: each is to see the copies that it zeroes a part of
                        ok = ok && mbar_wait_warp(&full[s], phase, &failed);
                        const int steps = zero_rows_past_end<Sh>(stages + s * Sh::kStageBytes, t.rows - whole * kGemmBK, lane);
                        if (kRelay && ok) {
                            ok = mbar_wait_warp<true>(&other[s], relayed >> s & 1, &failed);
                            relayed ^= 1u << s;
                        }
                        if (elect_one() && ok) issue(s, steps, whole);
                        __syncwarp();
                        if (++s == kStages) s = 0, phase ^= 1;
                    }
                ++acc_it;
            }
        } else if (kRelay) {
            // the pair's second CTA: its part of the stages that go past an expert's end
            while (walk.next(t)) {
                const int kb = walk.blocks(t);
                it += kb;
                if (t.rows % kGemmBK == 0) continue;
                const int s = (it - 1) % kStages;
                if (!mbar_wait_warp(&full[s], relayed >> s & 1, &failed)) break;
                relayed ^= 1u << s;
                zero_rows_past_end<Sh>(stages + s * Sh::kStageBytes, t.rows - (kb - 1) * kGemmBK, lane);
                if (lane == 0) mbar_arrive_cluster(cluster_smem_u32(&other[s], 0));
                __syncwarp();
            }
        }
    } else {
        // ---- epilogue: warp w reads lanes [32 (w mod 4), + 32) of the accumulators, one row a thread,
        // and two warps take the same rows' columns in turns of 32
        const int quarter = warp % 4, turn = (warp - 2) / 4;
        unsigned char *slab = slabs + (warp - 2) * kSlabBytes;
        const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
        uint32_t acc_it = 0;
        while (walk.next(t)) {
            const bool none = walk.blocks(t) == 0;
            const uint32_t slot = acc_it & 1;
            // the warp's first row within the tile; its columns of the tile
            const bool half = half_tile<OP, CG>(t);
            const int r0 = half ? (int)rank * (kGemmBM / 2) + quarter % 2 * 32 : (int)rank * kGemmBM + quarter * 32;
            const int c_first = half ? quarter / 2 * (Sh::kOutN / 2) : 0;
            const int N = p.N[t.problem];
            const int c_end = min(half ? c_first + Sh::kOutN / 2 : Sh::kOutN, N - t.n0);
            const int rows = min(t.valid - r0, 32);  // of this warp's 32 that count
            // where the tile's column 0 would be for this warp
            const uint32_t src = tmem + lanes + slot * NB - (half ? quarter / 2 * (NB / 2) : 0);
            const size_t row = Sh::kDW ? (size_t)t.e * p.M[t.problem] + t.m0 + r0 : (size_t)t.m0 + r0;
            int c = c_first + turn * kCols;
            // DGateUp: g and u are asked for a turn ahead, the first before the accumulator is there
            uint4 gq[4], uq[4];
            const auto ask = [&](int c) {
                if (OP != ExpertOp::kDGateUp || rows <= 0 || c >= c_end) return;
                slab_load(gq, lane, p.g + row * N, N, t.n0 + c, rows);
                slab_load(uq, lane, p.u + row * N, N, t.n0 + c, rows);
            };
            ask(c);
            if (!none) {
                bool ok = true;
                if (lane == 0) ok = mbar_wait_limited(&acc_full[slot], (acc_it / 2) & 1, &failed);
                if (!__shfl_sync(0xFFFFFFFFu, ok, 0)) break;
                ++acc_it;
                tmem_fence_after();
            }
            for (; rows > 0 && c < c_end; c += 2 * kCols) {
                const int n = t.n0 + c;
                uint32_t v[32], o[16];
                if constexpr (OP == ExpertOp::kDGateUp) {
                    uint32_t g[16], u[16];
                    slab_fill(slab, lane, gq);
                    slab_get(slab, lane, g);
                    __syncwarp();
                    slab_fill(slab, lane, uq);
                    slab_get(slab, lane, u);
                    __syncwarp();
                    ask(c + 2 * kCols);
                    tmem_load_32(src + c, v);
                    tmem_wait_ld(v);
                    if (p.saved_bf16)
                        gate_gradients<true>(v, g, u, o);
                    else
                        gate_gradients<false>(v, g, u, o);
                    slab_put(slab, lane, o);
                    slab_store(slab, lane, p.out[0] + row * N, N, n, rows);
                    slab_put(slab, lane, u);
                    slab_store(slab, lane, p.out[1] + row * N, N, n, rows);
                } else if constexpr (OP == ExpertOp::kGateUp) {
                    uint32_t w[32];
                    const uint32_t at = src + c / Sh::kGate * (2 * Sh::kGate) + c % Sh::kGate;
                    tmem_load_32(at, v);
                    tmem_load_32(at + Sh::kGate, w);
                    tmem_wait_ld(v);
                    tmem_wait_ld(w);
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float g0 = __uint_as_float(v[2 * i]), g1 = __uint_as_float(v[2 * i + 1]);
                        o[i] = bf16_pair(g0 * sigmoid(g0) * __uint_as_float(w[2 * i]),
                                         g1 * sigmoid(g1) * __uint_as_float(w[2 * i + 1]));
                    }
                    slab_put(slab, lane, o);
                    slab_store(slab, lane, p.out[0] + row * N, N, n, rows);
                    if (p.g) {
                        saved_pairs(v, o, p.saved_bf16);
                        slab_put(slab, lane, o);
                        slab_store(slab, lane, p.g + row * N, N, n, rows);
                        saved_pairs(w, o, p.saved_bf16);
                        slab_put(slab, lane, o);
                        slab_store(slab, lane, p.u + row * N, N, n, rows);
                    }
                } else {
                    if (!none) {
                        tmem_load_32(src + c, v);
                        tmem_wait_ld(v);
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i)
                        o[i] = none ? 0u : bf16_pair(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]));
                    slab_put(slab, lane, o);
                    slab_store(slab, lane, p.out[t.problem] + row * N, N, n, rows);
                }
            }
            if (!none) {
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
    }

    __syncthreads();
    if constexpr (CG == 2) {
        // a CTA that gave up tells the other one, whose memory its copies and MMAs may use
        if (threadIdx.x == 0 && failed) st_cluster(cluster_smem_u32(const_cast<int *>(&failed), rank ^ 1), 1);
        cluster_sync();  // no arrival may reach a CTA that has ended
    }
    // After a failure nobody has waited for what is under way, and it may have come after its warp had
    // finished: from here on no role adds to it or sets `failed`. Nothing may be left when a CTA ends.
    if (failed) {
        if (produces) {
            const uint32_t mine = warp == 0 ? 0 : warp - 1 - kEpilogueWarps;
            int gave_up = 0;
            if (rank == 0) {
                wait_for_fills(full, it, mine, kProducers, kStages);
            } else {
                for (int i = mine; kRelay && i < kStages; i += kProducers)
                    if (ever >> i & 1) mbar_wait_limited(&full[i], (relayed >> i & 1) ^ 1, &gave_up);
                // copies for which the first CTA's barrier was not armed any more
                for (int i = 0; i < 100; ++i) __nanosleep(10000);
            }
        } else if (warp == 1 && rank == 0) {  // MMAs read the stages and write TMEM
            if (elect_one()) mma_commit<CG>(&drained);
            __syncwarp();
            int gave_up = 0;
            mbar_wait_limited(&drained, 0, &gave_up);
        }
        __syncthreads();
        if constexpr (CG == 2) cluster_sync();
        if (threadIdx.x == 0) atomicOr(p.error, kErrExpertWait);
    }
    if (warp == 1) tmem_free<CG>(tmem, Sh::kTmemCols);
}

}  // namespace ep
