// norm_rows.cuh -- the norms around a block: a group of threads, a warp or a CTA, walks rows and holds each in
// registers, so that it is read once and written once, with its mean squares as sums over the group.
//
// HBM bounds these kernels, if the instructions they issue do not: so two values go to an instruction where
// there is one (f32x2), and what a call has (y, a norm of y, a gate with a value for every column) is a
// compile-time form. The rest is decided by branches that a whole CTA takes alike.
#pragma once

#include "pairs.cuh"
#include "tcgen05.cuh"  // SharedMemoryLimit

namespace ep {

constexpr int kNormWarps = 8;          // rows of a CTA where a row is one warp's
// CTAs of the backward pass, at most, each of which leaves a row of partial sums: two for every SM, or more of
// short rows, which then still are a small part of what the pass moves; and three rows for each, once every SM has one, as
// otherwise the partial sums are most of it (777 rows of 1000, backward, 11.6 -> 9.9 us, 1500 of 512 12.7 -> 10.0).
inline int norm_partials(const ep_norm_config &c) {
    const int64_t most = 304 * (int64_t)(c.H >= 4096 ? 1 : c.H >= 2048 ? 2 : 4), few = c.T / 3 > 152 ? c.T / 3 : 152;
    const int64_t n = few < most ? few : most;
    return (int)(c.T < n ? c.T : n);
}

struct NormArgs {
    const void *x;
    const uint4 *y, *w_post, *w_next;
    const void *gate;
    void *out;
    uint4 *n;
    float *rstd_post, *rstd_next;  // forward: written where given; backward: read
    const void *d_out;
    const uint4 *d_n;
    void *d_x, *d_gate;
    uint4 *d_y;
    float *partial;  // [CTA][sums][H]
    int32_t T, vecs, kind, sigmoid;
    int32_t next_at, y_at;  // where a row of partial sums holds them, in H; -1: not wanted
    float eps, scale, offset, inv_h;
};

// What a call has, as far as kernels are made for it.
constexpr int kFormY = 1, kFormPost = 2, kFormGate = 4;  // Gate: of channels or elements

// In norm_forward.cu and norm_backward.cu; *ctas: the CTAs that were launched.
cudaError_t launch_norm_forward(const NormArgs &p, bool f32, cudaStream_t s);
cudaError_t launch_norm_backward(const NormArgs &p, bool f32, int most, int *ctas, cudaStream_t s);

// Eight fp32 values as four pairs: the arithmetic below takes two at a time (f32x2 instructions), as the
// instructions issued are what bounds these kernels beside HBM.
struct V8 {
    uint64_t p[4];
};
__device__ __forceinline__ V8 unpack8(const uint4 &q) {
    const uint32_t u[4] = {q.x, q.y, q.z, q.w};
    V8 v;
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = (uint64_t)(u[i] & 0xFFFF0000u) << 32 | (uint64_t)(u[i] << 16);
    return v;
}
__device__ __forceinline__ uint4 pack8(const V8 &v) {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(u[i]) : "f"(high(v.p[i])), "f"(low(v.p[i])));
    return make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void times(V8 &v, const V8 &f) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = mul2(v.p[i], f.p[i]);
}
__device__ __forceinline__ void times(V8 &v, float f) {
    const uint64_t ff = pair(f, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = mul2(v.p[i], ff);
}
// sum += a b
__device__ __forceinline__ void dot(uint64_t &sum, const V8 &a, const V8 &b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) sum = fma2(a.p[i], b.p[i], sum);
}
// v = f a + v
__device__ __forceinline__ void add_scaled(V8 &v, float f, const V8 &a) {
    const uint64_t ff = pair(f, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = fma2(ff, a.p[i], v.p[i]);
}
// v += a b
__device__ __forceinline__ void add_product(V8 &v, const V8 &a, const V8 &b) {
#pragma unroll
    for (int i = 0; i < 4; ++i) v.p[i] = fma2(a.p[i], b.p[i], v.p[i]);
}

// Eight values of the residual stream, bf16 or float: `at` counts in eights.
template <bool F32>
struct Stream8 {
    uint4 q[F32 ? 2 : 1];
    __device__ __forceinline__ void load(const void *p, size_t at) {
        const uint4 *s = static_cast<const uint4 *>(p) + at * (F32 ? 2 : 1);
        q[0] = *s;
        if constexpr (F32) q[1] = s[1];
    }
    __device__ __forceinline__ void clear() {
        q[0] = make_uint4(0, 0, 0, 0);
        if constexpr (F32) q[1] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ V8 get() const {
        if constexpr (F32) {
            V8 v;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                v.p[2 * i] = (uint64_t)q[i].y << 32 | q[i].x;
                v.p[2 * i + 1] = (uint64_t)q[i].w << 32 | q[i].z;
            }
            return v;
        } else {
            return unpack8(q[0]);
        }
    }
    __device__ __forceinline__ static void store(void *p, size_t at, const V8 &v) {
        uint4 *d = static_cast<uint4 *>(p) + at * (F32 ? 2 : 1);
        if constexpr (F32) {
            // 32 bytes by one instruction where they lie so: two of 16 each write half of every sector (4096 rows of 4096,
            // normed and joined, 44 -> 41 us, backward 78 -> 75)
            if (reinterpret_cast<uintptr_t>(p) % 32 == 0) {
                asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(d), "l"(v.p[0]), "l"(v.p[1]), "l"(v.p[2]), "l"(v.p[3]) : "memory");
                return;
            }
#pragma unroll
            for (int i = 0; i < 2; ++i)
                st_v4(d + i, make_uint4((uint32_t)v.p[2 * i], (uint32_t)(v.p[2 * i] >> 32), (uint32_t)v.p[2 * i + 1],
                                        (uint32_t)(v.p[2 * i + 1] >> 32)));
        } else {
            st_v4(d, pack8(v));
        }
    }
};

// The gate's factor, in place, and its derivative. With q = exp(-|g|) neither cancels at either end.
__device__ __forceinline__ float gate_act(float g, bool sigmoid, float &slope) {
    slope = 1.0f;
    if (!sigmoid) return g;
    const float q = __expf(-fabsf(g)), a = __fdividef(1.0f, 1.0f + q);
    slope = q * a * a;
    return g >= 0.0f ? a : q * a;
}
__device__ __forceinline__ void gate_act(V8 &g, bool sigmoid, V8 &slope) {
    if (sigmoid) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float s0, s1;
            const float a0 = gate_act(low(g.p[i]), true, s0), a1 = gate_act(high(g.p[i]), true, s1);
            g.p[i] = pair(a0, a1);
            slope.p[i] = pair(s0, s1);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i) slope.p[i] = pair(1.0f, 1.0f);
    }
}
__device__ __forceinline__ void gate_act(V8 &g, bool sigmoid) {
    V8 slope;
    gate_act(g, sigmoid, slope);
}
// v times the norm's weights
__device__ __forceinline__ void weigh(V8 &v, const uint4 &weights, float offset) {
    V8 w = unpack8(weights);
    if (offset != 0.0f) {
        const uint64_t o = pair(offset, offset);
#pragma unroll
        for (int i = 0; i < 4; ++i) w.p[i] = add2(w.p[i], o);
    }
    times(v, w);
}

// The sums of N values over the group, in every thread of it: over the lanes, then each thread adds the
// warps' sums up for itself, four to a load (a second round of shuffles takes four times the instructions,
// which are what bounds these kernels). `scratch`: not that of the sum before this one, which slower warps may
// still read.
struct Scratch {
    float4 part[2][2][8];  // [turn][value][warp / 4]
};
template <bool WARP, int N>
__device__ __forceinline__ void group_sum(float (&v)[N], Scratch &scratch, int &turn) {
#pragma unroll
    for (int d = 16; d > 0; d /= 2)
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] += __shfl_xor_sync(0xFFFFFFFFu, v[k], d);
    if constexpr (!WARP) {
        const int warps = blockDim.x / 32;
        if (threadIdx.x % 32 == 0)
#pragma unroll
            for (int k = 0; k < N; ++k) reinterpret_cast<float *>(scratch.part[turn][k])[threadIdx.x / 32] = v[k];
        __syncthreads();
#pragma unroll
        for (int k = 0; k < N; ++k) v[k] = 0.0f;
        for (int i = 0; 4 * i < warps; ++i)
#pragma unroll
            for (int k = 0; k < N; ++k) {
                const float4 q = scratch.part[turn][k][i];
                v[k] += (q.x + q.y) + (q.z + q.w);
            }
        turn ^= 1;
    }
}
// Before the first sum: the places of warps that there are not. One barrier before they are read is that sum's own.
template <bool WARP>
__device__ __forceinline__ void clear_scratch(Scratch &scratch) {
    if (!WARP)
        for (int i = threadIdx.x; i < 128; i += blockDim.x)
            if (i % 32 >= (int)blockDim.x / 32) reinterpret_cast<float *>(scratch.part)[i] = 0.0f;
}
template <bool WARP>
__device__ __forceinline__ float group_sum(float v, Scratch &scratch, int &turn) {
    float one[1] = {v};
    group_sum<WARP, 1>(one, scratch, turn);
    return one[0];
}

// The thread's place: which row its group takes first, the step to the next, and its vectors
// i * stride + first of a row.
template <bool WARP>
struct Place {
    int first, stride, row, step;
    __device__ Place() {
        first = WARP ? threadIdx.x % 32 : threadIdx.x;
        stride = WARP ? 32 : blockDim.x;
        row = WARP ? blockIdx.x * (blockDim.x / 32) + threadIdx.x / 32 : blockIdx.x;
        step = WARP ? gridDim.x * (blockDim.x / 32) : gridDim.x;
    }
};

// What a group has in flight of its next rows: 16-byte pieces that a thread copies for itself into shared
// memory, a row or two ahead, and reads from there when their row's turn comes. Nobody else touches them, so
// no barrier goes with them. Piece i of array a in stage s lies at ((s arrays + a) NV + i) threads + thread:
// neighbours in a warp are neighbours in memory.
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
// Until at most `n` of the last groups are under way, n < 2.
__device__ __forceinline__ void copies_wait(int n) {
    if (n == 1)
        asm volatile("cp.async.wait_group 1;" ::: "memory");
    else
        asm volatile("cp.async.wait_group 0;" ::: "memory");
}

template <bool F32, int NV>
struct Ring {
    static constexpr int kStream = F32 ? 2 : 1;  // arrays of the residual stream: a second one for the upper halves of 8 floats
    uint32_t base, array_bytes, piece_bytes, stage_bytes;
    uint32_t gate, d_out, d_n;  // offsets within a stage; x is first, y next
    uint32_t factors;           // behind the stages: this thread's column factors, floats
    uint32_t y_ahead;           // y's places where it is a row further ahead: stages + 1 of them, between the two
    __device__ Ring(const void *smem, int stages, bool y, bool element, bool d, bool n, bool ahead = false) {
        piece_bytes = blockDim.x * 16;
        array_bytes = piece_bytes * NV;
        base = smem_u32(smem) + threadIdx.x * 16;
        uint32_t at = array_bytes * kStream + (y && !ahead ? array_bytes : 0);
        gate = at, at += element ? array_bytes : 0;
        d_out = at, at += d ? array_bytes * kStream : 0;
        d_n = at, at += n ? array_bytes : 0;
        stage_bytes = at;
        y_ahead = base + stages * at;
        factors = y_ahead + (ahead ? (stages + 1) * array_bytes : 0);
    }
    // What of z = f y r(y) is the same for all rows, a value a column: the norm's weights and a channel gate's
    // factor. KEPT: as floats, as they would be unpacked, offset and put through the sigmoid for every row.
    template <bool POST, bool GATE>
    static __device__ __forceinline__ V8 column_factors(const NormArgs &p, int v) {
        V8 f;
#pragma unroll
        for (int j = 0; j < 4; ++j) f.p[j] = pair(1.0f, 1.0f);
        if (POST) weigh(f, __ldg(p.w_post + v), p.offset);
        if (GATE && p.kind == EP_GATE_CHANNEL) {
            V8 a = unpack8(__ldg(static_cast<const uint4 *>(p.gate) + v));
            gate_act(a, p.sigmoid);
            times(f, a);
        }
        return f;
    }
    template <bool POST, bool GATE>
    __device__ __forceinline__ void keep_factors(const NormArgs &p, int first, int stride) const {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int v = i * stride + first;
            if (v >= p.vecs) continue;
            const V8 f = column_factors<POST, GATE>(p, v);
#pragma unroll
            for (int h = 0; h < 2; ++h)
                asm volatile("st.shared.v2.u64 [%0], {%1, %2};" ::"r"(factors + (2 * i + h) * piece_bytes), "l"(f.p[2 * h]), "l"(f.p[2 * h + 1]) : "memory");
        }
    }
    template <bool KEPT, bool POST, bool GATE>
    __device__ __forceinline__ V8 get_factors(const NormArgs &p, int i, int v) const {
        if constexpr (!KEPT) return column_factors<POST, GATE>(p, v);
        V8 f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
            asm volatile("ld.shared.v2.u64 {%0, %1}, [%2];" : "=l"(f.p[2 * h]), "=l"(f.p[2 * h + 1]) : "r"(factors + (2 * i + h) * piece_bytes));
        return f;
    }
    __host__ static int arrays(bool y, bool element, bool d, bool n) { return kStream + y + element + (d ? kStream : 0) + n; }
    static __device__ __forceinline__ void copy16(uint32_t to, const void *from) {
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
    }
    static __device__ __forceinline__ uint4 get16(uint32_t at) {
        uint4 q;
        asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(q.x), "=r"(q.y), "=r"(q.z), "=r"(q.w) : "r"(at));
        return q;
    }
    __device__ __forceinline__ uint32_t stage(int s) const { return base + s * stage_bytes; }
    __device__ __forceinline__ uint32_t y() const { return array_bytes * kStream; }
    __device__ __forceinline__ uint32_t y_place(int i) const { return y_ahead + i * array_bytes; }
    __device__ __forceinline__ void copy(uint32_t stage, uint32_t array, int i, const void *p, size_t at) const {
        copy16(stage + array + i * piece_bytes, static_cast<const uint4 *>(p) + at);
    }
    __device__ __forceinline__ void copy_stream(uint32_t stage, uint32_t array, int i, const void *p, size_t at) const {
        const uint4 *src = static_cast<const uint4 *>(p) + at * kStream;
        copy16(stage + array + i * piece_bytes, src);
        if constexpr (F32) copy16(stage + array + array_bytes + i * piece_bytes, src + 1);
    }
    __device__ __forceinline__ uint4 get(uint32_t stage, uint32_t array, int i) const { return get16(stage + array + i * piece_bytes); }
    __device__ __forceinline__ V8 get_stream(uint32_t stage, uint32_t array, int i) const {
        Stream8<F32> q;
        q.q[0] = get16(stage + array + i * piece_bytes);
        if constexpr (F32) q.q[1] = get16(stage + array + array_bytes + i * piece_bytes);
        return q.get();
    }
};

// Rows of more than 8192 values leave no room for column factors.
__host__ __device__ constexpr bool kept_factors(int threads) { return threads <= 512; }

// Shared memory that the rows in flight of a CTA may take.
constexpr size_t kRingBytes = 225 * 1024;

// Launches the kernel that LAUNCH::kernel<F32, FORM, WARP, NV, THREADS, AHEAD>() names, for rows of p.vecs vectors, with two rows
// in flight (three took 56 us instead of 50 for 4096 rows of 7168: what shared memory they take is L1's, where
// the weights are read from), one where two do not fit. least: bytes of shared memory that it needs anyway.
template <typename LAUNCH, bool F32, int FORM, bool WARP, int NV, int THREADS, bool AHEAD = false>
cudaError_t run_rows(const NormArgs &p, int arrays, size_t least, int most, int *ctas, cudaStream_t s) {
    const auto kernel = LAUNCH::template kernel<F32, FORM, WARP, NV, THREADS, AHEAD>();
    const int threads = WARP ? THREADS : (p.vecs + 32 * NV - 1) / (32 * NV) * 32;
    const size_t stage = (size_t)arrays * NV * threads * sizeof(uint4);
    const bool kept = kept_factors(THREADS) && (FORM & kFormPost || (FORM & kFormGate && p.kind == EP_GATE_CHANNEL));
    const size_t factors = kept ? (size_t)2 * NV * threads * sizeof(uint4) : 0;
    const size_t extra = factors + (AHEAD ? (size_t)NV * threads * sizeof(uint4) : 0);
    int stages = 2 * stage + extra <= kRingBytes ? 2 : 1;
    // Backward, floats: one row in flight if two of them take more than half an SM's shared memory: it has
    // two CTAs then, or L1 has the rest (4096 rows of 4096 76 -> 74 us, with a gate of elements 95 -> 79, of
    // 7168 130 -> 123; of 2048, which stay with two, 39 and 40; bf16 as often slower as faster).
    if (LAUNCH::template one_row<F32>() && 2 * stage + extra > 110 * 1024) stages = 1;
    const size_t smem = stages * stage + extra > least ? stages * stage + extra : least;
    static SharedMemoryLimit limit;
    const cudaError_t e = limit.allow(kernel, smem);
    if (e != cudaSuccess) return e;
    const int per_sm = max_blocks_per_sm((const void *)kernel, threads, smem), sms = current_device_sm_count();
    if (per_sm <= 0 || sms <= 0) return cudaErrorInvalidConfiguration;
    const int rows = WARP ? (p.T - 1) / kNormWarps + 1 : p.T;
    *ctas = min(min(rows, per_sm * sms), most);
    return launch_dependent(kernel, dim3((unsigned)*ctas), dim3((unsigned)threads), smem, s, p, stages);
}
template <typename LAUNCH, bool F32, int FORM>
cudaError_t run_form(const NormArgs &p, int arrays, bool sums, int most, int *ctas, cudaStream_t s) {
    // WARP: the CTA's sums over its rows come into shared memory at the end
    if (p.vecs <= 32)
        return run_rows<LAUNCH, F32, FORM, true, 1, 32 * kNormWarps>(p, arrays, sums ? (size_t)p.vecs * 64 : 0, most, ctas, s);
    if (p.vecs <= 256) return run_rows<LAUNCH, F32, FORM, false, 1, 256>(p, arrays, 0, most, ctas, s);
    // AHEAD from four rows a CTA on, as its first row takes one more barrier (bf16, 7168 wide with a channel gate: 600 rows 9.9
    // -> 10.6 us, 1216 16.6 -> 16.7, 4096 45.5 -> 44.0; float 83.4 -> 73.5, with a gate of elements 99 -> 79). What more of y it
    // holds takes bf16 rows beside a gate of elements from L1 (7168 wide 48.4 -> 54.5), and more than 8192 columns (16384 51 -> 56).
    if constexpr (LAUNCH::kAhead && FORM & kFormPost) {
        if (p.T >= 8 * current_device_sm_count() && (F32 || p.kind != EP_GATE_ELEMENT || p.vecs <= 512)) {
            if (p.vecs <= 512) return run_rows<LAUNCH, F32, FORM, false, 2, 256, true>(p, arrays, 0, most, ctas, s);
            if (p.vecs <= 1024) return run_rows<LAUNCH, F32, FORM, false, 2, 512, true>(p, arrays, 0, most, ctas, s);
            if constexpr (F32) return run_rows<LAUNCH, F32, FORM, false, 2, 1024, true>(p, arrays, 0, most, ctas, s);
        }
    }
    if (p.vecs <= 512) return run_rows<LAUNCH, F32, FORM, false, 2, 256>(p, arrays, 0, most, ctas, s);
    // Backward: by their registers two CTAs of 320 threads fit an SM, by their shared memory with up to four arrays or with one
    // stage (4096 rows of 5120, normed, bf16 82 -> 69 us; with five arrays, where one fits, 77 -> 115; as 384 threads 6144
    // wide 76 -> 112).
    if constexpr (!LAUNCH::kAhead)
        if (p.vecs <= 640 && (F32 || arrays <= 4)) return run_rows<LAUNCH, F32, FORM, false, 2, 320>(p, arrays, 0, most, ctas, s);
    if (p.vecs <= 1024) return run_rows<LAUNCH, F32, FORM, false, 2, 512>(p, arrays, 0, most, ctas, s);
    return run_rows<LAUNCH, F32, FORM, false, 2, 1024>(p, arrays, 0, most, ctas, s);
}
template <typename LAUNCH, bool F32>
cudaError_t run_any(const NormArgs &p, bool d, bool n, bool sums, int most, int *ctas, cudaStream_t s) {
    const bool element = p.kind == EP_GATE_ELEMENT, gate = element || p.kind == EP_GATE_CHANNEL;
    const int arrays = Ring<F32, 1>::arrays(p.y != nullptr, element, d, n);
    if (!p.y) return run_form<LAUNCH, F32, 0>(p, arrays, sums, most, ctas, s);
    if (p.w_post) {
        if (gate) return run_form<LAUNCH, F32, kFormY | kFormPost | kFormGate>(p, arrays, sums, most, ctas, s);
        return run_form<LAUNCH, F32, kFormY | kFormPost>(p, arrays, sums, most, ctas, s);
    }
    if (gate) return run_form<LAUNCH, F32, kFormY | kFormGate>(p, arrays, sums, most, ctas, s);
    return run_form<LAUNCH, F32, kFormY>(p, arrays, sums, most, ctas, s);
}

}  // namespace ep
