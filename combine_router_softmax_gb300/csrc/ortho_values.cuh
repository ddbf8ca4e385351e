// ortho_values.cuh -- how the matrices to be orthogonalised come in: scaled by 1 / (norm + eps), as two halves.
#pragma once

#include "ortho_gemm.cuh"
#include "values.cuh"

namespace ep {

// 1 / (norm + eps) as three factors, so that no product on the way leaves fp32's range.
struct OrthoScale {
    float f, p1, p2;
    __device__ float operator()(float v) const { return v * p1 * p2 * f; }
};
__device__ __forceinline__ OrthoScale ortho_scale(double squares, float eps) {
    OrthoScale s;
    if (squares >= 0x1p-100 && squares <= 0x1p100) {  // the usual case, without the few 64-bit units' square root
        s.f = 1.0f / (sqrtf((float)squares) + eps);
        s.p1 = s.p2 = 1.0f;
        return s;
    }
    const double by = sqrt(squares) + (double)eps;
    if (by > 0 && by < 1e300) {
        int e;
        const double f = frexp(by, &e);
        s.f = (float)(1.0 / f);
        s.p1 = ldexpf(1.0f, -e / 2);
        s.p2 = ldexpf(1.0f, -(e - e / 2));
    } else {  // 0 / 0, or not finite
        s.f = (float)(1.0 / by);
        s.p1 = s.p2 = 1.0f;
    }
    return s;
}

// Two values of X as they are held.
__device__ __forceinline__ void split_pair(float x0, float x1, uint32_t &hi, uint32_t &lo) {
    x0 *= kX, x1 *= kX;
    hi = half_pair(x0, x1);
    const float2 r = saved_values<false>(hi);
    lo = half_pair(x0 - r.x, x1 - r.y);
}

// Whether the bounds of X, A and B over the steps, from |singular values| <= 1 on, fit the halves; and, where `form` is given,
// what each step of matrices with so many rows does with X's lower half.
bool ortho_steps(const float *k, int32_t steps, int32_t rows, OrthoForm *form);

// Matrices that one cluster takes through all steps (ortho_fused.cu).
bool ortho_fits_fused(const ep_ortho_config &c);
// And that one does on every device: the others need the products' workspace, in case this device has no place for it.
bool ortho_fits_any_device(const ep_ortho_config &c);
// *ran: false, with cudaSuccess, where it has none.
cudaError_t launch_ortho_fused(const ep_ortho_config &c, const float *k, const void *m, ep_bf16 *out, bool *ran, cudaStream_t s);

}  // namespace ep
