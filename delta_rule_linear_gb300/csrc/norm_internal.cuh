// norm_internal.cuh -- declarations of the gated norm and the residual norm.
#pragma once

#include "kda_internal.cuh"
#include "launch_after.cuh"

namespace kda {

constexpr int kGatedNormMax = 1024;      // widest head row (a warp holds it)
constexpr int kResidualNormMax = 16384;  // widest token row (a CTA holds it)

struct NormView {
    void *p;
    long long t, h;   // element strides of the token and the head; D is contiguous
};

struct GatedNorm {
    NormView x, g, y;        // forward; act == 0: no gate (g.p == nullptr)
    NormView dy, dx, dg;     // backward
    const float *w;          // [D]
    float *dw, *part;        // [D]; [norm_parts, D] scratch
    long rows;               // tokens * heads
    int H, D, act;           // act: 0 none, 1 silu, 2 sigmoid
    int flat;                // every array is contiguous (set by the launcher)
    float eps, inv_d;
    DType dtype;
    int sms;
};

struct ResidualNorm {
    const void *x, *y;       // forward: residual stream, block output; backward: x' and y (or nullptr)
    const void *dn, *dxo;    // backward: gradients of n and x' (dxo may be nullptr: zeros)
    long long xs, ys, dns, dxs;   // row strides
    void *xo, *n;            // forward: x', n; backward: dx, dy (contiguous rows)
    const float *w, *cv;     // [D]; cv: per-channel scale or nullptr (the scalar c)
    float *dw, *dc, *part;   // [D], [D]; [norm_parts, D or 2 D] scratch
    long rows;
    int D;
    float c, eps, inv_d;
    DType res, dtype;        // x, x', dx; y, n, dy
    int sms;
};

// CTAs of a backward at most (each leaves one partial row of dw).
inline int norm_parts(int sms) { return 8 * sms; }

cudaError_t launch_gated_norm(const GatedNorm &a, bool bwd, cudaStream_t st);
cudaError_t launch_residual_norm(const ResidualNorm &a, bool bwd, cudaStream_t st);

}  // namespace kda
