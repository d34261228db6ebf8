// ssm_scan.cu -- the state space scan: prompts (equal lengths or packed) and single tokens.
//
//     dt_t = softplus(dt_t + bias),   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t . h_t + skip x_t) silu(gate_t)
//
// L = N / 4 lanes hold a channel, four states each (lane l: l, l + L, l + 2 L, l + 3 L), and walk a sequence.
#include <algorithm>

#include "ssm_internal.cuh"
#include "ssm_math.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

template <typename T> __device__ __forceinline__ float at(const SsmView &v, long b, long t, long e) {
    return to_f32(static_cast<const T *>(v.p)[b * v.b + t * v.t + e]);
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) ssm_walk_kernel(Ssm a, int cpg, int bpg) {
    const int CH = kThreads / L, N = 4 * L;
    const int g = blockIdx.x / bpg, cg = (blockIdx.x - g * bpg) * CH + threadIdx.x / L, l = threadIdx.x % L;
    const bool live = cg < cpg;
    const int d = g * cpg + (live ? cg : 0), n = blockIdx.y;
    long start = 0, len = a.s.T, b = n;
    if (a.s.cu) {
        start = min(max((long)a.s.cu[n], 0L), a.total);
        len = min(max((long)a.s.cu[n + 1] - a.s.cu[n], 0L), a.total - start);
        b = 0;
    }
    float A[4], h[4];
    for (int i = 0; i < 4; ++i) {
        A[i] = a.A[(long)d * N + l + L * i] * kLog2eF;
        h[i] = a.h0 ? a.h0[((long)n * a.D + d) * N + l + L * i] : 0.f;
    }
    const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
    for (long t = start; t < start + len; ++t) {
        float dt = at<T>(a.dt, b, t, d) + bias;
        if (a.softplus) dt = softplus<T>(dt);
        const float x = at<T>(a.x, b, t, d), u = dt * x;
        float y = 0.f;
        for (int i = 0; i < 4; ++i) {
            const int e = l + L * i;
            h[i] = fmaf(ex2(dt * A[i]), h[i], u * at<T>(a.B, b, t, g * a.B.g + e));
            y = fmaf(h[i], at<T>(a.C, b, t, g * a.C.g + e), y);
        }
        for (int off = L / 2; off; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        y = fmaf(skip, x, y);
        if (a.gate.p) {
            float z = at<T>(a.gate, b, t, d), rest;
            y *= z * sigmoid<T>(z, rest);
        }
        if (live && l == 0) static_cast<T *>(a.y.p)[b * a.y.b + t * a.y.t + d] = from_f32<T>(y);
    }
    if (a.hT && live)
        for (int i = 0; i < 4; ++i) a.hT[((long)n * a.D + d) * N + l + L * i] = h[i];
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(SsmStep a) {
    const int CH = kThreads / L, N = 4 * L;
    const int d0 = blockIdx.x * CH + threadIdx.x / L, l = threadIdx.x % L, n = blockIdx.y;
    const bool live = d0 < a.D;
    const int d = live ? d0 : 0, g = d / (a.D / a.G);
    auto val = [](const void *p, long i) { return to_f32(static_cast<const T *>(p)[i]); };
    float dt = val(a.dt, n * a.dtb + d) + (a.bias ? a.bias[d] : 0.f);
    if (a.softplus) dt = softplus<T>(dt);
    const float x = val(a.x, n * a.xb + d), u = dt * x;
    float *sp = a.state + ((long)n * a.D + d) * N + 4 * l;
    const float4 s = *reinterpret_cast<const float4 *>(sp);
    const float4 A = *reinterpret_cast<const float4 *>(a.A + (long)d * N + 4 * l);
    float h[4] = {s.x, s.y, s.z, s.w}, y = 0.f;
    const float Av[4] = {A.x, A.y, A.z, A.w};
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(ex2(dt * (Av[i] * kLog2eF)), h[i], u * val(a.B, n * a.Bb + g * a.Bg + 4 * l + i));
        y = fmaf(h[i], val(a.C, n * a.Cb + g * a.Cg + 4 * l + i), y);
    }
    for (int off = L / 2; off; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    if (!live) return;
    *reinterpret_cast<float4 *>(sp) = make_float4(h[0], h[1], h[2], h[3]);
    y = fmaf(a.skip ? a.skip[d] : 0.f, x, y);
    if (a.gate) {
        float z = val(a.gate, n * a.gb + d), rest;
        y *= z * sigmoid<T>(z, rest);
    }
    if (l == 0) static_cast<T *>(a.y)[n * a.yb + d] = from_f32<T>(y);
}

template <typename T, int L> cudaError_t run(const Ssm &a, cudaStream_t st) {
    const int cpg = a.D / a.G, CH = kThreads / L, bpg = (cpg + CH - 1) / CH;
    ssm_walk_kernel<T, L><<<dim3(bpg * a.G, a.s.nseq), kThreads, 0, st>>>(a, cpg, bpg);
    return cudaGetLastError();
}
template <typename T, int L> cudaError_t run_step(const SsmStep &a, cudaStream_t st) {
    ssm_step_kernel<T, L><<<dim3((a.D * L + kThreads - 1) / kThreads, a.nb), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T> cudaError_t go(const Ssm &a, cudaStream_t st) {
    return a.N == 8 ? run<T, 2>(a, st) : a.N == 16 ? run<T, 4>(a, st) : a.N == 32 ? run<T, 8>(a, st) : run<T, 16>(a, st);
}
template <typename T> cudaError_t go_step(const SsmStep &a, cudaStream_t st) {
    return a.N == 8 ? run_step<T, 2>(a, st) : a.N == 16 ? run_step<T, 4>(a, st) : a.N == 32 ? run_step<T, 8>(a, st) : run_step<T, 16>(a, st);
}

}  // namespace

size_t ssm_scratch_bytes(int, long, int, bool, int, int, int, int) { return 0; }
cudaError_t launch_ssm(const Ssm &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? go<__nv_bfloat16>(a, st) : go<float>(a, st);
}
cudaError_t launch_ssm_step(const SsmStep &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? go_step<__nv_bfloat16>(a, st) : go_step<float>(a, st);
}

}  // namespace kda
