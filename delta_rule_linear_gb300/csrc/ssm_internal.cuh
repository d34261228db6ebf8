// ssm_internal.cuh -- declarations of the state space scan.
//
//   dt_t = softplus(dt_t + bias) (or dt_t + bias),  h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,
//   y_t  = (C_t . h_t + skip x_t) silu(gate_t)      per (sequence, channel), h_t a vector of N states.
#pragma once

#include "linear_internal.cuh"

namespace kda {

// Channel rows [B, T, D] (g unused) or [B, T, G, N]: element strides, the last dimension contiguous.
struct SsmView {
    void *p;
    long long b, t, g;
};

struct Ssm {
    SsmView x, dt, gate, y;      // gate.p may be nullptr; backward: y holds d_y
    SsmView B, C;
    const float *A;              // [D, N]
    const float *skip, *bias;    // [D] or nullptr
    const float *h0;             // [nseq, D, N] or nullptr
    float *hT;                   // the same or nullptr
    LinSeqs s;
    long total;                  // token rows of a packed batch (equal length: T)
    int max_len;                 // bound on the longest sequence
    int D, G, N, softplus;
    DType dtype;
    void *ws;
    int sms;
    // backward
    SsmView dx, ddt, dgate, dB, dC;
    float *dA, *dskip, *dbias, *dh0;   // [D, N], [D], [D], [nseq, D, N]; all but dA may be nullptr
    const float *dhT;                  // [nseq, D, N] or nullptr
};

size_t ssm_scratch_bytes(int nseq, long total, int max_len, bool varlen, int D, int G, int N, int sms);
cudaError_t launch_ssm(const Ssm &a, cudaStream_t st);
size_t ssm_bwd_scratch_bytes(int nseq, long total, int max_len, bool varlen, int D, int G, int N, int sms);
cudaError_t launch_ssm_bwd(const Ssm &a, cudaStream_t st);

struct SsmStep {
    const void *x, *dt, *gate, *B, *C;
    void *y;
    long long xb, dtb, gb, Bb, Bg, Cb, Cg, yb;   // element strides of the request (and group)
    const float *A, *skip, *bias;
    float *state;                // [B, D, N], in place
    int nb, D, G, N, softplus;
    DType dtype;
    int sms;
};
cudaError_t launch_ssm_step(const SsmStep &a, cudaStream_t st);

}  // namespace kda
