// conv_internal.cuh -- declarations of the short causal convolution.
#pragma once

#include "linear_internal.cuh"

namespace kda {

// Channel rows [B, T, C]: element strides, channels contiguous.
struct ConvView {
    void *p;
    long long b, t;
};

struct Conv {
    ConvView x, y;           // backward: x and d_y
    ConvView dx;             // backward
    const float *w, *bias;   // [C, K]; [C] or nullptr
    const void *h0, *dhT;    // windows [nseq, K - 1, C] of x's type or nullptr
    void *hT, *dh0;          // the same or nullptr
    float *dw, *dbias;       // backward: [C, K], [C] or nullptr
    float *part;             // backward: [conv_parts, K + 1, C] scratch
    LinSeqs s;
    long total;              // token rows of a packed batch (equal length: T)
    int C, K, act;           // act: 0 none, 1 silu
    int blocks;              // blocks of channels (set by the launcher, as the next two)
    int run;                 // tokens a warp takes in a row
    long items;              // runs of the launch (a bound for packed sequences)
    DType dtype;
    int sms;
};

// Partial sums of the weights' gradients at most (rows of `part`): four CTAs per SM, of up to 128 channels.
inline int conv_parts(int C, int sms) {
    const int blocks = C / 128 + (C % 128 != 0);
    return 4 * sms > blocks ? 4 * sms / blocks : 1;
}

cudaError_t launch_conv(const Conv &a, cudaStream_t st);
cudaError_t launch_conv_bwd(const Conv &a, cudaStream_t st);

struct ConvStep {
    const void *x;
    void *y, *state;         // [B, C] (strides xb, yb), [B, K - 1, C] in place
    const float *w, *bias;
    long long xb, yb;
    int B, C, K, act;
    DType dtype;
    int sms;
};
cudaError_t launch_conv_step(const ConvStep &a, cudaStream_t st);

}  // namespace kda
