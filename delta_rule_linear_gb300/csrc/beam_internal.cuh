// beam_internal.cuh -- declarations of beam search's selection and of the reordering of states.
#pragma once

#include "kda_internal.cuh"
#include "launch_after.cuh"

namespace kda {

constexpr int kBeamMax = 32;        // beams kept (k) and beams reordered at most
constexpr int kBeamsIn = 128;       // beams selected from at most
constexpr int kBeamChunk = 512;     // logits of a chunk
constexpr int kBeamTake = 1024;     // logits that a warp takes at a time: two chunks
constexpr int kBeamStates = 32;     // arrays of a reordering launch

// Part of a row: its largest logit and the sum of exp(x - max).
struct BeamSum {
    double sum;
    float max;
};

struct BeamSelect {
    const void *logits;             // rows of V, strides sb (request) and sw (beam) in elements
    long long sb, sw;
    const float *scores;            // [B, W]
    const unsigned char *finished;  // [B, W] or nullptr
    float *out;                     // [B, k]
    int *parents, *tokens;          // [B, k]
    int B, W, V, k, eos;
    DType dtype;
    // scratch: each row's sums in `splits` parts, and the chunks' maxima [B W, nc]
    BeamSum *sums;
    float *cmax;
    int nc, splits;
    int sms;
};
inline int beam_takes(int V) { return (int)(((long)V + kBeamTake - 1) / kBeamTake); }
inline int beam_chunks(int V) { return beam_takes(V) * (kBeamTake / kBeamChunk); }      // (the last may be empty)
int beam_splits(long rows, int takes, int sms);
cudaError_t launch_beam_select(const BeamSelect &a, cudaStream_t st);

struct BeamReorder {
    char *p[kBeamStates];           // arrays [B, W, row bytes]
    long long bytes[kBeamStates];   // bytes of a row
    int unit[kBeamStates];          // bytes moved at a time (a power of two that divides row and address)
    unsigned first[kBeamStates + 1];// first CTA of the array (per request)
    int count;
    const int *parents;             // [B, W]
    int B, W;
};
cudaError_t launch_beam_reorder(BeamReorder &a, cudaStream_t st);

}  // namespace kda
