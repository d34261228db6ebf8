// linear_internal.cuh -- declarations of the linear-attention (no delta term) kernels.
//
// h_t = exp(decay_t) h_{t-1} + k_t v_t^T,  o_t = scale h_t^T q_t  per (sequence, value head).
#pragma once

#include "kda_internal.cuh"
#include "launch_after.cuh"

namespace kda {

// A token array [B, T, heads, D]: element strides, the last dimension contiguous.
struct LinView {
    const void *p;
    long long b, t, h;
};

// Sequences: equal-length batches (cu == nullptr: sequence n = batch entry n, T tokens) or
// packed (cu [nseq + 1] device prefix array, one batch entry).
struct LinSeqs {
    const int *cu;
    int nseq, T;
};

// The decay of (sequence row, value head): [B, T, HV] (t = HV), [HV] (b = t = 0) or none (p = nullptr).
struct LinDecay {
    const float *p;
    long long b, t;
};

// A sequence's tokens are walked in segments of `L` tokens; work item = one segment of one
// sequence, counted over the sequences in order.  An empty sequence has one (empty) segment.
struct LinItem {
    int n, p, nseg;   // sequence, segment of it, its segments
    int first;        // item of the sequence's segment 0
    long start;       // first token row
    int len;          // tokens of the sequence
};
// Decodes `item` (whole warps call it together); false: past the last item.
__device__ __forceinline__ bool lin_item(const LinSeqs &s, int L, int item, LinItem &it) {
    if (!s.cu) {
        it.nseg = s.T > L ? (s.T + L - 1) / L : 1;
        it.n = item / it.nseg;
        it.p = item - it.n * it.nseg;
        it.first = item - it.p;
        it.start = (long)it.n * s.T;
        it.len = s.T;
        return it.n < s.nseq;
    }
    const int lane = threadIdx.x & 31;
    int base = 0;
    for (int n0 = 0; n0 < s.nseq; n0 += 32) {
        const int n = n0 + lane;
        int segs = 0;
        if (n < s.nseq) {
            const int len = s.cu[n + 1] - s.cu[n];
            segs = len > L ? (len + L - 1) / L : 1;
        }
        int sum = segs;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, sum, off);
            if (lane >= off) sum += up;
        }
        const int all = __shfl_sync(0xffffffffu, sum, 31);
        if (item < base + all) {
            const unsigned hit = __ballot_sync(0xffffffffu, item < base + sum);
            const int src = __ffs(hit) - 1;
            it.n = n0 + src;
            it.nseg = __shfl_sync(0xffffffffu, segs, src);
            it.first = base + __shfl_sync(0xffffffffu, sum, src) - it.nseg;
            it.p = item - it.first;
            it.start = s.cu[it.n];
            it.len = s.cu[it.n + 1] - s.cu[it.n];
            return true;
        }
        base += all;
    }
    return false;
}
// Items of a launch: exact for equal lengths, a bound for packed sequences.
inline long lin_items(int nseq, long total, int max_len, bool varlen, int L) {
    if (!varlen) return (long)nseq * (max_len > L ? (max_len + L - 1) / L : 1);
    return max_len > L ? total / L + nseq : nseq;
}

// One forward problem.
struct LinFwd {
    LinView q, k, v, o;
    LinDecay g;
    LinSeqs s;
    const float *h0;      // [nseq, HV, dk, dv] or nullptr
    float *hT;            // the same or nullptr
    int H, HV, dk, dv;
    DType dtype;
    float scale;
    void *ws;             // segment memories (linear_*_scratch_bytes)
    WsHeader *hdr;
    long total;           // token rows of a packed batch (equal length: T)
    int max_len;          // bound on the longest sequence
    int sms;
};

// Decays below this are exactly 0 as factors (exp(-104) < 2^-150); clamping them to it keeps
// sums and differences of log decays finite, so a decay of -inf is a clean restart.  NaN stays.
constexpr float kMinDecay = -104.f;
__device__ __forceinline__ float clamp_decay(float d) { return d < kMinDecay ? kMinDecay : d; }

// CUDA-core token walk (linear_scan.cu): any supported shape and type.
size_t linear_scan_scratch_bytes(int nseq, int HV, int dk, int dv, long total, int max_len, bool varlen, int sms);
cudaError_t launch_linear_scan(const LinFwd &a, cudaStream_t st);

struct LinDecode {
    LinView q, k, v, o;   // b strides only (one token)
    const float *g;       // [B, HV] (gb = HV), [HV] (gb = 0) or nullptr
    long long gb;
    float *state;         // [B, HV, dk, dv], in place
    int B, H, HV, dk, dv;
    DType dtype;
    float scale;
    int sms;
};
cudaError_t launch_linear_decode(const LinDecode &a, cudaStream_t st);

// Gradients.
struct LinBwd {
    LinView q, k, v, d_o;       // inputs
    LinView dq, dk_, dv_;       // outputs, the inputs' type
    LinDecay g;
    float *dg;                  // [B, T, HV], [HV] when g is fixed per head, or nullptr
    const float *h0, *dhT;      // [B, HV, dk, dv] or nullptr
    float *dh0;                 // the same or nullptr
    int B, T, H, HV, dk, dv;
    DType dtype;
    float scale;
    void *ws;
    WsHeader *hdr;
    int sms;
};
size_t linear_scan_bwd_scratch_bytes(int B, int T, int H, int HV, int dk, int dv, int sms);
cudaError_t launch_linear_scan_bwd(const LinBwd &a, cudaStream_t st);

// Tensor-core chunked forms (linear_tc.cu): bf16, dk and dv in {64, 128}.
bool linear_tc_supported(int dk, int dv, DType dt);
size_t linear_tc_scratch_bytes(int nseq, int HV, int dk, int dv, long total, int max_len, bool varlen, int sms);
cudaError_t launch_linear_tc(const LinFwd &a, cudaStream_t st);
size_t linear_tc_bwd_scratch_bytes(int B, int T, int H, int HV, int dk, int dv, int sms);
cudaError_t launch_linear_tc_bwd(const LinBwd &a, cudaStream_t st);

// Reductions the backwards share (linear_scan.cu): the value heads of a shared q/k head added
// up, dq and dk at once (fp32 [rows, HV, D] -> out[rows, H, D] of the input type), and a fixed decay's
// gradient (per-token [B * T, HV] -> [HV]).
cudaError_t launch_fold_heads(const float *src0, const LinView &dst0, const float *src1, const LinView &dst1, DType dt,
                              int B, int T, int H, int m, int D, cudaStream_t st);
cudaError_t launch_sum_rows(const float *src, float *dst, long rows, int cols, cudaStream_t st);

}  // namespace kda
