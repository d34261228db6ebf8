// ssm_api.cu -- the C ABI of the short convolution, the state space scan and beam search: argument checks, workspace
// carving, dispatch.  Nothing here allocates device memory.
#include <initializer_list>

#include "../../include/kda.h"
#include "beam_internal.cuh"
#include "conv_internal.cuh"
#include "ssm_internal.cuh"

using namespace kda;

namespace {

constexpr int kSms = 152;       // the work is split for this part's SM count; the workspace queries make no CUDA call

bool al(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(kda_dtype d) { return d == KDA_F32 || d == KDA_BF16; }
unsigned size_of(kda_dtype d) { return d == KDA_BF16 ? 2 : 4; }
DType to_dtype(kda_dtype d) { return d == KDA_BF16 ? DType::BF16 : DType::F32; }
// Whether one of the outputs is one of the inputs (nullptr: not there).
bool any_in_place(std::initializer_list<const void *> outputs, std::initializer_list<const void *> inputs) {
    for (const void *o : outputs)
        for (const void *i : inputs)
            if (o && o == i) return true;
    return false;
}
kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

// Packed sequences: the device array, and the host copy where there is one (max_len: bound on the longest).
kda_status check_packed(const int *cu, const int *host, int N, int total, int &max_len) {
    if (N == 0 && total > 0) return KDA_ERR_INDEX;      // tokens of no sequence: nobody would write their outputs
    if (N > 0 && !cu) return KDA_ERR_NULL;
    if (!al(cu, 4)) return KDA_ERR_ALIGN;
    max_len = total;
    if (host) {
        if (host[0] != 0 || host[N] != total) return KDA_ERR_INDEX;
        max_len = 0;
        for (int n = 0; n < N; ++n) {
            const long L = (long)host[n + 1] - host[n];
            if (L < 0) return KDA_ERR_INDEX;
            if (L > max_len) max_len = (int)L;
        }
    }
    return KDA_OK;
}

// ------------------------------------------------------------------------------ convolution

kda_status conv_shape(long N, long T, int C, int K, kda_dtype dtype, int act) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (N < 0 || T < 0 || C <= 0 || K <= 0 || N * T > 0x7fffffffL || C > 1 << 20 || N > 1 << 24) return KDA_ERR_SHAPE;
    return K < 2 || K > 4 || act < 0 || act > 1 ? KDA_ERR_UNSUPPORTED : KDA_OK;
}
ConvView conv_view(const void *p, const long long *s, int i, long N, long T, int C) {
    ConvView v{const_cast<void *>(p), (long long)T * C, C};
    if (s && N > 1) v.b = s[2 * i];
    if (s && T > 1) v.t = s[2 * i + 1];
    return v;
}

kda_status conv_fwd(const void *x, const float *w, const float *bias, const void *h0, void *y, void *hT, const long long *strides,
                    const int *cu, int N, int T, long rows, int C, int K, kda_dtype dtype, int act, cudaStream_t st) {
    if (!w || (rows > 0 && (!x || !y))) return KDA_ERR_NULL;
    if (rows > 0 && y == x) return KDA_ERR_UNSUPPORTED;     // rows are read by more runs than the one that writes them
    const unsigned e = size_of(dtype);
    if (!al(x, e) || !al(y, e) || !al(h0, e) || !al(hT, e) || !al(w, 4) || !al(bias, 4)) return KDA_ERR_ALIGN;
    if (N == 0) return KDA_OK;
    Conv a{};
    a.x = conv_view(x, strides, 0, cu ? 1 : N, T, C);
    a.y = conv_view(y, strides, 1, cu ? 1 : N, T, C);
    a.w = w; a.bias = bias; a.h0 = h0; a.hT = hT;
    a.s.cu = cu; a.s.nseq = N; a.s.T = cu ? 0 : T; a.total = T;
    a.C = C; a.K = K; a.act = act; a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_conv(a, st));
}

// ------------------------------------------------------------------------------ scan

kda_status ssm_shape(long N, long T, int D, int G, int S, kda_dtype dtype) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (N < 0 || T < 0 || D <= 0 || G <= 0 || D % G || S <= 0 || N * T > 0x7fffffffL || D > 1 << 20 || N > 65535)
        return KDA_ERR_SHAPE;
    return S == 8 || S == 16 || S == 32 || S == 64 ? KDA_OK : KDA_ERR_UNSUPPORTED;
}
SsmView ssm_rows(const void *p, const long long *s, int i, long N, long T, int D) {
    SsmView v{const_cast<void *>(p), (long long)T * D, D, 0};
    if (s && N > 1) v.b = s[3 * i];
    if (s && T > 1) v.t = s[3 * i + 1];
    return v;
}
SsmView ssm_heads(const void *p, const long long *s, int i, long N, long T, int G, int S) {
    SsmView v = ssm_rows(p, s, i, N, T, G * S);
    v.g = s && G > 1 ? s[3 * i + 2] : S;
    return v;
}

struct SsmIn {
    const void *x, *dt, *B, *C, *gate;
    const float *A, *skip, *bias, *h0;
};
// Whether y is one of the inputs: a split sequence is read by two launches, of which the second writes; the rows of B and C
// are read by all CTAs of a group, the other arrays by all that have a channel.
bool in_place(const void *y, const SsmIn &p, const int *cu, long rows) {
    return rows > 0 && any_in_place({y}, {p.x, p.dt, p.B, p.C, p.gate, p.A, p.skip, p.bias, p.h0, cu});
}
// The arrays that every call has; strides in the order x, dt, B, C, gate.
kda_status ssm_in(Ssm &a, const SsmIn &p, const long long *s, const int *cu, int N, int T, long rows, int D, int G, int S,
                  kda_dtype dtype, int softplus) {
    if (!p.A || (rows > 0 && (!p.x || !p.dt || !p.B || !p.C))) return KDA_ERR_NULL;
    const unsigned e = size_of(dtype);
    for (const void *q : {p.x, p.dt, p.B, p.C, p.gate})
        if (!al(q, e)) return KDA_ERR_ALIGN;
    if (!al(p.A, 16) || !al(p.h0, 16) || !al(p.skip, 4) || !al(p.bias, 4)) return KDA_ERR_ALIGN;
    const long nb = cu ? 1 : N;
    a.x = ssm_rows(p.x, s, 0, nb, T, D);
    a.dt = ssm_rows(p.dt, s, 1, nb, T, D);
    a.B = ssm_heads(p.B, s, 2, nb, T, G, S);
    a.C = ssm_heads(p.C, s, 3, nb, T, G, S);
    a.gate = ssm_rows(p.gate, s, 4, nb, T, D);
    a.A = p.A; a.skip = p.skip; a.bias = p.bias; a.h0 = p.h0;
    a.s.cu = cu; a.s.nseq = N; a.s.T = cu ? 0 : T; a.total = T; a.max_len = T;
    a.D = D; a.G = G; a.N = S; a.softplus = softplus != 0; a.dtype = to_dtype(dtype); a.sms = kSms;
    return KDA_OK;
}

constexpr size_t kLeast = 256;      // bytes of the smallest workspace

}  // namespace

extern "C" {

kda_status kda_conv_fwd(const void *x, const float *weight, const float *bias, const void *initial_state, void *y,
                        void *final_state, const long long *strides, int B, int T, int C, int K, kda_dtype dtype,
                        int activation, kda_stream_t stream) {
    const kda_status c = conv_shape(B, T, C, K, dtype, activation);
    if (c != KDA_OK) return c;
    return conv_fwd(x, weight, bias, initial_state, y, final_state, strides, nullptr, B, T, (long)B * T, C, K, dtype,
                    activation, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_conv_varlen_fwd(const void *x, const float *weight, const float *bias, const int *cu_seqlens,
                               const int *cu_seqlens_host, const void *initial_state, void *y, void *final_state,
                               const long long *strides, int N, int total_T, int C, int K, kda_dtype dtype,
                               int activation, kda_stream_t stream) {
    kda_status c = conv_shape(N, 0, C, K, dtype, activation);
    if (c != KDA_OK) return c;
    if (total_T < 0) return KDA_ERR_SHAPE;
    int max_len;
    c = check_packed(cu_seqlens, cu_seqlens_host, N, total_T, max_len);
    if (c != KDA_OK) return c;
    return conv_fwd(x, weight, bias, initial_state, y, final_state, strides, cu_seqlens, N, total_T, total_T, C, K, dtype,
                    activation, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_conv_decode_step(const void *x, const float *weight, const float *bias, void *state, void *y,
                                const long long *strides, int B, int C, int K, kda_dtype dtype, int activation,
                                kda_stream_t stream) {
    const kda_status c = conv_shape(B, 1, C, K, dtype, activation);
    if (c != KDA_OK) return c;
    if (B == 0) return KDA_OK;
    if (!x || !weight || !state || !y) return KDA_ERR_NULL;
    const unsigned e = size_of(dtype);
    if (!al(x, e) || !al(y, e) || !al(state, e) || !al(weight, 4) || !al(bias, 4)) return KDA_ERR_ALIGN;
    ConvStep a{};
    a.x = x; a.y = y; a.state = state; a.w = weight; a.bias = bias;
    a.xb = strides ? strides[0] : C;
    a.yb = strides ? strides[1] : C;
    a.B = B; a.C = C; a.K = K; a.act = activation; a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_conv_step(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_conv_bwd_workspace(int C, int K) {
    if (conv_shape(0, 0, C, K, KDA_F32, 0) != KDA_OK) return 0;
    return kLeast + (size_t)conv_parts(C, kSms) * C * (K + 1) * 4;
}

kda_status kda_conv_bwd(const void *d_y, const void *x, const float *weight, const float *bias, const void *initial_state,
                        const void *dfinal_state, void *dx, float *dweight, float *dbias, void *dinitial_state,
                        const int *cu_seqlens, const long long *strides, int N, int T, int C, int K, kda_dtype dtype,
                        int activation, void *ws, size_t ws_bytes, kda_stream_t stream) {
    kda_status c = conv_shape(N, cu_seqlens ? 0 : T, C, K, dtype, activation);
    if (c != KDA_OK) return c;
    if (T < 0) return KDA_ERR_SHAPE;
    const long rows = cu_seqlens ? T : (long)N * T;
    if (cu_seqlens && N == 0 && T > 0) return KDA_ERR_INDEX;
    if (!weight || !dweight || (rows > 0 && (!x || !d_y || !dx))) return KDA_ERR_NULL;
    const unsigned e = size_of(dtype);
    for (const void *p : {d_y, x, initial_state, dfinal_state, (const void *)dx, (const void *)dinitial_state})
        if (!al(p, e)) return KDA_ERR_ALIGN;
    if (!al(weight, 4) || !al(bias, 4) || !al(dweight, 4) || !al(dbias, 4) || !al(cu_seqlens, 4)) return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_conv_bwd_workspace(C, K)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    // rows and windows are read by other runs than the one that writes them
    const auto tok = [&](const void *p) { return rows > 0 ? p : nullptr; };
    const auto seq = [&](const void *p) { return N > 0 ? p : nullptr; };
    if (any_in_place({tok(dx), dweight, dbias, seq(dinitial_state)},
                     {tok(d_y), tok(x), weight, bias, seq(initial_state), seq(dfinal_state), cu_seqlens}))
        return KDA_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {
        if (cudaMemsetAsync(dweight, 0, (size_t)C * K * 4, st) != cudaSuccess) return KDA_ERR_CUDA;
        return dbias ? done(cudaMemsetAsync(dbias, 0, (size_t)C * 4, st)) : KDA_OK;
    }
    Conv a{};
    const long nb = cu_seqlens ? 1 : N;
    a.x = conv_view(x, strides, 0, nb, T, C);
    a.y = conv_view(d_y, strides, 1, nb, T, C);
    a.dx = conv_view(dx, strides, 2, nb, T, C);
    a.w = weight; a.bias = bias; a.h0 = initial_state; a.dhT = dfinal_state; a.dh0 = dinitial_state;
    a.dw = dweight; a.dbias = dbias; a.part = static_cast<float *>(ws);
    a.s.cu = cu_seqlens; a.s.nseq = N; a.s.T = cu_seqlens ? 0 : T; a.total = T;
    a.C = C; a.K = K; a.act = activation; a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_conv_bwd(a, st));
}

size_t kda_ssm_chunk_fwd_workspace(int B, int T, int D, int G, int N, kda_dtype dtype) {
    if (ssm_shape(B, T, D, G, N, dtype) != KDA_OK) return 0;
    return kLeast + ssm_scratch_bytes(B, T, T, false, D, G, N, kSms);
}

size_t kda_ssm_varlen_fwd_workspace(int nseq, int total_T, int D, int G, int N, kda_dtype dtype) {
    if (ssm_shape(nseq, 0, D, G, N, dtype) != KDA_OK || total_T < 0) return 0;
    return kLeast + ssm_scratch_bytes(nseq, total_T, total_T, true, D, G, N, kSms);
}

kda_status kda_ssm_chunk_fwd(const void *x, const void *dt, const float *A, const void *B_in, const void *C_in,
                             const float *skip, const void *gate, const float *dt_bias, const float *initial_state, void *y,
                             float *final_state, const long long *strides, int B, int T, int D, int G, int N,
                             kda_dtype dtype, int softplus, void *ws, size_t ws_bytes, kda_stream_t stream) {
    kda_status c = ssm_shape(B, T, D, G, N, dtype);
    if (c != KDA_OK) return c;
    Ssm a{};
    c = ssm_in(a, {x, dt, B_in, C_in, gate, A, skip, dt_bias, initial_state}, strides, nullptr, B, T, (long)B * T, D, G, N, dtype,
               softplus);
    if (c != KDA_OK) return c;
    if ((long)B * T > 0 && !y) return KDA_ERR_NULL;
    if (in_place(y, {x, dt, B_in, C_in, gate, A, skip, dt_bias, initial_state}, nullptr, (long)B * T)) return KDA_ERR_UNSUPPORTED;
    if (!al(y, size_of(dtype)) || !al(final_state, 16)) return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_ssm_chunk_fwd_workspace(B, T, D, G, N, dtype)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    if (B == 0) return KDA_OK;
    a.y = ssm_rows(y, strides, 5, B, T, D);
    a.hT = final_state;
    a.ws = ws;
    return done(launch_ssm(a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_ssm_varlen_fwd(const void *x, const void *dt, const float *A, const void *B_in, const void *C_in,
                              const float *skip, const void *gate, const float *dt_bias, const int *cu_seqlens,
                              const int *cu_seqlens_host, const float *initial_state, void *y, float *final_state,
                              const long long *strides, int nseq, int total_T, int D, int G, int N, kda_dtype dtype,
                              int softplus, void *ws, size_t ws_bytes, kda_stream_t stream) {
    kda_status c = ssm_shape(nseq, 0, D, G, N, dtype);
    if (c != KDA_OK) return c;
    if (total_T < 0) return KDA_ERR_SHAPE;
    int max_len;
    c = check_packed(cu_seqlens, cu_seqlens_host, nseq, total_T, max_len);
    if (c != KDA_OK) return c;
    Ssm a{};
    c = ssm_in(a, {x, dt, B_in, C_in, gate, A, skip, dt_bias, initial_state}, strides, cu_seqlens, nseq, total_T, total_T, D, G, N,
               dtype, softplus);
    if (c != KDA_OK) return c;
    if (total_T > 0 && !y) return KDA_ERR_NULL;
    if (in_place(y, {x, dt, B_in, C_in, gate, A, skip, dt_bias, initial_state}, cu_seqlens, total_T)) return KDA_ERR_UNSUPPORTED;
    if (!al(y, size_of(dtype)) || !al(final_state, 16)) return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_ssm_varlen_fwd_workspace(nseq, total_T, D, G, N, dtype)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    if (nseq == 0) return KDA_OK;
    a.max_len = max_len;
    a.y = ssm_rows(y, strides, 5, 1, total_T, D);
    a.hT = final_state;
    a.ws = ws;
    return done(launch_ssm(a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_ssm_decode_step(const void *x, const void *dt, const float *A, const void *B_in, const void *C_in,
                               const float *skip, const void *gate, const float *dt_bias, float *state, void *y,
                               const long long *strides, int B, int D, int G, int N, kda_dtype dtype, int softplus,
                               kda_stream_t stream) {
    const kda_status c = ssm_shape(B, 1, D, G, N, dtype);
    if (c != KDA_OK) return c;
    if (B == 0) return KDA_OK;
    if (!x || !dt || !A || !B_in || !C_in || !state || !y) return KDA_ERR_NULL;
    const unsigned e = size_of(dtype);
    for (const void *p : {x, dt, B_in, C_in, gate, (const void *)y})
        if (!al(p, e)) return KDA_ERR_ALIGN;
    if (!al(A, 16) || !al(state, 16) || !al(skip, 4) || !al(dt_bias, 4)) return KDA_ERR_ALIGN;
    SsmStep a{};
    a.x = x; a.dt = dt; a.gate = gate; a.B = B_in; a.C = C_in; a.y = y;
    a.A = A; a.skip = skip; a.bias = dt_bias; a.state = state;
    const long long plain[8] = {D, D, (long long)G * N, N, (long long)G * N, N, D, D};
    const long long *s = strides ? strides : plain;
    a.xb = s[0]; a.dtb = s[1]; a.Bb = s[2]; a.Bg = s[3]; a.Cb = s[4]; a.Cg = s[5]; a.gb = s[6]; a.yb = s[7];
    a.nb = B; a.D = D; a.G = G; a.N = N; a.softplus = softplus != 0; a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_ssm_step(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_ssm_chunk_bwd_workspace(int nseq, int T, int packed, int D, int G, int N, kda_dtype dtype) {
    if (ssm_shape(nseq, packed ? 0 : T, D, G, N, dtype) != KDA_OK || T < 0) return 0;
    return kLeast + ssm_bwd_scratch_bytes(nseq, T, T, packed != 0, D, G, N, kSms);
}

kda_status kda_ssm_chunk_bwd(const void *d_y, const void *x, const void *dt, const float *A, const void *B_in, const void *C_in,
                             const float *skip, const void *gate, const float *dt_bias, const float *initial_state,
                             const float *dfinal_state, void *dx, void *ddt, float *dA, void *dB, void *dC, float *dskip,
                             void *dgate, float *ddt_bias, float *dinitial_state, const int *cu_seqlens,
                             const long long *strides, int nseq, int T, int D, int G, int N, kda_dtype dtype, int softplus,
                             void *ws, size_t ws_bytes, kda_stream_t stream) {
    kda_status c = ssm_shape(nseq, cu_seqlens ? 0 : T, D, G, N, dtype);
    if (c != KDA_OK) return c;
    if (T < 0) return KDA_ERR_SHAPE;
    if (cu_seqlens && nseq == 0 && T > 0) return KDA_ERR_INDEX;
    const long rows = cu_seqlens ? T : (long)nseq * T;
    Ssm a{};
    c = ssm_in(a, {x, dt, B_in, C_in, gate, A, skip, dt_bias, initial_state}, strides, cu_seqlens, nseq, T, rows, D, G, N, dtype,
               softplus);
    if (c != KDA_OK) return c;
    if (!dA || (rows > 0 && (!d_y || !dx || !ddt || !dB || !dC || (gate && !dgate)))) return KDA_ERR_NULL;
    const unsigned e = size_of(dtype);
    for (const void *p : {d_y, (const void *)dx, (const void *)ddt, (const void *)dB, (const void *)dC, (const void *)dgate})
        if (!al(p, e)) return KDA_ERR_ALIGN;
    if (!al(dA, 16) || !al(dfinal_state, 16) || !al(dinitial_state, 16) || !al(dskip, 4) || !al(ddt_bias, 4) || !al(cu_seqlens, 4))
        return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_ssm_chunk_bwd_workspace(nseq, T, cu_seqlens != nullptr, D, G, N, dtype)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    // arrays without rows have no address that counts
    const auto tok = [&](const void *p) { return rows > 0 ? p : nullptr; };
    const auto seq = [&](const void *p) { return nseq > 0 ? p : nullptr; };
    if (any_in_place({tok(dx), tok(ddt), tok(dB), tok(dC), gate ? tok(dgate) : nullptr, dA, dskip, ddt_bias, seq(dinitial_state)},
                     {tok(d_y), tok(x), tok(dt), tok(B_in), tok(C_in), tok(gate), A, skip, dt_bias, seq(initial_state),
                      seq(dfinal_state), cu_seqlens}))
        return KDA_ERR_UNSUPPORTED;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (nseq == 0) {
        if (cudaMemsetAsync(dA, 0, (size_t)D * N * 4, st) != cudaSuccess) return KDA_ERR_CUDA;
        if (dskip && cudaMemsetAsync(dskip, 0, (size_t)D * 4, st) != cudaSuccess) return KDA_ERR_CUDA;
        return ddt_bias ? done(cudaMemsetAsync(ddt_bias, 0, (size_t)D * 4, st)) : KDA_OK;
    }
    const long nb = cu_seqlens ? 1 : nseq;
    a.y = ssm_rows(d_y, strides, 5, nb, T, D);
    a.dx = ssm_rows(dx, nullptr, 0, nb, T, D);
    a.ddt = ssm_rows(ddt, nullptr, 0, nb, T, D);
    a.dgate = ssm_rows(gate ? dgate : nullptr, nullptr, 0, nb, T, D);
    a.dB = ssm_heads(dB, nullptr, 0, nb, T, G, N);
    a.dC = ssm_heads(dC, nullptr, 0, nb, T, G, N);
    a.dA = dA; a.dskip = dskip; a.dbias = ddt_bias; a.dh0 = dinitial_state; a.dhT = dfinal_state;
    a.ws = ws;
    return done(launch_ssm_bwd(a, st));
}

// ------------------------------------------------------------------------------ beams

static kda_status beam_shape(int B, int W, int V, int k, kda_dtype dtype) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (B < 0 || W <= 0 || V <= 0 || k <= 0 || (long)W * V > 0x7fffffffL || (long)B * W > 0xffffffL || k > (long)W * V)
        return KDA_ERR_SHAPE;
    return k > kBeamMax || W > kBeamsIn ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

size_t kda_beam_select_workspace(int B, int W, int V, kda_dtype dtype) {
    if (beam_shape(B, W, V, 1, dtype) != KDA_OK) return 0;
    const long rows = (long)B * W;
    const int nc = beam_chunks(V);
    return kLeast + rows * beam_splits(rows, beam_takes(V), kSms) * sizeof(BeamSum) + (size_t)rows * nc * 4;
}

kda_status kda_beam_select(const void *logits, const long long *strides, const float *scores, const unsigned char *finished,
                           int eos, float *out_scores, int *parents, int *tokens, int B, int W, int V, int k,
                           kda_dtype dtype, void *ws, size_t ws_bytes, kda_stream_t stream) {
    const kda_status c = beam_shape(B, W, V, k, dtype);
    if (c != KDA_OK) return c;
    if (finished && (eos < 0 || eos >= V)) return KDA_ERR_INDEX;
    if (B == 0) return KDA_OK;
    if (!logits || !scores || !out_scores || !parents || !tokens) return KDA_ERR_NULL;
    if (!al(logits, size_of(dtype)) || !al(scores, 4) || !al(out_scores, 4) || !al(parents, 4) || !al(tokens, 4)) return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_beam_select_workspace(B, W, V, dtype)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    BeamSelect a{};
    a.logits = logits;
    a.sb = strides ? strides[0] : (long long)W * V;
    a.sw = strides ? strides[1] : V;
    a.scores = scores; a.finished = finished; a.out = out_scores; a.parents = parents; a.tokens = tokens;
    a.B = B; a.W = W; a.V = V; a.k = k; a.eos = eos; a.dtype = to_dtype(dtype); a.sms = kSms;
    const long rows = (long)B * W;
    a.nc = beam_chunks(V);
    a.splits = beam_splits(rows, beam_takes(V), kSms);
    a.sums = static_cast<BeamSum *>(ws);
    a.cmax = reinterpret_cast<float *>(a.sums + rows * a.splits);
    return done(launch_beam_select(a, reinterpret_cast<cudaStream_t>(stream)));
}

kda_status kda_beam_reorder(void *const *states, const long long *row_bytes, int count, const int *parents, int B, int W,
                            kda_stream_t stream) {
    if (count < 0 || B < 0 || W <= 0 || B > 65535) return KDA_ERR_SHAPE;
    if (W > kBeamMax) return KDA_ERR_UNSUPPORTED;
    if (count > 0 && (!states || !row_bytes)) return KDA_ERR_NULL;
    for (int i = 0; i < count; ++i) {
        if (row_bytes[i] < 0) return KDA_ERR_SHAPE;
        if (B > 0 && row_bytes[i] > 0 && !states[i]) return KDA_ERR_NULL;
        const uintptr_t p = reinterpret_cast<uintptr_t>(states[i]), n = (uintptr_t)row_bytes[i] * B * W;
        for (int j = 0; j < i; ++j) {       // an array that is there twice would be moved twice
            const uintptr_t q = reinterpret_cast<uintptr_t>(states[j]), m = (uintptr_t)row_bytes[j] * B * W;
            if (n && m && p < q + m && q < p + n) return KDA_ERR_INDEX;
        }
    }
    if (B == 0 || count == 0 || W == 1) return KDA_OK;
    if (!parents) return KDA_ERR_NULL;
    if (!al(parents, 4)) return KDA_ERR_ALIGN;
    for (int i = 0; i < count; ++i) {       // every CTA reads them, others have written by then
        const uintptr_t p = reinterpret_cast<uintptr_t>(states[i]), q = reinterpret_cast<uintptr_t>(parents);
        if (row_bytes[i] && p < q + 4 * (uintptr_t)B * W && q < p + (uintptr_t)row_bytes[i] * B * W) return KDA_ERR_INDEX;
    }
    for (int i0 = 0; i0 < count; i0 += kBeamStates) {
        BeamReorder a{};
        a.count = count - i0 < kBeamStates ? count - i0 : kBeamStates;
        for (int i = 0; i < a.count; ++i) {
            a.p[i] = static_cast<char *>(states[i0 + i]);
            a.bytes[i] = row_bytes[i0 + i];
        }
        a.parents = parents; a.B = B; a.W = W;
        if (launch_beam_reorder(a, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess) return KDA_ERR_CUDA;
    }
    return KDA_OK;
}

}  // extern "C"
