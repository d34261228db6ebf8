// linear_api.cu -- the C ABI of linear attention with a decay per head and of the block norms:
// argument checks, workspace carving, dispatch.  Nothing here allocates device memory.
#include <math.h>

#include "../../include/kda.h"
#include "linear_internal.cuh"
#include "norm_internal.cuh"

using namespace kda;

namespace {

constexpr size_t kWsHeader = sizeof(WsHeader);
// The work is split for this part's SM count; the workspace queries make no CUDA call.
constexpr int kSms = 152;

bool head_ok(int d) { return d == 32 || d == 64 || d == 128; }
bool al(const void *p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(kda_dtype d) { return d == KDA_F32 || d == KDA_BF16; }
DType to_dtype(kda_dtype d) { return d == KDA_BF16 ? DType::BF16 : DType::F32; }
float pick_scale(float s, int dk) { return s > 0.f ? s : 1.0f / sqrtf((float)dk); }
kda_status done(cudaError_t e) { return e == cudaSuccess ? KDA_OK : KDA_ERR_CUDA; }

kda_status check_shape(long B, long T, int H, int HV, int dk, int dv, kda_dtype dtype) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (B < 0 || T < 0 || H <= 0 || HV < H || HV % H || dk <= 0 || dv <= 0) return KDA_ERR_SHAPE;
    if (!head_ok(dk) || !head_ok(dv)) return KDA_ERR_UNSUPPORTED;
    // launch limits: heads in grid.y, token rows and (sequence, head) pairs as int
    if (HV > 65535 || B * (long)HV > 0x3fffffffL || B * T > 0x7fffffffL) return KDA_ERR_SHAPE;
    return KDA_OK;
}

// The view of array `i` (strides NULL: contiguous [B, T, heads, D]).  False: a misaligned stride.
bool view(LinView &v, const void *p, const long long *strides, int i, long B, long T, int heads, int D, kda_dtype dt) {
    v.p = p;
    v.h = D;
    v.t = (long long)heads * D;
    v.b = (long long)T * heads * D;
    if (!strides) return true;
    const int unit = dt == KDA_BF16 ? 8 : 4;
    const long long *s = strides + 3 * i;
    if (B > 1) v.b = s[0];
    if (T > 1) v.t = s[1];
    if (heads > 1) v.h = s[2];
    return v.b % unit == 0 && v.t % unit == 0 && v.h % unit == 0;
}

// Whether the chunked tensor-core form takes this problem.  A chunk costs the same whatever it
// holds; the token walk costs less for a few tokens.  On the device, walk and chunk, 16 tokens: prefill of one
// sequence, 4 heads of 64 5.0 and 7.8 us, of 128 7.1 and 9.6, of 16 x 32 heads of 128 56 and 35; gradients 8.7 and 15.2,
// 9.2 and 21, 98 and 117.  32 tokens: prefill 7.0 and 7.9, 9.5 and 9.7, 77 and 35; gradients 10.8 and 15.0, 12.4 and 21,
// 175 and 121.  One limit serves both; gradients of one sequence with few heads would gain by the walk up to 64 tokens.
bool use_tc(int dk, int dv, kda_dtype dt, int max_len) {
    return linear_tc_supported(dk, dv, to_dtype(dt)) && max_len > 16;
}

size_t fwd_scratch(int n, long total, int max_len, bool varlen, int HV, int dk, int dv, kda_dtype dt) {
    // packed: the longest sequence may turn out short or long, so room for either form
    size_t a = linear_scan_scratch_bytes(n, HV, dk, dv, total, max_len, varlen, kSms);
    if (use_tc(dk, dv, dt, max_len)) {
        const size_t b = linear_tc_scratch_bytes(n, HV, dk, dv, total, max_len, varlen, kSms);
        a = varlen ? (a > b ? a : b) : b;
    }
    return kWsHeader + a;
}

kda_status run_fwd(LinFwd &a, void *ws, kda_dtype dt, cudaStream_t st) {
    a.hdr = static_cast<WsHeader *>(ws);
    a.ws = static_cast<char *>(ws) + kWsHeader;
    a.sms = kSms;
    if (a.s.nseq == 0) return KDA_OK;        // nothing to do: no pointer is touched
    if (a.max_len == 0) {
        if (cudaMemsetAsync(ws, 0, 2 * sizeof(int), st) != cudaSuccess) return KDA_ERR_CUDA;
        SeqBatch p{};
        p.h0 = a.h0; p.hT = a.hT; p.nseq = a.s.nseq; p.H = a.HV; p.dk = a.dk; p.dv = a.dv;
        return done(launch_state_passthrough(p, st));
    }
    if (!use_tc(a.dk, a.dv, dt, a.max_len)) return done(launch_linear_scan(a, st));
    return done(launch_linear_tc(a, st));
}

}  // namespace

extern "C" {

size_t kda_linear_chunk_fwd_workspace(int B, int T, int H, int HV, int dk, int dv, kda_dtype dtype) {
    if (check_shape(B, T, H, HV, dk, dv, dtype) != KDA_OK) return 0;
    return fwd_scratch(B, T, T, false, HV, dk, dv, dtype);
}

size_t kda_linear_varlen_fwd_workspace(int N, int total_T, int H, int HV, int dk, int dv, kda_dtype dtype) {
    if (check_shape(N, 0, H, HV, dk, dv, dtype) != KDA_OK || total_T < 0) return 0;
    return fwd_scratch(N, total_T, total_T, true, HV, dk, dv, dtype);
}

static kda_status linear_fwd(const void *q, const void *k, const void *v, const float *decay, int decay_fixed,
                             const float *h0, void *o, float *hT, const long long *strides, int B, int T, long rows,
                             int H, int HV, int dk, int dv, kda_dtype dtype, float scale, LinFwd &a) {
    if (rows > 0 && (!q || !k || !v || !o)) return KDA_ERR_NULL;
    if (!al(q, 16) || !al(k, 16) || !al(v, 16) || !al(o, 16) || !al(h0, 16) || !al(hT, 16) || !al(decay, 4))
        return KDA_ERR_ALIGN;
    if (!view(a.q, q, strides, 0, B, T, H, dk, dtype) || !view(a.k, k, strides, 1, B, T, H, dk, dtype) ||
        !view(a.v, v, strides, 2, B, T, HV, dv, dtype) || !view(a.o, o, strides, 3, B, T, HV, dv, dtype))
        return KDA_ERR_ALIGN;
    a.g.p = decay;
    a.g.b = decay_fixed ? 0 : (long long)T * HV;
    a.g.t = decay_fixed ? 0 : HV;
    a.h0 = h0; a.hT = hT; a.H = H; a.HV = HV; a.dk = dk; a.dv = dv;
    a.dtype = to_dtype(dtype); a.scale = pick_scale(scale, dk);
    return KDA_OK;
}

kda_status kda_linear_chunk_fwd(const void *q, const void *k, const void *v, const float *decay, int decay_fixed,
                                const float *initial_state, void *o, float *final_state, const long long *strides,
                                int B, int T, int H, int HV, int dk, int dv, kda_dtype dtype, float scale, void *ws,
                                size_t ws_bytes, kda_stream_t stream) {
    kda_status c = check_shape(B, T, H, HV, dk, dv, dtype);
    if (c != KDA_OK) return c;
    LinFwd a{};
    c = linear_fwd(q, k, v, decay, decay_fixed, initial_state, o, final_state, strides, B, T, (long)B * T, H, HV, dk,
                   dv, dtype, scale, a);
    if (c != KDA_OK) return c;
    if (!ws || ws_bytes < kda_linear_chunk_fwd_workspace(B, T, H, HV, dk, dv, dtype)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    a.s.nseq = B; a.s.T = T; a.total = T; a.max_len = T;
    return run_fwd(a, ws, dtype, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_linear_varlen_fwd(const void *q, const void *k, const void *v, const float *decay, int decay_fixed,
                                 const int *cu_seqlens, const int *cu_seqlens_host, const float *initial_state,
                                 void *o, float *final_state, const long long *strides, int N, int total_T, int H,
                                 int HV, int dk, int dv, kda_dtype dtype, float scale, void *ws, size_t ws_bytes,
                                 kda_stream_t stream) {
    kda_status c = check_shape(N, 0, H, HV, dk, dv, dtype);
    if (c != KDA_OK) return c;
    if (total_T < 0) return KDA_ERR_SHAPE;
    if (N == 0 && total_T > 0) return KDA_ERR_INDEX;      // tokens of no sequence: nobody would write their outputs
    if (N > 0 && !cu_seqlens) return KDA_ERR_NULL;
    if (!al(cu_seqlens, 4)) return KDA_ERR_ALIGN;
    LinFwd a{};
    c = linear_fwd(q, k, v, decay, decay_fixed, initial_state, o, final_state, strides, 1, total_T, total_T, H, HV,
                   dk, dv, dtype, scale, a);
    if (c != KDA_OK) return c;
    int max_len = total_T;
    if (cu_seqlens_host) {
        if (cu_seqlens_host[0] != 0 || cu_seqlens_host[N] != total_T) return KDA_ERR_INDEX;
        max_len = 0;
        for (int n = 0; n < N; ++n) {
            const long L = (long)cu_seqlens_host[n + 1] - cu_seqlens_host[n];
            if (L < 0) return KDA_ERR_INDEX;
            if (L > max_len) max_len = (int)L;
        }
    }
    if (!ws || ws_bytes < kda_linear_varlen_fwd_workspace(N, total_T, H, HV, dk, dv, dtype)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    a.s.cu = cu_seqlens; a.s.nseq = N; a.total = total_T; a.max_len = max_len;
    return run_fwd(a, ws, dtype, reinterpret_cast<cudaStream_t>(stream));
}

kda_status kda_linear_decode_step(const void *q, const void *k, const void *v, const float *decay, int decay_fixed,
                                  float *state, void *o, const long long *strides, int B, int H, int HV, int dk,
                                  int dv, kda_dtype dtype, float scale, kda_stream_t stream) {
    kda_status c = check_shape(B, 1, H, HV, dk, dv, dtype);
    if (c != KDA_OK) return c;
    if (B == 0) return KDA_OK;
    if (!q || !k || !v || !o || !state) return KDA_ERR_NULL;
    const unsigned e = dtype == KDA_BF16 ? 2 : 4;
    if (!al(q, e) || !al(k, e) || !al(v, e) || !al(o, e) || !al(state, 16) || !al(decay, 4)) return KDA_ERR_ALIGN;
    LinDecode a{};
    const void *ps[4] = {q, k, v, o};
    LinView *vs[4] = {&a.q, &a.k, &a.v, &a.o};
    for (int i = 0; i < 4; ++i) {
        const int heads = i < 2 ? H : HV, D = i < 2 ? dk : dv;
        vs[i]->p = ps[i];
        vs[i]->b = strides ? strides[2 * i] : (long long)heads * D;
        vs[i]->h = strides ? strides[2 * i + 1] : D;
    }
    a.g = decay; a.gb = decay_fixed ? 0 : HV;
    a.state = state; a.B = B; a.H = H; a.HV = HV; a.dk = dk; a.dv = dv;
    a.dtype = to_dtype(dtype); a.scale = pick_scale(scale, dk); a.sms = kSms;
    return done(launch_linear_decode(a, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_linear_chunk_bwd_workspace(int B, int T, int H, int HV, int dk, int dv, kda_dtype dtype) {
    if (check_shape(B, T, H, HV, dk, dv, dtype) != KDA_OK) return 0;
    return kWsHeader + (use_tc(dk, dv, dtype, T) ? linear_tc_bwd_scratch_bytes(B, T, H, HV, dk, dv, kSms)
                                                 : linear_scan_bwd_scratch_bytes(B, T, H, HV, dk, dv, kSms));
}

kda_status kda_linear_chunk_bwd(const void *q, const void *k, const void *v, const float *decay, int decay_fixed,
                                const float *initial_state, const void *d_o, const float *dfinal_state, void *dq,
                                void *dk_out, void *dv_out, float *ddecay, float *dinitial_state,
                                const long long *strides, int B, int T, int H, int HV, int dk, int dv,
                                kda_dtype dtype, float scale, void *ws, size_t ws_bytes, kda_stream_t stream) {
    kda_status c = check_shape(B, T, H, HV, dk, dv, dtype);
    if (c != KDA_OK) return c;
    const bool some = (long)B * T > 0;
    if (some && (!q || !k || !v || !d_o || !dq || !dk_out || !dv_out)) return KDA_ERR_NULL;
    for (const void *p : {q, k, v, d_o, (const void *)dq, (const void *)dk_out, (const void *)dv_out,
                          (const void *)initial_state, (const void *)dfinal_state, (const void *)dinitial_state})
        if (!al(p, 16)) return KDA_ERR_ALIGN;
    if (!al(decay, 4) || !al(ddecay, 4)) return KDA_ERR_ALIGN;
    LinBwd a{};
    if (!view(a.q, q, strides, 0, B, T, H, dk, dtype) || !view(a.k, k, strides, 1, B, T, H, dk, dtype) ||
        !view(a.v, v, strides, 2, B, T, HV, dv, dtype) || !view(a.d_o, d_o, strides, 3, B, T, HV, dv, dtype) ||
        !view(a.dq, dq, strides, 4, B, T, H, dk, dtype) || !view(a.dk_, dk_out, strides, 5, B, T, H, dk, dtype) ||
        !view(a.dv_, dv_out, strides, 6, B, T, HV, dv, dtype))
        return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_linear_chunk_bwd_workspace(B, T, H, HV, dk, dv, dtype)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    if (B == 0 && !(decay && decay_fixed && ddecay)) return KDA_OK;   // nothing to do: no pointer is touched
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (!some) {   // no token: the memory passes through, and so does its gradient
        if (cudaMemsetAsync(ws, 0, 2 * sizeof(int), st) != cudaSuccess) return KDA_ERR_CUDA;
        if (decay && decay_fixed && ddecay && cudaMemsetAsync(ddecay, 0, (size_t)HV * 4, st) != cudaSuccess)
            return KDA_ERR_CUDA;
        SeqBatch p{};
        p.h0 = dfinal_state; p.hT = dinitial_state; p.nseq = B; p.H = HV; p.dk = dk; p.dv = dv;
        return done(launch_state_passthrough(p, st));
    }
    a.g.p = decay;
    a.g.b = decay_fixed ? 0 : (long long)T * HV;
    a.g.t = decay_fixed ? 0 : HV;
    a.dg = ddecay; a.h0 = initial_state; a.dhT = dfinal_state; a.dh0 = dinitial_state;
    a.B = B; a.T = T; a.H = H; a.HV = HV; a.dk = dk; a.dv = dv;
    a.dtype = to_dtype(dtype); a.scale = pick_scale(scale, dk); a.sms = kSms;
    a.hdr = static_cast<WsHeader *>(ws);
    a.ws = static_cast<char *>(ws) + kWsHeader;
    if (!use_tc(dk, dv, dtype, T)) return done(launch_linear_scan_bwd(a, st));
    return done(launch_linear_tc_bwd(a, st));
}

// ------------------------------------------------------------------------------ norms

static kda_status check_gated(long N, int H, int D, kda_dtype dtype, int act) {
    if (!dtype_ok(dtype)) return KDA_ERR_DTYPE;
    if (N < 0 || H <= 0 || D <= 0 || N > 0x7fffffffffL / H) return KDA_ERR_SHAPE;
    if (D > kGatedNormMax || act < 0 || act > 2) return KDA_ERR_UNSUPPORTED;
    return KDA_OK;
}

static void norm_view(NormView &v, const void *p, const long long *strides, int i, int H, int D) {
    v.p = const_cast<void *>(p);
    v.t = strides ? strides[2 * i] : (long long)H * D;
    v.h = strides ? strides[2 * i + 1] : D;
}

kda_status kda_gated_norm_fwd(const void *x, const void *gate, const float *weight, void *y,
                              const long long *strides, long N, int H, int D, kda_dtype dtype, int activation,
                              float eps, kda_stream_t stream) {
    kda_status c = check_gated(N, H, D, dtype, activation);
    if (c != KDA_OK) return c;
    if (!weight || (N > 0 && (!x || !y || (activation && !gate)))) return KDA_ERR_NULL;
    const unsigned e = dtype == KDA_BF16 ? 2 : 4;
    if (!al(x, e) || !al(gate, e) || !al(y, e) || !al(weight, 4)) return KDA_ERR_ALIGN;
    if (N == 0) return KDA_OK;
    GatedNorm a{};
    norm_view(a.x, x, strides, 0, H, D);
    norm_view(a.g, activation ? gate : nullptr, strides, 1, H, D);
    norm_view(a.y, y, strides, 2, H, D);
    a.w = weight; a.rows = N * H; a.H = H; a.D = D; a.act = activation;
    a.eps = eps; a.inv_d = 1.f / (float)D; a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_gated_norm(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_gated_norm_bwd_workspace(int D) {
    return D > 0 && D <= kGatedNormMax ? (size_t)norm_parts(kSms) * D * 4 : 0;
}

kda_status kda_gated_norm_bwd(const void *d_y, const void *x, const void *gate, const float *weight, void *dx,
                              void *dgate, float *dweight, const long long *strides, long N, int H, int D,
                              kda_dtype dtype, int activation, float eps, void *ws, size_t ws_bytes,
                              kda_stream_t stream) {
    kda_status c = check_gated(N, H, D, dtype, activation);
    if (c != KDA_OK) return c;
    if (!weight || !dweight || (N > 0 && (!d_y || !x || !dx || (activation && (!gate || !dgate))))) return KDA_ERR_NULL;
    const unsigned e = dtype == KDA_BF16 ? 2 : 4;
    if (!al(d_y, e) || !al(x, e) || !al(gate, e) || !al(dx, e) || !al(dgate, e) || !al(weight, 4) || !al(dweight, 4))
        return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_gated_norm_bwd_workspace(D)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) return done(cudaMemsetAsync(dweight, 0, (size_t)D * 4, st));
    GatedNorm a{};
    norm_view(a.x, x, strides, 0, H, D);
    norm_view(a.g, activation ? gate : nullptr, strides, 1, H, D);
    norm_view(a.dy, d_y, strides, 2, H, D);
    norm_view(a.dx, dx, strides, 3, H, D);
    norm_view(a.dg, activation ? dgate : nullptr, strides, 4, H, D);
    a.w = weight; a.dw = dweight; a.part = static_cast<float *>(ws);
    a.rows = N * H; a.H = H; a.D = D; a.act = activation;
    a.eps = eps; a.inv_d = 1.f / (float)D; a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_gated_norm(a, true, st));
}

static kda_status check_residual(long N, int D, kda_dtype res, kda_dtype dtype) {
    if (!dtype_ok(res) || !dtype_ok(dtype) || (res == KDA_BF16 && dtype == KDA_F32)) return KDA_ERR_DTYPE;
    if (N < 0 || D <= 0 || N > 0x7fffffffL) return KDA_ERR_SHAPE;
    return D > kResidualNormMax ? KDA_ERR_UNSUPPORTED : KDA_OK;
}

kda_status kda_residual_norm_fwd(const void *x, const void *y, const float *weight, const float *scale_vec,
                                 float scale, void *x_out, void *n, long long xs, long long ys, long N, int D,
                                 kda_dtype res, kda_dtype dtype, float eps, kda_stream_t stream) {
    kda_status c = check_residual(N, D, res, dtype);
    if (c != KDA_OK) return c;
    if (!weight || (N > 0 && (!x || !y || !x_out || !n))) return KDA_ERR_NULL;
    const unsigned er = res == KDA_BF16 ? 2 : 4, e = dtype == KDA_BF16 ? 2 : 4;
    if (!al(x, er) || !al(x_out, er) || !al(y, e) || !al(n, e) || !al(weight, 4) || !al(scale_vec, 4)) return KDA_ERR_ALIGN;
    if (N == 0) return KDA_OK;
    ResidualNorm a{};
    a.x = x; a.y = y; a.xs = xs; a.ys = ys; a.xo = x_out; a.n = n; a.w = weight; a.cv = scale_vec; a.c = scale;
    a.rows = N; a.D = D; a.eps = eps; a.inv_d = 1.f / (float)D;
    a.res = to_dtype(res); a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_residual_norm(a, false, reinterpret_cast<cudaStream_t>(stream)));
}

size_t kda_residual_norm_bwd_workspace(int D) {
    return D > 0 && D <= kResidualNormMax ? (size_t)norm_parts(kSms) * 2 * D * 4 : 0;
}

kda_status kda_residual_norm_bwd(const void *d_n, const void *d_x_out, const void *x_out, const void *y,
                                 const float *weight, const float *scale_vec, float scale, void *dx, void *dy,
                                 float *dweight, float *dscale, long N, int D, kda_dtype res, kda_dtype dtype,
                                 float eps, void *ws, size_t ws_bytes, kda_stream_t stream) {
    kda_status c = check_residual(N, D, res, dtype);
    if (c != KDA_OK) return c;
    if (!weight || !dweight || (dscale && N > 0 && !y) || (y && !dscale) || (N > 0 && (!d_n || !x_out || !dx || !dy)))
        return KDA_ERR_NULL;
    const unsigned er = res == KDA_BF16 ? 2 : 4, e = dtype == KDA_BF16 ? 2 : 4;
    if (!al(d_x_out, er) || !al(x_out, er) || !al(dx, er) || !al(d_n, e) || !al(y, e) || !al(dy, e) || !al(weight, 4) ||
        !al(scale_vec, 4) || !al(dweight, 4) || !al(dscale, 4))
        return KDA_ERR_ALIGN;
    if (!ws || ws_bytes < kda_residual_norm_bwd_workspace(D)) return KDA_ERR_WORKSPACE;
    if (!al(ws, 16)) return KDA_ERR_ALIGN;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (N == 0) {
        if (cudaMemsetAsync(dweight, 0, (size_t)D * 4, st) != cudaSuccess) return KDA_ERR_CUDA;
        return dscale ? done(cudaMemsetAsync(dscale, 0, (size_t)D * 4, st)) : KDA_OK;
    }
    ResidualNorm a{};
    a.x = x_out; a.y = dscale ? y : nullptr; a.dn = d_n; a.dxo = d_x_out;
    a.xs = a.ys = a.dns = a.dxs = D;
    a.xo = dx; a.n = dy; a.w = weight; a.cv = scale_vec; a.c = scale; a.dw = dweight; a.dc = dscale;
    a.part = static_cast<float *>(ws);
    a.rows = N; a.D = D; a.eps = eps; a.inv_d = 1.f / (float)D;
    a.res = to_dtype(res); a.dtype = to_dtype(dtype); a.sms = kSms;
    return done(launch_residual_norm(a, true, st));
}

}  // extern "C"
