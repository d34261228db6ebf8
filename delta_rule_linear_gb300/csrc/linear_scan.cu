// linear_scan.cu -- linear attention with a decay per head, token by token on CUDA cores:
// the single-token step, the prefill walk for every supported type and shape, and the
// gradients as three such walks.
//
//     h_t = a_t h_{t-1} + k_t v_t^T,     o_t = s h_t^T q_t,      a_t = exp(decay_t)
//
// The memory h [dk, dv] stays in fp32 registers: a warp holds 8 value columns of all dk rows
// (lane l the rows l, l + 32, ...), so the update and the read-out cost 2 dk dv FMAs per token
// and head; the sums over the lanes for the 32 outputs of four tokens are 31 shuffles.  Four warps share
// one staged tile of 16 tokens.
//
// A walk is sequential over its tokens, so a long sequence with few heads is cut into
// segments: a first launch leaves every segment's memory as if it started from zero, and the
// second starts segment p from  sum_{p' < p} (decay of the segments between) local_{p'}, which
// it adds up itself (at most kMaxSegs - 1 reads).
//
// Gradients (D_t = dL/dh_t, collected backwards):
//     dq_t = s h_t do_t                                 = this walk on (q, k, v) := (do, v, k)
//     D_t  = a_{t+1} D_{t+1} + s q_t do_t^T
//     dv_t = D_t^T k_t                                  = the walk backwards on (k, q, do)
//     dk_t = D_t v_t                                    = the walk backwards on (v, do, q)
//     ddecay_t = a_t <h_{t-1}, D_t>
//              = <h_T, dh_T> + sum_{i >= t} (q_i . dq'_i - k_i . dk'_i)
// where ' leaves out token i's own pair: both dots then hold just what crosses token t (a term
// of token i's own pair would have to cancel between them, and under a strong decay it is far
// larger than the result).  The last sum runs in fp64.  A token that keeps nothing (a restart, the first one without an
// initial memory) has 0.
#include <algorithm>

#include "linear_internal.cuh"

namespace kda {
namespace {

// ------------------------------------------------------------------------------ single token
constexpr int kStepThreads = 256;

// One CTA per (request, value head): the [DK, DV] memory crosses HBM once in and once out, as
// 16-byte accesses that are all in flight before the first is used.  Bound by that traffic: 256 requests of
// 32 heads of 128 x 128 take 157 us, 6.9 TB/s, what a plain copy reaches; the arithmetic (3 flops per 4 bytes) is free.
template <typename T, int DK, int DV>
__global__ void __launch_bounds__(kStepThreads) linear_step_kernel(LinDecode a) {
    constexpr int TPR = DV / 4, RG = kStepThreads / TPR;   // threads per row, rows per pass
    constexpr int R = (DK + RG - 1) / RG;
    static_assert(DK % RG == 0, "rows tile the block");
    __shared__ float s_k[DK], s_q[DK];
    __shared__ __align__(16) float s_red[RG][DV];
    const int b = blockIdx.x / a.HV, hv = blockIdx.x % a.HV, hq = hv / (a.HV / a.H);
    const int tid = threadIdx.x, cg = tid % TPR, rg = tid / TPR;
    float *st = a.state + (size_t)blockIdx.x * DK * DV + 4 * cg;
    float4 S[R];
#pragma unroll
    for (int m = 0; m < R; ++m) S[m] = __ldcs(reinterpret_cast<const float4 *>(st + (size_t)(rg + RG * m) * DV));
    for (int i = tid; i < 2 * DK; i += kStepThreads) {
        if (i < DK)
            s_k[i] = to_f32(static_cast<const T *>(a.k.p)[b * a.k.b + hq * a.k.h + i]);
        else
            s_q[i - DK] = a.scale * to_f32(static_cast<const T *>(a.q.p)[b * a.q.b + hq * a.q.h + i - DK]);
    }
    const T *v = static_cast<const T *>(a.v.p) + b * a.v.b + hv * a.v.h + 4 * cg;
    const float v0 = to_f32(v[0]), v1 = to_f32(v[1]), v2 = to_f32(v[2]), v3 = to_f32(v[3]);
    const float al = a.g ? expf(a.g[b * a.gb + hv]) : 1.f;
    __syncthreads();
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int m = 0; m < R; ++m) {
        const int i = rg + RG * m;
        const float kk = s_k[i], qq = s_q[i];
        S[m].x = fmaf(S[m].x, al, kk * v0);
        S[m].y = fmaf(S[m].y, al, kk * v1);
        S[m].z = fmaf(S[m].z, al, kk * v2);
        S[m].w = fmaf(S[m].w, al, kk * v3);
        o.x = fmaf(S[m].x, qq, o.x);
        o.y = fmaf(S[m].y, qq, o.y);
        o.z = fmaf(S[m].z, qq, o.z);
        o.w = fmaf(S[m].w, qq, o.w);
        __stcs(reinterpret_cast<float4 *>(st + (size_t)i * DV), S[m]);
    }
    *reinterpret_cast<float4 *>(&s_red[rg][4 * cg]) = o;
    __syncthreads();
    if (tid < DV) {
        float sum = 0.f;
#pragma unroll
        for (int g = 0; g < RG; ++g) sum += s_red[g][tid];
        static_cast<T *>(const_cast<void *>(a.o.p))[b * a.o.b + hv * a.o.h + tid] = from_f32<T>(sum);
    }
}

// ------------------------------------------------------------------------------ token walk
constexpr int kTile = 16;        // tokens staged at a time
constexpr int kWalkThreads = 128;
constexpr int kCols = 32;        // value columns of a CTA
constexpr int kMaxSegs = 32;     // segments of a sequence (a start state adds up to 31 memories)
constexpr int kMinSeg = 32;      // tokens of a segment at least: 300 tokens, 4 heads of 32 x 64, fp32: 10.3 us, 13.7 with 64

struct Walk {
    LinView q, k, v, x;          // roles; x: the vector of the row dots (or p = nullptr)
    int gq, gk, gv, gx;          // value heads per head of each array
    void *o;                     // output [.., DV] or nullptr
    long long ob, ot, oh;
    int o_f32;                   // the output is fp32 whatever the inputs are
    LinDecay g;
    LinSeqs s;
    int rev;                     // walk the tokens from the last to the first
    int L;                       // tokens per segment
    float add_scale, out_scale;
    const float *h0;
    float *hT;
    long long si, sj;            // strides of h0 and hT: row (q/k channel), column
    int HV, DV;
    float *loc, *gam;            // per (item, head): local memory [DK, DV] and decay factor
    float *rd;                   // partial row dots [DV / 32][rows, HV] or nullptr
    long rows;                   // token rows (stride of rd's slices)
    WsHeader *hdr;               // no kernel here waits, so the first launch clears the error word
};

template <typename T> struct Vec;
template <> struct Vec<float> { static constexpr int N = 4; };
template <> struct Vec<__nv_bfloat16> { static constexpr int N = 8; };
template <typename T> __device__ __forceinline__ void put_vec(float *dst, const uint4 &w) {
    if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<uint4 *>(dst) = w;
    } else {
        float4 lo, hi;
        lo.x = __uint_as_float(w.x << 16); lo.y = __uint_as_float(w.x & 0xffff0000u);
        lo.z = __uint_as_float(w.y << 16); lo.w = __uint_as_float(w.y & 0xffff0000u);
        hi.x = __uint_as_float(w.z << 16); hi.y = __uint_as_float(w.z & 0xffff0000u);
        hi.z = __uint_as_float(w.w << 16); hi.w = __uint_as_float(w.w & 0xffff0000u);
        reinterpret_cast<float4 *>(dst)[0] = lo;
        reinterpret_cast<float4 *>(dst)[1] = hi;
    }
}

// Sums over the warp of x[0 .. N - 1]: half of the values go to the other half of the lanes, and so on; lane l ends with
// that of index l N / 32 in x[0].
template <int N, int LANES>
__device__ __forceinline__ void lane_sums(float *x, int lane) {
    if constexpr (LANES > 1) {
        constexpr int half = LANES / 2, keep = N > 1 ? N / 2 : 1;
        if constexpr (N > 1) {
            const bool up = lane & half;
#pragma unroll
            for (int i = 0; i < keep; ++i) {
                const float mine = up ? x[i + keep] : x[i], send = up ? x[i] : x[i + keep];
                x[i] = mine + __shfl_xor_sync(0xffffffffu, send, half);
            }
        } else {
            x[0] += __shfl_xor_sync(0xffffffffu, x[0], half);
        }
        lane_sums<keep, half>(x, lane);
    }
}

// OUT: the second launch (outputs, final memory); otherwise a segment's local memory.
// A gradient's three walks, in one launch (they are as short as their launches).
struct Walks {
    Walk w[3];
};

template <typename T, int DK, bool OUT, bool RD>
__device__ __forceinline__ void walk_tokens(const Walk &w) {
    constexpr int R = DK / 32, VN = Vec<T>::N;
    constexpr int QV = kTile * DK / VN;                      // 16-byte pieces of a q or k tile
    constexpr int NQ = (QV + kWalkThreads - 1) / kWalkThreads;
    constexpr int VV = kTile * kCols / VN;
    static_assert(VV <= kWalkThreads, "one piece of v per thread");
    __shared__ __align__(16) float s_q[kTile][DK], s_k[kTile][DK], s_v[kTile][kCols],
        s_o[kTile][kCols + 8];                               // rows apart in the banks
    __shared__ float s_a[kTile], s_qk[kTile];

    if constexpr (OUT) wait_for_previous();
    const int nsl = w.DV / kCols, sl = blockIdx.x % nsl, item = blockIdx.x / nsl, hv = blockIdx.y;
    if (blockIdx.x == 0 && hv == 0 && threadIdx.x == 0 && w.hdr) w.hdr->error = 0;
    LinItem it;
    if (!lin_item(w.s, w.L, item, it)) return;
    if (!OUT && it.p == it.nseg - 1) return;                 // nobody reads the last segment's memory
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int col0 = sl * kCols, c0 = col0 + 8 * warp;
    const int u0 = it.p * w.L, u1 = min(it.len, u0 + w.L);
    const int b = w.s.cu ? 0 : it.n;
    const long t_base = w.s.cu ? it.start : 0;               // token index inside batch entry b
    auto tok = [&](int u) { return t_base + (w.rev ? it.len - 1 - u : u); };
    const T *qp = static_cast<const T *>(w.q.p) + b * w.q.b + (hv / w.gq) * w.q.h;
    const T *kp = static_cast<const T *>(w.k.p) + b * w.k.b + (hv / w.gk) * w.k.h;
    const T *vp = static_cast<const T *>(w.v.p) + b * w.v.b + (hv / w.gv) * w.v.h + col0;
    const float *gp = w.g.p ? w.g.p + b * w.g.b + hv : nullptr;

    float h[R][8];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
        for (int c = 0; c < 8; ++c) h[r][c] = 0.f;
    if constexpr (OUT) {
        if (w.h0) {
            const float *p = w.h0 + ((size_t)it.n * w.HV + hv) * DK * w.DV;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < 8; ++c) h[r][c] = p[(lane + 32 * r) * w.si + (c0 + c) * w.sj];
        }
#pragma unroll 4
        for (int pp = 0; pp < it.p; ++pp) {                  // start state of this segment
            const size_t slot = (size_t)(it.first + pp) * w.HV + hv;
            const float ga = w.gam[slot];
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const float4 *l = reinterpret_cast<const float4 *>(w.loc + (slot * DK + lane + 32 * r) * w.DV + c0);
                const float4 x = l[0], y = l[1];
                h[r][0] = fmaf(h[r][0], ga, x.x); h[r][1] = fmaf(h[r][1], ga, x.y);
                h[r][2] = fmaf(h[r][2], ga, x.z); h[r][3] = fmaf(h[r][3], ga, x.w);
                h[r][4] = fmaf(h[r][4], ga, y.x); h[r][5] = fmaf(h[r][5], ga, y.y);
                h[r][6] = fmaf(h[r][6], ga, y.z); h[r][7] = fmaf(h[r][7], ga, y.w);
            }
        }
    }
    // the tile after the current one, in flight
    uint4 rq[NQ], rk[NQ], rv;
    float ra = 0.f;
    auto fetch = [&](int u) {
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int i = tid + j * kWalkThreads, t = i / (DK / VN), e = (i % (DK / VN)) * VN;
            rq[j] = rk[j] = make_uint4(0, 0, 0, 0);
            if (i < QV && u + t < u1) {
                const long row = tok(u + t);
                if (OUT) rq[j] = *reinterpret_cast<const uint4 *>(qp + row * w.q.t + e);
                rk[j] = *reinterpret_cast<const uint4 *>(kp + row * w.k.t + e);
            }
        }
        rv = make_uint4(0, 0, 0, 0);
        if (tid < VV) {
            const int t = tid / (kCols / VN), e = (tid % (kCols / VN)) * VN;
            if (u + t < u1) rv = *reinterpret_cast<const uint4 *>(vp + tok(u + t) * w.v.t + e);
        }
        if (tid < kTile) {
            // the factor before token u's update: its own decay, or (backwards) that of the
            // token visited before it
            const int ud = w.rev ? u + tid - 1 : u + tid;
            ra = (gp && u + tid < u1 && ud >= 0) ? gp[tok(ud) * w.g.t] : 0.f;
        }
    };
    float gsum = 0.f;
    if (u0 < u1) fetch(u0);
    for (int u = u0; u < u1; u += kTile) {
        __syncthreads();
#pragma unroll
        for (int j = 0; j < NQ; ++j) {
            const int i = tid + j * kWalkThreads;
            if (i < QV) {
                if (OUT) put_vec<T>(&s_q[0][0] + i * VN, rq[j]);
                put_vec<T>(&s_k[0][0] + i * VN, rk[j]);
            }
        }
        if (tid < VV) put_vec<T>(&s_v[0][0] + tid * VN, rv);
        if (tid < kTile) {
            s_a[tid] = expf(ra);
            gsum += ra;
        }
        __syncthreads();
        if (u + kTile < u1) fetch(u + kTile);
        const int nt = min(kTile, u1 - u);
        // four tokens at a time (rows past the segment are staged as zeros): their updates are a chain of one FMA
        // each, and their 32 outputs are summed over the lanes together, a shuffle for each
#pragma unroll 1
        for (int t0 = 0; t0 < nt; t0 += 4) {
            float acc[32], qk[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int t = t0 + j;
                const float a = s_a[t];
                float vv[8], kk[R];
                *reinterpret_cast<float4 *>(vv) = *reinterpret_cast<const float4 *>(&s_v[t][8 * warp]);
                *reinterpret_cast<float4 *>(vv + 4) = *reinterpret_cast<const float4 *>(&s_v[t][8 * warp + 4]);
#pragma unroll
                for (int r = 0; r < R; ++r) kk[r] = w.add_scale * s_k[t][lane + 32 * r];
                if constexpr (!OUT) {
#pragma unroll
                    for (int r = 0; r < R; ++r)
#pragma unroll
                        for (int c = 0; c < 8; ++c) h[r][c] = fmaf(h[r][c], a, kk[r] * vv[c]);
                } else {
#pragma unroll
                    for (int c = 0; c < 8; ++c) acc[8 * j + c] = 0.f;
                    qk[j] = 0.f;
#pragma unroll
                    for (int r = 0; r < R; ++r) {
                        const float qq = s_q[t][lane + 32 * r];
                        if constexpr (RD) qk[j] = fmaf(qq, kk[r], qk[j]);
#pragma unroll
                        for (int c = 0; c < 8; ++c) {
                            if constexpr (RD) {
                                h[r][c] *= a;
                                acc[8 * j + c] = fmaf(h[r][c], qq, acc[8 * j + c]);
                                h[r][c] = fmaf(kk[r], vv[c], h[r][c]);
                            } else {
                                h[r][c] = fmaf(h[r][c], a, kk[r] * vv[c]);
                                acc[8 * j + c] = fmaf(h[r][c], qq, acc[8 * j + c]);
                            }
                        }
                    }
                }
            }
            if constexpr (OUT) {
                lane_sums<32, 32>(acc, lane);                // lane l: token l / 8, column l % 8
                s_o[t0 + (lane >> 3)][8 * warp + (lane & 7)] = acc[0] * w.out_scale;
                if constexpr (RD) {
                    if (((t0 >> 2) & 3) == warp) {           // all warps hold q and k: they take turns
                        lane_sums<4, 32>(qk, lane);          // lanes 8 j and on: token j
                        if ((lane & 7) == 0) s_qk[t0 + (lane >> 3)] = qk[0] * w.out_scale;
                    }
                }
            }
        }
        if constexpr (OUT) {
            __syncthreads();
            if constexpr (RD) {
                // x . (output without the token's own pair), this CTA's 32 columns
                const int t = tid >> 3, e = (tid & 7) * 4;
                float d = 0.f;
                if (w.rd && t < nt) {
                    const T *xp = static_cast<const T *>(w.x.p) + b * w.x.b + (hv / w.gx) * w.x.h +
                                  tok(u + t) * w.x.t + col0 + e;
#pragma unroll
                    for (int j = 0; j < 4; ++j) d = fmaf(to_f32(xp[j]), s_o[t][e + j], d);
                }
#pragma unroll
                for (int off = 4; off; off >>= 1) d += __shfl_xor_sync(0xffffffffu, d, off);
                if (w.rd && t < nt && (tid & 7) == 0)
                    w.rd[(size_t)sl * w.rows * w.HV + ((size_t)(w.s.cu ? 0 : (long)it.n * w.s.T) + tok(u + t)) * w.HV +
                         hv] = d;
            }
            static_assert(kTile * kCols == 4 * kWalkThreads, "four columns to a thread");
            if (const int t = tid >> 3, c = (tid & 7) * 4; t < nt) {
                float4 val = *reinterpret_cast<const float4 *>(&s_o[t][c]);
                if constexpr (RD) {
                    const float4 vv = *reinterpret_cast<const float4 *>(&s_v[t][c]);
                    const float d = s_qk[t];
                    val.x = fmaf(d, vv.x, val.x); val.y = fmaf(d, vv.y, val.y);
                    val.z = fmaf(d, vv.z, val.z); val.w = fmaf(d, vv.w, val.w);
                }
                const long long off = b * w.ob + tok(u + t) * w.ot + hv * w.oh + col0 + c;
                if (sizeof(T) == 4 || w.o_f32)
                    *reinterpret_cast<float4 *>(static_cast<float *>(w.o) + off) = val;
                else {
                    const __nv_bfloat162 p[2] = {__floats2bfloat162_rn(val.x, val.y), __floats2bfloat162_rn(val.z, val.w)};
                    *reinterpret_cast<uint2 *>(static_cast<T *>(w.o) + off) = *reinterpret_cast<const uint2 *>(p);
                }
            }
        }
    }
    if constexpr (OUT) {
        if (w.hT && it.p == it.nseg - 1) {
            // backwards, the first token's own decay is still due
            const float a = (w.rev && gp && it.len > 0) ? expf(gp[tok(it.len - 1) * w.g.t]) : 1.f;
            float *p = w.hT + ((size_t)it.n * w.HV + hv) * DK * w.DV;
#pragma unroll
            for (int r = 0; r < R; ++r)
#pragma unroll
                for (int c = 0; c < 8; ++c) p[(lane + 32 * r) * w.si + (c0 + c) * w.sj] = a * h[r][c];
        }
    } else {
        const size_t slot = (size_t)item * w.HV + hv;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            float4 *l = reinterpret_cast<float4 *>(w.loc + (slot * DK + lane + 32 * r) * w.DV + c0);
            l[0] = make_float4(h[r][0], h[r][1], h[r][2], h[r][3]);
            l[1] = make_float4(h[r][4], h[r][5], h[r][6], h[r][7]);
        }
        if (sl == 0 && warp == 0) {
#pragma unroll
            for (int off = 16; off; off >>= 1) gsum += __shfl_xor_sync(0xffffffffu, gsum, off);
            if (lane == 0) w.gam[slot] = expf(gsum);
        }
    }
}

template <typename T, int DK, bool OUT, bool RD>
__global__ void __launch_bounds__(kWalkThreads) linear_walk_kernel(const __grid_constant__ Walks ws) {
    walk_tokens<T, DK, OUT, RD>(ws.w[blockIdx.z]);
}
// A gradient's walks where dk and dv differ: two with rows of DKA channels, the third with DKB.  One launch of these,
// whose CTAs run side by side: apart, with 301 tokens and 4 heads in fp32, each pair of launches takes 26 us.
template <typename T, int DKA, int DKB, bool OUT>
__global__ void __launch_bounds__(kWalkThreads) linear_walk3_kernel(const __grid_constant__ Walks ws) {
    if (blockIdx.z < 2)
        walk_tokens<T, DKA, OUT, OUT>(ws.w[blockIdx.z]);
    else
        walk_tokens<T, DKB, OUT, false>(ws.w[2]);
}

// Tokens per segment.  Whole sequences as long as they give every SM six CTAs (what hides the
// walk's latency); otherwise as many segments as get there, none below kMinSeg tokens.  A sequence of up to
// four of those is not cut: the second launch costs the host more than it saves (128 tokens, 4 heads
// of 64, fp32: a call takes 20.8 us, cut 24.5; replayed in a graph 17.3 and 13.3).
int walk_segment(int nseq, int HV, int nsl, long total, int max_len, bool varlen, int sms) {
    const long ctas = (long)nseq * HV * nsl, want = 6L * sms;
    if (max_len <= 4 * kMinSeg || ctas >= want) return std::max(max_len, 1);
    const long tokens = varlen ? total : (long)nseq * max_len;
    const long segs = std::max(1L, want / ((long)HV * nsl));
    long L = (tokens + segs - 1) / segs;
    L = std::max(L, (long)(max_len + kMaxSegs - 1) / kMaxSegs);
    L = std::max(L, (long)kMinSeg);
    return (int)((L + kTile - 1) / kTile * kTile);
}

// The segments' memories where there are several, and the outputs
cudaError_t run_pair(void (*local)(Walks), void (*out)(Walks), bool cut, dim3 grid, const Walks &ws, cudaStream_t st) {
    if (!cut) {
        out<<<grid, kWalkThreads, 0, st>>>(ws);
        return cudaGetLastError();
    }
    local<<<grid, kWalkThreads, 0, st>>>(ws);
    const cudaError_t e = cudaGetLastError();
    return e == cudaSuccess ? launch_after(out, grid, kWalkThreads, 0, st, ws) : e;
}

template <typename T, int DK>
cudaError_t run_walk_t(const Walk &w, long items, int max_len, cudaStream_t st) {
    const int nsl = w.DV / kCols;
    if (items * nsl > 0x7fffffffL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)(items * nsl), (unsigned)w.HV);
    Walks ws{};
    ws.w[0] = w;
    return run_pair(linear_walk_kernel<T, DK, false, false>, linear_walk_kernel<T, DK, true, false>, max_len > w.L, grid,
                    ws, st);
}
template <typename T>
cudaError_t run_walk(const Walk &w, int DK, long items, int max_len, cudaStream_t st) {
    switch (DK) {
        case 32: return run_walk_t<T, 32>(w, items, max_len, st);
        case 64: return run_walk_t<T, 64>(w, items, max_len, st);
        default: return run_walk_t<T, 128>(w, items, max_len, st);
    }
}

// The walks of a gradient, equal lengths: ws.w[0] and [1] with rows of DKA channels, [2] with DKB.  Where the
// three share one kernel, the one without row dots has a null pointer for them.
template <typename T, int DKA, int DKB>
cudaError_t run_walks_t(const Walks &ws, int T_len, cudaStream_t st) {
    long x = 0;
    bool cut = false;
    for (const Walk &w : ws.w) {
        x = std::max(x, lin_items(w.s.nseq, T_len, T_len, false, w.L) * (w.DV / kCols));
        cut = cut || T_len > w.L;
    }
    if (x > 0x7fffffffL) return cudaErrorInvalidValue;
    const dim3 grid((unsigned)x, (unsigned)ws.w[0].HV, 3);
    if constexpr (DKA == DKB)
        return run_pair(linear_walk_kernel<T, DKA, false, false>, linear_walk_kernel<T, DKA, true, true>, cut, grid, ws, st);
    else
        return run_pair(linear_walk3_kernel<T, DKA, DKB, false>, linear_walk3_kernel<T, DKA, DKB, true>, cut, grid, ws, st);
}
template <typename T, int DKA>
cudaError_t run_walks_b(const Walks &ws, int DKB, int T_len, cudaStream_t st) {
    switch (DKB) {
        case 32: return run_walks_t<T, DKA, 32>(ws, T_len, st);
        case 64: return run_walks_t<T, DKA, 64>(ws, T_len, st);
        default: return run_walks_t<T, DKA, 128>(ws, T_len, st);
    }
}
template <typename T>
cudaError_t run_walks(const Walks &ws, int DKA, int DKB, int T_len, cudaStream_t st) {
    switch (DKA) {
        case 32: return run_walks_b<T, 32>(ws, DKB, T_len, st);
        case 64: return run_walks_b<T, 64>(ws, DKB, T_len, st);
        default: return run_walks_b<T, 128>(ws, DKB, T_len, st);
    }
}

// ------------------------------------------------------------------------------ reductions
// ddecay from the row dots: one CTA per (batch entry, value head); every thread sums a run of
// tokens, the runs' sums are scanned from the end, and the runs are walked again.
constexpr int kGradThreads = 256;
struct Dgate {
    const float *rq, *rk;        // row dots, n slices each
    int n;
    const float *hT, *dhT;       // final memory and its gradient (or nullptr)
    LinDecay g;
    int h0;                      // there is an initial memory
    float *dg;
    int T, HV, cells;
    long rows;
};
__device__ __forceinline__ void sum_dgate(const Dgate &d, int pair) {
    __shared__ double s_run[kGradThreads / 32], s_anchor[kGradThreads / 32];
    const int b = pair / d.HV, hv = pair % d.HV, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t slice = (size_t)d.rows * d.HV;
    auto at = [&](int t) {
        const size_t i = ((size_t)b * d.T + t) * d.HV + hv;
        double x = 0.0;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (j < d.n) x += (double)__ldg(d.rq + j * slice + i) - (double)__ldg(d.rk + j * slice + i);
        return x;
    };
    const int run = (d.T + kGradThreads - 1) / kGradThreads, t0 = min(d.T, tid * run), t1 = min(d.T, t0 + run);
    double mine = 0.0, anchor = 0.0;
#pragma unroll 2
    for (int t = t0; t < t1; ++t) mine += at(t);
    if (d.dhT) {
        const float *p = d.hT + (size_t)pair * d.cells, *q = d.dhT + (size_t)pair * d.cells;
#pragma unroll 8
        for (int i = tid; i < d.cells; i += kGradThreads) anchor += (double)__ldg(p + i) * __ldg(q + i);
#pragma unroll
        for (int off = 16; off; off >>= 1) anchor += __shfl_xor_sync(0xffffffffu, anchor, off);
    }
    double sum = mine;                                       // over this and the warp's later runs
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const double x = __shfl_down_sync(0xffffffffu, sum, off);
        if (lane + off < 32) sum += x;
    }
    if (lane == 0) {
        s_run[warp] = sum;
        s_anchor[warp] = anchor;
    }
    __syncthreads();
    double acc = sum - mine;
#pragma unroll
    for (int i = 0; i < kGradThreads / 32; ++i) acc += s_anchor[i] + (i > warp ? s_run[i] : 0.0);
    const float *gp = d.g.p + b * d.g.b + hv;
    for (int t = t1 - 1; t >= t0; --t) {
        acc += at(t);
        // where nothing is kept the sum's terms cancel, all but their rounding
        const bool kept = (t > 0 || d.h0) && !(gp[(long long)t * d.g.t] < kMinDecay);
        d.dg[((size_t)b * d.T + t) * d.HV + hv] = kept ? (float)acc : 0.f;
    }
}

// The value heads of a shared q/k head added up: two arrays
struct Fold {
    const float *src[2];         // [rows, H, m, D]
    LinView dst[2];
    long n;                      // elements of a result
    int T, H, m, D;
};
template <typename T>
__device__ __forceinline__ void fold_heads(const Fold &f, int which, long first, long step) {
    const float *src = f.src[which];
    const LinView &dst = f.dst[which];
    for (long i = first; i < f.n; i += step) {
        const int c = (int)(i % f.D);
        const long rh = i / f.D;
        const int h = (int)(rh % f.H);
        const long row = rh / f.H;
        float sum = 0.f;
        for (int j = 0; j < f.m; ++j) sum += src[((row * f.H + h) * f.m + j) * f.D + c];
        static_cast<T *>(const_cast<void *>(dst.p))[(row / f.T) * dst.b + (row % f.T) * dst.t + h * dst.h + c] =
            from_f32<T>(sum);
    }
}
// What follows a gradient's walks, in one launch: the first CTAs take ddecay, the others the shared heads.
template <typename T>
__global__ void __launch_bounds__(kGradThreads) linear_tail_kernel(Dgate d, int pairs, Fold f) {
    wait_for_previous();
    if ((int)blockIdx.x < pairs) {
        sum_dgate(d, blockIdx.x);
        return;
    }
    const int at = blockIdx.x - pairs, per = (gridDim.x - pairs) / 2;
    fold_heads<T>(f, at >= per, (long)(at % per) * kGradThreads + threadIdx.x, (long)per * kGradThreads);
}
cudaError_t run_tail(const Dgate &d, int pairs, const Fold &f, DType dt, cudaStream_t st) {
    const long grid = pairs + 2 * std::min(2048L, (f.n + kGradThreads - 1) / kGradThreads);
    if (grid == 0) return cudaSuccess;
    return launch_after(dt == DType::BF16 ? linear_tail_kernel<__nv_bfloat16> : linear_tail_kernel<float>, (unsigned)grid,
                        kGradThreads, 0, st, d, pairs, f);
}

// dst[c] = sum over the rows of src[r, c]: one CTA per column, a fixed order, fp64 sums (a
// fixed decay's gradient adds up every token of the batch).
__global__ void __launch_bounds__(256) sum_rows_kernel(const float *src, float *dst, long rows, int cols) {
    __shared__ double s[256];
    wait_for_previous();
    double d = 0.0;
    for (long r = threadIdx.x; r < rows; r += 256) d += src[r * cols + blockIdx.x];
    s[threadIdx.x] = d;
    __syncthreads();
    for (int off = 128; off; off >>= 1) {
        if (threadIdx.x < off) s[threadIdx.x] += s[threadIdx.x + off];
        __syncthreads();
    }
    if (threadIdx.x == 0) dst[blockIdx.x] = (float)s[0];
}

size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

// bytes of the segment memories (and their decay factors) of one walk
size_t walk_scratch(int nseq, int HV, int dk, int dv, long total, int max_len, bool varlen, int L) {
    if (max_len <= L) return 0;
    const size_t slots = (size_t)lin_items(nseq, total, max_len, varlen, L) * HV;
    return round256(slots * dk * dv * 4) + round256(slots * 4);
}

}  // namespace

size_t linear_scan_scratch_bytes(int nseq, int HV, int dk, int dv, long total, int max_len, bool varlen, int sms) {
    if (varlen) {   // whatever the lengths turn out to be: the shortest segments the total allows
        const long ctas = (long)nseq * HV * (dv / kCols), want = 6L * sms;
        if (total <= 4 * kMinSeg || ctas >= want) return 0;
        const long L = walk_segment(nseq, HV, dv / kCols, total, 4 * kMinSeg + 1, true, sms);
        const size_t slots = (size_t)(total / L + nseq) * HV;
        return round256(slots * dk * dv * 4) + round256(slots * 4);
    }
    return walk_scratch(nseq, HV, dk, dv, total, max_len, varlen,
                        walk_segment(nseq, HV, dv / kCols, total, max_len, varlen, sms));
}

cudaError_t launch_linear_scan(const LinFwd &a, cudaStream_t st) {
    Walk w{};
    const bool varlen = a.s.cu != nullptr;
    const int m = a.HV / a.H;
    w.q = a.q; w.k = a.k; w.v = a.v;
    w.gq = w.gk = m; w.gv = w.gx = 1;
    w.o = const_cast<void *>(a.o.p); w.ob = a.o.b; w.ot = a.o.t; w.oh = a.o.h;
    w.g = a.g; w.s = a.s; w.hdr = a.hdr;
    w.add_scale = 1.f; w.out_scale = a.scale;
    w.h0 = a.h0; w.hT = a.hT; w.si = a.dv; w.sj = 1;
    w.HV = a.HV; w.DV = a.dv;
    // in place (h_T over h_0) every CTA must own its memory: no segments
    w.L = a.h0 && a.h0 == a.hT ? std::max(a.max_len, 1)
                                : walk_segment(a.s.nseq, a.HV, a.dv / kCols, a.total, a.max_len, varlen, a.sms);
    const long items = lin_items(a.s.nseq, a.total, a.max_len, varlen, w.L);
    w.loc = static_cast<float *>(a.ws);
    w.gam = reinterpret_cast<float *>(static_cast<char *>(a.ws) + round256((size_t)items * a.HV * a.dk * a.dv * 4));
    return a.dtype == DType::BF16 ? run_walk<__nv_bfloat16>(w, a.dk, items, a.max_len, st)
                                  : run_walk<float>(w, a.dk, items, a.max_len, st);
}

cudaError_t launch_fold_heads(const float *src0, const LinView &dst0, const float *src1, const LinView &dst1, DType dt,
                              int B, int T, int H, int m, int D, cudaStream_t st) {
    return run_tail(Dgate{}, 0, Fold{{src0, src1}, {dst0, dst1}, (long)B * T * H * D, T, H, m, D}, dt, st);
}

cudaError_t launch_sum_rows(const float *src, float *dst, long rows, int cols, cudaStream_t st) {
    return launch_after(sum_rows_kernel, cols, 256, 0, st, src, dst, rows, cols);
}

// Scratch of the gradients: [h_T][row dots of dq and dk][per-token ddecay when it is summed]
// [per-value-head dq, dk when heads are shared][segment memories of the three walks]
size_t linear_scan_bwd_scratch_bytes(int B, int T, int H, int HV, int dk, int dv, int sms) {
    size_t n = 0;
    const int dims[3][2] = {{dv, dk}, {dv, dk}, {dk, dv}};
    for (auto &d : dims)
        n += walk_scratch(B, HV, d[0], d[1], T, T, false, walk_segment(B, HV, d[1] / kCols, T, T, false, sms));
    const size_t rows = (size_t)B * T * HV;
    n += round256((size_t)B * HV * dk * dv * 4) + 2 * round256(rows * (dk / kCols) * 4) + round256(rows * 4);
    if (HV > H) n += 2 * round256(rows * dk * 4);
    return n;
}

cudaError_t launch_linear_scan_bwd(const LinBwd &a, cudaStream_t st) {
    const int m = a.HV / a.H;
    const size_t rows = (size_t)a.B * a.T * a.HV;
    char *p = static_cast<char *>(a.ws);
    auto carve = [&](size_t n) { char *r = p; p += round256(n); return reinterpret_cast<float *>(r); };
    float *hT = carve((size_t)a.B * a.HV * a.dk * a.dv * 4);
    float *rq = carve(rows * (a.dk / kCols) * 4), *rk = carve(rows * (a.dk / kCols) * 4);
    float *dgt = carve(rows * 4);
    float *fq = nullptr, *fk = nullptr;
    if (m > 1) {
        fq = carve(rows * a.dk * 4);
        fk = carve(rows * a.dk * 4);
    }
    const bool want_g = a.g.p && a.dg;
    auto walk = [&](int DK, int DV, const LinView &out, float *f32out) {
        Walk w{};
        w.hdr = a.hdr;
        w.g = a.g; w.s.nseq = a.B; w.s.T = a.T; w.HV = a.HV;
        w.rows = (long)a.B * a.T;
        w.DV = DV;
        w.L = walk_segment(a.B, a.HV, DV / kCols, a.T, a.T, false, a.sms);
        const size_t need = walk_scratch(a.B, a.HV, DK, DV, a.T, a.T, false, w.L);
        if (need) {
            const size_t slots = (size_t)lin_items(a.B, a.T, a.T, false, w.L) * a.HV;
            w.loc = carve(slots * DK * DV * 4);
            w.gam = carve(slots * 4);
        }
        w.o_f32 = f32out != nullptr;
        w.o = f32out ? static_cast<void *>(f32out) : const_cast<void *>(out.p);
        w.ob = f32out ? (long long)a.T * a.HV * DV : out.b;
        w.ot = f32out ? (long long)a.HV * DV : out.t;
        w.oh = f32out ? DV : out.h;
        return w;
    };
    Walks ws{};
    // dq: forwards on (do, v, k); memory transposed, [dv, dk]
    Walk &wq = ws.w[0] = walk(a.dv, a.dk, a.dq, fq);
    wq.q = a.d_o; wq.gq = 1; wq.k = a.v; wq.gk = 1; wq.v = a.k; wq.gv = m;
    wq.x = a.q; wq.gx = m; wq.rd = want_g ? rq : nullptr;
    wq.add_scale = 1.f; wq.out_scale = a.scale;
    wq.h0 = a.h0; wq.hT = want_g && a.dhT ? hT : nullptr; wq.si = 1; wq.sj = a.dv;
    // dk: backwards on (v, do, q), memory [dv, dk]
    Walk &wk = ws.w[1] = walk(a.dv, a.dk, a.dk_, fk);
    wk.rev = 1;
    wk.q = a.v; wk.gq = 1; wk.k = a.d_o; wk.gk = 1; wk.v = a.q; wk.gv = m;
    wk.x = a.k; wk.gx = m; wk.rd = want_g ? rk : nullptr;
    wk.add_scale = a.scale; wk.out_scale = 1.f;
    wk.h0 = a.dhT; wk.si = 1; wk.sj = a.dv;
    // dv: backwards on (k, q, do), memory [dk, dv]; its final memory is the initial one's gradient
    Walk &wv = ws.w[2] = walk(a.dk, a.dv, a.dv_, nullptr);
    wv.rev = 1;
    wv.q = a.k; wv.gq = m; wv.k = a.q; wv.gk = m; wv.v = a.d_o; wv.gv = wv.gx = 1;
    wv.add_scale = a.scale; wv.out_scale = 1.f;
    wv.h0 = a.dhT; wv.hT = a.dh0; wv.si = a.dv; wv.sj = 1;
    cudaError_t e = a.dtype == DType::BF16 ? run_walks<__nv_bfloat16>(ws, a.dv, a.dk, a.T, st)
                                           : run_walks<float>(ws, a.dv, a.dk, a.T, st);
    if (e != cudaSuccess) return e;
    const bool fixed = a.g.t == 0;
    Dgate d{rq, rk, a.dk / kCols, hT, a.dhT, a.g, a.h0 != nullptr, fixed ? dgt : a.dg, a.T, a.HV, a.dk * a.dv, (long)a.B * a.T};
    Fold f{};
    if (m > 1) f = Fold{{fq, fk}, {a.dq, a.dk_}, (long)a.B * a.T * a.H * a.dk, a.T, a.H, m, a.dk};
    e = run_tail(d, want_g ? a.B * a.HV : 0, f, a.dtype, st);
    if (e == cudaSuccess && want_g && fixed) e = launch_sum_rows(dgt, a.dg, (long)a.B * a.T, a.HV, st);
    return e;
}

namespace {
template <typename T, int DK>
cudaError_t step_dv(const LinDecode &a, cudaStream_t st) {
    const unsigned grid = (unsigned)(a.B * a.HV);
    switch (a.dv) {
        case 32: linear_step_kernel<T, DK, 32><<<grid, kStepThreads, 0, st>>>(a); break;
        case 64: linear_step_kernel<T, DK, 64><<<grid, kStepThreads, 0, st>>>(a); break;
        default: linear_step_kernel<T, DK, 128><<<grid, kStepThreads, 0, st>>>(a); break;
    }
    return cudaGetLastError();
}
template <typename T>
cudaError_t step_dk(const LinDecode &a, cudaStream_t st) {
    return a.dk == 32 ? step_dv<T, 32>(a, st) : a.dk == 64 ? step_dv<T, 64>(a, st) : step_dv<T, 128>(a, st);
}
}  // namespace

cudaError_t launch_linear_decode(const LinDecode &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? step_dk<__nv_bfloat16>(a, st) : step_dk<float>(a, st);
}

}  // namespace kda
