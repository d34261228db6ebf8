// ssm_bwd.cu -- gradients of the state space scan.
//
// With r_t = C_t . h_t + skip x_t, y_t = r_t silu(z_t), u_t = dt_t x_t, a_t = exp(dt_t A), p_t = dy_t silu(z_t):
//     g_t = C_t p_t + a_{t+1} g_{t+1}                      (the gradient of h_t; behind the last token dhT)
//     dC_t = sum_d p_t h_t,    dB_t = sum_d u_t g_t        (over the channels of the group)
//     s_t = g_t . B_t,   e_t = a_t g_t h_{t-1}
//     dx_t = dt_t s_t + skip p_t,   ddt_t = (x_t s_t + sum_n e_t A) softplus'(dt_t),   dz_t = dy_t r_t silu'(z_t)
//     dA = sum_t e_t dt_t,   dskip = sum p_t x_t,   dbias = sum ddt_t,   dh0 = a_1 g_1
//
// Chunks of 32 tokens are independent once the memory before a chunk and the gradient behind it are known, so:
//   1. every chunk by itself, forwards: the memory it leaves from an empty one, what its outputs send to the memory before
//      it, sum_t (a_1 .. a_t) C_t p_t, and the sum of its dt (its decay is exp(A sum dt));
//   2. the two chains over the chunks, one thread per (sequence, channel, state) and direction;
//   3. every chunk again: forwards from its memory, then backwards; dB and dC of up to 128 channels go out as partial sums;
//   4. the partial sums, in a fixed order.
// Per (token, channel, state) that is three exp2 and some 20 fp32 operations, in packed pairs of states, and the sums over
// states and channels; arithmetic and issue bound it.  Measured, bf16, 2 x 2048 tokens of 4096 channels of 16 states, gated: 113 + 32 +
// 385 + 11 us (237 MB, 35 us at the copy rate).
//
// A warp holds 64 / L channels (L = N / 4): a lane two channels and four states, so that sums over states meet over L lanes, in
// shuffles that halve the values at every step (a lane ends with one token's sums), and sums over channels over 32 / L, by columns
// through shared memory.  Memories of a chunk do not fit in registers: every fourth is kept in shared memory, and four tokens at
// a time are walked again from it.
#include <algorithm>

#include "linear_tc.cuh"
#include "run_item.cuh"
#include "ssm_internal.cuh"
#include "ssm_math.cuh"

namespace kda {
namespace {

constexpr int kWarps = 4, kThreads = 32 * kWarps;
constexpr int kTile = 32;                   // tokens of a chunk
constexpr float kLn2F = 0.6931471805599453f;
constexpr int kPartC = 128;                 // floats from the lanes' dB to their dC

template <typename T, int L> struct Lay {
    static constexpr int N = 4 * L, CL = 32 / L, CW = 2 * CL, CH = kWarps * CW;      // states; channel lanes, channels of a warp, of a CTA
    // floats: B and C of the chunk; per warp dt, u, p (each twice, for both channels of a lane), x, dt, dy, z as they came
    // (two channels each), memories kept (but the first), dB and dC
    static constexpr int HEADS = 2 * kTile * N, ROWS = kTile * CL * 12, RAW = kTile * CL * 2 * (int)sizeof(T),
                         KEPT = (kTile / 4 - 1) * 256, SUMS = kTile * 2 * N;
    static constexpr int WARP = ROWS + RAW + KEPT + SUMS;
    static constexpr size_t bytes(bool local) { return (size_t)(HEADS + kWarps * (local ? ROWS : WARP)) * 4; }
};

struct Bwd {
    Ssm a;
    int cpg, bpg, blocks;       // channels and CTAs of a group of heads, CTAs of all
    long chunks;                // (a bound for packed sequences)
    int slots;                  // CTAs that share a block of channels
    long rows;
    float *h, *g, *sums;        // [chunks, D, N] twice, [chunks, D]
    float *bc;                  // [bpg, rows, G, 2 N]
    float *pA, *pd;             // [slots, D, N], [slots, 2, D]
};

__device__ __forceinline__ bool chunk_item(const Bwd &w, long item, LinItem &it) {
    return run_item(w.a.s, w.a.total, kTile, item, it);
}

// Sums over GRP lanes (STRIDE apart) of CNT values each: a step sends one half and keeps the other, so that a lane ends with
// the sums of CNT / GRP values (of one, if there are fewer than lanes: neighbours have the same), from index first() on.
template <int CNT, int GRP, int STRIDE> struct Meet {
    static constexpr int LEFT = CNT > GRP ? CNT / GRP : 1;
    static __device__ __forceinline__ void sum(float (&v)[CNT]) {
        const int lane = threadIdx.x & 31;
        int n = CNT;
#pragma unroll
        for (int off = GRP / 2; off; off >>= 1) {
            if (n > 1) {
                n /= 2;
                const bool up = lane & (off * STRIDE);
#pragma unroll
                for (int i = 0; i < CNT / 2; ++i) {
                    if (i >= n) break;
                    const float send = up ? v[i] : v[i + n], keep = up ? v[i + n] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, send, off * STRIDE);
                }
            } else {
                v[0] += __shfl_xor_sync(0xffffffffu, v[0], off * STRIDE);
            }
        }
    }
    static constexpr int SAME = CNT < GRP ? GRP / CNT : 1;
    static __device__ __forceinline__ int first(int i) { return i / SAME * LEFT; }
    static __device__ __forceinline__ bool lead(int i) { return i % SAME == 0; }      // of the neighbours
};

// Two channels' elements as they lie in memory (n of them are there).  PAIRS: by one access.
template <typename T> struct Raw2 {
    uint32_t w[sizeof(T) / 2];
    __device__ __forceinline__ float operator[](int i) const {
        if constexpr (sizeof(T) == 4)
            return __uint_as_float(w[i]);
        else
            return __uint_as_float(i ? w[0] & 0xffff0000u : w[0] << 16);
    }
};
template <bool PAIRS, typename T> __device__ __forceinline__ Raw2<T> get2(const T *p, int n) {
    Raw2<T> r{};
    if constexpr (PAIRS) {
        if (n > 0) {
            if constexpr (sizeof(T) == 4) {
                const uint2 v = *reinterpret_cast<const uint2 *>(p);
                r.w[0] = v.x, r.w[1] = v.y;
            } else {
                r.w[0] = *reinterpret_cast<const uint32_t *>(p);
            }
        }
    } else if constexpr (sizeof(T) == 4) {
        if (n > 0) r.w[0] = __float_as_uint(p[0]);
        if (n > 1) r.w[1] = __float_as_uint(p[1]);
    } else {
        uint32_t x = 0, y = 0;
        if (n > 0) x = __bfloat16_as_ushort(p[0]);
        if (n > 1) y = __bfloat16_as_ushort(p[1]);
        r.w[0] = x | y << 16;
    }
    return r;
}
template <bool PAIRS, typename T> __device__ __forceinline__ void put2(T *p, int n, float x, float y) {
    if constexpr (PAIRS) {
        if (n <= 0) return;
        if constexpr (sizeof(T) == 4) {
            *reinterpret_cast<float2 *>(p) = make_float2(x, y);
        } else {
            *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(x, y);
        }
    } else {
        if (n > 0) p[0] = from_f32<T>(x);
        if (n > 1) p[1] = from_f32<T>(y);
    }
}

// Where a chunk lies in the arrays.
struct At {
    long b, row;        // batch entry, its first token
    int len;            // tokens of the chunk
};
template <typename T> __device__ __forceinline__ T *rows_at(const SsmView &v, const At &at, int t, long e) {
    return static_cast<T *>(v.p) + at.b * v.b + (at.row + t) * v.t + e;
}

// What both walks read: B and C (all warps together), and the warp's dt, u, p; KEEP: and its rows as they came.  All loads of
// a part go out before the first is used.
template <typename T, int L, bool PAIRS, bool KEEP>
__device__ __forceinline__ void bring(const Bwd &w, const At &at, int g, int d0, int live, float *heads, float *rows, float *raw) {
    using Y = Lay<T, L>;
    const Ssm &a = w.a;
    const int lane = threadIdx.x & 31;
    const int cp = lane % Y::CL, n = live - 2 * cp, tl = lane / Y::CL;
    const long d = d0 + 2 * cp;
    constexpr int U = 32 / L < 8 ? 32 / L : 8;         // tokens of a lane and part
    constexpr int HT = 2 * kTile * L / kThreads;        // quads of states of a thread
    Raw2<T> hq[HT][2];
#pragma unroll
    for (int j = 0; j < HT; ++j) {
        const int i = threadIdx.x + j * kThreads, q = i % L, t = i / L % kTile;
        const SsmView &v = i < kTile * L ? a.B : a.C;
        const T *p = rows_at<const T>(v, at, t, (long)g * v.g + 4 * q);
        hq[j][0] = get2<PAIRS, T>(p, t < at.len ? 2 : 0);
        hq[j][1] = get2<PAIRS, T>(p + 2, t < at.len ? 2 : 0);
    }
    float bias[2] = {0.f, 0.f};
    if (a.bias) {
        if (n > 0) bias[0] = a.bias[d];
        if (n > 1) bias[1] = a.bias[d + 1];
    }
#pragma unroll 1
    for (int t0 = 0; t0 < kTile; t0 += U * L) {
        Raw2<T> dt2[U], x2[U], y2[U], z2[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * L + tl, m = t < at.len ? n : 0;
            dt2[u] = get2<PAIRS, T>(rows_at<const T>(a.dt, at, t, d), m);
            x2[u] = get2<PAIRS, T>(rows_at<const T>(a.x, at, t, d), m);
            y2[u] = get2<PAIRS, T>(rows_at<const T>(a.y, at, t, d), m);
            z2[u] = get2<PAIRS, T>(rows_at<const T>(a.gate, at, t, d), a.gate.p ? m : 0);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int t = t0 + u * L + tl, m = t < at.len ? n : 0;
            float dt[2] = {dt2[u][0] + bias[0], dt2[u][1] + bias[1]}, p[2] = {y2[u][0], y2[u][1]}, rest;
            if (a.softplus) softplus<T>(dt[0], dt[1]);
            if (a.gate.p) {
                p[0] *= z2[u][0] * sigmoid<T>(z2[u][0], rest);
                p[1] *= z2[u][1] * sigmoid<T>(z2[u][1], rest);
            }
            // behind the last token, and in channels that are not there, nothing happens: dt = u = p = 0
            dt[0] = m > 0 ? dt[0] : 0.f, dt[1] = m > 1 ? dt[1] : 0.f;
            const float u0 = m > 0 ? dt[0] * x2[u][0] : 0.f, u1 = m > 1 ? dt[1] * x2[u][1] : 0.f;
            float4 *to = reinterpret_cast<float4 *>(rows) + (t * Y::CL + cp) * 3;
            to[0] = make_float4(dt[0], dt[0], dt[1], dt[1]);
            to[1] = make_float4(u0, u0, u1, u1);
            to[2] = make_float4(p[0], p[0], p[1], p[1]);
            if constexpr (KEEP) {
                Raw2<T> *r = reinterpret_cast<Raw2<T> *>(raw) + (t * Y::CL + cp) * 4;
                if constexpr (sizeof(T) == 2) {
                    *reinterpret_cast<uint4 *>(r) = make_uint4(x2[u].w[0], dt2[u].w[0], y2[u].w[0], z2[u].w[0]);
                } else {
                    reinterpret_cast<uint4 *>(r)[0] = make_uint4(x2[u].w[0], x2[u].w[1], dt2[u].w[0], dt2[u].w[1]);
                    reinterpret_cast<uint4 *>(r)[1] = make_uint4(y2[u].w[0], y2[u].w[1], z2[u].w[0], z2[u].w[1]);
                }
            }
        }
    }
#pragma unroll
    for (int j = 0; j < HT; ++j)        // B's quads, then C's, token by token: the order of the threads
        reinterpret_cast<float4 *>(heads)[threadIdx.x + j * kThreads] = make_float4(hq[j][0][0], hq[j][0][1], hq[j][1][0], hq[j][1][1]);
}

__device__ __forceinline__ Two ex2_2(Two x) {
    float a, b;
    each(x, a, b);
    return two(ex2(a), ex2(b));
}
__device__ __forceinline__ float both(Two x) {
    float a, b;
    each(x, a, b);
    return a + b;
}

// CTA = one chunk, kWarps warps' channels.
template <typename T, int L, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 4) ssm_bwd_local_kernel(const __grid_constant__ Bwd w) {
    using Y = Lay<T, L>;
    extern __shared__ __align__(16) float smem[];
    const Ssm &a = w.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, l = lane % L, cl = lane / L;
    const long item = blockIdx.x / w.blocks;
    const int cb = (int)(blockIdx.x - item * w.blocks), g = cb / w.bpg, c0 = (cb - g * w.bpg) * Y::CH + warp * Y::CW;
    LinItem it;
    if (!chunk_item(w, item, it)) return;
    const int t0 = min(it.p * kTile, it.len);
    const At at{a.s.cu ? 0L : it.n, (a.s.cu ? it.start : 0L) + t0, min(kTile, it.len - t0)};
    const int d0 = g * w.cpg + c0, live = w.cpg - c0;
    float *rows = smem + Y::HEADS + warp * Y::ROWS;
    bring<T, L, PAIRS, false>(w, at, g, d0, live, smem, rows, nullptr);
    __syncthreads();
    Two A[2][2], h[2][2], P[2][2], G[2][2];
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const long d = min(d0 + 2 * cl + c, a.D - 1);
        const float4 x = *reinterpret_cast<const float4 *>(a.A + d * Y::N + 4 * l);
        A[c][0] = two(x.x * kLog2eF, x.y * kLog2eF);
        A[c][1] = two(x.z * kLog2eF, x.w * kLog2eF);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            h[c][k] = G[c][k] = two(0.f, 0.f);
            P[c][k] = two(1.f, 1.f);
        }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll 4
    for (int t = 0; t < kTile; ++t) {
        const ulonglong2 B2 = *reinterpret_cast<const ulonglong2 *>(smem + t * Y::N + 4 * l);
        const ulonglong2 C2 = *reinterpret_cast<const ulonglong2 *>(smem + (t + kTile) * Y::N + 4 * l);
        const ulonglong2 *rp = reinterpret_cast<const ulonglong2 *>(rows) + (t * Y::CL + cl) * 3;
        const ulonglong2 dt2 = rp[0], u2 = rp[1], p2 = rp[2];
        const Two B[2] = {B2.x, B2.y}, C[2] = {C2.x, C2.y}, dt[2] = {dt2.x, dt2.y}, u[2] = {u2.x, u2.y}, p[2] = {p2.x, p2.y};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            float d0, d1;
            each(dt[c], d0, d1);
            sum[c] += d0;
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const Two f = ex2_2(mul2(dt[c], A[c][k]));
                h[c][k] = fma2(f, h[c][k], mul2(u[c], B[k]));
                P[c][k] = mul2(P[c][k], f);
                G[c][k] = fma2(P[c][k], mul2(p[c], C[k]), G[c][k]);
            }
        }
    }
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        if (2 * cl + c >= live) continue;
        const long d = d0 + 2 * cl + c, to = (item * a.D + d) * Y::N + 4 * l;
        *reinterpret_cast<ulonglong2 *>(w.h + to) = make_ulonglong2(h[c][0], h[c][1]);
        *reinterpret_cast<ulonglong2 *>(w.g + to) = make_ulonglong2(G[c][0], G[c][1]);
        if (l == 0) w.sums[item * a.D + d] = sum[c];
    }
}

// One thread per (sequence, channel, state) and direction (blockIdx.y): what a chunk left by itself becomes the memory before
// it, or the gradient behind it.
template <int N> __global__ void __launch_bounds__(256) ssm_bwd_chain_kernel(const __grid_constant__ Bwd w, int seq_blocks) {
    const Ssm &a = w.a;
    const int n = blockIdx.x / seq_blocks;
    const long e = (long)(blockIdx.x - n * seq_blocks) * 256 + threadIdx.x, DN = (long)a.D * N;
    // the sequence's chunks
    long first;
    int cnt;
    if (a.s.cu) {
        const int start = min(max(a.s.cu[n], 0), (int)a.total), len = min(a.s.cu[n + 1], (int)a.total) - start;
        cnt = len > kTile ? (len + kTile - 1) / kTile : 1;
        if (a.s.nseq <= kCounted) {
            __shared__ long s_first;
            if (threadIdx.x < 32) {
                long before = 0;
                for (int k = threadIdx.x; k < n; k += 32) {
                    const int len = (int)min((long)a.s.cu[k + 1] - a.s.cu[k], a.total);
                    before += len > kTile ? (len + kTile - 1) / kTile : 1;
                }
#pragma unroll
                for (int off = 16; off; off >>= 1) before += __shfl_xor_sync(0xffffffffu, before, off);
                if (threadIdx.x == 0) s_first = before;
            }
            __syncthreads();
            first = s_first;
        } else {
            first = first_of_many(a.s, a.total, kTile, n);
        }
        if (first >= w.chunks) return;
        cnt = (int)min((long)cnt, w.chunks - first);
    } else {
        cnt = a.s.T > kTile ? (a.s.T + kTile - 1) / kTile : 1;
        first = (long)n * cnt;
    }
    if (e >= DN) return;
    const bool back = blockIdx.y;
    const float A = a.A[e] * kLog2eF;
    const long d = e / N;
    const float *start = back ? a.dhT : a.h0;
    float v = start ? start[n * DN + e] : 0.f;
    float *arr = (back ? w.g : w.h) + e;
    constexpr int U = 16;
    for (int i0 = 0; i0 < cnt; i0 += U) {
        float x[U], s[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int i = min(i0 + u, cnt - 1);
            const long k = first + (back ? cnt - 1 - i : i);
            x[u] = arr[k * DN];
            s[u] = w.sums[k * a.D + d];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (i0 + u >= cnt) break;
            const long k = first + (back ? cnt - 1 - (i0 + u) : i0 + u);
            arr[k * DN] = v;
            v = fmaf(ex2(s[u] * A), v, x[u]);
        }
    }
    if (back && a.dh0) a.dh0[n * DN + e] = v;
}

template <typename T, int L, bool PAIRS>
__global__ void __launch_bounds__(kThreads, 2) ssm_bwd_grad_kernel(const __grid_constant__ Bwd w) {
    using Y = Lay<T, L>;
    extern __shared__ __align__(16) float smem[];
    const Ssm &a = w.a;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, l = lane % L, cl = lane / L;
    const int slot = blockIdx.x / w.blocks, cb = blockIdx.x - slot * w.blocks, g = cb / w.bpg, cg = cb - g * w.bpg;
    const int c0 = cg * Y::CH + warp * Y::CW, d0 = g * w.cpg + c0, live = w.cpg - c0;
    float *rows = smem + Y::HEADS + warp * Y::WARP, *raw = rows + Y::ROWS, *kept = raw + Y::RAW, *sums = kept + Y::KEPT;
    Two A[2][2], dA[2][2];
    float skip[2], bias[2], dskip[2] = {0.f, 0.f}, dbias[2] = {0.f, 0.f};
    const int n = live - 2 * cl;            // of the lane's two channels those that are there
#pragma unroll
    for (int c = 0; c < 2; ++c) {
        const long d = min(d0 + 2 * cl + c, a.D - 1);
        const float4 x = *reinterpret_cast<const float4 *>(a.A + d * Y::N + 4 * l);
        A[c][0] = two(x.x * kLog2eF, x.y * kLog2eF);
        A[c][1] = two(x.z * kLog2eF, x.w * kLog2eF);
        dA[c][0] = dA[c][1] = two(0.f, 0.f);
        skip[c] = a.skip && c < n ? a.skip[d] : 0.f;
        bias[c] = a.bias && c < n ? a.bias[d] : 0.f;
    }
    for (long item = slot; item < w.chunks; item += w.slots) {
        LinItem it;
        if (!chunk_item(w, item, it)) continue;
        const int t0 = min(it.p * kTile, it.len);
        const At at{a.s.cu ? 0L : it.n, (a.s.cu ? it.start : 0L) + t0, min(kTile, it.len - t0)};
        if (at.len == 0) continue;
        __syncthreads();        // the chunk before has been read
        bring<T, L, PAIRS, true>(w, at, g, d0, live, smem, rows, raw);
        Two h[2][2], G[2][2], start[2][2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const long from = (item * a.D + min(d0 + 2 * cl + c, a.D - 1)) * Y::N + 4 * l;
            ulonglong2 x = make_ulonglong2(0, 0), y = x;
            if (c < n) x = *reinterpret_cast<const ulonglong2 *>(w.h + from), y = *reinterpret_cast<const ulonglong2 *>(w.g + from);
            start[c][0] = h[c][0] = x.x, start[c][1] = h[c][1] = x.y;
            G[c][0] = y.x, G[c][1] = y.y;
        }
        __syncthreads();
        auto heads = [&](int t, Two (&B)[2]) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2 *>(smem + t * Y::N + 4 * l);
            B[0] = x.x, B[1] = x.y;
        };
        auto row = [&](int t, int k) { return *reinterpret_cast<const ulonglong2 *>(rows + ((t * Y::CL + cl) * 3 + k) * 4); };
        // forwards, every fourth memory kept
        for (int q = 0; q < kTile / 4 - 1; ++q) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 4 * q + k;
                Two B[2];
                heads(t, B);
                const ulonglong2 dt = row(t, 0), u = row(t, 1);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    h[0][s] = fma2(ex2_2(mul2(dt.x, A[0][s])), h[0][s], mul2(u.x, B[s]));
                    h[1][s] = fma2(ex2_2(mul2(dt.y, A[1][s])), h[1][s], mul2(u.y, B[s]));
                }
            }
            ulonglong2 *to = reinterpret_cast<ulonglong2 *>(kept) + q * 64 + lane;
            to[0] = make_ulonglong2(h[0][0], h[0][1]);
            to[32] = make_ulonglong2(h[1][0], h[1][1]);
        }
        // backwards, four tokens at a time
#pragma unroll 1
        for (int q = kTile / 4 - 1; q >= 0; --q) {
            if (4 * q >= at.len) continue;          // nothing happens there
            Two was[5][2][2], f[4][2][2];
            was[0][0][0] = start[0][0], was[0][0][1] = start[0][1], was[0][1][0] = start[1][0], was[0][1][1] = start[1][1];
            if (q) {
                const ulonglong2 *from = reinterpret_cast<const ulonglong2 *>(kept) + (q - 1) * 64 + lane;
                const ulonglong2 x = from[0], y = from[32];
                was[0][0][0] = x.x, was[0][0][1] = x.y, was[0][1][0] = y.x, was[0][1][1] = y.y;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = 4 * q + k;
                Two B[2];
                heads(t, B);
                const ulonglong2 dt = row(t, 0), u = row(t, 1);
#pragma unroll
                for (int s = 0; s < 2; ++s) {
                    f[k][0][s] = ex2_2(mul2(dt.x, A[0][s]));
                    f[k][1][s] = ex2_2(mul2(dt.y, A[1][s]));
                    was[k + 1][0][s] = fma2(f[k][0][s], was[k][0][s], mul2(u.x, B[s]));
                    was[k + 1][1][s] = fma2(f[k][1][s], was[k][1][s], mul2(u.y, B[s]));
                }
            }
            float *part = kept + max(q - 1, 0) * 256;       // 2 x 32 lanes x 4 values
            __syncwarp();
            float r[8], sB[8], sA[8];       // token, channel
#pragma unroll
            for (int k = 3; k >= 0; --k) {
                const int t = 4 * q + k;
                Two B[2], C[2];
                heads(t, B);
                heads(t + kTile, C);
                const ulonglong2 dt2 = row(t, 0), u2 = row(t, 1), p2 = row(t, 2);
                const Two dt[2] = {dt2.x, dt2.y}, u[2] = {u2.x, u2.y}, p[2] = {p2.x, p2.y};
                Two dB[2], dC[2];
#pragma unroll
                for (int c = 0; c < 2; ++c) {
                    Two rr, ss, sa;
#pragma unroll
                    for (int s = 0; s < 2; ++s) {
                        const Two now = was[k + 1][c][s];
                        rr = s ? fma2(now, C[s], rr) : mul2(now, C[s]);
                        dC[s] = c ? fma2(now, p[c], dC[s]) : mul2(now, p[c]);
                        G[c][s] = fma2(C[s], p[c], G[c][s]);
                        dB[s] = c ? fma2(G[c][s], u[c], dB[s]) : mul2(G[c][s], u[c]);
                        ss = s ? fma2(G[c][s], B[s], ss) : mul2(G[c][s], B[s]);
                        G[c][s] = mul2(G[c][s], f[k][c][s]);
                        const Two e = mul2(G[c][s], was[k][c][s]);
                        sa = s ? fma2(e, A[c][s], sa) : mul2(e, A[c][s]);
                        dA[c][s] = fma2(e, dt[c], dA[c][s]);
                    }
                    r[2 * k + c] = both(rr);
                    sB[2 * k + c] = both(ss);
                    sA[2 * k + c] = both(sa);
                }
                // over the channels: every lane leaves its eight values, and takes a column of them (the memory that was kept
                // for this part has been read)
                ulonglong2 *to = reinterpret_cast<ulonglong2 *>(part) + lane;
                to[0] = make_ulonglong2(dB[0], dB[1]);
                to[kPartC / 4] = make_ulonglong2(dC[0], dC[1]);
                __syncwarp();
                constexpr int COLS = 8 * L;         // of the warp: B or C, state
#pragma unroll
                for (int j = 0; j < (COLS + 31) / 32; ++j) {
                    const int col = lane + 32 * j, n = col % Y::N;
                    if (COLS >= 32 || col < COLS) {
                        const float *from = part + col / Y::N * kPartC + n;
                        float v[Y::CL];
#pragma unroll
                        for (int i = 0; i < Y::CL; ++i) v[i] = from[(i ^ col / Y::N) * 4 * L];     // dC's in another order: other banks
#pragma unroll
                        for (int half = Y::CL / 2; half; half /= 2)
#pragma unroll
                            for (int i = 0; i < half; ++i) v[i] += v[i + half];
                        sums[t * 2 * Y::N + col] = v[0];
                    }
                }
                __syncwarp();
            }
            using M = Meet<8, L, 1>;
            M::sum(r);
            M::sum(sB);
            M::sum(sA);
            // the lane's tokens: two channels of one or two of them, or one channel
            if (M::lead(l)) {
                constexpr int CNT = M::LEFT;
#pragma unroll
                for (int i = 0; i < CNT; i += 2) {
                    const int j = M::first(l) + i, t = 4 * q + (j >> 1), c1 = CNT == 1 ? (j & 1) : 0;
                    const long d = d0 + 2 * cl + c1;
                    const int m = t < at.len ? (CNT == 1 ? min(n - c1, 1) : n) : 0;
                    const Raw2<T> *rw = reinterpret_cast<const Raw2<T> *>(raw) + (t * Y::CL + cl) * 4;
                    const Raw2<T> x2 = rw[0], dt2 = rw[1], y2 = rw[2], z2 = rw[3];
                    float dx[2], ddt[2], dz[2];
#pragma unroll
                    for (int c = 0; c < (CNT > 1 ? 2 : 1); ++c) {
                        const int ch = CNT == 1 ? c1 : c;
                        const float sk = ch ? skip[1] : skip[0], bi = ch ? bias[1] : bias[0];
                        const float *rp = rows + (t * Y::CL + cl) * 12 + 2 * ch;
                        const float dt = rp[0], p = rp[8], x = ch ? x2[1] : x2[0];
                        float rest = 0.f, slope = 1.f;
                        if (a.softplus) slope = sigmoid<T>((ch ? dt2[1] : dt2[0]) + bi, rest);
                        dx[c] = fmaf(dt, sB[i + c], sk * p);
                        ddt[c] = fmaf(x, sB[i + c], kLn2F * sA[i + c]) * slope;
                        if (a.gate.p) {
                            const float z = ch ? z2[1] : z2[0], sg = sigmoid<T>(z, rest), rr = fmaf(sk, x, r[i + c]);
                            dz[c] = (ch ? y2[1] : y2[0]) * rr * fmaf(z * sg, rest, sg);
                        }
                        if (c < m) {
                            if (ch) {
                                dskip[1] = fmaf(p, x, dskip[1]);
                                dbias[1] += ddt[c];
                            } else {
                                dskip[0] = fmaf(p, x, dskip[0]);
                                dbias[0] += ddt[c];
                            }
                        }
                    }
                    put2<PAIRS && (CNT > 1), T>(rows_at<T>(a.dx, at, t, d), m, dx[0], dx[1]);
                    put2<PAIRS && (CNT > 1), T>(rows_at<T>(a.ddt, at, t, d), m, ddt[0], ddt[1]);
                    if (a.gate.p) put2<PAIRS && (CNT > 1), T>(rows_at<T>(a.dgate, at, t, d), m, dz[0], dz[1]);
                }
            }
        }
        __syncthreads();
        const long row0 = a.s.cu ? at.row : at.b * a.s.T + at.row;
        for (int i = threadIdx.x; i < at.len * 2 * Y::N; i += kThreads) {
            const float *from = smem + Y::HEADS + Y::WARP - Y::SUMS + i;
            constexpr int step = Y::WARP;
            const float v = (from[0] + from[step]) + (from[2 * step] + from[3 * step]);
            const int t = i / (2 * Y::N), k = i % (2 * Y::N);
            w.bc[(((long)cg * w.rows + row0 + t) * a.G + g) * 2 * Y::N + k] = v;
        }
    }
    // the lanes' sums over tokens
#pragma unroll
    for (int c = 0; c < 2; ++c) {
#pragma unroll
        for (int off = 1; off < L; off <<= 1) {
            dskip[c] += __shfl_xor_sync(0xffffffffu, dskip[c], off);
            dbias[c] += __shfl_xor_sync(0xffffffffu, dbias[c], off);
        }
        if (c >= n) continue;
        const long d = d0 + 2 * cl + c;
        *reinterpret_cast<ulonglong2 *>(w.pA + ((long)slot * a.D + d) * Y::N + 4 * l) = make_ulonglong2(dA[c][0], dA[c][1]);
        if (l == 0) {
            w.pd[(long)slot * 2 * a.D + d] = dskip[c];
            w.pd[((long)slot * 2 + 1) * a.D + d] = dbias[c];
        }
    }
}

// dB and dC from the blocks' sums (a thread per value of a token), and the parameters' gradients from the slots'.
template <typename T>
__global__ void __launch_bounds__(256) ssm_bwd_fold_kernel(const __grid_constant__ Bwd w, long bc_blocks) {
    const Ssm &a = w.a;
    if (blockIdx.x < bc_blocks) {
        const long id = (long)blockIdx.x * 256 + threadIdx.x, n2 = (long)a.G * 2 * a.N, all = w.rows * n2;
        if (id >= all) return;
        const long row = id / n2;
        const int e = (int)(id - row * n2);
        if (a.s.cu && (row < a.s.cu[0] || row >= a.s.cu[a.s.nseq])) return;
        float v = 0.f;
        for (int k = 0; k < w.bpg; ++k) v += w.bc[k * all + id];
        const int g = e / (2 * a.N), k = e % (2 * a.N);
        const long b = a.s.cu ? 0 : row / a.s.T, t = a.s.cu ? row : row - b * a.s.T;
        const SsmView &o = k < a.N ? a.dB : a.dC;
        static_cast<T *>(o.p)[b * o.b + t * o.t + g * o.g + k % a.N] = from_f32<T>(v);
        return;
    }
    const long id = (blockIdx.x - bc_blocks) * 256 + threadIdx.x, nA = (long)a.D * a.N;
    if (id >= nA + 2 * a.D) return;
    const float *from = id < nA ? w.pA + id : w.pd + (id - nA);
    const long step = id < nA ? nA : 2L * a.D;
    float v = 0.f;
    for (int s = 0; s < w.slots; ++s) v += from[s * step];
    if (id < nA)
        a.dA[id] = v;
    else if (id < nA + a.D) {
        if (a.dskip) a.dskip[id - nA] = v;
    } else if (a.dbias) {
        a.dbias[id - nA - a.D] = v;
    }
}

// Sizes and places of the scratch.
struct Plan {
    long rows, chunks;
    int cpg, bpg, blocks, slots;
    size_t mem, sums, bc, pA, pd;
};
Plan plan(int nseq, long total, int max_len, bool varlen, int D, int G, int N, int sms) {
    Plan p{};
    const int CH = kWarps * 64 / (N / 4);
    p.rows = varlen ? total : (long)nseq * max_len;
    p.chunks = varlen ? total / kTile + nseq : lin_items(nseq, max_len, max_len, false, kTile);      // as run_items
    p.cpg = D / G;
    p.bpg = (p.cpg + CH - 1) / CH;
    p.blocks = p.bpg * G;
    // four rounds of two CTAs per SM: ends meet, and the parameters' partial sums stay few
    p.slots = (int)std::max(1L, std::min(p.chunks, (8L * sms + p.blocks - 1) / p.blocks));
    p.mem = (size_t)p.chunks * D * N;
    p.sums = ((size_t)p.chunks * D + 3) / 4 * 4;
    p.bc = (size_t)p.bpg * p.rows * G * 2 * N;
    p.pA = (size_t)p.slots * D * N;
    p.pd = (size_t)p.slots * 2 * D;
    return p;
}

template <typename T> bool even(const SsmView &v, bool heads) {
    return !v.p || (reinterpret_cast<uintptr_t>(v.p) % (2 * sizeof(T)) == 0 && v.b % 2 == 0 && v.t % 2 == 0 && (!heads || v.g % 2 == 0));
}

template <typename T, int L, bool PAIRS> cudaError_t run(const Ssm &a, const Plan &p, cudaStream_t st) {
    using Y = Lay<T, L>;
    Bwd w{};
    w.a = a;
    w.cpg = p.cpg, w.bpg = p.bpg, w.blocks = p.blocks, w.chunks = p.chunks, w.slots = p.slots, w.rows = p.rows;
    w.h = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sizeof(WsHeader));
    w.g = w.h + p.mem;
    w.pA = w.g + p.mem;
    w.bc = w.pA + p.pA;
    w.sums = w.bc + p.bc;
    w.pd = w.sums + p.sums;
    const long ctas = p.chunks * p.blocks;
    const int seq_blocks = (int)(((long)a.D * a.N + 255) / 256);
    if (ctas > 0x7fffffffL || (long)a.s.nseq * seq_blocks > 0x7fffffffL) return cudaErrorInvalidValue;
    static lin::SmemOnce local_once, grad_once;
    cudaError_t e = local_once(ssm_bwd_local_kernel<T, L, PAIRS>, (int)Y::bytes(true));
    if (e != cudaSuccess) return e;
    e = grad_once(ssm_bwd_grad_kernel<T, L, PAIRS>, (int)Y::bytes(false));
    if (e != cudaSuccess) return e;
    ssm_bwd_local_kernel<T, L, PAIRS><<<(unsigned)ctas, kThreads, Y::bytes(true), st>>>(w);
    ssm_bwd_chain_kernel<4 * L><<<dim3((unsigned)(a.s.nseq * seq_blocks), 2), 256, 0, st>>>(w, seq_blocks);
    ssm_bwd_grad_kernel<T, L, PAIRS><<<(unsigned)(p.slots * p.blocks), kThreads, Y::bytes(false), st>>>(w);
    const long bc_blocks = (p.rows * a.G * 2 * a.N + 255) / 256, par_blocks = ((long)a.D * (a.N + 2) + 255) / 256;
    ssm_bwd_fold_kernel<T><<<(unsigned)(bc_blocks + par_blocks), 256, 0, st>>>(w, bc_blocks);
    return cudaGetLastError();
}
template <typename T, int L> cudaError_t run(const Ssm &a, cudaStream_t st) {
    const bool varlen = a.s.cu != nullptr;
    const Plan p = plan(a.s.nseq, a.total, varlen ? (int)a.total : a.s.T, varlen, a.D, a.G, a.N, a.sms);
    const bool pairs = p.cpg % 2 == 0 && even<T>(a.x, false) && even<T>(a.dt, false) && even<T>(a.gate, false) && even<T>(a.y, false) &&
                       even<T>(a.B, true) && even<T>(a.C, true) && even<T>(a.dx, false) && even<T>(a.ddt, false) && even<T>(a.dgate, false);
    return pairs ? run<T, L, true>(a, p, st) : run<T, L, false>(a, p, st);
}
template <typename T> cudaError_t go(const Ssm &a, cudaStream_t st) {
    return a.N == 8 ? run<T, 2>(a, st) : a.N == 16 ? run<T, 4>(a, st) : a.N == 32 ? run<T, 8>(a, st) : run<T, 16>(a, st);
}

}  // namespace

size_t ssm_bwd_scratch_bytes(int nseq, long total, int max_len, bool varlen, int D, int G, int N, int sms) {
    const Plan p = plan(nseq, total, max_len, varlen, D, G, N, sms);
    return 4 * (2 * p.mem + p.sums + p.bc + p.pA + p.pd);
}
cudaError_t launch_ssm_bwd(const Ssm &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? go<__nv_bfloat16>(a, st) : go<float>(a, st);
}

}  // namespace kda
