// beam.cu -- beam search: the k best continuations of a request's W beams, and the recurrent memories that follow them.
//
// Selection: total[w, v] = score_w + x_w[v] - lse_w, lse_w = log sum_v exp(x_w[v]); the k largest over all (w, v), ties to
// the lowest w V + v.  The logits are read once: a warp takes 1024 consecutive ones at a time, keeps the maxima of their
// two chunks of 512 and adds up exp(x - M) against the running maximum M of its chunks.  An element among the k best lies in one of the k
// chunks that come first when chunks are ordered by (maximum, position): every chunk before its own holds an element that
// comes before it.  So the second kernel, a CTA per request, orders the chunks' maxima and looks at k chunks only.
// Totals are compared as pairs of fp32, 48 bits: tokens of a beam, and of beams with equal rows, may be closer than an fp32 total's
// rounding.  Sums of exp are fp32 over a warp's terms (approximate exp2 of exponents rounded to fp32) and 64-bit from there on:
// lse is good to some 3e-7 (131,072 normal logits), so far are other beams told apart.
//
// Measured: 64 requests of 8 beams over 131,072 bf16 logits 23 us (134 MB, 19.8 us at the copy rate) and 15 us for the second kernel, whose
// small steps wait for one another; 35 us together.
//
// Reordering in place: a thread holds one 16-byte column of all W beams of a request, reads what the moved beams take
// and then writes it, so no beam is overwritten before it has been read and nothing is copied aside.
#include <algorithm>

#include "beam_internal.cuh"
#include "pack.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kPickThreads = 512, kPickWarps = kPickThreads / 32;

template <typename T> __device__ __forceinline__ const T *row_of(const BeamSelect &a, int b, int w) {
    return static_cast<const T *>(a.logits) + b * a.sb + w * a.sw;
}

// V consecutive elements from e on, p + e on a 16-byte boundary: those outside [0, n) count as -inf and are not touched.
template <typename T, int V> __device__ __forceinline__ uint4 get_some(const T *p, long e, long n) {
    if (e >= 0 && e + V <= n) return *reinterpret_cast<const uint4 *>(p + e);
    uint32_t u[4] = {};
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const T x = e + i >= 0 && e + i < n ? p[e + i] : from_f32<T>(-INFINITY);
        if constexpr (sizeof(T) == 4)
            u[i] = __float_as_uint(x);
        else
            u[i / 2] |= (uint32_t)__bfloat16_as_ushort(x) << 16 * (i & 1);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
}

// The 16 bytes that begin `bytes` (0 .. 15, a multiple of the element) into the 32 of lo and hi.
__device__ __forceinline__ uint4 from_byte(uint4 lo, uint4 hi, int bytes) {
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    if (bytes & 8) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (bytes & 4) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const int bits = (bytes & 3) * 8;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

// 1024 elements of a row, 16 bytes per lane and i: elements j 1024 + (32 i + lane) V on, whatever the row's address is, so that
// equal rows give equal sums.  A row off the 16-byte boundary is read from the boundary before it and shifted, with the
// next lane's bytes.
template <typename T, int V, int NI> __device__ __forceinline__ void get_chunk(const T *p, int j, int n, typename Pack<T, V>::Raw (&r)[NI]) {
    const int lane = threadIdx.x & 31, off = (int)(reinterpret_cast<uintptr_t>(p) % 16);
    const long e = (long)j * kBeamTake - off / (int)sizeof(T) + lane * V;
#pragma unroll
    for (int i = 0; i < NI; ++i) r[i].w[0] = get_some<T, V>(p, e + i * 32 * V, n);
    if (!off) return;
    uint4 over = get_some<T, V>(p, e - lane * V + NI * 32 * V, n);      // behind the chunk's last lane
#pragma unroll
    for (int i = NI - 1; i >= 0; --i) {
        const uint4 a = r[i].w[0];
        uint4 next;
        next.x = __shfl_down_sync(0xffffffffu, a.x, 1);
        next.y = __shfl_down_sync(0xffffffffu, a.y, 1);
        next.z = __shfl_down_sync(0xffffffffu, a.z, 1);
        next.w = __shfl_down_sync(0xffffffffu, a.w, 1);
        const uint4 first = make_uint4(__shfl_sync(0xffffffffu, a.x, 0), __shfl_sync(0xffffffffu, a.y, 0), __shfl_sync(0xffffffffu, a.z, 0),
                                       __shfl_sync(0xffffffffu, a.w, 0));
        r[i].w[0] = from_byte(a, lane == 31 ? over : next, off);
        over = first;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) beam_scan_kernel(BeamSelect a) {
    constexpr int V = 16 / sizeof(T), NI = kBeamTake / (32 * V);
    constexpr float kLog2e = 1.4426950408889634f;
    __shared__ float sm[kWarps], ss[kWarps];
    next_may_start();
    const int row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits;
    const int b = row / a.W, w = row - b * a.W, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    if (a.finished && a.finished[row]) return;
    const T *p = row_of<T>(a, b, w);
    float M = -INFINITY, S = 0.f;
    const int takes = (a.V + kBeamTake - 1) / kBeamTake;
    for (int j = split * kWarps + warp; j < takes; j += a.splits * kWarps) {
        typename Pack<T, V>::Raw r[NI];
        get_chunk<T, V, NI>(p, j, a.V, r);
        float half[2] = {-INFINITY, -INFINITY}, x[V];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            Pack<T, V>::open(r[i], x);
#pragma unroll
            for (int k = 0; k < V; ++k) half[2 * i / NI] = fmaxf(half[2 * i / NI], x[k]);
        }
        // lanes of the upper half go on with the second chunk's maximum
        const bool up = lane & 16;
        float m = fmaxf(up ? half[1] : half[0], __shfl_xor_sync(0xffffffffu, up ? half[0] : half[1], 16));
#pragma unroll
        for (int off = 8; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if ((lane & 15) == 0) a.cmax[(long)row * a.nc + 2 * j + (lane >> 4)] = m;
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 16));
        const float now = fmaxf(M, m), ref = now == -INFINITY ? 0.f : now;    // nothing but -inf so far: sums of 0
        float add = 0.f;
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            Pack<T, V>::open(r[i], x);
#pragma unroll
            for (int k = 0; k < V; ++k) {
                float e;
                asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"((x[k] - ref) * kLog2e));
                add += e;
            }
        }
        float shrink;
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(shrink) : "f"((M - ref) * kLog2e));
        S = fmaf(S, shrink, add);
        M = now;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) S += __shfl_xor_sync(0xffffffffu, S, off);
    if (lane == 0) {
        sm[warp] = M;
        ss[warp] = S;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        float m = sm[0];
#pragma unroll
        for (int i = 1; i < kWarps; ++i) m = fmaxf(m, sm[i]);
        const float ref = m == -INFINITY ? 0.f : m;
        double sum = 0.0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) sum += (double)(ss[i] * exp2f((sm[i] - ref) * kLog2e));
        a.sums[blockIdx.x] = {sum, m};
    }
}

// A total as the sum of two fp32 (48 bits), which orders it by whole numbers; fp64 is 64 times slower here.
__device__ __forceinline__ unsigned ordered(float x) {
    const unsigned u = __float_as_uint(x + 0.f);        // -0 is 0
    return u ^ ((unsigned)((int)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(unsigned u) { return __uint_as_float(u >> 31 ? u ^ 0x80000000u : ~u); }
struct Off {                // score - lse; hi = -inf: the beam's candidates are all -inf
    float hi, lo;
};
__device__ __forceinline__ unsigned long long key_of(float hi, float lo) { return (unsigned long long)ordered(hi) << 32 | ordered(lo); }
__device__ __forceinline__ unsigned long long key_of(const Off &o, float x) {
    const float s = o.hi + x;
    if (!(fabsf(s) < INFINITY)) return key_of(s != s ? -INFINITY : s, 0.f);
    const float b = s - o.hi, e = ((o.hi - (s - b)) + (x - b)) + o.lo, hi = s + e;      // s + the sum's error, exactly
    return key_of(hi, (s - hi) + e);
}

// log of a sum of exp (1 <= s < 2^40), 2^-44: s = 2^n f, log f = 2 artanh((f - 1) / (f + 1)) by its series, |r| < 0.172.
__device__ __forceinline__ double log_sum(double s) {
    int n = (int)((unsigned long long)__double_as_longlong(s) >> 52) - 1023;
    double f = __longlong_as_double((__double_as_longlong(s) & 0xfffffffffffffll) | 0x3ff0000000000000ll);
    if (f > 1.4142135623730951) {
        f *= 0.5;
        ++n;
    }
    const double d = f + 1.0;
    double q = 1.0f / (float)d;
    q = q * (2.0 - d * q);                  // 2^-46
    const double r = (f - 1.0) * q, r2 = r * r, r4 = r2 * r2;
    // the series in pairs: every operation of the chain takes as long as dozens in fp32
    const double p = (1.0 + r2 * (1.0 / 3)) + r4 * ((1.0 / 5 + r2 * (1.0 / 7)) + r4 * ((1.0 / 9 + r2 * (1.0 / 11)) + r4 * (1.0 / 13 + r2 * (1.0 / 15))));
    return (r + r) * p + n * 0.69314718055994530942;
}

// A candidate's place in the order: larger totals first, then lower indices.
struct Cand {
    unsigned long long key;     // of the total: larger is larger (0: none)
    unsigned at;                // w V + v, or a chunk's number
};
__device__ __forceinline__ bool before(const Cand &a, const Cand &b) { return a.key > b.key || (a.key == b.key && a.at < b.at); }
__device__ __forceinline__ Cand shuffled(const Cand &c, int from) {
    return {__shfl_sync(0xffffffffu, c.key, from), __shfl_sync(0xffffffffu, c.at, from)};
}

// The best 32 of what a warp has seen, in order over its lanes.
struct WarpList {
    Cand c;
    // lane pairs `stride` apart: the better one to the lower lane (up: to the upper)
    __device__ __forceinline__ void trade(int stride, bool up) {
        const Cand y = shuffled(c, (threadIdx.x & 31) ^ stride);
        const bool lower = !(threadIdx.x & stride);
        if (before(y, c) == (lower != up)) c = y;
    }
    // a first batch, one candidate of each lane
    __device__ __forceinline__ void start(Cand x) {
        c = x;
#pragma unroll
        for (int size = 2; size <= 32; size *= 2)
#pragma unroll
            for (int stride = size / 2; stride; stride /= 2) trade(stride, size < 32 && (threadIdx.x & size));
    }
    // lanes with `some` bring a candidate each; k: how many are wanted
    __device__ __forceinline__ void take(bool some, Cand x, int k) {
        const int lane = threadIdx.x & 31;
        for (;;) {
            const Cand worst = shuffled(c, k - 1);      // by the whole warp, whatever its lanes bring
            some = some && before(x, worst);
            const unsigned who = __ballot_sync(0xffffffffu, some);
            if (!who) return;
            const int src = __ffs(who) - 1;
            const Cand y = shuffled(x, src);
            if (lane == src) some = false;
            const int pos = __popc(__ballot_sync(0xffffffffu, before(c, y)));     // the list is in order
            const Cand up = shuffled(c, lane ? lane - 1 : 0);
            if (lane == pos) c = y;
            if (lane > pos) c = up;
        }
    }
};

// The best 32 of all warps' lists, in order, in warp 0's (two lists, one of them turned round, hold their best 32 in the
// better of each place, and five trades put those in order).
__device__ __forceinline__ void join(WarpList &l, Cand *other) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
#pragma unroll 1
    for (int half = kPickWarps / 2; half; half /= 2) {
        __syncthreads();
        if (warp >= half && warp < 2 * half) other[(warp - half) * 32 + lane] = l.c;
        __syncthreads();
        if (warp < half) {
            const Cand y = other[warp * 32 + 31 - lane];
            if (before(y, l.c)) l.c = y;
#pragma unroll
            for (int stride = 16; stride; stride /= 2) l.trade(stride, false);
        }
    }
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(BeamSelect a) {
    __shared__ Off off[kBeamsIn];
    __shared__ Cand other[kPickWarps / 2 * 32], top[kBeamMax];
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32, k = a.k;
    wait_for_previous();
    if ((int)threadIdx.x < a.W) {           // a beam each
        const int w = threadIdx.x;
        const long row = (long)b * a.W + w;
        const float score = a.scores[row];
        Off o{score, 0.f};
        if (!(a.finished && a.finished[row])) {
            const BeamSum *s = a.sums + row * a.splits;
            float m = -INFINITY;
#pragma unroll 4
            for (int i = 0; i < a.splits; ++i) m = fmaxf(m, s[i].max);
            double sum = 0.0;
#pragma unroll 4
            for (int i = 0; i < a.splits; ++i) {        // a part of -inf alone has a sum of 0
                const float part = s[i].max;
                sum += part == m || part == -INFINITY ? s[i].sum : s[i].sum * (double)exp2f((part - m) * 1.4426950408889634f);
            }
            o.hi = -INFINITY;
            if (m > -INFINITY && m < INFINITY && sum < INFINITY && score > -INFINITY && score < INFINITY) {
                const double t = (double)score - ((double)m + log_sum(sum));
                o.hi = (float)t;
                o.lo = (float)(t - (double)o.hi);
            }
        }
        if (!(o.hi == o.hi)) o.hi = -INFINITY;
        off[w] = o;
    }
    __syncthreads();
    const unsigned long long none = key_of(-INFINITY, 0.f);
    auto done = [&](int w) { return a.finished && a.finished[(long)b * a.W + w]; };
    // the k first chunks
    WarpList l;
    const int nall = a.W * a.nc;
    constexpr int AT_ONCE = 4;              // maxima of a lane, loaded together
    bool first = true;
    for (int i0 = warp * 32; first || i0 < nall; i0 += AT_ONCE * kPickThreads) {
        Cand x[AT_ONCE];
#pragma unroll
        for (int u = 0; u < AT_ONCE; ++u) {
            const int i = i0 + u * kPickThreads + lane, w = i / a.nc, j = i - w * a.nc;
            x[u] = {0, 0xffffffffu};
            if (i >= nall || j * kBeamChunk >= a.V) continue;       // (a row's last chunk may hold nothing)
            x[u].at = i;
            if (done(w))
                x[u].key = a.eos / kBeamChunk == j ? key_of(off[w].hi, off[w].lo) : none;
            else
                x[u].key = off[w].hi > -INFINITY ? key_of(off[w], a.cmax[((long)b * a.W + w) * a.nc + j]) : none;
        }
        // a lane's best first: what comes after the lanes' best ones is seldom wanted
        auto order = [&](Cand &p, Cand &q) {
            if (before(q, p)) {
                const Cand t = p;
                p = q;
                q = t;
            }
        };
        order(x[0], x[1]);
        order(x[2], x[3]);
        order(x[0], x[2]);
        order(x[1], x[3]);
        order(x[1], x[2]);
        if (first)
            l.start(x[0]);
        else
            l.take(x[0].key != 0, x[0], k);
        first = false;
#pragma unroll 1
        for (int u = 1; u < AT_ONCE; ++u) {
            x[0] = x[1];
#pragma unroll
            for (int q = 1; q + 1 < AT_ONCE; ++q) x[q] = x[q + 1];
            l.take(x[0].key != 0, x[0], k);
        }
    }
    join(l, other);
    if (threadIdx.x < k) top[threadIdx.x] = l.c;
    __syncthreads();
    // their elements, those that reach the k-th chunk's maximum
    const unsigned long long least = top[k - 1].key;
    l.c = {0, 0xffffffffu};
    constexpr int U = 8, parts = kBeamChunk / (32 * U);         // eight rows of 32 elements at a time, loaded together
    for (int i = warp; i < k * parts; i += kPickWarps) {
        const unsigned chunk = top[i / parts].at;
        if (chunk == 0xffffffffu) break;         // fewer chunks than k
        const int w = chunk / a.nc, e0 = (int)(chunk - w * a.nc) * kBeamChunk + i % parts * (32 * U) + lane;
        const Off o = off[w];
        const T *p = row_of<T>(a, b, w);
        T x[U];
#pragma unroll
        for (int u = 0; u < U; ++u) x[u] = e0 + 32 * u < a.V ? p[e0 + 32 * u] : from_f32<T>(0.f);
        const bool over = done(w);
#pragma unroll 1
        for (int u = 0; u < U; ++u) {
            T v = x[0];
#pragma unroll
            for (int q = 0; q + 1 < U; ++q) x[q] = x[q + 1];
            const int e = e0 + 32 * u;
            Cand c{0, (unsigned)(w * (long)a.V + e)};
            if (over)
                c.key = e == a.eos ? key_of(o.hi, o.lo) : none;
            else
                c.key = o.hi > -INFINITY ? key_of(o, to_f32(v)) : none;
            l.take(e < a.V && c.key >= least, c, k);
        }
    }
    join(l, other);
    if (threadIdx.x < k) {
        const long o = (long)b * k + threadIdx.x;
        a.out[o] = unordered((unsigned)(l.c.key >> 32));
        a.parents[o] = (int)(l.c.at / (unsigned)a.V);
        a.tokens[o] = (int)(l.c.at % (unsigned)a.V);
    }
}

// ------------------------------------------------------------------------------ reordering
template <typename U, int W> __device__ __forceinline__ void move_column(char *base, long long bytes, long col, const int *par, int n) {
    U v[W];
#pragma unroll
    for (int w = 0; w < W; ++w)
        if (w < n && par[w] != w) v[w] = *reinterpret_cast<const U *>(base + par[w] * bytes + col * (long)sizeof(U));
#pragma unroll
    for (int w = 0; w < W; ++w)
        if (w < n && par[w] != w) *reinterpret_cast<U *>(base + w * bytes + col * (long)sizeof(U)) = v[w];
}

template <int W>
__global__ void __launch_bounds__(kThreads) beam_reorder_kernel(const __grid_constant__ BeamReorder a) {
    __shared__ int par[W];
    const int b = blockIdx.y;
    if (threadIdx.x < W) {
        const int w = threadIdx.x;
        int p = w < a.W ? a.parents[(long)b * a.W + w] : w;
        par[w] = p < 0 || p >= a.W ? w : p;          // out of range: the beam stays
    }
    __syncthreads();
    int i = 0;
    while (i + 1 < a.count && blockIdx.x >= a.first[i + 1]) ++i;
    const long col = (long)(blockIdx.x - a.first[i]) * kThreads + threadIdx.x;
    const long long bytes = a.bytes[i];
    if (col * a.unit[i] >= bytes) return;
    char *base = a.p[i] + (long)b * a.W * bytes;
    switch (a.unit[i]) {
    case 16: move_column<uint4, W>(base, bytes, col, par, a.W); break;
    case 8: move_column<uint2, W>(base, bytes, col, par, a.W); break;
    case 4: move_column<unsigned, W>(base, bytes, col, par, a.W); break;
    case 2: move_column<unsigned short, W>(base, bytes, col, par, a.W); break;
    default: move_column<unsigned char, W>(base, bytes, col, par, a.W);
    }
}

template <int W> void go_reorder(const BeamReorder &a, cudaStream_t st) {
    beam_reorder_kernel<W><<<dim3(a.first[a.count], a.B), kThreads, 0, st>>>(a);
}

}  // namespace

int beam_splits(long rows, int nc, int sms) {
    const int most = (nc + kWarps - 1) / kWarps;        // a chunk for every warp
    int s = 1;
    while (s < most && rows * s < 8L * sms) ++s;
    return s;
}

cudaError_t launch_beam_select(const BeamSelect &a, cudaStream_t st) {
    const unsigned grid = (unsigned)((long)a.B * a.W * a.splits);
    if (a.dtype == DType::BF16)
        beam_scan_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
    else
        beam_scan_kernel<float><<<grid, kThreads, 0, st>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(a.dtype == DType::BF16 ? beam_pick_kernel<__nv_bfloat16> : beam_pick_kernel<float>, dim3((unsigned)a.B),
                        kPickThreads, 0, st, a);
}

cudaError_t launch_beam_reorder(BeamReorder &a, cudaStream_t st) {
    unsigned first = 0;
    for (int i = 0; i < a.count; ++i) {
        int u = 16;
        while ((reinterpret_cast<uintptr_t>(a.p[i]) | (uintptr_t)a.bytes[i]) & (u - 1)) u /= 2;
        a.unit[i] = u;
        a.first[i] = first;
        const long long ctas = (a.bytes[i] / u + kThreads - 1) / kThreads;
        if (ctas > 0x7fffffffL - first) return cudaErrorInvalidValue;
        first += (unsigned)ctas;
    }
    a.first[a.count] = first;
    if (!first || !a.B) return cudaSuccess;
    if (a.W <= 4) go_reorder<4>(a, st);
    else if (a.W <= 8) go_reorder<8>(a, st);
    else if (a.W <= 16) go_reorder<16>(a, st);
    else go_reorder<32>(a, st);
    return cudaGetLastError();
}

}  // namespace kda
