// beam.cu -- beam search: the k best continuations of a request's W beams, and the recurrent memories that follow them.
//
// Selection: total[w, v] = score_w + x_w[v] - lse_w, lse_w = log sum_v exp(x_w[v]); the k largest over all (w, v), ties to
// the lowest w V + v.  The logits are read once: a warp takes a chunk of 1024 consecutive ones, keeps the chunk's maximum
// and adds up exp(x - M) against the running maximum M of its chunks.  An element among the k best lies in one of the k
// chunks that come first when chunks are ordered by (maximum, position): every chunk before its own holds an element that
// comes before it.  So the second kernel, a CTA per request, orders the chunks' maxima and looks at k chunks only.
// Totals are formed and compared in 64 bits (candidates of different beams may be closer than an fp32 total's rounding);
// sums of exp are fp32 over a lane's few hundred terms and 64-bit from there on.
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

// Chunk j of a row, 16 bytes per lane and i: elements j 1024 + (32 i + lane) V on, whatever the row's address is, so that
// equal rows give equal sums.  A row off the 16-byte boundary is read from the boundary before it and shifted, with the
// next lane's bytes.
template <typename T, int V, int NI> __device__ __forceinline__ void get_chunk(const T *p, int j, int n, typename Pack<T, V>::Raw (&r)[NI]) {
    const int lane = threadIdx.x & 31, off = (int)(reinterpret_cast<uintptr_t>(p) % 16);
    const long e = (long)j * kBeamChunk - off / (int)sizeof(T) + lane * V;
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
    constexpr int V = 16 / sizeof(T), NI = kBeamChunk / (32 * V);
    constexpr float kLog2e = 1.4426950408889634f;
    __shared__ float sm[kWarps], ss[kWarps];
    next_may_start();
    const int row = blockIdx.x / a.splits, split = blockIdx.x - row * a.splits;
    const int b = row / a.W, w = row - b * a.W, lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    if (a.finished && a.finished[row]) return;
    const T *p = row_of<T>(a, b, w);
    float M = -INFINITY, S = 0.f;
    for (int j = split * kWarps + warp; j < a.nc; j += a.splits * kWarps) {
        typename Pack<T, V>::Raw r[NI];
        get_chunk<T, V, NI>(p, j, a.V, r);
        float m = -INFINITY, x[V];
#pragma unroll
        for (int i = 0; i < NI; ++i) {
            Pack<T, V>::open(r[i], x);
#pragma unroll
            for (int k = 0; k < V; ++k) m = fmaxf(m, x[k]);
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, off));
        if (lane == 0) a.cmax[(long)row * a.nc + j] = m;
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

// A candidate's place in the order: larger totals first, then lower indices.
struct Cand {
    unsigned long long key;     // of the total: larger is larger
    unsigned at;                // w V + v, or a chunk's number
};
__device__ __forceinline__ bool before(const Cand &a, const Cand &b) { return a.key > b.key || (a.key == b.key && a.at < b.at); }
__device__ __forceinline__ unsigned long long key_of(double x) {
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);    // -0 is 0
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double total_of(unsigned long long key) {
    return __longlong_as_double((long long)(key >> 63 ? key & 0x7fffffffffffffffull : ~key));
}

// The best of what a warp has seen, in order over its lanes.
struct WarpList {
    Cand c;
    __device__ __forceinline__ void clear() { c = {0, 0xffffffffu}; }
    // lanes with `some` bring a candidate each; k: how many are wanted
    __device__ __forceinline__ void take(bool some, Cand x, int k) {
        const int lane = threadIdx.x & 31;
        for (;;) {
            Cand worst;
            worst.key = __shfl_sync(0xffffffffu, c.key, k - 1);
            worst.at = __shfl_sync(0xffffffffu, c.at, k - 1);
            some = some && before(x, worst);
            const unsigned who = __ballot_sync(0xffffffffu, some);
            if (!who) return;
            const int src = __ffs(who) - 1;
            Cand y;
            y.key = __shfl_sync(0xffffffffu, x.key, src);
            y.at = __shfl_sync(0xffffffffu, x.at, src);
            if (lane == src) some = false;
            const int pos = __popc(__ballot_sync(0xffffffffu, before(c, y)));     // the list is in order
            const unsigned long long uk = __shfl_up_sync(0xffffffffu, c.key, 1);
            const unsigned ua = __shfl_up_sync(0xffffffffu, c.at, 1);
            if (lane == pos) c = y;
            if (lane > pos) c = {uk, ua};
        }
    }
};

// The k first of all warps' lists, in order, at out[0 .. k): every entry counts those before it.
__device__ __forceinline__ void join(WarpList &l, Cand *all, Cand *out, int k) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, n = kPickWarps * k;
    __syncthreads();
    if (lane < k) all[warp * k + lane] = l.c;
    __syncthreads();
    if ((int)threadIdx.x < n) {
        const Cand x = all[threadIdx.x];
        int rank = 0;
        for (int i = 0; i < n; ++i) rank += i != (int)threadIdx.x && (before(all[i], x) || (!before(x, all[i]) && i < (int)threadIdx.x));
        if (rank < k) out[rank] = x;
    }
    __syncthreads();
}

template <typename T>
__global__ void __launch_bounds__(kPickThreads) beam_pick_kernel(BeamSelect a) {
    __shared__ double off[kBeamsIn];        // score - lse; -inf: the beam's candidates are all -inf
    __shared__ Cand all[kPickWarps * kBeamMax], top[kBeamMax];
    const int b = blockIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x / 32, k = a.k;
    wait_for_previous();
    for (int w = warp; w < a.W; w += kPickWarps) {
        const long row = (long)b * a.W + w;
        const double score = a.scores[row];
        double o = score;
        if (!(a.finished && a.finished[row])) {
            const BeamSum *s = a.sums + row * a.splits;
            float m = -INFINITY;
            for (int i = lane; i < a.splits; i += 32) m = fmaxf(m, s[i].max);
#pragma unroll
            for (int q = 16; q; q >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, q));
            double sum = 0.0;
            for (int i = lane; i < a.splits; i += 32)      // a part of -inf alone has a sum of 0
                sum += s[i].max == m || s[i].max == -INFINITY ? s[i].sum : s[i].sum * exp((double)s[i].max - (double)m);
#pragma unroll
            for (int q = 16; q; q >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, q);
            o = score - ((double)m + log(sum));
            if (!(m > -INFINITY && m < INFINITY && sum < INFINITY)) o = -INFINITY;       // no distribution
        }
        if (!(o == o)) o = -INFINITY;
        if (lane == 0) off[w] = o;
    }
    __syncthreads();
    auto dead = [&](double o) { return o == -INFINITY; };
    auto done = [&](int w) { return a.finished && a.finished[(long)b * a.W + w]; };
    // the k first chunks
    WarpList l;
    l.clear();
    const int nall = a.W * a.nc;
    for (int i0 = warp * 32; i0 < nall; i0 += kPickThreads) {
        const int i = i0 + lane;
        const bool some = i < nall;
        Cand x{0, (unsigned)i};
        if (some) {
            const int w = i / a.nc, j = i - w * a.nc;
            double t = -INFINITY;
            if (done(w))
                t = a.eos / kBeamChunk == j ? off[w] : t;
            else if (!dead(off[w]))
                t = off[w] + (double)a.cmax[((long)b * a.W + w) * a.nc + j];
            x.key = key_of(t);
        }
        l.take(some, x, k);
    }
    join(l, all, top, k);
    // their elements: those that reach the k-th chunk's maximum are looked at in 64 bits
    const unsigned long long least = top[k - 1].at == 0xffffffffu ? 0 : top[k - 1].key;
    const double reach = total_of(least ? least : key_of(-INFINITY));
    l.clear();
    constexpr int parts = kBeamChunk / 32;
    for (int i = warp; i < k * parts; i += kPickWarps) {
        const unsigned chunk = top[i / parts].at;
        if (chunk == 0xffffffffu) break;         // fewer chunks than k
        const int w = chunk / a.nc, j = chunk - w * a.nc;
        const T *p = row_of<T>(a, b, w);
        const long e = (long)j * kBeamChunk + (i % parts) * 32 + lane;
        bool some = e < a.V;
        Cand x{0, (unsigned)(w * (long)a.V + e)};
        if (some) {
            double t = -INFINITY;
            if (done(w))
                t = e == a.eos ? off[w] : t;
            else if (!dead(off[w]))
                t = off[w] + (double)to_f32(p[e]);
            x.key = key_of(t);
            some = t >= reach;
        }
        l.take(some, x, k);
    }
    join(l, all, top, k);
    if (threadIdx.x < k) {
        const Cand x = top[threadIdx.x];
        const long o = (long)b * k + threadIdx.x;
        a.out[o] = (float)total_of(x.key);
        a.parents[o] = (int)(x.at / (unsigned)a.V);
        a.tokens[o] = (int)(x.at % (unsigned)a.V);
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
