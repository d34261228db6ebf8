// short_conv.cu -- the short causal convolution over tokens, one filter of K taps per channel.
//
//     p_t = bias + sum_j w_j x_{t-K+1+j},   y_t = act(p_t),   act = silu or none,
// with the K - 1 tokens before a sequence from its window (zeros without one), and after it the last K - 1 tokens as the
// next window.  Gradients, with q_t = dy_t act'(p_t) (p_t formed again):
//     dx_t = sum_j w_j q_{t+K-1-j},   dw_j = sum_t q_t x_{t-K+1+j},   dbias = sum_t q_t,
// where the last K - 1 tokens' dx takes the next window's gradient too, and dx of the tokens before the sequence is the
// window's gradient.
//
// A lane holds V = 4 channels in packed pairs (8 of them left registers for too few rows in flight: forwards 34 us at 2 x 2048 tokens
// of 4096 channels where 4 took 23), a warp 32 V of them, and walks a run of tokens of one sequence with the K last rows in
// registers, so that every row is read once, but for the K - 1 rows that a run shares with the next (L2 has them).  The
// sums are fp32 and rounded once.  The weights' gradients stay in registers over all runs of a lane, are added up over a
// CTA's warps in shared memory and over the CTAs by a second kernel, in a fixed order.
//
// Measured, bf16: forwards 15 us at that shape (67 MB, 9.9 us at the copy rate; 66 instructions a row and warp take 0.57 of the
// issue slots, and warps wait for their loads), 16 packed prompts of 40,000 tokens in all and 2048 channels 61 to 64 us, 5.3 to
// 5.1 TB/s; gradients 31 us (101 MB, 14.9 us; 128 registers, 16 warps an SM), the second kernel among it; in fp32 44 us (29.7).
#include <algorithm>

#include "conv_internal.cuh"
#include "run_item.cuh"
#include "ssm_math.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kWarps = kThreads / 32;

// V channels' values, in packed pairs where there are any.
template <int V> struct Ch {
    static constexpr int P = V / 2;
    Two p[P];
    __device__ __forceinline__ void set(const float (&x)[V]) {
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] = two(x[2 * i], x[2 * i + 1]);
    }
    __device__ __forceinline__ void get(float (&x)[V]) const {
#pragma unroll
        for (int i = 0; i < P; ++i) each(p[i], x[2 * i], x[2 * i + 1]);
    }
    __device__ __forceinline__ void add(const Ch &a) {
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] = add2(p[i], a.p[i]);
    }
    __device__ __forceinline__ void fma(const Ch &a, const Ch &b) {
#pragma unroll
        for (int i = 0; i < P; ++i) p[i] = fma2(a.p[i], b.p[i], p[i]);
    }
};
template <> struct Ch<1> {
    float p;
    __device__ __forceinline__ void set(const float (&x)[1]) { p = x[0]; }
    __device__ __forceinline__ void get(float (&x)[1]) const { x[0] = p; }
    __device__ __forceinline__ void add(const Ch &a) { p += a.p; }
    __device__ __forceinline__ void fma(const Ch &a, const Ch &b) { p = fmaf(a.p, b.p, p); }
};

template <typename T, int V> __device__ __forceinline__ Few<T, V> get(const T *p, bool live = true) {
    Few<T, V> r;
    r.template load<true>(p, live ? V : 0);
    return r;
}
template <typename T, int V> __device__ __forceinline__ Ch<V> open(const Few<T, V> &r) {
    float x[V];
#pragma unroll
    for (int i = 0; i < V; ++i) x[i] = r[i];
    Ch<V> c;
    c.set(x);
    return c;
}
template <typename T, int V> __device__ __forceinline__ void put(T *p, const float (&x)[V]) { Few<T, V>::template store<true>(p, x, V); }
template <int V> __device__ __forceinline__ Ch<V> zeros() {
    float x[V] = {};
    Ch<V> c;
    c.set(x);
    return c;
}

// Taps of the lane's channels [c, c + V), and their biases.
template <int V, int K, typename A> __device__ __forceinline__ void load_taps(const A &a, int c, bool live, Ch<V> (&w)[K], Ch<V> &b) {
    if constexpr (V == 4) {        // K 16-byte pieces (the launcher has seen to the alignment)
        float t[4 * K];
#pragma unroll
        for (int j = 0; j < K; ++j) {
            const float4 v = live ? reinterpret_cast<const float4 *>(a.w + (long)c * K)[j] : make_float4(0.f, 0.f, 0.f, 0.f);
            t[4 * j] = v.x, t[4 * j + 1] = v.y, t[4 * j + 2] = v.z, t[4 * j + 3] = v.w;
        }
        const float4 v = live && a.bias ? *reinterpret_cast<const float4 *>(a.bias + c) : make_float4(0.f, 0.f, 0.f, 0.f);
        b.set({v.x, v.y, v.z, v.w});
#pragma unroll
        for (int j = 0; j < K; ++j) w[j].set({t[j], t[K + j], t[2 * K + j], t[3 * K + j]});
    } else {
        b.set({live && a.bias ? a.bias[c] : 0.f});
#pragma unroll
        for (int j = 0; j < K; ++j) w[j].set({live ? a.w[(long)c * K + j] : 0.f});
    }
}

// Row t of the window before a sequence's tokens (t in [-(K - 1), -1]).
template <typename T, int V, int K>
__device__ __forceinline__ Ch<V> load_window(const void *h0, int n, int t, int C, int c) {
    return open<T, V>(get<T, V>(static_cast<const T *>(h0) + ((long)n * (K - 1) + (t + K - 1)) * C + c, h0 != nullptr));
}

// The window after sequence n: rows len - (K - 1) .. len - 1, read before any is written (hT may be h0).
template <typename T, int V, int K>
__device__ __forceinline__ void next_window(const Conv &a, int n, long start, int len, int c) {
    const T *xp = static_cast<const T *>(a.x.p) + (a.s.cu ? start * a.x.t : (long)n * a.x.b) + c;
    Few<T, V> r[K - 1];
#pragma unroll
    for (int i = 0; i < K - 1; ++i) {
        const int t = len - (K - 1) + i;
        if (t >= 0)
            r[i] = get<T, V>(xp + t * a.x.t);
        else
            r[i] = get<T, V>(static_cast<const T *>(a.h0) + ((long)n * (K - 1) + (t + K - 1)) * a.C + c, a.h0 != nullptr);
    }
    T *hp = static_cast<T *>(a.hT) + (long)n * (K - 1) * a.C + c;
#pragma unroll
    for (int i = 0; i < K - 1; ++i) r[i].keep(hp + (long)i * a.C);
}

// Run `item` of the launch; false: there is none.  (What run_item does, written out: called, 16 packed prompts of 40,000 tokens take
// 69.6 us instead of 63.4, with the same registers; the search is not what they go through.)
__device__ __forceinline__ bool conv_item(const Conv &a, long item, LinItem &it) {
    if (item >= a.items) return false;
    if (!a.s.cu) return lin_item(a.s, a.run, (int)item, it);
    if (a.s.nseq <= kCounted) {
        if (!lin_item(a.s, a.run, (int)item, it)) return false;
        it.start = min(max(it.start, 0L), a.total);
        it.len = (int)min((long)max(it.len, 0), a.total - it.start);
        return true;
    }
    const int lane = threadIdx.x & 31, total = (int)a.total;
    const auto place = [&](int n) { return min(max(a.s.cu[n], 0), total); };
    int lo = 0, n = a.s.nseq, step;         // the sequence is among lo .. lo + n
    do {
        step = (n + 31) / 32;
        const int k = lane * step;
        const unsigned some = __ballot_sync(0xffffffffu, k < n && place(lo + k) / a.run + lo + k <= item);
        if (!some) return false;
        const int last = (31 - __clz(some)) * step;
        lo += last;
        n = min(step, n - last);
    } while (step > 1);
    const int start = place(lo);
    it.n = lo;
    it.first = start / a.run + lo;
    it.p = (int)item - it.first;
    it.start = start;
    it.len = max(place(lo + 1) - start, 0);
    it.nseg = it.len > a.run ? (it.len + a.run - 1) / a.run : 1;
    return it.p < it.nseg;
}

// Warp = 32 V channels of one run.  The run that ends a sequence writes its next window (WINDOW_ONLY: nothing else).
template <typename T, int V, int K, bool WINDOW_ONLY>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 3) conv_fwd_kernel(Conv a) {
    const int group = blockIdx.x / a.blocks, c = ((blockIdx.x - group * a.blocks) * 32 + (threadIdx.x & 31)) * V;
    const bool live = c < a.C;
    LinItem it;
    if (!conv_item(a, (long)group * kWarps + threadIdx.x / 32, it)) return;
    const int t0 = it.p * a.run, t1 = min(it.len, t0 + a.run);
    if (a.hT && it.p == it.nseg - 1 && live && (WINDOW_ONLY || a.hT != a.h0)) next_window<T, V, K>(a, it.n, it.start, it.len, c);
    if (WINDOW_ONLY || !live || t0 >= t1) return;
    Ch<V> w[K], b, x[K];
    load_taps<V, K>(a, c, live, w, b);
    const T *xp = static_cast<const T *>(a.x.p) + (a.s.cu ? it.start * a.x.t : it.n * a.x.b) + c;
    T *yp = static_cast<T *>(a.y.p) + (a.s.cu ? it.start * a.y.t : it.n * a.y.b) + c;
#pragma unroll
    for (int j = 1; j < K; ++j) {
        const int t = t0 - K + j;
        x[j] = t >= 0 ? open<T, V>(get<T, V>(xp + t * a.x.t)) : load_window<T, V, K>(a.h0, it.n, t, a.C, c);
    }
    auto one = [&](int t, const Few<T, V> &raw) {
#pragma unroll
        for (int j = 0; j + 1 < K; ++j) x[j] = x[j + 1];
        x[K - 1] = open<T, V>(raw);
        Ch<V> p = b;
#pragma unroll
        for (int j = 0; j < K; ++j) p.fma(w[j], x[j]);
        float y[V];
        p.get(y);
        if (a.act) {
#pragma unroll
            for (int i = 0; i < V; ++i) {
                float rest;
                y[i] *= sigmoid<T>(y[i], rest);
            }
        }
        put<T, V>(yp + t * a.y.t, y);
    };
    constexpr int U = 4;                // rows ahead of those at work
    int t = t0;
    Few<T, V> now[U], next[U];
    auto fetch = [&](int t, Few<T, V> (&r)[U]) {
#pragma unroll
        for (int u = 0; u < U; ++u) r[u] = get<T, V>(xp + (t + u) * a.x.t);
    };
    if (t + U <= t1) fetch(t, now);
    for (; t + U <= t1; t += U) {
        if (t + 2 * U <= t1) fetch(t + U, next);
#pragma unroll
        for (int u = 0; u < U; ++u) one(t + u, now[u]);
#pragma unroll
        for (int u = 0; u < U; ++u) now[u] = next[u];
    }
    if (t < t1) {                       // what is left of the run, loaded together
#pragma unroll
        for (int u = 0; u < U - 1; ++u) now[u] = get<T, V>(xp + (t + u) * a.x.t, t + u < t1);
#pragma unroll
        for (int u = 0; u < U - 1; ++u)
            if (t + u < t1) one(t + u, now[u]);
    }
}

// A warp's lanes go over the items warp, warp + warps, ...; q of K rows and x of K rows in registers.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads, 2) conv_bwd_kernel(Conv a) {
    __shared__ float sum[kWarps / 2][32 * V + 1];
    next_may_start();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const int c = (blockIdx.x * 32 + lane) * V;
    const bool live = c < a.C;
    Ch<V> w[K], b, dw[K], db = zeros<V>();
    load_taps<V, K>(a, c, live, w, b);
#pragma unroll
    for (int j = 0; j < K; ++j) dw[j] = db;
    for (long item = (long)blockIdx.y * kWarps + warp; item < a.items; item += (long)gridDim.y * kWarps) {
        LinItem it;
        if (!conv_item(a, item, it) || !live || (it.p && it.p * a.run >= it.len)) continue;
        const int t0 = it.p * a.run, t1 = min(it.len, t0 + a.run);
        const T *xp = static_cast<const T *>(a.x.p) + (a.s.cu ? it.start * a.x.t : it.n * a.x.b) + c;
        const T *gp = static_cast<const T *>(a.y.p) + (a.s.cu ? it.start * a.y.t : it.n * a.y.b) + c;
        T *dp = static_cast<T *>(a.dx.p) + (a.s.cu ? it.start * a.dx.t : it.n * a.dx.b) + c;
        const long win = (long)it.n * (K - 1) * a.C + c;      // row -(K - 1) of the window
        Ch<V> x[K], q[K];
#pragma unroll
        for (int j = 1; j < K; ++j) {
            const int t = t0 - K + j;
            x[j] = t >= 0 ? open<T, V>(get<T, V>(xp + t * a.x.t)) : load_window<T, V, K>(a.h0, it.n, t, a.C, c);
        }
#pragma unroll
        for (int j = 0; j < K; ++j) q[j] = zeros<V>();
        // dx of row t - (K - 1) is whole once q_t is there; the first run goes on to the window's rows.  q of rows past
        // the run is formed here too (its share of the weights' gradients belongs to the next run).
        const int last = t1 + K - 1;
        // INNER: a row of the run whose dx row is of the run too, which needs no condition
        auto one = [&](int tt, const Few<T, V> &xr, const Few<T, V> &gr, auto inner) {
            constexpr bool INNER = decltype(inner)::value;
#pragma unroll
            for (int j = 0; j + 1 < K; ++j) {
                x[j] = x[j + 1];
                q[j] = q[j + 1];
            }
            x[K - 1] = open<T, V>(xr);
            float g[V];
#pragma unroll
            for (int i = 0; i < V; ++i) g[i] = gr[i];
            if (a.act) {
                Ch<V> pre = b;
#pragma unroll
                for (int j = 0; j < K; ++j) pre.fma(w[j], x[j]);
                float p[V], rest;
                pre.get(p);
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    const float s = sigmoid<T>(p[i], rest);
                    g[i] *= fmaf(p[i] * s, rest, s);
                }
            }
            if (!INNER) {
#pragma unroll
                for (int i = 0; i < V; ++i) g[i] = tt < it.len ? g[i] : 0.f;
            }
            q[K - 1].set(g);
            if (INNER || tt < t1) {
                db.add(q[K - 1]);
#pragma unroll
                for (int j = 0; j < K; ++j) dw[j].fma(q[K - 1], x[j]);
            }
            const int row = tt - (K - 1);
            if (INNER || row >= t0 || (t0 == 0 && a.dh0)) {
                Ch<V> d = zeros<V>();
                if (!INNER && a.dhT && tt >= it.len)        // a row of the next window
                    d = open<T, V>(get<T, V>(static_cast<const T *>(a.dhT) + win + (long)(tt - it.len) * a.C));
#pragma unroll
                for (int j = 0; j < K; ++j) d.fma(w[j], q[K - 1 - j]);
                float o[V];
                d.get(o);
                put<T, V>(INNER || row >= 0 ? dp + row * a.dx.t : static_cast<T *>(a.dh0) + win + (long)(row + K - 1) * a.C, o);
            }
        };
        // n rows from t on, loaded together
        constexpr int U = sizeof(T) == 2 ? 6 : 4;
        auto some = [&](int t, int n, auto most, auto inner) {
            constexpr int MOST = decltype(most)::value;
            Few<T, V> xr[MOST], gr[MOST];
#pragma unroll
            for (int u = 0; u < MOST; ++u) {
                const bool there = u < n && (decltype(inner)::value || t + u < it.len);
                xr[u] = get<T, V>(xp + (t + u) * a.x.t, there);
                gr[u] = get<T, V>(gp + (t + u) * a.y.t, there);
            }
#pragma unroll
            for (int u = 0; u < MOST; ++u)
                if (u < n) one(t + u, xr[u], gr[u], inner);
        };
        const std::true_type inner;
        const std::false_type edge;
        const std::integral_constant<int, K - 1> few;
        const std::integral_constant<int, U> many;
        some(t0, K - 1, few, edge);             // (of a short run: rows behind it)
        int t = t0 + K - 1;
        for (; t + U <= t1; t += U) some(t, U, many, inner);
        if (t < t1) some(t, t1 - t, many, inner);
        t = max(t1, t0 + K - 1);
        some(t, last - t, few, edge);
    }
    // the CTA's sums, in the order of its warps: 4 + 4 (two rounds), then the partial row
    const long row = (long)blockIdx.y * a.C * (K + 1);
#pragma unroll
    for (int j = 0; j <= K; ++j) {
        float v[V];
        (j < K ? dw[j < K ? j : 0] : db).get(v);
        __syncthreads();
        if (warp >= kWarps / 2)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[warp - kWarps / 2][lane * V + i] = v[i];
        __syncthreads();
        if (warp < kWarps / 2)
#pragma unroll
            for (int i = 0; i < V; ++i) sum[warp][lane * V + i] += v[i];
        __syncthreads();
        for (int e = threadIdx.x; e < 32 * V; e += kThreads) {
            const int ch = blockIdx.x * 32 * V + e;
            if (ch < a.C) a.part[row + (long)j * a.C + ch] = (sum[0][e] + sum[1][e]) + (sum[2][e] + sum[3][e]);
        }
    }
}

// dw, dbias from the partial rows; a warp sums 32 consecutive columns' parts in order, eight warps share a column.
__global__ void __launch_bounds__(kThreads) conv_fold_kernel(const float *part, int parts, int C, int K, float *dw, float *dbias) {
    __shared__ float s[kWarps][33];
    wait_for_previous();
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32;
    const long col = (long)blockIdx.x * 32 + lane, cols = (long)C * (K + 1);
    float v = 0.f;
    if (col < cols)
        for (int p = warp; p < parts; p += kWarps) v += part[p * cols + col];
    s[warp][lane] = v;
    __syncthreads();
    if (warp || col >= cols) return;
    v = 0.f;
#pragma unroll
    for (int k = 0; k < kWarps; ++k) v += s[k][lane];
    const int j = (int)(col / C), c = (int)(col - (long)j * C);
    if (j < K)
        dw[(long)c * K + j] = v;
    else if (dbias)
        dbias[c] = v;
}

// One token of a request, V channels per lane.
template <typename T, int V, int K>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(ConvStep a) {
    const int nv = a.C / V;
    const long id = blockIdx.x * (long)kThreads + threadIdx.x;
    if (id >= (long)nv * a.B) return;
    const int n = (int)(id / nv), c = (int)(id - (long)n * nv) * V;
    T *sp = static_cast<T *>(a.state) + (long)n * (K - 1) * a.C + c;
    Ch<V> w[K], b;
    Few<T, V> r[K];
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) r[j] = get<T, V>(sp + (long)j * a.C);
    r[K - 1] = get<T, V>(static_cast<const T *>(a.x) + n * a.xb + c);
    load_taps<V, K>(a, c, true, w, b);
#pragma unroll
    for (int j = 0; j < K; ++j) b.fma(w[j], open<T, V>(r[j]));
    float y[V];
    b.get(y);
    if (a.act) {
#pragma unroll
        for (int i = 0; i < V; ++i) {
            float rest;
            y[i] *= sigmoid<T>(y[i], rest);
        }
    }
    put<T, V>(static_cast<T *>(a.y) + n * a.yb + c, y);
#pragma unroll
    for (int j = 0; j + 1 < K; ++j) r[j + 1].keep(sp + (long)j * a.C);
}

constexpr int kLane = 4;            // channels of a lane where everything is aligned to them
template <typename T> bool by4(const void *p) { return reinterpret_cast<uintptr_t>(p) % (kLane * sizeof(T)) == 0; }
template <typename T> bool vec_view(const ConvView &v) { return by4<T>(v.p) && v.b % kLane == 0 && v.t % kLane == 0; }

// Tokens of a run: so many that the warps that stay resident (ctas to an SM) have one each, or the same number of them where
// they would pass 64 tokens; a last round of few warps would take as long as a full one (2 x 2048 tokens of 4096 channels in runs
// of 16 and 32: forwards 17, backwards 41 us; in runs of 27 and 57: 15 and 30).
int pick_run(const Conv &a, int V, long rows, int ctas) {
    const long blocks = (a.C + 32 * V - 1) / (32 * V), warps = std::max(1L, (long)ctas * a.sms / blocks) * kWarps;
    const long most = warps * ((rows + warps * 64 - 1) / (warps * 64));         // runs
    long run = std::max(8L, most ? (rows + most - 1) / most : 0);
    if (!a.s.cu)
        while (run < 64 && a.s.nseq * ((a.s.T + run - 1) / run) > most) ++run;   // sequences end in runs of their own
    return (int)run;
}

template <typename T, int V, int K> cudaError_t run_fwd(Conv a, cudaStream_t st) {
    const long rows = a.s.cu ? a.total : (long)a.s.nseq * a.s.T;
    a.run = pick_run(a, V, rows, sizeof(T) == 2 ? 4 : 3);
    a.items = run_items(a.s, a.total, a.run);
    a.blocks = (a.C + 32 * V - 1) / (32 * V);
    const long ctas = (a.items + kWarps - 1) / kWarps * a.blocks;
    if (ctas > 0x7fffffffL) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)ctas;
    conv_fwd_kernel<T, V, K, false><<<grid, kThreads, 0, st>>>(a);
    // the window is updated in place: after the tokens have been read
    if (a.hT && a.hT == a.h0) conv_fwd_kernel<T, V, K, true><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <typename T, int V, int K> cudaError_t run_bwd(Conv a, cudaStream_t st) {
    const long rows = a.s.cu ? a.total : (long)a.s.nseq * a.s.T;
    a.run = pick_run(a, V, rows, 2);
    a.items = run_items(a.s, a.total, a.run);
    const unsigned cb = (a.C + 32 * V - 1) / (32 * V);
    const long want = (long)std::max(1, std::min(conv_parts(a.C, a.sms), 4 * a.sms / (int)cb));
    const unsigned parts = (unsigned)std::min((a.items + kWarps - 1) / kWarps, want);
    conv_bwd_kernel<T, V, K><<<dim3(cb, parts), kThreads, 0, st>>>(a);
    const long cols = (long)a.C * (K + 1);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    return launch_after(conv_fold_kernel, dim3((unsigned)((cols + 31) / 32)), kThreads, 0, st, (const float *)a.part, (int)parts,
                        a.C, K, a.dw, a.dbias);
}

template <typename T, int K> cudaError_t go(const Conv &a, bool bwd, cudaStream_t st) {
    constexpr int V = kLane;
    const bool vec = a.C % V == 0 && by4<float>(a.w) && by4<float>(a.bias) && vec_view<T>(a.x) && vec_view<T>(a.y) && by4<T>(a.h0) &&
                     by4<T>(a.hT) && (!bwd || (vec_view<T>(a.dx) && by4<T>(a.dhT) && by4<T>(a.dh0)));
    if (bwd) return vec ? run_bwd<T, V, K>(a, st) : run_bwd<T, 1, K>(a, st);
    return vec ? run_fwd<T, V, K>(a, st) : run_fwd<T, 1, K>(a, st);
}
template <typename T> cudaError_t taps(const Conv &a, bool bwd, cudaStream_t st) {
    return a.K == 2 ? go<T, 2>(a, bwd, st) : a.K == 3 ? go<T, 3>(a, bwd, st) : go<T, 4>(a, bwd, st);
}

template <typename T, int V, int K> cudaError_t run_step(const ConvStep &a, cudaStream_t st) {
    const long n = (long)(a.C / V) * a.B;
    conv_step_kernel<T, V, K><<<(unsigned)((n + kThreads - 1) / kThreads), kThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T, int K> cudaError_t go_step(const ConvStep &a, cudaStream_t st) {
    constexpr int V = kLane;
    const bool vec = a.C % V == 0 && by4<float>(a.w) && by4<float>(a.bias) && by4<T>(a.x) && by4<T>(a.y) && by4<T>(a.state) &&
                     (a.B == 1 || (a.xb % V == 0 && a.yb % V == 0));
    return vec ? run_step<T, V, K>(a, st) : run_step<T, 1, K>(a, st);
}
template <typename T> cudaError_t taps_step(const ConvStep &a, cudaStream_t st) {
    return a.K == 2 ? go_step<T, 2>(a, st) : a.K == 3 ? go_step<T, 3>(a, st) : go_step<T, 4>(a, st);
}

}  // namespace

cudaError_t launch_conv(const Conv &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? taps<__nv_bfloat16>(a, false, st) : taps<float>(a, false, st);
}
cudaError_t launch_conv_bwd(const Conv &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? taps<__nv_bfloat16>(a, true, st) : taps<float>(a, true, st);
}
cudaError_t launch_conv_step(const ConvStep &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? taps_step<__nv_bfloat16>(a, st) : taps_step<float>(a, st);
}

}  // namespace kda
