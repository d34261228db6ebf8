// ssm_bwd.cu -- gradients of the state space scan.
//
// With r_t = C_t . h_t + skip x_t, y_t = r_t silu(z_t), u_t = dt_t x_t, a_t = exp(dt_t A), p_t = dy_t silu(z_t):
//     g_t = C_t p_t + a_{t+1} g_{t+1}                      (the gradient of h_t; behind the last token dhT)
//     dC_t = sum_d p_t h_t,    dB_t = sum_d u_t g_t        (over the channels of the group)
//     s_t = g_t . B_t,   e_t = a_t g_t h_{t-1}
//     dx_t = dt_t s_t + skip p_t,   ddt_t = (x_t s_t + sum_n e_t A) softplus'(dt_t),   dz_t = dy_t r_t silu'(z_t)
//     dA = sum_t e_t dt_t,   dskip = sum p_t x_t,   dbias = sum ddt_t,   dh0 = a_1 g_1
#include <algorithm>

#include "ssm_internal.cuh"
#include "ssm_math.cuh"

namespace kda {
namespace {

constexpr int kThreads = 128;

template <typename T> __device__ __forceinline__ float at(const SsmView &v, long b, long t, long e) {
    return to_f32(static_cast<const T *>(v.p)[b * v.b + t * v.t + e]);
}
template <typename T> __device__ __forceinline__ void put(const SsmView &v, long b, long t, long e, float x) {
    static_cast<T *>(v.p)[b * v.b + t * v.t + e] = from_f32<T>(x);
}

template <typename T, int L>
__global__ void __launch_bounds__(kThreads) ssm_bwd_walk_kernel(Ssm a, int cpg, int bpg, long rows, float *kept, float *part,
                                                                float *pA, float *pd) {
    const int CH = kThreads / L, N = 4 * L;
    const int g = blockIdx.x / bpg, cb = blockIdx.x - g * bpg, cg = cb * CH + threadIdx.x / L, l = threadIdx.x % L;
    const bool live = cg < cpg;
    const int d = g * cpg + (live ? cg : 0), n = blockIdx.y;
    long start = 0, len = a.s.T, b = n, row0 = (long)n * a.s.T;
    if (a.s.cu) {
        start = min(max((long)a.s.cu[n], 0L), a.total);
        len = min(max((long)a.s.cu[n + 1] - a.s.cu[n], 0L), a.total - start);
        b = 0;
        row0 = 0;
    }
    float A[4], A2[4], h[4], G[4], dA[4];
    for (int i = 0; i < 4; ++i) {
        A[i] = a.A[(long)d * N + l + L * i];
        A2[i] = A[i] * kLog2eF;
        dA[i] = 0.f;
        h[i] = a.h0 ? a.h0[((long)n * a.D + d) * N + l + L * i] : 0.f;
        G[i] = a.dhT ? a.dhT[((long)n * a.D + d) * N + l + L * i] : 0.f;
    }
    const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
    auto step = [&](long t, float &raw) {
        raw = at<T>(a.dt, b, t, d) + bias;
        return a.softplus ? softplus<T>(raw) : raw;
    };
    auto keep = [&](long t, int i) -> float & { return kept[((row0 + t) * a.D + d) * N + l + L * i]; };
    for (long t = start; t < start + len; ++t) {
        float raw;
        const float dt = step(t, raw), u = dt * at<T>(a.x, b, t, d);
        for (int i = 0; i < 4; ++i) {
            if (live) keep(t, i) = h[i];
            h[i] = fmaf(ex2(dt * A2[i]), h[i], u * at<T>(a.B, b, t, g * a.B.g + l + L * i));
        }
    }
    float dskip = 0.f, dbias = 0.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, warps = bpg * (kThreads / 32);
    for (long t = start + len - 1; t >= start; --t) {
        float raw;
        const float dt = step(t, raw), x = at<T>(a.x, b, t, d), u = dt * x, dy = live ? at<T>(a.y, b, t, d) : 0.f;
        float p = dy, z = 0.f, sg = 1.f, rest = 0.f;
        if (a.gate.p) {
            z = at<T>(a.gate, b, t, d);
            sg = sigmoid<T>(z, rest);
            p *= z * sg;
        }
        float r = 0.f, s = 0.f, sA = 0.f, bc[8];
        for (int i = 0; i < 4; ++i) {
            const float Bn = at<T>(a.B, b, t, g * a.B.g + l + L * i), Cn = at<T>(a.C, b, t, g * a.C.g + l + L * i);
            const float was = live ? keep(t, i) : 0.f, al = ex2(dt * A2[i]), now = fmaf(al, was, u * Bn);
            r = fmaf(now, Cn, r);
            G[i] = fmaf(Cn, p, G[i]);
            bc[i] = live ? u * G[i] : 0.f;
            bc[4 + i] = live ? p * now : 0.f;
            s = fmaf(G[i], Bn, s);
            G[i] *= al;
            const float e = G[i] * was;
            sA = fmaf(e, A[i], sA);
            dA[i] = fmaf(e, dt, dA[i]);
        }
        for (int off = L / 2; off; off >>= 1) {
            r += __shfl_xor_sync(0xffffffffu, r, off);
            s += __shfl_xor_sync(0xffffffffu, s, off);
            sA += __shfl_xor_sync(0xffffffffu, sA, off);
        }
        r = fmaf(skip, x, r);
        float ddt = fmaf(x, s, sA), other;
        if (a.softplus) ddt *= sigmoid<T>(raw, other);
        dskip = fmaf(p, x, dskip);
        dbias += ddt;
        if (live && l == 0) {
            put<T>(a.dx, b, t, d, fmaf(dt, s, skip * p));
            put<T>(a.ddt, b, t, d, ddt);
            if (a.gate.p) put<T>(a.dgate, b, t, d, dy * r * fmaf(z * sg, rest, sg));
        }
        for (int k = 0; k < 8; ++k)
            for (int off = 16; off >= L; off >>= 1) bc[k] += __shfl_xor_sync(0xffffffffu, bc[k], off);
        if (lane < L)
            for (int k = 0; k < 8; ++k)
                part[(((long)(cb * (kThreads / 32) + warp) * rows + row0 + t) * a.G + g) * 2 * N + (k / 4) * N + l + L * (k % 4)] = bc[k];
    }
    (void)warps;
    if (!live) return;
    for (int i = 0; i < 4; ++i) {
        if (a.dh0) a.dh0[((long)n * a.D + d) * N + l + L * i] = G[i];
        pA[((long)n * a.D + d) * N + l + L * i] = dA[i];
    }
    if (l == 0) {
        pd[((long)n * 2) * a.D + d] = dskip;
        pd[((long)n * 2 + 1) * a.D + d] = dbias;
    }
}

// dB, dC of row blockIdx.x from the warps' parts; the last blocks: dA, dskip, dbias from the sequences'
template <typename T>
__global__ void __launch_bounds__(kThreads) ssm_fold_bc_kernel(Ssm a, long rows, int warps, const float *part) {
    const long row = blockIdx.x;
    const int n2 = a.G * 2 * a.N;
    if (a.s.cu && (row < a.s.cu[0] || row >= a.s.cu[a.s.nseq])) return;
    for (int e = threadIdx.x; e < n2; e += kThreads) {
        float v = 0.f;
        for (int w = 0; w < warps; ++w) v += part[((long)w * rows + row) * n2 + e];
        const int g = e / (2 * a.N), k = e % (2 * a.N);
        const long b = a.s.cu ? 0 : row / a.s.T, t = a.s.cu ? row : row % a.s.T;
        const SsmView &o = k < a.N ? a.dB : a.dC;
        static_cast<T *>(o.p)[b * o.b + t * o.t + g * o.g + k % a.N] = from_f32<T>(v);
    }
}
__global__ void __launch_bounds__(kThreads) ssm_fold_par_kernel(Ssm a, const float *pA, const float *pd) {
    const long id = blockIdx.x * (long)kThreads + threadIdx.x, nA = (long)a.D * a.N;
    float v = 0.f;
    if (id < nA) {
        for (int n = 0; n < a.s.nseq; ++n) v += pA[n * nA + id];
        a.dA[id] = v;
    } else if (id < nA + 2 * a.D) {
        const long k = id - nA;
        for (int n = 0; n < a.s.nseq; ++n) v += pd[(long)n * 2 * a.D + k];
        if (k < a.D) {
            if (a.dskip) a.dskip[k] = v;
        } else if (a.dbias) {
            a.dbias[k - a.D] = v;
        }
    }
}

struct Plan {
    long rows;
    int cpg, bpg, warps;
    size_t kept, part, pA, pd;
};
Plan plan(int nseq, long rows, int D, int G, int N) {
    Plan p{};
    const int L = N / 4, CH = kThreads / L;
    p.rows = rows;
    p.cpg = D / G;
    p.bpg = (p.cpg + CH - 1) / CH;
    p.warps = p.bpg * (kThreads / 32);
    p.kept = (size_t)rows * D * N;
    p.part = (size_t)p.warps * rows * G * 2 * N;
    p.pA = (size_t)nseq * D * N;
    p.pd = (size_t)nseq * 2 * D;
    return p;
}

template <typename T, int L> cudaError_t run(const Ssm &a, cudaStream_t st) {
    const long rows = a.s.cu ? a.total : (long)a.s.nseq * a.s.T;
    const Plan p = plan(a.s.nseq, rows, a.D, a.G, a.N);
    float *kept = static_cast<float *>(a.ws), *part = kept + p.kept, *pA = part + p.part, *pd = pA + p.pA;
    ssm_bwd_walk_kernel<T, L><<<dim3(p.bpg * a.G, a.s.nseq), kThreads, 0, st>>>(a, p.cpg, p.bpg, rows, kept, part, pA, pd);
    if (rows > 0) ssm_fold_bc_kernel<T><<<(unsigned)rows, kThreads, 0, st>>>(a, rows, p.warps, part);
    ssm_fold_par_kernel<<<(unsigned)(((long)a.D * (a.N + 2) + kThreads - 1) / kThreads), kThreads, 0, st>>>(a, pA, pd);
    return cudaGetLastError();
}
template <typename T> cudaError_t go(const Ssm &a, cudaStream_t st) {
    return a.N == 8 ? run<T, 2>(a, st) : a.N == 16 ? run<T, 4>(a, st) : a.N == 32 ? run<T, 8>(a, st) : run<T, 16>(a, st);
}

}  // namespace

size_t ssm_bwd_scratch_bytes(int nseq, long total, int max_len, bool varlen, int D, int G, int N, int) {
    const Plan p = plan(nseq, varlen ? total : (long)nseq * max_len, D, G, N);
    return 4 * (p.kept + p.part + p.pA + p.pd);
}
cudaError_t launch_ssm_bwd(const Ssm &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? go<__nv_bfloat16>(a, st) : go<float>(a, st);
}

}  // namespace kda
