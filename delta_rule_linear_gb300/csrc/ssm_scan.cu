// ssm_scan.cu -- the state space scan: prompts (equal lengths or packed) and single tokens.
//
//     dt_t = softplus(dt_t + bias),   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t . h_t + skip x_t) silu(gate_t)
//
// The decay differs by channel and state, so nothing here is a matrix product: per (token, channel, state) there is one
// exp2 and four multiply-adds.  An SM does 32 exp2 and 128 fp32 operations a cycle, which are 32 such cells either way;
// 152 SMs 9.3e12 a second.  With 16 states that is below the rate at which HBM brings x, dt, gate and takes y, so the
// scan is bound by issue and arithmetic, and the kernel keeps everything else away from the warps that do it.
//
// A CTA walks 128 / L channels of one sequence (L = N / 4 lanes hold a channel, four states each), 32 tokens a tile, with
// four warps that only scan and four that only serve them, one barrier a tile:
//   serving warps load tile s (x, dt, B, C; the loads go out a tile ahead), apply softplus, and leave dt, dt x, B and C as
//     fp32 in shared memory, tokens side by side; they add up the lanes' parts of tile s - 2, and store y after skip and gate;
//   scanning warps read four tokens of dt, dt x, B, C at a time and work on packed pairs of tokens (exponents, inputs and
//     outputs; the memory itself goes from token to token), and leave every lane's part of y in shared memory, since
//     adding it up over the lanes by shuffles would cost them four times what storing it does.
// Few channels and a long sequence: its parts ("segments") run side by side.  A first launch walks all but a sequence's last
// segment from an empty memory and leaves the memory and the sum of dt; in the second, every CTA joins those before it,
// h <- exp(A sum dt) h + local, which costs the walk of the memories (not of y) twice.
#include <algorithm>

#include "ssm_internal.cuh"
#include "ssm_math.cuh"

namespace kda {
namespace {

constexpr int kThreads = 256, kServe = 128;     // threads of a CTA; of them, those that serve
constexpr int kTile = 32;                       // tokens
constexpr int kPitch = kTile + 4;               // floats from row to row: rows start four banks apart

// Layout of the shared memory, in floats.  Pads keep the rows that a warp's lanes touch at once in different banks.
template <int L> struct Lay {
    static constexpr int N = 4 * L, CH = 128 / L;               // states, channels of a CTA
    static constexpr int VC = CH >= 32 ? 8 : CH / 4;            // channels that a serving lane loads together
    static constexpr int NQ = CH / VC;
    static constexpr int QPAD = L == 2 ? 4 : L == 4 ? 8 : L == 8 ? 24 : 0;
    static constexpr int LPAD = L == 2 ? 16 : L == 4 ? 8 : 4;
    static constexpr int ROWS = CH * kPitch + NQ * QPAD, HEADS = N * kPitch, PART = CH * kPitch + LPAD;
    static constexpr int IN = 2 * ROWS + 2 * HEADS, OUT = L * PART;
    static constexpr size_t bytes(bool local) { return (size_t)(2 * IN + (local ? 0 : 2 * OUT)) * 4; }
    static __device__ __forceinline__ int row(int c) { return c * kPitch + c / VC * QPAD; }
    static constexpr int PC = L <= 4 ? 2 : 1;                   // channels that a serving lane finishes together
    static constexpr int IN_TASKS = kTile * NQ / kServe, BC_TASKS = L / 2;
    static constexpr int OUT_TASKS = CH / PC * (kTile / 4) > kServe ? CH / PC * (kTile / 4) / kServe : 1;
};

struct Walk {
    Ssm a;
    int cpg, bpg, blocks;       // channels and CTAs of a group, CTAs of all
    int seg;                    // tokens of a segment
    long items;
    float *local, *sums;        // [items, D, N], [items, D]; nullptr where nothing is split
};

// The segment `item`, with the rows a packed batch has (whatever its prefix array says, none outside them is touched).
__device__ __forceinline__ bool walk_item(const Walk &w, long item, LinItem &it) {
    if (!lin_item(w.a.s, w.seg, (int)item, it)) return false;
    if (w.a.s.cu) {
        it.start = min(max(it.start, 0L), w.a.total);
        it.len = (int)min((long)max(it.len, 0), w.a.total - it.start);
    }
    return true;
}

// VEC: rows and heads start on boundaries of what a lane loads, and groups hold whole loads.
template <typename T, int L, bool VEC, bool LOCAL>
__global__ void __launch_bounds__(kThreads, 2) ssm_scan_kernel(const __grid_constant__ Walk w) {
    using Y = Lay<L>;
    extern __shared__ __align__(16) float smem[];
    const Ssm &a = w.a;
    const long item = blockIdx.x / w.blocks;
    const int cb = (int)(blockIdx.x - item * w.blocks), g = cb / w.bpg, c0 = (cb - g * w.bpg) * Y::CH;   // first channel in the group
    if (LOCAL) next_may_start();
    LinItem it;
    if (!walk_item(w, item, it) || (LOCAL && it.p == it.nseg - 1)) {
        if (!LOCAL && w.local) wait_for_previous();
        return;
    }
    const int t0 = min(it.p * w.seg, it.len), len = min(w.seg, it.len - t0), nt = (len + kTile - 1) / kTile;
    const int d0 = g * w.cpg + c0, live = min(Y::CH, w.cpg - c0);      // channels d0 .. d0 + live
    const long b = a.s.cu ? 0 : it.n, row0 = (a.s.cu ? it.start : 0) + t0;
    float *in = smem, *out = smem + 2 * Y::IN;

    if (threadIdx.x >= kServe) {        // ---------------------------------------------------------------- scan
        const int tid = threadIdx.x - kServe, c = tid / L, l = tid % L;
        const int d = d0 + min(c, live - 1);
        const long at = ((long)it.n * a.D + d) * Y::N + l;
        float h[4];
        Two A[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float x = a.A[(long)d * Y::N + l + L * i] * kLog2eF;
            A[i] = two(x, x);
            h[i] = !LOCAL && a.h0 ? a.h0[at + L * i] : 0.f;
        }
        if (!LOCAL && w.local) {
            wait_for_previous();
            for (int p = 0; p < it.p; ++p) {
                const long k = it.first + p;
                const float s = w.sums[k * a.D + d];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float A1, A2;
                    each(A[i], A1, A2);
                    h[i] = fmaf(ex2(s * A1), h[i], w.local[(k * a.D + d) * Y::N + l + L * i]);
                }
            }
        }
        Two sum = two(0.f, 0.f);
        for (int s = 0; s <= nt + (LOCAL ? 0 : 1); ++s) {
            __syncthreads();
            if (s < 1 || s > nt) continue;
            const float *base = in + ((s - 1) & 1) * Y::IN;
            const float *dtp = base + Y::row(c), *dxp = dtp + Y::ROWS, *Bp = base + 2 * Y::ROWS + l * kPitch, *Cp = Bp + Y::HEADS;
            float *op = out + ((s - 1) & 1) * Y::OUT + l * Y::PART + c * kPitch;
#pragma unroll 4
            for (int t = 0; t < kTile; t += 4) {
                const ulonglong2 dt = *reinterpret_cast<const ulonglong2 *>(dtp + t), dx = *reinterpret_cast<const ulonglong2 *>(dxp + t);
                if (LOCAL) sum = add2(sum, add2(dt.x, dt.y));
                ulonglong2 y = make_ulonglong2(0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const ulonglong2 B = *reinterpret_cast<const ulonglong2 *>(Bp + L * i * kPitch + t);
                    const Two p0 = mul2(dt.x, A[i]), p1 = mul2(dt.y, A[i]), u0 = mul2(dx.x, B.x), u1 = mul2(dx.y, B.y);
                    float e0, e1, e2, e3, v0, v1, v2, v3;
                    each(p0, e0, e1);
                    each(p1, e2, e3);
                    each(u0, v0, v1);
                    each(u1, v2, v3);
                    const float h0 = fmaf(ex2(e0), h[i], v0), h1 = fmaf(ex2(e1), h0, v1), h2 = fmaf(ex2(e2), h1, v2);
                    h[i] = fmaf(ex2(e3), h2, v3);
                    if (!LOCAL) {
                        const ulonglong2 C = *reinterpret_cast<const ulonglong2 *>(Cp + L * i * kPitch + t);
                        y.x = i ? fma2(two(h0, h1), C.x, y.x) : mul2(two(h0, h1), C.x);
                        y.y = i ? fma2(two(h2, h[i]), C.y, y.y) : mul2(two(h2, h[i]), C.y);
                    }
                }
                if (!LOCAL) *reinterpret_cast<ulonglong2 *>(op + t) = y;
            }
        }
        if (c >= live) return;
        if (LOCAL) {
#pragma unroll
            for (int i = 0; i < 4; ++i) w.local[(item * a.D + d) * Y::N + l + L * i] = h[i];
            float s0, s1;
            each(sum, s0, s1);
            if (l == 0) w.sums[item * a.D + d] = s0 + s1;
        } else if (a.hT && it.p == it.nseg - 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a.hT[at + L * i] = h[i];
        }
        return;
    }

    // ------------------------------------------------------------------------------------------------ serve
    const int tid = threadIdx.x, lane = tid & 31, warp = tid / 32;
    const int q = tid % Y::NQ, cq = q * Y::VC, tq = tid / Y::NQ;       // input: channels cq.., token tq (+ kServe / NQ)
    float bias[Y::VC];
#pragma unroll
    for (int i = 0; i < Y::VC; ++i) bias[i] = a.bias && cq + i < live ? a.bias[d0 + cq + i] : 0.f;
    const T *xp = static_cast<const T *>(a.x.p) + b * a.x.b + row0 * a.x.t + d0;
    const T *dp = static_cast<const T *>(a.dt.p) + b * a.dt.b + row0 * a.dt.t + d0;
    const T *zp = static_cast<const T *>(a.gate.p) + (a.gate.p ? b * a.gate.b + row0 * a.gate.t + d0 : 0);
    const T *Bp = static_cast<const T *>(a.B.p) + b * a.B.b + row0 * a.B.t + g * a.B.g;
    const T *Cp = static_cast<const T *>(a.C.p) + b * a.C.b + row0 * a.C.t + g * a.C.g;
    T *yp = LOCAL ? nullptr : static_cast<T *>(a.y.p) + b * a.y.b + row0 * a.y.t + d0;
    Few<T, Y::VC> rx[Y::IN_TASKS], rd[Y::IN_TASKS];
    Few<T, 4> rh[Y::BC_TASKS];
    auto fetch = [&](int s) {
#pragma unroll
        for (int j = 0; j < Y::IN_TASKS; ++j) {
            const int t = s * kTile + tq + j * (kServe / Y::NQ), n = t < len ? live - cq : 0;
            rx[j].template load<VEC>(xp + (long)t * a.x.t + cq, n);
            rd[j].template load<VEC>(dp + (long)t * a.dt.t + cq, n);
        }
#pragma unroll
        for (int j = 0; j < Y::BC_TASKS; ++j) {      // token = lane; quad of states = the rest, B's then C's
            const int k = warp + 4 * j, t = s * kTile + lane;
            const bool isB = k < L;
            if (LOCAL && !isB) continue;
            rh[j].template load<VEC>(isB ? Bp + (long)t * a.B.t + 4 * k : Cp + (long)t * a.C.t + 4 * (k - L), t < len ? 4 : 0);
        }
    };
    // output: PC channels from co on, tokens 4 to .. 4 to + 3 (of the task's)
    int co, to;
    if (L <= 4) {
        co = 2 * ((lane & 3) | (lane >> 3) << 2);
        to = (lane >> 2 & 1) | warp << 1;
    } else if (L == 8) {
        co = lane & 15;
        to = lane >> 4 | warp << 1;
    } else {
        co = lane & 7;
        to = lane >> 3 | warp << 2;
    }
    const bool finishes = to < kTile / 4;
    float skip[Y::OUT_TASKS][Y::PC];
    Few<T, Y::PC> ox[Y::OUT_TASKS][4], oz[Y::OUT_TASKS][4];
#pragma unroll
    for (int j = 0; j < Y::OUT_TASKS; ++j)
#pragma unroll
        for (int i = 0; i < Y::PC; ++i) {
            const int c = co + j * 32 + i;
            skip[j][i] = a.skip && c < live ? a.skip[d0 + c] : 0.f;
        }
    auto fetch_out = [&](int s) {
#pragma unroll
        for (int j = 0; j < Y::OUT_TASKS; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int t = s * kTile + 4 * to + k, c = co + j * 32, n = finishes && t < len ? live - c : 0;
                ox[j][k].template load<VEC>(xp + (long)t * a.x.t + c, n);
                if (a.gate.p) oz[j][k].template load<VEC>(zp + (long)t * a.gate.t + c, n);
            }
    };
    fetch(0);
    for (int s = 0; s <= nt + (LOCAL ? 0 : 1); ++s) {
        __syncthreads();
        if (s < nt) {
            float *base = in + (s & 1) * Y::IN;
#pragma unroll
            for (int j = 0; j < Y::IN_TASKS; ++j) {
                const int tt = tq + j * (kServe / Y::NQ);
                const bool there = s * kTile + tt < len;        // behind the last token the memory stays: dt = 0
#pragma unroll
                for (int i = 0; i < Y::VC; ++i) {
                    float v = rd[j][i] + bias[i];
                    if (a.softplus) v = softplus<T>(v);
                    v = there ? v : 0.f;
                    float *to_row = base + Y::row(cq + i) + tt;
                    to_row[0] = v;
                    to_row[Y::ROWS] = there ? v * rx[j][i] : 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < Y::BC_TASKS; ++j) {
                const int k = warp + 4 * j;
                if (LOCAL && k >= L) continue;
                float *to_row = base + 2 * Y::ROWS + (k < L ? 4 * k * kPitch : Y::HEADS + 4 * (k - L) * kPitch) + lane;
#pragma unroll
                for (int i = 0; i < 4; ++i) to_row[i * kPitch] = rh[j][i];
            }
            if (s + 1 < nt) fetch(s + 1);
        }
        if (!LOCAL) {
            if (s >= 2 && finishes) {
                const float *base = out + (s & 1) * Y::OUT;
#pragma unroll
                for (int j = 0; j < Y::OUT_TASKS; ++j) {
                    const int c = co + j * 32;
                    Two y[Y::PC][2];
#pragma unroll
                    for (int i = 0; i < Y::PC; ++i) {
                        y[i][0] = y[i][1] = two(0.f, 0.f);
#pragma unroll
                        for (int l = 0; l < L; ++l) {
                            const ulonglong2 v = *reinterpret_cast<const ulonglong2 *>(base + l * Y::PART + (c + i) * kPitch + 4 * to);
                            y[i][0] = l ? add2(y[i][0], v.x) : v.x;
                            y[i][1] = l ? add2(y[i][1], v.y) : v.y;
                        }
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const int t = (s - 2) * kTile + 4 * to + k;
                        float v[Y::PC];
#pragma unroll
                        for (int i = 0; i < Y::PC; ++i) {
                            float v0, v1;
                            each(y[i][k / 2], v0, v1);
                            v[i] = fmaf(skip[j][i], ox[j][k][i], k & 1 ? v1 : v0);
                            if (a.gate.p) {
                                const float z = oz[j][k][i];
                                float rest;
                                v[i] *= z * sigmoid<T>(z, rest);
                            }
                        }
                        Few<T, Y::PC>::template store<VEC>(yp + (long)t * a.y.t + c, v, t < len ? live - c : 0);
                    }
                }
            }
            if (s >= 1 && s <= nt) fetch_out(s - 1);
        }
    }
}

constexpr int kStepThreads = 128;

template <typename T, int L>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(SsmStep a) {
    const int CH = kStepThreads / L, N = 4 * L;
    const int d0 = blockIdx.x * CH + threadIdx.x / L, l = threadIdx.x % L, n = blockIdx.y;
    const bool live = d0 < a.D;
    const int d = live ? d0 : 0, g = d / (a.D / a.G);
    auto val = [](const void *p, long i) { return to_f32(static_cast<const T *>(p)[i]); };
    float dt = val(a.dt, n * a.dtb + d) + (a.bias ? a.bias[d] : 0.f);
    if (a.softplus) dt = softplus<T>(dt);
    const float x = val(a.x, n * a.xb + d), u = dt * x;
    float *sp = a.state + ((long)n * a.D + d) * N + 4 * l;
    const float4 s = *reinterpret_cast<const float4 *>(sp);
    const float4 A = *reinterpret_cast<const float4 *>(a.A + (long)d * N + 4 * l);
    float h[4] = {s.x, s.y, s.z, s.w}, y = 0.f;
    const float Av[4] = {A.x, A.y, A.z, A.w};
    for (int i = 0; i < 4; ++i) {
        h[i] = fmaf(ex2(dt * (Av[i] * kLog2eF)), h[i], u * val(a.B, n * a.Bb + g * a.Bg + 4 * l + i));
        y = fmaf(h[i], val(a.C, n * a.Cb + g * a.Cg + 4 * l + i), y);
    }
    for (int off = L / 2; off; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
    if (!live) return;
    *reinterpret_cast<float4 *>(sp) = make_float4(h[0], h[1], h[2], h[3]);
    y = fmaf(a.skip ? a.skip[d] : 0.f, x, y);
    if (a.gate) {
        float z = val(a.gate, n * a.gb + d), rest;
        y *= z * sigmoid<T>(z, rest);
    }
    if (l == 0) static_cast<T *>(a.y)[n * a.yb + d] = from_f32<T>(y);
}

template <typename T> bool few_view(const SsmView &v, int n, bool heads) {      // rows start where n elements may be loaded at once
    const size_t bytes = std::min<size_t>(16, n * sizeof(T));
    const long long u = (long long)(bytes / sizeof(T));
    return !v.p || (reinterpret_cast<uintptr_t>(v.p) % bytes == 0 && v.b % u == 0 && v.t % u == 0 && (!heads || v.g % u == 0));
}

// Tokens of a segment: as many as a CTA would walk if the work were spread evenly, unless the longest sequence is not
// much longer than that.  0: no splitting.
int pick_segment(const Ssm &a, long rows, int max_len, int blocks) {
    const long even = rows * blocks / (2L * a.sms);
    if (max_len <= 256 || max_len <= 3 * even) return 0;
    return (int)std::max(128L, (even + kTile - 1) / kTile * kTile);
}
long split_items(int nseq, long rows, int blocks, int sms) {      // of any segment that pick_segment gives
    const long seg = std::max(128L, rows * blocks / (2L * sms));
    return rows / seg + nseq;
}

template <int L> int blocks_of(int D, int G) { return (D / G + Lay<L>::CH - 1) / Lay<L>::CH * G; }

template <typename T, int L, bool VEC> cudaError_t launch(const Ssm &a, cudaStream_t st) {
    using Y = Lay<L>;
    Walk w{};
    w.a = a;
    w.cpg = a.D / a.G;
    w.bpg = (w.cpg + Y::CH - 1) / Y::CH;
    w.blocks = w.bpg * a.G;
    const long rows = a.s.cu ? a.total : (long)a.s.nseq * a.s.T;
    const int max_len = a.s.cu ? a.max_len : a.s.T;
    w.seg = a.hT && a.hT == a.h0 ? 0 : pick_segment(a, rows, max_len, w.blocks);
    const bool split = w.seg > 0;
    if (!split) w.seg = std::max(max_len, 1);
    w.items = lin_items(a.s.nseq, a.s.cu ? a.total : a.s.T, max_len, a.s.cu != nullptr, w.seg);
    const long ctas = w.items * w.blocks;
    if (ctas > 0x7fffffffL) return cudaErrorInvalidValue;
    if (split) {
        w.local = static_cast<float *>(a.ws);
        w.sums = w.local + w.items * (long)a.D * a.N;
        const auto first = ssm_scan_kernel<T, L, VEC, true>;
        cudaError_t e = cudaFuncSetAttribute(first, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Y::bytes(true));
        if (e != cudaSuccess) return e;
        first<<<(unsigned)ctas, kThreads, Y::bytes(true), st>>>(w);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    const auto main = ssm_scan_kernel<T, L, VEC, false>;
    cudaError_t e = cudaFuncSetAttribute(main, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)Y::bytes(false));
    if (e != cudaSuccess) return e;
    if (split) return launch_after(main, dim3((unsigned)ctas), kThreads, Y::bytes(false), st, w);
    main<<<(unsigned)ctas, kThreads, Y::bytes(false), st>>>(w);
    return cudaGetLastError();
}

template <typename T, int L> cudaError_t run(const Ssm &a, cudaStream_t st) {
    using Y = Lay<L>;
    const int cpg = a.D / a.G;
    const bool vec = cpg % Y::VC == 0 && few_view<T>(a.x, Y::VC, false) && few_view<T>(a.dt, Y::VC, false) &&
                     few_view<T>(a.gate, Y::VC, false) && few_view<T>(a.y, Y::VC, false) && few_view<T>(a.B, 4, true) &&
                     few_view<T>(a.C, 4, true);
    return vec ? launch<T, L, true>(a, st) : launch<T, L, false>(a, st);
}
template <typename T, int L> cudaError_t run_step(const SsmStep &a, cudaStream_t st) {
    ssm_step_kernel<T, L><<<dim3((a.D * L + kStepThreads - 1) / kStepThreads, a.nb), kStepThreads, 0, st>>>(a);
    return cudaGetLastError();
}
template <typename T> cudaError_t go(const Ssm &a, cudaStream_t st) {
    return a.N == 8 ? run<T, 2>(a, st) : a.N == 16 ? run<T, 4>(a, st) : a.N == 32 ? run<T, 8>(a, st) : run<T, 16>(a, st);
}
template <typename T> cudaError_t go_step(const SsmStep &a, cudaStream_t st) {
    return a.N == 8 ? run_step<T, 2>(a, st) : a.N == 16 ? run_step<T, 4>(a, st) : a.N == 32 ? run_step<T, 8>(a, st) : run_step<T, 16>(a, st);
}

}  // namespace

size_t ssm_scratch_bytes(int nseq, long total, int max_len, bool varlen, int D, int G, int N, int sms) {
    const int blocks = N == 8 ? blocks_of<2>(D, G) : N == 16 ? blocks_of<4>(D, G) : N == 32 ? blocks_of<8>(D, G) : blocks_of<16>(D, G);
    if (max_len <= 256) return 0;
    return (size_t)split_items(nseq, varlen ? total : (long)nseq * max_len, blocks, sms) * D * (N + 1) * 4;
}
cudaError_t launch_ssm(const Ssm &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? go<__nv_bfloat16>(a, st) : go<float>(a, st);
}
cudaError_t launch_ssm_step(const SsmStep &a, cudaStream_t st) {
    return a.dtype == DType::BF16 ? go_step<__nv_bfloat16>(a, st) : go_step<float>(a, st);
}

}  // namespace kda
