// ssm_scan.cu -- the state space scan: prompts (equal lengths or packed) and single tokens.
//
//     dt_t = softplus(dt_t + bias),   h_t = exp(dt_t A) h_{t-1} + dt_t x_t B_t,   y_t = (C_t . h_t + skip x_t) silu(gate_t)
//
// The decay differs by channel and state, so the recurrence is no matrix product: per (token, channel, state) there is one
// exp2 and four multiply-adds.  An SM does 32 exp2 and 128 fp32 operations a cycle, which are 32 such cells either way;
// 152 SMs 9.3e12 a second.  With 16 states that is below the rate at which HBM brings x, dt, gate and takes y, so the
// scan is bound by issue and arithmetic, and everything else is kept away from the warps that do it.
//
// What they would wait for is shared memory: a load delivers 128 bytes a cycle to an SM whatever is the same in them, and
// B_t, C_t are wanted by every channel (8 bytes a cell: 40 cycles a token of 32 channels, where the arithmetic takes 17).  So
// the tensor cores spread them: D = E X with E [128 lanes, 16] one-hot rows that pick a lane's states and X [16, columns]
// the tokens' B and C as they lie in memory puts each lane's B and C into its TMEM row, as fp32 and exactly (one term
// of the sum is not zero; fp32 inputs go in as three bf16 parts), and tcgen05.ld reads TMEM beside the shared memory.
//
// A group of eight warps walks 128 / L channels of one sequence (L = N / 4 lanes hold a channel, four states each), 32 tokens
// a tile; four of its warps only scan and four only serve them, one barrier a tile:
//   serving warps load tiles ahead into a ring, lay B and C out and issue their product, apply softplus, and leave dt and
//     dt x as fp32 in shared memory, tokens side by side; they add up the lanes' parts of tile s - 2, and store y after skip
//     and gate;
//   scanning warps work on packed pairs of tokens (exponents, inputs, outputs; the memory itself goes from token to token)
//     and leave every lane's part of y in shared memory: adding it up by shuffles would cost four times what storing does.
// A CTA is one group, or two (over the same B and C) where there are more blocks of channels than SMs; it takes all of
// TMEM (two tiles of 256 columns), so there is one to an SM.
// Few channels and a long sequence: its parts ("segments") run side by side.  A first launch walks all but a sequence's last
// segment from an empty memory and leaves the memory and the sum of dt; in the second, every CTA joins those before it,
// h <- exp(A sum dt) h + local, which costs the walk of the memories (not of y) twice.
//
// Measured, bf16, 16 states, gated: 2 x 2048 tokens of 4096 channels 103 us (the cells alone 29 us, HBM 20; an earlier form with
// B and C from shared memory 156), 32,768 tokens 932 us (230 and 158); 0.65 of the issue slots in the former.  Per tile of the latter
// the scanning warps alone take 0.58 us, with what serves them 0.91.
#include <algorithm>

#include "linear_tc.cuh"
#include "run_item.cuh"
#include "ssm_internal.cuh"
#include "ssm_math.cuh"

namespace kda {
namespace {

using lin::Waits;
using namespace ptx;

constexpr int kServe = 128;                     // threads of a group that serve (as many scan)
constexpr int kTile = 32;                       // tokens
constexpr int kPitch = kTile + 4;               // floats from row to row: rows start four banks apart

// Layout of the shared memory, in floats.  Pads keep the rows that a warp's lanes touch at once in different banks.
template <typename T, int L> struct Lay {
    static constexpr int N = 4 * L, CH = 128 / L;               // states, channels of a group
    static constexpr int VC = CH >= 32 ? 8 : CH / 4;            // channels that a serving lane loads together
    static constexpr int NQ = CH / VC;
    static constexpr int QPAD = L == 2 ? 4 : L == 4 ? 8 : L == 8 ? 24 : 0;
    static constexpr int LPAD = L == 2 ? 16 : L == 4 ? 8 : 4;
    static constexpr int ROWS = CH * kPitch + NQ * QPAD, PART = ROWS + LPAD;
    static constexpr int IN = 2 * ROWS, OUT = L * PART;         // per group, two of each
    static __device__ __forceinline__ int row(int c) { return c * kPitch + c / VC * QPAD; }
    static constexpr int TASKS = kTile * NQ / kServe, BC_TASKS = L / 2;     // loads of a serving lane and tile
    // What serving lanes have loaded, in a ring of tiles: x (from two tiles back on, for the output), dt, gate; B and C.
    using Rows = Own<T, VC, kServe>;
    using Quad = Own<T, 4, kServe>;
    static constexpr int RING = sizeof(T) == 2 ? 5 : L == 2 || L == 16 ? 4 : 5, AHEAD = RING - 3;      // as many as fit
    static constexpr int RAW = 3 * TASKS * Rows::SIZE, RAW_BC = BC_TASKS * Quad::SIZE;      // bytes of a tile
    // The product's operands: rows of 128 bytes (K-major, 128-byte swizzle) whose four K steps of 16 hold tile buffer 0,
    // buffer 1 and E, KS steps each; a block of rows more for every four steps.
    static constexpr int PARTS = sizeof(T) == 2 ? 1 : 3, KS = (PARTS * L + 15) / 16, BLOCKS = (3 * KS + 3) / 4;
    static constexpr int XROWS(bool local) { return local ? 128 : 256; }
    static constexpr size_t bytes(int groups, bool local) {
        return 1024 + (size_t)BLOCKS * XROWS(local) * 128 + (size_t)RING * RAW_BC +
               (size_t)groups * ((2 * IN + (local ? 0 : 2 * OUT)) * 4 + RING * RAW);
    }
};

struct Walk {
    Ssm a;
    int cpg, bpg, blocks;       // channels and CTAs of a group of heads, CTAs of all
    int seg;                    // tokens of a segment (of any number where nothing is split)
    int pairs;                  // every array can be read by two elements
    long items;
    float *local, *sums;        // [items, D, N], [items, D]; nullptr where nothing is split
    WsHeader *hdr;
};

struct Ctl {
    uint64_t full[2];           // the tile's product is in TMEM
    uint32_t tmem;
    int fail;
};

// The segment `item`; where nothing is split, the sequence.  (Whatever a prefix array says, no row outside the batch is touched.)
__device__ __forceinline__ bool walk_item(const Walk &w, long item, LinItem &it) {
    const LinSeqs &s = w.a.s;
    if (w.local) return run_item(s, w.a.total, w.seg, item, it);
    it.n = it.first = (int)item;
    it.p = 0;
    it.nseg = 1;
    it.start = s.cu ? min(max((long)s.cu[it.n], 0L), w.a.total) : (long)it.n * s.T;
    it.len = s.cu ? (int)max(min((long)s.cu[it.n + 1], w.a.total) - it.start, 0L) : s.T;
    return true;
}

// Byte of K element k (16 a step) of row r, step `slot`, in the operands.
__device__ __forceinline__ uint32_t op_byte(int rows, int r, int slot, int k) {
    const int chunk = (slot & 3) * 2 + (k >> 3);
    return (uint32_t)((slot >> 2) * rows * 128 + r * 128 + ((chunk ^ (r & 7)) << 4) + (k & 7) * 2);
}
__device__ __forceinline__ uint64_t op_desc(uint32_t base, int rows, int slot) {
    return smem_desc(base + (uint32_t)((slot >> 2) * rows * 128 + (slot & 3) * 32), 16u, 1024u, kSwizzle128B);
}

// What a lane has asked of TMEM is there: nothing that uses it may come before.
template <int N> __device__ __forceinline__ void landed(uint32_t (&r)[N]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;");
#pragma unroll
    for (int i = 0; i < N; ++i) asm volatile("" : "+r"(r[i]));
}

// Threads of a CTA.  A lone group has few warps to change between, so what serves is split: four warps each for x and dt, for
// the outputs, and for B and C.
constexpr int threads_of(bool local, int groups) { return !local && groups == 1 ? 512 : 256 * groups; }

// VEC: rows and heads start on boundaries of what a lane loads, and groups hold whole loads.
template <typename T, int L, bool VEC, bool LOCAL, int GROUPS>
__global__ void __launch_bounds__(threads_of(LOCAL, GROUPS), 1) ssm_scan_kernel(const __grid_constant__ Walk w) {
    using Y = Lay<T, L>;
    constexpr int THREADS = threads_of(LOCAL, GROUPS), GT = THREADS / GROUPS;
    constexpr bool SPLIT = GT == 512;
    constexpr int HEADS = SPLIT ? 3 : 1;        // the role that brings B and C
    constexpr int XR = Y::XROWS(LOCAL), W = LOCAL ? 4 : 8;      // columns of X: 4 W of every four tokens, W of a state
    constexpr uint32_t COLS = LOCAL ? 256 : 512;
    extern __shared__ __align__(1024) uint8_t raw[];
    __shared__ Ctl ctl;
    const Ssm &a = w.a;
    const long item = blockIdx.x / w.blocks;
    const int cb = (int)(blockIdx.x - item * w.blocks), g = cb / w.bpg, sub = threadIdx.x / GT;
    const int c0 = ((cb - g * w.bpg) * GROUPS + sub) * Y::CH;           // the group's first channel among its heads'
    const int role = threadIdx.x % GT / 128;                            // 0 scan, 1 serve (SPLIT: x and dt), 2 the outputs, 3 B and C
    const int tid = threadIdx.x & 127, lane = tid & 31, warp = tid / 32;
    LinItem it;
    if (blockIdx.x == 0 && threadIdx.x == 0 && (LOCAL || !w.local)) w.hdr->error = 0;       // (no wait can run out this early)
    if (!walk_item(w, item, it) || (LOCAL && it.p == it.nseg - 1)) {
        if (LOCAL) next_may_start();
        if (!LOCAL && w.local) wait_for_previous();
        return;
    }
    const uint32_t x_base = (smem_u32(raw) + 1023u) & ~1023u;
    uint8_t *xs = raw + (x_base - smem_u32(raw));
    constexpr int GROUP = (2 * Y::IN + (LOCAL ? 0 : 2 * Y::OUT)) * 4 + Y::RING * Y::RAW;
    uint8_t *ring_bc = xs + Y::BLOCKS * XR * 128, *ring = ring_bc + Y::RING * Y::RAW_BC + sub * GROUP;
    float *in = reinterpret_cast<float *>(ring + Y::RING * Y::RAW), *out = in + 2 * Y::IN;
    if (threadIdx.x == 0) {
        mbar_init(&ctl.full[0], 1);
        mbar_init(&ctl.full[1], 1);
        ctl.fail = 0;
        fence_mbar_init();
    }
    for (int i = threadIdx.x; i < Y::BLOCKS * XR * 8; i += THREADS) reinterpret_cast<uint4 *>(xs)[i] = make_uint4(0, 0, 0, 0);
    fence_proxy_async();
    if (threadIdx.x >= 224 && threadIdx.x < 256) {
        tmem_alloc(&ctl.tmem, COLS);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (LOCAL) next_may_start();        // behind the allocation
    const uint32_t tm = ctl.tmem;
    if (threadIdx.x < 128) {            // E: lane m has state l of each quad, in all parts
#pragma unroll
        for (int p = 0; p < Y::PARTS; ++p) {
            const int k = p * L + tid % L;
            *reinterpret_cast<__nv_bfloat16 *>(xs + op_byte(XR, tid, 2 * Y::KS + k / 16, k & 15)) = __float2bfloat16_rn(1.f);
        }
        fence_proxy_async();
    }
    const Waits wt{&ctl.fail, w.hdr};
    const int t0 = min(it.p * w.seg, it.len), len = min(w.seg, it.len - t0), nt = (len + kTile - 1) / kTile;
    const int d0 = g * w.cpg + c0, live = min(Y::CH, w.cpg - c0);      // channels d0 .. d0 + live (none: live <= 0)
    const long b = a.s.cu ? 0 : it.n, row0 = (a.s.cu ? it.start : 0) + t0;
    const int last = nt + (LOCAL ? 0 : 1);

    if (role == 0) {    // ------------------------------------------------------------------------------------- scan
        const int c = tid / L, l = tid % L;
        const int d = min(d0 + min(c, max(live - 1, 0)), a.D - 1);
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
        const uint32_t mine = tm + ((uint32_t)(32 * warp) << 16);
        for (int s = 0; s <= last; ++s) {
            tc_fence_before();
            __syncthreads();
            if (s < 1 || s > nt) continue;
            const int k = s - 1;
            const float *dtp = in + (k & 1) * Y::IN + Y::row(c), *dxp = dtp + Y::ROWS;
            float *op = out + (k & 1) * Y::OUT + l * Y::PART + Y::row(c);
            const uint32_t from = mine + (k & 1) * XR;
            // The factors of the next four tokens are formed beside the memories of these, state by state: four exp2 hold their
            // unit for 16 cycles, as long as the chain of four multiply-adds takes.
            uint32_t bc[2][4 * W];
            float f[2][4][4];
            auto ask = [&](int t4) {
                if constexpr (LOCAL)
                    tmem_ld16(from + t4 * 16, bc[t4 & 1]);
                else
                    tmem_ld32(from + t4 * 32, bc[t4 & 1]);
            };
            auto factors = [&](const ulonglong2 &dt, int i, float (&e)[4]) {
                each(mul2(dt.x, A[i]), e[0], e[1]);
                each(mul2(dt.y, A[i]), e[2], e[3]);
#pragma unroll
                for (int k = 0; k < 4; ++k) e[k] = ex2(e[k]);
            };
            ulonglong2 dt = *reinterpret_cast<const ulonglong2 *>(dtp), dx = *reinterpret_cast<const ulonglong2 *>(dxp), dx_next = dx;
#pragma unroll
            for (int i = 0; i < 4; ++i) factors(dt, i, f[0][i]);
            wt.warp(&ctl.full[k & 1], (k >> 1) & 1, 1);
            tc_fence_after();
            ask(0);
#pragma unroll
            for (int t4 = 0; t4 < kTile / 4; ++t4) {
                const bool more = t4 + 1 < kTile / 4;
                if (LOCAL) sum = add2(sum, add2(dt.x, dt.y));
                if (more) {
                    dt = *reinterpret_cast<const ulonglong2 *>(dtp + 4 * t4 + 4);
                    dx_next = *reinterpret_cast<const ulonglong2 *>(dxp + 4 * t4 + 4);
                }
                uint32_t(&r)[4 * W] = bc[t4 & 1];
                landed(r);
                if (more) ask(t4 + 1);
                auto col = [&](int k0) { return two(__uint_as_float(r[k0]), __uint_as_float(r[k0 + 1])); };
                ulonglong2 y = make_ulonglong2(0, 0);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float(&e)[4] = f[t4 & 1][i];
                    float v0, v1, v2, v3;
                    each(mul2(dx.x, col(W * i)), v0, v1);
                    each(mul2(dx.y, col(W * i + 2)), v2, v3);
                    if (more) factors(dt, i, f[(t4 + 1) & 1][i]);
                    const float h0 = fmaf(e[0], h[i], v0), h1 = fmaf(e[1], h0, v1), h2 = fmaf(e[2], h1, v2);
                    h[i] = fmaf(e[3], h2, v3);
                    if constexpr (!LOCAL) {
                        y.x = i ? fma2(two(h0, h1), col(W * i + 4), y.x) : mul2(two(h0, h1), col(W * i + 4));
                        y.y = i ? fma2(two(h2, h[i]), col(W * i + 6), y.y) : mul2(two(h2, h[i]), col(W * i + 6));
                    }
                }
                if (!LOCAL) *reinterpret_cast<ulonglong2 *>(op + 4 * t4) = y;
                dx = dx_next;
            }
        }
        if (c < live) {
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
        }
    } else {            // ------------------------------------------------------------------------------------- serve
        const int q = tid % Y::NQ, cq = q * Y::VC, tq = tid / Y::NQ;       // channels cq .. cq + VC, token tq (+ kServe / NQ)
        float bias[Y::VC], skip[Y::VC];
#pragma unroll
        for (int i = 0; i < Y::VC; ++i) {
            bias[i] = a.bias && cq + i < live ? a.bias[d0 + cq + i] : 0.f;
            skip[i] = a.skip && cq + i < live ? a.skip[d0 + cq + i] : 0.f;
        }
        using Rows = typename Y::Rows;
        using Quad = typename Y::Quad;
        constexpr int NEXT = kServe / Y::NQ;        // tokens from a lane's load to its next
        // the lane's places in the tile that is fetched next, and in the one that is finished next
        const T *xp = static_cast<const T *>(a.x.p) + b * a.x.b + (row0 + tq) * a.x.t + d0 + cq;
        const T *dp = static_cast<const T *>(a.dt.p) + b * a.dt.b + (row0 + tq) * a.dt.t + d0 + cq;
        const T *zp = a.gate.p ? static_cast<const T *>(a.gate.p) + b * a.gate.b + (row0 + tq) * a.gate.t + d0 + cq : nullptr;
        const T *hp[Y::BC_TASKS];       // B and C: token = lane; quad of states = the rest, B's then C's
#pragma unroll
        for (int j = 0; j < Y::BC_TASKS; ++j) {
            const int k = warp + 4 * j;
            const SsmView &v = k < L ? a.B : a.C;
            hp[j] = static_cast<const T *>(v.p) + b * v.b + (row0 + lane) * v.t + g * v.g + 4 * (k < L ? k : k - L);
        }
        T *yp = LOCAL ? nullptr : static_cast<T *>(a.y.p) + b * a.y.b + (row0 + tq) * a.y.t + d0 + cq;
        const bool gated = zp != nullptr;
        int to_fetch = 0;               // tokens of the tiles fetched so far
        uint8_t *slot_in = ring, *slot_bc = ring_bc;
        auto fetch = [&]() {
            if (to_fetch < len) {
                uint8_t *slot = slot_in;
#pragma unroll
                for (int j = 0; j < Y::TASKS; ++j, slot += 3 * Rows::SIZE) {
                    const int n = to_fetch + tq + j * NEXT < len ? live - cq : 0;
                    if (!SPLIT || role == 1) {
                        Rows::template fetch<VEC>(slot, tid, xp + (long)(j * NEXT) * a.x.t, n, w.pairs);
                        Rows::template fetch<VEC>(slot + Rows::SIZE, tid, dp + (long)(j * NEXT) * a.dt.t, n, w.pairs);
                    }
                    if (!LOCAL && gated && (!SPLIT || role == 2)) Rows::template fetch<VEC>(slot + 2 * Rows::SIZE, tid, zp + (long)(j * NEXT) * a.gate.t, n, w.pairs);
                }
                if (!sub && role == HEADS) {
#pragma unroll
                    for (int j = 0; j < Y::BC_TASKS; ++j) {
                        const bool isB = warp + 4 * j < L;
                        if (LOCAL && !isB) continue;
                        Quad::template fetch<VEC>(slot_bc + j * Quad::SIZE, tid, hp[j], to_fetch + lane < len ? 4 : 0, w.pairs);
                        hp[j] += (long)kTile * (isB ? a.B.t : a.C.t);
                    }
                }
                to_fetch += kTile;
                xp += kTile * a.x.t;
                dp += kTile * a.dt.t;
                if (gated) zp += kTile * a.gate.t;
                const bool round = slot_in == ring + (Y::RING - 1) * Y::RAW;
                slot_in = round ? ring : slot_in + Y::RAW;
                slot_bc = round ? ring_bc : slot_bc + Y::RAW_BC;
            }
            copies_commit();
        };
        const uint8_t *slot_s = ring, *slot_s_bc = ring_bc, *slot_out = ring;      // of tile s, and of tile s - 2
        auto on = [&](const uint8_t *&slot, const uint8_t *first, int size) { slot = slot == first + (Y::RING - 1) * size ? first : slot + size; };
#pragma unroll
        for (int s = 0; s < Y::AHEAD; ++s) fetch();
        for (int s = 0; s <= last; ++s) {
            __syncthreads();
            copies_wait<Y::AHEAD - 1>();
            const int P = s & 1;
            if (s < nt) {
                if (!sub && role == HEADS) {        // B and C into the operand's rows (token, state, B or C), parts of L states side by side
                    const uint8_t *slot = slot_s_bc;
                    on(slot_s_bc, ring_bc, Y::RAW_BC);
#pragma unroll
                    for (int j = 0; j < Y::BC_TASKS; ++j) {
                        const int k = warp + 4 * j, quad = k < L ? k : k - L;
                        if (LOCAL && k >= L) continue;
                        const Few<T, 4> f = Quad::read(slot + j * Quad::SIZE, tid);
                        const int r0 = (lane >> 2) * 4 * W + (k < L ? 0 : 4) + (lane & 3);
#pragma unroll
                        for (int e = 0; e < 4; e += 2) {        // states 4 quad + e and the next: column i, K element l
                            const int n = 4 * quad + e, i = n / L, l = n % L;
                            if constexpr (sizeof(T) == 2) {
                                *reinterpret_cast<uint32_t *>(xs + op_byte(XR, r0 + i * W, P * Y::KS, l)) = f.w[e / 2];
                            } else {
                                float u = f[e], v = f[e + 1];
#pragma unroll
                                for (int p = 0; p < Y::PARTS; ++p) {
                                    const int kk = p * L + l;
                                    *reinterpret_cast<uint32_t *>(xs + op_byte(XR, r0 + i * W, P * Y::KS + kk / 16, kk & 15)) = lin::top2(u, v);
                                    u = lin::rest(u);
                                    v = lin::rest(v);
                                }
                            }
                        }
                    }
                    fence_proxy_async();
                    lin::named_sync(1, kServe);
                    if (tid == 0) {
                        tc_fence_after();
                        constexpr uint32_t id = idesc_bf16_f32(128, XR, false, false);
#pragma unroll
                        for (int p = 0; p < Y::KS; ++p) {
                            const uint64_t e = op_desc(x_base, XR, 2 * Y::KS + p), x = op_desc(x_base, XR, P * Y::KS + p);
                            if (p)
                                mma_ss<1>(tm + P * XR, e, x, id);
                            else
                                mma_ss<0>(tm + P * XR, e, x, id);
                        }
                        mma_commit(&ctl.full[P]);
                    }
                }
            }
            if (s < nt && role == 1) {
                float *base = in + P * Y::IN;
                const uint8_t *slot = slot_s;
                on(slot_s, ring, Y::RAW);
                const bool whole = (s + 1) * kTile <= len;
#pragma unroll
                for (int j = 0; j < Y::TASKS; ++j) {
                    const int tt = tq + j * NEXT;
                    const bool there = whole || s * kTile + tt < len;       // behind the last token the memory stays: dt = 0
                    const Few<T, Y::VC> x = Rows::read(slot + 3 * j * Rows::SIZE, tid), d = Rows::read(slot + (3 * j + 1) * Rows::SIZE, tid);
#pragma unroll
                    for (int i = 0; i < Y::VC; i += 2) {
                        float v[2] = {d[i] + bias[i], d[i + 1] + bias[i + 1]};
                        if (a.softplus) softplus<T>(v[0], v[1]);
                        float u[2] = {v[0] * x[i], v[1] * x[i + 1]};
                        if (!whole) {
#pragma unroll
                            for (int k = 0; k < 2; ++k) v[k] = there ? v[k] : 0.f, u[k] = there ? u[k] : 0.f;
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float *to_row = base + Y::row(cq + i + k) + tt;
                            to_row[0] = v[k];
                            to_row[Y::ROWS] = u[k];
                        }
                    }
                }
            }
            if (!LOCAL && s >= 2 && (!SPLIT || role == 2)) {
                const float *base = out + P * Y::OUT;
                const uint8_t *slot = slot_out;
                on(slot_out, ring, Y::RAW);
#pragma unroll
                for (int j = 0; j < Y::TASKS; ++j) {
                    const int tt = tq + j * NEXT, t = (s - 2) * kTile + tt;
                    const Few<T, Y::VC> x = Rows::read(slot + 3 * j * Rows::SIZE, tid);
                    Few<T, Y::VC> z;
                    if (gated) z = Rows::read(slot + (3 * j + 2) * Rows::SIZE, tid);
                    float v[Y::VC];
#pragma unroll
                    for (int i = 0; i < Y::VC; ++i) {
                        const float *part = base + Y::row(cq + i) + tt;
                        v[i] = part[0];
#pragma unroll
                        for (int l = 1; l < L; ++l) v[i] += part[l * Y::PART];
                        v[i] = fmaf(skip[i], x[i], v[i]);
                        if (gated) {
                            float rest;
                            v[i] *= z[i] * sigmoid<T>(z[i], rest);
                        }
                    }
                    Few<T, Y::VC>::template store<VEC>(yp + (long)(j * NEXT) * a.y.t, v, t < len ? live - cq : 0);
                }
                yp += kTile * a.y.t;
            }
            fetch();
        }
    }
    tc_fence_before();
    __syncthreads();
    if (threadIdx.x >= 224 && threadIdx.x < 256) {
        tc_fence_after();
        tmem_dealloc(tm, COLS);
    }
}

constexpr int kStepThreads = 128;

// One token: a lane has four states of a channel, for kStepReqs requests at a time (A, skip and bias are read once, all
// their loads are in flight together).
constexpr int kStepReqs = 4;
template <typename T, int L, bool VEC>
__global__ void __launch_bounds__(kStepThreads) ssm_step_kernel(SsmStep a) {
    constexpr int CH = kStepThreads / L, N = 4 * L, R = kStepReqs;
    const int d0 = blockIdx.x * CH + threadIdx.x / L, l = threadIdx.x % L;
    const bool live = d0 < a.D;
    const int d = live ? d0 : 0, g = a.G == 1 ? 0 : d / (a.D / a.G);
    auto val = [](const void *p, long i) { return to_f32(static_cast<const T *>(p)[i]); };
    float4 s[R];
    float dt[R], x[R], z[R];
    Few<T, 4> B[R], C[R];
    const int n0 = blockIdx.y * R;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        const int n = min(n0 + r, a.nb - 1);
        s[r] = *reinterpret_cast<const float4 *>(a.state + ((long)n * a.D + d) * N + 4 * l);
        dt[r] = val(a.dt, n * a.dtb + d);
        x[r] = val(a.x, n * a.xb + d);
        z[r] = a.gate ? val(a.gate, n * a.gb + d) : 0.f;
        B[r].template load<VEC>(static_cast<const T *>(a.B) + n * a.Bb + g * a.Bg + 4 * l, 4);
        C[r].template load<VEC>(static_cast<const T *>(a.C) + n * a.Cb + g * a.Cg + 4 * l, 4);
    }
    const float4 A = *reinterpret_cast<const float4 *>(a.A + (long)d * N + 4 * l);
    const float Av[4] = {A.x * kLog2eF, A.y * kLog2eF, A.z * kLog2eF, A.w * kLog2eF};
    const float bias = a.bias ? a.bias[d] : 0.f, skip = a.skip ? a.skip[d] : 0.f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
        if (n0 + r >= a.nb) break;
        float t = dt[r] + bias;
        if (a.softplus) t = softplus<T>(t);
        const float u = t * x[r];
        float h[4] = {s[r].x, s[r].y, s[r].z, s[r].w}, y = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            h[i] = fmaf(ex2(t * Av[i]), h[i], u * B[r][i]);
            y = fmaf(h[i], C[r][i], y);
        }
#pragma unroll
        for (int off = L / 2; off; off >>= 1) y += __shfl_xor_sync(0xffffffffu, y, off);
        if (!live) continue;
        *reinterpret_cast<float4 *>(a.state + ((long)(n0 + r) * a.D + d) * N + 4 * l) = make_float4(h[0], h[1], h[2], h[3]);
        y = fmaf(skip, x[r], y);
        if (a.gate) {
            float rest;
            y *= z[r] * sigmoid<T>(z[r], rest);
        }
        if (l == 0) static_cast<T *>(a.y)[(n0 + r) * a.yb + d] = from_f32<T>(y);
    }
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

template <int L> int blocks_of(int D, int G) { return (D / G + 128 / L - 1) / (128 / L) * G; }

template <typename T, int L, bool VEC, bool LOCAL, int GROUPS> cudaError_t start(const Walk &w, long ctas, bool after, cudaStream_t st) {
    static lin::SmemOnce once;
    constexpr size_t bytes = Lay<T, L>::bytes(GROUPS, LOCAL);
    constexpr int threads = threads_of(LOCAL, GROUPS);
    static_assert(bytes <= 232448 - 64, "shared memory");
    const auto kernel = ssm_scan_kernel<T, L, VEC, LOCAL, GROUPS>;
    const cudaError_t e = once(kernel, (int)bytes);
    if (e != cudaSuccess) return e;
    if (after) return launch_after(kernel, dim3((unsigned)ctas), threads, bytes, st, w);
    kernel<<<(unsigned)ctas, threads, bytes, st>>>(w);
    return cudaGetLastError();
}

template <typename T, int L, bool VEC> cudaError_t launch(const Ssm &a, cudaStream_t st) {
    using Y = Lay<T, L>;
    Walk w{};
    w.pairs = a.D / a.G % 2 == 0 && few_view<T>(a.x, 2, false) && few_view<T>(a.dt, 2, false) && few_view<T>(a.gate, 2, false) &&
              few_view<T>(a.B, 2, true) && few_view<T>(a.C, 2, true);
    w.a = a;
    w.hdr = static_cast<WsHeader *>(a.ws);
    w.cpg = a.D / a.G;
    const long rows = a.s.cu ? a.total : (long)a.s.nseq * a.s.T;
    const int max_len = a.s.cu ? a.max_len : a.s.T;
    w.seg = a.hT && a.hT == a.h0 ? 0 : pick_segment(a, rows, max_len, blocks_of<L>(a.D, a.G));
    const bool split = w.seg > 0;
    if (!split) w.seg = 0x7fffffff;
    w.items = split ? run_items(a.s, a.total, w.seg) : a.s.nseq;
    // two groups to a CTA where one would leave blocks waiting for an SM
    constexpr bool two_groups = sizeof(T) == 2 && L > 2;      // what two groups hold has to fit
    const bool pair = two_groups && w.items * blocks_of<L>(a.D, a.G) > a.sms && w.cpg > Y::CH;
    w.bpg = (w.cpg + Y::CH * (1 + pair) - 1) / (Y::CH * (1 + pair));
    w.blocks = w.bpg * a.G;
    const long ctas = w.items * w.blocks;
    if (ctas > 0x7fffffffL) return cudaErrorInvalidValue;
    if (split) {
        w.local = reinterpret_cast<float *>(static_cast<char *>(a.ws) + sizeof(WsHeader));
        w.sums = w.local + w.items * (long)a.D * a.N;
        Walk one = w;       // one group to a CTA: two of these share an SM
        one.bpg = (w.cpg + Y::CH - 1) / Y::CH;
        one.blocks = one.bpg * a.G;
        const cudaError_t e = start<T, L, VEC, true, 1>(one, one.items * one.blocks, false, st);
        if (e != cudaSuccess) return e;
    }
    if constexpr (two_groups)
        if (pair) return start<T, L, VEC, false, 2>(w, ctas, split, st);
    return start<T, L, VEC, false, 1>(w, ctas, split, st);
}

template <typename T, int L> cudaError_t run(const Ssm &a, cudaStream_t st) {
    using Y = Lay<T, L>;
    const int cpg = a.D / a.G;
    const bool vec = cpg % Y::VC == 0 && few_view<T>(a.x, Y::VC, false) && few_view<T>(a.dt, Y::VC, false) &&
                     few_view<T>(a.gate, Y::VC, false) && few_view<T>(a.y, Y::VC, false) && few_view<T>(a.B, 4, true) &&
                     few_view<T>(a.C, 4, true);
    return vec ? launch<T, L, true>(a, st) : launch<T, L, false>(a, st);
}
template <typename T, int L> cudaError_t run_step(const SsmStep &a, cudaStream_t st) {
    const dim3 grid((unsigned)(((long)a.D * L + kStepThreads - 1) / kStepThreads), (a.nb + kStepReqs - 1) / kStepReqs);
    const auto by4 = [](const void *p, long long b, long long g) { return reinterpret_cast<uintptr_t>(p) % (4 * sizeof(T)) == 0 && b % 4 == 0 && g % 4 == 0; };
    if (by4(a.B, a.Bb, a.Bg) && by4(a.C, a.Cb, a.Cg))
        ssm_step_kernel<T, L, true><<<grid, kStepThreads, 0, st>>>(a);
    else
        ssm_step_kernel<T, L, false><<<grid, kStepThreads, 0, st>>>(a);
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
