// linear_tc_bwd.cu -- gradients of linear attention with a decay per head on the tcgen05 tensor cores:
// bf16, dk, dv in {64, 128}, chunks of C = 128 tokens.
//
// With S the memory entering a chunk, R the gradient of the memory leaving it, G the chunk's running log
// decays, D_ij = e^{G_i - G_j} (j <= i), s = Q K^T, m = dO V^T and c the query scale:
//
//     dQ = diag(c e^G) dO S^T       + M K,          M_ij = c m_ij D_ij
//     dK = diag(e^{G_C - G}) V R^T  + M^T Q
//     dV = diag(e^{G_C - G}) K R    + P^T dO,       P_ij = c s_ij D_ij
//     S' = e^{G_C} S + K^T diag(e^{G_C - G}) V,     R' = e^{G_C} R + Q^T diag(c e^G) dO   (R': into the chunk)
//     ddecay_t = e^{G_C} <S, R> + sum_{i >= t} q_i . (first term of dQ)_i + sum_{j < t} k_j . (first term of dK)_j
//                + sum_{j < t <= i} W_ij,           W_ij = c s_ij m_ij D_ij
//
// (what crosses token t: the memory through the whole chunk, into a later token, from an earlier token
// out, or from an earlier to a later token; a sum over j < t <= i is a suffix sum of W's row sums less its
// column sums, j < i only).  Every term of ddecay comes from fp32 products of exact or two-part operands
// and is anchored in its own chunk, so nothing drifts along the sequence.
//
// For a group of (sequence, head) pairs, first every chunk's S and R (the two are one kernel on other
// operands: the weighted values go in as three bf16 parts, as in the forward), then everything else, all chunks
// at once.  S and R come
//   of enough pairs from one launch that walks the chunks, the memory in registers;
//   of few pairs from two: every chunk's own contribution, all chunks at once, then the two chains over
//   the chunks, elementwise and in place.
// A walk takes 1.4 to 2.1 us a chunk of d = 128 however many pairs fit the machine, the other way 0.11 us a
// chunk and pair or, where a group has room for few pairs, the latency of the chains (costs in `walks` below).  All
// gradients of 2 x 2048 tokens, 16 heads of 128, on the device: 92 us walked, 107 the other way; of 2048 tokens, 14
// heads: 55 and 46; of 2 x 2048 tokens, 16 heads of 64: 61 and 54; of 32,768 tokens, 16 heads of 128: 813 and 1252.  Of
// 12 shapes the choice is the faster one, in one 7 % off it (8192 tokens, 14 heads: 203 for 189).
// The contributions of a group stay within L2, where the chains read them: 2 x 64 KB a chunk at d = 128 and
// at most kGroupChunks chunks.  A walk's memories are read back once, and a wider group fills the machine: kWalkChunks
// of them (32,768 tokens, 16 heads: 814 us, with half as many 1187).  A larger problem is taken group by
// group through the same scratch.
//
// Every wait is bounded; a time-out is recorded in the workspace header and the CTA unwinds.
#include <algorithm>
#include <initializer_list>

#include "linear_tc.cuh"

namespace kda {
namespace {

using namespace lin;

// Chunks of a group: six for every SM, and 117 MB of memories at d = 128 (L2 is 129 MB)
constexpr long kGroupChunks = 912;
constexpr long kWalkChunks = 4864;     // 0.6 GB of memories at d = 128

struct BwdParams {
    LinDecay g;
    int HV, m, T, nch;
    long pair0;                 // first (sequence, head) pair of the group
    int pairs;
    float scale;
    const float *h0, *dhT;      // whole arrays
    float *dh0;
    float *S, *R, *alpha;       // [pairs * nch][DK, DV] twice, [pairs * nch]
    __nv_bfloat16 *dq, *dk, *dv;
    long long qs[3], ks[3], vs[3];   // strides of dq, dk, dv: batch, token, head
    float *fq, *fk;             // per-value-head fp32 dq, dk [B, T, HV, DK] when heads are shared
    float *dg;                  // per-token ddecay [B, T, HV] or nullptr
    WsHeader *hdr;
    int clear;                  // the call's first launch: clears the error word
};

// Weights of a lane's four tokens from their log2 decays: of their values in the memory that leaves the chunk
// (direction 0: the decays behind a token), of their output gradients in the one that enters it (direction 1: up to and
// with it, times the query scale).  `all` (lane 31): the chunk's factor.
__device__ __forceinline__ float4 chunk_weights(const float4 &d, int dir, float scale, int lane, float &all) {
    float4 x = d, y = make_float4(d.y + (d.z + d.w), d.z + d.w, d.w, 0.f);
    x.y += x.x; x.z += x.y; x.w += x.z;
    float up = x.w, down = d.x + y.x;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const float p = __shfl_up_sync(0xffffffffu, up, off), q = __shfl_down_sync(0xffffffffu, down, off);
        if (lane >= off) up += p;
        if (lane + off < 32) down += q;
    }
    float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
    if (lane == 0) before = 0.f;
    if (lane == 31) behind = 0.f;
    all = ex2(up);
    return dir ? make_float4(scale * ex2(x.x + before), scale * ex2(x.y + before), scale * ex2(x.z + before),
                             scale * ex2(x.w + before))
               : make_float4(ex2(y.x + behind), ex2(y.y + behind), ex2(y.z + behind), ex2(behind));
}

// ------------------------------------------------------------------------------ 1: contributions
// Warps 0-7: weighted values (thread = value channel, half of the tokens); 8-11: results; 12: decays
// and TMA; 13: products.  Items (direction, pair, chunk) go round the CTAs.
constexpr int kPartThreads = 14 * 32;

template <int DK, int DV>
struct PartCfg {
    static constexpr int KB = kC * DK * 2, VB = kC * DV * 2, STAGE = KB + VB;
    static constexpr int NST = STAGE > 48 * 1024 ? 3 : 4;
    static constexpr int ARR = NST * STAGE, CTL = ARR + NST * kC * 4, SMEM = CTL + 256;
    static constexpr int T_V = 128;             // result [128], then two sets of hi, mid, lo
    static_assert(T_V + 384 <= 512 && SMEM <= 232448, "TMEM, shared memory");
};
struct PartCtl {
    uint64_t full[4], empty[4], ready[2], used[2], d_full, d_free, last;
    uint32_t tmem;
    int fail;
};
static_assert(sizeof(PartCtl) <= 256, "control block");

template <int DK, int DV>
__global__ void __launch_bounds__(kPartThreads, 1)
linear_part_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, BwdParams w) {
    using Cf = PartCfg<DK, DV>;
    constexpr int NST = Cf::NST;
    extern __shared__ __align__(1024) uint8_t smem[];
    PartCtl *ctl = reinterpret_cast<PartCtl *>(smem + Cf::CTL);
    if ((smem_u32(smem) & 1023) || blockDim.x != kPartThreads) {
        if (threadIdx.x == 0) atomicCAS(&w.hdr->error, 0, kStatusDeviceTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (w.clear && blockIdx.x == 0 && tid == 0) w.hdr->error = 0;
    const int slots = w.pairs * w.nch, items = 2 * slots;
    const int mine = ((int)blockIdx.x < items) ? (items - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->ready[i], 256);
            mbar_init(&ctl->used[i], 1);
        }
        mbar_init(&ctl->d_full, 1);
        mbar_init(&ctl->d_free, 128);
        mbar_init(&ctl->last, 1);
        ctl->fail = 0;
        fence_mbar_init();
    }
    if (warp == 13) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ctl->tmem;
    const Waits wt{&ctl->fail, w.hdr};
    const uint32_t tlane = tm + ((uint32_t)(32 * (warp & 3)) << 16);
    float *wa = reinterpret_cast<float *>(smem + Cf::ARR);
    auto item_of = [&](int n) { return (int)blockIdx.x + n * (int)gridDim.x; };

    if (warp == 12) {
        for (int n = 0; n < mine; ++n) {
            const int s = n % NST, item = item_of(n), dir = item >= slots, slot = item - dir * slots;
            const int pi = slot / w.nch, c = slot - pi * w.nch, u = c * kC;
            const long pair = w.pair0 + pi;
            const int b = (int)(pair / w.HV), hv = (int)(pair % w.HV);
            const float *gp = w.g.p ? w.g.p + b * w.g.b + hv : nullptr;
            const float4 d = load_decay(w.g, gp, u + 4 * lane, w.T);
            float all;
            const float4 f = chunk_weights(d, dir, w.scale, lane, all);
            if (lane == 31 && !dir) w.alpha[slot] = all;
            if (n >= NST && !wt.warp(&ctl->empty[s], (n / NST - 1) & 1, 41)) break;
            *reinterpret_cast<float4 *>(wa + s * kC + 4 * lane) = f;
            __syncwarp();
            if (lane == 0) {
                uint8_t *st = smem + s * Cf::STAGE;
                mbar_expect_tx(&ctl->full[s], Cf::STAGE);
#pragma unroll
                for (int i = 0; i < DK / 64; ++i)
                    tma_load_4d(st + i * kC * 128, dir ? &mq : &mk, &ctl->full[s], 64 * i, hv / w.m, u, b);
#pragma unroll
                for (int i = 0; i < DV / 64; ++i)
                    tma_load_4d(st + Cf::KB + i * kC * 128, dir ? &mo : &mv, &ctl->full[s], 64 * i, hv, u, b);
            }
        }
    } else if (warp == 13) {
        constexpr uint32_t id = idesc_bf16_f32(128, DK, false, true);
        for (int n = 0; n < mine; ++n) {
            const int s = n % NST;
            if (!wt.warp(&ctl->full[s], (n / NST) & 1, 42) || !wt.warp(&ctl->ready[n & 1], (n >> 1) & 1, 43)) break;
            if (n > 0 && !wt.warp(&ctl->d_free, (n - 1) & 1, 44)) break;
            tc_fence_after();
            const uint64_t dk = desc_mnmajor_sw128(smem_u32(smem + s * Cf::STAGE), kC, 0);
            const uint32_t a = tm + Cf::T_V + (n & 1) * 192;
            if (lane == 0) {
                product_ts<false>(tm, a + 128, dk, id);
                product_ts<true>(tm, a + 64, dk, id);
                product_ts<true>(tm, a, dk, id);
                mma_commit(&ctl->used[n & 1]);
                mma_commit(&ctl->empty[s]);
                mma_commit(&ctl->d_full);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        const int ch = tid & 127, half = tid >> 7;
        const bool has = (ch & ~31) < DV;
        for (int n = 0; n < mine; ++n) {
            const int s = n % NST;
            if (!wt.warp(&ctl->full[s], (n / NST) & 1, 45)) break;
            if (n >= 2 && !wt.warp(&ctl->used[n & 1], ((n >> 1) - 1) & 1, 46)) break;
            tc_fence_after();
            const uint32_t a = tlane + Cf::T_V + (n & 1) * 192;
            if (has) put_values<3>(smem + s * Cf::STAGE + Cf::KB, wa + s * kC, ch, 64 * half, a, a + 64, a + 128);
            tc_fence_before();
            mbar_arrive(&ctl->ready[n & 1]);
        }
    } else {
        const int i = tid - 256;                // value channel
        for (int n = 0; n < mine; ++n) {
            const int item = item_of(n), dir = item >= slots, slot = item - dir * slots;
            float *p = (dir ? w.R : w.S) + (size_t)slot * DK * DV + i;
            if (!wt.warp(&ctl->d_full, n & 1, 47)) break;
            tc_fence_after();
#pragma unroll 1
            for (int cb = 0; cb < DK; cb += 32) {
                uint32_t x[32];
                tmem_ld32(tlane + cb, x);
                tmem_ld_wait();
                if (cb + 32 == DK) {
                    tc_fence_before();
                    mbar_arrive(&ctl->d_free);
                }
                if (i < DV)
#pragma unroll
                    for (int j = 0; j < 32; ++j) p[(cb + j) * DV] = __uint_as_float(x[j]);
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        if (lane == 0) mma_commit(&ctl->last);
        __syncwarp();
        (void)mbar_wait(&ctl->last, 0, kWaitNs);
        if (ctl->fail) {                        // let what is in flight land
            const uint64_t t = globaltimer_ns();
            while (globaltimer_ns() - t < 1000000ull) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------------ 2: the chains
// In place: a slot's contribution becomes the memory entering its chunk (S), or the gradient of the one
// leaving it (R).  Bound by L2: eight slots' loads are in flight per thread.
__global__ void __launch_bounds__(256) linear_chain_kernel(BwdParams w, int cells) {
    next_may_start();
    wait_for_previous();
    const int per = cells / 4, e = blockIdx.x * 256 + threadIdx.x;
    if (e >= per * w.pairs) return;
    const int pi = e / per, at = (e - pi * per) * 4;
    const bool rev = blockIdx.y;
    const size_t pc = (size_t)(w.pair0 + pi) * cells + at;
    const float *init = rev ? w.dhT : w.h0;
    float4 s = init ? *reinterpret_cast<const float4 *>(init + pc) : make_float4(0.f, 0.f, 0.f, 0.f);
    float *base = (rev ? w.R : w.S) + (size_t)pi * w.nch * cells + at;
    const float *al = w.alpha + (size_t)pi * w.nch;
    constexpr int U = 8;
    for (int c0 = 0; c0 < w.nch; c0 += U) {
        float4 x[U];
        float a[U];
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = rev ? w.nch - 1 - (c0 + i) : c0 + i;
            if (c0 + i < w.nch) {
                x[i] = *reinterpret_cast<const float4 *>(base + (size_t)c * cells);
                a[i] = al[c];
            }
        }
#pragma unroll
        for (int i = 0; i < U; ++i) {
            const int c = rev ? w.nch - 1 - (c0 + i) : c0 + i;
            if (c0 + i < w.nch) {
                *reinterpret_cast<float4 *>(base + (size_t)c * cells) = s;
                s.x = fmaf(a[i], s.x, x[i].x); s.y = fmaf(a[i], s.y, x[i].y);
                s.z = fmaf(a[i], s.z, x[i].z); s.w = fmaf(a[i], s.w, x[i].w);
            }
        }
    }
    if (rev && w.dh0) *reinterpret_cast<float4 *>(w.dh0 + pc) = s;
}

// ------------------------------------------------------------------------------ 1 and 2 at once: the walk
// A CTA walks the chunks of one (direction, pair) for 64 key channels: the memory stays in fp32 registers, is stored
// to each chunk's slot, decayed, and takes the chunk's contribution, a product of its own (24 steps of N = 64) in one of
// two TMEM accumulators, rounded to nearest.  Added up in the accumulator itself it would be cut 24 times a chunk, always
// towards 0: without decays that came to 1.2e-4 of the memory over 32,768 tokens (3e-7 now).  The products wait for nothing of the
// memory's, so what a chunk takes is the conversion of its weighted values: 14 instructions a pair of them, in either half
// of a memory's CTAs.
// Warps 0-7: weighted values; 8-11: the memory; 12: decays and TMA; 13: products.
template <int DV>
struct StateCfg {
    static constexpr int KB = kC * 128, VB = kC * DV * 2, STAGE = KB + VB, NST = 4;
    static constexpr int ARR = NST * STAGE, CTL = ARR + NST * kC * 4, SMEM = CTL + 256;
    static constexpr int T_V = 128;             // two accumulators [64], then two sets of hi, mid, lo
    static_assert(SMEM <= 232448, "shared memory");
};
struct StateCtl {
    uint64_t full[4], empty[4], ready[2], used[2], d_full[2], d_free[2], last;
    float alpha[4];
    uint32_t tmem;
    int fail;
};
static_assert(sizeof(StateCtl) <= 256, "control block");

template <int DK, int DV>
__global__ void __launch_bounds__(kPartThreads, 1)
linear_state_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, BwdParams w) {
    using Cf = StateCfg<DV>;
    constexpr int NST = Cf::NST, KS = DK / 64;
    extern __shared__ __align__(1024) uint8_t smem[];
    StateCtl *ctl = reinterpret_cast<StateCtl *>(smem + Cf::CTL);
    if ((smem_u32(smem) & 1023) || blockDim.x != kPartThreads) {
        if (threadIdx.x == 0) atomicCAS(&w.hdr->error, 0, kStatusDeviceTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (w.clear && blockIdx.x == 0 && tid == 0) w.hdr->error = 0;
    const int part = blockIdx.x % KS, dir = blockIdx.x / KS % 2, pi = blockIdx.x / (2 * KS), nch = w.nch;
    const long pair = w.pair0 + pi;
    const int b = (int)(pair / w.HV), hv = (int)(pair % w.HV);
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1 + 128);   // the product has read the tiles, the memory's threads the factor
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->ready[i], 256);
            mbar_init(&ctl->used[i], 1);
            mbar_init(&ctl->d_full[i], 1);
            mbar_init(&ctl->d_free[i], 128);
        }
        mbar_init(&ctl->last, 1);
        ctl->fail = 0;
        fence_mbar_init();
    }
    if (warp == 13) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    next_may_start();                           // the TMEM is this CTA's by now
    tc_fence_after();
    const uint32_t tm = ctl->tmem;
    const Waits wt{&ctl->fail, w.hdr};
    const uint32_t tlane = tm + ((uint32_t)(32 * (warp & 3)) << 16);
    float *wa = reinterpret_cast<float *>(smem + Cf::ARR);
    auto chunk_of = [&](int n) { return dir ? nch - 1 - n : n; };

    if (warp == 12) {
        const float *gp = w.g.p ? w.g.p + b * w.g.b + hv : nullptr;
        for (int n = 0; n < nch; ++n) {
            const int s = n % NST, u = chunk_of(n) * kC;
            float all;
            const float4 f = chunk_weights(load_decay(w.g, gp, u + 4 * lane, w.T), dir, w.scale, lane, all);
            if (n >= NST && !wt.warp(&ctl->empty[s], (n / NST - 1) & 1, 61)) break;
            *reinterpret_cast<float4 *>(wa + s * kC + 4 * lane) = f;
            if (lane == 31) ctl->alpha[s] = all;
            __syncwarp();
            if (lane == 0) {
                uint8_t *st = smem + s * Cf::STAGE;
                mbar_expect_tx(&ctl->full[s], Cf::STAGE);
                tma_load_4d(st, dir ? &mq : &mk, &ctl->full[s], 64 * part, hv / w.m, u, b);
#pragma unroll
                for (int i = 0; i < DV / 64; ++i)
                    tma_load_4d(st + Cf::KB + i * kC * 128, dir ? &mo : &mv, &ctl->full[s], 64 * i, hv, u, b);
            }
        }
    } else if (warp == 13) {
        constexpr uint32_t id = idesc_bf16_f32(128, 64, false, true);
        for (int n = 0; n < nch; ++n) {
            const int s = n % NST;
            if (!wt.warp(&ctl->full[s], (n / NST) & 1, 62) || !wt.warp(&ctl->ready[n & 1], (n >> 1) & 1, 63)) break;
            if (n >= 2 && !wt.warp(&ctl->d_free[n & 1], ((n >> 1) - 1) & 1, 64)) break;
            tc_fence_after();
            const uint64_t dk = desc_mnmajor_sw128(smem_u32(smem + s * Cf::STAGE), kC, 0);
            const uint32_t a = tm + Cf::T_V + (n & 1) * 192, d = tm + (n & 1) * 64;
            if (lane == 0) {
                product_ts<false>(d, a + 128, dk, id);
                product_ts<true>(d, a + 64, dk, id);
                product_ts<true>(d, a, dk, id);
                mma_commit(&ctl->used[n & 1]);
                mma_commit(&ctl->empty[s]);
                mma_commit(&ctl->d_full[n & 1]);
            }
            __syncwarp();
        }
    } else if (warp < 8) {
        const int ch = tid & 127, half = tid >> 7;
        const bool has = (ch & ~31) < DV;
        for (int n = 0; n < nch; ++n) {
            const int s = n % NST;
            if (!wt.warp(&ctl->full[s], (n / NST) & 1, 65)) break;
            if (n >= 2 && !wt.warp(&ctl->used[n & 1], ((n >> 1) - 1) & 1, 66)) break;
            tc_fence_after();
            const uint32_t a = tlane + Cf::T_V + (n & 1) * 192;
            if (has) put_values<3>(smem + s * Cf::STAGE + Cf::KB, wa + s * kC, ch, 64 * half, a, a + 64, a + 128);
            tc_fence_before();
            mbar_arrive(&ctl->ready[n & 1]);
        }
    } else {
        const int i = tid - 256;                // value channel
        const float *init = dir ? w.dhT : w.h0;
        const size_t own = (size_t)64 * part * DV + i;
        float x[2][32];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int j = 0; j < 32; ++j) x[k][j] = init && i < DV ? init[(size_t)pair * DK * DV + own + (32 * k + j) * DV] : 0.f;
        bool ok = true;
        for (int n = 0; n < nch; ++n) {
            const int s = n % NST;
            if (!(ok = wt.warp(&ctl->full[s], (n / NST) & 1, 67))) break;
            const float al = ctl->alpha[s];
            mbar_arrive(&ctl->empty[s]);
            float *p = (dir ? w.R : w.S) + ((size_t)pi * nch + chunk_of(n)) * DK * DV + own;
            if (i < DV)
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int j = 0; j < 32; ++j) p[(32 * k + j) * DV] = x[k][j];
            if (!(ok = wt.warp(&ctl->d_full[n & 1], (n >> 1) & 1, 68))) break;
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t y[32];
                tmem_ld32(tlane + (n & 1) * 64 + 32 * k, y);
                tmem_ld_wait();
#pragma unroll
                for (int j = 0; j < 32; ++j) x[k][j] = fmaf(al, x[k][j], __uint_as_float(y[j]));
            }
            tc_fence_before();
            mbar_arrive(&ctl->d_free[n & 1]);
        }
        if (dir && w.dh0 && ok && i < DV) {
            float *p = w.dh0 + (size_t)pair * DK * DV + own;
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int j = 0; j < 32; ++j) p[(32 * k + j) * DV] = x[k][j];
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 13) {
        if (lane == 0) mma_commit(&ctl->last);
        __syncwarp();
        (void)mbar_wait(&ctl->last, 0, kWaitNs);
        if (ctl->fail) {                        // let what is in flight land
            const uint64_t t = globaltimer_ns();
            while (globaltimer_ns() - t < 1000000ull) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------------ 3: gradients
// One chunk at a time per CTA.  Warps 0-15 compute (thread = token row of the TMEM lanes, a quarter of the
// columns), warp 16 loads and issues.  TMEM: K Q^T, V dO^T, Q K^T, dO V^T in four blocks of 128 columns; then P^T
// over the first, M^T over the second, M over the fourth, every quarter's packed pairs in the lower half
// of its own columns; dQ gathers in the third, dK in the fourth once M is used, dV in the second once
// M^T is.  Loops are kept rolled and what is used three times out of line: the chunk's code runs once per
// chunk, and instruction fetch is what a longer one waits for (8 warps and unrolled passes: 0.109 ms with
// 2 x 2048 tokens, 16 heads of 128, instead of 0.065).
// The first terms of dQ and dK are read back before their second terms are added, for their dots with q and k
// (S and R go in as two bf16 parts for those dots).  Row factors are left to the stores,
//     dQ_i = E_i [dO (e^{G_C} S)^T + sum_j m_ij w_j k_j],   E_i = c e^{G_i - G_C},
//     dK_j = w_j [V R^T + sum_i m_ij E_i q_i],   dV_j = w_j [K R + sum_i s_ij E_i do_i],   w_j = e^{G_C - G_j},
// which takes one multiplication per element and no exponential, as long as the chunk is mild (is_mild); otherwise
// every weight has its own exponent and the first terms are rescaled in place (99 us instead of 92 with 2 x 2048 tokens).
// 17 warps leave a thread 96 registers, of which 44 to 120 bytes spill.
constexpr int kGradThreads = 17 * 32;

template <int DK, int DV>
struct GradCfg {
    static constexpr int QB = kC * DK * 2, VB = kC * DV * 2, XB = DK * DV * 2;
    static constexpr int Q = 0, K = QB, V = 2 * QB, O = 2 * QB + VB, XH = 2 * QB + 2 * VB, XL = XH + XB;
    // G, E (in chunks that are not mild: what G's fp32 lost), w, then quarters of: r, c, q dots, k dots
    static constexpr int ARR = XL + XB;
    static constexpr int CTL = ARR + 19 * kC * 4, SMEM = CTL + 256;
    static_assert(SMEM <= 232448, "shared memory");
};
struct GradCtl {
    uint64_t full_qk, full_vo, m, go, sync, last;
    uint32_t tmem;
    int fail;
    int strong;
    float dot[16];
};
static_assert(sizeof(GradCtl) <= 256, "control block");

// 32 columns of a row of results times f, bf16, four lanes trading 16-byte pieces (rows u0 .. u0 + 3)
__device__ __noinline__ void store_rows(uint32_t taddr, float f, __nv_bfloat16 *p, long long ts, int rows, int lane) {
    uint32_t x[32];
    tmem_ld32(taddr, x);
    tmem_ld_wait();
    uint4 r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        uint32_t *pr = &r[j].x;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            pr[i] = pack_bf16(f * __uint_as_float(x[8 * j + 2 * i]), f * __uint_as_float(x[8 * j + 2 * i + 1]));
    }
    trade4(r, lane);
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (j < rows) *reinterpret_cast<uint4 *>(p + (long long)j * ts) = r[j];
}
// the same in fp32, a row to a thread (only where q/k heads are shared)
__device__ __noinline__ void store_row_f32(uint32_t taddr, float f, float *p, bool live) {
    uint32_t x[32];
    tmem_ld32(taddr, x);
    tmem_ld_wait();
    if (live)
#pragma unroll
        for (int j = 0; j < 32; j += 4)
            *reinterpret_cast<float4 *>(p + j) = make_float4(f * __uint_as_float(x[j]), f * __uint_as_float(x[j + 1]),
                                                             f * __uint_as_float(x[j + 2]), f * __uint_as_float(x[j + 3]));
}
// dot of 32 columns with columns c0 .. of row r of a bf16 tile
__device__ __noinline__ float dot_row(uint32_t taddr, const uint8_t *tile, int r, int c0) {
    float d0 = 0.f, d1 = 0.f;
    uint32_t x[32];
    tmem_ld32(taddr, x);
    tmem_ld_wait();
#pragma unroll
    for (int j = 0; j < 32; j += 8) {
        const uint4 t = *reinterpret_cast<const uint4 *>(tile + piece(kC, r, (c0 + j) / 8));
        const uint32_t *pt = &t.x;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d0 = fmaf(__uint_as_float(x[j + 2 * i]), __uint_as_float(pt[i] << 16), d0);
            d1 = fmaf(__uint_as_float(x[j + 2 * i + 1]), __uint_as_float(pt[i] & 0xffff0000u), d1);
        }
    }
    return d0 + d1;
}
// row factor on 32 columns in place
__device__ __noinline__ void scale_row(uint32_t taddr, float f) {
    uint32_t x[32];
    tmem_ld32(taddr, x);
    tmem_ld_wait();
#pragma unroll
    for (int i = 0; i < 32; ++i) x[i] = __float_as_uint(f * __uint_as_float(x[i]));
    tmem_st32(taddr, x);
    tmem_st_wait();
}

// Running sums of a lane's four log2 decays and all before them as sums of two floats, x + low.  A restart counts as -150,
// so that a few of them leave fp32 no bits for the decays between: 2^-24 of 2000 is 1e-4 of a weight.
struct Two {
    float h, l;
};
__device__ __forceinline__ Two add(const Two &a, const Two &b) {
    const float s = a.h + b.h, v = s - a.h, r = (a.h - (s - v)) + (b.h - v) + (a.l + b.l);   // what s lost, both tails
    const float h = s + r;
    return {h, r - (h - s)};
}
__device__ __noinline__ void running_sums(const float4 &d, int lane, float4 &x, float4 &low) {
    const Two a = {d.x, 0.f}, b = add(a, {d.y, 0.f}), c = add(b, {d.z, 0.f}), e = add(c, {d.w, 0.f});
    Two run = e;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
        const Two y = {__shfl_up_sync(0xffffffffu, run.h, off), __shfl_up_sync(0xffffffffu, run.l, off)};
        if (lane >= off) run = add(y, run);
    }
    Two before = {__shfl_up_sync(0xffffffffu, run.h, 1), __shfl_up_sync(0xffffffffu, run.l, 1)};
    if (lane == 0) before = {0.f, 0.f};
    const Two p = add(before, a), q = add(before, b), r = add(before, c), s = add(before, e);
    x = make_float4(p.h, q.h, r.h, s.h);
    low = make_float4(p.l, q.l, r.l, s.l);
}

template <int DK, int DV>
__global__ void __launch_bounds__(kGradThreads, 1)
linear_grad_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                   const __grid_constant__ CUtensorMap mv, const __grid_constant__ CUtensorMap mo, BwdParams w) {
    using Cf = GradCfg<DK, DV>;
    constexpr uint32_t R0 = 0, R1 = 128, R2 = 256, R3 = 384;
    constexpr int NX = DK * DV / 8 / 512;       // 8-value pieces of a memory per thread
    extern __shared__ __align__(1024) uint8_t smem[];
    GradCtl *ctl = reinterpret_cast<GradCtl *>(smem + Cf::CTL);
    if ((smem_u32(smem) & 1023) || blockDim.x != kGradThreads) {
        if (threadIdx.x == 0) atomicCAS(&w.hdr->error, 0, kStatusDeviceTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int slots = w.pairs * w.nch;
    if (tid == 0) {
        mbar_init(&ctl->full_qk, 1);
        mbar_init(&ctl->full_vo, 1);
        mbar_init(&ctl->m, 1);
        mbar_init(&ctl->go, 512);
        mbar_init(&ctl->sync, 512);
        mbar_init(&ctl->last, 1);
        ctl->fail = 0;
        fence_mbar_init();
    }
    if (warp == 16) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ctl->tmem;
    const Waits wt{&ctl->fail, w.hdr};

    if (warp == 16) {
        constexpr uint32_t ida = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t idx = idesc_bf16_f32(128, DK, false, false);
        constexpr uint32_t idk = idesc_bf16_f32(128, DK, false, true);
        constexpr uint32_t idv = idesc_bf16_f32(128, DV, false, true);
        const uint32_t sb = smem_u32(smem);
        const uint64_t q = desc_kmajor_sw128(sb + Cf::Q, kC, 0), k = desc_kmajor_sw128(sb + Cf::K, kC, 0),
                       v = desc_kmajor_sw128(sb + Cf::V, kC, 0), o = desc_kmajor_sw128(sb + Cf::O, kC, 0);
        const uint64_t qn = desc_mnmajor_sw128(sb + Cf::Q, kC, 0), kn = desc_mnmajor_sw128(sb + Cf::K, kC, 0),
                       on = desc_mnmajor_sw128(sb + Cf::O, kC, 0);
        const uint64_t xh = desc_kmajor_sw128(sb + Cf::XH, DK, 0), xl = desc_kmajor_sw128(sb + Cf::XL, DK, 0),
                       xn = desc_mnmajor_sw128(sb + Cf::XH, DK, 0);
        // tiles of the item at `slot`, as they become free: V, then Q and K, then dO
        auto load = [&](int slot, int what) {
            const int pi = slot / w.nch, u = (slot - pi * w.nch) * kC;
            const long pair = w.pair0 + pi;
            const int b = (int)(pair / w.HV), hv = (int)(pair % w.HV);
            if (lane == 0 && slot < slots) {
                if (what == 0) mbar_expect_tx(&ctl->full_vo, 2 * Cf::VB);
                if (what == 1) mbar_expect_tx(&ctl->full_qk, 2 * Cf::QB);
#pragma unroll
                for (int i = 0; i < DV / 64; ++i) {
                    if (what == 0) tma_load_4d(smem + Cf::V + i * kC * 128, &mv, &ctl->full_vo, 64 * i, hv, u, b);
                    if (what == 2) tma_load_4d(smem + Cf::O + i * kC * 128, &mo, &ctl->full_vo, 64 * i, hv, u, b);
                }
#pragma unroll
                for (int i = 0; i < DK / 64; ++i)
                    if (what == 1) {
                        tma_load_4d(smem + Cf::Q + i * kC * 128, &mq, &ctl->full_qk, 64 * i, hv / w.m, u, b);
                        tma_load_4d(smem + Cf::K + i * kC * 128, &mk, &ctl->full_qk, 64 * i, hv / w.m, u, b);
                    }
            }
            __syncwarp();
        };
        // token tile times token tile over D channels, both K-major
        auto gram_k = [&](uint32_t d, uint64_t a, uint64_t bb) { product_ss<DK / 16, kC, kC, false>(tm + d, a, bb, ida); };
        auto gram_v = [&](uint32_t d, uint64_t a, uint64_t bb) { product_ss<DV / 16, kC, kC, false>(tm + d, a, bb, ida); };
        // token tile [., dv] times X^T, the small part first
        auto into = [&](uint64_t a, uint32_t d) {
            product_ss<DV / 16, kC, DK, false>(tm + d, a, xl, idx);
            product_ss<DV / 16, kC, DK, true>(tm + d, a, xh, idx);
        };
        // A in TMEM times a token tile
        auto spread = [&](uint32_t d, uint32_t a, uint64_t bb, uint32_t id) { product_ts<true, true>(tm + d, tm + a, bb, id); };
        auto done = [&]() { mma_commit(&ctl->m); };
        int n = 0, ph = 0;                       // items; phases of `go` seen
        auto next = [&]() {
            const bool ok = wt.warp(&ctl->go, ph & 1, 52);
            ++ph;
            tc_fence_after();
            return ok;
        };
        for (int i = 0; i < 3; ++i) load(blockIdx.x, i);
        for (int slot = blockIdx.x; slot < slots; slot += gridDim.x, ++n) {
            if (!wt.warp(&ctl->full_qk, n & 1, 51)) break;
            tc_fence_after();
            if (lane == 0) {
                gram_k(R0, k, q);
                gram_k(R2, q, k);
            }
            __syncwarp();
            if (!wt.warp(&ctl->full_vo, n & 1, 50)) break;   // dO comes last
            if (lane == 0) {
                gram_v(R1, v, o);
                gram_v(R3, o, v);
                done();
            }
            __syncwarp();
            if (!next()) break;
            if (lane == 0) {
                into(o, R2);                     // dO S^T
                done();
            }
            __syncwarp();
            if (!next()) break;
            if (lane == 0) {
                spread(R2, R3, kn, idk);         // + M K
                into(v, R3);                     // V R^T
                done();
            }
            __syncwarp();
            if (!next()) break;
            load(slot + gridDim.x, 0);           // products with V are done
            if (lane == 0) {
                spread(R3, R1, qn, idk);         // + M^T Q
                product_ss<DK / 16, kC, 0, false>(tm + R1, k, xn, idv);   // K R
                done();
            }
            __syncwarp();
            if (!next()) break;
            load(slot + gridDim.x, 1);           // and with Q and K
            if (lane == 0) {
                spread(R1, R0, on, idv);         // + P^T dO
                done();
            }
            __syncwarp();
            if (!next()) break;
            load(slot + gridDim.x, 2);
        }
    } else {
        const int quad = warp & 3, part = warp >> 2, row = 32 * quad + lane;
        const uint32_t tl = tm + ((uint32_t)(32 * quad) << 16);
        float *ga = reinterpret_cast<float *>(smem + Cf::ARR);
        float *ae = ga + kC, *aw = ae + kC;
        float *ar = aw + kC + part * kC, *ac = ar + 4 * kC, *aq = ac + 4 * kC, *ak = aq + 4 * kC;   // this quarter's
        int ph = 0, sp = 0;                      // phases of `m` and `sync` seen
        auto done = [&](int where) {
            const bool ok = wt.warp(&ctl->m, ph & 1, where);
            ++ph;
            tc_fence_after();
            return ok;
        };
        auto meet = [&]() {
            mbar_arrive(&ctl->sync);
            const bool ok = wt.warp(&ctl->sync, sp & 1, 60);
            ++sp;
            return ok;
        };
        auto go = [&]() {
            tc_fence_before();
            mbar_arrive(&ctl->go);
        };
        // a memory's pieces of this thread, as two bf16 parts (16 bits) into the operand tiles
        auto put_x = [&](const float4 (&x)[2 * NX], float f0) {
#pragma unroll
            for (int p = 0; p < NX; ++p) {
                const int e = tid + 512 * p, r = e / (DV / 8), c = e % (DV / 8);
                const float f[8] = {f0 * x[2 * p].x, f0 * x[2 * p].y, f0 * x[2 * p].z, f0 * x[2 * p].w,
                                    f0 * x[2 * p + 1].x, f0 * x[2 * p + 1].y, f0 * x[2 * p + 1].z, f0 * x[2 * p + 1].w};
                uint4 h, l;
                uint32_t *ph_ = &h.x, *pl = &l.x;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ph_[i] = pack_bf16(f[2 * i], f[2 * i + 1]);   // rounded: dV takes this part alone
                    pl[i] = pack_bf16(f[2 * i] - __uint_as_float(ph_[i] << 16),
                                      f[2 * i + 1] - __uint_as_float(ph_[i] & 0xffff0000u));
                }
                *reinterpret_cast<uint4 *>(smem + Cf::XH + piece(DK, r, c)) = h;
                *reinterpret_cast<uint4 *>(smem + Cf::XL + piece(DK, r, c)) = l;
            }
        };
        float4 xs[2 * NX];
        auto get_s = [&](int slot) {
            const float4 *ps = reinterpret_cast<const float4 *>(w.S + (size_t)slot * DK * DV);
#pragma unroll
            for (int p = 0; p < NX; ++p) {
                xs[2 * p] = ps[2 * (tid + 512 * p)];
                xs[2 * p + 1] = ps[2 * (tid + 512 * p) + 1];
            }
        };
        wait_for_previous();                     // S and R (the other warp loads the call's inputs)
        if ((int)blockIdx.x < slots) get_s(blockIdx.x);
        int it = 0;
        for (int slot = blockIdx.x; slot < slots; slot += gridDim.x, ++it) {
            const int pi = slot / w.nch, u = (slot - pi * w.nch) * kC;
            const long pair = w.pair0 + pi;
            const int b = (int)(pair / w.HV), hv = (int)(pair % w.HV);
            const int live = w.T - u;            // tokens of the chunk (more: all 128)
            // ---- S (asked for at the end of the item before), the decays
            if (warp == 0) {
                const float *gp = w.g.p ? w.g.p + b * w.g.b + hv : nullptr;
                const float4 d = load_decay(w.g, gp, u + 4 * lane, w.T);
                float4 x = d;
                x.y += x.x; x.z += x.y; x.w += x.z;
                float up = x.w;
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float y = __shfl_up_sync(0xffffffffu, up, off);
                    if (lane >= off) up += y;
                }
                float before = __shfl_up_sync(0xffffffffu, up, 1);
                if (lane == 0) before = 0.f;
                x = make_float4(x.x + before, x.y + before, x.z + before, x.w + before);
                const float end = __shfl_sync(0xffffffffu, x.w, 31);
                const int strong = !__all_sync(0xffffffffu, is_mild(x, end));
                if (lane == 0) ctl->strong = strong;
                float4 e;
                if (strong)
                    running_sums(d, lane, x, e);
                else
                    e = make_float4(w.scale * ex2(x.x - end), w.scale * ex2(x.y - end), w.scale * ex2(x.z - end),
                                    w.scale * ex2(x.w - end));
                *reinterpret_cast<float4 *>(ga + 4 * lane) = x;
                *reinterpret_cast<float4 *>(ae + 4 * lane) = e;
                *reinterpret_cast<float4 *>(aw + 4 * lane) = make_float4(ex2(end - x.x), ex2(end - x.y), ex2(end - x.z), ex2(end - x.w));
            }
            if (!meet()) break;
            const float gr = ga[row], gc = ga[kC - 1];
            const bool strong = ctl->strong;
            const float lr = strong ? ae[row] : 0.f, lc = strong ? ae[kC - 1] : 0.f;
            // row factors of dQ and of dK, dV at the end; of the first terms in place
            const float fq = strong ? 1.f : ae[row], fk = strong ? 1.f : aw[row];
            const float iq = w.scale * ex2(gr), ik = ex2((gc - gr) + (lc - lr));
            put_x(xs, strong ? 1.f : ex2(gc));
            fence_proxy_async();                 // here, where the products are waited for (1500 clocks before `go`)
            if (!wt.warp(&ctl->full_qk, it & 1, 58) || !done(53)) break;   // Q and K are read here too
            // ---- P^T, M^T of this row j and its quarter of the i; M of this row i and its quarter of the j; sums of W
            float cs = 0.f, rs = 0.f;
#pragma unroll 1
            for (int i0 = 32 * part; i0 < 32 * part + 32; i0 += 16) {
                const uint32_t to = 32 * part + (i0 & 16) / 2;
                uint32_t p[8], q[8];
                if (part < quad) {               // all before the row's tokens
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = q[j] = 0u;
                } else {
                    uint32_t x[16], y[16];
                    tmem_ld16(tl + R0 + i0, x);
                    tmem_ld16(tl + R1 + i0, y);
                    float e[16];
                    if (!strong) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<float4 *>(e + j) = *reinterpret_cast<const float4 *>(ae + i0 + j);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) e[j] = w.scale * ex2((ga[i0 + j] - gr) + (ae[i0 + j] - lr));
                    }
                    if (part == quad) {          // nothing from before the row's own token, W not from it either
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (i0 + j < row) e[j] = 0.f;
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float sx = __uint_as_float(x[j]), c = __uint_as_float(y[j]) * e[j];
                        cs = fmaf(sx, part == quad && i0 + j == row ? 0.f : c, cs);
                        x[j] = __float_as_uint(sx * e[j]);
                        y[j] = __float_as_uint(c);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        p[j] = pack_bf16(__uint_as_float(x[2 * j]), __uint_as_float(x[2 * j + 1]));
                        q[j] = pack_bf16(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]));
                    }
                }
                tmem_st8(tl + R0 + to, p);
                tmem_st8(tl + R1 + to, q);
            }
#pragma unroll 1
            for (int j0 = 32 * part; j0 < 32 * part + 32; j0 += 16) {
                const uint32_t to = 32 * part + (j0 & 16) / 2;
                uint32_t p[8];
                if (part > quad) {               // all after the row's tokens
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = 0u;
                } else {
                    uint32_t x[16], y[16];
                    tmem_ld16(tl + R2 + j0, x);
                    tmem_ld16(tl + R3 + j0, y);
                    float e[16];
                    if (!strong) {
#pragma unroll
                        for (int j = 0; j < 16; j += 4)
                            *reinterpret_cast<float4 *>(e + j) = *reinterpret_cast<const float4 *>(aw + j0 + j);
                    } else {
#pragma unroll
                        for (int j = 0; j < 16; ++j) e[j] = w.scale * ex2((gr - ga[j0 + j]) + (lr - ae[j0 + j]));
                    }
                    if (part == quad) {
#pragma unroll
                        for (int j = 0; j < 16; ++j)
                            if (j0 + j > row) e[j] = 0.f;
                    }
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) {
                        const float c = __uint_as_float(y[j]) * e[j];
                        rs = fmaf(__uint_as_float(x[j]), part == quad && j0 + j == row ? 0.f : c, rs);
                        y[j] = __float_as_uint(c);
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) p[j] = pack_bf16(__uint_as_float(y[2 * j]), __uint_as_float(y[2 * j + 1]));
                }
                tmem_st8(tl + R3 + to, p);
            }
            ar[row] = fq * rs;
            ac[row] = fk * cs;
            tmem_st_wait();
            go();
            // ---- R; first term of dQ
            float4 xr[2 * NX];
            const float4 *pr = reinterpret_cast<const float4 *>(w.R + (size_t)slot * DK * DV);
#pragma unroll
            for (int p = 0; p < NX; ++p) {
                xr[2 * p] = pr[2 * (tid + 512 * p)];
                xr[2 * p + 1] = pr[2 * (tid + 512 * p) + 1];
            }
            float dot = 0.f;
#pragma unroll
            for (int p = 0; p < 2 * NX; ++p)
                dot = fmaf(xs[p].x, xr[p].x, fmaf(xs[p].y, xr[p].y, fmaf(xs[p].z, xr[p].z, fmaf(xs[p].w, xr[p].w, dot))));
#pragma unroll
            for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
            if (lane == 0) ctl->dot[warp] = dot;
            if (!done(54)) break;
            put_x(xr, 1.f);
            const bool onk = 32 * part < DK, onv = 32 * part < DV;   // this warp's 32 columns exist
            if (strong && onk) scale_row(tl + R2 + 32 * part, iq);
            aq[row] = onk ? fq * dot_row(tl + R2 + 32 * part, smem + Cf::Q, row, 32 * part) : 0.f;
            fence_proxy_async();                 // R's parts
            go();
            // ---- dQ out; first term of dK
            const int u0 = u + (row & ~3), rows = min(4, w.T - u0), l8 = 8 * (lane & 3);
            const long long tok = (long long)b * w.T + u + row;
            if (!done(55)) break;
            // dK's first term first: products 4 wait for it, nobody for dQ's stores
            if (strong && onk) scale_row(tl + R3 + 32 * part, ik);
            ak[row] = onk ? fk * dot_row(tl + R3 + 32 * part, smem + Cf::K, row, 32 * part) : 0.f;
            go();
            if (onk) {
                if (w.fq)
                    store_row_f32(tl + R2 + 32 * part, fq, w.fq + (tok * w.HV + hv) * DK + 32 * part, row < live);
                else
                    store_rows(tl + R2 + 32 * part, fq,
                               w.dq + b * w.qs[0] + (long long)u0 * w.qs[1] + hv * w.qs[2] + 32 * part + l8, w.qs[1], rows, lane);
            }
            // ---- dK out; first term of dV
            if (!done(56)) break;
            if (strong && onv) scale_row(tl + R1 + 32 * part, ik);
            go();
            if (onk) {
                if (w.fk)
                    store_row_f32(tl + R3 + 32 * part, fk, w.fk + (tok * w.HV + hv) * DK + 32 * part, row < live);
                else
                    store_rows(tl + R3 + 32 * part, fk,
                               w.dk + b * w.ks[0] + (long long)u0 * w.ks[1] + hv * w.ks[2] + 32 * part + l8, w.ks[1], rows, lane);
            }
            // ---- dV out
            if (!done(57)) break;
            if (onv)
                store_rows(tl + R1 + 32 * part, fk,
                           w.dv + b * w.vs[0] + (long long)u0 * w.vs[1] + hv * w.vs[2] + 32 * part + l8, w.vs[1], rows, lane);
            go();
            // the next item's S: 32 registers of it would not live through the calls above, which would wait for it
            if (slot + (int)gridDim.x < slots) get_s(slot + gridDim.x);
            // ---- ddecay, while the next chunk's first products run (every warp's sums and dots came before `done`;
            // they are written again after the next meeting, which this warp joins when it is through)
            if (w.dg && warp == 0) {
                const float *a0 = aw + kC;
                float f[4], kd[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = 4 * lane + i;
                    auto sum4 = [&](int which) {
                        const float *a = a0 + 4 * which * kC + t;
                        return (a[0] + a[kC]) + (a[2 * kC] + a[3 * kC]);
                    };
                    f[i] = sum4(0) - sum4(1) + sum4(2);
                    kd[i] = sum4(3);
                }
                float fs = (f[0] + f[1]) + (f[2] + f[3]), kk = (kd[0] + kd[1]) + (kd[2] + kd[3]);
                float down = fs, up = kk;    // over this and the later lanes; this and the earlier
#pragma unroll
                for (int off = 1; off < 32; off <<= 1) {
                    const float x = __shfl_down_sync(0xffffffffu, down, off), y = __shfl_up_sync(0xffffffffu, up, off);
                    if (lane + off < 32) down += x;
                    if (lane >= off) up += y;
                }
                float all = 0.f;
                for (int i = 0; i < 16; ++i) all += ctl->dot[i];
                float behind = __shfl_down_sync(0xffffffffu, down, 1), before = __shfl_up_sync(0xffffffffu, up, 1);
                if (lane == 31) behind = 0.f;
                if (lane == 0) before = 0.f;
                all *= ex2(gc);
                // a token that keeps nothing has 0, not what the sums' rounding leaves (restarts are in chunks that are not mild)
                float4 d = make_float4(0.f, 0.f, 0.f, 0.f);
                if (strong) d = load_decay(w.g, w.g.p + b * w.g.b + hv, u + 4 * lane, w.T);
                const float *pd = &d.x;
                float suf[4];
                suf[3] = behind + f[3]; suf[2] = suf[3] + f[2]; suf[1] = suf[2] + f[1]; suf[0] = suf[1] + f[0];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int t = u + 4 * lane + i;
                    const bool kept = (t > 0 || w.h0) && pd[i] > kMinDecay * kLog2e;
                    if (t < w.T) w.dg[((long long)b * w.T + t) * w.HV + hv] = kept || pd[i] != pd[i] ? all + suf[i] + before : 0.f;
                    before += kd[i];
                }
            }
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 16) {
        if (lane == 0) mma_commit(&ctl->last);
        __syncwarp();
        (void)mbar_wait(&ctl->last, 0, kWaitNs);
        if (ctl->fail) {                         // let what is in flight land
            const uint64_t t = globaltimer_ns();
            while (globaltimer_ns() - t < 1000000ull) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------------ host
// Whether the memories are walked: the time of either way, in us per chunk of a sequence (as measured).
bool walks(long pairs, int nch, int dk, int sms) {
    auto group = [&](long chunks) { return std::max(1L, std::min(pairs, chunks / nch)); };
    auto count = [&](long g) { return (double)((pairs + g - 1) / g); };
    const long gw = group(kWalkChunks), gc = group(kGroupChunks), ctas = gw * (dk / 64) * 2;
    const double each = gc * dk / 128.0;
    return count(gw) * (double)((ctas + sms - 1) / sms) * 2.0 < count(gc) * std::max(0.11 * each, 0.045 * each + 0.4);
}
long group_pairs(long pairs, int nch, int dk, int sms) {
    return std::max(1L, std::min(pairs, (walks(pairs, nch, dk, sms) ? kWalkChunks : kGroupChunks) / nch));
}

template <int DK, int DV>
cudaError_t run_groups(const LinBwd &a, BwdParams w, const CUtensorMap &mq, const CUtensorMap &mk, const CUtensorMap &mv,
                       const CUtensorMap &mo, cudaStream_t st) {
    using PC = PartCfg<DK, DV>;
    using GC = GradCfg<DK, DV>;
    using SC = StateCfg<DV>;
    static SmemOnce part_once, state_once, grad_once;
    cudaError_t e = part_once(linear_part_kernel<DK, DV>, PC::SMEM);
    if (e == cudaSuccess) e = state_once(linear_state_kernel<DK, DV>, SC::SMEM);
    if (e == cudaSuccess) e = grad_once(linear_grad_kernel<DK, DV>, GC::SMEM);
    if (e != cudaSuccess) return e;
    const long pairs = (long)a.B * a.HV, np = group_pairs(pairs, w.nch, DK, a.sms);
    constexpr int cells = DK * DV;
    for (long p0 = 0; p0 < pairs; p0 += np) {
        w.pair0 = p0;
        w.clear = p0 == 0;
        w.pairs = (int)std::min(np, pairs - p0);
        const int slots = w.pairs * w.nch;
        if (walks(pairs, w.nch, DK, a.sms)) {
            linear_state_kernel<DK, DV><<<w.pairs * 2 * (DK / 64), kPartThreads, SC::SMEM, st>>>(mq, mk, mv, mo, w);
            e = cudaGetLastError();
        } else {
            linear_part_kernel<DK, DV><<<std::min(2 * slots, a.sms), kPartThreads, PC::SMEM, st>>>(mq, mk, mv, mo, w);
            const dim3 grid((unsigned)(((long)w.pairs * (cells / 4) + 255) / 256), 2);
            e = cudaGetLastError();
            if (e == cudaSuccess) e = launch_after(linear_chain_kernel, grid, 256, 0, st, w, cells);
        }
        if (e == cudaSuccess)
            e = launch_after(linear_grad_kernel<DK, DV>, std::min(slots, a.sms), kGradThreads, GC::SMEM, st, mq, mk, mv, mo, w);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace

// Scratch: [S][R][chunk decays] of a group, [per-value-head dq, dk] when heads are shared, [per-token ddecay]
size_t linear_tc_bwd_scratch_bytes(int B, int T, int H, int HV, int dk, int dv, int sms) {
    const int nch = (T + kC - 1) / kC;
    const size_t slots = (size_t)group_pairs((long)B * HV, nch, dk, sms) * nch, rows = (size_t)B * T * HV;
    size_t n = 2 * round256(slots * dk * dv * 4) + round256(slots * 4) + round256(rows * 4);
    if (HV > H) n += 2 * round256(rows * dk * 4);
    return n;
}

cudaError_t launch_linear_tc_bwd(const LinBwd &a, cudaStream_t st) {
    BwdParams w{};
    const int m = a.HV / a.H;
    w.g = a.g; w.HV = a.HV; w.m = m; w.T = a.T; w.nch = (a.T + kC - 1) / kC; w.scale = a.scale;
    w.h0 = a.h0; w.dhT = a.dhT; w.dh0 = a.dh0; w.hdr = a.hdr;
    const size_t slots = (size_t)group_pairs((long)a.B * a.HV, w.nch, a.dk, a.sms) * w.nch, rows = (size_t)a.B * a.T * a.HV;
    char *p = static_cast<char *>(a.ws);
    auto carve = [&](size_t n) { char *r = p; p += round256(n); return reinterpret_cast<float *>(r); };
    w.S = carve(slots * a.dk * a.dv * 4);
    w.R = carve(slots * a.dk * a.dv * 4);
    w.alpha = carve(slots * 4);
    float *dgt = carve(rows * 4);
    if (m > 1) {
        w.fq = carve(rows * a.dk * 4);
        w.fk = carve(rows * a.dk * 4);
    }
    const bool want_g = a.g.p && a.dg, fixed = want_g && a.g.t == 0;
    w.dg = want_g ? (fixed ? dgt : a.dg) : nullptr;
    auto out = [](const LinView &v, __nv_bfloat16 *&q, long long (&s)[3]) {
        q = static_cast<__nv_bfloat16 *>(const_cast<void *>(v.p));
        s[0] = v.b; s[1] = v.t; s[2] = v.h;
    };
    out(a.dq, w.dq, w.qs);
    out(a.dk_, w.dk, w.ks);
    out(a.dv_, w.dv, w.vs);
    CUtensorMap mq, mk, mv, mo;
    if (!token_map(&mq, a.q, a.dk, a.H, a.T, a.B) || !token_map(&mk, a.k, a.dk, a.H, a.T, a.B) ||
        !token_map(&mv, a.v, a.dv, a.HV, a.T, a.B) || !token_map(&mo, a.d_o, a.dv, a.HV, a.T, a.B))
        return cudaErrorInvalidValue;
    cudaError_t e;
    if (a.dk == 128 && a.dv == 128) e = run_groups<128, 128>(a, w, mq, mk, mv, mo, st);
    else if (a.dk == 128) e = run_groups<128, 64>(a, w, mq, mk, mv, mo, st);
    else if (a.dv == 128) e = run_groups<64, 128>(a, w, mq, mk, mv, mo, st);
    else e = run_groups<64, 64>(a, w, mq, mk, mv, mo, st);
    if (e != cudaSuccess) return e;
    if (m > 1 && (e = launch_fold_heads(w.fq, a.dq, w.fk, a.dk_, a.dtype, a.B, a.T, a.H, m, a.dk, st)) != cudaSuccess) return e;
    return fixed ? launch_sum_rows(dgt, a.dg, (long)a.B * a.T, a.HV, st) : cudaSuccess;
}

}  // namespace kda
