// linear_tc.cu -- linear attention with a decay per head on the tcgen05 tensor cores: bf16,
// dk, dv in {64, 128}, chunks of C = 128 tokens.
//
// With G the running sum of the chunk's log decays (G_C its total), per (sequence, value head):
//
//     O = diag(e^G) Q S  +  P V,         P[i][j] = (q_i . k_j) e^{G_i - G_j}   (j <= i)
//     S_next = e^{G_C} S + K^T (diag(e^{G_C - G}) V)
//
// One CTA walks the chunks of one (sequence, head) or of one segment of it; the memory stays in registers in
// fp32 as S^T [dv, dk].  Per chunk four products of M = 128 rows (tokens, or value channels):
//
//     1  scores = Q K^T                     (operands as TMA writes them)
//     2  O = Q S_bf16                       (S rounded to a bf16 operand in shared memory)
//     3  O += P V                           (P written back to TMEM as the A operand)
//     4  Vw^T K,  Vw = hi + mid + lo        (three products; Vw^T written to TMEM as the A operand)
//
// What is rounded: P and the operand copy of S to bf16, each once, so O errs by three bf16
// roundings with its own (2.3e-3 of it, against 1.7e-3 for the last one alone); the memory itself
// must not, since a model carries it over tens of thousands of tokens and reads it back in fp32: the
// decayed values w v go in as the sum of three bf16s, which is w v as fp32 has it (two parts, 16
// bits, leave 2.4e-6 in the memory), k is exact, and a chunk's product is added to S in fp32 registers, rounded to
// nearest.  (Added up in the tensor cores' accumulator, S would be cut at each of the 24 steps of a chunk, always towards
// 0: 3.8e-5 of a memory kept over 32,768 tokens, against 3e-7.  It costs 1 % at dk = 128, nothing at 64.)
//
// Bound: 2 (2 dk + 2 dv) bytes per token and head through HBM; per chunk of d = 128 that is 128 KB,
// 5900 clocks of an SM's share at the measured 6.8 TB/s.  A chunk takes 6800 (8 x 4096 tokens, 19 heads: one CTA
// per SM, 128 us, 5.0 TB/s), of d = 64 5100 (half the bytes).  What the CTA itself is short of is TMEM and
// shared-memory bandwidth: beside the passes over values, memory and outputs a product's step of 16 takes 130 to
// 230 clocks (64 alone), and the passes take longer beside the products; and instruction fetch.  So the two
// products that can take their A operand from TMEM do, values are transposed by ldmatrix, products are issued from
// one-lane branches, and every role's loop is kept to a few hundred instructions (fully unrolled, the roles
// evicted each other's code and the walk took 1.5 times as long).
//
// Warps 0-3: scores -> P.  4-7: outputs.  8-15: the memory and its operand copy.  16-23: Vw.
// 24: decays and TMA.  25: issues the products.  (26 and 27 fill their warp group.)  The groups and the tensor pipe
// work on different stages of neighbouring chunks, so that none of their latencies adds up.
//
// Few heads and long sequences: a sequence is cut into segments.  A first launch (local kernel)
// leaves, for all but the last, the memory it adds from zero; the walk starts segment p from
// sum_{p'} (decay of the segments between) local_{p'}.  It reads k and v a second time, so the cut is
// chosen by a cost model (plan below).  The local kernel walks backwards, so that every weight is
// the product of the decays behind it and nothing needs rescaling, it leaves the segment's first
// tokens in L2, where the walk begins, and it stops once the weights are 0 in fp32.
//
// Every wait is bounded (2 s); a time-out is recorded in the workspace header and the CTA unwinds.
#include <algorithm>
#include <initializer_list>
#include <type_traits>

#include "linear_tc.cuh"

namespace kda {
namespace {

using namespace lin;

// The registers that warp groups trade have to be what the launch holds, or the trade never ends.
template <typename K>
cudaError_t check_regs(K *kernel, int regs) {
    cudaFuncAttributes f;
    const cudaError_t e = cudaFuncGetAttributes(&f, kernel);
    return e != cudaSuccess ? e : f.numRegs == regs ? cudaSuccess : cudaErrorInvalidConfiguration;
}

constexpr float kZeroWeight = -150.f;          // 2^x is 0 in fp32 below this
// A mild chunk (is_mild) is attended with e^{G_i - G_C} taken out of the row:
// O_i = e^{G_i - G_C} (q_i (e^{G_C} S) + sum_j s_ij w_j v_j), w_j = e^{G_C - G_j} the weights that the
// memory takes too: one accumulator and one factor per column, none beyond 2^62.  Stronger decays (a
// restart among them) get every weight e^{G_i - G_j} from its own exponent and the first term
// rescaled in between.
constexpr int kMaxSegs = 64;                   // segments of a sequence at most (equal lengths)
constexpr int kSortSeqs = 128;                 // packed sequences ranked by length up to this many

struct TcWalk {
    LinSeqs s;
    LinDecay g;
    int L;                  // tokens per segment (a multiple of kC)
    int HV, m;              // value heads, value heads per q/k head
    int sorted;             // packed, one segment each: take the sequences longest first
    float scale;
    const float *h0;
    float *hT;
    __nv_bfloat16 *o;
    long long ob, ot, oh;
    float *loc, *gam;       // per (item, head): [DK, DV], decay factor
    WsHeader *hdr;
    int clear;              // this launch is the call's first: it clears the error word
};

// The sequence of rank r by decreasing length (ties: lower index first); whole warp.
__device__ __forceinline__ int seq_by_rank(const LinSeqs &s, int r) {
    const int lane = threadIdx.x & 31;
    int found = -1;
    for (int n = lane; n < s.nseq; n += 32) {
        const int len = s.cu[n + 1] - s.cu[n];
        int rank = 0;
        for (int k = 0; k < s.nseq; ++k) {
            const int lk = s.cu[k + 1] - s.cu[k];
            rank += (lk > len || (lk == len && k < n)) ? 1 : 0;
        }
        if (rank == r) found = n;
    }
    const unsigned hit = __ballot_sync(0xffffffffu, found >= 0);
    return __shfl_sync(0xffffffffu, found, __ffs(hit) - 1);
}

__device__ __forceinline__ bool walk_item(const TcWalk &w, int item, LinItem &it) {
    if (w.sorted) {
        if (item >= w.s.nseq) return false;
        item = seq_by_rank(w.s, item);   // one segment each: item = sequence
    }
    return lin_item(w.s, w.L, item, it);
}

// ------------------------------------------------------------------------------ the walk
template <int DK, int DV>
struct WalkCfg {
    static constexpr int QB = kC * DK * 2, VB = kC * DV * 2;    // bytes of a q or k tile, of a v tile
    static constexpr int STAGE = 2 * QB + VB;                   // Q, K, V; two stages
    static constexpr int SB = 2 * STAGE;                        // the memory's operand copy
    static constexpr int ARR = SB + DK * DV * 2;                // per chunk parity: G [128], w [128]
    static constexpr int CTL = ARR + 2 * 2 * kC * 4;
    static constexpr int SMEM = CTL + 256;
    // TMEM columns: a chunk's product 4 [dv][dk] (first the start state), scores / P, O, the three parts of the decayed
    // values.  At d = 128 there is room for two of them, and hi follows lo once that is used
    static constexpr bool OWN_HI = DK + DV <= 192;
    static constexpr int T_S = 0, T_P = DK, T_O = DK + 128, T_V = DK + 128 + DV, T_HI = OWN_HI ? T_V + 128 : T_V;
    static_assert(T_V + (OWN_HI ? 192 : 128) <= 512, "TMEM");
    static_assert(SMEM <= 232448, "shared memory");
};

struct WalkCtl {
    uint64_t full[2], done[2], s_full, q_free, p_ready, r_ready, o_full, o_free, s_ready, v_ready, hi_ready, lo_done, kv_done,
        cleared, start, last;
    uint32_t tmem;
    int fail;
    int strong[2];   // the chunk is not mild
};
static_assert(sizeof(WalkCtl) <= 256, "control block");

constexpr int kWalkThreads = 28 * 32;
// dk = 128: a thread of the memory holds 64 of its channels, and registers are split by warp groups (four warps: P, outputs,
// twice the memory, twice the values, the rest).  What one gives up another takes; all there is, is what the launch holds.
// Calls do not go with that, so the waits are short ones, which cost 3 %; dk = 64 needs neither.
constexpr int kWalkRegs = 72, kRegsP = 48, kRegsO = 64, kRegsM = 96, kRegsV = 64, kRegsC = 72;
static_assert(kRegsP + kRegsO + 2 * kRegsM + 2 * kRegsV + kRegsC <= 7 * kWalkRegs, "more than the launch holds: an endless wait");
template <int DK, int N>
__device__ __forceinline__ void reg_split() {
    if constexpr (DK == 128 && N < kWalkRegs) reg_dec<N>();
    if constexpr (DK == 128 && N > kWalkRegs) reg_inc<N>();
}
__device__ __forceinline__ Waits walk_waits(WalkCtl *ctl, WsHeader *hdr, std::false_type) { return {&ctl->fail, hdr}; }
__device__ __forceinline__ ShortWaits walk_waits(WalkCtl *ctl, WsHeader *, std::true_type) { return {&ctl->fail}; }

template <int DK, int DV>
__global__ void __launch_bounds__(kWalkThreads, 1)
linear_chunk_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, TcWalk w) {
    using Cf = WalkCfg<DK, DV>;
    extern __shared__ __align__(1024) uint8_t smem[];
    WalkCtl *ctl = reinterpret_cast<WalkCtl *>(smem + Cf::CTL);
    if ((smem_u32(smem) & 1023) || blockDim.x != kWalkThreads) {   // what follows is laid out for these
        if (threadIdx.x == 0) atomicCAS(&w.hdr->error, 0, kStatusDeviceTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    // (no wait can run out before the first CTA has got here)
    if (w.clear && blockIdx.x == 0 && tid == 0) w.hdr->error = 0;
    const int hv = blockIdx.x % w.HV;
    LinItem it;
    if (!walk_item(w, blockIdx.x / w.HV, it)) return;
    const int t0 = it.p * w.L, t1 = min(it.len, t0 + w.L);      // tokens of the sequence
    const int nch = (t1 - t0 + kC - 1) / kC;
    const int b = w.s.cu ? 0 : it.n;
    const long tb = w.s.cu ? it.start : 0;                      // token of batch entry b

    if (tid == 0) {
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->done[i], 1);
        }
        for (uint64_t *x : {&ctl->s_full, &ctl->q_free, &ctl->o_full, &ctl->lo_done, &ctl->kv_done, &ctl->last}) mbar_init(x, 1);
        for (uint64_t *x : {&ctl->p_ready, &ctl->r_ready, &ctl->o_free}) mbar_init(x, 128);
        for (uint64_t *x : {&ctl->s_ready, &ctl->v_ready, &ctl->hi_ready, &ctl->cleared}) mbar_init(x, 256);
        mbar_init(&ctl->start, 512);
        ctl->fail = 0;
        fence_mbar_init();
    }
    if (warp == 25) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    if (warp == 24 && lane == 0) {
        tma_prefetch_desc(&mq);
        tma_prefetch_desc(&mk);
        tma_prefetch_desc(&mv);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm = ctl->tmem;
    const auto wt = walk_waits(ctl, w.hdr, std::integral_constant<bool, DK == 128>());
    const uint32_t tlane = tm + ((uint32_t)(32 * (warp & 3)) << 16);   // this warp's 32 TMEM lanes
    auto arr_g = [&](int c) { return reinterpret_cast<float *>(smem + Cf::ARR) + (c & 1) * 2 * kC; };
    auto stage = [&](int c) { return smem + (c & 1) * Cf::STAGE; };

    // The segment's start state, 32 key channels to each of four warp groups (one group alone spent
    // 1 us per 32 channels and earlier segment, all of it latency).
    const size_t pair = (size_t)it.n * w.HV + hv;
    if (warp < 16) {
        wait_for_previous();
        const int i = tid & 127, cb = 32 * (warp >> 2);
        if (nch > 0 && cb < DK && (i & ~31) < DV) {
            float acc[32];
            if (w.h0) {
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[j] = w.h0[(pair * DK + cb + j) * DV + i];
            } else {
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[j] = 0.f;
            }
#pragma unroll 1
            for (int pp = 0; pp < it.p; ++pp) {
                const size_t slot = (size_t)(it.first + pp) * w.HV + hv;
                const float ga = w.gam[slot];
                const float *l = w.loc + (slot * DK + cb) * DV + i;
#pragma unroll
                for (int j = 0; j < 32; ++j) acc[j] = fmaf(acc[j], ga, l[j * DV]);
            }
            uint32_t x[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(acc[j]);
            tmem_st32(tlane + Cf::T_S + cb, x);
            tmem_st_wait();
        }
        tc_fence_before();
        mbar_arrive(&ctl->start);
    }

    if (warp >= 24) reg_split<DK, kRegsC>();
    if (warp == 24) {
        // ---- decays and loads
        const float *gp = w.g.p ? w.g.p + b * w.g.b + tb * w.g.t + hv : nullptr;
        float4 d = load_decay(w.g, gp, t0 + 4 * lane, t1);
        for (int c = 0; c < nch; ++c) {
            const int s = c & 1, u = t0 + c * kC;
            float4 x = d;                       // running sums
            x.y += x.x; x.z += x.y; x.w += x.z;
            // sums of the decays behind a token (its weight in the memory)
            float4 e = make_float4(d.y + (d.z + d.w), d.z + d.w, d.w, 0.f);
            float up = x.w, down = d.x + e.x;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float y = __shfl_up_sync(0xffffffffu, up, off), z = __shfl_down_sync(0xffffffffu, down, off);
                if (lane >= off) up += y;
                if (lane + off < 32) down += z;
            }
            float before = __shfl_up_sync(0xffffffffu, up, 1), behind = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 0) before = 0.f;
            if (lane == 31) behind = 0.f;
            x.x += before; x.y += before; x.z += before; x.w += before;
            e = make_float4(ex2(e.x + behind), ex2(e.y + behind), ex2(e.z + behind), ex2(behind));
            const int strong = !__all_sync(0xffffffffu, is_mild(x, __shfl_sync(0xffffffffu, x.w, 31)));
            if (c >= 2 && !wt.warp(&ctl->done[s], ((c >> 1) - 1) & 1, 1)) break;
            float *ga = arr_g(c);
            *reinterpret_cast<float4 *>(ga + 4 * lane) = x;
            *reinterpret_cast<float4 *>(ga + kC + 4 * lane) = e;
            __syncwarp();
            if (lane == 0) {
                uint8_t *st = stage(c);
                uint64_t *bar = &ctl->full[s];
                ctl->strong[s] = strong;
                mbar_expect_tx(bar, Cf::STAGE);
                const int row = (int)(tb + u), hq = hv / w.m;
#pragma unroll
                for (int i = 0; i < DK / 64; ++i) tma_load_4d(st + i * kC * 128, &mq, bar, 64 * i, hq, row, b);
#pragma unroll
                for (int i = 0; i < DK / 64; ++i) tma_load_4d(st + Cf::QB + i * kC * 128, &mk, bar, 64 * i, hq, row, b);
#pragma unroll
                for (int i = 0; i < DV / 64; ++i) tma_load_4d(st + 2 * Cf::QB + i * kC * 128, &mv, bar, 64 * i, hv, row, b);
            }
            if (c + 1 < nch) d = load_decay(w.g, gp, u + kC + 4 * lane, t1);
        }
    } else if (warp == 25) {
        // ---- products
        constexpr uint32_t id1 = idesc_bf16_f32(128, 128, false, false);
        constexpr uint32_t id2 = idesc_bf16_f32(128, DV, false, false);
        constexpr uint32_t id3 = idesc_bf16_f32(128, DV, false, true);
        constexpr uint32_t id4 = idesc_bf16_f32(128, DK, false, true);   // dv = 64: rows 64.. are nobody's
        const uint64_t ds = desc_kmajor_sw128(smem_u32(smem + Cf::SB), DV, 0);
        // product 1 of chunk c: its scores lie where P(c - 1) did
        auto scores = [&](int c) {
            if (!wt.warp(&ctl->full[c & 1], (c >> 1) & 1, 3)) return false;
            tc_fence_after();
            const uint32_t q = smem_u32(stage(c));
            const uint64_t dq = desc_kmajor_sw128(q, kC, 0), dk = desc_kmajor_sw128(q + Cf::QB, kC, 0);
            if (lane == 0) {
                product_ss<DK / 16, kC, kC, false>(tm + Cf::T_P, dq, dk, id1);
                mma_commit(&ctl->s_full);
            }
            __syncwarp();
            return true;
        };
        // Product 1 of the next chunk comes after 4 (where it can, product 3 too): they fill the pipe while
        // the memory (waiting for 4) is turned into the next operand
        bool ok = nch > 0 && scores(0);
        uint32_t ph_r = 0;
        for (int c = 0; ok && c < nch; ++c) {
            const uint32_t ph = c & 1;
            const uint32_t q = smem_u32(stage(c));
            const uint64_t dq = desc_kmajor_sw128(q, kC, 0), dk = desc_mnmajor_sw128(q + Cf::QB, kC, 0),
                           dv = desc_mnmajor_sw128(q + 2 * Cf::QB, kC, 0);
            if (!wt.warp(&ctl->s_ready, ph, 4) || !wt.warp(&ctl->o_free, ph, 5)) break;
            tc_fence_after();
            if (lane == 0) {
                product_ss<DK / 16, kC, DV, false>(tm + Cf::T_O, dq, ds, id2);
                mma_commit(&ctl->q_free);
            }
            __syncwarp();
            // product 3, once P is there
            auto outputs = [&]() {
                if (!wt.warp(&ctl->p_ready, ph, 8)) return false;
                if (ctl->strong[ph]) {
                    if (!wt.warp(&ctl->r_ready, ph_r, 9)) return false;
                    ph_r ^= 1;
                }
                tc_fence_after();
                if (lane == 0) {
                    product_ts<true>(tm + Cf::T_O, tm + Cf::T_P, dv, id3);
                    mma_commit(&ctl->o_full);
                }
                __syncwarp();
                return true;
            };
            if (!wt.warp(&ctl->v_ready, ph, 6)) break;
            tc_fence_after();
            if (lane == 0) {
                product_ts<false>(tm + Cf::T_S, tm + Cf::T_V, dk, id4);
                if (!Cf::OWN_HI) mma_commit(&ctl->lo_done);
                product_ts<true>(tm + Cf::T_S, tm + Cf::T_V + 64, dk, id4);
            }
            __syncwarp();
            if (!Cf::OWN_HI) {                   // while hi is written over lo
                if (!outputs()) break;
                if (!wt.warp(&ctl->hi_ready, ph, 7)) break;
                tc_fence_after();
            }
            if (lane == 0) {
                product_ts<true>(tm + Cf::T_S, tm + Cf::T_HI, dk, id4);
                mma_commit(&ctl->kv_done);
            }
            __syncwarp();
            if (Cf::OWN_HI && !outputs()) break;
            if (lane == 0) mma_commit(&ctl->done[ph]);
            __syncwarp();
            if (c + 1 < nch) ok = scores(c + 1);
        }
    } else if (warp < 4) {
        // ---- scores -> P (thread = token row)
        reg_split<DK, kRegsP>();
        const int row = tid;
        for (int c = 0; c < nch; ++c) {
            const float *ga = arr_g(c), *wa = ga + kC;
            if (!wt.warp(&ctl->full[c & 1], (c >> 1) & 1, 10)) break;
            if (!wt.warp(&ctl->s_full, c & 1, 11)) break;
            tc_fence_after();
            const float gi = ga[row];
            const bool strong = ctl->strong[c & 1];
            // 16 columns at a time, written as 8 columns of packed pairs over scores read already
#pragma unroll 1
            for (int j0 = 0; j0 < 32 * (warp + 1); j0 += 16) {
                uint32_t x[16], p[8];
                tmem_ld16(tlane + Cf::T_P + j0, x);
                tmem_ld_wait();
                if (!strong) {
#pragma unroll
                    for (int j = 0; j < 16; j += 4) {
                        const float4 e = *reinterpret_cast<const float4 *>(wa + j0 + j);
                        x[j] = __float_as_uint(__uint_as_float(x[j]) * e.x);
                        x[j + 1] = __float_as_uint(__uint_as_float(x[j + 1]) * e.y);
                        x[j + 2] = __float_as_uint(__uint_as_float(x[j + 2]) * e.z);
                        x[j + 3] = __float_as_uint(__uint_as_float(x[j + 3]) * e.w);
                    }
                } else {
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        x[j] = __float_as_uint(__uint_as_float(x[j]) * (w.scale * ex2(gi - ga[j0 + j])));
                }
                // nothing after the row's own token (only the last 32 columns hold any)
                const int keep = j0 >= 32 * warp ? row - j0 : 16;
#pragma unroll
                for (int j = 0; j < 16; j += 2)
                    p[j / 2] = pack_bf16(j <= keep ? __uint_as_float(x[j]) : 0.f, j + 1 <= keep ? __uint_as_float(x[j + 1]) : 0.f);
                tmem_st8(tlane + Cf::T_P + j0 / 2, p);
            }
#pragma unroll 1
            for (int j0 = 16 * (warp + 1); j0 < 64; j0 += 8) {  // tokens after the row
                const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
                tmem_st8(tlane + Cf::T_P + j0, zero);
            }
            tmem_st_wait();
            tc_fence_before();
            mbar_arrive(&ctl->p_ready);
        }
    } else if (warp < 8) {
        // ---- outputs (thread = token row)
        reg_split<DK, kRegsO>();
        const int row = tid - 128;
        float gi = 0.f, gc = 0.f;              // G of the row and of the chunk and the chunk's kind, read a
        bool next_strong = false;              // chunk ahead (their places are reused)
        if (nch > 0 && wt.warp(&ctl->full[0], 0, 12)) {
            gi = arr_g(0)[row];
            gc = arr_g(0)[kC - 1];
            next_strong = ctl->strong[0];
            mbar_arrive(&ctl->o_free);         // nothing to read yet
        }
        for (int c = 0; c < nch; ++c) {
            const bool strong = next_strong;
            float gs = w.scale * ex2(strong ? gi : gi - gc);
            const int u0 = t0 + c * kC + (row & ~3);       // first row of the four lanes that trade pieces
            __nv_bfloat16 *op = w.o + b * w.ob + (tb + u0) * w.ot + hv * w.oh + 8 * (lane & 3);
            if (c + 1 < nch) {
                if (!wt.warp(&ctl->full[(c + 1) & 1], ((c + 1) >> 1) & 1, 13)) break;
                gi = arr_g(c + 1)[row];
                gc = arr_g(c + 1)[kC - 1];
                next_strong = ctl->strong[(c + 1) & 1];
            }
            if (strong) {                                   // the first term takes its factor before P V is added
                if (!wt.warp(&ctl->q_free, c & 1, 14)) break;
                tc_fence_after();
#pragma unroll 1
                for (int cb = 0; cb < DV; cb += 32) {
                    uint32_t x[32];
                    tmem_ld32(tlane + Cf::T_O + cb, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) x[j] = __float_as_uint(gs * __uint_as_float(x[j]));
                    tmem_st32(tlane + Cf::T_O + cb, x);
                }
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&ctl->r_ready);
                gs = 1.f;
            }
            if (!wt.warp(&ctl->o_full, c & 1, 15)) break;
            tc_fence_after();
#pragma unroll 1
            for (int cb = 0; cb < DV; cb += 32) {
                uint32_t x[32];
                tmem_ld32(tlane + Cf::T_O + cb, x);
                tmem_ld_wait();
                if (cb + 32 == DV) {       // the accumulator is free before the last stores go out
                    tc_fence_before();
                    mbar_arrive(&ctl->o_free);
                }
                // Stored as they lie, a row to a thread, 16-byte stores would touch 32 lines each and stall
                // for thousands of clocks; four lanes trade 16-byte pieces, so that they hold 64
                // bytes of one row at a time.
                uint4 r[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    uint32_t *pr = &r[j].x;
#pragma unroll
                    for (int i = 0; i < 4; ++i)
                        pr[i] = pack_bf16(gs * __uint_as_float(x[8 * j + 2 * i]), gs * __uint_as_float(x[8 * j + 2 * i + 1]));
                }
                trade4(r, lane);
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (u0 + j < t1) *reinterpret_cast<uint4 *>(op + (long long)j * w.ot + cb) = r[j];
            }
        }
    } else if (warp < 16) {
        // ---- the memory (thread = value channel i, TMEM lane i, half of the key channels; dv = 64: half of the warps)
        reg_split<DK, kRegsM>();
        constexpr int NB = DK / 64;                // blocks of 32 key channels
        const int i = tid & 127, k0 = (warp >> 2 & 1) * (DK / 2);
        const bool mine = (i & ~31) < DV;
        uint8_t *sb = smem + Cf::SB;
        float S[NB][32], alpha = 0.f;
        // what the start, or the last chunk's products, left in TMEM is added
        auto add = [&]() {
#pragma unroll
            for (int n = 0; n < NB; ++n)
#pragma unroll
                for (int h = 0; h < 32; h += 16) {
                    uint32_t x[16];
                    tmem_ld16(tlane + Cf::T_S + k0 + 32 * n + h, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 16; ++j) S[n][h + j] = fmaf(alpha, S[n][h + j], __uint_as_float(x[j]));
                }
        };
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int j = 0; j < 32; ++j) S[n][j] = 0.f;
        for (int c = 0; c < nch; ++c) {
            if (!wt.warp(&ctl->full[c & 1], (c >> 1) & 1, 16)) break;
            const float next = ex2(arr_g(c)[kC - 1]), beta = ctl->strong[c & 1] ? 1.f : next;
            if (c == 0 ? !wt.warp(&ctl->start, 0, 25)
                       : !wt.warp(&ctl->q_free, (c - 1) & 1, 17) || !wt.warp(&ctl->kv_done, (c - 1) & 1, 18)) break;
            tc_fence_after();
            if (mine) {
                add();
                // operand: row i, 32 key channels at a time
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int j = 0; j < 32; j += 8) {
                        uint4 p;
                        uint32_t *pp = &p.x;
#pragma unroll
                        for (int k = 0; k < 4; ++k) pp[k] = pack_bf16(beta * S[n][j + 2 * k], beta * S[n][j + 2 * k + 1]);
                        *reinterpret_cast<uint4 *>(sb + piece(DV, i, (k0 + 32 * n + j) / 8)) = p;
                    }
                fence_proxy_async();
                tc_fence_before();
            }
            alpha = next;
            mbar_arrive(&ctl->s_ready);
        }
        // the final memory
        if (w.hT && it.p == it.nseg - 1 && mine) {
            float *hp = w.hT + (pair * DK + k0) * DV + i;
            if (nch == 0) {                    // an empty sequence keeps its memory
                for (int j = 0; j < DK / 2; ++j) hp[j * DV] = w.h0 ? w.h0[(pair * DK + k0 + j) * DV + i] : 0.f;
            } else if (wt.warp(&ctl->kv_done, (nch - 1) & 1, 19)) {
                tc_fence_after();
                add();
#pragma unroll
                for (int n = 0; n < NB; ++n)
#pragma unroll
                    for (int j = 0; j < 32; ++j) hp[(32 * n + j) * DV] = S[n][j];
            }
        }
    } else if (warp < 24) {
        // ---- decayed values (thread = value channel, half of the tokens)
        reg_split<DK, kRegsV>();
        const int ch = tid & 127, half = (tid - 512) >> 7;
        const bool mine = (ch & ~31) < DV;
        for (int c = 0; c < nch; ++c) {
            if (!wt.warp(&ctl->full[c & 1], (c >> 1) & 1, 20)) break;
            const float *wa = arr_g(c) + kC;
            uint8_t *k = stage(c) + Cf::QB, *v = stage(c) + 2 * Cf::QB;
            if (c > 0 && !wt.warp(&ctl->kv_done, (c - 1) & 1, 21)) break;   // the last chunk's are used
            const int live = t1 - t0 - c * kC;
            if (live < kC) {
                // rows past the sequence may hold anything: cleared in K and V by the 256 threads, each half of
                // one row (of both tiles' own widths), before any of them reads V
                if (!wt.warp(&ctl->s_full, c & 1, 22)) break;               // product 1 reads K
                if (ch >= live) {
#pragma unroll 1
                    for (int p = half * (DK / 16); p < (half + 1) * (DK / 16); ++p)
                        *reinterpret_cast<uint4 *>(k + piece(kC, ch, p)) = make_uint4(0, 0, 0, 0);
#pragma unroll 1
                    for (int p = half * (DV / 16); p < (half + 1) * (DV / 16); ++p)
                        *reinterpret_cast<uint4 *>(v + piece(kC, ch, p)) = make_uint4(0, 0, 0, 0);
                }
                fence_proxy_async();
                mbar_arrive(&ctl->cleared);                                 // only a sequence's last chunk comes here
                if (!wt.warp(&ctl->cleared, 0, 24)) break;
            }
            tc_fence_after();
            if (mine) put_values<Cf::OWN_HI ? 3 : 1>(v, wa, ch, 64 * half, tlane + Cf::T_HI, tlane + Cf::T_V + 64, tlane + Cf::T_V);
            tc_fence_before();
            mbar_arrive(&ctl->v_ready);
            if constexpr (Cf::OWN_HI) continue;
            if (!wt.warp(&ctl->lo_done, c & 1, 23)) break;
            tc_fence_after();
            if (mine) put_values<2>(v, wa, ch, 64 * half, tlane + Cf::T_HI, 0, 0);
            tc_fence_before();
            mbar_arrive(&ctl->hi_ready);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 25) {
        // nothing of this CTA's is in flight once its last product and loads have landed (a bounded
        // wait: after a time-out they may not have)
        if (lane == 0) mma_commit(&ctl->last);
        __syncwarp();
        (void)mbar_wait(&ctl->last, 0, kWaitNs);
        if (const int where = ctl->fail) {
            if (DK == 128 && lane == 0 && atomicCAS(&w.hdr->error, 0, kStatusDeviceTimeout) == 0) w.hdr->where = where;
            const uint64_t t = globaltimer_ns();
            while (globaltimer_ns() - t < 1000000ull) {
            }
        }
        __syncwarp();
        tc_fence_after();
        tmem_dealloc(tm, 512);
    }
}

// ------------------------------------------------------------------------------ local memories
template <int DK, int DV>
struct LocalCfg {
    static constexpr int KB = kC * DK * 2, VB = kC * DV * 2;
    static constexpr int STAGE = KB + VB;                      // K, V
    static constexpr int NST = STAGE > 48 * 1024 ? 3 : 4;
    static constexpr int ARR = NST * STAGE;                    // per stage: w [128]
    static constexpr int CTL = ARR + NST * kC * 4;
    static constexpr int SMEM = CTL + 256;
    static constexpr int T_V = DK;                             // a chunk's product [DK], two sets of hi, mid, lo
    static_assert(T_V + 384 <= 512 && SMEM <= 232448, "TMEM, shared memory");
};
struct LocalCtl {
    uint64_t full[4], empty[4], ready[2], used[2], d_full, d_free;
    uint32_t tmem;
    int fail;
    int cmd[4];        // 1: a chunk, 0: no more
    float red[8], top[8];
};
static_assert(sizeof(LocalCtl) <= 256, "control block");

// The memory one segment adds from zero, in registers as in the walk.  Warps 0-7: weighted values (thread = channel,
// half of the tokens), the segment's total decay; 8: decays and TMA, from the segment's last chunk to its first; 9:
// products; 12-19: the memory (thread = channel, half of the key channels); 10 and 11 bring these to their TMEM lanes.
constexpr int kLocalThreads = 20 * 32;

template <int DK, int DV>
__global__ void __launch_bounds__(kLocalThreads, 1)
linear_local_kernel(const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, TcWalk w) {
    using Cf = LocalCfg<DK, DV>;
    constexpr int NST = Cf::NST;
    extern __shared__ __align__(1024) uint8_t smem[];
    LocalCtl *ctl = reinterpret_cast<LocalCtl *>(smem + Cf::CTL);
    if ((smem_u32(smem) & 1023) || blockDim.x != kLocalThreads) {
        if (threadIdx.x == 0) atomicCAS(&w.hdr->error, 0, kStatusDeviceTimeout);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (w.clear && blockIdx.x == 0 && tid == 0) w.hdr->error = 0;
    const int hv = blockIdx.x % w.HV, item = blockIdx.x / w.HV;
    LinItem it;
    if (!lin_item(w.s, w.L, item, it) || it.p == it.nseg - 1) return;   // nobody reads the last segment's
    const int t0 = it.p * w.L, nch = w.L / kC;                          // whole chunks: not the last segment
    const int b = w.s.cu ? 0 : it.n;
    const long tb = w.s.cu ? it.start : 0;
    const float *gp = w.g.p ? w.g.p + b * w.g.b + tb * w.g.t + hv : nullptr;
    if (tid == 0) {
        for (int i = 0; i < NST; ++i) {
            mbar_init(&ctl->full[i], 1);
            mbar_init(&ctl->empty[i], 1 + 256);     // the product has read the tiles, the memory's threads the command
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ctl->ready[i], 256);
            mbar_init(&ctl->used[i], 1);
        }
        mbar_init(&ctl->d_full, 1);
        mbar_init(&ctl->d_free, 256);
        ctl->fail = 0;
        fence_mbar_init();
    }
    if (warp == 9) {
        tmem_alloc(&ctl->tmem, 512);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    next_may_start();                       // the TMEM is this CTA's by now (one that returned above has its say too)
    tc_fence_after();
    const uint32_t tm = ctl->tmem;
    const Waits wt{&ctl->fail, w.hdr};
    float *wa = reinterpret_cast<float *>(smem + Cf::ARR);

    if (warp == 8) {
        float tail = 0.f;                       // decays behind the chunk
        float4 d = load_decay(w.g, gp, t0 + (nch - 1) * kC + 4 * lane, 0x7fffffff);
        int n = 0, c = nch - 1;
        bool known = false, never_up = false;
        for (; c >= 0; --c, ++n) {
            const int s = n % NST, u = t0 + c * kC;
            // sums of the decays behind each token: a suffix sum without the token's own
            float4 x = make_float4(d.y + (d.z + d.w), d.z + d.w, d.w, 0.f);
            float down = x.x + d.x;
#pragma unroll
            for (int off = 1; off < 32; off <<= 1) {
                const float y = __shfl_down_sync(0xffffffffu, down, off);
                if (lane + off < 32) down += y;
            }
            const float all = __shfl_sync(0xffffffffu, down, 0);
            float behind = __shfl_down_sync(0xffffffffu, down, 1);
            if (lane == 31) behind = 0.f;
            behind += tail;
            // with no positive decay in the segment the weights only fall from here on
            if (tail < kZeroWeight) {
                if (!known) {
                    named_sync(1, 288);         // the totals are in
                    known = true;
                    never_up = true;
                    for (int i = 0; i < 8; ++i) never_up = never_up && ctl->top[i] <= 0.f;
                }
                if (never_up) break;
            }
            if (n >= NST && !wt.warp(&ctl->empty[s], (n / NST - 1) & 1, 31)) break;
            *reinterpret_cast<float4 *>(wa + s * kC + 4 * lane) =
                make_float4(ex2(x.x + behind), ex2(x.y + behind), ex2(x.z + behind), ex2(x.w + behind));
            __syncwarp();
            if (lane == 0) {
                ctl->cmd[s] = 1;
                uint8_t *st = smem + s * Cf::STAGE;
                mbar_expect_tx(&ctl->full[s], Cf::STAGE);
                const int row = (int)(tb + u), hq = hv / w.m;
#pragma unroll
                for (int i = 0; i < DK / 64; ++i) tma_load_4d(st + i * kC * 128, &mk, &ctl->full[s], 64 * i, hq, row, b);
#pragma unroll
                for (int i = 0; i < DV / 64; ++i)
                    tma_load_4d(st + Cf::KB + i * kC * 128, &mv, &ctl->full[s], 64 * i, hv, row, b);
            }
            tail += all;
            if (c > 0) d = load_decay(w.g, gp, u - kC + 4 * lane, 0x7fffffff);
        }
        if (!known) named_sync(1, 288);
        // tell the others
        const int s = n % NST;
        if (n < NST || wt.warp(&ctl->empty[s], (n / NST - 1) & 1, 32)) {
            if (lane == 0) {
                ctl->cmd[s] = 0;
                mbar_arrive(&ctl->full[s]);
            }
        }
    } else if (warp == 9) {
        constexpr uint32_t id = idesc_bf16_f32(128, DK, false, true);
        for (int n = 0;; ++n) {
            const int s = n % NST;
            if (!wt.warp(&ctl->full[s], (n / NST) & 1, 33)) break;
            if (!ctl->cmd[s]) break;
            if (!wt.warp(&ctl->ready[n & 1], (n >> 1) & 1, 34)) break;
            if (n > 0 && !wt.warp(&ctl->d_free, (n - 1) & 1, 37)) break;
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
    } else if (warp >= 12) {
        constexpr int NB = DK / 64;             // blocks of 32 key channels
        const int ch = tid & 127, k0 = ((warp >> 2) & 1) * (DK / 2);
        const bool mine = (ch & ~31) < DV;
        const uint32_t tlane = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        float S[NB][32];
#pragma unroll
        for (int i = 0; i < NB; ++i)
#pragma unroll
            for (int j = 0; j < 32; ++j) S[i][j] = 0.f;
        bool ok;
        for (int n = 0;; ++n) {
            const int s = n % NST;
            ok = wt.warp(&ctl->full[s], (n / NST) & 1, 38);
            if (!ok || !ctl->cmd[s]) break;
            mbar_arrive(&ctl->empty[s]);
            ok = wt.warp(&ctl->d_full, n & 1, 39);
            if (!ok) break;
            tc_fence_after();
            if (mine) {
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    uint32_t x[32];
                    tmem_ld32(tlane + k0 + 32 * i, x);
                    tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < 32; ++j) S[i][j] += __uint_as_float(x[j]);
                }
            }
            tc_fence_before();
            mbar_arrive(&ctl->d_free);
        }
        if (ok && mine) {
            float *lp = w.loc + (((size_t)item * w.HV + hv) * DK + k0) * DV + ch;
#pragma unroll
            for (int i = 0; i < NB; ++i)
#pragma unroll
                for (int j = 0; j < 32; ++j) lp[(32 * i + j) * DV] = S[i][j];
        }
    } else if (warp < 8) {
        // total decay of the segment, in a fixed order; its largest decay
        float sum = 0.f, top = -INFINITY;
        for (int u = tid; u < w.L; u += 256) {
            const float x = gp ? clamp_decay(gp[(long long)(t0 + u) * w.g.t]) * kLog2e : 0.f;
            sum += x;
            top = x > top || x != x ? x : top;
        }
#pragma unroll
        for (int off = 16; off; off >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, off);
            const float y = __shfl_xor_sync(0xffffffffu, top, off);
            top = y > top || y != y ? y : top;
        }
        if (lane == 0) {
            ctl->red[warp] = sum;
            ctl->top[warp] = top;
        }
        named_sync(2, 256);
        named_arrive(1, 288);                   // the producer warp may look at them
        if (tid == 0) {
            float all = 0.f;
            for (int i = 0; i < 8; ++i) all += ctl->red[i];
            w.gam[(size_t)item * w.HV + hv] = ex2(all);
        }
        const int ch = tid & 127, half = tid >> 7;
        const bool mine = (ch & ~31) < DV;
        const uint32_t tlane = tm + ((uint32_t)(32 * (warp & 3)) << 16);
        for (int n = 0;; ++n) {
            const int s = n % NST;
            if (!wt.warp(&ctl->full[s], (n / NST) & 1, 35)) break;
            if (!ctl->cmd[s]) break;
            if (n >= 2 && !wt.warp(&ctl->used[n & 1], ((n >> 1) - 1) & 1, 36)) break;
            tc_fence_after();
            const uint32_t a = tlane + Cf::T_V + (n & 1) * 192;
            if (mine) put_values<3>(smem + s * Cf::STAGE + Cf::KB, wa + s * kC, ch, 64 * half, a, a + 64, a + 128);
            tc_fence_before();
            mbar_arrive(&ctl->ready[n & 1]);
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 9) {
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

// ------------------------------------------------------------------------------ host
// Chunks per segment.  In units of one chunk of the walk (3.7 us at d = 128, 2.6 at 64), a CTA costs about 3 to set up,
// fill and drain, a chunk of the local kernel 0.5, its launch 1, a start state 0.2 per earlier segment; every
// (sequence, head) that finds no SM waits for the next wave.  Equal lengths: the cut with the least of it, and
// of cuts within 5 % the coarsest (a long segment's local memory stops early where decays are strong: B=1 T=32768
// H=32, 4 segments 0.30 ms, 8 segments 0.36 ms).  Of all cuts of ten shapes, 2048 to 32,768 tokens, 1 to 128 heads, it
// picks the fastest or one within 1 %, in one 9 % (8192 tokens, 4 heads of 128: 39.0 us for 35.9).
// Packed sequences: whole ones while the
// longest is no more than an SM's share of the work (taken longest first they then fill the SMs evenly),
// else segments of half an SM's share.
int plan_chunks(int nseq, int HV, long total, int max_len, bool varlen, int sms) {
    const int nch = std::max(1, (max_len + kC - 1) / kC);
    const long pairs = (long)nseq * HV;
    if (varlen) {
        const double share = (double)(total / kC + nseq) * HV / sms;
        if (nch <= share + 2.0 || nch <= 8) return nch;
        return std::min(nch, std::max(4, (int)(share / 2 + 0.5)));
    }
    int best = nch;
    double cost = 1e30;
    for (int p = 1; p <= std::min(nch, kMaxSegs); ++p) {
        const int lc = (nch + p - 1) / p, segs = (nch + lc - 1) / lc;
        double t = (double)((pairs * segs + sms - 1) / sms) * (lc + 3.0);
        if (segs > 1) t += (double)((pairs * (segs - 1) + sms - 1) / sms) * (0.5 * lc + 3.0) + 1.0 + 0.2 * (segs - 1);
        if (t < 0.95 * cost) {
            cost = t;
            best = lc;
        }
    }
    return best;
}

template <int DK, int DV>
cudaError_t go(const LinFwd &a, const TcWalk &w, long items, bool split, const CUtensorMap &mq, const CUtensorMap &mk,
               const CUtensorMap &mv, cudaStream_t st) {
    using WC = WalkCfg<DK, DV>;
    using LC = LocalCfg<DK, DV>;
    if (items * a.HV > 0x7fffffffL) return cudaErrorInvalidValue;
    const unsigned grid = (unsigned)(items * a.HV);
    static SmemOnce local_once, walk_once;
    cudaError_t e;
    TcWalk first = w;
    first.clear = 1;
    if (split) {
        if ((e = local_once(linear_local_kernel<DK, DV>, LC::SMEM)) != cudaSuccess) return e;
        linear_local_kernel<DK, DV><<<grid, kLocalThreads, LC::SMEM, st>>>(mk, mv, first);
        if ((e = cudaGetLastError()) != cudaSuccess) return e;
    }
    if ((e = walk_once(linear_chunk_kernel<DK, DV>, WC::SMEM)) != cudaSuccess) return e;
    if constexpr (DK == 128) {
        static const cudaError_t held = check_regs(linear_chunk_kernel<DK, DV>, kWalkRegs);
        if (held != cudaSuccess) return held;
    }
    if (split) return launch_after(linear_chunk_kernel<DK, DV>, grid, kWalkThreads, WC::SMEM, st, mq, mk, mv, w);
    linear_chunk_kernel<DK, DV><<<grid, kWalkThreads, WC::SMEM, st>>>(mq, mk, mv, first);
    return cudaGetLastError();
}

}  // namespace

bool linear_tc_supported(int dk, int dv, DType dt) {
    return dt == DType::BF16 && (dk == 64 || dk == 128) && (dv == 64 || dv == 128);
}

size_t linear_tc_scratch_bytes(int nseq, int HV, int dk, int dv, long total, int max_len, bool varlen, int sms) {
    size_t slots;
    if (varlen) {   // whatever the lengths turn out to be: the shortest segments plan_chunks cuts
        const double share = (double)(total / kC + nseq) * HV / sms;
        const long lc = std::max(4, (int)(share / 2 + 0.5));
        slots = (size_t)(total / (lc * kC) + nseq) * HV;
    } else {
        const int lc = plan_chunks(nseq, HV, total, max_len, false, sms);
        if ((long)lc * kC >= max_len) return 0;
        slots = (size_t)lin_items(nseq, total, max_len, false, lc * kC) * HV;
    }
    return round256(slots * dk * dv * 4) + round256(slots * 4);
}

cudaError_t launch_linear_tc(const LinFwd &a, cudaStream_t st) {
    const bool varlen = a.s.cu != nullptr;
    int lc = plan_chunks(a.s.nseq, a.HV, a.total, a.max_len, varlen, a.sms);
    if (a.h0 && a.h0 == a.hT) lc = (a.max_len + kC - 1) / kC;   // in place: every CTA owns its memory
    TcWalk w{};
    w.s = a.s; w.g = a.g; w.L = lc * kC; w.HV = a.HV; w.m = a.HV / a.H;
    w.scale = a.scale; w.h0 = a.h0; w.hT = a.hT;
    w.o = static_cast<__nv_bfloat16 *>(const_cast<void *>(a.o.p));
    w.ob = a.o.b; w.ot = a.o.t; w.oh = a.o.h; w.hdr = a.hdr;
    const bool split = a.max_len > w.L;
    w.sorted = varlen && !split && a.s.nseq > 1 && a.s.nseq <= kSortSeqs;
    const long items = lin_items(a.s.nseq, a.total, a.max_len, varlen, w.L);
    w.loc = static_cast<float *>(a.ws);
    w.gam = reinterpret_cast<float *>(static_cast<char *>(a.ws) + round256((size_t)items * a.HV * a.dk * a.dv * 4));
    const long B = varlen ? 1 : a.s.nseq;
    CUtensorMap mq, mk, mv;
    if (!token_map(&mq, a.q, a.dk, a.H, a.total, B) || !token_map(&mk, a.k, a.dk, a.H, a.total, B) ||
        !token_map(&mv, a.v, a.dv, a.HV, a.total, B))
        return cudaErrorInvalidValue;
    if (a.dk == 128 && a.dv == 128) return go<128, 128>(a, w, items, split, mq, mk, mv, st);
    if (a.dk == 128) return go<128, 64>(a, w, items, split, mq, mk, mv, st);
    if (a.dv == 128) return go<64, 128>(a, w, items, split, mq, mk, mv, st);
    return go<64, 64>(a, w, items, split, mq, mk, mv, st);
}

}  // namespace kda
