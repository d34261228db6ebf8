// linear_tc.cuh -- what the tensor-core kernels of linear attention (linear_tc.cu, linear_tc_bwd.cu) share:
// chunk constants, bounded waits, operand layouts, the three-part operand, tensor maps.
#pragma once

#include <atomic>

#include "linear_internal.cuh"
#include "linear_ptx.cuh"
#include "tma_host.cuh"

namespace kda {
namespace lin {

using namespace ptx;

constexpr int kC = 128;                        // tokens per chunk
constexpr uint64_t kWaitNs = 2000000000ull;
constexpr int kStatusDeviceTimeout = 8;        // KDA_ERR_DEVICE_TIMEOUT
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kMildSpan = 62.f;

// 2^x (ex2.approx: 2 ulp; results below 2^-126 are 0)
__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// Whether a chunk's weights e^{G_i - G_j} factor over rows and columns, e^{G_i - G_C} e^{G_C - G_j}: its running log2
// decays (a lane's four, `end` the last of all) lie within kMildSpan of the chunk's start and of its end, so that no
// factor passes 2^62.  Decays that only fall are mild by the first alone; ones that fall and grow again would have
// columns of up to 2^124, which times a score passes fp32 where no result does.
__device__ __forceinline__ bool is_mild(const float4 &x, float end) {
    const float top = fmaxf(fmaxf(x.x, x.y), fmaxf(x.z, x.w)), low = fminf(fminf(x.x, x.y), fminf(x.z, x.w));
    return fmaxf(top, top - end) <= kMildSpan && fminf(low, low - end) >= -kMildSpan;
}
__device__ __forceinline__ void named_sync(int id, int count) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(count) : "memory");
}
__device__ __forceinline__ void named_arrive(int id, int count) {
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(count) : "memory");
}

// A CTA's failure flag and its bounded waits: once one has run out, the others return at once.
struct Waits {
    volatile int *fail;
    WsHeader *hdr;
    __device__ __forceinline__ bool wait(uint64_t *bar, uint32_t parity, int where) const {
        return mbar_try_wait(bar, parity) || slow(bar, parity, where);
    }
    // out of line: the roles' loops have to stay in the instruction caches
    __device__ __noinline__ bool slow(uint64_t *bar, uint32_t parity, int where) const {
        if (*fail) return false;
        const uint64_t t0 = globaltimer_ns();
        while (true) {
#pragma unroll 1
            for (int i = 0; i < 64; ++i)
                if (mbar_try_wait(bar, parity)) return true;
            if (*fail) return false;
            if (globaltimer_ns() - t0 > kWaitNs) break;
        }
        *fail = 1;
        if (atomicCAS(&hdr->error, 0, kStatusDeviceTimeout) == 0) hdr->where = where;
        return false;
    }
    // for a whole warp, which goes on or leaves together
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity, int where) const {
        return __all_sync(0xffffffffu, wait(bar, parity, where));
    }
};

// The same without a call, which goes with no setmaxnreg, and in few instructions: the time from the timer's lower half
// (it comes round after 4.3 s), a failure left in `fail` for the CTA's end to record.
struct ShortWaits {
    volatile int *fail;
    __device__ __forceinline__ bool warp(uint64_t *bar, uint32_t parity, int where) const {
        bool ok = mbar_try_wait(bar, parity);
        if (!ok) {
            const uint32_t t0 = now();
#pragma unroll 1
            do ok = mbar_try_wait(bar, parity);
            while (!ok && !*fail && now() - t0 < (uint32_t)kWaitNs);
            if (!ok && !*fail) *fail = where;
        }
        return __all_sync(0xffffffffu, ok);
    }
    static __device__ __forceinline__ uint32_t now() {
        uint32_t t;
        asm volatile("mov.u32 %0, %globaltimer_lo;" : "=r"(t));
        return t;
    }
};

// A decayed value x = w v in fp32 goes in as the sum of three bf16s: each takes the top 8 bits of what is
// left (a truncation, so the rest is exact), together x's 24.  Their products are added up from the smallest part on: the
// accumulator cuts every step towards 0, by its own size, which is next to nothing until the large part comes (8 of
// the 24 steps; the other way round a chunk's product lost three times as much).
__device__ __forceinline__ uint32_t top2(float a, float b) {
    return __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x7632);
}
__device__ __forceinline__ float rest(float a) { return a - __uint_as_float(__float_as_uint(a) & 0xffff0000u); }
// byte offset of 16-byte piece c of row r in a bf16 tile [rows][D] (blocks of 64 channels, 128-byte swizzle)
__device__ __forceinline__ uint32_t piece(int rows, int r, int c) {
    return (uint32_t)((c >> 3) * rows * 128 + r * 128 + (((c & 7) ^ (r & 7)) << 4));
}
// The decayed values of the warp's 32 channels (from `ch`, its TMEM lanes), tokens t0 .. t0 + 63, as A-operand
// words (two tokens each) into column t0 / 2 of each part.  PARTS: bit 0 mid and lo, bit 1 hi.  The tile is
// token-major: ldmatrix transposes it into the layout that a 16x128b store takes (lane l holds channel l / 4,
// tokens 2 (l % 4) and the next of each 8), 16 channels by 32 tokens a step.
template <int PARTS>
__device__ __forceinline__ void put_values(const uint8_t *v, const float *wa, int ch, int t0, uint32_t hi, uint32_t mid,
                                           uint32_t lo) {
    const int lane = threadIdx.x & 31, row = ((lane >> 4) << 3) | (lane & 7);
    const uint32_t base = smem_u32(v) + (ch >> 6) * kC * 128 + row * 128;
    const int c = ((ch >> 3) & 4) + ((lane >> 3) & 1);        // 16-byte piece of the row
    wa += 2 * (lane & 3);
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
        const int t = t0 + (u >> 1) * 32;
        const uint32_t at = base + t * 128 + (((c + 2 * (u & 1)) ^ (lane & 7)) << 4);
        uint32_t r[8], h[8], m[8], l[8];
        ldsm4t(at, r);
        ldsm4t(at + 16 * 128, r + 4);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const float2 w = *reinterpret_cast<const float2 *>(wa + t + (j >> 1) * 8);
            const float x = w.x * __uint_as_float(r[j] << 16), y = w.y * __uint_as_float(r[j] & 0xffff0000u);
            if constexpr (PARTS & 2) h[j] = top2(x, y);
            if constexpr (PARTS & 1) {
                const float rx = rest(x), ry = rest(y);
                m[j] = top2(rx, ry);
                l[j] = top2(rest(rx), rest(ry));
            }
        }
        const uint32_t to = ((uint32_t)(u & 1) << 20) + t / 2;  // 16 lanes on
        if constexpr (PARTS & 1) {
            tmem_st_16x128(lo + to, l);
            tmem_st_16x128(mid + to, m);
        }
        if constexpr (PARTS & 2) tmem_st_16x128(hi + to, h);
    }
    tmem_st_wait();
}

// One product: a sum over K in steps of 16, issued by one lane.  A step moves a descriptor's start address, in
// 16-byte units: a K-major tile of ROWS rows by 32 bytes inside a block of 64 channels, an MN-major one (ROWS = 0)
// by 16 rows of 128 bytes.
constexpr uint64_t op_step(int ks, int rows) {
    return rows ? (uint64_t)((ks >> 2) * rows * 8 + (ks & 3) * 2) : (uint64_t)ks * 128;
}
template <int STEPS, int RA, int RB, bool ADD>
__device__ __forceinline__ void product_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id) {
    if constexpr (ADD)
        mma_ss<1>(d, a, b, id);
    else
        mma_ss<0>(d, a, b, id);
#pragma unroll
    for (int ks = 1; ks < STEPS; ++ks) mma_ss<1>(d, a + op_step(ks, RA), b + op_step(ks, RB), id);
}
// A in TMEM, 8 columns a step (QUARTERS: of every 32 columns the first 16), B MN-major, 128 tokens
template <bool ADD, bool QUARTERS = false>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id) {
    if constexpr (ADD)
        mma_ts<1>(d, a, b, id);
    else
        mma_ts<0>(d, a, b, id);
#pragma unroll
    for (int ks = 1; ks < kC / 16; ++ks)
        mma_ts<1>(d, a + (QUARTERS ? 32 * (ks >> 1) + 8 * (ks & 1) : 8 * ks), b + op_step(ks, 0), id);
}

// Lane t of a group of four starts with four pieces of its own row and ends with piece t of the
// four rows.
__device__ __forceinline__ void trade4(uint4 (&r)[4], int lane) {
#pragma unroll
    for (int b = 1; b < 4; b <<= 1) {
        const bool up = lane & b;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (j & b) continue;
            uint32_t *lo = &r[j].x, *hi = &r[j | b].x;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? lo[i] : hi[i], b);
                if (up) lo[i] = got; else hi[i] = got;
            }
        }
    }
}

// log2 decays of tokens u .. u + 3 of the sequence (u >= limit: 0)
__device__ __forceinline__ float4 load_decay(const LinDecay &g, const float *gp, int u, int limit) {
    float4 d;
    float *p = &d.x;
#pragma unroll
    for (int i = 0; i < 4; ++i) p[i] = (gp && u + i < limit) ? clamp_decay(gp[(long long)(u + i) * g.t]) * kLog2e : 0.f;
    return d;
}

// ---- host
inline bool token_map(CUtensorMap *map, const LinView &v, int D, int heads, long T, long B, int rows = kC) {
    const uint64_t dims[4] = {(uint64_t)D, (uint64_t)heads, (uint64_t)T, (uint64_t)B};
    const uint64_t st[3] = {(uint64_t)v.h * 2, (uint64_t)v.t * 2, (uint64_t)v.b * 2};
    const uint32_t box[4] = {64, 1, (uint32_t)rows, 1};
    return make_tensor_map(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, v.p, dims, st, box, true);
}

// A kernel's dynamic shared memory limit, raised once per device.
struct SmemOnce {
    std::atomic<unsigned long long> done{0};
    template <typename K> cudaError_t operator()(K *kernel, int bytes) {
        int dev = 0;
        cudaError_t e = cudaGetDevice(&dev);
        if (e != cudaSuccess) return e;
        const unsigned long long bit = 1ull << (dev & 63);
        if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
        return e;
    }
};

inline size_t round256(size_t n) { return (n + 255) & ~size_t(255); }

}  // namespace lin
}  // namespace kda
