// silu_mul.hip -- SiLU-mul on bf16 rows and its gradient, between the two
// grouped products of the bf16 experts on gfx950.
//
//   act = g u s,  dg = d u s (1 + g (1 - s)),  du = d g s,  s = 1 / (1 + e^-g)
//
// in fp32, each output rounded once to bf16.  e^-g may reach infinity (then
// s = 0 and every product with a finite factor is 0) or 0 (s = 1), without a
// clamp: large |g| of either sign come out right while s (g >= -87) and d u are
// values that fp32 holds.  Below, s counts as 0 and an output is off by less
// than 2^-118 times its other factors; splitting s over the factors removes
// that and cost 5-20% of the time (130 to 16384 tokens).  The hardware
// exponential and reciprocal are off by a few 2^-24 (1 + |g|) relative, against
// the 2^-8 of the rounding to bf16.
//
// Bound by HBM: 6 bytes per act element forward, 10 backward.  Only valid rows
// are walked: every block scans the experts' row counts in LDS, takes a
// contiguous share of the valid rows and walks it in 16-byte chunks, each
// thread keeping the expert of its row, so padding costs nothing.
#include "moe_device.hpp"
#include "moe_internal.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float sigmoid(float g) { return __builtin_amdgcn_rcpf(1.0f + __expf(-g)); }

__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
    return uint4{f32x2_to_bf16x2(v[0], v[1]), f32x2_to_bf16x2(v[2], v[3]), f32x2_to_bf16x2(v[4], v[5]),
                 f32x2_to_bf16x2(v[6], v[7])};
}

template <bool BWD>
__global__ __launch_bounds__(kThreads) void k_silu(const uint16_t* h, const uint16_t* __restrict__ dact,
                                                   int64_t rows, int n, const int32_t* __restrict__ offsets,
                                                   const int32_t* __restrict__ counts, int El, uint16_t* out) {
    constexpr int kPer = kMaxLocalExperts / kThreads;
    __shared__ int s_pre[kMaxLocalExperts + 1];   // valid rows before expert e
    __shared__ int s_lo[kMaxLocalExperts];        // its first row
    __shared__ int64_t s_wsum[kThreads / kWave];
    int64_t total = rows;
    if (offsets != nullptr) {
        // 64-bit sums, stored capped at `rows`: segments that overlap (offsets
        // out of order) cannot push the walk past its tables
        int64_t sum = 0;
        int c[kPer], off[kPer + 1], num[kPer];   // loaded without conditions, so together
        const int rows32 = (int)rows;
#pragma unroll
        for (int j = 0; j <= kPer; ++j) off[j] = offsets[min((int)threadIdx.x * kPer + j, El)];
#pragma unroll
        for (int j = 0; j < kPer; ++j) num[j] = counts[min((int)threadIdx.x * kPer + j, El - 1)];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = threadIdx.x * kPer + j;
            const int end = max(0, min(off[j + 1], rows32)), lo = max(0, min(off[j], end));
            c[j] = e < El ? min(max(num[j], 0), end - lo) : 0;
            if (e < El) s_lo[e] = lo;
            sum += c[j];
        }
        const int64_t incl = wave_inclusive_scan(sum);
        const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
        if (lane == kWave - 1) s_wsum[wave] = incl;
        __syncthreads();
        int64_t run = incl - sum;
        for (int w = 0; w < wave; ++w) run += s_wsum[w];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = threadIdx.x * kPer + j;
            if (e < El) s_pre[e] = (int)(run < rows ? run : rows);
            run += c[j];
        }
        if (threadIdx.x == kThreads - 1) s_pre[El] = (int)(run < rows ? run : rows);
        __syncthreads();
        total = s_pre[El];
    }
    // the block's rows: total / grid of them, the first total mod grid blocks one more
    const uint32_t per = (uint32_t)total / gridDim.x, more = (uint32_t)total - per * gridDim.x;
    const int64_t v_lo = (int64_t)(blockIdx.x * per + min(blockIdx.x, more));
    const int64_t v_hi = v_lo + per + (blockIdx.x < more);
    if (v_lo >= v_hi) return;
    const int nch = n / 8;
    const int step_r = kThreads / nch, step_c = kThreads - step_r * nch;
    int64_t v = v_lo + threadIdx.x / nch;
    int c = threadIdx.x % nch;
    int e = 0;
    if (offsets != nullptr) {
        // the last expert with s_pre[e] <= the block's first row; the walk goes on from there
        const int lane = threadIdx.x & (kWave - 1);
        e = -1;
        for (int j = 0; j < El; j += kWave) e += __popcll(ballot(j + lane < El && s_pre[min(j + lane, El)] <= v_lo));
    }
    for (; v < v_hi;) {
        int64_t r = v;
        if (offsets != nullptr) {
            while (s_pre[e + 1] <= v) ++e;   // v < s_pre[El], so this ends at e < El
            r = s_lo[e] + (v - s_pre[e]);
        }
        float g[8], u[8];
        const int64_t at = r * 2 * n + c * 8;
        bf16x8_to_f32(load_once16(h + at), g);
        bf16x8_to_f32(load_once16(h + at + n), u);
        if constexpr (BWD) {
            float d[8], dg[8], du[8];
            bf16x8_to_f32(load_once16(dact + r * n + c * 8), d);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float s = sigmoid(g[i]);
                dg[i] = d[i] * u[i] * (s * (1.0f + g[i] * (1.0f - s)));
                du[i] = d[i] * (g[i] * s);
            }
            store_once16(out + at, pack8(dg));
            store_once16(out + at + n, pack8(du));
        } else {
            float act[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) act[i] = g[i] * sigmoid(g[i]) * u[i];
            store_once16(out + r * n + c * 8, pack8(act));
        }
        v += step_r;
        c += step_c;
        if (c >= nch) {
            c -= nch;
            ++v;
        }
    }
}

// Two chunks a thread of the buffer's rows (which of them are valid the host
// does not know) until there are 128 blocks per CU, then more: many short
// blocks keep the streams' pages close together, until every block's scan of
// the counts tells.  131072 valid rows of 147328, 768 wide, forward / backward
// us: 32 blocks per CU 105 / 181, 64 97 / 170, 128 92 / 161, 192 111 / 156;
// 16000 valid rows of 32256: one chunk a thread 24 / 27, two 16.5 / 22, three
// 14.6 / 23, six 14.5 / 23; 128 of 4096: 3.6 / 3.7 and 3.05 / 3.4; 1400 of
// 1520, 1504 wide: 5.1 / 6.2, 4.8 / 6.5 and 5.6 / 7.1.
unsigned grid_for(int64_t rows, int n, int num_cus) {
    int64_t b = (rows * (n / 8) + 2 * kThreads - 1) / (2 * kThreads);
    b = b > 128 * num_cus ? 128 * num_cus : b;
    return (unsigned)(b < 1 ? 1 : b);
}

}  // namespace

hipError_t launch_silu_mul(const uint16_t* h, int64_t rows, int n, const int32_t* offsets, const int32_t* counts,
                           int El, uint16_t* act, int num_cus, hipStream_t s) {
    k_silu<false><<<grid_for(rows, n, num_cus), kThreads, 0, s>>>(h, nullptr, rows, n, offsets, counts, El, act);
    return hipGetLastError();
}

hipError_t launch_silu_mul_bwd(const uint16_t* h, const uint16_t* dact, int64_t rows, int n, const int32_t* offsets,
                               const int32_t* counts, int El, uint16_t* dh, int num_cus, hipStream_t s) {
    k_silu<true><<<grid_for(rows, n, num_cus), kThreads, 0, s>>>(h, dact, rows, n, offsets, counts, El, dh);
    return hipGetLastError();
}

}  // namespace moe
