// unpermute_bwd.hip -- gradient of the weighted unpermute on gfx950:
//
//   dy[row, c] = bf16(w[t,k] dout[t,c]),  dw[t,k] = sum_c y[row,c] dout[t,c],
//   row = inv_perm[t,k]
//
// Bound by HBM: every y row read once, every dy row written once (16384
// tokens, top-8, 2048 columns: 1.14 GB in 219 us, 5.2 TB/s).  One wave takes a
// token and a share of its picks, so dw needs no sum across waves and its
// order is fixed; it loads up to four 512-column slabs of a row before it uses
// the first (without: 222-226 us).
#include "moe_device.hpp"
#include "moe_internal.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 20;   // along the tokens: a launch holds fewer than 2^32 threads

__global__ __launch_bounds__(kThreads) void k_unpermute_bwd(const uint16_t* __restrict__ dout,
                                                            const uint16_t* __restrict__ y, int64_t y_rows,
                                                            const int32_t* __restrict__ inv_perm,
                                                            const float* __restrict__ topk_w, int64_t Mc, int K,
                                                            int topk, uint16_t* __restrict__ dy,
                                                            float* __restrict__ dweights) {
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (topk + (int)gridDim.y - 1) / (int)gridDim.y;
    const int k_end = min(topk, ((int)blockIdx.y + 1) * per);
    constexpr int kSlabs = 4;   // 512-column slabs in flight
    int64_t t = (int64_t)blockIdx.x * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (; t < Mc; t += (int64_t)gridDim.x * (kThreads / kWave)) {
        for (int k = (int)blockIdx.y * per; k < k_end; ++k) {
            const int64_t row = inv_perm[t * topk + k];
            float acc = 0.0f;
            if (row >= 0 && row < y_rows) {
                const float w = topk_w[t * topk + k];
                for (int c0 = lane * 8; c0 < K; c0 += kSlabs * kWave * 8) {
                    uint4 yv[kSlabs], dv[kSlabs];
#pragma unroll
                    for (int b = 0; b < kSlabs; ++b) {
                        const int c = c0 + b * kWave * 8 < K ? c0 + b * kWave * 8 : c0;
                        yv[b] = load_once16(y + row * K + c);
                        dv[b] = *reinterpret_cast<const uint4*>(dout + t * K + c);
                    }
#pragma unroll
                    for (int b = 0; b < kSlabs; ++b) {
                        const int c = c0 + b * kWave * 8;
                        if (c >= K) break;
                        float d[8], v[8];
                        bf16x8_to_f32(dv[b], d);
                        bf16x8_to_f32(yv[b], v);
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            acc = __builtin_fmaf(v[i], d[i], acc);
                            d[i] *= w;
                        }
                        store_once16(dy + row * K + c, uint4{f32x2_to_bf16x2(d[0], d[1]), f32x2_to_bf16x2(d[2], d[3]),
                                                         f32x2_to_bf16x2(d[4], d[5]), f32x2_to_bf16x2(d[6], d[7])});
                    }
                }
            }
#pragma unroll
            for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m, kWave);
            if (lane == 0) dweights[t * topk + k] = acc;
        }
    }
}

}  // namespace

hipError_t launch_unpermute_bwd(const uint16_t* dout, const uint16_t* y, int64_t y_rows, const int32_t* inv_perm,
                                const float* topk_w, int64_t Mc, int K, int topk, uint16_t* dy, float* dweights,
                                int num_cus, hipStream_t s) {
    int64_t bx = (Mc + kThreads / kWave - 1) / (kThreads / kWave);
    bx = bx < kMaxBlocks ? bx : kMaxBlocks;
    // a token's picks over several waves until there are 64 blocks per CU
    // (8 blocks: 223 us, 32: 221, 64: 219 at 16384 tokens; level at 130)
    int64_t by = (64 * (int64_t)num_cus + bx - 1) / bx;
    by = by > topk ? topk : by;
    k_unpermute_bwd<<<dim3((unsigned)bx, (unsigned)by), kThreads, 0, s>>>(dout, y, y_rows, inv_perm, topk_w, Mc, K,
                                                                          topk, dy, dweights);
    return hipGetLastError();
}

}  // namespace moe
