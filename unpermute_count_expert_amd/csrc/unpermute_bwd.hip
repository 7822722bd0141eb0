// unpermute_bwd.hip -- gradient of the weighted unpermute on gfx950:
//
//   dy[row, c] = bf16(w[t,k] dout[t,c]),  dw[t,k] = sum_c y[row,c] dout[t,c],
//   row = inv_perm[t,k]
//
// Bound by HBM: every y row read once, every dy row written once.  One wave
// takes a token and a share of its picks, so dw needs no sum across waves and
// its order is fixed.
#include "moe_device.hpp"
#include "moe_internal.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void k_unpermute_bwd(const uint16_t* __restrict__ dout,
                                                            const uint16_t* __restrict__ y, int64_t y_rows,
                                                            const int32_t* __restrict__ inv_perm,
                                                            const float* __restrict__ topk_w, int64_t Mc, int K,
                                                            int topk, uint16_t* __restrict__ dy,
                                                            float* __restrict__ dweights) {
    const int lane = threadIdx.x & (kWave - 1);
    const int64_t t = (int64_t)blockIdx.x * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    if (t >= Mc) return;
    const int per = (topk + (int)gridDim.y - 1) / (int)gridDim.y;
    const int k_end = min(topk, ((int)blockIdx.y + 1) * per);
    for (int k = (int)blockIdx.y * per; k < k_end; ++k) {
        const int64_t row = inv_perm[t * topk + k];
        float acc = 0.0f;
        if (row >= 0 && row < y_rows) {
            const float w = topk_w[t * topk + k];
            for (int c = lane * 8; c < K; c += kWave * 8) {
                float d[8], v[8];
                bf16x8_to_f32(*reinterpret_cast<const uint4*>(dout + t * K + c), d);
                bf16x8_to_f32(load_once16(y + row * K + c), v);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    acc = __builtin_fmaf(v[i], d[i], acc);
                    d[i] *= w;
                }
                store_once16(dy + row * K + c, uint4{f32x2_to_bf16x2(d[0], d[1]), f32x2_to_bf16x2(d[2], d[3]),
                                                     f32x2_to_bf16x2(d[4], d[5]), f32x2_to_bf16x2(d[6], d[7])});
            }
        }
#pragma unroll
        for (int m = 32; m > 0; m >>= 1) acc += __shfl_xor(acc, m, kWave);
        if (lane == 0) dweights[t * topk + k] = acc;
    }
}

}  // namespace

hipError_t launch_unpermute_bwd(const uint16_t* dout, const uint16_t* y, int64_t y_rows, const int32_t* inv_perm,
                                const float* topk_w, int64_t Mc, int K, int topk, uint16_t* dy, float* dweights,
                                int num_cus, hipStream_t s) {
    const int64_t bx = (Mc + kThreads / kWave - 1) / (kThreads / kWave);
    // few tokens: their picks over several waves, until the CUs have eight blocks each
    int64_t by = (8 * (int64_t)num_cus + bx - 1) / bx;
    by = by > topk ? topk : by;
    k_unpermute_bwd<<<dim3((unsigned)bx, (unsigned)by), kThreads, 0, s>>>(dout, y, y_rows, inv_perm, topk_w, Mc, K,
                                                                          topk, dy, dweights);
    return hipGetLastError();
}

}  // namespace moe
