// checkpoint.hip -- what a training step keeps of a forward call in 8 bits, and
// the rows of the backward pass, on gfx950.
//
// A block of 32 values along a row has one scale, the least power of two that
// brings its largest magnitude to e4m3's 448 or below (one byte, E8M0), and 32
// e4m3 codes.  A power of two costs e4m3 no precision (it has its own
// exponents) and makes code * scale a bf16 number exactly, so nothing is
// rounded when a checkpoint is restored.
//
// All kernels here are bound by HBM.
#include "moe_device.hpp"
#include "moe_internal.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int64_t kMaxBlocks = 1 << 20;   // a launch holds fewer than 2^32 threads

// The largest of a lane's value over its quad of lanes.
__device__ __forceinline__ uint32_t quad_max(uint32_t m) {
    m = max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0xb1, 0xf, 0xf, false));   // lanes 1 0 3 2
    return max(m, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)m, 0x4e, 0xf, 0xf, false));   // lanes 2 3 0 1
}

__device__ __forceinline__ uint2 encode8(const float (&v)[8], float scale) {
    return uint2{f32x4_to_e4m3_scaled(v[0], v[1], v[2], v[3], scale),
                 f32x4_to_e4m3_scaled(v[4], v[5], v[6], v[7], scale)};
}

__device__ __forceinline__ uint4 decode8(uint2 c, float scale) {
    const f32x4 x = e4m3x4_to_f32_scaled(c.x, scale), y = e4m3x4_to_f32_scaled(c.y, scale);
    return uint4{f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(y[0], y[1]),
                 f32x2_to_bf16x2(y[2], y[3])};
}

// Rows are whole blocks, so the matrix is one line of them: a lane takes eight
// values, a quad of lanes a block, each thread kSets of its octets in flight.
constexpr int kSets = 4;
__global__ __launch_bounds__(kThreads) void k_encode(const uint16_t* __restrict__ x, int64_t octets,
                                                     uint8_t* __restrict__ q, uint8_t* __restrict__ scales) {
    const int64_t stride = (int64_t)gridDim.x * kThreads * kSets;
    for (int64_t o0 = (int64_t)blockIdx.x * kThreads * kSets + threadIdx.x; o0 < octets; o0 += stride) {
        uint4 in[kSets];
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const int64_t o = o0 + s * kThreads;
            in[s] = load_once16(x + (o < octets ? o : o0) * 8);
        }
#pragma unroll
        for (int s = 0; s < kSets; ++s) {
            const int64_t o = o0 + s * kThreads;   // of a quad, all four or none are below octets
            float v[8];
            bf16x8_to_f32(in[s], v);
            uint32_t m = 0;
#pragma unroll
            for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(v[i]) & 0x7fffffffu);
            const uint32_t e = e8m0_of(quad_max(m));
            if (o >= octets) break;
            const uint2 c = encode8(v, e8m0_value(e));
            *reinterpret_cast<uint2*>(q + o * 8) = c;
            if ((threadIdx.x & 3) == 0) scales[o >> 2] = (uint8_t)e;
        }
    }
}

// out[inv_perm[t, k]] = token t's row, bf16 as it is or restored from 8 bits,
// and row_weights[inv_perm[t, k]] = topk_w[t, k]; inv_perm null: out[t].  One
// wave takes a token and a share of its picks and reads its row once for them,
// kSlabs slabs of 512 columns at a time.  NT: non-temporal stores.
template <bool CODES, bool NT>
__global__ __launch_bounds__(kThreads) void k_rows(const void* __restrict__ x, const uint8_t* __restrict__ scales,
                                                   const int32_t* __restrict__ inv_perm,
                                                   const float* __restrict__ topk_w, int64_t Mc, int K, int topk,
                                                   uint16_t* __restrict__ out, int64_t out_rows,
                                                   float* __restrict__ row_weights) {
    constexpr int kSlabs = 4;
    const int lane = threadIdx.x & (kWave - 1);
    const int per = (topk + (int)gridDim.y - 1) / (int)gridDim.y;
    const int k_lo = (int)blockIdx.y * per, k_end = min(topk, k_lo + per);
    int64_t t = (int64_t)blockIdx.x * (kThreads / kWave) + __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    for (; t < Mc; t += (int64_t)gridDim.x * (kThreads / kWave)) {
        for (int c0 = lane * 8; c0 - lane * 8 < K; c0 += kSlabs * kWave * 8) {
            uint4 v[kSlabs];
            if constexpr (CODES) {
                uint2 q[kSlabs];
                uint32_t s[kSlabs];
#pragma unroll
                for (int b = 0; b < kSlabs; ++b) {
                    const int64_t at = t * K + min(c0 + b * kWave * 8, K - 8);
                    q[b] = *reinterpret_cast<const uint2*>(static_cast<const uint8_t*>(x) + at);
                    s[b] = scales[at >> 5];
                }
#pragma unroll
                for (int b = 0; b < kSlabs; ++b) v[b] = decode8(q[b], e8m0_value(s[b]));
            } else {
#pragma unroll
                for (int b = 0; b < kSlabs; ++b)
                    v[b] = *reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(x) + t * K +
                                                           min(c0 + b * kWave * 8, K - 8));
            }
            for (int k = k_lo; k < k_end; ++k) {
                const int64_t row = inv_perm ? inv_perm[t * topk + k] : t;
                if (row < 0 || row >= out_rows) continue;
#pragma unroll
                for (int b = 0; b < kSlabs; ++b) {
                    const int c = c0 + b * kWave * 8;
                    if (c >= K) break;
                    if constexpr (NT) store_once16(out + row * K + c, v[b]);
                    else *reinterpret_cast<uint4*>(out + row * K + c) = v[b];
                }
                if (row_weights && c0 == 0) row_weights[row] = topk_w[t * topk + k];
            }
        }
    }
}

// dweights[t, k] = the sum of dots[inv_perm[t, k], :], sixteen lanes a pair, in
// a fixed order.
__global__ __launch_bounds__(kThreads) void k_dots(const float* __restrict__ dots, int nd, int64_t rows,
                                                   const int32_t* __restrict__ inv_perm, int64_t pairs,
                                                   float* __restrict__ dweights) {
    const int l = threadIdx.x & 15;
    for (int64_t p = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 4; p < pairs;
         p += (int64_t)gridDim.x * (kThreads / 16)) {
        const int64_t row = inv_perm[p];
        float sum = 0.0f;
        if (row >= 0 && row < rows)
            for (int i = l; i < nd; i += 16) sum += dots[row * nd + i];
#pragma unroll
        for (int m = 8; m > 0; m >>= 1) sum += __shfl_xor(sum, m, 16);
        if (l == 0) dweights[p] = sum;
    }
}

}  // namespace

hipError_t launch_checkpoint(const uint16_t* x, int64_t values, uint8_t* q, uint8_t* scales, hipStream_t s) {
    const int64_t octets = values / 8, per = kThreads * kSets;
    int64_t b = (octets + per - 1) / per;
    b = b < kMaxBlocks ? b : kMaxBlocks;
    k_encode<<<(unsigned)b, kThreads, 0, s>>>(x, octets, q, scales);
    return hipGetLastError();
}

// x: bf16 rows (scales null) or e4m3 codes
hipError_t launch_rows(const void* x, const uint8_t* scales, const int32_t* inv_perm, const float* topk_w, int64_t Mc,
                       int K, int topk, uint16_t* out, int64_t out_rows, float* row_weights, int num_cus,
                       hipStream_t s) {
    int64_t bx = (Mc + kThreads / kWave - 1) / (kThreads / kWave);
    bx = bx < kMaxBlocks ? bx : kMaxBlocks;
    // a token's picks over several waves until there are 8 blocks per CU
    int64_t by = (8 * (int64_t)num_cus + bx - 1) / bx;
    by = by > topk ? topk : by;
    // Plain stores where the rows written fit the 256 MB behind the L2s, from
    // where the next product reads them, non-temporal ones past that.  2048
    // columns, top-8, bf16 and restored rows, us, calls back to back: 4096 tokens
    // plain 31 and 23, non-temporal 29 and 27; 16384 tokens 161 and 112, 106 and
    // 105 (bf16 rows after the backward pass's other kernels 126).
    const bool nt = (int64_t)K * 2 * Mc * topk > (int64_t)256 << 20;
    auto* k = scales ? (nt ? k_rows<true, true> : k_rows<true, false>) : (nt ? k_rows<false, true> : k_rows<false, false>);
    k<<<dim3((unsigned)bx, (unsigned)by), kThreads, 0, s>>>(x, scales, inv_perm, topk_w, Mc, K, topk, out, out_rows,
                                                            row_weights);
    return hipGetLastError();
}

hipError_t launch_topk_weights_bwd(const float* dots, int nd, int64_t rows, const int32_t* inv_perm, int64_t pairs,
                                   float* dweights, hipStream_t s) {
    int64_t b = (pairs + kThreads / 16 - 1) / (kThreads / 16);
    b = b < kMaxBlocks ? b : kMaxBlocks;
    k_dots<<<(unsigned)b, kThreads, 0, s>>>(dots, nd, rows, inv_perm, pairs, dweights);
    return hipGetLastError();
}

}  // namespace moe
