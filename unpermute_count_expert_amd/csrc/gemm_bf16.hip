// gemm_bf16.hip -- grouped bf16 products over ragged expert segments for
// gfx950, with the gradients by the rows and by the weights:
//
//   forward  out[r,n] = sum_k a[r,k] w[e,n,k]          (contraction: k)
//   dgrad    dx[r,k]  = sum_n dy[r,n] w[e,n,k]         (contraction: n)
//   wgrad    dw[e,n,k] (+)= sum_{r of e} dy[r,n] a[r,k] (contraction: e's rows)
//
// fp32 sums, one rounding to bf16.
#include "moe_device.hpp"
#include "moe_internal.hpp"

namespace moe {
namespace {

enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };

// rows [lo, hi) of expert e, cut at the next segment and at cap_rows
__device__ __forceinline__ void segment(const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts,
                                        int64_t cap_rows, int e, int64_t& lo, int64_t& hi) {
    const int64_t next = offsets[e + 1];
    const int64_t end = next < 0 ? 0 : (next < cap_rows ? next : cap_rows);
    lo = offsets[e];
    lo = lo < 0 ? 0 : (lo > end ? end : lo);
    const int64_t c = counts[e] < 0 ? 0 : counts[e];
    hi = lo + c < end ? lo + c : end;
}

// One 64x64 output tile per 256-thread block, both operands staged in LDS
// with the contraction index innermost, 4x4 outputs per thread.
template <int MODE>
__global__ __launch_bounds__(256) void k_tile64(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
                                                const int32_t* __restrict__ offsets,
                                                const int32_t* __restrict__ counts, int64_t cap_rows, int n_out,
                                                int k_in, int f32, int accumulate, void* __restrict__ out) {
    constexpr int T = 64, D = 16;
    __shared__ float sA[T][D + 1], sB[T][D + 1];
    const int e = blockIdx.z;
    int64_t lo, hi;
    segment(offsets, counts, cap_rows, e, lo, hi);
    const int64_t rows = hi - lo;
    const int64_t M = MODE == kWgrad ? n_out : rows;
    const int N = MODE == kFwd ? n_out : k_in;
    const int64_t C = MODE == kFwd ? k_in : MODE == kDgrad ? n_out : rows;
    const uint16_t* we = MODE == kWgrad ? b + lo * k_in : b + (int64_t)e * n_out * k_in;
    const uint16_t* ae = a + lo * (MODE == kFwd ? k_in : n_out);
    const int n0 = blockIdx.x * T;
    const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
    for (int64_t m0 = (int64_t)blockIdx.y * T; m0 < M; m0 += (int64_t)gridDim.y * T) {
        float acc[4][4] = {};
        for (int64_t c0 = 0; c0 < C; c0 += D) {
            for (int i = threadIdx.x; i < T * D; i += 256) {
                // the index that is contiguous in memory runs fastest over the lanes
                const int ia = MODE == kWgrad ? i % T : i / D, ca = MODE == kWgrad ? i / T : i % D;
                const int ib = MODE == kFwd ? i / D : i % T, cb = MODE == kFwd ? i % D : i / T;
                const int64_t m = m0 + ia, n = n0 + ib;
                float va = 0.0f, vb = 0.0f;
                if (m < M && c0 + ca < C)
                    va = bf16_to_f32(MODE == kWgrad ? ae[(c0 + ca) * n_out + m] : ae[m * C + c0 + ca]);
                if (n < N && c0 + cb < C)
                    vb = bf16_to_f32(MODE == kFwd ? we[n * k_in + c0 + cb] : we[(c0 + cb) * k_in + n]);
                sA[ia][ca] = va;
                sB[ib][cb] = vb;
            }
            __syncthreads();
            for (int d = 0; d < D; ++d)
#pragma unroll
                for (int i = 0; i < 4; ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j) acc[i][j] = __builtin_fmaf(sA[ty + 16 * i][d], sB[tx + 16 * j][d], acc[i][j]);
            __syncthreads();
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int64_t m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
                if (m >= M || n >= N) continue;
                const int64_t at = (MODE == kWgrad ? (int64_t)e * n_out + m : lo + m) * N + n;
                if (f32) {
                    float* o = static_cast<float*>(out) + at;
                    *o = accumulate ? *o + acc[i][j] : acc[i][j];
                } else {
                    static_cast<uint16_t*>(out)[at] = f32_to_bf16(acc[i][j]);
                }
            }
    }
}

template <int MODE>
hipError_t launch(const uint16_t* a, const uint16_t* b, const int32_t* offsets, const int32_t* counts, int El,
                  int64_t cap_rows, int n_out, int k_in, bool f32, bool acc, void* out, hipStream_t s) {
    const int N = MODE == kFwd ? n_out : k_in;
    const int64_t M = MODE == kWgrad ? n_out : cap_rows / El + 64;
    int64_t gy = (M + 63) / 64;
    gy = gy > 65535 ? 65535 : gy;
    k_tile64<MODE><<<dim3((N + 63) / 64, (unsigned)gy, El), 256, 0, s>>>(a, b, offsets, counts, cap_rows, n_out, k_in,
                                                                       f32, acc, out);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* w, const int32_t* offsets, const int32_t* counts,
                            int El, int64_t cap_rows, int n_out, int k_in, int64_t rows_hint, uint16_t* out,
                            int num_cus, hipStream_t s) {
    return launch<kFwd>(a, w, offsets, counts, El, cap_rows, n_out, k_in, false, false, out, s);
}
hipError_t launch_gemm_bf16_dgrad(const uint16_t* dy, const uint16_t* w, const int32_t* offsets,
                                  const int32_t* counts, int El, int64_t cap_rows, int n_out, int k_in,
                                  int64_t rows_hint, uint16_t* dx, int num_cus, hipStream_t s) {
    return launch<kDgrad>(dy, w, offsets, counts, El, cap_rows, n_out, k_in, false, false, dx, s);
}
hipError_t launch_gemm_bf16_wgrad(const uint16_t* dy, const uint16_t* a, const int32_t* offsets,
                                  const int32_t* counts, int El, int64_t cap_rows, int n_out, int k_in,
                                  int64_t rows_hint, bool f32, bool accumulate, void* dw, int num_cus, hipStream_t s) {
    return launch<kWgrad>(dy, a, offsets, counts, El, cap_rows, n_out, k_in, f32, accumulate, dw, s);
}

}  // namespace moe
