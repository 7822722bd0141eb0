// grad_clip.hip -- global gradient norm over many tensors, and clipping, for
// gfx950:
//
//   S = sum over tensors and elements of g^2,
//   c = min(1, max_norm / (sqrt(S) + 1e-6)),  out = g c.
//
// Squares and sums are fp64: the square of any fp32 value is exact enough
// there and neither overflows nor vanishes, and the kernel still runs at the
// rate of the reads.  No atomics: every block writes one partial sum, one
// block adds the partials in a fixed order, so equal calls give equal bits.
// The tensor list goes by value in the kernel arguments (a launch holds up to
// 128 tensors), so nothing is copied to the device and a captured graph keeps
// it.
//
// Bound by HBM.  604 M fp32 values (2.4 GB): the sum 383 us (6.3 TB/s read),
// the clip into other memory 850 us (5.7 TB/s read and written).  The sum's
// blocks walk 16 KB items and write one partial each (2048 at most); the clip
// has nothing to add up and takes an 8 KB item a block (16 KB items on 2048
// blocks: 897 us), from the list's end, which the sum has left in the
// memory-side cache (from the start: 1% more).  Short lists are bound by their
// launches (3.4 us of host each), so one of up to three items is summed by one
// block into its place (8100 fp32 values: 4.4 us against 6.7; eight items in
// one block take 11.5).
#include "moe_device.hpp"
#include "moe_internal.hpp"

namespace moe {
namespace {

constexpr int kThreads = 256;
constexpr int kVec = 16;                          // bytes per lane and load
constexpr int kSumChunk = 4 * kThreads * kVec;    // bytes of one work item
constexpr int kClipChunk = 2 * kThreads * kVec;
constexpr int kOneBlock = 3;                     // items that one block sums alone
constexpr int kClipBlocks = 65536;

struct List {
    const void* grad[kGradTensors];
    void* out[kGradTensors];
    int64_t numel[kGradTensors];
    int32_t first[kGradTensors + 1];   // work items before tensor i
    uint64_t f32[kGradTensors / 64];   // bit i: tensor i is fp32, else bf16
    int num;
};
static_assert(sizeof(List) <= 3840, "fits the 4 KB of kernel arguments");

// The work item's tensor (uniform over the block) and byte range, aligned
// down to 16 bytes in memory at both ends but the tensor's own.
struct Item {
    int i;
    int es;              // element size
    uintptr_t g, lo, hi; // tensor start, this item's bytes [lo, hi)
};

// The lane's part of `first`: a wave finds an item's tensor from it with two
// ballots, after one load's time instead of a chain of seven.
struct Firsts {
    int v[kGradTensors / kWave];
};

__device__ __forceinline__ Firsts firsts_of(const List& L) {
    Firsts f;
#pragma unroll
    for (int j = 0; j < kGradTensors / kWave; ++j) {
        const int i = j * kWave + (threadIdx.x & (kWave - 1));
        f.v[j] = i < L.num ? L.first[i] : INT32_MAX;
    }
    return f;
}

template <int CHUNK>
__device__ __forceinline__ Item item_of(const List& L, const Firsts& f, int64_t q) {
    int lo = -1;   // the last tensor with first[i] <= q
#pragma unroll
    for (int v : f.v) lo += __popcll(ballot(v <= q));
    Item it;
    it.i = lo;
    it.es = (L.f32[lo >> 6] >> (lo & 63)) & 1 ? 4 : 2;
    it.g = reinterpret_cast<uintptr_t>(L.grad[lo]);
    const uintptr_t end = it.g + (uintptr_t)L.numel[lo] * it.es;
    const uintptr_t base = (it.g & ~uintptr_t(kVec - 1)) + (uintptr_t)(q - L.first[lo]) * CHUNK;
    it.lo = base < it.g ? it.g : base;
    it.hi = base + CHUNK < end ? base + CHUNK : end;
    return it;
}

// sum of squares of the elements in a 16-byte vector
__device__ __forceinline__ double sq16(const uint4& v, bool f32) {
    const uint32_t u[4] = {v.x, v.y, v.z, v.w};
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (f32) {
            const double x = __uint_as_float(u[i]);
            s = __builtin_fma(x, x, s);
        } else {
            const double x = __uint_as_float(u[i] << 16), y = __uint_as_float(u[i] & 0xffff0000u);
            s = __builtin_fma(x, x, s);
            s = __builtin_fma(y, y, s);
        }
    }
    return s;
}

__device__ __forceinline__ float load_el(uintptr_t p, int es) {
    return es == 4 ? *reinterpret_cast<const float*>(p) : bf16_to_f32(*reinterpret_cast<const uint16_t*>(p));
}

__device__ __forceinline__ double block_sum(double v) {
    __shared__ double s_w[kThreads / kWave];
#pragma unroll
    for (int m = 32; m > 0; m >>= 1) v += __shfl_xor(v, m, kWave);
    if ((threadIdx.x & (kWave - 1)) == 0) s_w[threadIdx.x / kWave] = v;
    __syncthreads();
    double r = 0.0;
#pragma unroll
    for (int w = 0; w < kThreads / kWave; ++w) r += s_w[w];
    return r;
}

__global__ __launch_bounds__(kThreads) void k_sumsq(List L, double* __restrict__ partials) {
    double acc = 0.0;
    const Firsts firsts = firsts_of(L);
    for (int64_t q = blockIdx.x; q < L.first[L.num]; q += gridDim.x) {
        const Item it = item_of<kSumChunk>(L, firsts, q);
        const uintptr_t vlo = (it.lo + kVec - 1) & ~uintptr_t(kVec - 1), vhi = it.hi & ~uintptr_t(kVec - 1);
        for (uintptr_t p = vlo + threadIdx.x * kVec; p < vhi; p += kThreads * kVec)
            acc += sq16(*reinterpret_cast<const uint4*>(p), it.es == 4);
        // ragged ends of the tensor: at most 7 elements each (with no whole
        // vector between them the two meet at vlo or vhi)
        const uintptr_t head = vlo < it.hi ? vlo : it.hi, tail = vhi > head ? vhi : head;
        for (uintptr_t p = it.lo + threadIdx.x * it.es; p < head; p += kThreads * it.es) {
            const double x = load_el(p, it.es);
            acc = __builtin_fma(x, x, acc);
        }
        for (uintptr_t p = tail + threadIdx.x * it.es; p < it.hi; p += kThreads * it.es) {
            const double x = load_el(p, it.es);
            acc = __builtin_fma(x, x, acc);
        }
    }
    const double s = block_sum(acc);
    if (threadIdx.x == 0) partials[blockIdx.x] = s;
}

__global__ __launch_bounds__(kThreads) void k_sum_partials(const double* __restrict__ partials, int num,
                                                           double* __restrict__ sumsq) {
    double acc = 0.0;
    for (int i = threadIdx.x; i < num; i += kThreads) acc += partials[i];
    const double s = block_sum(acc);
    if (threadIdx.x == 0) sumsq[0] = s;
}

__global__ __launch_bounds__(kThreads) void k_clip(List L, const double* __restrict__ sumsq, float max_norm,
                                                   float* __restrict__ norm) {
    const Firsts firsts = firsts_of(L);
    // The norm of finite gradients may lie past the largest fp32 value and the
    // factor below the smallest normal one: the factor is fp64, and where it is
    // that small the products are, too.
    const double root = __builtin_sqrt(sumsq[0]);
    const float nrm = (float)root;
    if (norm != nullptr && blockIdx.x == 0 && threadIdx.x == 0) norm[0] = nrm;
    double c64 = 1.0;
    if (!(nrm + 1e-6f <= max_norm && nrm < HUGE_VALF)) {
        const double ratio = max_norm / (root + 1e-6);
        c64 = ratio >= 1.0 ? 1.0 : ratio;   // a NaN ratio stays NaN
    }
    const float c = (float)c64;
    const bool wide = c64 > 0.0 && c64 < 0x1p-126;
    for (int64_t q = blockIdx.x; q < L.first[L.num]; q += gridDim.x) {
        const Item it = item_of<kClipChunk>(L, firsts, L.first[L.num] - 1 - q);
        const uintptr_t o = reinterpret_cast<uintptr_t>(L.out[it.i]);
        if (o == it.g && c == 1.0f) continue;
        const bool f32 = it.es == 4;
        auto one = [&](uintptr_t p) {
            const float x = load_el(p, it.es);
            const float v = wide ? (float)(x * c64) : x * c;
            if (f32) *reinterpret_cast<float*>(o + (p - it.g)) = v;
            else *reinterpret_cast<uint16_t*>(o + (p - it.g)) = f32_to_bf16(v);
        };
        if (wide || ((o - it.g) & (kVec - 1)) != 0) {   // or the two are not aligned alike
            for (uintptr_t p = it.lo + threadIdx.x * it.es; p < it.hi; p += kThreads * it.es) one(p);
            continue;
        }
        const uintptr_t vlo = (it.lo + kVec - 1) & ~uintptr_t(kVec - 1), vhi = it.hi & ~uintptr_t(kVec - 1);
        for (uintptr_t p = vlo + threadIdx.x * kVec; p < vhi; p += kThreads * kVec) {
            uint4 v = *reinterpret_cast<const uint4*>(p);
            uint32_t u[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                u[i] = f32 ? __float_as_uint(__uint_as_float(u[i]) * c)
                           : f32x2_to_bf16x2(__uint_as_float(u[i] << 16) * c, __uint_as_float(u[i] & 0xffff0000u) * c);
            store_once16(reinterpret_cast<void*>(o + (p - it.g)), uint4{u[0], u[1], u[2], u[3]});
        }
        const uintptr_t head = vlo < it.hi ? vlo : it.hi, tail = vhi > head ? vhi : head;
        for (uintptr_t p = it.lo + threadIdx.x * it.es; p < head; p += kThreads * it.es) one(p);
        for (uintptr_t p = tail + threadIdx.x * it.es; p < it.hi; p += kThreads * it.es) one(p);
    }
}

// The next launch's tensors; returns its work items: a tensor's are the
// chunk-byte windows, from its 16-byte aligned-down start, that it touches.
int64_t fill(List& L, const moe_grad_tensor* t, int num, int chunk) {
    L.num = num;
    for (uint64_t& w : L.f32) w = 0;
    int64_t items = 0;
    for (int i = 0; i < num; ++i) {
        L.grad[i] = t[i].grad;
        L.out[i] = t[i].out;
        L.numel[i] = t[i].numel;
        L.first[i] = (int32_t)items;
        const bool f32 = t[i].dtype == MOE_DTYPE_F32;
        L.f32[i >> 6] |= (uint64_t)f32 << (i & 63);
        const int64_t bytes = t[i].numel * (f32 ? 4 : 2);
        const int64_t skew = (int64_t)(reinterpret_cast<uintptr_t>(t[i].grad) & (kVec - 1));
        if (bytes > 0) items += (skew + bytes + chunk - 1) / chunk;
    }
    L.first[num] = (int32_t)items;
    return items;
}

}  // namespace

hipError_t launch_grad_sumsq(const moe_grad_tensor* t, int num, double* sumsq, double* partials, hipStream_t s) {
    int np = 0;
    for (int i = 0; i < num; i += kGradTensors) {
        List L;
        const int64_t items = fill(L, t + i, num - i < kGradTensors ? num - i : kGradTensors, kSumChunk);
        if (num <= kGradTensors && items > 0 && items <= kOneBlock) {   // its partial sum is the sum
            k_sumsq<<<1, kThreads, 0, s>>>(L, sumsq);
            return hipGetLastError();
        }
        const int grid = (int)(items < kGradBlocks ? items : kGradBlocks);
        if (grid == 0) continue;
        k_sumsq<<<grid, kThreads, 0, s>>>(L, partials + np);
        np += grid;
    }
    k_sum_partials<<<1, kThreads, 0, s>>>(partials, np, sumsq);
    return hipGetLastError();
}

hipError_t launch_grad_clip(const moe_grad_tensor* t, int num, const double* sumsq, float max_norm, float* norm,
                            hipStream_t s) {
    for (int i = 0; i < num || i == 0; i += kGradTensors) {
        List L;
        const int64_t items = fill(L, t + i, num - i < kGradTensors ? num - i : kGradTensors, kClipChunk);
        const int grid = (int)(items < kClipBlocks ? (items > 0 ? items : 1) : kClipBlocks);
        k_clip<<<grid, kThreads, 0, s>>>(L, sumsq, max_norm, i == 0 ? norm : nullptr);
    }
    return hipGetLastError();
}

}  // namespace moe
