// gemm_bf16.hip -- grouped bf16 products over ragged expert segments for
// gfx950, with the gradients by the rows and by the weights:
//
//   forward  out[r,n] = sum_k a[r,k] w[e,n,k]           (contraction: k)
//   dgrad    dx[r,k]  = sum_n dy[r,n] w[e,n,k]          (contraction: n)
//   wgrad    dw[e,n,k] (+)= sum_{r of e} dy[r,n] a[r,k] (contraction: e's rows)
//
// fp32 sums, one rounding to bf16.
//
// Design:
//  * One kernel for the three: an output tile of BM x 256 per 512-thread
//    block (8 waves, 2 x 4, each 16*MI x 64 of it in 16x16x32 MFMAs), the
//    contraction in steps of 64.  An operand whose contraction index is
//    contiguous in memory (rows of a or dy; w in the forward) lies in LDS as
//    128-byte rows and is read 16 bytes a lane; one whose output index is
//    contiguous (w in dgrad, both in wgrad) lies as it is in memory, one
//    contraction index a row, and is transposed on the way to the registers
//    by ds_read_b64_tr_b16.  So no operand is ever transposed in memory.
//  * Operands move global -> LDS by buffer loads with LDS destination through
//    a ring of stages.  The buffer descriptor ends at the segment's (or the
//    matrix's) last byte, so everything past it, ragged rows and the tail of
//    the contraction included, arrives as zeros without a read: rows past a
//    segment never meet the sum, whatever they hold, and the per-lane
//    offsets are the same in every tile.
//  * The weight-side fragment is the MFMA's first operand, so a lane holds
//    four consecutive columns of one row; for bf16 two column blocks are
//    exchanged between neighbouring 16-lane rows (v_permlane16_swap) to 16
//    bytes a store.
//  * Persistent grid, tiles dealt to the XCDs in contiguous eighths of the
//    (expert, m-tile, n-tile) sequence, the operand stream running ahead
//    across tile boundaries.
#include "moe_device.hpp"
#include "moe_internal.hpp"

namespace moe {
namespace {

enum { kFwd = 0, kDgrad = 1, kWgrad = 2 };

constexpr int BN = 256;
constexpr int BK = 64;
constexpr int kThreads = 512;
constexpr int kWaves = kThreads / kWave;

typedef short v4s __attribute__((ext_vector_type(4)));
typedef short v8s __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;

// rows [lo, hi) of expert e, cut at the next segment and at cap_rows
__device__ __forceinline__ void segment(const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts,
                                        int64_t cap_rows, int e, int& lo, int& hi) {
    const int64_t next = offsets[e + 1];
    const int64_t end = next < 0 ? 0 : (next < cap_rows ? next : cap_rows);
    int64_t l = offsets[e];
    l = l < 0 ? 0 : (l > end ? end : l);
    const int64_t c = counts[e] < 0 ? 0 : counts[e];
    lo = (int)l;
    hi = (int)(l + c < end ? l + c : end);
}

template <int N>
__device__ __forceinline__ void wait_loads_barrier() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

// 16 bytes a lane from base + voff to LDS byte lds + 16 * lane; zeros where
// voff + 16 > bytes
__device__ __forceinline__ void dma16(const void* base, uint32_t bytes, uint32_t voff, uint32_t lds) {
    const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, (int)bytes, 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(uintptr_t)lds, 16, (int)voff, 0, 0, 0);
}

// ---- the two LDS layouts of an operand stage of W output indexes ------------
// Rows: 128 bytes for each output index, the 16-byte chunk c of row r at
// position c ^ (r mod 8) ^ (r / 8 mod 2): 16 lanes reading a chunk of 16 rows
// touch 16 distinct bank groups.
__device__ __forceinline__ int swz(int c, int r) { return c ^ (r & 7) ^ ((r >> 3) & 1); }
// Columns: 2 * W bytes for each contraction index k, the 32-byte slot s (16
// output indexes) at slot s ^ hx(k): the eight contraction rows that half a
// wave's transposing read touches lie in eight distinct slots.
__device__ __forceinline__ int hx(int k) { return (k & 3) | (((k >> 3) & 1) << 2); }

// The global byte offset that lane `lane` of the idx-th 1 KB of a stage
// fetches (ld: bytes between rows in memory).
template <bool T, int W>
__device__ __forceinline__ uint32_t dma_offset(int idx, int lane, int ld) {
    if constexpr (T) {
        constexpr int RB = 2 * W;
        const int byte = idx * 1024 + lane * 16;
        const int k = byte / RB, pos = (byte % RB) >> 4;
        return (uint32_t)(k * ld + ((((pos >> 1) ^ hx(k)) << 1) | (pos & 1)) * 16);
    } else {
        const int r = idx * 8 + (lane >> 3);
        return (uint32_t)(r * ld + swz(lane & 7, r) * 16);
    }
}

// A lane's fragment of 16 output indexes (o0 + 16 * b, b the block) by 32
// contraction indexes (half ks of the stage): base address for block 0 and
// half 0, then by xor and immediate offsets.
template <bool T, int W>
struct Frag {
    uint32_t base;
    __device__ __forceinline__ void init(int o0, int lane) {
        if constexpr (T) {
            const int k = 8 * (lane >> 4) + ((lane & 15) >> 2);
            base = (uint32_t)(k * 2 * W + (((o0 >> 4) ^ hx(k)) << 5) + (lane & 3) * 8);
        } else {
            const int r = o0 + (lane & 15);
            base = (uint32_t)(r * 128 + (swz(lane >> 4, r) << 4));
        }
    }
    __device__ __forceinline__ v8bf read(const uint8_t* stage, int b, int ks) const {
        if constexpr (T) {
            // (slot ^ hx) ^ b: o0 / 16 is a multiple of the block count, so xor adds b to the slot
            typedef __attribute__((address_space(3))) v4s* lp;
            const uint32_t at = (uint32_t)(uintptr_t)stage + (base ^ (uint32_t)(b << 5)) + ks * 32 * 2 * W;
            const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)at);
            const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lp)(uintptr_t)(at + 4 * 2 * W));
            return __builtin_bit_cast(v8bf, v8s{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w});
        } else {
            return *reinterpret_cast<const v8bf*>(stage + (base ^ (uint32_t)(ks << 6)) + b * 2048);
        }
    }
};

// One block's tiles t, t + nslots, ... of the (expert, m-tile, n-tile)
// sequence, walked without divisions; all fields are wave-uniform.
struct Cursor {
    int64_t t;
    int tm, tn, e, lo, hi;
    bool valid;
};

template <int MODE, int MI, bool F32>
__global__ __launch_bounds__(kThreads, 1) void k_gemm(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
                                                      const int32_t* __restrict__ offsets,
                                                      const int32_t* __restrict__ counts, int El, int64_t cap_rows,
                                                      int n_out, int k_in, int accumulate, void* __restrict__ out) {
    constexpr int BM = 32 * MI;
    constexpr bool AT = MODE == kWgrad, BT = MODE != kFwd;
    constexpr int kStageA = BM * BK * 2, kStage = kStageA + BN * BK * 2;
    constexpr int kStages = MI == 8 ? 2 : 3;
    constexpr int kADma = BM / 64, kBDma = 4;
    constexpr int kPer = kMaxLocalExperts / kThreads;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kStages * kStage];
    __shared__ int s_tpre[kMaxLocalExperts + 1];   // first m-tile of expert e
    __shared__ int s_lo[kMaxLocalExperts], s_hi[kMaxLocalExperts];
    __shared__ int s_wsum[kWaves];

    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int N = MODE == kFwd ? n_out : k_in;        // output columns
    const int ntm_w = (n_out + BM - 1) / BM;          // wgrad: m-tiles of an expert

    int nt[kPer], tsum = 0;
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = tid * kPer + j;
        nt[j] = 0;
        if (e < El) {
            int lo, hi;
            segment(offsets, counts, cap_rows, e, lo, hi);
            s_lo[e] = lo;
            s_hi[e] = hi;
            // an expert without rows has a gradient of zeros to write, or nothing to add
            nt[j] = MODE == kWgrad ? (accumulate && hi == lo ? 0 : ntm_w) : (hi - lo + BM - 1) / BM;
        }
        tsum += nt[j];
    }
    const int incl = wave_inclusive_scan(tsum);
    if (lane == kWave - 1) s_wsum[wave] = incl;
    __syncthreads();
    int run = incl - tsum;
    for (int w = 0; w < wave; ++w) run += s_wsum[w];
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const int e = tid * kPer + j;
        if (e < El) s_tpre[e] = run;
        run += nt[j];
    }
    if (tid == kThreads - 1) s_tpre[El] = run;
    __syncthreads();

    const int mtiles = __builtin_amdgcn_readfirstlane(s_tpre[El]);
    const int ntn = (N + BN - 1) / BN;
    const int xcd = blockIdx.x & 7, nslots = gridDim.x >> 3;
    const int64_t total = (int64_t)mtiles * ntn;
    const int64_t t_hi = total * (xcd + 1) / 8;
    const int step_q = nslots / ntn, step_r = nslots - step_q * ntn;

    auto fill = [&](Cursor& c) __attribute__((always_inline)) {
        c.lo = __builtin_amdgcn_readfirstlane(s_lo[c.e]);
        c.hi = __builtin_amdgcn_readfirstlane(s_hi[c.e]);
    };
    auto start = [&](Cursor& c) __attribute__((always_inline)) {
        c.t = total * xcd / 8 + (blockIdx.x >> 3);
        c.valid = c.t < t_hi;
        c.tm = c.tn = c.e = c.lo = c.hi = 0;
        if (!c.valid) return;
        c.tm = (int)(c.t / ntn);
        c.tn = (int)(c.t - (int64_t)c.tm * ntn);
        int lo = 0, hi = El - 1;   // the last expert with s_tpre[e] <= tm
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (s_tpre[mid] <= c.tm) lo = mid; else hi = mid - 1;
        }
        c.e = __builtin_amdgcn_readfirstlane(lo);
        fill(c);
    };
    auto next = [&](Cursor& c) __attribute__((always_inline)) {
        c.t += nslots;
        c.valid = c.t < t_hi;
        if (!c.valid) return;
        c.tn += step_r;
        c.tm += step_q;
        if (c.tn >= ntn) {
            c.tn -= ntn;
            ++c.tm;
        }
        bool moved = false;
        while (c.e + 1 < El && s_tpre[c.e + 1] <= c.tm) {
            ++c.e;
            moved = true;
        }
        c.e = __builtin_amdgcn_readfirstlane(c.e);
        if (moved) fill(c);
    };
    // first output row of a tile (a row of the buffer; wgrad: a weight row),
    // the end of its valid rows, and its contraction length
    auto m_first = [&](const Cursor& c) __attribute__((always_inline)) {
        const int m = (c.tm - __builtin_amdgcn_readfirstlane(s_tpre[c.e])) * BM;
        return MODE == kWgrad ? m : c.lo + m;
    };
    auto depth = [&](const Cursor& c) __attribute__((always_inline)) {
        return MODE == kFwd ? k_in : MODE == kDgrad ? n_out : c.hi - c.lo;
    };

    // ---- the operand stream --------------------------------------------------
    const int ldA = 2 * (MODE == kFwd ? k_in : n_out), ldB = 2 * k_in;   // bytes
    uint32_t voA[kADma], voB[kBDma];
    int cA[kADma], cB[kBDma];   // row layout: the 16-byte chunk, masked past the contraction's end
#pragma unroll
    for (int j = 0; j < kADma; ++j) {
        const int idx = wave * kADma + j;
        voA[j] = dma_offset<AT, BM>(idx, lane, ldA);
        cA[j] = swz(lane & 7, idx * 8 + (lane >> 3)) * 8;
    }
#pragma unroll
    for (int j = 0; j < kBDma; ++j) {
        const int idx = wave * kBDma + j;
        voB[j] = dma_offset<BT, BN>(idx, lane, ldB);
        cB[j] = swz(lane & 7, idx * 8 + (lane >> 3)) * 8;
    }
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    Cursor d;
    start(d);
    const uint8_t *dA = nullptr, *dB = nullptr;
    int d_left = 0, d_slot = 0;
    int d_mrows = 0, d_ncols = 0;   // output rows and columns from the tile's origin on
    int pending = 0;                // steps issued and not yet consumed
    auto d_tile = [&]() __attribute__((always_inline)) {
        const int m0 = m_first(d), n0 = d.tn * BN;
        d_left = depth(d);
        d_mrows = (MODE == kWgrad ? n_out : d.hi) - m0;
        d_ncols = N - n0;
        const uint8_t* A = reinterpret_cast<const uint8_t*>(a);
        const uint8_t* B = reinterpret_cast<const uint8_t*>(b);
        dA = MODE == kWgrad ? A + (int64_t)d.lo * ldA + m0 * 2 : A + (int64_t)m0 * ldA;
        dB = MODE == kFwd ? B + ((int64_t)d.e * n_out + n0) * ldB
           : MODE == kDgrad ? B + (int64_t)d.e * n_out * ldB + n0 * 2
                            : B + (int64_t)d.lo * ldB + n0 * 2;
    };
    if (d.valid) d_tile();
    auto issue = [&]() __attribute__((always_inline)) {
        const int kk = d_left < BK ? d_left : BK;
        // bytes from the base that belong to the operand; a row layout's rows
        // all lie inside it, a column layout's last row ends with its width
        const uint32_t bytesA = AT ? (kk > 0 ? (uint32_t)((kk - 1) * ldA + d_mrows * 2) : 0u)
                                   : (uint32_t)(((d_mrows < BM ? d_mrows : BM) - 1) * ldA + d_left * 2);
        const uint32_t bytesB = BT ? (kk > 0 ? (uint32_t)((kk - 1) * ldB + d_ncols * 2) : 0u)
                                   : (uint32_t)(((d_ncols < BN ? d_ncols : BN) - 1) * ldB + d_left * 2);
        const uint32_t at = lds0 + d_slot * kStage;
        const bool tail = d_left < BK;
#pragma unroll
        for (int j = 0; j < kADma; ++j) {
            uint32_t v = voA[j];
            if (!AT && tail) v |= cA[j] >= d_left ? 0x80000000u : 0u;   // past any descriptor: zeros
            dma16(dA, bytesA, v, at + (wave * kADma + j) * 1024);
        }
#pragma unroll
        for (int j = 0; j < kBDma; ++j) {
            uint32_t v = voB[j];
            if (!BT && tail) v |= cB[j] >= d_left ? 0x80000000u : 0u;
            dma16(dB, bytesB, v, at + kStageA + (wave * kBDma + j) * 1024);
        }
        dA += AT ? (int64_t)BK * ldA : BK * 2;
        dB += BT ? (int64_t)BK * ldB : BK * 2;
        d_left -= BK;
        d_slot = d_slot + 1 == kStages ? 0 : d_slot + 1;
        ++pending;
        if (d_left <= 0) {
            next(d);
            if (d.valid) d_tile();
        }
    };

    const int wm = wave >> 2, wn = wave & 3;
    Frag<AT, BM> fA;
    Frag<BT, BN> fB;
    fA.init(wm * 16 * MI, lane);
    fB.init(wn * 64, lane);

#pragma unroll
    for (int s = 0; s < kStages - 1; ++s)
        if (d.valid) issue();

    Cursor c;
    start(c);
    int slot = 0;
    while (c.valid) {
        const int m0 = m_first(c) + wm * 16 * MI;
        const int m_end = MODE == kWgrad ? n_out : c.hi;
        const int n0 = c.tn * BN + wn * 64;
        const bool mine = m0 < m_end && n0 < N;   // else nothing of this wave's part is stored
        v4f acc[MI][4];
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        int left = depth(c);
        do {
            if (kStages == 2 || pending < 2) wait_loads_barrier<0>();
            else wait_loads_barrier<kADma + kBDma>();
            if (d.valid) issue();
            --pending;
            if (mine) {
                const uint8_t* st = smem + slot * kStage;
#pragma unroll
                for (int ks = 0; ks < 2; ++ks) {
                    v8bf bf[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) bf[j] = fB.read(st + kStageA, j, ks);
#pragma unroll
                    for (int i = 0; i < MI; ++i) {
                        const v8bf af = fA.read(st, i, ks);
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[j], af, acc[i][j], 0, 0, 0);
                    }
                }
            }
            slot = slot + 1 == kStages ? 0 : slot + 1;
            left -= BK;
        } while (left > 0);

        if (mine) {
            const int g = lane >> 4;
            const int64_t row0 = MODE == kWgrad ? (int64_t)c.e * n_out + m0 : m0;
#pragma unroll
            for (int i = 0; i < MI; ++i) {
                const int r = 16 * i + (lane & 15);
                const bool ok = m0 + r < m_end;
                if constexpr (F32) {
                    float* o = static_cast<float*>(out) + (row0 + r) * N;
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const int col = n0 + 16 * j + 4 * g;
                        if (ok && col < N) {
                            v4f v = acc[i][j];
                            if (accumulate) v += *reinterpret_cast<const v4f*>(o + col);
                            *reinterpret_cast<v4f*>(o + col) = v;
                        }
                    }
                } else {
                    uint16_t* o = static_cast<uint16_t*>(out) + (row0 + r) * N;
#pragma unroll
                    for (int p = 0; p < 2; ++p) {
                        const v4f x = acc[i][2 * p], y = acc[i][2 * p + 1];
                        const auto w0 = __builtin_amdgcn_permlane16_swap(f32x2_to_bf16x2(x[0], x[1]),
                                                                         f32x2_to_bf16x2(y[0], y[1]), false, false);
                        const auto w1 = __builtin_amdgcn_permlane16_swap(f32x2_to_bf16x2(x[2], x[3]),
                                                                         f32x2_to_bf16x2(y[2], y[3]), false, false);
                        const int col = n0 + 32 * p + 16 * (g & 1) + 8 * (g >> 1);
                        if (ok && col < N) store_once16(o + col, uint4{w0[0], w1[0], w0[1], w1[1]});
                    }
                }
            }
        }
        next(c);
    }
}

template <int MODE, bool F32>
hipError_t launch(const uint16_t* a, const uint16_t* b, const int32_t* offsets, const int32_t* counts, int El,
                  int64_t cap_rows, int n_out, int k_in, int64_t rows_hint, int acc, void* out, int num_cus,
                  hipStream_t s) {
    const unsigned grid = (unsigned)((num_cus + 7) / 8 * 8);   // whole rounds over the eight XCDs
    auto go = [&](auto* kern) {
        kern<<<grid, kThreads, 0, s>>>(a, b, offsets, counts, El, cap_rows, n_out, k_in, acc, out);
    };
    if constexpr (MODE == kWgrad) {
        go(k_gemm<MODE, 8, F32>);
    } else {
        if (rows_hint >= (int64_t)104 * El) go(k_gemm<MODE, 8, F32>);
        else if (rows_hint >= (int64_t)48 * El) go(k_gemm<MODE, 4, F32>);
        else go(k_gemm<MODE, 2, F32>);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* w, const int32_t* offsets, const int32_t* counts,
                            int El, int64_t cap_rows, int n_out, int k_in, int64_t rows_hint, uint16_t* out,
                            int num_cus, hipStream_t s) {
    return launch<kFwd, false>(a, w, offsets, counts, El, cap_rows, n_out, k_in, rows_hint, 0, out, num_cus, s);
}
hipError_t launch_gemm_bf16_dgrad(const uint16_t* dy, const uint16_t* w, const int32_t* offsets,
                                  const int32_t* counts, int El, int64_t cap_rows, int n_out, int k_in,
                                  int64_t rows_hint, uint16_t* dx, int num_cus, hipStream_t s) {
    return launch<kDgrad, false>(dy, w, offsets, counts, El, cap_rows, n_out, k_in, rows_hint, 0, dx, num_cus, s);
}
hipError_t launch_gemm_bf16_wgrad(const uint16_t* dy, const uint16_t* a, const int32_t* offsets,
                                  const int32_t* counts, int El, int64_t cap_rows, int n_out, int k_in,
                                  int64_t rows_hint, bool f32, bool accumulate, void* dw, int num_cus, hipStream_t s) {
    if (f32)
        return launch<kWgrad, true>(dy, a, offsets, counts, El, cap_rows, n_out, k_in, rows_hint, accumulate, dw,
                                    num_cus, s);
    return launch<kWgrad, false>(dy, a, offsets, counts, El, cap_rows, n_out, k_in, rows_hint, 0, dw, num_cus, s);
}

}  // namespace moe
