// gemm_bf16.hip -- grouped bf16 products over ragged expert segments for
// gfx950, with the gradients by the rows and by the weights:
//
//   forward  out[r,n] = sum_k a[r,k] w[e,n,k]           (contraction: k)
//   dgrad    dx[r,k]  = sum_n dy[r,n] w[e,n,k]          (contraction: n)
//   wgrad    dw[e,n,k] (+)= sum_{r of e} dy[r,n] a[r,k] (contraction: e's rows)
//
// fp32 sums, one rounding to bf16.  Two kernels:
//
// k_tiles, for experts of more than a few rows.
//  * An output tile of 256 (or 128) x 256 per 512-thread block, one block per
//    CU, the contraction in steps of 64: eight waves, 2 x 4, each with 128
//    (64) x 64 of the tile in 16x16x32 MFMAs.
//  * Operands move global -> LDS by buffer loads with LDS destination, in
//    granules of 8 KB: 64 output indexes by 64 contraction indexes.  An
//    operand whose contraction index is contiguous in memory (rows of a or
//    dy; w in the forward) lies in its granules as 64 rows of 128 bytes and
//    is read 16 bytes a lane; one whose output index is contiguous (w in
//    dgrad, both in wgrad) lies as in memory, one contraction index a row,
//    and is transposed on its way to the registers by ds_read_b64_tr_b16.  So
//    nothing is ever transposed in memory, and both layouts read without
//    bank conflicts (counted: 6 to 19 cycles a block and launch, the same for
//    4096 and 16384 tokens: the tables at its start).
//  * The buffer descriptor of a granule ends with the last byte that belongs
//    to it, so ragged rows, the tail of the contraction and whole granules
//    past the tile arrive as zeros without a read; rows past a segment never
//    meet a sum, whatever they hold, and a lane's offsets are the same in
//    every tile.
//  * Two groups of four waves, one of each on every SIMD, run one phase
//    apart: while one group reads a step's fragments into registers (all of
//    them, 96 VGPRs) and issues loads, the other multiplies from its
//    registers; a barrier swaps the roles.  A granule is free as soon as its
//    readers have it in registers, long before they have multiplied it, so a
//    ring of 19 granules (152 KB, the LDS but for the tile tables) keeps up
//    to 104 KB in flight, most of it for three phases.  What was measured on
//    the way (16384 tokens, top-8, 128 experts, 1536 x 2048, forward): two
//    whole stages of 64 KB, all waves in step, 0.89 ms; loads alone 0.69 ms,
//    multiplies alone 0.64 ms.  The ring takes the loads alone to 0.45 ms,
//    the groups the multiplies alone to 0.55 ms and both together to 0.75 ms
//    (1100 TFLOP/s).  Past that the clock gives: at 64% of the MFMA rate it
//    is down to 1.5-1.8 GHz, and a step's fragment reads and loads take the
//    LDS as many cycles (98 KB out and 32 KB in a phase, 128 bytes a cycle)
//    as the phase's MFMAs take the matrix units.  dgrad runs at 1070, wgrad
//    at 910 (fp32 gradients; accumulating 770) and 1060 TFLOP/s (bf16).
//  * Not kept: four waves of 128 x 128 with fragments double-buffered (one
//    wave per SIMD; 0.96 ms), steps of 32 in four stages (0.96 ms, half-line
//    reads), a prefetch of later steps into L2 (slower by its own reads: the
//    loads are bound by their number), raised wave priority around the
//    multiplies (level), loads issued by the multiplying group as well (0.82
//    ms: its issue slots are what the MFMAs need), leaving out the multiplies
//    of a tile's row blocks past the last valid row (level: such tiles wait
//    for their weights), waits that count the stores in flight instead of
//    letting them drain (level), the last round's tiles in quarters where
//    those fill it (8 experts of 4096 x 4096: 3-9% faster; 128 experts, 8192
//    and more tokens: level to 3% slower), a weight gradient's finished tile
//    kept in registers and stored a row block a step (128-row tiles, 5-45%
//    slower: stores go fastest all at once).
//  * The weight-side fragment is the MFMA's first operand, so a lane holds
//    four consecutive columns of one row; for bf16 two column blocks are
//    exchanged between neighbouring 16-lane rows (v_permlane16_swap) to 16
//    bytes a store, through a descriptor that ends with the last valid row.
//  * Persistent grid; tiles dealt to the XCDs in contiguous eighths of the
//    (expert, n-tile, m-tile) sequence, m-tiles fastest: an expert's weights
//    are then read by tiles that run together (n-tiles fastest: forward 1-5%
//    and weight gradient 5% slower), and the operand stream runs ahead across
//    tile boundaries.
//
// k_few, for a few rows per expert (decoding), where the weights' bytes are
// the time and 256-column tiles would leave most CUs idle: 16 rows by 32 (64
// in dgrad) columns per four waves that split the contraction, each wave
// streaming its own share through its own three LDS stages without barriers,
// the four sums added in a fixed order.  One token, top-8, 1536 x 2048 (50 MB
// of weights): 11.9 us against 31 us on k_tiles.
#include <algorithm>
#include <cmath>

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
typedef unsigned v4u __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_ptr;
typedef __attribute__((address_space(3))) const v8bf* lds_v8;
typedef __attribute__((address_space(3))) v4s* lds_v4;

// rows [lo, hi) of an expert's segment, cut at the next one and at cap_rows
__device__ __forceinline__ void cut(int offset, int next_offset, int count, int64_t cap_rows, int& lo, int& hi) {
    const int64_t next = next_offset;
    const int64_t end = next < 0 ? 0 : (next < cap_rows ? next : cap_rows);
    int64_t l = offset;
    l = l < 0 ? 0 : (l > end ? end : l);
    const int64_t c = count < 0 ? 0 : count;
    lo = (int)l;
    hi = (int)(l + c < end ? l + c : end);
}
__device__ __forceinline__ void segment(const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts,
                                        int64_t cap_rows, int e, int& lo, int& hi) {
    cut(offsets[e], offsets[e + 1], counts[e], cap_rows, lo, hi);
}
// the segments of experts 2 t and 2 t + 1, no rows past El; loaded without
// conditions, so together
__device__ __forceinline__ void segments(const int32_t* __restrict__ offsets, const int32_t* __restrict__ counts,
                                         int64_t cap_rows, int El, int t, int (&lo)[2], int (&hi)[2]) {
    int off[3], num[2];
#pragma unroll
    for (int j = 0; j < 3; ++j) off[j] = offsets[min(2 * t + j, El)];
#pragma unroll
    for (int j = 0; j < 2; ++j) num[j] = counts[min(2 * t + j, El - 1)];
#pragma unroll
    for (int j = 0; j < 2; ++j) cut(off[j], off[j + 1], 2 * t + j < El ? num[j] : 0, cap_rows, lo[j], hi[j]);
}

// Exclusive prefix over the experts of nt (two consecutive experts a thread)
// into pre[0 .. El), and the total, both capped at `most`: disjoint segments
// never reach the cap, and overlapping ones (offsets out of order) cannot
// push a sum past it.  wsum: LDS scratch of kWaves values.  All 512 threads
// call it; it ends with a barrier.
__device__ __forceinline__ int expert_prefix(const int (&nt)[2], int El, int64_t most, int* pre, int64_t* wsum) {
    const int lane = threadIdx.x & (kWave - 1), wave = threadIdx.x / kWave;
    const int64_t sum = (int64_t)nt[0] + nt[1];
    const int64_t incl = wave_inclusive_scan(sum);
    if (lane == kWave - 1) wsum[wave] = incl;
    __syncthreads();
    int64_t run = incl - sum, total = 0;
    for (int w = 0; w < kWaves; ++w) {
        const int64_t v = wsum[w];
        if (w < wave) run += v;
        total += v;
    }
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        const int e = threadIdx.x * 2 + j;
        if (e < El) pre[e] = (int)(run < most ? run : most);
        run += nt[j];
    }
    __syncthreads();
    return __builtin_amdgcn_readfirstlane((int)(total < most ? total : most));
}

// 16 bytes a lane from base + voff to LDS byte lds + 16 * lane; zeros where
// they do not lie in the first `bytes` bytes
__device__ __forceinline__ void dma16(const void* base, int bytes, uint32_t voff, uint32_t lds) {
    const __amdgpu_buffer_rsrc_t r =
        __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), 0, max(bytes, 0), 0x00020000);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)(uintptr_t)lds, 16, (int)voff, 0, 0, 0);
}
constexpr int kNonTemporal = 2;              // the buffer instructions' cache bits
constexpr uint32_t kNowhere = 0x80000000u;   // an offset past every descriptor: zeros, or not stored

template <int N>
__device__ __forceinline__ void wait_loads() {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
__device__ __forceinline__ void barrier() { asm volatile("s_barrier" ::: "memory"); }
__device__ __forceinline__ void sched_fence() { __builtin_amdgcn_sched_barrier(0); }

// ---- LDS layouts -------------------------------------------------------------
// Row layout: 128 bytes for each output index, the 16-byte chunk c of row r at
// position c ^ (r mod 8) ^ (r / 8 mod 2).  A 128-bit LDS read serves sixteen
// lanes at a time, half of them from one 16-lane row of the wave and half
// from the next, so neighbouring lane rows read chunks two apart: lane row g
// takes chunk 2 g in the first half of a step and 2 g + 1 in the second.
__device__ __forceinline__ int swz(int c, int r) { return c ^ (r & 7) ^ ((r >> 3) & 1); }
// Column layout: 128 bytes (64 output indexes) for each contraction index k,
// the 32-byte slot s at slot s ^ fx(k): the eight contraction rows that half
// a wave's transposing read touches (k = 16 g + 0..3) lie in eight distinct
// slots of two adjacent rows.
__device__ __forceinline__ int fx(int k) { return ((k >> 1) & 1) | (((k >> 4) & 1) << 1); }

// 16 output indexes by 32 contraction indexes at LDS byte `at` (column
// layout): contraction rows k..k+3 and k+4..k+7 of the lane's row group.
// __restrict__ tells the compiler that what is read here is not what a load
// in flight writes (each granule has its own wait); without it, it waits for
// every load to LDS before the first transposing read of a step.
__device__ __forceinline__ v8bf read_columns(lds_v4 __restrict__ p) {
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16(p + 512 / sizeof(v4s));
    return __builtin_bit_cast(v8bf, v8s{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w});
}

// two 16-column blocks' sums, four consecutive columns a lane in each, as 16
// bytes of bf16: lane row g then holds columns 16 (g mod 2) + 8 (g / 2) .. + 7
__device__ __forceinline__ v4u pack_pair(const v4f& x, const v4f& y) {
    const auto w0 = __builtin_amdgcn_permlane16_swap(f32x2_to_bf16x2(x[0], x[1]), f32x2_to_bf16x2(y[0], y[1]), false, false);
    const auto w1 = __builtin_amdgcn_permlane16_swap(f32x2_to_bf16x2(x[2], x[3]), f32x2_to_bf16x2(y[2], y[3]), false, false);
    return v4u{w0[0], w1[0], w0[1], w1[1]};
}

// ---- k_tiles -----------------------------------------------------------------
constexpr int kGran = 8192;   // a granule
constexpr int kRing = 19;     // granules in the ring
constexpr int kTab = 2048;    // ints beside it: together the CU's 160 KB

// One block's tiles t, t + nslots, ... ; all fields are wave-uniform.
struct Cursor {
    int64_t t;
    int e;           // the place of the tile's expert in the walk
    int x, lo, hi;   // the expert and its rows
    int tm, tn;      // the tile's place among the expert's m-tiles and n-tiles
    bool valid;
};

// NA: granules of the row operand per wave group (the tile has 128 * NA rows).
// A step's granules are numbered p = 0 .. P - 1: group 0's NA of the row
// operand, four of the weight-side operand (one per wave column), group 1's
// NA.  Granule p of the block's step i lies in ring slot (P i + p) mod kRing.
//
// Phases.  In phase 2 i group 0 reads the fragments of step i (group 1
// multiplies step i - 1), in phase 2 i + 1 group 1 reads them (group 0
// multiplies).  Group 0's own NA granules are free after phase 2 i, the other
// NA + 4 after phase 2 i + 1, and each slot is refilled in the next phase, by
// the reading group: with R = kRing mod P, group 1 in its phases moves the
// granules R .. R + NA - 1 of each step, group 0 the others.  The waits count
// the loads that a wave has issued after the one needed; they are exact,
// because past the last tile the stream goes on with loads of zero bytes.
// F32: fp32 outputs; ACC: added to what is there.
template <int MODE, int NA, bool F32, bool ACC, bool TURN>   // TURN: forward only
__global__ __launch_bounds__(kThreads, 1) void k_tiles(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
                                                       const int32_t* __restrict__ offsets,
                                                       const int32_t* __restrict__ counts, int El, int64_t cap_rows,
                                                       int n_out, int k_in, void* __restrict__ out) {
    constexpr int MI = 4 * NA, BM = 128 * NA, NJ = 4;
    constexpr bool AT = MODE == kWgrad, BT = MODE != kFwd;   // column layout
    constexpr int P = 2 * NA + 4, R = kRing % P;
    constexpr int kAhead = (kRing - NA - 4) / P;   // the step that the first even phase goes on loading
    static_assert(R <= 4 && (kRing - NA - 4) % P == R + NA, "the phases' shares of a step");
    // loads (two a granule and wave) issued after the last one needed: group
    // 0 before even and odd phases, group 1 before even ones (its granules
    // are all needed there)
    constexpr int kEven0 = 2 * (NA + R + (kAhead - 1) * (NA + 4)), kOdd0 = 2 * (R + kAhead * (NA + 4));
    constexpr int kEven1 = 2 * kAhead * NA;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kRing * kGran];
    __shared__ int s_tab[kTab];

    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int grp = wave >> 2, wn = wave & 3;
    const int N = MODE == kFwd ? n_out : k_in;   // output columns

    // The experts in the order their tiles are walked, and, where they fit,
    // their rows.  Forward and dgrad: as they come, with the first m-tile of
    // each.  wgrad: every expert has the same tiles, whose time goes with the
    // expert's rows, so longest first, in classes of 256 rows (within a class
    // as they come: the writes of short experts, most of their time, lose 6%
    // in random order).
    const bool rows_in_lds = 3 * El <= kTab;
    int* s_at = s_tab;   // first m-tile of an expert (wgrad: the expert at a place)
    int* s_lo = s_tab + El;
    int* s_hi = s_lo + El;
    const int ntm_w = (n_out + BM - 1) / BM;   // wgrad: m-tiles of every expert
    int lo[2], hi[2], nt[2];
    segments(offsets, counts, cap_rows, El, tid, lo, hi);
#pragma unroll
    for (int j = 0; j < 2; ++j) nt[j] = (hi[j] - lo[j] + BM - 1) / BM;
    int mtiles;
    bool alike = true;
    if constexpr (MODE == kWgrad) {
        // an expert without rows has a gradient of zeros to write, or (class
        // 0) nothing to add
        auto class_of = [](int rows) __attribute__((always_inline)) { return rows > 0 ? (rows + 255) / 256 : ACC ? 0 : 1; };
        int lo0, hi0, mine[2];
        segment(offsets, counts, cap_rows, 0, lo0, hi0);
        const int class0 = class_of(hi0 - lo0);
#pragma unroll
        for (int j = 0; j < 2; ++j) mine[j] = tid * 2 + j < El ? class_of(hi[j] - lo[j]) : class0;
        int* s_same = reinterpret_cast<int*>(smem);   // of each wave: its experts are of class0
        const bool same = __all(mine[0] == class0 && mine[1] == class0);
        if (lane == 0) s_same[wave] = same && class0 > 0;
        __syncthreads();
        for (int w = 0; w < kWaves; ++w) alike = alike && s_same[w] != 0;
        int walked = El, at[2] = {tid * 2, tid * 2 + 1};
        if (!alike) {   // places by class
            int4* s_class = reinterpret_cast<int4*>(smem + 1024);   // El, then -1 up to a multiple of 4
            const int quads = (El + 3) / 4;
#pragma unroll
            for (int j = 0; j < 2; ++j)
                if (tid * 2 + j < quads * 4) reinterpret_cast<int*>(s_class)[tid * 2 + j] = tid * 2 + j < El ? mine[j] : -1;
            __syncthreads();
            walked = at[0] = at[1] = 0;
#pragma unroll 4
            for (int q = 0; q < quads; ++q) {
                const int4 c = s_class[q];
                const int other[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    walked += other[i] > 0;
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        at[j] += other[i] > mine[j] || (other[i] == mine[j] && q * 4 + i < tid * 2 + j);
                }
            }
            walked = __builtin_amdgcn_readfirstlane(walked);
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            if (tid * 2 + j >= El) continue;
            s_at[at[j]] = tid * 2 + j;
            if (rows_in_lds) {
                s_lo[at[j]] = lo[j];
                s_hi[at[j]] = hi[j];
            }
        }
        mtiles = ntm_w * walked;
        __syncthreads();   // the places are read, and the ring loaded, from here on
    } else {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int e = tid * 2 + j;
            if (rows_in_lds && e < El) {
                s_lo[e] = lo[j];
                s_hi[e] = hi[j];
            }
        }
        mtiles = expert_prefix(nt, El, cap_rows / BM + El, s_at, reinterpret_cast<int64_t*>(smem));
    }

    // Which tiles are this block's: those of an XCD lie side by side, so that
    // its blocks share operands in its L2.  Where tiles cost alike: the XCD's
    // eighth of the sequence.  Where they do not: of every round of gridDim.x
    // tiles the XCD's eighth, so that each has its share of the long ones
    // (4096 tokens on hot experts, 2048 x 768: 363 us in eighths, 165 dealt; 512
    // tokens, all short, 1536 x 2048, fp32: 253 and 263).
    const int ntn = (N + BN - 1) / BN;
    const int xcd = blockIdx.x & 7, nslots = gridDim.x >> 3;
    const int64_t total = (int64_t)mtiles * ntn;
    const int64_t t_lo = alike ? total * xcd / 8 : xcd * nslots;
    const int64_t t_hi = alike ? total * (xcd + 1) / 8 : total;
    const int t_step = alike ? nslots : (int)gridDim.x;

    auto place = [&](Cursor& c) __attribute__((always_inline)) {   // c.t lies in the expert at place c.e
        const int first = MODE == kWgrad ? c.e * ntm_w : __builtin_amdgcn_readfirstlane(s_at[c.e]);
        const int end = MODE == kWgrad ? first + ntm_w
                        : c.e + 1 < El ? __builtin_amdgcn_readfirstlane(s_at[c.e + 1]) : mtiles;
        const uint32_t mt = (uint32_t)(end - first);
        const uint32_t local = (uint32_t)(c.t - (int64_t)first * ntn);
        c.tn = (int)(local / mt);
        c.tm = (int)(local - (uint32_t)c.tn * mt);
        c.x = MODE == kWgrad ? __builtin_amdgcn_readfirstlane(s_at[c.e]) : c.e;
        int lo, hi;
        if (rows_in_lds) {
            lo = s_lo[c.e];
            hi = s_hi[c.e];
        } else {
            segment(offsets, counts, cap_rows, c.x, lo, hi);
        }
        c.lo = __builtin_amdgcn_readfirstlane(lo);
        c.hi = __builtin_amdgcn_readfirstlane(hi);
    };
    auto start = [&](Cursor& c) __attribute__((always_inline)) {
        c.t = t_lo + (blockIdx.x >> 3);
        c.valid = c.t < t_hi;
        c.tm = c.tn = c.e = c.x = c.lo = c.hi = 0;
        if (!c.valid) return;
        if constexpr (MODE == kWgrad) {
            c.e = (int)((uint32_t)c.t / (uint32_t)(ntm_w * ntn));
        } else {
            int lo = 0, hi = El - 1;   // the last expert whose first tile is not after t
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if ((int64_t)s_at[mid] * ntn <= c.t) lo = mid; else hi = mid - 1;
            }
            c.e = __builtin_amdgcn_readfirstlane(lo);
        }
        place(c);
    };
    auto next = [&](Cursor& c) __attribute__((always_inline)) {
        c.t += t_step;
        c.valid = c.t < t_hi;
        if (!c.valid) return;
        if constexpr (MODE == kWgrad) {
            c.e = (int)((uint32_t)c.t / (uint32_t)(ntm_w * ntn));   // at most 1024 * 512 * 256 tiles
        } else {
            while (c.e + 1 < El && (int64_t)s_at[c.e + 1] * ntn <= c.t) ++c.e;
            c.e = __builtin_amdgcn_readfirstlane(c.e);
        }
        place(c);
    };
    // a tile's first output row (a row of the buffer; wgrad: of the expert's
    // weights) and its contraction's length
    auto m_first = [&](const Cursor& c) __attribute__((always_inline)) {
        return MODE == kWgrad ? c.tm * BM : c.lo + c.tm * BM;
    };
    auto depth = [&](const Cursor& c) __attribute__((always_inline)) {
        return MODE == kFwd ? k_in : MODE == kDgrad ? n_out : c.hi - c.lo;
    };

    // ---- the operand stream -------------------------------------------------
    const int ldA = 2 * (MODE == kFwd ? k_in : n_out), ldB = 2 * k_in;   // bytes between rows in memory
    // A granule is eight kilobytes of eight rows; wave wn of a group moves
    // kilobytes 2 wn and 2 wn + 1, whose rows lie 8 * ld apart (and whose row
    // layout swaps neighbouring chunks).
    const int gr = wn * 16 + (lane >> 3);
    const int crow = swz(lane & 7, gr), ccol = ((((lane & 7) >> 1) ^ fx(gr)) << 1) | (lane & 1);
    const uint32_t voA = (uint32_t)(gr * ldA + (AT ? ccol : crow) * 16);
    const uint32_t voB = MODE == kFwd ? voA : (uint32_t)(gr * ldB + (BT ? ccol : crow) * 16);
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    Cursor d;
    start(d);
    if (!d.valid) return;   // no tile for this block
    const uint8_t *dA, *dB;   // the step's operands
    int d_left, tA, tB;       // contraction left; operand bytes that do not depend on the step
    // TURN: neighbouring tiles start a step apart and go round the
    // contraction.  In step they would all read the same 128 bytes of their
    // rows at a time, which for rows of 4 KB lie on a few of the memory's
    // channels.  Forward, 1536 x 2048, 128 experts, rows per expert and us in
    // step and turned: 16 150-182 and 139, 64 162-189 and 155, 187 227 and 191;
    // where the products bound, the turn only costs the rows' reuse: 256 272 and
    // 277, 1024 738 and 764.
    const int nsteps = (k_in + BK - 1) / BK;
    int d_cnt = 0;            // TURN: the tile's steps left
    int d_q = 0;              // ring slot of the step's granule 0
    const int gA = AT ? 128 : 64 * ldA, gB = BT ? 128 : 64 * ldB;   // bytes between granules in memory
    auto d_tile = [&]() __attribute__((always_inline)) {
        const int m0 = m_first(d), n0 = d.tn * BN;
        d_left = depth(d);
        const int mrows = min((MODE == kWgrad ? n_out : d.hi) - m0, BM), ncols = min(N - n0, BN);
        tA = AT ? mrows * 2 : (mrows - 1) * ldA;
        tB = BT ? ncols * 2 : (ncols - 1) * ldB;
        const uint8_t* A = reinterpret_cast<const uint8_t*>(a);
        const uint8_t* B = reinterpret_cast<const uint8_t*>(b);
        dA = MODE == kWgrad ? A + (int64_t)d.lo * ldA + m0 * 2 : A + (int64_t)m0 * ldA;
        dB = MODE == kFwd ? B + ((int64_t)d.x * n_out + n0) * ldB
           : MODE == kDgrad ? B + (int64_t)d.x * n_out * ldB + n0 * 2
                            : B + (int64_t)d.lo * ldB + n0 * 2;
        if constexpr (TURN) {
            d_cnt = nsteps;
            const int first = (int)((uint32_t)(d.e * ntn + d.tn) % (uint32_t)nsteps);
            dA += first * BK * 2;
            dB += first * BK * 2;
            d_left -= first * BK;
        }
    };
    d_tile();
    auto put = [&](int p) __attribute__((always_inline)) {   // granule p of the step
        const bool isA = p < NA || p >= NA + 4;
        const int g = p < NA ? p : isA ? p - 4 : p - NA;
        const bool T = isA ? AT : BT;
        const int ld = isA ? ldA : ldB, go = g * (isA ? gA : gB);
        // from the step's first byte to the last one that belongs to it
        const int bytes = T ? (min(d_left, BK) - 1) * ld + (isA ? tA : tB) : d_left * 2 + (isA ? tA : tB);
        const int q = d_q + p >= kRing ? d_q + p - kRing : d_q + p;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            uint32_t v = (isA ? voA : voB) + (T || h == 0 ? 0 : 16 - ((crow & 1) << 5));
            if (!T && d_left < BK)   // the contraction's tail: the chunks past it read as zeros
                v |= (crow ^ h) * 8 >= d_left ? kNowhere : 0u;
            const int at = go + h * 8 * ld;
            dma16((isA ? dA : dB) + at, bytes - at, v, lds0 + q * kGran + wn * 2048 + h * 1024);
        }
    };
    auto advance = [&]() __attribute__((always_inline)) {
        dA += AT ? (int64_t)BK * ldA : BK * 2;
        dB += BT ? (int64_t)BK * ldB : BK * 2;
        d_left -= BK;
        d_q = d_q + P >= kRing ? d_q + P - kRing : d_q + P;
        if (TURN && --d_cnt > 0) {
            if (d_left <= 0) {
                dA -= nsteps * BK * 2;
                dB -= nsteps * BK * 2;
                d_left = k_in;
            }
        } else if (TURN || d_left <= 0) {
            if (d.valid) next(d);
            if (d.valid) {
                d_tile();
            } else {   // past the last tile: zero bytes
                d_left = 0;
                d_cnt = 1;
                tA = tB = -(1 << 30);
            }
        }
    };
    auto even_puts = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int p = R + NA; p < P; ++p) put(p);
        advance();
#pragma unroll
        for (int p = 0; p < R; ++p) put(p);
    };
    auto odd_puts = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int p = R; p < R + NA; ++p) put(p);
        advance();
    };
    // A reading phase's loads: issued before its transposing reads, which are
    // many (a wave's 48 in wgrad, 32 with the rows' in dgrad), or after its
    // plain reads (24).  16384 tokens, 1536 x 2048: dgrad 765 us before, 782
    // after; wgrad fp32 881 and 978, bf16 765 and 852; forward 768 and 746.
    auto puts = [&]() __attribute__((always_inline)) {
        if (grp == 0) even_puts();
        else odd_puts();
    };
    // the ring but for what the first even phase loads
    if (grp == 0) {
#pragma unroll
        for (int q = 0; q < kRing - NA - 4; ++q) {
            if (q % P < R || q % P >= R + NA) put(q % P);
            if (q % P == P - 1) advance();
        }
    } else {
#pragma unroll
        for (int q = 0; q <= kAhead; ++q) odd_puts();
    }

    // ---- the compute side ---------------------------------------------------
    const int kc = 16 * (lane >> 4) + ((lane & 15) >> 2);   // column layout: the lane's contraction row
    const uint32_t col = (uint32_t)(kc * 128 + (fx(kc) << 5) + (lane & 3) * 8);
    const uint32_t row = (uint32_t)((lane & 15) * 128 + (swz(2 * (lane >> 4), lane & 15) << 4));
    const uint32_t rA = AT ? col : row, rB = BT ? col : row;   // the lane's byte in a granule
    int c_q = 0;   // ring slot of the step's granule 0
    auto granule = [&](int p) __attribute__((always_inline)) {
        return lds0 + (c_q + p >= kRing ? c_q + p - kRing : c_q + p) * kGran;
    };
    // block blk (16 output indexes) and half ks of a granule's contraction
    auto frag = [&](bool T, uint32_t at, int blk, int ks) __attribute__((always_inline)) {
        return T ? read_columns((lds_v4)(uintptr_t)((at ^ (uint32_t)(blk << 5)) + ks * 1024))
                 : *(lds_v8)(uintptr_t)((at ^ (uint32_t)(ks << 4)) + blk * 2048);
    };
    v4f acc[MI][NJ];
    auto load = [&](v8bf (&fa)[2][MI], v8bf (&fb)[2][NJ]) __attribute__((always_inline)) {
        const uint32_t bB = granule(NA + wn) + rB;
#pragma unroll
        for (int ks = 0; ks < 2; ++ks) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) fb[ks][j] = frag(BT, bB, j, ks);
#pragma unroll
            for (int g = 0; g < NA; ++g) {
                const uint32_t bA = granule((grp ? NA + 4 : 0) + g) + rA;
#pragma unroll
                for (int i = 0; i < 4; ++i) fa[ks][4 * g + i] = frag(AT, bA, i, ks);
            }
        }
    };
    auto multiply = [&](const v8bf (&fa)[2][MI], const v8bf (&fb)[2][NJ]) __attribute__((always_inline)) {
#pragma unroll
        for (int ks = 0; ks < 2; ++ks)
#pragma unroll
            for (int i = 0; i < MI; ++i)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[i][j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[ks][j], fa[ks][i], acc[i][j], 0, 0, 0);
    };
    // This wave's part of a tile.
    struct Part {
        int m0, m_end, n0, e;
        bool mine;   // any of it is valid
    } done = {0, 0, 0, 0, false};
    auto part_of = [&](const Cursor& c) __attribute__((always_inline)) {
        Part t;
        t.m0 = m_first(c) + grp * 64 * NA;
        t.m_end = MODE == kWgrad ? n_out : c.hi;
        t.n0 = c.tn * BN + wn * 64;
        t.e = c.x;
        t.mine = t.m0 < t.m_end && t.n0 < N;
        return t;
    };
    // Its outputs, `rows` rows at a time, each time through a descriptor that
    // ends with the last valid row; columns past the width go nowhere.
    constexpr int ES = F32 ? 4 : 2, kPieces = F32 ? NJ : NJ / 2, kCols = F32 ? 16 : 32;   // 64-byte pieces of a row
    const int g = lane >> 4, c0 = F32 ? 4 * g : 16 * (g & 1) + 8 * (g >> 1);
    struct Rows {
        uint8_t* o;
        int w, bytes;   // columns from n0 on, bytes to the end of the last valid row
    };
    auto rows_of = [&](const Part& t) __attribute__((always_inline)) {
        const int64_t row0 = MODE == kWgrad ? (int64_t)t.e * n_out + t.m0 : t.m0;
        Rows x;
        x.o = static_cast<uint8_t*>(out) + (row0 * N + t.n0) * ES;
        x.w = N - t.n0;
        x.bytes = ((min(t.m_end - t.m0, 16 * MI) - 1) * N + x.w) * ES;
        return x;
    };
    auto from_row = [&](const Rows& x, int r) __attribute__((always_inline)) {
        return __builtin_amdgcn_make_buffer_rsrc(x.o + (int64_t)r * N * ES, 0, max(x.bytes - r * N * ES, 0), 0x00020000);
    };
    // A gradient's bytes are most of a short batch's time.  There (kLines) the
    // lanes eight apart trade halves of two neighbouring pieces, so that a
    // store writes eight rows of whole 128-byte lines instead of sixteen of
    // half lines (512 tokens, 1536 x 2048: fp32 gradients 437 -> 253 us, bf16
    // 224 -> 148; forward and dgrad are level or 2% slower with it), and
    // non-temporal where the rows are whole lines (4096 tokens on hot experts,
    // 2048 x 768, bf16: 150 us, plainly 202).  Where they are not, a piece's
    // two half-filled lines have to meet their other halves in L2: plain
    // stores (725 tokens, 704 x 1256: fp32 208 -> 107 us, bf16 104 -> 43).
    // The rows' products are written once and read soon: plainly in the
    // forward (16384 tokens, 736 against 746 us non-temporal; 60 experts of
    // 408 x 336, 31 against 37), non-temporal in dgrad (4096 tokens on hot
    // experts 150 against 155 us, widths of half lines 3% slower).
    const bool whole = ((reinterpret_cast<uintptr_t>(out) | (uintptr_t)(N * ES)) & 127) == 0;
    auto put16 = [&](const v4u& v, const __amdgpu_buffer_rsrc_t& r, uint32_t at) __attribute__((always_inline)) {
        if (MODE == kDgrad || (MODE == kWgrad && whole))
            __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, kNonTemporal);
        else
            __builtin_amdgcn_raw_buffer_store_b128(v, r, at, 0, 0);
    };
    // ACC adds what is there to the finished sums, one rounding at its magnitude
    // (starting the sums at it would round at it every 32 rows).  It is read
    // in the stores' own pieces, kOld row blocks ahead of its use: the step's
    // fragments are dead here and leave the registers.  Bound by its bytes, 8 an
    // element (4096 tokens, 1536 x 2048: 606 us, 5.7 TB/s; one, two and four
    // blocks ahead: 627, 620, 606), non-temporal as the stores are (read
    // plainly 678; 725 tokens, 704 x 1256, whose rows are not whole lines: 204,
    // non-temporal 233).
    constexpr int kOld = 4;
    auto get16 = [&](const __amdgpu_buffer_rsrc_t& r, uint32_t at) __attribute__((always_inline)) {
        return __builtin_bit_cast(v4f, whole ? __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kNonTemporal)
                                             : __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, 0));
    };
    auto store = [&]() __attribute__((always_inline)) {
        if (!done.mine) return;
        constexpr bool kLines = MODE == kWgrad;
        static_assert(!ACC || (kLines && F32), "accumulating: fp32 weight gradients");
        const Rows x = rows_of(done);
        const bool up = kLines && (lane & 8);
        const int c1 = c0 + (up ? kCols : 0);
        const uint32_t v = (uint32_t)(((lane & (kLines ? 7 : 15)) * N + c1) * ES);
        auto at = [&](int p) __attribute__((always_inline)) { return c1 + kCols * p < x.w ? v + kCols * ES * p : kNowhere; };
        v4f old[ACC ? MI : 1][ACC ? kPieces : 1];
        auto fetch = [&](int i) __attribute__((always_inline)) {
#pragma unroll
            for (int p = 0; p < kPieces; p += 2)
#pragma unroll
                for (int h = 0; h < 2; ++h) old[i][p + h] = get16(from_row(x, 16 * i + 8 * h), at(p));
        };
        if constexpr (ACC) {
#pragma unroll
            for (int i = 0; i < kOld; ++i) fetch(i);
        }
#pragma unroll
        for (int i = 0; i < MI; ++i) {
            if constexpr (ACC)
                if (i + kOld < MI) fetch(i + kOld);
#pragma unroll
            for (int p = 0; p < kPieces; p += 2) {
                v4u lo, hi;
                if constexpr (F32) {
                    lo = __builtin_bit_cast(v4u, acc[i][p]);
                    hi = __builtin_bit_cast(v4u, acc[i][p + 1]);
                } else {
                    lo = pack_pair(acc[i][2 * p], acc[i][2 * p + 1]);
                    hi = pack_pair(acc[i][2 * p + 2], acc[i][2 * p + 3]);
                }
                if constexpr (kLines) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        const uint32_t got = __builtin_amdgcn_update_dpp(0u, up ? lo[q] : hi[q], 0x128, 0xf, 0xf, false);   // row_ror:8
                        lo[q] = up ? got : lo[q];
                        hi[q] = up ? hi[q] : got;
                    }
                    if constexpr (ACC) {
                        lo = __builtin_bit_cast(v4u, __builtin_bit_cast(v4f, lo) + old[i][p]);
                        hi = __builtin_bit_cast(v4u, __builtin_bit_cast(v4f, hi) + old[i][p + 1]);
                    }
                    put16(lo, from_row(x, 16 * i), at(p));
                    put16(hi, from_row(x, 16 * i + 8), at(p));
                } else {
                    put16(lo, from_row(x, 16 * i), at(p));
                    put16(hi, from_row(x, 16 * i), at(p + 1));
                }
            }
            sched_fence();
        }
    };
    auto begin = [&]() __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < MI; ++i)
#pragma unroll
            for (int j = 0; j < NJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    };

    // Before a group's reading phase, and before its multiplying phase: the
    // loads whose data the coming phase reads, whoever reads it, then the
    // barrier that publishes every wave's.
    auto to_read = [&]() __attribute__((always_inline)) {
        sched_fence();
        if (grp == 0) wait_loads<kEven0>();
        else wait_loads<63>();   // nothing of group 1's: LDS reads only
        barrier();
        sched_fence();
    };
    auto to_multiply = [&]() __attribute__((always_inline)) {
        sched_fence();
        if (grp == 0) wait_loads<kOdd0>();
        else wait_loads<kEven1>();
        barrier();
        sched_fence();
    };
    Cursor c;
    start(c);
    bool have = false;             // a finished tile's sums are in registers
    if (grp != 0) to_multiply();   // group 1 runs one phase behind
    while (c.valid) {
        const Part t = part_of(c);
        int left = depth(c);
        bool first = true;
        do {   // an expert without rows: one step, of zeros
            to_read();
            if (BT) puts();
            sched_fence();
            if (first) {
                if (have) store();
                sched_fence();
                done = t;
                begin();
                first = false;
                have = true;
            }
            v8bf fa[2][MI], fb[2][NJ];   // the step's fragments: dead between steps, where the stores need registers
            // (ACC: read whether they are used or not; else what the last step
            // left would pass for them, and the registers are taken in store())
            if (ACC || t.mine) load(fa, fb);
            if (!BT) puts();
            c_q = c_q + P >= kRing ? c_q + P - kRing : c_q + P;
            to_multiply();
            if (t.mine) multiply(fa, fb);
            left -= BK;
        } while (left > 0);
        next(c);
    }
    if (grp == 0) to_read();   // as many barriers as group 1
    if (have) store();
    wait_loads<0>();   // no load may still write this block's LDS when it ends
}

// ---- k_few -------------------------------------------------------------------
constexpr int kFewStages = 3;

// A unit: 16 rows of an expert by NC columns.  A block works on two units at a
// time, four waves each; wave kw of a unit takes its steps kw, kw + 4, ...
// (KS of the contraction each: 4 KB of weights and the rows' part).  MODE:
// forward (row layouts, 32 columns) or dgrad (weights in column layout, 64
// columns, so that a step still reads whole 128-byte lines).
template <int MODE>
__global__ __launch_bounds__(kThreads, 1) void k_few(const uint16_t* __restrict__ a, const uint16_t* __restrict__ b,
                                                     const int32_t* __restrict__ offsets,
                                                     const int32_t* __restrict__ counts, int El, int64_t cap_rows,
                                                     int n_out, int k_in, uint16_t* __restrict__ out) {
    static_assert(MODE == kFwd || MODE == kDgrad, "the contraction is not the ragged axis");
    constexpr bool BT = MODE == kDgrad;
    constexpr int NC = BT ? 64 : 32, KS = BT ? 32 : 64;
    constexpr int NJ = NC / 16, KK = KS / 32;
    constexpr int kW = 4096, kStep = kW + 16 * KS * 2;        // a stage: weights, rows
    constexpr int kADma = 16 * KS * 2 / 1024, kDma = 4 + kADma;   // loads a step
    __shared__ __attribute__((aligned(1024))) uint8_t smem[kWaves * kFewStages * kStep];
    __shared__ __attribute__((aligned(16))) float s_red[2][3][16 * NC];
    __shared__ int s_tpre[kMaxLocalExperts];   // first 16-row tile of each expert
    const int tid = threadIdx.x;
    const int lane = tid & (kWave - 1);
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int uw = wave >> 2, kw = wave & 3;
    const int N = MODE == kFwd ? n_out : k_in, C = MODE == kFwd ? k_in : n_out;
    int lo2[2], hi2[2], nt[2];
    segments(offsets, counts, cap_rows, El, tid, lo2, hi2);
#pragma unroll
    for (int j = 0; j < 2; ++j) nt[j] = (hi2[j] - lo2[j] + 15) / 16;
    const int tiles = expert_prefix(nt, El, cap_rows / 16 + El, s_tpre, reinterpret_cast<int64_t*>(smem));
    const int ncu = (N + NC - 1) / NC;
    const int64_t units = (int64_t)tiles * ncu;
    const int64_t first = 2 * (int64_t)blockIdx.x, stride = 2 * (int64_t)gridDim.x;
    if (first >= units) return;
    const int S = (C + KS - 1) / KS;
    const int steps = (S - kw + 3) / 4;   // this wave's steps of every unit; may be none

    struct Unit {
        int e, m0, rows, n0;   // rows 0: past the last unit
    };
    auto unit_of = [&](int64_t u) __attribute__((always_inline)) {
        Unit x = {0, 0, 0, 0};
        if (u >= units) return x;
        const int t = (int)(u / ncu);
        x.n0 = (int)(u - (int64_t)t * ncu) * NC;
        int at = 0;   // experts whose first tile is not after t
        for (int j = 0; j < El; j += kWave)
            at += __popcll(ballot(j + lane < El && s_tpre[min(j + lane, El - 1)] <= t));
        x.e = __builtin_amdgcn_readfirstlane(at - 1);
        int lo, hi;
        segment(offsets, counts, cap_rows, x.e, lo, hi);
        x.m0 = __builtin_amdgcn_readfirstlane(lo + 16 * (t - s_tpre[x.e]));
        x.rows = min(16, __builtin_amdgcn_readfirstlane(hi) - x.m0);
        return x;
    };

    // the operand stream of this wave: weights in kilobytes of eight rows
    // (columns of the output, or contraction indexes), then the rows
    const int ldA = 2 * C, ldB = 2 * k_in;
    const int rw = lane >> 3;
    const int cB = BT ? ((((lane & 7) >> 1) ^ ((rw >> 1) & 1)) << 1) | (lane & 1) : swz(lane & 7, rw);
    const uint32_t voB = (uint32_t)(rw * ldB + cB * 16);
    const int ra = BT ? lane >> 2 : lane >> 3;
    const int cA = BT ? (lane & 3) ^ ((ra >> 2) & 3) : swz(lane & 7, ra);
    const uint32_t voA = (uint32_t)(ra * ldA + cA * 16);
    const uint32_t ring = (uint32_t)(uintptr_t)smem + wave * kFewStages * kStep;
    int64_t d_u = first + uw;
    Unit d = unit_of(d_u);
    int d_j = 0, d_slot = 0;
    auto issue = [&]() __attribute__((always_inline)) {
        const int k0 = (kw + 4 * d_j) * KS, left = d.rows > 0 ? C - k0 : 0;
        const uint32_t at = ring + d_slot * kStep;
        const uint8_t* W = reinterpret_cast<const uint8_t*>(b) + (int64_t)d.e * n_out * ldB +
                           (BT ? (int64_t)k0 * ldB + d.n0 * 2 : (int64_t)d.n0 * ldB + k0 * 2);
        const int wb = left <= 0 ? 0 : BT ? (min(left, KS) - 1) * ldB + (N - d.n0) * 2
                                          : (min(N - d.n0, NC) - 1) * ldB + left * 2;
#pragma unroll
        for (int h = 0; h < 4; ++h) {
            // the next eight rows swap neighbouring chunks (row layout) or pairs of slots (column layout)
            uint32_t v = voB + ((h & 1) == 0 ? 0 : BT ? 64 - ((cB & 4) << 5) : 16 - ((cB & 1) << 5));
            if (!BT && left < KS) v |= (cB ^ (h & 1)) * 8 >= left ? kNowhere : 0u;
            dma16(W + h * 8 * ldB, wb - h * 8 * ldB, v, at + h * 1024);
        }
        const uint8_t* A = reinterpret_cast<const uint8_t*>(a) + (int64_t)d.m0 * ldA + k0 * 2;
        const int ab = left <= 0 ? 0 : (d.rows - 1) * ldA + left * 2;
#pragma unroll
        for (int h = 0; h < kADma; ++h) {
            uint32_t v = voA + (h == 0 ? 0 : 16 - ((cA & 1) << 5));
            if (left < KS) v |= (cA ^ h) * 8 >= left ? kNowhere : 0u;
            dma16(A + h * 8 * ldA, ab - h * 8 * ldA, v, at + kW + h * 1024);
        }
        d_slot = d_slot + 1 == kFewStages ? 0 : d_slot + 1;
        if (++d_j >= steps) {
            d_j = 0;
            d_u += stride;
            d = unit_of(d_u);
        }
    };
    if (steps > 0) {
#pragma unroll
        for (int s = 0; s < kFewStages; ++s) issue();
    }

    const int g = lane >> 4;
    const int kc = 8 * g + ((lane & 15) >> 2);   // column layout: the lane's contraction row
    const uint32_t rB = BT ? (uint32_t)(kc * 128 + ((((kc >> 1) & 1) | ((kc >> 3) & 1) << 1) << 5) + (lane & 3) * 8)
                           : (uint32_t)((lane & 15) * 128 + (swz(2 * g, lane & 15) << 4));
    const uint32_t rA = BT ? (uint32_t)((lane & 15) * 64 + ((g ^ (((lane & 15) >> 2) & 3)) << 4))
                           : (uint32_t)((lane & 15) * 128 + (swz(2 * g, lane & 15) << 4));
    int slot = 0;
    for (int64_t u = first + uw; u - uw < units; u += stride) {
        v4f acc[NJ];
#pragma unroll
        for (int j = 0; j < NJ; ++j) acc[j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
        for (int s = 0; s < steps; ++s) {
            sched_fence();
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(kDma * (kFewStages - 1)) : "memory");   // this step's loads
            sched_fence();
            const uint32_t at = ring + slot * kStep;
            v8bf fa[KK], fb[KK][NJ];
#pragma unroll
            for (int ks = 0; ks < KK; ++ks) {
                fa[ks] = *(lds_v8)(uintptr_t)(at + kW + (rA ^ (uint32_t)(ks << 4)));
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    fb[ks][j] = BT ? read_columns((lds_v4)(uintptr_t)(at + (rB ^ (uint32_t)(j << 5))))
                                   : *(lds_v8)(uintptr_t)(at + (rB ^ (uint32_t)(ks << 4)) + j * 2048);
            }
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // the stage is in registers: refill it
            sched_fence();
            issue();
#pragma unroll
            for (int ks = 0; ks < KK; ++ks)
#pragma unroll
                for (int j = 0; j < NJ; ++j)
                    acc[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[ks][j], fa[ks], acc[j], 0, 0, 0);
            slot = slot + 1 == kFewStages ? 0 : slot + 1;
        }
        if (kw > 0) {
#pragma unroll
            for (int j = 0; j < NJ; ++j) *reinterpret_cast<v4f*>(&s_red[uw][kw - 1][(j * kWave + lane) * 4]) = acc[j];
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
        if (kw == 0) {
            const Unit x = unit_of(u);
#pragma unroll
            for (int j = 0; j < NJ; ++j)
#pragma unroll
                for (int w = 0; w < 3; ++w)
                    acc[j] += *reinterpret_cast<const v4f*>(&s_red[uw][w][(j * kWave + lane) * 4]);
            const int w = N - x.n0;   // columns from n0 on
            const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
                out + (int64_t)x.m0 * N + x.n0, 0, x.rows > 0 ? ((x.rows - 1) * N + w) * 2 : 0, 0x00020000);
#pragma unroll
            for (int p = 0; p < NJ / 2; ++p) {
                const int c = 32 * p + 16 * (g & 1) + 8 * (g >> 1);
                const uint32_t v = c < w ? (uint32_t)(((lane & 15) * N + c) * 2) : kNowhere;
                __builtin_amdgcn_raw_buffer_store_b128(pack_pair(acc[2 * p], acc[2 * p + 1]), r, v, 0, 0);
            }
        }
        asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");   // s_red may be written again
    }
    wait_loads<0>();   // no load may still write this block's LDS when it ends
}

// Which kernel.  Where there are many weights their bytes bound both alike;
// what tells the kernels apart is how well their units of work fill the CUs
// and how long one takes.  The rule compares estimates of that in
// microseconds, for rows_hint rows spread evenly and a part of a tile more an
// expert for raggedness; the constants are fitted to 538 measured calls (1 to
// 131072 rows, 4 to 128 experts, widths of 128 to 4096, even and skewed
// routing; those under 8 us were fitted as 8), in which the choice is 1.2%
// slower than the best of the three on average (by rows per expert alone 9%),
// over 20% slower in 15 and 52% at worst (four experts of 2048 x 1024 or 60 to
// 128 narrow ones, where a part of a round decides; 30 experts of 1232 x 1056
// under skew 36%, as the rows are taken to lie evenly).  Measured (k_few, 128
// rows, 256 rows; r rows per expert):
//   128 experts, 1536 x 2048, forward   r 4  138 139 142   r 16 158 143 144
//                                       r 96 480 160 162   r 128 616 211 177
//                             dgrad     r 4  149 142 141   r 16 171 145 140
//                                       r 96 465 155 168   r 128 608 215 171
//   8 experts, 4096 x 4096, forward     r 8   52  70  83   r 32  67  61  79   r 250 351 144 94
//   8 experts, 1504 x 488, forward      r 1    6  12  15
//   8 experts, 624 x 176, dgrad         r 139  7  14  18
//   16 experts, 352 x 200, forward      r 275 17  11  13
//   4 experts, 376 x 1360, forward      r 41   9  24  31
//   32 experts, 1792 x 1376, forward    r 106 113 57  71
// The gradient by the weights has whole matrices as output tiles, whatever the
// rows (it reads no hint); 256-row ones where they save more than two fifths
// of the rounds (290 calls: 1.2% slower than the better on average, 24% at
// worst, always 256 rows 11%; 16 experts of 352 x 200, 4404 rows: 42 us with
// 128 rows, 59 with 256; 128 of 264 x 360, 16384 rows: 63 and 86; 128 of
// 1536 x 2048, 32768 rows, bf16: 340 and 288).
// Forward tiles turn (TURN) up to 208 rows per expert, 128-row ones always.
template <int MODE, bool F32, bool ACC>
hipError_t launch(const uint16_t* a, const uint16_t* b, const int32_t* offsets, const int32_t* counts, int El,
                  int64_t cap_rows, int n_out, int k_in, int64_t rows_hint, void* out, int num_cus, hipStream_t s) {
    const unsigned grid = (unsigned)((num_cus + 7) / 8 * 8);   // the same number of blocks on each of the eight XCDs
    auto tiles = [&](auto* kernel) {
        kernel<<<grid, kThreads, 0, s>>>(a, b, offsets, counts, El, cap_rows, n_out, k_in, out);
    };
    const double cus = num_cus;
    const int ntn = ((MODE == kFwd ? n_out : k_in) + BN - 1) / BN;   // n-tiles
    if constexpr (MODE == kWgrad) {
        const double rounds1 = std::ceil((double)El * ((n_out + 127) / 128) * ntn / cus);
        const double rounds2 = std::ceil((double)El * ((n_out + 255) / 256) * ntn / cus);
        if (3 * rounds1 <= 5 * rounds2) tiles(k_tiles<MODE, 1, F32, ACC, false>);
        else tiles(k_tiles<MODE, 2, F32, ACC, false>);
    } else {
        constexpr int NC = MODE == kDgrad ? 64 : 32, KS = MODE == kDgrad ? 32 : 64;   // k_few's columns and step
        const int N = MODE == kFwd ? n_out : k_in, C = MODE == kFwd ? k_in : n_out;
        const double experts = rows_hint < El ? (double)rows_hint : El, r = (double)rows_hint / experts;
        const double bytes = experts * N * C * 2 / 5.5e6;   // the weights' time
        const double units = experts * std::max(1.0, r / 16 + 0.75) * ((N + NC - 1) / NC) / (2 * cus);
        const double few = 3.5 + std::max(1.0, units) *
                                     (1.5 + (MODE == kDgrad ? 1.2 : 0.85) * ((C + 4 * KS - 1) / (4 * KS)));
        // rounds of tiles; 128 rows unless 256 save more than a fifth of them
        const double rounds1 = experts * std::max(1.0, r / 128 + 0.5) * ntn / cus;
        const double rounds2 = experts * std::max(1.0, r / 256 + 0.5) * ntn / cus;
        const bool low = 4 * std::ceil(rounds1) <= 5 * std::ceil(rounds2);
        const double walk = 6.5 + std::max(1.0, low ? rounds1 : rounds2) *
                                      (1.7 + (low ? 0.8 : 1.1) * ((C + BK - 1) / BK));
        if (std::max(few, bytes) <= std::max(walk, bytes + 1))
            k_few<MODE><<<grid, kThreads, 0, s>>>(a, b, offsets, counts, El, cap_rows, n_out, k_in,
                                                  static_cast<uint16_t*>(out));
        else if (low) tiles(k_tiles<MODE, 1, F32, ACC, MODE == kFwd>);
        else if (MODE == kFwd && rows_hint < (int64_t)208 * El) tiles(k_tiles<MODE, 2, F32, ACC, MODE == kFwd>);
        else tiles(k_tiles<MODE, 2, F32, ACC, false>);
    }
    return hipGetLastError();
}

}  // namespace

hipError_t launch_gemm_bf16(const uint16_t* a, const uint16_t* w, const int32_t* offsets, const int32_t* counts,
                            int El, int64_t cap_rows, int n_out, int k_in, int64_t rows_hint, uint16_t* out,
                            int num_cus, hipStream_t s) {
    return launch<kFwd, false, false>(a, w, offsets, counts, El, cap_rows, n_out, k_in, rows_hint, out, num_cus, s);
}
hipError_t launch_gemm_bf16_dgrad(const uint16_t* dy, const uint16_t* w, const int32_t* offsets,
                                  const int32_t* counts, int El, int64_t cap_rows, int n_out, int k_in,
                                  int64_t rows_hint, uint16_t* dx, int num_cus, hipStream_t s) {
    return launch<kDgrad, false, false>(dy, w, offsets, counts, El, cap_rows, n_out, k_in, rows_hint, dx, num_cus, s);
}
hipError_t launch_gemm_bf16_wgrad(const uint16_t* dy, const uint16_t* a, const int32_t* offsets,
                                  const int32_t* counts, int El, int64_t cap_rows, int n_out, int k_in,
                                  bool f32, bool accumulate, void* dw, int num_cus, hipStream_t s) {
    auto* go = !f32 ? launch<kWgrad, false, false> : accumulate ? launch<kWgrad, true, true> : launch<kWgrad, true, false>;
    return go(dy, a, offsets, counts, El, cap_rows, n_out, k_in, /*rows_hint=*/0, dw, num_cus, s);
}

}  // namespace moe
