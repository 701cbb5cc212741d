// Per-tensor-scaled FP8 GEMM with fused bias and bf16 output, on the sm_100a
// 5th-generation tensor cores (tcgen05, kind::f8f6f4).
//
// Method: AstrAI commit logs -- astrai/extension/fp8.py @f4c44ebf (bias added
// in fp32 before the single bf16 rounding; 3-D operands with stride-0
// broadcast; bf16-only output), tests/extension/test_fp8_mma.py @cebdd45d
// (bias_scale slot: bf16 bias when null, dequantized fp8 bias otherwise) and
// csrc/kernels/fp8/gemm.cuh @5e76fbd1 (the NT / NN / TN operand layouts of a
// linear layer's forward, dX and dW).
//
// Design (B200-first; the pages' sm_89 mma.sync / ldmatrix / cp.async / PRMT
// kernel is prior art only):
//  * persistent CTAs (one per SM at most), each walking output tiles
//    BM x BN = 128 x {64,128,256}, or 256 x 256 on an SM pair (tcgen05
//    cta_group::2, clusters of two, no TMA multicast), in groups of M-tile
//    rows walked M-fastest, so that the tiles running together share their
//    A and B panels in L2;
//  * 6 warps with fixed roles: warp 0 issues TMA loads (one lane), warp 1
//    owns TMEM and issues tcgen05.mma (one lane), warps 2-5 run the epilogue
//    (one per TMEM lane quarter);
//  * operands arrive by TMA in 128-byte-swizzled shared-memory stages of
//    BK = 128 bytes of K, in their stored orientation: K-major for A in
//    NT/NN and B in NT, MN-major for A in TN and B in NN/TN (the tensor core
//    reads MN-major 8-bit operands directly, so dX / dW need no transposed
//    copies). TMA zero-fills every M, N, K tail and batch end;
//  * each stage is 4 MMAs of 128 x BN x 32 accumulating in TMEM (fp32);
//    tcgen05.commit releases the stage back to the producer;
//  * two TMEM accumulators (2 x BN columns): the epilogue of tile i overlaps
//    the main loop of tile i+1;
//  * epilogue: tcgen05.ld 32 columns at a time, y = acc * (1/sa)(1/sb) +
//    bias in fp32 (one fma), one round-to-nearest-even to bf16, staged as
//    128 x 32 tiles in shared memory and written by one TMA store each (TMA
//    clips the M / N tails);
//  * short problems (M <= 32, NT and NN) swap the operands, C^T = B^T A^T,
//    so that C's few rows become an MMA N of 16 or 32;
//  * split K: a tile's k-blocks are shared by several CTAs, whose fp32
//    partials go through a caller workspace (the last CTA to finish adds
//    them), through the library's static scratch, or, for short problems
//    without a workspace, to split 0 of a cluster through distributed shared
//    memory; partials are always added in split order;
//  * grouped launches: up to 4 problems (a linear's dX and dW) share one
//    persistent grid, each work unit looking up its problem in a table;
//  * every mbarrier wait is bounded by a time limit; a wait that gives up
//    records FP8_ERR_DEVICE_TIMEOUT in the library's device error word and the
//    CTA stops issuing work and exits through the normal teardown.

#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include <cuda_fp16.h>

#include <algorithm>
#include <mutex>

#include "act.cuh"
#include "common.cuh"
#include "sm100.cuh"

namespace fp8lite {
namespace {

using namespace sm100;

// Set by a bounded wait that gave up. Each source file that instantiates a
// kernel of this header has its own word; fp8_last_device_error reads them all.
__device__ uint32_t g_device_error = 0;

constexpr int BM = 128;
constexpr int BK = 128;  // bytes = elements of K per stage
constexpr int kEpiThreads = 128;            // 4 epilogue warps, one per TMEM lane quarter
constexpr int kThreads = 64 + kEpiThreads;  // producer warp, MMA warp, epilogue
// An activation epilogue on unswapped tiles runs sixteen warps (at 96
// registers a thread: the file serves a block in steps of four warps, 20 here).
__host__ __device__ constexpr int epi_threads(bool ep, bool swap) { return ep && !swap ? 4 * kEpiThreads : kEpiThreads; }
constexpr int kActRegs = 96;
constexpr uint64_t kWaitLimitNs = 2000000000ull;  // 2 s per wait

struct GemmParams {
    int M, N, K;
    int m_tiles, n_tiles, k_blocks, total_tiles;
    int group_m;  // tiles are walked in groups of this many M-tile rows
    int a_bcast, b_bcast;
    uint32_t idesc;
    const float* sa;
    const float* sb;
    const void* bias;
    const float* bias_scale;
    int bias_kind;  // 0 none, 1 bf16, 2 fp8
    int bias_fmt;
    uint16_t* out;
    int64_t stride_c;
    int vec_store;  // 16-byte stores allowed (N, stride_c multiples of 8, base aligned)
    int tma_store;  // tiles leave through shared memory and TMA stores (same conditions)
    // split K: every tile is `split` work units of up to kb_per k-blocks each
    int split, kb_per, total_units;
    // swapped short problems: the splits of a tile run as one cluster and the
    // others' fp32 partials reach split 0 through its shared memory (no workspace)
    int csplit;
    float* ws;         // fp32 partial slots: [tile][rank][split] x (128 x BN)
    uint32_t* ws_cnt;  // per (tile, rank): {units arrived, partials written}
    // FP8 output (fp8_mm_out8): format, delayed-scaling ring, the scale used, the amax
    int out_fmt;
    fp8_ring* out_ring;
    float* out_scale;
    float* out_amax;
};

// Grouped launch (fp8_mm_grouped): several independent problems share one
// persistent grid. Work units [unit_end of the previous entry, unit_end) are
// the tiles of entry i; each role looks its unit's entry up here. An entry is
// a problem, or a column range of one: the host may give a problem's last
// columns their own entry with 128-wide tiles, so that the tiles of the
// grid's last round are cheaper.
constexpr int kMaxGroup = FP8_MM_MAX_GROUP;
constexpr int kMaxEntries = kMaxGroup + 1;
struct GroupProblem {
    CUtensorMap ta, tb, tc;  // operand maps and the output's store map
    int M, N, k_blocks, m_tiles, n_tiles, unit_end;
    int a_mn, b_mn;
    uint32_t idesc;
    int bias_kind, bias_fmt, tma_store, vec_store;
    int bn, n_base;  // this entry's tile width (128 or the launch's BN) and first output column
    const float* sa;
    const float* sb;
    const void* bias;
    const float* bias_scale;
    uint16_t* out;
};
template <bool GROUP>
struct GroupTab {};  // single-problem launches carry no table
template <>
struct GroupTab<true> {
    GroupProblem q[kMaxEntries];
    int count;
};

// Activation epilogue (fp8_mm_act, fp8_mm_act_out8): the activation, the bf16
// residual added after it, and where z (the activation's input) is kept.
template <bool EP>
struct EpArgs {};  // other launches carry none of it
template <>
struct EpArgs<true> {
    CUtensorMap tz;            // store map of preact (fast launches)
    int act;
    int fast;                  // whole tiles: every pointer, stride and N aligned for 16-byte accesses
    const uint16_t* residual;  // may be the output itself
    int64_t stride_r;
    uint16_t* preact;          // laid out as the output
};

// The i-th work unit of a CTA whose first unit is unit0, the persistent grid
// holding unit_step CTAs (pairs). A grouped launch walks its rounds in
// alternating directions: CTA c takes unit c of the first round, unit
// step-1-c of the second, and so on. Its units come longest K first, so the
// CTAs that drew the short tiles of one round take the first units of the
// next, and no CTA stacks a second tile on a long one while others idle.
template <bool GROUP>
__device__ __forceinline__ int unit_of(int i, int unit0, int unit_step) {
    return i * unit_step + ((GROUP && (i & 1)) ? unit_step - 1 - unit0 : unit0);
}

// The problem that work unit u of a grouped launch belongs to, and the
// unit's tile index within it.
__device__ __forceinline__ const GroupProblem& group_problem(const GroupTab<true>& g, int u, int& t) {
    int i = 0;
    while (i + 1 < g.count && u >= g.q[i].unit_end) ++i;
    t = i == 0 ? u : u - g.q[i - 1].unit_end;
    return g.q[i];
}

// Wait for phase `parity` of the mbarrier at `bar`, giving up after
// `limit_ns`: then the library's device error word is set and false returned.
__device__ __forceinline__ bool wait_bounded_cluster(uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait_cluster(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait_cluster(bar, parity)) return true;
        if ((i & 1023u) == 0 && globaltimer_ns() - t0 > limit_ns) {
            atomicOr(&g_device_error, 1u);
            return false;
        }
    }
}

__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, uint64_t limit_ns = kWaitLimitNs) {
    if (mbar_try_wait(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        if (mbar_try_wait(bar, parity)) return true;
        if ((i & 1023u) == 0 && globaltimer_ns() - t0 > limit_ns) {
            atomicOr(&g_device_error, 1u);
            return false;
        }
    }
}

// wait_bounded by every lane of a warp, with one verdict for all of them.
__device__ __forceinline__ bool wait_bounded_warp(uint32_t bar, uint32_t parity) {
    return __all_sync(0xffffffffu, wait_bounded(bar, parity));
}

// True in one lane of the (fully active) warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "elect.sync _|p, 0xffffffff;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint32_t ld_acquire_u32(const uint32_t* ptr) {
    uint32_t v;
    asm volatile("ld.acquire.gpu.global.u32 %0, [%1];" : "=r"(v) : "l"(ptr) : "memory");
    return v;
}

__device__ __forceinline__ void red_release_add(uint32_t* ptr, uint32_t v) {
    asm volatile("red.release.gpu.global.add.u32 [%0], %1;" ::"l"(ptr), "r"(v) : "memory");
}

// Wait until the counter at `ptr` reaches `want`, giving up (device error
// word set, false returned) after `limit_ns`.
__device__ __forceinline__ bool wait_count(const uint32_t* ptr, uint32_t want, uint64_t limit_ns = kWaitLimitNs) {
    if (ld_acquire_u32(ptr) >= want) return true;
    const uint64_t t0 = globaltimer_ns();
    for (uint32_t i = 1;; ++i) {
        __nanosleep(32);
        if (ld_acquire_u32(ptr) >= want) return true;
        if ((i & 255u) == 0 && globaltimer_ns() - t0 > limit_ns) {
            atomicOr(&g_device_error, 1u);
            return false;
        }
    }
}

// One FP8 code -> fp32 (exact: every E4M3 / E5M2 value is an fp16 value).
__device__ __forceinline__ float fp8_to_f32(uint8_t c, int fmt) {
    uint32_t h;
    const uint16_t in = c;
    if (fmt == FP8_E4M3) {
        asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(in));
    } else {
        asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(h) : "h"(in));
    }
    return __half2float(__ushort_as_half(uint16_t(h & 0xFFFFu)));
}

// Two fp32 values to a pair of FP8 codes (nearest-even, saturating), the
// first in the low byte.
__device__ __forceinline__ uint32_t cvt_fp8x2(int fmt, float lo, float hi) {
    uint16_t r;
    if (fmt == FP8_E4M3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else                 asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint32_t pack_bf16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
    uint16_t h;
    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
    return h;
}

__device__ __forceinline__ float bf16_value(uint16_t h) { return __uint_as_float(uint32_t(h) << 16); }

// Shared-memory plan of one CTA. CTAS = 2: an MMA pair, each CTA holding its
// 128 rows of A and BN/2 columns of B per stage.
// STG: staging tiles of the epilogue.
template <int BN, int STAGES, int CTAS, int STG = 3>
struct Smem {
    static constexpr int kABytes = BM * BK;
    static constexpr int kBBytes = (BN / CTAS) * BK;
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStageTx = CTAS * kStageBytes;  // bytes landing on the leader's full barrier
    // three 128-row x 32-column bf16 staging tiles (64-byte swizzle), used in
    // turn, so that a chunk waits only for the store two chunks back; 24 KB
    // in all, so that a waiting kernel's small blocks still fit on the SM
    // beside this CTA. An activation epilogue takes four: 2 KB for each of its
    // sixteen warps
    static constexpr int kStgBufs = STG;
    static constexpr int kStgPending = 1;  // stores that may still be reading their tile when one more is issued
    static_assert(STG >= 3, "");
    static constexpr int kStgBytes = BM * 32 * 2;
    static constexpr int kStgOffset = STAGES * kStageBytes;  // a multiple of 1024
    static constexpr int kBiasOffset = kStgOffset + kStgBufs * kStgBytes;  // BN fp32 bias values
    static constexpr bool kAct = STG == 4;  // an activation epilogue: 32 bias values for each of its warps
    static constexpr int kBarOffset = kBiasOffset + (kAct ? 2048 : BN * 4);
    // full[S], empty[S], tmem_full[2], tmem_empty[2], then the TMEM slot and the split ticket
    static constexpr int kBytes = kBarOffset + (2 * STAGES + 4) * 8 + 16;
    // room to align the base to 1024. The base is declared so; an activation
    // epilogue has no full KB left for one that is not, and gives up then
    static constexpr int kAlloc = kAct ? 227 * 1024 : kBytes + 1024;
    static constexpr uint32_t kTmemCols = 2 * BN < 32 ? 32 : 2 * BN;
    static_assert(kStgOffset % 1024 == 0, "staging tiles need 1024-byte alignment");
    static_assert(kAlloc <= 227 * 1024 && kBytes <= kAlloc, "shared memory per CTA");
};

// Whether a CTA's plan fits its shared memory from the aligned base on (for
// every thread of the grid alike). If not, the device error word is set.
template <typename L>
__device__ __forceinline__ bool smem_fits(const uint8_t* raw, const uint8_t* base) {
    if (base - raw + L::kBytes <= L::kAlloc) return true;
    atomicOr(&g_device_error, 1u);
    return false;
}

// The tile walk's scalars, read once into registers.
struct TileWalk {
    int m_tiles, n_tiles, group_m;
};

// Tile order: batch outermost; inside a batch, groups of `group_m` M-tile
// rows, walked M-fastest within the group, then N. A wave of concurrently
// running tiles then covers a compact block of rows and columns whose A and B
// panels stay resident in L2 (an M-fastest walk over all rows streams the
// whole A through L2 every wave).
__device__ __forceinline__ void tile_coords(int t, const TileWalk& w, int& mb, int& nb, int& b) {
    const int per_batch = w.m_tiles * w.n_tiles;
    b = t / per_batch;
    const int r = t - b * per_batch;
    const int per_group = w.group_m * w.n_tiles;
    const int g = r / per_group;
    const int first_m = g * w.group_m;
    const int rows = min(w.group_m, w.m_tiles - first_m);
    const int i = r - g * per_group;
    mb = first_m + i % rows;
    nb = i / rows;
}

// The same without the divisions that a small problem does not need.
__device__ __forceinline__ void tile_coords_lazy(int t, const TileWalk& w, int& mb, int& nb, int& b) {
    b = 0;
    const int per_batch = w.m_tiles * w.n_tiles;
    if (t >= per_batch) {
        b = t / per_batch;
        t -= b * per_batch;
    }
    int first_m = 0;
    const int per_group = w.group_m * w.n_tiles;
    if (t >= per_group) {
        const int g = t / per_group;
        first_m = g * w.group_m;
        t -= g * per_group;
    }
    const int rows = min(w.group_m, w.m_tiles - first_m);
    nb = t / rows;
    mb = first_m + t - nb * rows;
}

// Keeps a value's computation (a kernel-parameter read) at this point of the
// program: the first read of each parameter is a slow constant-cache miss, so
// the kernel issues them all together while its set-up runs.
template <typename T>
__device__ __forceinline__ T pin(T v) {
    asm volatile("" : "+r"(v));
    return v;
}

// Named barrier 1: the epilogue warps.
template <int T = kEpiThreads>
__device__ __forceinline__ void epilogue_bar() {
    asm volatile("bar.sync 1, %0;" ::"n"(T) : "memory");
}

// Barrier 1, returning whether any epilogue thread passed true.
template <int T = kEpiThreads>
__device__ __forceinline__ bool epilogue_bar_or(bool v) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred q, p;\n\t"
        "setp.ne.u32 q, %1, 0;\n\t"
        "bar.red.or.pred p, 1, %2, q;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r)
        : "r"(uint32_t(v)), "n"(T)
        : "memory");
    return r != 0;
}

// One 128 x 32 bf16 block of the epilogue: to the staging tile whose last
// store is known to have read it (64-byte swizzle: 16-byte piece j of row r at
// (j ^ (r / 2 mod 4)) * 16, so the 8 lanes of a store phase hit distinct
// banks), then one TMA store by the lead thread, which clips the M / N tails
// of the output. n_st counts the stores issued so far (they take the staging
// tiles in turn).
template <typename L>
__device__ __forceinline__ void stage_and_store(uint32_t stg0, int n_st, int row_in_tile, const float (&y)[32],
                                                bool store_lead, const CUtensorMap* map_c, int col0, int m0, int b) {
    const uint32_t stg = stg0 + uint32_t(n_st % L::kStgBufs) * L::kStgBytes;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t addr = stg + row_in_tile * 64 + ((j ^ ((row_in_tile >> 1) & 3)) << 4);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(pack_bf16x2(y[8 * j + 0], y[8 * j + 1])),
                     "r"(pack_bf16x2(y[8 * j + 2], y[8 * j + 3])), "r"(pack_bf16x2(y[8 * j + 4], y[8 * j + 5])),
                     "r"(pack_bf16x2(y[8 * j + 6], y[8 * j + 7]))
                     : "memory");
    }
    fence_proxy_async_smem();
    // the store two blocks back has read its tile, which the next block
    // reuses (only the newest store may still be reading); the barrier
    // publishes that and this block
    if (store_lead) bulk_wait_read<L::kStgPending>();
    epilogue_bar();
    if (store_lead) {
        tma_store_3d(map_c, stg, col0, m0, b);
        bulk_commit();
    }
}

// One output tile of an activation epilogue (unswapped), as one of its warps
// sees it. Rows below m_end and columns below N exist; `out`, `preact` and
// `residual` point at the row 0 and column 0 that row0 and col_first count
// from.
struct ActTile {
    const CUtensorMap* map_out;
    const CUtensorMap* map_z;
    void* out;                 // bf16, or codes
    uint16_t* preact;          // or NULL
    const uint16_t* residual;  // or NULL; may be out
    float* s_bias;             // 32 values of this warp: the block's bias (0 and left alone without one)
    uint32_t t_row;            // accumulator: this warp's lanes, the tile's first column
    uint32_t stg;              // this warp's staging tile (2 KB)
    float inv, s_out;
    int act, out_fmt;
    bool has_bias;
    int row0, m_end;  // this warp's first row
    int col_first, N, b;
    bool tma_out, tma_z;  // blocks of 32 rows leave by TMA
    bool vec_out, vec_z;  // else: 16-byte pieces of rows may be written (vec_z: preact, and residual read)
    bool has;             // there is an accumulator (else the products are 0)
};

// 16-byte piece j of row r of a 32-row staging tile of bf16 (64-byte swizzle)
// and of codes (32-byte swizzle): the lanes of a phase hit distinct banks.
__device__ __forceinline__ uint32_t stg_bf16(uint32_t stg, int r, int j) { return stg + r * 64 + ((j ^ ((r >> 1) & 3)) << 4); }
__device__ __forceinline__ uint32_t stg_code(uint32_t stg, int r, int j) { return stg + r * 32 + ((j ^ ((r >> 2) & 1)) << 4); }

__device__ __forceinline__ void sts128(uint32_t a, uint32_t x, uint32_t y, uint32_t z, uint32_t w) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(x), "r"(y), "r"(z), "r"(w) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}

// The warp's staging tile is free again: the TMA store of it, if any, has read it.
__device__ __forceinline__ void act_stage_free(int lane) {
    if (lane == 0) bulk_wait_read<0>();
    __syncwarp();
}

// The staged block to global memory: by TMA, which clips what the map does
// not hold, or row by row as far as rows and columns exist. PIECES: 16-byte
// pieces of a staged row (4 for bf16, 2 for codes, which leave by TMA or
// byte by byte).
template <int PIECES>
__device__ __forceinline__ void act_store(const ActTile& t, void* dst, const CUtensorMap* map, bool tma, bool vec,
                                          int col0, int lane) {
    constexpr int kElem = PIECES / 2;  // bytes of a value
    auto slot = [&](int r, int j) { return PIECES == 4 ? stg_bf16(t.stg, r, j) : stg_code(t.stg, r, j); };
    uint8_t* d = static_cast<uint8_t*>(dst);
    if (tma) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(map, t.stg, col0, t.row0, t.b);
            bulk_commit();
        }
    } else if (PIECES == 4 && vec) {
        __syncwarp();
        const int piece = lane % PIECES, col = col0 + piece * (16 / kElem);
#pragma unroll
        for (int r = lane / PIECES; r < 32; r += 32 / PIECES) {
            const uint4 w = lds128(slot(r, piece));
            if (t.row0 + r < t.m_end && col < t.N)
                *reinterpret_cast<uint4*>(d + (int64_t(t.row0 + r) * t.N + col) * kElem) = w;
        }
    } else {
        __syncwarp();
        const int at = lane * kElem;  // byte of a staged row: one column a lane
#pragma unroll 1
        for (int r = 0; r < 32 && t.row0 + r < t.m_end; ++r) {
            const uint32_t addr = slot(r, at >> 4) + (at & 15);
            uint16_t v;
            if (kElem == 2) asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
            else            asm volatile("{\n\t.reg .b32 w;\n\tld.shared.u8 w, [%1];\n\tcvt.u16.u32 %0, w;\n\t}" : "=h"(v) : "r"(addr) : "memory");
            if (col0 + lane < t.N) {
                const int64_t o = int64_t(t.row0 + r) * t.N + col0 + lane;
                if (kElem == 2) reinterpret_cast<uint16_t*>(d)[o] = v;
                else            d[o] = uint8_t(v);
            }
        }
    }
}

__device__ __forceinline__ void act_stage(uint32_t stg, const float (&y)[32], int lane) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
        sts128(stg_bf16(stg, lane, j), pack_bf16x2(y[8 * j + 0], y[8 * j + 1]), pack_bf16x2(y[8 * j + 2], y[8 * j + 3]),
               pack_bf16x2(y[8 * j + 4], y[8 * j + 5]), pack_bf16x2(y[8 * j + 6], y[8 * j + 7]));
}

// A warp's part of an activation epilogue: its 32 rows of the tile, every
// fourth block of 32 columns. Sixteen warps share a tile (four to a TMEM lane
// quarter and to a scheduler), because the epilogue is bound by latency: a
// block is a chain of TMEM load, MUFU, staging and store, which one warp a
// scheduler left bare (2048 x 4096 x 1024, GELU to codes with preact: 24.7 us
// with four warps, 16.3 with sixteen). Each warp stages and stores its own blocks, so that the
// warps drift apart and overlap; nothing is shared between them, and no
// barrier holds them together. Per block: z = acc * inv + bias, kept as bf16 if asked
// for, then act(z) + residual as bf16, or act(z) as FP8 codes under the output
// ring's scale (m_out: their amax so far). The residual arrives as 64-byte row
// pieces (a warp's load covers 8 rows), the first block's before the
// accumulator is there, and passes through the staging tile, where each
// thread finds its own row.
constexpr int kActPhases = 4;

// Blocks of 32 columns that a warp may have in a tile.
template <int BN>
constexpr int kActBlocks = (BN / 32 + kActPhases - 1) / kActPhases;

struct ActResidual {
    uint4 v[4];
    // rows (lane / 4) + 8 j of block c, 16-byte piece lane % 4
    __device__ __forceinline__ void load(const ActTile& t, int c, int lane) {
        const int col = t.col_first + c * 32 + (lane & 3) * 8;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int r = t.row0 + (lane >> 2) + 8 * j;
            v[j] = (r < t.m_end && col < t.N)
                       ? __ldcg(reinterpret_cast<const uint4*>(t.residual + int64_t(r) * t.N + col))
                       : make_uint4(0, 0, 0, 0);
        }
    }
};

// bias: this lane's column of each of the warp's blocks.
template <int BN, int ACT, bool OUT8>
__device__ __forceinline__ void act_blocks(const ActTile& t, ActResidual& res, const float (&bias)[kActBlocks<BN>],
                                           float& m_out, int phase, int lane) {
    const int left = (t.N - t.col_first + 31) / 32;
    const int nch = left < BN / 32 ? left : BN / 32;
#pragma unroll 1
    for (int c = phase; c < nch; c += kActPhases) {
        const int col0 = t.col_first + c * 32;
        uint32_t acc[32];
        if (t.has_bias) {
            __syncwarp();  // the previous block's readers are done
            t.s_bias[lane] = c < kActPhases ? bias[0] : bias[kActBlocks<BN> - 1];
        }
        if (t.has) {
            __syncwarp();
            tmem_ld<32>(t.t_row + c * 32, acc);
            tmem_ld_wait_tied(acc);
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) acc[i] = 0u;
        }
        __syncwarp();
        float y[32];
#pragma unroll
        for (int i = 0; i < 32; i += 4) {
            const float4 v = *reinterpret_cast<const float4*>(t.s_bias + i);
            split(fma2(f2(__uint_as_float(acc[i]), __uint_as_float(acc[i + 1])), f2(t.inv), f2(v.x, v.y)), y[i], y[i + 1]);
            split(fma2(f2(__uint_as_float(acc[i + 2]), __uint_as_float(acc[i + 3])), f2(t.inv), f2(v.z, v.w)), y[i + 2],
                  y[i + 3]);
        }
        if (t.preact) {
            act_stage_free(lane);
            act_stage(t.stg, y, lane);
            act_store<4>(t, t.preact, t.map_z, t.tma_z, t.vec_z, col0, lane);
        }
        if (ACT != FP8_ACT_NONE) act_each<ACT>(y);
        if (!OUT8 && t.residual) {
            act_stage_free(lane);
            if (t.vec_z) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sts128(stg_bf16(t.stg, (lane >> 2) + 8 * j, lane & 3), res.v[j].x, res.v[j].y, res.v[j].z, res.v[j].w);
                if (c + kActPhases < nch) res.load(t, c + kActPhases, lane);
            } else {
#pragma unroll 1
                for (int r = 0; r < 32; ++r) {
                    const bool in = t.row0 + r < t.m_end && col0 + lane < t.N;
                    const uint16_t v = in ? t.residual[int64_t(t.row0 + r) * t.N + col0 + lane] : uint16_t(0);
                    asm volatile("st.shared.u16 [%0], %1;" ::"r"(stg_bf16(t.stg, r, lane >> 3) + (lane & 7) * 2), "h"(v)
                                 : "memory");
                }
            }
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const uint4 w = lds128(stg_bf16(t.stg, lane, j));
                const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    split(add2(f2(y[8 * j + 2 * k], y[8 * j + 2 * k + 1]),
                               f2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xFFFF0000u))),
                          y[8 * j + 2 * k], y[8 * j + 2 * k + 1]);
            }
        }
        if constexpr (OUT8) {
            const bool row_in = t.row0 + lane < t.m_end;
            uint32_t w[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                uint32_t h[2];
#pragma unroll
                for (int k = 0; k < 4; k += 2) {
                    const float v0 = y[4 * j + k], v1 = y[4 * j + k + 1];
                    // columns past N hold bias 0 and products of zeros: act(0) = 0 does not raise the amax
                    if (row_in) asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m_out) : "f"(v0), "f"(v1));
                    float q0, q1;
                    split(mul2(f2(v0, v1), f2(t.s_out)), q0, q1);
                    h[k / 2] = cvt_fp8x2(t.out_fmt, q0, q1);
                }
                w[j] = h[0] | (h[1] << 16);
            }
            act_stage_free(lane);
            sts128(stg_code(t.stg, lane, 0), w[0], w[1], w[2], w[3]);
            sts128(stg_code(t.stg, lane, 1), w[4], w[5], w[6], w[7]);
            act_store<2>(t, t.out, t.map_out, t.tma_out, t.vec_out, col0, lane);
        } else {
            if (!t.residual) act_stage_free(lane);
            act_stage(t.stg, y, lane);
            act_store<4>(t, t.out, t.map_out, t.tma_out, t.vec_out, col0, lane);
        }
    }
}

template <int BN, bool OUT8>
__device__ __forceinline__ void act_tile(const ActTile& t, ActResidual& res, const float (&bias)[kActBlocks<BN>],
                                         float& m_out, int phase, int lane) {
    if (t.row0 >= t.m_end) return;  // no row of this warp exists
    switch (t.act) {
        case FP8_ACT_NONE: act_blocks<BN, FP8_ACT_NONE, OUT8>(t, res, bias, m_out, phase, lane); break;
        case FP8_ACT_RELU: act_blocks<BN, FP8_ACT_RELU, OUT8>(t, res, bias, m_out, phase, lane); break;
        case FP8_ACT_GELU: act_blocks<BN, FP8_ACT_GELU, OUT8>(t, res, bias, m_out, phase, lane); break;
        case FP8_ACT_GELU_TANH: act_blocks<BN, FP8_ACT_GELU_TANH, OUT8>(t, res, bias, m_out, phase, lane); break;
        default: act_blocks<BN, FP8_ACT_SILU, OUT8>(t, res, bias, m_out, phase, lane); break;
    }
}

// The amax of an FP8 output, over every epilogue thread of the grid: one
// atomicMax a CTA, then a ticket; the CTA holding the last one folds it into
// the output's ring. T: epilogue threads of the CTA; red: shared memory that
// no epilogue thread uses any more after the first barrier.
template <int T>
__device__ __forceinline__ void out8_finish(const GemmParams& p, float m_out, float* s_bias, int warp, int lane, int etid) {
    uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m_out));
    epilogue_bar<T>();  // the bias slots are free now
    uint32_t* red = reinterpret_cast<uint32_t*>(s_bias);
    if (lane == 0) red[warp - 2] = bits;
    epilogue_bar<T>();
    if (etid != 0) return;
    bits = red[0];
    for (int w = 1; w < T / 32; ++w) bits = max(bits, red[w]);
    fp8_ring* ring = p.out_ring;
    if (bits != 0u) atomicMax(&ring->amax_bits, bits);
    const uint32_t ticket = atom_add_acq_rel(&ring->ticket, 1u);
    if (ticket != gridDim.x - 1) return;
    volatile fp8_ring* rr = ring;
    float h[FP8_RING_HISTORY];
    const uint32_t idx = ring_read(rr, h);
    const float a = __uint_as_float(atomicExch(&ring->amax_bits, 0u));
    ring_fold(rr, h, idx, a, fmt_max(p.out_fmt));
    if (p.out_amax) *p.out_amax = a;
    rr->ticket = 0u;
}

// The epilogue role of an activation launch (unswapped tiles). What a tile
// needs from global memory is asked for one tile early: its bias (a lane
// fetches a column of each of its warp's blocks), and its residual as a
// prefetch into L2, whose first block each warp then loads before the
// accumulator is there.
template <int BN, int CTAS, bool OUT8>
__device__ __forceinline__ void act_epilogue(const GemmParams& p, const EpArgs<true>& ep, const CUtensorMap* map_c,
                                             float* s_bias, uint32_t stg0, uint32_t tmem_base, uint32_t bar_tfull,
                                             uint32_t bar_tempty, uint32_t rank, int unit0, int unit_step,
                                             int total_units, const TileWalk& walk, int M, int N, int tma_store,
                                             int warp, int lane) {
    constexpr int ET = epi_threads(true, false);
    griddep_wait();
    griddep_launch();
    const int q = warp & 3, phase = (warp - 2) >> 2;
    const int etid = threadIdx.x - 64;
    const float bscale = p.bias_kind == 2 ? __ldg(p.bias_scale) : 1.0f;
    float m_out = 0.0f;
    ActTile t;
    t.map_out = map_c;
    t.map_z = &ep.tz;
    t.s_bias = s_bias + (warp - 2) * 32;
    t.s_bias[lane] = 0.0f;
    t.has_bias = p.bias_kind != 0;
    t.stg = stg0 + uint32_t(warp - 2) * 2048u;
    t.inv = (1.0f / __ldg(p.sa)) * (1.0f / __ldg(p.sb));
    t.s_out = 1.0f;
    if (OUT8) {  // the ring's scale before this call: the fold waits for every CTA's ticket
        t.s_out = *reinterpret_cast<volatile float*>(&p.out_ring->scale);
        if (blockIdx.x == 0 && etid == 0) *p.out_scale = t.s_out;
    }
    t.act = ep.act;
    t.out_fmt = p.out_fmt;
    t.m_end = M;
    t.N = N;
    t.tma_out = t.vec_out = tma_store;
    t.tma_z = t.vec_z = ep.fast;
    t.has = true;
    const bool res_vec = !OUT8 && ep.residual && ep.fast;
    float bias[kActBlocks<BN>] = {}, bias_next[kActBlocks<BN>] = {};
    auto ask_bias = [&](int nb) {
#pragma unroll
        for (int i = 0; i < kActBlocks<BN>; ++i) {
            const int col = nb * BN + (phase + i * kActPhases) * 32 + lane;
            if (col >= N || p.bias_kind == 0) bias_next[i] = 0.0f;
            else if (p.bias_kind == 1) bias_next[i] = bf16_value(__ldg(static_cast<const uint16_t*>(p.bias) + col));
            else bias_next[i] = __fdiv_rn(fp8_to_f32(__ldg(static_cast<const uint8_t*>(p.bias) + col), p.bias_fmt), bscale);
        }
    };
    int mb = 0, nb = 0, b = 0;
    if (unit0 < total_units) {
        tile_coords_lazy(unit0, walk, mb, nb, b);
        ask_bias(nb);
    }
    bool failed = false;
    int it = 0;
    for (int u = unit0; u < total_units; u += unit_step, ++it) {
        const int buf = it & 1;
        t.row0 = (mb * CTAS + int(rank)) * BM + q * 32;
        t.col_first = nb * BN;
        t.b = b;
        t.out = OUT8 ? static_cast<void*>(reinterpret_cast<uint8_t*>(p.out) + int64_t(b) * p.stride_c)
                     : static_cast<void*>(p.out + int64_t(b) * p.stride_c);
        t.preact = ep.preact ? ep.preact + int64_t(b) * p.stride_c : nullptr;
        t.residual = ep.residual ? ep.residual + int64_t(b) * ep.stride_r : nullptr;
        ActResidual res;
        if (res_vec) res.load(t, phase, lane);
#pragma unroll
        for (int i = 0; i < kActBlocks<BN>; ++i) bias[i] = bias_next[i];
        if (u + unit_step < total_units) {
            tile_coords_lazy(u + unit_step, walk, mb, nb, b);
            ask_bias(nb);
            const int64_t row = int64_t(mb * CTAS + int(rank)) * BM + q * 32 + lane;
            if (res_vec && row < M) {
                const uint16_t* r = ep.residual + int64_t(b) * ep.stride_r + row * N;
#pragma unroll
                for (int c = phase * 32; c < BN; c += kActPhases * 32)
                    if (nb * BN + c < N) asm volatile("prefetch.global.L2 [%0];" ::"l"(r + nb * BN + c));
            }
        }
        if (!failed) failed = !wait_bounded_warp(bar_tfull + 8 * buf, (it >> 1) & 1);
        if (failed) continue;  // the other warps find it out for themselves
        tc_fence_after();
        t.t_row = tmem_base + (uint32_t(q * 32) << 16) + buf * BN;
        act_tile<BN, OUT8>(t, res, bias, m_out, phase, lane);
        tc_fence_before();
        // release the accumulator to the MMA issuer (the pair's leader)
        if (CTAS == 1) mbar_arrive(bar_tempty + 8 * buf);
        else           mbar_arrive_cluster(map_to_rank(bar_tempty + 8 * buf, 0));
    }
    if (lane == 0) bulk_wait_read<0>();  // the staging tiles outlive the stores that read them
    if (OUT8) out8_finish<ET>(p, m_out, s_bias, warp, lane, etid);
}

// One kernel for both tile shapes: CTAS = 1 computes 128 x BN tiles per CTA;
// CTAS = 2 runs as clusters of two CTAs on two SMs computing 256 x BN tiles
// with tcgen05 cta_group::2 -- the leader issues the MMAs, each CTA loads its
// own 128 rows of A and BN/2 columns of B (halving each SM's operand
// traffic) and writes its own 128 output rows.
//
// Epilogue: 4 warps, one per TMEM lane quarter. Every 32 columns of the tile
// become a 128 x 32 bf16 tile in shared memory that one thread writes with a
// single TMA store (8 stores for a 128 x 256 tile).
//
// GROUP: the units are the tiles of up to kMaxEntries table entries (one SM
// per tile, no split, no batches); operand majors, maps, tile width, first
// column, scales, bias and output come from the entry of each unit, A_MN /
// B_MN only give the defaults and BN is the widest tile.
template <int BN, bool A_MN, bool B_MN, int STAGES, bool HAS_BIAS, int CTAS, bool SPLIT, bool SWAP, bool OUT8,
          bool GROUP = false, bool EP = false>
__global__ void __maxnreg__(EP && !SWAP ? kActRegs : 168)
fp8_gemm_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                const __grid_constant__ CUtensorMap tm_c, const GemmParams p,
                const __grid_constant__ GroupTab<GROUP> grp, const __grid_constant__ EpArgs<EP> ep) {
    using L = Smem<BN, STAGES, CTAS, EP ? 4 : 3>;
    constexpr int ET = epi_threads(EP, SWAP);
    static_assert(!EP || (HAS_BIAS && !GROUP), "an activation epilogue always has its bias slots");
    static_assert(!(B_MN && CTAS == 2 && BN != 256), "MN-major B halves must be whole 128-byte atoms");
    static_assert(!GROUP || (CTAS == 1 && !SPLIT && !SWAP && !OUT8), "grouped launches use plain one-SM tiles");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if constexpr (L::kAct) {
        if (!smem_fits<L>(smem_raw, smem)) return;
    }
    const uint32_t s_base = smem_addr(smem);
    const uint32_t s_a = s_base;
    const uint32_t s_b = s_base + STAGES * L::kABytes;
    const uint32_t bar_full = s_base + L::kBarOffset;
    const uint32_t bar_empty = bar_full + STAGES * 8;
    const uint32_t bar_tfull = bar_empty + STAGES * 8;
    const uint32_t bar_tempty = bar_tfull + 2 * 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBarOffset + (2 * STAGES + 4) * 8);
    uint32_t* ticket_slot = tmem_slot + 1;  // split K: the epilogue's arrival ticket
    const uint32_t bar_red = smem_addr(tmem_slot + 2);  // cluster split: the other splits' partials are in
    float* s_bias = reinterpret_cast<float*>(smem + L::kBiasOffset);

    const int warp = threadIdx.x >> 5;
    const int lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_ctarank() : 0u;  // 0 = the pair's leader
    const bool leader = rank == 0;
    const int unit0 = blockIdx.x / CTAS;     // this CTA's first work unit (a pair shares it)
    const int unit_step = gridDim.x / CTAS;  // units advance by the number of CTAs (pairs)

    // every parameter the roles read, fetched together now
    const int total_units = pin(p.total_units);
    const int k_blocks = pin(p.k_blocks);
    const int split = SPLIT ? pin(p.split) : 1;  // without SPLIT the split-K code compiles away
    const int kb_per = SPLIT ? pin(p.kb_per) : k_blocks;
    const TileWalk walk = {pin(p.m_tiles), pin(p.n_tiles), pin(p.group_m)};
    const int a_bcast = pin(p.a_bcast), b_bcast = pin(p.b_bcast);
    const uint32_t idesc = pin(p.idesc);
    int M = pin(p.M), N = pin(p.N);  // per unit in a grouped launch
    int tma_store = pin(p.tma_store), vec_store = pin(p.vec_store);
    const int csplit = (SWAP && SPLIT) ? pin(p.csplit) : 0;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, CTAS * ET);
        }
        if (csplit) mbar_init(bar_red, uint32_t(split - 1) * kEpiThreads);
        fence_mbar_init();
        if constexpr (GROUP) {
            for (int i = 0; i < grp.count; ++i) {
                tma_prefetch(&grp.q[i].ta);
                tma_prefetch(&grp.q[i].tb);
                if (grp.q[i].tma_store) tma_prefetch(&grp.q[i].tc);
            }
        } else {
            tma_prefetch(&tm_a);
            tma_prefetch(&tm_b);
            if (tma_store) tma_prefetch(&tm_c);
            if constexpr (EP) {
                if (ep.fast && ep.preact) tma_prefetch(&ep.tz);
            }
        }
    }
    if (warp == 1) {
        tmem_alloc<CTAS>(smem_addr(tmem_slot), L::kTmemCols);
        tmem_relinquish<CTAS>();
    }
    tc_fence_before();
    __syncthreads();
    // the cluster's barriers exist before any remote arrive
    if (CTAS == 2 || csplit) cluster_sync();
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    // The prologue above overlaps the previous kernel's tail; operands,
    // scales and the output are touched only after it has completed. Each
    // role waits for it separately, so that the producer can work out its
    // first unit's tile (pure arithmetic on the parameters) before.

    if (warp == 0) {
        // ------------------------------------------------ TMA producer ---
        // The whole warp walks the units and waits on the barriers, so the
        // loop's values stay warp-uniform; one elected lane issues the loads.
        const bool issuer = elect_one();
        struct Plan {
            const CUtensorMap* map_a;
            const CUtensorMap* map_b;
            int kb0, kb1, m0, n0, ba, bb, ebn;
            uint32_t stage_tx;
            bool a_mn, b_mn;
        };
        // the loads of work unit u: maps, k-block range, tile origin, batch
        auto plan = [&](int u) {
            Plan pl;
            int t = u / split;
            pl.map_a = &tm_a;
            pl.map_b = &tm_b;
            pl.a_mn = A_MN;
            pl.b_mn = B_MN;
            TileWalk w = walk;
            int kbs = k_blocks;
            int n_base = 0;
            pl.ebn = BN;  // the unit's tile width
            if constexpr (GROUP) {
                const GroupProblem& q = group_problem(grp, u, t);
                pl.map_a = &q.ta;
                pl.map_b = &q.tb;
                pl.a_mn = q.a_mn;
                pl.b_mn = q.b_mn;
                w = {q.m_tiles, q.n_tiles, walk.group_m};
                kbs = q.k_blocks;
                pl.ebn = q.bn;
                n_base = q.n_base;
            }
            pl.kb0 = GROUP ? 0 : (u - t * split) * kb_per;
            pl.kb1 = GROUP ? kbs : min(k_blocks, pl.kb0 + kb_per);
            int mb, nb, b;
            tile_coords(t, w, mb, nb, b);
            pl.ba = a_bcast ? 0 : b;
            pl.bb = b_bcast ? 0 : b;
            pl.m0 = mb * BM * CTAS + int(rank) * BM;
            pl.n0 = n_base + nb * pl.ebn + int(rank) * (BN / CTAS);
            pl.stage_tx = GROUP ? uint32_t(L::kABytes + pl.ebn * BK) : uint32_t(L::kStageTx);
            return pl;
        };
        Plan pl = {};
        if (unit0 < total_units) pl = plan(unit0);  // before the wait: it reads no memory
        griddep_wait();
        griddep_launch();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int i = 0, u = unit0; u < total_units && ok;) {
            const CUtensorMap* map_a = pl.map_a;
            const CUtensorMap* map_b = pl.map_b;
            const bool a_mn = pl.a_mn, b_mn = pl.b_mn;
            const int kb0 = pl.kb0, kb1 = pl.kb1, m0 = pl.m0, n0 = pl.n0, ba = pl.ba, bb = pl.bb, ebn = pl.ebn;
            const uint32_t stage_tx = pl.stage_tx;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!wait_bounded_warp(bar_empty + 8 * stage, phase ^ 1)) { ok = false; break; }
                const uint32_t full = bar_full + 8 * stage;
                const uint32_t da = s_a + stage * L::kABytes;
                const uint32_t db = s_b + stage * L::kBBytes;
                if (issuer) {
                    if (leader) mbar_arrive_expect_tx(full, stage_tx);
                    if (CTAS == 1) {
                        if (a_mn) tma_load_3d(da, map_a, full, m0, kb * BK, ba);
                        else      tma_load_3d(da, map_a, full, kb * BK, m0, ba);
                        if (b_mn) {
#pragma unroll
                            for (int h = 0; h < BN / 128; ++h)
                                if (h * 128 < ebn) tma_load_3d(db + h * 128 * BK, map_b, full, n0 + h * 128, kb * BK, bb);
                        } else {
                            tma_load_3d(db, map_b, full, kb * BK, n0, bb);
                        }
                    } else {
                        const uint32_t lfull = map_to_rank(full, 0);  // the leader's barrier
                        if (A_MN) tma_load_3d_pair(da, &tm_a, lfull, m0, kb * BK, ba);
                        else      tma_load_3d_pair(da, &tm_a, lfull, kb * BK, m0, ba);
                        if (B_MN) tma_load_3d_pair(db, &tm_b, lfull, n0, kb * BK, bb);
                        else      tma_load_3d_pair(db, &tm_b, lfull, kb * BK, n0, bb);
                    }
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
            u = unit_of<GROUP>(++i, unit0, unit_step);
            if (u < total_units) pl = plan(u);
        }
        // drain: wait until the MMAs released every stage still in use
        for (int i = 0; i < STAGES && ok; ++i) {
            if (!wait_bounded_warp(bar_empty + 8 * stage, phase ^ 1)) break;
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
    } else if (warp == 1) {
        // --------------------------------------------------- MMA issuer ---
        griddep_wait();
        griddep_launch();
        // As the producer: the warp walks and waits together, one elected
        // lane issues every MMA and commit (a commit tracks the MMAs of the
        // thread that issues it, so it is always the same lane).
        const bool issuer = elect_one();
        if (leader) {
            int stage = 0;
            uint32_t phase = 0;
            int it = 0;
            bool ok = true;
            for (int u = unit0; u < total_units && ok; u = unit_of<GROUP>(++it, unit0, unit_step)) {
                int t = u / split;
                bool a_mn = A_MN, b_mn = B_MN;
                uint32_t id = idesc;
                int kbs = k_blocks;
                if constexpr (GROUP) {
                    const GroupProblem& q = group_problem(grp, u, t);
                    a_mn = q.a_mn;
                    b_mn = q.b_mn;
                    id = q.idesc;
                    kbs = q.k_blocks;
                }
                const int kb0 = GROUP ? 0 : (u - t * split) * kb_per;
                const int kb1 = GROUP ? kbs : min(k_blocks, kb0 + kb_per);
                const int buf = it & 1;
                const uint32_t acc_phase = (it >> 1) & 1;
                if (!wait_bounded_warp(bar_tempty + 8 * buf, acc_phase ^ 1)) break;
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * BN;
                const uint64_t a_desc0 = a_mn ? smem_desc_sw128(s_a, 128 * BK, 1024) : smem_desc_sw128(s_a, 16, 1024);
                const uint64_t b_desc0 = b_mn ? smem_desc_sw128(s_b, 128 * BK, 1024) : smem_desc_sw128(s_b, 16, 1024);
                const uint64_t a_step = a_mn ? 256u : 2u, b_step = b_mn ? 256u : 2u;
                for (int kb = kb0; kb < kb1; ++kb) {
                    // the stage's operands arrive through the async proxy and
                    // complete on this barrier: the MMAs may read them without
                    // a tcgen05 fence (that is needed only after the epilogue's
                    // hand-back of the accumulator, above)
                    if (!wait_bounded_warp(bar_full + 8 * stage, phase)) { ok = false; break; }
                    // the stage's descriptors: stage 0's plus the stage offset in
                    // the start-address field (16-byte units; no carry out of it,
                    // shared memory is below 256 KB). Each next 32-deep K slice is
                    // +32 bytes inside the swizzle atom (K-major) or 32 rows of
                    // 128 bytes further (MN-major).
                    const uint64_t adesc = a_desc0 + uint64_t(stage) * (L::kABytes >> 4);
                    const uint64_t bdesc = b_desc0 + uint64_t(stage) * (L::kBBytes >> 4);
                    if (issuer) {
                        mma_kblock_f8f6f4<CTAS>(d_tmem, adesc, bdesc, a_step, b_step, id, kb != kb0);
                        // release the stage (in both CTAs of a pair)
                        if (CTAS == 1) mma_commit(bar_empty + 8 * stage);
                        else           mma_commit_pair(bar_empty + 8 * stage);
                    }
                    __syncwarp();
                    if (++stage == STAGES) { stage = 0; phase ^= 1; }
                }
                if (issuer) {
                    if (CTAS == 1) mma_commit(bar_tfull + 8 * buf);
                    else           mma_commit_pair(bar_tfull + 8 * buf);
                }
                __syncwarp();
            }
        }
    } else {
        // ----------------------------------------------------- epilogue ---
        if constexpr (EP && !SWAP) {
            act_epilogue<BN, CTAS, OUT8>(p, ep, &tm_c, s_bias, s_base + L::kStgOffset, tmem_base, bar_tfull, bar_tempty, rank,
                                         unit0, unit_step, total_units, walk, M, N, tma_store, warp, lane);
        } else {
            griddep_wait();
            griddep_launch();
            const int q = warp & 3;             // TMEM lane quarter this warp may access
            const int row_in_tile = q * 32 + lane;
            const int etid = threadIdx.x - 64;  // 0 .. kEpiThreads-1
            const bool store_lead = etid == 0;  // issues the TMA stores
            const uint32_t stg0 = s_base + L::kStgOffset;
            int n_st = 0;  // TMA stores issued so far (they take the staging tiles in turn)
            float inv = (1.0f / __ldg(p.sa)) * (1.0f / __ldg(p.sb));
            int bias_kind = p.bias_kind, bias_fmt = p.bias_fmt;
            const void* bias_ptr = p.bias;
            float bscale = (HAS_BIAS && bias_kind == 2) ? __ldg(p.bias_scale) : 1.0f;
            uint16_t* out_base = p.out;
            const CUtensorMap* map_c = &tm_c;
            // FP8 output: the ring's scale before this call (every CTA reads it
            // before any CTA can fold: the fold waits for all CTAs' tickets)
            float s_out = 1.0f, m_out = 0.0f;
            if (OUT8) {
                s_out = *reinterpret_cast<volatile float*>(&p.out_ring->scale);
                if (blockIdx.x == 0 && etid == 0) *p.out_scale = s_out;
            }
            bool failed = false;
            int it = 0;
            for (int u = unit0; u < total_units; u = unit_of<GROUP>(++it, unit0, unit_step)) {
                int t = u / split;
                const int split_id = u - t * split;
                TileWalk w = walk;
                int ebn = BN, n_base = 0;  // the unit's tile width and first column
                if constexpr (GROUP) {
                    const GroupProblem& q = group_problem(grp, u, t);
                    w = {q.m_tiles, q.n_tiles, walk.group_m};
                    ebn = q.bn;
                    n_base = q.n_base;
                    M = q.M;
                    N = q.N;
                    tma_store = q.tma_store;
                    vec_store = q.vec_store;
                    map_c = &q.tc;
                    out_base = q.out;
                    bias_kind = q.bias_kind;
                    bias_fmt = q.bias_fmt;
                    bias_ptr = q.bias;
                    inv = (1.0f / __ldg(q.sa)) * (1.0f / __ldg(q.sb));
                    bscale = (HAS_BIAS && bias_kind == 2) ? __ldg(q.bias_scale) : 1.0f;
                }
                int mb, nb, b;
                tile_coords(t, w, mb, nb, b);
                const int buf = it & 1;
                const uint32_t acc_phase = (it >> 1) & 1;
                const int m0 = mb * BM * CTAS + int(rank) * BM;  // this CTA's first output row
                if (HAS_BIAS && !SWAP) {
                    // the tile's BN bias values, dequantized once into shared memory
                    epilogue_bar();  // the previous tile's readers are done
                    for (int j = etid; j < ebn; j += kEpiThreads) {
                        const int col = n_base + nb * ebn + j;
                        float v = 0.0f;
                        if (col < N && bias_kind != 0) {  // a grouped launch may mix problems with and without bias
                            if (bias_kind == 1) {
                                v = __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(bias_ptr) + col)) << 16);
                            } else {
                                v = __fdiv_rn(fp8_to_f32(__ldg(static_cast<const uint8_t*>(bias_ptr) + col), bias_fmt),
                                              bscale);
                            }
                        }
                        s_bias[j] = v;
                    }
                    epilogue_bar();
                }
                // a swapped activation asks for its residual's first 16 rows of C and
                // for its bias while the accumulator is still being made
                float act_bias = 0.0f, act_res[16];
                if constexpr (EP && SWAP) {
                    const int col = m0 + row_in_tile;  // of C
#pragma unroll
                    for (int i = 0; i < 16; ++i) act_res[i] = 0.0f;
                    if (col < M && (!csplit || split_id == 0)) {
                        const uint16_t* res = ep.residual ? ep.residual + int64_t(b) * ep.stride_r + col : nullptr;
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (res && nb * BN + i < N) act_res[i] = bf16_value(res[int64_t(nb * BN + i) * M]);
                        if (bias_kind == 1)
                            act_bias = bf16_value(__ldg(static_cast<const uint16_t*>(bias_ptr) + col));
                        else if (bias_kind == 2)
                            act_bias = __fdiv_rn(fp8_to_f32(__ldg(static_cast<const uint8_t*>(bias_ptr) + col), bias_fmt),
                                                 bscale);
                    }
                }
                // every lane waits, then all epilogue warps agree (and each warp
                // reconverges) before the warp-collective TMEM loads. After a wait
                // gave up, they all keep walking the units without waiting, so that
                // they still meet at every named barrier.
                if (!failed) failed = !wait_bounded(bar_tfull + 8 * buf, acc_phase);
                failed = epilogue_bar_or(failed);
                if (failed) continue;
                tc_fence_after();
                const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16) + buf * BN;
                // Split K: the unit that arrives last at its tile finishes it; the
                // others leave their fp32 partial in the workspace. Slot layout:
                // 16-byte piece v of CW-column chunk c of tile row r sits at
                // ((c * CW / 4 + v) * 128 + r) * 16, so each store and load
                // instruction of a warp covers 512 contiguous bytes.
                constexpr int CW = SWAP ? 16 : 32;  // accumulator columns per TMEM load
                const float4* slots = nullptr;
                if (SPLIT && split > 1 && csplit) {
                    // cluster split: CTA r of the cluster is split r of the tile
                    // (one tile per cluster); splits 1.. push their partials into
                    // split 0's staging area (free in swapped launches), slot r - 1,
                    // laid out as the workspace's slots, and arrive on its barrier
                    if (split_id != 0) {
                        const uint32_t dst = map_to_rank(stg0 + uint32_t(split_id - 1) * (BM * BN * 4), 0);
#pragma unroll 1
                        for (int c = 0; c < BN / CW; ++c) {
                            if (nb * BN + c * CW >= N) break;  // uniform; split 0 skips it too
                            uint32_t r[CW];
                            tmem_ld<CW>(t_row + c * CW, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int v = 0; v < CW / 4; ++v)
                                st_cluster_v4(dst + uint32_t(((c * (CW / 4) + v) * 128 + row_in_tile) * 16),
                                              __uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                              __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3]));
                        }
                        mbar_arrive_cluster(map_to_rank(bar_red, 0));  // release: the stores above come first
                        tc_fence_before();
                        mbar_arrive(bar_tempty + 8 * buf);
                        continue;
                    }
                    if (!failed) failed = !wait_bounded_cluster(bar_red, 0);
                    failed = epilogue_bar_or(failed);
                    if (failed) continue;
                } else if (SPLIT && split > 1) {
                    uint32_t* cnt = p.ws_cnt + 2 * (t * CTAS + int(rank));
                    slots = reinterpret_cast<const float4*>(p.ws) + size_t(t * CTAS + int(rank)) * split * (BM * BN / 4);
                    if (etid == 0) *ticket_slot = atomicAdd(cnt, 1u);
                    epilogue_bar();
                    const bool last = *ticket_slot == uint32_t(split - 1);
                    if (!last) {
                        float4* mine = const_cast<float4*>(slots) + size_t(split_id) * (BM * BN / 4);
#pragma unroll 1
                        for (int c = 0; c < BN / CW; ++c) {
                            if (nb * BN + c * CW >= N) break;  // uniform; the finisher skips it too
                            uint32_t r[CW];
                            tmem_ld<CW>(t_row + c * CW, r);
                            tmem_ld_wait();
#pragma unroll
                            for (int v = 0; v < CW / 4; ++v)
                                __stcg(mine + (c * (CW / 4) + v) * 128 + row_in_tile,
                                       make_float4(__uint_as_float(r[4 * v]), __uint_as_float(r[4 * v + 1]),
                                                   __uint_as_float(r[4 * v + 2]), __uint_as_float(r[4 * v + 3])));
                        }
                        __threadfence();
                        epilogue_bar();
                        if (etid == 0) red_release_add(cnt + 1, 1u);
                        tc_fence_before();
                        if (CTAS == 1) mbar_arrive(bar_tempty + 8 * buf);
                        else           mbar_arrive_cluster(map_to_rank(bar_tempty + 8 * buf, 0));
                        continue;
                    }
                    if (etid == 0) {
                        wait_count(cnt + 1, uint32_t(split - 1));
                        cnt[0] = 0u;  // the tile's counters are ready for the next call
                        cnt[1] = 0u;
                    }
                    epilogue_bar();
                }
                const int row = m0 + row_in_tile;
                // swapped operands: this thread's TMEM lane is output column `row`
                // of C (the kernel's M is C's N), its accumulator columns are C's rows
                float bias_row = (EP && SWAP) ? act_bias : 0.0f;
                if (SWAP && HAS_BIAS && !EP && row < M) {
                    if (bias_kind == 1)
                        bias_row = __uint_as_float(uint32_t(__ldg(static_cast<const uint16_t*>(bias_ptr) + row)) << 16);
                    else
                        bias_row = __fdiv_rn(fp8_to_f32(__ldg(static_cast<const uint8_t*>(bias_ptr) + row), bias_fmt),
                                             bscale);
                }
                uint16_t* orow = SWAP ? out_base + int64_t(b) * p.stride_c + row
                                      : out_base + int64_t(b) * p.stride_c + int64_t(row) * N;
                if constexpr (!SPLIT && !SWAP && !OUT8) {
                    if (tma_store) {
                        // The common case, pipelined: chunk c + 1's accumulator
                        // columns leave TMEM while chunk c is converted, staged and
                        // stored (two register sets, the wait tied to the set it
                        // waits for).
                        const int col_first = n_base + nb * ebn;
                        const int left = (N - col_first + 31) / 32;
                        const int nch = left < ebn / 32 ? left : ebn / 32;
                        auto emit = [&](const uint32_t (&r)[32], int c) {
                            float y[32];
#pragma unroll
                            for (int i = 0; i < 32; ++i) {
                                const float bias = HAS_BIAS ? s_bias[c * 32 + i] : 0.0f;
                                y[i] = fmaf(__uint_as_float(r[i]), inv, bias);
                            }
                            stage_and_store<L>(stg0, n_st, row_in_tile, y, store_lead, map_c, col_first + c * 32, m0, b);
                            ++n_st;
                        };
                        uint32_t ra[32], rb[32];
                        tmem_ld<32>(t_row, ra);
                        tmem_ld_wait_tied(ra);
#pragma unroll 1
                        for (int c = 0; c < nch; c += 2) {
                            __syncwarp();
                            if (c + 1 < nch) tmem_ld<32>(t_row + (c + 1) * 32, rb);
                            emit(ra, c);
                            if (c + 1 >= nch) break;
                            tmem_ld_wait_tied(rb);
                            __syncwarp();
                            if (c + 2 < nch) tmem_ld<32>(t_row + (c + 2) * 32, ra);
                            emit(rb, c + 1);
                            if (c + 2 < nch) tmem_ld_wait_tied(ra);
                        }
                        tc_fence_before();
                        if (CTAS == 1) mbar_arrive(bar_tempty + 8 * buf);
                        else           mbar_arrive_cluster(map_to_rank(bar_tempty + 8 * buf, 0));
                        continue;
                    }
                }
#pragma unroll 1
                for (int c = 0; c < ebn / CW; ++c) {
                    const int col0 = n_base + nb * ebn + c * CW;
                    if (col0 >= N) break;  // uniform over the epilogue warps
                    uint32_t r[CW];
                    tmem_ld<CW>(t_row + c * CW, r);
                    tmem_ld_wait();
                    if (SPLIT && split > 1) {
                        // the sum over the splits in split order, whatever order
                        // they arrived in (the result does not depend on timing)
                        float acc[CW];
#pragma unroll 1
                        for (int sp = 0; sp < split; ++sp) {
                            if (sp == split_id) {
#pragma unroll
                                for (int i = 0; i < CW; ++i)
                                    acc[i] = sp == 0 ? __uint_as_float(r[i]) : acc[i] + __uint_as_float(r[i]);
                            } else if (csplit) {
                                const uint32_t src = stg0 + uint32_t(sp - 1) * (BM * BN * 4) +
                                                     uint32_t(((c * (CW / 4)) * 128 + row_in_tile) * 16);
#pragma unroll
                                for (int v = 0; v < CW / 4; ++v) {
                                    float4 x;
                                    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                                                 : "=f"(x.x), "=f"(x.y), "=f"(x.z), "=f"(x.w)
                                                 : "r"(src + uint32_t(v * 128 * 16)));
                                    acc[4 * v] = acc[4 * v] + x.x;
                                    acc[4 * v + 1] = acc[4 * v + 1] + x.y;
                                    acc[4 * v + 2] = acc[4 * v + 2] + x.z;
                                    acc[4 * v + 3] = acc[4 * v + 3] + x.w;
                                }
                            } else {
                                const float4* src =
                                    slots + size_t(sp) * (BM * BN / 4) + c * (CW / 4) * 128 + row_in_tile;
#pragma unroll
                                for (int v = 0; v < CW / 4; ++v) {
                                    const float4 x = __ldcg(src + v * 128);
                                    acc[4 * v] = sp == 0 ? x.x : acc[4 * v] + x.x;
                                    acc[4 * v + 1] = sp == 0 ? x.y : acc[4 * v + 1] + x.y;
                                    acc[4 * v + 2] = sp == 0 ? x.z : acc[4 * v + 2] + x.z;
                                    acc[4 * v + 3] = sp == 0 ? x.w : acc[4 * v + 3] + x.w;
                                }
                            }
                        }
#pragma unroll
                        for (int i = 0; i < CW; ++i) r[i] = __float_as_uint(acc[i]);
                    }
                    if constexpr (SWAP) {
                        // C[col0 + i][row]: lanes hold consecutive columns, so each
                        // store instruction of a warp writes 64 contiguous bytes
                        if constexpr (EP) {
                            // the same, through the activation: z to preact, act(z) + residual to out
                            float y[CW];
#pragma unroll
                            for (int i = 0; i < CW; ++i) y[i] = fmaf(__uint_as_float(r[i]), inv, bias_row);
                            if (row < M) {
                                if (ep.preact) {
                                    uint16_t* z = ep.preact + (orow - out_base);
#pragma unroll
                                    for (int i = 0; i < CW; ++i)
                                        if (col0 + i < N) z[int64_t(col0 + i) * M] = bf16_bits(y[i]);
                                }
                                act_apply(ep.act, y);
                                if (ep.residual && c > 0) {
                                    const uint16_t* res = ep.residual + int64_t(b) * ep.stride_r + row;
#pragma unroll
                                    for (int i = 0; i < CW; ++i)
                                        act_res[i] = col0 + i < N ? bf16_value(res[int64_t(col0 + i) * M]) : 0.0f;
                                }
                                if (ep.residual) {
#pragma unroll
                                    for (int i = 0; i < CW; ++i) y[i] += act_res[i];
                                }
#pragma unroll
                                for (int i = 0; i < CW; ++i)
                                    if (col0 + i < N) orow[int64_t(col0 + i) * M] = bf16_bits(y[i]);
                            }
                        } else if (row < M) {
#pragma unroll
                            for (int i = 0; i < CW; ++i) {
                                if (col0 + i >= N) break;
                                const float y = fmaf(__uint_as_float(r[i]), inv, bias_row);
                                uint16_t h;
                                asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(y));
                                orow[int64_t(col0 + i) * M] = h;
                            }
                        }
                    } else {
                        float y[CW];
#pragma unroll
                        for (int i = 0; i < CW; ++i) {
                            const float bias = HAS_BIAS ? s_bias[c * CW + i] : 0.0f;
                            y[i] = fmaf(__uint_as_float(r[i]), inv, bias);
                        }
                        if constexpr (OUT8) {
                            // q = sat_rne(fp32(y * s_out)); the amax is over the
                            // unquantized y of this call's own outputs only
                            if (row < M) {
                                uint32_t w[8];
#pragma unroll
                                for (int j = 0; j < 8; ++j) {
#pragma unroll
                                    for (int k = 0; k < 4; ++k)
                                        if (col0 + 4 * j + k < N) m_out = fmaxf(m_out, fabsf(y[4 * j + k]));
                                    w[j] = cvt_fp8x2(p.out_fmt, __fmul_rn(y[4 * j], s_out), __fmul_rn(y[4 * j + 1], s_out)) |
                                           (cvt_fp8x2(p.out_fmt, __fmul_rn(y[4 * j + 2], s_out),
                                                      __fmul_rn(y[4 * j + 3], s_out)) << 16);
                                }
                                uint8_t* dst = reinterpret_cast<uint8_t*>(out_base) + int64_t(b) * p.stride_c +
                                               int64_t(row) * N + col0;
                                if (vec_store && col0 + 32 <= N) {
                                    reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
                                    reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
                                } else {
#pragma unroll
                                    for (int i = 0; i < 32; ++i)
                                        if (col0 + i < N) dst[i] = uint8_t(w[i >> 2] >> (8 * (i & 3)));
                                }
                            }
                        } else if (tma_store) {
                            // the 128 x 32 bf16 block goes to the staging tile whose last
                            // store is known to have read it (64-byte swizzle: 16-byte
                            // piece j of row r at (j ^ (r / 2 mod 4)) * 16, so the 8
                            // lanes of a store phase hit distinct banks); then one TMA
                            // store, which clips the M / N tails of the output
                            const uint32_t stg = stg0 + uint32_t(n_st % L::kStgBufs) * L::kStgBytes;
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                const uint32_t addr = stg + row_in_tile * 64 + ((j ^ ((row_in_tile >> 1) & 3)) << 4);
                                asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr),
                                             "r"(pack_bf16x2(y[8 * j + 0], y[8 * j + 1])),
                                             "r"(pack_bf16x2(y[8 * j + 2], y[8 * j + 3])),
                                             "r"(pack_bf16x2(y[8 * j + 4], y[8 * j + 5])),
                                             "r"(pack_bf16x2(y[8 * j + 6], y[8 * j + 7]))
                                             : "memory");
                            }
                            fence_proxy_async_smem();
                            // the store two blocks back has read its tile, which the next
                            // block reuses (only the newest store may still be reading);
                            // the barrier publishes that and this block
                            if (store_lead) bulk_wait_read<L::kStgPending>();
                            epilogue_bar();
                            if (store_lead) {
                                tma_store_3d(map_c, stg, col0, m0, b);
                                bulk_commit();
                            }
                            ++n_st;
                        } else if (row < M) {
                            if (vec_store && col0 + 32 <= N) {
                                uint4* dst = reinterpret_cast<uint4*>(orow + col0);
#pragma unroll
                                for (int v = 0; v < 4; ++v) {
                                    uint4 x;
                                    x.x = pack_bf16x2(y[8 * v + 0], y[8 * v + 1]);
                                    x.y = pack_bf16x2(y[8 * v + 2], y[8 * v + 3]);
                                    x.z = pack_bf16x2(y[8 * v + 4], y[8 * v + 5]);
                                    x.w = pack_bf16x2(y[8 * v + 6], y[8 * v + 7]);
                                    dst[v] = x;
                                }
                            } else {
#pragma unroll
                                for (int i = 0; i < 32; i += 2) {
                                    const uint32_t x = pack_bf16x2(y[i], y[i + 1]);
                                    if (col0 + i < N) orow[col0 + i] = uint16_t(x & 0xFFFFu);
                                    if (col0 + i + 1 < N) orow[col0 + i + 1] = uint16_t(x >> 16);
                                }
                            }
                        }
                    }
                }
                tc_fence_before();
                // release the accumulator to the MMA issuer (the pair's leader)
                if (CTAS == 1) mbar_arrive(bar_tempty + 8 * buf);
                else           mbar_arrive_cluster(map_to_rank(bar_tempty + 8 * buf, 0));
            }
            // the staging tiles must outlive the stores that read them; the global
            // writes themselves complete with the grid (a dependent kernel's
            // griddepcontrol.wait and stream order both see them)
            if ((GROUP || tma_store) && store_lead) bulk_wait_read<0>();
            if constexpr (OUT8) {
                out8_finish<kEpiThreads>(p, m_out, s_bias, warp, lane, etid);
            }
        }
    }

    tc_fence_before();
    __syncthreads();
    if (CTAS == 2) cluster_sync();  // neither CTA leaves while the other may still signal it
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<CTAS>(tmem_base, L::kTmemCols);
    }
}

// ------------------------------------------------------------- host side ---

// Reads and clears this source file's device error word on the current device.
inline bool take_error_word(uint32_t* v) {
    if (cudaMemcpyFromSymbol(v, g_device_error, sizeof(*v)) != cudaSuccess) return false;
    const uint32_t zero = 0;
    return *v == 0 || cudaMemcpyToSymbol(g_device_error, &zero, sizeof(zero)) == cudaSuccess;
}

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                   const cuuint64_t*, const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave,
                                   CUtensorMapSwizzle, CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
    static EncodeTiledFn fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<EncodeTiledFn>(f);
    });
    return fn;
}

// 3-D map over uint8 codes: (inner, outer, batch) with a 128-byte swizzle.
// A broadcast operand (batch stride 0) gets a batch extent of 1.
bool make_map(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer, uint64_t batch,
              uint64_t batch_stride_bytes, uint32_t box_inner, uint32_t box_outer) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    const uint64_t pitch = inner;
    if (batch_stride_bytes == 0) {
        batch = 1;
        batch_stride_bytes = ((pitch * outer + 15) / 16) * 16;
    }
    cuuint64_t dims[3] = {inner, outer, batch};
    cuuint64_t strides[2] = {pitch, batch_stride_bytes};
    cuuint32_t box[3] = {box_inner, box_outer, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// 3-D map over the bf16 output (N, M, batch), 32-column x 128-row boxes with
// a 64-byte swizzle matching the epilogue's staging tiles (32 rows for a warp
// of an activation epilogue).
bool make_out_map(CUtensorMap* map, void* base, uint64_t n, uint64_t m, uint64_t batch, uint64_t batch_stride_bytes,
                  uint32_t box_rows = BM) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    if (batch <= 1 || batch_stride_bytes == 0) {
        batch = 1;
        batch_stride_bytes = ((n * m * 2 + 15) / 16) * 16;
    }
    cuuint64_t dims[3] = {n, m, batch};
    cuuint64_t strides[2] = {n * 2, batch_stride_bytes};
    cuuint32_t box[3] = {32, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_64B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

// 3-D map over FP8 output codes (N, M, batch), 32-column x 32-row boxes with
// a 32-byte swizzle.
bool make_out8_map(CUtensorMap* map, void* base, uint64_t n, uint64_t m, uint64_t batch, uint64_t batch_stride) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    if (batch <= 1 || batch_stride == 0) {
        batch = 1;
        batch_stride = (n * m + 15) / 16 * 16;
    }
    cuuint64_t dims[3] = {n, m, batch};
    cuuint64_t strides[2] = {n, batch_stride};
    cuuint32_t box[3] = {32, 32, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, base, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
              CU_TENSOR_MAP_SWIZZLE_32B, CU_TENSOR_MAP_L2_PROMOTION_NONE, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
           CUDA_SUCCESS;
}

struct HostArgs {
    int fa, fb;
    const void* b8;
    int64_t batch, stride_b;
};

template <int BN, bool A_MN, bool B_MN, int STAGES, bool HAS_BIAS, int CTAS, bool SPLIT, bool SWAP, bool OUT8,
          bool EP = false>
fp8_status launch_one(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, GemmParams p,
                      const HostArgs& h, cudaStream_t st, const EpArgs<EP>& ep = {}) {
    using L = Smem<BN, STAGES, CTAS, EP ? 4 : 3>;
    auto kern = fp8_gemm_kernel<BN, A_MN, B_MN, STAGES, HAS_BIAS, CTAS, SPLIT, SWAP, OUT8, false, EP>;
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc) != cudaSuccess)
            return FP8_ERR_CUDA;
        attr_set[dev] = true;
    }
    p.idesc = sm100::instr_desc_f8(h.fa, h.fb, A_MN ? 1 : 0, B_MN ? 1 : 0, BM * CTAS, BN);
    p.m_tiles = (p.M + BM * CTAS - 1) / (BM * CTAS);
    p.n_tiles = (p.N + BN - 1) / BN;
    const int64_t tiles = int64_t(p.m_tiles) * p.n_tiles * h.batch;
    p.total_tiles = int(tiles);
    p.group_m = CTAS == 2 ? 8 : 16;  // about sqrt(concurrent tiles) rows per group
    p.kb_per = (p.k_blocks + p.split - 1) / p.split;
    const int64_t work = tiles * p.split;
    p.total_units = int(work);
    const int64_t units_max = sm_count() / CTAS;
    const int units = int(work < units_max ? work : units_max);
    // a cluster split runs each tile's splits as one cluster (every unit in
    // the grid's one round, so the grid is a whole number of clusters)
    const int cluster = p.csplit ? p.split : CTAS;
    return launch_pdl(kern, units * CTAS, 64 + epi_threads(EP, SWAP), L::kAlloc, st, cluster, ta, tb, tc, p,
                      GroupTab<false>{}, ep);
}

template <int BN, bool A_MN, bool B_MN, int STAGES, int CTAS, bool SWAP = false, bool OUT8 = false, bool EP = false>
fp8_status launch(const CUtensorMap& ta, const CUtensorMap& tb, GemmParams p, const HostArgs& h, cudaStream_t st,
                  const EpArgs<EP>& ep = {}) {
    CUtensorMap tc = {};
    if (p.tma_store && !(EP && OUT8 ? make_out8_map(&tc, p.out, p.N, p.M, h.batch, uint64_t(p.stride_c))
                                    : make_out_map(&tc, p.out, p.N, p.M, h.batch, uint64_t(p.stride_c) * 2,
                                                   EP ? 32 : BM)))
        return FP8_ERR_CUDA;
    if constexpr (EP) {  // always with bias slots; only a swapped problem splits (as a cluster)
        if constexpr (SWAP) {
            if (p.split > 1)
                return launch_one<BN, A_MN, B_MN, STAGES, true, CTAS, true, SWAP, false, true>(ta, tb, tc, p, h, st, ep);
        }
        return launch_one<BN, A_MN, B_MN, STAGES, true, CTAS, false, SWAP, OUT8, true>(ta, tb, tc, p, h, st, ep);
    } else if constexpr (OUT8) {  // no split, no swap
        return p.bias_kind ? launch_one<BN, A_MN, B_MN, STAGES, true, CTAS, false, false, true>(ta, tb, tc, p, h, st)
                           : launch_one<BN, A_MN, B_MN, STAGES, false, CTAS, false, false, true>(ta, tb, tc, p, h, st);
    } else {
        if (p.split > 1)
            return p.bias_kind
                       ? launch_one<BN, A_MN, B_MN, STAGES, true, CTAS, true, SWAP, false>(ta, tb, tc, p, h, st)
                       : launch_one<BN, A_MN, B_MN, STAGES, false, CTAS, true, SWAP, false>(ta, tb, tc, p, h, st);
        return p.bias_kind ? launch_one<BN, A_MN, B_MN, STAGES, true, CTAS, false, SWAP, false>(ta, tb, tc, p, h, st)
                           : launch_one<BN, A_MN, B_MN, STAGES, false, CTAS, false, SWAP, false>(ta, tb, tc, p, h, st);
    }
}

// Tile choice for 148 SMs by a small cost model: a persistent grid walks
// ceil(units / CTAs) rounds of work units, each costing its k-blocks times
// the per-k-block time of that tile shape, plus the one epilogue left exposed
// at the end. The per-k-block and epilogue constants were fitted on B200 to
// this kernel: 128x256 0.48, 128x128 0.40, 128x64 0.30 and an SM pair's
// 256x256 0.43. While its tensor core runs, an SM takes in operands at about
// 65 bytes per clock, so a one-SM k-block costs more than its MMAs (a
// 128 x 128 k-block loads 32 KB for half the MMA work of a 128 x 256 one,
// which loads 48 KB), and the wider tile costs less per output. Pairs of
// 256 x 256 are used only with at least one such tile per SM (below that
// their coarser grain loses) and at least 16 k-blocks: with 4 or 8 (K = 512,
// 1024) each CTA's 128 x 256 epilogue outlasts its main loop and pairs lost
// to one SM's 128 x 256 on every shape measured (4096^2 x 1024 18.9 against
// 20.4 us, 64 x 512^3 16.2 against 19.3), while from 16 on they won
// (4096^2 x 2048 28.5 against 31.0). The pair's 256 x 128 tile (24 KB per SM per
// k-block) measured slower than one SM's 128 x 128 on the shapes it could
// serve and is not chosen.
//
// Split K (split_req >= 2, with a workspace): a tile becomes `split` units
// over consecutive k-block ranges; the unit that finishes last adds the
// others' fp32 partials and runs the epilogue. The automatic choice
// (split_req = 0) does not split these unswapped tiles: on every shape
// measured on B200 the partials' round trip through L2 cost more than the
// shorter main loop saved (short problems, swapped below, do split).
constexpr size_t kSplitCntBytes = 4096;  // two counters per (tile, CTA of the tile)
constexpr int kMaxSplit = 4;

struct TileChoice {
    bool pair;
    int bn;
    int split;  // 0: the requested split is not possible for this problem
};

inline size_t split_ws_bytes(int64_t tiles, int ctas, int bn, int split) {
    return kSplitCntBytes + size_t(tiles) * ctas * split * BM * bn * sizeof(float);
}

inline int64_t tile_count(int64_t M, int64_t N, int64_t batch, bool pair, int bn) {
    const int64_t rows = BM * (pair ? 2 : 1);
    return ((M + rows - 1) / rows) * ((N + bn - 1) / bn) * batch;
}

inline TileChoice choose_tile(int64_t M, int64_t N, int64_t K, int64_t batch, bool b_mn, int64_t sms,
                              int split_req) {
    const int64_t kb = (K + BK - 1) / BK;
    const int split = split_req < 2 ? 1 : split_req;
    const int64_t kb_per = (kb + split - 1) / split;
    if (split > 1 && (split - 1) * kb_per >= kb) return {false, 256, 0};  // every unit needs k-blocks
    auto cost = [&](bool pair, int bn, double t_k, double t_epi) {
        const int ctas = pair ? 2 : 1;
        const int64_t units = sms / ctas;
        const int64_t tiles = tile_count(M, N, batch, pair, bn);
        if (split > 1 && size_t(tiles) * ctas * 2 * sizeof(uint32_t) > kSplitCntBytes) return 1e30;
        const int64_t rounds = (tiles * split + units - 1) / units;
        return double(rounds) * double(kb_per) * t_k + t_epi;
    };
    if (split == 1 && M > BM && N > 128 && kb >= 16 && tile_count(M, N, batch, true, 256) >= sms)
        return {true, 256, 1};
    const bool pair_ok = M > BM;  // a pair's second CTA would hold only padding otherwise
    const TileChoice c[4] = {{false, 256, split}, {false, 128, split}, {false, 64, split}, {true, 256, split}};
    const double t[4] = {cost(false, 256, 0.48, 2.0), cost(false, 128, 0.40, 1.0),
                         b_mn ? 1e30 : cost(false, 64, 0.30, 0.5),
                         (split > 1 && pair_ok && N > 128) ? cost(true, 256, 0.43, 2.0) : 1e30};
    TileChoice best = {false, 256, 0};
    double best_cost = 1e30;
    for (int i = 0; i < 4; ++i)
        if (t[i] < best_cost) { best = c[i]; best_cost = t[i]; }
    // With at most 4 k-blocks a 128 x 256 tile's epilogue (about 2.1 us)
    // outlasts its main loop while a 128 x 128 tile's (about 1.1 us) does not,
    // so the rounds times the epilogue decide between the two widths. Measured
    // on B200 over ten such shapes, this picks the faster of them in every case
    // with a clear difference: 128 for 64 x 512^3 (15.1 us against 16.2) and
    // 4096^2 x 512 (14.1 against 14.7), 256 for 2048^2 x 256 (5.4 against 5.6)
    // and 4096 x 2048 x 128 (7.1 against 7.9), among others.
    if (!best.pair && (best.bn == 256 || best.bn == 128) && split == 1 && kb <= 4) {
        const int64_t r256 = (tile_count(M, N, batch, false, 256) + sms - 1) / sms;
        const int64_t r128 = (tile_count(M, N, batch, false, 128) + sms - 1) / sms;
        best = {false, double(r128) * 1.1 < double(r256) * 2.1 ? 128 : 256, 1};
    }
    return best;
}

template <bool A_MN, bool B_MN, bool OUT8 = false, bool EP = false>
fp8_status dispatch(const CUtensorMap& ta, GemmParams p, const HostArgs& h, void* ws, size_t ws_bytes,
                    int split_req, cudaStream_t st, const EpArgs<EP>& ep = {}) {
    const TileChoice tc = choose_tile(p.M, p.N, p.K, h.batch, B_MN, sm_count(), split_req);
    if (tc.split == 0) return FP8_ERR_UNSUPPORTED;
    const bool pair = tc.pair;
    const int bn = tc.bn;
    p.split = tc.split;
    if (tc.split > 1) {
        const int64_t tiles = tile_count(p.M, p.N, h.batch, pair, bn);
        if (!ws || ws_bytes < split_ws_bytes(tiles, pair ? 2 : 1, bn, tc.split)) return FP8_ERR_INVALID_ARG;
        p.ws_cnt = static_cast<uint32_t*>(ws);
        p.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kSplitCntBytes);
    }
    CUtensorMap tb;
    const uint64_t sb_bytes = uint64_t(h.stride_b);
    const uint32_t b_box_n = pair ? bn / 2 : bn;  // N extent one CTA loads
    const bool ok = B_MN ? make_map(&tb, h.b8, p.N, p.K, h.batch, sb_bytes, 128, BK)
                         : make_map(&tb, h.b8, p.K, p.N, h.batch, sb_bytes, BK, b_box_n);
    if (!ok) return FP8_ERR_CUDA;
    if (pair) return launch<256, A_MN, B_MN, 6, 2, false, OUT8, EP>(ta, tb, p, h, st, ep);
    if (bn == 256) return launch<256, A_MN, B_MN, 4, 1, false, OUT8, EP>(ta, tb, p, h, st, ep);
    if (bn == 128) return launch<128, A_MN, B_MN, 6, 1, false, OUT8, EP>(ta, tb, p, h, st, ep);
    if constexpr (!B_MN) return launch<64, A_MN, B_MN, 8, 1, false, OUT8, EP>(ta, tb, p, h, st, ep);
    return FP8_ERR_UNSUPPORTED;
}

// Swapped operands for short problems (M <= 32, N >= 128, NT or NN): the
// kernel computes C^T = B^T A^T, so that C's N runs along the tensor core's
// 128-row M and C's few rows become an MMA N of 16 or 32; the epilogue
// writes C transposed. (TN is excluded: its A would become an MN-major B
// operand narrower than a 128-byte swizzle atom. From 33 rows on, the
// unswapped 128 x 64 tile was as fast or faster on B200: at 64 x 8192 x 2048
// it keeps 128 SMs busy where the swapped 128 x 64 tiles keep 64.)
inline bool swap_ab(int64_t M, int64_t N, fp8_layout layout) {
    return M <= 32 && N >= 128 && layout != FP8_TN;
}

inline int swap_bn(int64_t M) { return M <= 16 ? 16 : 32; }

// The split a swapped problem takes (0: the requested split is impossible).
// Automatic (split_req 0): few 128-column tiles with a long K leave most SMs
// idle, and their partials are small (128 x 16..64 fp32), so splitting pays
// where the main loop it saves exceeds the fix-up: about 0.28 us per k-block
// saved against 2.2 + 0.02 * BN * split us, with every unit in one round (both
// constants measured on B200 over 1, 8, 16, 32 and 64-row problems).
inline int swap_split(int64_t M, int64_t N, int64_t K, int64_t batch, int split_req, int64_t sms) {
    const int64_t kb = (K + BK - 1) / BK;
    const int64_t tiles = ((N + BM - 1) / BM) * batch;
    auto possible = [&](int s) {
        const int64_t kb_per = (kb + s - 1) / s;
        return (s - 1) * kb_per < kb && size_t(tiles) * 2 * sizeof(uint32_t) <= kSplitCntBytes;
    };
    if (split_req == 1) return 1;
    if (split_req >= 2) return possible(split_req) ? split_req : 0;
    const int bn = swap_bn(M);
    int best = 1;
    double best_gain = 0.0;
    for (int s = 2; s <= kMaxSplit; ++s) {
        if (!possible(s) || tiles * s > sms) continue;
        const double gain = double(kb - (kb + s - 1) / s) * 0.28 - (2.2 + 0.02 * bn * s);
        if (gain > best_gain) { best = s; best_gain = gain; }
    }
    return best;
}

template <bool A_MN, bool EP = false>
fp8_status dispatch_swap(const uint8_t* a8, int fa, const uint8_t* b8, int fb, int64_t M, int64_t N, int64_t K,
                         int64_t batch, int64_t stride_a, int64_t stride_b, GemmParams p, void* ws, size_t ws_bytes,
                         int split_req, cudaStream_t st, const EpArgs<EP>& ep = {}) {
    const int bn = swap_bn(M);
    // The automatic choice without a workspace splits as a cluster: the
    // splits' partials go through split 0's staging area, which holds three
    // 128 x 16 partials or one 128 x 32 one.
    p.csplit = 0;
    if (split_req == 0 && !ws) {
        const int s_max = bn == 16 ? 4 : 2;
        int s = swap_split(M, N, K, batch, 0, sm_count());
        s = s > s_max ? s_max : s;
        p.split = s;
        p.csplit = s > 1;
    } else {
        p.split = swap_split(M, N, K, batch, split_req, sm_count());
    }
    if (p.split == 0) return FP8_ERR_UNSUPPORTED;
    if (p.split > 1 && !p.csplit) {
        const int64_t tiles = ((N + BM - 1) / BM) * batch;
        if (!ws || ws_bytes < split_ws_bytes(tiles, 1, bn, p.split)) {
            if (split_req >= 2) return FP8_ERR_INVALID_ARG;
            p.split = 1;  // an automatic split that does not fit the workspace is dropped
        }
    }
    if (p.split > 1 && !p.csplit) {
        p.ws_cnt = static_cast<uint32_t*>(ws);
        p.ws = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kSplitCntBytes);
    }
    // the kernel's problem: M' = N rows of A' = B, N' = M columns of B' = A
    p.M = int(N);
    p.N = int(M);
    p.a_bcast = stride_b == 0;
    p.b_bcast = stride_a == 0;
    p.tma_store = 0;
    p.vec_store = 0;
    CUtensorMap ta, tb;
    const bool ok_a = A_MN ? make_map(&ta, b8, N, K, batch, uint64_t(stride_b), 128, BK)
                           : make_map(&ta, b8, K, N, batch, uint64_t(stride_b), BK, BM);
    const bool ok_b = make_map(&tb, a8, K, M, batch, uint64_t(stride_a), BK, uint32_t(bn));
    if (!ok_a || !ok_b) return FP8_ERR_CUDA;
    const HostArgs h = {fb, fa, a8, batch, stride_a};
    if (bn == 16) return launch<16, A_MN, false, 10, 1, true, false, EP>(ta, tb, p, h, st, ep);
    return launch<32, A_MN, false, 9, 1, true, false, EP>(ta, tb, p, h, st, ep);
}

// The argument checks that every single-problem entry point shares. out_align:
// bytes that the output must be aligned to.
inline fp8_status check_mm(const void* a8, int fa, const void* b8, int fb, const float* sa, const float* sb, int layout,
                           int64_t M, int64_t N, int64_t K, int64_t batch, int64_t stride_a, int64_t stride_b,
                           int64_t stride_c, const void* bias, const float* bias_scale, int bias_fmt, const void* out,
                           int out_align) {
    if (!valid_fmt(fa) || !valid_fmt(fb)) return FP8_ERR_INVALID_ARG;
    if (layout != FP8_NT && layout != FP8_NN && layout != FP8_TN) return FP8_ERR_INVALID_ARG;
    if (!a8 || !b8 || !sa || !sb || !out) return FP8_ERR_INVALID_ARG;
    if (M < 1 || N < 1 || K < 1 || batch < 1) return FP8_ERR_INVALID_ARG;
    if (stride_a < 0 || stride_b < 0 || stride_c < 0) return FP8_ERR_INVALID_ARG;
    if (bias_scale && !bias) return FP8_ERR_INVALID_ARG;
    if (bias && bias_scale && !valid_fmt(bias_fmt)) return FP8_ERR_INVALID_ARG;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31) ||
        batch >= (int64_t(1) << 31))
        return FP8_ERR_UNSUPPORTED;
    if (batch > 1 && stride_c < M * N) return FP8_ERR_INVALID_ARG;
    const int64_t tiles = ((M + BM - 1) / BM) * ((N + 63) / 64) * batch;
    if (tiles >= (int64_t(1) << 31)) return FP8_ERR_UNSUPPORTED;
    // contiguous extent of each operand = TMA row pitch in bytes
    if ((layout == FP8_TN ? M : K) % 16 != 0 || (layout != FP8_NT ? N : K) % 16 != 0) return FP8_ERR_ALIGNMENT;
    if (!aligned(a8, 16) || !aligned(b8, 16)) return FP8_ERR_ALIGNMENT;
    if (stride_a % 16 != 0 || stride_b % 16 != 0) return FP8_ERR_ALIGNMENT;
    if (!aligned(out, out_align) || !aligned(sa, 4) || !aligned(sb, 4)) return FP8_ERR_ALIGNMENT;
    if (bias && !bias_scale && !aligned(bias, 2)) return FP8_ERR_ALIGNMENT;
    return FP8_OK;
}

}  // namespace
}  // namespace fp8lite
