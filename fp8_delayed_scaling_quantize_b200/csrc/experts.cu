// FP8 products grouped by expert: the rows of a token-sorted matrix belong to
// experts in turn, expert e's being [offsets[e], offsets[e+1]), and every
// expert has its own weight. The offsets live on the device: the host knows
// the total and the number of experts only, and nothing is synchronised.
//
//   NT, NN   out[r] = act(A[r] op(B[e]) / (sa sb_e) + bias_e),  r in e's rows
//   TN       out[e] = A[rows of e]^T B[rows of e] / (sa sb)
//
// Bound by what moves rather than by the MMAs: an SM takes 48 KB for a 128 x 256
// tile's k-block, and few k-blocks stand against the output's bytes. Measured on
// B200 (16384 rows to 32 experts of 4096 x 1024, unequal): NT with SiLU and
// preact 102-104 us, 403 MB at 3.9 TB/s of which 268 written (without either 88
// us), NN 70 us, 0.60 of the FP8 rate, TN 98 us, 268 of 352 MB written (the same
// stores alone reach 4.7 TB/s, 57 us); 64 of 80 rows to 64 experts of 2048 x 1024
// 16.5 us, 7 TB/s as counted, each weight read once.
//
// One persistent launch. Each warp of a CTA works out from the offsets which
// expert a unit belongs to (struct Experts) and walks the CTA's share of the
// units; the roles, pipeline and epilogue are those of gemm_kernel.cuh.
//
//  * A tile that reaches past its expert's last row loads the next expert's
//    rows too; their results are dropped at the store, which writes such a
//    tile in 16-byte row pieces and a whole tile by TMA.
//  * In TN the rows are the contraction, and an expert's last block of 128 may
//    hold rows of the next one. Of a block of t < 128 rows only the ceil(t / 32)
//    MMA slices (32 rows each) that hold rows of the expert are issued, and the
//    MMA warp first clears the last slice's other rows in shared memory, in
//    both operands: a NaN code in either would reach the sum through a zero.
//  * Few rows an expert (swapped): the weight's columns run along the tensor
//    core's 128 rows and 16 or 32 token rows are its N, so that a weight tile
//    is read once for all of them and no operand is padded to 128 tokens.

#include "gemm_kernel.cuh"

#include "errors.h"

using namespace fp8lite;

namespace fp8lite {

bool experts_error(uint32_t* v) { return take_error_word(v); }

namespace {

constexpr int kMaxExperts = FP8_MM_MAX_EXPERTS;

enum ExpertKind { kRowsNT = 0, kRowsNN = 1, kSumTN = 2 };

struct ExpertParams {
    const int32_t* offsets;
    int experts, rows;  // rows: of the token matrices
    int M, N, K;        // of one output (ROWS: M unused; SUM: K unused)
    int m_tiles, n_tiles, k_blocks;
    uint32_t idesc;
    const float* sa;
    const float* sb;
    int sb_stride;
    const uint16_t* bias;
    int act;
    uint16_t* preact;
    uint16_t* out;
    int fast;  // N and the pointers allow 16-byte accesses and TMA stores
};

// One tile of work.
struct Item {
    int e;          // expert
    int m0, m_end;  // ROWS: first row of the tile and the expert's end; SUM: first row of the tile in the output, M
    int n0;         // first output column (swapped: of 128)
    int kbs;        // k-blocks
    int k_row, k_end;  // SUM: the expert's rows
};

// Where the experts' rows begin and end, looked up by a whole warp (every lane
// calls every function, with the same arguments). A lane stands for `per`
// consecutive experts and knows the tiles before them, so that a lookup is a
// ballot over the lanes and one over the experts of the lane found, whose
// offsets come from L1 then: no table in shared memory, and no block barrier
// before the first load. Offsets are limited to [0, rows] and to no less than
// the one before (a running maximum), so that no offsets lead an access out
// of the matrices.
template <int TILE>  // rows of a tile
struct Experts {
    const int32_t* offsets;
    int experts, rows, per, lane;
    int before;  // maximum of the offsets before this lane's
    int tiles;   // tiles up to and with this lane's experts
    int mine;    // this lane's
    // the expert found last: its tiles [t0, t1), units [u0, u1) and rows [lo, hi)
    int e, t0, t1, u0, u1, lo, hi;

    __device__ __forceinline__ int at(int i) const { return min(max(__ldg(offsets + min(i, experts)), 0), rows); }
    __device__ __forceinline__ static int count(int lo, int hi) { return (hi - lo + TILE - 1) / TILE; }

    __device__ __forceinline__ void init(const ExpertParams& p) {
        offsets = p.offsets;
        experts = p.experts;
        rows = p.rows;
        per = (experts + 31) / 32;
        lane = threadIdx.x & 31;
        e = -1;
        t0 = t1 = u0 = u1 = 0;
        const int first = lane * per;
        int m = 0;
        for (int i = 0; i < per; ++i) m = max(m, at(first + i));
        before = __shfl_up_sync(0xffffffffu, m, 1);
        if (lane == 0) before = 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before = max(before, v);
        }
        mine = 0;
        int prev = max(before, at(first));
        for (int i = 0; i < per; ++i) {  // past the last expert at() repeats the last offset: no tiles
            const int next = max(prev, at(first + i + 1));
            mine += count(prev, next);
            prev = next;
        }
        tiles = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, tiles, o);
            if (lane >= o) tiles += v;
        }
    }

    __device__ __forceinline__ int total() const { return __shfl_sync(0xffffffffu, tiles, 31); }

    // Offsets of the experts of lane `l`: lane j gets [v, next) of expert l * per + j.
    __device__ __forceinline__ void group(int l, int& v, int& next) const {
        v = max(at(l * per + min(lane, per)), __shfl_sync(0xffffffffu, before, l));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o) v = max(v, w);
        }
        next = __shfl_down_sync(0xffffffffu, v, 1);
        if (lane >= per) next = v;
    }

    // The expert that unit u belongs to, `per_tile` units to a tile.
    __device__ __forceinline__ void find_unit(int u, int per_tile) {
        if (u >= u0 && u < u1) return;
        const int t = u / per_tile;
        const int l = __ffs(__ballot_sync(0xffffffffu, tiles > t)) - 1;
        const int base = __shfl_sync(0xffffffffu, tiles - mine, l);
        int v, next;
        group(l, v, next);
        const int n = count(v, next);
        int sum = n;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int w = __shfl_up_sync(0xffffffffu, sum, o);
            if (lane >= o) sum += w;
        }
        const int k = __ffs(__ballot_sync(0xffffffffu, base + sum > t)) - 1;
        e = l * per + k;
        lo = __shfl_sync(0xffffffffu, v, k);
        hi = __shfl_sync(0xffffffffu, next, k);
        t1 = base + __shfl_sync(0xffffffffu, sum, k);
        t0 = t1 - __shfl_sync(0xffffffffu, n, k);
        u0 = t0 * per_tile;
        u1 = t1 * per_tile;
    }

    // The same where every expert has `per_expert` units.
    __device__ __forceinline__ void find_expert(int u, int per_expert) {
        if (u >= u0 && u < u1) return;
        const int x = u / per_expert;
        int v, next;
        group(x / per, v, next);
        e = x;
        u0 = x * per_expert;
        u1 = u0 + per_expert;
        lo = __shfl_sync(0xffffffffu, v, x % per);
        hi = __shfl_sync(0xffffffffu, next, x % per);
    }
};

// Work unit u.
template <int BN, int KIND, bool SWAP, int TILE>
__device__ __forceinline__ Item item_of(Experts<TILE>& x, const ExpertParams& p, int u) {
    Item it;
    int mb, nb, b;
    if constexpr (KIND == kSumTN) {
        x.find_expert(u, p.m_tiles * p.n_tiles);
        tile_coords_lazy(u - x.u0, TileWalk{p.m_tiles, p.n_tiles, 16}, mb, nb, b);
        it.m0 = mb * TILE;
        it.m_end = p.M;
        it.n0 = nb * BN;
        it.k_row = x.lo;
        it.k_end = x.hi;
        it.kbs = (x.hi - x.lo + BK - 1) / BK;
    } else {
        x.find_unit(u, p.n_tiles);
        if constexpr (SWAP) {
            nb = (u - x.u0) / (x.t1 - x.t0);  // the row tiles of one weight tile one after the other
            mb = u - x.u0 - nb * (x.t1 - x.t0);
            it.n0 = nb * BM;
        } else {
            tile_coords_lazy(u - x.u0, TileWalk{x.t1 - x.t0, p.n_tiles, 16}, mb, nb, b);
            it.n0 = nb * BN;
        }
        it.m0 = x.lo + mb * TILE;
        it.m_end = x.hi;
        it.k_row = it.k_end = 0;
        it.kbs = p.k_blocks;
    }
    it.e = x.e;
    return it;
}

constexpr int kSliceRows = 32;  // K of one MMA

// Rows [from, to) of a 128-column operand tile, 128 bytes each in shared
// memory (the swizzle stays within a row), become zeros: a whole warp.
__device__ __forceinline__ void clear_rows(uint8_t* tile, int from, int to, int lane) {
    for (int i = from * 128 + lane * 16; i < to * 128; i += 32 * 16)
        *reinterpret_cast<uint4*>(tile + i) = make_uint4(0u, 0u, 0u, 0u);
}

// KIND, SWAP: see the head of the file. BN: output columns of a tile, or
// token rows of a swapped one. CTAS = 2: a pair of CTAs on 256 x BN tiles
// (cta_group::2): each loads its 128 rows of A and half of B and writes its
// own 128 rows of the output, so an SM takes in a third less per MMA.
template <int BN, int KIND, int STAGES, bool SWAP, int CTAS>
__global__ void __maxnreg__(SWAP ? 168 : kActRegs)
expert_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_z, const ExpertParams p) {
    using L = Smem<BN, STAGES, CTAS, SWAP ? 3 : 4>;
    static_assert(CTAS == 1 || (BN == 256 && !SWAP), "a pair's half of an MN-major B is one 128-byte atom");
    static_assert(CTAS == 1 || KIND != kSumTN, "the leader's MMA warp could not clear the other CTA's rows");
    constexpr int ET = epi_threads(true, SWAP);
    constexpr int TILE = SWAP ? BN : BM * CTAS;
    // majors of the MMA's operands: K-major unless the stored rows run along K
    constexpr bool A_MN = SWAP ? KIND == kRowsNN : KIND == kSumTN;
    constexpr bool B_MN = !SWAP && KIND != kRowsNT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    if constexpr (L::kAct) {
        if (!smem_fits<L>(smem_raw, smem)) return;
    }
    const uint32_t s_a = smem_addr(smem);
    const uint32_t s_b = s_a + STAGES * L::kABytes;
    const uint32_t bar_full = s_a + L::kBarOffset;
    const uint32_t bar_empty = bar_full + STAGES * 8;
    const uint32_t bar_tfull = bar_empty + STAGES * 8;
    const uint32_t bar_tempty = bar_tfull + 2 * 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBarOffset + (2 * STAGES + 4) * 8);
    float* s_bias = reinterpret_cast<float*>(smem + L::kBiasOffset);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = CTAS == 2 ? cluster_ctarank() : 0u;  // 0 = the pair's leader
    const bool leader = rank == 0;
    const int unit0 = blockIdx.x / CTAS, unit_step = gridDim.x / CTAS;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, CTAS * ET);
        }
        fence_mbar_init();
        tma_prefetch(&tm_a);
        tma_prefetch(&tm_b);
        if (p.fast && !SWAP) {
            tma_prefetch(&tm_c);
            if (p.preact) tma_prefetch(&tm_z);
        }
    }
    if (warp == 1) {
        tmem_alloc<CTAS>(smem_addr(tmem_slot), L::kTmemCols);
        tmem_relinquish<CTAS>();
    }
    tc_fence_before();
    __syncthreads();
    if (CTAS == 2) cluster_sync();  // the pair's barriers exist before any remote arrive
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    griddep_wait();
    griddep_launch();
    Experts<TILE> x;
    x.init(p);
    const int units = KIND == kSumTN ? p.experts * p.m_tiles * p.n_tiles : x.total() * p.n_tiles;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer ---
        const bool issuer = elect_one();
        int stage = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = unit0; u < units && ok; u += unit_step) {
            const Item it = item_of<BN, KIND, SWAP>(x, p, u);
            for (int kb = 0; kb < it.kbs; ++kb) {
                if (!wait_bounded_warp(bar_empty + 8 * stage, phase ^ 1)) { ok = false; break; }
                const uint32_t full = bar_full + 8 * stage;
                const uint32_t da = s_a + stage * L::kABytes, db = s_b + stage * L::kBBytes;
                if (issuer) {
                    if (leader) mbar_arrive_expect_tx(full, uint32_t(L::kStageTx));
                    // a pair's loads complete on the leader's barrier
                    const uint32_t bar = CTAS == 2 ? map_to_rank(full, 0) : full;
                    auto load = [&](uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2) {
                        if (CTAS == 2) tma_load_3d_pair(dst, map, bar, c0, c1, c2);
                        else           tma_load_3d(dst, map, bar, c0, c1, c2);
                    };
                    constexpr int kAtoms = BN / CTAS / 128;  // 128-column atoms of an MN-major B
                    const int m0 = it.m0 + int(rank) * BM, n0 = it.n0 + int(rank) * (BN / CTAS);
                    if constexpr (KIND == kSumTN) {
                        const int first = it.k_row + kb * BK;
                        load(da, &tm_a, m0, first, 0);
#pragma unroll
                        for (int h = 0; h < kAtoms; ++h) load(db + h * 128 * BK, &tm_b, n0 + h * 128, first, 0);
                    } else if constexpr (SWAP) {
                        if (A_MN) load(da, &tm_b, it.n0, kb * BK, it.e);
                        else      load(da, &tm_b, kb * BK, it.n0, it.e);
                        load(db, &tm_a, kb * BK, it.m0, 0);
                    } else {
                        load(da, &tm_a, kb * BK, m0, 0);
                        if (B_MN) {
#pragma unroll
                            for (int h = 0; h < kAtoms; ++h) load(db + h * 128 * BK, &tm_b, n0 + h * 128, kb * BK, it.e);
                        } else {
                            load(db, &tm_b, kb * BK, n0, it.e);
                        }
                    }
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
        }
        // drain: wait until the MMAs released every stage still in use
        for (int i = 0; i < STAGES && ok; ++i) {
            if (!wait_bounded_warp(bar_empty + 8 * stage, phase ^ 1)) break;
            if (++stage == STAGES) { stage = 0; phase ^= 1; }
        }
    } else if (warp == 1) {
        // --------------------------------------------------- MMA issuer ---
        const bool issuer = elect_one();
        const uint64_t a_desc0 = A_MN ? smem_desc_sw128(s_a, 128 * BK, 1024) : smem_desc_sw128(s_a, 16, 1024);
        const uint64_t b_desc0 = B_MN ? smem_desc_sw128(s_b, 128 * BK, 1024) : smem_desc_sw128(s_b, 16, 1024);
        int stage = 0, done = 0;
        uint32_t phase = 0;
        bool ok = leader;  // a pair's MMAs are its leader's
        for (int u = unit0; u < units && ok; u += unit_step) {
            const Item it = item_of<BN, KIND, SWAP>(x, p, u);
            if (it.kbs == 0) continue;  // an expert without rows: the epilogue writes its zeros
            const int buf = done & 1;
            if (!wait_bounded_warp(bar_tempty + 8 * buf, ((done >> 1) & 1) ^ 1)) break;
            tc_fence_after();
            for (int kb = 0; kb < it.kbs; ++kb) {
                if (!wait_bounded_warp(bar_full + 8 * stage, phase)) { ok = false; break; }
                const uint64_t a_desc = a_desc0 + uint64_t(stage) * (L::kABytes >> 4);
                const uint64_t b_desc = b_desc0 + uint64_t(stage) * (L::kBBytes >> 4);
                int left = BK;  // SUM: the expert's rows in the block
                if constexpr (KIND == kSumTN) {
                    left = it.k_end - (it.k_row + kb * BK);
                    if (left < BK && left % kSliceRows != 0) {
                        const int to = (left + kSliceRows - 1) / kSliceRows * kSliceRows;
                        clear_rows(smem + stage * L::kABytes, left, to, lane);
#pragma unroll
                        for (int h = 0; h < BN / 128; ++h)
                            clear_rows(smem + STAGES * L::kABytes + stage * L::kBBytes + h * 128 * BK, left, to, lane);
                        fence_proxy_async_smem();
                        __syncwarp();
                    }
                }
                if (issuer) {
                    if (KIND == kSumTN && left < BK) {
                        for (int k = 0; k * kSliceRows < left; ++k)
                            mma_slice_f8f6f4(tmem_base + buf * BN, a_desc + uint64_t(k) * 256u, b_desc + uint64_t(k) * 256u,
                                             p.idesc, (kb | k) != 0);
                    } else {
                        mma_kblock_f8f6f4<CTAS>(tmem_base + buf * BN, a_desc, b_desc, A_MN ? 256u : 2u, B_MN ? 256u : 2u,
                                                p.idesc, kb != 0);
                    }
                    if (CTAS == 2) mma_commit_pair(bar_empty + 8 * stage);
                    else           mma_commit(bar_empty + 8 * stage);
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
            if (issuer) {
                if (CTAS == 2) mma_commit_pair(bar_tfull + 8 * buf);
                else           mma_commit(bar_tfull + 8 * buf);
            }
            __syncwarp();
            ++done;
        }
    } else {
        // ----------------------------------------------------- epilogue ---
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int row_in_tile = q * 32 + lane;
        const int phase = (warp - 2) >> 2;
        const uint32_t stg0 = s_a + L::kStgOffset;
        const float inv_a = 1.0f / __ldg(p.sa);
        int done = 0;
        float unused = 0.0f;
        ActResidual none;
        bool failed = false;
        if constexpr (!SWAP) s_bias[(warp - 2) * 32 + lane] = 0.0f;
        // what a unit needs from global memory is asked for one unit early
        Item next = {};
        float scale_next = 1.0f;
        constexpr int kBlocks = SWAP ? 1 : kActBlocks<BN>;
        float bias[kBlocks] = {}, bias_next[kBlocks] = {};  // this lane's column of each block (swapped: its column)
        auto ask = [&](int u) {
            next = item_of<BN, KIND, SWAP>(x, p, u);
            scale_next = __ldg(p.sb + int64_t(next.e) * p.sb_stride);
            if (!p.bias) return;
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) {
                const int col = next.n0 + (SWAP ? row_in_tile : (phase + i * kActPhases) * 32 + lane);
                bias_next[i] = col < p.N ? bf16_value(__ldg(p.bias + int64_t(next.e) * p.N + col)) : 0.0f;
            }
        };
        if (unit0 < units) ask(unit0);
        for (int u = unit0; u < units; u += unit_step) {
            const Item it = next;
            const float inv = inv_a * (1.0f / scale_next);
#pragma unroll
            for (int i = 0; i < kBlocks; ++i) bias[i] = bias_next[i];
            if (u + unit_step < units) ask(u + unit_step);
            const bool has = it.kbs > 0;
            const int buf = done & 1;
            if (has) {
                if (!failed) failed = !wait_bounded_warp(bar_tfull + 8 * buf, (done >> 1) & 1);
                if (failed) continue;  // the other warps find it out for themselves
                tc_fence_after();
            }
            const uint32_t t_row = tmem_base + (uint32_t(q * 32) << 16) + buf * BN;
            if constexpr (SWAP) {
                // TMEM lane: output column n0 + row_in_tile; accumulator columns: token rows
                const int col = it.n0 + row_in_tile;
#pragma unroll 1
                for (int c = 0; c < BN / 16; ++c) {
                    const int r0 = it.m0 + c * 16;
                    if (r0 >= it.m_end) break;
                    uint32_t r[16];
                    tmem_ld<16>(t_row + c * 16, r);
                    tmem_ld_wait();
                    float y[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) y[i] = fmaf(__uint_as_float(r[i]), inv, bias[0]);
                    if (col < p.N) {
                        const int64_t at = int64_t(r0) * p.N + col;
                        if (p.preact) {
#pragma unroll
                            for (int i = 0; i < 16; ++i)
                                if (r0 + i < it.m_end) p.preact[at + int64_t(i) * p.N] = bf16_bits(y[i]);
                        }
                        act_apply(p.act, y);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            if (r0 + i < it.m_end) p.out[at + int64_t(i) * p.N] = bf16_bits(y[i]);
                    }
                }
            } else {
                ActTile t;
                t.map_out = &tm_c;
                t.map_z = &tm_z;
                t.out = KIND == kSumTN ? p.out + int64_t(it.e) * p.M * p.N : p.out;
                t.preact = p.preact;
                t.residual = nullptr;
                t.s_bias = s_bias + (warp - 2) * 32;
                t.has_bias = KIND != kSumTN && p.bias != nullptr;
                t.t_row = t_row;
                t.stg = stg0 + uint32_t(warp - 2) * 2048u;
                t.inv = inv;
                t.s_out = 1.0f;
                t.act = p.act;
                t.out_fmt = 0;
                t.row0 = it.m0 + int(rank) * BM + q * 32;
                t.m_end = it.m_end;
                t.col_first = it.n0;
                t.N = p.N;
                t.b = KIND == kSumTN ? it.e : 0;
                // a warp whose rows end inside its 32 writes them row by row
                t.tma_out = t.tma_z = p.fast && (KIND == kSumTN || t.row0 + 32 <= it.m_end);
                t.vec_out = t.vec_z = p.fast;
                t.has = has;
                if constexpr (KIND == kSumTN) {
                    if (t.row0 < t.m_end) act_blocks<BN, FP8_ACT_NONE, false>(t, none, bias, unused, phase, lane);
                } else {
                    act_tile<BN, false>(t, none, bias, unused, phase, lane);
                }
            }
            if (has) {
                tc_fence_before();
                if (CTAS == 2) mbar_arrive_cluster(map_to_rank(bar_tempty + 8 * buf, 0));
                else           mbar_arrive(bar_tempty + 8 * buf);
                ++done;
            }
        }
        if (!SWAP && lane == 0) bulk_wait_read<0>();  // the staging tiles outlive the stores that read them
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

// Zeros in the rows of no expert: where the offsets leave none, as they mostly
// do, the launch reads two offsets and ends (16384 x 4096: 1.1 us where
// writing all rows takes 34). Otherwise the rows end at the largest offset: it
// is offsets[experts] unless they decrease, and where the products end then.
__global__ void zero_rest_kernel(uint4* out, int64_t rows, int64_t pitch, const int32_t* offsets, int experts) {
    griddep_wait();
    griddep_launch();
    const int end = int(rows);
    const int64_t lo = min(max(__ldg(offsets), 0), end);
    int top = min(max(__ldg(offsets + experts), 0), end);
    if (lo == 0 && top == end) return;
#pragma unroll 4
    for (int i = threadIdx.x & 31; i < experts; i += 32) top = max(top, min(__ldg(offsets + i), end));
    const int64_t hi = __reduce_max_sync(0xffffffffu, top);
    const int64_t before = lo * pitch, n = before + (rows - hi) * pitch;
    for (int64_t i = int64_t(blockIdx.x) * blockDim.x + threadIdx.x; i < n; i += int64_t(gridDim.x) * blockDim.x)
        out[i < before ? i : i - before + hi * pitch] = make_uint4(0u, 0u, 0u, 0u);
}

template <int BN, int KIND, int STAGES, bool SWAP, int CTAS = 1>
fp8_status launch_experts(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const CUtensorMap& tz,
                          ExpertParams p, int fa, int fb, int64_t most_units, cudaStream_t st) {
    using L = Smem<BN, STAGES, CTAS, SWAP ? 3 : 4>;
    auto kern = expert_kernel<BN, KIND, STAGES, SWAP, CTAS>;
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc) != cudaSuccess)
            return FP8_ERR_CUDA;
        attr_set[dev] = true;
    }
    p.idesc = SWAP ? instr_desc_f8(fb, fa, KIND == kRowsNN, 0, BM, BN)
                   : instr_desc_f8(fa, fb, KIND == kSumTN, KIND != kRowsNT, BM * CTAS, BN);
    const int64_t slots = sm_count() / CTAS;
    const int grid = int(most_units < slots ? most_units : slots) * CTAS;
    return launch_pdl(kern, grid, 64 + epi_threads(true, SWAP), L::kAlloc, st, CTAS, ta, tb, tc, tz, p);
}

// Whether an SM pair's 256 x 256 tiles serve NT and NN. They take in less per
// MMA but pad an expert's last rows to 256 and halve the grid's grain, so they
// pay with many rows an expert and a long main loop. Measured on B200 (us, one
// SM against pairs): 8 experts of 2048 rows, 4096 x 2048 121 -> 111, its dX
// (32 k-blocks) 114 -> 107; but with 8 k-blocks 67 -> 71 even for one expert of
// 16384 rows, and 32 experts of 512 rows 82 -> 92, dX 68.5 -> 70.9.
inline bool use_pair(int64_t rows, int64_t N, int64_t K, int64_t experts) {
    return N > 128 && K / BK >= 16 && rows >= 1024 * experts;
}

// Whether 128-wide tiles serve NT and NN, for about `m` rows of tiles and `kb`
// k-blocks each: rounds of the grid times the k-blocks at the tile's rate, plus
// the last epilogue (the constants of choose_tile). Measured on B200 (us, 256
// wide against 128): 4 experts of 100 rows, 2048 x 2048 12.5 -> 9.9, of 250
// rows, 1024 x 1024 8.8 -> 7.3; but 8 of 500 rows, 2048 x 1024 14.6 -> 17.2.
inline bool narrow_rows(double m, int64_t N, double kb) {
    auto cost = [&](int bn, double t_k, double t_epi) {
        const double rounds = m * double((N + bn - 1) / bn) / double(sm_count());
        const double whole = rounds < 4.0 ? double(int64_t(rounds + 0.999)) : rounds;
        return (whole < 1.0 ? 1.0 : whole) * kb * t_k + t_epi;
    };
    return cost(128, 0.40, 1.0) < cost(256, 0.48, 2.0);
}

// TN writes more than it multiplies, and wide tiles write faster: 128-wide ones
// only where 256-wide ones would leave half of the SMs without any (2 experts,
// 1024 x 512, 32 wide tiles: 5.9 -> 5.1 us; 16 of 512 x 512, 128 of them: 6.2 -> 6.7).
inline bool narrow_sum(int64_t experts, int64_t M, int64_t N) {
    return experts * ((M + BM - 1) / BM) * ((N + 255) / 256) * 2 <= sm_count();
}

}  // namespace
}  // namespace fp8lite

extern "C" fp8_status fp8_experts_zero_rest(void* out, int64_t rows, int64_t row_bytes, int32_t experts,
                                            const int32_t* offsets, void* stream) {
    if (rows < 0 || row_bytes < 1 || experts < 1 || !offsets || (rows > 0 && !out)) return FP8_ERR_INVALID_ARG;
    if (experts > kMaxExperts || rows >= (int64_t(1) << 31) || row_bytes >= (int64_t(1) << 32)) return FP8_ERR_UNSUPPORTED;
    if (row_bytes % 16 != 0 || !aligned(out, 16) || !aligned(offsets, 4)) return FP8_ERR_ALIGNMENT;
    if (rows == 0) return FP8_OK;
    const int64_t pitch = row_bytes / 16, blocks = (rows * pitch + 255) / 256;
    const int grid = int(blocks < 4 * int64_t(sm_count()) ? blocks : 4 * int64_t(sm_count()));
    return launch_pdl(zero_rest_kernel, grid, 256, 0, as_stream(stream), 1, static_cast<uint4*>(out), rows, pitch, offsets,
                      int(experts));
}

extern "C" fp8_status fp8_mm_experts(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa,
                                     const float* sb, int32_t sb_stride, fp8_layout layout, int64_t M, int64_t N,
                                     int64_t K, int32_t experts, const int32_t* offsets, const void* bias, fp8_act act,
                                     void* preact, void* out, void* stream) {
    if (!valid_fmt(fa) || !valid_fmt(fb) || !valid_act(int(act))) return FP8_ERR_INVALID_ARG;
    if (layout != FP8_NT && layout != FP8_NN && layout != FP8_TN) return FP8_ERR_INVALID_ARG;
    const bool sum = layout == FP8_TN;
    const int64_t rows = sum ? K : M;
    if (N < 1 || (sum ? M : K) < 1 || rows < 0 || experts < 1) return FP8_ERR_INVALID_ARG;
    if (sb_stride != 0 && (sb_stride != 1 || sum)) return FP8_ERR_INVALID_ARG;
    if (sum && (bias || preact || act != FP8_ACT_NONE)) return FP8_ERR_INVALID_ARG;
    // without token rows the token matrices may be NULL
    if (!sa || !sb || !offsets || (rows > 0 && !a8) || ((rows > 0 || !sum) && !b8) || ((rows > 0 || sum) && !out))
        return FP8_ERR_INVALID_ARG;
    if (preact && preact == out) return FP8_ERR_INVALID_ARG;
    if (experts > kMaxExperts || M > kMaxExtent || N > kMaxExtent || K > kMaxExtent)
        return FP8_ERR_UNSUPPORTED;
    if ((sum ? M : K) % 16 != 0 || (layout != FP8_NT && N % 16 != 0)) return FP8_ERR_ALIGNMENT;
    if (!aligned(a8, 16) || !aligned(b8, 16) || !aligned(out, 2) || !aligned(preact, 2) || !aligned(bias, 2))
        return FP8_ERR_ALIGNMENT;
    if (!aligned(sa, 4) || !aligned(sb, 4) || !aligned(offsets, 4)) return FP8_ERR_ALIGNMENT;
    cudaStream_t st = as_stream(stream);
    if (rows == 0) {  // no tokens: nothing to write, or nothing to sum
        if (!sum) return FP8_OK;
        return cudaMemsetAsync(out, 0, size_t(experts) * M * N * 2, st) == cudaSuccess ? FP8_OK : FP8_ERR_CUDA;
    }
    ExpertParams p = {};
    p.offsets = offsets;
    p.experts = experts;
    p.rows = int(rows);
    p.M = int(M);
    p.N = int(N);
    p.K = int(K);
    p.k_blocks = int((K + BK - 1) / BK);
    p.sa = sa;
    p.sb = sb;
    p.sb_stride = sb_stride;
    p.bias = static_cast<const uint16_t*>(bias);
    p.act = int(act);
    p.preact = static_cast<uint16_t*>(preact);
    p.out = static_cast<uint16_t*>(out);
    p.fast = N % 8 == 0 && aligned(out, 16) && aligned(preact, 16);
    CUtensorMap ta = {}, tb = {}, tc = {}, tz = {};
    // tiles at most: every expert may end inside one
    auto most = [&](int64_t tile) {
        const int64_t with_rows = experts < rows ? experts : rows;
        return rows / tile + with_rows;
    };
    constexpr int64_t kMost = int64_t(1) << 31;
    if (sum) {
        const int bn = narrow_sum(experts, M, N) ? 128 : 256;
        p.m_tiles = int((M + BM - 1) / BM);
        p.n_tiles = int((N + bn - 1) / bn);
        const int64_t units = int64_t(experts) * p.m_tiles * p.n_tiles;
        if (units >= kMost) return FP8_ERR_UNSUPPORTED;
        if (!make_map(&ta, a8, M, rows, 1, 0, 128, BK) || !make_map(&tb, b8, N, rows, 1, 0, 128, BK)) return FP8_ERR_CUDA;
        if (p.fast && !make_out_map(&tc, out, N, M, experts, uint64_t(M) * N * 2, 32)) return FP8_ERR_CUDA;
        if (bn == 256) return launch_experts<256, kSumTN, 4, false>(ta, tb, tc, tz, p, fa, fb, units, st);
        return launch_experts<128, kSumTN, 6, false>(ta, tb, tc, tz, p, fa, fb, units, st);
    }
    const bool nn = layout == FP8_NN;
    // Few rows an expert: swapped tiles of 16 or 32 token rows
    if (N >= 128 && rows <= int64_t(32) * experts) {
        const int bn = rows <= int64_t(8) * experts ? 16 : 32;
        p.n_tiles = int((N + BM - 1) / BM);
        if (most(bn) * p.n_tiles >= kMost) return FP8_ERR_UNSUPPORTED;
        const bool ok = make_map(&ta, a8, K, rows, 1, 0, BK, uint32_t(bn)) &&
                        (nn ? make_map(&tb, b8, N, K, experts, uint64_t(N) * K, 128, BK)
                            : make_map(&tb, b8, K, N, experts, uint64_t(N) * K, BK, BM));
        if (!ok) return FP8_ERR_CUDA;
        const int64_t units = most(bn) * p.n_tiles;
        if (bn == 16)
            return nn ? launch_experts<16, kRowsNN, 10, true>(ta, tb, tc, tz, p, fa, fb, units, st)
                      : launch_experts<16, kRowsNT, 10, true>(ta, tb, tc, tz, p, fa, fb, units, st);
        return nn ? launch_experts<32, kRowsNN, 9, true>(ta, tb, tc, tz, p, fa, fb, units, st)
                  : launch_experts<32, kRowsNT, 9, true>(ta, tb, tc, tz, p, fa, fb, units, st);
    }
    const bool pair = use_pair(rows, N, K, experts);
    // an expert's last tile is half empty on average
    const double m_tiles = double(rows) / BM + 0.5 * double(experts < rows ? experts : rows);
    const int bn = pair || !narrow_rows(m_tiles, N, double(p.k_blocks)) ? 256 : 128;
    p.n_tiles = int((N + bn - 1) / bn);
    const int64_t units = most(BM * (pair ? 2 : 1)) * p.n_tiles;
    if (units >= kMost) return FP8_ERR_UNSUPPORTED;
    const bool ok = make_map(&ta, a8, K, rows, 1, 0, BK, BM) &&
                    (nn ? make_map(&tb, b8, N, K, experts, uint64_t(N) * K, 128, BK)
                        : make_map(&tb, b8, K, N, experts, uint64_t(N) * K, BK, uint32_t(pair ? bn / 2 : bn)));
    if (!ok) return FP8_ERR_CUDA;
    if (p.fast && !make_out_map(&tc, out, N, rows, 1, 0, 32)) return FP8_ERR_CUDA;
    if (p.fast && preact && !make_out_map(&tz, preact, N, rows, 1, 0, 32)) return FP8_ERR_CUDA;
    if (pair)
        return nn ? launch_experts<256, kRowsNN, 6, false, 2>(ta, tb, tc, tz, p, fa, fb, units, st)
                  : launch_experts<256, kRowsNT, 6, false, 2>(ta, tb, tc, tz, p, fa, fb, units, st);
    if (bn == 256)
        return nn ? launch_experts<256, kRowsNN, 4, false>(ta, tb, tc, tz, p, fa, fb, units, st)
                  : launch_experts<256, kRowsNT, 4, false>(ta, tb, tc, tz, p, fa, fb, units, st);
    return nn ? launch_experts<128, kRowsNN, 6, false>(ta, tb, tc, tz, p, fa, fb, units, st)
              : launch_experts<128, kRowsNT, 6, false>(ta, tb, tc, tz, p, fa, fb, units, st);
}
