// FP8 products grouped by expert: the rows of a token-sorted matrix belong to
// experts in turn, expert e's being [offsets[e], offsets[e+1]), and every
// expert has its own weight. The offsets live on the device: the host knows
// the total and the number of experts only, and nothing is synchronised.
//
//   NT, NN   out[r] = act(A[r] op(B[e]) / (sa sb_e) + bias_e),  r in e's rows
//   TN       out[e] = A[rows of e]^T B[rows of e] / (sa sb)
//
// One persistent launch. Each CTA turns the offsets into a table of tiles per
// expert in shared memory (clamped to the matrix and made monotone first, so
// that no offsets can lead an access out of it) and walks its share of the
// units; the roles, pipeline and epilogue are those of gemm_kernel.cuh.
//
//  * A tile that reaches past its expert's last row loads the next expert's
//    rows too; their results are dropped at the store, which writes such a
//    tile in 16-byte row pieces and a whole tile by TMA.
//  * In TN the rows are the contraction, so a block of 128 may hold no row of
//    another expert. Its tensor map has two row dimensions of the same pitch:
//    the block's first row, and 128 rows from there. A block of t < 128 rows
//    starts at row t - 128 of the second: rows below 0 are out of bounds and
//    arrive as zeros, the last t are the expert's (both operands alike, so
//    the order of the sum is all that changes).
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
    int m0, m_end;  // ROWS: first row of the tile and the expert's end; SUM: first row of the output, M
    int n0;         // first output column (swapped: of 128)
    int kbs;        // k-blocks
    int k_row, k_end;  // SUM: the expert's rows
};

// The tile table of a CTA.
struct Table {
    int off[kMaxExperts + 1];
    int tiles[kMaxExperts + 1];  // tiles (ROWS) before each expert
};

// Fills the table (every thread of the block calls it). TILE: rows of a tile.
template <int TILE>
__device__ __forceinline__ void build_table(Table& tab, const ExpertParams& p) {
    const int n = p.experts + 1;
    for (int i = threadIdx.x; i < n; i += blockDim.x) tab.off[i] = min(max(__ldg(p.offsets + i), 0), p.rows);
    __syncthreads();
    if (threadIdx.x < 32) {
        const int lane = threadIdx.x, per = (n + 31) / 32;
        const int lo = min(lane * per, n), hi = min(lo + per, n);
        // running maximum: expert e ends where the next begins, never before it
        int m = 0;
        for (int i = lo; i < hi; ++i) m = max(m, tab.off[i]);
        int before = __shfl_up_sync(0xffffffffu, m, 1);
        if (lane == 0) before = 0;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, before, o);
            if (lane >= o) before = max(before, v);
        }
        m = before;
        for (int i = lo; i < hi; ++i) tab.off[i] = m = max(m, tab.off[i]);
        __syncwarp();
        int sum = 0;
        for (int i = lo; i < hi && i < p.experts; ++i) sum += (tab.off[i + 1] - tab.off[i] + TILE - 1) / TILE;
        int at = sum;
        for (int o = 1; o < 32; o <<= 1) {
            const int v = __shfl_up_sync(0xffffffffu, at, o);
            if (lane >= o) at += v;
        }
        at -= sum;
        for (int i = lo; i < hi; ++i) {
            tab.tiles[i] = at;
            if (i < p.experts) at += (tab.off[i + 1] - tab.off[i] + TILE - 1) / TILE;
        }
    }
    __syncthreads();
}

// Work unit u; `e` is the caller's cursor (units come in rising order).
template <int BN, int KIND, bool SWAP>
__device__ __forceinline__ Item item_of(const Table& tab, const ExpertParams& p, int u, int& e) {
    Item it;
    int mb, nb, b;
    if constexpr (KIND == kSumTN) {
        const int per = p.m_tiles * p.n_tiles;
        e = u / per;
        tile_coords(u - e * per, TileWalk{p.m_tiles, p.n_tiles, 16}, mb, nb, b);
        it.m0 = mb * BM;
        it.m_end = p.M;
        it.n0 = nb * BN;
        it.k_row = tab.off[e];
        it.k_end = tab.off[e + 1];
        it.kbs = (it.k_end - it.k_row + BK - 1) / BK;
    } else {
        while (u >= tab.tiles[e + 1] * p.n_tiles) ++e;
        const int t = u - tab.tiles[e] * p.n_tiles, mt = tab.tiles[e + 1] - tab.tiles[e];
        if constexpr (SWAP) {
            mb = t % mt;  // the row tiles of one weight tile one after the other
            nb = t / mt;
            it.m0 = tab.off[e] + mb * BN;
            it.n0 = nb * BM;
        } else {
            tile_coords(t, TileWalk{mt, p.n_tiles, 16}, mb, nb, b);
            it.m0 = tab.off[e] + mb * BM;
            it.n0 = nb * BN;
        }
        it.m_end = tab.off[e + 1];
        it.k_row = it.k_end = 0;
        it.kbs = p.k_blocks;
    }
    it.e = e;
    return it;
}

template <int BN, int STAGES>
struct ExpertSmem : Smem<BN, STAGES, 1, 3> {
    using Base = Smem<BN, STAGES, 1, 3>;
    static constexpr int kTableOffset = (Base::kBytes + 15) / 16 * 16;
    static constexpr int kTotal = kTableOffset + int(sizeof(Table)) + 1024;
    static_assert(kTotal <= 227 * 1024, "shared memory per CTA");
};

// KIND, SWAP: see the head of the file. BN: output columns of a tile, or
// token rows of a swapped one.
template <int BN, int KIND, int STAGES, bool SWAP>
__global__ void __maxnreg__(168)
expert_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
              const __grid_constant__ CUtensorMap tm_c, const __grid_constant__ CUtensorMap tm_z, const ExpertParams p) {
    using L = ExpertSmem<BN, STAGES>;
    // majors of the MMA's operands: K-major unless the stored rows run along K
    constexpr bool A_MN = SWAP ? KIND == kRowsNN : KIND == kSumTN;
    constexpr bool B_MN = !SWAP && KIND != kRowsNT;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    const uint32_t s_a = smem_addr(smem);
    const uint32_t s_b = s_a + STAGES * L::kABytes;
    const uint32_t bar_full = s_a + L::kBarOffset;
    const uint32_t bar_empty = bar_full + STAGES * 8;
    const uint32_t bar_tfull = bar_empty + STAGES * 8;
    const uint32_t bar_tempty = bar_tfull + 2 * 8;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBarOffset + (2 * STAGES + 4) * 8);
    float* s_bias = reinterpret_cast<float*>(smem + L::kBiasOffset);
    Table& tab = *reinterpret_cast<Table*>(smem + L::kTableOffset);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

    if (warp == 0 && lane == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(bar_full + 8 * s, 1);
            mbar_init(bar_empty + 8 * s, 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(bar_tfull + 8 * b, 1);
            mbar_init(bar_tempty + 8 * b, kEpiThreads);
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
        tmem_alloc<1>(smem_addr(tmem_slot), L::kTmemCols);
        tmem_relinquish<1>();
    }
    griddep_wait();  // the offsets are read next
    griddep_launch();
    tc_fence_before();
    build_table<SWAP ? BN : BM>(tab, p);  // ends with a block barrier
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;
    const int units = KIND == kSumTN ? p.experts * p.m_tiles * p.n_tiles : tab.tiles[p.experts] * p.n_tiles;

    if (warp == 0) {
        // ------------------------------------------------ TMA producer ---
        const bool issuer = elect_one();
        int stage = 0, e = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const Item it = item_of<BN, KIND, SWAP>(tab, p, u, e);
            for (int kb = 0; kb < it.kbs; ++kb) {
                if (!wait_bounded_warp(bar_empty + 8 * stage, phase ^ 1)) { ok = false; break; }
                const uint32_t full = bar_full + 8 * stage;
                const uint32_t da = s_a + stage * L::kABytes, db = s_b + stage * L::kBBytes;
                if (issuer) {
                    mbar_arrive_expect_tx(full, uint32_t(L::kStageBytes));
                    if constexpr (KIND == kSumTN) {
                        const int first = it.k_row + kb * BK;
                        const int r0 = min(it.k_end - first, BK) - BK;  // 0, or negative in the last block
                        tma_load_3d(da, &tm_a, full, it.m0, r0, first);
#pragma unroll
                        for (int h = 0; h < BN / 128; ++h)
                            tma_load_3d(db + h * 128 * BK, &tm_b, full, it.n0 + h * 128, r0, first);
                    } else if constexpr (SWAP) {
                        if (A_MN) tma_load_3d(da, &tm_b, full, it.n0, kb * BK, it.e);
                        else      tma_load_3d(da, &tm_b, full, kb * BK, it.n0, it.e);
                        tma_load_3d(db, &tm_a, full, kb * BK, it.m0, 0);
                    } else {
                        tma_load_3d(da, &tm_a, full, kb * BK, it.m0, 0);
                        if (B_MN) {
#pragma unroll
                            for (int h = 0; h < BN / 128; ++h)
                                tma_load_3d(db + h * 128 * BK, &tm_b, full, it.n0 + h * 128, kb * BK, it.e);
                        } else {
                            tma_load_3d(db, &tm_b, full, kb * BK, it.n0, it.e);
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
        int stage = 0, e = 0, done = 0;
        uint32_t phase = 0;
        bool ok = true;
        for (int u = blockIdx.x; u < units && ok; u += gridDim.x) {
            const Item it = item_of<BN, KIND, SWAP>(tab, p, u, e);
            if (it.kbs == 0) continue;  // an expert without rows: the epilogue writes its zeros
            const int buf = done & 1;
            if (!wait_bounded_warp(bar_tempty + 8 * buf, ((done >> 1) & 1) ^ 1)) break;
            tc_fence_after();
            for (int kb = 0; kb < it.kbs; ++kb) {
                if (!wait_bounded_warp(bar_full + 8 * stage, phase)) { ok = false; break; }
                if (issuer) {
                    mma_kblock_f8f6f4<1>(tmem_base + buf * BN, a_desc0 + uint64_t(stage) * (L::kABytes >> 4),
                                         b_desc0 + uint64_t(stage) * (L::kBBytes >> 4), A_MN ? 256u : 2u,
                                         B_MN ? 256u : 2u, p.idesc, kb != 0);
                    mma_commit(bar_empty + 8 * stage);
                }
                __syncwarp();
                if (++stage == STAGES) { stage = 0; phase ^= 1; }
            }
            if (issuer) mma_commit(bar_tfull + 8 * buf);
            __syncwarp();
            ++done;
        }
    } else {
        // ----------------------------------------------------- epilogue ---
        const int q = warp & 3;  // TMEM lane quarter this warp may access
        const int row_in_tile = q * 32 + lane;
        const int etid = threadIdx.x - 64;
        const bool store_lead = etid == 0;
        const uint32_t stg0 = s_a + L::kStgOffset;
        const float inv_a = 1.0f / __ldg(p.sa);
        int n_st = 0, e = 0, done = 0;
        bool failed = false;
        for (int u = blockIdx.x; u < units; u += gridDim.x) {
            const Item it = item_of<BN, KIND, SWAP>(tab, p, u, e);
            const float inv = inv_a * (1.0f / __ldg(p.sb + int64_t(it.e) * p.sb_stride));
            const bool has = it.kbs > 0;
            const int buf = done & 1;
            if constexpr (!SWAP && KIND != kSumTN) {
                epilogue_bar();  // the previous tile's readers are done
                for (int j = etid; j < BN; j += kEpiThreads) {
                    const int col = it.n0 + j;
                    s_bias[j] = (p.bias && col < p.N) ? bf16_value(__ldg(p.bias + int64_t(it.e) * p.N + col)) : 0.0f;
                }
                epilogue_bar();
            }
            float bias_row = 0.0f;
            if (SWAP && p.bias && it.n0 + row_in_tile < p.N)
                bias_row = bf16_value(__ldg(p.bias + int64_t(it.e) * p.N + it.n0 + row_in_tile));
            if (has) {
                if (!failed) failed = !wait_bounded(bar_tfull + 8 * buf, (done >> 1) & 1);
                failed = epilogue_bar_or(failed);
                if (failed) continue;
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
                    for (int i = 0; i < 16; ++i) y[i] = fmaf(__uint_as_float(r[i]), inv, bias_row);
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
                const int row = it.m0 + row_in_tile;
                uint16_t* out = KIND == kSumTN ? p.out + int64_t(it.e) * p.M * p.N : p.out;
                const int left = (p.N - it.n0 + 31) / 32;
                const int nch = left < BN / 32 ? left : BN / 32;
                const bool whole = p.fast && (KIND == kSumTN || it.m0 + BM <= it.m_end);
                // one 128 x 32 block to global memory
                auto put = [&](const float (&y)[32], uint16_t* dst, const CUtensorMap* map, int col0) {
                    if (whole) {
                        stage_and_store<L>(stg0, n_st, row_in_tile, y, store_lead, map, col0, it.m0,
                                           KIND == kSumTN ? it.e : 0);
                        ++n_st;
                    } else if (p.fast) {
                        // an expert's last rows: staged by the warp for itself, then 64-byte row pieces
                        const uint32_t stg = stg0 + uint32_t(n_st % L::kStgBufs) * L::kStgBytes;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
                            asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                                             stg + row_in_tile * 64 + ((j ^ ((row_in_tile >> 1) & 3)) << 4)),
                                         "r"(pack_bf16x2(y[8 * j + 0], y[8 * j + 1])),
                                         "r"(pack_bf16x2(y[8 * j + 2], y[8 * j + 3])),
                                         "r"(pack_bf16x2(y[8 * j + 4], y[8 * j + 5])),
                                         "r"(pack_bf16x2(y[8 * j + 6], y[8 * j + 7]))
                                         : "memory");
                        __syncwarp();
                        const int piece = lane & 3, col = col0 + piece * 8;
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const int r = q * 32 + (lane >> 2) + 8 * j;
                            uint4 w;
                            asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                                         : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                                         : "r"(stg + r * 64 + ((piece ^ ((r >> 1) & 3)) << 4))
                                         : "memory");
                            if (it.m0 + r < it.m_end && col < p.N)
                                *reinterpret_cast<uint4*>(dst + int64_t(it.m0 + r) * p.N + col) = w;
                        }
                        // every TMA store has read its tile before the next block is staged: this
                        // block issues none, so a store three back could be the newest one pending
                        if (store_lead) bulk_wait_read<0>();
                        epilogue_bar();
                        ++n_st;
                    } else if (row < it.m_end) {
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (col0 + i < p.N) dst[int64_t(row) * p.N + col0 + i] = bf16_bits(y[i]);
                    }
                };
#pragma unroll 1
                for (int c = 0; c < nch; ++c) {
                    const int col0 = it.n0 + c * 32;
                    float y[32];
                    if (has) {
                        uint32_t r[32];
                        __syncwarp();
                        tmem_ld<32>(t_row + c * 32, r);
                        tmem_ld_wait();
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            y[i] = KIND == kSumTN ? __uint_as_float(r[i]) * inv
                                                  : fmaf(__uint_as_float(r[i]), inv, s_bias[c * 32 + i]);
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) y[i] = 0.0f;
                    }
                    if constexpr (KIND != kSumTN) {
                        if (p.preact) put(y, p.preact, &tm_z, col0);
                        act_apply(p.act, y);
                    }
                    put(y, out, &tm_c, col0);
                }
            }
            if (has) {
                tc_fence_before();
                mbar_arrive(bar_tempty + 8 * buf);
                ++done;
            }
        }
        if (store_lead) bulk_wait_read<0>();  // the staging tiles outlive the stores that read them
    }

    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        tmem_dealloc<1>(tmem_base, L::kTmemCols);
    }
}

// Token rows as blocks of up to 128 that may start at any row: (columns, row
// within the block, first row), both row dimensions one row apart.
bool make_block_map(CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows) {
    EncodeTiledFn fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {cols, uint64_t(BK), rows};
    cuuint64_t strides[2] = {cols, cols};
    cuuint32_t box[3] = {128, uint32_t(BK), 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int BN, int KIND, int STAGES, bool SWAP>
fp8_status launch_experts(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc, const CUtensorMap& tz,
                          ExpertParams p, int fa, int fb, int64_t most_units, cudaStream_t st) {
    using L = ExpertSmem<BN, STAGES>;
    auto kern = expert_kernel<BN, KIND, STAGES, SWAP>;
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kTotal) != cudaSuccess)
            return FP8_ERR_CUDA;
        attr_set[dev] = true;
    }
    p.idesc = SWAP ? instr_desc_f8(fb, fa, KIND == kRowsNN, 0, BM, BN)
                   : instr_desc_f8(fa, fb, KIND == kSumTN, KIND != kRowsNT, BM, BN);
    const int grid = int(most_units < sm_count() ? most_units : sm_count());
    return launch_pdl(kern, grid, kThreads, L::kTotal, st, 1, ta, tb, tc, tz, p);
}

}  // namespace
}  // namespace fp8lite

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
    if (!sa || !sb || !offsets || !b8 || (rows > 0 && !a8) || ((rows > 0 || sum) && !out)) return FP8_ERR_INVALID_ARG;
    if (experts > kMaxExperts || M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31))
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
        constexpr int BN = 256;
        p.m_tiles = int((M + BM - 1) / BM);
        p.n_tiles = int((N + BN - 1) / BN);
        const int64_t units = int64_t(experts) * p.m_tiles * p.n_tiles;
        if (units >= kMost) return FP8_ERR_UNSUPPORTED;
        if (!make_block_map(&ta, a8, M, rows) || !make_block_map(&tb, b8, N, rows)) return FP8_ERR_CUDA;
        if (p.fast && !make_out_map(&tc, out, N, M, experts, uint64_t(M) * N * 2)) return FP8_ERR_CUDA;
        return launch_experts<BN, kSumTN, 4, false>(ta, tb, tc, tz, p, fa, fb, units, st);
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
    constexpr int BN = 256;
    p.n_tiles = int((N + BN - 1) / BN);
    const int64_t units = most(BM) * p.n_tiles;
    if (units >= kMost) return FP8_ERR_UNSUPPORTED;
    const bool ok = make_map(&ta, a8, K, rows, 1, 0, BK, BM) &&
                    (nn ? make_map(&tb, b8, N, K, experts, uint64_t(N) * K, 128, BK)
                        : make_map(&tb, b8, K, N, experts, uint64_t(N) * K, BK, BN));
    if (!ok) return FP8_ERR_CUDA;
    if (p.fast && !make_out_map(&tc, out, N, rows, 1, 0)) return FP8_ERR_CUDA;
    if (p.fast && preact && !make_out_map(&tz, preact, N, rows, 1, 0)) return FP8_ERR_CUDA;
    return nn ? launch_experts<BN, kRowsNN, 4, false>(ta, tb, tc, tz, p, fa, fb, units, st)
              : launch_experts<BN, kRowsNT, 4, false>(ta, tb, tc, tz, p, fa, fb, units, st);
}
