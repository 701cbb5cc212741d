// Gradient through an activation, quantized as it is formed: dz = g act'(z) in
// fp32, its FP8 codes under a delayed ring, and the bias gradient sum_i dz[i][j].
//
// Bound by HBM: 5 bytes an element (g and z in bf16 read, one code written).
// Measured on B200 with SiLU at 32768 x 4096: 119.4 us, 5.6 TB/s, 0.86 of the
// measured copy; 2048 x 4096 with GELU tanh (42 MB) 13.9 us, 3.0 TB/s: the launch,
// the first trip to HBM and the sums' exchange; 37 x 1040 4.0 us, the same alone.
//
// Split: a cluster of up to 16 CTAs owns a strip of columns, its CTAs taking
// row blocks in turn, so that a column's sum is finished inside the cluster:
// each thread adds its rows, the warps meet in shared memory, and rank 0 adds
// the other CTAs' sums through distributed shared memory. Every sum has one
// fixed order, in fp32, with no workspace and no atomics; the cluster's amax
// takes the same way, so the ring sees one atomic per cluster. A thread covers
// 8 columns (16 bytes of g and of z, 8 of codes) of a few rows at a time.
//
// Rows of experts (fp8_act_grad_experts): a cluster takes every `parts`-th
// expert of its strip and finishes each one's sums before the next. Whole experts
// are dealt out, so the time follows the routing: 16384 x 4096 with SiLU, 32
// experts, 66 us with equal ones, 94 to 115 with shares spread as exp(normal),
// 284 with all rows in one (64 of 576 CTAs stream); without an activation 37, 47
// to 56, 122. 512 experts of 8 rows, 2048 wide, take 60 us: a barrier or three each.

#include <cuda_runtime.h>

#include "act.cuh"
#include "common.cuh"
#include "sm100.cuh"

namespace fp8lite {
namespace {

using namespace sm100;

constexpr int kThreads = 256;  // of a CTA; tall, narrow tensors take twice as many
constexpr int kPerSm = 4;      // CTAs of an SM
constexpr int64_t kTallRows = 8192;  // from here on twice the threads may pay
constexpr int kPortableRanks = 8;  // CTAs of a cluster that every device holds
constexpr int kMaxRanks = 16;      // by opt-in, where the device holds them

struct GradArgs {
    const uint4* g;
    const uint4* z;
    int64_t rows;
    int64_t pitch;  // 16-byte pieces of a row
    uint2* out8;
    fp8_ring* ring;
    float* amax_out;
    float* scale_out;
    uint16_t* dbias;
    int fmt;
    int defer;
    int ranks;  // CTAs of a cluster
    // rows of experts: offsets[experts + 1], or NULL (one range, all rows)
    const int32_t* offsets;
    int experts;
    int parts;  // clusters of a strip
};

__device__ __forceinline__ float lo_f32(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f32(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

template <int FMT>
__device__ __forceinline__ uint32_t cvt2(float lo, float hi) {
    uint16_t r;
    if (FMT == FP8_E4M3) asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    else                 asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}

template <int FMT>
__device__ __forceinline__ uint2 codes8(const F2 (&d)[4], float s) {
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float lo, hi;
        split(mul2(d[i], f2(s)), lo, hi);
        c[i] = cvt2<FMT>(lo, hi);
    }
    return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// max(m, |lo|, |hi|); NaN is ignored.
__device__ __forceinline__ float max_abs(float m, F2 v) {
    float lo, hi;
    split(v, lo, hi);
    asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(m) : "f"(lo), "f"(hi));
    return m;
}

// The cluster's amax (bmax: this CTA's, rank 0 of it) to the ring; the cluster
// that holds the last ticket finishes the call. One thread.
__device__ __forceinline__ void publish_amax(const GradArgs& a, float* bmax) {
    float v = *bmax;
    for (int r = 1; r < a.ranks; ++r) v = fmaxf(v, ld_cluster_f32(map_to_rank(smem_addr(bmax), uint32_t(r))));
    fp8_ring* ring = a.ring;
    if (v != 0.0f) atomicMax(&ring->amax_bits, __float_as_uint(v));
    const uint32_t ticket = atom_add_acq_rel(&ring->ticket, 1u);
    if (ticket != gridDim.x / a.ranks - 1) return;
    volatile fp8_ring* rr = ring;
    if (a.defer) {
        if (a.amax_out) *a.amax_out = __uint_as_float(*reinterpret_cast<volatile uint32_t*>(&ring->amax_bits));
    } else {
        float h[FP8_RING_HISTORY];
        const uint32_t idx = ring_read(rr, h);
        const float top = __uint_as_float(atomicExch(&ring->amax_bits, 0u));
        ring_fold(rr, h, idx, top, fmt_max(a.fmt));
        if (a.amax_out) *a.amax_out = top;
    }
    rr->ticket = 0u;
}

// W: columns of a strip (64, 32 or 16). THREADS: of a CTA. EXPERTS: the rows
// belong to experts (a kernel of its own: the plain form's loads in flight leave
// no registers for the offsets; 32768 x 4096 GELU 147 -> 149 us with both in one).
template <int ACT, int W, int THREADS, bool EXPERTS>
__global__ void __launch_bounds__(THREADS, kPerSm * kThreads / THREADS) act_grad_kernel(const GradArgs a) {
    constexpr int kWarps = THREADS / 32;
    // rows in flight per thread: with z as many as 64 registers hold; without it
    // twice that (32768 x 4096 without an activation: 79 us with two, 66 with four)
    constexpr int kRows = ACT == FP8_ACT_NONE ? 4 : 2;
    constexpr int kTpr = W / 8;                 // threads of a row
    constexpr int kBlockRows = THREADS / kTpr;  // rows of a block's pass
    __shared__ float part[kWarps][W];
    __shared__ float colsum[W];
    __shared__ uint32_t wmax[kWarps];
    __shared__ float bmax;
    __shared__ float s_scale;
    __shared__ int s_before[EXPERTS ? kWarps : 1];
    griddep_wait();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int rank = int(blockIdx.x) % a.ranks;
    const int64_t cluster = int64_t(blockIdx.x) / a.ranks;
    const int64_t strip = cluster / a.parts;
    const int part0 = int(cluster - strip * a.parts);
    const int64_t piece = strip * kTpr + threadIdx.x % kTpr;  // this thread's 8 columns
    const bool in = piece < a.pitch;
    const int64_t step = int64_t(a.ranks) * kBlockRows;  // rows between two of this thread
    const int64_t stride = step * a.pitch;
    const int64_t first = int64_t(rank) * kBlockRows + threadIdx.x / kTpr;  // this thread's first row of a range
    const uint4* pg = nullptr;  // the row to load next
    const uint4* pz = nullptr;
    uint4 g[kRows], z[kRows];
    auto load = [&](int u) {
        g[u] = __ldg(pg);
        pg += stride;
        if (ACT != FP8_ACT_NONE) {
            z[u] = __ldg(pz);
            pz += stride;
        }
    };
    float s = 0.0f, m = 0.0f;
    for (int e = part0; e < (EXPERTS ? a.experts : 1); e += a.parts) {
        int64_t lo = 0, hi = a.rows;
        if constexpr (EXPERTS) {
            // Offsets are limited to [0, rows] and to no less than the ones before
            // them, as in the experts' products. Each warp keeps the running
            // maximum, in shared memory: a register more would cost 2 %.
            volatile int* before = &s_before[warp];
            const int rows = int(a.rows);
            const int end = min(__ldg(a.offsets + e + 1), rows);
            int top = e == part0 ? 0 : *before;
#pragma unroll 4
            for (int i = (e == part0 ? 0 : e - a.parts + 1) + lane; i <= e; i += 32)
                top = max(top, min(__ldg(a.offsets + i), rows));
            top = __reduce_max_sync(0xffffffffu, top);
            *before = top;
            __syncwarp();
            lo = top;
            hi = max(top, end);
        } else if constexpr (ACT == FP8_ACT_NONE || ACT == FP8_ACT_RELU || ACT == FP8_ACT_SILU) {
            // constants to the compiler, which schedules these loops better without
            // knowing them (us, SiLU 32768 x 4096 122.2 -> 119.0; GELU would take 146 -> 155)
            asm volatile("" : "+l"(lo), "+l"(hi));
        }
        const int64_t row = lo + first;
        int n = in && row < hi ? int((hi - row + step - 1) / step) : 0;  // rows left
        const int64_t at = row * a.pitch + piece;
        pg = a.g + at;
        pz = a.z + at;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
            if (u < n) load(u);  // before the scale is known: the loads do not need it
        if (e == part0) {
            if (threadIdx.x == 0) {
                s_scale = *reinterpret_cast<volatile float*>(&a.ring->scale);
                if (blockIdx.x == 0) *a.scale_out = s_scale;
            }
            __syncthreads();
            s = s_scale;
        }
        F2 sum[4] = {0, 0, 0, 0};
        uint2* out = a.out8 + at;
        while (n > 0) {
#pragma unroll
            for (int u = 0; u < kRows; ++u) {
                if (u < n) {
                    const uint32_t gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
                    const uint32_t zw[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
                    F2 d[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        d[i] = f2(lo_f32(gw[i]), hi_f32(gw[i]));
                        if (ACT != FP8_ACT_NONE) d[i] = mul2(d[i], act_slope<ACT>(zw[i]));
                    }
                    if (u + kRows < n) load(u);  // the registers are free: the row kRows further on
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        m = max_abs(m, d[i]);
                        sum[i] = add2(sum[i], d[i]);
                    }
                    *out = a.fmt == FP8_E4M3 ? codes8<FP8_E4M3>(d, s) : codes8<FP8_E5M2>(d, s);
                    out += stride;
                }
            }
            n -= kRows;
        }
        // The block's column sums and, after its last range, its amax; then the
        // cluster's: rank 0 takes them in rank order.
        const bool last = !EXPERTS || e + a.parts >= a.experts;
        if (!a.dbias && !last) continue;
        if (a.dbias) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                float v0, v1;
                split(sum[i], v0, v1);
#pragma unroll
                for (int o = kTpr; o < 32; o <<= 1) {
                    v0 += __shfl_xor_sync(0xffffffffu, v0, o);
                    v1 += __shfl_xor_sync(0xffffffffu, v1, o);
                }
                if (lane < kTpr) {
                    part[warp][lane * 8 + 2 * i] = v0;
                    part[warp][lane * 8 + 2 * i + 1] = v1;
                }
            }
        }
        if (last) {
            griddep_launch();
            const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(m));
            if (lane == 0) wmax[warp] = bits;
        }
        __syncthreads();
        if (a.dbias && threadIdx.x < W) {
            float v = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) v += part[w][threadIdx.x];
            colsum[threadIdx.x] = v;
        }
        if (last && threadIdx.x >= THREADS - 32) {
            const uint32_t bits = __reduce_max_sync(0xffffffffu, lane < kWarps ? wmax[lane] : 0u);
            if (lane == 0) bmax = __uint_as_float(bits);
        }
        if (a.ranks > 1) cluster_sync();
        else             __syncthreads();
        if (rank == 0) {
            if (last && threadIdx.x == THREADS - 32) publish_amax(a, &bmax);
            if (a.dbias && threadIdx.x < W) {
                float v = colsum[threadIdx.x];
                const uint32_t mine = smem_addr(&colsum[threadIdx.x]);
                for (int r = 1; r < a.ranks; ++r) v += ld_cluster_f32(map_to_rank(mine, uint32_t(r)));
                const int64_t c = strip * W + threadIdx.x;
                if (c < a.pitch * 8) {
                    uint16_t h;
                    asm("cvt.rn.bf16.f32 %0, %1;" : "=h"(h) : "f"(v));
                    a.dbias[int64_t(e) * a.pitch * 8 + c] = h;
                }
            }
        }
        // rank 0 has read what the others hold before it changes or they leave
        if (a.ranks > 1) cluster_sync();
        else             __syncthreads();
    }
}

// Clusters of `cluster` CTAs that the current device holds at a time: 0 if none
// of its GPCs has the SMs for one.
int max_clusters(void (*kern)(GradArgs), int threads, int cluster) {
    cudaLaunchAttribute attr = {};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = unsigned(cluster);
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(unsigned(cluster));
    cfg.blockDim = dim3(unsigned(threads));
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kern, &cfg) == cudaSuccess) return n;
    cudaGetLastError();  // clears it
    return 0;
}

template <int ACT, int W, int THREADS, bool EXPERTS>
fp8_status launch_kernel(GradArgs a, int64_t strips, cudaStream_t st) {
    auto kern = act_grad_kernel<ACT, W, THREADS, EXPERTS>;
    if (a.ranks > kPortableRanks) {
        static int fits[64] = {0};  // 1: the device holds such a cluster, -1: it does not
        int dev = 0;
        if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
        if (fits[dev] == 0) {
            if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess)
                return FP8_ERR_CUDA;
            fits[dev] = max_clusters(kern, THREADS, kMaxRanks) > 0 ? 1 : -1;
        }
        if (fits[dev] < 0) a.ranks = kPortableRanks;
    }
    return launch_pdl(kern, dim3(unsigned(strips * a.parts * a.ranks)), THREADS, 0, st, a.ranks, a);
}

template <int ACT, int W, int THREADS>
fp8_status launch_act(const GradArgs& a, int64_t strips, cudaStream_t st) {
    return a.offsets ? launch_kernel<ACT, W, THREADS, true>(a, strips, st)
                     : launch_kernel<ACT, W, THREADS, false>(a, strips, st);
}

template <int W, int THREADS = kThreads>
fp8_status launch_width(const GradArgs& a, int act, int64_t strips, cudaStream_t st) {
    switch (act) {
        case FP8_ACT_NONE:      return launch_act<FP8_ACT_NONE, W, THREADS>(a, strips, st);
        case FP8_ACT_RELU:      return launch_act<FP8_ACT_RELU, W, THREADS>(a, strips, st);
        case FP8_ACT_GELU:      return launch_act<FP8_ACT_GELU, W, THREADS>(a, strips, st);
        case FP8_ACT_GELU_TANH: return launch_act<FP8_ACT_GELU_TANH, W, THREADS>(a, strips, st);
        default:                return launch_act<FP8_ACT_SILU, W, THREADS>(a, strips, st);
    }
}

}  // namespace
}  // namespace fp8lite

using namespace fp8lite;

namespace fp8lite {
namespace {

fp8_status act_grad_impl(const void* g, const void* z, int64_t rows, int64_t cols, int experts, const int32_t* offsets,
                         int act, int fmt, fp8_ring* ring, uint32_t flags, uint8_t* out8, float* amax_out,
                         float* scale_out, void* dbias, void* stream) {
    if (!valid_act(act) || !valid_fmt(fmt)) return FP8_ERR_INVALID_ARG;
    if (flags != 0 && flags != FP8_QUANTIZE_DEFER_FOLD) return FP8_ERR_INVALID_ARG;
    if (rows < 0 || cols < 1 || cols >= (int64_t(1) << 31) || rows >= (int64_t(1) << 31) ||
        rows >= (int64_t(1) << 40) / cols)
        return FP8_ERR_INVALID_ARG;
    if (!ring || !scale_out) return FP8_ERR_INVALID_ARG;
    if (rows > 0 && (!g || !out8 || (act != FP8_ACT_NONE && !z))) return FP8_ERR_INVALID_ARG;
    if (cols % 8 != 0) return FP8_ERR_ALIGNMENT;
    if (!aligned(g, 16) || !aligned(z, 16) || !aligned(out8, 16) || !aligned(dbias, 2)) return FP8_ERR_ALIGNMENT;
    if (!aligned(ring, 4) || !aligned(amax_out, 4) || !aligned(scale_out, 4) || !aligned(offsets, 4))
        return FP8_ERR_ALIGNMENT;
    GradArgs a = {};
    a.g = static_cast<const uint4*>(g);
    a.z = static_cast<const uint4*>(z);
    a.rows = rows;
    a.pitch = cols / 8;
    a.out8 = reinterpret_cast<uint2*>(out8);
    a.ring = ring;
    a.amax_out = amax_out;
    a.scale_out = scale_out;
    a.dbias = static_cast<uint16_t*>(dbias);
    a.fmt = fmt;
    a.defer = flags == FP8_QUANTIZE_DEFER_FOLD;
    a.offsets = offsets;
    a.experts = experts;
    // Strips of 64 columns (a row piece is one 128-byte line) unless they are
    // too few to give every SM two CTAs. Then as many CTAs as stay resident
    // together: experts first (their sums need no exchange), and to an expert
    // as many CTAs of a cluster as its mean rows can feed. Clusters of 16 only
    // where the narrowest strips would leave SMs idle in clusters of 8:
    // measured on B200 (SiLU, us, 8 against 16) 32768 x 128 20.9 -> 14.3, but
    // 2048 x 1024 8.8 -> 11.4 and 32768 x 1040 42 -> 51 (fewer of them fit a
    // GPC together).
    const int64_t sms = sm_count();
    const auto strips = [&](int w) { return (cols + w - 1) / w; };
    // Tall tensors of 296 to 1024 columns, whose clusters of 8 would not fill the
    // SMs with wider strips, take CTAs of twice the threads instead (us, ReLU /
    // GELU tanh / none): 65536 x 1024 82 / 78 / 66 -> 58 / 67 / 37, 16384 x 1024
    // 22.8 / 23.5 / 17.3 -> 19.4 / 22.2 / 14.6, 65536 x 320 45 / 49 / 33 -> 38 /
    // 39 / 28; at 2048 rows they lost (1024 columns 8.3 / 8.8 / 6.9 -> 8.3 / 9.2 /
    // 7.3) and past 1024 columns too (4096 x 1040 10.4 -> 12.1: a 33rd cluster).
    const bool tall = experts == 1 && strips(16) * 8 >= sms && cols <= 1024 && rows >= kTallRows;
    const int threads = tall ? 2 * kThreads : kThreads;
    const int64_t slots = kPerSm * kThreads / threads * sms;
    const int w = tall                                  ? (strips(32) * 8 >= sms ? 32 : 16)
                  : strips(64) * experts * 8 >= 2 * sms ? 64
                  : strips(32) * experts * 8 >= 2 * sms ? 32
                                                        : 16;
    const int max_ranks = strips(16) * experts * 8 < sms ? kMaxRanks : kPortableRanks;
    const int64_t n = strips(w);
    a.parts = int(n * experts <= slots ? experts : slots / n < 1 ? 1 : slots / n);
    const int64_t block_rows = threads / (w / 8);
    const int64_t blocks = (rows / experts + block_rows - 1) / block_rows;
    a.ranks = 1;
    while (a.ranks < max_ranks && a.ranks < blocks && n * a.parts * a.ranks * 2 <= slots) a.ranks *= 2;
    cudaStream_t st = as_stream(stream);
    if (tall)
        return w == 32 ? launch_width<32, 2 * kThreads>(a, act, n, st) : launch_width<16, 2 * kThreads>(a, act, n, st);
    if (w == 64) return launch_width<64>(a, act, n, st);
    if (w == 32) return launch_width<32>(a, act, n, st);
    return launch_width<16>(a, act, n, st);
}

}  // namespace
}  // namespace fp8lite

extern "C" fp8_status fp8_act_grad(const void* g, const void* z, int64_t rows, int64_t cols, fp8_act act, fp8_fmt fmt,
                                   fp8_ring* ring, uint32_t flags, uint8_t* out8, float* amax_out, float* scale_out,
                                   void* dbias, void* stream) {
    return act_grad_impl(g, z, rows, cols, 1, nullptr, int(act), int(fmt), ring, flags, out8, amax_out, scale_out, dbias,
                         stream);
}

extern "C" fp8_status fp8_act_grad_experts(const void* g, const void* z, int64_t rows, int64_t cols, int32_t experts,
                                           const int32_t* offsets, fp8_act act, fp8_fmt fmt, fp8_ring* ring,
                                           uint32_t flags, uint8_t* out8, float* amax_out, float* scale_out,
                                           void* dbias, void* stream) {
    if (experts < 1 || !offsets) return FP8_ERR_INVALID_ARG;
    if (experts > FP8_MM_MAX_EXPERTS) return FP8_ERR_UNSUPPORTED;
    return act_grad_impl(g, z, rows, cols, experts, offsets, int(act), int(fmt), ring, flags, out8, amax_out, scale_out,
                         dbias, stream);
}
