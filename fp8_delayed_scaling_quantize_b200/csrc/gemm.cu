// Entry points of the per-tensor-scaled FP8 GEMM (the kernel and its tile
// choice are in gemm_kernel.cuh): argument checks, the plain, FP8-output,
// split-K and grouped launches, and the device error word.

#include "gemm_kernel.cuh"
#include "errors.h"

using namespace fp8lite;

namespace fp8lite {
namespace {

// Diagnostic: one thread waits, through the same bounded wait the GEMM
// uses, on a shared-memory barrier that nothing ever arrives at.
__global__ void selftest_wait_kernel(uint64_t limit_ns) {
    __shared__ __align__(8) uint64_t bar;
    const uint32_t b = smem_addr(&bar);
    mbar_init(b, 1);
    fence_mbar_init();
    wait_bounded(b, 0, limit_ns);
}

// The FP8 output of fp8_mm_out8 (none for the bf16 entry points).
inline int choose_group_bn(const int64_t* M, const int64_t* N, const int64_t* kb, int count, int64_t sms);
inline int choose_narrow_tail(const int64_t* M, const int64_t* N, const int64_t* kb, int count, int64_t sms);
fp8_status mm_grouped_impl(const fp8_mm_problem* probs, int32_t count, void* stream);

struct Out8 {
    bool on;
    fp8_fmt fmt;
    fp8_ring* ring;
    float* amax;
    float* scale;
};

fp8_status mm_impl(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa, const float* sb,
                   fp8_layout layout, int64_t M, int64_t N, int64_t K, int64_t batch, int64_t stride_a,
                   int64_t stride_b, int64_t stride_c, const void* bias, const float* bias_scale, fp8_fmt bias_fmt,
                   void* out, void* workspace, size_t workspace_bytes, int32_t split_k, const Out8& o8,
                   void* stream) {
    if (split_k < 0 || split_k > kMaxSplit) return FP8_ERR_INVALID_ARG;
    if (workspace && !aligned(workspace, 16)) return FP8_ERR_ALIGNMENT;
    if (o8.on && (!valid_fmt(o8.fmt) || !o8.ring || !o8.scale)) return FP8_ERR_INVALID_ARG;
    const fp8_status st0 = check_mm(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias,
                                    bias_scale, bias_fmt, out, o8.on ? 1 : 4);
    if (st0 != FP8_OK) return st0;
    const bool a_mn = layout == FP8_TN;
    const bool b_mn = layout != FP8_NT;
    if (o8.on && (!aligned(o8.ring, 4) || !aligned(o8.scale, 4) || !aligned(o8.amax, 4))) return FP8_ERR_ALIGNMENT;
    if (batch == 1) { stride_a = 0; stride_b = 0; }

    GemmParams p = {};
    p.M = int(M);
    p.N = int(N);
    p.K = int(K);
    p.k_blocks = int((K + BK - 1) / BK);
    p.a_bcast = stride_a == 0;
    p.b_bcast = stride_b == 0;
    p.sa = sa;
    p.sb = sb;
    p.bias = bias;
    p.bias_scale = bias_scale;
    p.bias_kind = bias ? (bias_scale ? 2 : 1) : 0;
    p.bias_fmt = bias_fmt;
    p.out = static_cast<uint16_t*>(out);
    p.stride_c = stride_c;
    p.split = 1;
    if (o8.on) {  // byte codes, 16-byte vector stores where rows allow
        p.out_fmt = int(o8.fmt);
        p.out_ring = o8.ring;
        p.out_amax = o8.amax;
        p.out_scale = o8.scale;
        p.vec_store = (N % 16 == 0) && (stride_c % 16 == 0) && aligned(out, 16);
        p.tma_store = 0;
    } else {
        p.vec_store = (N % 8 == 0) && (stride_c % 8 == 0) && aligned(out, 16);
        p.tma_store = p.vec_store;
    }
    cudaStream_t st = as_stream(stream);
    // One problem whose 128 x 256 tiles leave the persistent grid's last round
    // part-empty runs as a grouped launch of one, where its rightmost columns
    // can take 128-wide tiles (choose_narrow_tail); the result is the same.
    if (!o8.on && batch == 1 && split_k <= 1 && !swap_ab(M, N, layout)) {
        const TileChoice tc = choose_tile(M, N, K, 1, b_mn, sm_count(), split_k);
        const int64_t kb1 = (K + BK - 1) / BK;
        // only where it was measured to win: at least 8 k-blocks and at most
        // two rounds of 256-wide tiles (NT 2048 x 3072 x 1024: 11.52 -> 11.01 us);
        // with more rounds or fewer k-blocks the plain 128 x 256 launch was
        // faster (4096^2 x 1024 18.9 against 21.6 us, 2048^2 x 256 5.4 against 5.6)
        if (!tc.pair && tc.bn == 256 && tc.split == 1 && kb1 >= 8 &&
            tile_count(M, N, 1, false, 256) <= 2 * int64_t(sm_count()) &&
            choose_group_bn(&M, &N, &kb1, 1, sm_count()) == 256 && choose_narrow_tail(&M, &N, &kb1, 1, sm_count()) > 0) {
            const fp8_mm_problem one = {a8, b8, sa, sb, bias, bias_scale, out, M, N, K,
                                        int32_t(fa), int32_t(fb), int32_t(layout), int32_t(bias_fmt)};
            return mm_grouped_impl(&one, 1, stream);
        }
    }
    if (!o8.on && swap_ab(M, N, layout))
        return layout == FP8_NN ? dispatch_swap<true>(a8, fa, b8, fb, M, N, K, batch, stride_a, stride_b, p, workspace,
                                                      workspace_bytes, split_k, st)
                                : dispatch_swap<false>(a8, fa, b8, fb, M, N, K, batch, stride_a, stride_b, p,
                                                       workspace, workspace_bytes, split_k, st);

    CUtensorMap ta;
    bool ok = a_mn ? make_map(&ta, a8, M, K, batch, uint64_t(stride_a), 128, BK)
                   : make_map(&ta, a8, K, M, batch, uint64_t(stride_a), BK, BM);
    if (!ok) return FP8_ERR_CUDA;
    const HostArgs h = {int(fa), int(fb), b8, batch, stride_b};
    if (o8.on) {
        switch (layout) {
            case FP8_NT: return dispatch<false, false, true>(ta, p, h, nullptr, 0, 1, st);
            case FP8_NN: return dispatch<false, true, true>(ta, p, h, nullptr, 0, 1, st);
            default:     return dispatch<true, true, true>(ta, p, h, nullptr, 0, 1, st);
        }
    }
    switch (layout) {
        case FP8_NT: return dispatch<false, false>(ta, p, h, workspace, workspace_bytes, split_k, st);
        case FP8_NN: return dispatch<false, true>(ta, p, h, workspace, workspace_bytes, split_k, st);
        default:     return dispatch<true, true>(ta, p, h, workspace, workspace_bytes, split_k, st);
    }
}


// ------------------------------------------------------- grouped launch ---

template <int BN, int STAGES, bool HAS_BIAS>
fp8_status launch_group(const GroupTab<true>& g, int total_units, cudaStream_t st) {
    using L = Smem<BN, STAGES, 1>;
    auto kern = fp8_gemm_kernel<BN, false, false, STAGES, HAS_BIAS, 1, false, false, false, true>;
    static bool attr_set[64] = {false};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return FP8_ERR_CUDA;
    if (!attr_set[dev]) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kAlloc) != cudaSuccess)
            return FP8_ERR_CUDA;
        attr_set[dev] = true;
    }
    // the kernel-wide parameters a grouped launch still reads: the unit
    // count, the walk's group height, and valid scale pointers for the
    // epilogue's set-up (every unit reloads its own problem's scales)
    GemmParams p = {};
    p.total_units = total_units;
    p.total_tiles = total_units;
    p.split = 1;
    p.group_m = 16;
    p.a_bcast = 1;
    p.b_bcast = 1;
    p.sa = g.q[0].sa;
    p.sb = g.q[0].sb;
    const int units = total_units < sm_count() ? total_units : sm_count();
    const CUtensorMap none = {};
    return launch_pdl(kern, units, kThreads, L::kAlloc, st, 1, none, none, none, p, g, EpArgs<false>{});
}

// Tile width of a grouped launch: the persistent grid hands out the units in
// rounds of `grid`, alternating direction (unit_of), so the launch lasts as
// long as its busiest CTA; this is that CTA's k-blocks (times the per-k-block
// cost of the tile width) plus one exposed epilogue, the same cost model as a
// single problem's choice. Past a few thousand units the rounds even out and
// the estimate is rounds x the longest K.
inline int choose_group_bn(const int64_t* M, const int64_t* N, const int64_t* kb, int count, int64_t sms) {
    constexpr int64_t kMaxSlots = 1024, kSimUnits = 8192;
    int best_bn = 256;
    double best = 1e30;
    for (int bn : {256, 128}) {
        const double t_k = bn == 256 ? 0.48 : 0.40, t_epi = bn == 256 ? 2.0 : 1.0;
        int64_t total = 0, kb_max = 0;
        for (int i = 0; i < count; ++i) {
            total += ((M[i] + BM - 1) / BM) * ((N[i] + bn - 1) / bn);
            kb_max = kb[i] > kb_max ? kb[i] : kb_max;
        }
        const int64_t slots = sms < kMaxSlots ? sms : kMaxSlots;
        const int64_t grid = total < slots ? total : slots;
        int64_t worst = 0;
        if (total > kSimUnits) {
            worst = ((total + grid - 1) / grid) * kb_max;
        } else {
            int64_t load[kMaxSlots] = {0};
            int64_t u = 0;
            for (int i = 0; i < count; ++i) {
                const int64_t tiles = ((M[i] + BM - 1) / BM) * ((N[i] + bn - 1) / bn);
                for (int64_t k = 0; k < tiles; ++k, ++u) {
                    const int64_t round = u / grid, pos = u - round * grid;
                    load[(round & 1) ? grid - 1 - pos : pos] += kb[i];
                }
            }
            for (int64_t c = 0; c < grid; ++c) worst = load[c] > worst ? load[c] : worst;
        }
        const double c = double(worst) * t_k + t_epi;
        if (c < best) { best = c; best_bn = bn; }
    }
    return best_bn;
}

// How many of the last problem's 256-wide column tiles (counted from its
// right edge) to run as 128-wide tiles in a 256-wide grouped launch. The
// launch's last round often holds fewer tiles than there are CTAs; a 128-wide
// tile costs about 0.28 us per k-block against 0.45 us for a 256-wide one
// (measured on B200 with this kernel), so narrower tiles at the end shorten
// the busiest CTA. Each choice is evaluated on the exact unit-to-CTA
// assignment (unit_of); 0 keeps every tile 256 wide.
inline int choose_narrow_tail(const int64_t* M, const int64_t* N, const int64_t* kb, int count, int64_t sms) {
    constexpr int64_t kMaxSlots = 1024, kSimUnits = 8192;
    const int last = count - 1;
    const int64_t n256 = (N[last] + 255) / 256;
    int best_k = 0;
    double best = 1e30;
    for (int64_t k = 0; k <= n256; ++k) {
        const int64_t n1 = (n256 - k) * 256;  // columns left 256 wide
        int64_t units[kMaxEntries], cost[kMaxEntries];  // per entry: tiles, and their cost in 0.01 us
        int e = 0;
        for (int i = 0; i < last; ++i, ++e) {
            units[e] = ((M[i] + BM - 1) / BM) * ((N[i] + 255) / 256);
            cost[e] = kb[i] * 45;
        }
        const int64_t mt = (M[last] + BM - 1) / BM;
        units[e] = mt * (n1 / 256);
        cost[e++] = kb[last] * 45;
        units[e] = mt * ((N[last] - n1 + 127) / 128);
        cost[e++] = kb[last] * 28;
        int64_t total = 0;
        for (int i = 0; i < e; ++i) total += units[i];
        if (total > kSimUnits) return 0;
        const int64_t slots = sms < kMaxSlots ? sms : kMaxSlots;
        const int64_t grid = total < slots ? total : slots;
        int64_t load[kMaxSlots] = {0};
        int64_t u = 0;
        for (int i = 0; i < e; ++i)
            for (int64_t t = 0; t < units[i]; ++t, ++u) {
                const int64_t round = u / grid, pos = u - round * grid;
                load[(round & 1) ? grid - 1 - pos : pos] += cost[i];
            }
        int64_t worst = 0;
        for (int64_t c = 0; c < grid; ++c) worst = load[c] > worst ? load[c] : worst;
        if (double(worst) < best - 1e-9) { best = double(worst); best_k = int(k); }
    }
    return best_k;
}

fp8_status mm_grouped_impl(const fp8_mm_problem* probs, int32_t count, void* stream) {
    if (!probs || count < 1 || count > kMaxGroup) return FP8_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const fp8_mm_problem& q = probs[i];
        if (!valid_fmt(q.fmt_a) || !valid_fmt(q.fmt_b)) return FP8_ERR_INVALID_ARG;
        if (q.layout != FP8_NT && q.layout != FP8_NN && q.layout != FP8_TN) return FP8_ERR_INVALID_ARG;
        if (!q.a8 || !q.b8 || !q.sa || !q.sb || !q.out) return FP8_ERR_INVALID_ARG;
        if (q.M < 1 || q.N < 1 || q.K < 1) return FP8_ERR_INVALID_ARG;
        if (q.bias_scale && !q.bias) return FP8_ERR_INVALID_ARG;
        if (q.bias && q.bias_scale && !valid_fmt(q.bias_fmt)) return FP8_ERR_INVALID_ARG;
        if (q.M >= (int64_t(1) << 31) || q.N >= (int64_t(1) << 31) || q.K >= (int64_t(1) << 31))
            return FP8_ERR_UNSUPPORTED;
        const bool a_mn = q.layout == FP8_TN, b_mn = q.layout != FP8_NT;
        if ((a_mn ? q.M : q.K) % 16 != 0 || (b_mn ? q.N : q.K) % 16 != 0) return FP8_ERR_ALIGNMENT;
        if (!aligned(q.a8, 16) || !aligned(q.b8, 16)) return FP8_ERR_ALIGNMENT;
        if (!aligned(q.out, 4) || !aligned(q.sa, 4) || !aligned(q.sb, 4)) return FP8_ERR_ALIGNMENT;
        if (q.bias && !q.bias_scale && !aligned(q.bias, 2)) return FP8_ERR_ALIGNMENT;
    }
    // longest K first: the first wave of the persistent grid starts the
    // tiles that take longest, the shorter ones fill in behind them
    int order[kMaxGroup];
    for (int i = 0; i < count; ++i) order[i] = i;
    std::stable_sort(order, order + count, [&](int x, int y) { return probs[x].K > probs[y].K; });
    int64_t M[kMaxGroup], N[kMaxGroup], kb[kMaxGroup];
    for (int i = 0; i < count; ++i) {
        M[i] = probs[order[i]].M;
        N[i] = probs[order[i]].N;
        kb[i] = (probs[order[i]].K + BK - 1) / BK;
    }
    const int bn = choose_group_bn(M, N, kb, count, sm_count());
    // entries: every problem with bn-wide tiles; in a 256-wide launch the last
    // problem's rightmost columns may form one more entry with 128-wide tiles
    const int narrow = bn == 256 ? choose_narrow_tail(M, N, kb, count, sm_count()) : 0;
    GroupTab<true> g = {};
    int64_t units = 0;
    bool any_bias = false;
    int e = 0;
    for (int i = 0; i < count; ++i) {
        const fp8_mm_problem& q = probs[order[i]];
        const bool a_mn = q.layout == FP8_TN, b_mn = q.layout != FP8_NT;
        // column ranges of this problem: [0, n1) at bn, [n1, N) at 128
        const int64_t n1 = (i == count - 1 && narrow > 0) ? ((q.N + 255) / 256 - narrow) * 256 : q.N;
        for (int part = 0; part < 2; ++part) {
            const int64_t c0 = part == 0 ? 0 : n1, c1 = part == 0 ? n1 : q.N;
            if (c1 <= c0) continue;
            const int ebn = part == 0 ? bn : 128;
            GroupProblem& d = g.q[e++];
            const bool ok = (a_mn ? make_map(&d.ta, q.a8, q.M, q.K, 1, 0, 128, BK)
                                  : make_map(&d.ta, q.a8, q.K, q.M, 1, 0, BK, BM)) &&
                            (b_mn ? make_map(&d.tb, q.b8, q.N, q.K, 1, 0, 128, BK)
                                  : make_map(&d.tb, q.b8, q.K, q.N, 1, 0, BK, uint32_t(ebn)));
            if (!ok) return FP8_ERR_CUDA;
            d.M = int(q.M);
            d.N = int(q.N);
            d.k_blocks = int(kb[i]);
            d.m_tiles = int((q.M + BM - 1) / BM);
            d.n_tiles = int((c1 - c0 + ebn - 1) / ebn);
            d.bn = ebn;
            d.n_base = int(c0);
            units += int64_t(d.m_tiles) * d.n_tiles;
            if (units >= (int64_t(1) << 31)) return FP8_ERR_UNSUPPORTED;
            d.unit_end = int(units);
            d.a_mn = a_mn;
            d.b_mn = b_mn;
            d.idesc = sm100::instr_desc_f8(q.fmt_a, q.fmt_b, a_mn, b_mn, BM, ebn);
            d.bias_kind = q.bias ? (q.bias_scale ? 2 : 1) : 0;
            d.bias_fmt = q.bias_fmt;
            any_bias = any_bias || q.bias;
            d.vec_store = (q.N % 8 == 0) && aligned(q.out, 16);
            d.tma_store = d.vec_store;
            if (d.tma_store && !make_out_map(&d.tc, q.out, q.N, q.M, 1, 0)) return FP8_ERR_CUDA;
            d.sa = q.sa;
            d.sb = q.sb;
            d.bias = q.bias;
            d.bias_scale = q.bias_scale;
            d.out = static_cast<uint16_t*>(q.out);
        }
    }
    g.count = e;
    cudaStream_t st = as_stream(stream);
    if (bn == 256)
        return any_bias ? launch_group<256, 4, true>(g, int(units), st) : launch_group<256, 4, false>(g, int(units), st);
    return any_bias ? launch_group<128, 6, true>(g, int(units), st) : launch_group<128, 6, false>(g, int(units), st);
}
}  // namespace
}  // namespace fp8lite

extern "C" fp8_status fp8_mm_ws(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa,
                                const float* sb, fp8_layout layout, int64_t M, int64_t N, int64_t K, int64_t batch,
                                int64_t stride_a, int64_t stride_b, int64_t stride_c, const void* bias,
                                const float* bias_scale, fp8_fmt bias_fmt, void* out, void* workspace,
                                size_t workspace_bytes, int32_t split_k, void* stream) {
    const Out8 none = {false, FP8_E4M3, nullptr, nullptr, nullptr};
    return mm_impl(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias, bias_scale,
                   bias_fmt, out, workspace, workspace_bytes, split_k, none, stream);
}

extern "C" fp8_status fp8_mm_out8(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa,
                                  const float* sb, fp8_layout layout, int64_t M, int64_t N, int64_t K, int64_t batch,
                                  int64_t stride_a, int64_t stride_b, int64_t stride_c, const void* bias,
                                  const float* bias_scale, fp8_fmt bias_fmt, fp8_fmt out_fmt, fp8_ring* out_ring,
                                  uint8_t* out8, float* out_amax, float* out_scale, void* stream) {
    const Out8 o8 = {true, out_fmt, out_ring, out_amax, out_scale};
    return mm_impl(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias, bias_scale,
                   bias_fmt, out8, nullptr, 0, 1, o8, stream);
}

extern "C" fp8_status fp8_mm(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa,
                             const float* sb, fp8_layout layout, int64_t M, int64_t N, int64_t K, int64_t batch,
                             int64_t stride_a, int64_t stride_b, int64_t stride_c, const void* bias,
                             const float* bias_scale, fp8_fmt bias_fmt, void* out, void* stream) {
    return fp8_mm_ws(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias, bias_scale,
                     bias_fmt, out, nullptr, 0, 0, stream);
}

extern "C" size_t fp8_mm_workspace_size(int64_t M, int64_t N, int64_t K, int64_t batch, fp8_layout layout,
                                        int32_t split_k) {
    if (M < 1 || N < 1 || K < 1 || batch < 1 || split_k < 0 || split_k > kMaxSplit) return 0;
    if (M >= (int64_t(1) << 31) || N >= (int64_t(1) << 31) || K >= (int64_t(1) << 31) || batch >= (int64_t(1) << 31))
        return 0;
    if (layout != FP8_NT && layout != FP8_NN && layout != FP8_TN) return 0;
    if (swap_ab(M, N, layout)) {
        const int split = swap_split(M, N, K, batch, split_k, sm_count());
        if (split < 2) return 0;
        return split_ws_bytes(((N + BM - 1) / BM) * batch, 1, swap_bn(M), split);
    }
    const TileChoice tc = choose_tile(M, N, K, batch, layout != FP8_NT, sm_count(), split_k);
    if (tc.split < 2) return 0;
    return split_ws_bytes(tile_count(M, N, batch, tc.pair, tc.bn), tc.pair ? 2 : 1, tc.bn, tc.split);
}

// Library-owned split-K scratch for fp8_mm_splitk_static: the counter block
// (kSplitCntBytes) followed by the fp32 partial tiles. One array per device
// that loads the library, held until the process exits, shared by every call
// on that device. Host code may not use the symbol itself as a pointer: on
// the host it names a stand-in, not device memory, so the device address is
// looked up once per device (scratch_address) and passed to the kernel.
constexpr size_t kStaticScratchBytes = size_t(32) << 20;
__device__ __align__(256) uint8_t g_splitk_scratch[kStaticScratchBytes];

namespace fp8lite {
namespace {

// The scratch's device address on the current device, looked up on the first
// call made with that device current and kept for later calls. The lookup may
// load the library's GEMM module on that device, which stream capture does not
// allow: the first call on a device must come before any capture.
void* scratch_address() {
    constexpr int kMaxDevices = 64;
    static void* addr[kMaxDevices] = {};
    static std::mutex mu;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) return nullptr;
    std::lock_guard<std::mutex> lock(mu);
    if (!addr[dev]) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_splitk_scratch) != cudaSuccess) return nullptr;
        addr[dev] = p;
    }
    return addr[dev];
}

}  // namespace
}  // namespace fp8lite

extern "C" fp8_status fp8_mm_splitk_static(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb,
                                           const float* sa, const float* sb, fp8_layout layout, int64_t M, int64_t N,
                                           int64_t K, int64_t batch, int64_t stride_a, int64_t stride_b,
                                           int64_t stride_c, const void* bias, const float* bias_scale,
                                           fp8_fmt bias_fmt, void* out, int32_t split_k, void* stream) {
    if (split_k < 2 || split_k > kMaxSplit) return FP8_ERR_INVALID_ARG;
    const size_t need = fp8_mm_workspace_size(M, N, K, batch, layout, split_k);
    if (need > kStaticScratchBytes) return FP8_ERR_UNSUPPORTED;
    void* scratch = scratch_address();
    if (!scratch) return FP8_ERR_CUDA;
    // The counters must be zero when the GEMM starts. A completed call leaves
    // them zero, but a call whose bounded wait gave up may not; clearing them
    // on the caller's stream makes every call start clean. The partial tiles
    // need no clearing: each is written before it is read.
    if (need > 0 && cudaMemsetAsync(scratch, 0, kSplitCntBytes, as_stream(stream)) != cudaSuccess)
        return FP8_ERR_CUDA;
    // fp8_mm_ws validates the rest (and reports a split the problem cannot take)
    return fp8_mm_ws(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias, bias_scale,
                     bias_fmt, out, scratch, kStaticScratchBytes, split_k, stream);
}

extern "C" fp8_status fp8_last_device_error(void) {
    if (cudaDeviceSynchronize() != cudaSuccess) return FP8_ERR_CUDA;
    uint32_t v[3] = {0, 0, 0};
    if (!take_error_word(&v[0]) || !gemm_act_error(&v[1]) || !experts_error(&v[2])) return FP8_ERR_CUDA;
    return (v[0] | v[1] | v[2]) ? FP8_ERR_DEVICE_TIMEOUT : FP8_OK;
}

extern "C" fp8_status fp8_selftest_wait_timeout(uint32_t limit_us, void* stream) {
    if (limit_us == 0 || limit_us > 1000000u) return FP8_ERR_INVALID_ARG;
    selftest_wait_kernel<<<1, 1, 0, as_stream(stream)>>>(uint64_t(limit_us) * 1000ull);
    return launch_status();
}

extern "C" fp8_status fp8_mm_grouped(const fp8_mm_problem* problems, int32_t count, void* stream) {
    return mm_grouped_impl(problems, count, stream);
}
