// FP8 GEMM with an activation and a residual in its epilogue: the kernel of
// gemm_kernel.cuh with its EP epilogue (act_tile, and the swapped one).
//
//   z = acc / (sa sb) + bias;  out = bf16(act(z) + residual), preact = bf16(z)
//
// The product, its tiles and their choice are those of fp8_mm. What the
// epilogue adds is, per output, the activation's two MUFU instructions and
// about ten others, 2 bytes of residual read and 2 of preact written.
//
// Measured on B200 (graph replay, operands from HBM; the tensor cores' share is
// of twice the measured bf16 rate, 3256 TF/s):
//   8192^3 ReLU, bias, residual                375-390 us, 0.87-0.90 of the tensor
//   2048 x 4096 x 1024 GELU tanh, preact, out8  16.3 us: the last tile's epilogue and
//                two rounds of tiles (bf16 out without activation 12.2, GELU + 2.1,
//                preact + 1, codes + 1)
//   2048 x 1024 x 4096 bias, residual           12.6 us: one round of 32 k-blocks
//   1001 x 1040 x 2064 NN residual              10.8 us: 72 tiles of 17 k-blocks
//   1 x 4096 x 4096 SiLU, residual               7.7 us, 2.15 TB/s: launch, one trip
//                to HBM and the exchange in the cluster

#include "gemm_kernel.cuh"

#include "errors.h"

using namespace fp8lite;

namespace fp8lite {

bool gemm_act_error(uint32_t* v) { return take_error_word(v); }

namespace {

struct ActOut {
    int act;
    const void* residual;
    int64_t stride_r;
    void* preact;
    bool out8;
    int out_fmt;
    fp8_ring* ring;
    float* amax;
    float* scale;
};

fp8_status mm_act_impl(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa, const float* sb,
                       fp8_layout layout, int64_t M, int64_t N, int64_t K, int64_t batch, int64_t stride_a,
                       int64_t stride_b, int64_t stride_c, const void* bias, const float* bias_scale, fp8_fmt bias_fmt,
                       const ActOut& o, void* out, void* stream) {
    if (!valid_act(o.act)) return FP8_ERR_INVALID_ARG;
    if (o.out8 && (!valid_fmt(o.out_fmt) || !o.ring || !o.scale)) return FP8_ERR_INVALID_ARG;
    const fp8_status ok = check_mm(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias,
                                   bias_scale, bias_fmt, out, o.out8 ? 1 : 4);
    if (ok != FP8_OK) return ok;
    if (M > kMaxExtent || N > kMaxExtent || K > kMaxExtent) return FP8_ERR_UNSUPPORTED;
    if (o.residual && (o.stride_r < 0 || (batch > 1 && o.stride_r != 0 && o.stride_r < M * N)))
        return FP8_ERR_INVALID_ARG;
    // out and preact are written as the tiles come: only a residual laid out as out may be out
    if (o.preact && (o.preact == out || o.preact == o.residual)) return FP8_ERR_INVALID_ARG;
    if (o.residual == out && batch > 1 && o.stride_r != stride_c) return FP8_ERR_INVALID_ARG;
    if (!aligned(o.residual, 2) || !aligned(o.preact, 2)) return FP8_ERR_ALIGNMENT;
    if (o.out8 && (!aligned(o.ring, 4) || !aligned(o.scale, 4) || !aligned(o.amax, 4))) return FP8_ERR_ALIGNMENT;
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
    if (o.out8) {
        p.out_fmt = o.out_fmt;
        p.out_ring = o.ring;
        p.out_amax = o.amax;
        p.out_scale = o.scale;
        p.tma_store = N % 16 == 0 && stride_c % 16 == 0 && aligned(out, 16);
    }
    EpArgs<true> ep = {};
    ep.act = o.act;
    ep.residual = static_cast<const uint16_t*>(o.residual);
    ep.stride_r = batch == 1 ? 0 : o.stride_r;
    ep.preact = static_cast<uint16_t*>(o.preact);
    cudaStream_t st = as_stream(stream);
    if (!o.out8 && swap_ab(M, N, layout))
        return layout == FP8_NN ? dispatch_swap<true, true>(a8, fa, b8, fb, M, N, K, batch, stride_a, stride_b, p,
                                                            nullptr, 0, 0, st, ep)
                                : dispatch_swap<false, true>(a8, fa, b8, fb, M, N, K, batch, stride_a, stride_b, p,
                                                             nullptr, 0, 0, st, ep);
    ep.fast = N % 8 == 0 && stride_c % 8 == 0 && (o.out8 || aligned(out, 16)) &&
              (!o.residual || (ep.stride_r % 8 == 0 && aligned(o.residual, 16))) && aligned(o.preact, 16);
    if (!o.out8) p.tma_store = ep.fast;
    if (ep.fast && o.preact && !make_out_map(&ep.tz, o.preact, N, M, batch, uint64_t(stride_c) * 2, 32)) return FP8_ERR_CUDA;

    CUtensorMap ta;
    const bool a_mn = layout == FP8_TN;
    if (!(a_mn ? make_map(&ta, a8, M, K, batch, uint64_t(stride_a), 128, BK)
               : make_map(&ta, a8, K, M, batch, uint64_t(stride_a), BK, BM)))
        return FP8_ERR_CUDA;
    const HostArgs h = {int(fa), int(fb), b8, batch, stride_b};
    if (o.out8) {
        switch (layout) {
            case FP8_NT: return dispatch<false, false, true, true>(ta, p, h, nullptr, 0, 1, st, ep);
            case FP8_NN: return dispatch<false, true, true, true>(ta, p, h, nullptr, 0, 1, st, ep);
            default:     return dispatch<true, true, true, true>(ta, p, h, nullptr, 0, 1, st, ep);
        }
    }
    switch (layout) {
        case FP8_NT: return dispatch<false, false, false, true>(ta, p, h, nullptr, 0, 1, st, ep);
        case FP8_NN: return dispatch<false, true, false, true>(ta, p, h, nullptr, 0, 1, st, ep);
        default:     return dispatch<true, true, false, true>(ta, p, h, nullptr, 0, 1, st, ep);
    }
}

}  // namespace
}  // namespace fp8lite

extern "C" fp8_status fp8_mm_act(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa,
                                 const float* sb, fp8_layout layout, int64_t M, int64_t N, int64_t K, int64_t batch,
                                 int64_t stride_a, int64_t stride_b, int64_t stride_c, const void* bias,
                                 const float* bias_scale, fp8_fmt bias_fmt, fp8_act act, const void* residual,
                                 int64_t stride_r, void* preact, void* out, void* stream) {
    const ActOut o = {int(act), residual, stride_r, preact, false, 0, nullptr, nullptr, nullptr};
    return mm_act_impl(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias, bias_scale,
                       bias_fmt, o, out, stream);
}

extern "C" fp8_status fp8_mm_act_out8(const uint8_t* a8, fp8_fmt fa, const uint8_t* b8, fp8_fmt fb, const float* sa,
                                      const float* sb, fp8_layout layout, int64_t M, int64_t N, int64_t K,
                                      int64_t batch, int64_t stride_a, int64_t stride_b, int64_t stride_c,
                                      const void* bias, const float* bias_scale, fp8_fmt bias_fmt, fp8_act act,
                                      void* preact, fp8_fmt out_fmt, fp8_ring* out_ring, uint8_t* out8,
                                      float* out_amax, float* out_scale, void* stream) {
    const ActOut o = {int(act), nullptr, 0, preact, true, int(out_fmt), out_ring, out_amax, out_scale};
    return mm_act_impl(a8, fa, b8, fb, sa, sb, layout, M, N, K, batch, stride_a, stride_b, stride_c, bias, bias_scale,
                       bias_fmt, o, out8, stream);
}
