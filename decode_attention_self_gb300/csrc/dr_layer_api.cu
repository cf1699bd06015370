// extern "C" boundary of the operators between a layer's attention calls: argument checks and launches.  As in
// dr_api.cu, nothing here allocates device memory or synchronises with the host.
#include <math.h>

#include "dr_layer.h"

namespace {

// The kernels look a tile past the last token in 32-bit numbers; tensor maps take strides below 2^40 bytes.  K: a bounded wait
// (2^32 cycles) spans the products of up to two tiles, at 2^24 so 2^19 chunks of 64, of 300 to 520 cycles from L2 (1400 where
// every operand comes from memory): a sixth of the limit.
constexpr int kMaxTokens = 0x7FFFF000, kMaxK = 1 << 24;
constexpr int64_t kMaxStride = 1LL << 37;

bool aligned(const void *p, int bytes) { return reinterpret_cast<uintptr_t>(p) % (uintptr_t)bytes == 0; }

bool aligned_rows(const void *p, int64_t stride_bytes) { return aligned(p, 16) && stride_bytes % 16 == 0; }

dr_status from_cuda(cudaError_t e) { return e == cudaSuccess ? DR_OK : DR_ERR_CUDA; }

// dr_linear's checks and launch; stall_tile >= 0 only from the test hook.
dr_status linear_call(const void *x, int64_t x_stride, const void *W, const dr_linear_opts *opts, int T, int K, int N,
                      const dr_linear_out *outs, int n_outs, dr_dtype out_dtype, int32_t *err_flag, bool stall,
                      int stall_tile, void *stream) {
    if (!x || !W || !outs || T < 1 || T > kMaxTokens || K < 8 || K > kMaxK || K % 8 != 0 || N < 1) return DR_ERR_INVALID_ARG;
    if (n_outs < 1 || n_outs > DR_LINEAR_MAX_OUTS) return DR_ERR_INVALID_ARG;
    if (!aligned(x, 16) || !aligned(W, 16) || x_stride < K || x_stride % 8 != 0 || x_stride > kMaxStride)
        return DR_ERR_INVALID_ARG;
    if (out_dtype != DR_BF16 && out_dtype != DR_F32) return DR_ERR_INVALID_ARG;
    const int e = out_dtype == DR_F32 ? 4 : 2;
    dr::LinearParams p;
    p.act = DR_ACT_NONE;
    p.gated = 0;
    p.bias = nullptr;
    p.residual = nullptr;
    p.res_stride = 0;
    if (opts) {
        if (opts->act < DR_ACT_NONE || opts->act > DR_ACT_SILU) return DR_ERR_INVALID_ARG;
        if (opts->gated != 0 && opts->gated != 1) return DR_ERR_INVALID_ARG;
        if (!aligned(opts->bias, 16) || !aligned(opts->residual, e)) return DR_ERR_INVALID_ARG;
        p.act = opts->act;
        p.gated = opts->gated;
        p.bias = static_cast<const uint16_t *>(opts->bias);
        p.residual = opts->residual;
        p.res_stride = opts->residual_stride;
        // one residual, one output; in place only row by row
        if (p.residual && (n_outs != 1 || p.res_stride < N || p.res_stride > kMaxStride ||
                           (p.residual == outs[0].ptr && p.res_stride != outs[0].stride && T > 1)))
            return DR_ERR_INVALID_ARG;
    }
    if (N > 0x3FFFFFFF) return DR_ERR_INVALID_ARG;   // weight rows are counted in 32 bits
    p.vec_out = 1;
    int64_t at = 0;
    for (int i = 0; i < n_outs; ++i) {
        const dr_linear_out &o = outs[i];
        if (!o.ptr || o.cols < 1 || o.stride < o.cols || o.stride > kMaxStride || !aligned(o.ptr, e)) return DR_ERR_INVALID_ARG;
        if (o.ptr == x || o.ptr == W || o.ptr == (opts ? opts->bias : nullptr)) return DR_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (outs[j].ptr == o.ptr) return DR_ERR_INVALID_ARG;
        if (i + 1 < n_outs && o.cols % 64 != 0) return DR_ERR_INVALID_ARG;
        if (!aligned_rows(o.ptr, o.stride * e)) p.vec_out = 0;
        if (at + o.cols > N) return DR_ERR_INVALID_ARG;
        p.out[i].ptr = o.ptr;
        p.out[i].stride = o.stride;
        p.out[i].col0 = (int)at;
        p.out[i].cols = o.cols;
        at += o.cols;
    }
    if (at != N) return DR_ERR_INVALID_ARG;
    for (int i = n_outs; i < DR_LINEAR_MAX_OUTS; ++i) p.out[i] = p.out[0];
    p.vec_res = p.residual && aligned_rows(p.residual, p.res_stride * e);
    p.x = static_cast<const uint16_t *>(x);
    p.x_stride = x_stride;
    p.W = static_cast<const uint16_t *>(W);
    p.n_outs = n_outs;
    p.T = T;
    p.K = K;
    p.N = N;
    p.out_f32 = out_dtype == DR_F32;
    p.err = err_flag;
    if (stall) {
        const int sms = dr::current_device_sms();
        if (sms <= 0) return DR_ERR_CUDA;
        const int tiles = dr::linear_tiles(p, sms);
        if (tiles == 0) return DR_ERR_UNSUPPORTED;
        if (stall_tile >= tiles) return DR_ERR_INVALID_ARG;
        p.stall_tile = stall_tile;
    }
    return from_cuda(dr::launch_linear(p, static_cast<cudaStream_t>(stream)));
}

bool bad_rows(const void *ptr, int64_t stride, dr_dtype type, int Dm) {
    return !aligned(ptr, 16) || stride < Dm || stride % (type == DR_F32 ? 4 : 8) != 0;
}

bool fill_norm(dr::NormParams &out, const dr_norm *n) {
    out.kind = DR_NORM_NONE;
    out.eps = 0.f;
    out.weight = out.bias = nullptr;
    if (!n || n->kind == DR_NORM_NONE) return true;
    if (n->kind != DR_NORM_LAYER && n->kind != DR_NORM_RMS) return false;
    if (!(n->eps >= 0.f) || isinf(n->eps) || !aligned(n->weight, 16) || !aligned(n->bias, 16)) return false;
    out.kind = n->kind;
    out.eps = n->eps;
    out.weight = static_cast<const uint16_t *>(n->weight);
    out.bias = static_cast<const uint16_t *>(n->bias);
    return true;
}

}  // namespace

extern "C" {

dr_status dr_linear(const void *x, int64_t x_stride, const void *W, const dr_linear_opts *opts, int T, int K, int N,
                    const dr_linear_out *outs, int n_outs, dr_dtype out_dtype, int32_t *err_flag, void *stream) {
    return linear_call(x, x_stride, W, opts, T, K, N, outs, n_outs, out_dtype, err_flag, false, -1, stream);
}

dr_status dr_linear_stall_test(const void *x, int64_t x_stride, const void *W, const dr_linear_opts *opts, int T, int K,
                               int N, const dr_linear_out *outs, int n_outs, dr_dtype out_dtype, int32_t *err_flag,
                               int stall_tile, void *stream) {
    if (stall_tile < 0) return DR_ERR_INVALID_ARG;
    return linear_call(x, x_stride, W, opts, T, K, N, outs, n_outs, out_dtype, err_flag, true, stall_tile, stream);
}

dr_status dr_residual_norm(const void *x, int64_t x_stride, dr_dtype x_dtype, const dr_norm *post, const void *gate,
                           int64_t gate_stride, float scale, const void *residual, int64_t residual_stride, void *h,
                           int64_t h_stride, dr_dtype h_dtype, const dr_norm *pre, void *y, int64_t y_stride,
                           dr_dtype y_dtype, int T, int Dm, void *stream) {
    if (!x || (!h && !y) || T < 1 || T > kMaxTokens || Dm < 8 || Dm % 8 != 0) return DR_ERR_INVALID_ARG;
    if ((x_dtype != DR_BF16 && x_dtype != DR_F32) || (h_dtype != DR_BF16 && h_dtype != DR_F32) ||
        (y_dtype != DR_BF16 && y_dtype != DR_F32))
        return DR_ERR_INVALID_ARG;
    if (bad_rows(x, x_stride, x_dtype, Dm) || (residual && bad_rows(residual, residual_stride, h_dtype, Dm)) ||
        (h && bad_rows(h, h_stride, h_dtype, Dm)) || (y && bad_rows(y, y_stride, y_dtype, Dm)))
        return DR_ERR_INVALID_ARG;
    if (gate && (!aligned(gate, 16) || gate_stride % 8 != 0 || (gate_stride != 0 && gate_stride < Dm)))
        return DR_ERR_INVALID_ARG;
    if (!(scale == scale) || isinf(scale)) return DR_ERR_INVALID_ARG;
    // in place only element by element
    const auto other = [&](const void *out, int64_t out_stride, dr_dtype out_type, const void *in, int64_t in_stride, dr_dtype in_type) {
        return out && out == in && (out_type != in_type || (T > 1 && out_stride != in_stride));
    };
    if (other(h, h_stride, h_dtype, residual, residual_stride, h_dtype) || other(h, h_stride, h_dtype, x, x_stride, x_dtype) ||
        other(y, y_stride, y_dtype, residual, residual_stride, h_dtype) || other(y, y_stride, y_dtype, x, x_stride, x_dtype))
        return DR_ERR_INVALID_ARG;
    if (gate && (gate == h || gate == y)) return DR_ERR_INVALID_ARG;
    if (h && h == y) return DR_ERR_INVALID_ARG;
    dr::ResidualNormParams p;
    if (!fill_norm(p.post, post) || !fill_norm(p.pre, pre)) return DR_ERR_INVALID_ARG;
    if (Dm > 16384) return DR_ERR_UNSUPPORTED;
    p.x = x;
    p.residual = residual;
    p.h = h;
    p.y = y;
    p.gate = static_cast<const uint16_t *>(gate);
    p.x_stride = x_stride;
    p.res_stride = residual_stride;
    p.h_stride = h_stride;
    p.y_stride = y_stride;
    p.gate_stride = gate_stride;
    p.x_f32 = x_dtype == DR_F32;
    p.res_f32 = h_dtype == DR_F32;
    p.y_f32 = y_dtype == DR_F32;
    p.scale = scale;
    p.T = T;
    p.Dm = Dm;
    return from_cuda(dr::launch_residual_norm(p, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
