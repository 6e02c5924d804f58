// C ABI of the norm, the quantiser and the products with block scales.  Every check happens before the
// first HIP call.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstring>

#include "../../include/dlfusion.h"
#include "block_scale.h"
#include "checks.h"
#include "kernels.h"
#include "status.h"

namespace {

using dlf::aligned;
using dlf::any_overlap;
using dlf::fail;
using dlf::ok;
using dlf::rows_bytes;
using dlf::Span;

constexpr int32_t kMaxCols = 1 << 23;
constexpr int64_t kMaxStride = int64_t(1) << 31;
constexpr int32_t kMaxScaleStride = 1 << 20;     // 256 rows of scales are below 2^31 bytes, a buffer's size

bool known(dlf_dtype d) { return d == DLF_F32 || d == DLF_BF16 || d == DLF_FP8_E4M3; }
size_t size_of(dlf_dtype d) { return d == DLF_F32 ? 4 : d == DLF_BF16 ? 2 : 1; }
int64_t blocks_of(int64_t cols) { return (cols + dlf::kScaleBlock - 1) / dlf::kScaleBlock; }

// rows, cols and the inputs' type of the row operators
dlf_status check_rows(int64_t rows, int32_t cols, dlf_dtype dtype) {
    if (!known(dtype)) return fail(DLF_ERR_INVALID_ARG, "unknown dtype");
    if (dtype == DLF_FP8_E4M3) return fail(DLF_ERR_UNSUPPORTED, "the rows are bf16 or fp32");
    if (rows < 0 || cols < 1) return fail(DLF_ERR_INVALID_ARG, "rows must be >= 0, cols >= 1");
    if (cols > kMaxCols || rows >= (int64_t(1) << 31))
        return fail(DLF_ERR_UNSUPPORTED, "cols must be at most 2^23, rows below 2^31");
    return ok();
}

dlf_status check_stride(int64_t stride, int64_t width) {
    if (stride < width) return fail(DLF_ERR_INVALID_ARG, "a row stride is below its row");
    if (stride > kMaxStride) return fail(DLF_ERR_UNSUPPORTED, "row strides must be at most 2^31");
    return ok();
}

dlf_status check_scale_stride(int32_t stride, int64_t cols) {
    if (stride < blocks_of(cols)) return fail(DLF_ERR_INVALID_ARG, "a row of scales has fewer entries than the row has blocks");
    if (stride % 4 != 0) return fail(DLF_ERR_UNSUPPORTED, "scale strides must be multiples of 4");
    if (stride > kMaxScaleStride) return fail(DLF_ERR_UNSUPPORTED, "scale strides must be at most 2^20");
    return ok();
}

dlf_status hip_status(hipError_t e, const char* what) {
    return e == hipSuccess ? ok() : fail(DLF_ERR_HIP, "%s: %s", what, hipGetErrorString(e));
}

// Magnitude's e4m3 code, nearest with ties to even, saturating; v >= 0 and finite.
uint8_t e4m3_code(double v) {
    if (v >= 448.0) return 0x7E;
    if (v == 0.0) return 0;
    int e = 0;
    std::frexp(v, &e);                          // v in [2^(e-1), 2^e)
    const int lead = e - 1 < -6 ? -6 : e - 1;   // subnormal codes share the spacing of 2^-6
    const double q = std::nearbyint(std::ldexp(v, 3 - lead));   // eighths of 2^lead; 16 carries into the exponent
    return static_cast<uint8_t>((lead + 6) * 8 + static_cast<int>(q));
}

}  // namespace

extern "C" dlf_status dlf_rms_norm(const dlf_rms_norm_desc* d, const void* x, const void* residual, const float* weight,
                                   void* sum, void* y, float* y_scale, void* stream) {
    if (!d) return fail(DLF_ERR_INVALID_ARG, "norm descriptor is NULL");
    dlf_status st = check_rows(d->rows, d->cols, d->dtype);
    if (st != DLF_OK) return st;
    if (!known(d->out_dtype)) return fail(DLF_ERR_INVALID_ARG, "unknown dtype");
    // below, squares that fp32 holds with fewer bits, or not at all, would count beside it
    if (!std::isfinite(d->eps) || d->eps < 0x1p-100f) return fail(DLF_ERR_INVALID_ARG, "eps must be finite and at least 2^-100");
    if ((st = check_stride(d->x_stride, d->cols)) != DLF_OK || (st = check_stride(d->y_stride, d->cols)) != DLF_OK) return st;
    if (residual && (st = check_stride(d->residual_stride, d->cols)) != DLF_OK) return st;
    if (sum && (st = check_stride(d->sum_stride, d->cols)) != DLF_OK) return st;
    if (y_scale) {
        if (d->out_dtype != DLF_FP8_E4M3) return fail(DLF_ERR_INVALID_ARG, "block scales are those of an e4m3 output");
        if ((st = check_scale_stride(d->scale_stride, d->cols)) != DLF_OK) return st;
    } else if (d->out_dtype == DLF_FP8_E4M3 && (!std::isfinite(d->out_inv_scale) || d->out_inv_scale <= 0.0f)) {
        return fail(DLF_ERR_INVALID_ARG, "out_inv_scale must be finite and > 0");
    }
    if (d->rows == 0) return ok();
    if (!x || !y) return fail(DLF_ERR_INVALID_ARG, "x and y must be non-NULL");
    for (const void* p : {x, residual, static_cast<const void*>(weight), static_cast<const void*>(sum),
                          static_cast<const void*>(y), static_cast<const void*>(y_scale)})
        if (!aligned(p, 16)) return fail(DLF_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
    const size_t size = size_of(d->dtype);
    const Span xs{x, rows_bytes(d->rows, d->x_stride, d->cols, size)};
    const Span rs{residual, rows_bytes(d->rows, d->residual_stride, d->cols, size)};
    const Span ws{weight, static_cast<size_t>(d->cols) * 4};
    const Span ss{sum, rows_bytes(d->rows, d->sum_stride, d->cols, size)};
    const Span ys{y, rows_bytes(d->rows, d->y_stride, d->cols, size_of(d->out_dtype))};
    const Span cs{y_scale, rows_bytes(d->rows, d->scale_stride, d->scale_stride, 4)};
    // an output that is an input itself: each element is written by the thread that has read it
    auto itself = [&](const void* out, int64_t stride, const void* in, int64_t in_stride) {
        return out == in && stride == in_stride;
    };
    auto clash = [&](const Span& o, int64_t stride, bool same_type) {
        return (dlf::overlaps(o, xs) && !(same_type && itself(o.p, stride, x, d->x_stride))) ||
               (dlf::overlaps(o, rs) && !(same_type && itself(o.p, stride, residual, d->residual_stride)));
    };
    if (clash(ss, d->sum_stride, true) || clash(ys, d->y_stride, d->out_dtype == d->dtype) ||
        any_overlap({cs}, {xs, rs}) || any_overlap({ss, ys, cs}, {ws}))
        return fail(DLF_ERR_ALIAS, "an output overlaps an input or another output");
    dlf::RmsNormArgs a{};
    a.x = x;
    a.residual = residual;
    a.weight = weight;
    a.sum = sum;
    a.y = y;
    a.scale = y_scale;
    a.rows = d->rows;
    a.x_stride = d->x_stride;
    a.residual_stride = d->residual_stride;
    a.sum_stride = d->sum_stride;
    a.y_stride = d->y_stride;
    a.cols = d->cols;
    a.scale_stride = d->scale_stride;
    a.eps = d->eps;
    a.inv_scale = d->out_inv_scale;
    a.inv_cols = 1.0 / d->cols;
    const int out = d->out_dtype == DLF_F32 ? dlf::kOutF32 : d->out_dtype == DLF_BF16 ? dlf::kOutBf16 : dlf::kOutFp8;
    return hip_status(dlf::launch_rms_norm(a, d->dtype == DLF_F32, out, static_cast<hipStream_t>(stream)), "dlf_rms_norm");
}

extern "C" dlf_status dlf_quant_blocks(const dlf_quant_blocks_desc* d, const void* x, uint8_t* codes, float* scale,
                                       void* stream) {
    if (!d) return fail(DLF_ERR_INVALID_ARG, "quantiser descriptor is NULL");
    dlf_status st = check_rows(d->rows, d->cols, d->dtype);
    if (st != DLF_OK) return st;
    if ((st = check_stride(d->x_stride, d->cols)) != DLF_OK || (st = check_stride(d->codes_stride, d->cols)) != DLF_OK ||
        (st = check_scale_stride(d->scale_stride, d->cols)) != DLF_OK)
        return st;
    if (d->rows * blocks_of(d->cols) >= (int64_t(1) << 31)) return fail(DLF_ERR_UNSUPPORTED, "2^31 blocks or more");
    if (d->rows == 0) return ok();
    if (!x || !codes || !scale) return fail(DLF_ERR_INVALID_ARG, "x, codes and scale must be non-NULL");
    if (!aligned(x, 16) || !aligned(codes, 16) || !aligned(scale, 16))
        return fail(DLF_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
    if (any_overlap({{codes, rows_bytes(d->rows, d->codes_stride, d->cols, 1)},
                     {scale, rows_bytes(d->rows, d->scale_stride, d->scale_stride, 4)}},
                    {{x, rows_bytes(d->rows, d->x_stride, d->cols, size_of(d->dtype))}}))
        return fail(DLF_ERR_ALIAS, "an output overlaps an input or another output");
    dlf::QuantBlocksArgs a{};
    a.x = x;
    a.codes = codes;
    a.scale = scale;
    a.x_stride = d->x_stride;
    a.codes_stride = d->codes_stride;
    a.row_blocks = static_cast<int>(blocks_of(d->cols));
    a.blocks = static_cast<uint32_t>(d->rows * a.row_blocks);
    a.cols = d->cols;
    a.scale_stride = d->scale_stride;
    return hip_status(dlf::launch_quant_blocks(a, d->dtype == DLF_F32, static_cast<hipStream_t>(stream)), "dlf_quant_blocks");
}

namespace {

// the descriptor's checks; fills the kernels' sizes and their plan
dlf_status check_gemm_desc(const dlf_gemm_blocks_desc* d, dlf::GemmBlocksArgs* g) {
    if (!d) return fail(DLF_ERR_INVALID_ARG, "gemm descriptor is NULL");
    if (d->act < DLF_ACT_NONE || d->act > DLF_ACT_GELU_ERF)
        return fail(DLF_ERR_INVALID_ARG, "unknown activation %d", static_cast<int>(d->act));
    if (d->m < 0 || d->n < 0 || d->k < 0) return fail(DLF_ERR_INVALID_ARG, "negative dimension");
    if (d->k % 16 != 0) return fail(DLF_ERR_UNSUPPORTED, "k must be a multiple of 16");
    if (d->n > kMaxCols || d->k > kMaxCols || d->m > (int64_t(1) << 24) || d->m * d->n >= (int64_t(1) << 37))
        return fail(DLF_ERR_UNSUPPORTED, "n and k must be at most 2^23, m at most 2^24, m * n below 2^37");
    dlf_status st = check_scale_stride(d->a_scale_stride, d->k);
    if (st != DLF_OK || (st = check_scale_stride(d->b_scale_stride, d->k)) != DLF_OK) return st;
    *g = dlf::GemmBlocksArgs{};
    g->m = d->m;
    g->n = d->n;
    g->k = d->k;
    g->a_scale_stride = d->a_scale_stride;
    g->b_scale_stride = d->b_scale_stride;
    dlf::plan_gemm_blocks(g);
    return ok();
}

size_t gemm_ws_bytes(const dlf::GemmBlocksArgs& g) {
    return g.parts > 1 ? static_cast<size_t>(g.parts) * static_cast<size_t>(g.m) * static_cast<size_t>(g.part_stride) * 4 : 0;
}

// both products; act as launch_gemm_blocks takes it
dlf_status run_gemm(const dlf_gemm_blocks_desc* d, dlf::GemmBlocksArgs& g, const void* a, const float* a_scale, const void* b, const float* b_scale,
                    const float* shift, const void* residual, int act, void* c, void* workspace, size_t workspace_bytes,
                    void* stream, const char* what) {
    if (d->m == 0 || d->n == 0) return ok();
    const bool gated = act >= dlf::kActSiluMul;
    if (!c || (d->k > 0 && (!a || !a_scale || !b || !b_scale)))
        return fail(DLF_ERR_INVALID_ARG, "a, b, their scales and c must be non-NULL");
    for (const void* p : {a, static_cast<const void*>(a_scale), b, static_cast<const void*>(b_scale),
                          static_cast<const void*>(shift), residual, static_cast<const void*>(c),
                          static_cast<const void*>(workspace)})
        if (!aligned(p, 16)) return fail(DLF_ERR_INVALID_ARG, "device pointers must be 16-byte aligned");
    const size_t need = gemm_ws_bytes(g);
    if (need > 0 && (!workspace || workspace_bytes < need))
        return fail(DLF_ERR_INVALID_ARG, "workspace of %zu bytes needed (dlf_gemm_blocks_workspace_bytes), got %zu", need,
                    workspace ? workspace_bytes : size_t(0));
    const size_t m = static_cast<size_t>(d->m), n = static_cast<size_t>(d->n), k = static_cast<size_t>(d->k);
    const int64_t slabs = gated ? 2 * ((d->n + 2 * dlf::kScaleBlock - 1) / (2 * dlf::kScaleBlock)) : blocks_of(d->n);
    const Span cs{c, m * (gated ? n / 2 : n) * 2}, ws{workspace, need};
    if (any_overlap({cs, ws}, {{a, m * k}, {b, n * k}, {a_scale, rows_bytes(d->m, d->a_scale_stride, d->a_scale_stride, 4)},
                               {b_scale, rows_bytes(slabs, d->b_scale_stride, d->b_scale_stride, 4)}, {shift, n * 4},
                               {residual, m * n * 2}}))
        return fail(DLF_ERR_ALIAS, "the output or the workspace overlaps an operand");
    g.a = static_cast<const uint8_t*>(a);
    g.a_scale = a_scale;
    g.b = static_cast<const uint8_t*>(b);
    g.b_scale = b_scale;
    g.shift = shift;
    g.residual = static_cast<const uint16_t*>(residual);
    g.c = static_cast<uint16_t*>(c);
    g.part = static_cast<float*>(workspace);
    return hip_status(dlf::launch_gemm_blocks(g, act, static_cast<hipStream_t>(stream)), what);
}

}  // namespace

extern "C" dlf_status dlf_gemm_blocks_workspace_bytes(const dlf_gemm_blocks_desc* d, size_t* bytes) {
    if (!bytes) return fail(DLF_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    dlf::GemmBlocksArgs g;
    const dlf_status st = check_gemm_desc(d, &g);
    if (st == DLF_OK && d->m > 0 && d->n > 0) *bytes = gemm_ws_bytes(g);
    return st;
}

extern "C" dlf_status dlf_gemm_blocks(const dlf_gemm_blocks_desc* d, const void* a, const float* a_scale, const void* b,
                                      const float* b_scale, const float* col_shift, const void* residual, void* c,
                                      void* workspace, size_t workspace_bytes, void* stream) {
    dlf::GemmBlocksArgs g;
    const dlf_status st = check_gemm_desc(d, &g);
    if (st != DLF_OK) return st;
    const int act = d->act == DLF_ACT_RELU ? dlf::kActRelu : d->act == DLF_ACT_GELU_TANH ? dlf::kActGelu
                    : d->act == DLF_ACT_GELU_ERF ? dlf::kActGeluErf : dlf::kActNone;
    return run_gemm(d, g, a, a_scale, b, b_scale, col_shift, residual, act, c, workspace, workspace_bytes, stream, "dlf_gemm_blocks");
}

extern "C" dlf_status dlf_gemm_blocks_gated(const dlf_gemm_blocks_desc* d, const void* a, const float* a_scale, const void* b,
                                            const float* b_scale, const float* col_shift, dlf_gate gate, void* c,
                                            void* workspace, size_t workspace_bytes, void* stream) {
    dlf::GemmBlocksArgs g;
    const dlf_status st = check_gemm_desc(d, &g);
    if (st != DLF_OK) return st;
    if (gate < DLF_GATE_SILU || gate > DLF_GATE_GELU_ERF)
        return fail(DLF_ERR_INVALID_ARG, "unknown gate %d", static_cast<int>(gate));
    if (d->act != DLF_ACT_NONE) return fail(DLF_ERR_INVALID_ARG, "the gate is the activation: act must be NONE");
    if (d->n % 2 != 0) return fail(DLF_ERR_INVALID_ARG, "n counts gate and up rows: it must be even");
    const int act = gate == DLF_GATE_SILU ? dlf::kActSiluMul : gate == DLF_GATE_GELU_TANH ? dlf::kActGeluMul : dlf::kActGeluErfMul;
    return run_gemm(d, g, a, a_scale, b, b_scale, col_shift, nullptr, act, c, workspace, workspace_bytes, stream,
                    "dlf_gemm_blocks_gated");
}

extern "C" dlf_status dlf_quant_blocks_weights(int64_t n, int64_t k, const float* w, int32_t gated, int32_t scale_stride,
                                               uint8_t* codes, float* scale) {
    if (n < 0 || k < 0 || n > kMaxCols || k > kMaxCols) return fail(DLF_ERR_INVALID_ARG, "n and k must be 0 .. 2^23");
    if (gated != 0 && gated != 1) return fail(DLF_ERR_INVALID_ARG, "gated must be 0 or 1");
    if (gated && n % 2 != 0) return fail(DLF_ERR_INVALID_ARG, "n counts gate and up rows: it must be even");
    const int64_t blocks = blocks_of(k);
    if (scale_stride < blocks || scale_stride % 4 != 0)
        return fail(DLF_ERR_INVALID_ARG, "scale_stride must be a multiple of 4 and hold ceil(k / 128) scales");
    if (n == 0) return ok();
    if (!scale || (k > 0 && (!w || !codes))) return fail(DLF_ERR_INVALID_ARG, "NULL pointer argument");
    constexpr int64_t kB = dlf::kScaleBlock;
    const int64_t slabs = gated ? 2 * ((n + 2 * kB - 1) / (2 * kB)) : blocks_of(n);
    if (any_overlap({{codes, static_cast<size_t>(n * k)}, {scale, static_cast<size_t>(slabs * scale_stride) * 4}},
                    {{w, static_cast<size_t>(n * k) * 4}}))
        return fail(DLF_ERR_ALIAS, "an output overlaps the weights or the other output");
    for (int64_t i = 0; i < n * k; ++i)
        if (!std::isfinite(w[i])) return fail(DLF_ERR_INVALID_ARG, "weight %lld is not finite", static_cast<long long>(i));
    for (int64_t s = 0; s < slabs; ++s) {
        // the slab's rows: first, first + step, ..., below end
        const int64_t step = gated ? 2 : 1, first = gated ? s / 2 * 2 * kB + s % 2 : s * kB;
        const int64_t end = first + step * kB < n ? first + step * kB : n;
        for (int64_t t = 0; t < scale_stride; ++t) {
            float* const to = scale + s * scale_stride + t;
            *to = 0.0f;
            if (t >= blocks) continue;
            const int64_t k0 = t * kB, k1 = k0 + kB < k ? k0 + kB : k;
            double top = dlf::kLeastMax;
            for (int64_t r = first; r < end; r += step)
                for (int64_t j = k0; j < k1; ++j) top = std::fmax(top, std::fabs(static_cast<double>(w[r * k + j])));
            *to = static_cast<float>(top / 448.0);
            const double inv = static_cast<double>(*to);
            for (int64_t r = first; r < end; r += step)
                for (int64_t j = k0; j < k1; ++j) {
                    const double v = static_cast<double>(w[r * k + j]) / inv;
                    codes[r * k + j] = static_cast<uint8_t>(e4m3_code(std::fabs(v)) | (std::signbit(v) ? 0x80 : 0));
                }
        }
    }
    return ok();
}
