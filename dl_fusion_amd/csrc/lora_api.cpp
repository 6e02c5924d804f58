// C ABI of the low-rank adapters beside a projection.  Every check happens before the first HIP call.
#include <hip/hip_runtime.h>

#include <cstdint>

#include "../../include/dlfusion.h"
#include "checks.h"
#include "kernels.h"
#include "status.h"

namespace {

using dlf::aligned;
using dlf::any_overlap;
using dlf::fail;
using dlf::ok;
using dlf::rows_bytes;

// the descriptor's checks; fills the kernels' sizes
dlf_status check_lora_desc(const dlf_lora_desc* d, dlf::LoraArgs* a) {
    if (!d) return fail(DLF_ERR_INVALID_ARG, "lora descriptor is NULL");
    if (d->dtype != DLF_BF16) {
        if (d->dtype != DLF_F32 && d->dtype != DLF_FP8_E4M3) return fail(DLF_ERR_INVALID_ARG, "unknown dtype");
        return fail(DLF_ERR_UNSUPPORTED, "the adapters are bf16 only");
    }
    if (d->m < 0 || d->n < 0 || d->k < 0 || d->rank < 0 || d->adapters < 0 || d->requests < 0)
        return fail(DLF_ERR_INVALID_ARG, "negative dimension");
    if (d->rank == 0 || d->rank % 8 != 0 || d->rank > 128)
        return fail(DLF_ERR_UNSUPPORTED, "rank must be a positive multiple of 8, at most 128 (got %d)", d->rank);
    if (d->n % 8 != 0 || d->k % 8 != 0) return fail(DLF_ERR_UNSUPPORTED, "n and k must be multiples of 8");
    if (d->n > (1 << 23) || d->k > (1 << 23)) return fail(DLF_ERR_UNSUPPORTED, "n and k must be at most 2^23");
    if (d->m > (int64_t(1) << 24)) return fail(DLF_ERR_UNSUPPORTED, "m must be at most 2^24");
    if (d->x_stride < d->k || d->base_stride < d->n || d->out_stride < d->n)
        return fail(DLF_ERR_INVALID_ARG, "a row stride is below its row");
    const int64_t lim = int64_t(1) << 31;
    if (d->x_stride % 8 != 0 || d->base_stride % 8 != 0 || d->out_stride % 8 != 0 || d->x_stride > lim ||
        d->base_stride > lim || d->out_stride > lim)
        return fail(DLF_ERR_UNSUPPORTED, "row strides must be multiples of 8, at most 2^31");
    *a = dlf::LoraArgs{};
    a->x_stride = d->x_stride;
    a->base_stride = d->base_stride;
    a->out_stride = d->out_stride;
    a->m = static_cast<int>(d->m);
    a->n = d->n;
    a->k = d->k;
    a->rank = d->rank;
    a->adapters = d->adapters;
    a->requests = d->requests;
    a->parts = d->m > 0 ? dlf::lora_parts(a->m, a->k, a->rank, a->adapters) : 1;
    return ok();
}

size_t lora_h_bytes(const dlf::LoraArgs& a) {
    return static_cast<size_t>(a.parts) * static_cast<size_t>(a.m) * static_cast<size_t>(a.rank) * 4;
}

size_t lora_ws_bytes(const dlf::LoraArgs& a) { return a.m > 0 ? lora_h_bytes(a) + 1024 : 0; }

}  // namespace

extern "C" dlf_status dlf_lora_workspace_bytes(const dlf_lora_desc* d, size_t* bytes) {
    if (!bytes) return fail(DLF_ERR_INVALID_ARG, "bytes is NULL");
    *bytes = 0;
    dlf::LoraArgs a;
    const dlf_status st = check_lora_desc(d, &a);
    if (st != DLF_OK) return st;
    *bytes = d->n > 0 ? lora_ws_bytes(a) : 0;
    return ok();
}

extern "C" dlf_status dlf_lora_add(const dlf_lora_desc* d, const void* x, const void* a_w, const void* b_w,
                                   const float* scale, const int32_t* ids, const int32_t* row_map, const void* base,
                                   void* out, void* workspace, size_t workspace_bytes, void* stream) {
    dlf::LoraArgs a;
    const dlf_status st = check_lora_desc(d, &a);
    if (st != DLF_OK || d->m == 0 || d->n == 0) return st;
    if (!ids || !out || (d->k > 0 && !x) || (d->adapters > 0 && (!b_w || (d->k > 0 && !a_w))))
        return fail(DLF_ERR_INVALID_ARG, "x, a, b, ids and out must be non-NULL");
    if (!aligned(x, 16) || !aligned(a_w, 16) || !aligned(b_w, 16) || !aligned(base, 16) || !aligned(out, 16) ||
        !aligned(scale, 4) || !aligned(ids, 4) || !aligned(row_map, 4))
        return fail(DLF_ERR_INVALID_ARG, "device pointers must be 16-byte aligned (int32 and fp32 arrays 4)");
    const size_t need = lora_ws_bytes(a);
    if (!workspace || workspace_bytes < need)
        return fail(DLF_ERR_INVALID_ARG, "workspace of %zu bytes needed (dlf_lora_workspace_bytes), got %zu", need,
                    workspace ? workspace_bytes : size_t(0));
    if (!aligned(workspace, 16)) return fail(DLF_ERR_INVALID_ARG, "workspace must be 16-byte aligned");
    const size_t m = static_cast<size_t>(d->m), adapters = static_cast<size_t>(d->adapters);
    const size_t rank = static_cast<size_t>(d->rank);
    const dlf::Span xs{x, rows_bytes(d->m, d->x_stride, d->k, 2)};
    const dlf::Span as{a_w, adapters * rank * static_cast<size_t>(d->k) * 2};
    const dlf::Span bs{b_w, adapters * rank * static_cast<size_t>(d->n) * 2};
    const dlf::Span ss{scale, adapters * 4}, ms{row_map, m * 4};
    const dlf::Span is{ids, (row_map ? static_cast<size_t>(d->requests) : m) * 4};
    const dlf::Span ys{base, rows_bytes(d->m, d->base_stride, d->n, 2)};
    const dlf::Span os{out, rows_bytes(d->m, d->out_stride, d->n, 2)}, ws{workspace, need};
    const bool in_place = base == out && d->base_stride == d->out_stride;
    if (any_overlap({os, ws}, {xs, as, bs, ss, ms, is}) || (!in_place && dlf::overlaps(os, ys)) || dlf::overlaps(ws, ys))
        return fail(DLF_ERR_ALIAS, "the output or the workspace overlaps an operand");
    a.x = static_cast<const uint16_t*>(x);
    a.a = static_cast<const uint16_t*>(a_w);
    a.b = static_cast<const uint16_t*>(b_w);
    a.scale = scale;
    a.ids = ids;
    a.row_map = row_map;
    a.base = static_cast<const uint16_t*>(base);
    a.out = static_cast<uint16_t*>(out);
    a.h = static_cast<float*>(workspace);
    a.nowhere = static_cast<uint16_t*>(workspace) + lora_h_bytes(a) / 2;
    const hipError_t e = dlf::launch_lora(a, static_cast<hipStream_t>(stream));
    if (e != hipSuccess) return fail(DLF_ERR_HIP, "dlf_lora_add: %s", hipGetErrorString(e));
    return ok();
}
