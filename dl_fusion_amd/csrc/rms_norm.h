// Root-mean-square norm of rows with the residual's addition, and the quantiser of rows into e4m3 codes
// with a scale for each 128 columns.
//
//     h = x [+ residual],  sum = h,  y = h / sqrt(mean(h^2) + eps) * weight
//
// Both read each value once and write each output once, and have nothing to compute beside: HBM bounds them,
// or the launch where there are few rows.  A thread holds 8 neighbouring columns at a time, so that a row
// is read in whole lines and 16 neighbouring lanes hold a block of 128 columns: its largest magnitude is a
// maximum over those lanes, no LDS.
//
// On the device, from a graph: 8192 rows of 4096 bf16 columns with residual and sum into codes 42 to 44 us (5.4 to 5.6 TB/s; a copy
// reaches 5.2), 64 rows 3.3 to 3.5 us, one row into bf16 2.6 to 2.9 us, against 2.2 us of an empty kernel; the quantiser 8192 rows of
// 4096 columns 20 us (5.0 TB/s), 64 rows 2.3.  Rows that do not start at 16 bytes cost up to a quarter more (8192 x 4096, us: stride
// 4096 | 4097, bf16 output 45 | 57, codes 44 | 51; 4095 columns close together 61 and 56; fp32 rows nothing).  Two kinds of rows are
// far from their bytes: short ones, a wave each however few lanes they fill (262144 x 128 without residual 75 us, 26 of bytes), and
// those above 16384 columns, which are read twice (1024 x 20000 with residual and sum 43 us, 32 of bytes).
#pragma once

#include "block_scale.h"
#include "kernels.h"

namespace dlf {
namespace {

enum : int { kYBf16 = 0, kYF32 = 1, kYStatic = 2, kYBlocks = 3 };

// 16 bytes at any address that the element type allows: rows of odd width or stride start anywhere, and the
// hardware takes such loads.
typedef u32x4_t u32x4_any_t __attribute__((aligned(2)));
typedef f32x4_t f32x4_any_t __attribute__((aligned(4)));
typedef uint32_t u32x2_any_t __attribute__((ext_vector_type(2), aligned(1)));

template <bool STREAM, typename V>
__device__ __forceinline__ V get(const V* p) {
    if constexpr (STREAM) return __builtin_nontemporal_load(p);
    else return *p;
}
template <bool STREAM, typename V>
__device__ __forceinline__ void put(V* p, V v) {
    if constexpr (STREAM) __builtin_nontemporal_store(v, p);
    else *p = v;
}

// 8 values as they lie in memory: loaded and looked at in two steps, so that the loads of all tensors are on their way together.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    u32x4_t x;
    template <bool STREAM>
    __device__ __forceinline__ void load(const uint16_t* p) { x = get<STREAM>(reinterpret_cast<const u32x4_any_t*>(p)); }
    __device__ __forceinline__ void to(float* v) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(x[i] << 16);
            v[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        }
    }
};
template <>
struct Raw8<float> {
    f32x4_t a, b;
    template <bool STREAM>
    __device__ __forceinline__ void load(const float* p) {
        a = get<STREAM>(reinterpret_cast<const f32x4_any_t*>(p));
        b = get<STREAM>(reinterpret_cast<const f32x4_any_t*>(p + 4));
    }
    __device__ __forceinline__ void to(float* v) const {
#pragma unroll
        for (int i = 0; i < 4; ++i) { v[i] = a[i]; v[4 + i] = b[i]; }
    }
};
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ float load1(const float* p) { return *p; }

// Columns at .. at + 7 of a row, zeros behind its end.  What reaches past the end is loaded as the row's last 8 values and moved
// down in registers (end_chunk), so that no load stands behind a branch (8192 rows of 4095 columns, us: value by value 75,
// so 51).  Rows of less than 8 columns are SHORT, and loaded value by value.  A chunk that begins past the end is zeros.
template <bool STREAM, typename T>
__device__ __forceinline__ Raw8<T> load_chunk(const T* row, int at, int cols) {
    Raw8<T> r;
    r.template load<STREAM>(row + (at + 8 <= cols ? at : cols - 8));
    return r;
}
__device__ __forceinline__ void end_chunk(int at, int cols, float* v) {
    const int back = at + 8 - cols;
    if (back > 0) {
#pragma unroll
        for (int d = 1; d < 8; d *= 2)
#pragma unroll
            for (int i = 0; i < 8; ++i) v[i] = back & d ? (i + d < 8 ? v[i + d] : 0.0f) : v[i];
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] = back < 8 ? v[i] : 0.0f;
    }
}

template <bool STREAM>
__device__ __forceinline__ void store_chunk(uint16_t* p, int n, const float* v) {
    if (n >= 8) {
        u32x4_t x;
#pragma unroll
        for (int i = 0; i < 4; ++i) x[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
        put<STREAM, u32x4_any_t>(reinterpret_cast<u32x4_any_t*>(p), x);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = f32_to_bf16(v[i]);
    }
}
template <bool STREAM>
__device__ __forceinline__ void store_chunk(float* p, int n, const float* v) {
    if (n >= 8) {
        put<STREAM, f32x4_any_t>(reinterpret_cast<f32x4_any_t*>(p), f32x4_t{v[0], v[1], v[2], v[3]});
        put<STREAM, f32x4_any_t>(reinterpret_cast<f32x4_any_t*>(p + 4), f32x4_t{v[4], v[5], v[6], v[7]});
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = v[i];
    }
}
template <bool STREAM>
__device__ __forceinline__ void store_codes(uint8_t* p, int n, const float* v, float inv) {
    const uint32_t lo = e4m3_x4(v, inv), hi = e4m3_x4(v + 4, inv);
    if (n >= 8) {
        put<STREAM, u32x2_any_t>(reinterpret_cast<u32x2_any_t*>(p), u32x2_any_t{lo, hi});
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) p[i] = static_cast<uint8_t>((i < 4 ? lo : hi) >> (8 * (i & 3)));
    }
}

// The block of the 16 lanes that hold 8 columns each: its scale, and the codes.  Lanes past the row's end
// hold zeros.
template <bool STREAM>
__device__ __forceinline__ void store_block(const float* v, int n, int lane, uint8_t* codes, float* scale) {
    float top = kLeastMax;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = fmaxf(top, finite_abs(v[i]));
#pragma unroll
    for (int d = 8; d > 0; d >>= 1) top = fmaxf(top, __shfl_xor(top, d));
    if (n > 0) {
        if ((lane & 15) == 0) *scale = top / 448.0f;
        store_codes<STREAM>(codes, n, v, 448.0f / top);
    }
}

// 1 / sqrt(m), rounded once; 0 of an infinity.  The instruction is off by 2^-24 (measured), one Newton step squares that.  In
// fp32 the mean, eps, the root and its reciprocal round four times, and take longer (4099 x 1023 fp32, error against 64 bits and
// time in a graph: 5.9e-8 and 9.2 us | 5.1e-8 and 8.9 us).
__device__ __forceinline__ float rsqrt_once(double m) {
    const double r = __builtin_amdgcn_rsq(m);
    return m < INFINITY || m != m ? static_cast<float>(fma(fma(-m * r, r, 1.0), 0.5 * r, r)) : 0.0f;
}

// A row per group of TPR threads, V chunks of 8 columns a thread in registers; V = 0: rows beyond that, read
// again from memory for the second pass.  Each element is read by the thread that writes it, and written after
// both passes have read it or in place of it: sum and y may be an input itself.
template <typename T, int OUT, int TPR, int V, bool STREAM, bool SHORT = false>
__global__ __launch_bounds__(TPR == 64 ? 256 : TPR, V == 1 ? 8 : 4) void rms_norm_kernel(const RmsNormArgs p) {
    constexpr int kRows = TPR == 64 ? 4 : 1;        // a workgroup has several rows only where a row is a wave's: no barrier
    constexpr int kWaves = TPR / 64;
    __shared__ float part[kWaves];
    const int tid = kRows > 1 ? static_cast<int>(threadIdx.x) % TPR : static_cast<int>(threadIdx.x), lane = tid & 63;
    const int cols = p.cols;
    const float* const w = p.weight;
    // every thread of a workgroup takes as many turns: the barriers below are met by all
    for (int64_t row0 = static_cast<int64_t>(blockIdx.x) * kRows; row0 < p.rows; row0 += static_cast<int64_t>(gridDim.x) * kRows) {
        const int64_t row = kRows > 1 ? row0 + __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) / TPR) : row0;  // uniform
        if (kRows > 1 && row >= p.rows) return;
        const T* const x = static_cast<const T*>(p.x) + row * p.x_stride;
        const T* const res = p.residual ? static_cast<const T*>(p.residual) + row * p.residual_stride : nullptr;
        T* const sum = p.sum ? static_cast<T*>(p.sum) + row * p.sum_stride : nullptr;
        auto load_h = [&](int at, float* h) __attribute__((always_inline)) {
            if constexpr (SHORT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    h[i] = load1(x + (i < cols ? i : 0));
                    if (res) h[i] += load1(res + (i < cols ? i : 0));
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] = at + i < cols ? h[i] : 0.0f;
                return;
            }
            const Raw8<T> a = load_chunk<STREAM>(x, at, cols);
            Raw8<T> b;
            if (res) b = load_chunk<STREAM>(res, at, cols);
            // both on their way before the first is waited for (8192 rows of 4096 columns, us: 45.7 | 41.8)
            __builtin_amdgcn_sched_barrier(0);
            a.to(h);
            if (res) {
                float r[8];
                b.to(r);
#pragma unroll
                for (int i = 0; i < 8; ++i) h[i] += r[i];
            }
            end_chunk(at, cols, h);
        };
        auto all_sum = [&](float s) __attribute__((always_inline)) {
#pragma unroll
            for (int d = 32; d > 0; d >>= 1) s += __shfl_xor(s, d);
            if constexpr (kWaves > 1) {
                __syncthreads();                        // the last sum has been read
                if (lane == 0) part[tid / 64] = s;
                __syncthreads();
                s = 0.0f;
#pragma unroll
                for (int i = 0; i < kWaves; ++i) s += part[i];
            }
            return s;
        };
        // The weights of a single chunk come with the row, and not behind its sum.  (Those of two would take 88 registers instead of
        // 66, and waves with them: 4096 rows of 8192 columns, us: 53.4 | 48.1.)
        constexpr bool kEarly = V == 1 && !SHORT;
        Raw8<float> early[kEarly ? V : 1];
        float h[V > 0 ? V : 1][8];
        auto squares = [&](float factor) __attribute__((always_inline)) {
            auto add = [&](float s, const float* v) __attribute__((always_inline)) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    const float u = v[i] * factor;
                    s = fmaf(u, u, s);
                }
                return s;
            };
            float s = 0.0f;
            if constexpr (V > 0) {
#pragma unroll
                for (int j = 0; j < V; ++j) s = add(s, h[j]);
            } else {
                // thousands of values a thread: chunks are added in 64 bits (in fp32 alone, 2^23 columns of 1.1 were off by 470 2^-24)
                double all = 0.0;
                for (int at = 8 * tid; at < cols; at += 8 * TPR) {
                    load_h(at, h[0]);
                    all += static_cast<double>(add(0.0f, h[0]));
                }
                s = static_cast<float>(all);
            }
            return all_sum(s);
        };
        if constexpr (V > 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
                const int at = 8 * (tid + j * TPR);
                if (kEarly && w) early[kEarly ? j : 0] = load_chunk<false>(w, at, cols);
                load_h(at, h[j]);
            }
        }
        float total = squares(1.0f);
        float factor = 1.0f;
        double eps = p.eps;
        if (__builtin_expect(total == INFINITY, 0)) {
            // past fp32's range, or an infinity among them: the row, and eps with it, 2^-80 times as large (2^23 squares of
            // 2^48 fit); h * r itself would need an r below the normal numbers
            factor = 0x1p-80f;
            eps *= 0x1p-160;
            total = squares(factor);
        }
        const float r = rsqrt_once(static_cast<double>(total) * p.inv_cols + eps);
        auto finish = [&](int at, int j, const float* v) __attribute__((always_inline)) {
            const int n = cols - at;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = v[i] * factor * r;
            if (w) {
                float f[8];
                if constexpr (SHORT) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = i < n ? load1(w + i) : 0.0f;
                } else {
                    if constexpr (kEarly) early[j].to(f);
                    else load_chunk<false>(w, at, cols).to(f);
                    end_chunk(at, cols, f);
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) y[i] *= f[i];
            }
            if (sum && n > 0) store_chunk<STREAM>(sum + at, n, v);
            if constexpr (OUT == kYBlocks) {
                if (n < 8) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) y[i] = i < n ? y[i] : 0.0f;     // 0 x infinity past the end
                }
                store_block<STREAM>(y, n, lane, static_cast<uint8_t*>(p.y) + row * p.y_stride + at,
                            p.scale + row * p.scale_stride + at / kScaleBlock);
            } else if (n > 0) {
                if constexpr (OUT == kYBf16) store_chunk<STREAM>(static_cast<uint16_t*>(p.y) + row * p.y_stride + at, n, y);
                else if constexpr (OUT == kYF32) store_chunk<STREAM>(static_cast<float*>(p.y) + row * p.y_stride + at, n, y);
                else store_codes<STREAM>(static_cast<uint8_t*>(p.y) + row * p.y_stride + at, n, y, p.inv_scale);
            }
        };
        if constexpr (V > 0) {
#pragma unroll
            for (int j = 0; j < V; ++j) finish(8 * (tid + j * TPR), j, h[j]);
        } else {
            // all lanes of a block's 16 go together
            for (int base = 0; base < cols; base += 8 * TPR) {
                const int at = base + 8 * tid;
                load_h(at, h[0]);
                finish(at, 0, h[0]);
            }
        }
    }
}

// 16 lanes a block of 128 columns, blocks numbered row by row; U of them a thread, whose loads are all on their way
// before the first is used.
template <typename T, int U, bool STREAM, bool SHORT = false>
__global__ __launch_bounds__(256) void quant_blocks_kernel(const QuantBlocksArgs p) {
    const int lane = static_cast<int>(threadIdx.x) & 15;
    for (uint32_t first = blockIdx.x * (16 * U) + threadIdx.x / 16; first < p.blocks; first += gridDim.x * (16 * U)) {
        Raw8<T> raw[U];
        uint32_t row[U], b[U];
        int at[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t block = first + 16 * u < p.blocks ? first + 16 * u : first;     // the first again: as it is
            row[u] = block / static_cast<uint32_t>(p.row_blocks);
            b[u] = block - row[u] * static_cast<uint32_t>(p.row_blocks);
            at[u] = static_cast<int>(b[u]) * kScaleBlock + 8 * lane;
            if constexpr (!SHORT) raw[u] = load_chunk<STREAM>(static_cast<const T*>(p.x) + row[u] * p.x_stride, at[u], p.cols);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float v[8];
            if constexpr (SHORT) {
#pragma unroll
                for (int i = 0; i < 8; ++i) v[i] = at[u] + i < p.cols ? load1(static_cast<const T*>(p.x) + row[u] * p.x_stride + i) : 0.0f;
            } else {
                raw[u].to(v);
                end_chunk(at[u], p.cols, v);
            }
            store_block<STREAM>(v, p.cols - at[u], lane, p.codes + row[u] * p.codes_stride + at[u],
                                p.scale + static_cast<int64_t>(row[u]) * p.scale_stride + b[u]);
        }
    }
}

constexpr unsigned kMostGroups = 1u << 20;      // workgroups of a launch; what is beyond comes round again

// Bytes from which on loads and stores are non-temporal: what is written does not stay in the 32 MB of the L2s anyway.
// Measured with a residual, 4096 columns, bf16 to codes (us, cached | non-temporal): 512 rows 5.2 | 5.3, 2048 13.4 | 13.9,
// 4096 28.0 | 25.5, 8192 51.7 | 46.1; the quantiser, 11008 columns: 4096 rows 31.4 | 28.9, 8192 59.7 | 54.8.
constexpr int64_t kStreamBytes = int64_t(64) << 20;

// One chunk of 8 columns a thread up to 4096 columns: a row is short, its few barriers and loads one after another are what it
// takes (64 rows of 4096: 256 threads 4.4 us, 512 3.5, 1024 4.4; 8192 rows 46.5 | 46.1 | 46.6).  Beyond, 512 threads: 1024 take
// 4.4 us instead of 4.8 for 64 rows of 8192, but 63 instead of 48 for 4096 rows.
template <typename T, int OUT, bool STREAM>
hipError_t launch(const RmsNormArgs& a, hipStream_t s) {
    auto go = [&](auto kernel, int tpr) {
        const int rows = tpr == 64 ? 4 : 1;
        const int64_t groups = (a.rows + rows - 1) / rows;
        kernel<<<groups < kMostGroups ? static_cast<unsigned>(groups) : kMostGroups, tpr == 64 ? 256 : tpr, 0, s>>>(a);
        return hipGetLastError();
    };
    if (a.cols < 8) return go(rms_norm_kernel<T, OUT, 64, 1, STREAM, true>, 64);
    if (a.cols <= 512) return go(rms_norm_kernel<T, OUT, 64, 1, STREAM>, 64);
    if (a.cols <= 1024) return go(rms_norm_kernel<T, OUT, 128, 1, STREAM>, 128);
    if (a.cols <= 2048) return go(rms_norm_kernel<T, OUT, 256, 1, STREAM>, 256);
    if (a.cols <= 4096) return go(rms_norm_kernel<T, OUT, 512, 1, STREAM>, 512);
    if (a.cols <= 8192) return go(rms_norm_kernel<T, OUT, 512, 2, STREAM>, 512);
    if (a.cols <= 16384) return go(rms_norm_kernel<T, OUT, 512, 4, STREAM>, 512);
    return go(rms_norm_kernel<T, OUT, 1024, 0, STREAM>, 1024);
}

template <typename T, int OUT>
hipError_t launch_stream(const RmsNormArgs& a, hipStream_t s) {
    const int64_t bytes = a.rows * a.cols * (sizeof(T) * (1 + (a.residual != nullptr) + (a.sum != nullptr)) + (OUT == kYF32 ? 4 : OUT == kYBf16 ? 2 : 1));
    return bytes >= kStreamBytes ? launch<T, OUT, true>(a, s) : launch<T, OUT, false>(a, s);
}

template <typename T>
hipError_t launch_out(const RmsNormArgs& a, int out, hipStream_t s) {
    switch (out) {
        case kOutBf16: return launch_stream<T, kYBf16>(a, s);
        case kOutF32: return launch_stream<T, kYF32>(a, s);
        default: return a.scale ? launch_stream<T, kYBlocks>(a, s) : launch_stream<T, kYStatic>(a, s);
    }
}

template <typename T>
hipError_t launch_quant(const QuantBlocksArgs& a, hipStream_t s) {
    const bool stream = a.cols >= 8 && static_cast<int64_t>(a.blocks) * kScaleBlock * (sizeof(T) + 1) >= kStreamBytes;
    // two blocks a thread cost 0.5 us where there are few, and gain 4% where there are many
    const unsigned each = stream ? 32 : 16, all = (a.blocks + each - 1) / each, groups = all < kMostGroups ? all : kMostGroups;
    if (a.cols < 8) quant_blocks_kernel<T, 1, false, true><<<groups, 256, 0, s>>>(a);
    else if (stream) quant_blocks_kernel<T, 2, true><<<groups, 256, 0, s>>>(a);
    else quant_blocks_kernel<T, 1, false><<<groups, 256, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace
}  // namespace dlf
