// Low-rank adapters of many requests beside a shared projection:
//     out[i] = base[i] + scale[a] (x[i] A_a^T) B_a^T,   a the adapter of row i.
//
// Two kernels, since the second product needs the first one's sum over all of k: h = x A^T in fp32
// through a workspace (m x rank, small beside x and out), then out.  2 m rank (k + n) flops over x,
// base, out and the used adapters' weights: at rank 64 about 60 flops a byte, so both are bound by
// what they read, and the matrix cores serve to keep everything else out of the way.
//
// Rows of one adapter are gathered per tile of 64 rows: a wave holds the tile's adapters one a lane,
// and a ballot gives the rows that share the first one left, so any order of rows is served, a run of
// one adapter in one pass over the tile, 64 different ones in 64 passes of one row each (each reads
// only its own weights, which has to happen anyway).  The passes of a tile are spread over gridDim's
// slots where there are few tiles.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"

namespace dlf {
namespace {

constexpr int kTileRows = 64;
constexpr int kWaves = 4;

// The adapter of row `row`, -1 for none.
__device__ __forceinline__ int adapter_of(const LoraArgs& p, int row) {
    if (row >= p.m) return -1;
    int at = row;
    if (p.row_map) {
        at = p.row_map[row];
        if (at < 0 || at >= p.requests) return -1;
    }
    const int id = p.ids[at];
    return id >= 0 && id < p.adapters ? id : -1;
}

// f(adapter, lanes) for every different adapter of the wave's 64 rows (-1 among them) whose turn is
// this slot's; `there`: the lanes that have a row.
template <class Fn>
__device__ __forceinline__ void for_each_adapter(int id, uint64_t there, int slot, int slots, Fn&& f) {
    int turn = 0;
    while (there) {
        const int cur = __builtin_amdgcn_readlane(id, __builtin_ctzll(there));
        const uint64_t same = __ballot(id == cur) & there;
        there &= ~same;
        if (turn == slot) f(cur, same);
        turn = turn + 1 == slots ? 0 : turn + 1;
    }
}

// In lane i the place (0..63) of the i-th set bit of `lanes`; past the last one, of the first.
__device__ __forceinline__ int nth_lane(uint64_t lanes, int lane) {
    const int rank = __popcll(lanes & ((uint64_t(1) << lane) - 1));
    const int first = __builtin_ctzll(lanes);
    int place = first;
    const int to = lanes >> lane & 1 ? rank : 63;      // lane 63's value is used only when all 64 are set
    const int got = __builtin_amdgcn_ds_permute(4 * to, lane);
    if (lane < __popcll(lanes)) place = got;
    return place;
}

// ---- h = x A^T: a workgroup takes a tile, an adapter and a slice of k ----
// RF: 16-rank fragments.  The products are computed transposed (ranks x rows), so that a lane ends up
// with four neighbouring ranks of one row.  Operands come straight from memory: a lane's 16 bytes of a
// row are its MFMA operand.  The waves take k in turns of 64 (a cache line of a row) and are added
// through LDS.
template <int RF>
__global__ __launch_bounds__(64 * kWaves, RF == 8 ? 1 : 2) void lora_shrink_kernel(const LoraArgs p) {
    constexpr int kRound = 4;      // fragments a wave hands over at a time
    __shared__ f32x4_t sum_s[kWaves][kRound][64];
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int row0 = static_cast<int>(blockIdx.x) * kTileRows;
    const int part = static_cast<int>(blockIdx.z);
    const int units = (p.k + 63) / 64;
    const int u0 = static_cast<int>(static_cast<int64_t>(units) * part / p.parts);
    const int u1 = static_cast<int>(static_cast<int64_t>(units) * (part + 1) / p.parts);
    const int id = adapter_of(p, row0 + lane);

    auto pass = [&](auto nf_c, int cur, uint64_t same) {
        constexpr int NF = decltype(nf_c)::value;      // 16-row fragments
        const int count = __popcll(same);
        const int place = nth_lane(same, lane);
        const uint16_t* xr[NF];
        int row[NF];
#pragma unroll
        for (int f = 0; f < NF; ++f) {
            // places past the last row repeat the first: computed, never stored
            row[f] = row0 + __shfl(place, 16 * f + li);
            xr[f] = p.x + row[f] * p.x_stride + 8 * g;
        }
        const uint16_t* ar[RF];
#pragma unroll
        for (int c = 0; c < RF; ++c) {
            const int rk = 16 * c + li < p.rank ? 16 * c + li : p.rank - 1;
            ar[c] = p.a + (static_cast<int64_t>(cur) * p.rank + rk) * p.k + 8 * g;
        }
        f32x4_t acc[RF][NF];
#pragma unroll
        for (int c = 0; c < RF; ++c)
#pragma unroll
            for (int f = 0; f < NF; ++f) acc[c][f] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
        for (int u = u0 + wave; u < u1; u += kWaves) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                const int k0 = 64 * u + 32 * s;
                u32x4_t xv[NF], av[RF];
                const bool in = k0 + 8 * g < p.k;       // k is a multiple of 8
#pragma unroll
                for (int f = 0; f < NF; ++f) xv[f] = in ? *reinterpret_cast<const u32x4_t*>(xr[f] + k0) : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                for (int c = 0; c < RF; ++c) av[c] = in ? *reinterpret_cast<const u32x4_t*>(ar[c] + k0) : u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                for (int c = 0; c < RF; ++c)
#pragma unroll
                    for (int f = 0; f < NF; ++f)
                        acc[c][f] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, av[c]),
                                                                            __builtin_bit_cast(bf16x8_t, xv[f]), acc[c][f], 0, 0, 0);
            }
        }
        // lane: ranks 16 c + 4 g .. + 3 of row fragment f's row li
        constexpr int kAll = RF * NF;
#pragma unroll
        for (int r = 0; r < kAll; r += kRound) {
            __syncthreads();
#pragma unroll
            for (int i = 0; i < kRound; ++i)
                if (r + i < kAll) sum_s[wave][i][lane] = acc[(r + i) / NF][(r + i) % NF];
            __syncthreads();
            // wave w adds fragment r + w of all four
            if (r + wave < kAll) {
                f32x4_t v = sum_s[0][wave][lane];
#pragma unroll
                for (int w = 1; w < kWaves; ++w) v += sum_s[w][wave][lane];
                const int c = (r + wave) / NF, f = (r + wave) % NF;
                const int rk = 16 * c + 4 * g;
                const int at = 16 * f + li;
                int to = row[0];
#pragma unroll
                for (int i = 1; i < NF; ++i) to = f == i ? row[i] : to;
                if (at < count && rk < p.rank)
                    *reinterpret_cast<f32x4_t*>(p.h + (static_cast<int64_t>(part) * p.m + to) * p.rank + rk) = v;
            }
        }
    };
    for_each_adapter(id, __ballot(row0 + lane < p.m), static_cast<int>(blockIdx.y), static_cast<int>(gridDim.y),
                     [&](int cur, uint64_t same) {
                         if (cur < 0) return;
                         if (__popcll(same) <= 16) pass(std::integral_constant<int, 1>{}, cur, same);
                         else pass(std::integral_constant<int, 4>{}, cur, same);
                     });
}

// ---- out = base + scale h B^T: a workgroup takes a tile, an adapter and 256 columns, a wave 64 ----
// RS: steps of 32 ranks.  Again transposed (columns x rows).  Fragment i's row m stands for column
// 16 (m / 4) + 4 i + m % 4 of the wave's 64, so that the four fragments leave a lane with 16
// neighbouring columns of its row: base and out move 32 bytes a lane, a line a row.
template <int RS>
__global__ __launch_bounds__(64 * kWaves) void lora_expand_kernel(const LoraArgs p) {
    const int lane = static_cast<int>(threadIdx.x) & 63, wave = static_cast<int>(threadIdx.x) >> 6;
    const int li = lane & 15, g = lane >> 4;
    const int row0 = static_cast<int>(blockIdx.x) * kTileRows;
    const int n0 = static_cast<int>(blockIdx.y) * 64 * kWaves + 64 * wave;
    if (n0 >= p.n) return;
    const int id = adapter_of(p, row0 + lane);
    for_each_adapter(id, __ballot(row0 + lane < p.m), static_cast<int>(blockIdx.z), static_cast<int>(gridDim.z),
                     [&](int cur, uint64_t same) {
        const int count = __popcll(same);
        const int place = nth_lane(same, lane);
        bf16x8_t bf[4][RS];
        float scale = 1.0f;
        if (cur >= 0) {
            if (p.scale) scale = p.scale[cur];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                int col = n0 + 16 * (li / 4) + 4 * i + (li & 3);
                col = col < p.n ? col : p.n - 1;
                const uint16_t* const br = p.b + (static_cast<int64_t>(cur) * p.n + col) * p.rank;
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    u32x4_t v{0u, 0u, 0u, 0u};
                    if (32 * s + 8 * g < p.rank) v = *reinterpret_cast<const u32x4_t*>(br + 32 * s + 8 * g);
                    bf[i][s] = __builtin_bit_cast(bf16x8_t, v);
                }
            }
        }
        for (int f = 0; 16 * f < count; ++f) {
            const int row = row0 + __shfl(place, 16 * f + li);
            const bool mine = 16 * f + li < count;
            const int col = n0 + 16 * g;
            u32x4_t base[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                base[i] = u32x4_t{0u, 0u, 0u, 0u};
                if (p.base && mine && col + 8 * i < p.n)
                    base[i] = *reinterpret_cast<const u32x4_t*>(p.base + row * p.base_stride + col + 8 * i);
            }
            f32x4_t acc[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            if (cur >= 0) {
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    // the row's 8 values of h: the parts' sum, scaled, as hi + lo in bf16 (one rounding's
                    // 2^-9 would be as large as the output's own)
                    u32x4_t hi{0u, 0u, 0u, 0u}, lo{0u, 0u, 0u, 0u};
                    if (32 * s + 8 * g < p.rank) {
                        f32x4_t v[2] = {{0.0f, 0.0f, 0.0f, 0.0f}, {0.0f, 0.0f, 0.0f, 0.0f}};
                        for (int q = 0; q < p.parts; ++q) {
                            const float* const hr = p.h + (static_cast<int64_t>(q) * p.m + row) * p.rank + 32 * s + 8 * g;
                            v[0] += *reinterpret_cast<const f32x4_t*>(hr);
                            v[1] += *reinterpret_cast<const f32x4_t*>(hr + 4);
                        }
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const float x = v[e / 2][2 * (e & 1)] * scale, y = v[e / 2][2 * (e & 1) + 1] * scale;
                            hi[e] = pack_bf16x2(x, y);
                            lo[e] = pack_bf16x2(x - __uint_as_float(hi[e] << 16), y - __uint_as_float(hi[e] & 0xFFFF0000u));
                        }
                    }
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[i][s], __builtin_bit_cast(bf16x8_t, hi), acc[i], 0, 0, 0);
                        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(bf[i][s], __builtin_bit_cast(bf16x8_t, lo), acc[i], 0, 0, 0);
                    }
                }
            }
            // lane: columns 4 i + e of its 16, row li
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                u32x4_t y;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const f32x4_t a = acc[2 * i + e / 2];
                    y[e] = pack_bf16x2(a[2 * (e & 1)] + __uint_as_float(base[i][e] << 16),
                                       a[2 * (e & 1) + 1] + __uint_as_float(base[i][e] & 0xFFFF0000u));
                }
                if (mine && col + 8 * i < p.n)
                    *reinterpret_cast<u32x4_t*>(p.out + row * p.out_stride + col + 8 * i) = y;
            }
        }
    });
}

int tiles_of(int m) { return (m + kTileRows - 1) / kTileRows; }

// Passes of a tile side by side: as many as it can have, while the tiles alone leave the chip idle.
int slots_of(int m, int adapters, int others) {
    const int tiles = tiles_of(m);
    int most = m < kTileRows ? m : kTileRows;
    if (most > adapters + 1) most = adapters + 1;
    const int64_t want = 2048 / (static_cast<int64_t>(tiles) * others);
    return want < 1 ? 1 : want < most ? static_cast<int>(want) : most;
}

}  // namespace

int lora_parts(int m, int k, int adapters) {
    const int tiles = tiles_of(m);
    int parts = 1024 / (tiles * slots_of(m, adapters, 4));    // tiles <= 2^18, and one slot beyond 512 tiles
    const int most = (k + 255) / 256;       // at least one turn of every wave
    if (parts > 16) parts = 16;
    if (parts > most) parts = most;
    return parts < 1 ? 1 : parts;
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
    const unsigned tiles = static_cast<unsigned>(tiles_of(a.m));
    const dim3 g1(tiles, static_cast<unsigned>(slots_of(a.m, a.adapters, 4)), static_cast<unsigned>(a.parts));
    const int rf = (a.rank + 15) / 16;
    if (rf <= 1) lora_shrink_kernel<1><<<g1, 64 * kWaves, 0, s>>>(a);
    else if (rf <= 2) lora_shrink_kernel<2><<<g1, 64 * kWaves, 0, s>>>(a);
    else if (rf <= 4) lora_shrink_kernel<4><<<g1, 64 * kWaves, 0, s>>>(a);
    else lora_shrink_kernel<8><<<g1, 64 * kWaves, 0, s>>>(a);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int ntiles = (a.n + 64 * kWaves - 1) / (64 * kWaves);
    const dim3 g2(tiles, static_cast<unsigned>(ntiles), static_cast<unsigned>(slots_of(a.m, a.adapters, ntiles)));
    if (a.rank <= 32) lora_expand_kernel<1><<<g2, 64 * kWaves, 0, s>>>(a);
    else if (a.rank <= 64) lora_expand_kernel<2><<<g2, 64 * kWaves, 0, s>>>(a);
    else lora_expand_kernel<4><<<g2, 64 * kWaves, 0, s>>>(a);
    return hipGetLastError();
}

}  // namespace dlf
