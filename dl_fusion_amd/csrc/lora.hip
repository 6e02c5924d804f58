// Low-rank adapters of many requests beside a shared projection:
//     out[i] = base[i] + scale[a] (x[i] A_a^T) B_a^T,   a the adapter of row i.
//
// The second product needs the first one's sum over all of k: h = x A^T in fp32 goes through a workspace
// (m x rank, small beside x and out) from one kernel to the next; for a small batch one kernel does both.
// 2 m rank (k + n) flops over x, base, out and the used adapters' weights: at rank 64 about 60 flops a
// byte, so both are bound by what they read and, where that is little, by the chain of a workgroup's
// start (ids, rows, operands).  8192 rows of 4096 at rank 64, 8 adapters: 58 us for 210 MB, 3.6 TB/s;
// 96 rows of 64 adapters at rank 16: 15 us for 15 MB; one row at rank 8: 7.0 us.
//
// Rows of one adapter are gathered per tile of 64 rows: a wave holds the tile's adapters one a lane,
// and a ballot gives the rows that share the first one left, so any order of rows is served, a run of
// one adapter in one pass over the tile, 64 different ones in 64 passes of one row each (each reads
// only its own weights, which has to happen anyway).  The passes of a tile are spread over gridDim's
// slots where there are few tiles.
#include <type_traits>

#include "device_common.h"
#include "kernels.h"
#include "mma_common.h"

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

// The same by at most 16 rows of an adapter at a time, each such group a turn of its own.
template <class Fn>
__device__ __forceinline__ void for_each_16(int id, int lane, uint64_t there, int slot, int slots, Fn&& f) {
    const int rows = __popcll(there);       // the first lanes
    int before = 0;                         // rows before this one that share its adapter
    auto count = [&](auto first_c, auto last_c) {
#pragma unroll
        for (int j = decltype(first_c)::value; j < decltype(last_c)::value; ++j)
            before += lane > j && id == __builtin_amdgcn_readlane(id, j);
    };
    if (rows > 1) count(std::integral_constant<int, 0>{}, std::integral_constant<int, 15>{});
    if (rows > 16) count(std::integral_constant<int, 15>{}, std::integral_constant<int, 63>{});
    uint64_t firsts = __ballot((before & 15) == 0) & there;
    for (int turn = 0; firsts; ++turn, firsts &= firsts - 1) {
        if (turn < slot) continue;
        const int l = __builtin_ctzll(firsts);
        const int cur = __builtin_amdgcn_readlane(id, l), from = __builtin_amdgcn_readlane(before, l);
        f(cur, __ballot(id == cur && before >= from && before < from + 16) & there);
        slot += slots;
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

// A lane's MFMA operand is 16 bytes of one row, and the 16 lanes next to each other have 16 rows: taken
// straight from memory that is 64 accesses of the cache a load.  So x, A and B go to LDS by loads whose
// neighbouring lanes take neighbouring bytes, no register between, and come back with one 16-byte read
// a lane; out goes the same way back.
//
// The first product's ring.  RF and NF: fragments of 16 ranks and of 16 rows.  80 KB, so that a CU holds
// two workgroups: one alone is bound by the way from a barrier over LDS to the products, 3.6 TB/s of x.
template <int RF, int NF>
struct Ring {
    static constexpr int kSlice = NF == 1 && RF <= 4 ? 128 : 64;    // k
    static constexpr int kRow = 2 * kSlice;                         // bytes of a row of a slice
    static constexpr int kChunks = kSlice / 8;
    static constexpr int kFrag = 16 * kRow;
    static constexpr int kStage = (RF + NF) * kFrag;
    static constexpr int kDepth = (80 << 10) / kStage < 8 ? (80 << 10) / kStage : 8;
    // 1 KB loads, and those of a wave: where there are fewer than waves, some do the same
    static constexpr int kX = NF * kFrag / 1024, kA = RF * kFrag / 1024;
    static constexpr int kXLoads = (kX + kWaves - 1) / kWaves, kALoads = (kA + kWaves - 1) / kWaves;
    static constexpr int kLoads = kXLoads + kALoads;
    // chunk c of a row lies at place c ^ swizzle(row), so that 16 lanes' reads fall on all banks
    static __device__ __forceinline__ int swizzle(int row) { return kChunks == 16 ? row & 15 : row >> 1 & 7; }
};
constexpr int kRingBytes = 80 << 10;

// Waits for the oldest loads while `younger` groups of N loads each, and E operations more, may be
// outstanding.
template <int N, int MOST, int E = 0>
__device__ __forceinline__ void wait_groups(int younger) {
    if constexpr (MOST == 0) {
        wait_vmcnt<E>();
    } else {
        if (younger >= MOST) wait_vmcnt<N * MOST + E>();
        else wait_groups<N, MOST - 1, E>(younger);
    }
}

// sum of A x^T over k0 .. k1 (k0 a multiple of 128) for the rows of a pass and one adapter: done(c, f, v)
// gets ranks 16 c + 4 g .. + 3 of row 16 f + li (computed transposed, ranks x rows, so that a lane ends up
// with neighbouring ranks of a row).  Slices go through a ring in LDS that is filled kDepth - 1 ahead.
// With 64 rows a wave has 16 of them and all k; with 16 it has one step of 32 k of each slice (and, of 8
// fragments of ranks, half), and the waves' sums are added at the end.
template <int RF, int NF, class Fn>
__device__ __forceinline__ void multiply(const LoraArgs& p, uint8_t* lds, int wave, int lane, int row0, int place, int cur,
                                         int k0, int k1, Fn&& done) {
    using R = Ring<RF, NF>;
    constexpr int D = R::kDepth, S = R::kSlice / 32;
    static_assert(D >= 3 && (D - 2) * R::kLoads < 64 && D * R::kStage <= kRingBytes, "ring");
    const int li = lane & 15, g = lane >> 4;
    const int in = lane / R::kChunks, to_chunk = lane % R::kChunks;     // of a load
    const int n = (k1 - k0 + R::kSlice - 1) / R::kSlice;
    const uint16_t* xr[R::kXLoads];
    int xc[R::kXLoads], x_to[R::kXLoads];
#pragma unroll
    for (int j = 0; j < R::kXLoads; ++j) {
        x_to[j] = (wave + kWaves * j) % R::kX;
        const int row = x_to[j] * (1024 / R::kRow) + in;    // places past the last row repeat the first
        xr[j] = p.x + (row0 + __shfl(place, row)) * p.x_stride;
        xc[j] = 8 * (to_chunk ^ R::swizzle(row));
    }
    const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(p.a + static_cast<int64_t>(cur) * p.rank * p.k,
                                                  static_cast<uint32_t>(p.rank) * static_cast<uint32_t>(p.k) * 2);   // <= 2^31
    uint32_t ao[R::kALoads];        // elements
    int ac[R::kALoads], a_to[R::kALoads];
#pragma unroll
    for (int j = 0; j < R::kALoads; ++j) {
        a_to[j] = (wave + kWaves * j) % R::kA;
        const int rk = a_to[j] * (1024 / R::kRow) + in;
        ao[j] = static_cast<uint32_t>(rk < p.rank ? rk : p.rank - 1) * static_cast<uint32_t>(p.k);
        ac[j] = 8 * (to_chunk ^ R::swizzle(rk));
    }
    auto issue = [&](int i, int slot) {
        uint8_t* const to = lds + slot * R::kStage;
        const int k = k0 + R::kSlice * i;
        const int last = k + R::kSlice <= p.k ? 0x7FFFFFFF : p.k - 8;       // k past the last is masked when it is read
#pragma unroll
        for (int j = 0; j < R::kXLoads; ++j) load_lds16_stream(xr[j] + (k + xc[j] < last ? k + xc[j] : last), to + 1024 * x_to[j]);
#pragma unroll
        for (int j = 0; j < R::kALoads; ++j)
            load_lds16_buf(ar, 2 * (ao[j] + static_cast<uint32_t>(k + ac[j] < last ? k + ac[j] : last)),
                           to + NF * R::kFrag + 1024 * a_to[j]);
    };
    constexpr bool kHalf = NF == 1 && S == 2;           // a wave has half of the ranks
    static_assert(NF == 4 || S == 4 || RF % 2 == 0, "a step a wave");
    constexpr int kSteps = NF == 1 ? 1 : S, kC = kHalf ? RF / 2 : RF;
    const int s_own = kHalf ? wave & 1 : wave, c_own = kHalf ? (wave >> 1) * kC : 0;
    uint32_t at[kSteps];                                // where a lane's operands lie in 16 rows
#pragma unroll
    for (int s = 0; s < kSteps; ++s)
        at[s] = static_cast<uint32_t>(R::kRow * li + 16 * ((4 * (NF == 1 ? s_own : s) + g) ^ R::swizzle(li)));
    f32x4_t acc[kC];
#pragma unroll
    for (int c = 0; c < kC; ++c) acc[c] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
    auto slice = [&](const uint8_t* from, int k, auto tail_c) {
        u32x4_t x[kSteps], w[kSteps][kC];
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
            x[s] = *reinterpret_cast<const u32x4_t*>(from + (NF == 1 ? 0 : R::kFrag * wave) + at[s]);
#pragma unroll
            for (int c = 0; c < kC; ++c) w[s][c] = *reinterpret_cast<const u32x4_t*>(from + R::kFrag * (NF + c_own + c) + at[s]);
            if (decltype(tail_c)::value && k + 32 * (NF == 1 ? s_own : s) + 8 * g >= p.k) {
                x[s] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                for (int c = 0; c < kC; ++c) w[s][c] = u32x4_t{0u, 0u, 0u, 0u};
            }
        }
#pragma unroll
        for (int s = 0; s < kSteps; ++s)
#pragma unroll
            for (int c = 0; c < kC; ++c)
                acc[c] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[s][c]),
                                                                 __builtin_bit_cast(bf16x8_t, x[s]), acc[c], 0, 0, 0);
    };
#pragma unroll
    for (int i = 0; i < D - 1; ++i)
        if (i < n) issue(i, i);
    int slot = 0;
    for (int i = 0; i < n; ++i) {
        // this wave's loads of slice i have landed, after the barrier everybody's; and slice i - 1 has been
        // read by everybody
        wait_groups<R::kLoads, D - 2>(n - 1 - i);
        barrier();
        if (i + D - 1 < n) issue(i + D - 1, slot == 0 ? D - 1 : slot - 1);
        const int k = k0 + R::kSlice * i;
        if (k + R::kSlice <= p.k) slice(lds + slot * R::kStage, k, std::false_type{});
        else slice(lds + slot * R::kStage, k, std::true_type{});
        slot = slot + 1 == D ? 0 : slot + 1;
    }
    wait_vmcnt<0>();
    barrier();              // the ring is free
    if constexpr (NF == 4) {
#pragma unroll
        for (int c = 0; c < RF; ++c) done(c, wave, acc[c]);
    } else {
        f32x4_t* const sum = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
        for (int c = 0; c < kC; ++c) sum[(wave * kC + c) * 64 + lane] = acc[c];
        __syncthreads();
        // wave w adds fragments w, w + 4
#pragma unroll
        for (int c0 = 0; c0 < RF; c0 += kWaves) {
            const int c = c0 + wave;
            if (c < RF) {
                const int w0 = kHalf ? 2 * (c / kC) : 0;
                f32x4_t v = sum[(w0 * kC + c % kC) * 64 + lane];
#pragma unroll
                for (int w = 1; w < (kHalf ? 2 : kWaves); ++w) v += sum[((w0 + w) * kC + c % kC) * 64 + lane];
                done(c, 0, v);
            }
        }
        __syncthreads();    // and free again
    }
}

// The same for at most 16 rows and 32 ranks, each wave by itself: it takes a quarter of the k through a ring
// of its own of `DEPTH` slices of 64, no barrier but at the end, where the waves' sums are added.  One row at
// rank 8 and k = 4096: 32 barriers less are 2 us.
template <int RF, int DEPTH, class Fn>
__device__ __forceinline__ void multiply_alone(const LoraArgs& p, uint8_t* lds, int wave, int lane, int row0, int place, int cur,
                                               int k0, int k1, Fn&& done) {
    using R = Ring<RF, 4>;              // its rows of 64 k
    constexpr int kStage = (1 + RF) * R::kFrag, kLoads = 2 + 2 * RF;
    static_assert(R::kSlice == 64 && DEPTH >= 3 && (DEPTH - 2) * kLoads < 64, "ring");
    const int li = lane & 15, g = lane >> 4;
    const int in = lane / R::kChunks, to_chunk = lane % R::kChunks;
    const int units = (k1 - k0 + 63) / 64, first = units * wave / kWaves, n = units * (wave + 1) / kWaves - first;
    uint8_t* const ring = lds + wave * DEPTH * kStage;
    const uint16_t* xr[2];
    int c[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
        xr[j] = p.x + (row0 + __shfl(place, 8 * j + in)) * p.x_stride;      // places past the last row repeat the first
        c[j] = 8 * (to_chunk ^ R::swizzle(8 * j + in));
    }
    const __amdgpu_buffer_rsrc_t ar = buffer_rsrc(p.a + static_cast<int64_t>(cur) * p.rank * p.k,
                                                  static_cast<uint32_t>(p.rank) * static_cast<uint32_t>(p.k) * 2);   // <= 2^31
    uint32_t ao[2 * RF];        // elements
#pragma unroll
    for (int j = 0; j < 2 * RF; ++j) {
        const int rk = 8 * j + in;
        ao[j] = static_cast<uint32_t>(rk < p.rank ? rk : p.rank - 1) * static_cast<uint32_t>(p.k);
    }
    auto issue = [&](int i, int slot) {
        uint8_t* const to = ring + slot * kStage;
        const int k = k0 + 64 * (first + i);
        const int last = k + 64 <= p.k ? 0x7FFFFFFF : p.k - 8;      // k past the last is masked when it is read
#pragma unroll
        for (int j = 0; j < 2 * RF; ++j)
            load_lds16_buf(ar, 2 * (ao[j] + static_cast<uint32_t>(k + c[j & 1] < last ? k + c[j & 1] : last)), to + R::kFrag + 1024 * j);
#pragma unroll
        for (int j = 0; j < 2; ++j) load_lds16(xr[j] + (k + c[j] < last ? k + c[j] : last), to + 1024 * j);
    };
    uint32_t at[2];
#pragma unroll
    for (int s = 0; s < 2; ++s) at[s] = static_cast<uint32_t>(R::kRow * li + 16 * ((4 * s + g) ^ R::swizzle(li)));
    f32x4_t acc[RF];
#pragma unroll
    for (int r = 0; r < RF; ++r) acc[r] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int i = 0; i < DEPTH - 1; ++i)
        if (i < n) issue(i, i);
    int slot = 0;
    for (int i = 0; i < n; ++i) {
        wait_groups<kLoads, DEPTH - 2>(n - 1 - i);
        const uint8_t* const from = ring + slot * kStage;
        u32x4_t x[2], w[2][RF];
#pragma unroll
        for (int s = 0; s < 2; ++s) {
            x[s] = *reinterpret_cast<const u32x4_t*>(from + at[s]);
#pragma unroll
            for (int r = 0; r < RF; ++r) w[s][r] = *reinterpret_cast<const u32x4_t*>(from + R::kFrag * (1 + r) + at[s]);
        }
        const int k = k0 + 64 * (first + i);
        if (k + 64 > p.k) {
#pragma unroll
            for (int s = 0; s < 2; ++s)
                if (k + 32 * s + 8 * g >= p.k) {
                    x[s] = u32x4_t{0u, 0u, 0u, 0u};
#pragma unroll
                    for (int r = 0; r < RF; ++r) w[s][r] = u32x4_t{0u, 0u, 0u, 0u};
                }
        }
#pragma unroll
        for (int s = 0; s < 2; ++s)
#pragma unroll
            for (int r = 0; r < RF; ++r)
                acc[r] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, w[s][r]),
                                                                 __builtin_bit_cast(bf16x8_t, x[s]), acc[r], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);      // slice i has been read; slice i - 1's place is refilled
        if (i + DEPTH - 1 < n) issue(i + DEPTH - 1, slot == 0 ? DEPTH - 1 : slot - 1);
        slot = slot + 1 == DEPTH ? 0 : slot + 1;
    }
    wait_vmcnt<0>();
    __syncthreads();
    f32x4_t* const sum = reinterpret_cast<f32x4_t*>(lds);
#pragma unroll
    for (int r = 0; r < RF; ++r) sum[(wave * RF + r) * 64 + lane] = acc[r];
    __syncthreads();
    if (wave < RF) {
        f32x4_t v = sum[wave * 64 + lane];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) v += sum[(w * RF + wave) * 64 + lane];
        done(wave, 0, v);
    }
    __syncthreads();        // the ring is free
}

// Between LDS writes and reads of one wave's lanes: they are done in program order, and the compiler has
// to keep that order.
__device__ __forceinline__ void wave_fence() {
    __builtin_amdgcn_wave_barrier();
    asm volatile("" ::: "memory");
}

// ---- h = x A^T into the workspace: a workgroup takes a tile, an adapter and a range of slices ----
template <int RF>
__global__ __launch_bounds__(64 * kWaves, 2) void lora_shrink_kernel(const LoraArgs p) {
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int row0 = static_cast<int>(blockIdx.x) * kTileRows;
    const int part = static_cast<int>(blockIdx.y);
    const int units = (p.k + 127) / 128;
    const int k0 = 128 * static_cast<int>(static_cast<int64_t>(units) * part / p.parts);
    int k1 = 128 * static_cast<int>(static_cast<int64_t>(units) * (part + 1) / p.parts);
    k1 = k1 < p.k ? k1 : p.k;
    const int id = adapter_of(p, row0 + lane);
    const int slot = static_cast<int>(gridDim.z - 1 - blockIdx.z);      // second passes first: they are few
    for_each_adapter(id, __ballot(row0 + lane < p.m), slot, static_cast<int>(gridDim.z), [&](int cur, uint64_t same) {
        if (cur < 0) return;
        const int count = __popcll(same), place = nth_lane(same, lane);
        auto store = [&](int c, int f, f32x4_t v) {
            const int to = row0 + __shfl(place, 16 * f + li), rk = 16 * c + 4 * g;
            if (16 * f + li < count && rk < p.rank)
                *reinterpret_cast<f32x4_t*>(p.h + (static_cast<int64_t>(part) * p.m + to) * p.rank + rk) = v;
        };
        if (count > 16) multiply<RF, 4>(p, lds, wave, lane, row0, place, cur, k0, k1, store);
        else if constexpr (RF <= 2) multiply_alone<RF, RF == 1 ? 5 : 3>(p, lds, wave, lane, row0, place, cur, k0, k1, store);
        else multiply<RF, 1>(p, lds, wave, lane, row0, place, cur, k0, k1, store);
    });
}

// ---- out = base + scale h B^T: a workgroup takes a tile, an adapter and a range of blocks of 64 columns
// (32 at ranks above 64, for two workgroups a CU) ----
// Again transposed (columns x rows), so that base and out are added and rounded once.  A block of B is
// one run of memory, taken to LDS in lines; in every 16 chunks of it, chunk c lies at place c ^ (the 16's
// number & 15).  The products pass through LDS 16 rows at a time, so that base and out move in lines.
// h is held in registers for all columns, as hi + lo in bf16: one rounding's 2^-8 would be as large as
// the output's own.
// More than 16 rows: a wave has 16 of them and all columns; B and base go through a ring of blocks, as the
// first product's slices do.  Up to 16 rows: the waves take the blocks in turns, a few at a time each.
// SELF: for a small batch, 16 rows of an adapter at a time: the workgroup computes the adapter's h by itself.
// Every range of the columns reads A again, from L2, which saves a launch and h's way through memory.  Else h
// comes from the workspace.
template <int RF, bool SELF>
struct OutLds {
    static constexpr int kSteps = (RF + 1) / 2;             // of 32 ranks
    static constexpr int kCols = kSteps == 4 ? 32 : 64;     // of a block
    static constexpr int kB = kCols * (SELF ? 16 * RF : 32 * kSteps) * 2;   // bytes of a block of B
    static constexpr int kBase = kTileRows * kCols * 2;     // and of base
    // Blocks in the ring, for two workgroups a CU: five at ranks 33..64 are 96 KB, and 8192 rows at rank 64 take 75 us
    // instead of 61 (three: 60; at ranks 65..128 three, four and five are 90, 91 and 91)
    static constexpr int kDepth = kSteps == 2 ? 4 : 5;
    static constexpr int kOwn = 16 * kCols * 4;             // a wave's 16 rows of products, fp32
    // Blocks that a wave has of its own at a time.  As many as leave two workgroups a CU: four at ranks 33..64 take
    // 64 rows of 64 adapters from 21 us to 25.  Fewer are level: 1024 rows of 64 adapters at rank 16, 1, 2 and 4 blocks
    // 76, 78 and 79; 96 rows in one launch, 1 and 2 blocks 15.7 and 15.2.
    static constexpr int kOwnBlocks = kSteps == 1 && !SELF ? 4 : 2;
    static constexpr int kMany = kDepth * (kB + kBase), kFew = kWaves * kOwnBlocks * kB;
    // Slices of multiply_alone().  At rank 16 a fourth leaves one workgroup a CU: 96 rows of 64 adapters 19.5 us instead
    // of 15.2, one row level.  At rank 32 there is one anyway: 16 rows of 16 adapters 9.3, with three 9.9.
    static constexpr int kSelfDepth = RF == 1 ? 3 : 4;
    static constexpr int kPitch = 32 * kSteps + 8;          // bf16 values of a row of h: 16 rows in different banks
    static constexpr int kH = SELF ? 2 * 16 * kPitch * 2 : 0;
    // SELF: the first product's ring is free when products come, and holds them
    static constexpr int kSelf = kWaves * kSelfDepth * (1 + RF) * 2048;
    static constexpr int kRings = SELF ? kFew : kMany > kFew ? kMany : kFew;
    static constexpr int kBytes = kH + kRings + (SELF ? kSelf : kWaves * kOwn);
    static_assert(kWaves * kOwn <= kSelf, "own");
};

template <int RF, bool SELF>
__global__ __launch_bounds__(64 * kWaves, 2) void lora_out_kernel(const LoraArgs p) {
    using L = OutLds<RF, SELF>;
    constexpr int RS = L::kSteps;
    extern __shared__ __attribute__((aligned(16))) uint8_t lds[];
    const int lane = static_cast<int>(threadIdx.x) & 63;
    const int wave = __builtin_amdgcn_readfirstlane(static_cast<int>(threadIdx.x) >> 6);
    const int li = lane & 15, g = lane >> 4;
    const int row0 = static_cast<int>(blockIdx.x) * kTileRows;
    constexpr int C = L::kCols, F = C / 16, U = C / 32;    // columns, fragments and 1 KB loads of 16 rows of a block
    const int blocks = (p.n + C - 1) / C;
    const int cb0 = static_cast<int>(static_cast<int64_t>(blocks) * blockIdx.y / gridDim.y);
    const int cb1 = static_cast<int>(static_cast<int64_t>(blocks) * (blockIdx.y + 1) / gridDim.y);
    const int id = adapter_of(p, row0 + lane);
    uint16_t* const h_s = reinterpret_cast<uint16_t*>(lds);     // SELF: hi, then lo
    uint8_t* const rings = lds + L::kH;
    uint8_t* const own = lds + L::kH + L::kRings + wave * L::kOwn;

    // what a lane moves of 16 rows: row o_row (+ 16 / U for the second load), 8 columns
    const int o_row = lane / (C / 8), o_col = 8 * (lane % (C / 8));
    const int block_bytes = C * p.rank * 2, block_kb = (block_bytes + 1023) / 1024;
    // KB j of block cb; what lies past the adapter's end comes as zeros, and KB past the block's too: many() loads
    // those, so that its loads are as many at every rank, few() leaves them as they are
    auto load_b = [&](__amdgpu_buffer_rsrc_t br, int cb, int j, uint8_t* to) {
        const uint32_t q = static_cast<uint32_t>(64 * j + lane);
        const uint32_t at = static_cast<uint32_t>(cb) * static_cast<uint32_t>(block_bytes) + 16 * (q ^ (q >> 4 & 15));
        load_lds16_buf(br, j < block_kb ? at : kOutOfRange, to + 1024 * j);
    };
    // hi stops at bf16's largest value, so that a value just beyond it has its rest in lo, an infinity is lo's (a lo of
    // inf - inf would be NaN), and NaN as well
    auto split = [](const f32x4_t& v, float scale, uint32_t* hi, uint32_t* lo) {
        constexpr float kTop = 0x1.FEp127f;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
            const float x = v[2 * e] * scale, y = v[2 * e + 1] * scale;
            hi[e] = pack_bf16x2(__builtin_amdgcn_fmed3f(x, -kTop, kTop), __builtin_amdgcn_fmed3f(y, -kTop, kTop));
            lo[e] = pack_bf16x2(x - __uint_as_float(hi[e] << 16), y - __uint_as_float(hi[e] & 0xFFFF0000u));
        }
    };
    // ranks 32 s + 8 g .. of a row of h, from the workspace
    auto load_h = [&](int row, float scale, u32x4_t (&hi)[RS], u32x4_t (&lo)[RS]) {
        f32x4_t v[RS][2];
        const float* from[RS];
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            v[s][0] = v[s][1] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
            // ranks past the last repeat a valid one, and are cleared below
            from[s] = p.h + static_cast<int64_t>(row) * p.rank + (32 * s + 8 * g < p.rank ? 32 * s + 8 * g : 0);
        }
        constexpr int kTogether = 8 / RS;      // parts whose loads are in flight together
        const int64_t step = static_cast<int64_t>(p.m) * p.rank;
        for (int q0 = 0; q0 < p.parts; q0 += kTogether) {
            f32x4_t t[kTogether][RS][2];
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    const float* const at = from[s] + (q0 + j < p.parts ? q0 + j : q0) * step;
                    t[j][s][0] = *reinterpret_cast<const f32x4_t*>(at);
                    t[j][s][1] = *reinterpret_cast<const f32x4_t*>(at + 4);
                }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int j = 0; j < kTogether; ++j)
                if (q0 + j < p.parts)
#pragma unroll
                    for (int s = 0; s < RS; ++s) {
                        v[s][0] += t[j][s][0];
                        v[s][1] += t[j][s][1];
                    }
        }
#pragma unroll
        for (int s = 0; s < RS; ++s) {
            uint32_t h[4], l[4];
            split(v[s][0], scale, h, l);
            split(v[s][1], scale, h + 2, l + 2);
            const bool in = 32 * s + 8 * g < p.rank;
            hi[s] = in ? u32x4_t{h[0], h[1], h[2], h[3]} : u32x4_t{0u, 0u, 0u, 0u};
            lo[s] = in ? u32x4_t{l[0], l[1], l[2], l[3]} : u32x4_t{0u, 0u, 0u, 0u};
        }
    };
    // where a lane's operands of a block of B lie: column 16 i + li, ranks 32 s + 8 g ..
    uint32_t b_at[RS][F];
#pragma unroll
    for (int s = 0; s < RS; ++s)
#pragma unroll
        for (int i = 0; i < F; ++i) {
            const uint32_t q = static_cast<uint32_t>((16 * i + li) * (p.rank / 8) + 4 * s + g);
            b_at[s][i] = 16 * (q ^ (q >> 4 & 15));
        }
    // The steps of 32 ranks from the smallest rank that comes here on (of 65..128 ranks, the third and the
    // fourth) may have lanes past the last rank: what these read is another column's or nobody's, and is cleared,
    // since an infinity or NaN there would not vanish against the zeros of h.
    constexpr int kWhole = RF == 8 ? 2 : RF == 4 ? 1 : 0;
    // the wave's own LDS: 16-byte chunk c of row r
    auto own_at = [&](int r, int c) {
        return reinterpret_cast<f32x4_t*>(own + 4 * C * r + 16 * (c ^ (C == 64 ? r & 15 : r >> 1 & 7)));
    };
    // 16 rows by the columns of the block in LDS at b, into the wave's own LDS
    auto products = [&](const uint8_t* b, const u32x4_t (&hi)[RS], const u32x4_t (&lo)[RS]) {
        u32x4_t bf[RS][F];
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int i = 0; i < F; ++i) bf[s][i] = *reinterpret_cast<const u32x4_t*>(b + b_at[s][i]);
#pragma unroll
        for (int s = kWhole; s < RS; ++s) {
            const bool past = 32 * s + 8 * g >= p.rank;
#pragma unroll
            for (int i = 0; i < F; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) bf[s][i][e] = past ? 0u : bf[s][i][e];
        }
        f32x4_t y[F];
#pragma unroll
        for (int i = 0; i < F; ++i) y[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int s = 0; s < RS; ++s)
#pragma unroll
            for (int part = 0; part < 2; ++part)
#pragma unroll
                for (int i = 0; i < F; ++i)
                    y[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, bf[s][i]),
                                                                   __builtin_bit_cast(bf16x8_t, part ? lo[s] : hi[s]), y[i], 0, 0, 0);
        // A weight of infinity has become NaN where lo is 0 or against hi.  So where there is a NaN, once more with the
        // weights that are not finite apart: hi meets them alone, lo something finite of their sign.
        f32x4_t all = y[0];
#pragma unroll
        for (int i = 1; i < F; ++i) all += y[i];
        if (__builtin_expect(__ballot(__builtin_isnan(all[0] + all[1] + all[2] + all[3])) != 0, 0)) {
#pragma unroll
            for (int i = 0; i < F; ++i) {
                y[i] = f32x4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
                for (int s = 0; s < RS; ++s) {
                    u32x4_t finite, apart, sign;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const uint32_t w = bf[s][i][e], bad = not_finite_bf16x2(w);
                        finite[e] = w & ~bad;
                        apart[e] = w & bad;
                        sign[e] = finite[e] | (bad & (w & 0x80008000u | 0x3F803F80u));      // 1 or -1
                    }
                    auto add = [&](const u32x4_t& b16, const u32x4_t& h16) {
                        y[i] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, b16),
                                                                       __builtin_bit_cast(bf16x8_t, h16), y[i], 0, 0, 0);
                    };
                    add(finite, hi[s]);
                    add(sign, lo[s]);
                    add(apart, hi[s]);
                }
            }
        }
        // lane: row li, columns 16 i + 4 g .. + 3
        wave_fence();
#pragma unroll
        for (int i = 0; i < F; ++i) *own_at(li, 4 * i + g) = y[i];
        wave_fence();
    };
    // the lane's 8 columns of its row of load u, with base, rounded
    auto finish = [&](int u, const u32x4_t& base) {
        const int r = 16 / U * u + o_row;
        const f32x4_t t[2] = {*own_at(r, o_col / 4), *own_at(r, o_col / 4 + 1)};
        u32x4_t v;
#pragma unroll
        for (int e = 0; e < 4; ++e)
            v[e] = pack_bf16x2(t[e / 2][2 * (e & 1)] + __uint_as_float(base[e] << 16),
                               t[e / 2][2 * (e & 1) + 1] + __uint_as_float(base[e] & 0xFFFF0000u));
        return v;
    };
    auto load_base = [&](int64_t row, bool mine, int col) {
        u32x4_t v{0u, 0u, 0u, 0u};
        if (p.base && mine && col < p.n) v = *reinterpret_cast<const u32x4_t*>(p.base + row * p.base_stride + col);
        return v;
    };
    auto b_of = [&](int cur) {
        return buffer_rsrc(p.b + static_cast<int64_t>(cur) * p.n * p.rank,
                           static_cast<uint32_t>(p.n) * static_cast<uint32_t>(p.rank) * 2);     // <= 2^31
    };

    auto few = [&](int cur, uint64_t same) {
        const int count = __popcll(same), place = nth_lane(same, lane);
        const float scale = p.scale ? p.scale[cur] : 1.0f;
        const __amdgpu_buffer_rsrc_t br = b_of(cur);
        uint8_t* const ring = rings + wave * L::kOwnBlocks * L::kB;
        int row[U];
        bool mine[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = 16 / U * u + o_row;
            row[u] = row0 + __shfl(place, at);
            mine[u] = at < count;
        }
        u32x4_t base[L::kOwnBlocks][U];
        auto fetch = [&](int first) {
#pragma unroll
            for (int d = 0; d < L::kOwnBlocks; ++d) {
                const int cb = first + kWaves * d;
                if (cb >= cb1) continue;
                for (int j = 0; j < block_kb; ++j) load_b(br, cb, j, ring + d * L::kB);
#pragma unroll
                for (int u = 0; u < U; ++u) base[d][u] = load_base(row[u], mine[u], C * cb + o_col);
            }
        };
        fetch(cb0 + wave);      // on its way while h is made
        u32x4_t hi[RS], lo[RS];
        if constexpr (SELF) {
            multiply_alone<RF, L::kSelfDepth>(p, lds + L::kH + L::kRings, wave, lane, row0, place, cur, 0, p.k, [&](int c, int, f32x4_t v) {
                uint32_t h[2], l[2];
                split(v, scale, h, l);
                const int at = li * L::kPitch + 16 * c + 4 * g;
                *reinterpret_cast<uint2*>(h_s + at) = make_uint2(h[0], h[1]);
                *reinterpret_cast<uint2*>(h_s + 16 * L::kPitch + at) = make_uint2(l[0], l[1]);
            });
            __syncthreads();
#pragma unroll
            for (int s = 0; s < RS; ++s) {
                hi[s] = lo[s] = u32x4_t{0u, 0u, 0u, 0u};
                if (32 * s + 8 * g < p.rank) {      // ranks past the last have nothing in LDS
                    hi[s] = *reinterpret_cast<const u32x4_t*>(h_s + li * L::kPitch + 32 * s + 8 * g);
                    lo[s] = *reinterpret_cast<const u32x4_t*>(h_s + (16 + li) * L::kPitch + 32 * s + 8 * g);
                }
            }
        } else {
            load_h(row0 + __shfl(place, li), scale, hi, lo);
        }
        for (int first = cb0 + wave; first < cb1; first += kWaves * L::kOwnBlocks) {
            if (first > cb0 + wave) fetch(first);
            wait_vmcnt<0>();
#pragma unroll
            for (int d = 0; d < L::kOwnBlocks; ++d) {
                const int cb = first + kWaves * d;
                if (cb >= cb1) continue;
                products(ring + d * L::kB, hi, lo);
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    const u32x4_t v = finish(u, base[d][u]);
                    if (mine[u] && C * cb + o_col < p.n)
                        *reinterpret_cast<u32x4_t*>(p.out + row[u] * p.out_stride + C * cb + o_col) = v;
                }
            }
        }
        __syncthreads();        // SELF: h is made again by the next pass; else the rings are laid out anew
    };

    auto many = [&](int cur, uint64_t same) {
        constexpr int D = L::kDepth, kBLoads = L::kB / 1024 / kWaves;
        const int count = __popcll(same), place = nth_lane(same, lane);
        const float scale = p.scale ? p.scale[cur] : 1.0f;
        const __amdgpu_buffer_rsrc_t br = b_of(cur);
        bool mine[U];
        const uint16_t* from[U];
        uint16_t* to[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int at = 16 * wave + 16 / U * u + o_row;
            const int64_t row = row0 + __shfl(place, at);       // places past the last row repeat the first: loaded, never used
            mine[u] = at < count;
            from[u] = p.base + row * p.base_stride;
            to[u] = p.out + row * p.out_stride;
        }
        auto issue = [&](int cb, int slot) {
            uint8_t* const block = rings + slot * (L::kB + L::kBase);
#pragma unroll
            for (int j = 0; j < kBLoads; ++j) load_b(br, cb, kWaves * j + wave, block);
            const int col = C * cb + o_col < p.n ? C * cb + o_col : p.n - 8;
            if (p.base) {
#pragma unroll
                for (int u = 0; u < U; ++u) load_lds16_stream(from[u] + col, block + L::kB + 1024 * (U * wave + u));
            }
        };
        const int n = cb1 - cb0;
#pragma unroll
        for (int i = 0; i < D - 1; ++i)
            if (i < n) issue(cb0 + i, i);
        u32x4_t hi[RS], lo[RS];
        load_h(row0 + __shfl(place, 16 * wave + li), scale, hi, lo);
        int slot = 0;
        for (int i = 0; i < n; ++i) {
            // as in multiply(); the stores of the D - 1 blocks before this one are younger than its loads
            if (i >= D - 1) {
                if (p.base) wait_groups<kBLoads + U, D - 2, U * (D - 1)>(n - 1 - i);
                else wait_groups<kBLoads, D - 2, U * (D - 1)>(n - 1 - i);
            } else {
                if (p.base) wait_groups<kBLoads + U, D - 2>(n - 1 - i);
                else wait_groups<kBLoads, D - 2>(n - 1 - i);
            }
            barrier();
            if (i + D - 1 < n) issue(cb0 + i + D - 1, slot == 0 ? D - 1 : slot - 1);
            const uint8_t* const block = rings + slot * (L::kB + L::kBase);
            products(block, hi, lo);
#pragma unroll
            for (int u = 0; u < U; ++u) {
                u32x4_t base{0u, 0u, 0u, 0u};
                if (p.base) base = *reinterpret_cast<const u32x4_t*>(block + L::kB + 1024 * (U * wave + u) + 16 * lane);
                const u32x4_t v = finish(u, base);
                // every store is done by some address, so that the waits can count them: lanes without an
                // output write to the workspace's last KB, which nobody reads
                const int col = C * (cb0 + i) + o_col;
                uint16_t* const at = mine[u] && col < p.n ? to[u] + col : p.nowhere + 8 * lane;
                *reinterpret_cast<u32x4_t*>(at) = v;
            }
            slot = slot + 1 == D ? 0 : slot + 1;
        }
        __syncthreads();        // the rings are laid out anew by the next pass
    };

    const int slot = static_cast<int>(gridDim.z - 1 - blockIdx.z);      // second passes first: they are few
    auto pass = [&](int cur, uint64_t same) {
        if (cur < 0) {      // rows without an adapter: base, or zeros
            const int count = __popcll(same), place = nth_lane(same, lane);
            for (int at0 = 0; at0 < count; at0 += 16 / U) {
                const int64_t row = row0 + __shfl(place, at0 + o_row & 63);
                for (int cb = cb0 + wave; cb < cb1; cb += kWaves) {
                    const int col = C * cb + o_col;
                    const u32x4_t v = load_base(row, at0 + o_row < count, col);
                    if (at0 + o_row < count && col < p.n) *reinterpret_cast<u32x4_t*>(p.out + row * p.out_stride + col) = v;
                }
            }
        } else if (SELF || __popcll(same) <= 16) {
            few(cur, same);
        } else if constexpr (!SELF) {
            many(cur, same);
        }
    };
    const uint64_t there = __ballot(row0 + lane < p.m);
    if constexpr (SELF) for_each_16(id, lane, there, slot, static_cast<int>(gridDim.z), pass);
    else for_each_adapter(id, there, slot, static_cast<int>(gridDim.z), pass);
}

int tiles_of(int m) { return (m + kTileRows - 1) / kTileRows; }

// Passes that a tile can have, at most.
int passes_of(int m, int adapters) {
    const int rows = m < kTileRows ? m : kTileRows;
    return rows < adapters + 1 ? rows : adapters + 1;
}

// Passes that get workgroups of their own when the work is split.  In up to 4 tiles (a decode batch) any
// row may have an adapter of its own, or all rows one; more rows are taken to be runs, which costs where they are not:
// 512 rows of 64 adapters in any order at rank 64 take 84 us, 512 of one run 21.  256 rows of 64 adapters
// at rank 64, all different | all one (us): with 4 passes 58 | 22, 16 46 | 29, 64 47 | 87, so 64 in all tiles.
int expected_passes(int m, int adapters) {
    const int most = passes_of(m, adapters), tiles = tiles_of(m);
    return tiles > 4 ? 1 : most < kTileRows / tiles ? most : kTileRows / tiles;
}

// Passes of a tile side by side, where `others` workgroups share each: as many as it can have, while that
// leaves CUs idle, and in a large batch a second one for the tiles that two runs share.
int slots_of(int m, int adapters, int others) {
    const int64_t want = 512 / (static_cast<int64_t>(tiles_of(m)) * others);
    const int most = passes_of(m, adapters);
    return want < 2 ? (most < 2 ? most : 2) : want < most ? static_cast<int>(want) : most;
}

int at_most(int v, int most) { return v < 1 || most < 1 ? 1 : v < most ? v : most; }

// Workgroups that a kernel is split into: three quarters of the 512 that the chip holds (two a CU by their
// LDS), so that the second passes of tiles that two runs share find room beside the first.  With 256 | 384 | 512 (us, n =
// k = 4096, runs of 900 rows): 8192 rows at rank 64 75 | 61 | 76, at rank 16 61 | 50 | 61, at rank 128 105 | 91 | 115.  Fewer
// rows would like 256: 4096 at rank 64 37 | 38 | 45, 2048 27 | 29 | 32, in runs of 100 29 | 35 | 35; the host does not see
// runs.
constexpr int kWorkgroups = 384;

template <int RF>
void launch_shrink(const LoraArgs& a, hipStream_t s) {
    const dim3 grid(static_cast<unsigned>(tiles_of(a.m)), static_cast<unsigned>(a.parts),
                    static_cast<unsigned>(slots_of(a.m, a.adapters, a.parts)));
    lora_shrink_kernel<RF><<<grid, 64 * kWaves, kRingBytes, s>>>(a);
}

// Multiples of 16 tiles, once some CUs get a second workgroup, run slower than their neighbours, which an
// empty tile mends by making the number odd (measured; the cause is not known).  Without it | with it (us): rank 64, n =
// 4096, 2048 rows 33 | 29, 4096 rows 43 | 38; n = 11008, 1024 rows 37 | 31, 2048 50 | 41, 4096 77 | 68; rank 128, 4096 rows, n
// = 11008 116 | 99; rank 16 38 | 34.  At other numbers of tiles it costs where the sum becomes a multiple of 16 (4032 rows
// at rank 64 41 | 46), and up to one workgroup a CU (1024 rows, n = 4096 22 | 25; 16384 138 | 142).
template <int RF, bool SELF>
void launch_out(const LoraArgs& a, int slots, int ranges, hipStream_t s) {
    const int tiles = tiles_of(a.m), empty = tiles % 16 == 0 && tiles * ranges > 256 ? 1 : 0;
    const dim3 grid(static_cast<unsigned>(tiles + empty), static_cast<unsigned>(ranges), static_cast<unsigned>(slots));
    lora_out_kernel<RF, SELF><<<grid, 64 * kWaves, OutLds<RF, SELF>::kBytes, s>>>(a);
}

}  // namespace

// Every range of the second kernel reads all parts of h, so that many of them cost.  2048 rows at rank 64 (us):
// 4 parts 36, 8 39, 12 46; 512 rows 23.0, 21.0, 16 parts 23.1; 2048 rows at rank 16 31.3, 29.8, 33.6.
int lora_parts(int m, int k, int rank, int adapters) {
    const int most = (k + 255) / 256, cap = rank <= 32 || tiles_of(m) <= 8 ? 8 : 4;
    return at_most(kWorkgroups / at_most(tiles_of(m) * expected_passes(m, adapters), kWorkgroups), most < cap ? most : cap);
}

hipError_t launch_lora(const LoraArgs& a, hipStream_t s) {
    const int blocks = (a.n + 63) / 64;
    // One launch (us as called, against two) at n = k = 4096: one row at rank 8 7.8 | 11.0, 16 rows of 16 adapters
    // at rank 32 9.3 | 12.8; 96 rows at rank 16, of 64 adapters 14.7 | 18.6, of one 10.1 | 12.4; 256 rows of one run
    // 10.6 | 13.5, of 64 adapters 21.0 | 24.7.  A workgroup alone reads its A: one row at rank 32, k = 6144 9.8 | 11.0,
    // 8192 11.4 | 11.2, 11008 13.4 | 10.6 (without the call 9.4 | 8.4, 11.4 | 8.6, 13.6 | 8.9).
    if (a.m <= 256 && a.rank <= 32 && a.k <= 6144) {
        // groups of 16 rows that a tile can have, at most: one begun for each adapter, the others full
        const int most = passes_of(a.m, a.adapters);
        const int passes = most + ((a.m < kTileRows ? a.m : kTileRows) - most) / 16;
        // rank 16 leaves room for two workgroups a CU
        const int ranges = at_most((a.rank <= 16 ? kWorkgroups : 256) / (passes * tiles_of(a.m)), (blocks + kWaves - 1) / kWaves);
        if (a.rank <= 16) launch_out<1, true>(a, passes, ranges, s);
        else launch_out<2, true>(a, passes, ranges, s);
        return hipGetLastError();
    }
    if (a.rank <= 16) launch_shrink<1>(a, s);
    else if (a.rank <= 32) launch_shrink<2>(a, s);
    else if (a.rank <= 64) launch_shrink<4>(a, s);
    else launch_shrink<8>(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    const int split = at_most(tiles_of(a.m) * expected_passes(a.m, a.adapters), kWorkgroups);
    // Ranges of 4 blocks give each wave one where few rows share an adapter.  Shorter ones pay up to one workgroup
    // a CU, counting a second pass in all but small batches: at rank 64 (us, against 4 blocks) 52 rows, n = 4096
    // 15.2 | 17.4, 1024 rows, n = 1024 19.6 | 21.5, but 300 rows in runs of 40 21.6 | 21.0 (without that pass 23.9).
    // Up to kWorkgroups as well: 512 rows, n = 4096 22.6 | 21.0, 2097 rows, n = 1608 30 | 27.
    const int of_4 = (blocks + kWaves - 1) / kWaves;
    const int one_a_cu = at_most(256 / (tiles_of(a.m) > 4 ? 2 * split : split), blocks);
    const int ranges = at_most(kWorkgroups / split, of_4 > one_a_cu ? of_4 : one_a_cu);
    const int slots = slots_of(a.m, a.adapters, ranges);
    if (a.rank <= 32) launch_out<2, false>(a, slots, ranges, s);
    else if (a.rank <= 64) launch_out<4, false>(a, slots, ranges, s);
    else launch_out<8, false>(a, slots, ranges, s);
    return hipGetLastError();
}

}  // namespace dlf
