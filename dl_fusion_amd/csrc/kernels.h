// Internal interface between the C-ABI layer (api.cpp) and the HIP kernels.
// Nothing here is exported from the shared library.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace dlf {

// Route and tile switches (tuning and tests).  They are read from the environment once, when
// the library is loaded, and again by dlf_tuning_reload():
//   DLF_TILE=<n>            force MFMA tile n (a kTile* value the route has)
//   DLF_GEMM=tiled|stream   the tiled MFMA kernel, or the streaming kernel wherever it applies
//   DLF_CONV=generic|stream the implicit GEMM for every conv, or the weight-streaming halo kernel
//                           for every 3x3 stride-1 conv
//   DLF_STREAM_NB=128|256|384  the streaming kernel's column block, where built and dividing N
//   DLF_FFN_TOK=32|64       the fused FFN's token block
//   DLF_FFN_SPLIT=<s>       the fused FFN's d_ff parts (0 or 1: no split)
struct Options {
    int tile;        // forced tile, or -1
    int gemm;        // 0 the library's choice, 1 tiled only, 2 streaming where it applies
    int conv;        // 0 the library's choice, 1 implicit GEMM, 2 weight-streaming halo kernel
    int stream_nb;   // 0, or the forced column block
    int ffn_tok;     // 0, or the forced token block
    int ffn_split;   // 0 the library's choice, 1 no split, >= 2 that many parts
};
const Options& options();
void reload_options();

// Arguments of the MFMA GEMM / implicit-GEMM kernel.  C[m][n] = sum_k A[m][k] B[n][k]
// followed by the register epilogue.  For a convolution, A is gathered on the fly
// from the NHWC input (row m = (img, ho, wo), k = (r*KW + s)*Cin + ci).
struct MmaArgs {
    const void* a;          // dense: A [M][K]; conv: x [N][H][W][Cin]
    const void* b;          // B [N][K] (OHWI-flattened weights)
    const float* scale;     // [N] per-column multiplier or nullptr (= 1)
    const float* shift;     // [N] per-column bias / shift or nullptr (= 0)
    const uint16_t* res;    // bf16 residual [M][N] or nullptr
    void* c;                // output [M][N]
    int64_t M;
    int N, K;
    float out_inv_scale;    // fp8 output: fp32(1/s_y)
    float dequant;          // fp32 output of the plain fp8 GEMM: s_x * s_w
    // split store (parts > 1): columns [p * part_cols, (p + 1) * part_cols) go to outs[p], each
    // [M][part_cols]; part_cols is a multiple of one 16-byte chunk of output.  parts == 1: c.
    int parts, part_cols;
    void* outs[4];
    // convolution geometry (A gather); unused by the dense kernel
    int H, W, Cin, Ho, Wo, KW, SH, SW, PH, PW;
};

// Output tile shapes of the MFMA kernel (rows x columns of C per workgroup).  The 256 x 256
// tile serves the dense GEMM only; the implicit-GEMM convolution takes the other three.
enum MmaTile : int {
    kTile256x256 = 0,   // 4x4 waves of 64x64, one barrier per two K slices
    kTile128x128 = 1,   // 2x2 waves of 64x64
    kTile128x64 = 2,    // 2x2 waves of 64x32
    kTile64x64 = 3,     // 2x2 waves of 32x32
    kTileCount = 4
};
int mma_tile_rows(int tile);
int mma_tile_cols(int tile);

// out: kOutBf16 / kOutFp8 / kOutF32; act: kActNone / kActRelu / kActGelu.
hipError_t launch_mma_bf16(const MmaArgs& args, bool conv, int act, int tile, hipStream_t stream);
hipError_t launch_mma_fp8(const MmaArgs& args, int act, int out, int tile, hipStream_t stream);
// Streaming GEMM for memory-bound shapes (bf16, no scale, one output): K of 128 or 256, N a
// multiple of 128 (column blocks of 128 to 384, at most 32 of them), A and C below 2 GB.
bool gemm_stream_ok(const MmaArgs& args);
// ... and where it is faster than the tiled kernel (from 4M outputs)
bool gemm_stream_pays(const MmaArgs& args);
hipError_t launch_gemm_stream(const MmaArgs& args, int act, hipStream_t stream);
// instantiation groups of the MFMA kernel (one translation unit each); wide: rows of 8 MB or
// more, read by 64-bit global addresses
hipError_t launch_mma_bf16_dense(const MmaArgs& args, bool wide, int act, int tile, hipStream_t stream);
hipError_t launch_mma_bf16_gated(const MmaArgs& args, bool wide, int act, int tile, hipStream_t stream);
hipError_t launch_mma_bf16_conv(const MmaArgs& args, int act, int tile, hipStream_t stream);
hipError_t launch_mma_fp8_q(const MmaArgs& args, bool wide, int act, int tile, hipStream_t stream);
hipError_t launch_mma_fp8_b(const MmaArgs& args, bool wide, int act, int out, int tile, hipStream_t stream);

// fp32 direct convolution with the same epilogue (bias -> residual -> act).
struct ConvF32Args {
    const float* x;
    const float* w;
    const float* bias;      // nullable
    const float* res;       // nullable
    float* y;
    int M;                  // n * ho * wo (<= 2^30, checked on the host)
    int Cout, K;
    int H, W, Cin, Ho, Wo, KW, SH, SW, PH, PW;
};
hipError_t launch_conv_f32(const ConvF32Args& args, int act, hipStream_t stream);

// bf16 3x3 stride-1 pad-1 convolution with the input halo resident in LDS.
struct HaloArgs {
    const uint16_t* x;      // [N][H][W][Cin]
    const uint16_t* w;      // [Cout][3][3][Cin]
    const float* bias;      // [Cout] or nullptr
    const uint16_t* res;    // [N][H][W][Cout] or nullptr
    uint16_t* y;            // [N][H][W][Cout]
    int N, H, W, Cin, Cout;
    int co_tiles;           // Cout / 64
};
struct HaloPlan {
    int kind;        // 0: one row tile per workgroup, weights streamed; 1: Cin = 64, weights resident;
                     // 2: small images, one image x 32 output channels per workgroup
    int th;          // output rows per tile
    int row_tiles;   // ceil(H / th)
    int wf;          // 32-pixel fragments per wave (1 or 2)
    int halo_kb;     // LDS reserved for one halo
    int per_xcd;     // kind 1: spatial tiles per XCD
};
// False when the shape does not qualify (Cin = 64 or a multiple of 128, Cout a
// multiple of 64, the halo of one output row within 96 KB; or, for kind 2, Cin a
// multiple of 64, Cout of 32 and a small image).  resident_ok = false restricts the
// plan to the streaming kernel (kind 0).
bool conv_halo_plan(int N, int H, int W, int Cin, int Cout, bool resident_ok, HaloPlan* plan);
hipError_t launch_conv_halo(const HaloArgs& args, const HaloPlan& plan, int act, hipStream_t stream);

// bf16 convolution for inputs with few channels (c_in <= 4, e.g. a ResNet stem): weights and
// the input patch of `th` output rows re-laid in LDS with 4-channel pixels, one workgroup
// per CU with compute and store waves.
struct SmallCArgs {
    const uint16_t* x;      // [N][H][W][Cin]
    const uint16_t* w;      // [Cout][KH][KW][Cin]
    const float* bias;      // [Cout] or nullptr
    const uint16_t* res;    // [N][Ho][Wo][Cout] or nullptr
    uint16_t* y;            // [N][Ho][Wo][Cout]
    int N, H, W, Cin, Cout, KH, KW, SH, SW, PH, PW, Ho, Wo;
    int kwp;                // KW + toff rounded up to a multiple of 4
    int pw;                 // patch width in pixels (even)
    int pwl;                // patch column of image column 0: PW rounded up to even
    int toff;               // pwl - PW: kernel column s is tap s + toff
    int th;                 // output rows per workgroup
    int row_tiles;          // ceil(Ho / th)
    int co_blocks;          // ceil(Cout / 64)
};
// False when the shape does not qualify (Cin <= 4, Cout a multiple of 32, W*Cin a multiple
// of 8, KW + toff <= 16, and the weights of 64 channels, 64 KB of staged output and the
// patch of one output row within 160 KB of LDS); fills everything but the pointers.
bool conv_smallc_plan(int N, int H, int W, int Cin, int Cout, int KH, int KW, int SH, int SW, int PH, int PW,
                      int Ho, int Wo, SmallCArgs* args);
hipError_t launch_conv_smallc(const SmallCArgs& args, int act, hipStream_t stream);

// Feed-forward block FC1 -> act -> FC2 (+ b2, + residual) in one kernel; weights packed in
// MFMA fragment order (dlf_ffn_pack).
struct FfnArgs {
    const uint16_t* x;      // [M][D]
    const uint16_t* w1p;    // W1 [F][D], packed
    const float* b1;        // [F] or nullptr
    const uint16_t* w2p;    // W2 [D][F], packed
    const float* b2;        // [D] or nullptr
    const uint16_t* res;    // [M][D] or nullptr
    uint16_t* y;            // [M][D]
    int64_t M;
    int D, F;               // D in {256, 512, 768, 1024}; F a positive multiple of 256
    // parts S > 1: S workgroups a token block, each over 1/S of d_ff, write fp32 partial sums
    // of y to ws [S][M][D], which a second kernel adds with b2 and the residual
    int parts;
    float* ws;
};
// the d_ff parts the fused FFN splits into for these sizes (1 = no split); DLF_FFN_SPLIT=<S>
// forces S (0 or 1: no split) where a split is built
int ffn_parts(int64_t M, int D, int F);
hipError_t launch_ffn(const FfnArgs& args, int act, hipStream_t stream);

// A launch has fewer than 2^32 threads along x: workgroups of 256 have to stay below this.
constexpr int64_t kMaxWorkgroups = int64_t(1) << 24;

// Page plan: block tables and slot maps from request lengths (dlf_page_plan).
struct PagePlanArgs {
    const int32_t* cached;      // [requests]
    const int32_t* fresh;       // [requests]
    const int32_t* free_pages;  // [free_cap]
    const int32_t* free_head;   // nullable (= 0)
    int32_t* table;             // [requests][max_pages]
    int32_t* starts;            // [requests + 1]
    int32_t* lens;              // [requests]
    int64_t* slots;             // [token_cap]
    int32_t* rows;              // [token_cap] or nullptr
    int32_t* counts;            // [4]
    int requests, page_size, max_pages, token_cap, free_cap;
};
hipError_t launch_page_plan(const PagePlanArgs& args, hipStream_t stream);

// New keys and values into the paged cache's slots (dlf_paged_store).
struct PagedStoreArgs {
    const uint16_t* src[2];     // k, v: [tokens][kv_heads][head_dim], rows stride[] apart
    void* cache[2];             // [pages][kv_heads][page_size][head_dim]
    const int64_t* slots;       // [tokens]
    int64_t stride[2];
    float inv_scale[2];         // fp8 cache
    int64_t tokens;
    int64_t slot_count;         // pages * page_size (< 2^31)
    int kv_heads, head_dim, page_size;
    bool fp8;
};
int paged_store_tokens(int kv_heads, int head_dim);   // tokens that a workgroup takes
hipError_t launch_paged_store(const PagedStoreArgs& args, hipStream_t stream);

// Attention of one new token per request over the paged cache (dlf_paged_attention).
struct PagedAttnArgs {
    const uint16_t* q;          // [requests][heads][head_dim], requests q_stride apart
    const uint8_t* k;           // [pages][kv_heads][page_size][head_dim]
    const uint8_t* v;
    const int32_t* table;       // [requests][max_pages]
    const int32_t* lens;        // [requests]
    uint16_t* out;              // [requests][heads][head_dim]
    float* lse;                 // [requests][heads] or nullptr
    // workspace, unused where aim is 0
    float* part_o;              // [items + aim][min(group, 16)][head_dim]: the pieces' sums
    float* part_ml;             // the same rows' maximum and sum
    int32_t* pieces;            // [requests][2]: a request's first piece among all requests', and its pieces
    int64_t q_stride;
    int requests, heads, kv_heads, page_size, pages, max_pages, window;
    int group;                  // heads / kv_heads
    int head_tiles;             // ceil(group / 16)
    int aim;                    // pieces that the items are cut into if they are long, 0: none is cut
    int least;                  // tiles that are not cut further
    float score_scale;          // softmax_scale * k_scale * log2(e)
    float v_scale;
};
void plan_paged_attention(PagedAttnArgs* args, int row_bytes, int max_len);   // fills aim and least
hipError_t launch_paged_attention(const PagedAttnArgs& args, int head_dim, bool fp8, hipStream_t stream);

// Low-rank adapters beside a projection (dlf_lora_add).
struct LoraArgs {
    const uint16_t* x;          // [m][k], rows x_stride apart
    const uint16_t* a;          // [adapters][rank][k]
    const uint16_t* b;          // [adapters][n][rank]
    const float* scale;         // [adapters] or nullptr (= 1)
    const int32_t* ids;         // [m], or [requests] with a row map
    const int32_t* row_map;     // [m] or nullptr
    const uint16_t* base;       // [m][n], rows base_stride apart, or nullptr
    uint16_t* out;              // [m][n], rows out_stride apart
    float* h;                   // workspace: [parts][m][rank] partial sums of x A^T
    uint16_t* nowhere;          // and 1 KB after them
    int64_t x_stride, base_stride, out_stride;
    int m, n, k, rank, adapters, requests;
    int parts;                  // k slices of the first product (lora_parts)
};
int lora_parts(int m, int k, int rank, int adapters);
hipError_t launch_lora(const LoraArgs& args, hipStream_t stream);

// Root-mean-square norm of rows (dlf_rms_norm).
struct RmsNormArgs {
    const void* x;              // [rows][cols], fp32 or bf16
    const void* residual;       // nullable
    const float* weight;        // [cols] or nullptr (= 1)
    void* sum;                  // nullable
    void* y;
    float* scale;               // [rows][scale_stride], block scales of an e4m3 y, or nullptr
    int64_t rows;               // < 2^31
    int64_t x_stride, residual_stride, sum_stride, y_stride;
    int cols, scale_stride;
    float eps, inv_scale;
    double inv_cols;            // 1 / cols
};
// out: kOutBf16 / kOutF32 / kOutFp8 (block scales where scale is given, else inv_scale)
hipError_t launch_rms_norm(const RmsNormArgs& args, bool f32, int out, hipStream_t stream);
hipError_t launch_rms_norm_f32(const RmsNormArgs& args, int out, hipStream_t stream);

// Rows into e4m3 codes with a scale for each 128 columns (dlf_quant_blocks).
struct QuantBlocksArgs {
    const void* x;              // [rows][cols], fp32 or bf16
    uint8_t* codes;
    float* scale;               // [rows][scale_stride]
    int64_t x_stride, codes_stride;
    uint32_t blocks;            // of all rows, < 2^31
    int cols, row_blocks, scale_stride;
};
hipError_t launch_quant_blocks(const QuantBlocksArgs& args, bool f32, hipStream_t stream);
hipError_t launch_quant_blocks_f32(const QuantBlocksArgs& args, hipStream_t stream);

// Product of e4m3 matrices with block scales (dlf_gemm_blocks, dlf_gemm_blocks_gated).
struct GemmBlocksArgs {
    const uint8_t* a;           // [m][k]
    const float* a_scale;       // [m][a_scale_stride]
    const uint8_t* b;           // [n][k]
    const float* b_scale;       // [ceil(n / 128)][b_scale_stride]; gated: [2 ceil(n / 256)]
    const float* shift;         // [n] or nullptr
    const uint16_t* residual;   // [m][n] or nullptr
    uint16_t* c;                // [m][n]; gated: [m][n / 2]
    int64_t m;
    int n, k;
    int a_scale_stride, b_scale_stride;
    int kind;                   // kGemmBlocks*
    // the sum over k in parts (> 1: each goes to the workspace, and a second kernel joins them)
    int parts, part_blocks;     // part_blocks: blocks of 128 of a part, a multiple of 4 where there are several
    int part_stride;            // n, rounded up to a multiple of 4
    float* part;                // [parts][m][part_stride]
};
// the kernels: up to 16 or 32 rows of a, 16 rows of b a workgroup or 32, and tiles
enum : int {
    kGemmBlocks16 = 0, kGemmBlocks16Wide = 1, kGemmBlocks32 = 2, kGemmBlocks32Wide = 3,
    kGemmBlocksTile64 = 4, kGemmBlocksTile128 = 5, kGemmBlocksTile128Deep = 6, kGemmBlocksTile256 = 7
};
void plan_gemm_blocks(GemmBlocksArgs* args);    // fills kind, parts, part_blocks and part_stride from m, n and k
// act: kAct*, or kActSiluMul.. for the gated form
hipError_t launch_gemm_blocks_skinny(const GemmBlocksArgs& args, int act, hipStream_t stream);
hipError_t launch_gemm_blocks_join(const GemmBlocksArgs& args, int act, hipStream_t stream);
hipError_t launch_gemm_blocks(const GemmBlocksArgs& args, int act, hipStream_t stream);

// Shader-clock probe: workgroups x 4 waves of back-to-back bf16 MFMAs; stamps[4 b + 0..3] =
// s_memtime before / after, s_memrealtime before / after, for workgroup b.
hipError_t launch_clock_probe(int workgroups, int iters, uint64_t* stamps, hipStream_t stream);

// Elementwise passes of the unfused chain.  dt: 0 fp32, 1 bf16.
hipError_t launch_bn_apply(int64_t rows, int64_t c, int dt, const void* y, const float* gamma,
                           const float* beta, const float* mean, const float* var, float eps,
                           void* z, hipStream_t stream);
hipError_t launch_scale_shift(int64_t rows, int64_t c, int dt, const void* y, const float* scale,
                              const float* shift, void* z, hipStream_t stream);
hipError_t launch_add(int64_t count, int dt, const void* a, const void* b, void* out,
                      hipStream_t stream);
hipError_t launch_act(int64_t count, int dt, int act, const void* in, void* out, hipStream_t stream);
hipError_t launch_quant(int64_t count, const float* in, float inv_scale, uint8_t* codes,
                        hipStream_t stream);

}  // namespace dlf
