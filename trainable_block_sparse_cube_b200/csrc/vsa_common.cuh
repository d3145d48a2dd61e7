// Shared definitions of the VSA kernels (device side) and their launchers.
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cstdint>

namespace vsa {

// Bits of the device error word kept in the workspace.
enum : int { kErrTimeout = 1, kErrBadIndex = 2 };

constexpr int kCube = 64;  // tokens per 4x4x4 cube

// Raster token index of in-cube slot r of cube c (cube and slot numbering as
// documented in include/vsa.h).
__host__ __device__ __forceinline__ int cube_token(int c, int r, int H, int W) {
  const int Hc = H >> 2, Wc = W >> 2;
  const int ct = c / (Hc * Wc), ch = (c / Wc) % Hc, cw = c % Wc;
  const int t = 4 * ct + (r >> 4), h = 4 * ch + ((r >> 2) & 3), w = 4 * cw + (r & 3);
  return (t * H + h) * W + w;
}

struct GatherParams {
  const __nv_bfloat16* src[3];  // q, k, v raster [BH, N, D]
  __nv_bfloat16* dst[3];        // cube-major [BH, C, 64, D]; null: pool only for that tensor
  float* pool[3];               // [BH, C, D] cube means
  __nv_bfloat16* split[3];      // [3, BH, C, D] the means as three bf16 terms (hi, mid, lo)
  int BH, C, H, W, N;
};

struct CoarseParams {
  // 3-D maps (128-byte swizzle) over the bf16 three-term splits:
  //   tm_qs, tm_ks: [3 * BH][C][D], boxes of 128 rows x 64 channels;
  //   tm_vs: [3 * BH][C][D], boxes of 64 rows x 64 channels;
  //   tm_ps: [3 * BH][C][Cp], boxes of 128 rows x 64 columns.
  CUtensorMap tm_qs, tm_ks, tm_vs, tm_ps;
  float* s;            // [BH, C, C] scores
  __nv_bfloat16* psplit;  // [3, BH, C, Cp] coarse probabilities as bf16 terms (hi, mid, lo)
  int p_terms;         // terms of P written: 2 (the forward's output product), 3 (the backward's products)
  float* oc;           // [BH, C, D]
  float* oc_copy;      // optional second destination of oc (may be null)
  int Cp;              // C rounded up to a multiple of 8 (row pitch of psplit)
  int* err;
  unsigned long long wait_ns;
  int32_t* idx;        // [BH, C, kcap]
  int32_t* cnt;        // [BH, C]
  int BH, C, D, kcap;
  int topk;            // > 0: top-K; 0: top-p
  float top_p;
  int kmin, kmax;
  int do_select;       // 0: only probabilities (selection supplied by the caller)
  float scale;         // 1/sqrt(D)
};

struct FineParams {
  // tm_out: 5-D map over the raster out [BH][T][H][W][D] bf16; a box is one
  // cube's 4 x 4 x 4 tokens by 64 channels, in the 128-byte swizzle.
  // tm_k, tm_v: 2-D maps over the cube-major copies (rows of D bf16, 64 x 64 boxes).
  CUtensorMap tm_k, tm_v;
  CUtensorMap tm_out;
  const __nv_bfloat16* q;        // [BH, N, D] raster (query cubes are read from here)
  const int32_t* idx;            // [BH, C, kcap]
  const int32_t* cnt;            // [BH, C] or null (then every row has kcap ids)
  const int32_t* order;          // [BH * C] item order (schedule.cu), or null: items in index order
  const float* oc;               // [BH, C, D]
  const float* gate_c;           // [BH, N]
  const float* gate_f;           // [BH, N]
  __nv_bfloat16* out;            // [BH, N, D] or null
  float* out_fine;               // [BH, N, D] or null
  float* o_fine;                 // [BH, N, D] fp32 fine output saved for the backward pass, or null
  float* lse;                    // [BH, N] natural-log softmax denominators saved for the backward pass, or null
  int* err;
  unsigned long long wait_ns;
  int BH, C, H, W, N, kcap, n_items;
  float scale_log2;              // log2(e)/sqrt(D)
  int debug_stall;
};

// ---------------------------------------------------------------- backward pass
// Per-token preparation of the backward pass (one warp per query cube).
struct PrepParams {
  const __nv_bfloat16* dout;   // [BH, N, D] raster, gradient of the gated output
  const float* ofine;          // [BH, N, D] raster, fp32 fine output saved by the forward
  const float* lse;            // [BH, N] raster, natural-log softmax denominators saved by the forward
  const float* gate_c;         // [BH, N]
  const float* gate_f;         // [BH, N]
  const float* oc;             // [BH, C, D] coarse output (recomputed)
  __nv_bfloat16* do_cube;      // [BH, C, 64, D] gate_f * dout, cube-major (bf16)
  float* qstat;                // [BH, C, 2, 64]: lse * log2(e) and delta = bf16(gate_f dout) . ofine
  float* doc;                  // [BH, C, D] gradient of the coarse output
  __nv_bfloat16* docsplit;     // [3, BH, C, D] the same as three bf16 terms (hi, mid, lo)
  float* dlc;                  // [BH, C] doc . oc per cube
  float* dgate_c;              // [BH, N]
  float* dgate_f;              // [BH, N]
  int BH, C, H, W, N;
};

// Backward of the coarse attention on the pooled tokens: four C x C x D
// products per head on the tensor cores, each fp32 operand as three bf16
// terms (as in the forward's coarse products).
struct CoarseBwdParams {
  // 3-D maps [3 * BH][rows][cols] over three-term bf16 operands, 128-byte swizzle, boxes {64 cols, rows}:
  CUtensorMap tm_doc128, tm_vb128;         // dOc, vbar [C][D], 128-row boxes (dS product: A, B K-major)
  CUtensorMap tm_ds128;                    // dS [C][Cp], 128-row boxes (dqbar product: A K-major)
  CUtensorMap tm_kb64, tm_qb64, tm_doc64;  // kbar, qbar, dOc [C][D], 64-row boxes (B operands, N-major)
  CUtensorMap tm_ds64, tm_p64;             // dS, P [C][Cp], 64-row boxes (A MN-major: dkbar, dvbar products)
  const __nv_bfloat16* psplit;  // [3, BH, C, Cp] coarse probabilities (three terms), read by the dS epilogue
  __nv_bfloat16* dssplit;       // [3, BH, C, Cp] dS = P (dOc vbar^T - delta_c) as three terms (written)
  int Cp;
  const float* dlc;             // [BH, C]
  float* dqbar;                 // [BH, C, D] gradients of the pooled q, k, v
  float* dkbar;
  float* dvbar;
  int* err;
  unsigned long long wait_ns;
  int BH, C, D;
  float scale;                  // 1/sqrt(D)
};

// Transposed selection lists: for every KV cube, the query cubes that selected it.
struct TlistParams {
  const int32_t* idx;   // [BH, C, kcap]
  const int32_t* cnt;   // [BH, C] or null (every row holds kcap ids)
  uint32_t* bitmap;     // [BH, C, W32] bit i of row j: query cube i selected KV cube j
  int32_t* tcnt;        // [BH, C]
  int32_t* toff;        // [BH, C] absolute offsets into tlist
  int32_t* tlist;       // [BH * C * kcap] ascending query-cube ids per KV cube
  int* err;
  int BH, C, kcap, W32;
};

// Block-sparse fine attention backward (tcgen05). The dQ kernel walks query
// cubes over their selected KV cubes; the dK/dV kernel walks KV cubes over
// the query cubes that selected them.
struct BwdFineParams {
  // 2-D maps over cube-major copies [BH * C * 64][D] bf16, 64 x 64 boxes, 128-byte swizzle
  CUtensorMap tm_q, tm_k, tm_v, tm_do;
  // 5-D store maps over raster outputs [BH][T][H][W][D] bf16: dQ kernel tm_out0 = dq;
  // dK/dV kernel tm_out0 = dk, tm_out1 = dv
  CUtensorMap tm_out0, tm_out1;
  const int32_t* list;   // dQ: idx [BH * C, kcap]; dK/dV: the flat transposed lists
  const int32_t* cnt;    // dQ: counts or null (kcap each); dK/dV: tcnt
  const int32_t* off;    // dK/dV: toff; dQ: null
  const int32_t* order;  // [BH * C] item order (schedule.cu), or null: items in index order
  const float* qstat;    // [BH * C, 2, 64]
  const float* cpart0;   // [BH * C, D] coarse-path gradient rows: dQ kernel dq_bar; dK/dV kernel dk_bar
  const float* cpart1;   // dK/dV kernel dv_bar
  int* err;
  unsigned long long wait_ns;
  int BH, C, H, W, N, kcap, n_items;
  float scale_log2;      // log2(e) / sqrt(D)
  float scale;           // 1 / sqrt(D)
};

// ---------------------------------------------------------------- rotary positions, norm
constexpr int kRopeAxes = 4, kRopePairs = 128;

// q or k of a rotation: strided views [B, heads, N, D] (element strides, channels contiguous).
struct RopeTensor {
  const void* in;
  const void* dy;      // norm backward: gradient of the output
  void* out;
  const float* w;      // norm weight [D] or null (ones)
  int heads;           // 0: no such tensor
  long long in_b, in_h, in_n, dy_b, dy_h, dy_n, out_b, out_h, out_n;
};

// Division of numbers below 2^31 by a number known on the host:
// n / d = n m >> s, m the whole number above 2^s / d, s = 31 + log2 d rounded up.
struct Divisor {
  uint32_t m = 0;
  int s = 0;
  Divisor() = default;
  explicit Divisor(uint32_t d) {
    for (s = 31; (1ull << (s - 31)) < d; ++s) {}
    m = (uint32_t)((1ull << s) / d + 1);
  }
  __device__ __forceinline__ uint32_t operator()(uint32_t n) const { return (uint32_t)((uint64_t)n * m >> s); }
};

// One pair of channels: the axis it turns with, and how far for one position.
struct RopePair {
  uint32_t lo, hi;  // fraction of a turn, in 2^-64
  uint32_t whole;   // whole turns, modulo 2^32 (they count between whole positions)
  int axis;
};

struct RopeParams {
  RopeTensor t[2];          // q, k
  int B, N, D;
  int rot, interleaved;     // rotated leading channels; pairs (2i, 2i + 1) or (i, i + rot/2)
  int axes;
  RopePair pairs[kRopePairs];
  int pos_kind;             // 0: raster grid of H x W frames; 1: int32 list; 2: fp32 list
  int H, W, origin[3];
  Divisor by_h, by_w;       // of a raster grid
  const void* pos;          // list [B or 1, N, axes]
  long long pos_batch;      // elements between batches of the list (0: one list for all)
  int back;                 // rotate by the opposite angle
  int norm;
  float eps;
  int wide;                 // every 8 fp32 channels of the outputs start on a 32-byte boundary
  float* partial;           // norm backward: [grid, 2, D] weight gradients of the blocks
  int tiles, groups;        // work split, set by the launcher
  unsigned units;
  Divisor by_groups, by_tiles;
};

cudaError_t launch_rope(RopeParams p, int type, int num_sms, cudaStream_t st);
size_t norm_rope_partial_bytes(int D, int num_sms);
cudaError_t launch_norm_rope_backward(RopeParams p, int type, float* dwq, float* dwk, int num_sms, cudaStream_t st);

// ---------------------------------------------------------------- linear product
enum : int { kActNone = 0, kActSilu = 1, kActGelu = 2, kActGeluTanh = 3 };

// A strided 16-bit tensor [B, heads, N, D] seen as B x N rows of heads * D channels.
struct RowsView {
  void* data;
  int heads, D;
  long long s_b, s_h, s_n;
};

// The tiles' order: blocks of kTileGroup row tiles by all columns (see linear.cu).
constexpr int kTileGroup = 8;
struct TileOrder {
  int rows = 0, cols = 0, block = 0;  // row tiles of all batches, column tiles, tiles of a block
  Divisor by_block;
  TileOrder() = default;
  TileOrder(int r, int c) : rows(r), cols(c), block(kTileGroup * c), by_block(kTileGroup * c) {}
};

// Test hook: operands are left unloaded, or the odd CTAs load theirs only after the wait for them ran out.
enum : int { kStallUnloaded = 1, kStallLate = 2 };

// out = A B^T on the tensor cores. A and B are 4-D maps (channel of a head,
// row, head, batch) in 128-byte swizzle with boxes of 64 channels. A K-major operand is read along
// its channels, an MN-major one along its rows.
struct GemmParams {
  CUtensorMap ta, tb;
  RowsView out, residual, z;  // residual, z: data null for none
  float* partial;           // parts of split tiles [splits, rest, 256, bn]
  int wide;                 // out, residual, z and partial are accessed in aligned 32-byte pieces
  int a_d, b_d;             // channels of a head of A, B
  int a_rows;               // rows of A's boxes (K-major)
  int stages, stage_bytes;  // ring of operand stages: A's tile, then B's at tile_a
  int tile_a;
  int bn;                   // columns of a tile: a multiple of 32, 64 to 256
  int batches, row_tiles;   // batches x row_tiles tiles of 256 rows
  int rows;                 // rows of a batch
  int F;                    // columns
  TileOrder order;
  Divisor by_row_tiles, by_rest;
  int kblocks;              // 64-long blocks of the contraction
  int kblocks_batch;        // kGemmWeight: blocks of a batch of rows
  int whole, rest, splits;  // tiles computed in one go, and those computed in parts of the contraction
  const float* bias;        // [F] or null
  int act;
  int stall;                // test hook: kStall...
  unsigned long long wait_ns;
  unsigned failures;        // word that counts waits that ran out
  long long units;          // whole + rest x splits
};

// Sums the parts of the split tiles (number first, first + 1, ...) and applies the epilogue.
struct FinishParams {
  const float* partial;     // [splits, rest, 256, bn]
  int first, rest, splits, bn, row_tiles, rows, F;
  TileOrder order;
  const float* bias;
  int act;
  RowsView residual, z, out;   // data null: none
};

struct FewRowsParams {
  RowsView x, residual, z, out;
  const void* w;
  long long w_stride;
  const float* bias;
  int act, rows, batches, K, F;
};

// dz = dout act'(z) (with an activation) and column sums of dz in fp32.
struct SlopeParams {
  RowsView dout, z;
  void* dz;                 // [batches * rows, F], with an activation
  float* partial;           // [blocks_y, F] column sums (db itself, if there is one) or null
  int act, batches, rows, F;
  Divisor by_rows;
  int blocks_y;
};

enum : int { kGemmForward = 0, kGemmInput = 1, kGemmWeight = 2 };
constexpr int kFewRows = 32;
constexpr int kGemmMaxStages = 16;
// type: 0 bf16, 1 fp16
cudaError_t launch_linear_gemm(const GemmParams& p, int kind, int type, int num_sms, cudaStream_t st);
cudaError_t launch_linear_finish(const FinishParams& p, int type, cudaStream_t st);
cudaError_t launch_linear_few_rows(const FewRowsParams& p, int type, cudaStream_t st);
cudaError_t launch_linear_slope(const SlopeParams& p, int type, float* db, cudaStream_t st);
// The current device's counts of waits that ran out in linear products: word 0
// those captured into graphs, the others those of streams (synchronises `st`).
constexpr int kLinearFailureWords = 256;
cudaError_t linear_failures(unsigned (&counts)[kLinearFailureWords], cudaStream_t st);

cudaError_t launch_gather(const GatherParams& p, int D, int num_sms, cudaStream_t st);
cudaError_t launch_coarse(const CoarseParams& p, cudaStream_t st);
cudaError_t launch_fine(const FineParams& p, int D, int grid, cudaStream_t st);
cudaError_t launch_bwd_prep(const PrepParams& p, int D, cudaStream_t st);
cudaError_t launch_coarse_bwd(const CoarseBwdParams& p, cudaStream_t st);
cudaError_t launch_tlists(const TlistParams& p, cudaStream_t st);
cudaError_t launch_fine_dq(const BwdFineParams& p, int D, int grid, cudaStream_t st);
cudaError_t launch_fine_dkv(const BwdFineParams& p, int D, int grid, cudaStream_t st);
cudaError_t launch_schedule(const int32_t* len, int32_t* order, int BH, int C, int maxlen, cudaStream_t st);
cudaError_t launch_l2_read(const void* buf, size_t bytes, int passes, int* status, int grid, cudaStream_t st);

}  // namespace vsa
