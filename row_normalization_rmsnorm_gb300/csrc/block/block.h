// block.h -- parameters and launchers of the block-boundary kernels
// (block.cuh), which also run the norms whose input is kept as an 8-bit
// checkpoint (ckpt.cuh).
#pragma once

#include "../launch.h"

namespace gb300norm {

// Streamed row inputs.  The forward reads X, R (residual) and, when gate rows
// are streamed, G; the backward R (the gradient of h), DY, X and H (saved rows
// or checkpoints) and G.
enum BlockStream : int { SX = 0, SR = 1, SG = 2, SDY = 3, SH = 4, kBlockStreams = 5 };

struct BlockParams {
  const char* in[kBlockStreams];     // null = absent
  int64_t in_stride[kBlockStreams];  // bytes between rows
  uint32_t soff[kBlockStreams];      // offset in a stage
  uint32_t stage_bytes;
  int room_x;                        // the launch shape counts x's stream, read or not
  int part;                          // columns of a slice when a row is split
  int64_t min_stride;                // smallest in_stride of the rows of the activations' type
  // outputs: h and y (forward), the gradients of the residual and of x
  // (backward); null = not wanted
  char* out_a;  int64_t a_stride;    // h / d residual
  char* out_b;  int64_t b_stride;    // y / dx
  char* xq;  char* hq;  int64_t q_stride;   // checkpoints (forward)
  char* dg;  int64_t dg_stride;      // gate gradient rows (bytes)
  // per column
  const void* w1;                    // norm of the block's output, null = none
  const void* w2;                    // norm of h, null = none
  const void* bias;                  // LayerNorm bias, nullable
  const void* gate;  int64_t gate_stride;   // gate held per column, elements between rows
  int w_code, gate_code, fmt;        // element types; checkpoint format
  // per row
  float* rs1_out;  float* rs2_out;  float* mean_out;
  const float* rs1;  const float* rs2;
  // weight-gradient partial rows, FP32, [row groups][N]; the gate's: head and
  // tail rows of each row group (see block_bwd_kernel)
  float* ws1;  float* ws2;  float* ws_head;  float* ws_tail;
  // from one row of a row group to its next: rows, and bytes of each output
  int64_t row_step, a_step, b_step, q_step, dg_step;
  int64_t M;
  int64_t R;         // rows per gate row
  int64_t n_gates;   // gate rows
  int N;
  float alpha, beta, offset, eps;
  int post, pre;     // norm of the block's output / norm of h present
  int seg;           // rows are dealt out in contiguous ranges (several gate rows, R > 1, backward)
  int* status;
  int hold_last;
};

// First row of row group c when M rows are dealt out in G contiguous ranges,
// and the group that holds a row.
__host__ __device__ inline int64_t seg_begin(int64_t c, int64_t M, int64_t G) { return M * c / G; }
__host__ __device__ inline int64_t seg_owner(int64_t row, int64_t M, int64_t G) { return ((row + 1) * G + M - 1) / M - 1; }

struct BlockFlags {
  bool ln = false;      // h's norm is LayerNorm
  bool norm = false;    // RMSNorm or fused add: no first norm, gate and scales
  bool grow = false;    // gate rows are streamed
  bool q8 = false;      // checkpoints: written (forward) or read (backward)
  bool acc = false;     // weight (or broadcast gate) gradients wanted (backward)
  bool aligned = false; // every streamed row starts on 16 bytes
};

// *grid receives the number of row groups (partial rows written).
int launch_block_fwd(const BlockParams&, int dtype, const BlockFlags&, const DevInfo&, cudaStream_t, int* grid);
int launch_block_bwd(const BlockParams&, int dtype, const BlockFlags&, const DevInfo&, cudaStream_t, int* grid);

// One translation unit per type, direction and group of flags.
template <class T, bool Q8> int launch_block_fwd_t(const BlockParams&, const BlockFlags&, const DevInfo&, cudaStream_t, int*);
template <class T, bool Q8, bool ACC>
int launch_block_bwd_t(const BlockParams&, const BlockFlags&, const DevInfo&, cudaStream_t, int*);

// The column sums of a backward's G partial rows: dw1, dw2 (null = not wanted; of
// dw_code) and the gradient (p.dg) of a gate with fewer rows than M (n_gates of
// them, 0: not wanted).
int launch_block_reduce(const BlockParams&, void* dw1, void* dw2, int dw_code, int G, cudaStream_t);

int launch_ckpt_encode(const char* x, int64_t x_stride, char* q, int64_t q_stride, int64_t M, int64_t N, int fmt,
                       int dtype, const DevInfo&, cudaStream_t);
int launch_ckpt_decode(const char* q, int64_t q_stride, char* x, int64_t x_stride, int64_t M, int64_t N, int fmt,
                       int dtype, const DevInfo&, cudaStream_t);

// Bytes a row may have: 8 CTAs a row, each with two stages of five streams of a
// slice in shared memory (160 KB of 227).
constexpr int64_t kBlockMaxRowBytes = 131072;

}  // namespace gb300norm
