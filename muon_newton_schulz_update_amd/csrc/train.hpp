// Descriptors shared by the training-step kernels (train_kernels.hip,
// head_kernels.hip) and their host code (train_api.cpp).
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/libmuon.h"

namespace muon {

// ---------------------------------------------------------------------------
// Tensor lists (gradient norm, scaling, AdamW). A list travels in the kernel
// arguments, up to kListMax tensors a launch, so a call uploads nothing and
// can be captured in a graph; longer lists take more launches.
// ---------------------------------------------------------------------------
constexpr int kChunk = 8192;      // elements per work item of a list kernel
constexpr int kNormMax = 88;      // tensors per norm or scale launch
constexpr int kAdamMax = 32;      // tensors per AdamW launch
constexpr int kNormChunk = 32768; // the norm kernel's (1024 threads, four pieces of eight elements each)
constexpr int kNormBlocks = 512;  // blocks of a norm launch at most (one partial each)

struct ListItem {      // one tensor: 40 bytes
  const void* src;
  int64_t ld;          // row stride, elements
  int64_t cols;
  int64_t n;           // rows * cols
  int32_t dt;          // MUON_F32 / MUON_BF16
  int32_t flat;        // 1: one contiguous run with 16-byte aligned start
};
struct NormList {
  int32_t n;
  int32_t chunk0[kNormMax + 1];   // first work item of each tensor
  ListItem t[kNormMax];
};
static_assert(sizeof(NormList) <= 4000, "kernel arguments");

// One destination beside one source (scaling).
constexpr int kScaleMax = 56;
struct ScaleItem {
  const void* src;
  void* dst;
  int64_t ld_src, ld_dst, cols, n;
  int32_t dt;          // bit 0: source bf16, bit 1: destination bf16, bit 2: flat
};
struct ScaleList {
  int32_t n;
  int32_t chunk0[kScaleMax + 1];
  ScaleItem t[kScaleMax];
};
static_assert(sizeof(ScaleList) <= 4000, "kernel arguments");

struct AdamItem {
  const void* g;
  float* m;
  float* v;
  void* w;
  void* copy;          // or null
  int64_t ld[5];       // of g, m, v, w, copy
  int64_t cols, n;
  int32_t dt;          // bit 0: g bf16, bit 1: w bf16, bit 2: copy bf16, bit 3: flat
};
struct AdamList {
  int32_t n;
  int32_t chunk0[kAdamMax + 1];
  AdamItem t[kAdamMax];
};
static_assert(sizeof(AdamList) <= 4000, "kernel arguments");

struct AdamConst {
  float beta1, c1;      // 1 - beta1
  float beta2, c2;
  float keep;           // 1 - lr weight_decay
  float lr1;            // lr / (1 - beta1^step)
  float rs2;            // 1 / sqrt(1 - beta2^step)
  float eps;
};
// Step and rate that are read from the device when the kernel runs, and what
// AdamConst's dependent members are made of (both pointers null: not used).
struct AdamClock {
  const int64_t* step_at;
  const float* lr_at;
  int64_t step;
  double lr, weight_decay;
  double log2_b1, log2_b2;
};

// The norm kernel's state in the handle's workspace.
struct NormState {
  uint32_t ticket;      // blocks done; the last one of a call sets it back to 0
  uint32_t pad[3];
  double part[1];       // one partial per block of every launch of the call
};

hipError_t launch_norm(const NormList& L, int blocks, int chunks, NormState* st, int part0, int total_blocks,
                       float max_norm, float* norm, float* coef, hipStream_t s);
hipError_t launch_norm_reset(NormState* st, hipStream_t s);
hipError_t launch_norm_empty(float max_norm, float* norm, float* coef, hipStream_t s);
hipError_t launch_scale(const ScaleList& L, int chunks, const float* coef, int in_place, hipStream_t s);
hipError_t launch_adamw(const AdamList& L, int chunks, const AdamConst& c, const AdamClock& clock, const float* scale,
                        hipStream_t s);

// ---------------------------------------------------------------------------
// Head cross entropy. The valid tokens (target != ignore_index) are gathered
// into a compact order and taken in pieces of at most `piece` tokens.
//
// Panel layout of the per-piece matrices (rows = tokens, contraction over
// either index): blocks of 64 tokens; in a block, columns in 16-byte chunks,
// chunk after chunk, each chunk for the block's 64 tokens in turn. A stage of
// a product over tokens or over columns is then whole kilobytes either way.
// ---------------------------------------------------------------------------
constexpr int kPanelRows = 64;
// Kept exponentials of 16-bit inputs, in [2^-63, 1]: the fp32 pattern's 6 low
// bits of exponent and 10 high bits of mantissa, rounded half up; kCodeBase is
// the pattern of 2^-63 shifted down.
constexpr uint32_t kCodeBase = 64u << 10;
template <typename T>
__host__ __device__ inline int64_t panel_at(int64_t row, int64_t col, int64_t ld) {
  constexpr int ch = 16 / (int)sizeof(T);
  return ((row / kPanelRows) * (ld / ch) + col / ch) * (kPanelRows * ch) + (row % kPanelRows) * ch + col % ch;
}

struct HeadArgs {
  const void* h;   int64_t ld_h;
  const void* w;   int64_t ld_w;      // the caller's weight, or its padded copy
  const void* w_src; int64_t ld_src;  // the weight to copy, or null
  void* dh;        int64_t ld_dh;
  void* dw;        int64_t ld_dw;
  int32_t n, v, d;                    // tokens, vocabulary, width
  int32_t dp, vp;                     // padded width (64 or 32 elements), padded vocabulary (256)
  int32_t w_cols;                     // columns of w: d, or dp of a padded copy
  int32_t vtile, n_vt;                // vocabulary columns per statistic of a token, statistics
  int32_t piece, row0;                // tokens per piece (buffers), first compact token of this piece
  int32_t rows_max;                   // tokens of this piece if none is ignored
  const void* targets;
  int64_t ignore;
  int32_t target_bytes;
  int32_t per_token;                  // reduction none
  int32_t mean;
  int32_t half;                       // 16-bit inputs
  float softcap, cap_inv;             // soft cap (0: none) and 1 / cap
  // workspace
  int32_t* count;                     // [0] valid tokens
  int32_t* idx;                       // compact -> token
  int32_t* tgt;                       // compact -> target, -1: out of range
  float* lossc;                       // compact losses
  void* hp;                           // piece x dp panels of the gathered hidden states
  void* e;                            // piece x vp panels: exponentials (times the soft cap's slope), then the logits' gradient
  float* tmax;                        // n_vt x piece: each tile's largest logit of the row, without the target's
  float* tsum;                        // n_vt x piece: sum of its exponentials over that reference, without the target's
  float* zt;                          // piece: the target's logit
  float* zf;                          // piece: the soft cap's slope there (with a soft cap)
  float4* rs;                         // piece: {reference, factor, target's gradient, what its rounding lost}
  float* part;                        // dH partial sums: split x piece x dp
  int32_t split;                      // parts of the vocabulary in dH
  float* wpart;                       // dW partial sums: wsplit x v x dp
  int32_t wsplit;                     // parts of the piece's tokens in dW
  int32_t logit_tile, grad_tile;      // tile edges of the products
  int32_t gather;                     // the logits read the hidden rows themselves
  int32_t rows_direct;                // hidden rows are whole 16-byte pieces within 2 GiB
  float* dwacc;                       // v x dp fp32 sum over pieces, or null: one piece
  int32_t first, last;                // this piece starts / ends the sum over pieces
  float* loss;                        // caller's: one value, or n
  const float* grad_out;              // device, or null (1)
};

// Picks the tile edges, the statistics' columns and the splits, from the sizes
// and from which gradients are wanted (before the workspace is laid out).
void head_plan(HeadArgs& a, int dt);
hipError_t launch_head_compact(const HeadArgs& a, hipStream_t s);
hipError_t launch_head_pack(const HeadArgs& a, int dt, hipStream_t s);
hipError_t launch_head_logits(const HeadArgs& a, int dt, int keep, hipStream_t s);
hipError_t launch_head_merge(const HeadArgs& a, int grad, hipStream_t s);
hipError_t launch_head_dlogits(const HeadArgs& a, int dt, hipStream_t s);
hipError_t launch_head_gradients(const HeadArgs& a, int dt, hipStream_t s);   // dh and dw, each if not null
hipError_t launch_head_gradients_out(const HeadArgs& a, int dt, hipStream_t s);

}  // namespace muon
