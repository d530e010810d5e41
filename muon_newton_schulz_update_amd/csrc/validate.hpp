// Host-only validation helpers shared by the C-ABI entry points.
#pragma once
#include <stdint.h>

#include "../../include/libmuon.h"

namespace muon {

constexpr int kMaxDim = 65536;                 // rows, cols
constexpr int kMaxShort = 16384;               // min(rows, cols)
constexpr int64_t kMaxElems = int64_t(1) << 31;
constexpr int kMaxBatch = 65535;               // matrices per call
constexpr int64_t kMaxLd = int64_t(1) << 40;   // row stride in elements (keeps every offset far from overflow)

int check_config(const muon_config* c, char* msg, int len);
int check_polar(int n, const muon_matrix* in, const muon_matrix* out, const muon_config* cfg, char* msg, int len);
int check_update(int n, const muon_matrix* g, const muon_matrix* m, const muon_matrix* w, const muon_matrix* uo,
                 const muon_config* cfg, char* msg, int len);

// Training-step entry points (train_api.cpp).
constexpr int64_t kMaxListElems = int64_t(1) << 42;   // elements of one tensor of a list
constexpr int kMaxVocab = 1 << 22;
int check_norm(int n, const muon_matrix* g, const muon_matrix* out, float max_norm, const float* norm,
               const float* coef, int writes, char* msg, int len);
int check_scale(int n, const muon_matrix* in, const muon_matrix* out, const float* coef, char* msg, int len);
int check_adamw(int n, const muon_matrix* g, const muon_matrix* m, const muon_matrix* v, const muon_matrix* w,
                const muon_matrix* copy, const muon_adamw_config* cfg, const float* scale, char* msg, int len);
int check_loss(const muon_matrix* hidden, const muon_matrix* weight, const void* targets, int target_bytes,
               const muon_loss_config* cfg, const float* grad_out, const float* loss, const muon_matrix* dhidden,
               const muon_matrix* dweight, int grad, char* msg, int len);

}  // namespace muon
