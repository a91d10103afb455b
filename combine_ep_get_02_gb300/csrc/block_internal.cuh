// Internal declarations of the norm in front of the router, of activations kept in 8 bits,
// and of the experts' layer of a few tokens.
#pragma once

#include "moe_internal.cuh"

namespace ep {

// ---- norm -----------------------------------------------------------------------

constexpr int kNormMaxHidden = 16384;
constexpr float kNormMinEps = 1e-20f, kNormMaxEps = 1e38f;  // the largest mean of squares, 2^125, and eps stay in fp32

struct NormArgs {
  const void* x;            // [rows][H] bf16 or fp32
  const void* residual;     // the same, or null
  const uint16_t* weight;   // [H] or null (ones)
  void* sum;                // x + residual, or null
  uint16_t* y;              // [rows][H] or null
  uint8_t* codes;           // [rows][H] or null
  float* sf;                // [rows][G], or words of packed bytes
  int64_t rows;
  int H, sf_pack;
  float eps;
};

struct NormGradArgs {
  const void* sum;
  const uint16_t* weight;
  const uint8_t* mask;      // [rows] or null
  const uint16_t* d_y;
  const void* d_sum;        // gradient that arrives at the sum itself, or null
  void* d_x;                // may be null
  float* d_weight;          // may be null
  float* part;              // workspace [CTAs][H]
  uint32_t* err;
  int64_t rows;
  int H;
  float eps;
};

// CTAs of a gradient's launch at most, and with it partial sums of d_weight in the workspace
constexpr int kNormGradCtas = 608;

cudaError_t launch_norm(const NormArgs& a, int x_fp32, int num_sms, cudaStream_t stream);
cudaError_t launch_norm_grad(const NormGradArgs& a, int x_fp32, int num_sms, cudaStream_t stream);

// ---- rows kept in 8 bits ------------------------------------------------------------

struct CheckpointArgs {
  Groups groups;
  int F, sf_pack;
  const void* in;   // bf16 rows, or codes
  void* out;        // codes, or bf16 rows
  float* sf;
  uint32_t* err;
};

struct CheckpointGradArgs {
  Groups groups;
  int N, Z, act, sf_pack;
  const uint8_t* codes;
  const float* sf;
  const uint16_t* d_h;
  uint16_t* h;      // may be null
  uint16_t* d_z;    // may be null
  float* part;      // workspace; null without d_bias
  uint32_t* done;
  float* d_bias;    // may be null
  uint32_t* err;
};

cudaError_t launch_checkpoint(const CheckpointArgs& a, bool back, int num_sms, cudaStream_t stream);
cudaError_t launch_checkpoint_grad(const CheckpointGradArgs& a, int num_sms, cudaStream_t stream);

// ---- the experts' layer of a few tokens -----------------------------------------------

constexpr int kLayerMaxTokens = 64;
// Up to as many tokens h is kept as the sum of two bf16: the 8 columns of a product then have room for both terms.
constexpr int kLayerPairTokens = 4;
constexpr int kLayerMaxSplit = 8;  // parts that an output tile's sum over experts is taken in at most

struct LayerArgs {
  const uint16_t* x;          // [T][H]
  const int64_t* idx;         // [T][K]
  const float* w;             // [T][K]
  const void* up;             // [E][Z][H] bf16 or codes
  const float* up_sf;         // [E][ceil(Z / 128)][H / 128] or null
  const uint16_t* up_bias;    // [E][Z] or null
  const void* down;           // [E][H][I]
  const float* down_sf;       // [E][H / 128][I / 128] or null
  const uint16_t* down_bias;  // [E][H] or null
  const uint16_t* residual;   // [T][H] or null
  uint16_t* out;              // [T][H]
  uint16_t* h;                // workspace [lanes][I], up to kLayerPairTokens tokens [2][lanes][I]
  float* part;                // workspace [kLayerMaxSplit][T][H]
  uint32_t* done;             // workspace [H / 16]: parts of a tile that are there (the first kernel zeroes them)
  uint32_t* err;
  int T, E, K, H, I, Z, act;
  int device_sms;
};

cudaError_t launch_layer(const LayerArgs& a, bool fp8, int num_sms, cudaStream_t stream);

}  // namespace ep
