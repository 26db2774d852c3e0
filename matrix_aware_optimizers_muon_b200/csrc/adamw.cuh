// AdamW over lists of tensors (fp32 or 8-bit moments), the conversion of the
// moments, and clipping by the global gradient norm: launch tables shared by
// the entry points (adamw_api.cu) and the kernels (adamw.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace mo {

constexpr int AW_BLOCK = 256;      // elements that share a scale of the 8-bit moments
constexpr int AW_THREADS = 32;     // a CTA is one warp, which works on one block at a time
constexpr int AW_RUN = 8;          // most blocks of a run (fp32 moments: AW_RUN32)
constexpr int AW_RUN32 = 2;
constexpr int AW_MAX = 350;        // tensors per launch (the table travels in the kernel's parameters)
constexpr int AW_SHORT = 96;       // tensors that a launch with fewer parameters takes

enum AwType : unsigned char { AW_F32 = 0, AW_BF16 = 1, AW_F16 = 2, AW_NONE = 3 };

// One tensor.  All tensors of a table have the types of the first, and either
// all of them or none have vec 2.  Which pointers are used depends on the kernel:
//   adamw    W, G, M, V (fp32), C (optional low-precision copy of W)
//   adamw8   W, G, M, V (codes), MS, VS (scales), C
//   pack     G = first moment, C = second moment (read), M, V, MS, VS (written)
//   unpack   M, V, MS, VS (read), W = first moment, C = second moment (written)
//   norm     G;  scale: G, C = output
struct AwTensor {
  void* W;
  const void* G;
  void* M;
  void* V;
  void* C;
  unsigned char* MS;
  unsigned char* VS;
  long long numel;
  float lr_scale, wd;
  unsigned index;                  // place in the caller's list (noise stream)
  unsigned first;                  // its first run among those of the table
  AwType wt, gt, ct;
  unsigned char vec;               // 2: every pointer is aligned to 8 elements, 1: the 8-bit codes are
};

template <int N>
struct AwTableOf {
  int n;
  int run;                         // blocks of a run, the work that a CTA takes at a time
  unsigned runs;
  AwTensor t[N];
};
using AwTable = AwTableOf<AW_MAX>;

struct AwHyper {
  float b1, c1, b2, c2;            // beta, 1 - beta
  float eps;
  float lr, rate, root;            // lr, lr / (1 - b1^t), 1 / sqrt(1 - b2^t) of a step given by the host
  float log_b1, log_b2;            // for a step read on the device
  int bias, stochastic;
  int first;                       // 8-bit moments: the first is rounded stochastically too
  unsigned least_scale;            // scale byte from which on betas times the scale are normal numbers
  unsigned long long seed;
  long long step;
  const float* lr_dev;
  const long long* step_dev;
  const float* gscale;
  const int* skip;
};

struct ClipArgs {
  double* partial;                 // one sum of squares per CTA
  int parts;                       // number of partial sums
  int finish_here;                 // the scale launch sums them itself
  float max_norm;
  const float* scale;              // optional factor of the gradients
  float* norm;
  float* factor;
  int* nonfinite;                  // optional
};

constexpr int CLIP_MAX_CTAS = 8192;   // partial sums of one call
constexpr int FEW_PARTS = 512;        // partial sums that one warp takes
constexpr int FINISH_THREADS = 256;

// Blocks of a run, at most `most`, for a list of so many blocks on `sms` SMs: twice
// as long while that leaves half of `warps` runs for each SM.
// Steps and moments: 64 (see run_of).  Gradients, whose kernels take four blocks at
// a time and where few runs mean few partial sums: 2 (65 tensors of 4096: 5.0 us
// captured and 13.0 with the host; with 64 6.2 and 15.0).
constexpr int STEP_RUNS = 64, GRAD_RUNS = 2;
int run_of(long long blocks, int most, int warps, int sms);
cudaError_t launch_adamw(const AwTable& t, const AwHyper& h, cudaStream_t s);
cudaError_t launch_adamw8(const AwTable& t, const AwHyper& h, cudaStream_t s);
cudaError_t launch_pack(const AwTable& t, const AwHyper& h, cudaStream_t s);
cudaError_t launch_unpack(const AwTable& t, cudaStream_t s);
// CTAs of the norm launch (its number of partial sums), at most `most`
int clip_norm_ctas(const AwTable& t, int most);
cudaError_t launch_clip_norm(const AwTable& t, double* partial, int ctas, cudaStream_t s);
cudaError_t launch_clip_finish(const ClipArgs& a, cudaStream_t s);
cudaError_t launch_clip_scale(const AwTable& t, const ClipArgs& a, cudaStream_t s);

}  // namespace mo
