// Linear attention with a decay for each head: what the entry points (linattn.cu) and
// the tensor-core kernel (linattn_tc.cu) share.
//
// Everything is one pass, run with different operands:
//   out_i = scale * sum_j w(i, j) (a_i . b_j) c_j + (what the state brought in adds),
// w = gamma^{|i - j|} over the tokens j of i's document up to i (forwards) or from i on
// (backwards in time, `rev`), with the state F = sum_j gamma^{..} b_j c_j^T [Da, Dc]:
//   O  : a = q,  b = k,  c = v,  forwards;     F = S
//   gq : a = gO, b = v,  c = k,  forwards;     F = S^T
//   gv : a = k,  b = q,  c = gO, backwards;    F = R = sum gamma^{..} q gO^T
//   gk : a = v,  b = gO, c = q,  backwards;    F = R^T
// Forwards, F after a token is S at that token; row i of a chunk sees the state from
// before the chunk with gamma^{i+1}.  Backwards, F is R at the token last taken; the
// state's gradient enters before the last token without a decay of its own (`rev`
// passes take one factor less in the row's last chunk).
#pragma once

#include <cuda_runtime.h>

#include "common.cuh"

namespace ipttt {
namespace la {

struct Pass {
  const void *a, *b, *c;         // [B*T tokens][heads][width], strides in elements
  long long lda, ldb, ldc;
  int ga, gb, gc;                // head h of the pass reads head h / g of the operand
  void* out;                     // null: the pass leaves only each segment's state (in seg_state)
  long long ldo;
  int out_f32;                   // out is fp32 whatever the operands' type
  const float* init;             // [B][H] states before the first token taken, or null
  int init_t, seg_t;             // init, seg_in are stored transposed ([Dc][Da])
  float init_mul;                // factor on init
  float* fin;                    // [B][H][Da][Dc] state after the last token taken, or null
  int fin_scale;                 // fin gets scale * gamma * F: the gradient of S0 from R
  const float* log_decay;        // [H]
  const uint32_t* starts;        // bit t % 32 of word [b][t / 32]: token t starts a document; null: none
  long long words;               // words of a row
  // [B][H][segs][Da][Dc] (segs > 1): the segments' own states, or (prefixed) the states they start from
  const float* seg_in;
  float* seg_state;              // the same array, written when out is null
  int prefixed;
  int segs, seg_chunks, chunk;   // segments of a row, chunks of each (the last may have fewer), tokens of a chunk
  int after_states;              // the launch before is the pass for this one's segment states
  int fine;                      // the state goes out: formed to fp32's accuracy, see linattn_tc.cu
  int whole;                     // (row, head) pairs b * H + h below this are not cut into segments
  int B, T, H, Da, Dc;
  int rev;
  float scale;
  int* status;
};

// The weight of what a token does not see: another document's, or any past where gamma is 0 (below
// the smallest fp32 number).  It is left out, not multiplied by 0, which would make NaN of a value
// that is not finite; a weight that underflows is 0 and does make NaN of an infinity, which
// the definition keeps.
constexpr float kNone = -1.0f;
__device__ __forceinline__ float decay_pow(float g, int n) { return n <= 0 ? 1.0f : expf(g * (float)n); }

// A power of gamma that a state is multiplied by again and again.  Its rounding to fp32 would be the same
// each time and grow with the tokens remembered (5e-6 of a state at 16k); so what a factor's
// rounding left goes into the next one, and any number of them is off by two roundings.
struct Fade {
  float hi, lo, inv;  // hi + lo is the power, inv = 1 / hi
};
__device__ __forceinline__ Fade fade_of(float g, int n) {
  const double x = exp((double)g * n);
  Fade f;
  f.hi = (float)x;
  f.lo = f.hi > 0.0f ? (float)(x - f.hi) : 0.0f;
  f.inv = f.hi > 1e-30f ? 1.0f / f.hi : 0.0f;  // below it no state remembers two of them
  return f;
}
__device__ __forceinline__ float fade_next(const Fade& f, float& left) {
  const float t = fmaf(f.hi, left, f.lo), x = f.hi + t;
  left = ((f.hi - x) + t) * f.inv;
  return x;
}

// The CUDA-core pass (any widths up to 256, fp32 or bf16 operands), chunks of 32 tokens.
constexpr int kSimtChunk = 32;
cudaError_t run_simt(const Pass& p, int dtype, cudaStream_t st);
int simt_segments(int B, int T, int H, int width, int* seg_chunks);

// The tensor-core pass (bf16 operands, widths of 64 and 128), chunks of 128 tokens.
constexpr int kTcChunk = 128;
bool tc_takes(int Da, int Dc);
cudaError_t run_tc(const Pass& p, cudaStream_t st);
int tc_segments(int B, int T, int H, int* seg_chunks, int* whole);

}  // namespace la
}  // namespace ipttt
