// Softmax cross entropy of a linear head in pieces of the vocabulary
// (ipttt_xent_forward, ipttt_xent_backward).
//
// Mathematics: each row's logits l = H W^T are folded into maxima m and sums s = sum
// exp(l - m) as they are formed, and dropped; lse = m + log s and loss = lse - l[target].
// Backward, by pieces of the vocabulary: the piece's logits again, p = (exp(l - lse) -
// onehot) gloss, then gH += p W_piece and gW_piece = p^T H.
// bf16: tensor-core GEMMs (gemm.cu) whose epilogues do the softmax's part on the
// accumulators: the forward's leaves (m, s) for each 128 columns of a row, the
// backward's writes p in bf16.  Bound by the tensor cores: 2 N V d operations forwards,
// 6 N V d backwards (2 N V d of them to form the logits again).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"
#include "gemm.h"

namespace ipttt {
namespace {

constexpr int kThreads = 256;

// ------------------------------------------------------------------ fp32 products

// out[slice][m][n] = sum over the slice of k of A(m, k) B(k, n), fp32 FMA.  An operand is
// either K-major (A[m * lda + k]) or MN-major (A[k * lda + m]); K-major operands have
// K a multiple of 4, MN-major ones rows readable up to a multiple of 4 columns.
// 64 x 128 tiles of 128 threads, 8 x 8 products a thread (strips of 4 rows and columns, 32 and 64
// apart), 16 k a step, the next step's operands in registers meanwhile.  The 64-row tiles
// waste less of the odd row counts of a small model than 128 would, and give enough
// blocks for four an SM.  300 tokens, 10007 words, d = 512: 84 us for the logits (37 TFLOP/s),
// 71 for gH, 76 for gW; one product an instruction took 87, 80 and 88, 128 x 128 tiles of 256
// threads 111, 132 and 97.
// Up to 16 rows (a batch of a few tokens against the whole vocabulary) take 16-row tiles, 2 x 8
// products a thread: loss and gradients of 16 tokens, 50000 words, d = 1024, 394 us (595 in
// 64-row tiles); 32 tokens 628 us in 64-row tiles (712 in 16-row ones).
constexpr int SM = 64, SN = 128, SK = 16, kGemmThreads = 128;
constexpr int kFewRows = 16;  // at most so many rows take 16-row tiles
struct Sgemm {
  const float *A, *B;
  float* out;
  long long lda, ldb, ldo, osz;
  int M, N, K, slices;
  int a_cols, b_cols;  // MN-major operands: readable columns
  int add;             // add to out
};

// The block's part of an operand for 16 k: WIDTH rows (or columns) from r0 on.
template <bool KMAJOR, int WIDTH> struct Fetch {
  static constexpr int N = (WIDTH * SK / 4 + kGemmThreads - 1) / kGemmThreads;
  static constexpr bool WHOLE = N * kGemmThreads * 4 == WIDTH * SK;  // else threads past the end idle
  float4 v[N];
  __device__ __forceinline__ void load(const float* X, long long ld, int rows, int cols, int k1, int r0, int k0) {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = threadIdx.x + u * kGemmThreads;
      v[u] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (!WHOLE && i >= WIDTH * SK / 4) continue;
      if (KMAJOR) {
        const int r = r0 + i / 4, k = k0 + 4 * (i % 4);
        if (r < rows && k < k1) v[u] = *reinterpret_cast<const float4*>(X + r * ld + k);
      } else {
        const int k = k0 + i / (WIDTH / 4), r = r0 + 4 * (i % (WIDTH / 4));
        if (k < k1 && r < cols) v[u] = *reinterpret_cast<const float4*>(X + k * ld + r);
      }
    }
  }
  __device__ __forceinline__ void place(float (*s)[WIDTH + 4]) const {
#pragma unroll
    for (int u = 0; u < N; ++u) {
      const int i = threadIdx.x + u * kGemmThreads;
      if (!WHOLE && i >= WIDTH * SK / 4) continue;
      if (KMAJOR) {
        const int r = i / 4, k = 4 * (i % 4);
        s[k][r] = v[u].x;
        s[k + 1][r] = v[u].y;
        s[k + 2][r] = v[u].z;
        s[k + 3][r] = v[u].w;
      } else {
        *reinterpret_cast<float4*>(&s[i / (WIDTH / 4)][4 * (i % (WIDTH / 4))]) = v[u];
      }
    }
  }
};

// d += a b on two fp32 numbers at once (each rounded as fmaf).
__device__ __forceinline__ void fma2(unsigned long long& d, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

template <bool AK, bool BK, int TM>
__global__ void __launch_bounds__(kGemmThreads, 4) k_sgemm(const Sgemm g) {
  constexpr int R = TM / 8;  // rows a thread
  __shared__ __align__(16) float as[2][SK][TM + 4], bs[2][SK][SN + 4];
  const int nt = (g.N + SN - 1) / SN;
  const int m0 = blockIdx.x / nt * TM, n0 = blockIdx.x % nt * SN;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;  // 16 x 8 threads
  const int blocks = (g.K + SK - 1) / SK;
  const int kb0 = (int)((long long)blocks * blockIdx.z / g.slices), kb1 = (int)((long long)blocks * (blockIdx.z + 1) / g.slices);
  unsigned long long pair[R][4] = {};  // products of two columns each
  Fetch<AK, TM> av;
  Fetch<BK, SN> bv;
  if (kb0 < kb1) {
    av.load(g.A, g.lda, g.M, g.a_cols, g.K, m0, kb0 * SK);
    bv.load(g.B, g.ldb, g.N, g.b_cols, g.K, n0, kb0 * SK);
    av.place(as[0]);
    bv.place(bs[0]);
  }
  __syncthreads();
  for (int kb = kb0; kb < kb1; ++kb) {
    const int cur = (kb - kb0) & 1;
    const bool more = kb + 1 < kb1;
    if (more) {
      av.load(g.A, g.lda, g.M, g.a_cols, g.K, m0, (kb + 1) * SK);
      bv.load(g.B, g.ldb, g.N, g.b_cols, g.K, n0, (kb + 1) * SK);
    }
#pragma unroll
    for (int k = 0; k < SK; ++k) {
      float x[R];
      if constexpr (R == 8) {
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(&as[cur][k][4 * ty]);
        *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(&as[cur][k][32 + 4 * ty]);
      } else {
        *reinterpret_cast<float2*>(x) = *reinterpret_cast<const float2*>(&as[cur][k][2 * ty]);
      }
      const ulonglong2 y0 = *reinterpret_cast<const ulonglong2*>(&bs[cur][k][4 * tx]);
      const ulonglong2 y1 = *reinterpret_cast<const ulonglong2*>(&bs[cur][k][64 + 4 * tx]);
#pragma unroll
      for (int i = 0; i < R; ++i) {
        unsigned long long xx;
        asm("mov.b64 %0, {%1, %1};" : "=l"(xx) : "f"(x[i]));
        fma2(pair[i][0], xx, y0.x);
        fma2(pair[i][1], xx, y0.y);
        fma2(pair[i][2], xx, y1.x);
        fma2(pair[i][3], xx, y1.y);
      }
    }
    if (more) {
      av.place(as[cur ^ 1]);
      bv.place(bs[cur ^ 1]);
    }
    __syncthreads();
  }
  float acc[R][8];
#pragma unroll
  for (int i = 0; i < R; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      asm("mov.b64 {%0, %1}, %2;" : "=f"(acc[i][2 * j]), "=f"(acc[i][2 * j + 1]) : "l"(pair[i][j]));
  float* out = g.out + blockIdx.z * g.osz;
#pragma unroll
  for (int i = 0; i < R; ++i) {
    const int m = m0 + (R == 8 ? (i / 4) * 32 + 4 * ty + i % 4 : 2 * ty + i);
    if (m >= g.M) continue;
#pragma unroll
    for (int j = 0; j < 8; j += 4) {
      const int n = n0 + (j / 4) * 64 + 4 * tx;
      float* o = out + m * g.ldo + n;
      if (n + 4 <= g.N) {  // rows are a multiple of 4 apart
        float4 v = make_float4(acc[i][j], acc[i][j + 1], acc[i][j + 2], acc[i][j + 3]);
        if (g.add) {
          const float4 w = *reinterpret_cast<const float4*>(o);
          v = make_float4(w.x + v.x, w.y + v.y, w.z + v.z, w.w + v.w);
        }
        *reinterpret_cast<float4*>(o) = v;
      } else {
        for (int e = 0; e < 4 && n + e < g.N; ++e) o[e] = g.add ? o[e] + acc[i][j + e] : acc[i][j + e];
      }
    }
  }
}

template <bool AK, bool BK>
cudaError_t sgemm(const Sgemm& g, cudaStream_t st) {
  const int tm = g.M <= kFewRows ? 16 : SM;
  const long long tiles = (long long)((g.N + SN - 1) / SN) * ((g.M + tm - 1) / tm);
  if (tiles > 0x7fffffffLL) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)tiles, 1, g.slices);
  if (tm == 16) k_sgemm<AK, BK, 16><<<grid, kGemmThreads, 0, st>>>(g);
  else k_sgemm<AK, BK, SM><<<grid, kGemmThreads, 0, st>>>(g);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ the rows' statistics and gradients

// (maximum, sum) of two sets of logits.  fmaxf leaves NaN out, the sums do not: a NaN as a set's maximum or
// sum makes the sum NaN.  At its own maximum a sum stays as it is (an infinity minus itself is
// NaN): a logit of infinity gives an infinite lse, logits of -infinity alone one of -infinity.
__device__ __forceinline__ float2 merge(float2 a, float2 b) {
  const float m = fmaxf(a.x, b.x);
  return make_float2(m, (a.x == m ? a.y : a.y * expf(a.x - m)) + (b.x == m ? b.y : b.y * expf(b.x - m)));
}

__device__ __forceinline__ float2 block_merge(float2 v, float2* sh) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = merge(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = v;
  __syncthreads();
  v = sh[0];
  for (int i = 1; i < kThreads / 32; ++i) v = merge(v, sh[i]);
  return v;
}

// A row's lse, and its loss where it takes part.
__device__ __forceinline__ void finish_row(int n, float2 v, float target_logit, int V, const int64_t* targets, int64_t ignore,
                                           float* loss, float* lse, int* status) {
  const int64_t t = targets[n];
  const float s = v.x + logf(v.y);
  lse[n] = s;
  const bool out = t < 0 || t >= V;
  if (out && t != ignore) set_status(status, IPTTT_ERR_ARG);
  loss[n] = out || t == ignore ? 0.0f : s - target_logit;
}

// fp32: one block a row: the piece's logits into the row's running maximum and sum, and its
// target's logit.  The last piece writes lse and loss.
__global__ void __launch_bounds__(kThreads) k_row_stats(const float* l, long long ld, int v0, int cols, int V, int last,
                                                      const int64_t* targets, int64_t ignore, float2* run, float* tl,
                                                      float* loss, float* lse, int* status) {
  __shared__ float2 sh[kThreads / 32];
  const int n = blockIdx.x;
  const float* x = l + (long long)n * ld;
  float2 v = make_float2(-INFINITY, 0.0f);
  for (int i = threadIdx.x; i < cols; i += kThreads) v = merge(v, make_float2(x[i], 1.0f));
  v = block_merge(v, sh);
  if (threadIdx.x != 0) return;
  if (v0 > 0) v = merge(run[n], v);
  run[n] = v;
  const int64_t t = targets[n];
  if (t >= v0 && t < v0 + cols) tl[n] = x[t - v0];
  if (last) finish_row(n, v, tl[n], V, targets, ignore, loss, lse, status);
}

// bf16: the GEMM's (maximum, sum) of every 128 columns, part[parts][N], into lse and loss.
// 8 rows a block, 32 threads a row.
__global__ void __launch_bounds__(kThreads) k_row_join(const float2* part, int parts, int N, int V, const int64_t* targets,
                                                     int64_t ignore, const float* tl, float* loss, float* lse,
                                                     int* status) {
  __shared__ float2 sh[8][33];
  const int r = threadIdx.x % 8, k = threadIdx.x / 8, n = blockIdx.x * 8 + r;
  float2 v = make_float2(-INFINITY, 0.0f);
  if (n < N)
    for (int i = k; i < parts; i += 32) v = merge(v, part[(long long)i * N + n]);
  sh[r][k] = v;
  __syncthreads();
  // warp w joins row w
  const int row = threadIdx.x / 32, at = blockIdx.x * 8 + row;
  v = sh[row][threadIdx.x % 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
    v = merge(v, make_float2(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  if (threadIdx.x % 32 == 0 && at < N) finish_row(at, v, tl[at], V, targets, ignore, loss, lse, status);
}

// bf16: p is formed with gloss divided by its largest magnitude, unit[0], which goes onto the
// products' fp32 results instead.  For a mean every row's gloss is the same, and the target's p
// - 1, nearly -1, is then as good as exact, where -gloss would be off by the same rounding in
// every row.  Also reports targets that are neither in the vocabulary nor the one to leave out.
// One block.
__global__ void __launch_bounds__(1024) k_unit(const int64_t* targets, const float* gloss, int N, int V, int64_t ignore,
                                               float* unit, int* status) {
  __shared__ float sh[32];
  float top = 0.0f;
  for (int n = threadIdx.x; n < N; n += 1024) {
    const int64_t t = targets[n];
    if (t == ignore) continue;
    if (t < 0 || t >= V) set_status(status, IPTTT_ERR_ARG);
    else top = fmaxf(top, fabsf(gloss[n]));
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if (threadIdx.x % 32 == 0) sh[threadIdx.x / 32] = top;
  __syncthreads();
  if (threadIdx.x < 32) {
    top = sh[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    // no gradient at all, or one that is not finite, is left as it is
    if (threadIdx.x == 0) unit[0] = top > 0.0f && top < INFINITY ? top : 1.0f;
  }
}

// fp32: p = (exp(l - lse) - onehot) gloss for the piece's columns; 0 in the padding.
__global__ void __launch_bounds__(kThreads) k_row_grad(float* l, long long ld, int v0, int cols, int padded, int V,
                                                     const int64_t* targets, int64_t ignore, const float* lse,
                                                     const float* gloss, int* status) {
  const int n = blockIdx.x;
  const int64_t t = targets[n];
  const bool out = t < 0 || t >= V;
  if (out && t != ignore && threadIdx.x == 0) set_status(status, IPTTT_ERR_ARG);
  const bool on = !out && t != ignore;
  const float s = lse[n], g = on ? gloss[n] : 0.0f;
  for (int i = threadIdx.x; i < padded; i += kThreads) {
    float v = 0.0f;
    if (on && i < cols) v = (expf(l[(long long)n * ld + i] - s) - (t - v0 == i ? 1.0f : 0.0f)) * g;
    l[(long long)n * ld + i] = v;
  }
}

// H with zeros in the rows that take no part, for gW = p^T H alone: p is 0 there, but 0 times
// a value that is not finite (padding that was never written) would reach every row of gW.
// Rows of `units` 16-byte units.  8192 rows of 2560 bf16: 84 MB moved beside the 200 times
// that the products take.
__global__ void __launch_bounds__(kThreads) k_live_rows(const uint4* H, uint4* out, long long n, int units, int V,
                                                      const int64_t* targets, int64_t ignore) {
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads) {
    const int64_t t = targets[i / units];
    out[i] = t != ignore && t >= 0 && t < V ? H[i] : make_uint4(0u, 0u, 0u, 0u);
  }
}

// gH (in T) = the sum of the fp32 slices, in slice order, times *unit (null: 1).  Rows that take no part
// get 0 whatever W holds: p is 0 there, and 0 times a word that is not finite NaN, so a sum that is
// not finite asks for its row's target (asking always: 353 -> 357 us for 300 tokens in fp32).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_sum_slices(const float* part, T* out, long long n, int slices, const float* unit,
                                                       int d, int V, const int64_t* targets, int64_t ignore) {
  const float f = unit ? *unit : 1.0f;
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads) {
    float s = part[i];
    for (int q = 1; q < slices; ++q) s += part[q * n + i];
    if (!isfinite(s)) {
      const int64_t t = targets[i / d];
      if (t == ignore || t < 0 || t >= V) s = 0.0f;
    }
    out[i] = from_f<T>(s * f);
  }
}

// ------------------------------------------------------------------ sizes

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

// Of a piece's p (fp32: of its logits, p in their place).  128 to 512 MB are within 1% at 8192 tokens of
// 65536 words; more tokens make a piece fewer words (131072: 1024), whose gW product has fewer tiles than
// SMs and whose gH is added up more often: not measured there, `piece` may say otherwise.
constexpr size_t kPieceBytes = size_t(256) << 20;

ipttt_status check(const ipttt_xent_params* p) {
  if (!p) return IPTTT_ERR_ARG;
  if (p->dtype != IPTTT_F32 && p->dtype != IPTTT_BF16) return IPTTT_ERR_DTYPE;
  if (p->N <= 0 || p->V <= 0 || p->d <= 0 || p->piece < 0 || p->piece % 256 != 0) return IPTTT_ERR_ARG;
  if (p->d % (p->dtype == IPTTT_BF16 ? 32 : 4) != 0) return IPTTT_ERR_UNSUPPORTED;
  if (p->N > (1 << 24) || p->V > (1 << 26) || p->d > (1 << 16)) return IPTTT_ERR_SHAPE;
  return IPTTT_OK;
}

struct Work {
  int piece;  // vocabulary rows at a time, a multiple of 256
  int slices; // partial sums of gH: slices of a piece's columns
  size_t p, part, tl, gH, unit, live, total;  // p: fp32 logits and p, or bf16 p; live: H's rows that take part
};

Work work_of(const ipttt_xent_params& p, bool backward) {
  Work w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  const long long all = ((long long)p.V + 255) / 256 * 256;
  const bool tc = p.dtype == IPTTT_BF16;
  const long long row = (long long)p.N * (tc ? 2 : 4);
  w.piece = p.piece ? p.piece : (int)std::max<long long>(256, std::min<long long>(all, kPieceBytes / row / 256 * 256));
  w.piece = (int)std::min<long long>(w.piece, all);
  if (!(tc && !backward)) w.p = take(row * w.piece);
  if (!backward) {
    w.part = take((size_t)p.N * sizeof(float2) * (tc ? all / 128 : 1));
    w.tl = take((size_t)p.N * 4);
  } else {
    // slices of K for gH's product, each of at least 256 columns: in bf16 enough to fill the SMs
    // twice, in fp32 the number that comes out fastest by the busiest SM's blocks (fewer than four
    // leave its pipe idle for part of the time) and the sum of the slices (one takes 50 /
    // piece of the product's time).  1000 tokens of 2560, 8000 words: 801 us in 6 slices, 1215 in
    // one; 300 of 512, 10007: 74 in 29 (580 blocks), 105 in 7 (140).
    const int rows = tc ? 128 : p.N <= kFewRows ? 16 : SM;
    const long long tiles = (long long)((p.N + rows - 1) / rows) * ((p.d + 127) / 128);
    const int most = std::max(1, std::min(w.piece / 256, 32));
    w.slices = tc ? (int)std::max<long long>(1, std::min<long long>(296 / tiles, most)) : 1;
    double best = 0.0;
    for (int s = 1; !tc && s <= most; ++s) {
      const long long busiest = (tiles * s + 147) / 148;
      const double pace = busiest >= 4 ? 1.0 : 0.2 + 0.2 * (double)busiest;
      const double time = (double)busiest * 148 / (pace * (double)(tiles * s)) + 50.0 * s / w.piece;
      if (s > 1 && time >= best) continue;
      best = time;
      w.slices = s;
    }
    w.gH = take((size_t)p.N * p.d * 4 * w.slices);
    w.unit = take(4);
    w.live = take((size_t)p.N * p.d * (tc ? 2 : 4));
  }
  w.total = off;
  return w;
}

// The logits of vocabulary rows [v0, v0 + cols), fp32.
cudaError_t logits_of(const ipttt_xent_params& p, const void* H, const void* W, int v0, int cols, float* out, long long ld,
                      cudaStream_t st) {
  Sgemm g{static_cast<const float*>(H), static_cast<const float*>(W) + (long long)v0 * p.d, out, p.d, p.d, ld, 0,
          p.N, cols, p.d, 1, 0, 0, 0};
  return sgemm<true, true>(g, st);
}

// H W^T over vocabulary rows [v0, v0 + cols), bf16, with a softmax epilogue.
gemm::Args logits_args(const ipttt_xent_params& p, const void* H, const void* W, const int64_t* targets, int v0, int cols) {
  gemm::Args a{};
  a.A = {H, (uint64_t)p.d, (uint64_t)p.N, 1};
  a.Bop = {static_cast<const __nv_bfloat16*>(W) + (long long)v0 * p.d, (uint64_t)p.d, (uint64_t)cols, 1};
  a.mode = gemm::GM_PLAIN;
  a.M = p.N;
  a.N = (cols + 31) / 32 * 32;
  a.K = p.d;
  a.softmax.targets = targets;
  a.softmax.ignore = p.ignore_index;
  a.softmax.V = p.V;
  a.softmax.v0 = v0;
  a.softmax.cols = cols;
  a.status = device_status();
  return a;
}

bool aligned(std::initializer_list<const void*> ps, unsigned bytes) {
  uintptr_t any = 0;
  for (const void* q : ps) any |= reinterpret_cast<uintptr_t>(q);
  return any % bytes == 0;
}

cudaError_t forward(const ipttt_xent_params& p, const Work& w, const void* H, const void* W, const int64_t* targets,
                    float* loss, float* lse, uint8_t* ws, int* launches, cudaStream_t st) {
  float2* part = reinterpret_cast<float2*>(ws + w.part);
  float* tl = reinterpret_cast<float*>(ws + w.tl);
  if (p.dtype == IPTTT_BF16) {
    gemm::Args a = logits_args(p, H, W, targets, 0, p.V);
    a.out_kind = gemm::GO_ROW_STATS;
    a.softmax.part = part;
    a.softmax.target_logit = tl;
    const cudaError_t e = gemm::run(a, device_sms(), st);
    if (e != cudaSuccess) return e;
    k_row_join<<<(p.N + 7) / 8, kThreads, 0, st>>>(part, (p.V + 127) / 128, p.N, p.V, targets, p.ignore_index, tl, loss,
                                                     lse, device_status());
    *launches += 2;
    return cudaGetLastError();
  }
  float* l = reinterpret_cast<float*>(ws + w.p);
  for (int v0 = 0; v0 < p.V; v0 += w.piece) {
    const int cols = std::min(w.piece, p.V - v0);
    const cudaError_t e = logits_of(p, H, W, v0, cols, l, w.piece, st);
    if (e != cudaSuccess) return e;
    k_row_stats<<<p.N, kThreads, 0, st>>>(l, w.piece, v0, cols, p.V, v0 + cols == p.V, targets, p.ignore_index,
                                          part, tl, loss, lse, device_status());
    *launches += 2;
  }
  return cudaGetLastError();
}

cudaError_t backward(const ipttt_xent_params& p, const Work& w, const void* H, const void* W, const int64_t* targets,
                     const float* lse, const float* gloss, void* gH, void* gW, uint8_t* ws, int* launches,
                     cudaStream_t st) {
  float* acc = reinterpret_cast<float*>(ws + w.gH);
  const long long nd = (long long)p.N * p.d;
  const bool tc = p.dtype == IPTTT_BF16;
  float* unit = reinterpret_cast<float*>(ws + w.unit);
  if (tc) {
    k_unit<<<1, 1024, 0, st>>>(targets, gloss, p.N, p.V, p.ignore_index, unit, device_status());
    ++*launches;
  }
  void* live = ws + w.live;
  const int units = p.d * (tc ? 2 : 4) / 16;
  const long long all_units = (long long)p.N * units;
  k_live_rows<<<(unsigned)std::min<long long>((all_units + kThreads - 1) / kThreads, 148 * 16), kThreads, 0, st>>>(
      static_cast<const uint4*>(H), static_cast<uint4*>(live), all_units, units, p.V, targets, p.ignore_index);
  ++*launches;
  int all_slices = 0;
  for (int v0 = 0; v0 < p.V; v0 += w.piece) {
    const int cols = std::min(w.piece, p.V - v0);
    const int slices = std::max(1, std::min(w.slices, cols / 256));
    if (v0 == 0) all_slices = slices;  // a shorter last piece adds to the first ones
    cudaError_t e;
    if (!tc) {
      float* l = reinterpret_cast<float*>(ws + w.p);
      const float* Wf = static_cast<const float*>(W) + (long long)v0 * p.d;
      e = logits_of(p, H, W, v0, cols, l, w.piece, st);
      if (e != cudaSuccess) return e;
      k_row_grad<<<p.N, kThreads, 0, st>>>(l, w.piece, v0, cols, w.piece, p.V, targets, p.ignore_index, lse, gloss,
                                           device_status());
      // p's columns past the vocabulary are zero, and W's rows past it are not read
      Sgemm a{l, Wf, acc, w.piece, p.d, p.d, nd, p.N, p.d, cols, slices, 0, p.d, v0 > 0};
      e = sgemm<true, false>(a, st);
      if (e != cudaSuccess) return e;
      Sgemm b{l, static_cast<const float*>(live), static_cast<float*>(gW) + (long long)v0 * p.d, w.piece, p.d, p.d, 0,
              cols, p.d, p.N, 1, w.piece, p.d, 0};
      e = sgemm<false, false>(b, st);
      if (e != cudaSuccess) return e;
      *launches += 4;
      continue;
    }
    __nv_bfloat16* pb = reinterpret_cast<__nv_bfloat16*>(ws + w.p);
    gemm::Args l = logits_args(p, H, W, targets, v0, cols);
    l.out_kind = gemm::GO_ROW_GRAD;
    l.out = pb;
    l.ldo = w.piece;
    l.softmax.lse = lse;
    l.softmax.gloss = gloss;
    l.softmax.unit = unit;
    e = gemm::run(l, device_sms(), st);
    if (e != cudaSuccess) return e;
    gemm::Args a{};
    a.A = {pb, (uint64_t)cols, (uint64_t)p.N, 1, (uint64_t)w.piece};
    a.Bop = {static_cast<const __nv_bfloat16*>(W) + (long long)v0 * p.d, (uint64_t)p.d, (uint64_t)cols, 1};
    a.b_mn = 1;
    a.mode = gemm::GM_PLAIN;
    a.M = p.N;
    a.N = p.d;
    a.K = cols;
    a.out_kind = v0 > 0 ? gemm::GO_F32_ADD : gemm::GO_F32;
    a.out = acc;
    a.ldo = p.d;
    a.osz = nd;
    a.ksplit = slices;
    a.status = device_status();
    e = gemm::run(a, device_sms(), st);
    if (e != cudaSuccess) return e;
    gemm::Args b{};
    b.A = {pb, (uint64_t)cols, (uint64_t)p.N, 1, (uint64_t)w.piece};
    b.a_mn = 1;
    b.Bop = {live, (uint64_t)p.d, (uint64_t)p.N, 1};
    b.b_mn = 1;
    b.mode = gemm::GM_PLAIN;
    b.M = cols;
    b.N = p.d;
    b.K = p.N;
    b.out_kind = gemm::GO_BF16;
    b.scale = unit;
    b.out = static_cast<__nv_bfloat16*>(gW) + (long long)v0 * p.d;
    b.ldo = p.d;
    b.status = device_status();
    e = gemm::run(b, device_sms(), st);
    if (e != cudaSuccess) return e;
    *launches += 3;
  }
  const unsigned grid = (unsigned)std::min<long long>((nd + kThreads - 1) / kThreads, 148 * 16);
  if (tc)
    k_sum_slices<<<grid, kThreads, 0, st>>>(acc, static_cast<__nv_bfloat16*>(gH), nd, all_slices, unit, p.d, p.V, targets,
                                              p.ignore_index);
  else
    k_sum_slices<<<grid, kThreads, 0, st>>>(acc, static_cast<float*>(gH), nd, all_slices, static_cast<const float*>(nullptr), p.d,
                                              p.V, targets, p.ignore_index);
  ++*launches;
  return cudaGetLastError();
}

}  // namespace
}  // namespace ipttt

using namespace ipttt;

extern "C" {

size_t ipttt_xent_workspace_size(const ipttt_xent_params* p) {
  return check(p) == IPTTT_OK ? work_of(*p, false).total : 0;
}

size_t ipttt_xent_backward_workspace_size(const ipttt_xent_params* p) {
  return check(p) == IPTTT_OK ? work_of(*p, true).total : 0;
}

ipttt_status ipttt_xent_forward(const ipttt_xent_params* p, const void* H, const void* W, const int64_t* targets,
                                float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  const ipttt_status rc = check(p);
  if (rc != IPTTT_OK) return rc;
  if (!H || !W || !targets || !loss || !lse) return IPTTT_ERR_ARG;
  if (shared_pointer({loss, lse, workspace}, {H, W, targets})) return IPTTT_ERR_ARG;
  if (!aligned({H, W}, 16) || !aligned({targets}, 8) || !aligned({loss, lse}, 4)) return IPTTT_ERR_ALIGN;
  const Work w = work_of(*p, false);
  if (!workspace || workspace_bytes < w.total) return IPTTT_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return IPTTT_ERR_ALIGN;
  int launches = 0;
  const cudaError_t e = forward(*p, w, H, W, targets, loss, lse, static_cast<uint8_t*>(workspace), &launches,
                                static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail("xent_forward", e);
  count_launches(launches);
  return IPTTT_OK;
}

ipttt_status ipttt_xent_backward(const ipttt_xent_params* p, const void* H, const void* W, const int64_t* targets,
                                 const float* lse, const float* gloss, void* gH, void* gW, void* workspace,
                                 size_t workspace_bytes, void* stream) {
  const ipttt_status rc = check(p);
  if (rc != IPTTT_OK) return rc;
  if (!H || !W || !targets || !lse || !gloss || !gH || !gW) return IPTTT_ERR_ARG;
  if (shared_pointer({gH, gW, workspace}, {H, W, targets, lse, gloss})) return IPTTT_ERR_ARG;
  if (!aligned({H, W, gH, gW}, 16) || !aligned({targets}, 8) || !aligned({lse, gloss}, 4)) return IPTTT_ERR_ALIGN;
  const Work w = work_of(*p, true);
  if (!workspace || workspace_bytes < w.total) return IPTTT_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return IPTTT_ERR_ALIGN;
  int launches = 0;
  const cudaError_t e = backward(*p, w, H, W, targets, lse, gloss, gH, gW, static_cast<uint8_t*>(workspace), &launches,
                                 static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail("xent_backward", e);
  count_launches(launches);
  return IPTTT_OK;
}

}  // extern "C"
