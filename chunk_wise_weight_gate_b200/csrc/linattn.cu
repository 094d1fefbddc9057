// Linear attention with a decay for each head: entry points, the pass on the CUDA
// cores (fp32, and widths that the tensor-core pass does not take), the single-token
// step, and the sum of a shared head's gradients.  linattn.h has the mathematics.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>
#include <atomic>

#include "linattn.h"
#include "tc.cuh"

namespace ipttt {
namespace la {

namespace {

constexpr int kThreads = 256;
constexpr int kMaxWidth = 256;
constexpr int kMaxSegs = 148;      // segments of a row
// The tensor-core pass sums up to so many segments' states itself, which saves a launch (full clocks):
// 2 rows of 20 heads of 128 x 8192 tokens 118 us (136 by k_prefix), 20 heads of 32768 tokens, 7
// segments, 198 (206; under load 227 to 240).  Above it k_prefix does: 10 heads of 32768 tokens 124 us (134 summed by
// every segment), 2 heads 55 (102), 2 heads of 131072 tokens 109 (169).
constexpr int kDirectStates = 8;
constexpr long long kSmemSm = 233472;  // shared memory of an SM
constexpr int L = kSimtChunk;
constexpr int kSlice = 64;  // columns of the state a block holds
constexpr int kSp = L + 4;  // row stride of a chunk's products

__device__ __forceinline__ float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  const float2 a = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.x));
  const float2 b = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v.y));
  return make_float4(a.x, a.y, b.x, b.y);
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(v.x, v.y), b = __floats2bfloat162_rn(v.z, v.w);
  uint2 u;
  u.x = *reinterpret_cast<const uint32_t*>(&a);
  u.y = *reinterpret_cast<const uint32_t*>(&b);
  *reinterpret_cast<uint2*>(p) = u;
}
__device__ __forceinline__ void fma4(float4& acc, float s, float4 v) {
  acc.x = fmaf(s, v.x, acc.x);
  acc.y = fmaf(s, v.y, acc.y);
  acc.z = fmaf(s, v.z, acc.z);
  acc.w = fmaf(s, v.w, acc.w);
}
__device__ __forceinline__ bool finite4(float4 v) { return isfinite(v.x) && isfinite(v.y) && isfinite(v.z) && isfinite(v.w); }
__device__ __forceinline__ float4 scale4(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }

// ------------------------------------------------------------------ document starts

// The start bits of 32 tokens a thread, from the sorted list of offsets b*T + t: the first start at
// or after its tokens by search, then those before their end.  (One kernel, where
// clearing the words and marking every start takes two.)  Every entry is checked by some thread.
__global__ void k_mark(uint32_t* words, long long wpr, int B, int T, const int32_t* ds, int n, int* status) {
  const long long i = blockIdx.x * (long long)blockDim.x + threadIdx.x;
  for (long long k = i; k < n; k += (long long)gridDim.x * blockDim.x)
    if (ds[k] < 0 || ds[k] >= (long long)B * T || (k > 0 && ds[k - 1] >= ds[k])) set_status(status, IPTTT_ERR_ARG);
  if (i >= B * wpr) return;
  const int t0 = (int)(i % wpr) * 32;
  uint32_t bits = 0u;
  if (t0 < T) {
    const long long base = i / wpr * T + t0, end = base + min(32, T - t0);
    int lo = 0, hi = n;
    while (lo < hi) {
      const int mid = (lo + hi) / 2;
      if (ds[mid] < base) lo = mid + 1;
      else hi = mid;
    }
    for (; lo < n && ds[lo] < end; ++lo)
      if (ds[lo] >= base) bits |= 1u << (int)(ds[lo] - base);
  }
  words[i] = bits;
}

// ------------------------------------------------------------------ the pass on the CUDA cores

size_t simt_smem(int Da) {
  return sizeof(float) * ((size_t)Da * kSlice + 2 * (size_t)L * (Da + 4) + (size_t)L * kSlice + L * kSp + 3 * L + 4);
}

// One block walks a segment's chunks of 32 tokens for one (row, head) and 64 columns
// of c, with its columns of the state in shared memory: the chunk's a, b and c are
// staged as fp32, the 32 x 32 products a . b under the decay formed, the chunk's
// output written and the state advanced.  Bound by the reads of shared memory and the
// latency of a chunk's steps: 4 heads of 128 x 8192 tokens, fp32, 203 us (20 TFLOP/s of some
// 70).  So a thread holds 2 x 4 outputs and reads their operands four at a time, and 4 x 4
// of the state, a row of c read once for four of its rows;
// and a batch of loads is under way before its first store.  2 rows of 6 heads of 64 x 96, 777
// tokens, backwards: 140 us (324 with a row of c read for each row of the state, a scalar an
// operand and a load at a time, 183 with the loads alone like that).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_pass(const Pass p) {
  extern __shared__ __align__(16) float smem[];
  const int Da = p.Da, lda = Da + 4;
  float* F = smem;                      // [Da][kSlice]
  float* sa = F + (size_t)Da * kSlice;  // [L][lda]
  float* sb = sa + (size_t)L * lda;     // [L][lda]
  float* sc = sb + (size_t)L * lda;     // [L][kSlice]
  float* sp = sc + L * kSlice;          // [L][kSp]
  float* pw = sp + L * kSp;         // [L + 1] powers of gamma
  float* win = pw + L + 1;              // [L] the state's weight in each row
  float* wout = win + L;                // [L] each row's weight in the new state
  float* fade = wout + L;               // [3] the factor of a whole chunk

  const int b = blockIdx.y / p.H, h = blockIdx.y % p.H;
  const int seg = blockIdx.z;
  const int c0 = blockIdx.x * kSlice;
  const int tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const float g = p.log_decay[h];
  if (threadIdx.x == 0 && !(g <= 0.0f)) set_status(p.status, IPTTT_ERR_ARG);
  if (threadIdx.x <= L) pw[threadIdx.x] = decay_pow(g, threadIdx.x);
  if (threadIdx.x == L) {
    const Fade f = fade_of(g, L);
    fade[0] = f.hi;
    fade[1] = f.lo;
    fade[2] = f.inv;
  }
  float left = 0.0f;
  const bool no_past = decay_pow(g, 1) == 0.0f;
  const T* A = static_cast<const T*>(p.a) + (long long)b * p.T * p.lda + (long long)(h / p.ga) * Da;
  const T* Bm = static_cast<const T*>(p.b) + (long long)b * p.T * p.ldb + (long long)(h / p.gb) * Da;
  const T* C = static_cast<const T*>(p.c) + (long long)b * p.T * p.ldc + (long long)(h / p.gc) * p.Dc;
  const uint32_t* words = p.starts ? p.starts + b * p.words : nullptr;
  const bool only_state = p.out == nullptr;
  if (only_state && seg == (p.rev ? 0 : p.segs - 1)) return;  // no segment comes after it

  const int nchunks = (p.T + L - 1) / L;
  const int first = seg * p.seg_chunks, last = min(nchunks, first + p.seg_chunks);
  const size_t bh = (size_t)b * p.H + h, nstate = (size_t)Da * p.Dc;
  // the state the segment starts from: the initial one, or what k_prefix has left for it
  const int c = c0 + 4 * tx;
  {
    const float* from = p.segs > 1 ? p.seg_in + (bh * p.segs + seg) * nstate : p.init ? p.init + bh * nstate : nullptr;
    const int turned = p.segs > 1 ? p.seg_t : p.init_t;
    const float mul = p.segs > 1 ? 1.0f : p.init_mul;
    for (int r = ty; r < Da; r += 16) {
      float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (!only_state && from && c < p.Dc) {
        if (!turned) f = load4(from + (size_t)r * p.Dc + c);
        else f = make_float4(from[(size_t)c * Da + r], from[(size_t)(c + 1) * Da + r], from[(size_t)(c + 2) * Da + r],
                             from[(size_t)(c + 3) * Da + r]);
      }
      store4(F + r * kSlice + 4 * tx, scale4(f, mul));
    }
  }

  for (int n = 0; n < last - first; ++n) {
    const int ch = p.rev ? last - 1 - n : first + n;
    const int t0 = ch * L, len = min(L, p.T - t0);
    const uint32_t w = words ? words[ch] : 0u;  // one word of starts a chunk
    const int first_start = w ? __ffs(w) - 1 : L, last_start = w ? 31 - __clz(w) : 0;
    const int lag = p.rev && t0 + len == p.T ? 1 : 0;
    __syncthreads();  // the last chunk's readers
    const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    // all loads of a batch before its first store: one at a time, each would wait for HBM by itself
    float4 vc[2];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int r = ty + 16 * u;
      vc[u] = r < len && c < p.Dc ? load4(C + (t0 + r) * p.ldc + c) : zero;
    }
    for (int q0 = 4 * tx; q0 < Da; q0 += 128) {
      float4 va[4], vb[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = ty + 16 * (u & 1), q = q0 + 64 * (u >> 1);
        const bool on = r < len && q < Da;
        vb[u] = on ? load4(Bm + (t0 + r) * p.ldb + q) : zero;
        va[u] = on && !only_state ? load4(A + (t0 + r) * p.lda + q) : zero;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = ty + 16 * (u & 1), q = q0 + 64 * (u >> 1);
        if (q >= Da) continue;
        store4(sb + r * lda + q, vb[u]);
        if (!only_state) store4(sa + r * lda + q, va[u]);
      }
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) store4(sc + (ty + 16 * u) * kSlice + 4 * tx, vc[u]);
    if (threadIdx.x < L) {
      const int i = threadIdx.x;
      const bool in = p.rev ? i >= last_start : i < first_start;
      const bool out = p.rev ? i < first_start : i >= last_start;
      const int ni = p.rev ? len - i - lag : i + 1, no = p.rev ? i : len - 1 - i;
      win[i] = in && i < len && !(no_past && ni > 0) ? pw[ni] : kNone;
      wout[i] = out && i < len && !(no_past && no > 0) ? pw[no] : kNone;
    }
    __syncthreads();
    if (!only_state) {
      float s[2][2] = {};
      int from[2], to[2];  // the tokens of row i's document on the side the pass looks at: [from, to)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = ty + 16 * u;
        const uint32_t below = w & ((2u << i) - 1u), above = i == 31 ? 0u : w >> (i + 1);
        from[u] = p.rev || no_past ? i : (below ? 31 - __clz(below) : 0);
        to[u] = p.rev && !no_past ? (above ? i + __ffs(above) : L) : i + 1;
      }
      for (int d = 0; d < Da; d += 4) {
        float4 x[2], y[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          x[u] = *reinterpret_cast<const float4*>(sa + (ty + 16 * u) * lda + d);
          y[u] = *reinterpret_cast<const float4*>(sb + (tx + 16 * u) * lda + d);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int v = 0; v < 2; ++v)
            s[u][v] = fmaf(x[u].x, y[v].x, fmaf(x[u].y, y[v].y, fmaf(x[u].z, y[v].z, fmaf(x[u].w, y[v].w, s[u][v]))));
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = ty + 16 * u;
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const int j = tx + 16 * v;
          sp[i * kSp + j] = j >= from[u] && j < to[u] ? s[u][v] * pw[abs(i - j)] : 0.0f;
        }
      }
      __syncthreads();
      float4 o[2], e[2];
      o[0] = o[1] = e[0] = e[1] = zero;
      // acc[u] += row ty + 16 u of x [.][ld] times y [n][kSlice]
      auto rows_times = [&](float4* acc, const float* x, int ld, const float* y, int n) {
#pragma unroll 2
        for (int d = 0; d < n; d += 4) {
          const float4 x0 = load4(x + ty * ld + d), x1 = load4(x + (ty + 16) * ld + d);
          float4 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = load4(y + (d + k) * kSlice + 4 * tx);
          fma4(acc[0], x0.x, v[0]);
          fma4(acc[1], x1.x, v[0]);
          fma4(acc[0], x0.y, v[1]);
          fma4(acc[1], x1.y, v[1]);
          fma4(acc[0], x0.z, v[2]);
          fma4(acc[1], x1.z, v[2]);
          fma4(acc[0], x0.w, v[3]);
          fma4(acc[1], x1.w, v[3]);
        }
      };
      rows_times(o, sp, kSp, sc, L);
      rows_times(e, sa, lda, F, Da);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int i = ty + 16 * u;
        if (i >= len || c >= p.Dc) continue;
        if (!finite4(o[u])) {  // 0 times a value of a token that the row does not see is NaN: those it sees alone
          o[u] = zero;
          for (int j = from[u]; j < min(to[u], len); ++j) fma4(o[u], sp[i * kSp + j], load4(sc + j * kSlice + 4 * tx));
        }
        if (win[i] >= 0.0f) fma4(o[u], win[i], e[u]);
        const long long at = ((long long)b * p.T + t0 + i) * p.ldo + (long long)h * p.Dc + c;
        const float4 r = scale4(o[u], p.scale);
        if (p.out_f32) store4(static_cast<float*>(p.out) + at, r);
        else store4(static_cast<T*>(p.out) + at, r);
      }
      __syncthreads();
    }
    float keep = len - lag == L ? fade_next({fade[0], fade[1], fade[2]}, left) : pw[len - lag];
    if (w || (no_past && len > lag)) keep = kNone;
    // four rows of the state at a time, so that a row of c is read once for them
    for (int r0 = ty; r0 < Da; r0 += 64) {
      float4 f[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int r = r0 + 16 * u;
        f[u] = keep >= 0.0f && r < Da ? scale4(load4(F + r * kSlice + 4 * tx), keep) : zero;
      }
#pragma unroll 4
      for (int j = 0; j < len; ++j) {
        const float x = wout[j];
        if (x < 0.0f) continue;
        const float4 v = scale4(load4(sc + j * kSlice + 4 * tx), x);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (r0 + 16 * u < Da) fma4(f[u], sb[j * lda + r0 + 16 * u], v);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (r0 + 16 * u < Da) store4(F + (r0 + 16 * u) * kSlice + 4 * tx, f[u]);
    }
  }

  float* dst = nullptr;
  float mul = 1.0f;
  bool none = false;
  if (only_state) {
    dst = p.seg_state + (bh * p.segs + seg) * nstate;
  } else if (p.fin && (p.rev ? seg == 0 : seg == p.segs - 1)) {
    dst = p.fin + bh * nstate;
    if (p.fin_scale) {
      mul = p.scale * decay_pow(g, 1);
      none = no_past;
    }
  }
  if (dst && c < p.Dc) {
    for (int r = ty; r < Da; r += 16) {  // a thread's own elements: no barrier since they were written
      const float4 f = load4(F + r * kSlice + 4 * tx);
      store4(dst + (size_t)r * p.Dc + c, none ? make_float4(0.0f, 0.0f, 0.0f, 0.0f) : scale4(f, mul));
    }
  }
}

// The segments' own states of a (row, head), seg_state, in place into the state that each segment
// starts from: forwards in order (backwards in the opposite one), the state brought along times
// gamma for every token of a segment, 0 where a document starts in it, plus the segment's own.  One
// thread takes four elements.  4.7 us for 12 heads of 13 states of 64 x 96.  (Every segment's block summing the
// states before it reads them segments^2 / 2 times, most of the time of a long row in many.)
__global__ void __launch_bounds__(kThreads) k_prefix(const Pass p) {
  __shared__ float keep[kMaxSegs], keep_lo[kMaxSegs];
  const size_t bh = p.whole + blockIdx.y, nstate = (size_t)p.Da * p.Dc;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  tc::launch_dependents();  // the pass may set itself up meanwhile
  const float g = p.log_decay[h];
  const uint32_t* words = p.starts ? p.starts + b * p.words : nullptr;
  for (int s = threadIdx.x; s < p.segs; s += kThreads) {
    const int lo = s * p.seg_chunks * p.chunk, hi = min(p.T, lo + p.seg_chunks * p.chunk);
    uint32_t any = 0;
    for (int w = lo / 32; words && 32 * w < hi; ++w) any |= words[w];
    const int n = hi - lo - (p.rev && hi == p.T ? 1 : 0);
    const Fade f = fade_of(g, n);
    keep[s] = any || (decay_pow(g, 1) == 0.0f && n > 0) ? kNone : f.hi;
    keep_lo[s] = f.lo;
  }
  __syncthreads();
  const size_t e = 4 * ((size_t)blockIdx.x * kThreads + threadIdx.x);
  if (e >= nstate) return;
  float4 f = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (p.init) {
    const int r = (int)(e / p.Dc), c = (int)(e % p.Dc);
    const float* in = p.init + bh * nstate;
    f = p.init_t ? make_float4(in[(size_t)c * p.Da + r], in[(size_t)(c + 1) * p.Da + r], in[(size_t)(c + 2) * p.Da + r],
                               in[(size_t)(c + 3) * p.Da + r])
                 : load4(in + e);
    f = scale4(f, p.init_mul);
  }
  float* x = p.seg_state + bh * p.segs * nstate + e;
  constexpr int AHEAD = 8;
  for (int n0 = 0; n0 < p.segs; n0 += AHEAD) {
    float4 own[AHEAD];
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {  // the last one's own state is nobody's
      const int s = p.rev ? p.segs - 1 - n0 - u : n0 + u;
      if (n0 + u < p.segs - 1) own[u] = load4(x + (size_t)s * nstate);
    }
#pragma unroll
    for (int u = 0; u < AHEAD; ++u) {
      if (n0 + u >= p.segs) continue;
      const int s = p.rev ? p.segs - 1 - n0 - u : n0 + u;
      store4(x + (size_t)s * nstate, f);
      if (n0 + u == p.segs - 1) continue;
      const float k = keep[s];
      if (k < 0.0f) {  // whatever f holds
        f = own[u];
      } else {
        float4 y = own[u];
        fma4(y, keep_lo[s], f);
        fma4(y, k, f);
        f = y;
      }
    }
  }
}

// ------------------------------------------------------------------ shared heads

// out[token][hk] = the sum over the group's heads, in head order, of part[token][hk * G + g] (fp32).
template <typename T>
__global__ void __launch_bounds__(kThreads) k_sum_heads(const float* part, T* out, long long tokens, int Hkv, int G, int D,
                                                      long long ldo) {
  const int dq = D / 4;
  const long long per = (long long)Hkv * dq, n = tokens * per;
  for (long long i = blockIdx.x * (long long)kThreads + threadIdx.x; i < n; i += (long long)gridDim.x * kThreads) {
    const long long t = i / per;
    const int e = (int)(i % per), hk = e / dq, q = 4 * (e % dq);
    const float* x = part + ((t * Hkv + hk) * G) * (long long)D + q;
    float4 s = load4(x);
    for (int g = 1; g < G; ++g) {
      const float4 y = load4(x + (long long)g * D);
      s = make_float4(s.x + y.x, s.y + y.y, s.z + y.z, s.w + y.w);
    }
    store4(out + t * ldo + (long long)hk * D + q, s);
  }
}

// ------------------------------------------------------------------ one token

// S <- gamma S + k v^T and o = scale q S for one (row, head) and COLS columns of the state
// a block.  Bound by HBM: the state is read and written once; a thread has all its
// rows' loads in flight before it uses one.
template <typename T, int COLS, int ROWS>
__global__ void __launch_bounds__(kThreads) k_step(float* S, const T* q, const T* k, const T* v, const float* log_decay,
                                                 const int32_t* starts, T* o, int H, int G, int Dk, int Dv,
                                                 long long ldq, long long ldk, long long ldv, long long ldo,
                                                 float scale, int* status) {
  constexpr int LANES = COLS / 4, GROUPS = kThreads / LANES;  // a group of LANES threads takes a row of the state
  __shared__ __align__(16) float part[GROUPS][COLS];
  __shared__ float sq[kMaxWidth], sk[kMaxWidth];
  const int b = blockIdx.x / H, h = blockIdx.x % H;
  const int grp = threadIdx.x / LANES, c = blockIdx.y * COLS + 4 * (threadIdx.x % LANES);
  const float g = log_decay[h];
  if (threadIdx.x == 0 && !(g <= 0.0f)) set_status(status, IPTTT_ERR_ARG);
  const float gamma = decay_pow(g, 1);
  const bool fresh = (starts && starts[b] != 0) || gamma == 0.0f;  // no past, whatever the state holds
  const T* qp = q + b * ldq + (long long)h * Dk;
  const T* kp = k + b * ldk + (long long)(h / G) * Dk;
  for (int i = threadIdx.x; i < Dk; i += kThreads) {
    sq[i] = to_f(qp[i]);
    sk[i] = to_f(kp[i]);
  }
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float* st = S + ((size_t)blockIdx.x * Dk) * Dv + c;
  const bool on = c < Dv;
  float4 vv = zero, acc = zero;
  if (on) vv = load4(v + b * ldv + (long long)(h / G) * Dv + c);
  bool waited = false;
  for (int r0 = grp; r0 < Dk || !waited; r0 += GROUPS * ROWS) {
    float4 s[ROWS];
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int r = r0 + u * GROUPS;
      s[u] = on && !fresh && r < Dk ? load4(st + (size_t)r * Dv) : zero;
    }
    if (!waited) {  // sq and sk; the state's loads are under way
      __syncthreads();
      waited = true;
    }
#pragma unroll
    for (int u = 0; u < ROWS; ++u) {
      const int r = r0 + u * GROUPS;
      if (!on || r >= Dk) continue;
      float4 x = scale4(s[u], gamma);
      fma4(x, sk[r], vv);
      fma4(acc, sq[r], x);
      store4(st + (size_t)r * Dv, x);
    }
  }
  *reinterpret_cast<float4*>(&part[grp][4 * (threadIdx.x % LANES)]) = acc;
  __syncthreads();
  const int e = blockIdx.y * COLS + threadIdx.x;
  if (threadIdx.x < COLS && e < Dv) {
    float s = 0.0f;
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) s += part[i][threadIdx.x];
    o[b * ldo + (long long)h * Dv + e] = from_f<T>(s * scale);
  }
}

template <typename T>
cudaError_t launch_step(const ipttt_linattn_params& p, float* S, const void* q, const void* k, const void* v,
                        const float* ld, const int32_t* starts, void* o, int* status, cudaStream_t st) {
  const int blocks = p.B * p.H, G = p.H / p.Hkv;
  // half rows of the state (of 128) where (row, head) pairs alone nearly fill the SMs, else quarter
  // rows: 80 pairs of 128 x 128, with the state in L2, 3.3 us in quarters, 3.5 in halves; 140
  // pairs 4.1 and 3.8, 240 pairs 5.8 and 5.3.  From HBM, 640 pairs: 16.8 us with 64 columns and
  // 4 loads ahead a thread, 18.0 with 32 columns, 17.4 with 128 and 8 loads, 20.3 with 128
  // and 16 (12.9 at the copy bandwidth).
  if (blocks >= 128)
    k_step<T, 64, 4><<<dim3(blocks, (p.Dv + 63) / 64), kThreads, 0, st>>>(
        S, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), ld, starts, static_cast<T*>(o),
        p.H, G, p.Dk, p.Dv, p.ldq, p.ldk, p.ldv, p.ldo, p.scale, status);
  else
    k_step<T, 32, 4><<<dim3(blocks, (p.Dv + 31) / 32), kThreads, 0, st>>>(
        S, static_cast<const T*>(q), static_cast<const T*>(k), static_cast<const T*>(v), ld, starts, static_cast<T*>(o),
        p.H, G, p.Dk, p.Dv, p.ldq, p.ldk, p.ldv, p.ldo, p.scale, status);
  return cudaGetLastError();
}

}  // namespace

// One cut for all passes of a call (`width`: the wider of Dk and Dv), so that the pass for gk can
// take the states of the one for gv.
int simt_segments(int B, int T, int H, int width, int* seg_chunks) {
  const int n = (T + L - 1) / L;
  const long long blocks = (long long)B * H * ((width + kSlice - 1) / kSlice), sms = 148;
  // The number of segments that comes out fastest, in two-hundredths of a chunk's time: an SM
  // holds up to three blocks (two at width 128), each more of them slowing all by 0.3; a block starts
  // in half a chunk's time, the pass for the segments' states takes 0.3 of the time a chunk and
  // its launch a quarter of one.  fp32, backwards: 4 heads of 128 x 8192 tokens 529 us in 37
  // segments (795 in 25, 720 in 50), 12 heads of 64 x 96, 777 tokens, 141 in 13 (276 in 4, 142 in
  // 25), 160 heads of 128 x 512 tokens 1284 in 3 (1402 in one).
  const long long room = std::min<long long>(3, kSmemSm / (long long)(simt_smem(width) + 1024));
  auto time = [&](long long count, long long work) {  // work in twentieths of a chunk
    const long long full = count / (sms * room), rest = (count % (sms * room) + sms - 1) / sms;
    return work * (full * (10 + 3 * (room - 1)) + (rest ? 10 + 3 * (rest - 1) : 0));
  };
  long long best = 0;
  for (int s = 1; s <= std::min(n, kMaxSegs); ++s) {
    const int each = (n + s - 1) / s, segs = (n + each - 1) / each;
    if (segs != s) continue;
    long long t = time(blocks * segs, 20 * each + 10);
    if (segs > 1) t += time(blocks * (segs - 1), 6 * each + 10) + 50;
    if (best == 0 || t < best) {
      best = t;
      *seg_chunks = each;
    }
  }
  return (n + *seg_chunks - 1) / *seg_chunks;
}

cudaError_t run_simt(const Pass& p, int dtype, cudaStream_t st) {
  const size_t smem = simt_smem(p.Da);
  const dim3 grid((p.Dc + kSlice - 1) / kSlice, p.B * p.H, p.segs);
  static std::atomic<bool> ready[64];  // room for the widest heads, once a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    const int most = (int)simt_smem(kMaxWidth);
    e = cudaFuncSetAttribute(k_pass<__nv_bfloat16>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k_pass<float>, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    if (e != cudaSuccess) return e;
    ready[dev].store(true);
  }
  if (dtype == IPTTT_BF16) k_pass<__nv_bfloat16><<<grid, kThreads, smem, st>>>(p);
  else k_pass<float><<<grid, kThreads, smem, st>>>(p);
  return cudaGetLastError();
}

// ------------------------------------------------------------------ entry points

namespace {

size_t al256(size_t x) { return (x + 255) & ~size_t(255); }

ipttt_status check(const ipttt_linattn_params* p) {
  if (!p) return IPTTT_ERR_ARG;
  if (p->dtype != IPTTT_F32 && p->dtype != IPTTT_BF16) return IPTTT_ERR_DTYPE;
  if (p->B <= 0 || p->T <= 0 || p->H <= 0 || p->Hkv <= 0 || p->Dk <= 0 || p->Dv <= 0) return IPTTT_ERR_ARG;
  if (p->H % p->Hkv != 0 || !isfinite(p->scale) || p->scale == 0.0f) return IPTTT_ERR_ARG;
  if (p->Dk % 8 != 0 || p->Dv % 8 != 0 || p->Dk > kMaxWidth || p->Dv > kMaxWidth) return IPTTT_ERR_UNSUPPORTED;
  if ((long long)p->B * p->T > (1ll << 30) || (long long)p->B * p->H > 65535 || p->H > 65535) return IPTTT_ERR_SHAPE;
  struct { long long ld, packed; } lds[] = {
      {p->ldq, (long long)p->H * p->Dk},   {p->ldk, (long long)p->Hkv * p->Dk}, {p->ldv, (long long)p->Hkv * p->Dv},
      {p->ldo, (long long)p->H * p->Dv},   {p->ldgq, (long long)p->H * p->Dk},  {p->ldgk, (long long)p->Hkv * p->Dk},
      {p->ldgv, (long long)p->Hkv * p->Dv}};
  for (const auto& x : lds)
    if (x.ld != 0 && (x.ld < x.packed || x.ld % 8 != 0 || x.ld > (1ll << 31))) return IPTTT_ERR_ARG;
  return IPTTT_OK;
}

// The parameters with every stride filled in.
ipttt_linattn_params filled(const ipttt_linattn_params& p) {
  ipttt_linattn_params f = p;
  auto set = [](int64_t& ld, long long packed) { if (ld == 0) ld = packed; };
  set(f.ldq, (long long)p.H * p.Dk);
  set(f.ldk, (long long)p.Hkv * p.Dk);
  set(f.ldv, (long long)p.Hkv * p.Dv);
  set(f.ldo, (long long)p.H * p.Dv);
  set(f.ldgq, (long long)p.H * p.Dk);
  set(f.ldgk, (long long)p.Hkv * p.Dk);
  set(f.ldgv, (long long)p.Hkv * p.Dv);
  return f;
}

bool aligned16(std::initializer_list<const void*> ps) {
  uintptr_t any = 0;
  for (const void* q : ps) any |= reinterpret_cast<uintptr_t>(q);
  return any % 16 == 0;
}

// bf16 of their widths always, short rows too: 20 heads of 128, 8192 tokens 73 us (958 on the CUDA
// cores), 64 tokens 7.1 (24.2; with states 13.3 and 25.2), one token 6.8 (9.2; 13.3 and 10.4), 1280 rows and
// heads of one token 52 (111).
bool on_tensor_cores(const ipttt_linattn_params& p) { return p.dtype == IPTTT_BF16 && tc_takes(p.Dk, p.Dv); }

struct Work {
  size_t starts, seg, S0, parts, total;
  long long words;
  int segs, seg_chunks;  // segments of a row, chunks of each
  int whole;             // (row, head) pairs that are not cut
  int prefixed;          // the segments' states are summed into those that they start from
};

Work work_of(const ipttt_linattn_params& p, bool backward) {
  Work w{};
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t o = off;
    off += al256(bytes);
    return o;
  };
  w.words = (p.T + kTcChunk - 1) / kTcChunk * (kTcChunk / 32);
  w.starts = take((size_t)p.B * w.words * 4);
  w.segs = on_tensor_cores(p) ? tc_segments(p.B, p.T, p.H, &w.seg_chunks, &w.whole)
                              : simt_segments(p.B, p.T, p.H, std::max(p.Dk, p.Dv), &w.seg_chunks);
  w.prefixed = !on_tensor_cores(p) || w.segs > kDirectStates;
  w.seg = take(w.segs > 1 ? (size_t)p.B * p.H * w.segs * p.Dk * p.Dv * 4 : 0);
  w.S0 = take(!backward && w.segs > 1 && !w.prefixed ? (size_t)p.B * p.H * p.Dk * p.Dv * 4 : 0);
  w.parts = take(backward && p.H != p.Hkv ? (size_t)p.B * p.T * p.H * std::max(p.Dk, p.Dv) * 4 : 0);
  w.total = std::max<size_t>(off, 256);
  return w;
}

cudaError_t run_prefix(const Pass& p, cudaStream_t st) {
  k_prefix<<<dim3((unsigned)((p.Da * p.Dc / 4 + kThreads - 1) / kThreads), p.B * p.H - p.whole), kThreads, 0, st>>>(p);
  return cudaGetLastError();
}

cudaError_t run_one(const ipttt_linattn_params& p, const Pass& q, cudaStream_t st) {
  return on_tensor_cores(p) ? run_tc(q, st) : run_simt(q, p.dtype, st);
}

// A pass, after its segments' own states where the row is cut into segments (have: they are in
// `seg` already).
cudaError_t run_pass(const ipttt_linattn_params& p, Pass q, float* seg, bool have, int* launches, cudaStream_t st) {
  if (q.segs > 1 && !have) {
    Pass s = q;
    s.out = nullptr;
    s.seg_state = seg;
    cudaError_t e = run_one(p, s, st);
    if (e != cudaSuccess) return e;
    ++*launches;
    q.after_states = 1;
    if (q.prefixed) {
      e = run_prefix(s, st);
      if (e != cudaSuccess) return e;
      ++*launches;
    }
  }
  q.seg_in = seg;
  ++*launches;
  return run_one(p, q, st);
}

// The start bits of the call, or null where no start is listed.
cudaError_t mark_starts(const ipttt_linattn_params& p, const Work& w, uint8_t* ws, const int32_t* ds, int n, int* status,
                        const uint32_t** out, int* launches, cudaStream_t st) {
  *out = nullptr;
  if (n == 0) return cudaSuccess;
  uint32_t* words = reinterpret_cast<uint32_t*>(ws + w.starts);
  k_mark<<<(unsigned)((p.B * w.words + 127) / 128), 128, 0, st>>>(words, w.words, p.B, p.T, ds, n, status);
  ++*launches;
  *out = words;
  return cudaGetLastError();
}

}  // namespace
}  // namespace la
}  // namespace ipttt

using namespace ipttt;
using namespace ipttt::la;

extern "C" {

size_t ipttt_linattn_workspace_size(const ipttt_linattn_params* p) {
  return check(p) == IPTTT_OK ? work_of(*p, false).total : 0;
}

size_t ipttt_linattn_backward_workspace_size(const ipttt_linattn_params* p) {
  return check(p) == IPTTT_OK ? work_of(*p, true).total : 0;
}

ipttt_status ipttt_linattn_forward(const ipttt_linattn_params* pp, const void* q, const void* k, const void* v,
                                   const float* log_decay, const int32_t* doc_starts, int32_t n_doc_starts,
                                   const float* S0_opt, void* O, float* S_final_opt, void* workspace,
                                   size_t workspace_bytes, void* stream) {
  const ipttt_status rc = check(pp);
  if (rc != IPTTT_OK) return rc;
  if (!q || !k || !v || !log_decay || !O || n_doc_starts < 0 || (n_doc_starts > 0 && !doc_starts)) return IPTTT_ERR_ARG;
  if (shared_pointer({O, workspace}, {q, k, v, log_decay, doc_starts, S0_opt, S_final_opt}) ||
      shared_pointer({S_final_opt}, {q, k, v, log_decay, doc_starts}))
    return IPTTT_ERR_ARG;
  if (!aligned16({q, k, v, O, S0_opt, S_final_opt})) return IPTTT_ERR_ALIGN;
  const Work w = work_of(*pp, false);
  if (!workspace || workspace_bytes < w.total) return IPTTT_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return IPTTT_ERR_ALIGN;
  const ipttt_linattn_params p = filled(*pp);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* status = device_status();
  int launches = 0;
  Pass a{};
  a.B = p.B;
  a.T = p.T;
  a.H = p.H;
  a.log_decay = log_decay;
  a.words = w.words;
  a.scale = p.scale;
  a.init_mul = 1.0f;
  a.status = status;
  const int G = p.H / p.Hkv;
  a.a = q;
  a.lda = p.ldq;
  a.ga = 1;
  a.b = k;
  a.ldb = p.ldk;
  a.gb = G;
  a.c = v;
  a.ldc = p.ldv;
  a.gc = G;
  a.Da = p.Dk;
  a.Dc = p.Dv;
  a.out = O;
  a.ldo = p.ldo;
  a.init = S0_opt;
  a.fin = S_final_opt;
  a.fine = S_final_opt != nullptr;
  a.segs = w.segs;
  a.seg_chunks = w.seg_chunks;
  a.whole = w.whole;
  a.prefixed = w.prefixed;
  a.chunk = on_tensor_cores(p) ? kTcChunk : kSimtChunk;
  cudaError_t e = mark_starts(p, w, ws, doc_starts, n_doc_starts, status, &a.starts, &launches, st);
  if (e == cudaSuccess && S0_opt && S0_opt == S_final_opt && a.segs > 1 && !w.prefixed) {
    // the last segment may write the final state before the others have read the first
    a.init = reinterpret_cast<const float*>(ws + w.S0);
    e = cudaMemcpyAsync(ws + w.S0, S0_opt, (size_t)p.B * p.H * p.Dk * p.Dv * 4, cudaMemcpyDeviceToDevice, st);
  }
  if (e == cudaSuccess) e = run_pass(p, a, reinterpret_cast<float*>(ws + w.seg), false, &launches, st);
  if (e != cudaSuccess) return cuda_fail("linattn_forward", e);
  count_launches(launches);
  return IPTTT_OK;
}

ipttt_status ipttt_linattn_backward(const ipttt_linattn_params* pp, const void* q, const void* k, const void* v,
                                    const float* log_decay, const int32_t* doc_starts, int32_t n_doc_starts,
                                    const float* S0_opt, const void* gO, const float* gS_final_opt, void* gq, void* gk,
                                    void* gv, float* gS0_opt, void* workspace, size_t workspace_bytes, void* stream) {
  const ipttt_status rc = check(pp);
  if (rc != IPTTT_OK) return rc;
  if (!q || !k || !v || !log_decay || !gO || !gq || !gk || !gv || n_doc_starts < 0 || (n_doc_starts > 0 && !doc_starts))
    return IPTTT_ERR_ARG;
  if (gS_final_opt && !isfinite(1.0f / pp->scale)) return IPTTT_ERR_ARG;  // R is kept without the scale: gS_final / scale enters it
  // (gS0 too: it is written before gS_final's last reader)
  if (shared_pointer({gq, gk, gv, gS0_opt, workspace}, {q, k, v, log_decay, doc_starts, S0_opt, gO, gS_final_opt}))
    return IPTTT_ERR_ARG;
  if (!aligned16({q, k, v, gO, gq, gk, gv, S0_opt, gS_final_opt, gS0_opt})) return IPTTT_ERR_ALIGN;
  const Work w = work_of(*pp, true);
  if (!workspace || workspace_bytes < w.total) return IPTTT_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return IPTTT_ERR_ALIGN;
  const ipttt_linattn_params p = filled(*pp);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* seg = reinterpret_cast<float*>(ws + w.seg);
  float* parts = reinterpret_cast<float*>(ws + w.parts);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int* status = device_status();
  int launches = 0;
  const int G = p.H / p.Hkv;
  Pass base{};
  base.B = p.B;
  base.T = p.T;
  base.H = p.H;
  base.log_decay = log_decay;
  base.words = w.words;
  base.scale = p.scale;
  base.segs = w.segs;
  base.seg_chunks = w.seg_chunks;
  base.whole = w.whole;
  base.prefixed = w.prefixed;
  base.chunk = on_tensor_cores(p) ? kTcChunk : kSimtChunk;
  base.status = status;
  cudaError_t e = mark_starts(p, w, ws, doc_starts, n_doc_starts, status, &base.starts, &launches, st);

  struct Arg {
    const void* x;
    long long ld;
    int g;
  };
  const Arg xq{q, p.ldq, 1}, xk{k, p.ldk, G}, xv{v, p.ldv, G}, xg{gO, p.ldo, 1};
  auto pass_of = [&](const Arg& a, const Arg& b, const Arg& c, int Da, int Dc) {
    Pass s = base;
    s.a = a.x;
    s.lda = a.ld;
    s.ga = a.g;
    s.b = b.x;
    s.ldb = b.ld;
    s.gb = b.g;
    s.c = c.x;
    s.ldc = c.ld;
    s.gc = c.g;
    s.Da = Da;
    s.Dc = Dc;
    return s;
  };
  // a gradient of k or v: straight to the output, or per head in fp32 and then summed over the group
  auto shared = [&](Pass s, void* out, long long ldo, int D, bool have) {
    s.rev = 1;
    s.init = gS_final_opt;
    s.init_mul = 1.0f / p.scale;
    if (G == 1) {
      s.out = out;
      s.ldo = ldo;
      return run_pass(p, s, seg, have, &launches, st);
    }
    s.out = parts;
    s.out_f32 = 1;
    s.ldo = (long long)p.H * D;
    const cudaError_t err = run_pass(p, s, seg, have, &launches, st);
    if (err != cudaSuccess) return err;
    const long long tokens = (long long)p.B * p.T, n = tokens * p.Hkv * (D / 4);
    const unsigned grid = (unsigned)std::min<long long>((n + kThreads - 1) / kThreads, 148 * 16);
    if (p.dtype == IPTTT_BF16)
      k_sum_heads<<<grid, kThreads, 0, st>>>(parts, static_cast<__nv_bfloat16*>(out), tokens, p.Hkv, G, D, ldo);
    else
      k_sum_heads<<<grid, kThreads, 0, st>>>(parts, static_cast<float*>(out), tokens, p.Hkv, G, D, ldo);
    ++launches;
    return cudaGetLastError();
  };

  if (e == cudaSuccess) {
    Pass s = pass_of(xg, xv, xk, p.Dv, p.Dk);  // gq, the state transposed
    s.init = S0_opt;
    s.init_mul = 1.0f;
    s.init_t = 1;
    s.out = gq;
    s.ldo = p.ldgq;
    e = run_pass(p, s, seg, false, &launches, st);
  }
  if (e == cudaSuccess) {
    Pass s = pass_of(xk, xq, xg, p.Dk, p.Dv);  // gv, and R's last value gives gS0
    s.fin = gS0_opt;
    s.fine = gS0_opt != nullptr;
    s.fin_scale = 1;
    e = shared(s, gv, p.ldgv, p.Dv, false);
  }
  if (e == cudaSuccess) {
    Pass s = pass_of(xv, xg, xq, p.Dv, p.Dk);  // gk, R transposed
    s.init_t = 1;
    s.seg_t = 1;      // the segments' R of the pass for gv serve here too
    e = shared(s, gk, p.ldgk, p.Dk, true);
  }
  if (e != cudaSuccess) return cuda_fail("linattn_backward", e);
  count_launches(launches);
  return IPTTT_OK;
}

ipttt_status ipttt_linattn_step(const ipttt_linattn_params* pp, float* S, const void* q, const void* k, const void* v,
                                const float* log_decay, const int32_t* starts_opt, void* o, void* stream) {
  const ipttt_status rc = check(pp);
  if (rc != IPTTT_OK) return rc;
  if (pp->T != 1 || !S || !q || !k || !v || !log_decay || !o) return IPTTT_ERR_ARG;
  if (shared_pointer({S, o}, {q, k, v, log_decay, starts_opt})) return IPTTT_ERR_ARG;
  if (!aligned16({S, q, k, v, o})) return IPTTT_ERR_ALIGN;
  const ipttt_linattn_params p = filled(*pp);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p.dtype == IPTTT_BF16
                            ? launch_step<__nv_bfloat16>(p, S, q, k, v, log_decay, starts_opt, o, device_status(), st)
                            : launch_step<float>(p, S, q, k, v, log_decay, starts_opt, o, device_status(), st);
  if (e != cudaSuccess) return cuda_fail("linattn_step", e);
  count_launches(1);
  return IPTTT_OK;
}

}  // extern "C"
