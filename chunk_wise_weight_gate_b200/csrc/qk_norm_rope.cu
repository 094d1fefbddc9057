// Norms of queries and keys for each head with the position rotation, in one pass
// (ipttt_qk_norm_rope) and its gradients (ipttt_qk_norm_rope_backward).
//
// Mathematics, per vector x [D] with weight w: r = 1/sqrt(mean(x^2) + eps), xh = x r,
// z = xh w; each pair of z's first R elements turns by position * inv_freq.  Backward:
// gz = the pairs of gy turned back, gw = sum gz xh, gx = r (gz w - xh mean(gz w xh)).
//
// Bound by HBM: 16 bytes in and 16 out per 8 bf16 elements, some 100 instructions.
// Layout: a lane holds 8 elements of a vector as two quads, chosen so that both
// halves of a pair lie in the same lane: elements 4l.. and R/2 + 4l.. (pairs
// (i, i + R/2)), or 8l..8l+7 (pairs (2i, 2i+1)); lanes from R/8 on hold the elements
// that do not turn, 8 in a row.  So the rotation needs no exchange between lanes,
// and the norm one reduction over the 8, 16 or 32 lanes of a vector.  A block takes
// a few tokens with all their heads, so that the sines and cosines (one per
// token and pair: angle reduced to a turn in 64 bits, sincospif of the rest)
// are computed once and shared by the heads through shared memory.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"

namespace ipttt {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 4;        // tokens of a tile (1 where there are few)
constexpr int kMaxD = 256;
constexpr int kGradBlocks = 592;  // most blocks (= partial weight gradients) of the backward: 4 per SM

struct QkArgs {
  const void *q, *k, *wq, *wk, *gqo, *gko;
  const double* inv_freq;
  const long long* pos;
  void *qo, *ko;                 // forward: the outputs; backward: gq, gk
  long long ldq, ldk, ldqo, ldko, ldgq, ldgk;
  float* parts;                  // backward: [2][blocks][D]
  long long tokens;
  int Hq, Hk, D, R, interleaved, tile;
  float eps;
};

// Four consecutive elements as fp32.
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

__device__ __forceinline__ float dot4(float4 a, float4 b) { return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w; }
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
__device__ __forceinline__ float4 scale4(float4 a, float s) { return make_float4(a.x * s, a.y * s, a.z * s, a.w * s); }

// Turns the four pairs held in (a, b) by the angles whose cosines and sines are c and s.
__device__ __forceinline__ void turn(float4& a, float4& b, float4 c, float4 s, bool interleaved) {
  const float4 x = a, y = b;
  if (interleaved) {  // pairs (x.x, x.y), (x.z, x.w), (y.x, y.y), (y.z, y.w)
    a = make_float4(x.x * c.x - x.y * s.x, x.y * c.x + x.x * s.x, x.z * c.y - x.w * s.y, x.w * c.y + x.z * s.y);
    b = make_float4(y.x * c.z - y.y * s.z, y.y * c.z + y.x * s.z, y.z * c.w - y.w * s.w, y.w * c.w + y.z * s.w);
  } else {
    a = make_float4(x.x * c.x - y.x * s.x, x.y * c.y - y.y * s.y, x.z * c.z - y.z * s.z, x.w * c.w - y.w * s.w);
    b = make_float4(y.x * c.x + x.x * s.x, y.y * c.y + x.y * s.y, y.z * c.z + x.z * s.z, y.w * c.w + x.w * s.w);
  }
}

// The sum over the G lanes of a vector (all lanes of the warp take part).
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// A lane's two quads within a vector, and its first pair.
struct LanePlace {
  int o0, o1, pair;
  bool rotates, used;
};
__device__ __forceinline__ LanePlace place_of(const QkArgs& a, int l) {
  LanePlace p;
  p.used = 8 * l < a.D;
  p.rotates = 8 * l < a.R;
  p.pair = 4 * l;
  const bool halves = p.rotates && !a.interleaved;
  p.o0 = halves ? 4 * l : 8 * l;
  p.o1 = halves ? a.R / 2 + 4 * l : 8 * l + 4;
  return p;
}

// cos and sin of every (token, pair) of the tile that starts at token t0.
__device__ __forceinline__ void fill_angles(const QkArgs& a, long long t0, int n, float* cs, float* sn) {
  const int half = a.R / 2;
  for (int i = threadIdx.x; i < n * half; i += kThreads) {
    const int t = i / half, f = i % half;
    const double turns = (double)a.pos[t0 + t] * (a.inv_freq[f] * 0.15915494309189533577);  // 1 / (2 pi)
    float s, c;
    sincospif(2.0f * (float)(turns - rint(turns)), &s, &c);
    cs[t * (kMaxD / 2) + f] = c;
    sn[t * (kMaxD / 2) + f] = s;
  }
}

template <typename T, int G>
__device__ __forceinline__ void forward_heads(const QkArgs& a, const LanePlace& lp, long long t0, int n, int H,
                                              const T* x, long long ldx, const T* w, T* y, long long ldy,
                                              const float* cs, const float* sn) {
  constexpr int kVecs = kThreads / G;  // vectors a block has in hand
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float4 w0 = lp.used ? load4(w + lp.o0) : zero, w1 = lp.used ? load4(w + lp.o1) : zero;
  const int total = n * H;
  // every lane of a warp runs the same number of steps: the sums need them all
  for (int v0 = 0; v0 < total; v0 += kVecs) {
    const int v = v0 + threadIdx.x / G;
    const bool on = v < total && lp.used;
    const int t = on ? v / H : 0, h = on ? v % H : 0;
    float4 x0 = zero, x1 = zero;
    if (on) {
      const T* xp = x + (t0 + t) * ldx + (long long)h * a.D;
      x0 = load4(xp + lp.o0);
      x1 = load4(xp + lp.o1);
    }
    const float r = rsqrtf(group_sum<G>(dot4(x0, x0) + dot4(x1, x1)) / a.D + a.eps);
    if (!on) continue;
    float4 y0 = mul4(scale4(x0, r), w0), y1 = mul4(scale4(x1, r), w1);
    if (lp.rotates) {
      const float4 c = *reinterpret_cast<const float4*>(cs + t * (kMaxD / 2) + lp.pair);
      const float4 s = *reinterpret_cast<const float4*>(sn + t * (kMaxD / 2) + lp.pair);
      turn(y0, y1, c, s, a.interleaved);
    }
    T* yp = y + (t0 + t) * ldy + (long long)h * a.D;
    store4(yp + lp.o0, y0);
    store4(yp + lp.o1, y1);
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) k_qk_forward(const QkArgs a) {
  __shared__ __align__(16) float cs[kTokens * kMaxD / 2], sn[kTokens * kMaxD / 2];
  const LanePlace lp = place_of(a, threadIdx.x % G);
  const long long t0 = (long long)blockIdx.x * a.tile;
  const int n = (int)min((long long)a.tile, a.tokens - t0);
  fill_angles(a, t0, n, cs, sn);
  __syncthreads();
  forward_heads<T, G>(a, lp, t0, n, a.Hq, static_cast<const T*>(a.q), a.ldq, static_cast<const T*>(a.wq),
                      static_cast<T*>(a.qo), a.ldqo, cs, sn);
  forward_heads<T, G>(a, lp, t0, n, a.Hk, static_cast<const T*>(a.k), a.ldk, static_cast<const T*>(a.wk),
                      static_cast<T*>(a.ko), a.ldko, cs, sn);
}

// As forward_heads; the lane's share of the weight gradient is added to g0, g1.
template <typename T, int G>
__device__ __forceinline__ void backward_heads(const QkArgs& a, const LanePlace& lp, long long t0, int n, int H,
                                               const T* x, long long ldx, const T* w, const T* gy, long long ldgy,
                                               T* gx, long long ldgx, const float* cs, const float* sn, float4& g0,
                                               float4& g1) {
  constexpr int kVecs = kThreads / G;
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  const float4 w0 = lp.used ? load4(w + lp.o0) : zero, w1 = lp.used ? load4(w + lp.o1) : zero;
  const int total = n * H;
  for (int v0 = 0; v0 < total; v0 += kVecs) {
    const int v = v0 + threadIdx.x / G;
    const bool on = v < total && lp.used;
    const int t = on ? v / H : 0, h = on ? v % H : 0;
    float4 x0 = zero, x1 = zero, z0 = zero, z1 = zero;
    if (on) {
      const T* xp = x + (t0 + t) * ldx + (long long)h * a.D;
      const T* gp = gy + (t0 + t) * ldgy + (long long)h * a.D;
      x0 = load4(xp + lp.o0);
      x1 = load4(xp + lp.o1);
      z0 = load4(gp + lp.o0);
      z1 = load4(gp + lp.o1);
      if (lp.rotates) {  // back: the same pairs by the opposite angle
        const float4 c = *reinterpret_cast<const float4*>(cs + t * (kMaxD / 2) + lp.pair);
        const float4 s = *reinterpret_cast<const float4*>(sn + t * (kMaxD / 2) + lp.pair);
        turn(z0, z1, c, scale4(s, -1.0f), a.interleaved);
      }
    }
    const float4 u0 = mul4(z0, w0), u1 = mul4(z1, w1);
    const float ss = group_sum<G>(dot4(x0, x0) + dot4(x1, x1));
    const float ux = group_sum<G>(dot4(u0, x0) + dot4(u1, x1));
    if (!on) continue;
    const float r = rsqrtf(ss / a.D + a.eps);
    x0 = scale4(x0, r);
    x1 = scale4(x1, r);
    const float m = ux * r / a.D;  // mean(u xh)
    T* op = gx + (t0 + t) * ldgx + (long long)h * a.D;
    store4(op + lp.o0, make_float4(r * (u0.x - x0.x * m), r * (u0.y - x0.y * m), r * (u0.z - x0.z * m),
                                   r * (u0.w - x0.w * m)));
    store4(op + lp.o1, make_float4(r * (u1.x - x1.x * m), r * (u1.y - x1.y * m), r * (u1.z - x1.z * m),
                                   r * (u1.w - x1.w * m)));
    g0 = make_float4(fmaf(z0.x, x0.x, g0.x), fmaf(z0.y, x0.y, g0.y), fmaf(z0.z, x0.z, g0.z), fmaf(z0.w, x0.w, g0.w));
    g1 = make_float4(fmaf(z1.x, x1.x, g1.x), fmaf(z1.y, x1.y, g1.y), fmaf(z1.z, x1.z, g1.z), fmaf(z1.w, x1.w, g1.w));
  }
}

// The block's sum of every element's weight gradient, in the order of its groups of lanes.
template <int G>
__device__ __forceinline__ void store_parts(const LanePlace& lp, float4 g0, float4 g1, float* sh, float* out, int D) {
  constexpr int kVecs = kThreads / G;
  __syncthreads();  // sh's last readers
  if (lp.used) {
    float* s = sh + (threadIdx.x / G) * kMaxD;
    *reinterpret_cast<float4*>(s + lp.o0) = g0;
    *reinterpret_cast<float4*>(s + lp.o1) = g1;
  }
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kThreads) {
    float sum = 0.0f;
    for (int q = 0; q < kVecs; ++q) sum += sh[q * kMaxD + e];
    out[e] = sum;
  }
}

template <typename T, int G>
__global__ void __launch_bounds__(kThreads) k_qk_backward(const QkArgs a) {
  __shared__ __align__(16) float cs[kTokens * kMaxD / 2], sn[kTokens * kMaxD / 2];
  extern __shared__ __align__(16) float sh[];  // [kThreads / G][kMaxD]
  const LanePlace lp = place_of(a, threadIdx.x % G);
  const float4 zero = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  float4 q0 = zero, q1 = zero, k0 = zero, k1 = zero;
  const long long tiles = (a.tokens + a.tile - 1) / a.tile;
  for (long long i = blockIdx.x; i < tiles; i += gridDim.x) {
    const long long t0 = i * a.tile;
    const int n = (int)min((long long)a.tile, a.tokens - t0);
    __syncthreads();  // the last tile's angles have been read
    fill_angles(a, t0, n, cs, sn);
    __syncthreads();
    backward_heads<T, G>(a, lp, t0, n, a.Hq, static_cast<const T*>(a.q), a.ldq, static_cast<const T*>(a.wq),
                         static_cast<const T*>(a.gqo), a.ldqo, static_cast<T*>(a.qo), a.ldgq, cs, sn, q0, q1);
    backward_heads<T, G>(a, lp, t0, n, a.Hk, static_cast<const T*>(a.k), a.ldk, static_cast<const T*>(a.wk),
                         static_cast<const T*>(a.gko), a.ldko, static_cast<T*>(a.ko), a.ldgk, cs, sn, k0, k1);
  }
  store_parts<G>(lp, q0, q1, sh, a.parts + (size_t)blockIdx.x * a.D, a.D);
  store_parts<G>(lp, k0, k1, sh, a.parts + (size_t)(gridDim.x + blockIdx.x) * a.D, a.D);
}

// gw[e] = the blocks' partial sums in block order, in 64 bits; one block of 32 x 8
// threads takes 32 elements of gwq (y = 0) or gwk (y = 1).
__global__ void k_qk_weight_grad(const float* parts, float* gwq, float* gwk, int blocks, int D) {
  __shared__ double sh[8][32];
  const int e = blockIdx.x * 32 + threadIdx.x;
  double s = 0.0;
  if (e < D)
    for (int i = threadIdx.y; i < blocks; i += 8) s += parts[((size_t)blockIdx.y * blocks + i) * D + e];
  sh[threadIdx.y][threadIdx.x] = s;
  __syncthreads();
  if (threadIdx.y == 0 && e < D) {
    for (int q = 1; q < 8; ++q) s += sh[q][threadIdx.x];
    (blockIdx.y == 0 ? gwq : gwk)[e] = (float)s;
  }
}

ipttt_status check(const ipttt_qk_params* p) {
  if (!p) return IPTTT_ERR_ARG;
  if (p->dtype != IPTTT_F32 && p->dtype != IPTTT_BF16) return IPTTT_ERR_DTYPE;
  if (p->B <= 0 || p->T <= 0 || p->Hq <= 0 || p->Hk <= 0 || p->D <= 0 || p->R < 0) return IPTTT_ERR_ARG;
  if (!(p->eps > 0.0f) || !isfinite(p->eps) || (p->interleaved != 0 && p->interleaved != 1)) return IPTTT_ERR_ARG;
  if (p->D % 8 != 0 || p->R % 8 != 0 || p->R > p->D || p->D > kMaxD) return IPTTT_ERR_UNSUPPORTED;
  if ((long long)p->B * p->T > (1ll << 30) || p->Hq > (1 << 16) || p->Hk > (1 << 16)) return IPTTT_ERR_SHAPE;
  const long long wq = (long long)p->Hq * p->D, wk = (long long)p->Hk * p->D;
  for (long long ld : {(long long)p->ldq, (long long)p->ldqo, (long long)p->ldgq})
    if (ld != 0 && (ld < wq || ld % 8 != 0 || ld > (1ll << 31))) return IPTTT_ERR_ARG;
  for (long long ld : {(long long)p->ldk, (long long)p->ldko, (long long)p->ldgk})
    if (ld != 0 && (ld < wk || ld % 8 != 0 || ld > (1ll << 31))) return IPTTT_ERR_ARG;
  return IPTTT_OK;
}

QkArgs args_of(const ipttt_qk_params& p) {
  QkArgs a{};
  const long long wq = (long long)p.Hq * p.D, wk = (long long)p.Hk * p.D;
  auto ld = [](long long v, long long packed) { return v ? v : packed; };
  a.ldq = ld(p.ldq, wq);
  a.ldk = ld(p.ldk, wk);
  a.ldqo = ld(p.ldqo, wq);
  a.ldko = ld(p.ldko, wk);
  a.ldgq = ld(p.ldgq, wq);
  a.ldgk = ld(p.ldgk, wk);
  a.tokens = (long long)p.B * p.T;
  a.Hq = p.Hq;
  a.Hk = p.Hk;
  a.D = p.D;
  a.R = p.R;
  a.interleaved = p.interleaved;
  a.eps = p.eps;
  // four tokens share a block's angle pass, unless that leaves SMs without a block
  a.tile = a.tokens >= (long long)kTokens * kGradBlocks ? kTokens : 1;
  return a;
}

int lanes_of(int D) { return D <= 64 ? 8 : D <= 128 ? 16 : 32; }

int grad_blocks(const QkArgs& a) {
  return (int)std::min<long long>(kGradBlocks, (a.tokens + a.tile - 1) / a.tile);
}

template <typename T>
cudaError_t launch_forward(const QkArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)((a.tokens + a.tile - 1) / a.tile);
  switch (lanes_of(a.D)) {
    case 8: k_qk_forward<T, 8><<<grid, kThreads, 0, st>>>(a); break;
    case 16: k_qk_forward<T, 16><<<grid, kThreads, 0, st>>>(a); break;
    default: k_qk_forward<T, 32><<<grid, kThreads, 0, st>>>(a); break;
  }
  return cudaGetLastError();
}

template <typename T>
cudaError_t launch_backward(const QkArgs& a, cudaStream_t st) {
  const unsigned grid = (unsigned)grad_blocks(a);
  switch (lanes_of(a.D)) {
    case 8: k_qk_backward<T, 8><<<grid, kThreads, (kThreads / 8) * kMaxD * 4, st>>>(a); break;
    case 16: k_qk_backward<T, 16><<<grid, kThreads, (kThreads / 16) * kMaxD * 4, st>>>(a); break;
    default: k_qk_backward<T, 32><<<grid, kThreads, (kThreads / 32) * kMaxD * 4, st>>>(a); break;
  }
  return cudaGetLastError();
}

bool aligned16(std::initializer_list<const void*> ps) {
  uintptr_t any = 0;
  for (const void* q : ps) any |= reinterpret_cast<uintptr_t>(q);
  return any % 16 == 0;
}

}  // namespace
}  // namespace ipttt

using namespace ipttt;

extern "C" {

ipttt_status ipttt_qk_norm_rope(const ipttt_qk_params* p, const void* q, const void* k, const void* wq, const void* wk,
                                const double* inv_freq, const int64_t* positions, void* q_out, void* k_out,
                                void* stream) {
  const ipttt_status rc = check(p);
  if (rc != IPTTT_OK) return rc;
  if (!q || !k || !wq || !wk || !q_out || !k_out || (p->R > 0 && (!inv_freq || !positions))) return IPTTT_ERR_ARG;
  if (!aligned16({q, k, wq, wk, q_out, k_out}) || reinterpret_cast<uintptr_t>(inv_freq) % 8 ||
      reinterpret_cast<uintptr_t>(positions) % 8)
    return IPTTT_ERR_ALIGN;
  QkArgs a = args_of(*p);
  // in place means the same elements: another stride would write vectors not yet read
  if ((q == q_out && a.ldq != a.ldqo) || (k == k_out && a.ldk != a.ldko)) return IPTTT_ERR_ARG;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.inv_freq = inv_freq;
  a.pos = reinterpret_cast<const long long*>(positions);
  a.qo = q_out;
  a.ko = k_out;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == IPTTT_BF16 ? launch_forward<__nv_bfloat16>(a, st) : launch_forward<float>(a, st);
  if (e != cudaSuccess) return cuda_fail("qk_norm_rope", e);
  count_launches(1);
  return IPTTT_OK;
}

size_t ipttt_qk_norm_rope_backward_workspace_size(const ipttt_qk_params* p) {
  if (check(p) != IPTTT_OK) return 0;
  const QkArgs a = args_of(*p);
  return ((size_t)2 * grad_blocks(a) * a.D * sizeof(float) + 255) & ~size_t(255);
}

ipttt_status ipttt_qk_norm_rope_backward(const ipttt_qk_params* p, const void* q, const void* k, const void* wq,
                                         const void* wk, const double* inv_freq, const int64_t* positions,
                                         const void* gqo, const void* gko, void* gq, void* gk, float* gwq, float* gwk,
                                         void* workspace, size_t workspace_bytes, void* stream) {
  const ipttt_status rc = check(p);
  if (rc != IPTTT_OK) return rc;
  if (!q || !k || !wq || !wk || !gqo || !gko || !gq || !gk || !gwq || !gwk ||
      (p->R > 0 && (!inv_freq || !positions)))
    return IPTTT_ERR_ARG;
  if (!aligned16({q, k, wq, wk, gqo, gko, gq, gk, gwq, gwk}) || reinterpret_cast<uintptr_t>(inv_freq) % 8 ||
      reinterpret_cast<uintptr_t>(positions) % 8)
    return IPTTT_ERR_ALIGN;
  if (!workspace || workspace_bytes < ipttt_qk_norm_rope_backward_workspace_size(p)) return IPTTT_ERR_WORKSPACE;
  if (reinterpret_cast<uintptr_t>(workspace) % 256) return IPTTT_ERR_ALIGN;
  QkArgs a = args_of(*p);
  if ((gq == gqo && a.ldgq != a.ldqo) || (gk == gko && a.ldgk != a.ldko)) return IPTTT_ERR_ARG;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.inv_freq = inv_freq;
  a.pos = reinterpret_cast<const long long*>(positions);
  a.gqo = gqo;
  a.gko = gko;
  a.qo = gq;
  a.ko = gk;
  a.parts = static_cast<float*>(workspace);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = p->dtype == IPTTT_BF16 ? launch_backward<__nv_bfloat16>(a, st) : launch_backward<float>(a, st);
  if (e == cudaSuccess) {
    k_qk_weight_grad<<<dim3((a.D + 31) / 32, 2), dim3(32, 8), 0, st>>>(a.parts, gwq, gwk, grad_blocks(a), a.D);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return cuda_fail("qk_norm_rope_backward", e);
  count_launches(2);
  return IPTTT_OK;
}

}  // extern "C"
