// Norms of queries and keys for each head with the position rotation, in one pass
// (ipttt_qk_norm_rope) and its gradients (ipttt_qk_norm_rope_backward).
//
// Mathematics, per vector x [D] with weight w: r = 1/sqrt(mean(x^2) + eps), xh = x r,
// z = xh w; each pair of z's first R elements turns by position * inv_freq.  Backward:
// gz = the pairs of gy turned back, gw = sum gz xh, gx = r (gz w - xh mean(gz w xh)).
//
// Bound by HBM (each element read and written once) as long as the instructions keep up: a first
// form with 8 elements a lane took 256 instructions for 512 bytes in and out of a warp, and
// ran at the rate those issue (172 us for 32768 tokens of 32 + 8 heads of 128, bf16, where
// the bytes take 103).  So a lane holds 16 elements of a vector where the widths allow
// (8 elsewhere), in two strips chosen so that both halves of every pair lie in the same
// lane: the rotation needs no exchange between lanes, and the norm one sum over the 4 to
// 32 lanes of a vector.  (Arithmetic two elements an instruction took more instructions, not
// fewer: pairing registers up costs moves.)  Strips: elements
// from E/2 l and from R/2 + E/2 l on (pairs (i, i + R/2)), or E l.. and E l + E/2.. (pairs
// (2i, 2i+1), and elements that do not turn).  A block takes a tile of tokens at a time with
// all their heads; a group of lanes stays with one token, whose sines and cosines
// (angle reduced to a turn in 64 bits) are computed once for all heads and then stay in
// registers.  Now 116 us at full clocks, 118 to 123 under load, for those 32768 tokens (671 MB, 5.5 to
// 5.8 TB/s; 83 to 89% of the copy bandwidth), 5.4 for 300, 3.5 for 16.  Backwards, 3 x 4099
// tokens of 20 + 4 heads of 128, half of each turned: 68 to 72 us with the weights' sum (227 MB,
// 3.2 TB/s).  What bounds it is latency: two blocks of 8 warps an SM, a barrier on either side
// of a tile's angles and one round of loads ahead leave half of the issue slots and 60% of DRAM's
// time unused (stalls of an instruction at 16384 tokens: 2.3 for loads, 1.2 at barriers).
// In fp32 the forms of 16 elements a lane spill (forwards 700 bytes a thread at 80 registers,
// backwards 88); the bf16 ones do not.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <algorithm>

#include "common.cuh"

namespace ipttt {
namespace {

constexpr int kThreads = 256;
constexpr int kTokens = 8;        // tokens of a forward tile (1 where there are few)
constexpr int kMaxTokens = 32;    // of a backward tile
constexpr int kMaxD = 256;
constexpr int kForwardBlocks = 444, kBackwardBlocks = 296;  // most blocks: 3 and 2 per SM, as their registers allow

struct QkArgs {
  const void *q, *k, *wq, *wk, *gqo, *gko;
  const double* inv_freq;
  const long long* pos;
  void *qo, *ko;                 // forward: the outputs; backward: gq, gk
  long long ldq, ldk, ldqo, ldko, ldgq, ldgk;
  float* parts;                  // backward: [blocks][D]
  int qblocks, blocks;           // backward: blocks that take q, all blocks
  int qshift, kshift;            // backward: their tiles' tokens
  long long tokens;
  int Hq, Hk, D, R, interleaved;
  int shift;                     // tiles of 1 << shift tokens
  float eps, inv_d;
};

// N elements (4 or 8) as they lie in memory, as fp32, and back.
template <typename T, int N> struct Strip;
template <int N> struct Strip<float, N> {
  float4 v[N / 4];
  __device__ __forceinline__ void load(const float* p) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) v[i] = reinterpret_cast<const float4*>(p)[i];
  }
  __device__ __forceinline__ void unpack(float* x) const {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      x[4 * i] = v[i].x;
      x[4 * i + 1] = v[i].y;
      x[4 * i + 2] = v[i].z;
      x[4 * i + 3] = v[i].w;
    }
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i)
      reinterpret_cast<float4*>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
  }
};
template <int N> struct Strip<__nv_bfloat16, N> {
  uint32_t v[N / 2];
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    if constexpr (N == 8) *reinterpret_cast<uint4*>(v) = *reinterpret_cast<const uint4*>(p);
    else *reinterpret_cast<uint2*>(v) = *reinterpret_cast<const uint2*>(p);
  }
  __device__ __forceinline__ void unpack(float* x) const {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      x[2 * i] = __uint_as_float(v[i] << 16);
      x[2 * i + 1] = __uint_as_float(v[i] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
    uint32_t w[N / 2];
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    if constexpr (N == 8) *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(w);
    else *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(w);
  }
};

// A lane's E elements of a vector: two strips of E/2.
template <typename T, int E> struct Piece {
  Strip<T, E / 2> a, b;
  __device__ __forceinline__ void load(const T* p, int o0, int o1) {
    a.load(p + o0);
    b.load(p + o1);
  }
  __device__ __forceinline__ void unpack(float* x) const {
    a.unpack(x);
    b.unpack(x + E / 2);
  }
  static __device__ __forceinline__ void store(T* p, int o0, int o1, const float* x) {
    Strip<T, E / 2>::store(p + o0, x);
    Strip<T, E / 2>::store(p + o1, x + E / 2);
  }
};

// The cosines and sines of a lane's E/2 pairs (in order), read once for its token; BACK turns the
// other way.  Lanes whose elements do not turn keep c = 1, s = 0.
template <int E, bool BACK> struct Turn {
  float c[E / 2], s[E / 2];
  __device__ __forceinline__ void none() {
#pragma unroll
    for (int i = 0; i < E / 2; ++i) {
      c[i] = 1.0f;
      s[i] = 0.0f;
    }
  }
  __device__ __forceinline__ void read(const float* cs, const float* sn) {
#pragma unroll
    for (int i = 0; i < E / 8; ++i) {
      *reinterpret_cast<float4*>(c + 4 * i) = reinterpret_cast<const float4*>(cs)[i];
      *reinterpret_cast<float4*>(s + 4 * i) = reinterpret_cast<const float4*>(sn)[i];
    }
  }
  __device__ __forceinline__ void apply(float* x, bool interleaved) const {
    constexpr float sign = BACK ? -1.0f : 1.0f;
    if (!interleaved) {  // strip 0 holds the first halves, strip 1 the second
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float a = x[i], b = x[E / 2 + i];
        x[i] = fmaf(-sign * b, s[i], a * c[i]);
        x[E / 2 + i] = fmaf(sign * a, s[i], b * c[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < E / 2; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = fmaf(-sign * b, s[i], a * c[i]);
        x[2 * i + 1] = fmaf(sign * a, s[i], b * c[i]);
      }
    }
  }
};

// The sum over the G lanes of a vector (all lanes of the warp take part).
template <int G>
__device__ __forceinline__ float group_sum(float v) {
#pragma unroll
  for (int o = G / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a lane's strips lie within a vector, and its first pair.
struct LanePlace {
  int o0, o1, pair;
  bool rotates, used;
};
template <int E>
__device__ __forceinline__ LanePlace place_of(const QkArgs& a, int l) {
  LanePlace p;
  p.used = E * l < a.D;
  p.rotates = E * l < a.R;
  p.pair = E / 2 * l;
  const bool halves = p.rotates && !a.interleaved;
  p.o0 = halves ? E / 2 * l : E * l;
  p.o1 = halves ? a.R / 2 + E / 2 * l : E * l + E / 2;
  return p;
}

// cos and sin of every (token, pair) of the tile that starts at token t0.  The turns are reduced in
// 64 bits whatever the type; bf16 then takes the hardware's sine and cosine (off by 2^-21
// at most on [-pi, pi], far below its rounding of 2^-8), which with the accurate ones
// would be a third of all instructions.
template <typename T>
__device__ __forceinline__ void fill_angles(const QkArgs& a, long long t0, int n, float* cs, float* sn) {
  if (a.R == 0) return;  // there may be no positions
  for (int t = threadIdx.x >> 6; t < n; t += kThreads / 64) {
    const double pos = (double)a.pos[t0 + t];
    for (int f = threadIdx.x & 63; f < a.R / 2; f += 64) {
      const double turns = pos * (a.inv_freq[f] * 0.15915494309189533577);  // 1 / (2 pi)
      const float part = (float)(turns - rint(turns));
      float s, c;
      if constexpr (sizeof(T) == 2) __sincosf(6.283185307179586f * part, &s, &c);
      else sincospif(2.0f * part, &s, &c);
      cs[t * (kMaxD / 2) + f] = c;
      sn[t * (kMaxD / 2) + f] = s;
    }
  }
}

// A group of lanes takes the heads first, first + step, ... of its token of one operand.  Lanes that
// hold no elements keep the zeros they start with; a group past the last head keeps what it
// has, which goes nowhere.
template <typename T, int E> struct Heads {
  const T* x;
  int H, first, step;
  bool on;  // the lane holds elements, and the token is there
  __device__ __forceinline__ void load(Piece<T, E>& raw, const LanePlace& lp, int D, int h0) const {
    if (on && h0 + first < H) raw.load(x + (h0 + first) * D, lp.o0, lp.o1);
  }
};

template <typename T, int E>
__device__ __forceinline__ void load_weight(float* wv, const T* w, const LanePlace& lp) {
  Piece<T, E> pw{};
  if (lp.used) pw.load(w, lp.o0, lp.o1);
  pw.unpack(wv);
}

// Every lane of a warp runs the same number of rounds: the sums need them all.  raw holds the
// first two rounds' elements; a round's place is filled again, two rounds ahead, once it
// has been read.
template <typename T, int E, int G>
__device__ __forceinline__ void forward_heads(const QkArgs& a, const LanePlace& lp, const Turn<E, false>& turn,
                                              const Heads<T, E>& hd, Piece<T, E> (&raw)[2], const T* w, T* y) {
  float wv[E];
  load_weight<T, E>(wv, w, lp);
#pragma unroll 1
  for (int h0 = 0; h0 < hd.H; h0 += 2 * hd.step) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      const int h = h0 + u * hd.step + hd.first;
      float v[E], ss[2] = {};
      raw[u].unpack(v);
      hd.load(raw[u], lp, a.D, h0 + (u + 2) * hd.step);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        ss[i & 1] = fmaf(v[i], v[i], ss[i & 1]);
        v[i] *= wv[i];
      }
      const float r = rsqrtf(group_sum<G>(ss[0] + ss[1]) * a.inv_d + a.eps);
      turn.apply(v, a.interleaved);
#pragma unroll
      for (int i = 0; i < E; ++i) v[i] *= r;
      if (hd.on && h < hd.H) Piece<T, E>::store(y + h * a.D, lp.o0, lp.o1, v);
    }
  }
}

template <typename T, int E, int G>
__global__ void __launch_bounds__(kThreads, 3) k_qk_forward(const QkArgs a) {
  constexpr int kGroups = kThreads / G;
  __shared__ __align__(16) float cs[kTokens * kMaxD / 2], sn[kTokens * kMaxD / 2];
  const LanePlace lp = place_of<E>(a, threadIdx.x % G);
  const int grp = threadIdx.x / G, t = grp & ((1 << a.shift) - 1), first = grp >> a.shift, step = kGroups >> a.shift;
  for (long long t0 = (long long)blockIdx.x << a.shift; t0 < a.tokens; t0 += (long long)gridDim.x << a.shift) {
    const int n = (int)min(1ll << a.shift, a.tokens - t0);
    const long long tok = t0 + t;
    const bool on = t < n && lp.used;
    const Heads<T, E> hq{static_cast<const T*>(a.q) + tok * a.ldq, a.Hq, first, step, on};
    const Heads<T, E> hk{static_cast<const T*>(a.k) + tok * a.ldk, a.Hk, first, step, on};
    Piece<T, E> raw[2] = {};
    hq.load(raw[0], lp, a.D, 0);
    hq.load(raw[1], lp, a.D, step);
    __syncthreads();  // the last tile's angles have been read
    fill_angles<T>(a, t0, n, cs, sn);  // while the first elements are on their way
    __syncthreads();
    Turn<E, false> turn;
    if (lp.rotates && t < n) turn.read(cs + t * (kMaxD / 2) + lp.pair, sn + t * (kMaxD / 2) + lp.pair);
    else turn.none();
    forward_heads<T, E, G>(a, lp, turn, hq, raw, static_cast<const T*>(a.wq), static_cast<T*>(a.qo) + tok * a.ldqo);
    hk.load(raw[0], lp, a.D, 0);
    hk.load(raw[1], lp, a.D, step);
    forward_heads<T, E, G>(a, lp, turn, hk, raw, static_cast<const T*>(a.wk), static_cast<T*>(a.ko) + tok * a.ldko);
  }
}

// The block's sum of every element's weight gradient, in the order of its groups of lanes.
template <int E, int G>
__device__ __forceinline__ void store_parts(const LanePlace& lp, const float* gw, float* sh, float* out, int D) {
  constexpr int kGroups = kThreads / G;
  if (lp.used) Piece<float, E>::store(sh + (threadIdx.x / G) * (G * E), lp.o0, lp.o1, gw);
  __syncthreads();
  for (int e = threadIdx.x; e < D; e += kThreads) {
    float sum = 0.0f;
    for (int q = 0; q < kGroups; ++q) sum += sh[q * (G * E) + e];
    out[e] = sum;
  }
}

// The first a.qblocks blocks take q, the rest k (in proportion to their heads), so that a thread holds one
// operand's weight and weight gradient alone: with both, registers spill.  A round of x and
// gy is on its way while the last one is worked on.
template <typename T, int E, int G>
__global__ void __launch_bounds__(kThreads, 2) k_qk_backward(const QkArgs a) {
  constexpr int kGroups = kThreads / G;
  __shared__ __align__(16) float cs[kMaxTokens * kMaxD / 2], sn[kMaxTokens * kMaxD / 2];
  __shared__ __align__(16) float sh[kThreads * E];  // [kGroups][G E]
  const bool is_q = (int)blockIdx.x < a.qblocks;
  const int block = is_q ? blockIdx.x : blockIdx.x - a.qblocks, blocks = is_q ? a.qblocks : gridDim.x - a.qblocks;
  const T* x = static_cast<const T*>(is_q ? a.q : a.k);
  const T* gy = static_cast<const T*>(is_q ? a.gqo : a.gko);
  T* gx = static_cast<T*>(is_q ? a.qo : a.ko);
  const long long ldx = is_q ? a.ldq : a.ldk, ldgy = is_q ? a.ldqo : a.ldko, ldgx = is_q ? a.ldgq : a.ldgk;
  const int H = is_q ? a.Hq : a.Hk, shift = is_q ? a.qshift : a.kshift;
  const LanePlace lp = place_of<E>(a, threadIdx.x % G);
  const int grp = threadIdx.x / G, t = grp & ((1 << shift) - 1), first = grp >> shift, step = kGroups >> shift;
  float wv[E], gw[E] = {};
  load_weight<T, E>(wv, static_cast<const T*>(is_q ? a.wq : a.wk), lp);
  for (long long t0 = (long long)block << shift; t0 < a.tokens; t0 += (long long)blocks << shift) {
    const long long tok = t0 + t;
    const int n = (int)min(1ll << shift, a.tokens - t0);
    const bool on = t < n && lp.used;
    const Heads<T, E> hx{x + tok * ldx, H, first, step, on}, hg{gy + tok * ldgy, H, first, step, on};
    T* out = gx + tok * ldgx;
    Piece<T, E> rx{}, rg{};
    hx.load(rx, lp, a.D, 0);
    hg.load(rg, lp, a.D, 0);
    __syncthreads();  // the last tile's angles have been read
    fill_angles<T>(a, t0, n, cs, sn);
    __syncthreads();
    Turn<E, true> turn;
    if (lp.rotates && t < n) turn.read(cs + t * (kMaxD / 2) + lp.pair, sn + t * (kMaxD / 2) + lp.pair);
    else turn.none();
#pragma unroll 1
    for (int h0 = 0; h0 < H; h0 += step) {
      const int h = h0 + first;
      float v[E], z[E], ss[2] = {}, ux[2] = {};
      rx.unpack(v);
      rg.unpack(z);
      hx.load(rx, lp, a.D, h0 + step);
      hg.load(rg, lp, a.D, h0 + step);
      turn.apply(z, a.interleaved);
#pragma unroll
      for (int i = 0; i < E; ++i) {
        ss[i & 1] = fmaf(v[i], v[i], ss[i & 1]);
        ux[i & 1] = fmaf(z[i] * wv[i], v[i], ux[i & 1]);
      }
      const float r = rsqrtf(group_sum<G>(ss[0] + ss[1]) * a.inv_d + a.eps);
      const float m = -group_sum<G>(ux[0] + ux[1]) * r * a.inv_d;  // -mean(gz w xh)
      if (on && h < H) {
#pragma unroll
        for (int i = 0; i < E; ++i) {
          const float xh = v[i] * r;
          gw[i] = fmaf(z[i], xh, gw[i]);
          z[i] = fmaf(xh, m, z[i] * wv[i]) * r;
        }
        Piece<T, E>::store(out + h * a.D, lp.o0, lp.o1, z);
      }
    }
  }
  store_parts<E, G>(lp, gw, sh, a.parts + (size_t)blockIdx.x * a.D, a.D);
}

// gw[e] = the blocks' partial sums, in 64 bits and a fixed order; one block of 32 x 32
// threads takes 32 elements of gwq (y = 0) or gwk (y = 1).
__global__ void __launch_bounds__(1024) k_qk_weight_grad(const float* parts, float* gwq, float* gwk, int qblocks,
                                                         int blocks, int D) {
  __shared__ double sh[32][33];
  const int e = blockIdx.x * 32 + threadIdx.x;
  const int lo = blockIdx.y == 0 ? 0 : qblocks, hi = blockIdx.y == 0 ? qblocks : blocks;
  double s = 0.0;
  if (e < D) {
#pragma unroll 4
    for (int i = lo + threadIdx.y; i < hi; i += 32) s += parts[(size_t)i * D + e];
  }
  sh[threadIdx.x][threadIdx.y] = s;
  __syncthreads();
  // warp y sums element y
  s = sh[threadIdx.y][threadIdx.x];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < D) (blockIdx.y == 0 ? gwq : gwk)[out] = (float)s;
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
  a.inv_d = 1.0f / (float)p.D;
  // a token a tile while every block has one at most, else eight, whose angles and loads share a
  // block's latency: 32 + 8 heads of 128, 300 tokens 5.4 us (6.2 by eights), 1184 tokens 6.7 by
  // eights (12.9 one by one), 32768 tokens 116 (298).  Measured at those heads alone: with one head
  // of q and k three quarters of a tile's groups of lanes have none
  a.shift = a.tokens > kForwardBlocks ? 3 : 0;
  static_assert(kTokens == 8, "shift");
  return a;
}

long long tiles_of(const QkArgs& a) { return (a.tokens + (1ll << a.shift) - 1) >> a.shift; }

// Lanes and elements a lane of a vector: 16 elements where D and R are multiples of 16, else 8; the
// fewest lanes that hold D.
struct Form {
  int elements, lanes;
};
Form form_of(int D, int R) {
  const int e = D % 16 == 0 && R % 16 == 0 ? 16 : 8;
  const int base = 64 / e;
  return {e, D <= 64 ? base : D <= 128 ? 2 * base : 4 * base};
}

// The backward's tiles and blocks.  A tile holds so many tokens (up to 32) that a group of lanes has
// at least four heads of its token, and that every block still has one; the blocks, as many as
// run at once, are shared between q and k by what their tiles cost: the rounds of
// heads, and about two rounds for the angles and the first loads.
void share_blocks(QkArgs& a) {
  const int groups = kThreads / form_of(a.D, a.R).lanes, most = kBackwardBlocks;
  auto shift_of = [&](int H) {
    int s = 0;
    while ((2 << s) <= std::min(groups, kMaxTokens) && (groups >> s) > std::max(1, H / 4) &&
           (a.tokens >> (s + 1)) >= most / 2)
      ++s;
    return s;
  };
  auto tiles = [&](int shift) { return (a.tokens + (1ll << shift) - 1) >> shift; };
  auto cost = [&](int H, int shift) {
    const int step = groups >> shift;
    return tiles(shift) * ((H + step - 1) / step + 2);
  };
  a.qshift = shift_of(a.Hq);
  a.kshift = shift_of(a.Hk);
  const long long cq = cost(a.Hq, a.qshift), ck = cost(a.Hk, a.kshift);
  const int k = (int)std::min<long long>(most - 1, std::max<long long>(1, (most * ck + (cq + ck) / 2) / (cq + ck)));
  a.qblocks = (int)std::min<long long>(most - k, tiles(a.qshift));
  a.blocks = a.qblocks + (int)std::min<long long>(k, tiles(a.kshift));
}

struct Forward {
  template <typename T, int E, int G>
  static void launch(const QkArgs& a, cudaStream_t st) {
    k_qk_forward<T, E, G><<<(unsigned)std::min<long long>(kForwardBlocks, tiles_of(a)), kThreads, 0, st>>>(a);
  }
};
struct Backward {
  template <typename T, int E, int G>
  static void launch(const QkArgs& a, cudaStream_t st) {
    k_qk_backward<T, E, G><<<(unsigned)a.blocks, kThreads, 0, st>>>(a);
  }
};

template <typename K, typename T>
cudaError_t launch(const QkArgs& a, cudaStream_t st) {
  const Form f = form_of(a.D, a.R);
  if (f.elements == 16) {
    if (f.lanes == 4) K::template launch<T, 16, 4>(a, st);
    else if (f.lanes == 8) K::template launch<T, 16, 8>(a, st);
    else K::template launch<T, 16, 16>(a, st);
  } else {
    if (f.lanes == 8) K::template launch<T, 8, 8>(a, st);
    else if (f.lanes == 16) K::template launch<T, 8, 16>(a, st);
    else K::template launch<T, 8, 32>(a, st);
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
  if ((q == q_out && a.ldq != a.ldqo) || (k == k_out && a.ldk != a.ldko) || q == k_out || k == q_out ||
      shared_pointer({q_out, k_out}, {wq, wk, inv_freq, positions}))
    return IPTTT_ERR_ARG;
  a.q = q;
  a.k = k;
  a.wq = wq;
  a.wk = wk;
  a.inv_freq = inv_freq;
  a.pos = reinterpret_cast<const long long*>(positions);
  a.qo = q_out;
  a.ko = k_out;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const cudaError_t e = p->dtype == IPTTT_BF16 ? launch<Forward, __nv_bfloat16>(a, st) : launch<Forward, float>(a, st);
  if (e != cudaSuccess) return cuda_fail("qk_norm_rope", e);
  count_launches(1);
  return IPTTT_OK;
}

size_t ipttt_qk_norm_rope_backward_workspace_size(const ipttt_qk_params* p) {
  if (check(p) != IPTTT_OK) return 0;
  QkArgs a = args_of(*p);
  share_blocks(a);
  return ((size_t)a.blocks * a.D * sizeof(float) + 255) & ~size_t(255);
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
  if ((gq == gqo && a.ldgq != a.ldqo) || (gk == gko && a.ldgk != a.ldko) || (gq == q && a.ldgq != a.ldq) ||
      (gk == k && a.ldgk != a.ldk) || gq == k || gq == gko || gk == q || gk == gqo ||
      shared_pointer({gq, gk, gwq, gwk, workspace}, {wq, wk, inv_freq, positions}) ||
      shared_pointer({gwq, gwk, workspace}, {q, k, gqo, gko}))
    return IPTTT_ERR_ARG;
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
  share_blocks(a);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  cudaError_t e = p->dtype == IPTTT_BF16 ? launch<Backward, __nv_bfloat16>(a, st) : launch<Backward, float>(a, st);
  if (e == cudaSuccess) {
    k_qk_weight_grad<<<dim3((a.D + 31) / 32, 2), dim3(32, 32), 0, st>>>(a.parts, gwq, gwk, a.qblocks, a.blocks, a.D);
    e = cudaGetLastError();
  }
  if (e != cudaSuccess) return cuda_fail("qk_norm_rope_backward", e);
  count_launches(2);
  return IPTTT_OK;
}

}  // extern "C"
