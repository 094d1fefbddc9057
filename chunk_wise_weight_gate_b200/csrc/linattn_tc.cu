// The linear-attention pass on the tensor cores (bf16 operands, widths 64 and 128):
// linattn.h has the mathematics of a pass.
//
// A persistent CTA per SM takes work items (row, head, segment) and walks a segment's
// chunks of 128 tokens.  Per chunk, all on tcgen05 with fp32 accumulators in TMEM:
//   (1) SC = A B^T                 128 x 128 products of the chunk's tokens
//   (2) O1 = A F                   what the state before the chunk gives each token
//   (3) O2 = P C                   P = SC under the decay and the masks, bf16, in TMEM
//   (4) D  = (w B)^T C             the chunk's own addition to the state
// out = scale (O2 + w_in O1); F <- keep F + D in fp32 registers.  w B, each row times its
// decay to the chunk's end, is split in two bf16 halves (hi + lo): the state is off by 4e-6 of
// its norm, far below what its operand copy loses.  P and that copy are rounded to bf16
// once, like the inputs and outputs are (outputs off by 2.3e-3 where their own rounding
// makes 1.7e-3).  Where the state itself goes out (FINE), w B is three parts: B times the power of
// two nearest to w, exact, and two of the rest, a third of w at most: 7e-7, for a third more of
// (4)'s products; lower parts of 64 tokens at a time share the place of the one.  8 x 2047 tokens
// of 24 heads with states: 126.2 us, 112.4 in two parts (one box in turn).
//
// Roles: warp 0 issues the TMA loads, a thread of warp 1 the MMAs (1) to (3), a thread of
// warp 2 those of (4); 8 warps turn SC into P (two a quarter of the rows, 64 columns
// each) and write the output (through the a tile's place and TMA stores); 8 warps scale
// and split B in place, hold the state (a row and a strip of columns a thread) and write
// its bf16 copy, the B operand of (2).  Every wait is bounded and reports IPTTT_ERR_TIMEOUT; where
// a waiter may be a whole chunk behind, a pair of barriers is taken in turn (a parity
// tells a phase only from its neighbours).
//
// What bounds it, at width 128: a chunk moves 131 KB (3.0 us an SM at the measured copy bandwidth
// over 148 SMs) and takes 2600 clocks of tensor pipe (N = 128: 64 clocks a MMA).  Shared
// memory is full (two a tiles, three b and c tiles, the lo half, the state's copy: 224 KB),
// so a tile's load starts less than a chunk ahead, and a chunk takes 3.3 to 3.7 us: 148 heads of 2048
// tokens 64 us, 310 MB at 4.8 TB/s (73% of the copy bandwidth).  Measured on the way there: descriptors
// rebuilt for each MMA cost its issuing thread 100 clocks a MMA; loops unrolled as far as they go
// overran the instruction caches (a third of all stalls); one issuing thread instead of
// two: 68 us; tiles brought into L2 ahead of their loads: 72 us.
//
// Masked places are products with 0, which is NaN for a value that is not finite.  An item that held one
// is done again at the end, token by token (`walk`).  Telling by the state alone, and the masks, cost
// 2 x 8192 tokens of 20 heads backwards 0.4% (337.6 -> 339.0 us, one box in turn) and 32768 forwards
// nothing; looking at the outputs too cost 2% more, a walk within the item with its state in
// registers 5%.  Rows of one chunk pay more: 1280 of 64 wide 36.5 -> 43.6 us with P's lower part.
//
// Rows are cut into segments when rows and heads alone leave SMs idle: a first pass (STATES) forms
// each segment's own state from b and c alone (1.5 to 1.7 us a chunk: 64 KB, HBM), and the full
// pass starts each segment from their sum under the decay (many segments: from what k_prefix left).
#include <cuda_bf16.h>

#include <algorithm>
#include <atomic>

#include "linattn.h"
#include "linattn_smem.h"
#include "tc.cuh"
#include "tc_kernels.h"

namespace ipttt {
namespace la {

using namespace ipttt::tc;

namespace {

constexpr int CH = kTcChunk;
constexpr int kOutWarp = 4;  // first of the 8 warps that turn scores into P and write the output

enum Kind { FORWARD = 0, REVERSE = 1, STATES = 2 };  // STATES: a segment's own state alone, either way

template <int DA, int DC, bool STATE>
struct Cfg {
  using Mem = Smem<DA, DC, STATE>;
  static constexpr int SLOT = Mem::SLOT;
  static constexpr int NS = Mem::NS;
  static constexpr int SMEM = Mem::BYTES;
  static constexpr int NC = DA * DC / 256;   // state columns a thread holds
  static constexpr int SW = STATE ? 4 : 12;  // first of the 8 state warps
  static constexpr int THREADS = 32 * (SW + 8);
};
// Registers a thread of the full pass's three groups (640 threads, 96 each at launch): the
// state's owners need more than an even share, the others less.
constexpr int kRegsIssue = 64, kRegsOut = 88, kRegsState = 120, kRegsLaunch = 96;
static_assert(128 * kRegsIssue + 256 * kRegsOut + 256 * kRegsState <= 640 * kRegsLaunch, "register split");
// TMEM columns
constexpr int kSC = 0, kO1 = 128;
__host__ __device__ constexpr int col_o2(int dc) { return 128 + dc; }
__host__ __device__ constexpr int col_d(int dc) { return 128 + 2 * dc; }

struct TcArgs {
  CUtensorMap ma, mb, mc, mo;
  Pass p;
  int items;
};

struct Item {
  int b, h, seg, segs, first, last;  // chunks [first, last) of segment seg out of segs
};

// Work items: the (row, head) pairs that are not cut, then the segments of the others, the
// pairs fastest (heads side by side in memory are walked at the same time).
__device__ __forceinline__ Item item_of(const Pass& p, int i) {
  Item t;
  const int n = (p.T + CH - 1) / CH;
  int bh;
  if (p.out && i < p.whole) {
    bh = i;
    t.seg = 0;
    t.segs = 1;
    t.first = 0;
    t.last = n;
  } else {
    const int j = p.out ? i - p.whole : i, cut = p.B * p.H - p.whole;
    bh = p.whole + j % cut;
    // a pass for states alone leaves out the segment that nothing follows
    t.seg = j / cut + (!p.out && p.rev ? 1 : 0);
    t.segs = p.segs;
    t.first = t.seg * p.seg_chunks;
    t.last = min(n, t.first + p.seg_chunks);
  }
  t.b = bh / p.H;
  t.h = bh % p.H;
  return t;
}

// The document starts of a chunk of 128 tokens, as bits.
struct Starts {
  uint4 w;
  __device__ __forceinline__ bool any() const { return (w.x | w.y | w.z | w.w) != 0; }
  __device__ __forceinline__ int first() const {  // CH if none
    return w.x ? __ffs(w.x) - 1 : w.y ? 31 + __ffs(w.y) : w.z ? 63 + __ffs(w.z) : w.w ? 95 + __ffs(w.w) : CH;
  }
  __device__ __forceinline__ int last() const {  // 0 if none
    return w.w ? 127 - __clz(w.w) : w.z ? 95 - __clz(w.z) : w.y ? 63 - __clz(w.y) : w.x ? 31 - __clz(w.x) : 0;
  }
  // the bits of tokens [0, n)
  __device__ __forceinline__ Starts below(int n) const {
    auto m = [n](int k) { return n >= 32 * k + 32 ? 0xffffffffu : n <= 32 * k ? 0u : (1u << (n - 32 * k)) - 1u; };
    return {make_uint4(w.x & m(0), w.y & m(1), w.z & m(2), w.w & m(3))};
  }
  __device__ __forceinline__ Starts from(int n) const {
    const Starts b = below(n);
    return {make_uint4(w.x ^ b.w.x, w.y ^ b.w.y, w.z ^ b.w.z, w.w ^ b.w.w)};
  }
};

__device__ __forceinline__ Starts starts_of(const Pass& p, int b, int ch) {
  if (!p.starts) return {make_uint4(0u, 0u, 0u, 0u)};
  return {*reinterpret_cast<const uint4*>(p.starts + b * p.words + 4 * ch)};
}

// The nearest start on the far side of a segment, for one warp (every lane gets it): forwards the
// last start before token `at` (-1: none), backwards the first start from token `at` on (T: none).
__device__ __forceinline__ int nearest_start_warp(const Pass& p, int b, int at, int lane) {
  int best = p.rev ? p.T : -1;
  if (!p.starts) return best;
  const uint32_t* w = p.starts + b * p.words;
  if (p.rev) {
    for (int i = at / 32 + lane; i < p.words; i += 32) {
      const uint32_t m = i == at / 32 ? w[i] & (0xffffffffu << (at % 32)) : w[i];
      if (m) best = min(best, 32 * i + __ffs(m) - 1);
    }
    return __reduce_min_sync(0xffffffffu, best);
  }
  for (int i = lane; 32 * i < at; i += 32) {
    const uint32_t m = i == at / 32 ? w[i] & ((1u << (at % 32)) - 1u) : w[i];
    if (m) best = max(best, 32 * i + 31 - __clz(m));
  }
  return __reduce_max_sync(0xffffffffu, best);
}

// Factor with which segment s's own state, and the initial state (s = -1), reach the
// segment of tokens [lo, hi): kNone where a document starts between, or there is no past.
__device__ __forceinline__ float reach(const Pass& p, float g, int s, int lo, int hi, int start) {
  bool seen;
  int n;  // tokens between
  if (p.rev) {
    const int s0 = s * p.seg_chunks * CH;
    seen = s < 0 ? start >= p.T : s0 <= start;
    n = s < 0 ? p.T - 1 - hi : s0 - hi;
  } else {
    const int end = s < 0 ? 0 : (s + 1) * p.seg_chunks * CH;
    seen = s < 0 ? start < 0 : end > start;
    n = lo - end;
  }
  return seen && (n <= 0 || decay_pow(g, 1) != 0.0f) ? decay_pow(g, n) : kNone;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// Zeros on the far side of the diagonal block's row `lane`, 32 bf16 numbers, whatever they are: not times 0
// alone, as products of tokens far apart in size may overflow.  (PTX shifts by more than 31 leave 0.)
__device__ __forceinline__ void far_side_off(uint32_t (&w)[16], int lane, bool rev) {
#pragma unroll
  for (int e = 0; e < 16; ++e) {
    const int bits = rev ? max(16 * (2 * e + 2 - lane), 0) : max(16 * (lane + 1 - 2 * e), 0);  // kept, from the near side
    uint32_t off;
    if (rev) asm("shr.u32 %0, %1, %2;" : "=r"(off) : "r"(0xffffffffu), "r"(bits));
    else asm("shl.b32 %0, %1, %2;" : "=r"(off) : "r"(0xffffffffu), "r"(bits));
    w[e] &= ~off;
  }
}

// What the roles tell one another besides barriers; from W_ODD on, a bit for each item of the block.
enum Word { W_TMEM = 0, W_ABORT = 1, W_TILES = 2, W_A_TILES = 3, W_ODD = 4 };

// mbar_wait_or_abort in few instructions: there are some twenty waits in the kernel.
__device__ __forceinline__ bool wait_for(uint64_t* bar, uint32_t parity, volatile uint32_t* words) {
  bool done = mbar_try_wait(bar, parity);
  if (!done) {
    const uint64_t t0 = global_timer_ns();
#pragma unroll 1
    do done = mbar_try_wait(bar, parity);
    while (!done && !words[W_ABORT] && global_timer_ns() - t0 < kWaitLimitNs);
  }
  return done;
}

// Where an item's last state goes (null: nowhere), and the factor on it; none: it is 0, as there is no
// past that it could be the gradient of.
struct Last {
  float* dst;
  float mul;
  bool none;
};
template <bool STATE>
__device__ __forceinline__ Last last_of(const Pass& p, const Item& it, float g) {
  const size_t bh = (size_t)it.b * p.H + it.h, nstate = (size_t)p.Da * p.Dc;
  Last to = {nullptr, 1.0f, false};
  if (STATE) {
    to.dst = p.seg_state + (bh * p.segs + it.seg) * nstate;
  } else if (p.fin && (p.rev ? it.seg == 0 : it.seg == it.segs - 1)) {
    to.dst = p.fin + bh * nstate;
    if (p.fin_scale) {
      to.mul = p.scale * decay_pow(g, 1);
      to.none = decay_pow(g, 1) == 0.0f;
    }
  }
  return to;
}

// An item by the recurrence itself, token by token, on the 256 threads of the state warps (tid).  For items
// alone that hold a value that is not finite: 0 times it, in masked places, is NaN, and the chunk's
// other tokens and documents must not take it.  A thread has a column of the state, tid % DC, and
// ROWS of its rows from tid / DC * ROWS on; the state lies in F (shared memory, as registers would
// cost the chunks' loop), kWalk tokens at a time in `room`, as fp32.  A barrier joins the threads,
// `met` times so far; false: a wait gave up.  2.0 us a token at width 128 (32768 tokens of 20 heads, a
// bad value in each item: 9.5 ms): the shared memory's and the batches' latency.
template <int DA, int DC, bool STATE>
__device__ __forceinline__ bool walk(const Pass& p, const Item& it, float* F, float* room, int tid, uint64_t* bar,
                                     uint32_t& met, volatile uint32_t* words) {
  constexpr int ROWS = DA * DC / 256, GROUPS = 256 / DC;
  float *sa = room, *sb = sa + kWalk * DA, *sc = sb + kWalk * DA;  // [kWalk][DA], [kWalk][DA], [kWalk][DC]
  float* so = sc + kWalk * DC;                                     // [kWalk][GROUPS][DC]
  const int col = tid % DC, r0 = tid / DC * ROWS;
  const size_t bh = (size_t)it.b * p.H + it.h, nstate = (size_t)DA * DC;
  const int lo = it.first * CH, hi = min(p.T, it.last * CH);
  const uint32_t* starts = p.starts ? p.starts + it.b * p.words : nullptr;
  const float g = p.log_decay[it.h];
  const Fade gamma = fade_of(g, 1);
  float left = 0.0f;
  float* f = F + r0 * DC + col;  // the thread's first element; its rows are DC apart
  auto meet = [&] {
    __syncwarp();
    if (tid % 32 == 0) mbar_arrive(bar);
    return __all_sync(0xffffffffu, wait_for(bar, met++ & 1u, words)) != 0;
  };
#pragma unroll 1
  for (int e = 0; e < ROWS; ++e) f[e * DC] = 0.0f;
  if constexpr (!STATE) {
    const bool prefixed = p.prefixed && it.segs > 1;
    auto add = [&](const float* src, int transposed, float w) {
#pragma unroll 1
      for (int e = 0; e < ROWS; ++e)
        f[e * DC] = fmaf(w, src[transposed ? (size_t)col * DA + r0 + e : (size_t)(r0 + e) * DC + col], f[e * DC]);
    };
    const int start = nearest_start_warp(p, it.b, p.rev ? hi : lo, tid & 31);
    // s = -1: the initial state; then the segments before this one on the pass's way
    for (int s = prefixed ? it.segs : -1; s < it.segs; s = s < 0 && p.rev ? it.seg + 1 : s + 1) {
      if (s >= 0 && !p.rev && s >= it.seg) break;
      const float w = reach(p, g, s, lo, hi, start);
      if (s < 0 && p.init && w >= 0.0f) add(p.init + bh * nstate, p.init_t, p.init_mul * w);
      if (s >= 0 && w >= 0.0f) add(p.seg_in + (bh * p.segs + s) * nstate, p.seg_t, w);
    }
    if (prefixed) add(p.seg_in + (bh * p.segs + it.seg) * nstate, p.seg_t, 1.0f);
  }
  const __nv_bfloat16* A = static_cast<const __nv_bfloat16*>(p.a) + (long long)it.b * p.T * p.lda + (long long)(it.h / p.ga) * DA;
  const __nv_bfloat16* B = static_cast<const __nv_bfloat16*>(p.b) + (long long)it.b * p.T * p.ldb + (long long)(it.h / p.gb) * DA;
  const __nv_bfloat16* C = static_cast<const __nv_bfloat16*>(p.c) + (long long)it.b * p.T * p.ldc + (long long)(it.h / p.gc) * DC;
  if (!meet()) return false;
#pragma unroll 1
  for (int n0 = 0; n0 < hi - lo; n0 += kWalk) {
    const int n = min(kWalk, hi - lo - n0);
    auto token = [&](int k) { return p.rev ? hi - 1 - n0 - k : lo + n0 + k; };
    const int word = token(0) / 32;  // the starts of the tokens lie in two words at most
    const uint32_t bits0 = starts ? starts[word] : 0u, bits1 = starts ? starts[token(n - 1) / 32] : 0u;
    // all of a thread's loads before its stores
    constexpr int PA = kWalk * DA / 256, PC = kWalk * DC / 256;
    float va[PA], vb[PA], vc[PC];
#pragma unroll
    for (int u = 0; u < PA; ++u) {
      const int i = tid + 256 * u, t = token(i / DA);
      va[u] = !STATE && i < n * DA ? to_f(A[t * p.lda + i % DA]) : 0.0f;
      vb[u] = i < n * DA ? to_f(B[t * p.ldb + i % DA]) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < PC; ++u) {
      const int i = tid + 256 * u;
      vc[u] = i < n * DC ? to_f(C[token(i / DC) * p.ldc + i % DC]) : 0.0f;
    }
#pragma unroll
    for (int u = 0; u < PA; ++u) {
      if constexpr (!STATE) sa[tid + 256 * u] = va[u];
      sb[tid + 256 * u] = vb[u];
    }
#pragma unroll
    for (int u = 0; u < PC; ++u) sc[tid + 256 * u] = vc[u];
    if (!meet()) return false;
#pragma unroll 1
    for (int k = 0; k < n; ++k) {
      const int t = token(k);
      const bool start = ((t / 32 == word ? bits0 : bits1) >> (t % 32) & 1u) != 0;
      // no decay before the last token, whose state's gradient comes in as it is
      const float keep = p.rev && t == p.T - 1 ? 1.0f : fade_next(gamma, left);
      const bool drop = keep == 0.0f || (!p.rev && start);
      const bool ends = p.rev && start;  // the document, on the way back
      const float c = sc[k * DC + col];
      float o = 0.0f;
#pragma unroll 1
      for (int e0 = 0; e0 < ROWS; e0 += 16) {  // all loads of 16 rows before their stores
        float x[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) x[e] = f[(e0 + e) * DC];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          x[e] = fmaf(sb[k * DA + r0 + e0 + e], c, drop ? 0.0f : keep * x[e]);
          if constexpr (!STATE) o = fmaf(sa[k * DA + r0 + e0 + e], x[e], o);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) f[(e0 + e) * DC] = ends ? 0.0f : x[e];
      }
      if constexpr (!STATE) so[(k * GROUPS + tid / DC) * DC + col] = o;
    }
    if (!meet()) return false;
    if constexpr (!STATE) {
#pragma unroll 1
      for (int i = tid; i < n * DC; i += 256) {
        const int k = i / DC, d = i % DC;
        float o = 0.0f;
#pragma unroll
        for (int q = 0; q < GROUPS; ++q) o += so[(k * GROUPS + q) * DC + d];
        const long long at = ((long long)it.b * p.T + token(k)) * p.ldo + (long long)it.h * DC + d;
        if (p.out_f32) static_cast<float*>(p.out)[at] = p.scale * o;
        else static_cast<__nv_bfloat16*>(p.out)[at] = __float2bfloat16_rn(p.scale * o);
      }
    }
  }
  const Last to = last_of<STATE>(p, it, g);
#pragma unroll 1
  for (int e = 0; to.dst && e < ROWS; ++e) to.dst[(size_t)(r0 + e) * DC + col] = to.none ? 0.0f : to.mul * f[e * DC];
  return true;
}

template <int DA, int DC, int KIND, bool FINE, bool BRIEF>
__global__ void __launch_bounds__(Cfg<DA, DC, KIND == STATES>::THREADS, 1) k_pass_tc(const __grid_constant__ TcArgs ta) {
  constexpr bool STATE = KIND == STATES;
  using Cf = Cfg<DA, DC, STATE>;
  using Mem = typename Cf::Mem;
  constexpr int NS = Cf::NS, SLOT = Cf::SLOT, NC = Cf::NC;
  const Pass& p = ta.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* a_buf = smem;                  // [2][SLOT], chunks in turn
  uint8_t* ring = smem + Mem::at_ring;    // [NS][SLOT]: b, c, b, c, ...
  uint8_t* lo_buf = smem + Mem::at_lo;
  uint8_t* f_buf = smem + Mem::at_f;
  float* tabs = reinterpret_cast<float*>(smem + Mem::at_tabs);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + Mem::at_bars);
  uint64_t *full = bars, *empty = bars + NS;
  // Pairs are taken in turn by even and odd chunks, where a waiter may be a chunk behind.
  uint64_t* sc_full = bars + 2 * NS;     // [2]
  uint64_t* conv_done = sc_full + 2;     // [2][2]: chunk, half of its tokens
  uint64_t* d_full = sc_full + 6;        // [2]
  uint64_t *a_full = sc_full + 8, *a_empty = sc_full + 10;  // [2]: the a buffers
  uint64_t *p_ready = sc_full + 12, *f_ready = sc_full + 13, *o_full = sc_full + 14, *o_free = sc_full + 15;
  uint64_t *tab_ready = sc_full + 16, *f_free = sc_full + 17, *drain = sc_full + 18;
  uint64_t *item_end = sc_full + 19, *all_done = sc_full + 20, *meet = sc_full + 21;
  uint64_t* lo_free = sc_full + 22;  // [2]
  static_assert(Mem::bars(NS) == 2 * NS + 24, "the barriers above");
  volatile uint32_t* words = reinterpret_cast<volatile uint32_t*>(smem + Mem::at_words);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) % 1024 != 0) {  // the swizzled tiles need it; uniform over the block
    if (threadIdx.x == 0) set_status(p.status, IPTTT_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], STATE ? 1 : 2);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sc_full[s], 1);
      mbar_init(&conv_done[2 * s], 8);
      mbar_init(&conv_done[2 * s + 1], 8);
      mbar_init(&d_full[s], 1);
      mbar_init(&lo_free[s], 1);
      mbar_init(&a_full[s], 1);
      mbar_init(&a_empty[s], 8);
    }
    mbar_init(p_ready, 8);
    mbar_init(f_ready, 8);
    mbar_init(f_free, 1);
    mbar_init(o_full, 1);
    mbar_init(o_free, 8);
    mbar_init(tab_ready, STATE ? 8 : 16);
    mbar_init(drain, STATE ? 1 : 2);
    mbar_init(item_end, 8);
    mbar_init(all_done, STATE ? 8 : 16);
    mbar_init(meet, 8);
    for (int w = W_ABORT; w < Mem::WORDS; ++w) words[w] = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    if (!STATE) {
      prefetch_tmap(&ta.ma);
      if (!p.out_f32) prefetch_tmap(&ta.mo);
    }
    prefetch_tmap(&ta.mb);
    prefetch_tmap(&ta.mc);
  }
  if (warp == 1) {
    tmem_alloc(reinterpret_cast<uint32_t*>(smem + Mem::at_words) + W_TMEM, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = words[W_TMEM];
  // The pass may start while the one for its segments' states still runs (it reads them at
  // its cut segments' starts, and ends after it in any case).
  if (STATE) launch_dependents();
  const bool rev = STATE ? p.rev != 0 : KIND == REVERSE;
  const int step = rev ? -1 : 1;
  // STATES has room for two chunks' lo halves and D, so that a chunk's scaling runs beside the last one's (4)
  constexpr uint32_t d_col = STATE ? 0 : col_d(DC), two_col = STATE ? DC : 0, two_lo = STATE ? 256 * DA / 16 : 0;
  auto mark_odd = [&](uint32_t n) { atomicOr(reinterpret_cast<uint32_t*>(smem + Mem::at_words) + W_ODD + n / 32, 1u << n % 32); };
  auto is_odd = [&](uint32_t n) { return (words[W_ODD + n / 32] >> n % 32 & 1u) != 0; };
  bool ok = true;
  // a wait that gives up ends the block's work: every role leaves its loops
#define LA_WAIT(bar, parity)                                  \
  if (!wait_for(bar, (parity) & 1u, words)) {           \
    ok = false;                                               \
    break;                                                    \
  }
  // of all lanes of a warp alike: what follows are warp-wide TMEM accesses
#define LA_WAIT_WARP(bar, parity)                                                      \
  if (!__all_sync(0xffffffffu, wait_for(bar, (parity) & 1u, words))) {           \
    ok = false;                                                                        \
    break;                                                                             \
  }

  if (warp < kOutWarp) {
    if constexpr (!STATE) regs_dec<kRegsIssue>();
    if (warp == 0 && lane == 0) {
      uint32_t tl = 0, cc = 0;
      auto load = [&](uint8_t* dst, const CUtensorMap* m, uint64_t* bar, int width, int x, int ch, int b) {
        mbar_arrive_expect_tx(bar, 256 * width);
        for (int q = 0; q < width / 64; ++q) tma_load_3d(dst + q * 16384, m, bar, x + 64 * q, ch * CH, b);
      };
      for (int i = blockIdx.x; ok && i < ta.items; i += gridDim.x) {
        const Item it = item_of(p, i);
        for (int n = 0; n < it.last - it.first; ++n, ++cc) {
          const int ch = rev ? it.last - 1 - n : it.first + n;
          LA_WAIT(&empty[tl % NS], (tl / NS) ^ 1u);
          load(ring + tl % NS * SLOT, &ta.mb, &full[tl % NS], DA, it.h / p.gb * DA, ch, it.b);
          ++tl;
          if constexpr (!STATE) {
            LA_WAIT(&a_empty[cc & 1], (cc >> 1) ^ 1u);
            load(a_buf + (cc & 1) * SLOT, &ta.ma, &a_full[cc & 1], DA, it.h / p.ga * DA, ch, it.b);
            words[W_A_TILES] = cc + 1;
          }
          LA_WAIT(&empty[tl % NS], (tl / NS) ^ 1u);
          load(ring + tl % NS * SLOT, &ta.mc, &full[tl % NS], DC, it.h / p.gc * DC, ch, it.b);
          ++tl;
        }
      }
      words[W_TILES] = tl;
    } else if ((warp == 1 || warp == 2) && lane == 0 && !(STATE && warp == 1)) {
      // Two threads issue the MMAs, warp 1's (1), (2) and (3), warp 2's (4): issuing takes longer than
      // the tensor pipe does, and (4) is on the path that bounds a chunk, from state to state.
      constexpr uint32_t id1 = idesc_bf16(128, 128, false, false), id2 = idesc_bf16(128, DC, false, true),
                         id3 = idesc_bf16(128, DC, false, true), id4 = idesc_bf16(128, DC, true, true);
      // width 64: rows 64-127 of (4) repeat rows 0-63 (the second block of 64 is the first)
      constexpr uint32_t lbo4 = DA == 128 ? 16384 : 0;
      // Descriptors of each tile's first K step; a step adds to the address field (16-byte
      // units).  Built once: made anew for each MMA they cost the issuing thread some 100
      // clocks a MMA, where the tensor pipe takes 64.
      auto k_major = [](const uint8_t* t) { return sdesc_sw128(smem_u32(t), 16, 1024); };
      auto mn_major = [](const uint8_t* t, uint32_t lbo) { return sdesc_sw128(smem_u32(t), lbo, 1024); };
      uint32_t total = 0;  // chunks this block walks
      for (int i = blockIdx.x; i < ta.items; i += gridDim.x) {
        const Item it = item_of(p, i);
        total += it.last - it.first;
      }
      const uint64_t c_mn = mn_major(ring, 16384);
      auto tile = [](uint32_t n) { return n % NS; };
      if (warp == 1) {
        const uint64_t a_k = k_major(a_buf), b_k = k_major(ring), f_mn = mn_major(f_buf, DA * 128);
        for (uint32_t c = 0; c < total; ++c) {
          const uint32_t sb = tile(2 * c), sc = tile(2 * c + 1);
          const uint64_t da = a_k + (c & 1) * (SLOT / 16), db = b_k + sb * (SLOT / 16), dc = c_mn + sc * (SLOT / 16);
          LA_WAIT(&full[sb], 2 * c / NS);
          LA_WAIT(&a_full[c & 1], c >> 1);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < DA / 16; ++k)
            mma_bf16(tm + kSC, da + (k / 4) * 1024 + (k % 4) * 2, db + (k / 4) * 1024 + (k % 4) * 2, id1, k > 0);
          mma_commit(&sc_full[c & 1]);
          mma_commit(&empty[sb]);
          LA_WAIT(f_ready, c);
          LA_WAIT(o_free, c ^ 1u);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < DA / 16; ++k)
            mma_bf16(tm + kO1, da + (k / 4) * 1024 + (k % 4) * 2, f_mn + k * 128, id2, k > 0);
          mma_commit(f_free);
          LA_WAIT(p_ready, c);
          LA_WAIT(&full[sc], (2 * c + 1) / NS);
          tc_fence_after();
          // P lies in columns 0-31 and 64-95 of the scores' place (BRIEF: its lower part in the latter)
#pragma unroll
          for (int k = 0; k < CH / 16; ++k)
            mma_bf16_ta(tm + col_o2(DC), tm + kSC + 8 * k + (k < 4 ? 0 : 32), dc + (BRIEF && k >= 4 ? k - 4 : k) * 128, id3, k > 0);
          mma_commit(&empty[sc]);
          mma_commit(o_full);
        }
      } else {
        const uint64_t b_mn = mn_major(ring, lbo4), lo_mn = mn_major(lo_buf, lbo4), part_mn = mn_major(lo_buf, lbo4 / 2);
        for (uint32_t c = 0; c < total; ++c) {
          const uint32_t sb = tile(2 * c), sc = tile(2 * c + 1);
          const uint64_t db = b_mn + sb * (SLOT / 16), dc = c_mn + sc * (SLOT / 16), dl = lo_mn + (c & 1) * two_lo;
          const uint32_t d = tm + d_col + two_col * (c & 1);
          LA_WAIT(&full[sc], (2 * c + 1) / NS);
          LA_WAIT(&conv_done[2 * (c & 1)], c >> 1);  // the first 64 tokens (and the last chunk's D has been read)
          tc_fence_after();
          if constexpr (FINE) {
            // the lower parts first: the next half's take their place meanwhile
            auto half = [&](int h) {
              const int slot = Mem::LO_SLOTS == 2 ? h : 0;
              const uint64_t l1 = part_mn + slot * (2 * Mem::LO_PART / 16), l2 = l1 + Mem::LO_PART / 16;
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_bf16(d, l1 + k * 128, dc + (4 * h + k) * 128, id4, h + k > 0);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_bf16(d, l2 + k * 128, dc + (4 * h + k) * 128, id4, 1);
              mma_commit(&lo_free[slot]);
#pragma unroll
              for (int k = 0; k < 4; ++k) mma_bf16(d, db + (4 * h + k) * 128, dc + (4 * h + k) * 128, id4, 1);
            };
            half(0);
            LA_WAIT(&conv_done[2 * (c & 1) + 1], c >> 1);
            tc_fence_after();
            half(1);
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16(d, db + k * 128, dc + k * 128, id4, k > 0);
#pragma unroll
            for (int k = 0; k < 4; ++k) mma_bf16(d, dl + k * 128, dc + k * 128, id4, 1);
            LA_WAIT(&conv_done[2 * (c & 1) + 1], c >> 1);
            tc_fence_after();
#pragma unroll
            for (int k = 4; k < 8; ++k) mma_bf16(d, db + k * 128, dc + k * 128, id4, 1);
#pragma unroll
            for (int k = 4; k < 8; ++k) mma_bf16(d, dl + k * 128, dc + k * 128, id4, 1);
          }
          mma_commit(&d_full[c & 1]);
          mma_commit(&empty[sb]);
          mma_commit(&empty[sc]);
        }
      }
      mma_commit(drain);
      mbar_wait(drain, 0);
    }
  } else if (warp < Cf::SW) {
    if constexpr (!STATE) {
      regs_dec<kRegsOut>();
      // two warps a quarter of the rows: each has 64 columns of the scores and half of the output's
      constexpr int HC = DC / 2;
      const int quarter = warp & 3, half = (warp - kOutWarp) >> 2, row = quarter * 32 + lane;
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      const uint32_t sc_addr = tm + kSC + lanes + 64 * half, o1_addr = tm + kO1 + lanes + HC * half,
                     o2_addr = tm + col_o2(DC) + lanes + HC * half;
      uint32_t cc = 0, ic = 0;
      for (int i = blockIdx.x; ok && i < ta.items; i += gridDim.x, ++ic) {
        const Item it = item_of(p, i);
        const float* pw = tabs + (ic & 1) * kTab + 128;
        if (lane == 0) mbar_arrive(tab_ready);
        LA_WAIT_WARP(tab_ready, ic);
        Starts next = starts_of(p, it.b, rev ? it.last - 1 : it.first);
        for (int n = 0; n < it.last - it.first; ++n, ++cc) {
          const int ch = rev ? it.last - 1 - n : it.first + n;
          const int t0 = ch * CH, len = min(CH, p.T - t0);
          const Starts st = next;  // read a chunk ahead
          if (n + 1 < it.last - it.first) next = starts_of(p, it.b, ch + step);
          const bool any = st.any();
          // the tokens the row looks at: [from, to); whether the state before the chunk reaches it
          int from = rev ? row : 0, to = rev ? CH : row + 1;
          bool in = true;
          if (any) {
            if (rev) {
              to = st.from(row + 1).first();
              in = row >= st.last();
            } else {
              from = st.below(row + 1).last();
              in = row < st.first();
            }
          }
          LA_WAIT_WARP(&sc_full[cc & 1], cc >> 1);
          if (cc > 0 && lane == 0) {  // the last chunk's output has left the a tile's place
            bulk_wait_read<0>();
            mbar_arrive(&a_empty[(cc - 1) & 1]);
          }
          __syncwarp();
          tc_fence_after();
          // 32 columns at a time; P takes the place of scores already read.  (Loops stay rolled:
          // unrolled, the roles' code overran the instruction caches, a third of all stalls.)
#pragma unroll 1
          for (int q = 0; q < (BRIEF && half == 1 ? 0 : 2); ++q) {
            const int block = 2 * half + q;
            uint32_t w[16];
            if (rev ? block < quarter : block > quarter) {  // on the other side of every row of the warp
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = 0u;
              tmem_st16(sc_addr + 16 * q, w);
              if constexpr (BRIEF) tmem_st16(sc_addr + 64 + 16 * q, w);
              continue;
            }
            uint32_t v[32];
            tmem_ld32(sc_addr + 32 * q, v);
            if (block == quarter) {  // the diagonal: gamma^|row - j|, 0 on the far side
              const float* wt = pw + (rev ? -lane : lane);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * wt[rev ? e : -e]);
            } else {  // a factor of the column times one of the row, neither above 1
              const float rf = rev ? pw[32 * block - row] : pw[row - 32 * block - 31];
              const float4* col = reinterpret_cast<const float4*>(rev ? pw : pw - 128 + kPw);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float4 c = col[e];
                v[4 * e] = __float_as_uint(__uint_as_float(v[4 * e]) * c.x * rf);
                v[4 * e + 1] = __float_as_uint(__uint_as_float(v[4 * e + 1]) * c.y * rf);
                v[4 * e + 2] = __float_as_uint(__uint_as_float(v[4 * e + 2]) * c.z * rf);
                v[4 * e + 3] = __float_as_uint(__uint_as_float(v[4 * e + 3]) * c.w * rf);
              }
            }
            auto masked = [&] {
              // bit j of the mask: column j of the block is in the row's document and on its side
              const int lo = min(max(from - 32 * block, 0), 32), hi = min(max(to - 32 * block, 0), 32);
              const uint32_t below_hi = hi == 32 ? 0xffffffffu : (1u << hi) - 1u;
              const uint32_t mask = lo == 32 ? 0u : below_hi & (0xffffffffu << lo);
#pragma unroll
              for (int e = 0; e < 16; ++e)
                w[e] &= (mask >> (2 * e) & 1u ? 0x0000ffffu : 0u) | (mask >> (2 * e) & 2u ? 0xffff0000u : 0u);
            };
#pragma unroll
            for (int e = 0; e < 16; ++e) w[e] = pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
            if (block == quarter) far_side_off(w, lane, rev);
            if constexpr (BRIEF) {  // what the rounding left, before either is masked
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                v[2 * e] = __float_as_uint(__uint_as_float(v[2 * e]) - __uint_as_float(w[e] << 16));
                v[2 * e + 1] = __float_as_uint(__uint_as_float(v[2 * e + 1]) - __uint_as_float(w[e] & 0xffff0000u));
              }
            }
            if (any) masked();
            tmem_st16(sc_addr + 16 * q, w);
            if constexpr (BRIEF) {
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = pack2(__uint_as_float(v[2 * e]), __uint_as_float(v[2 * e + 1]));
              if (block == quarter) far_side_off(w, lane, rev);
              if (any) masked();
              tmem_st16(sc_addr + 64 + 16 * q, w);
            }
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready);

          const int lag = rev && t0 + len == p.T ? 1 : 0;
          const bool write = row < len;
          const float win = in && write ? pw[rev ? len - row - lag : row + 1] : kNone;
          const float s1 = win * p.scale;
          // the output goes out through the a tile's place: (1) and (2) are done with it
          uint8_t* stage = a_buf + (cc & 1) * SLOT + half * (256 * HC);
          LA_WAIT_WARP(o_full, cc);
          tc_fence_after();
#pragma unroll 1
          for (int q = 0; q < HC / 16; ++q) {
            uint32_t x[16], y[16];
            tmem_ld16(o2_addr + 16 * q, x);
            tmem_ld16(o1_addr + 16 * q, y);
            tmem_ld_wait();
            float o[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = p.scale * __uint_as_float(x[e]);
            if (!any || win >= 0.0f) {  // rows of another document take nothing of the state, whatever is in it
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = fmaf(s1, __uint_as_float(y[e]), o[e]);
            }
            if (p.out_f32) {
              if (write) {
                float4* g = reinterpret_cast<float4*>(static_cast<float*>(p.out) +
                                                      ((long long)it.b * p.T + t0 + row) * p.ldo + (long long)it.h * DC +
                                                      HC * half + 16 * q);
#pragma unroll
                for (int e = 0; e < 4; ++e) g[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
              }
            } else {  // rows of HC columns, swizzled as the store's map is
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int unit = (2 * q + e) ^ (HC == 64 ? row & 7 : (row >> 1) & 3);
                *reinterpret_cast<uint4*>(stage + row * (2 * HC) + unit * 16) =
                    make_uint4(pack2(o[8 * e], o[8 * e + 1]), pack2(o[8 * e + 2], o[8 * e + 3]),
                               pack2(o[8 * e + 4], o[8 * e + 5]), pack2(o[8 * e + 6], o[8 * e + 7]));
              }
            }
            __syncwarp();
          }
          tc_fence_before();  // the accumulators are free
          __syncwarp();
          if (lane == 0) mbar_arrive(o_free);
          if (!p.out_f32) {
            fence_proxy_async_smem();
            __syncwarp();
            const int t = t0 + 32 * quarter;  // rows past T are left out by the map
            if (lane == 0 && t < p.T) {
              tma_store_3d(&ta.mo, stage + quarter * (64 * HC), it.h * DC + HC * half, t, it.b);
              bulk_commit();
            }
          }
        }
      }
      if (lane == 0) {
        bulk_wait<0>();
        mbar_arrive(all_done);
      }
    }
  } else {
    if constexpr (!STATE) regs_inc<kRegsState>();
    const int tid = threadIdx.x - Cf::SW * 32;
    const int quarter = warp & 3, half = (warp - Cf::SW) >> 2;
    const int row = DA == 128 ? quarter * 32 + lane : (quarter & 1) * 32 + lane;
    const int c0 = (DA == 128 ? half : half * 2 + (quarter >> 1)) * NC;  // its columns: [c0, c0 + NC)
    const uint32_t d_addr = tm + d_col + ((uint32_t)(quarter * 32) << 16) + c0;
    uint32_t tl = 0, cc = 0, ic = 0, in_place = 0;
    float f[NC];
    for (int i = blockIdx.x; ok && i < ta.items; i += gridDim.x, ++ic) {
      const Item it = item_of(p, i);
      const size_t bh = (size_t)it.b * p.H + it.h;
      const float g = p.log_decay[it.h];
      if (tid == 0 && !(g <= 0.0f)) set_status(p.status, IPTTT_ERR_ARG);
      float* pw = tabs + (ic & 1) * kTab + 128;
      pw[tid - 128] = tid < 128 ? 0.0f : decay_pow(g, tid - 128);
      if (tid < 32) pw[kPw - 128 + tid] = decay_pow(g, 31 - tid);
      if (tid == 32) {
        if constexpr (FINE) {
          const Fade fd = fade_of(g, CH);
          pw[128] = fd.hi;
          pw[129] = fd.lo;
          pw[130] = fd.inv;
        } else {
          pw[128] = decay_pow(g, 128);
        }
      }
      float left = 0.0f;
      __syncwarp();
      if (lane == 0) mbar_arrive(tab_ready);
      const int lo = it.first * CH, hi = min(p.T, it.last * CH);

#pragma unroll
      for (int e = 0; e < NC; ++e) f[e] = 0.0f;
      if constexpr (!STATE) {
        const bool prefixed = p.prefixed && it.segs > 1;
        const int start = !prefixed && (p.init || it.segs > 1) ? nearest_start_warp(p, it.b, rev ? hi : lo, lane) : 0;
        auto add = [&](const float* src, int transposed, float w) {
          if (transposed) {
#pragma unroll
            for (int e = 0; e < NC; ++e) f[e] = fmaf(w, src[(size_t)(c0 + e) * DA + row], f[e]);
          } else {
#pragma unroll
            for (int e = 0; e < NC; e += 4) {
              const float4 x = *reinterpret_cast<const float4*>(src + (size_t)row * DC + c0 + e);
              f[e] = fmaf(w, x.x, f[e]);
              f[e + 1] = fmaf(w, x.y, f[e + 1]);
              f[e + 2] = fmaf(w, x.z, f[e + 2]);
              f[e + 3] = fmaf(w, x.w, f[e + 3]);
            }
          }
        };
        if (p.init && !prefixed) {
          const float w = reach(p, g, -1, lo, hi, start);
          if (w >= 0.0f) add(p.init + bh * DA * DC, p.init_t, p.init_mul * w);
        }
        const int s0 = rev ? it.seg + 1 : 0, s1 = rev ? it.segs : it.seg;
        if (s0 < s1 || prefixed) wait_for_launch_before();
        if (prefixed) add(p.seg_in + (bh * p.segs + it.seg) * DA * DC, p.seg_t, 1.0f);
        for (int s = s0; s < s1 && !prefixed; ++s) {
          const float w = reach(p, g, s, lo, hi, start);
          if (w >= 0.0f) add(p.seg_in + (bh * p.segs + s) * DA * DC, p.seg_t, w);
        }
      }
      LA_WAIT_WARP(tab_ready, ic);

      // Masked places of b and c are multiplied by 0.  That is NaN for a value that is not finite: whatever
      // its weight, D is then not finite, nor is the state until a document starts.  An item that met
      // one is done again, by the recurrence itself.  (One of a touches its own row alone, where it
      // belongs.)
      auto look = [&] {
        float odd = 0.0f;
#pragma unroll
        for (int e = 0; e < NC; ++e) odd = fmaf(f[e], 0.0f, odd);
        if (isnan(odd)) mark_odd(ic);
      };
      // f <- keep f + D of chunk number c
      auto advance = [&](float keep, uint32_t c) {
        tc_fence_after();
        const uint32_t addr = d_addr + two_col * (c & 1);
        if (keep < 0.0f) {  // whatever f holds
          look();
          __syncwarp();  // what follows is of the whole warp
          keep = 0.0f;
#pragma unroll
          for (int e = 0; e < NC; ++e) f[e] = 0.0f;
        }
        constexpr int STEP = NC < 32 ? NC : 32;
#pragma unroll
        for (int q = 0; q < NC / STEP; ++q) {
          uint32_t r[STEP];
          if constexpr (STEP == 16) tmem_ld16(addr + STEP * q, r);
          else tmem_ld32(addr + STEP * q, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < STEP; ++e) f[STEP * q + e] = fmaf(keep, f[STEP * q + e], __uint_as_float(r[e]));
        }
      };
      // each row's weight in a chunk as wh + wl (FINE: + wm) in bf16; a thread's 16-byte units lie in four
      // rows, two a half chunk
      __nv_bfloat162 wh[2], wl[2], wm[FINE ? 2 : 1];
      auto half_of = [](__nv_bfloat162 x, int i) { return i == 0 ? __low2bfloat162(x) : __high2bfloat162(x); };
      auto weights = [&](int ch, const Starts& st) {
        const int len = min(CH, p.T - ch * CH);
        // rows that reach the state at the chunk's far end
        const int from = rev ? 0 : st.last(), to = rev ? min(len, st.first()) : len;
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          float w[2], x[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int j = (tid >> 3) + 32 * (2 * m + i);
            w[i] = j >= from && j < to ? pw[rev ? j : len - 1 - j] : 0.0f;
            if constexpr (FINE) {  // the nearest power of two first
              x[i] = __uint_as_float((__float_as_uint(w[i]) + 0x00400000u) & 0x7f800000u);
              w[i] -= x[i];
            }
          }
          if constexpr (FINE) wm[m] = __floats2bfloat162_rn(x[0], x[1]);
          wh[m] = __floats2bfloat162_rn(w[0], w[1]);
          wl[m] = __floats2bfloat162_rn(w[0] - __low2float(wh[m]), w[1] - __high2float(wh[m]));
        }
      };
      float keep = 0.0f;
      Starts next = starts_of(p, it.b, rev ? it.last - 1 : it.first);
      weights(rev ? it.last - 1 : it.first, next);
      for (int n = 0; n < it.last - it.first; ++n, ++cc, tl += 2) {
        const int ch = rev ? it.last - 1 - n : it.first + n;
        const int t0 = ch * CH, len = min(CH, p.T - t0);
        const Starts st = next;  // read a chunk ahead
        if (n + 1 < it.last - it.first) next = starts_of(p, it.b, ch + step);
        const bool any = st.any();
        const int lag = rev && t0 + len == p.T ? 1 : 0;
        const uint32_t sb = tl % NS;
        if constexpr (!STATE) {
          // the operand copy of the state, [Dc / 64][Da][64] in 128-byte swizzled rows, once the last
          // chunk's (2) has read the old one
          if (cc > 0) LA_WAIT_WARP(f_free, cc - 1);
          uint8_t* fb = f_buf + (c0 / 64) * (DA * 128) + row * 128;
#pragma unroll
          for (int e = 0; e < NC / 8; ++e) {
            const int unit = (c0 % 64) / 8 + e;
            *reinterpret_cast<uint4*>(fb + ((unit ^ (row & 7)) * 16)) =
                make_uint4(pack2(f[8 * e], f[8 * e + 1]), pack2(f[8 * e + 2], f[8 * e + 3]),
                           pack2(f[8 * e + 4], f[8 * e + 5]), pack2(f[8 * e + 6], f[8 * e + 7]));
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(f_ready);
        }
        LA_WAIT_WARP(&full[sb], tl / NS);
        uint8_t* bt = ring + sb * SLOT + tid * 16;
        uint8_t* lt = lo_buf + (cc & 1) * (two_lo * 16) + tid * 16;
        if constexpr (!STATE) LA_WAIT_WARP(&sc_full[cc & 1], cc >> 1);  // (1) has read B: it may be overwritten
        // hi = bf16(b wh); b wh - hi is a bf16 number, so lo = bf16(b wl + (b wh - hi)) loses 2^-8 of lo
        // alone.  FINE: b times the power of two, exact, in b's place, and hi and lo of the rest, a third of the
        // weight at most.  64 tokens at a time: the first half's (4) starts while the second is scaled.
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          constexpr int SLOTS = Mem::LO_SLOTS;
          const int slot = SLOTS == 2 ? half : 0;
          uint4 v[DA / 32];
#pragma unroll
          for (int m = 0; m < DA / 32; ++m)
            v[m] = *reinterpret_cast<const uint4*>(bt + (2 * half + (m & 1) + 4 * (m >> 1)) * 4096);
          if constexpr (FINE) {
            // the exact parts first, while the half chunk before is multiplied out of the others' place
#pragma unroll
            for (int m = 0; m < DA / 32; ++m) {
              const __nv_bfloat162 top = half_of(wm[half], m & 1);
              const uint32_t u[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
              uint32_t t[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const __nv_bfloat162 t2 = __hmul2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]), top);
                t[e] = *reinterpret_cast<const uint32_t*>(&t2);
              }
              *reinterpret_cast<uint4*>(bt + (2 * half + (m & 1) + 4 * (m >> 1)) * 4096) = make_uint4(t[0], t[1], t[2], t[3]);
            }
            if (2 * cc + half >= SLOTS) LA_WAIT_WARP(&lo_free[slot], (2 * cc + half) / SLOTS - 1);
          }
#pragma unroll
          for (int m = 0; m < DA / 32; ++m) {
            const __nv_bfloat162 h = half_of(wh[half], m & 1), l = half_of(wl[half], m & 1);
            const uint32_t u[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
            uint32_t hi4[4], lo4[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const __nv_bfloat162 x = *reinterpret_cast<const __nv_bfloat162*>(&u[e]);
              const __nv_bfloat162 h2 = __hmul2(x, h);
              const __nv_bfloat162 l2 = __hfma2(x, l, __hfma2(x, h, __hneg2(h2)));
              hi4[e] = *reinterpret_cast<const uint32_t*>(&h2);
              lo4[e] = *reinterpret_cast<const uint32_t*>(&l2);
            }
            const int at = (2 * half + (m & 1) + 4 * (m >> 1)) * 4096, in_part = ((m & 1) + 2 * (m >> 1)) * 4096;
            uint8_t* hi_at = FINE ? lo_buf + slot * (2 * Mem::LO_PART) + tid * 16 + in_part : bt + at;
            uint8_t* lo_at = FINE ? hi_at + Mem::LO_PART : lt + at;
            *reinterpret_cast<uint4*>(hi_at) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
            *reinterpret_cast<uint4*>(lo_at) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
          }
          fence_proxy_async_smem();
          tc_fence_before();  // the last chunk's D has been read
          __syncwarp();
          if (lane == 0) mbar_arrive(&conv_done[2 * (cc & 1) + half]);
        }
        if (FINE && !ok) break;
        float keep_now = pw[len - lag];
        if (FINE && len - lag == CH) keep_now = fade_next({keep_now, pw[129], pw[130]}, left);
        if (any) keep_now = kNone;
        if (n + 1 < it.last - it.first) weights(ch + step, next);
        if constexpr (STATE) {
          if (n > 0) {
            LA_WAIT_WARP(&d_full[(cc - 1) & 1], (cc - 1) >> 1);
            advance(keep, cc - 1);
          }
          keep = keep_now;
        } else {
          LA_WAIT_WARP(&d_full[cc & 1], cc >> 1);
          advance(keep_now, cc);
        }
      }
      if (!ok) break;
      if constexpr (STATE) {
        LA_WAIT_WARP(&d_full[(cc - 1) & 1], (cc - 1) >> 1);
        advance(keep, cc - 1);
      }
      if (!ok) break;
      look();
      __syncwarp();
      const Last to = last_of<STATE>(p, it, g);
      bool write = to.dst != nullptr;
      if (!STATE && write && p.fin == p.init && it.segs == 1) {
        // an item that is done again starts from the state that this would replace
        if (lane == 0) mbar_arrive(item_end);
        LA_WAIT_WARP(item_end, in_place);
        ++in_place;
        write = !is_odd(ic);
      }
      if (write) {
        float* dst = to.dst + (size_t)row * DC + c0;
#pragma unroll
        for (int e = 0; e < NC; e += 4)
          *reinterpret_cast<float4*>(dst + e) = make_float4(to.mul * f[e], to.mul * f[e + 1], to.mul * f[e + 2], to.mul * f[e + 3]);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(all_done);
    do {  // (left by a wait that gives up)
      if (!ok) break;
      LA_WAIT_WARP(all_done, 0);  // the outputs have been written
      uint32_t met = 0;
#pragma unroll 1
      for (uint32_t w = 0; ok && 32 * w < ic; ++w) {
#pragma unroll 1
        for (uint32_t bits = words[W_ODD + w]; ok && bits != 0; bits &= bits - 1) {
          const int k = 32 * (int)w + __ffs(bits) - 1;
          ok = walk<DA, DC, STATE>(p, item_of(p, blockIdx.x + k * gridDim.x), reinterpret_cast<float*>(smem),
                                   reinterpret_cast<float*>(lo_buf), tid, meet, met, words);
        }
      }
    } while (false);
  }
#undef LA_WAIT
#undef LA_WAIT_WARP
  if (!ok) {
    words[W_ABORT] = 1;
    set_status(p.status, IPTTT_ERR_TIMEOUT);
  }

  __syncthreads();
  if (!STATE && threadIdx.x == 0) wait_for_launch_before();
  if (words[W_ABORT] && threadIdx.x == 0) {
    // copies that were issued land before the block's shared memory is given back
    const uint32_t n = words[W_TILES], na = words[W_A_TILES];
    for (uint32_t t = n > (uint32_t)NS ? n - NS : 0; t < n; ++t) mbar_wait(&full[t % NS], (t / NS) & 1);
    for (uint32_t t = na > 2 ? na - 2 : 0; t < na; ++t) mbar_wait(&a_full[t & 1], (t >> 1) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

template <int DA, int DC, int KIND, bool FINE, bool BRIEF>
cudaError_t launch(const TcArgs& a, cudaStream_t st) {
  using Cf = Cfg<DA, DC, KIND == STATES>;
  // once a device: the shared memory, and a check of the registers.  The register split takes what
  // the launch gives: with less, the state's warps would wait for good.
  static std::atomic<bool> ready[64];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev].load()) {
    e = cudaFuncSetAttribute(k_pass_tc<DA, DC, KIND, FINE, BRIEF>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cf::SMEM);
    if (e != cudaSuccess) return e;
    cudaFuncAttributes at;
    e = cudaFuncGetAttributes(&at, k_pass_tc<DA, DC, KIND, FINE, BRIEF>);
    if (e != cudaSuccess) return e;
    if (KIND != STATES && at.numRegs < kRegsLaunch) return cudaErrorInvalidConfiguration;
    ready[dev].store(true);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  const int blocks = std::min(a.items, device_sms());
  if (blocks <= 0 || (a.items + blocks - 1) / blocks > kMostItems) return cudaErrorInvalidConfiguration;
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(Cf::THREADS);
  cfg.dynamicSmemBytes = Cf::SMEM;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = a.p.after_states ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, k_pass_tc<DA, DC, KIND, FINE, BRIEF>, a);
}

// Rows of up to 64 tokens leave half of P's place empty: it takes what the rounding of P to bf16 left
// (BRIEF).  In short rows that rounding is common to a row of o and does not average out: one
// token's o = scale (q . k) v would be off by up to 2^-8 as a whole, besides its own rounding.
template <int DA, int DC, bool FINE, bool BRIEF>
cudaError_t launch(const TcArgs& a, cudaStream_t st) {
  return a.p.rev ? launch<DA, DC, REVERSE, FINE, BRIEF>(a, st) : launch<DA, DC, FORWARD, FINE, BRIEF>(a, st);
}

template <int DA, int DC, bool FINE>
cudaError_t launch(const TcArgs& a, cudaStream_t st) {
  if (!a.p.out) return launch<DA, DC, STATES, FINE, false>(a, st);
  return a.p.T <= CH / 2 ? launch<DA, DC, FINE, true>(a, st) : launch<DA, DC, FINE, false>(a, st);
}

template <int DA, int DC>
cudaError_t launch(const TcArgs& a, cudaStream_t st) {
  return a.p.fine ? launch<DA, DC, true>(a, st) : launch<DA, DC, false>(a, st);
}

}  // namespace

bool tc_takes(int Da, int Dc) { return (Da == 64 || Da == 128) && (Dc == 64 || Dc == 128); }

int tc_segments(int B, int T, int H, int* seg_chunks, int* whole) {
  const int n = (T + CH - 1) / CH;
  const long long bh = (long long)B * H, sms = 148;
  // Time in quarters of a chunk of the full pass: what the busiest SM walks, an item's start
  // taken as 1.5 chunks, the pass for the segments' states at half the time a chunk, and
  // its launch as one chunk.  Pairs that fill the SMs evenly stay whole; the rest
  // are cut into the number of segments that comes out fastest.
  auto cost = [&](long long uncut, int segs) {
    const long long cut = bh - uncut, each = (n + segs - 1) / segs;
    const long long waves = (cut * segs + sms - 1) / sms, waves_s = (cut * (segs - 1) + sms - 1) / sms;
    return (uncut + sms - 1) / sms * (4 * n + 6) + waves * (4 * each + 6) + (segs > 1 && cut ? waves_s * (2 * each + 6) + 4 : 0);
  };
  const long long even = bh / sms * sms;
  long long best = cost(0, 1);
  int segs = 1;
  *whole = 0;
  for (int s = 2; s <= std::min(n, 148); ++s)
    for (long long u : {0ll, even})
      if (u < bh && cost(u, s) < best) {
        best = cost(u, s);
        segs = s;
        *whole = (int)u;
      }
  *seg_chunks = (n + segs - 1) / segs;
  return (n + *seg_chunks - 1) / *seg_chunks;
}

cudaError_t run_tc(const Pass& p, cudaStream_t st) {
  TcArgs a = {};  // (a map that the pass does not use stays empty)
  a.p = p;
  a.items = (p.B * p.H - p.whole) * (p.out ? p.segs : p.segs - 1) + (p.out ? p.whole : 0);
  if (a.items <= 0) return cudaSuccess;
  auto map = [&](CUtensorMap* m, const void* base, long long ld, int g, int width) {
    return tck::make_map_bf16_ld(m, base, (uint64_t)(p.H / g) * width, p.T, p.B, ld, 64, CH);
  };
  if (p.out && !map(&a.ma, p.a, p.lda, p.ga, p.Da)) return cudaErrorInvalidValue;
  if (p.out && !p.out_f32 &&
      !tck::make_map_bf16_ld(&a.mo, p.out, (uint64_t)p.H * p.Dc, p.T, p.B, p.ldo, p.Dc / 2, 32, p.Dc == 64))
    return cudaErrorInvalidValue;
  if (!map(&a.mb, p.b, p.ldb, p.gb, p.Da) || !map(&a.mc, p.c, p.ldc, p.gc, p.Dc)) return cudaErrorInvalidValue;
  if (p.Da == 128) return p.Dc == 128 ? launch<128, 128>(a, st) : launch<128, 64>(a, st);
  return p.Dc == 128 ? launch<64, 128>(a, st) : launch<64, 64>(a, st);
}

}  // namespace la
}  // namespace ipttt
