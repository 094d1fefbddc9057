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
// decay to the chunk's end, is split in two bf16 halves (hi + lo, 2^-17 relative), so
// the fp32 state is good to fp32-like accuracy; P and the operand copy of F are
// rounded to bf16 once, like the inputs and outputs are.
// Roles: warp 0 issues the TMA loads into a ring of tiles, one thread of warp 1 the
// MMAs; warps 2-5 turn SC into P and write the output; warps 6-13 scale and split B
// in place, hold the state (a row and a strip of columns a thread) and write its bf16
// copy, the B operand of the next chunk's (2).
// Per chunk of width 128: 131 KB of HBM traffic (20 us a GB/s per SM: 3.0 us at the
// measured copy bandwidth over 148 SMs) against some 2600 clocks (1.4 us) of tensor
// pipe, so HBM bounds it as long as the loads run ahead: the ring holds 5 tiles of 32 KB.
#include <cuda_bf16.h>

#include <algorithm>

#include "linattn.h"
#include "tc.cuh"
#include "tc_kernels.h"

namespace ipttt {
namespace la {

using namespace ipttt::tc;

namespace {

constexpr int CH = kTcChunk;
constexpr int kStateWarp = 6;  // warps 2-5: scores and output; from here: the state
constexpr int kTcThreads = 14 * 32;
constexpr int kTab = 256;  // tab[127 + n] = gamma^n for 0 <= n <= 128, 0 below

template <int DA, int DC, bool STATE>
struct Cfg {
  static constexpr int SLOT = 256 * (DA > DC ? DA : DC);
  static constexpr int LO = 256 * DA;                // lo half of the scaled B
  static constexpr int FB = STATE ? 0 : DA * DC * 2;  // bf16 state
  static constexpr int MISC = 2 * kTab * 4 + 512;
  static constexpr int FIT = (232448 - LO - FB - MISC) / SLOT;
  static constexpr int NS = FIT < 8 ? FIT : 8;
  static constexpr int SMEM = NS * SLOT + LO + FB + MISC;
  static constexpr int NC = DA * DC / 256;           // state columns a thread holds
  static constexpr int TPC = STATE ? 2 : 3;          // tiles a chunk
};
// TMEM columns
constexpr int kSC = 0, kO1 = 128;
__host__ __device__ constexpr int col_o2(int dc) { return 128 + dc; }
__host__ __device__ constexpr int col_d(int dc) { return 128 + 2 * dc; }

struct TcArgs {
  CUtensorMap ma, mb, mc;
  Pass p;
  int items;
};

struct Item {
  int b, h, seg, first, last;  // chunks [first, last)
};

__device__ __forceinline__ Item item_of(const Pass& p, int i) {
  Item t;
  t.h = i % p.H;
  const int r = i / p.H;
  // a pass for states alone leaves out the segment that nothing follows
  const int segs = p.out ? p.segs : p.segs - 1;
  t.seg = r % segs + (!p.out && p.rev ? 1 : 0);
  t.b = r / segs;
  const int n = (p.T + CH - 1) / CH;
  t.first = t.seg * p.seg_chunks;
  t.last = min(n, t.first + p.seg_chunks);
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

// nearest_start for one warp (every lane gets it).
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

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

template <int N>
__device__ __forceinline__ void tmem_load(uint32_t addr, uint32_t (&r)[N]) {
  if constexpr (N == 16) tmem_ld16(addr, r);
  else tmem_ld32(addr, r);
}

template <int DA, int DC, bool STATE>
__global__ void __launch_bounds__(kTcThreads, 1) k_pass_tc(const __grid_constant__ TcArgs ta) {
  using Cf = Cfg<DA, DC, STATE>;
  constexpr int NS = Cf::NS, SLOT = Cf::SLOT, TPC = Cf::TPC, NC = Cf::NC;
  const Pass& p = ta.p;
  extern __shared__ __align__(1024) uint8_t smem[];
  uint8_t* lo_buf = smem + NS * SLOT;
  uint8_t* f_buf = lo_buf + Cf::LO;
  float* tabs = reinterpret_cast<float*>(f_buf + Cf::FB);
  uint64_t* bars = reinterpret_cast<uint64_t*>(tabs + 2 * kTab);
  uint64_t *full = bars, *empty = bars + NS;
  uint64_t *sc_full = bars + 2 * NS, *p_ready = sc_full + 1, *conv_done = sc_full + 2, *d_full = sc_full + 3;
  uint64_t *f_ready = sc_full + 4, *o_full = sc_full + 5, *o_free = sc_full + 6, *tab_ready = sc_full + 7;
  uint64_t* drain = sc_full + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  uint32_t* issued = tmem_slot + 2;  // tiles whose loads were issued

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (smem_u32(smem) % 1024 != 0) {  // the swizzled tiles need it; uniform over the block
    if (threadIdx.x == 0) set_status(p.status, IPTTT_ERR_CUDA);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < NS; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(sc_full, 1);
    mbar_init(p_ready, 4);
    mbar_init(conv_done, 8);
    mbar_init(d_full, 1);
    mbar_init(f_ready, 8);
    mbar_init(o_full, 1);
    mbar_init(o_free, 4);
    mbar_init(tab_ready, STATE ? 8 : 12);
    mbar_init(drain, 1);
    *abort_flag = 0;
    *issued = 0;
    fence_mbar_init();
  }
  if (warp == 0 && lane == 0) {
    if (!STATE) prefetch_tmap(&ta.ma);
    prefetch_tmap(&ta.mb);
    prefetch_tmap(&ta.mc);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tm = *tmem_slot;
  bool ok = true;
  // a wait that gives up ends the block's work: every role leaves its loops
#define LA_WAIT(bar, parity)                                  \
  if (!mbar_wait_or_abort(bar, (parity) & 1u, abort_flag)) { \
    ok = false;                                               \
    break;                                                    \
  }

  // of all lanes of a warp alike: what follows are warp-wide TMEM accesses
#define LA_WAIT_WARP(bar, parity)                                                            \
  if (!__all_sync(0xffffffffu, mbar_wait_or_abort(bar, (parity) & 1u, abort_flag))) { \
    ok = false;                                                                              \
    break;                                                                                   \
  }

  if (warp == 0) {
    if (lane == 0) {
      uint32_t tl = 0;
      for (int i = blockIdx.x; ok && i < ta.items; i += gridDim.x) {
        const Item it = item_of(p, i);
        for (int n = 0; ok && n < it.last - it.first; ++n) {
          const int ch = p.rev ? it.last - 1 - n : it.first + n;
          for (int k = 0; k < TPC; ++k, ++tl) {
            const int s = tl % NS;
            LA_WAIT(&empty[s], (tl / NS) ^ 1u);
            const bool is_a = !STATE && k == 1, is_c = k == TPC - 1;
            const CUtensorMap* m = is_a ? &ta.ma : is_c ? &ta.mc : &ta.mb;
            const int width = is_c ? DC : DA;
            const int x = it.h / (is_a ? p.ga : is_c ? p.gc : p.gb) * width;
            mbar_arrive_expect_tx(&full[s], 256 * width);
            for (int q = 0; q < width / 64; ++q)
              tma_load_3d(smem + s * SLOT + q * 16384, m, &full[s], x + 64 * q, ch * CH, it.b);
          }
        }
      }
      *issued = tl;
      if (!ok) {
        *abort_flag = 1;
        set_status(p.status, IPTTT_ERR_TIMEOUT);
      }
    }
  } else if (warp == 1) {
    if (lane == 0) {
      constexpr uint32_t id1 = idesc_bf16(128, 128, false, false), id2 = idesc_bf16(128, DC, false, true),
                         id3 = idesc_bf16(128, DC, false, true), id4 = idesc_bf16(128, DC, true, true);
      // width 64: rows 64-127 of (4) repeat rows 0-63 (the second block of 64 is the first)
      constexpr uint32_t lbo4 = DA == 128 ? 16384 : 0;
      const uint32_t base = smem_u32(smem), lo_addr = smem_u32(lo_buf), f_addr = smem_u32(f_buf);
      uint32_t tl = 0, cc = 0;
      for (int i = blockIdx.x; ok && i < ta.items; i += gridDim.x) {
        const Item it = item_of(p, i);
        for (int n = it.first; ok && n < it.last; ++n, ++cc, tl += TPC) {
          const uint32_t sb = tl % NS, sa = (tl + 1) % NS, sc = (tl + TPC - 1) % NS;
          const uint32_t ab = base + sb * SLOT, aa = base + sa * SLOT, ac = base + sc * SLOT;
          if constexpr (!STATE) {
            LA_WAIT(&full[sb], tl / NS);
            LA_WAIT(&full[sa], (tl + 1) / NS);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < DA / 16; ++k)
              mma_bf16(tm + kSC, sdesc_sw128(aa + (k / 4) * 16384 + (k % 4) * 32, 16, 1024),
                       sdesc_sw128(ab + (k / 4) * 16384 + (k % 4) * 32, 16, 1024), id1, k > 0);
            mma_commit(sc_full);
            LA_WAIT(f_ready, cc);
            LA_WAIT(o_free, cc ^ 1u);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < DA / 16; ++k)
              mma_bf16(tm + kO1, sdesc_sw128(aa + (k / 4) * 16384 + (k % 4) * 32, 16, 1024),
                       sdesc_sw128(f_addr + k * 2048, DA * 128, 1024), id2, k > 0);
            mma_commit(&empty[sa]);
          }
          LA_WAIT(conv_done, cc);
          LA_WAIT(&full[sc], (tl + TPC - 1) / NS);
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < CH / 16; ++k)
            mma_bf16(tm + col_d(DC), sdesc_sw128(ab + k * 2048, lbo4, 1024), sdesc_sw128(ac + k * 2048, 16384, 1024), id4,
                     k > 0);
#pragma unroll
          for (int k = 0; k < CH / 16; ++k)
            mma_bf16(tm + col_d(DC), sdesc_sw128(lo_addr + k * 2048, lbo4, 1024), sdesc_sw128(ac + k * 2048, 16384, 1024),
                     id4, 1);
          mma_commit(&empty[sb]);
          if constexpr (STATE) mma_commit(&empty[sc]);
          mma_commit(d_full);
          if constexpr (!STATE) {
            LA_WAIT(p_ready, cc);
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < CH / 16; ++k)
              mma_bf16_ta(tm + col_o2(DC), tm + kSC + 8 * k, sdesc_sw128(ac + k * 2048, 16384, 1024), id3, k > 0);
            mma_commit(&empty[sc]);
            mma_commit(o_full);
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        set_status(p.status, IPTTT_ERR_TIMEOUT);
      }
      mma_commit(drain);
      mbar_wait(drain, 0);
    }
  } else if (warp < kStateWarp) {
    if constexpr (!STATE) {
      const int quarter = warp & 3, row = quarter * 32 + lane;
      const uint32_t lanes = (uint32_t)(quarter * 32) << 16;
      uint32_t cc = 0, ic = 0;
      for (int i = blockIdx.x; ok && i < ta.items; i += gridDim.x, ++ic) {
        const Item it = item_of(p, i);
        const float* tab = tabs + (ic & 1) * kTab;
        if (lane == 0) mbar_arrive(tab_ready);
        LA_WAIT_WARP(tab_ready, ic);
        for (int n = 0; n < it.last - it.first; ++n, ++cc) {
          const int ch = p.rev ? it.last - 1 - n : it.first + n;
          const int t0 = ch * CH, len = min(CH, p.T - t0);
          const Starts st = starts_of(p, it.b, ch);
          const bool any = st.any();
          // the tokens the row looks at: [from, to)
          int from = p.rev ? row : 0, to = p.rev ? CH : row + 1;
          bool in = true;
          if (any) {
            if (p.rev) {
              to = st.from(row + 1).first();
              in = row >= st.last();
            } else {
              from = st.below(row + 1).last();
              in = row < st.first();
            }
          }
          LA_WAIT_WARP(sc_full, cc);
          tc_fence_after();
          const float* wt = tab + 127 + (p.rev ? -row : row);
          const int dir = p.rev ? 1 : -1;
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            uint32_t w[16];
            if (p.rev ? q < quarter : q > quarter) {  // wholly on the other side of every row of the warp
#pragma unroll
              for (int e = 0; e < 16; ++e) w[e] = 0u;
            } else {
              uint32_t r[32];
              tmem_ld32(tm + kSC + lanes + 32 * q, r);
              tmem_ld_wait();
#pragma unroll
              for (int e = 0; e < 16; ++e) {
                const int j = 32 * q + 2 * e;
                float x = __uint_as_float(r[2 * e]) * wt[dir * j], y = __uint_as_float(r[2 * e + 1]) * wt[dir * (j + 1)];
                x = j >= from && j < to ? x : 0.0f;
                y = j + 1 >= from && j + 1 < to ? y : 0.0f;
                w[e] = pack2(x, y);
              }
            }
            tmem_st16(tm + kSC + lanes + 16 * q, w);
          }
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(p_ready);

          const int lag = p.rev && t0 + len == p.T ? 1 : 0;
          const bool write = row < len;
          const float win = in && write ? tab[127 + (p.rev ? len - row - lag : row + 1)] : 0.0f;
          const float s1 = win * p.scale;
          const long long at = ((long long)it.b * p.T + t0 + row) * p.ldo + (long long)it.h * DC;
          LA_WAIT_WARP(o_full, cc);
          tc_fence_after();
#pragma unroll
          for (int q = 0; q < DC / 32; ++q) {
            uint32_t x[32], y[32];
            tmem_ld32(tm + col_o2(DC) + lanes + 32 * q, x);
            tmem_ld32(tm + kO1 + lanes + 32 * q, y);
            tmem_ld_wait();
            if (q == DC / 32 - 1) {  // the last read: the accumulators are free
              tc_fence_before();
              __syncwarp();
              if (lane == 0) mbar_arrive(o_free);
            }
            if (write) {
#pragma unroll
              for (int e = 0; e < 32; ++e) {
                const float o = p.scale * __uint_as_float(x[e]);
                x[e] = __float_as_uint(win != 0.0f ? fmaf(s1, __uint_as_float(y[e]), o) : o);
              }
              if (p.out_f32) {
                uint4* o = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + at + 32 * q);
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = make_uint4(x[4 * e], x[4 * e + 1], x[4 * e + 2], x[4 * e + 3]);
              } else {
                uint4* o = reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.out) + at + 32 * q);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float* f = reinterpret_cast<const float*>(x) + 8 * e;
                  o[e] = make_uint4(pack2(f[0], f[1]), pack2(f[2], f[3]), pack2(f[4], f[5]), pack2(f[6], f[7]));
                }
              }
            }
            __syncwarp();
          }
        }
      }
      if (!ok) {
        *abort_flag = 1;
        set_status(p.status, IPTTT_ERR_TIMEOUT);
      }
    }
  } else {
    const int tid = threadIdx.x - kStateWarp * 32;
    const int quarter = warp & 3, half = (warp - kStateWarp) >> 2;
    const int row = DA == 128 ? quarter * 32 + lane : (quarter & 1) * 32 + lane;
    const int c0 = (DA == 128 ? half : half * 2 + (quarter >> 1)) * NC;  // its columns: [c0, c0 + NC)
    const uint32_t d_addr = tm + col_d(DC) + ((uint32_t)(quarter * 32) << 16) + c0;
    uint32_t tl = 0, cc = 0, ic = 0;
    float f[NC];
    for (int i = blockIdx.x; ok && i < ta.items; i += gridDim.x, ++ic) {
      const Item it = item_of(p, i);
      const size_t bh = (size_t)it.b * p.H + it.h;
      const float g = p.log_decay[it.h];
      if (tid == 0 && !(g <= 0.0f)) set_status(p.status, IPTTT_ERR_ARG);
      float* tab = tabs + (ic & 1) * kTab;
      tab[tid] = tid < 127 ? 0.0f : decay_pow(g, tid - 127);
      __syncwarp();
      if (lane == 0) mbar_arrive(tab_ready);
      const int lo = it.first * CH, hi = min(p.T, it.last * CH);

      // the state the segment starts from, and its operand copy
      auto store_f = [&]() {
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
      };
#pragma unroll
      for (int e = 0; e < NC; ++e) f[e] = 0.0f;
      if constexpr (!STATE) {
        const int start = p.init || p.segs > 1 ? nearest_start_warp(p, it.b, p.rev ? hi : lo, lane) : 0;
        auto add = [&](const float* src, int transposed, float w) {
          if (w == 0.0f) return;
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
        if (p.init) add(p.init + bh * DA * DC, p.init_t, p.init_mul * reach(p, g, -1, lo, hi, start, CH));
        const int s0 = p.rev ? it.seg + 1 : 0, s1 = p.rev ? p.segs : it.seg;
        for (int s = s0; s < s1; ++s)
          add(p.seg_in + (bh * p.segs + s) * DA * DC, p.seg_t, reach(p, g, s, lo, hi, start, CH));
        store_f();
      }
      LA_WAIT_WARP(tab_ready, ic);

      for (int n = 0; n < it.last - it.first; ++n, ++cc, tl += TPC) {
        const int ch = p.rev ? it.last - 1 - n : it.first + n;
        const int t0 = ch * CH, len = min(CH, p.T - t0);
        const Starts st = starts_of(p, it.b, ch);
        const bool any = st.any();
        const int lag = p.rev && t0 + len == p.T ? 1 : 0;
        // rows that reach the state at the chunk's far end
        const int out_from = p.rev ? 0 : st.last(), out_to = p.rev ? min(len, st.first()) : len;
        const uint32_t sb = tl % NS;
        LA_WAIT_WARP(&full[sb], tl / NS);
        uint8_t* bt = smem + sb * SLOT + tid * 16;
        uint8_t* lt = lo_buf + tid * 16;
        uint4 v[DA / 16];
#pragma unroll
        for (int m = 0; m < DA / 16; ++m) v[m] = *reinterpret_cast<const uint4*>(bt + m * 4096);
        if constexpr (!STATE) LA_WAIT_WARP(sc_full, cc);  // (1) has read B: it may be overwritten
#pragma unroll
        for (int m = 0; m < DA / 16; ++m) {
          const int j = (tid >> 3) + 32 * (m & 3);  // the token of this 16-byte unit
          const bool on = j >= out_from && j < out_to;
          const float w = tab[127 + (on ? (p.rev ? j : len - 1 - j) : 0)];
          const uint32_t u[4] = {v[m].x, v[m].y, v[m].z, v[m].w};
          uint32_t hi4[4], lo4[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float2 x = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&u[e]));
            x.x = on ? x.x * w : 0.0f;
            x.y = on ? x.y * w : 0.0f;
            hi4[e] = pack2(x.x, x.y);
            const float2 h2 = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&hi4[e]));
            lo4[e] = pack2(x.x - h2.x, x.y - h2.y);
          }
          *reinterpret_cast<uint4*>(bt + m * 4096) = make_uint4(hi4[0], hi4[1], hi4[2], hi4[3]);
          *reinterpret_cast<uint4*>(lt + m * 4096) = make_uint4(lo4[0], lo4[1], lo4[2], lo4[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();  // the last chunk's D has been read
        __syncwarp();
        if (lane == 0) mbar_arrive(conv_done);

        LA_WAIT_WARP(d_full, cc);
        tc_fence_after();
        const float keep = any ? 0.0f : tab[127 + len - lag];
        constexpr int STEP = NC < 32 ? NC : 32;
#pragma unroll
        for (int q = 0; q < NC / STEP; ++q) {
          uint32_t r[STEP];
          tmem_load<STEP>(d_addr + STEP * q, r);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < STEP; ++e) {
            float& x = f[STEP * q + e];
            x = keep != 0.0f ? fmaf(keep, x, __uint_as_float(r[e])) : __uint_as_float(r[e]);
          }
        }
        if constexpr (!STATE) {
          if (n + 1 < it.last - it.first) store_f();  // (2) of this chunk has read the old copy: d_full came after it
        }
      }
      if (!ok) break;
      float* dst = nullptr;
      float mul = 1.0f;
      if constexpr (STATE) {
        dst = p.seg_state + (bh * p.segs + it.seg) * DA * DC;
      } else if (p.fin && (p.rev ? it.seg == 0 : it.seg == p.segs - 1)) {
        dst = p.fin + bh * DA * DC;
        if (p.fin_scale) mul = p.scale * decay_pow(g, 1);
      }
      if (dst) {
#pragma unroll
        for (int e = 0; e < NC; e += 4)
          *reinterpret_cast<float4*>(dst + (size_t)row * DC + c0 + e) =
              make_float4(mul * f[e], mul * f[e + 1], mul * f[e + 2], mul * f[e + 3]);
      }
    }
    if (!ok) {
      *abort_flag = 1;
      set_status(p.status, IPTTT_ERR_TIMEOUT);
    }
  }
#undef LA_WAIT
#undef LA_WAIT_WARP

  __syncthreads();
  if (*abort_flag && threadIdx.x == 0) {
    // copies that were issued land before the block's shared memory is given back
    const uint32_t n = *issued;
    for (uint32_t t = n > (uint32_t)NS ? n - NS : 0; t < n; ++t) mbar_wait(&full[t % NS], (t / NS) & 1);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tm, 512);
  }
}

template <int DA, int DC, bool STATE>
cudaError_t launch(const TcArgs& a, cudaStream_t st) {
  constexpr int smem = Cfg<DA, DC, STATE>::SMEM;
  static_assert(smem <= 232448 && Cfg<DA, DC, STATE>::NS >= 2 * Cfg<DA, DC, STATE>::TPC - 1, "ring");
  const cudaError_t e =
      cudaFuncSetAttribute(k_pass_tc<DA, DC, STATE>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  k_pass_tc<DA, DC, STATE><<<std::min(a.items, device_sms()), kTcThreads, smem, st>>>(a);
  return cudaGetLastError();
}

template <int DA, int DC>
cudaError_t launch(const TcArgs& a, cudaStream_t st) {
  return a.p.out ? launch<DA, DC, false>(a, st) : launch<DA, DC, true>(a, st);
}

}  // namespace

bool tc_takes(int Da, int Dc) { return (Da == 64 || Da == 128) && (Dc == 64 || Dc == 128); }

int tc_segments(int B, int T, int H, int* seg_chunks) {
  const int n = (T + CH - 1) / CH;
  const long long bh = (long long)B * H;
  // Chunks the busiest SM walks, in the pass and (at two thirds of the time) in the pass for
  // the segments' states, with two more an item for its start; the fewest win.
  auto cost = [&](int segs) {
    const long long each = (n + segs - 1) / segs;
    const long long waves = (bh * segs + 147) / 148, waves_s = (bh * (segs - 1) + 147) / 148;
    return waves * (each + 2) * 3 + (segs > 1 ? waves_s * (each + 2) * 2 + 6 : 0);
  };
  int best = 1;
  for (int s = 2; s <= std::min(n, 148); ++s)
    if (cost(s) < cost(best)) best = s;
  *seg_chunks = (n + best - 1) / best;
  return (n + *seg_chunks - 1) / *seg_chunks;
}

cudaError_t run_tc(const Pass& p, cudaStream_t st) {
  TcArgs a;
  a.p = p;
  a.items = p.B * p.H * (p.out ? p.segs : p.segs - 1);
  if (a.items <= 0) return cudaSuccess;
  auto map = [&](CUtensorMap* m, const void* base, long long ld, int g, int width) {
    return tck::make_map_bf16_ld(m, base, (uint64_t)(p.H / g) * width, p.T, p.B, ld, 64, CH);
  };
  if (p.out && !map(&a.ma, p.a, p.lda, p.ga, p.Da)) return cudaErrorInvalidValue;
  if (!map(&a.mb, p.b, p.ldb, p.gb, p.Da) || !map(&a.mc, p.c, p.ldc, p.gc, p.Dc)) return cudaErrorInvalidValue;
  if (p.Da == 128) return p.Dc == 128 ? launch<128, 128>(a, st) : launch<128, 64>(a, st);
  return p.Dc == 128 ? launch<64, 128>(a, st) : launch<64, 64>(a, st);
}

}  // namespace la
}  // namespace ipttt
