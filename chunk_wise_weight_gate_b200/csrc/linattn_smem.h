// Shared memory of the tensor-core pass of linear attention (linattn_tc.cu), plain C++: the
// kernel takes its addresses from here, and a host test walks every form.
#pragma once

namespace ipttt {
namespace la {

// Per head: pw[128 + n] = gamma^n for 0 <= n <= 128 and 0 for n < 0, what fade_next takes besides gamma^128, then
// (from kPw on) gamma^{31 - n}, n < 32.
constexpr int kPw = 260, kTab = kPw + 32;
constexpr int kSmemBlock = 232448;  // most shared memory of a block
constexpr int kWalk = 8;            // tokens at a time, where an item is walked token by token
constexpr int kMostItems = 1024;    // of a block

// The form of widths DA (a, b) and DC (c); STATE: a segment's own state alone.  In order:
//   a tiles [NA][SLOT], ring [NS][SLOT], lo half, state's copy, tables [2][kTab], barriers, words.
template <int DA, int DC, bool STATE>
struct Smem {
  static constexpr int SLOT = 256 * (DA > DC ? DA : DC);  // a tile of 128 tokens (an a tile, then the output in its place)
  static constexpr int NA = STATE ? 0 : 2;
  // The scaled B's lower parts: of a chunk in one (STATES: of two chunks in turn), or, where the state is an
  // output, in two of half a chunk each (STATES: of two half chunks in turn).
  static constexpr int LO = 256 * DA * (STATE ? 2 : 1);
  static constexpr int LO_SLOTS = STATE ? 2 : 1, LO_PART = LO / LO_SLOTS / 2;  // the latter: half chunks, bytes of a part
  static constexpr int FB = STATE ? 0 : DA * DC * 2;      // bf16 state
  static constexpr int TABS = 2 * kTab * 4;
  static constexpr int MOST = 6;                          // tiles of the ring at most
  static constexpr int bars(int ns) { return 2 * ns + 24; }  // full, empty for each tile, and the others
  static constexpr int WORDS = 4 + kMostItems / 32;  // TMEM address, abort flag, tiles issued (ring, a), a bit for each item
  static constexpr int tail(int ns) { return (8 * bars(ns) + 4 * WORDS + 15) / 16 * 16; }
  static constexpr int FIXED = NA * SLOT + LO + FB + TABS + tail(MOST);
  static constexpr int FIT = (kSmemBlock - FIXED) / SLOT;
  static constexpr int NS = FIT < MOST ? FIT : MOST;
  static constexpr int at_ring = NA * SLOT, at_lo = at_ring + NS * SLOT, at_f = at_lo + LO, at_tabs = at_f + FB,
                       at_bars = at_tabs + TABS, at_words = at_bars + 8 * bars(NS), END = at_words + 4 * WORDS;
  static constexpr int BYTES = at_bars + tail(NS);
  // The walk by tokens (values that are not finite) has the fp32 state in the tiles' place, and in the lo
  // half's kWalk tokens' a, b and c and their outputs' parts.
  static_assert(4 * DA * DC <= at_lo && 4 * kWalk * (2 * DA + DC + 256) <= LO, "room for the walk");
  static_assert(NS >= 3 && END <= BYTES && BYTES <= kSmemBlock && at_bars % 8 == 0, "shared memory");
};

}  // namespace la
}  // namespace ipttt
