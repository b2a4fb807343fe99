// How the shares of a segment that pa_decode_int4 cut between CTAs are joined: which slots, how many, which counter.
// Plain arithmetic on values that do not change during a call, the same for every thread, so that the state of one
// segment's join cannot disturb another's; compiled for the device (decode_int4.cu) and, by the tests, for the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PA_HD __host__ __device__ __forceinline__
#else
#define PA_HD inline
#endif

namespace pa {

constexpr int kGroup = 8;  // CTAs whose shares of a segment are joined first, where a segment has many
// CTAs of a grid, at most.  The counters' room is this large whatever the sizes, so that a workspace serves calls of
// any sizes in turn: nothing of one call's results lies where the next one counts.
constexpr int kMaxGrid = 1024;

// Floor division of a >= 0 by b > 0; `narrow` (uniform) says both fit in 32 bits: the 64-bit one is a long sequence.
PA_HD long long udiv(long long a, long long b, bool narrow) {
  return narrow ? (long long)((uint32_t)a / (uint32_t)b) : a / b;
}

// A cut segment: its number (sequence times KV heads plus head) and the CTAs that hold tiles of it, one share each.
// The share of CTA c lies in slot seg + c: a CTA holds at most one share of a segment, and neighbouring segments
// share at most one CTA, so no slot is used twice.
struct Cut {
  long long seg;
  int c0, n;  // the first of its CTAs, and how many; n 0: no segment
};

// The CTAs of the tiles on places [tile0, tile0 + tiles) of a line of `total` places, of which CTA c of `ctas` takes
// [total c / ctas, total (c + 1) / ctas).
PA_HD Cut cut_of(long long seg, long long tile0, int tiles, long long ctas, long long total, bool narrow) {
  Cut k;
  k.seg = seg;
  k.c0 = (int)udiv((tile0 + 1) * ctas - 1, total, narrow);
  k.n = (int)udiv((tile0 + tiles) * ctas - 1, total, narrow) - k.c0 + 1;
  return k;
}

// One round of a segment's join: n shares count at `counter`; whoever counts last joins them.
struct Round {
  long long slot0, slots;  // share 0 is in slot0, share i > 0 in slots + i * step; a joint share goes to slot0
  int n, step, counter;
  bool again;  // the joint share counts in the next round (else it is the segment's result)
};

// The join of cut segment k as CTA `cta`, which holds a share of it, takes part in it: its first round (0) or its last (1).
// A segment with many shares is joined by groups of kGroup CTAs first (one SM reads shares at little more than 100 GB/s):
// the first round joins the shares of cta's group, the last the groups' joint shares.
// Counters [3 kMaxGrid]: a CTA holds the first tile of one cut segment at most, so the segment's own counter is that
// of its first CTA; and a later share of one segment at most, so a group's is that of its first CTA, apart where the
// group starts with the segment's first share.
PA_HD Round join_round(int round, const Cut& k, int cta) {
  Round r;
  const bool grouped = k.n > 2 * kGroup;
  if (round == 0 && grouped) {
    const int from = cta / kGroup * kGroup, end = k.c0 + k.n, first = from > k.c0 ? from : k.c0;
    r.slot0 = r.slots = k.seg + first;
    r.n = (from + kGroup < end ? from + kGroup : end) - first;
    r.step = 1;
    r.counter = (first == k.c0 ? kMaxGrid : 2 * kMaxGrid) + first;
    r.again = true;
  } else {
    r.slot0 = k.seg + k.c0;
    r.slots = grouped ? k.seg + k.c0 / kGroup * kGroup : r.slot0;
    r.n = grouped ? (k.c0 + k.n - 1) / kGroup - k.c0 / kGroup + 1 : k.n;
    r.step = grouped ? kGroup : 1;
    r.counter = k.c0;
    r.again = false;
  }
  return r;
}

}  // namespace pa
