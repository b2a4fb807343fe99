// The joining of pa_decode_int4's cut segments on the host: CTAs that take their steps in random order go through the
// rounds of csrc/join_int4.h; every segment has to get each of its shares exactly once, nothing may be read
// before it is written, and every counter has to end at zero.  "planted": the same with a mistake in the model, the
// state of the CTA's second segment overwritten by the first one's second round; it has to be found.

#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <map>
#include <random>
#include <vector>

#include "join_int4.h"

using namespace pa;

namespace {

constexpr int kTile = 32, kStart = 2;  // as in decode_int4.cu

struct Seg {
  long long start;  // on the line
  int tiles;
};

// What a CTA still has to do: one entry per step, so that CTAs' steps may be interleaved in any order.
struct Cta {
  int id;
  Cut cut[2];
  Round state[2];  // planted mistake only: rounds kept in variables
  bool done[2];
  int which = 0, round = 0, at = 0;  // at: 0 write, 1 count, 2 join, 3 count again, 4 over
};

struct Model {
  std::vector<Cta> ctas;
  std::vector<int> counters = std::vector<int>(3 * kMaxGrid, 0);
  std::map<long long, std::vector<int>> slots;      // shares (CTAs) that a slot's content is made of
  std::map<long long, std::vector<int>> results;    // segment -> the shares in its result
  std::map<long long, Cut> cuts;
  bool planted = false, bad = false;

  bool count(const Round& r) {
    if (r.counter < 0 || r.counter >= 3 * kMaxGrid) return bad = true, false;
    if (++counters[r.counter] != r.n) return false;
    counters[r.counter] = 0;
    return true;
  }

  void step(Cta& c) {
    if (c.at == 0) {  // the CTA's shares
      for (const Cut& k : c.cut)
        if (k.n) {
          if (slots.count(k.seg + c.id)) bad = true;  // a slot used twice
          slots[k.seg + c.id] = {c.id};
        }
      c.at = 1;
    } else if (c.at == 1) {
      for (int w = 0; w < 2; ++w) {
        if (c.cut[w].n) c.state[w] = join_round(0, c.cut[w], c.id);
        c.done[w] = c.cut[w].n && count(c.state[w]);
      }
      c.at = 2;
    } else if (c.at == 2) {  // join, for the segment `which`
      while (c.which < 2 && !c.done[c.which]) ++c.which, c.round = 0;
      if (c.which == 2) return void(c.at = 4);
      const Cut& k = c.cut[c.which];
      const Round r = planted ? c.state[c.which] : join_round(c.round, k, c.id);
      std::vector<int> sum;
      for (int i = 0; i < r.n; ++i) {
        const long long s = i == 0 ? r.slot0 : r.slots + (long long)i * r.step;
        if (!slots.count(s)) return void(bad = true);  // not written yet
        sum.insert(sum.end(), slots[s].begin(), slots[s].end());
      }
      if (r.again && !(planted && c.round)) {
        slots[r.slot0] = sum;
        c.at = 3;
      } else {
        if (results.count(k.seg)) bad = true;  // written twice
        results[k.seg] = sum;
        ++c.which, c.round = 0;
      }
    } else if (c.at == 3) {  // the joint share counts
      ++c.round;
      const Round up = join_round(c.round, c.cut[c.which], c.id);
      if (planted)
        for (int w = 0; w < 2; ++w)  // the mistake: of both segments
          if (c.cut[w].n) {
            const bool again = c.state[w].again;
            c.state[w] = join_round(1, c.cut[w], c.id);
            c.state[w].again = again;
          }
      c.done[c.which] = count(up);
      c.at = 2;
    }
  }

  bool right() {
    if (bad || results.size() != cuts.size()) return false;
    for (int c : counters)
      if (c) return false;
    for (auto& [seg, k] : cuts) {
      std::vector<int> sum = results[seg];  // the order of the line, each once
      if ((int)sum.size() != k.n) return false;
      for (int i = 0; i < k.n; ++i)
        if (sum[i] != k.c0 + i) return false;
    }
    return true;
  }
};

// The line of sequences of these lengths, cut for `grid` CTAs as the kernel cuts it; runs the join in a random order.
// Returns whether it was right; *grouped: whether a segment was joined in groups.
bool run(const std::vector<long long>& lens, int kv_heads, int grid, bool planted, std::mt19937_64& rng, bool* grouped) {
  std::vector<Seg> segs;
  std::vector<long long> number;
  long long total = 0;
  for (size_t b = 0; b < lens.size(); ++b)
    for (int g = 0; g < kv_heads; ++g)
      if (lens[b] > 0) {
        const int tiles = (int)((lens[b] + kTile - 1) / kTile);
        segs.push_back({total, tiles});
        number.push_back((long long)b * kv_heads + g);
        total += tiles + kStart;
      }
  const long long ctas = std::min<long long>(grid, total);
  Model m;
  m.planted = planted;
  size_t s0 = 0;
  for (int c = 0; c < ctas; ++c) {
    Cta cta;
    cta.id = c;
    cta.cut[0] = cta.cut[1] = Cut{0, 0, 0};
    const long long x0 = total * c / ctas, x1 = total * (c + 1) / ctas;
    std::vector<std::pair<Cut, bool>> runs;  // segments with tiles in [x0, x1), and whether all of them
    while (s0 < segs.size() && segs[s0].start + kStart + segs[s0].tiles <= x0) ++s0;
    for (size_t s = s0; s < segs.size(); ++s) {
      const long long t0 = segs[s].start + kStart, t1 = t0 + segs[s].tiles;
      if (t0 >= x1) break;
      const bool narrow = (total + 1) * (ctas + 1) < (1ll << 32);
      const Cut k = cut_of(number[s], t0, segs[s].tiles, ctas, total, narrow);
      runs.push_back({k, t0 >= x0 && t1 <= x1});
      // a share exactly where cut_of says that there is one
      if ((std::max(t0, x0) < std::min(t1, x1)) != (c >= k.c0 && c < k.c0 + k.n)) return false;
    }
    for (size_t r = 0; r < runs.size(); ++r)
      if (!runs[r].second) {
        if (r != 0 && r + 1 != runs.size()) return false;  // the first or the last only
        cta.cut[r == 0 ? 0 : 1] = runs[r].first;
        m.cuts[runs[r].first.seg] = runs[r].first;
        *grouped |= runs[r].first.n > 2 * kGroup;
      }
    m.ctas.push_back(cta);
  }
  std::vector<int> left;
  for (int c = 0; c < (int)m.ctas.size(); ++c) left.push_back(c);
  // in bursts: a CTA that has begun often goes on, as on a GPU, but any order may come
  size_t at = 0;
  while (!left.empty()) {
    if (rng() % 4 == 0 || at >= left.size()) at = rng() % left.size();
    m.step(m.ctas[left[at]]);
    if (m.bad) return false;
    if (m.ctas[left[at]].at == 4) left.erase(left.begin() + at);
  }
  return m.right();
}

}  // namespace

int main(int argc, char** argv) {
  const bool planted = argc > 1 && !strcmp(argv[1], "planted");
  std::mt19937_64 rng(7);
  int wrong = 0, joined = 0;
  struct Fixed {
    std::vector<long long> lens;
    int kv_heads, grid;
  };
  std::vector<Fixed> all = {{{32000, 16000}, 2, 148}, {{100000, 3000}, 8, 148}, {{64000, 1000}, 1, 148},
                            {{50000, 20000}, 1, 74},  {{8192, 8000, 64, 1}, 2, 148}, {{8193, 30, 30}, 2, 38},
                            {{100001}, 2, 74},        {{20000}, 1, 1024},     {{1 << 30, 5}, 2, 512}};
  std::vector<Fixed> runs;
  for (const Fixed& f : all)
    for (int i = 0; i < 200; ++i) runs.push_back(f);
  for (int i = 0; i < 3000; ++i) {  // few or many sequences, one to millions of tokens, any grid
    Fixed f;
    const int batch = 1 + rng() % (rng() % 4 ? 8 : 60);
    for (int b = 0; b < batch; ++b) f.lens.push_back(rng() % 10 ? 1 + rng() % (1ll << (4 + rng() % 18)) : 0);
    f.lens[0] = std::max(f.lens[0], 1ll);
    f.kv_heads = 1 + rng() % 8;
    f.grid = 1 + rng() % (rng() % 8 ? 160 : 1024);
    runs.push_back(f);
  }
  for (const Fixed& f : runs) {
    bool grouped = false;
    const bool ok = run(f.lens, f.kv_heads, f.grid, planted, rng, &grouped);
    wrong += !ok;
    joined += grouped;
    if (!ok && !planted) {
      fprintf(stderr, "wrong: %zu sequences, first of %lld tokens, %d KV heads, %d CTAs\n", f.lens.size(), f.lens[0],
              f.kv_heads, f.grid);
      return 1;
    }
  }
  if (joined < 500) return fprintf(stderr, "only %d runs joined a segment in groups\n", joined), 1;
  printf("%d wrong\n", wrong);
  return 0;
}
