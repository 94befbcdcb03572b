// The line of work of a batch of prompts (csrc/prompt.h) checked on the host: places of items
// against a count one by one, and for random batches that the parts cover every tile once, that
// every piece has a slot of its own and that the join reads just the pieces that were written.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <random>
#include <set>
#include <tuple>
#include <vector>

#include "../mla_decode_attention_folded_gb300/csrc/prompt.h"

using namespace mlafold;
using namespace mlafold::prompt;

static int fails = 0;
#define CHECK(c)                                            \
  do {                                                      \
    if (!(c)) {                                             \
      std::printf("line %d: %s\n", __LINE__, #c);           \
      if (++fails > 10) std::exit(1);                       \
    }                                                       \
  } while (0)

int main(int argc, char** argv) {
  const int rounds = argc > 1 ? std::atoi(argv[1]) : 1000;
  std::mt19937 g(1);
  auto pick = [&](int lo, int hi) { return std::uniform_int_distribution<int>(lo, hi)(g); };
  auto size = [&] { return pick(0, 3) ? pick(0, 700) : pick(0, 1) ? pick(0, 20000) : pick(0, 3); };
  long long cut_batches = 0, whole_batches = 0, joins = 0, tails = 0;
  for (int round = 0; round < rounds; ++round) {
    const int R = pick(1, pick(0, 2) ? 6 : 30), H = pick(1, 9), ctas = pick(0, 1) ? 152 : pick(1, 200);
    std::vector<Request> q(R);
    std::vector<long long> first(R + 1, 0);
    std::vector<int> of(R);                        // heads, or pairs of heads, of a request
    const bool allowed = pick(0, 1);
    int longest = 0;
    for (int r = 0; r < R; ++r) {
      q[r].n = size();
      q[r].m = pick(0, 1) ? q[r].n : size();
      q[r].causal = round & 1;
      long long at = 0;
      for (int u = 0; u < items(q[r]); ++u) {
        CHECK(before(q[r], u) == at);
        int most = 0;                              // tiles that some row of the item sees
        for (int i = u * kRows; i < q[r].n && i < (u + 1) * kRows; ++i) {
          long long lim = q[r].causal ? (long long)i + 1 + q[r].m - q[r].n : q[r].m;
          lim = lim < 0 ? 0 : lim > q[r].m ? q[r].m : lim;
          CHECK(lim == limit(q[r], i));
          most = std::max(most, (int)cdiv(lim, 128));
        }
        CHECK(item_tiles(q[r], u) == std::max(most, 1));
        CHECK(item_at(q[r], at) == u && item_at(q[r], at + item_tiles(q[r], u) + kExtra - 1) == u);
        longest = std::max(longest, item_tiles(q[r], u));
        at += item_tiles(q[r], u) + kExtra;
      }
      CHECK(places(q[r]) == at);
      const int I = items(q[r]);
      CHECK(!I || std::max(item_tiles(q[r], I - 1), I > 1 ? item_tiles(q[r], I - 2) : 0) >=
                      item_tiles(q[r], 0));
      of[r] = units(q[r], H, allowed);
      CHECK(twins(q[r], allowed) == (allowed && q[r].n <= kHalf));
      CHECK(twins(q[r], allowed) ? 2 * of[r] - H >= 0 && 2 * of[r] - H < 2 : of[r] == H);
      first[r + 1] = first[r] + at * of[r];
      if (at) {
        const long long x = std::uniform_int_distribution<long long>(0, at * of[r] - 1)(g);
        CHECK(head_at(x, at, of[r]) == x / at);
      }
    }
    const long long total = first[R];
    const bool whole_batch = whole_items(total, longest, ctas);
    const long long len = whole_batch ? 0 : cdiv(total, parts_of(total, ctas));
    const int parts = whole_batch ? 0 : (int)cdiv(total, len);
    CHECK(parts >= 0 && parts <= ctas);
    if (!parts) {
      ++whole_batches;
      // Every item is claimed once, the longest first within a group of heads.
      for (int r = 0; r < R; ++r) {
        std::set<std::pair<int, int>> seen;
        const int I = items(q[r]), wide = pick(1, 500);
        for (int x = 0; x < I * of[r]; ++x) {
          int head, u;
          claimed_item(q[r], of[r], wide, x, head, u);
          CHECK(head >= 0 && head < of[r] && u >= 0 && u < I && seen.insert({head, u}).second);
        }
      }
      continue;
    }
    ++cut_batches;
    CHECK(part_at(total, len, 0) == 0 && part_at(total, len, parts) == total);
    auto find = [&](long long x) {
      int r = 0;
      while (first[r + 1] <= x) ++r;
      return r;
    };
    std::map<int, std::tuple<long long, int, int>> slots;    // slot -> item's first place, tiles
    std::map<long long, int> done;                           // item's first place -> tiles done
    std::set<long long> whole;
    std::map<int, std::pair<int, long long>> noted;          // part -> last part, item's first place
    std::map<long long, int> size_of;
    for (int p = 0; p < parts; ++p) {
      long long at = part_at(total, len, p);
      const long long end = part_at(total, len, p + 1);
      CHECK(end > at);
      while (at < end) {
        const int r = find(at);
        const long long x = at - first[r], per = places(q[r]), head = head_at(x, per, of[r]);
        const long long rest = x - head * per;
        const int u = item_at(q[r], rest), tiles = item_tiles(q[r], u);
        const int t0 = (int)(rest - before(q[r], u));
        const long long left = std::min(end - at, (long long)(tiles + kExtra - t0)), start = at - t0;
        at += left;
        if (t0 >= tiles) continue;
        const int t1 = (int)std::min((long long)tiles, t0 + left);
        CHECK(t1 > t0 && done[start] == t0);
        done[start] = t1;
        int slot = -1;
        if (t0 > 0) slot = 2 * p;
        else if (t1 < tiles) {
          slot = 2 * p + 1;
          int last = p + 1;
          while (last + 1 < parts && part_at(total, len, last + 1) < start + tiles) ++last;
          CHECK(!noted.count(p));
          noted[p] = {last, start};
          size_of[start] = tiles;
        }
        if (slot >= 0) {
          CHECK(!slots.count(slot) && slot < 2 * ctas);
          slots[slot] = std::make_tuple(start, t0, t1);
          if (slot & 1) ++tails;
        } else {
          whole.insert(start);
        }
      }
    }
    std::set<int> read;
    for (const auto& jn : noted) {
      const int part = jn.first, last = jn.second.first;
      const long long start = jn.second.second;
      int tiles = 0;
      ++joins;
      for (int p = part; p <= last; ++p) {
        const int slot = p == part ? 2 * p + 1 : 2 * p;
        CHECK(slots.count(slot) && std::get<0>(slots[slot]) == start && read.insert(slot).second);
        CHECK(std::get<1>(slots[slot]) == tiles);
        tiles = std::get<2>(slots[slot]);
      }
      CHECK(tiles == size_of[start] && !whole.count(start));
    }
    CHECK(read.size() == slots.size());
  }
  std::printf("%lld %lld %lld %lld\n", cut_batches, whole_batches, joins, tails);
  return fails ? 1 : 0;
}
