// The shared-prefix decode's line of work (csrc/prefix.h) on the host: random shapes, lengths
// and plans, true ones, ones of other lengths and arbitrary words. The kernels' own
// functions say whether a plan serves; one that does is walked part by part, as
// wide_kernel walks it, and read as the merge reads it.
#include <algorithm>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <set>
#include <utility>
#include <vector>

#include "../mla_decode_attention_folded_gb300/csrc/prefix.h"

using namespace mlafold;

#define CHECK(x)                                                          \
  do {                                                                    \
    if (!(x)) {                                                           \
      std::printf("case %d: line %d: %s\n", at_case, __LINE__, #x);       \
      std::exit(1);                                                       \
    }                                                                     \
  } while (0)

int at_case = 0;

int main(int argc, char** argv) {
  const int cases = argc > 1 ? std::atoi(argv[1]) : 1000;
  std::mt19937 g(1);
  const auto rnd = [&](int lo, int hi) {
    return (int)(lo + (long long)(g() % (unsigned)(hi - lo + 1)));
  };
  long pieces = 0, served = 0, unserved = 0, longer = 0;
  for (int t = 1; t < 100000; ++t) CHECK(wide_own_tiles((int)wide_own_span(t)) == t);
  for (at_case = 0; at_case < cases; ++at_case) {
    WideArgs a{};
    a.R = rnd(1, 20);
    a.M = rnd(1, 300);
    a.N = (long long)a.R * a.M;
    a.prefix_pages = rnd(1, 40);
    a.max_pages = rnd(1, 120);
    a.num_pages = 1000;
    a.units = rnd(0, 3) ? rnd(1, 76) : rnd(1, 1024);
    a.blocks = (int)cdiv(a.N, kWideRows);
    a.own_blocks = (int)cdiv(a.M, kWideRows);
    a.own_tiles = (int)cdiv((long long)a.max_pages * kPage, kWideKeys);
    a.own_most = (int)wide_own_most(a.R, a.own_blocks, a.max_pages);
    const long long slots = (long long)a.units + a.blocks + (long long)a.R * a.own_blocks - 1;
    std::vector<int32_t> table((size_t)a.R * a.max_pages + a.prefix_pages);
    a.block_table = table.data();
    a.prefix_table = table.data() + (size_t)a.R * a.max_pages;
    const int prefix = rnd(-5, a.prefix_pages * kPage + 50);
    std::vector<int> lens(a.R), plan(a.R + 1, 0);
    for (int r = 0; r < a.R; ++r) {
      lens[r] = wide_len(rnd(0, 3) ? rnd(0, a.max_pages * kPage + 9) : 0, a.max_pages);
      CHECK(lens[r] >= 0 && wide_tiles(lens[r]) == (lens[r] + kWideKeys - 1) / kWideKeys &&
            wide_tiles(lens[r]) <= a.own_tiles);
    }
    const auto lay_out = [&](const std::vector<int>& of) {
      for (int r = 0; r < a.R; ++r) plan[r + 1] = plan[r] + wide_places(of[r], a.own_blocks);
    };
    lay_out(lens);
    const int mode = rnd(0, 8);
    if (mode == 1) for (auto& x : plan) x = (int)g();
    if (mode == 2) for (auto& x : plan) x = rnd(-10, 200);
    if (mode == 3) plan[rnd(0, a.R)] = (int)g();
    if (mode == 4) plan[rnd(0, a.R)] = rnd(-5, 100);
    if (mode == 5) for (int r = 0; r < a.R; ++r) plan[r] = rnd(0, plan[a.R]);
    if (mode == 6) for (int r = 0; r < a.R; ++r) plan[r] = rnd(0, 1) ? plan[r] : (int)g();
    if (mode >= 7) {                       // a plan of other lengths; 8: of longer ones
      std::vector<int> other(a.R);
      for (int r = 0; r < a.R; ++r)
        other[r] = wide_len(mode == 8 ? lens[r] + rnd(0, 600) : rnd(0, a.max_pages * kPage),
                            a.max_pages);
      lay_out(other);
    }

    // What a plan that serves is, from its words one by one.
    bool none = plan[0] != 0 && plan[0] != kPlanAnew, few = false;
    plan[0] = none ? plan[0] : 0;
    for (int r = 0; r < a.R; ++r) {
      bool is = false;
      for (int t = 0; t <= a.own_tiles && !is; ++t)
        if ((long long)plan[r + 1] - (r ? plan[r] : 0) == (t ? a.own_blocks * wide_own_span(t) : 0)) {
          is = true;
          few |= t < wide_tiles(lens[r]);
        }
      none |= !is;
    }
    int flaw = wide_ends_flaw(plan[0], plan[a.R], a.own_most);
    for (int r = 0; r < a.R; ++r)
      flaw |= wide_flaw(r ? plan[r] : 0, plan[r + 1], lens[r], a.own_blocks, a.own_tiles);
    CHECK((flaw != 0) == (none || few));
    if (!none) CHECK(!(flaw & kPlanNone));
    if (mode == 0 || mode == 8) CHECK(flaw == 0);
    plan[0] = 0;
    if (flaw != 0) {                       // as the kernels do then
      lay_out(lens);
      ++unserved;
    } else {
      ++served;
      longer += mode == 8;
    }

    // Parts: every tile of every segment once, every slot its own.
    std::set<int> used;
    std::set<std::pair<int, int>> done;    // segment, tile
    for (int u = 0; u < a.units; ++u) {
      WideWalk walk(a, plan.data(), lens.data(), prefix, u);
      if (walk.pos >= walk.end) continue;
      CHECK(walk.pos >= 0);
      WidePiece p;
      while (walk.next(p)) {
        ++pieces;
        CHECK(p.slot >= 0 && p.slot % kWideRows == 0 && p.slot / kWideRows < slots);
        CHECK(used.insert(p.slot / kWideRows).second);
        const int segment = p.slot / kWideRows - u;
        CHECK(p.count > 0 && p.tile >= 0 && p.row0 >= 0 && p.row0 < a.N && p.row_end <= a.N);
        if (segment < a.blocks) {
          CHECK(p.table == a.prefix_table && p.len == wide_len(prefix, a.prefix_pages));
          CHECK(p.row0 == segment * kWideRows && p.row_end == a.N);
        } else {
          const int r = (segment - a.blocks) / a.own_blocks, j = (segment - a.blocks) % a.own_blocks;
          CHECK(r < a.R && p.table == a.block_table + (size_t)r * a.max_pages && p.len == lens[r]);
          CHECK(p.row0 == r * a.M + j * kWideRows && p.row_end == (r + 1) * a.M);
          CHECK(p.tile + p.count <= a.own_tiles);
        }
        for (int t = p.tile; t < p.tile + p.count; ++t) CHECK(done.insert({segment, t}).second);
      }
    }
    const int prefix_tiles = wide_tiles(wide_len(prefix, a.prefix_pages));
    for (int b = 0; b < a.blocks; ++b)
      for (int t = 0; t < prefix_tiles; ++t) CHECK(done.count({b, t}));
    for (int r = 0; r < a.R; ++r)
      for (int j = 0; j < a.own_blocks; ++j)
        for (int t = 0; t < wide_tiles(lens[r]); ++t)
          CHECK(done.count({a.blocks + r * a.own_blocks + j, t}));

    // The merge: the consecutive slots that it reads of each segment are those written.
    const WideLine line(prefix, plan[a.R], a.prefix_pages, a.blocks, a.units);
    size_t read = 0;
    const auto take = [&](int first, int tiles, int segment) {
      const int u0 = line.unit_of(first), u1 = line.unit_of(first + tiles - 1);
      CHECK(u0 >= 0 && u1 >= u0 && u1 < a.units);
      for (int u = u0; u <= u1; ++u, ++read) CHECK(used.count(u + segment));
    };
    if (line.prefix_tiles > 0)
      for (int b = 0; b < a.blocks; ++b)
        take(b * (line.prefix_tiles + kWideCost), line.prefix_tiles, b);
    for (int r = 0; r < a.R; ++r) {
      const int span = (plan[r + 1] - plan[r]) / a.own_blocks;
      for (int j = 0; span > 0 && j < a.own_blocks; ++j)
        take(line.prefix_places + plan[r] + j * span, wide_own_tiles(span),
             a.blocks + r * a.own_blocks + j);
    }
    CHECK(read == used.size());
  }
  std::printf("pieces %ld served %ld of which longer %ld unserved %ld\n", pieces, served, longer,
              unserved);
  return 0;
}
