// The selection's kernels on the host (blocks/hip/hip_runtime.h), a block's waves in both
// orders, against a sort: what they keep must not depend on which wave comes first.
#include "k_evict.hip"

#include <cstdio>
#include <numeric>
#include <random>

using namespace lora;

namespace {

enum Kind { kEqual, kZeros, kNear, kTies, kSpread };
const char* const kNames[] = {"equal", "mostly zero", "close", "ties", "spread"};

struct Case {
  int H, T, nb;
  std::vector<int32_t> lens, table;
  int n_pages;
  std::vector<float> weights;
  int64_t w_ld;
};

Case make(int H, int T, int nb, std::vector<int32_t> lens, Kind kind, bool gaps, unsigned seed) {
  std::mt19937 rng(seed);
  Case c{H, T, nb, lens, {}, 7, {}, (int64_t)nb * T};
  const int S = (int)lens.size();
  c.table.resize((size_t)S * 2 * H * nb);
  for (auto& id : c.table) id = gaps && rng() % 16 == 0 ? -1 : (int32_t)(rng() % 7);
  c.weights.resize((size_t)S * H * c.w_ld);
  std::normal_distribution<float> normal;
  for (auto& w : c.weights) {
    switch (kind) {
      case kEqual: w = 0.25f; break;
      case kZeros: w = rng() % 50 ? 0.f : std::exp(normal(rng)); break;
      case kNear: w = __uint_as_float(0x3f800000u + rng() % 100000u); break;
      case kTies: w = (float)(rng() % 4); break;
      case kSpread: w = std::exp(2.f * normal(rng)); break;
    }
  }
  return c;
}

bool check(const Case& c, int budget, int sinks, int recent) {
  const int S = (int)c.lens.size(), ld = budget + 2;
  std::vector<int32_t> q_start(S + 1, 0), keep((size_t)S * c.H * ld, -9), n_keep(S, -9);
  SelectArgs a{};
  a.kv.n_pages = c.n_pages;
  a.kv.T = c.T;
  div_init(c.T, a.kv.div_m, a.kv.div_s);
  a.kv.H = c.H;
  a.kv.n_seqs = S;
  a.kv.nb = c.nb;
  a.kv.q_start = q_start.data();
  a.kv.kv_len = c.lens.data();
  a.kv.table = c.table.data();
  a.weights = c.weights.data();
  a.w_ld = c.w_ld;
  a.budget = budget;
  a.sinks = sinks;
  a.recent = recent;
  a.keep = keep.data();
  a.keep_ld = ld;
  a.n_keep = n_keep.data();
  std::vector<uint4> ws(select_workspace(S, c.H, (int64_t)c.nb * c.T) / 16 + 1, uint4{~0u, ~0u, ~0u, ~0u});
  a.ws = reinterpret_cast<char*>(ws.data());
  launch_select(a, nullptr);
  if (!blocks::fault.empty()) {
    std::printf("%s\n", blocks::fault.c_str());
    return false;
  }
  for (int s = 0; s < S; ++s) {
    std::vector<std::vector<int>> there(c.H);
    size_t k = (size_t)budget;
    for (int h = 0; h < c.H; ++h) {
      const int32_t* ktab = &c.table[((size_t)s * 2 * c.H + h) * c.nb];
      for (int j = 0; j < c.lens[s]; ++j)
        if (ktab[j / c.T] >= 0 && ktab[(size_t)c.H * c.nb + j / c.T] >= 0) there[h].push_back(j);
      k = std::min(k, there[h].size());
    }
    if (n_keep[s] != (int)k) {
      std::printf("sequence %d keeps %d of %zu\n", s, n_keep[s], k);
      return false;
    }
    for (int h = 0; h < c.H; ++h) {
      const float* w = &c.weights[((size_t)s * c.H + h) * c.w_ld];
      auto first = [&](int j) { return j < sinks || j >= c.lens[s] - recent; };
      auto& t = there[h];
      std::stable_sort(t.begin(), t.end(), [&](int x, int y) {
        return first(x) != first(y) ? first(x) : (!first(x) && w[x] > w[y]);
      });
      t.resize(k);
      std::sort(t.begin(), t.end());
      const int32_t* got = &keep[((size_t)s * c.H + h) * ld];
      if (!std::equal(t.begin(), t.end(), got) || got[k] != -9) {
        std::printf("sequence %d, head %d: another list\n", s, h);
        return false;
      }
    }
  }
  return true;
}

}  // namespace

int main() {
  struct Shape {
    int H, T, nb;
    std::vector<int32_t> lens;
  };
  std::vector<int32_t> many(129, 0);   // more heads of sequences than a launch of large blocks takes
  many[3] = 5000;
  std::vector<int32_t> more = many;
  more[3] = 16384;
  more[77] = 9001;
  const Shape shapes[] = {
      {3, 32, 64, {2048, 700, 0, 65}},    // each of the launches of one block a head ..
      {2, 32, 128, {4096, 2049}},
      {2, 64, 128, {8192, 1500}},
      {2, 64, 128, many},
      {2, 64, 256, {16384, 1025}},
      {2, 64, 256, more},
      {8, 16, 640, {10240, 3}},           // .. one whose page ids are looked at ahead ..
      {2, 64, 400, {25600, 8193, 40}},    // .. and those over chunks
  };
  int cases = 0;
  for (const Shape& sh : shapes)
    for (int kind = kEqual; kind <= kSpread; ++kind)
      for (int gaps = 0; gaps < 2; ++gaps) {
        const int most = *std::max_element(sh.lens.begin(), sh.lens.end());
        const Case c = make(sh.H, sh.T, sh.nb, sh.lens, (Kind)kind, gaps != 0, 1u + (unsigned)kind);
        for (const blocks::Order order : {blocks::kForward, blocks::kBackward}) {
          blocks::order = order;
          const int budget = most / 3;
          if (!check(c, budget, 4, budget / 4)) {
            std::printf("%d heads of up to %d tokens, weights %s, %s, waves %s\n", sh.H, most, kNames[kind],
                        gaps ? "pages missing" : "all pages there", order == blocks::kForward ? "forward" : "backward");
            return 1;
          }
          ++cases;
        }
      }
  std::printf("%d cases\n", cases);
  return 0;
}
