// The cuts of products: whatever number of rows the device counts, the splits that it then
// takes fit the grid and the partial sums' memory, and every k is in one split.
//   product_plan_check            checks
//   product_plan_check m n k ways prints the cut
#include <cstdio>
#include <cstdlib>

#include "act/product.h"

using namespace zero::act;

static int failures = 0;

static void check(bool ok, const char* what, uint64_t m, uint64_t n, uint64_t k, uint64_t c) {
  if (ok) return;
  ++failures;
  std::printf("%s: m %llu n %llu k %llu count %llu\n", what, (unsigned long long)m,
              (unsigned long long)n, (unsigned long long)k, (unsigned long long)c);
}

static void one(uint64_t m, uint64_t n, uint64_t k, const MulWays& ways) {
  const MulPlan p = plan_product(m, n, k, ways);
  check(p.tile == 256 || p.tile == 128 || (p.tile == 32 && ways.few_rows), "tile", m, n, k, m);
  check(p.splits >= 1 && p.splits <= p.most && p.most <= 32, "splits", m, n, k, m);
  check(ways.split || p.most == 1, "splits that may not be", m, n, k, m);
  check(ways.counted || p.most == p.splits, "splits without a count", m, n, k, m);
  uint64_t wgs = p.tiles * p.splits;
  if (p.most > p.splits && wgs < p.fill) wgs = p.fill;          // the grid
  const uint64_t room = partial_rows(p, m);
  const uint64_t counts[] = {0, 1, 31, 32, 33, m / 3, m / 2, m - 1, m};
  for (uint64_t c : counts) {
    if (c > m || (!ways.counted && c != m)) continue;
    const MulPlan q = plan_of(p, c, n);
    const uint32_t s = splits_of(p.splits, p.most, p.fill, static_cast<uint32_t>(q.tiles));
    check(s >= 1 && s <= p.most, "splits of a count", m, n, k, c);
    check(q.tiles * s <= wgs, "more workgroups than the grid", m, n, k, c);
    check(s == 1 || s * c <= room, "partial sums outside their memory", m, n, k, c);
    const uint64_t per = ((k + s - 1) / s + kMulDepth - 1) / kMulDepth * kMulDepth;
    check(per * s >= k, "k that no split has", m, n, k, c);
  }
}

int main(int argc, char** argv) {
  if (argc == 5) {
    const char* w = argv[4];
    const MulPlan p = plan_product(strtoull(argv[1], 0, 10), strtoull(argv[2], 0, 10),
                                   strtoull(argv[3], 0, 10),
                                   {w[0] == '1', w[1] == '1', w[2] == '1', w[3] == '1'});
    std::printf("tile %d splits %u most %u tiles %llu\n", p.tile, p.splits, p.most,
                (unsigned long long)p.tiles);
    return 0;
  }
  const uint64_t sizes[] = {1, 7, 31, 32, 33, 100, 255, 257, 700, 1025, 4096, 5003, 131072, 500001};
  for (uint64_t m : sizes)
    for (uint64_t n : sizes)
      for (uint64_t k : sizes)
        for (int w = 0; w < 16; ++w) one(m, n, k, {(w & 1) != 0, (w & 2) != 0, (w & 4) != 0, w >= 8});
  uint64_t seed = 1;
  const auto next = [&](uint64_t most) {
    seed = seed * 6364136223846793005ull + 1442695040888963407ull;
    return 1 + (seed >> 33) % (1ull << (1 + (seed >> 20) % most));
  };
  for (int i = 0; i < 200000; ++i) {
    const uint64_t m = next(20), n = next(20), k = next(20);
    one(m, n, k, {(i & 1) != 0, (i & 2) != 0, (i & 4) != 0, (i & 8) != 0});
  }
  if (failures) return 1;
  std::printf("product plan check ok\n");
  return 0;
}
