// What the host decides for the operators on token IDs (lm_layout.cpp), under
// AddressSanitizer and UndefinedBehaviorSanitizer: workspace layouts and
// divisors on the limits and on seeded random sizes.  One check by name per
// run; built and run by tests/test_lm_layout.py.
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <algorithm>
#include <random>
#include <utility>
#include <vector>

#include "lm_internal.h"

using namespace bpe;

#define CHECK(c)                                                      \
  do {                                                                \
    if (!(c)) {                                                       \
      fprintf(stderr, "check failed: %s (line %d)\n", #c, __LINE__); \
      exit(3);                                                        \
    }                                                                 \
  } while (0)

static std::mt19937_64 rng(20261206);

// Between lo and hi, spread over the logarithm.
static int64_t between(int64_t lo, int64_t hi) {
  const double x = std::uniform_real_distribution<double>(0, 1)(rng);
  const double v = (double)lo * __builtin_pow((double)hi / (double)lo, x);
  return std::min(hi, std::max(lo, (int64_t)v));
}

// Regions in order, aligned, each as large as what goes into it; digits that
// hold every value; tiles that hold every ID.
static void check_layout(int64_t n, int64_t V, int64_t D) {
  const GradLayout L = grad_layout(n, V, D);
  CHECK(L.bits >= 1 && L.bits <= kDigitBits && L.passes * L.bits < 32);
  CHECK(V >> (L.passes * L.bits) == 0);
  CHECK(L.sort_tiles >= 1 && L.sort_tiles <= kSortTiles);
  const int64_t per = (int64_t)kSortTile * L.sort_steps;
  CHECK(L.sort_tiles * per >= n && (L.sort_tiles - 1) * per < n);
  CHECK(L.tile >= 8 && L.tile <= kGradTile);
  CHECK((int64_t)L.tiles * L.tile >= n && (int64_t)(L.tiles - 1) * L.tile < n);
  const std::vector<std::pair<size_t, size_t>> regions = {
      {L.key0, (size_t)n * 4}, {L.key1, (size_t)n * 4}, {L.pos0, (size_t)n * 4},
      {L.pos1, (size_t)n * 4}, {L.counts, ((size_t)L.sort_tiles << L.bits) * 4},
      {L.touched, ((size_t)V + 15) / 16 * 16},  // cleared in whole 16-byte groups
      {L.part, (size_t)L.tiles * 2 * (size_t)D * 4}};
  size_t end = 0;
  for (const auto &r : regions) {
    CHECK(r.first % 256 == 0 && r.first >= end);
    end = r.first + r.second;
  }
  CHECK(L.total >= end);
}

static void layout() {
  for (int64_t n : {(int64_t)1, (int64_t)kGradDirect + 1, (int64_t)kGradSmall, (int64_t)BPE_MAX_IDS})
    for (int64_t V : {(int64_t)1, (int64_t)511, (int64_t)512, (int64_t)BPE_MAX_ROWS})
      for (int64_t D : {1, 7, 8, 513, BPE_MAX_WIDTH}) check_layout(n, V, D);
  for (int i = 0; i < 20000; ++i)
    check_layout(between(1, BPE_MAX_IDS), between(1, BPE_MAX_ROWS), between(1, BPE_MAX_WIDTH));
}

static void divisor() {
  for (int i = 0; i < 3000; ++i) {
    const int32_t bs = i < 300 ? i + 2 : (int32_t)between(2, INT32_MAX);
    uint32_t magic;
    int32_t shift;
    block_divisor(bs, &magic, &shift);
    CHECK(shift >= 0 && shift < 31);
    for (int j = 0; j < 300; ++j) {
      const int64_t q = between(1, (int64_t)INT32_MAX / bs + 1);
      for (int64_t x : {q * bs - 1, q * bs, (int64_t)(rng() >> 33), (int64_t)INT32_MAX - j, (int64_t)j})
        if (x <= INT32_MAX)
          CHECK((int64_t)(((uint64_t)x * magic >> 32) >> shift) == x / bs);
    }
  }
}

// The logits' variant goes by the lists' lengths, not by the room for them.
static void variant() {
  bpe_logits_args a = {};
  for (int64_t rows : {1, 24, 256})
    for (int64_t prompt : {0, 600, 4096, 5000, 75000}) {
      a.rows = rows;
      a.vocab = 128256;
      a.n_prompt = rows * prompt;
      a.made_width = 0;
      const bool wide = logits_wide(a);
      CHECK(wide == (prompt > 4096));
      for (int64_t width : {1, 256, 4096, 8192, 1 << 20}) {
        a.made_width = width;
        CHECK(logits_wide(a) == wide);
      }
    }
}

// A forward that passes the checks has launches of fewer than 2^32 threads, and
// the header's bound is the one that is checked.
static void embed_limit() {
  const int64_t most = ((int64_t)1 << 34) - 1024;
  int fits = 0, not_ = 0;
  for (int i = 0; i < 100000; ++i) {
    const int ot = (int)(rng() % 3);
    const int64_t n = between(1, BPE_MAX_IDS), size = ot == BPE_F32 ? 4 : 2;
    int64_t D = between(8, BPE_MAX_WIDTH);
    if (i % 2) D = std::min<int64_t>(BPE_MAX_WIDTH, std::max<int64_t>(8, most / n * 16 / size + (int64_t)(rng() % 41) - 20));
    const int64_t vectors = n * ((D * size + 15) / 16);
    CHECK(embed_fits(n, D, ot) == (vectors <= most));
    if (!embed_fits(n, D, ot)) {
      ++not_;
      continue;
    }
    ++fits;
    CHECK((vectors + kEmbedUnits - 1) / kEmbedUnits * 256 < (int64_t)1 << 32);
    // by sorted IDs: four waves per workgroup
    const int64_t E = 16 / size, waves = (n + 63) / 64 * ((D + 64 * E - 1) / (64 * E));
    CHECK((waves + 3) / 4 * 256 < (int64_t)1 << 32);
  }
  CHECK(fits > 1000 && not_ > 1000);
  for (int64_t D = 1; D < 8; ++D) CHECK(embed_fits(BPE_MAX_IDS, D, BPE_F32));
}

// A gradient that passes the checks has launches of fewer than 2^32 threads,
// and the header's bound is the one that is checked.
static void grad_limit() {
  int fits = 0, not_ = 0;
  for (int i = 0; i < 100000; ++i) {
    const int64_t n = between(kGradDirect + 1, BPE_MAX_IDS), V = between(1, BPE_MAX_ROWS);
    int64_t D = between(1, BPE_MAX_WIDTH);
    if (i % 2) D = std::min<int64_t>(BPE_MAX_WIDTH, ((int64_t)1 << 32) / n * 512 + (int64_t)(rng() % 1025) + 1);
    const GradLayout L = grad_layout(n, V, D);
    const int64_t slabs = (D + 511) / 512;
    CHECK(grad_fits(n, V, D) == ((n + 255) / 256 * slabs < (int64_t)1 << 24));
    if (!grad_fits(n, V, D)) {
      ++not_;
      continue;
    }
    ++fits;
    CHECK(((L.tiles * slabs + 3) / 4 + (V + kZeroRows - 1) / kZeroRows) * 256 < (int64_t)1 << 32);
    CHECK(L.tiles * slabs * 256 < (int64_t)1 << 32);
  }
  CHECK(fits > 1000 && not_ > 1000);
  CHECK(grad_fits(BPE_MAX_IDS, BPE_MAX_ROWS, 8) && grad_fits(BPE_MAX_IDS, 1, 1536));
  CHECK(!grad_fits(BPE_MAX_IDS, 1, 1537));
}

// The launch of the logits that pass the checks has fewer than 2^32 threads,
// also where the lists choose wide workgroups, and the header's bound is the
// one that is checked.
static void logits_limit() {
  bpe_logits_args a = {};
  int fits = 0, wide = 0;
  for (int i = 0; i < 200000; ++i) {
    a.vocab = i % 2 ? between(1, 9000) : between(1, BPE_MAX_ROWS);
    const int64_t slabs = (a.vocab + 4095) / 4096;
    a.rows = i % 3 ? between(1, BPE_MAX_IDS) : ((int64_t)1 << 24) / slabs + (int64_t)(rng() % 5) - 2;
    if (a.rows < 1) continue;
    a.n_prompt = a.rows * between(1, 100000);
    a.made_width = between(1, 1 << 20);
    CHECK(logits_fit(a) == (a.rows * slabs < (int64_t)1 << 24));
    if (!logits_fit(a)) continue;
    ++fits;
    wide += logits_wide(a);
    const int64_t per = logits_wide(a) ? 8192 : 4096, threads = logits_wide(a) ? 1024 : 256;
    CHECK((a.vocab + per - 1) / per * a.rows * threads < (int64_t)1 << 32);
  }
  CHECK(fits > 1000 && wide > 1000);
  a.rows = (int64_t)1 << 22;
  a.vocab = 100;
  a.n_prompt = a.rows * 5000;
  CHECK(logits_fit(a) && !logits_wide(a));
  --a.rows;
  CHECK(logits_wide(a));
}

int main(int argc, char **argv) {
  const std::pair<const char *, void (*)()> checks[] = {
      {"layout", layout},           {"divisor", divisor},       {"variant", variant},
      {"embed_limit", embed_limit}, {"grad_limit", grad_limit}, {"logits_limit", logits_limit}};
  for (const auto &c : checks)
    if (argc == 2 && !strcmp(argv[1], c.first)) {
      c.second();
      printf("passed\n");
      return 0;
    }
  fprintf(stderr, "no such check\n");
  return 2;
}
