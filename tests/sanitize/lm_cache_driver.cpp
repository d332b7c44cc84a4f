// What the host decides for a cache of few bits (lm_layout.cpp), and the searches
// that its kernels make with a caller's offsets and tables (lm_internal.h), under
// AddressSanitizer and UndefinedBehaviorSanitizer.  One check by name per run;
// built and run by tests/test_lm_cache_layout.py.
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

static std::mt19937_64 rng(20261209);
static int64_t below(int64_t n) { return (int64_t)(rng() % (uint64_t)n); }

static int32_t divide(const Divisor &d, int32_t x) {
  return d.d == 1 ? x : (int32_t)(((uint64_t)x * d.magic >> 32) >> d.shift);
}

// Every element of a token belongs to one lane, groups of lanes do not cross a
// wave, and a workgroup's tokens fit its list.
static void shape() {
  for (int i = 0; i < 20000; ++i) {
    CacheArgs a = {};
    a.c.heads = i % 3 ? 1 + (int)below(64) : 1 + (int)below(BPE_MAX_HEADS);
    a.c.dim = 1 + (int)below(BPE_MAX_DIM);
    a.c.group = kCacheMinGroup << below(6);
    a.c.format = (int)below(3);
    for (bool write : {true, false}) {
      const int ot = (int)below(3), vec = write ? kCacheVec : cache_read_vec(a.c.dim, ot);
      cache_shape(&a, write, ot);
      CHECK(1 << a.group_log2 == a.c.group);
      CHECK(a.groups * a.c.group >= a.c.dim && (a.groups - 1) * a.c.group < a.c.dim);
      CHECK(a.per_head.d * vec >= a.c.dim);
      CHECK(a.per_token.d == a.per_head.d * a.c.heads && a.per_token.d <= 1 << 18);
      CHECK(a.tokens >= 1 && a.tokens <= kCacheTokens);
      if (write) {
        const int lanes = a.c.group / kCacheVec;
        CHECK(lanes >= 2 && lanes <= 64 && a.per_head.d % lanes == 0);
        CHECK(a.per_head.d / lanes == a.groups);
      }
      const int count = a.tokens * a.per_token.d;
      for (int j = 0; j < 50; ++j) {
        const int x = (int)below(count);
        CHECK(divide(a.per_token, x) == x / a.per_token.d);
        CHECK(divide(a.per_head, x % a.per_token.d) == x % a.per_token.d / a.per_head.d);
      }
    }
  }
}

// What is refused, and what the limits let through.
static void refusals() {
  uint8_t codes;
  float scales;
  bpe_cache good = {&codes, &scales, 10, 16 * 128, 16, 16, 128, 128, BPE_E4M3};
  CHECK(cache_ok(good));
  auto with = [&](auto change) {
    bpe_cache c = good;
    change(c);
    return cache_ok(c);
  };
  CHECK(!with([](bpe_cache &c) { c.format = 3; }));
  CHECK(!with([](bpe_cache &c) { c.format = -1; }));
  CHECK(!with([](bpe_cache &c) { c.heads = 0; }));
  CHECK(!with([](bpe_cache &c) { c.heads = BPE_MAX_HEADS + 1; }));
  CHECK(!with([](bpe_cache &c) { c.dim = 0; }));
  CHECK(!with([](bpe_cache &c) { c.dim = BPE_MAX_DIM + 1; }));
  for (int g : {0, -16, 8, 24, 127, 1024}) CHECK(!with([&](bpe_cache &c) { c.group = g; }));
  CHECK(!with([](bpe_cache &c) { c.n_slots = -1; }));
  CHECK(!with([](bpe_cache &c) { c.codes = nullptr; }));
  CHECK(!with([](bpe_cache &c) { c.scales = nullptr; }));
  CHECK(with([](bpe_cache &c) { c.scales = nullptr, c.codes = nullptr, c.n_slots = 0; }));
  CHECK(!with([](bpe_cache &c) { c.codes_stride -= 1; }));
  CHECK(!with([](bpe_cache &c) { c.scales_stride -= 1; }));
  CHECK(with([](bpe_cache &c) { c.codes_stride = 1 << 22, c.scales_stride = 1 << 20; }));
  CHECK(!with([](bpe_cache &c) { c.codes_stride = (1 << 22) + 1; }));
  CHECK(!with([](bpe_cache &c) { c.scales_stride = (1 << 20) + 1; }));
  CHECK(!with([](bpe_cache &c) { c.format = BPE_UINT4, c.scales_stride = 31; }));
  CHECK(with([](bpe_cache &c) { c.format = BPE_UINT4, c.scales_stride = 32, c.codes_stride = 1024; }));
  CHECK(with([](bpe_cache &c) { c.heads = 1024, c.dim = 1024, c.group = 16, c.codes_stride = 1 << 20,
                                c.scales_stride = 1 << 17, c.format = BPE_UINT4; }));
  const int64_t G = (int64_t)1 << 32;
  CHECK(cache_tokens_ok(good, 5, 16 * 128, 128) && cache_tokens_ok(good, 1, 0, 128));
  CHECK(cache_tokens_ok(good, 5, 128, 5 * 128) && !cache_tokens_ok(good, 5, 128, 5 * 128 - 1));
  CHECK(!cache_tokens_ok(good, 5, 16 * 128 - 1, 128) && !cache_tokens_ok(good, 5, 0, 128));
  CHECK(!cache_tokens_ok(good, -1, 2048, 128) && !cache_tokens_ok(good, 5, 2048, 127));
  CHECK(cache_tokens_ok(good, 5, G, 128) && !cache_tokens_ok(good, 5, G + 1, 128));
  CHECK(!cache_tokens_ok(good, 1, 0, G + 1));
  bpe_cache one = good;
  one.heads = 1;
  CHECK(cache_tokens_ok(one, 5, 128, 0) && cache_tokens_ok(one, BPE_MAX_IDS - 64, 128, -7));
  CHECK(!cache_tokens_ok(one, BPE_MAX_IDS - 63, 128, 0));
}

// The launch of the tokens that pass the checks has fewer than 2^32 threads, and the
// header's bound is the one that is checked.
static void limit() {
  int fits = 0, not_ = 0;
  for (int i = 0; i < 200000; ++i) {
    CacheArgs a = {};
    a.c.heads = i % 3 ? 1 + (int)below(16) : 1 + (int)below(BPE_MAX_HEADS);
    a.c.dim = i % 5 ? 1 + (int)below(BPE_MAX_DIM) : 1 + (int)below(40);
    a.c.group = kCacheMinGroup << below(6);
    const bool write = i % 2;
    const int ot = (int)below(3), vec = ot == BPE_F32 && a.c.dim % 4 == 0 ? 4 : 8;
    cache_shape(&a, write, ot);
    const int64_t most = BPE_MAX_IDS - kCacheTokens;
    a.n = i % 7 ? std::min(most, ((int64_t)1 << 33) / a.per_token.d + below(5) - 2) : 1 + below(most);
    const int64_t per = write ? (int64_t)a.groups * a.c.group / 8 : (a.c.dim + vec - 1) / vec;
    CHECK(cache_fits(a) == (a.n * a.c.heads * per < (int64_t)1 << 33));
    if (!cache_fits(a)) {
      ++not_;
      continue;
    }
    ++fits;
    CHECK(cache_workgroups(a) * a.tokens >= a.n && cache_workgroups(a) * kCacheThreads < (int64_t)1 << 32);
  }
  CHECK(fits > 1000 && not_ > 1000);
}

// The request of a token, with empty requests, and in range for offsets of any
// values and order.
static void request() {
  for (int i = 0; i < 20000; ++i) {
    const int64_t R = 1 + below(i % 5 ? 30 : 500);
    std::vector<int64_t> off(R + 1);
    int64_t at = below(4);
    for (auto &o : off) {
      o = at;
      at += below(3) ? below(6) : 0;
    }
    for (int j = 0; j < 20; ++j) {
      const int64_t t = below(off[R] + 5);
      int64_t want = 0;
      while (want < R && off[want + 1] <= t) ++want;
      CHECK(cache_request(off.data(), 0, R, t) == want);
      CHECK(cache_request(off.data(), below(want + 1), want + below(R - want + 1), t) == want);
    }
    for (auto &o : off) o = below(5) ? below(100) - 20 : (int64_t)rng();
    for (int j = 0; j < 20; ++j) {
      const int64_t r0 = below(R + 1), r1 = below(R + 1);
      const int64_t r = cache_request(off.data(), r0, r1, (int64_t)rng() >> below(64));
      CHECK(r >= r0 && r <= std::max(r0, r1));
    }
  }
}

// The slot of a position: within the cache whatever the table holds, -1 and a
// bit otherwise.
static void slot() {
  for (int i = 0; i < 200000; ++i) {
    const int32_t bs = i % 3 ? 1 + (int32_t)below(64) : 1 + (int32_t)below(INT32_MAX);
    const Divisor d = divisor(bs);
    const int64_t width = below(6), n_slots = below(2000);
    std::vector<int32_t> row(width);
    for (auto &e : row) e = below(3) ? (int32_t)below(200) - 20 : (int32_t)rng();
    const int64_t p = below(3) ? below(400) : below(INT32_MAX);
    uint32_t status = 0;
    const int64_t got = cache_slot(row.data(), width, bs, n_slots, p, divide(d, (int32_t)p), &status);
    const int64_t block = p / bs;
    if (block >= width) {
      CHECK(got == -1 && status == BPE_STATUS_TABLE_FULL);
    } else if (row[block] < 0) {
      CHECK(got == -1 && status == 0);
    } else if ((int64_t)row[block] * bs + p % bs >= n_slots) {
      CHECK(got == -1 && status == BPE_STATUS_BAD_SLOT);
    } else {
      CHECK(got == (int64_t)row[block] * bs + p % bs && got >= 0 && got < n_slots && status == 0);
    }
  }
}

// The gradient of a loss is one launch of fewer than 2^32 threads, and the header's
// bound is the one that is checked.
static void gradient() {
  int fits = 0;
  for (int i = 0; i < 100000; ++i) {
    const int64_t V = 1 + below(i % 2 ? 20000 : BPE_MAX_ROWS), slabs = (V + 8191) / 8192;
    const int64_t n = i % 3 ? 1 + below(1 << 22) : ((int64_t)1 << 24) / slabs + below(5) - 2;
    CHECK(distill_grad_fits(n, V) == (n * slabs < (int64_t)1 << 24));
    if (!distill_grad_fits(n, V)) continue;
    ++fits;
    CHECK((V + kDistillSlab - 1) / kDistillSlab * n * kDistillThreads < (int64_t)1 << 32);
  }
  CHECK(fits > 1000);
}

// A row's regions cover it, whole waves of them, and a launch that passes the checks
// has fewer than 2^32 threads.
static void regions() {
  for (int i = 0; i < 100000; ++i) {
    const int64_t V = i < 5000 ? i + 1 : 1 + below(i % 2 ? 300000 : BPE_MAX_ROWS);
    const int64_t n = verify_regions(V), t = verify_tiles(V);
    CHECK(n >= 4 && n % 4 == 0 && n <= kVerifyMostRegions && t >= 1);
    CHECK(n * t * kVerifyTile >= V && (t == 1 || n == kVerifyMostRegions));
    CHECK((n - 4) * t * kVerifyTile < V || t > 1);
    for (int64_t r : {1, 256, 257, 100000})
      if (verify_alone(r, V)) CHECK(n <= kVerifyAlone / kVerifyTile && t == 1);
    const int64_t R = 1 + below(1 << 20), per = std::min<int64_t>(256, (V + 8191) / 8192);
    CHECK(verify_workgroups(R, V) == R * per);
    CHECK(launch_fits(verify_workgroups(R, V), kVerifyThreads) == (R * per < (int64_t)1 << 24));
  }
}

int main(int argc, char **argv) {
  const std::pair<const char *, void (*)()> checks[] = {
      {"shape", shape}, {"refusals", refusals}, {"limit", limit}, {"request", request}, {"slot", slot}, {"gradient", gradient}, {"regions", regions}};
  for (const auto &c : checks)
    if (argc == 2 && !strcmp(argv[1], c.first)) {
      c.second();
      printf("passed\n");
      return 0;
    }
  fprintf(stderr, "no such check\n");
  return 2;
}
