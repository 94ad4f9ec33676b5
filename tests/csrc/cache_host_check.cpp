// Host-side checks of the paged cache's arithmetic (csrc/serving.h), compiled with the host
// compiler by tests/test_cache_host.py.  Prints "ok" or the first failure and exits non-zero.
#include <cstdio>
#include <vector>

#include "serving.h"

static int fail(const char* what, long long a, long long b, long long c) {
  std::printf("FAIL %s %lld %lld %lld\n", what, a, b, c);
  return 1;
}

struct Batch {
  std::vector<int> indptr, kv;
};

static int check_cut(const ra::CacheDims& c, const Batch& t, int blocks, int tile, int min_steps,
                     long long min_rows, long long max_rows) {
  auto work = [&](int b) {
    return ra::seq_work(c, t.indptr[b], t.indptr[b + 1], t.kv[b], tile, min_rows, max_rows);
  };
  long long total = 0;
  std::vector<long long> base(c.B);
  for (int b = 0; b < c.B; ++b) {
    base[b] = total;
    total += work(b).total;
  }
  // every step of every item exactly once, in order; the followers of a split item's first
  // block are the blocks that hold its other steps
  std::vector<int> seen((size_t)total, 0);
  const long long per = ra::steps_per_block(total, blocks, min_steps);
  std::vector<long long> owner((size_t)total, -1);
  struct Split {
    long long item_end;
    int block, followers;
  };
  std::vector<Split> splits;
  for (int blk = 0; blk < blocks; ++blk) {
    ra::Run r{};
    r.per = per;
    r.whole = ra::whole_steps(per, tile);
    r.begin = blk * per < total ? blk * per : total;
    r.end = r.begin + per < total ? r.begin + per : total;
    for (int b = 0; b < c.B; ++b)
      if (r.begin >= base[b] && r.begin < base[b] + work(b).total) r.b = b, r.base = base[b];
    ra::Walk<decltype(work)> walk(work, r, c.B, c.Hkv);
    ra::Segment s;
    int segments = 0, split_here = 0;
    while (walk.next(s)) {
      const ra::SeqWork w = work(s.b);
      const int n = w.tiles > s.tile ? w.tile_steps(s.tile) : 0;
      if (s.h < 0 || s.h >= c.Hkv || s.tile < 0 || s.tile >= w.tiles || s.s0 < 0 ||
          s.s0 >= s.s1 || s.s1 > n)
        return fail("segment range", blk, s.b, s.s0);
      const long long item = base[s.b] + s.h * w.per_head + w.steps_before(s.tile);
      if (n <= r.whole && (s.s0 != 0 || s.s1 != n)) return fail("short item split", blk, s.b, n);
      if (w.steps_before(s.tile + 1) - w.steps_before(s.tile) != n)
        return fail("steps_before", s.b, s.tile, n);
      // the tile's steps hold every key that one of its rows sees
      const long long row0 = (long long)s.tile * tile, rows = (long long)w.qn * w.G;
      const long long row1 = row0 + tile < rows ? row0 + tile - 1 : rows - 1;
      const ra::KeyRange k0 = ra::row_keys(c, w, row0, w.G), k1 = ra::row_keys(c, w, row1, w.G);
      if (s.key0 % ra::kBlock || s.key0 < 0 || (k0.lo < k0.hi && s.key0 > k0.lo) ||
          k1.hi > s.key0 + (long long)n * ra::kStep)
        return fail("keys outside the steps", s.b, s.tile, k1.hi);
      for (int k = s.s0; k < s.s1; ++k) {
        if (seen[(size_t)(item + k)]++) return fail("step twice", blk, s.b, k);
        owner[(size_t)(item + k)] = blk;
      }
      // a block's partial slots: only its first segment may come over, only its last go on
      if (!s.first && segments > 0) return fail("came over late", blk, s.b, s.s0);
      if (split_here) return fail("segment after one that goes on", blk, s.b, s.s0);
      if (!s.last) split_here = 1;
      if (s.first && !s.last) {
        if (s.followers < 1) return fail("no followers", blk, s.b, s.s0);
        splits.push_back({item + n, blk, s.followers});
      } else if (s.followers) {
        return fail("followers of a whole item", blk, s.b, s.followers);
      }
      ++segments;
    }
  }
  for (long long k = 0; k < total; ++k)
    if (!seen[(size_t)k]) return fail("step missed", k, total, blocks);
  for (const Split& s : splits)
    if (owner[(size_t)(s.item_end - 1)] != s.block + s.followers)
      return fail("followers", s.block, s.followers, s.item_end);
  return 0;
}

int main() {
  ra::CacheDims c{};
  c.Hq = 8, c.Hkv = 2, c.d = 128, c.pages = 1 << 20, c.page_blocks = 4, c.max_pages = 4096;
  c.causal = 1, c.max_q = 1 << 20, c.T = 1 << 20, c.scale = 0.1f;
  // lengths from nothing to long, more sequences than a block has threads, other kernels'
  // sequences and faulty ones in between
  unsigned seed = 12345;
  auto rnd = [&](int n) { return (int)((seed = seed * 1664525u + 1013904223u) >> 8) % n; };
  for (int trial = 0; trial < 400; ++trial) {
    c.Hkv = 1 + trial % 2, c.Hq = c.Hkv * (1 + rnd(8));
    c.B = trial % 7 == 0 ? 1 : 1 + rnd(trial % 5 == 0 ? 300 : 20);
    c.window = trial % 4 == 1 ? 1 + rnd(5000) : 0;
    c.causal = trial % 6 != 5 || c.window;
    Batch t;
    t.indptr.push_back(trial % 3 == 0 ? rnd(5) : 0);
    for (int b = 0; b < c.B; ++b) {
      const int kind = rnd(10);
      const int qn = kind == 0 ? 0 : kind < 6 ? 1 : 1 + rnd(kind < 9 ? 40 : 2000);
      t.indptr.push_back(t.indptr.back() + qn);
      const int len = rnd(8);
      t.kv.push_back(len == 0 ? 0 : len < 5 ? rnd(600) : len < 7 ? rnd(60000) : 262145 + rnd(9));
    }
    for (int tile : {1, 8, 16, 256})
      for (int blocks : {1, 148, 592}) {
        if (check_cut(c, t, blocks, tile, 1 + trial % 3, 0, 1ll << 62)) return 1;
        if (check_cut(c, t, blocks, tile, 1, 64, 1ll << 62)) return 1;
        if (check_cut(c, t, blocks, tile, 2, 0, 64)) return 1;
      }
  }
  for (int a : {1, 2})
    for (int m = 1; m < 40; ++m) {
      long long sum = 0;
      for (int t = 0; t < 300; ++t) {
        sum += (long long)a * t / m;
        if (ra::floor_sum(t, a, m) != sum) return fail("floor_sum", t, a, m);
      }
    }
  c.Hq = 8, c.Hkv = 2;
  // faults: nothing of a faulty sequence is ever followed
  c.B = 1, c.window = 0, c.causal = 1, c.T = 100, c.max_q = 50, c.max_pages = 4, c.pages = 7;
  struct F { int q0, q1, L, want; };
  for (const F& f : {F{0, 10, 256, 0}, F{0, 10, 257, RA_CACHE_BAD_LENGTH},
                     F{0, 10, -1, RA_CACHE_BAD_LENGTH}, F{-1, 10, 20, RA_CACHE_BAD_INDPTR},
                     F{10, 9, 20, RA_CACHE_BAD_INDPTR}, F{60, 101, 50, RA_CACHE_BAD_INDPTR},
                     F{0, 51, 60, RA_CACHE_BAD_INDPTR}, F{50, 100, 0, 0}, F{5, 5, 0, 0}}) {
    if (ra::sequence_fault(c, f.q0, f.q1, f.L) != f.want) return fail("fault", f.q0, f.q1, f.L);
    if (f.want && ra::seq_work(c, f.q0, f.q1, f.L, 8, 0, 1 << 20).total)
      return fail("faulty sequence has work", f.q0, f.q1, f.L);
  }
  for (int page : {0, 6}) if (!ra::page_ok(c, page)) return fail("page_ok", page, 0, 0);
  for (int page : {-1, 7, 1 << 30, -2147483647 - 1})
    if (ra::page_ok(c, page)) return fail("page followed", page, 0, 0);
  // visible keys: never outside 0..L, empty before the first cached token
  for (int L : {0, 1, 5, 300})
    for (int qn : {1, 3, 9})
      for (int win : {0, 1, 4, 1000})
        for (int causal : {0, 1}) {
          if (win && !causal) continue;
          c.causal = causal, c.window = win, c.max_pages = 100;
          const ra::SeqWork w = ra::seq_work(c, 0, qn, L, 8, 0, 1 << 20);
          for (int row = 0; row < qn * 4; ++row) {
            const ra::KeyRange k = ra::row_keys(c, w, row, 4);
            const int pos = L - qn + row / 4;
            int n = 0;
            for (int j = 0; j < L; ++j) {
              const bool see = !causal || (j <= pos && (!win || j > pos - win));
              n += see;
              if (see != (j >= k.lo && j < k.hi)) return fail("row_keys", L, row, j);
            }
            if (n == 0 && k.lo < k.hi) return fail("empty row", L, row, k.lo);
          }
        }
  // offsets past 32 bits: the last byte of the last block of the largest cache
  c.pages = 1 << 30, c.Hkv = 1024, c.page_blocks = 256, c.d = 128;
  const long double bytes = (long double)c.pages * c.Hkv * c.page_blocks * ra::block_bytes(128);
  if ((long double)ra::block_at(c, c.pages - 1, c.Hkv - 1, c.page_blocks - 1) +
          ra::block_bytes(128) != bytes)
    return fail("block_at", 0, 0, 0);
  if (ra::block_bytes(64) != 1152 || ra::block_bytes(128) != 2304 || ra::block_bytes(64) % 16)
    return fail("block_bytes", ra::block_bytes(64), ra::block_bytes(128), 0);
  std::printf("ok\n");
  return 0;
}
