// Index arithmetic of decode.h at the ends of its ranges, on the host: prints
// "ok", or the first value that is wrong.
#include <cstdio>
#include <cstdlib>

#include "../int8_quantized_amd/csrc/decode.h"

using namespace q8ta;

static uint64_t state = 88172645463325252ull;
static uint64_t next() {
  state ^= state << 13;
  state ^= state >> 7;
  state ^= state << 17;
  return state;
}

static void division(uint32_t d) {
  const FastDiv f = make_fastdiv(d);
  const uint32_t last = 0x7fffffffu;
  auto check = [&](uint64_t n) {
    if (n <= last && fast_div((uint32_t)n, f) != (uint32_t)n / d) {
      printf("%llu / %u\n", (unsigned long long)n, d);
      exit(1);
    }
  };
  for (uint64_t n : {(uint64_t)0, (uint64_t)1, (uint64_t)last, (uint64_t)last - 1, (uint64_t)d - 1, (uint64_t)d, (uint64_t)d + 1})
    check(n);
  const uint64_t most = last / d;
  for (int i = 0; i < 300; ++i) {   // next to multiples, the largest among them
    const uint64_t m = (i < 50 ? most - (i < (int)most ? i : 0) : next() % (most + 1)) * d;
    if (m) check(m - 1);
    check(m);
    check(m + d - 1);
  }
}

static void ends(int64_t total, int64_t grain) {
  const int grains = total < 1 ? 1 : (int)((total - 1) / grain + 1);
  for (int64_t g1 : {(int64_t)1, (int64_t)grains / 2, (int64_t)grains - 1, (int64_t)grains}) {
    if (g1 < 1 || g1 > grains) continue;
    const int64_t want = total < g1 * grain ? total : g1 * grain;
    if (grains_end((int)total, grains, (int)grain, (int)g1) != want) {
      printf("end of %lld x %lld of %lld\n", (long long)g1, (long long)grain, (long long)total);
      exit(1);
    }
  }
}

int main() {
  const uint32_t most = 0x7fffffffu;
  for (uint32_t d = 1; d <= 5000; ++d) division(d);
  for (int b = 1; b < 31; ++b)
    for (int o = -2; o <= 2; ++o)
      if (((int64_t)1 << b) + o >= 1) division((1u << b) + o);
  for (int i = 0; i < 20000; ++i) division(1 + (uint32_t)(next() % most));
  division(most);
  const int64_t longest = ((int64_t)1 << 31) - 1024;   // the cache rows of a request
  for (int64_t grain = 64; grain < longest; grain *= 2)
    for (int64_t t : {(int64_t)0, (int64_t)1, grain - 1, grain, grain + 1, longest / 2, longest - 1, longest})
      ends(t, grain);
  ends(longest, longest);
  for (int i = 0; i < 100000; ++i) ends((int64_t)(next() % (longest + 1)), 1 + (int64_t)(next() % longest));
  puts("ok");
}
