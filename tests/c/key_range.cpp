// The narrowing of key_range.h over random keys, to the border and the number of keys that stay, against sorted keys.
#include "key_range.h"

#include <algorithm>
#include <cstdio>
#include <cstring>
#include <random>
#include <vector>

constexpr uint32_t kNan = 0xfffffffeu;         // the largest key of a slot that is not protected

static uint32_t key_of(float w) {
  uint32_t b;
  std::memcpy(&b, &w, 4);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}

// Whether the loop ends with as many keys kept as there should be, from the largest on.
static bool check(const std::vector<uint32_t>& keys, int keep, int which) {
  sa::KeyRange r{*std::min_element(keys.begin(), keys.end()), *std::max_element(keys.begin(), keys.end())};
  int left = keep, equal = (int)keys.size();
  uint32_t border = r.low;
  int rounds = 0;
  for (; left < equal && r.low < r.high; ++rounds) {
    const int shift = r.shift();
    std::vector<int> hist(sa::KeyRange::kBins, 0);
    for (uint32_t k : keys)
      if (r.holds(k)) ++hist.at(r.bin(k, shift));
    int above = 0, bin = sa::KeyRange::kBins - 1;
    while (above + hist.at(bin) < left) above += hist.at(bin--);
    r.take((uint32_t)bin, shift);
    left -= above;
    equal = hist[bin];
    border = r.low;
  }
  // keys above the border stay, and of those equal to it the first `left` (all, where they are as many)
  int more = 0, same = 0;
  for (uint32_t k : keys) {
    more += k > border;
    same += k == border;
  }
  const int kept = left < equal ? more + std::min(same, left) : more + same;
  std::vector<uint32_t> sorted = keys;
  std::sort(sorted.begin(), sorted.end(), std::greater<uint32_t>());
  const uint32_t last = sorted[keep - 1];      // the smallest key that stays
  const bool ok = kept == keep && rounds <= 3 && border <= last && (left == equal || border == last);
  if (!ok) std::printf("set %d, %zu keys, keep %d: border %08x kept %d (last %08x), %d rounds\n", which, keys.size(), keep, border, kept, last, rounds);
  return ok;
}

int main() {
  std::mt19937 gen(1);
  int wrong = 0, sets = 0;
  for (int i = 0; i < 20000; ++i, ++sets) {
    const int n = 2 + (int)(gen() % 60), nans = (int)(gen() % (n + 1)), kind = (int)(gen() % 6);
    std::vector<uint32_t> keys(n);
    std::exponential_distribution<float> positive(1.0f);
    std::normal_distribution<float> any(0.0f, 2.0f);
    for (uint32_t& k : keys) switch (kind) {
        case 0: k = key_of(positive(gen)); break;                    // gathered weights
        case 1: k = key_of(any(gen)); break;
        case 2: k = std::min((uint32_t)gen(), kNan); break;                     // any key
        case 3: k = kNan - (uint32_t)(gen() % 3000); break;                       // the top of the range
        case 4: k = (uint32_t)(gen() % 3000); break;                              // the bottom
        default: k = key_of(0.5f + 1e-6f * (float)(gen() % 9)); break;  // close together, ties
      }
    for (int j = 0; j < nans; ++j) keys[j] = kNan;
    std::shuffle(keys.begin(), keys.end(), gen);
    const int keep = 1 + (int)(gen() % (n - 1));
    if (!check(keys, keep, i) && ++wrong == 10) break;
  }
  std::printf("%d of %d sets wrong\n", wrong, sets);
  return wrong != 0;
}
