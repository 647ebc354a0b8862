// The work lists of the 4-bit and the latent decode, cut into ranges.
#pragma once

namespace pkv {

// A list of `total` entries cut into `parts` ranges whose sizes differ by one at
// most, with one division.
struct EvenSplit {
  long long size;  // of a range behind the first `longer`, which have one more
  int longer, parts;
  __device__ __forceinline__ EvenSplit(long long total, int n) : parts(n) {
    size = (long long)((unsigned long long)total / unsigned(n));
    longer = int(total - size * n);
  }
  __device__ __forceinline__ long long begin(int part) const { return part * size + (part < longer ? part : longer); }
  // The range of entry x (0 <= x < total).
  __device__ __forceinline__ int of(long long x) const {
    const long long rest = x - longer * (size + 1);
    int part = rest < 0 ? int(float(x) / float(size + 1)) : longer + int(float(rest) / float(size));
    part = min(parts - 1, part);  // but for the quotient's rounding
    while (part > 0 && begin(part) > x) --part;
    while (part + 1 < parts && begin(part + 1) <= x) ++part;
    return part;
  }
};

}  // namespace pkv
