// Which form of the 4-bit products serves a call, and how much of x a cluster's CTA stages.  Plain C++ on 64-bit
// sizes: channels go up to 2^28, so that a share's bytes pass 32 bits.
#pragma once
#include <cstdint>

namespace csa2 {
namespace mv {
namespace tc {

constexpr int kPlanChan = 128;             // channels of a block
constexpr int64_t kXBytes = 128 * 1024;    // x staged by a CTA, at most

// Bytes of x that each of C CTAs stages for `tok` token rows of n_kb channel blocks (f16, in whole kilobytes).
inline int64_t x_bytes(int64_t n_kb, int C, int tok) {
  return ((n_kb + C - 1) / C * tok * kPlanChan * 2 + 1023) / 1024 * 1024;
}
// Four CTAs share the channels (two and eight measured slower), or eight, where four do not hold x: up to 32768
// channels for 16 rows, 16384 for 32.  0: no cluster holds x, or has a channel block for each CTA.
inline int cluster(int64_t n_kb, int tok) {
  for (int C = 4; C <= 8; C *= 2)
    if (C <= n_kb && x_bytes(n_kb, C, tok) <= kXBytes) return C;
  return 0;
}

struct Plan {
  int tok, C;  // token rows of a pass (16 or 32) and CTAs of a cluster; tok = 0: matvec_kernel
};
// The tensor-memory form where there is enough weight to pay for its set-up.  Measured, us, this form against the
// other: 32 rows x 16384 x 8192 29 / 65, 24 x 4096 x 4096 10.6 / 12.6, 32 x 512 x 4096 9.5 / 9.3,
// 16 x 16384 x 8192 25 / 30, 16 x 8192 x 4096 11.8 / 12.0, 8 x 16384 x 8192 25 / 20.
inline Plan plan(int m, int64_t n_rb, int64_t n_kb) {
  const int64_t blocks = n_rb * n_kb;
  if (!((m > 16 && blocks >= 2048) || (m > 8 && blocks >= 16384))) return {0, 0};
  if (m > 16)
    if (const int C = cluster(n_kb, 32)) return {32, C};
  // more channels of 32 rows than a cluster holds: 16 rows at a time (4096 x 32768 68 us, the other form 100)
  if (const int C = cluster(n_kb, 16)) return {16, C};
  return {0, 0};
}

}  // namespace tc
}  // namespace mv
}  // namespace csa2
