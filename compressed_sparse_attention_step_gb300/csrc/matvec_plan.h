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
// channels for 16 rows, 16384 for 32.  0: no cluster holds x.
inline int cluster(int64_t n_kb, int tok) {
  for (int C = 4; C <= 8; C *= 2)
    if (x_bytes(n_kb, C, tok) <= kXBytes) return C;
  return 0;
}

struct Plan {
  int tok, C;  // token rows of a pass (16 or 32) and CTAs of a cluster; tok = 0: matvec_kernel
};
// The tensor-memory form where there is enough weight to pay for its set-up, and enough channels to pay for a step's
// end.  Measured, us, this form against the other, weights from HBM (rows x outputs x channels):
//   17 x  4096 x 4096  9.9 / 10.2   17 x 2048 x 4096  9.5 /  8.5   17 x 8192 x 2048 11.1 /  9.5   17 x 16384 x 512 14.7 / 7.8
//   24 x  4096 x 4096 10.7 / 10.9   24 x 2048 x 4096 10.3 /  9.1   24 x 8192 x 2560 12.8 / 11.0   24 x 1024 x 4096 10.2 / 7.4
//   32 x  4096 x 4096 11.1 / 12.8   32 x 2048 x 4096 10.5 / 11.1   32 x 8192 x 2048 12.3 / 11.6   32 x 16384 x 1024 16.5 / 13.2
//   32 x 8192 x 8192 18.8 / 28.2    32 x 512 x 16384 12.9 / 16.2   32 x 16384 x 2560 19.3 / 21.9  32 x 1024 x 4096 10.4 / 8.7
//    9 x 16384 x 8192 24.9 / 25.4    9 x 8192 x 8192 15.8 / 15.6    9 x 8192 x 6144 13.8 / 13.1    9 x 16384 x 4096 17.0 / 15.7
//   16 x 16384 x 8192 24.9 / 27.5   16 x 8192 x 8192 15.9 / 16.5   16 x 8192 x 6144 13.9 / 14.1   16 x 16384 x 4096 17.1 / 16.9
//   16 x 32768 x 2048 23.7 / 18.0    8 x 16384 x 8192 25 / 20
inline Plan plan(int m, int64_t n_rb, int64_t n_kb) {
  const int64_t blocks = n_rb * n_kb;
  const bool many = m > 16 && blocks >= 2048 && n_kb >= (m > 24 ? 16 : 32);
  if (!many && !(m > 8 && blocks >= 16384 && n_kb >= 64)) return {0, 0};
  if (m > 16)
    if (const int C = cluster(n_kb, 32)) return {32, C};
  // more channels of 32 rows than a cluster holds: 16 rows at a time (4096 x 32768 68 us, the other form 100)
  if (const int C = cluster(n_kb, 16)) return {16, C};
  return {0, 0};
}

}  // namespace tc
}  // namespace mv
}  // namespace csa2
