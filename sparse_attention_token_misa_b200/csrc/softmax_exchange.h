// What the softmax warpgroups of latent_mla.cu tell one another through shared
// memory, and the named barriers that order it.
//
// Two warpgroups of 128 threads take a cluster's tiles in turn (tile number n: group
// n & 1).  Threads tid and tid ^ 64 of a group have the same head and one half of a
// tile's rows each.  Three places, each written and read over and over:
//   maxima     [group][128]: a tile's maximum of a thread's half, read by the other half.
//   reference  [group][64]: a head's reference m after a tile, read at the next one.
//   sums       [turn][128]: an item's sums of the group that does not finish it.
//
// A place may be written again once all that read it have arrived at a barrier that
// the writer waits at:
//   maxima     read at tile n, written by the same group at n + 2.  Between them all its
//              threads pass the reference barrier of tile n - 1 (behind the read) or, at
//              the cluster's first tile, which has none, the maxima barrier once more.
//   reference  read at tile n + 1 before that tile's arrival, which the writer waits for
//              at n + 2 before it writes.
//   sums       read when item i is finished, written at item i + 2 at the earliest: item
//              i + 1 has a tile of the group that finished i, or is handed over by it.
// tests/test_softmax_exchange.py runs this file's code on the host and looks for
// accesses that no barrier orders.
//
// Io: store / load (offset in the exchange area, 32 bits), sync and arrive (barrier,
// threads).  The kernel's is shared memory and bar.sync / bar.arrive.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define MISA_EXCHANGE_FN __device__ __forceinline__
#else
#define MISA_EXCHANGE_FN inline
#endif

namespace misa {

constexpr int kBarMax = 1, kBarRef = 3, kBarSum = 5;   // barriers by group, by group, by turn
constexpr uint32_t kExMax = 0, kExRef = kExMax + 1024, kExSum = kExRef + 512, kExBytes = kExSum + 1024;

template <class Io>
struct SoftmaxExchange {
  Io io;
  uint32_t group;
  int tid;   // in the warpgroup

  // The tile's maximum in the other half of its rows.
  MISA_EXCHANGE_FN uint32_t other_half(uint32_t max_here) {
    io.store(kExMax + group * 512 + tid * 4, max_here);
    io.sync(kBarMax + group, 128);
    return io.load(kExMax + group * 512 + (tid ^ 64) * 4);
  }
  // The head's reference after tile n - 1, `none` at an item's first tile.
  MISA_EXCHANGE_FN uint32_t reference_before(uint32_t n, uint32_t first, uint32_t none) {
    if (n > 0) {
      io.sync(kBarRef + (group ^ 1u), 256);
      if (n > first) none = io.load(kExRef + (group ^ 1u) * 256 + (tid & 63) * 4);
    } else {
      io.sync(kBarMax + group, 128);   // in its place: this tile's maxima have been read
    }
    return none;
  }
  MISA_EXCHANGE_FN void set_reference(uint32_t m) {
    if (tid < 64) io.store(kExRef + group * 256 + (tid & 63) * 4, m);
    io.arrive(kBarRef + group, 256);
  }
  // An item's sums to the group that finishes it.
  MISA_EXCHANGE_FN void hand_over(uint32_t turn, uint32_t sum) {
    io.store(kExSum + turn * 512 + tid * 4, sum);
    io.arrive(kBarSum + turn, 256);
  }
  // Finishing it: this group's sum of the other half (the maxima's place is free
  // behind the first barrier, and again behind the last), then the other group's
  // of both.
  MISA_EXCHANGE_FN uint32_t other_half_sum(uint32_t turn, uint32_t sum) {
    io.sync(kBarMax + group, 128);
    io.store(kExMax + group * 512 + tid * 4, sum);
    io.sync(kBarSum + turn, 256);
    const uint32_t other = io.load(kExMax + group * 512 + (tid ^ 64) * 4);
    io.sync(kBarMax + group, 128);
    return other;
  }
  MISA_EXCHANGE_FN uint32_t handed_over(uint32_t turn, int half) {   // 0: this thread's, 1: the other half's
    return io.load(kExSum + turn * 512 + (tid ^ (half * 64)) * 4);
  }
};

}  // namespace misa
