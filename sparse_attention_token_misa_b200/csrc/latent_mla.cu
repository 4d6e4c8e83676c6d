// Attention over a latent cache held in 16, 8 or 4 bits: the listed rows of each
// query, or all rows of its prefix (include/misa_latent.h), on the 5th-generation
// tensor cores.
//
//   out[t, h] = sum_i p_i v_i / sum_i p_i,  p_i = exp(scale * q[t, h] . k_i)
//
// A query's 128 heads need 147 KB of queries and 256 KB of fp32 output at once,
// more than one SM holds beside the rows.  So a cluster of two CTAs takes a query
// (or a part of its rows), 64 heads each, and their tensor cores work as a pair
// (cta_group::2, M = 128): each CTA brings half of the operand that both multiply
// by, which halves the shared memory reads that bound a 64-head tile otherwise.
//
// Rows come in tiles of 64.  Per tile:
//  1. CTA u brings rows [32 u, 32 u + 32) of the tile to shared memory as bf16, in 9
//     blocks of 64 entries: quantised rows widened (exactly) in registers, bf16 rows
//     by TMA.  S = Q K^T reads these blocks.  S in TMEM: lane l < 64 has head l
//     against rows 0..31, lane 64 + l the same head against rows 32..63.
//  2. Softmax in one pass with a running reference m: when a tile's maximum is
//     more than 2^8 above 2^m, the sums so far are scaled and m moves (p stays
//     below 2^8, exact enough in bf16 and fp32).  p goes to shared memory as bf16.
//  3. O += P V needs entries [256 u, 256 u + 256) of all 64 rows in CTA u: eight
//     warps of each CTA write the blocks it brought to the CTA that multiplies them,
//     from registers (rows of 64 entries in 128-byte swizzled atoms serve both
//     products, K-major in one and MN-major in the other).  So a row is read from L2
//     and widened once.  O stays in TMEM, 256 columns.
// Every operand has two stages and S four places: a tile's way from its rows through
// the softmax to O takes about 6000 cycles, three times its share of the tensor cores
// (with one stage of 128 rows, or S held back until the O before it, the latency of
// that way was the speed: mx8 3.4 us for 128 rows).
//
// What bounds a tile is shared memory, which both products read at its full rate:
// S 36 x 24 cycles (queries and rows, 3 KB at 128 bytes a cycle), O 4 x 2 x 48, and
// rows and values written (bf16: and copied) once more, about 2000 cycles in all.
// Measured, 74 queries of one cache, for 128 rows of it: bf16 2.1 us (1.26 PFLOP/s,
// 0.76 of cuBLAS's measured rate in a burst, 0.90 of its sustained one), mx8 2.5 to
// 2.7, mx4 2.4 to 2.7, where the eight warps that widen rows take longer than that.  More of them were slower (16: mx8 2.9), and so were
// spilled registers: shared memory leaves L1 little room for a stack.
//
// A cluster stays on its SMs and takes one item in 74 (a query, or a part of its
// rows), each role on its own: the rows of the next item come while the output of
// this one leaves.  (A cluster an item spent 9 us on starting, queries and output
// around 3 us a tile; now an item costs 3 to 4 besides its tiles.)  Few queries: the rows of each are split
// over several items, whose partial sums a second kernel joins in a fixed order.
//
// Roles (640 threads a CTA): two warpgroups softmax and output (what they tell one
// another, and in what order, is in softmax_exchange.h), eight warps that bring
// quantised rows or copy bf16 ones, one warp that has TMEM and, in the first CTA,
// issues S, one that issues O, and two that ask for what comes by TMA and pass on what
// has landed.  Shared memory is addressed from one 32-bit base: with a pointer a
// barrier the kernel spilled.  Code is kept small (loops, not copies): at 140 KB the
// instruction caches, which many SMs share, halved the speed.  Waits are bounded.
#include <algorithm>

#include "kv_format.cuh"
#include "launch.h"
#include "misa_device.cuh"
#include "softmax_exchange.h"

namespace misa {

namespace {

constexpr int kDqk = MISA_MLA_DQK, kDv = MISA_MLA_DV;
constexpr int kTile = 64;                         // rows of a tile
constexpr int kRows = 32;                         // ... that one CTA brings
constexpr int kHeads = 64;                        // heads of a CTA
constexpr int kBlocks = kDqk / 64;                // 9
constexpr uint32_t kQBlock = kHeads * 128;        // 64 heads x 64 entries
constexpr uint32_t kKBlock = kRows * 128;         // 32 rows x 64 entries
constexpr uint32_t kVBlock = kTile * 128;         // 64 rows x 64 entries
constexpr uint32_t kKStage = kBlocks * kKBlock;   // S operand: the CTA's rows
constexpr uint32_t kVStage = 4 * kVBlock;         // O operand: 256 entries of all rows
constexpr uint32_t kPStage = kHeads * 128;
constexpr uint32_t kOffQ = 0;
constexpr uint32_t kOffK = kOffQ + kBlocks * kQBlock;   // [2]: stage = a tile's number modulo 2
constexpr uint32_t kOffV = kOffK + 2 * kKStage;         // [2]
constexpr uint32_t kOffP = kOffV + 2 * kVStage;         // [2]
// barriers, one a stage (of the first CTA where it says so)
constexpr uint32_t kKFull = kOffP + 2 * kPStage;  // first CTA: quantised rows brought by both, bf16 ones by the other
constexpr uint32_t kKHere = kKFull + 16;          // bf16: this CTA's rows landed
constexpr uint32_t kKEmpty = kKHere + 16;         // multiplied
constexpr uint32_t kCopied = kKEmpty + 16;        // bf16: read by those that copy to O's operand
constexpr uint32_t kVFull = kCopied + 16;         // first CTA: both CTAs' values are there
constexpr uint32_t kVLanded = kVFull + 16;        // this CTA's values of the other one's rows
constexpr uint32_t kVEmpty = kVLanded + 16;       // multiplied
constexpr uint32_t kSFull = kVEmpty + 16;         // [4] S complete
constexpr uint32_t kSEmpty = kSFull + 32;         // [4] first CTA: S read by both
constexpr uint32_t kPFull = kSEmpty + 32;         // first CTA: P written (and O scaled) by both
constexpr uint32_t kPvDone = kPFull + 16;         // O += P V complete
constexpr uint32_t kOEmpty = kPvDone + 16;        // (one) first CTA: O of the item before read by both
constexpr uint32_t kQFull = kOEmpty + 8;          // (one) this CTA's queries landed
constexpr uint32_t kQReady = kQFull + 8;          // (one) first CTA: queries landed (bf16: the other CTA's)
constexpr uint32_t kQEmpty = kQReady + 8;         // (one) the item's last S complete
constexpr uint32_t kDone = kQEmpty + 8;           // (one) every MMA of both warps that issue them retired
constexpr uint32_t kOffTmem = kDone + 8;
constexpr uint32_t kOffExchange = (kOffTmem + 8 + 15) / 16 * 16;   // maxima, references, sums (softmax_exchange.h)
constexpr int kSmemBytes = kOffExchange + kExBytes;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
// Warps: 0-7 softmax and output, 8-15 bring quantised rows or copy bf16 ones, 16-19 the rest.
constexpr int kRowWarp0 = 8, kRowWarps = 8, kMmaWarp = kRowWarp0 + kRowWarps;
constexpr int kThreads = (kMmaWarp + 4) * 32;
constexpr uint32_t kTmemS = 256;                  // O: columns 0..255, S: four places of 32 columns
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 64);
constexpr uint32_t kIdescO = idesc_bf16_f32(128, 256) | (1u << 16);   // values MN-major

// ---------------------------------------------------------------- shared memory by address
__device__ __forceinline__ void bar_init(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
__device__ __forceinline__ void arrive_here(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.release.cta.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}
// Arrive on CTA `rank`'s barrier.  The release is the CTA's: what this warp wrote is
// its own CTA's shared memory, which its own SM's tensor core reads, and
// fence.proxy.async has ordered that.  (A release of the cluster's scope would wait
// for the loads under way and for a round trip to L2, about 1000 cycles.)
__device__ __forceinline__ void arrive_in(uint32_t bar, uint32_t rank) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, %1;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(bar),
      "r"(rank)
      : "memory");
}
// The address of the same place in CTA `rank`, and a 16-byte store there that a
// barrier of that CTA counts.
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, uint32_t rank) {
  uint32_t a;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(addr), "r"(rank));
  return a;
}
__device__ __forceinline__ void st_async16(uint32_t remote, uint4 v, uint32_t remote_bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];" ::"r"(remote),
               "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(remote_bar)
               : "memory");
}
// Whether the phase of `parity` is over (may sleep a while first).
__device__ __forceinline__ bool try_phase(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\tmbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
__device__ __forceinline__ uint32_t ld_shared(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared(uint32_t a, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(a), "r"(v) : "memory");
}
__device__ __forceinline__ void st_shared16(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
// Waits until the phase of `parity` is over; gives up after about two seconds
// (counted in cycles: the nanosecond timer is read through the pipe that the
// softmax's exponentials need).
constexpr uint32_t kWaitCycles = 3900000000u, kDrainCycles = 20000000u;
__device__ __forceinline__ bool wait_one(uint32_t bar, uint32_t parity, uint32_t* err) {
  if (try_phase(bar, parity)) return true;
  const uint32_t t0 = clock();
  while (!try_phase(bar, parity))
    if (static_cast<uint32_t>(clock()) - t0 > kWaitCycles) {
      record_error(err, MISA_DEVERR_TIMEOUT);
      return false;
    }
  return true;
}
// The wait at the end of a cluster's work, which may take as long as all of it: its
// limit counts from the last time that O went on.
__device__ __forceinline__ bool wait_all(uint32_t sb, uint32_t* err) {
  uint32_t t0 = clock();
  bool seen = try_phase(sb + kPvDone, 0);
  while (!try_phase(sb + kDone, 0)) {
    const bool now = try_phase(sb + kPvDone, 0);
    if (now != seen) t0 = clock();
    seen = now;
    if (static_cast<uint32_t>(clock()) - t0 > kWaitCycles) {
      record_error(err, MISA_DEVERR_TIMEOUT);
      return false;
    }
  }
  return true;
}
// A wait of a whole warp: one outcome for all lanes.
__device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity, uint32_t* err) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, err));
}

// ---------------------------------------------------------------- the pair
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.relaxed.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// One product with operands kA and kB bytes behind those of the descriptors (added
// here: worked out ahead of the loop, the descriptors of a tile fill the registers).
template <uint32_t kA, uint32_t kB>
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "add.s64 x, %1, %5;\n\tadd.s64 y, %2, %6;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "n"(kA >> 4), "n"(kB >> 4)
      : "memory");
}
// Arrive on this barrier of both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint32_t bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(bar),
      "h"(static_cast<uint16_t>(3))
      : "memory");
}
__device__ __forceinline__ bool elect_one() {
  uint32_t e;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(e));
  return e != 0;
}
__device__ __forceinline__ uint64_t sw128_mnmajor_desc(uint32_t smem_addr, uint32_t lbo) {
  return static_cast<uint64_t>((smem_addr >> 4) & 0x3FFFu) | (static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16) |
         (static_cast<uint64_t>(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
__device__ __forceinline__ void tma_2d(uint32_t dst, const void* map, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void tma_3d(uint32_t dst, const void* map, uint32_t bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(dst),
      "l"(map), "r"(bar), "r"(x), "r"(y), "r"(z)
      : "memory");
}
__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  tmem_ld16(taddr, r);
  tmem_ld16(taddr + 16, r + 16);
}
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm volatile("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));   // (in order: it keeps the registers down)
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void tma_l2_3d(const void* map, int x, int y, int z) {
  asm volatile("cp.async.bulk.prefetch.tensor.3d.L2.global.tile [%0, {%1, %2, %3}];" ::"l"(map), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// ---------------------------------------------------------------- items
struct MlaParams {
  LatentArgs a;
  int nsplit, items; // items: T * nsplit
  uint32_t by_nsplit;   // ceil(2^32 / nsplit) (nsplit > 1)
  float* part_o;     // [T][nsplit][512 / 4][Hq][4] (nsplit > 1)
  float* part_ml;    // [T][nsplit][Hq][2]: m (log2 units), l
};
// An item: tiles [tile0, tile1) of the n row slots of query t.  Items run from the last
// query to the first: a prompt's later queries have more rows, and short lists end evenly.
struct Work {
  int t, split;
  int n, tile0, tile1;
  int seq;
  const uint8_t* base;      // cache of the query's sequence
  const int32_t* idx;       // its listed rows, or NULL: slot s is row s
  int L;
};
// n / nsplit, exact for n * nsplit < 2^32.
__device__ __forceinline__ int over_splits(const MlaParams& p, int n) {
  return p.nsplit == 1 ? n : static_cast<int>(__umulhi(static_cast<uint32_t>(n), p.by_nsplit));
}
// What global memory says of an item; read early, looked at when the item starts.
struct Peek {
  int t, seq, len;
};
__device__ __forceinline__ Peek peek(const MlaParams& p, int item) {
  Peek k = {0, 0, 0};
  if (item < p.items) {
    k.t = p.a.T - 1 - over_splits(p, item);
    k.seq = __ldg(p.a.seq_of + k.t);
    k.len = p.a.idx ? p.a.k : __ldg(p.a.prefix_len + k.t);
  }
  return k;
}
__device__ __forceinline__ Work work_of(const MlaParams& p, int item, Peek k) {
  Work w;
  w.t = k.t;
  w.split = item - (p.a.T - 1 - k.t) * p.nsplit;
  w.L = static_cast<int>(p.a.L);
  w.idx = p.a.idx ? p.a.idx + static_cast<int64_t>(w.t) * p.a.idx_stride : nullptr;
  w.n = p.a.idx ? k.len : max(min(k.len, w.L), 0);
  w.seq = k.seq;
  if (k.seq < 0 || k.seq >= p.a.nseq) w.seq = w.n = 0;
  w.base = static_cast<const uint8_t*>(p.a.cache) + static_cast<int64_t>(w.seq) * p.a.seq_stride;
  const int tiles = (w.n + kTile - 1) / kTile;
  const int share = over_splits(p, tiles + p.nsplit - 1);
  w.tile0 = min(w.split * share, tiles);
  w.tile1 = min(w.tile0 + share, tiles);
  return w;
}
// The items of a cluster, one after the other: there and back through the clusters, so
// that the first does not have the longest of every round of a prompt.
struct Round {
  int item, hop, next_hop;
  __device__ __forceinline__ Round() {
    const int c = static_cast<int>(blockIdx.x >> 1), clusters = static_cast<int>(gridDim.x >> 1);
    item = c;
    hop = 2 * (clusters - c) - 1;
    next_hop = 2 * c + 1;
  }
  __device__ __forceinline__ void next() {
    item += hop;
    const int h = hop;
    hop = next_hop;
    next_hop = h;
  }
};
// Those that have rows.
struct Items {
  Round r;        // of the item behind `w`
  Peek ahead;     // ... and what it is
  Work w;
  __device__ __forceinline__ explicit Items(const MlaParams& p) { ahead = peek(p, r.item); }
  // On to the next one.
  __device__ __forceinline__ bool next(const MlaParams& p) {
    do {
      if (r.item >= p.items) return false;
      w = work_of(p, r.item, ahead);
      r.next();
      ahead = peek(p, r.item);
    } while (w.tile1 == w.tile0);
    return true;
  }
};
// Row of slot s, -1 where there is none.
__device__ __forceinline__ int32_t row_of(const Work& w, int s) {
  if (s >= w.n) return -1;
  if (!w.idx) return s;
  const int32_t id = __ldg(w.idx + s);
  return id >= 0 && id < w.L ? id : -1;
}

template <int kFmt>
__device__ __forceinline__ uint2 load_code(const uint8_t* row, int entry) {   // 8 entries from `entry` on
  if (kFmt == MISA_KV_MX8) return __ldg(reinterpret_cast<const uint2*>(row + entry));
  return make_uint2(__ldg(reinterpret_cast<const uint32_t*>(row + entry / 2)), 0u);
}

// A tile's number over all items of the cluster: its stage and its phase there.
struct Turn {
  uint32_t n = 0;
  __device__ __forceinline__ uint32_t at() const { return 8 * (n & 1); }        // its barrier of two
  __device__ __forceinline__ uint32_t stage() const { return n & 1; }
  __device__ __forceinline__ uint32_t parity() const { return (n >> 1) & 1; }   // of the phase that ends with this tile
  __device__ __forceinline__ uint32_t before() const { return parity() ^ 1u; }  // of the one that ended two tiles ago
  // The same of S, which has four places.
  __device__ __forceinline__ uint32_t at4() const { return 8 * (n & 3); }
  __device__ __forceinline__ uint32_t place4() const { return n & 3; }
  __device__ __forceinline__ uint32_t parity4() const { return (n >> 2) & 1; }
};

// Brings quantised rows, 256 threads: thread = (row r0, piece of 8 entries) of each
// block.  A piece is widened once and written twice: to S's operand and, as soon as
// there is room, to O's in the CTA that multiplies it.  An absent row is any row's codes
// with scales of zero.  The codes of the next tile are asked for as soon as the
// registers are free: behind the first writes they came late (mx8, 16 x 32,768 rows:
// 178 and 192 us).
template <int kFmt>
__device__ __forceinline__ bool bring_rows(const MlaParams& p, uint32_t rank, int tid, uint32_t sb) {
  constexpr int kRow = kv_row_bytes(kFmt);
  const int r0 = tid >> 3, piece = tid & 7, own = static_cast<int>(rank) * kRows + r0;
  const uint32_t turn = (piece ^ (r0 & 7)) << 4;
  const uint32_t kdst0 = sb + kOffK + r0 * 128 + turn, vdst0 = sb + kOffV + own * 128 + turn;
  const uint32_t far0 = in_cta(vdst0, rank ^ 1u), far_bar0 = in_cta(sb + kVLanded, rank ^ 1u);
  const uint32_t sel = 0x4440u | (piece >> 2);   // the piece's byte of a block's two scale bytes
  Turn n;
  for (Items it(p); it.next(p);) {
    const Work& w = it.w;
    uint2 code[8];
    uint4 scale, rope;
    auto id_of = [&](int tile) {
      const int s = tile * kTile + own;
      return tile < w.tile1 && s < w.n ? w.idx ? __ldg(w.idx + s) : s : -1;
    };
    int32_t id = id_of(w.tile0);
    auto load = [&](int tile) {   // ask for this thread's pieces of a tile, and for its row of the one behind
      if (piece == 0 && (id < -1 || id >= w.L)) record_error(p.a.err, MISA_DEVERR_BAD_INDEX);
      const bool here = id >= 0 && id < w.L;
      const uint8_t* src = w.base + static_cast<int64_t>(here ? id : 0) * kRow;
#pragma unroll
      for (int b = 0; b < 8; ++b) code[b] = load_code<kFmt>(src, b * 64 + piece * 8);
      scale = rope = make_uint4(0u, 0u, 0u, 0u);
      if (here) {
        scale = __ldg(reinterpret_cast<const uint4*>(src + kv_code_bytes(kFmt)));
        rope = __ldg(reinterpret_cast<const uint4*>(src + kv_rope_offset(kFmt) + piece * 16));
      }
      id = id_of(tile + 1);
    };
    load(w.tile0);
#pragma unroll 1
    for (int tile = w.tile0; tile < w.tile1; ++tile, ++n.n) {
      uint4 y[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const uint32_t word = b < 2 ? scale.x : b < 4 ? scale.y : b < 6 ? scale.z : scale.w;
        y[b] = kv_decode8<kFmt>(code[b].x, code[b].y, kv_scale(__byte_perm(word, 0u, sel + 2 * (b & 1))));
      }
      const uint4 y8 = rope;
      load(tile + 1);
      if (!wait_warp(sb + kKEmpty + n.at(), n.before(), p.a.err)) return false;
      const uint32_t kdst = kdst0 + n.stage() * kKStage;
#pragma unroll
      for (int b = 0; b < 8; ++b) st_shared16(kdst + b * kKBlock, y[b]);
      st_shared16(kdst + 8 * kKBlock, y8);
      fence_proxy_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) arrive_in(sb + kKFull + n.at(), 0);
      if (!wait_warp(sb + kVEmpty + n.at(), n.before(), p.a.err)) return false;
      const uint32_t vofs = n.stage() * kVStage, far_bar = far_bar0 + n.at();
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if ((b >> 2) == static_cast<int>(rank)) st_shared16(vdst0 + vofs + (b & 3) * kVBlock, y[b]);
        else st_async16(far0 + vofs + (b & 3) * kVBlock, y[b], far_bar);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) arrive_in(sb + kVFull + n.at(), 0);
    }
  }
  return true;
}

// Copies this CTA's rows of a bf16 cache, 256 threads as above, to O's operand.
// Absent rows are cleared: P is 0 there, but 0 times a stale NaN is not.
__device__ __forceinline__ bool copy_rows(const MlaParams& p, uint32_t rank, int tid, uint32_t sb) {
  const int r0 = tid >> 3, piece = tid & 7, own = static_cast<int>(rank) * kRows + r0;
  const uint32_t turn = (piece ^ (r0 & 7)) << 4;
  const uint32_t src0 = sb + kOffK + r0 * 128 + turn, vdst0 = sb + kOffV + own * 128 + turn;
  const uint32_t far0 = in_cta(vdst0, rank ^ 1u), far_bar0 = in_cta(sb + kVLanded, rank ^ 1u);
  Turn n;
  for (Items it(p); it.next(p);)
#pragma unroll 1
    for (int tile = it.w.tile0; tile < it.w.tile1; ++tile, ++n.n) {
      if (!wait_warp(sb + kKHere + n.at(), n.parity(), p.a.err)) return false;
      uint4 y[8];
#pragma unroll
      for (int b = 0; b < 8; ++b) y[b] = ld_shared16(src0 + n.stage() * kKStage + b * kKBlock);
      if (tile * kTile + own >= it.w.n) {
#pragma unroll
        for (int b = 0; b < 8; ++b) y[b] = make_uint4(0u, 0u, 0u, 0u);
      }
      fence_proxy_async_smem();   // read before TMA may write there again
      __syncwarp();
      if ((threadIdx.x & 31) == 0) arrive_here(sb + kCopied + n.at());
      if (!wait_warp(sb + kVEmpty + n.at(), n.before(), p.a.err)) return false;
      const uint32_t vofs = n.stage() * kVStage;
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        if ((b >> 2) == static_cast<int>(rank)) st_shared16(vdst0 + vofs + (b & 3) * kVBlock, y[b]);
        else st_async16(far0 + vofs + (b & 3) * kVBlock, y[b], far_bar0 + n.at());
      }
      fence_proxy_async_smem();
      __syncwarp();
      if ((threadIdx.x & 31) == 0) arrive_in(sb + kVFull + n.at(), 0);
    }
  return true;
}

// Passes on to the first CTA what the other one has written here, a warp.
__device__ __forceinline__ bool pass_values(const MlaParams& p, int lane, uint32_t sb) {
  if (lane == 0) {
    bar_expect(sb + kVLanded, kVStage / 2);
    bar_expect(sb + kVLanded + 8, kVStage / 2);
  }
  Turn n;
  for (Items it(p); it.next(p);)
#pragma unroll 1
    for (int tile = it.w.tile0; tile < it.w.tile1; ++tile, ++n.n) {
      if (!wait_warp(sb + kVLanded + n.at(), n.parity(), p.a.err)) return false;
      if (lane == 0) {
        bar_expect(sb + kVLanded + n.at(), kVStage / 2);   // for the tile after the next
        asm volatile("fence.proxy.async;" ::: "memory");
        arrive_in(sb + kVFull + n.at(), 0);
      }
    }
  return true;
}

// Brings the queries of this CTA's heads, and asks the quantised rows of tiles ahead
// into L2, a warp: in a prefix one request for the CTA's rows, else line by line.
__device__ __forceinline__ void load_queries(const MlaParams& p, uint32_t rank, int t, const CUtensorMap* q_map, uint32_t sb) {
  bar_expect(sb + kQFull, kBlocks * kQBlock);
#pragma unroll 1
  for (int b = 0; b < kBlocks; ++b)
    tma_2d(sb + kOffQ + b * kQBlock, q_map, sb + kQFull, b * 64, t * p.a.Hq + static_cast<int>(rank) * kHeads);
}
constexpr int kAhead = 4;   // tiles (2, 8 and 12: the same within 3 %)
template <int kFmt>
__device__ __forceinline__ bool look_ahead(const MlaParams& p, uint32_t rank, int lane, const CUtensorMap* q_map, uint32_t sb) {
  constexpr int kRow = kv_row_bytes(kFmt);
  uint32_t items = 0;
  Turn n;
  for (Items it(p); it.next(p); ++items) {
    const Work& w = it.w;
    if (!wait_warp(sb + kQEmpty, (items & 1) ^ 1u, p.a.err)) return false;
    if (elect_one()) load_queries(p, rank, w.t, q_map, sb);
    __syncwarp();
    if (!wait_warp(sb + kQFull, items & 1, p.a.err)) return false;
    if (lane == 0) arrive_in(sb + kQReady, 0);
    for (int tile = w.tile0; tile < w.tile1; ++tile, ++n.n) {
      // Goes on with the tiles: S of this one waits for the arrival, so that no phase
      // can pass by unseen.
      if (!wait_warp(sb + kKEmpty + n.at(), n.before(), p.a.err)) return false;
      if (lane == 0) arrive_in(sb + kKFull + n.at(), 0);
      if (tile + kAhead >= w.tile1) continue;
      const int first = (tile + kAhead) * kTile + static_cast<int>(rank) * kRows;
      if (!w.idx) {
        const int rows = min(kRows, w.n - first);
        if (lane == 0 && rows > 0)
          asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(w.base + static_cast<int64_t>(first) * kRow), "r"(rows * kRow)
                       : "memory");
        continue;
      }
      const int32_t id = row_of(w, first + lane);
      if (id < 0) continue;
      const uint8_t* row = w.base + static_cast<int64_t>(id) * kRow;
#pragma unroll 1
      for (int o = 0; o < kRow; o += 128) asm volatile("prefetch.global.L2 [%0];" ::"l"(row + o));
    }
  }
  return true;
}

// Of a bf16 cache, brings queries and rows by TMA; one thread.
__device__ __forceinline__ bool ask_rows(const MlaParams& p, uint32_t rank, const CUtensorMap* q_map, const CUtensorMap* map, uint32_t sb) {
  uint32_t items = 0;
  Turn n;
  for (Items it(p); it.next(p); ++items) {
    for (int tile = it.w.tile0; tile < it.w.tile1; ++tile, ++n.n) {
      const int row = tile * kTile + static_cast<int>(rank) * kRows;
      const uint32_t bar = sb + kKHere + n.at();
      if (!wait_one(sb + kKEmpty + n.at(), n.before(), p.a.err) || !wait_one(sb + kCopied + n.at(), n.before(), p.a.err)) return false;
      bar_expect(bar, kKStage);
#pragma unroll 1
      for (int b = 0; b < kBlocks; ++b) {
        tma_3d(sb + kOffK + n.stage() * kKStage + b * kKBlock, map, bar, b * 64, row, it.w.seq);
        if (tile + kAhead < it.w.tile1) tma_l2_3d(map, b * 64, row + kAhead * kTile, it.w.seq);
      }
      if (tile == it.w.tile0) {   // the first rows need not wait for the place of the queries
        if (!wait_one(sb + kQEmpty, (items & 1) ^ 1u, p.a.err)) return false;
        load_queries(p, rank, it.w.t, q_map, sb);
      }
    }
  }
  return true;
}
// Passes on to the first CTA what has landed in the second, one thread.
__device__ __forceinline__ bool pass_rows(const MlaParams& p, uint32_t sb) {
  uint32_t items = 0;
  Turn n;
  for (Items it(p); it.next(p); ++items) {
    if (!wait_one(sb + kQFull, items & 1, p.a.err)) return false;
    arrive_in(sb + kQReady, 0);
#pragma unroll 1
    for (int tile = it.w.tile0; tile < it.w.tile1; ++tile, ++n.n) {
      if (!wait_one(sb + kKHere + n.at(), n.parity(), p.a.err)) return false;
      arrive_in(sb + kKFull + n.at(), 0);
    }
  }
  return true;
}

// Issue the products of both CTAs, two warps of the first: S of one tile after the
// other, and O += P V.  Each waits for its own operands; the tensor core takes what
// comes first.  (One warp for both had to look at six barriers in turn, at 50 to 90
// cycles each: it saw an operand 300 to 800 cycles late.)  All lanes wait, one issues.
template <bool kQuant>
__device__ __forceinline__ bool multiply_rows(const MlaParams& p, uint32_t tmem, uint32_t sb) {
  const bool leader = elect_one();
  bool ok = false;
  Turn n;
  uint32_t items = 0;
  for (Items it(p); it.next(p); ++items) {
    if (!wait_warp(sb + kQReady, items & 1, p.a.err) || (!kQuant && !wait_warp(sb + kQFull, items & 1, p.a.err))) goto done;
#pragma unroll 1
    for (int left = it.w.tile1 - it.w.tile0; left > 0; --left, ++n.n) {
      if (!wait_warp(sb + kSEmpty + n.at4(), n.parity4() ^ 1u, p.a.err) || !wait_warp(sb + kKFull + n.at(), n.parity(), p.a.err) ||
          (!kQuant && !wait_warp(sb + kKHere + n.at(), n.parity(), p.a.err)))
        goto done;
      if (leader) {
        tc_fence_after();
        const uint32_t d = tmem + kTmemS + n.place4() * 32;
        uint64_t q = sw128_kmajor_desc(sb + kOffQ), k = sw128_kmajor_desc(sb + kOffK + n.stage() * kKStage);
        uint32_t add = 0;
#pragma unroll 1
        for (int b = 0; b < kBlocks; b += 3) {
          umma_pair<0, 0>(d, q, k, kIdescS, add);
          umma_pair<32, 32>(d, q, k, kIdescS, 1);
          umma_pair<64, 64>(d, q, k, kIdescS, 1);
          umma_pair<96, 96>(d, q, k, kIdescS, 1);
          umma_pair<kQBlock, kKBlock>(d, q, k, kIdescS, 1);
          umma_pair<kQBlock + 32, kKBlock + 32>(d, q, k, kIdescS, 1);
          umma_pair<kQBlock + 64, kKBlock + 64>(d, q, k, kIdescS, 1);
          umma_pair<kQBlock + 96, kKBlock + 96>(d, q, k, kIdescS, 1);
          umma_pair<2 * kQBlock, 2 * kKBlock>(d, q, k, kIdescS, 1);
          umma_pair<2 * kQBlock + 32, 2 * kKBlock + 32>(d, q, k, kIdescS, 1);
          umma_pair<2 * kQBlock + 64, 2 * kKBlock + 64>(d, q, k, kIdescS, 1);
          umma_pair<2 * kQBlock + 96, 2 * kKBlock + 96>(d, q, k, kIdescS, 1);
          add = 1;
          q += 3 * kQBlock >> 4;
          k += 3 * kKBlock >> 4;
        }
        commit_pair(sb + kSFull + n.at4());
        commit_pair(sb + kKEmpty + n.at());
        if (left == 1) commit_pair(sb + kQEmpty);
      }
      __syncwarp();
    }
  }
  ok = true;
done:
  if (leader) commit_pair(sb + kDone);
  __syncwarp();
  return ok;
}
__device__ __forceinline__ bool multiply_values(const MlaParams& p, uint32_t tmem, uint32_t sb) {
  const bool leader = elect_one();
  bool ok = false;
  Turn n;
  uint32_t items = 0;
  for (Items it(p); it.next(p); ++items) {
    if (!wait_warp(sb + kOEmpty, (items & 1) ^ 1u, p.a.err)) goto done;
#pragma unroll 1
    for (int tile = it.w.tile0; tile < it.w.tile1; ++tile, ++n.n) {
      if (!wait_warp(sb + kVFull + n.at(), n.parity(), p.a.err) || !wait_warp(sb + kPFull + n.at(), n.parity(), p.a.err)) goto done;
      if (leader) {
        tc_fence_after();
        const uint64_t w = sw128_kmajor_desc(sb + kOffP + n.stage() * kPStage);
        const uint64_t v = sw128_mnmajor_desc(sb + kOffV + n.stage() * kVStage, kVBlock);
        const uint32_t add = tile > it.w.tile0;
        umma_pair<0, 0>(tmem, w, v, kIdescO, add);                      // 16 rows, entries 0 .. 127 of each half
        umma_pair<0, 2 * kVBlock>(tmem + 128, w, v, kIdescO, add);
        umma_pair<32, 2048>(tmem, w, v, kIdescO, 1);
        umma_pair<32, 2 * kVBlock + 2048>(tmem + 128, w, v, kIdescO, 1);
        umma_pair<64, 4096>(tmem, w, v, kIdescO, 1);
        umma_pair<64, 2 * kVBlock + 4096>(tmem + 128, w, v, kIdescO, 1);
        umma_pair<96, 6144>(tmem, w, v, kIdescO, 1);
        umma_pair<96, 2 * kVBlock + 6144>(tmem + 128, w, v, kIdescO, 1);
        commit_pair(sb + kVEmpty + n.at());
        commit_pair(sb + kPvDone + n.at());
      }
      __syncwarp();
    }
  }
  ok = true;
done:
  if (leader) commit_pair(sb + kDone);
  __syncwarp();
  return ok;
}

__device__ __forceinline__ void named_bar_arrive(int id, int nthreads) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(nthreads) : "memory");
}
// The softmax warpgroups' exchange area and its barriers.
struct ExchangeIo {
  uint32_t base;
  __device__ __forceinline__ void store(uint32_t at, uint32_t v) const { st_shared(base + at, v); }
  __device__ __forceinline__ uint32_t load(uint32_t at) const { return ld_shared(base + at); }
  __device__ __forceinline__ void sync(int id, int nthreads) const { named_bar_sync(id, nthreads); }
  __device__ __forceinline__ void arrive(int id, int nthreads) const { named_bar_arrive(id, nthreads); }
};

// Softmax and output, two warpgroups: each takes every other tile, so that one's
// loads, barriers and fences pass while the other one counts; between them goes the
// reference m alone, early in a tile.  tid: in the warpgroup; its warp w has TMEM
// lanes 32 w.., two lanes a head, one for each half of a tile's rows and of O.
__device__ __forceinline__ bool softmax(const MlaParams& p, uint32_t rank, uint32_t group, int tid, uint32_t tmem, uint32_t sb) {
  const LatentArgs& a = p.a;
  uint32_t* err = a.err;
  const int warp = tid >> 5, lane = tid & 31;
  const int half = warp >> 1;                     // rows [32 half, 32 half + 32) of a tile, entries 256 half .. of O
  const int hl = (warp & 1) * 32 + lane;          // head of this CTA
  const int h = static_cast<int>(rank) * kHeads + hl;
  const int h0 = static_cast<int>(rank) * kHeads + (warp & 1) * 32;   // first head of the warp
  const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
  const float kNegInf = -__int_as_float(0x7f800000);
  // A scale of 0 takes the scores away first (a NaN or an infinity becomes NaN, as in
  // 0 * s) and then weighs by 1, so that -inf times the scale stays -inf for the rows
  // that are not there.  (With the smallest normal number in place of 0, scores of 1e37
  // still weighed rows apart.)
  const bool flat = a.scale_log2 == 0.f;
  const float c = flat ? 1.f : a.scale_log2;
  const uint32_t my_p = sb + kOffP + group * kPStage;
  SoftmaxExchange<ExchangeIo> exchange = {{sb + kOffExchange}, group, tid};
  bool ok = true;
  Turn n;
  uint32_t items = 0;                              // that have rows, so far
  Round r;
  Peek ahead = peek(p, r.item);
  while (r.item < p.items) {
    const Work w = work_of(p, r.item, ahead);
    if (tid == 0 && group == 0 && rank == 0 && (ahead.seq < 0 || ahead.seq >= a.nseq)) record_error(err, MISA_DEVERR_BAD_SEQ);
    r.next();
    ahead = peek(p, r.item);
    const int ntiles = w.tile1 - w.tile0;
    const int64_t row0 = (p.nsplit > 1 ? static_cast<int64_t>(w.t) * p.nsplit + w.split : static_cast<int64_t>(w.t)) * a.Hq;
    if (ntiles == 0) {   // no rows: zeros, and a sum of nothing
      if (group == 0) {
        if (h < a.Hq && half == 0) {
          if (p.nsplit > 1) *reinterpret_cast<float2*>(p.part_ml + (row0 + h) * 2) = make_float2(kNegInf, 0.f);
          else if (a.lse) a.lse[row0 + h] = kNegInf;
        }
        for (int x = tid; p.nsplit == 1 && x < kHeads * 64; x += 128)
          if (static_cast<int>(rank) * kHeads + (x >> 6) < a.Hq)
            reinterpret_cast<uint4*>(a.out + (row0 + rank * kHeads) * kDv)[x] = make_uint4(0u, 0u, 0u, 0u);
      }
      continue;
    }
    const uint32_t first = n.n, end = n.n + ntiles;
    n.n += (n.n ^ group) & 1;                      // the first tile of this warpgroup
    float m_prev = kNegInf, m = kNegInf, l = 0.f;  // m: the reference that l is relative to
    auto row_at = [&](uint32_t t) {                // this lane's row of the half of tile number t
      return t < end ? row_of(w, (w.tile0 + static_cast<int>(t - first)) * kTile + half * 32 + lane) : -1;
    };
    int32_t here = row_at(n.n);
#pragma unroll 1
    for (; n.n < end; n.n += 2) {
      const uint32_t live = __ballot_sync(0xffffffffu, here >= 0);   // rows of this half that exist
      // A wait that gave up ends the work, not the loop: the barriers stay paired.
      ok = ok && wait_warp(sb + kSFull + n.at4(), n.parity4(), err);
      uint32_t s[32];
      float mx = kNegInf;
      if (ok) {
        tc_fence_after();
        tmem_ld32(t_lane + kTmemS + n.place4() * 32, s);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_in(sb + kSEmpty + n.at4(), 0);
        if (__builtin_expect(flat, 0)) {
#pragma unroll
          for (int j = 0; j < 32; ++j) s[j] = __float_as_uint(__uint_as_float(s[j]) * 0.f);
        }
        if (live != 0xffffffffu) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (!((live >> j) & 1u)) s[j] = 0xff800000u;
        }
        float x[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
#pragma unroll
        for (int j = 0; j < 32; ++j) x[j & 3] = fmaxf(x[j & 3], __uint_as_float(s[j]));
        mx = fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3]));
      }
      here = row_at(n.n + 2);
      // the other half of the tile's rows for the same head
      mx = fmaxf(mx, __uint_as_float(exchange.other_half(__float_as_uint(mx)))) * c;
      // the reference after the tile before, moved if this tile is far above it
      m_prev = __uint_as_float(exchange.reference_before(n.n, first, 0xff800000u));
      const bool moved = mx > m_prev + 8.f || (m_prev == kNegInf && mx > kNegInf);
      const float m_new = moved ? mx : m_prev;
      exchange.set_reference(__float_as_uint(m_new));
      if (m_new != m) {
        l *= m == kNegInf ? 0.f : ex2(m - m_new);
        m = m_new;
      }
      const float mr = m == kNegInf ? 0.f : m;
      float l0 = 0.f, l1 = 0.f;
#pragma unroll
      for (int j = 0; j < 32; j += 2) {   // (the packed pairs take the place of the scores)
        const float x = ex2(fmaf(__uint_as_float(s[j]), c, -mr)), y = ex2(fmaf(__uint_as_float(s[j + 1]), c, -mr));
        l0 += x;
        l1 += y;
        s[j >> 1] = pack_bf16(x, y);
      }
      l += l0 + l1;
      ok = ok && wait_warp(sb + kPvDone + n.at(), n.before(), err);   // O of two tiles ago has read this place of P
      if (!ok) continue;
#pragma unroll
      for (int u = 0; u < 4; ++u)
        st_shared16(my_p + hl * 128 + (((half * 4 + u) ^ (hl & 7)) << 4), make_uint4(s[4 * u], s[4 * u + 1], s[4 * u + 2], s[4 * u + 3]));
      if (n.n > first && __any_sync(0xffffffffu, moved)) {   // O so far, once it is complete
        Turn last = n;
        --last.n;
        ok = wait_warp(sb + kPvDone + last.at(), last.parity(), err);
        const float f = !moved ? 1.f : m_prev == kNegInf ? 0.f : ex2(m_prev - m_new);
        tc_fence_after();
#pragma unroll 1
        for (int o = 0; o < 256; o += 16) {
          uint32_t v[16];
          tmem_ld16(t_lane + o, v);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 16; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
          tmem_st16(t_lane + o, v);
        }
        asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        tc_fence_before();
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) arrive_in(sb + kPFull + n.at(), 0);
    }
    n.n = end;
    const uint32_t turn = items & 1;
    ++items;
    if (((end - 1) & 1) != group) {   // the other warpgroup finishes the item
      exchange.hand_over(turn, __float_as_uint(l));
      continue;
    }
    // The sums of both warpgroups and both halves: the other warpgroup's are relative
    // to the reference before the last tile.
    l += __uint_as_float(exchange.other_half_sum(turn, __float_as_uint(l)));
    if (ntiles > 1) {
      const float other = __uint_as_float(exchange.handed_over(turn, 0)) + __uint_as_float(exchange.handed_over(turn, 1));
      l += other * (m_prev == m ? 1.f : m_prev == kNegInf ? 0.f : ex2(m_prev - m));
    }
    Turn last;
    last.n = end - 1;
    ok = ok && wait_warp(sb + kPvDone + last.at(), last.parity(), err);
    tc_fence_after();
    // Output, 16 entries of O at a time.  Partial sums go out as they lie, a head a
    // lane (the scratch has the heads side by side).  For bf16 each warp turns its 32
    // heads' pieces round in its 2 KB of this warpgroup's place of P, so that four lanes
    // store 64 bytes of a row, while the next entries come from TMEM.
    const bool any = l > 0.f || l != l;
    if (h < a.Hq && half == 0) {
      if (p.nsplit > 1) *reinterpret_cast<float2*>(p.part_ml + (row0 + h) * 2) = make_float2(any ? m : kNegInf, l);
      else if (a.lse) a.lse[row0 + h] = any ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
    }
    uint32_t v[16];
    tmem_ld16(t_lane, v);
    if (p.nsplit > 1) {
      float4* out = reinterpret_cast<float4*>(p.part_o) + row0 * (kDv / 4) + static_cast<int64_t>(half) * 64 * a.Hq + h;
#pragma unroll 1
      for (int o = 16; o <= 256; o += 16) {
        tmem_wait_ld();
        if (ok && h < a.Hq) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            out[j * a.Hq] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]), __uint_as_float(v[4 * j + 2]),
                                        __uint_as_float(v[4 * j + 3]));
        }
        out += 4 * a.Hq;
        __syncwarp();
        if (o < 256) tmem_ld16(t_lane + o, v);
      }
    } else {
      const uint32_t turn_p = my_p + warp * 2048, at = turn_p + lane * 64, swz = (lane >> 1) & 3;
      const float inv = any ? 1.f / l : 0.f;
      uint8_t* out = reinterpret_cast<uint8_t*>(a.out + (row0 + h0) * kDv + half * 256) + (lane >> 2) * (kDv * 2) + (lane & 3) * 16;
      const int rows = ok ? a.Hq - h0 - (lane >> 2) : 0;   // from this lane's first on
#pragma unroll 1
      for (int o = 16; o <= 256; o += 16) {
        tmem_wait_ld();
        uint32_t x[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = pack_bf16(__uint_as_float(v[2 * j]) * inv, __uint_as_float(v[2 * j + 1]) * inv);
        if (o < 256) tmem_ld16(t_lane + o, v);
        const uint32_t second = ((o >> 3) & 2) ^ 2;   // 32 entries a store
#pragma unroll
        for (int j = 0; j < 2; ++j)
          st_shared16(at + (((second + j) ^ swz) << 4), make_uint4(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3]));
        if (!second) continue;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int r = j * 8 + (lane >> 2);
          if (j * 8 < rows)
            *reinterpret_cast<uint4*>(out + j * 8 * kDv * 2) = ld_shared16(turn_p + r * 64 + (((lane & 3) ^ ((r >> 1) & 3)) << 4));
        }
        out += 64;
        __syncwarp();
      }
    }
    tc_fence_before();
    __syncwarp();
    if (lane == 0) arrive_in(sb + kOEmpty, 0);   // O has been read
  }
  return ok;
}

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
latent_mla_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap row_map, const MlaParams p) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];   // swizzled operands
  const uint32_t sb = smem_u32(smem_raw);
  constexpr bool kQuant = kFmt != MISA_KV_BF16;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  if (tid == 0) {
    for (uint32_t at = 0; at < 16; at += 8) {
      bar_init(sb + kKFull + at, kQuant ? 2 * (kRowWarps + 1) : 1);   // bring_rows and look_ahead, or pass_rows
      bar_init(sb + kKHere + at, 1);
      bar_init(sb + kKEmpty + at, 1);
      bar_init(sb + kCopied + at, kRowWarps);
      bar_init(sb + kVFull + at, 2 * (kRowWarps + 1));                // and pass_values
      bar_init(sb + kVLanded + at, 1);
      bar_init(sb + kVEmpty + at, 1);
      for (uint32_t two = 0; two < 32; two += 16) {
        bar_init(sb + kSFull + two + at, 1);
        bar_init(sb + kSEmpty + two + at, 8);
      }
      bar_init(sb + kPFull + at, 8);
      bar_init(sb + kPvDone + at, 1);
    }
    bar_init(sb + kOEmpty, 8);
    bar_init(sb + kQFull, 1);
    bar_init(sb + kQReady, kQuant ? 2 : 1);
    bar_init(sb + kQEmpty, 1);
    bar_init(sb + kDone, 2);
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(sb + kOffTmem) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    if (lane == 0) {
      tma_prefetch_desc(&q_map);
      if (kFmt == MISA_KV_BF16) tma_prefetch_desc(&row_map);
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the other CTA's barriers (fence_mbar_init) are ready for arrivals
  tc_fence_after();
  const uint32_t tmem = ld_shared(sb + kOffTmem);
  pdl_wait_inputs();
  pdl_allow_next();

  bool ok = true;
  if (warp == kMmaWarp) {
    if (rank == 0) ok = multiply_rows<kQuant>(p, tmem, sb);
    ok = wait_all(sb, p.a.err) && ok;   // nothing reads this CTA's memory any more
    __syncwarp();
  } else if (warp == kMmaWarp + 3) {
    if (rank == 0) {
      ok = multiply_values(p, tmem, sb);
    } else if (!kQuant) {
      if (elect_one()) ok = pass_rows(p, sb);
      __syncwarp();
    }
  } else if (warp == kMmaWarp + 1) {
    ok = pass_values(p, lane, sb);
  } else if (warp == kMmaWarp + 2) {
    if constexpr (kQuant) {
      ok = look_ahead<kFmt>(p, rank, lane, &q_map, sb);
    } else {
      if (elect_one()) ok = ask_rows(p, rank, &q_map, &row_map, sb);
      __syncwarp();
    }
  } else if (warp >= kRowWarp0) {
    if constexpr (kQuant) ok = bring_rows<kFmt>(p, rank, tid - kRowWarp0 * 32, sb);
    else ok = copy_rows(p, rank, tid - kRowWarp0 * 32, sb);
  } else {
    ok = softmax(p, rank, warp >> 2, tid & 127, tmem, sb);
  }

  tc_fence_before();
  if (__syncthreads_or(!ok)) {
    // A wait gave up: copies that a role had asked for (by TMA, or st.async to the other
    // CTA) may be under way.  Neither CTA leaves before they have had some 10 ms to land;
    // nothing waits for them by barrier, since one of those did not come.
    const uint32_t t0 = clock();
    while (static_cast<uint32_t>(clock()) - t0 < kDrainCycles) {
    }
  }
  cluster_sync_all();   // neither CTA leaves while the other may still arrive on its barriers
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Joins the splits of a query: out[t, h] = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c.
// A CTA takes 8 heads; each of its threads 4 x 4 entries of all splits in order, or, of
// many splits, 4 entries of every fourth, and then the four sums in order.
constexpr int kMaxSplits = 128;
constexpr int kJoinHeads = 8, kJoinThreads = 256;
constexpr int join_steps(int parts) { return parts == 1 ? 4 : 1; }
constexpr int join_entries(int parts) { return kJoinThreads / parts / kJoinHeads * 4 * join_steps(parts); }   // of a CTA
template <int kParts>
__global__ void __launch_bounds__(kJoinThreads)
latent_join_kernel(const float* __restrict__ part_o, const float* __restrict__ part_ml, int Hq, int nsplit,
                   uint16_t* __restrict__ out, float* __restrict__ lse) {
  constexpr int kSteps = join_steps(kParts), kEntries = join_entries(kParts), kWidth = kJoinThreads / kParts;
  __shared__ float sW[kJoinHeads][kMaxSplits + 1], sL[kJoinHeads][kMaxSplits + 1];
  __shared__ float4 sO[kParts][kWidth];
  pdl_wait_inputs();
  pdl_allow_next();
  const int groups = (Hq + kJoinHeads - 1) / kJoinHeads;
  const int block = static_cast<int>(blockIdx.x / (kDv / kEntries)), t = block / groups, h0 = (block - t * groups) * kJoinHeads;
  const int tid = threadIdx.x;
  const float kNegInf = -__int_as_float(0x7f800000);
  const int64_t row0 = static_cast<int64_t>(t) * nsplit * Hq;
  for (int x = tid; x < nsplit * kJoinHeads; x += kJoinThreads) {
    const int c = x / kJoinHeads, h = x % kJoinHeads;
    const float2 ml = h0 + h < Hq ? *reinterpret_cast<const float2*>(part_ml + (row0 + static_cast<int64_t>(c) * Hq + h0 + h) * 2)
                                  : make_float2(kNegInf, 0.f);
    sW[h][c] = ml.x;
    sL[h][c] = ml.y;
  }
  __syncthreads();
  const int h = tid % kJoinHeads, part = tid / kWidth;
  const int e4 = static_cast<int>(blockIdx.x % (kDv / kEntries)) * (kEntries / 4) + tid % kWidth / kJoinHeads;
  float m = kNegInf;
  for (int c = 0; c < nsplit; ++c) m = fmaxf(m, sW[h][c]);
  __syncthreads();
  for (int c = tid / kJoinHeads; c < nsplit; c += kJoinThreads / kJoinHeads)
    // no rows: its O was not written; a sum without a maximum is NaN and stays so
    sW[h][c] = sL[h][c] == 0.f ? 0.f : sW[h][c] == kNegInf ? 1.f : exp2f(sW[h][c] - m);
  __syncthreads();
  float4 acc[kSteps];
#pragma unroll
  for (int u = 0; u < kSteps; ++u) acc[u] = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* src = reinterpret_cast<const float4*>(part_o) + row0 * (kDv / 4) + static_cast<int64_t>(e4) * Hq + h0 + h;   // (a head that is not there: every sum is 0)
  constexpr int kStride = kWidth / kJoinHeads;   // of a thread's steps
#pragma unroll 4
  for (int c = part; c < nsplit; c += kParts) {
    const bool some = sL[h][c] != 0.f;
    const float w = sW[h][c];
#pragma unroll
    for (int u = 0; u < kSteps; ++u) {
      const float4 o = some ? __ldcs(src + (static_cast<int64_t>(c) * (kDv / 4) + u * kStride) * Hq) : make_float4(0.f, 0.f, 0.f, 0.f);
      acc[u].x += w * o.x;
      acc[u].y += w * o.y;
      acc[u].z += w * o.z;
      acc[u].w += w * o.w;
    }
  }
  if constexpr (kParts > 1) {
    sO[part][tid % kWidth] = acc[0];
    __syncthreads();
    if (part) return;
#pragma unroll
    for (int u = 1; u < kParts; ++u) {
      const float4 o = sO[u][tid];
      acc[0].x += o.x;
      acc[0].y += o.y;
      acc[0].z += o.z;
      acc[0].w += o.w;
    }
  }
  if (h0 + h >= Hq) return;
  float l = 0.f;
  for (int c = 0; c < nsplit; ++c) l += sW[h][c] * sL[h][c];
  const bool any = l > 0.f || l != l;
  const float inv = any ? 1.f / l : 0.f;
  const int64_t row = static_cast<int64_t>(t) * Hq + h0 + h;
#pragma unroll
  for (int u = 0; u < kSteps; ++u)
    reinterpret_cast<uint2*>(out + row * kDv)[e4 + u * kStride] =
        make_uint2(pack_bf16(acc[u].x * inv, acc[u].y * inv), pack_bf16(acc[u].z * inv, acc[u].w * inv));
  if (lse && e4 == 0) lse[row] = any ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
}

// Clusters that run at once on the 148 SMs of a B200.  No cluster waits for another, so
// a device with fewer SMs would only run them in turn.
constexpr int kSlots = 74;

// How many items share a query's rows: the split that makes the busiest cluster's list
// shortest, counted in tiles (1.1 to 1.35 us).  The constants fit whole calls, not their
// parts: an item more in a cluster's list takes 3 to 4 us, but a part of a query also
// writes fp32 sums (256 KB at 128 heads) that the join reads again, and the 16 tiles an
// item stand for that too.  Measured, rows in L2: 64 queries of 2048 mx8 rows 50.5 us
// whole and 65.2 in halves; 32 queries 48.5 whole, 34.9 in halves, 47.2 in thirds; 16 of
// 32,768 rows 174 in four parts, 278 in five, 173 in nine.
// n is the room for rows (k, or L): lengths are on the device.  A cache with far more
// room than rows is split too often: 32 queries of 2048 mx8 rows take 35 us with room for
// up to 32,768 rows and 70 with room for 131,072 (nine parts each).
constexpr int kItemTiles = 16, kJoinTiles = 6;
constexpr int kMaxParts = 4 * kSlots;   // of all queries together
int64_t tiles_of(int64_t n) { return (n + kTile - 1) / kTile; }
int pick_splits(int T, int64_t n) {
  const int64_t tiles = tiles_of(n);
  int best = 1;
  int64_t best_cost = -1;
  for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
    if (s > 1 && static_cast<int64_t>(T) * s > kMaxParts) break;
    const int64_t rounds = (static_cast<int64_t>(T) * s + kSlots - 1) / kSlots;
    const int64_t cost = rounds * ((tiles + s - 1) / s + kItemTiles) + (s > 1 ? kJoinTiles : 0);
    if (best_cost < 0 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}
size_t part_bytes(int64_t parts, int Hq) { return static_cast<size_t>(parts) * Hq * (kDv + 2) * sizeof(float); }

}  // namespace

size_t latent_mla_scratch_bytes(int T, int Hq, int64_t n) {
  const int s = pick_splits(T, n);
  return s > 1 ? part_bytes(static_cast<int64_t>(T) * s, Hq) : 0;
}

// Fewer queries or rows may be split into more parts than many (2048 rows: 32 queries
// into 64 parts, 64 queries not at all), so the bound goes over all T' <= T; for each
// it takes what pick_splits may choose at most, which does not fall with n.
size_t latent_mla_scratch_bound(int T, int Hq, int64_t n) {
  int64_t most = 0;
  for (int t = 1; t <= T && 2 * t <= kMaxParts; ++t) {
    const int64_t s = std::min({static_cast<int64_t>(kMaxSplits), tiles_of(n), static_cast<int64_t>(kMaxParts / t)});
    if (s > 1) most = std::max(most, t * s);
  }
  return part_bytes(most, Hq);
}

cudaError_t launch_latent_mla(const LatentArgs& a, cudaStream_t stream) {
  MlaParams p;
  p.a = a;
  p.nsplit = pick_splits(a.T, a.idx ? a.k : a.L);
  p.part_o = static_cast<float*>(a.scratch);
  p.part_ml = p.part_o + static_cast<size_t>(a.T) * p.nsplit * a.Hq * kDv;
  CUtensorMap qmap;
  if (!encode_2d_map(&qmap, true, a.q, kDqk, static_cast<uint64_t>(a.T) * a.Hq, kDqk * 2, 64, kHeads, true))
    return cudaErrorInvalidValue;
  CUtensorMap rmap = qmap;   // (quantised rows go by plain loads)
  if (a.fmt == MISA_KV_BF16 &&
      !encode_3d_map(&rmap, a.cache, kDqk, static_cast<uint64_t>(a.L), static_cast<uint64_t>(a.nseq), kDqk * 2,
                     a.nseq > 1 ? static_cast<uint64_t>(a.seq_stride) : static_cast<uint64_t>(a.L) * kDqk * 2, 64, kRows))
    return cudaErrorInvalidValue;
  auto kern = a.fmt == MISA_KV_BF16  ? latent_mla_kernel<MISA_KV_BF16>
              : a.fmt == MISA_KV_MX8 ? latent_mla_kernel<MISA_KV_MX8>
                                     : latent_mla_kernel<MISA_KV_MX4>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), kSmemBytes);
  if (e != cudaSuccess) return e;
  p.items = a.T * p.nsplit;
  p.by_nsplit = p.nsplit > 1 ? static_cast<uint32_t>(((1ull << 32) + p.nsplit - 1) / p.nsplit) : 0u;
  const int clusters = p.items < kSlots ? p.items : kSlots;
  e = launch_pdl(kern, dim3(static_cast<unsigned>(clusters) * 2), dim3(kThreads), kSmemBytes, stream, 0, qmap, rmap, p);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  // Many splits to few queries: more threads to each sum.
  const int parts = p.nsplit > 8 ? 4 : 1;
  return launch_pdl(parts == 4 ? latent_join_kernel<4> : latent_join_kernel<1>,
                    dim3(static_cast<unsigned>(a.T) * ((a.Hq + kJoinHeads - 1) / kJoinHeads) * (kDv / join_entries(parts))),
                    dim3(kJoinThreads), 0, stream, 0, static_cast<const float*>(p.part_o), static_cast<const float*>(p.part_ml),
                    a.Hq, p.nsplit, a.out, a.lse);
}

}  // namespace misa
