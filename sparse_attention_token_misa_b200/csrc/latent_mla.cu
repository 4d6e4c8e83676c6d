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
// by, which halves the shared memory reads that bound a 64-head tile otherwise
// (per 16 of the sum: 32 cycles for 128 heads x 128 rows, 64 for 128 x 256
// values, the tensor rate; 48 and 80 cycles where one SM reads both operands).
//
// Rows come in tiles of 128.  Per tile:
//  1. S = Q K^T: CTA u holds rows [64 u, 64 u + 64) of the tile, all 576 entries,
//     in 9 blocks of 64 (3 units of 3 blocks in a ring).  S in TMEM: lane l < 64
//     has head l against rows 0..63, lane 64 + l the same head against 64..127.
//  2. Softmax in one pass with a running reference m: when a tile's maximum is
//     more than 2^8 above 2^m, the sums so far are scaled and m moves (p stays
//     below 2^8, exact enough in bf16 and fp32).  p goes to shared memory as bf16.
//  3. O += P V: CTA u brings entries [256 u, 256 u + 256) of all 128 rows, as units
//     of 32 rows in a ring (rows of 64 entries in 128-byte swizzled atoms, read
//     MN-major, so nothing is transposed).  O stays in TMEM, 256 columns.
// S has two places, so that the products of tile i + 1 run while the softmax of
// tile i does.  Quantised rows become bf16 (exactly) on the way from global to
// shared memory, in registers; bf16 rows are copied asynchronously.  Rows two
// tiles ahead are asked into L2.
//
// Few queries: the rows of each are split over several clusters, whose partial
// sums a second kernel joins in a fixed order.
//
// Roles (416 threads a CTA): warps 0-3 softmax and output (a lane of TMEM each),
// warp 4 TMEM and, in the first CTA, the MMAs, warps 5-8 bring the rows of S,
// warps 9-12 those of O.  Waits are bounded.
#include "kv_format.cuh"
#include "launch.h"
#include "misa_device.cuh"

namespace misa {

namespace {

constexpr int kDqk = MISA_MLA_DQK, kDv = MISA_MLA_DV;
constexpr int kTile = 128;                        // rows of a tile
constexpr int kHeads = 64;                        // heads of a CTA
constexpr int kBlocks = kDqk / 64;                // 9
constexpr int kBlockBytes = 64 * 128;             // 64 rows (heads) x 64 bf16
constexpr int kKUnits = 3, kKUnitBlocks = 3;      // ring of S operands: one tile
constexpr int kVUnits = 4, kVUnitRows = 32;       // ring of O operands: one tile
constexpr int kVAtom = kVUnitRows * 128;          // 32 rows x 64 entries
constexpr int kVUnitBytes = 4 * kVAtom;           // 32 rows x 256 entries
constexpr int kOffQ = 0;
constexpr int kOffK = kOffQ + kBlocks * kBlockBytes;
constexpr int kOffV = kOffK + kBlocks * kBlockBytes;
constexpr int kOffP = kOffV + kVUnits * kVUnitBytes;
constexpr int kOffBar = kOffP + 2 * kBlockBytes;
constexpr int kNumBars = 2 * kKUnits + 2 * kVUnits + 2 + 2 + 5;
constexpr int kOffTmem = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffTmem + 8;
constexpr int kOffRed = (kOffAbort + 8 + 15) / 16 * 16;   // [2][128] floats
constexpr int kSmemBytes = kOffRed + 2 * 128 * 4 + 1024;
static_assert(kSmemBytes <= 232448, "shared memory of a CTA");
constexpr int kMmaWarp = 4, kKWarp0 = 5, kVWarp0 = 9, kThreads = 13 * 32;
constexpr int kTmemS = 256;                       // O: columns 0..255, S: two places of 64 columns
constexpr uint32_t kIdescS = idesc_bf16_f32(128, 128);
constexpr uint32_t kIdescO = idesc_bf16_f32(128, 256) | (1u << 16);   // values MN-major

// ---------------------------------------------------------------- the pair
__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}
// Arrive on the first CTA's barrier.  The release is the CTA's: what this warp
// wrote is its own CTA's shared memory, which its own SM's tensor core reads, and
// fence.proxy.async has ordered that.  (A release of the cluster's scope would wait
// for the loads of the next unit and for a round trip to L2, about 1000 cycles.)
__device__ __forceinline__ void arrive_leader(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .b32 a;\n\tmapa.shared::cluster.u32 a, %0, 0;\n\t"
      "mbarrier.arrive.shared::cluster.b64 _, [a];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
// A wait of a whole warp: one outcome for all lanes.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, uint32_t* err, volatile uint32_t* abort) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, err, abort));
}
__device__ __forceinline__ void umma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
      : "memory");
}
// Arrive on this barrier of both CTAs when the MMAs issued so far are done.
__device__ __forceinline__ void commit_pair(uint64_t* bar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          smem_u32(bar)),
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
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ void l2_prefetch(const void* p) { asm volatile("prefetch.global.L2 [%0];" ::"l"(p)); }

// ---------------------------------------------------------------- rows
// The work of a cluster: query t, tiles [tile0, tile1) of its n row slots.
struct Work {
  int t;
  int n, tile0, tile1;
  const uint8_t* base;      // cache of the query's sequence
  const int32_t* idx;       // its listed rows, or NULL: slot s is row s
  int64_t L;
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

// Signals a unit: this lane's writes are visible to the tensor core, and the warp
// arrives once.
__device__ __forceinline__ void unit_ready(uint64_t* bar) {
  fence_proxy_async_smem();
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive_leader(bar);
}

// Brings the S operand, 128 threads: thread = (row r0 + 16 i, piece) of each block.
template <int kFmt>
__device__ __forceinline__ void bring_keys(const Work& w, uint32_t rank, int tid, uint8_t* sK, uint64_t* full,
                                           uint64_t* empty, uint32_t* err, volatile uint32_t* abort) {
  constexpr int kRow = kv_row_bytes(kFmt);
  const int r0 = tid >> 3, piece = tid & 7;
  uint8_t* dst0 = sK + r0 * 128 + ((piece ^ (r0 & 7)) << 4);   // rows 16 apart: the same swizzle
  const int own = static_cast<int>(rank) * 64;
  auto prefetch = [&](int tile) {
    // (lines of 128 bytes, two threads a row; one bulk prefetch a row is issued lane
    // by lane and took a warp 3000 cycles a tile)
    if (tile >= w.tile1) return;
    const int32_t id = row_of(w, tile * kTile + own + (tid >> 1));
    if (id < 0) return;
    const uint8_t* row = w.base + static_cast<int64_t>(id) * kRow;
#pragma unroll
    for (int o = 0; o < kRow; o += 256)
      if (o + (tid & 1) * 128 < kRow) l2_prefetch(row + o + (tid & 1) * 128);
  };
  prefetch(w.tile0);
  prefetch(w.tile0 + 1);
  int32_t ids[4];
  auto load_ids = [&](int tile) {
#pragma unroll
    for (int i = 0; i < 4; ++i) ids[i] = tile < w.tile1 ? row_of(w, tile * kTile + own + r0 + 16 * i) : -1;
  };
  load_ids(w.tile0);

  if constexpr (kFmt == MISA_KV_BF16) {
    int pending = -1;   // unit whose copies are under way
    uint32_t ph = 0;
    for (int tile = w.tile0; tile < w.tile1; ++tile, ph ^= 1u) {
      prefetch(tile + 2);
      const uint8_t* src[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) src[i] = w.base + static_cast<int64_t>(max(ids[i], 0)) * kRow + piece * 16;
      for (int g = 0; g < kKUnits; ++g) {
        if (pending >= 0 && !__all_sync(0xffffffffu, mbar_try_wait(&empty[g], ph ^ 1u))) {
          cp_async_wait_group<0>();
          unit_ready(&full[pending]);
          pending = -1;
        }
        if (!wait_warp(&empty[g], ph ^ 1u, err, abort)) { cp_async_wait_group<0>(); return; }
#pragma unroll
        for (int bb = 0; bb < kKUnitBlocks; ++bb) {
          const int b = g * kKUnitBlocks + bb;
#pragma unroll
          for (int i = 0; i < 4; ++i) cp_async_16(dst0 + b * kBlockBytes + i * 2048, src[i] + b * 128, ids[i] >= 0);
        }
        cp_async_commit();
        if (pending >= 0) {
          cp_async_wait_group<1>();
          unit_ready(&full[pending]);
        }
        pending = g;
      }
      load_ids(tile + 1);
    }
    cp_async_wait_group<0>();
    if (pending >= 0) unit_ready(&full[pending]);
  } else {
    // Absent rows: any row's codes with scales of zero, and no rotary entries.
    uint2 cur[kKUnitBlocks * 4];    // codes of the unit at hand (the rotary block apart)
    uint4 rope[4], scales[4];
    bool absent[4];
    const uint8_t* src[4];
    auto point = [&] {
#pragma unroll
      for (int i = 0; i < 4; ++i) src[i] = w.base + static_cast<int64_t>(max(ids[i], 0)) * kRow;
    };
    auto load_unit = [&](int g, uint2* c) {
#pragma unroll
      for (int bb = 0; bb < kKUnitBlocks; ++bb) {
        const int b = g * kKUnitBlocks + bb;
        if (b == kBlocks - 1) continue;
#pragma unroll
        for (int i = 0; i < 4; ++i) c[bb * 4 + i] = load_code<kFmt>(src[i], b * 64 + piece * 8);
      }
    };
    auto load_rest = [&] {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        scales[i] = __ldg(reinterpret_cast<const uint4*>(src[i] + kv_code_bytes(kFmt)));
        rope[i] = __ldg(reinterpret_cast<const uint4*>(src[i] + kv_rope_offset(kFmt) + piece * 16));
        absent[i] = ids[i] < 0;
      }
    };
    point();
    load_unit(0, cur);
    load_rest();
    load_ids(w.tile0 + 1);
    const uint32_t sel = 0x4440u | (piece >> 2);   // the piece's byte of a block's two scale bytes
    uint32_t ph = 0;
    for (int tile = w.tile0; tile < w.tile1; ++tile, ph ^= 1u) {
      prefetch(tile + 2);
#pragma unroll
      for (int g = 0; g < kKUnits; ++g) {
        uint2 nxt[kKUnitBlocks * 4];
        if (g + 1 < kKUnits) {
          load_unit(g + 1, nxt);
        } else {
          point();
          load_unit(0, nxt);
        }
        if (!wait_warp(&empty[g], ph ^ 1u, err, abort)) return;
        if (g == 0) {   // (here, not where they are loaded: this waits for them)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (absent[i]) scales[i] = rope[i] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int bb = 0; bb < kKUnitBlocks; ++bb) {
          const int b = g * kKUnitBlocks + bb;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint4 y;
            if (b == kBlocks - 1) {
              y = rope[i];
            } else {
              const uint32_t sw = b < 2 ? scales[i].x : b < 4 ? scales[i].y : b < 6 ? scales[i].z : scales[i].w;
              const uint2 c = cur[bb * 4 + i];
              y = kv_decode8<kFmt>(c.x, c.y, kv_scale(__byte_perm(sw, 0u, sel + (b & 1) * 2)));
            }
            *reinterpret_cast<uint4*>(dst0 + b * kBlockBytes + i * 2048) = y;
          }
        }
        unit_ready(&full[g]);
#pragma unroll
        for (int j = 0; j < kKUnitBlocks * 4; ++j) cur[j] = nxt[j];
      }
      load_rest();                // of the rows `src` points at now
      load_ids(tile + 2);
    }
  }
}

// Brings the O operand, 128 threads: entries [256 rank, 256 rank + 256) of units of 32 rows.
template <int kFmt>
__device__ __forceinline__ void bring_values(const Work& w, uint32_t rank, int tid, uint8_t* sV, uint64_t* full,
                                             uint64_t* empty, uint32_t* err, volatile uint32_t* abort) {
  constexpr int kRow = kv_row_bytes(kFmt);
  const int r0 = tid >> 3, piece = tid & 7;
  uint8_t* dst0 = sV + r0 * 128 + ((piece ^ (r0 & 7)) << 4);
  int32_t ids[2];
  auto load_ids = [&](int tile, int g) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      ids[i] = tile < w.tile1 ? row_of(w, tile * kTile + g * kVUnitRows + r0 + 16 * i) : -1;
  };
  load_ids(w.tile0, 0);

  if constexpr (kFmt == MISA_KV_BF16) {
    int pending = -1;
    uint32_t ph = 0;
    for (int tile = w.tile0; tile < w.tile1; ++tile, ph ^= 1u) {
      for (int g = 0; g < kVUnits; ++g) {
        if (pending >= 0 && !__all_sync(0xffffffffu, mbar_try_wait(&empty[g], ph ^ 1u))) {
          cp_async_wait_group<0>();
          unit_ready(&full[pending]);
          pending = -1;
        }
        if (!wait_warp(&empty[g], ph ^ 1u, err, abort)) { cp_async_wait_group<0>(); return; }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint8_t* src = w.base + static_cast<int64_t>(max(ids[i], 0)) * kRow + rank * 512 + piece * 16;
#pragma unroll
          for (int a = 0; a < 4; ++a) cp_async_16(dst0 + g * kVUnitBytes + a * kVAtom + i * 2048, src + a * 128, ids[i] >= 0);
        }
        cp_async_commit();
        if (pending >= 0) {
          cp_async_wait_group<1>();
          unit_ready(&full[pending]);
        }
        pending = g;
        if (g + 1 < kVUnits) load_ids(tile, g + 1);
        else load_ids(tile + 1, 0);
      }
    }
    cp_async_wait_group<0>();
    if (pending >= 0) unit_ready(&full[pending]);
  } else {
    uint2 cur[8], scales[2];
    const uint8_t* src[2];
    bool absent[2];
    auto load_unit = [&](uint2* c, uint2* s) {   // of the rows `ids`
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        src[i] = w.base + static_cast<int64_t>(max(ids[i], 0)) * kRow;
        s[i] = __ldg(reinterpret_cast<const uint2*>(src[i] + kv_code_bytes(kFmt) + rank * 8));
        absent[i] = ids[i] < 0;
#pragma unroll
        for (int a = 0; a < 4; ++a) c[i * 4 + a] = load_code<kFmt>(src[i], static_cast<int>(rank) * 256 + a * 64 + piece * 8);
      }
    };
    load_unit(cur, scales);
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (absent[i]) scales[i] = make_uint2(0u, 0u);
    load_ids(w.tile0, 1);
    const uint32_t sel = 0x4440u | (piece >> 2);
    uint32_t ph = 0;
    for (int tile = w.tile0; tile < w.tile1; ++tile, ph ^= 1u) {
#pragma unroll
      for (int g = 0; g < kVUnits; ++g) {
        uint2 nxt[8], nscales[2];
        load_unit(nxt, nscales);
        if (g + 2 < kVUnits) load_ids(tile, g + 2);
        else load_ids(tile + 1, g + 2 - kVUnits);
        if (!wait_warp(&empty[g], ph ^ 1u, err, abort)) return;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int a = 0; a < 4; ++a) {
            const uint2 c = cur[i * 4 + a];
            *reinterpret_cast<uint4*>(dst0 + g * kVUnitBytes + a * kVAtom + i * 2048) =
                kv_decode8<kFmt>(c.x, c.y, kv_scale(__byte_perm(a < 2 ? scales[i].x : scales[i].y, 0u, sel + (a & 1) * 2)));
          }
        unit_ready(&full[g]);
#pragma unroll
        for (int j = 0; j < 8; ++j) cur[j] = nxt[j];
#pragma unroll
        for (int i = 0; i < 2; ++i) scales[i] = absent[i] ? make_uint2(0u, 0u) : nscales[i];
      }
    }
  }
}

struct MlaParams {
  LatentArgs a;
  int nsplit;
  float* part_o;     // [T][nsplit][Hq][512] (nsplit > 1)
  float* part_ml;    // [T][nsplit][Hq][2]: m (log2 units), l
};

template <int kFmt>
__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
latent_mla_kernel(const __grid_constant__ CUtensorMap q_map, const MlaParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t *sQ = smem + kOffQ, *sK = smem + kOffK, *sV = smem + kOffV, *sP = smem + kOffP;
  uint64_t* kfull = reinterpret_cast<uint64_t*>(smem + kOffBar);   // first CTA: unit brought by both
  uint64_t* kempty = kfull + kKUnits;    // unit multiplied
  uint64_t* vfull = kempty + kKUnits;    // first CTA
  uint64_t* vempty = vfull + kVUnits;
  uint64_t* sfull = vempty + kVUnits;    // [2] S complete
  uint64_t* sempty = sfull + 2;          // [2] first CTA: S read by both
  uint64_t* pfull = sempty + 2;          // first CTA: P written (and O scaled) by both
  uint64_t* pvdone = pfull + 1;          // O += P V complete
  uint64_t* qfull = pfull + 2;           // this CTA's queries landed
  uint64_t* qready = pfull + 3;          // first CTA: both CTAs' queries landed
  uint64_t* done = pfull + 4;            // every MMA retired
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kOffTmem);
  volatile uint32_t* abort = reinterpret_cast<volatile uint32_t*>(smem + kOffAbort);
  float* sRed = reinterpret_cast<float*>(smem + kOffRed);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank();
  const int item = static_cast<int>(blockIdx.x >> 1);
  if (tid == 0) {
    for (int i = 0; i < kKUnits; ++i) { mbar_init(&kfull[i], 8); mbar_init(&kempty[i], 1); }
    for (int i = 0; i < kVUnits; ++i) { mbar_init(&vfull[i], 8); mbar_init(&vempty[i], 1); }
    for (int i = 0; i < 2; ++i) { mbar_init(&sfull[i], 1); mbar_init(&sempty[i], 8); }
    mbar_init(pfull, 8);
    mbar_init(pvdone, 1);
    mbar_init(qfull, 1);
    mbar_init(qready, 2);
    mbar_init(done, 1);
    *abort = 0u;
    fence_mbar_init();
  }
  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_u32(tmem_slot)) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    if (lane == 0) tma_prefetch_desc(&q_map);
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // the other CTA's barriers are ready for arrivals
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  pdl_wait_inputs();
  pdl_allow_next();

  const LatentArgs& a = p.a;
  uint32_t* err = a.err;
  Work w;
  w.t = item / p.nsplit;
  const int split = item - w.t * p.nsplit;
  w.L = a.L;
  w.idx = a.idx ? a.idx + static_cast<int64_t>(w.t) * a.idx_stride : nullptr;
  int64_t n = a.idx ? a.k : min(static_cast<int64_t>(a.prefix_len[w.t]), a.L);
  int64_t seq = a.seq_of[w.t];
  if (seq < 0 || seq >= a.nseq) {
    if (tid == 0) record_error(err, MISA_DEVERR_BAD_SEQ);
    seq = 0;
    n = 0;
  }
  w.n = static_cast<int>(max(n, static_cast<int64_t>(0)));
  w.base = static_cast<const uint8_t*>(a.cache) + seq * a.seq_stride;
  const int tiles = (w.n + kTile - 1) / kTile;
  const int share = (tiles + p.nsplit - 1) / p.nsplit;
  w.tile0 = min(split * share, tiles);
  w.tile1 = min(w.tile0 + share, tiles);
  const int ntiles = w.tile1 - w.tile0;

  if (warp >= kVWarp0) {
    if (ntiles > 0) bring_values<kFmt>(w, rank, tid - kVWarp0 * 32, sV, vfull, vempty, err, abort);
  } else if (warp >= kKWarp0) {
    if (ntiles > 0) {
      // ids that name no row: each slot is looked at by one thread of its CTA
      if (w.idx) {
        for (int s = w.tile0 * kTile + tid - kKWarp0 * 32; s < min(w.n, w.tile1 * kTile); s += 128)
          if (rank == 0 && (w.idx[s] < -1 || w.idx[s] >= w.L)) record_error(err, MISA_DEVERR_BAD_INDEX);
      }
      bring_keys<kFmt>(w, rank, tid - kKWarp0 * 32, sK, kfull, kempty, err, abort);
    }
  } else if (warp == kMmaWarp) {
    if (ntiles > 0 && elect_one()) {
      mbar_arrive_expect_tx(qfull, kBlocks * kBlockBytes);
      for (int b = 0; b < kBlocks; ++b)
        tma_load_2d(sQ + b * kBlockBytes, &q_map, qfull, b * 64, w.t * a.Hq + static_cast<int>(rank) * kHeads);
      const bool landed = mbar_wait(qfull, 0, err, abort);
      if (landed) arrive_leader(qready);
      if (rank == 0) {
        const uint32_t qa = smem_u32(sQ), ka = smem_u32(sK), va = smem_u32(sV), pa = smem_u32(sP);
        auto scores = [&](int i) {   // S of tile i (counted from the cluster's first)
          if (!mbar_wait(&sempty[i & 1], ((i >> 1) & 1) ^ 1u, err, abort)) return false;
          const uint32_t d = tmem + kTmemS + (i & 1) * 64;
          for (int g = 0; g < kKUnits; ++g) {
            if (!mbar_wait(&kfull[g], i & 1, err, abort)) return false;
            tc_fence_after();
#pragma unroll
            for (int bb = 0; bb < kKUnitBlocks; ++bb)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk) {
                const uint32_t at = (g * kKUnitBlocks + bb) * kBlockBytes + kk * 32;
                umma_pair(d, sw128_kmajor_desc(qa + at), sw128_kmajor_desc(ka + at), kIdescS, (g | bb | kk) ? 1u : 0u);
              }
            commit_pair(&kempty[g]);
          }
          commit_pair(&sfull[i & 1]);
          return true;
        };
        auto values = [&](int i) {
          if (!mbar_wait(pfull, i & 1, err, abort)) return false;
          for (int g = 0; g < kVUnits; ++g) {
            if (!mbar_wait(&vfull[g], i & 1, err, abort)) return false;
            tc_fence_after();
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              const int step = g * 2 + kk;   // 16 rows
              const uint64_t ad = sw128_kmajor_desc(pa + (step >> 2) * kBlockBytes + (step & 3) * 32);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                umma_pair(tmem + j * 128, ad, sw128_mnmajor_desc(va + g * kVUnitBytes + j * 2 * kVAtom + kk * 2048, kVAtom),
                          kIdescO, (i | step) ? 1u : 0u);
            }
            commit_pair(&vempty[g]);
          }
          commit_pair(pvdone);
          return true;
        };
        bool ok = landed && mbar_wait(qready, 0, err, abort) && scores(0);
        for (int i = 0; i < ntiles && ok; ++i) {
          if (i + 1 < ntiles) ok = scores(i + 1);
          ok = ok && values(i);
        }
        commit_pair(done);
      }
      mbar_wait(done, 0, err, nullptr);   // both: nothing reads this CTA's memory any more
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------ softmax and output
    const int half = warp >> 1;                     // rows [64 half, 64 half + 64) of a tile, entries 256 half .. of O
    const int hl = (warp & 1) * 32 + lane;          // head of this CTA
    const int h = static_cast<int>(rank) * kHeads + hl;
    const uint32_t t_lane = tmem + (static_cast<uint32_t>(warp * 32) << 16);
    const float kNegInf = -__int_as_float(0x7f800000);
    const float c = a.scale_log2;
    float m = kNegInf, l = 0.f;
    bool ok = true;
    for (int i = 0; i < ntiles; ++i) {
      // rows of this half that exist: two words, the same in the whole warp
      uint32_t live[2];
#pragma unroll
      for (int j = 0; j < 2; ++j)
        live[j] = __ballot_sync(0xffffffffu, row_of(w, (w.tile0 + i) * kTile + half * 64 + j * 32 + lane) >= 0);
      // a wait that gave up ends the work, not the loop: the warps' barriers stay paired
      ok = ok && wait_warp(&sfull[i & 1], (i >> 1) & 1, err, abort);
      uint32_t s[64];
      if (ok) {
        tc_fence_after();
        tmem_ld32(t_lane + kTmemS + (i & 1) * 64, s);
        tmem_ld32(t_lane + kTmemS + (i & 1) * 64 + 32, s + 32);
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) arrive_leader(&sempty[i & 1]);
      }
      float mx = kNegInf;
      if ((live[0] & live[1]) == 0xffffffffu) {
#pragma unroll
        for (int j = 0; j < 64; ++j) mx = fmaxf(mx, __uint_as_float(s[j]));
      } else {
#pragma unroll
        for (int j = 0; j < 64; ++j) {
          if (!((live[j >> 5] >> (j & 31)) & 1u)) s[j] = 0xff800000u;
          mx = fmaxf(mx, __uint_as_float(s[j]));
        }
      }
      // the other half of the tile's rows for the same head
      float* red = sRed + (i & 1) * 128;
      red[warp * 32 + lane] = mx;
      named_bar_sync(1, 128);
      mx = fmaxf(mx, red[((warp ^ 2) * 32) + lane]) * c;
      if (mx != mx) mx = kNegInf;    // scale 0 and nothing live: 0 * -inf
      float f = 1.f;
      if (mx > m + 8.f || (m == kNegInf && mx > kNegInf)) {
        f = m == kNegInf ? 0.f : ex2(m - mx);
        m = mx;
        l *= f;
      }
      const float mr = m == kNegInf ? 0.f : m;
      uint32_t pk[32];
      float l0 = 0.f, l1 = 0.f;
      const bool masked = (live[0] & live[1]) != 0xffffffffu;
#pragma unroll
      for (int j = 0; j < 64; j += 2) {
        float x = ex2(fmaf(__uint_as_float(s[j]), c, -mr)), y = ex2(fmaf(__uint_as_float(s[j + 1]), c, -mr));
        if (masked) {
          if (!((live[j >> 5] >> (j & 31)) & 1u)) x = 0.f;
          if (!((live[j >> 5] >> ((j & 31) + 1)) & 1u)) y = 0.f;
        }
        l0 += x;
        l1 += y;
        pk[j >> 1] = pack_bf16(x, y);
      }
      l += l0 + l1;
      if (i > 0) ok = ok && wait_warp(pvdone, (i - 1) & 1, err, abort);
      if (!ok) continue;
      if (i > 0) {
        tc_fence_after();
        if (__any_sync(0xffffffffu, f != 1.f)) {
#pragma unroll 1
          for (int o = 0; o < 256; o += 32) {
            uint32_t v[32];
            tmem_ld32(t_lane + o, v);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = __float_as_uint(__uint_as_float(v[j]) * f);
            tmem_st16(t_lane + o, v);
            tmem_st16(t_lane + o + 16, v + 16);
          }
          asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
        }
      }
      uint8_t* prow = sP + half * kBlockBytes + hl * 128;
#pragma unroll
      for (int u = 0; u < 8; ++u)
        *reinterpret_cast<uint4*>(prow + ((u ^ (hl & 7)) << 4)) =
            make_uint4(pk[4 * u], pk[4 * u + 1], pk[4 * u + 2], pk[4 * u + 3]);
      tc_fence_before();
      unit_ready(pfull);
    }
    // both halves' sums; a barrier apart from the last tile's exchange
    named_bar_sync(1, 128);
    sRed[warp * 32 + lane] = l;
    named_bar_sync(1, 128);
    l += sRed[((warp ^ 2) * 32) + lane];
    if (ntiles > 0) {
      ok = ok && wait_warp(pvdone, (ntiles - 1) & 1, err, abort);
      tc_fence_after();
    }
    const int64_t row = p.nsplit > 1 ? (static_cast<int64_t>(w.t) * p.nsplit + split) * a.Hq + h
                                     : static_cast<int64_t>(w.t) * a.Hq + h;
    const bool any = l > 0.f || l != l;
    if (p.nsplit > 1) {
      if (h < a.Hq && half == 0) {
        p.part_ml[row * 2] = any ? m : kNegInf;
        p.part_ml[row * 2 + 1] = l;
      }
      if (ntiles > 0 && ok) {
#pragma unroll 1
        for (int o = 0; o < 256; o += 32) {
          uint32_t v[32];
          tmem_ld32(t_lane + o, v);
          tmem_wait_ld();
          if (h < a.Hq) {
            float4* dst = reinterpret_cast<float4*>(p.part_o + row * kDv + half * 256 + o);
#pragma unroll
            for (int j = 0; j < 8; ++j)
              dst[j] = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                   __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
          }
        }
      }
    } else {
      const float inv = any ? 1.f / l : 0.f;
      if (a.lse && h < a.Hq && half == 0) a.lse[row] = any ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
#pragma unroll 1
      for (int o = 0; o < 256; o += 32) {
        uint32_t v[32];
        if (ntiles > 0 && ok) {
          tmem_ld32(t_lane + o, v);
          tmem_wait_ld();
        }
        if (h < a.Hq) {
          uint4* dst = reinterpret_cast<uint4*>(a.out + row * kDv + half * 256 + o);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t q[4];
#pragma unroll
            for (int u = 0; u < 4; ++u)
              q[u] = any ? pack_bf16(__uint_as_float(v[8 * j + 2 * u]) * inv, __uint_as_float(v[8 * j + 2 * u + 1]) * inv) : 0u;
            dst[j] = make_uint4(q[0], q[1], q[2], q[3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // neither CTA leaves while the other may still arrive on its barriers
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;" ::"r"(tmem) : "memory");
}

// Joins the splits of a query: out[t, h] = sum_c 2^(m_c - m) O_c / sum_c 2^(m_c - m) l_c
// in split order.  One CTA of 128 threads per (t, h), 4 entries a thread.
constexpr int kMaxSplits = 128;
__global__ void __launch_bounds__(128)
latent_join_kernel(const float* __restrict__ part_o, const float* __restrict__ part_ml, int Hq, int nsplit,
                   uint16_t* __restrict__ out, float* __restrict__ lse) {
  __shared__ float sM[kMaxSplits], sL[kMaxSplits];
  pdl_wait_inputs();
  pdl_allow_next();
  const int t = static_cast<int>(blockIdx.x) / Hq, h = static_cast<int>(blockIdx.x) - t * Hq;
  const int tid = threadIdx.x;
  const float kNegInf = -__int_as_float(0x7f800000);
  const int64_t row0 = static_cast<int64_t>(t) * nsplit * Hq + h;
  if (tid < nsplit) {
    const float2 ml = *reinterpret_cast<const float2*>(part_ml + (row0 + static_cast<int64_t>(tid) * Hq) * 2);
    sM[tid] = ml.x;
    sL[tid] = ml.y;
  }
  __syncthreads();
  float m = kNegInf;
  for (int c = 0; c < nsplit; ++c) m = fmaxf(m, sM[c]);
  float l = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < nsplit; ++c) {
    if (sL[c] == 0.f) continue;      // no rows: its O was not written
    const float w = sM[c] == kNegInf ? 1.f : exp2f(sM[c] - m);   // a sum without a maximum is NaN and stays so
    const float4 o = __ldcs(reinterpret_cast<const float4*>(part_o + (row0 + static_cast<int64_t>(c) * Hq) * kDv) + tid);
    l += w * sL[c];
    acc.x += w * o.x;
    acc.y += w * o.y;
    acc.z += w * o.z;
    acc.w += w * o.w;
  }
  const bool any = l > 0.f || l != l;
  const float inv = any ? 1.f / l : 0.f;
  const int64_t row = static_cast<int64_t>(t) * Hq + h;
  reinterpret_cast<uint2*>(out + row * kDv)[tid] = make_uint2(pack_bf16(acc.x * inv, acc.y * inv), pack_bf16(acc.z * inv, acc.w * inv));
  if (lse && tid == 0) lse[row] = any ? (m + log2f(l)) * 0.69314718055994531f : kNegInf;
}

// Clusters that run at once on the 148 SMs of a B200.
constexpr int kSlots = 74;

// How many clusters share a query's rows.  A cluster's time is its tiles and about
// three tiles' worth of set-up and output, a join costs about two more; the split
// that makes the waves of all clusters shortest is taken.
int pick_splits(int T, int64_t n) {
  const int64_t tiles = (n + kTile - 1) / kTile;
  int best = 1;
  int64_t best_cost = -1;
  for (int s = 1; s <= kMaxSplits && s <= tiles; ++s) {
    if (s > 1 && static_cast<int64_t>(T) * s > 2 * kSlots) break;
    const int64_t waves = (static_cast<int64_t>(T) * s + kSlots - 1) / kSlots;
    const int64_t cost = waves * ((tiles + s - 1) / s + 3) + (s > 1 ? 2 : 0);
    if (best_cost < 0 || cost < best_cost) {
      best = s;
      best_cost = cost;
    }
  }
  return best;
}

}  // namespace

size_t latent_mla_scratch_bytes(int T, int Hq, int64_t n) {
  const int s = pick_splits(T, n);
  return s > 1 ? static_cast<size_t>(T) * s * Hq * (kDv + 2) * sizeof(float) : 0;
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
  auto kern = a.fmt == MISA_KV_BF16  ? latent_mla_kernel<MISA_KV_BF16>
              : a.fmt == MISA_KV_MX8 ? latent_mla_kernel<MISA_KV_MX8>
                                     : latent_mla_kernel<MISA_KV_MX4>;
  cudaError_t e = ensure_dynamic_smem(reinterpret_cast<const void*>(kern), kSmemBytes);
  if (e != cudaSuccess) return e;
  e = launch_pdl(kern, dim3(static_cast<unsigned>(a.T) * p.nsplit * 2), dim3(kThreads), kSmemBytes, stream, 0, qmap, p);
  if (e != cudaSuccess || p.nsplit == 1) return e;
  return launch_pdl(latent_join_kernel, dim3(static_cast<unsigned>(a.T) * a.Hq), dim3(128), 0, stream, 0,
                    static_cast<const float*>(p.part_o), static_cast<const float*>(p.part_ml), a.Hq, p.nsplit, a.out, a.lse);
}

}  // namespace misa
