// prefill_fp4.cu -- tensor-core paged attention of prefill chunks over the 4-bit
// cache.
//
// Page "LLM推論エンジンvLLMの内部構造を徹底解説": section "エンジンの中核" -- a
// prefill is compute-bound; section "高度な機能群" -- a chunk attends to the
// context cached before it as well as to itself; section "PagedAttentionの仕組み"
// -- keys are read through the sequence's block table.
//
// Work items, tiles and the softmax are those of the bf16 prefill kernel: two
// 128-row Q tiles that read the same keys, 128 keys at a time, S and O in tensor
// memory, P written back over S.  What differs is how the operands arrive:
//
//   warps 8, 10 - 12, 14, 15  read the codes and scales of the tile's eight blocks one
//               phase ahead into registers (4.5 bits a value: 18 KB a tile),
//               convert them to f16 -- code * scale is exact there -- and store
//               them as the 128-byte swizzled K and V tiles that tcgen05.mma
//               reads; slots past the sequence are stored as zeros.  They run
//               on issue slots that the softmax leaves free.
//   warp 8      also loads the bf16 Q tiles by TMA, and takes the items
//   warps 0..7  turn their query rows to f16 in place, each row times a power of
//               two that brings its largest value into [1, 2) (bf16's bits fit),
//               then run the softmax; P is f16, 2^7 times itself (at most 2^15),
//               so that its small values keep their bits
//   warp 9      MMA issuer
//
// Bound: the softmax's exponentials and the MMAs that wait for them (half of the
// cycles each), not the cache's bytes.  Four chunks of 1024 over 2712 .. 5048 tokens
// (32 + 8 heads of 128): 232 us in a short burst, 61 % of the bf16 rate, against 230 of
// the bf16 prefill kernel on a bf16 cache; 254 us, 56 %, in a long loop.
//
// A CTA's first item goes by its number, the others it takes from a counter as
// the one before has two tiles left: the list is heaviest first, so the CTAs
// end close together.
//
// Fewer items than half the SMs are cut along their keys: a cluster of two to eight
// CTAs takes an item, each an equal stretch of its tiles, and each joins an equal
// share of its rows from the others' shared memory.  One chunk of 512 over 8192
// tokens, 64 items: 77.5 us, 133 without; two of 247 over up to 2953 on one kv-head,
// 32 items: 26.2, 53.7 without.  (The join takes 5 us; parts stored to the CTA that
// joins them, 16 bytes a lane, instead of loaded by it: 79.5 and 29.)
//
// Every mbarrier wait is bounded by a time limit; a wait that runs out sets a
// status bit in the workspace and the CTA winds down instead of hanging.
#include <cuda.h>
#include <float.h>
#include <math.h>

#include "pa_fastmath.cuh"
#include "pa_fp4.cuh"
#include "pa_internal.cuh"
#include "pa_prefill_plan.cuh"
#include "pa_tcgen05.cuh"
#include "pa_tma.cuh"
#include "pa_wait.cuh"

namespace pa {
namespace {

constexpr int kTileBlocks = KT / kBlockSize;    // 8 cache blocks per tile
// K and V tiles.  V(t) is needed a round after K(t), and the stages of both free
// up together at a round's end: with two K stages the next K tile was late.
constexpr int kKStages = 3, kVStages = 2;
constexpr int kThreads = 512;                   // 16 warps = 4 warpgroups
// Six producers: 8, 10, 11, 12, 14, 15.  Four chunks of 1024 over 2712 .. 5048
// tokens: 358 us with three producers in 384 threads (a producer warp is bound
// by its own latencies), 256 with six, 255 with seven, 247 with none of their
// conversions.
constexpr int kWarpQ = 8, kWarpMma = 9, kWarpIdle = 13;
constexpr int kProducers = 6;
// Registers: 2 x 128 x 192 + 2 x 128 x 64 = 512 x 128 (184 and 72: 276 us, the
// softmax's row of scores no longer fits)
constexpr int kRegsLaunch = 128, kRegsSoftmax = 192, kRegsOther = 64;
static_assert(2 * 128 * kRegsSoftmax + 256 * kRegsOther <= kThreads * kRegsLaunch,
              "register split exceeds the launch allocation");
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemO = 0, kTmemS = 256;    // + 128 * half
constexpr float kRescaleThreshold = 8.0f;       // log2 units: move the max only past 2^8
constexpr float kPShift = 7.0f;                 // P is held times 2^7
constexpr int kMaxCluster = 8;                  // CTAs that share an item
constexpr int kMaxChains = 8;                   // independent max chains over a row of scores

template <int D>
struct Layout {
  static constexpr int kPanels = D / 64;            // 64-wide slices of D
  static constexpr int kPanelBytes = 128 * 128;     // 128 rows x 128 bytes, of Q, K or V
  static constexpr int kBytes = kPanels * kPanelBytes;  // one Q, K or V tile
  static constexpr int q_off = 0;                   // two Q tiles (the two halves)
  static constexpr int k_off = q_off + 2 * kBytes;
  static constexpr int v_off = k_off + kKStages * kBytes;
  static constexpr int bar_off = v_off + kVStages * kBytes;
  static constexpr int used = bar_off + 256;
  // one CTA per SM (its tensor memory is all of the SM's)
  static constexpr int total = (used < 120 * 1024 ? 120 * 1024 : used) + 1024;
  static_assert(total <= 227 * 1024, "shared memory of one CTA");
  static_assert(bar_off - k_off >= 2 * 128 * (4 * D + 8), "a part in the place of K and V");
};

// Where a part's row r lies in the stages of K and V once they are read: O in fp32,
// its 16-byte units xor the row (the lanes of a store are 32 rows), and behind all
// rows each one's maximum and sum.
template <int D>
__device__ __forceinline__ uint32_t part_at(uint32_t at, int r, int unit) {
  return at + r * (4 * D) + ((unit ^ (r & (D / 4 - 1))) << 4);
}
template <int D>
__device__ __forceinline__ uint32_t part_ml(uint32_t at, int r) {
  return at + 2 * 128 * 4 * D + r * 8;
}

// mbarrier indices
enum : int {
  kBarQFull = 0,                    // the bf16 Q tiles have arrived
  kBarQReady,                       // and are f16
  kBarQEmpty,
  kBarKFull,                        // + stage
  kBarKEmpty = kBarKFull + kKStages,
  kBarVFull = kBarKEmpty + kKStages,
  kBarVEmpty = kBarVFull + kVStages,
  kBarSFull = kBarVEmpty + kVStages,  // + half
  kBarPFull = kBarSFull + 2,
  kBarODone = kBarPFull + 2,
  kBarItem = kBarODone + 2,          // + ring slot of items
  kBarDrain = kBarItem + 8,          // the MMAs under way when a role gave up
  kNumBars
};
constexpr int kItemRing = 8;
static_assert(kNumBars * 8 <= 256, "barriers must fit their 256-byte area");

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// The eight codes of a word times `scale`, as one 16-byte unit of a swizzled tile
__device__ __forceinline__ void store_unit(uint32_t addr, uint32_t word, __half2 scale) {
  __half2 x[4];
  e2m1x8_to_half2(word, x);
  uint32_t r[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 y = __hmul2(x[i], scale);
    r[i] = *reinterpret_cast<const uint32_t*>(&y);
  }
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3])
               : "memory");
}

// One lane's share of the K or the V of a cache block: two pieces of codes, 16
// bytes each at D = 128, 8 at D = 64, and their scales.
//
// A piece of K is 2 or 4 units (8 dims, 16 bytes of f16) of one token, a piece
// of V that of two tokens.  The unit's place in a 128-byte swizzled tile is its
// number xor the row's low three bits: with the lane's part of both in `at`, a
// store takes one xor with a constant.  Lanes are dealt to pieces, and the
// units of a V piece ordered by lane, so that the eight lanes that store at
// once meet different banks.
template <int D>
struct Share {
  uint32_t w[2][D / 32];
  uint32_t s[2];

  // K: piece `i` of a lane is token 8 i + token_k, chunk c of the row (D / 4
  // dims, one or two scales)
  static __device__ __forceinline__ int chunk_k(int lane) {
    return D == 128 ? (lane & 1) | (lane >> 2 & 2) : lane & 3;
  }
  static __device__ __forceinline__ int token_k(int lane) {
    return D == 128 ? (lane >> 1 & 3) | (lane >> 2 & 4) : lane >> 2;
  }
  // offset in a K tile of this lane's unit 0 in a block's first row of 8
  static __device__ __forceinline__ uint32_t at_k(int lane) {
    const int c = chunk_k(lane), token = token_k(lane);
    return D == 128 ? (c >> 1) * Layout<D>::kPanelBytes + token * 128 +
                          (((c & 1) * 4 ^ token) << 4)
                    : token * 128 + ((2 * c ^ token) << 4);
  }
  // V: piece `i` is tokens 4 t + 2 i, + 1 of chunk c (D / 8 dims), c = lane / 4,
  // t = lane % 4; lanes of t >= 2 store their odd units (at D = 64, their
  // second piece) first
  static __device__ __forceinline__ uint32_t at_v(int lane) {
    const int c = lane >> 2, t = lane & 3;
    return D == 128 ? (c >> 2) * Layout<D>::kPanelBytes + t * 512 +
                          ((2 * (c & 3) ^ 4 * (t & 1) ^ t >> 1) << 4)
                    : t * 512 + ((c ^ 4 * (t & 1)) << 4);
  }

  // `tile`: the block's, or null (zeros)
  __device__ __forceinline__ void load_k(const uint8_t* tile, int lane) {
    const int at = token_k(lane) * 4 + chunk_k(lane);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (D == 128) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (tile) v = *(const uint4*)(tile + i * 512 + at * 16);
        s[i] = tile ? *(const uint16_t*)(tile + Fp4Tile<D>::ks_off + i * 64 + at * 2) : 0;
        w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
      } else {
        uint2 v = make_uint2(0, 0);
        if (tile) v = *(const uint2*)(tile + i * 256 + at * 8);
        s[i] = tile ? tile[Fp4Tile<D>::ks_off + i * 32 + at] : 0;
        w[i][0] = v.x; w[i][1] = v.y;
      }
    }
  }
  __device__ __forceinline__ void load_v(const uint8_t* tile, int lane) {
    const int c = lane >> 2, t = lane & 3;
    // the scales of tokens 4 t .. 4 t + 3
    s[0] = tile ? *(const uint32_t*)(tile + Fp4Tile<D>::vs_off + (D == 128 ? c : c >> 1) * 16 +
                                     4 * t)
                : 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (D == 128) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (tile) v = *(const uint4*)(tile + Fp4Tile<D>::v_off + i * 512 + lane * 16);
        w[i][0] = v.x; w[i][1] = v.y; w[i][2] = v.z; w[i][3] = v.w;
      } else {
        uint2 v = make_uint2(0, 0);
        if (tile) v = *(const uint2*)(tile + Fp4Tile<D>::v_off + i * 256 + lane * 8);
        w[i][0] = v.x; w[i][1] = v.y;
      }
    }
  }
  // Into the 16 rows at `at` (the block's first row's offset in the tile plus
  // at_k / at_v); of tokens from `held` on, zeros.
  __device__ __forceinline__ void store_k(uint32_t at, int held, int lane) const {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint32_t bytes = 8 * i + token_k(lane) < held ? s[i] : 0u;
      const __half2 two = e4m3x2_to_half2(bytes);
      const __half2 lo = __low2half2(two), hi = __high2half2(two);
#pragma unroll
      for (int j = 0; j < D / 32; ++j)
        store_unit((at ^ (j << 4)) + i * 1024, w[i][j], D == 128 && j >= 2 ? hi : lo);
    }
  }
  __device__ __forceinline__ void store_v(uint32_t at, int held, int lane) const {
    const int t = lane & 3;
    const bool turn = t >= 2;
    uint32_t bytes = s[0];
    const int n = held - 4 * t;  // of this lane's four tokens
    if (n < 4) bytes = n <= 0 ? 0u : bytes & (0xffffffffu >> (32 - 8 * n));
    if (D == 64 && turn) {       // pieces in the other order
      at = (at ^ 32) + 256;
      bytes = bytes << 16 | bytes >> 16;
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const __half2 two = e4m3x2_to_half2(i ? bytes >> 16 : bytes & 0xffffu);
      const __half2 scale[2] = {__low2half2(two), __high2half2(two)};
#pragma unroll
      for (int k = 0; k < 2; ++k) {  // token of the pair
        if constexpr (D == 128) {
          const uint32_t a = w[i][2 * k], b = w[i][2 * k + 1];
#pragma unroll
          for (int j = 0; j < 2; ++j)
            store_unit((at ^ ((2 * i + k ^ j) << 4)) + (2 * i + k) * 128,
                       turn == (j == 0) ? b : a, scale[k]);
        } else {
          const uint32_t row = i == 0 ? at : turn ? (at ^ 32) - 256 : (at ^ 32) + 256;
          store_unit((row ^ (k << 4)) + k * 128, turn ? w[1 - i][k] : w[i][k], scale[k]);
        }
      }
    }
  }
};

// A cluster of several CTAs shares an item: each takes an equal stretch of its
// tiles, and joins an equal share of its rows.
__device__ __forceinline__ int cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return (int)r;
}
__device__ __forceinline__ int cluster_ctas() {
  uint32_t n;
  asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(n));
  return (int)n;
}
// every thread of the cluster, its shared-memory writes before the others' reads
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// this CTA's shared-memory address in CTA `rank` of the cluster
__device__ __forceinline__ uint32_t in_cta(uint32_t addr, int rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
// the tiles of an item that this CTA takes: all of them, but in a cluster
template <bool kSplit>
__device__ __forceinline__ int first_tile(int ntiles) {
  return kSplit ? cluster_rank() * ntiles / cluster_ctas() : 0;
}
template <bool kSplit>
__device__ __forceinline__ int end_tile(int ntiles) {
  return kSplit ? (cluster_rank() + 1) * ntiles / cluster_ctas() : ntiles;
}

// An item of the list, with the key tiles that the device's lengths give it: a list
// made on the host is as old as the captured call that it is part of.
__device__ __forceinline__ ItemInfo item_now(const AttnParams& p, const PrefillWork& work, int w,
                                             int pair_heads) {
  ItemInfo it = load_item(p, work, w);
  const int last_row = min((it.qt0 + (pair_heads ? 1 : 2)) * QT, it.ql) - 1;
  const int wide = (p.max_blocks_per_seq + kTileBlocks - 1) / kTileBlocks;
  it.ntiles = min(max(it.L - it.ql + last_row, 0) / KT + 1, wide);
  return it;
}

// The tiles of a CTA's items one after the other, as the producers walk them
template <bool kSplit>
struct TileCursor {
  int k = -1, t = 0, ntiles = 0;  // item of this CTA, tile in it, end of its tiles
  int w;                          // its place in the list
  int kvh, L, nblk;
  const int32_t* table;
  bool done = false;
  // item(k): the place of this CTA's item k in the list, past its end if none
  template <typename Item>
  __device__ __forceinline__ void next(const AttnParams& p, const PrefillWork& work, int pair_heads,
                                       int num_items, Item item) {
    if (done) return;
    while (++t >= ntiles) {
      w = item(++k);
      if (w >= num_items) {
        done = true;
        return;
      }
      const ItemInfo it = item_now(p, work, w, pair_heads);
      t = first_tile<kSplit>(it.ntiles) - 1;
      ntiles = end_tile<kSplit>(it.ntiles);
      kvh = it.head0 / p.group;
      L = it.L;
      nblk = (it.L + kBlockSize - 1) / kBlockSize;
      table = p.block_tables + (int64_t)it.seq * p.max_blocks_per_seq;
    }
  }
  // lane b < 8: the id of the tile's block b, or -1 (past the sequence, or
  // outside the pool)
  __device__ __forceinline__ int ids(const AttnParams& p, int lane) const {
    const int b = t * kTileBlocks + lane;
    int id = -1;
    if (!done && lane < kTileBlocks && b < nblk && b < p.max_blocks_per_seq) id = table[b];
    return id < p.num_blocks ? id : -1;
  }
};

template <int D, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
prefill_fp4_kernel(const AttnParams p, const float v_scale, const __grid_constant__ CUtensorMap tm_q,
                   int pair_heads, const __grid_constant__ PrefillWork work) {
  using LY = Layout<D>;
  constexpr int kPanels = LY::kPanels;
  extern __shared__ unsigned char smem_raw[];
  __shared__ uint32_t sh_tmem_base;
  __shared__ int sh_abort;
  __shared__ int sh_loaded;  // the last item whose Q was asked for
  __shared__ int sh_item[kItemRing];

  // (from one lane: the compiler then keeps what follows from it, above all the
  // MMA issuer's descriptors, in uniform registers; with the elected lane of its
  // branches, 254 -> 234 us at the case named above)
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
  const uint32_t base = ((uint32_t)__cvta_generic_to_shared(smem_raw) + 1023u) & ~1023u;
  const uint32_t sQ = base + LY::q_off, sK = base + LY::k_off, sV = base + LY::v_off,
                 sBar = base + LY::bar_off;
  auto bar = [&](int i) { return sBar + 8u * (uint32_t)i; };
  volatile int* abort_flag = &sh_abort;

  if (threadIdx.x == 0) {
    sh_abort = 0;
    sh_loaded = -1;
    mbar_init(bar(kBarQFull), 1);
    mbar_init(bar(kBarQReady), 8);  // one arrival per softmax warp
    mbar_init(bar(kBarQEmpty), 1);
    for (int i = 0; i < kKStages; ++i) {
      mbar_init(bar(kBarKFull + i), kProducers);
      mbar_init(bar(kBarKEmpty + i), 1);
    }
    for (int i = 0; i < kVStages; ++i) {
      mbar_init(bar(kBarVFull + i), kProducers);
      mbar_init(bar(kBarVEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(kBarSFull + i), 1);
      mbar_init(bar(kBarPFull + i), 4);  // one arrival per softmax warp of the half
      mbar_init(bar(kBarODone + i), 1);
    }
    for (int i = 0; i < kItemRing; ++i) mbar_init(bar(kBarItem + i), 1);
    mbar_init(bar(kBarDrain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    prefetch_tmap(&tm_q);
  }
  if (warp == kWarpMma) {
    tmem_alloc((uint32_t)__cvta_generic_to_shared(&sh_tmem_base), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, sh_tmem_base, 0);

  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int num_items = work.count > 0 ? work.count : p.ws_items[0].x;
  int* status = p.ws_status;
  // the place in the list of this CTA's item k.  (A slot of the ring is written
  // again eight items later, which every role must have reached by then.)
  auto item_at = [&](int k) {
    int w = INT32_MAX;
    if (wait_bar_warp(bar(kBarItem + k % kItemRing), (k / kItemRing) & 1, abort_flag, status))
      w = *(volatile int*)&sh_item[k % kItemRing];
    return __shfl_sync(0xffffffffu, w, 0);
  };

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsOther));
    if (warp != kWarpMma && warp != kWarpIdle) {
      // ============ producers: K and V tiles from codes; warp 8 the Q tiles too ============
      // A phase is the K or the V of a tile.  A warp takes one or two of the
      // phase's blocks, every sixth; the codes of the phase after are
      // loaded as each block of this one has been stored.
      const int me = warp == kWarpQ ? 0 : warp - (warp < kWarpIdle ? 9 : 10);  // 0 .. 5
      const int k0 = me, v0 = kProducers - 1 - me;  // its first block of a K / V phase
      const uint8_t* cache = (const uint8_t*)p.k_cache;
      // warp 8, lane 0: item k of this CTA is number w of the list
      auto publish = [&](int k, int w) {
        sh_item[k % kItemRing] = w;
        mbar_arrive(bar(kBarItem + k % kItemRing));
        // the last CTA to run out of items leaves the counters at zero
        if (!kSplit && w >= num_items && atomicAdd(p.ws_header + kWsDone, 1) == (int)gridDim.x - 1)
          p.ws_header[kWsClaim] = p.ws_header[kWsDone] = 0;
      };
      if (warp == kWarpQ && lane == 0) {
        publish(0, kSplit ? blockIdx.x / cluster_ctas() : blockIdx.x);
        if (kSplit) publish(1, INT32_MAX);  // one item to a cluster
      }
      TileCursor<kSplit> cur, nxt;
      nxt.next(p, work, pair_heads, num_items, item_at);
      int ids_n = nxt.ids(p, lane);
      auto tile_of = [&](int ids, int b, int kvh) -> const uint8_t* {
        const int id = __shfl_sync(0xffffffffu, ids, b & 7);
        return b < kTileBlocks && id >= 0
                   ? cache + ((int64_t)id * p.num_kv_heads + kvh) * Fp4Tile<D>::bytes
                   : nullptr;
      };
      Share<D> sh[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) sh[i].load_k(tile_of(ids_n, k0 + kProducers * i, nxt.kvh), lane);
      uint32_t g = 0;  // global tile counter
      bool ok = true;
      int item = -1;
      while (!nxt.done && ok) {
        cur = nxt;
        const int ids = ids_n;
        if (warp == kWarpQ && cur.k != item) {
          // ---- the item's two Q tiles
          item = cur.k;
          if (lane == 0) {
            if (item > 0) ok = wait_bar(bar(kBarQEmpty), (item - 1) & 1, abort_flag, status);
            if (ok) {
              const ItemInfo it = load_item(p, work, cur.w);
              mbar_expect_tx(bar(kBarQFull), 2 * LY::kBytes);
              sh_loaded = item;
              for (int h = 0; h < 2; ++h) {
                const int head = pair_heads ? it.head0 + h : it.head0;
                const int qt = pair_heads ? it.qt0 : it.qt0 + h;
                for (int pn = 0; pn < kPanels; ++pn)
                  tma_load_3d(sQ + h * LY::kBytes + pn * LY::kPanelBytes, &tm_q, 64 * pn, head,
                              it.q0 + qt * QT, bar(kBarQFull));
              }
            }
          }
          ok = __shfl_sync(0xffffffffu, ok, 0);
          if (!ok) break;
        }
        // the item after this one, when two of its tiles are left; made known at
        // the end of the first of them, when the counter has answered
        const bool take = !kSplit && warp == kWarpQ && lane == 0 && cur.t == max(cur.ntiles - 2, 0);
        int taken = 0;
        if (take) {
          taken = (int)gridDim.x + atomicAdd(p.ws_header + kWsClaim, 1);
          if (cur.ntiles == 1) publish(cur.k + 1, taken);
        }
        nxt.next(p, work, pair_heads, num_items, item_at);
        ids_n = nxt.ids(p, lane);
        const int key0 = cur.t * KT;
#pragma unroll
        for (int phase = 0; phase < 2 && ok; ++phase) {
          const uint32_t nst = phase ? kVStages : kKStages;
          const int st = g % nst;
          const int full = (phase ? kBarVFull : kBarKFull) + st;
          const int empty = (phase ? kBarVEmpty : kBarKEmpty) + st;
          if (g >= nst) {
            ok = wait_bar_warp(bar(empty), ((g / nst) - 1) & 1, abort_flag, status);
            if (!ok) break;
          }
          const uint32_t dst = phase ? sV + st * LY::kBytes + Share<D>::at_v(lane)
                                     : sK + st * LY::kBytes + Share<D>::at_k(lane);
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int b = (phase ? v0 : k0) + kProducers * i;
            if (b < kTileBlocks) {
              const int held = cur.L - key0 - b * kBlockSize;  // tokens of the block
              if (phase)
                sh[i].store_v(dst + b * 2048, held, lane);
              else
                sh[i].store_k(dst + b * 2048, held, lane);
            }
            // the same slot of the next phase: this tile's V, the next one's K
            if (phase)
              sh[i].load_k(tile_of(ids_n, k0 + kProducers * i, nxt.kvh), lane);
            else
              sh[i].load_v(tile_of(ids, v0 + kProducers * i, cur.kvh), lane);
          }
          fence_proxy_async_smem();  // the stores, before the tensor core reads them
          __syncwarp();
          if (elect_one()) mbar_arrive(bar(full));
        }
        if (take && cur.ntiles > 1) publish(cur.k + 1, taken);
        __syncwarp();
        ++g;
      }
    } else if (warp == kWarpMma) {
      // =========================== MMA issuer ===========================
      // (as in the bf16 kernel: P.V of tile g-1 before Q K^T of tile g, per half)
      constexpr uint32_t idesc_qk = instr_desc(128, KT, 0, 0, 0);
      constexpr uint32_t idesc_pv = instr_desc(128, D, 0, 1, 0);
      const uint64_t dq0 = smem_desc(sQ, 16, 1024);
      const uint64_t dk0 = smem_desc(sK, 16, 1024);
      const uint64_t dv0 = smem_desc(sV, LY::kPanelBytes, 1024);
      uint32_t g = 0;
      bool ok = true;
      auto issue_pv = [&](int h, uint32_t gt, bool first_of_item) {  // O_h += P_h V (tile gt)
        ok = wait_bar_warp(bar(kBarPFull + h), gt & 1, abort_flag, status);
        if (!ok) return;
        tc_fence_after();
        if (elect_one()) {
          const uint64_t dv = dv0 + (uint64_t)(((gt % kVStages) * LY::kBytes) >> 4);
          const uint32_t dst = tmem + kTmemO + 128 * h;
          const uint32_t pa = tmem + kTmemS + 128 * h;
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            umma_bf16_ts(dst, pa + 8 * kk, dv + (uint64_t)((kk * 2048) >> 4), idesc_pv,
                         (first_of_item && kk == 0) ? 0u : 1u);
          umma_commit(bar(kBarODone + h));
        }
        __syncwarp();
      };
      auto issue_qk = [&](int h, uint32_t gt) {  // S_h = Q_h K^T (tile gt)
        if (elect_one()) {
          const uint64_t dk = dk0 + (uint64_t)(((gt % kKStages) * LY::kBytes) >> 4);
          const uint64_t dq = dq0 + (uint64_t)((h * LY::kBytes) >> 4);
          const uint32_t dst = tmem + kTmemS + 128 * h;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t o = ((kk / 4) * LY::kPanelBytes + (kk % 4) * 32) >> 4;
            umma_bf16(dst, dq + o, dk + o, idesc_qk, kk > 0 ? 1u : 0u);
          }
          umma_commit(bar(kBarSFull + h));
        }
        __syncwarp();
      };
      for (int k = 0; ok; ++k) {
        const int w = item_at(k);
        if (w >= num_items) break;
        const ItemInfo it = item_now(p, work, w, pair_heads);
        const int t0 = first_tile<kSplit>(it.ntiles), t1 = end_tile<kSplit>(it.ntiles);
        if (kSplit && t0 == t1) continue;  // fewer tiles than CTAs: no Q comes
        ok = wait_bar_warp(bar(kBarQReady), k & 1, abort_flag, status);
        const uint32_t g_first = g;
        for (int t = t0; t < t1 && ok; ++t, ++g) {
          ok = wait_bar_warp(bar(kBarKFull + g % kKStages), (g / kKStages) & 1, abort_flag, status);
          if (ok && t > t0)
            ok = wait_bar_warp(bar(kBarVFull + (g - 1) % kVStages), ((g - 1) / kVStages) & 1,
                               abort_flag, status);
          if (!ok) break;
          tc_fence_after();
          for (int h = 0; h < 2 && ok; ++h) {
            if (t > t0) issue_pv(h, g - 1, g - 1 == g_first);  // P_h of the previous tile
            if (ok) issue_qk(h, g);
          }
          if (ok && elect_one()) {
            umma_commit(bar(kBarKEmpty + g % kKStages));
            if (t > t0) umma_commit(bar(kBarVEmpty + (g - 1) % kVStages));
            if (t == t1 - 1) umma_commit(bar(kBarQEmpty));
          }
          __syncwarp();
        }
        if (ok && t1 > t0) {  // P.V of the item's last tile
          const uint32_t gl = g - 1;
          ok = wait_bar_warp(bar(kBarVFull + gl % kVStages), (gl / kVStages) & 1, abort_flag, status);
          if (ok) tc_fence_after();
          for (int h = 0; h < 2 && ok; ++h) issue_pv(h, gl, gl == g_first);
          if (ok && elect_one()) umma_commit(bar(kBarVEmpty + gl % kVStages));
          __syncwarp();
        }
      }
    }
  } else {
    // =========================== softmax (two halves) ===========================
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    const int h = warp >> 2;                   // which Q tile
    const int quarter = warp & 3;              // TMEM lanes 32*quarter .. +31
    const int row = quarter * 32 + lane;       // query row of this thread in its tile
    const uint32_t lane_addr = (uint32_t)(quarter * 32) << 16;
    const uint32_t tS = tmem + lane_addr + kTmemS + 128 * h;
    const uint32_t tO = tmem + lane_addr + kTmemO + 128 * h;
    uint32_t g = 0;
    bool ok = true;
    // this row of item k's Q from bf16 to f16 in place, times 2^-e (e: the
    // exponent of its largest value, as far as 2^-e is a normal number); sets the
    // scale of the row's scores
    float sl2_next = 0.f;
    float m_run = -INFINITY, l_run = 0.f;  // this row's running max and sum
    auto convert_q = [&](int k) {
      ok = wait_bar_warp(bar(kBarQFull), k & 1, abort_flag, status);
      if (!ok) return;
      uint32_t q[D / 2];
      const uint32_t line = sQ + h * LY::kBytes + row * 128;
#pragma unroll
      for (int u = 0; u < D / 8; ++u)
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                     : "=r"(q[4 * u]), "=r"(q[4 * u + 1]), "=r"(q[4 * u + 2]), "=r"(q[4 * u + 3])
                     : "r"(line + (u / 8) * LY::kPanelBytes + (((u % 8) ^ (row & 7)) << 4)));
      uint32_t top = 0;  // the largest magnitude's bits (bf16 order is that of its bits)
#pragma unroll
      for (int i = 0; i < D / 2; ++i)
        top = max(top, max(q[i] & 0x7fffu, q[i] >> 16 & 0x7fffu));
      const int e = min(max((int)(top >> 7) - 127, -126), 126);
      const float f = exp2i(-e);
      // (a scale below the smallest normal number would make NaN of a masked score)
      sl2_next = fmaxf(p.scale_log2 * exp2i(e), FLT_MIN);
#pragma unroll
      for (int u = 0; u < D / 8; ++u) {
#pragma unroll
        for (int i = 4 * u; i < 4 * u + 4; ++i)
          q[i] = pack_f16x2(__uint_as_float(q[i] << 16) * f,
                            __uint_as_float(q[i] & 0xffff0000u) * f);
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(
                         line + (u / 8) * LY::kPanelBytes + (((u % 8) ^ (row & 7)) << 4)),
                     "r"(q[4 * u]), "r"(q[4 * u + 1]), "r"(q[4 * u + 2]), "r"(q[4 * u + 3])
                     : "memory");
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (elect_one()) mbar_arrive(bar(kBarQReady));
    };
    {
      const int w = item_at(0);
      bool any = w < num_items;
      if (kSplit && any) {
        const int n = item_now(p, work, w, pair_heads).ntiles;
        any = first_tile<kSplit>(n) < end_tile<kSplit>(n);
      }
      if (any) convert_q(0);
    }
    for (int k = 0; ok; ++k) {
      const int w = item_at(k);
      if (w >= num_items) break;
      const ItemInfo it = item_now(p, work, w, pair_heads);
      const int t0 = first_tile<kSplit>(it.ntiles), t1 = end_tile<kSplit>(it.ntiles);
      const int head = pair_heads ? it.head0 + h : it.head0;
      const int qt = pair_heads ? it.qt0 : it.qt0 + h;
      const int jq = qt * QT + row;
      const bool row_valid = jq < it.ql;
      const int pos = row_valid ? it.L - it.ql + jq : -1;  // last visible key
      const int min_pos = it.L - it.ql + qt * QT;          // smallest position in the tile
      const float sl2 = sl2_next;
      m_run = -INFINITY;
      l_run = 0.f;
      const uint32_t g_first = g;
      for (int t = t0; t < t1 && ok; ++t, ++g) {
        // S_h of tile g is complete; so is P.V of tile g-1 (issued before it)
        ok = wait_bar_warp(bar(kBarSFull + h), g & 1, abort_flag, status);
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[KT];
        tmem_ld32_at<0>(tS, sr);
        tmem_ld32_at<32>(tS + 32, sr);
        tmem_ld32_at<64>(tS + 64, sr);
        tmem_ld32_at<96>(tS + 96, sr);
        tmem_ld_wait();
        float s[KT];
#pragma unroll
        for (int n = 0; n < KT; ++n) s[n] = __uint_as_float(sr[n]);
        // ---- keys past this row's last visible one are out
        if (t * KT + KT - 1 > min_pos) {
          const int lim = pos - t * KT;
#pragma unroll
          for (int n = 0; n < KT; ++n) s[n] = n <= lim ? s[n] : -INFINITY;
        }
        // ---- row max of the raw scores: kMaxChains independent chains of
        // three-input maxima, then a tree
        float mc[kMaxChains];
#pragma unroll
        for (int q = 0; q < kMaxChains; ++q) mc[q] = fmaxf(s[2 * q], s[2 * q + 1]);
#pragma unroll
        for (int n = 2 * kMaxChains; n < KT; n += 2 * kMaxChains) {
#pragma unroll
          for (int q = 0; q < kMaxChains; ++q) mc[q] = max3(mc[q], s[n + 2 * q], s[n + 2 * q + 1]);
        }
#pragma unroll
        for (int c = kMaxChains; c > 1; c /= 2) {
#pragma unroll
          for (int q = 0; q < c / 2; ++q) mc[q] = fmaxf(mc[q], mc[q + c / 2]);
        }
        const float mx = sl2 * mc[0];
        // ---- running max (log2 units): moved only when it grows past the threshold
        float alpha = 1.f;
        if (mx > m_run + kRescaleThreshold || (m_run == -INFINITY && mx > -INFINITY)) {
          alpha = (m_run == -INFINITY) ? 0.f : ex2(m_run - mx);
          m_run = mx;
        }
        const float neg_base = (m_run == -INFINITY) ? 0.f : kPShift - m_run;
        // ---- P = 2^7 exp2(S * scale * log2(e) - max) on pairs of columns; two
        // f16 per word, written over the first half of S
        const uint64_t scale2 = f2(sl2, sl2), base2 = f2(neg_base, neg_base);
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t pw[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) {
            const int n = 64 * c + 2 * j;
            const uint64_t x = fma2(f2(s[n], s[n + 1]), scale2, base2);
            float x0, x1;
            f2_split(x, x0, x1);
            const uint64_t e = f2(ex2(x0), ex2(x1));  // masked: ex2(-inf) = 0
            acc[j & 3] = add2(acc[j & 3], e);
            float e0, e1;
            f2_split(e, e0, e1);
            pw[j] = pack_f16x2(e0, e1);
          }
          tmem_st32(tS + 32 * c, pw);
        }
        float sum;
        {
          float a0, a1;
          f2_split(add2(add2(acc[0], acc[1]), add2(acc[2], acc[3])), a0, a1);
          sum = a0 + a1;
        }
        l_run = l_run * alpha + sum;
        // ---- O carries the old max: rescale it (P.V of tile g-1 is complete)
        if (g != g_first && __any_sync(0xffffffffu, alpha != 1.f)) {
          const uint64_t alpha2 = f2(alpha, alpha);
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t orr[32];
            tmem_ld32(tO + c * 32, orr);
            tmem_ld_wait();
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              uint32_t lo, hi;
              u2_split(mul2(u2(orr[2 * e], orr[2 * e + 1]), alpha2), lo, hi);
              orr[2 * e] = lo;
              orr[2 * e + 1] = hi;
            }
            tmem_st32(tO + c * 32, orr);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (elect_one()) mbar_arrive(bar(kBarPFull + h));
      }
      if constexpr (kSplit) {
        if (ok && t1 > t0) ok = wait_bar_warp(bar(kBarODone + h), (g - 1) & 1, abort_flag, status);
        break;  // one item to a cluster
      }
      // the next item's Q while this one's last P.V runs
      if (ok && item_at(k + 1) < num_items) convert_q(k + 1);
      if (!ok || it.ntiles == 0) continue;
      // ---- epilogue: O / l to global memory
      ok = wait_bar_warp(bar(kBarODone + h), (g - 1) & 1, abort_flag, status);
      if (!ok) break;
      tc_fence_after();
      const float inv = v_scale / l_run;
      __nv_bfloat16* orow =
          (__nv_bfloat16*)p.out + ((int64_t)(it.q0 + jq) * p.num_q_heads + head) * D;
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orr[32];
        tmem_ld32(tO + c * 32, orr);
        tmem_ld_wait();
        if (row_valid) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 pk;
            pk.x = pack_bf16x2(__uint_as_float(orr[8 * v + 0]) * inv, __uint_as_float(orr[8 * v + 1]) * inv);
            pk.y = pack_bf16x2(__uint_as_float(orr[8 * v + 2]) * inv, __uint_as_float(orr[8 * v + 3]) * inv);
            pk.z = pack_bf16x2(__uint_as_float(orr[8 * v + 4]) * inv, __uint_as_float(orr[8 * v + 5]) * inv);
            pk.w = pack_bf16x2(__uint_as_float(orr[8 * v + 6]) * inv, __uint_as_float(orr[8 * v + 7]) * inv);
            *reinterpret_cast<uint4*>(orow + c * 32 + 8 * v) = pk;
          }
        }
      }
      // the next item's first P.V overwrites O: every lane has read it
      tc_fence_before();
    }
    if constexpr (kSplit) {
      // ---- this CTA's part of O, and each row's max and sum, where K and V were
      asm volatile("bar.sync 1, 256;" ::: "memory");  // the other half's MMAs too
      tc_fence_after();
      const bool part = __all_sync(0xffffffffu, ok && g > 0);
      const int r = h * QT + row;
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t orr[32];
        tmem_ld32(tO + c * 32, orr);
        tmem_ld_wait();
#pragma unroll
        for (int v = 0; v < 8; ++v)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(part_at<D>(sK, r, 8 * c + v)),
                       "r"(part ? orr[4 * v] : 0u), "r"(part ? orr[4 * v + 1] : 0u),
                       "r"(part ? orr[4 * v + 2] : 0u), "r"(part ? orr[4 * v + 3] : 0u)
                       : "memory");
      }
      asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(part_ml<D>(sK, r)), "f"(m_run),
                   "f"(l_run)
                   : "memory");
      tc_fence_before();
    }
  }

  // ---- wind down: every role is done (or gave up); free TMEM
  tc_fence_before();
  __syncthreads();
  if (sh_abort) {  // whoever gave up: the Q load and the MMAs under way end first
    if (threadIdx.x == 0 && sh_loaded >= 0)
      drain_bar(bar(kBarQFull), sh_loaded & 1, globaltimer());
    if (warp == kWarpMma) {
      if (elect_one()) umma_commit(bar(kBarDrain));
      __syncwarp();
      drain_bar(bar(kBarDrain), 0, globaltimer());
      __syncwarp();
    }
  }
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }

  if constexpr (kSplit) {
    // ---- the parts of the cluster's CTAs joined, an equal share of the rows each
    const int ctas = cluster_ctas(), w = (int)blockIdx.x / ctas;
    __syncwarp();
    cluster_sync();
    if (warp < 8 && w < num_items) {  // (the others keep too few registers)
      const ItemInfo it = load_item(p, work, w);
      constexpr int kUnits = D / 4, kRows = 2;  // (rows of a thread at once)
      const int rank = cluster_rank(), row0 = rank * 2 * QT / ctas;
      const int row1 = (rank + 1) * 2 * QT / ctas, u = threadIdx.x % kUnits;
      for (int r0 = row0 + threadIdx.x / kUnits; r0 < row1; r0 += kRows * 256 / kUnits) {
        int r[kRows];
        float m[kRows], l[kRows], y[kRows][4];
#pragma unroll
        for (int e = 0; e < kRows; ++e) {
          r[e] = min(r0 + e * 256 / kUnits, row1 - 1);
          m[e] = -INFINITY;
          l[e] = y[e][0] = y[e][1] = y[e][2] = y[e][3] = 0.f;
        }
#pragma unroll 2
        for (int i = 0; i < ctas; ++i) {  // (each CTA begins with its own part)
          const int c = rank + i < ctas ? rank + i : rank + i - ctas;
          float mc[kRows], lc[kRows], o[kRows][4];
#pragma unroll
          for (int e = 0; e < kRows; ++e) {
            asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];"
                         : "=f"(mc[e]), "=f"(lc[e])
                         : "r"(in_cta(part_ml<D>(sK, r[e]), c)));
            asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                         : "=f"(o[e][0]), "=f"(o[e][1]), "=f"(o[e][2]), "=f"(o[e][3])
                         : "r"(in_cta(part_at<D>(sK, r[e], u), c)));
          }
#pragma unroll
          for (int e = 0; e < kRows; ++e) {
            // (a part without a key that the row sees, or whose scores are all NaN,
            // has no maximum: its O is 0, or NaN)
            const float top = fmaxf(m[e], mc[e]);
            const float f = m[e] == top ? 1.f : ex2(m[e] - top);
            const float fc = mc[e] == -INFINITY ? 0.f : ex2(mc[e] - top);
            m[e] = top;
            l[e] = l[e] * f + lc[e] * fc;
#pragma unroll
            for (int k = 0; k < 4; ++k) y[e][k] = fmaf(o[e][k], fc, y[e][k] * f);
          }
        }
#pragma unroll
        for (int e = 0; e < kRows; ++e) {
          const int h = r[e] / QT, head = pair_heads ? it.head0 + h : it.head0;
          const int jq = (pair_heads ? it.qt0 : it.qt0 + h) * QT + r[e] % QT;
          if (jq >= it.ql || r0 + e * 256 / kUnits >= row1) continue;
          const float inv = v_scale / l[e];
          uint2 pk;
          pk.x = pack_bf16x2(y[e][0] * inv, y[e][1] * inv);
          pk.y = pack_bf16x2(y[e][2] * inv, y[e][3] * inv);
          *reinterpret_cast<uint2*>((__nv_bfloat16*)p.out +
                                    ((int64_t)(it.q0 + jq) * p.num_q_heads + head) * D + 4 * u) = pk;
        }
      }
    }
    __syncwarp();
    cluster_sync();  // the others have read this CTA's shared memory
  }
}

template <int D>
cudaError_t launch_d(const AttnParams& p, float v_scale, int max_query_len,
                     const int32_t* seq_lens_host, const int32_t* query_start_loc_host,
                     cudaStream_t stream, int max_ctas) {
  CUtensorMap tq;
  if (!make_map(&tq, p.q, D, p.num_q_heads, p.num_tokens, (uint64_t)D * 2,
                (uint64_t)p.num_q_heads * D * 2, 1, QT))
    return cudaErrorInvalidValue;
  const int pair_heads = (p.group % 2 == 0) ? 1 : 0;
  static thread_local PrefillWork work;  // 16 KB: kept off the stack
  int upper = 0;
  cudaError_t e = prefill_work_list(&work, &upper, p, max_query_len, -1, seq_lens_host,
                                    query_start_loc_host, pair_heads, stream);
  if (e != cudaSuccess) return e;
  const int smem = Layout<D>::total;
  static std::atomic<int> smem_done[64], split_smem_done[64];
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(max(1, min(min(device_sm_count(), max_ctas), upper)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  // items: those of the list, or what the step's sizes allow
  const int64_t most = min((int64_t)p.num_seqs * ((max_query_len + QT - 1) / QT),
                           (int64_t)p.num_tokens / QT + p.num_seqs) *
                       (pair_heads ? p.num_q_heads / 2 : p.num_q_heads);
  const int64_t items = work.count > 0 ? work.count : most;
  const int tiles = work.count > 0 ? work.items[0].w : (p.max_seq_len + KT - 1) / KT;
  const int ctas = prefill_fp4_cluster((double)items, tiles, max_ctas);
  if (ctas > 1) {
    auto kernel = prefill_fp4_kernel<D, true>;
    e = raise_smem_limit(kernel, smem, split_smem_done);
    if (e != cudaSuccess) return e;
    cfg.gridDim = dim3((unsigned)(items * ctas));
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, kernel, p, v_scale, tq, pair_heads, work);
  }
  auto kernel = prefill_fp4_kernel<D, false>;
  e = raise_smem_limit(kernel, smem, smem_done);
  if (e != cudaSuccess) return e;
  return cudaLaunchKernelEx(&cfg, kernel, p, v_scale, tq, pair_heads, work);
}

}  // namespace

// Clusters of n CTAs that the device holds at once, asked for once per device (74
// of two, 33 of four, 15 of eight at 148 SMs); 0 if it does not say
static int resident_clusters(int n) {
  static std::atomic<int> known[64][kMaxCluster + 1];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
  int held = known[dev][n].load(std::memory_order_relaxed);
  if (held == 0) {
    static std::atomic<int> smem_done[64];
    auto kernel = prefill_fp4_kernel<128, true>;
    if (raise_smem_limit(kernel, Layout<128>::total, smem_done) != cudaSuccess) return 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = n;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(n);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<128>::total;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaOccupancyMaxActiveClusters(&held, kernel, &cfg) != cudaSuccess) return 0;
    known[dev][n].store(held, std::memory_order_relaxed);
  }
  return held;
}

int prefill_fp4_cluster(double items, double tiles, int sms) {
  int best = 1;
  if (sms < device_sm_count() || 2 * items > sms) return best;  // beside the decode kernel; full
  double best_cost = tiles;
  for (int n = 2; n <= kMaxCluster && items * n <= sms; ++n) {
    const double cost = ceil(tiles / n) + kPrefillJoinTiles;
    if (cost < best_cost && items <= resident_clusters(n)) {
      best_cost = cost;
      best = n;
    }
  }
  return best;
}

cudaError_t launch_prefill_fp4(const AttnParams& p, float v_scale, int head_dim,
                               int max_query_len, const int32_t* seq_lens_host,
                               const int32_t* query_start_loc_host, cudaStream_t stream,
                               int max_ctas) {
  cudaError_t e = head_dim == 64
                      ? launch_d<64>(p, v_scale, max_query_len, seq_lens_host,
                                     query_start_loc_host, stream, max_ctas)
                      : launch_d<128>(p, v_scale, max_query_len, seq_lens_host,
                                      query_start_loc_host, stream, max_ctas);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace pa
