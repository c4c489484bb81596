// decode_fp4.cu -- paged attention over the 4-bit cache for few query rows per
// kv-head, bound by the cache's bytes.
//
// Page "LLM推論エンジンvLLMの内部構造を徹底解説", section "エンジンの中核": a decode
// runs the newest token against the cache and is bound by memory bandwidth;
// section "PagedAttentionの仕組み": the keys are read block by block through the
// sequence's block table.
//
//   o = sum_j softmax_j(scale q . k_j) v_j,  k_j = code_j * scale_j (pa_fp4.cuh)
//
// Work.  A unit is one (sequence, kv-head, group of R = 8 or 16 query rows).
// The blocks of all units in order form one line; the CTAs (one per SM) take
// equal stretches of it, and the warps of a CTA equal stretches of the CTA's.
// Every CTA derives the line from the device's own lengths (a block-wide scan),
// so nothing depends on host copies and a captured call follows the lengths at
// its replay.  A warp that holds a whole unit writes its output; parts of a
// unit in several warps are joined in shared memory, parts in several CTAs in
// the workspace by the CTA that arrives last.  The parts and their order depend
// on the lengths alone, so equal calls give equal bits.
//
// A warp streams its blocks' tiles (2304 or 1152 contiguous bytes) by bulk
// copies through a ring of its own, one mbarrier per stage, and runs ahead of
// its arithmetic over unit ends.  Per tile, with keys and value dims on the
// MMA's M side and query rows on its N side (mma.sync m16n8k16, f16 -> fp32):
//   S^T = K Q^T   codes converted to f16 and scaled, exact (six bits)
//   online softmax in fp32, exp2 domain; the running max moves only when a
//                 score passes it by 2^8
//   O^T += V^T P^T  P in f16, 2^7 times itself so that its small values keep
//                 their bits (at most 2^15), transposed in registers
// The query goes in as f16 too, each row times a power of two that brings its
// largest value into [1, 2): bf16's eight bits fit (of values under 2^-14 of the
// largest, those above 2^-25 of it); fp32 queries and their probabilities are split
// into two f16 terms each, 22 bits in all.
//
// Bound: the cache's bytes and the instructions that convert them, together.  192
// contexts of 256 .. 8192 tokens (32 + 8 heads of 128, 917 MB): 167.5 us, 84 % of
// the copy rate, issue slots 56 %, in a short burst; 188 us, 75 %, in a long loop,
// where the power limit holds the SM clock down; 8 of 32768 .. 131072 (855 MB): 152
// and 174 us, 86 and 75 %.  At D = 64 a byte takes 1.33 times the instructions: 256 of
// 8192 (604 MB) 132 and 141 us, 70 and 65 %.  With 16 rows 246 registers leave 8 warps
// at D = 128: 256 of 16384 on one kv-head (604 MB) 162 and 165 us, 57 %; at D = 64, 512
// of them 190 us, 49 %.  Few short contexts are bound by the chain of dependent reads
// (lengths, block ids, tiles, parts): one of 77 tokens 7.2 us, 64 of 128 .. 2048 at
// D = 64 14.5 us.
#include <float.h>
#include <math.h>

#include "pa_fastmath.cuh"
#include "pa_fp4.cuh"
#include "pa_wait.cuh"

namespace pa {
namespace {

constexpr float kRescale = 8.f;   // log2 units: the running max moves only past 2^8
constexpr float kPShift = 7.f;    // P is held times 2^7

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::
          "r"(dst), "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}
__device__ __forceinline__ uint32_t bits(__half2 h) { return *reinterpret_cast<uint32_t*>(&h); }
// 2^e, -126 <= e <= 127
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }
// the eight codes of a word as f16 pairs, times s
__device__ __forceinline__ void deq8(uint32_t w, __half2 s, uint32_t (&d)[4]) {
  __half2 x[4];
  e2m1x8_to_half2(w, x);
#pragma unroll
  for (int i = 0; i < 4; ++i) d[i] = bits(__hmul2(x[i], s));
}

// shape of one kernel
template <int D_, int NT_, int QP_>
struct Shape {
  static constexpr int D = D_, NT = NT_, QP = QP_;
  static constexpr int R = 8 * NT;                 // query rows of a unit
  static constexpr int kWarps = D * NT * QP <= 64 ? 16 : D * NT * QP <= 128 ? 12 : 8;
  static constexpr int kTile = Fp4Tile<D>::bytes;
  static constexpr int kPart = R * D * 4;          // one partial O
  // stages of one warp's ring, two tiles each: what the shared memory beside
  // the parts holds
  static constexpr int kStages = (211 * 1024 / kWarps - kPart) / (2 * kTile);
  static constexpr int kRing = kStages * 2 * kTile;
  static constexpr int kSteps = D / 16;            // MMA k-steps of S, M-tiles of O
  static constexpr int kChunkK = D / 4;            // dims of a lane's K chunk
  static constexpr int ring_off = 0;
  static constexpr int part_off = ring_off + kWarps * kRing;  // first parts
  static constexpr int total = part_off + kWarps * kPart;
  // Units up to this many blocks are not cut between CTAs: joining a cut unit
  // costs its CTA two more round trips to memory (3 to 5 us, by its rows), the
  // unequal stretches at most this many blocks over the warps of a CTA.  64
  // contexts of 128 .. 2048 at D = 64, 8 rows: 14.2 us, with half of it 16.0, with
  // half as much again 14.1; 33 of 40 .. 3060 with up to 13 drafted tokens, 16 rows:
  // 16.4, 18.6 and 16.4.  Around it: 64 of 128 blocks each 14.7 us (half 19.3, more
  // 14.7), of 129 blocks 18.9 (18.8, 15.2); 33 of 193 blocks, 16 rows, 22.2 (22.2,
  // 16.9); 30 of 96 and of 97 blocks on 8 kv-heads at D = 128 16.9 and 21.0 (20.5 and
  // 21.0, 16.9 and 17.5).
  static constexpr int kWhole = R * kWarps;
  // Parts of a unit that one CTA joins at once; of more, groups of so many first.
  // Two steps cost 2 to 4 us more than one of as many parts as that: four
  // contexts of 7236 .. 28944 at D = 64, 30 parts, 16.0 us, 21.1 in two steps.
  static constexpr int kJoin = 32, kGroup = 12;
  static_assert(kFp4MaxCtas <= 32 * kGroup && kJoin <= 32, "a lane per part");
  static_assert(kRing * kWarps >= R * 33 * 4, "the weights of a join");
  static_assert(kStages >= 3 && kRing >= kPart, "a warp's last part takes its ring's place");
};

// where a part of a unit belongs
struct PartMeta {
  int unit_start, nblk;       // of the unit, on the line of blocks
  int q0, head, row0, nrows;  // the unit's first query row of the kv-head, and its rows
  int valid, ended;           // holds a part; the part reaches the unit's end
};

// a sequence as the kernel sees it: its units' blocks on the line
struct Seq {
  int q0, ql, L, nblk, rgs;
};
// The parts of one unit that this CTA joins
struct Run {
  unsigned mine;         // the warps whose first parts belong to it
  int w0;                // the warp whose last part starts the unit (or, of a unit that
                         // starts in an earlier CTA, whose first part is the first here)
  int before, complete;  // starts in an earlier CTA; starts and ends here
};

// A join under way: the CTA of its first part, CTAs from one part to the next, and
// their number; whether the unit starts with it, and is whole after it
struct Join {
  int first, apart, n, starts, whole;
};

template <typename S>
struct Shared {
  unsigned long long bars[S::kWarps * S::kStages];
  PartMeta meta[S::kWarps][2];
  float ml[S::kWarps][2][S::R][2];
  // of the sequences under way: q0, ql, L (as read), and their blocks on the
  // line summed over the warp that read them
  int4 seqs[S::kWarps * 32];
  Run runs[S::kWarps + 1];
  int cut[2];  // this CTA's stretch
  int abort;
  Join join[2];
  int last[2];  // this CTA arrived last at its first, its last unit
};

template <int R>
__device__ __forceinline__ Seq make_seq(const Fp4AttnParams& p, int q0, int ql, int L) {
  const bool mine = ql > 0 && ql <= L && L <= p.max_seq_len && ql <= p.max_q;
  return Seq{q0, ql, L, mine ? (L + kBlockSize - 1) / kBlockSize : 0,
             mine ? (ql * p.group + R - 1) / R : 0};
}
template <int R>
__device__ __forceinline__ Seq load_seq(const Fp4AttnParams& p, int s) {
  const int q0 = p.query_start_loc[s];
  return make_seq<R>(p, q0, p.query_start_loc[s + 1] - q0, p.seq_lens[s]);
}

// a / b for 0 <= a, 0 < b.  The first quotient is off by at most 2^31 * 2^-22, and
// by one where a < 2^22; a second step brings the others there.
__device__ __forceinline__ int divide(int a, int b) {
  const float inv = __fdividef(1.f, (float)b);
  int q = (int)((float)a * inv);
  int r = a - q * b;
  if (a >= 1 << 22) {
    const int more = (int)((float)r * inv);
    q += more;
    r -= more * b;
  }
  return q + (r >= b) - (r < 0);
}
// query token of a row of a kv-head: row / group
__device__ __forceinline__ int token_of(const Fp4AttnParams& p, int row) {
  return p.group_inv ? (int)__umulhi((unsigned)row, p.group_inv) : row;
}

// A position on the line, walked block by block over units and sequences.
template <int R>
struct Cursor {
  int s;            // sequence
  Seq q;
  int head, rg, blk;
  int unit_start;
  // at position `pos` of the line, in sequence seq whose first unit starts at pre
  __device__ __forceinline__ void begin(const Seq& sq, int seq, int pre, int pos) {
    s = seq;
    q = sq;
    const int o = pos - pre;
    const int u = divide(o, q.nblk);
    blk = o - u * q.nblk;
    head = q.rgs == 1 ? u : divide(u, q.rgs);
    rg = u - head * q.rgs;
    unit_start = pos - blk;
  }
  // the next unit (only called while blocks of this line remain)
  __device__ __forceinline__ void next_unit(const Fp4AttnParams& p) {
    unit_start += q.nblk;
    blk = 0;
    if (++rg < q.rgs) return;
    rg = 0;
    if (++head < p.num_kv_heads) return;
    head = 0;
    const int lane = threadIdx.x & 31;
    int at = s + 1;
    while (at < p.num_seqs) {
      const int mine = at + lane;
      const Seq c = mine < p.num_seqs ? load_seq<R>(p, mine) : Seq{0, 0, 0, 0, 0};
      const unsigned any = __ballot_sync(0xffffffffu, c.nblk > 0);
      if (any) {
        const int from = __ffs(any) - 1;
        s = at + from;
        q.q0 = __shfl_sync(0xffffffffu, c.q0, from);
        q.ql = __shfl_sync(0xffffffffu, c.ql, from);
        q.L = __shfl_sync(0xffffffffu, c.L, from);
        q.nblk = __shfl_sync(0xffffffffu, c.nblk, from);
        q.rgs = __shfl_sync(0xffffffffu, c.rgs, from);
        return;
      }
      at += 32;
    }
  }
};

template <typename T>
__device__ __forceinline__ void store_dims(T* dst, const float* x);
template <>
__device__ __forceinline__ void store_dims<float>(float* dst, const float* x) {
  *(float4*)dst = make_float4(x[0], x[1], x[2], x[3]);
}
template <>
__device__ __forceinline__ void store_dims<__nv_bfloat16>(__nv_bfloat16* dst, const float* x) {
  __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *(uint2*)dst = make_uint2(*(uint32_t*)&a, *(uint32_t*)&b);
}
template <typename T, int N>
__device__ __forceinline__ void store_row(T* dst, const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; i += 4) store_dims<T>(dst + i, x + i);
}

template <typename S, typename T>
__global__ void __launch_bounds__(S::kWarps * 32, 1) decode_fp4_kernel(const Fp4AttnParams p) {
  constexpr int D = S::D, NT = S::NT, QP = S::QP, R = S::R, W = S::kWarps, K = S::kSteps;
  using Tile = Fp4Tile<D>;
  extern __shared__ __align__(1024) unsigned char smem[];
  __shared__ Shared<S> sh;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int g = lane >> 2, t = lane & 3;
  volatile int* abort_flag = &sh.abort;

  if (threadIdx.x == 0) sh.abort = 0;
  if (threadIdx.x < W) sh.meta[threadIdx.x][0].valid = sh.meta[threadIdx.x][1].valid = 0;
  for (int i = threadIdx.x; i < W * S::kStages; i += W * 32)
    mbar_init((uint32_t)__cvta_generic_to_shared(&sh.bars[i]), 1);
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---- the line of blocks (under 2^31 of them, which the host checks): its
  // length, this CTA's stretch of it and this warp's stretch of that, one step
  // each.  Up to W * 32 sequences stay in shared memory between the steps; more
  // are gone over again in each.  What one warp can find out, one warp does:
  // four warps share a scheduler, and all would wait for all of them.
  const bool resident = p.num_seqs <= W * 32;
  int per = 0, cta0 = 0, cta1 = 0;
  auto warp_start = [&](int w) { return cta0 + (int)((unsigned)(cta1 - cta0) * w / W); };
  Cursor<R> cu{};  // the arithmetic's
  int upto = 0, from = 0;   // lane w: where warp w's sequences end and start on the line
  int cost = 0, start = 0;  // of this thread's sequence: its blocks, and where they start
#pragma unroll 1
  for (int step = 0; step < 3; ++step) {
    int base = 0;
#pragma unroll 1
    for (int s0 = 0; s0 < p.num_seqs; s0 += W * 32) {
      if (step == 0 || !resident) {
        const int s = s0 + threadIdx.x;
        const Seq sq = s < p.num_seqs ? load_seq<R>(p, s) : Seq{};
        cost = sq.nblk * sq.rgs * p.num_kv_heads;
        int sum = cost;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, sum, o);
          if (lane >= o) sum += y;
        }
        if (s0 > 0 || step > 0) __syncthreads();  // the ones before have been searched
        sh.seqs[threadIdx.x] = make_int4(sq.q0, sq.ql, sq.L, sum);
        __syncthreads();
        const int own = lane < W ? sh.seqs[lane * 32 + 31].w : 0;
        upto = own;
#pragma unroll
        for (int o = 1; o < W; o <<= 1) {
          const int y = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += y;
        }
        upto += base;
        from = upto - own;
        start = __shfl_sync(0xffffffffu, from, warp) + sum - cost;
      }
      const int end = __shfl_sync(0xffffffffu, upto, W - 1);
      // the sequence (of those in shared memory) that holds position `at`, and
      // where it starts
      auto find = [&](int at, Seq* sq, int* pre) {
        const int w = __ffs(__ballot_sync(0xffffffffu, upto > at)) - 1;
        const int before = __shfl_sync(0xffffffffu, from, w);
        const int mine = sh.seqs[w * 32 + lane].w + before;
        const int i = w * 32 + __ffs(__ballot_sync(0xffffffffu, mine > at)) - 1;
        const int4 q = sh.seqs[i];
        *sq = make_seq<R>(p, q.x, q.y, q.z);
        *pre = q.w + before - sq->nblk * sq->rgs * p.num_kv_heads;
        return i;
      };
      if (step == 1) {  // by the thread whose sequence holds the end of a stretch:
        // moved to one of a short unit
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          const unsigned in = (blockIdx.x + i) * (unsigned)per - start;
          if (in >= (unsigned)cost) continue;
          const int nblk = (sh.seqs[threadIdx.x].z + kBlockSize - 1) / kBlockSize;
          const int r = (int)in - divide((int)in, nblk) * nblk;
          sh.cut[i] = start + (int)in + (nblk > S::kWhole ? 0 : 2 * r < nblk ? -r : nblk - r);
        }
      }
      if (step == 2) {
        const int at = warp_start(warp);
        if (at >= base && at < end) {
          Seq sq;
          int pre;
          const int s = s0 + find(at, &sq, &pre);
          cu.begin(sq, s, pre, at);
        }
      }
      base = end;
    }
    if (step == 0) {
      // at least a block per warp: fewer CTAs take a short line
      per = max(divide(base + (int)gridDim.x - 1, (int)gridDim.x), W);
      if ((long long)blockIdx.x * per >= base) return;
      if (threadIdx.x < 2) sh.cut[threadIdx.x] = base;
      __syncthreads();
    }
    if (step == 1) {
      __syncthreads();
      cta0 = sh.cut[0];
      cta1 = sh.cut[1];
      if (cta0 >= cta1) return;
    }
  }

  const int pos0 = warp_start(warp), pos1 = warp_start(warp + 1);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem + S::ring_off) + warp * S::kRing;
  const uint32_t bars = (uint32_t)__cvta_generic_to_shared(&sh.bars[warp * S::kStages]);
  bool ok = true;

  if (pos1 > pos0) {
    // ---- loads: in pairs of blocks of one unit (the last of an odd number
    // alone), a ring ahead of the arithmetic and with a cursor of their own.
    // Lane i holds the tiles of the i-th pair of a window of 32, and the block
    // ids of the window after it, on their way from the block table.
    Cursor<R> ld = cu;
    int ahead = pos1 - pos0;            // blocks not yet in a window
    int left = 0;                       // pairs of this window not yet issued
    int at_lane = 0, put = 0;           // the next one, and its stage
    int tile0 = 0, tile1 = 0;           // (second tile -1: none)
    int next0 = 0, next1 = 0, next_head = 0, next_pairs = 0;
    auto clamp_id = [&](int id) { return min(max(id, 0), p.num_blocks - 1); };  // never outside the pool
    auto look_ahead = [&]() {
      int n = 0, blk = -1, seq = 0;
      bool both = false;
      while (n < 32 && ahead > 0) {
        const int here = min(ld.q.nblk - ld.blk, ahead);      // blocks of this unit
        const int pairs = min((here + 1) / 2, 32 - n);
        if (lane >= n && lane < n + pairs) {
          blk = ld.blk + 2 * (lane - n);
          both = 2 * (lane - n) + 1 < here;
          seq = ld.s;
          next_head = ld.head;
        }
        n += pairs;
        const int took = min(2 * pairs, here);
        ahead -= took;
        ld.blk += took;
        if (ld.blk == ld.q.nblk && ahead > 0) ld.next_unit(p);
      }
      next_pairs = n;
      const int32_t* ids = p.block_tables + (int64_t)seq * p.max_blocks_per_seq;
      next0 = blk >= 0 ? ids[blk] : 0;
      next1 = both ? ids[blk + 1] : INT32_MIN;
    };
    auto install = [&]() {
      left = next_pairs;
      at_lane = 0;
      tile0 = clamp_id(next0) * p.num_kv_heads + next_head;
      tile1 = next1 == INT32_MIN ? -1 : clamp_id(next1) * p.num_kv_heads + next_head;
      next_pairs = 0;
    };
    auto issue = [&]() {  // the next pair of the window
      if (lane == at_lane) {
        const uint32_t bar = bars + 8 * put, dst = ring + put * 2 * S::kTile;
        mbar_expect_tx(bar, tile1 < 0 ? S::kTile : 2 * S::kTile);
        bulk_load(dst, p.kv_cache + (int64_t)tile0 * S::kTile, S::kTile, bar);
        if (tile1 >= 0)
          bulk_load(dst + S::kTile, p.kv_cache + (int64_t)tile1 * S::kTile, S::kTile, bar);
      }
      ++at_lane;
      --left;
      put = put + 1 == S::kStages ? 0 : put + 1;
    };

    // ---- the units of this stretch
    int pos = pos0;
    int at = 0, phase = 0;  // stage of the next block, and its barrier's parity
    bool first = true;
    while (pos < pos1 && ok) {
      const int blk0 = cu.blk;
      const int nb = min(cu.q.nblk - blk0, pos1 - pos);
      const int nrows = min(R, cu.q.ql * p.group - cu.rg * R);
      // -- the query rows (the B operand): row g (+8), this lane's chunk of dims
      constexpr int kVecs = S::kChunkK * (int)sizeof(T) / 16;
      uint4 raw[NT][kVecs];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = n * 8 + g;
        const int rr = cu.rg * R + row, j = token_of(p, rr);
        const T* src = (const T*)p.q +
                       ((int64_t)(cu.q.q0 + j) * p.num_q_heads + cu.head * p.group +
                        (rr - j * p.group)) * D +
                       t * S::kChunkK;
#pragma unroll
        for (int i = 0; i < kVecs; ++i)
          raw[n][i] = row < nrows ? ((const uint4*)src)[i] : make_uint4(0, 0, 0, 0);
      }
      if (first) {  // the first tiles' loads leave while the query's are under way
        look_ahead();
        install();
#pragma unroll 1
        for (int i = 0; i < S::kStages && left > 0; ++i) issue();
        if (ahead > 0) look_ahead();
        first = false;
      }
      uint32_t qf[QP][NT][K][2];
      float sl2[NT][2];  // log2(e) scale of the scores of rows 2t, 2t+1 (+8)
      int lim[NT][2];    // their last visible key
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        float x[S::kChunkK];
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
          const uint32_t u[4] = {raw[n][i].x, raw[n][i].y, raw[n][i].z, raw[n][i].w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (sizeof(T) == 2) {
              x[8 * i + 2 * k] = __uint_as_float(u[k] << 16);
              x[8 * i + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
            } else {
              x[4 * i + k] = __uint_as_float(u[k]);
            }
          }
        }
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < S::kChunkK; ++i) mx = fmaxf(mx, fabsf(x[i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the exponent of the row's largest value, as far as 2^-e is a normal
        // number (beyond: nearly so; infinities and NaN stay what they are)
        const int e = min(max((__float_as_int(mx) >> 23) - 127, -126), 126);
        const float f = exp2i(-e);
#pragma unroll
        for (int i = 0; i < S::kChunkK; ++i) x[i] *= f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float a = x[4 * k + 2 * h], b = x[4 * k + 2 * h + 1];
            const __half2 hi = __floats2half2_rn(a, b);
            qf[0][n][k][h] = bits(hi);
            if constexpr (QP == 2)
              qf[QP - 1][n][k][h] =
                  bits(__floats2half2_rn(a - __low2float(hi), b - __high2float(hi)));
          }
        }
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int er = __shfl_sync(0xffffffffu, e, (2 * t + c) * 4);
          // (a scale below the smallest normal number would make NaN of a masked score)
          sl2[n][c] = fmaxf(p.scale_log2 * exp2i(er), FLT_MIN);
          const int r2 = cu.rg * R + n * 8 + 2 * t + c;
          lim[n][c] = n * 8 + 2 * t + c < nrows ? cu.q.L - cu.q.ql + token_of(p, r2) : cu.q.L - 1;
        }
      }

      float o[NT][K][4];
      float m[NT][2], l[NT][2], base[NT][2];  // (base: what an exponent adds, 7 - m)
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[n][i][c] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = base[n][0] = base[n][1] = 0.f;
      }

      // -- two blocks at a time (the second of the last pair may be none: its
      // scores are all masked, and its V counts as 0)
      const int ta = 4 * (g >> 1) + (g & 1);  // K rows: tokens ta, ta + 2; V: 4t .. 4t + 3
      for (int b = 0; b < nb; b += 2) {
        const int two = nb - b == 1 ? 1 : 2;
        uint32_t kw[2][2][K / 2], vw[2][2][K / 2], ks[2][2], vs[2];
        if (!__all_sync(0xffffffffu, mbar_try_wait(bars + 8 * at, phase))) {
          ok = wait_bar(bars + 8 * at, phase, abort_flag, p.ws_status);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
        const unsigned char* stage = smem + S::ring_off + warp * S::kRing + at * 2 * S::kTile;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const unsigned char* tile = stage + i * S::kTile;
          if constexpr (D == 128) {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint4 a = *(const uint4*)(tile + (ta + 2 * h) * 64 + t * 16);
              kw[i][h][0] = a.x; kw[i][h][1] = a.y; kw[i][h][2] = a.z; kw[i][h][3] = a.w;
              const uint4 v = *(const uint4*)(tile + Tile::v_off + h * 512 + lane * 16);
              vw[i][h][0] = v.x; vw[i][h][1] = v.y; vw[i][h][2] = v.z; vw[i][h][3] = v.w;
              ks[i][h] = *(const uint16_t*)(tile + Tile::ks_off + (ta + 2 * h) * 8 + 2 * t);
            }
            vs[i] = *(const uint32_t*)(tile + Tile::vs_off + g * 16 + 4 * t);
          } else {
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint2 a = *(const uint2*)(tile + (ta + 2 * h) * 32 + t * 8);
              kw[i][h][0] = a.x; kw[i][h][1] = a.y;
              const uint2 v = *(const uint2*)(tile + Tile::v_off + h * 256 + lane * 8);
              vw[i][h][0] = v.x; vw[i][h][1] = v.y;
              ks[i][h] = *(tile + Tile::ks_off + (ta + 2 * h) * 4 + t);
            }
            vs[i] = *(const uint32_t*)(tile + Tile::vs_off + (g >> 1) * 16 + 4 * t);
          }
        }
        if (++at == S::kStages) {
          at = 0;
          phase ^= 1;
        }
        __syncwarp();  // the stage is free once every lane holds its part of it
        if (left == 0 && next_pairs > 0) {
          install();
          if (ahead > 0) look_ahead();
        }
        if (left > 0) issue();

        // -- S^T = K Q^T (one chain of MMAs per block and row tile: a second
        // costs its sums, 138.8 against 132.2 us for 256 contexts of 8192 at D 64)
        float x[2][NT][4];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) x[i][n][c] = 0.f;
          __half2 k2[2][2];  // [token][group of the chunk]
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __half2 pair = e4m3x2_to_half2(ks[i][h]);
            k2[h][0] = __low2half2(pair);
            k2[h][1] = __high2half2(pair);
          }
#pragma unroll
          for (int w = 0; w < K / 2; ++w) {
            const int grp = D == 128 ? w / 2 : 0;
            uint32_t a[2][4];
            deq8(kw[i][0][w], k2[0][grp], a[0]);
            deq8(kw[i][1][w], k2[1][grp], a[1]);
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int qp = 0; qp < QP; ++qp)
                  mma_f16(x[i][n], a[0][2 * j], a[1][2 * j], a[0][2 * j + 1], a[1][2 * j + 1],
                          qf[qp][n][2 * w + j][0], qf[qp][n][2 * w + j][1]);
          }
        }
        // -- keys past a row's last visible one are out
        const int key0 = (blk0 + b) * kBlockSize;
        if (key0 + 2 * kBlockSize > cu.q.L - cu.q.ql + 1 || two == 1) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int key = i < two ? key0 + i * kBlockSize : INT32_MAX - 64;
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int c = 0; c < 4; ++c)
                if (key + ta + (c & 2) > lim[n][c & 1]) x[i][n][c] = -INFINITY;
            // V of slots that hold no token: whatever they hold counts as 0
            const int held = cu.q.L - key - 4 * t;
            if (held < 4) vs[i] = held <= 0 ? 0u : vs[i] & (0xffffffffu >> (32 - 8 * held));
          }
        }
        // -- the running max (in log2 units) moves when a score passes it by 2^8
        float mx[NT][2];
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            mx[n][c] = sl2[n][c] * fmaxf(max3(x[0][n][c], x[0][n][c + 2], x[1][n][c]), x[1][n][c + 2]);
            // (a max of -inf is passed by every score but -inf)
            over |= mx[n][c] > m[n][c] + kRescale;
          }
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float v = mx[n][c];
#pragma unroll
              for (int s = 4; s < 32; s <<= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, s));
              if (v > m[n][c] + kRescale) {
                const float f = ex2(m[n][c] - v);
                m[n][c] = v;
                base[n][c] = kPShift - v;
                l[n][c] *= f;
#pragma unroll
                for (int i = 0; i < K; ++i) {
                  o[n][i][c] *= f;
                  o[n][i][c + 2] *= f;
                }
              }
            }
        }
        // -- P^T in f16
        uint32_t pf[2][QP][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float e[4];
            const uint64_t sc2 = f2(sl2[n][0], sl2[n][1]), ba2 = f2(base[n][0], base[n][1]);
            f2_split(fma2(f2(x[i][n][0], x[i][n][1]), sc2, ba2), e[0], e[1]);
            f2_split(fma2(f2(x[i][n][2], x[i][n][3]), sc2, ba2), e[2], e[3]);
#pragma unroll
            for (int c = 0; c < 4; ++c) e[c] = ex2(e[c]);
            f2_split(add2(f2(l[n][0], l[n][1]), add2(f2(e[0], e[1]), f2(e[2], e[3]))), l[n][0],
                     l[n][1]);
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const __half2 hi = __floats2half2_rn(e[2 * h], e[2 * h + 1]);
              pf[i][0][n][h] = transpose8(bits(hi));
              if constexpr (QP == 2)
                pf[i][QP - 1][n][h] = transpose8(bits(__floats2half2_rn(
                    e[2 * h] - __low2float(hi), e[2 * h + 1] - __high2float(hi))));
            }
          }
        }
        // -- O^T += V^T P^T: the codes of a pair of tokens side by side in a
        // byte (even dims, odd dims), converted and scaled
        constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const __half2 v2[2] = {e4m3x2_to_half2(vs[i] & 0xffffu), e4m3x2_to_half2(vs[i] >> 16)};
#pragma unroll
          for (int w = 0; w < K / 4; ++w) {
            uint32_t ev[2][4], od[2][4];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t a = vw[i][h][w], c = vw[i][h][K / 4 + w];
              deq8((a & kLow) | ((c << 4) & ~kLow), v2[h], ev[h]);
              deq8(((a >> 4) & kLow) | (c & ~kLow), v2[h], od[h]);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int n = 0; n < NT; ++n)
#pragma unroll
                for (int qp = 0; qp < QP; ++qp)
                  mma_f16(o[n][4 * w + k], ev[0][k], od[0][k], ev[1][k], od[1][k],
                          pf[i][qp][n][0], pf[i][qp][n][1]);
          }
        }
      }
      if (!ok) break;

      // ---- the stretch's part of this unit
      const bool whole = nb == cu.q.nblk;
      const int slot = blk0 != 0 ? 0 : 1;
      pos += nb;
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          float sum = l[n][c];
#pragma unroll
          for (int s = 4; s < 32; s <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
          const int row = n * 8 + 2 * t + c;
          if (row >= nrows) continue;
          float y[2 * K];
          const float f = whole ? p.v_scale / sum : 1.f;
#pragma unroll
          for (int i = 0; i < K; ++i) {
            y[2 * i] = o[n][i][c] * f;
            y[2 * i + 1] = o[n][i][c + 2] * f;
          }
          if (whole) {
            const int rr = cu.rg * R + row, j = token_of(p, rr);
            store_row((T*)p.out +
                          ((int64_t)(cu.q.q0 + j) * p.num_q_heads + cu.head * p.group +
                           (rr - j * p.group)) * D +
                          g * (D / 8),
                      y);
          } else {
            // the last part takes the place of the ring, which is drained
            float* part = (float*)(slot == 0 ? smem + S::part_off + warp * S::kPart
                                             : smem + S::ring_off + warp * S::kRing);
            store_row(part + row * D + g * (D / 8), y);
            if (g == 0) {
              sh.ml[warp][slot][row][0] = m[n][c];
              sh.ml[warp][slot][row][1] = sum;
            }
          }
        }
      if (!whole && lane == 0) {
        PartMeta& pm = sh.meta[warp][slot];
        pm.unit_start = cu.unit_start;
        pm.nblk = cu.q.nblk;
        pm.q0 = cu.q.q0;
        pm.head = cu.head;
        pm.row0 = cu.rg * R;
        pm.nrows = nrows;
        pm.ended = blk0 + nb == cu.q.nblk;
        pm.valid = 1;
      }
      if (pos < pos1) cu.next_unit(p);
    }
    if (!ok) {  // the stages from the one waited for on to the last one issued
      const uint64_t t0 = globaltimer();
      do {
        drain_bar(bars + 8 * at, phase, t0);
        if (++at == S::kStages) {
          at = 0;
          phase ^= 1;
        }
      } while (at != put);
    }
  }
  __syncthreads();
  if (sh.abort) return;

  // ---- join the parts.  A run: the parts of one unit here, in order: the last
  // part of the warp where it starts and first parts of the warps after it
  // (slot w), or only first parts, of a unit that starts in an earlier CTA
  // (slot W)
  const bool v0 = lane < W && sh.meta[lane < W ? lane : 0][0].valid;
  const bool v1 = lane < W && sh.meta[lane < W ? lane : 0][1].valid;
  const unsigned firsts = __ballot_sync(0xffffffffu, v0);
  const unsigned starts = __ballot_sync(0xffffffffu, v1);
  const unsigned ends = __ballot_sync(0xffffffffu, v0 && sh.meta[lane < W ? lane : 0][0].ended);
  // the first warp with a first part, if no unit starts in a warp before it
  const int lead = firsts ? __ffs(firsts) - 1 : 31;
  const bool carried = firsts && (starts & ((1u << lead) - 1)) == 0;
  const int nruns = __popc(starts) + carried;
  // a weight per run, row and part, written over the part's maximum
  for (int i = threadIdx.x; i < (W + 1) * R; i += W * 32) {
    const int slot = i / R, row = i % R;
    const bool before = slot == W;
    if (before ? !carried : !(starts >> slot & 1)) continue;
    const int w0 = before ? lead : slot;
    unsigned mine = firsts & (~0u << (before ? w0 : w0 + 1));
    const unsigned end = ends & mine;
    if (end) mine &= (end & -end) | ((end & -end) - 1);
    const bool complete = end && !before;
    if (row == 0)
      sh.runs[before ? 0 : __popc(starts & ((1u << slot) - 1)) + carried] =
          Run{mine, w0, before, complete};
    if (row >= sh.meta[w0][before ? 0 : 1].nrows) continue;
    // without branches: the lanes' runs differ (what a place holds that is not of
    // the run is loaded and dropped)
    float* start = sh.ml[w0][1][row];
    float m[W + 1], sum = 0.f;
    // (a part whose scores are all NaN has no maximum and no weight, but its O is
    // NaN, and so is the sum with it)
    m[W] = before ? -INFINITY : start[0];
    float mx = m[W];
#pragma unroll
    for (int w = 0; w < W; ++w) {
      m[w] = mine >> w & 1 ? sh.ml[w][0][row][0] : -INFINITY;
      mx = fmaxf(mx, m[w]);
    }
#pragma unroll
    for (int w = 0; w <= W; ++w) {
      float* ml = w < W ? sh.ml[w % W][0][row] : start;
      const float wt = m[w] == -INFINITY ? 0.f : ex2(m[w] - mx);
      const float l = ml[1];
      sum += wt == 0.f ? 0.f : wt * l;
      if (w < W ? mine >> w & 1 : !before) ml[0] = wt;
    }
    if (complete) {
      start[1] = p.v_scale / sum;  // (its own sum has been read)
    } else {
      const int64_t at = (int64_t)(blockIdx.x * 2 + !before) * 16 + row;
      *(float2*)(p.ws_ml + at * 2) = make_float2(mx, sum);
    }
  }
  __syncthreads();
  // four dims of a row per thread
  constexpr int kQuads = D / 4;
  for (int i = threadIdx.x; i < nruns * R * kQuads; i += W * 32) {
    const Run run = sh.runs[i / (R * kQuads)];
    const PartMeta& pm = sh.meta[run.w0][run.before ? 0 : 1];
    const int row = i / kQuads % R, off = row * D + i % kQuads * 4;
    if (row >= pm.nrows) continue;
    const unsigned mine = run.mine;
    float y[4] = {0.f, 0.f, 0.f, 0.f};
    auto add = [&](float f, const float4& v) {
      y[0] = fmaf(f, v.x, y[0]);
      y[1] = fmaf(f, v.y, y[1]);
      y[2] = fmaf(f, v.z, y[2]);
      y[3] = fmaf(f, v.w, y[3]);
    };
    if (!run.before)
      add(sh.ml[run.w0][1][row][0],
          *(const float4*)((const float*)(smem + S::ring_off + run.w0 * S::kRing) + off));
#pragma unroll 1
    for (unsigned left = mine; left;) {  // four parts' loads together
      float4 v[4];
      float f[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int w = __ffs(left) - 1;
        left &= left - 1;
        f[e] = 0.f;
        v[e] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w >= 0) {
          f[e] = sh.ml[w][0][row][0];
          v[e] = *(const float4*)((const float*)(smem + S::part_off + w * S::kPart) + off);
        }
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) add(f[e], v[e]);
    }
    if (run.complete) {
      const float f = sh.ml[run.w0][1][row][1];
#pragma unroll
      for (int k = 0; k < 4; ++k) y[k] *= f;
      const int rr = pm.row0 + row, j = token_of(p, rr);
      store_dims<T>((T*)p.out + ((int64_t)(pm.q0 + j) * p.num_q_heads + pm.head * p.group +
                                 (rr - j * p.group)) * D + i % kQuads * 4,
                    y);
    } else {
      *(float4*)(p.ws_o + ((int64_t)(blockIdx.x * 2 + !run.before) * 16 * D + off)) =
          make_float4(y[0], y[1], y[2], y[3]);
    }
  }
  // the units that other CTAs hold parts of too: one from before this CTA, one
  // that goes on after it
  const Run& tail = sh.runs[max(nruns - 1, 0)];
  const bool pending[2] = {nruns > 0 && sh.runs[0].before, nruns > 0 && !tail.before && !tail.complete};
  if (!pending[0] && !pending[1]) return;

  // ---- a unit in several CTAs: the one that arrives last joins its parts, in
  // the order of the CTAs; of many parts, the last of each group of CTAs joins the
  // group's first, in the place of its first part.  (Two contexts of 8270 and 33083
  // on one kv-head, fp32, 148 parts: 16.8 us, 34.6 when one warp per row took them all.)
  unsigned open = (pending[0] ? 1u : 0u) | (pending[1] ? 2u : 0u);
  float* weight = (float*)(smem + S::ring_off);  // [row][part], of the join under way
  float* total = weight + R * 32;                // [row]: their maximum, and sum
#pragma unroll 1
  for (int level = 0; level < 2; ++level) {
    __syncthreads();
    if (threadIdx.x < 2) {
      int mine = 0;
      if (open >> threadIdx.x & 1) {
        // the unit's CTAs, and the parts that are joined at this level
        const PartMeta& f = threadIdx.x == 0 ? sh.meta[sh.runs[0].w0][0] : sh.meta[tail.w0][1];
        const int c0 = divide(f.unit_start, per);
        const int all = divide(f.unit_start + f.nblk - 1, per) - c0 + 1;
        const bool grouped = all > S::kJoin, whole = !grouped || level == 1;
        int first = c0, n = all;
        if (grouped) {
          n = (all + S::kGroup - 1) / S::kGroup;
          if (level == 0) {
            first += ((int)blockIdx.x - c0) / S::kGroup * S::kGroup;
            n = min(S::kGroup, c0 + all - first);
          }
        }
        int* counter = p.ws_counters + (whole ? c0 : kFp4MaxCtas + 2 * first + (first == c0));
        __threadfence();  // this CTA's parts, before its arrival
        mine = atomicAdd(counter, 1) == n - 1;
        __threadfence();  // and the others' after theirs
        if (mine) *counter = 0;  // every part has arrived: zero for the next call
        sh.join[threadIdx.x] = Join{first, grouped && whole ? S::kGroup : 1, n, first == c0, whole};
      }
      sh.last[threadIdx.x] = mine;
    }
    __syncthreads();
#pragma unroll 1
    for (int side = 0; side < 2; ++side) {
      if (!sh.last[side]) open &= ~(1u << side);
      if (!(open >> side & 1)) continue;
      const PartMeta& f = side == 0 ? sh.meta[sh.runs[0].w0][0] : sh.meta[tail.w0][1];
      const Join join = sh.join[side];
      const int n = join.n;
      const bool whole = join.whole;
      // rows of part i in the workspace (a unit's first part is its CTA's last)
      auto slot = [&](int i) {
        return ((join.first + i * join.apart) * 2 + (i == 0 && join.starts)) * 16;
      };
      // four dims of a row per thread; the first parts' loads leave while the
      // weights are made
      int i = threadIdx.x;
      const int quads = f.nrows * kQuads;
      constexpr int kBatch = 12;
      float4 v[kBatch];
      auto load = [&](int k) {
        const float4* src = (const float4*)p.ws_o + i;
#pragma unroll
        for (int e = 0; e < kBatch; ++e) v[e] = __ldcg(src + slot(min(k + e, n - 1)) * kQuads);
      };
      if (i < quads) load(0);
      constexpr int kTimes = (R + W - 1) / W;  // rows of a warp; a lane per part (at most 32)
      float2 mls[kTimes];
#pragma unroll
      for (int e = 0; e < kTimes; ++e)
        mls[e] = lane < n && warp + e * W < f.nrows
                     ? __ldcg((const float2*)(p.ws_ml + (slot(lane) + warp + e * W) * 2))
                     : make_float2(-INFINITY, 0.f);
      __syncthreads();  // the join before has read its weights
#pragma unroll
      for (int e = 0; e < kTimes; ++e) {
        const int row = warp + e * W;
        if (row >= f.nrows) break;
        const float2 ml = mls[e];
        float mx = ml.x;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
        const float wt = ml.x == -INFINITY ? 0.f : ex2(ml.x - mx);
        float sum = wt == 0.f ? 0.f : wt * ml.y;
#pragma unroll
        for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
        weight[row * 32 + lane] = wt;
        if (lane == 0) {
          total[row] = whole ? p.v_scale / sum : 1.f;
          if (!whole) *(float2*)(p.ws_ml + (slot(0) + row) * 2) = make_float2(mx, sum);
        }
      }
      __syncthreads();
#pragma unroll 1
      while (i < quads) {
        const int row = i / kQuads, off = row * D + i % kQuads * 4;
        float y[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
        for (int k = 0;;) {
#pragma unroll
          for (int e = 0; e < kBatch; ++e) {
            if (k + e >= n) break;
            const float w = weight[row * 32 + k + e];
            y[0] = fmaf(w, v[e].x, y[0]);
            y[1] = fmaf(w, v[e].y, y[1]);
            y[2] = fmaf(w, v[e].z, y[2]);
            y[3] = fmaf(w, v[e].w, y[3]);
          }
          k += kBatch;
          if (k >= n) break;
          load(k);
        }
        if (whole) {
          const float s = total[row];
#pragma unroll
          for (int k = 0; k < 4; ++k) y[k] *= s;
          const int rr = f.row0 + row, j = token_of(p, rr);
          store_dims<T>((T*)p.out + ((int64_t)(f.q0 + j) * p.num_q_heads + f.head * p.group +
                                     (rr - j * p.group)) * D + i % kQuads * 4,
                        y);
        } else {  // (only this thread reads these elements of the parts)
          *(float4*)(p.ws_o + slot(0) * D + off) = make_float4(y[0], y[1], y[2], y[3]);
        }
        i += W * 32;
        if (i < quads) load(0);
      }
      if (whole) open &= ~(1u << side);
    }
    if (!open) return;
  }
}

template <int D, int NT, int QP, typename T>
cudaError_t launch_shape(const Fp4AttnParams& p, cudaStream_t stream, int max_ctas) {
  using S = Shape<D, NT, QP>;
  auto kernel = decode_fp4_kernel<S, T>;
  static std::atomic<int> smem_done[64];
  cudaError_t e = raise_smem_limit(kernel, S::total, smem_done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(min(min(device_sm_count(), kFp4MaxCtas), max_ctas));
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = S::total;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_decode_fp4(const Fp4AttnParams& p, int head_dim, bool f32, int rows,
                              cudaStream_t stream, int max_ctas) {
  cudaError_t e;
  const bool wide = rows > 8;
  if (f32) {
    if (head_dim == 64)
      e = wide ? launch_shape<64, 2, 2, float>(p, stream, max_ctas) : launch_shape<64, 1, 2, float>(p, stream, max_ctas);
    else
      e = wide ? launch_shape<128, 2, 2, float>(p, stream, max_ctas)
               : launch_shape<128, 1, 2, float>(p, stream, max_ctas);
  } else {
    if (head_dim == 64)
      e = wide ? launch_shape<64, 2, 1, __nv_bfloat16>(p, stream, max_ctas)
               : launch_shape<64, 1, 1, __nv_bfloat16>(p, stream, max_ctas);
    else
      e = wide ? launch_shape<128, 2, 1, __nv_bfloat16>(p, stream, max_ctas)
               : launch_shape<128, 1, 1, __nv_bfloat16>(p, stream, max_ctas);
  }
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace pa
