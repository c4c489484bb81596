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
// largest value into [1, 2): bf16's eight bits fit; fp32 queries and their
// probabilities are split into two f16 terms each, 22 bits in all.
#include <math.h>

#include "pa_fastmath.cuh"
#include "pa_fp4.cuh"
#include "pa_wait.cuh"

namespace pa {
namespace {

constexpr float kRescale = 8.f;   // log2 units: the running max moves only past 2^8
constexpr float kPShift = 7.f;    // P is held times 2^7
constexpr int kMaxWarps = 16;

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
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
// code pair in byte I of w, as f16, times s
template <int I>
__device__ __forceinline__ uint32_t deq(uint32_t w, __half2 s) {
  return bits(__hmul2(e2m1x2_to_half2(w >> (8 * I) & 255u), s));
}

// shape of one kernel
template <int D_, int NT_, int QP_>
struct Shape {
  static constexpr int D = D_, NT = NT_, QP = QP_;
  static constexpr int R = 8 * NT;                 // query rows of a unit
  static constexpr bool kSmall = D * NT * QP <= 128;  // fits 128 registers a thread
  static constexpr int kWarps = kSmall ? 16 : 8;
  static constexpr int kTile = Fp4Tile<D>::bytes;
  static constexpr int kStages = (kSmall ? 4 : 8) * (128 / D);
  static constexpr int kRing = kStages * kTile;    // one warp's ring
  static constexpr int kPart = R * D * 4;          // one partial O
  static constexpr int kSteps = D / 16;            // MMA k-steps of S, M-tiles of O
  static constexpr int kChunkK = D / 4;            // dims of a lane's K chunk
  static constexpr int ring_off = 0;
  static constexpr int part_off = ring_off + kWarps * kRing;  // first parts
  static constexpr int total = part_off + kWarps * kPart;
  static_assert(kRing >= kPart, "a warp's last part takes its ring's place");
  static_assert(total <= 220 * 1024, "shared memory of one CTA");
};

// where a part of a unit belongs
struct PartMeta {
  long long unit_start;  // of the unit, on the line of blocks
  int nblk;
  int seq, head, rg;     // row group
  int valid, ended;      // holds a part; the part reaches the unit's end
};

template <typename S>
struct Shared {
  unsigned long long bars[S::kWarps * S::kStages];
  PartMeta meta[S::kWarps][2];
  float ml[S::kWarps][2][S::R][2];
  long long scan[kMaxWarps + 1];
  long long start_pre[kMaxWarps];
  int start_seq[kMaxWarps];
  int abort;
  int last[2];
};

// a sequence as the kernel sees it: its units' blocks on the line
struct Seq {
  int q0, ql, L, nblk, rgs;
};
template <int R>
__device__ __forceinline__ Seq load_seq(const Fp4AttnParams& p, int s) {
  Seq r;
  r.q0 = p.query_start_loc[s];
  r.ql = p.query_start_loc[s + 1] - r.q0;
  r.L = p.seq_lens[s];
  const long long rows = (long long)r.ql * p.group;
  const bool mine = r.ql > 0 && r.ql <= r.L && r.L <= p.max_seq_len && rows <= p.max_rows;
  r.nblk = mine ? (r.L + kBlockSize - 1) / kBlockSize : 0;
  r.rgs = mine ? (int)((rows + R - 1) / R) : 0;
  return r;
}
template <int R>
__device__ __forceinline__ long long seq_cost(const Fp4AttnParams& p, int s) {
  const Seq q = load_seq<R>(p, s);
  return (long long)q.nblk * q.rgs * p.num_kv_heads;
}

// inclusive block-wide sum of one value per thread; *total gets the whole sum
template <int kWarps>
__device__ __forceinline__ long long block_scan(long long x, long long* sh, long long* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) sh[warp] = x;
  __syncthreads();
  long long before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    const long long y = sh[w];
    if (w < warp) before += y;
    all += y;
  }
  *total = all;
  return x + before;
}

// A position on the line, walked block by block over units and sequences.
template <int R>
struct Cursor {
  int s;            // sequence
  Seq q;
  int head, rg, blk;
  long long unit_start;
  __device__ __forceinline__ void begin(const Fp4AttnParams& p, int seq, long long pre,
                                        long long pos) {
    s = seq;
    q = load_seq<R>(p, s);
    const long long o = pos - pre;
    const long long u = o / q.nblk;
    blk = (int)(o - u * q.nblk);
    head = (int)(u / q.rgs);
    rg = (int)(u - (long long)head * q.rgs);
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

  // ---- the line of blocks, and this CTA's and its warps' stretches of it
  long long total = 0;
  for (int s0 = 0; s0 < p.num_seqs; s0 += W * 32) {
    const int s = s0 + threadIdx.x;
    long long part;
    block_scan<W>(s < p.num_seqs ? seq_cost<R>(p, s) : 0, sh.scan, &part);
    total += part;
  }
  // at least a block per warp: fewer CTAs take a short line
  const long long per = max((total + gridDim.x - 1) / (long long)gridDim.x, (long long)W);
  const long long cta0 = blockIdx.x * per, cta1 = min(total, cta0 + per);
  if (cta0 >= total) return;
  const int len = (int)(cta1 - cta0);
  auto warp_start = [&](int w) { return cta0 + (long long)len * w / W; };
  {
    long long base = 0;
    for (int s0 = 0; s0 < p.num_seqs && base < cta1; s0 += W * 32) {
      const int s = s0 + threadIdx.x;
      const long long c = s < p.num_seqs ? seq_cost<R>(p, s) : 0;
      long long part;
      const long long end = base + block_scan<W>(c, sh.scan, &part);
      if (c > 0 && end > cta0 && end - c < cta1)
        for (int w = 0; w < W; ++w) {
          const long long at = warp_start(w);
          if (at >= end - c && at < end) {
            sh.start_seq[w] = s;
            sh.start_pre[w] = end - c;
          }
        }
      base += part;
    }
  }
  __syncthreads();

  const long long pos0 = warp_start(warp), pos1 = warp_start(warp + 1);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(smem + S::ring_off) + warp * S::kRing;
  const uint32_t bars = (uint32_t)__cvta_generic_to_shared(&sh.bars[warp * S::kStages]);
  bool ok = true;

  if (pos1 > pos0) {
    // ---- loads: a cursor of their own, kStages blocks ahead of the arithmetic
    Cursor<R> ld;
    ld.begin(p, sh.start_seq[warp], sh.start_pre[warp], pos0);
    int left = (int)(pos1 - pos0);  // blocks not yet issued
    int issued = 0;
    int ids = 0, ids_at = -1;       // lane i: the id of block ids_at + i of the sequence
    auto issue = [&]() {
      if (ids_at < 0 || ld.blk >= ids_at + 32) {
        ids_at = ld.blk;
        const int b = min(ids_at + lane, ld.q.nblk - 1);
        ids = p.block_tables[(int64_t)ld.s * p.max_blocks_per_seq + b];
        ids = min(max(ids, 0), p.num_blocks - 1);  // never outside the pool
      }
      const int id = __shfl_sync(0xffffffffu, ids, ld.blk - ids_at);
      if (lane == 0) {
        const int st = issued % S::kStages;
        mbar_expect_tx(bars + 8 * st, S::kTile);
        bulk_load(ring + st * S::kTile,
                  p.kv_cache + ((int64_t)id * p.num_kv_heads + ld.head) * S::kTile, S::kTile,
                  bars + 8 * st);
      }
      ++issued;
      --left;
      if (++ld.blk == ld.q.nblk) {
        const int was = ld.s;
        if (left > 0) ld.next_unit(p);
        if (ld.s != was || ids_at > 0) ids_at = -1;
      }
    };
    for (int i = 0; i < S::kStages && left > 0; ++i) issue();

    // ---- the units of this stretch
    Cursor<R> cu;
    cu.begin(p, sh.start_seq[warp], sh.start_pre[warp], pos0);
    long long pos = pos0;
    int done = 0;
    while (pos < pos1 && ok) {
      const int blk0 = cu.blk;
      const int nb = (int)min((long long)(cu.q.nblk - blk0), pos1 - pos);
      const int nrows = min(R, cu.q.ql * p.group - cu.rg * R);
      // -- the query rows (the B operand): row g (+8), this lane's chunk of dims
      uint32_t qf[QP][NT][K][2];
      float sl2[NT][2];  // log2(e) scale of the scores of rows 2t, 2t+1 (+8)
      int lim[NT][2];    // their last visible key
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const int row = n * 8 + g;
        const int rr = cu.rg * R + row;
        float x[S::kChunkK];
        if (row < nrows) {
          const int j = rr / p.group;
          const T* src = (const T*)p.q +
                         ((int64_t)(cu.q.q0 + j) * p.num_q_heads + cu.head * p.group +
                          (rr - j * p.group)) * D +
                         t * S::kChunkK;
#pragma unroll
          for (int i = 0; i < S::kChunkK; i += 16 / (int)sizeof(T)) {
            const uint4 w = *(const uint4*)(src + i);
            const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              if constexpr (sizeof(T) == 2) {
                x[i + 2 * k] = __uint_as_float(u[k] << 16);
                x[i + 2 * k + 1] = __uint_as_float(u[k] & 0xffff0000u);
              } else {
                x[i + k] = __uint_as_float(u[k]);
              }
            }
          }
        } else {
#pragma unroll
          for (int i = 0; i < S::kChunkK; ++i) x[i] = 0.f;
        }
        float mx = 0.f;
#pragma unroll
        for (int i = 0; i < S::kChunkK; ++i) mx = fmaxf(mx, fabsf(x[i]));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the exponent of the row's largest value; 0 for a row of zeros and
        // (as they are) for infinities.  Two factors: 2^-e alone may overflow
        const int e = mx > 0.f && mx < INFINITY ? ilogbf(mx) : 0;
        const int e1 = -e / 2;
        const float f1 = __int_as_float((127 + e1) << 23), f2 = __int_as_float((127 - e - e1) << 23);
#pragma unroll
        for (int i = 0; i < S::kChunkK; ++i) x[i] = x[i] * f1 * f2;
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
          sl2[n][c] = ldexpf(p.scale_log2, er);
          const int r2 = cu.rg * R + n * 8 + 2 * t + c;
          lim[n][c] = n * 8 + 2 * t + c < nrows ? cu.q.L - cu.q.ql + r2 / p.group : cu.q.L - 1;
        }
      }

      float o[NT][K][4];
      float m[NT][2], l[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int i = 0; i < K; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[n][i][c] = 0.f;
        m[n][0] = m[n][1] = -INFINITY;
        l[n][0] = l[n][1] = 0.f;
      }

      for (int b = 0; b < nb; ++b, ++done) {
        const int st = done % S::kStages;
        ok = wait_bar(bars + 8 * st, (done / S::kStages) & 1, abort_flag, p.ws_status);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const unsigned char* tile = smem + S::ring_off + warp * S::kRing + st * S::kTile;
        // -- this lane's codes and scales: K of tokens ta and ta + 2, V of
        // tokens 4t .. 4t + 3
        const int ta = 4 * (g >> 1) + (g & 1);
        uint32_t kw[2][K / 2], vw[2][K / 2];
        uint32_t ks[2], vs;
        if constexpr (D == 128) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint4 a = *(const uint4*)(tile + (ta + 2 * h) * 64 + t * 16);
            kw[h][0] = a.x; kw[h][1] = a.y; kw[h][2] = a.z; kw[h][3] = a.w;
            const uint4 v = *(const uint4*)(tile + Tile::v_off + h * 512 + lane * 16);
            vw[h][0] = v.x; vw[h][1] = v.y; vw[h][2] = v.z; vw[h][3] = v.w;
            ks[h] = *(const uint16_t*)(tile + Tile::ks_off + (ta + 2 * h) * 8 + 2 * t);
          }
          vs = *(const uint32_t*)(tile + Tile::vs_off + g * 16 + 4 * t);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint2 a = *(const uint2*)(tile + (ta + 2 * h) * 32 + t * 8);
            kw[h][0] = a.x; kw[h][1] = a.y;
            const uint2 v = *(const uint2*)(tile + Tile::v_off + h * 256 + lane * 8);
            vw[h][0] = v.x; vw[h][1] = v.y;
            ks[h] = *(tile + Tile::ks_off + (ta + 2 * h) * 4 + t);
          }
          vs = *(const uint32_t*)(tile + Tile::vs_off + (g >> 1) * 16 + 4 * t);
        }
        __syncwarp();  // the stage is free once every lane holds its part of it
        if (left > 0) issue();

        // -- S^T = K Q^T in two chains of MMAs
        float sc[NT][2][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[n][0][c] = sc[n][1][c] = 0.f;
        __half2 k2[2][2];  // [token][group of the chunk]
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const __half2 two = e4m3x2_to_half2(ks[h]);
          k2[h][0] = __low2half2(two);
          k2[h][1] = __high2half2(two);
        }
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int grp = D == 128 ? k / 4 : 0;
          const uint32_t w0 = kw[0][k / 2] >> (16 * (k & 1)), w1 = kw[1][k / 2] >> (16 * (k & 1));
          const uint32_t a0 = deq<0>(w0, k2[0][grp]), a1 = deq<0>(w1, k2[1][grp]);
          const uint32_t a2 = deq<1>(w0, k2[0][grp]), a3 = deq<1>(w1, k2[1][grp]);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int qp = 0; qp < QP; ++qp)
              mma_f16(sc[n][k & 1], a0, a1, a2, a3, qf[qp][n][k][0], qf[qp][n][k][1]);
        }
        // -- scores in log2 units; keys past a row's last visible one are out
        float x[NT][4];
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) x[n][c] = (sc[n][0][c] + sc[n][1][c]) * sl2[n][c & 1];
        const int key0 = (blk0 + b) * kBlockSize;
        if (key0 + kBlockSize > cu.q.L - cu.q.ql + 1) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (key0 + ta + (c & 2) > lim[n][c & 1]) x[n][c] = -INFINITY;
          // V of slots that hold no token yet: whatever they hold counts as 0
          const int held = cu.q.L - key0 - 4 * t;
          if (held < 4) vs = held <= 0 ? 0u : vs & (0xffffffffu >> (32 - 8 * held));
        }
        // -- the running max moves when a score passes it by 2^8
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c)
            over |= fmaxf(x[n][c], x[n][c + 2]) > m[n][c] + kRescale ||
                    (m[n][c] == -INFINITY && fmaxf(x[n][c], x[n][c + 2]) > -INFINITY);
        if (__any_sync(0xffffffffu, over)) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              float mx = fmaxf(x[n][c], x[n][c + 2]);
#pragma unroll
              for (int s = 4; s < 32; s <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
              if (mx > m[n][c] + kRescale || (m[n][c] == -INFINITY && mx > -INFINITY)) {
                const float f = ex2(m[n][c] - mx);
                m[n][c] = mx;
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
        uint32_t pf[QP][NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float e[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const float base = m[n][c & 1] == -INFINITY ? 0.f : m[n][c & 1] - kPShift;
            e[c] = ex2(x[n][c] - base);
          }
          l[n][0] += e[0] + e[2];
          l[n][1] += e[1] + e[3];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const __half2 hi = __floats2half2_rn(e[2 * h], e[2 * h + 1]);
            pf[0][n][h] = transpose8(bits(hi));
            if constexpr (QP == 2)
              pf[QP - 1][n][h] = transpose8(bits(__floats2half2_rn(
                  e[2 * h] - __low2float(hi), e[2 * h + 1] - __high2float(hi))));
          }
        }
        // -- O^T += V^T P^T: the codes of a pair of tokens side by side in a
        // byte (even dims, odd dims), converted and scaled
        const __half2 v2[2] = {e4m3x2_to_half2(vs & 0xffffu), e4m3x2_to_half2(vs >> 16)};
        constexpr uint32_t kLow = 0x0f0f0f0fu;
#pragma unroll
        for (int w = 0; w < K / 4; ++w) {
          uint32_t ev[2], od[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t a = vw[h][w], c = vw[h][K / 4 + w];
            ev[h] = (a & kLow) | ((c << 4) & ~kLow);
            od[h] = ((a >> 4) & kLow) | (c & ~kLow);
          }
          auto step = [&](auto ic) {
            constexpr int i = decltype(ic)::value;
            const uint32_t a0 = deq<i>(ev[0], v2[0]), a1 = deq<i>(od[0], v2[0]);
            const uint32_t a2 = deq<i>(ev[1], v2[1]), a3 = deq<i>(od[1], v2[1]);
#pragma unroll
            for (int n = 0; n < NT; ++n)
#pragma unroll
              for (int qp = 0; qp < QP; ++qp)
                mma_f16(o[n][4 * w + i], a0, a1, a2, a3, pf[qp][n][0], pf[qp][n][1]);
          };
          step(std::integral_constant<int, 0>{});
          step(std::integral_constant<int, 1>{});
          step(std::integral_constant<int, 2>{});
          step(std::integral_constant<int, 3>{});
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
            const int rr = cu.rg * R + row, j = rr / p.group;
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
        pm.seq = cu.s;
        pm.head = cu.head;
        pm.rg = cu.rg;
        pm.ended = blk0 + nb == cu.q.nblk;
        pm.valid = 1;
      }
      if (pos < pos1) cu.next_unit(p);
    }
  }
  __syncthreads();
  if (sh.abort) return;

  // ---- join the parts.  A run: the parts of one unit in this CTA, in order:
  // the last part of the warp where it starts (or the first part of warp 0, of
  // a unit that starts in an earlier CTA) and the first parts that follow
  unsigned starts, firsts, ends;
  {
    const bool in = lane < W;
    const bool v0 = in && sh.meta[lane][0].valid, v1 = in && sh.meta[lane][1].valid;
    firsts = __ballot_sync(0xffffffffu, v0);
    ends = __ballot_sync(0xffffffffu, v0 && sh.meta[lane][0].ended);
    starts = __ballot_sync(0xffffffffu, v1);
  }
  // a unit from an earlier CTA: its run starts at the first warp with a first
  // part before any unit starts here
  const int lead = firsts ? __ffs(firsts) - 1 : 32;
  const bool carried = lead < 32 && (starts & ((1u << lead) - 1)) == 0;
  const int nruns = __popc(starts) + (carried ? 1 : 0);
  unsigned rest = starts;
  bool pending[2] = {false, false};   // a part of a unit that other CTAs hold too
  PartMeta far[2];
  for (int r = 0; r < nruns; ++r) {
    const bool from_before = carried && r == 0;
    int w0;
    if (from_before) {
      w0 = lead;
    } else {
      w0 = __ffs(rest) - 1;
      rest &= rest - 1;
    }
    // the warps whose first parts belong to the run
    unsigned mine = firsts & (from_before ? ~0u << w0 : w0 == 31 ? 0u : ~0u << (w0 + 1));
    const unsigned end = ends & mine;
    const bool ended = end != 0;
    if (ended) mine &= (end & -end) | ((end & -end) - 1);
    const PartMeta& pm = sh.meta[w0][from_before ? 0 : 1];
    const Seq q = load_seq<R>(p, pm.seq);
    const int nrows = min(R, q.ql * p.group - pm.rg * R);
    const bool complete = ended && !from_before;
    const int side = from_before ? 0 : 1;
    if (!complete) {
      pending[side] = true;
      far[side] = pm;
    }
    for (int row = warp; row < nrows; row += W) {
      // weights of the parts: lane w that of warp w's first part, lane 31 that
      // of the part the unit starts with
      float mi = -INFINITY, li = 0.f;
      const bool first = lane < W && (mine >> lane & 1);
      const bool last = !from_before && lane == 31;
      if (first || last) {
        const float* ml = sh.ml[last ? w0 : lane][last ? 1 : 0][row];
        mi = ml[0];
        li = ml[1];
      }
      float mx = mi;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      const float wt = mi == -INFINITY ? 0.f : ex2(mi - mx);
      float sum = li * wt;
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
      float y[D / 32];
#pragma unroll
      for (int i = 0; i < D / 32; ++i) y[i] = 0.f;
      auto add = [&](const float* part, float f) {
#pragma unroll
        for (int i = 0; i < D / 32; ++i) y[i] = fmaf(f, part[row * D + lane * (D / 32) + i], y[i]);
      };
      if (!from_before)
        add((const float*)(smem + S::ring_off + w0 * S::kRing), __shfl_sync(0xffffffffu, wt, 31));
      for (unsigned left = mine; left; left &= left - 1) {
        const int w = __ffs(left) - 1;
        add((const float*)(smem + S::part_off + w * S::kPart), __shfl_sync(0xffffffffu, wt, w));
      }
      if (complete) {
        const int rr = pm.rg * R + row, j = rr / p.group;
        T* dst = (T*)p.out + ((int64_t)(q.q0 + j) * p.num_q_heads + pm.head * p.group +
                              (rr - j * p.group)) * D + lane * (D / 32);
#pragma unroll
        for (int i = 0; i < D / 32; ++i) dst[i] = (T)(y[i] * (p.v_scale / sum));
      } else {
        const int64_t at = (int64_t)(blockIdx.x * 2 + side) * 16 + row;
#pragma unroll
        for (int i = 0; i < D / 32; ++i) p.ws_o[at * D + lane * (D / 32) + i] = y[i];
        if (lane == 0) {
          p.ws_ml[at * 2] = mx;
          p.ws_ml[at * 2 + 1] = sum;
        }
      }
    }
  }
  if (!pending[0] && !pending[1]) return;

  // ---- a unit in several CTAs: the one that arrives last joins its parts, in
  // the order of the CTAs
  __threadfence();
  __syncthreads();
  if (threadIdx.x < 2) {
    int mine = 0;
    if (pending[threadIdx.x]) {
      const PartMeta& f = far[threadIdx.x];
      const int c0 = (int)(f.unit_start / per), c1 = (int)((f.unit_start + f.nblk - 1) / per);
      mine = atomicAdd(p.ws_counters + c0, 1) == c1 - c0;
      if (mine) p.ws_counters[c0] = 0;  // every part has arrived: zero for the next call
    }
    sh.last[threadIdx.x] = mine;
  }
  __syncthreads();
#pragma unroll 1
  for (int side = 0; side < 2; ++side) {
    if (!sh.last[side]) continue;
    __threadfence();
    const PartMeta f = far[side];
    const Seq q = load_seq<R>(p, f.seq);
    const int nrows = min(R, q.ql * p.group - f.rg * R);
    const int c0 = (int)(f.unit_start / per), c1 = (int)((f.unit_start + f.nblk - 1) / per);
    for (int row = warp; row < nrows; row += W) {
      auto at = [&](int c) { return (int64_t)(c * 2 + (c == c0 ? 1 : 0)) * 16 + row; };
      float mx = -INFINITY;
      for (int c = c0 + lane; c <= c1; c += 32) mx = fmaxf(mx, __ldcg(p.ws_ml + at(c) * 2));
#pragma unroll
      for (int s = 16; s > 0; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
      float y[D / 32], sum = 0.f;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) y[i] = 0.f;
#pragma unroll 4
      for (int c = c0; c <= c1; ++c) {
        const float mi = __ldcg(p.ws_ml + at(c) * 2);
        const float wt = mi == -INFINITY ? 0.f : ex2(mi - mx);
        sum = fmaf(wt, __ldcg(p.ws_ml + at(c) * 2 + 1), sum);
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
          y[i] = fmaf(wt, __ldcg(p.ws_o + at(c) * D + lane * (D / 32) + i), y[i]);
      }
      const int rr = f.rg * R + row, j = rr / p.group;
      T* dst = (T*)p.out + ((int64_t)(q.q0 + j) * p.num_q_heads + f.head * p.group +
                            (rr - j * p.group)) * D + lane * (D / 32);
#pragma unroll
      for (int i = 0; i < D / 32; ++i) dst[i] = (T)(y[i] * (p.v_scale / sum));
    }
  }
}

template <int D, int NT, int QP, typename T>
cudaError_t launch_shape(const Fp4AttnParams& p, cudaStream_t stream) {
  using S = Shape<D, NT, QP>;
  auto kernel = decode_fp4_kernel<S, T>;
  static std::atomic<int> smem_done[64];
  cudaError_t e = raise_smem_limit(kernel, S::total, smem_done);
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(min(device_sm_count(), kFp4MaxCtas));
  cfg.blockDim = dim3(S::kWarps * 32);
  cfg.dynamicSmemBytes = S::total;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_decode_fp4(const Fp4AttnParams& p, int head_dim, bool f32, int rows,
                              cudaStream_t stream) {
  cudaError_t e;
  const bool wide = rows > 8;
  if (f32) {
    if (head_dim == 64)
      e = wide ? launch_shape<64, 2, 2, float>(p, stream) : launch_shape<64, 1, 2, float>(p, stream);
    else
      e = wide ? launch_shape<128, 2, 2, float>(p, stream)
               : launch_shape<128, 1, 2, float>(p, stream);
  } else {
    if (head_dim == 64)
      e = wide ? launch_shape<64, 2, 1, __nv_bfloat16>(p, stream)
               : launch_shape<64, 1, 1, __nv_bfloat16>(p, stream);
    else
      e = wide ? launch_shape<128, 2, 1, __nv_bfloat16>(p, stream)
               : launch_shape<128, 1, 1, __nv_bfloat16>(p, stream);
  }
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace pa
