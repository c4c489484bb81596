// rope_append.cu -- a step's new rows on their way into the cache: queries and
// keys rotated to their positions, keys and values stored through the slot
// mapping, in the input's type or in 4 bits; and rows of a 4-bit cache back as
// values.
//
// Page "LLM推論エンジンvLLMの内部構造を徹底解説", section "PagedAttentionの仕組み": KV
// lives in 16-token blocks and position indices tell the tokens of the
// flattened step apart; a token's slot names its block and offset.
//
// Rotation by the angle of (position, pair) of the first `rotary_dim` dims:
//   y1 = x1 cos - x2 sin,  y2 = x2 cos + x1 sin
// over the pairs (i, i + rotary_dim / 2), or (2 i, 2 i + 1) when interleaved.
// In fp32, each product and sum rounded on its own (no contraction into an
// FMA), so that the stored bits follow from the formula alone; then rounded
// once to the row's type, or to a 4-bit group.
//
// Quantisation of 16 dims x of one token: s = e4m3(min(max|x| / (6 g), 448)),
// codes e2m1(x / (s g)), g the tensor's scale.  Both quotients are rounded as IEEE's:
// a value half-way between two codes then goes to the even code, where a
// product with a rounded reciprocal alone would send it either way.  A NaN makes its
// group's scale NaN.
//
// Bound: HBM bytes for prompts, latency for a few tokens.  A lane holds two
// 8-dim vectors of one head row (both sides of its rotation pairs: nothing is
// exchanged between lanes except the 4-bit groups' maxima), D / 16 lanes a row.
// A warp takes U row sets of one token, their loads issued together, and reads
// that token's cos / sin once for them.
#include <math.h>

#include "pa_fp4.cuh"

namespace pa {
namespace {

// Small CTAs: a warp is done after two round trips to memory, and its place is
// free at once (8 warps: 46.8 us for 8192 tokens of 32 + 2 x 8 heads of 128 in
// bf16, 205 MB; 4 warps: 41.7, both with one item per warp)
constexpr int kWarps = 4;

// eight consecutive elements
__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = __ldg((const float4*)p), b = __ldg((const float4*)p + 1);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
__device__ __forceinline__ void store8(float* p, const float (&x)[8]) {
  ((float4*)p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  ((float4*)p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&x)[8]) {
  uint4 w;
  __nv_bfloat162 h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
  w.x = *(uint32_t*)&h[0]; w.y = *(uint32_t*)&h[1];
  w.z = *(uint32_t*)&h[2]; w.w = *(uint32_t*)&h[3];
  *(uint4*)p = w;
}
// a row vector as it lies in memory, and its values
template <typename T>
struct Raw8 {
  uint4 w[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) w[i] = ((const uint4*)p)[i];
  }
  __device__ __forceinline__ void store(T* p) const {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) / 2; ++i) ((uint4*)p)[i] = w[i];
  }
  __device__ __forceinline__ void values(float (&x)[8]) const {
    if constexpr (sizeof(T) == 2) {
      const uint32_t u[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = __uint_as_float(u[i] << 16);
        x[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
      }
    } else {
      const uint32_t u[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(u[i]);
    }
  }
};

__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float absmax8(const float (&x)[8]) {
  float m = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) m = max_nan(m, fabsf(x[i]));
  return m;
}
// scale byte of a group whose largest magnitude is amax (six_g = 6 g)
__device__ __forceinline__ uint32_t group_scale(float amax, float six_g) {
  return __nv_cvt_float_to_fp8(__fdiv_rn(amax, six_g), __NV_SATFINITE, __NV_E4M3);
}
// eight codes under that scale, dim 2j in the low half of byte j
__device__ __forceinline__ uint32_t codes8(const float (&x)[8], uint32_t scale, float g) {
  const float product = __fmul_rn(e4m3_to_float(scale), g);
  float y[8];
  // One correctly rounded reciprocal and two residual steps give each quotient as the
  // division rounds it (Markstein 1990: q + (x - q d) RN(1 / d) rounds right from a q
  // within a unit of the last place), where nothing overflows and no residual that
  // matters underflows: scales that neither saturate nor are NaN (quotients below 16),
  // tensor scales of middle size.  4099 tokens of 32 + 2 x 8 heads of 128: 23.7 us, with
  // a division per value 24.7.
  if (scale < 126 && (product == 0.f || (product >= 0x1p-60f && product <= 0x1p60f))) {
    const float r = product > 0.f ? __frcp_rn(product) : 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      float q = __fmul_rn(x[i], r);
      q = fmaf(fmaf(-q, product, x[i]), r, q);
      y[i] = fmaf(fmaf(-q, product, x[i]), r, q);
    }
  } else {
    const float d = product > 0.f ? product : INFINITY;
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __fdiv_rn(x[i], d);
  }
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= (uint32_t)__nv_cvt_float2_to_fp4x2(make_float2(y[2 * i], y[2 * i + 1]), __NV_E2M1,
                                            cudaRoundNearest)
         << (8 * i);
  return w;
}

// U: row sets per warp (their loads are in flight together)
template <typename T, int D, bool kFp4, int U>
__global__ void __launch_bounds__(kWarps * 32)
rope_append_kernel(const RopeAppendParams p, int chunks, int64_t items) {
  using Tile = Fp4Tile<D>;
  constexpr int kLanes = D / 16;          // lanes of a row
  constexpr int kRows = 32 / kLanes;      // rows of a row set
  // launched as a programmatic dependent of the work before it on the stream,
  // and lets the work after it be launched: see the other kernels
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int lane = threadIdx.x & 31;
  const int l = lane % kLanes, sub = lane / kLanes;
  const int nk = p.num_q_heads, nv = nk + p.num_kv_heads, n = nv + p.num_kv_heads;

  // this lane's two vectors of a row: the two sides of its rotation pairs; of
  // the dims past rotary_dim, one from each half
  const int half_pairs = p.rotary_dim / 16;
  const bool rotated = l < half_pairs;
  int va, vb;
  if (p.interleaved) {
    va = 2 * l;
    vb = va + 1;
  } else {
    va = rotated ? l : half_pairs + l;
    vb = va + (rotated ? half_pairs : kLanes - half_pairs);
  }

  // An item is U row sets of one token.  Its slot and position are read one
  // item ahead, so that its rows and angles are one round trip away.
  const int64_t step = (int64_t)gridDim.x * kWarps;
  int64_t item = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (item >= items) return;
  int64_t tok = item / chunks, slot = p.slot_mapping[tok];
  int64_t pos = p.rotary_dim > 0 ? p.positions[tok] : 0;
#pragma unroll 1
  while (true) {
    const int row0 = (int)(item - tok * chunks) * (kRows * U) + sub;
    Raw8<T> a[U], b[U];
  #pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = min(row0 + u * kRows, n - 1);  // past the last row: that row again, unused
      const T* src = r < nk   ? (const T*)p.q + tok * p.q_stride + (int64_t)r * D
                     : r < nv ? (const T*)p.k + tok * p.k_stride + (int64_t)(r - nk) * D
                              : (const T*)p.v + tok * p.v_stride + (int64_t)(r - nv) * D;
      a[u].load(src + 8 * va);
      b[u].load(src + 8 * vb);
    }
    const bool stored = slot >= 0 && slot < (int64_t)p.num_blocks * kBlockSize;
    const int64_t blk = slot / kBlockSize;
    const int off = (int)(slot % kBlockSize);
    // without an angle the token is left out
    const bool placed = p.rotary_dim == 0 || (pos >= 0 && pos < p.max_position);
    float c[8], s[8];
    if (placed && rotated && row0 < nv) {
      const float* t = p.cos_sin + pos * p.rotary_dim + 8 * l;
      load8(t, c);
      load8(t + p.rotary_dim / 2, s);
    }
    // the next item's
    const int64_t item2 = item + step, tok1 = tok;
    if (item2 < items) {
      tok = item2 / chunks;
      slot = p.slot_mapping[tok];
      pos = p.rotary_dim > 0 ? p.positions[tok] : 0;
    }
  #pragma unroll
    for (int u = 0; u < U; ++u) {
      const int r = row0 + u * kRows;
      // every lane of the warp stays in the loop: the 4-bit groups' maxima are
      // exchanged between lanes of a row
      const bool live = placed && r < n && (r < nk || stored);
      float x[8], y[8];
      a[u].values(x);
      b[u].values(y);
      const bool turn = rotated && r < nv;
      if (turn) {
        if (p.interleaved) {
  #pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float x0 = x[2 * j], x1 = x[2 * j + 1], y0 = y[2 * j], y1 = y[2 * j + 1];
            x[2 * j] = __fsub_rn(__fmul_rn(x0, c[j]), __fmul_rn(x1, s[j]));
            x[2 * j + 1] = __fadd_rn(__fmul_rn(x1, c[j]), __fmul_rn(x0, s[j]));
            y[2 * j] = __fsub_rn(__fmul_rn(y0, c[4 + j]), __fmul_rn(y1, s[4 + j]));
            y[2 * j + 1] = __fadd_rn(__fmul_rn(y1, c[4 + j]), __fmul_rn(y0, s[4 + j]));
          }
        } else {
  #pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float x0 = x[j], y0 = y[j];
            x[j] = __fsub_rn(__fmul_rn(x0, c[j]), __fmul_rn(y0, s[j]));
            y[j] = __fadd_rn(__fmul_rn(y0, c[j]), __fmul_rn(x0, s[j]));
          }
        }
      }
      if constexpr (kFp4) {
        const bool is_v = r >= nv;
        const int h = r - (is_v ? nv : nk);
        const float g = is_v ? p.v_scale : p.k_scale, six_g = is_v ? p.v_six : p.k_six;
        // interleaved: a lane holds a whole group; else each half of a group
        // lies with the neighbouring lane
        // (asked of the warp's rows, not of this lane's)
        if (row0 - sub + u * kRows + kRows > nk) {
          float ma = absmax8(x), mb = absmax8(y);
          const float oa = __shfl_xor_sync(0xffffffffu, ma, 1);
          const float ob = __shfl_xor_sync(0xffffffffu, mb, 1);
          if (p.interleaved) {
            ma = mb = max_nan(ma, mb);
          } else {
            ma = max_nan(ma, oa);
            mb = max_nan(mb, ob);
          }
          if (live && r >= nk) {
            uint8_t* tile = (uint8_t*)p.k_cache + (blk * p.num_kv_heads + h) * (int64_t)Tile::bytes;
            const uint32_t sa = group_scale(ma, six_g), sb = group_scale(mb, six_g);
            const uint32_t wa = codes8(x, sa, g), wb = codes8(y, sb, g);
            if (is_v) {
              *(uint32_t*)(tile + Tile::v_word(off, va)) = wa;
              *(uint32_t*)(tile + Tile::v_word(off, vb)) = wb;
              if (va % 2 == 0) tile[Tile::v_scale(off, va / 2)] = (uint8_t)sa;
              if (vb % 2 == 0) tile[Tile::v_scale(off, vb / 2)] = (uint8_t)sb;
            } else {
              *(uint32_t*)(tile + Tile::k_word(off, va)) = wa;
              *(uint32_t*)(tile + Tile::k_word(off, vb)) = wb;
              if (va % 2 == 0) tile[Tile::k_scale(off, va / 2)] = (uint8_t)sa;
              if (vb % 2 == 0) tile[Tile::k_scale(off, vb / 2)] = (uint8_t)sb;
            }
            continue;
          }
        }
      }
      if (!live) continue;
      T* dst;
      if (r < nk) {
        dst = (T*)p.q_out + (tok1 * nk + r) * (int64_t)D;
      } else {
        const int h = r - (r < nv ? nk : nv);
        dst = (T*)(r < nv ? p.k_cache : p.v_cache) +
              ((blk * p.num_kv_heads + h) * kBlockSize + off) * (int64_t)D;
      }
      if (turn) {
        store8(dst + 8 * va, x);
        store8(dst + 8 * vb, y);
      } else {  // bit-exact copy
        a[u].store(dst + 8 * va);
        b[u].store(dst + 8 * vb);
      }
    }
    if (item2 >= items) break;
    item = item2;
  }
}

// One thread per (row, kv-head, 16-dim group): K and V.
template <typename T, int D>
__global__ void __launch_bounds__(256)
gather_fp4_kernel(const GatherFp4Params p, int64_t threads) {
  using Tile = Fp4Tile<D>;
  asm volatile("griddepcontrol.launch_dependents;\n" ::: "memory");
  asm volatile("griddepcontrol.wait;\n" ::: "memory");
  const int64_t i = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  if (i >= threads) return;
  const int g = (int)(i % Tile::kGroups);
  const int64_t rh = i / Tile::kGroups;
  const int h = (int)(rh % p.num_kv_heads);
  const int64_t slot = p.slots[rh / p.num_kv_heads];
  if (slot < 0 || slot >= (int64_t)p.num_blocks * kBlockSize) return;
  const uint8_t* tile = p.kv_cache +
                        (slot / kBlockSize * p.num_kv_heads + h) * (int64_t)Tile::bytes;
  const int off = (int)(slot % kBlockSize);
  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    w[j] = *(const uint32_t*)(tile + Tile::k_word(off, 2 * g + j));
    w[2 + j] = *(const uint32_t*)(tile + Tile::v_word(off, 2 * g + j));
  }
  const float s[2] = {e4m3_to_float(tile[Tile::k_scale(off, g)]),
                      e4m3_to_float(tile[Tile::v_scale(off, g)])};
  T* dst[2] = {(T*)p.k_out, (T*)p.v_out};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float sc = s[j / 2], own = j < 2 ? p.k_scale : p.v_scale;
    float x[8];
    __half2 two[4];
    e2m1x8_to_half2(w[j], two);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float2 f = __half22float2(two[e]);
      x[2 * e] = __fmul_rn(f.x * sc, own);  // code * scale is exact
      x[2 * e + 1] = __fmul_rn(f.y * sc, own);
    }
    store8(dst[j / 2] + rh * D + 16 * g + 8 * (j % 2), x);
  }
}

// CTAs of a kernel that one SM holds, asked for once per kernel and device
template <typename Kernel>
int resident_ctas(Kernel kernel, int threads, std::atomic<int> (&known)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 1;
  int n = known[dev].load(std::memory_order_relaxed);
  if (n == 0) {
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, 0) != cudaSuccess ||
        n < 1)
      return 1;
    known[dev].store(n, std::memory_order_relaxed);
  }
  return n;
}

cudaLaunchConfig_t dependent_launch(int64_t grid, int threads, cudaStream_t stream,
                                    cudaLaunchAttribute* attr) {
  attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr->val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(threads);
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cfg;
}

template <typename T, int D, bool kFp4>
cudaError_t launch_rope(const RopeAppendParams& p, cudaStream_t stream) {
  constexpr int kRows = 32 / (D / 16);
  // row sets per warp once every SM has its fill of warps: more loads in
  // flight against more registers (8192 bf16 tokens as above: 43.1 us with two,
  // 41.7 with three or four, one item per warp; quantising, 4099 tokens: 27.8, 33.1, 33.8)
  constexpr int kWide = kFp4 ? 2 : 3;
  static std::atomic<int> known1[64], known[64];
  const int n = p.num_q_heads + 2 * p.num_kv_heads;
  cudaLaunchAttribute attr;
  auto go = [&](auto kernel, int u, std::atomic<int> (&known)[64]) {
    const int chunks = (n + kRows * u - 1) / (kRows * u);
    const int64_t items = (int64_t)p.num_tokens * chunks;
    // one wave of CTAs exactly (8192 bf16 tokens as above: 37.2 us, 84 % of the
    // copy rate; with one
    // more per SM than fits 48.0, with one less 41.4)
    const int64_t grid =
        min((items + kWarps - 1) / kWarps,
            (int64_t)device_sm_count() * resident_ctas(kernel, kWarps * 32, known));
    cudaLaunchConfig_t cfg = dependent_launch(grid, kWarps * 32, stream, &attr);
    return cudaLaunchKernelEx(&cfg, kernel, p, chunks, items);
  };
  if ((int64_t)p.num_tokens * n <= (int64_t)device_sm_count() * 64 * kRows)
    return go(rope_append_kernel<T, D, kFp4, 1>, 1, known1);
  return go(rope_append_kernel<T, D, kFp4, kWide>, kWide, known);
}

}  // namespace

cudaError_t launch_rope_append(const RopeAppendParams& p, int head_dim, bool f32, bool fp4,
                               cudaStream_t stream) {
  cudaError_t e;
  if (f32)
    e = head_dim == 64 ? (fp4 ? launch_rope<float, 64, true>(p, stream)
                              : launch_rope<float, 64, false>(p, stream))
                       : (fp4 ? launch_rope<float, 128, true>(p, stream)
                              : launch_rope<float, 128, false>(p, stream));
  else
    e = head_dim == 64 ? (fp4 ? launch_rope<__nv_bfloat16, 64, true>(p, stream)
                              : launch_rope<__nv_bfloat16, 64, false>(p, stream))
                       : (fp4 ? launch_rope<__nv_bfloat16, 128, true>(p, stream)
                              : launch_rope<__nv_bfloat16, 128, false>(p, stream));
  return e == cudaSuccess ? cudaGetLastError() : e;
}

cudaError_t launch_gather_fp4(const GatherFp4Params& p, int head_dim, bool f32,
                              cudaStream_t stream) {
  const int64_t threads = (int64_t)p.num_rows * p.num_kv_heads * (head_dim / 16);
  cudaLaunchAttribute attr;
  cudaLaunchConfig_t cfg = dependent_launch((threads + 255) / 256, 256, stream, &attr);
  cudaError_t e;
  if (f32)
    e = head_dim == 64 ? cudaLaunchKernelEx(&cfg, gather_fp4_kernel<float, 64>, p, threads)
                       : cudaLaunchKernelEx(&cfg, gather_fp4_kernel<float, 128>, p, threads);
  else
    e = head_dim == 64
            ? cudaLaunchKernelEx(&cfg, gather_fp4_kernel<__nv_bfloat16, 64>, p, threads)
            : cudaLaunchKernelEx(&cfg, gather_fp4_kernel<__nv_bfloat16, 128>, p, threads);
  return e == cudaSuccess ? cudaGetLastError() : e;
}

}  // namespace pa
