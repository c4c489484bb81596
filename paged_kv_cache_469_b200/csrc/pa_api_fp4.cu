// pa_api_fp4.cu -- the C ABI of the rotating append and of the 4-bit cache:
// host-side argument checks and dispatch (declared in include/pa.h).
#include <math.h>

#include "pa.h"
#include "pa_fp4.cuh"
#include "pa_internal.cuh"

using namespace pa;

namespace {

bool supported_dim(int d) { return d == 64 || d == 128; }
bool positive(float x) { return x > 0.f && isfinite(x); }

// [first row .. last row] of `heads` x `head_dim` elements, `stride` elements apart
Range rows_range(const void* p, int rows, int64_t stride, int heads, int head_dim, int elem) {
  return Range{p, rows > 0 ? ((size_t)(rows - 1) * stride + (size_t)heads * head_dim) * elem : 0};
}

int rope_append_impl(void* q_out, const void* q, int64_t q_stride, const void* k,
                     int64_t k_stride, const void* v, int64_t v_stride, void* k_cache,
                     void* v_cache, const int64_t* slot_mapping, const int64_t* positions,
                     const float* cos_sin, int64_t max_position, int rotary_dim, int interleaved,
                     int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                     int block_size, int num_blocks, pa_dtype dtype, bool fp4, float k_scale,
                     float v_scale, struct CUstream_st* stream) {
  if (num_tokens < 0 || num_q_heads < 0 || num_kv_heads <= 0 || num_blocks < 0 ||
      max_position < 0 || rotary_dim < 0 || rotary_dim > head_dim)
    return PA_ERR_INVALID;
  if (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16) return PA_ERR_UNSUPPORTED;
  if (block_size != kBlockSize || !supported_dim(head_dim)) return PA_ERR_UNSUPPORTED;
  if (num_q_heads + 2 * (int64_t)num_kv_heads > 1 << 30) return PA_ERR_UNSUPPORTED;  // 32-bit rows
  // a lane's two vectors are the two sides of eight rotation pairs; the 4-bit
  // groups pair neighbouring lanes
  if (rotary_dim % (fp4 && !interleaved ? 32 : 16) != 0) return PA_ERR_UNSUPPORTED;
  if (fp4 && (!positive(k_scale) || !positive(v_scale) || !isfinite(6.f * k_scale) ||
              !isfinite(6.f * v_scale)))
    return PA_ERR_INVALID;
  const int elem = dtype == PA_DTYPE_F32 ? 4 : 2;
  const int64_t strides[3] = {q_stride, k_stride, v_stride};
  for (int64_t s : strides)
    if (s < 0 || s > INT64_MAX / 16 || s * elem % 16 != 0) return PA_ERR_INVALID;
  if (num_tokens == 0) return PA_OK;
  if (!k || !v || !k_cache || (!fp4 && !v_cache) || !slot_mapping) return PA_ERR_INVALID;
  if (num_q_heads > 0 && (!q || !q_out)) return PA_ERR_INVALID;
  if (rotary_dim > 0 && (!positions || !cos_sin)) return PA_ERR_INVALID;
  const void* ptrs[7] = {q, q_out, k, v, k_cache, v_cache, cos_sin};
  for (const void* p : ptrs)
    if (!aligned_to(p, 16)) return PA_ERR_INVALID;
  if (!aligned_to(slot_mapping, 8) || !aligned_to(positions, 8)) return PA_ERR_INVALID;
  if (num_q_heads > 0) {
    // in place, or apart from every input: rows are read and written by
    // different warps in any order
    const int64_t row = (int64_t)num_q_heads * head_dim;
    const Range out = rows_range(q_out, num_tokens, row, num_q_heads, head_dim, elem);
    const bool in_place = q_out == q && (q_stride == row || num_tokens == 1);
    if ((!in_place && out.overlaps(rows_range(q, num_tokens, q_stride, num_q_heads, head_dim, elem))) ||
        out.overlaps(rows_range(k, num_tokens, k_stride, num_kv_heads, head_dim, elem)) ||
        out.overlaps(rows_range(v, num_tokens, v_stride, num_kv_heads, head_dim, elem)))
      return PA_ERR_INVALID;
  }
  RopeAppendParams p{};
  p.q_out = q_out;
  p.q = q;
  p.k = k;
  p.v = v;
  p.q_stride = q_stride;
  p.k_stride = k_stride;
  p.v_stride = v_stride;
  p.k_cache = k_cache;
  p.v_cache = v_cache;
  p.slot_mapping = slot_mapping;
  p.positions = positions;
  p.cos_sin = cos_sin;
  p.max_position = max_position;
  p.rotary_dim = rotary_dim;
  p.interleaved = interleaved != 0;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.num_blocks = num_blocks;
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.k_six = 6.f * k_scale;
  p.v_six = 6.f * v_scale;
  return launch_rope_append(p, head_dim, dtype == PA_DTYPE_F32, fp4, (cudaStream_t)stream) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

// Workspace of attention over a 4-bit cache: the 256-byte header, the arrival
// counters (of a CTA's unit, and two of groups of CTAs), two partial results per CTA, and the prefill work list.
struct Fp4Workspace {
  int max_items;
  size_t counters_off, ml_off, o_off, items_off, total;
};
Fp4Workspace fp4_workspace(int num_seqs, int num_tokens, int num_q_heads, int head_dim) {
  Fp4Workspace w{};
  w.counters_off = 256;
  w.ml_off = w.counters_off + kFp4MaxCtas * 3 * sizeof(int);
  w.o_off = w.ml_off + (size_t)kFp4MaxCtas * 2 * 16 * 2 * sizeof(float);
  w.items_off = w.o_off + (size_t)kFp4MaxCtas * 2 * 16 * head_dim * sizeof(float);
  // a sequence's query tiles times the heads at most, one item each
  const int64_t items =
      ((int64_t)num_tokens / kPrefillQTile + min(num_seqs, num_tokens)) * num_q_heads;
  w.max_items = (int)min(items, (int64_t)1 << 30);
  w.total = w.items_off + ((size_t)w.max_items + 1) * sizeof(int4);
  return w;
}

// What the two attention kernels cost, measured at 148 SMs.  The decode kernel
// reads the keys again for every 16 query rows (8 where no sequence has more) and
// spreads them over all SMs; the prefill kernel takes 128 query tokens of two
// heads at once, an item, on one SM.
struct Fp4Costs {
  double block_ns[2];  // SM-nanoseconds per block and group of 8, of 16 rows
  double tile_ns;      // per item and 128 keys
  int even_q, odd_q;   // with every SM at work the kernels cost the same at about so
                       // many query tokens: where the heads pair up, where they do not
};
Fp4Costs fp4_costs(int head_dim) {
  return head_dim == 128 ? Fp4Costs{{60., 93.}, 1950., 24, 44} : Fp4Costs{{38., 50.}, 1800., 36, 72};
}
constexpr double kLaunchNs = 8000.;  // a kernel's start and end

// The prefill kernel's work of a step.
struct PrefillLoad {
  double items = 0., tiles = 0., longest = 0.;
  // its time on n SMs: the items are given out heaviest first
  double ns(int n, double tile_ns) const {
    if (items <= 0.) return 0.;
    const int ctas = prefill_fp4_cluster(items, longest, n);  // of an item
    if (ctas > 1) return tile_ns * (ceil(longest / ctas) + kPrefillJoinTiles) + kLaunchNs;
    return tile_ns * (items <= n ? longest : max(longest, tiles / n + longest / 2)) + kLaunchNs;
  }
};
struct Fp4Split {
  int decode_q;         // most query tokens of a sequence of the decode kernel
  double decode_sm_ns;  // its work
  PrefillLoad prefill;
  double decode_ns(int n) const {
    return decode_sm_ns > 0. ? decode_sm_ns / n + kLaunchNs : 0.;
  }
};

// Divides a step's sequences between the kernels by their query tokens.  Few
// prefill items leave SMs idle even with their keys cut: one chunk of 64 tokens (32 +
// 8 heads of 128) over 32768 keys takes 100 us there (500 uncut) and 160 on the decode
// kernel, one of 48 over 4096 about 41 and 30.  Without the host copies a step is
// taken for one of equal lengths.
Fp4Split fp4_split(int num_seqs, int num_tokens, int max_query_len, int max_seq_len,
                   int num_q_heads, int num_kv_heads, int head_dim, const int32_t* seq_lens_host,
                   const int32_t* query_start_loc_host) {
  const int group = num_q_heads / num_kv_heads;
  const bool paired = group % 2 == 0;
  const Fp4Costs c = fp4_costs(head_dim);
  const int base = paired ? c.even_q : c.odd_q;
  if (max_query_len <= base) return Fp4Split{base, 0., {}};
  // the candidates, and the step's sequences between one and the next
  constexpr int kBins = 8;
  const int most[kBins] = {base, 48, 96, 160, 256, 400, 640, INT32_MAX};
  double blocks[kBins][2] = {};  // block reads in groups of 8, of 16 rows
  int rows[kBins] = {};
  PrefillLoad load[kBins];
  auto add = [&](int ql, int L, double times) {
    int b = 0;
    while (ql > most[b]) ++b;
    const double kt = (L + kPrefillKvTile - 1) / kPrefillKvTile;
    const double nblk = times * ((L + kBlockSize - 1) / kBlockSize) * num_kv_heads;
    const int qt = (ql + kPrefillQTile - 1) / kPrefillQTile;
    const double items = times * (paired ? qt * (num_q_heads / 2.) : (qt + 1) / 2 * (double)num_q_heads);
    const int64_t r = (int64_t)ql * group;
    blocks[b][0] += nblk * ((r + 7) / 8);
    blocks[b][1] += nblk * ((r + 15) / 16);
    rows[b] = max(rows[b], (int)min(r, (int64_t)64));
    load[b].items += items;
    load[b].tiles += items * kt;
    load[b].longest = max(load[b].longest, kt);
  };
  if (seq_lens_host && query_start_loc_host) {
    for (int s = 0; s < num_seqs; ++s) {
      const int ql = query_start_loc_host[s + 1] - query_start_loc_host[s];
      if (ql > 0) add(ql, seq_lens_host[s], 1.);
    }
  } else {
    add(max_query_len, max_seq_len, max(1, min(num_seqs, num_tokens / max_query_len)));
  }
  const int sms = device_sm_count();
  Fp4Split best{base, 0., {}};
  double best_ns = INFINITY, reads[2] = {0., 0.};
  int most_rows = 0;
  for (int k = 0; k < kBins; ++k) {
    reads[0] += blocks[k][0];
    reads[1] += blocks[k][1];
    most_rows = max(most_rows, rows[k]);
    const int wide = most_rows > 8;
    Fp4Split s{most[k], reads[wide] * c.block_ns[wide], {}};
    for (int j = k + 1; j < kBins; ++j) {
      s.prefill.items += load[j].items;
      s.prefill.tiles += load[j].tiles;
      s.prefill.longest = max(s.prefill.longest, load[j].longest);
    }
    const double ns = s.decode_ns(sms) + s.prefill.ns(sms, c.tile_ns);
    if (ns < best_ns) {
      best_ns = ns;
      best = s;
    }
  }
  return best;
}

// SMs for the prefill kernel when both run side by side, each on its own; 0 where
// that is not expected to end sooner than one after the other.
int fp4_prefill_sms(const Fp4Split& s, int head_dim) {
  const double tile_ns = fp4_costs(head_dim).tile_ns;
  const int sms = device_sm_count();
  double best_ns = 0.95 * (s.decode_ns(sms) + s.prefill.ns(sms, tile_ns));
  int best = 0;
  for (int n = 4; n < sms; n += 4) {
    const double ns = max(s.prefill.ns(n, tile_ns), s.decode_ns(sms - n));
    if (ns < best_ns) {
      best_ns = ns;
      best = n;
    }
  }
  return best;
}

}  // namespace

extern "C" int pa_rope_append(void* q_out, const void* q, int64_t q_stride, const void* k,
                              int64_t k_stride, const void* v, int64_t v_stride, void* k_cache,
                              void* v_cache, const int64_t* slot_mapping,
                              const int64_t* positions, const float* cos_sin,
                              int64_t max_position, int rotary_dim, int interleaved,
                              int num_tokens, int num_q_heads, int num_kv_heads, int head_dim,
                              int block_size, int num_blocks, pa_dtype dtype,
                              struct CUstream_st* stream) {
  return rope_append_impl(q_out, q, q_stride, k, k_stride, v, v_stride, k_cache, v_cache,
                          slot_mapping, positions, cos_sin, max_position, rotary_dim, interleaved,
                          num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                          dtype, false, 1.f, 1.f, stream);
}

extern "C" int pa_rope_append_fp4(void* q_out, const void* q, int64_t q_stride, const void* k,
                                  int64_t k_stride, const void* v, int64_t v_stride,
                                  void* kv_cache, float k_scale, float v_scale,
                                  const int64_t* slot_mapping, const int64_t* positions,
                                  const float* cos_sin, int64_t max_position, int rotary_dim,
                                  int interleaved, int num_tokens, int num_q_heads,
                                  int num_kv_heads, int head_dim, int block_size, int num_blocks,
                                  pa_dtype dtype, struct CUstream_st* stream) {
  return rope_append_impl(q_out, q, q_stride, k, k_stride, v, v_stride, kv_cache, nullptr,
                          slot_mapping, positions, cos_sin, max_position, rotary_dim, interleaved,
                          num_tokens, num_q_heads, num_kv_heads, head_dim, block_size, num_blocks,
                          dtype, true, k_scale, v_scale, stream);
}

extern "C" int pa_gather_fp4(void* k_out, void* v_out, const void* kv_cache, float k_scale,
                             float v_scale, const int64_t* slots, int num_rows, int num_kv_heads,
                             int head_dim, int block_size, int num_blocks, pa_dtype dtype,
                             struct CUstream_st* stream) {
  if (num_rows < 0 || num_kv_heads <= 0 || num_blocks < 0) return PA_ERR_INVALID;
  if (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16) return PA_ERR_UNSUPPORTED;
  if (block_size != kBlockSize || !supported_dim(head_dim)) return PA_ERR_UNSUPPORTED;
  if (!positive(k_scale) || !positive(v_scale)) return PA_ERR_INVALID;
  if (num_rows == 0) return PA_OK;
  if (!k_out || !v_out || !kv_cache || !slots) return PA_ERR_INVALID;
  if (!aligned_to(k_out, 16) || !aligned_to(v_out, 16) || !aligned_to(kv_cache, 16) ||
      !aligned_to(slots, 8))
    return PA_ERR_INVALID;
  const int elem = dtype == PA_DTYPE_F32 ? 4 : 2;
  const int64_t row = (int64_t)num_kv_heads * head_dim;
  const Range out[2] = {rows_range(k_out, num_rows, row, num_kv_heads, head_dim, elem),
                        rows_range(v_out, num_rows, row, num_kv_heads, head_dim, elem)};
  const Range cache{kv_cache, (size_t)num_blocks * num_kv_heads * 18 * head_dim};
  if (out[0].overlaps(out[1]) || out[0].overlaps(cache) || out[1].overlaps(cache))
    return PA_ERR_INVALID;
  const GatherFp4Params p{k_out,    v_out,        (const uint8_t*)kv_cache, slots,
                          num_rows, num_kv_heads, num_blocks,               k_scale,
                          v_scale};
  return launch_gather_fp4(p, head_dim, dtype == PA_DTYPE_F32, (cudaStream_t)stream) ==
                 cudaSuccess
             ? PA_OK
             : PA_ERR_CUDA;
}

extern "C" size_t pa_attention_fp4_workspace_size(int num_seqs, int num_tokens, int num_q_heads,
                                                  int num_kv_heads, int head_dim) {
  if (num_seqs < 0 || num_tokens < 0 || num_kv_heads <= 0 || num_q_heads <= 0) return 0;
  if (num_q_heads % num_kv_heads != 0 || !supported_dim(head_dim)) return 0;
  return fp4_workspace(num_seqs, num_tokens, num_q_heads, head_dim).total;
}

extern "C" int pa_attention_varlen_fp4(
    void* out, const void* q, const void* kv_cache, float k_scale, float v_scale,
    const int32_t* block_tables, int max_blocks_per_seq, const int32_t* seq_lens,
    const int32_t* query_start_loc, int num_seqs, int num_tokens, int max_query_len,
    int max_seq_len, int num_q_heads, int num_kv_heads, int head_dim, int block_size,
    int num_blocks, float scale, pa_dtype dtype, void* workspace, size_t workspace_bytes,
    const int32_t* seq_lens_host, const int32_t* query_start_loc_host,
    struct CUstream_st* stream) {
  if (num_seqs < 0 || num_tokens < 0 || max_query_len < 0 || max_seq_len < 0 ||
      num_q_heads <= 0 || num_kv_heads <= 0 || num_blocks < 0 || max_blocks_per_seq < 0)
    return PA_ERR_INVALID;
  if (dtype != PA_DTYPE_F32 && dtype != PA_DTYPE_BF16) return PA_ERR_UNSUPPORTED;
  if (block_size != kBlockSize || !supported_dim(head_dim)) return PA_ERR_UNSUPPORTED;
  if (num_q_heads % num_kv_heads != 0) return PA_ERR_INVALID;
  const int group = num_q_heads / num_kv_heads;
  if (group > kDecodeRows) return PA_ERR_UNSUPPORTED;
  if (!positive(scale) || !positive(k_scale) || !positive(v_scale) || !positive(scale * k_scale))
    return PA_ERR_INVALID;
  if (max_query_len > max_seq_len) return PA_ERR_INVALID;
  if ((long)max_blocks_per_seq * kBlockSize < (long)max_seq_len) return PA_ERR_INVALID;
  if (num_seqs == 0 || num_tokens == 0) return PA_OK;
  if (!out || !q || !kv_cache || num_blocks == 0 || !block_tables || !seq_lens ||
      !query_start_loc)
    return PA_ERR_INVALID;
  if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(kv_cache, 16) ||
      !aligned_to(block_tables, 4) || !aligned_to(seq_lens, 4) || !aligned_to(query_start_loc, 4))
    return PA_ERR_INVALID;
  // a unit's rows are read by several CTAs while others write theirs
  {
    const size_t bytes = (size_t)num_tokens * num_q_heads * head_dim *
                         (dtype == PA_DTYPE_F32 ? 4 : 2);
    if (Range{out, bytes}.overlaps(Range{q, bytes})) return PA_ERR_INVALID;
  }
  const bool hints = seq_lens_host && query_start_loc_host;
  if (hints) {
    if (query_start_loc_host[0] != 0 || query_start_loc_host[num_seqs] != num_tokens)
      return PA_ERR_INVALID;
    for (int s = 0; s < num_seqs; ++s) {
      const int ql = query_start_loc_host[s + 1] - query_start_loc_host[s];
      const int L = seq_lens_host[s];
      if (ql < 0 || ql > L || L > max_seq_len || ql > max_query_len) return PA_ERR_INVALID;
    }
  }
  // ---- which kernels the step needs
  const bool f32 = dtype == PA_DTYPE_F32;
  const Fp4Split split =
      f32 ? Fp4Split{INT32_MAX, 0., {}}
          : fp4_split(num_seqs, num_tokens, max_query_len, max_seq_len, num_q_heads, num_kv_heads,
                      head_dim, hints ? seq_lens_host : nullptr,
                      hints ? query_start_loc_host : nullptr);
  const int decode_q = split.decode_q;  // most query tokens of a sequence of the decode kernel
  int longest = min(max_query_len, decode_q);  // of the decode kernel's
  bool any_decode = true, any_prefill = max_query_len > decode_q;
  if (hints) {
    longest = 0;
    any_prefill = false;
    for (int s = 0; s < num_seqs; ++s) {
      const int ql = query_start_loc_host[s + 1] - query_start_loc_host[s];
      if (ql > decode_q)
        any_prefill = true;
      else
        longest = max(longest, ql);
    }
    any_decode = longest > 0;
  }
  // query rows per kv-head that choose the decode kernel's row group: where prompt
  // chunks are in the step and lengths are not known, the rest is taken for
  // one-token decodes (192 of them and 4 chunks of 512: 358 -> 279 us; any length
  // is computed right by either group)
  const int64_t rows = (int64_t)(any_prefill && !hints ? 1 : longest) * group;
  // the prefill plan keeps a counter per 128-key tile in shared memory
  if (any_prefill && max_blocks_per_seq / (kPrefillKvTile / kBlockSize) > 50000)
    return PA_ERR_UNSUPPORTED;
  // the decode kernel's line of blocks is counted in 32 bits
  const double groups =
      num_seqs + min((double)num_tokens, (double)num_seqs * longest) * group / (rows > 8 ? 16 : 8);
  if (any_decode && groups * num_kv_heads * ((max_seq_len + kBlockSize - 1) / kBlockSize) >= 2147483648.0)
    return PA_ERR_UNSUPPORTED;
  const Fp4Workspace w = fp4_workspace(num_seqs, num_tokens, num_q_heads, head_dim);
  if (!workspace || workspace_bytes < w.total || !aligned_to(workspace, 16)) return PA_ERR_INVALID;
  char* ws = (char*)workspace;
  Fp4AttnParams p{};
  p.out = out;
  p.q = q;
  p.kv_cache = (const uint8_t*)kv_cache;
  p.block_tables = block_tables;
  p.seq_lens = seq_lens;
  p.query_start_loc = query_start_loc;
  p.max_blocks_per_seq = max_blocks_per_seq;
  p.max_seq_len = max_seq_len;
  p.num_seqs = num_seqs;
  p.num_tokens = num_tokens;
  p.num_q_heads = num_q_heads;
  p.num_kv_heads = num_kv_heads;
  p.group = group;
  p.group_inv = group == 1 ? 0u : (unsigned)(((1ull << 32) + group - 1) / group);
  p.num_blocks = num_blocks;
  p.scale_log2 = scale * k_scale * 1.4426950408889634f;
  p.v_scale = v_scale;
  p.max_q = decode_q;
  p.ws_status = (int*)ws;
  p.ws_counters = (int*)(ws + w.counters_off);
  p.ws_ml = (float*)(ws + w.ml_off);
  p.ws_o = (float*)(ws + w.o_off);
  const cudaStream_t st = (cudaStream_t)stream;
  const int sms = device_sm_count();
  auto run_decode = [&](int ctas) {
    return launch_decode_fp4(p, head_dim, f32, (int)min(rows, (int64_t)INT32_MAX), st, ctas) ==
           cudaSuccess;
  };
  if (!any_prefill) return !any_decode || run_decode(sms) ? PA_OK : PA_ERR_CUDA;
  AttnParams a{};
  a.out = out;
  a.q = q;
  a.k_cache = kv_cache;
  a.block_tables = block_tables;
  a.seq_lens = seq_lens;
  a.query_start_loc = query_start_loc;
  a.max_blocks_per_seq = max_blocks_per_seq;
  a.max_seq_len = max_seq_len;
  a.num_seqs = num_seqs;
  a.num_tokens = num_tokens;
  a.num_q_heads = num_q_heads;
  a.num_kv_heads = num_kv_heads;
  a.group = group;
  a.num_blocks = num_blocks;
  a.scale_log2 = p.scale_log2;
  a.ws_status = a.ws_header = p.ws_status;
  a.ws_items = (int4*)(ws + w.items_off);
  a.max_items = w.max_items;
  a.decode_max_rows = (int)min((int64_t)decode_q * group, (int64_t)INT32_MAX);
  auto run_prefill = [&](cudaStream_t on, int ctas) {
    return launch_prefill_fp4(a, v_scale, head_dim, max_query_len, seq_lens_host,
                              query_start_loc_host, on, ctas) == cudaSuccess;
  };
  // both kinds of work, known from the host copies: side by side, since one is
  // bound by the cache's bytes and the other by arithmetic
  const int prefill_ctas = hints && any_decode ? fp4_prefill_sms(split, head_dim) : 0;
  ForkStreams* fork = prefill_ctas > 0 ? fork_streams(st) : nullptr;
  if (!fork)
    return (!any_decode || run_decode(sms)) && run_prefill(st, sms) ? PA_OK : PA_ERR_CUDA;
  return side_by_side(*fork, st, [&](cudaStream_t side) { return run_prefill(side, prefill_ctas); },
                      [&] { return run_decode(sms - prefill_ctas); })
             ? PA_OK
             : PA_ERR_CUDA;
}
