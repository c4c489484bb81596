// pa_prefill_plan.cuh -- the prefill kernels' work list: items of two 128-row Q
// tiles, heaviest first, built on the host from its copies of the lengths or by
// a one-CTA kernel in the workspace.
#pragma once

#include "pa_internal.cuh"

namespace pa {
namespace {

constexpr int QT = kPrefillQTile;               // 128 query rows per Q tile
constexpr int KT = kPrefillKvTile;              // 128 keys per K/V tile

// A work item is two 128-row Q tiles that read the same keys: two q-heads of
// one kv-head (pair_heads), or two consecutive query tiles of one q-head.
struct ItemInfo {
  int seq, qt0, head0, ntiles;
  int q0, ql, L;
};

// A work list the host built from its copies of the step's lengths, passed as
// a kernel parameter (count 0: the list is in the workspace, built by
// prefill_plan_kernel).
constexpr int kParamItems = 1024;
struct PrefillWork {
  int count;
  int pad[3];
  int4 items[kParamItems];
};

__device__ __forceinline__ ItemInfo load_item(const AttnParams& p, const PrefillWork& work,
                                              int w) {
  const int4 it = work.count > 0 ? work.items[w] : p.ws_items[1 + w];
  ItemInfo r;
  r.seq = it.x; r.qt0 = it.y; r.head0 = it.z; r.ntiles = it.w;
  r.q0 = p.query_start_loc[r.seq];
  r.ql = p.query_start_loc[r.seq + 1] - r.q0;
  r.L = p.seq_lens[r.seq];
  return r;
}

// item index of the k-th item of CTA c (boustrophedon over rounds of gridDim)
__device__ __forceinline__ int item_index(int k) {
  const int g = gridDim.x, c = blockIdx.x;
  return k * g + ((k & 1) ? (g - 1 - c) : c);
}

// One CTA: list the prefill items of every sequence with q_len * group >
// decode_max_rows, heaviest (most key tiles) first (a counting sort on the tile count), and
// store the count in ws_items[0].x.  An item pairs two q-heads of one kv-head
// (pair_heads: the group is even) or two consecutive query tiles of one
// q-head; its tile count covers the later of its two query tiles.
__host__ __device__ __forceinline__ void prefill_item_range(int L, int ql, int pair_heads,
                                                            int i, int* last_row_pos) {
  const int hi_tile = pair_heads ? i : 2 * i + 1;
  const int last_row = min((hi_tile + 1) * QT, ql) - 1;
  *last_row_pos = L - ql + last_row;
}

__global__ void __launch_bounds__(1024)
prefill_plan_kernel(const AttnParams p, int max_tiles, int pair_heads) {
  extern __shared__ int hist[];  // [max_tiles + 1] counters, then running offsets
  // the prefill kernel may be launched at once: it waits for this grid before
  // it reads the work list
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
  for (int i = threadIdx.x; i <= max_tiles; i += blockDim.x) hist[i] = 0;
  __syncthreads();
  const int per_tile = pair_heads ? p.num_q_heads / 2 : p.num_q_heads;  // items per (seq, tile)
  const int lane = threadIdx.x & 31;
  // fn(sequence, item of it, key tiles): a lane reads a sequence, and its warp goes
  // over the items of those that have any
  auto for_each_item = [&](auto fn) {
    for (int s0 = threadIdx.x - lane; s0 < p.num_seqs; s0 += blockDim.x) {
      int ql = 0, L = 0;
      if (s0 + lane < p.num_seqs) {
        ql = p.query_start_loc[s0 + lane + 1] - p.query_start_loc[s0 + lane];
        L = p.seq_lens[s0 + lane];
      }
      const bool mine = !(ql * p.group <= p.decode_max_rows || ql > L);
      for (unsigned left = __ballot_sync(0xffffffffu, mine); left; left &= left - 1) {
        const int from = __ffs(left) - 1;
        const int ql1 = __shfl_sync(0xffffffffu, ql, from), L1 = __shfl_sync(0xffffffffu, L, from);
        const int nq = (ql1 + QT - 1) / QT;
        const int ni = pair_heads ? nq : (nq + 1) / 2;
        for (int i = lane; i < ni; i += 32) {
          int last;
          prefill_item_range(L1, ql1, pair_heads, i, &last);
          fn(s0 + from, i, min(last / KT + 1, max_tiles));
        }
      }
    }
  };
  // pass 1: histogram of items by tile count
  for_each_item([&](int, int, int nt) { atomicAdd(&hist[nt], per_tile); });
  __syncthreads();
  if (threadIdx.x < 32) {  // exclusive offsets, descending tile count
    int run = 0;
    for (int hi = max_tiles; hi >= 0; hi -= 32) {
      const int nt = hi - lane;
      const int c = nt >= 0 ? hist[nt] : 0;
      int sum = c;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, sum, o);
        if (lane >= o) sum += y;
      }
      if (nt >= 0) hist[nt] = run + sum - c;
      run += __shfl_sync(0xffffffffu, sum, 31);
    }
    if (lane == 0) p.ws_items[0] = make_int4(min(run, p.max_items), 0, 0, 0);
  }
  __syncthreads();
  // pass 2: scatter
  for_each_item([&](int s, int i, int nt) {
    const int at = atomicAdd(&hist[nt], per_tile);
    for (int h = 0; h < per_tile; ++h) {
      if (at + h >= p.max_items) break;
      p.ws_items[1 + at + h] = pair_heads ? make_int4(s, i, 2 * h, nt) : make_int4(s, 2 * i, h, nt);
    }
  });
}

// The work list of prefill_plan_kernel, built on the host from its copies of
// the step's lengths: the same items, heaviest first.  False when there are
// more items than a kernel parameter holds.
bool host_work_list(PrefillWork* work, const AttnParams& p, const int32_t* seq_lens_host,
                    const int32_t* query_start_loc_host, int max_tiles, int pair_heads) {
  const int per_tile = pair_heads ? p.num_q_heads / 2 : p.num_q_heads;
  static thread_local int hist[1 << 16];
  if (max_tiles + 1 > (1 << 16)) return false;
  for (int i = 0; i <= max_tiles; ++i) hist[i] = 0;
  long total = 0;
  auto for_each_item = [&](auto fn) {
    for (int s = 0; s < p.num_seqs; ++s) {
      const int ql = query_start_loc_host[s + 1] - query_start_loc_host[s];
      const int L = seq_lens_host[s];
      if (ql * p.group <= p.decode_max_rows || ql > L) continue;
      const int nq = (ql + QT - 1) / QT;
      const int ni = pair_heads ? nq : (nq + 1) / 2;
      for (int i = 0; i < ni; ++i) {
        int last;
        prefill_item_range(L, ql, pair_heads, i, &last);
        fn(s, i, min(last / KT + 1, max_tiles));
      }
    }
  };
  for_each_item([&](int, int, int nt) { hist[nt] += per_tile; total += per_tile; });
  if (total > kParamItems || total > p.max_items) return false;
  int run = 0;
  for (int nt = max_tiles; nt >= 0; --nt) {
    const int c = hist[nt];
    hist[nt] = run;
    run += c;
  }
  for_each_item([&](int s, int i, int nt) {
    int at = hist[nt];
    hist[nt] += per_tile;
    for (int h = 0; h < per_tile; ++h, ++at)
      work->items[at] = pair_heads ? make_int4(s, i, 2 * h, nt) : make_int4(s, 2 * i, h, nt);
  });
  work->count = (int)total;
  return total > 0;
}

// The work list of one launch: from the host copies when given and small
// enough (a kernel parameter), else built on the device.  *upper: at most so
// many items (num_items, when the caller knows it, is >= 0).
inline cudaError_t prefill_work_list(PrefillWork* work, int* upper, const AttnParams& p,
                                     int max_query_len, int num_items,
                                     const int32_t* seq_lens_host,
                                     const int32_t* query_start_loc_host, int pair_heads,
                                     cudaStream_t stream) {
  const int tiles = (p.max_blocks_per_seq * kBlockSize + KT - 1) / KT;
  work->count = 0;
  if (!(seq_lens_host && query_start_loc_host &&
        host_work_list(work, p, seq_lens_host, query_start_loc_host, tiles, pair_heads))) {
    work->count = 0;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(1024);
    cfg.dynamicSmemBytes = (tiles + 1) * sizeof(int);
    cfg.stream = stream;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cfg.dynamicSmemBytes > 48 * 1024) {
      static std::atomic<int> plan_smem_done[64];
      cudaError_t e = raise_smem_limit(prefill_plan_kernel, (int)cfg.dynamicSmemBytes,
                                       plan_smem_done);
      if (e != cudaSuccess) return e;
    }
    cudaError_t e = cudaLaunchKernelEx(&cfg, prefill_plan_kernel, p, tiles, pair_heads);
    if (e != cudaSuccess) return e;
  }
  *upper = work->count > 0 ? work->count
           : num_items >= 0 ? num_items
                            : (int)min((long)p.max_items,
                                       (long)p.num_seqs * ((max_query_len + QT - 1) / QT) *
                                           p.num_q_heads);
  return cudaSuccess;
}

}  // namespace
}  // namespace pa
