// Page tables and slot maps from request lengths (tw_update_page_table).
//
// A serving step changes the lengths of a batch: finished requests shrink to
// nothing, rejected drafts shrink by a few tokens, the others grow by a token
// or a prompt.  From the old and the new lengths alone this kernel gives the
// pages that are no longer needed back to a stack of free pages, takes pages
// for the growth from its top, enters them in the page table and writes, for
// every new token, the cache slot its K/V rows go to.  With
//   pages(n) = max(ceil(n / 16), keep)          (keep: pages of a shared prefix)
//   give_b = max(0, pages(old_b) - pages(new_b)),
//   take_b = max(0, pages(new_b) - pages(old_b)) if new_b and its slots fit, else 0
// page i that b gives goes to stack place F + sum_{b' < b} give_b' + i, and the
// j-th page that b takes comes from place A - 1 - (sum_{b' < b} take_b' + j),
// F the stack's height before and A = F + sum give.  A sequence is served when
// the takes up to and with its own do not pass A; these sums only rise, so the
// served takes are a prefix of the batch's.
//
// The work is a few hundred KB of 32-bit words at most, so what bounds it is
// latency: the launch, one round trip for the lengths, the scans, one for the
// stack.  One launch does all: every CTA of one thread-block cluster forms the
// same sums in its own shared memory (a few words per sequence, cheaper than
// exchanging them), and the cluster shares out the pages and the slots.  The
// one dependence between CTAs, that given pages are on the stack before they
// are taken from it, and that every CTA has read the lengths and the height
// before the results are written (the results may lie over them), is the
// cluster's barrier.
#include "tw_bulk.cuh"
#include "tw_common.cuh"
#include "tw_kernels.h"

namespace tw {

constexpr int kPtThreads = 1024;
constexpr int kPtPer = kPtMaxBatch / kPtThreads;   // sequences per thread in the scans

struct PtSmem {
  int64_t scan64[32];
  int scan32[32];
  // then int old_len[B], new_len[B], tok_end[B], give_end[B], take_end[B]
};

// Inclusive scan over the block's threads; *total gets the sum.  Every warp
// scans the warps' totals for itself.
template <typename T>
__device__ __forceinline__ T block_scan(T v, T* sh, T* total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += t;
  }
  __syncthreads();   // sh may still be read by an earlier scan
  if (lane == 31) sh[warp] = v;
  __syncthreads();
  T w = lane < nw ? sh[lane] : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const T t = __shfl_up_sync(0xffffffffu, w, o);
    if (lane >= o) w += t;
  }
  *total = __shfl_sync(0xffffffffu, w, nw - 1);
  const T before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
  return v + (warp ? before : 0);
}

// First index whose (ascending) end is above x; n if none.
__device__ __forceinline__ int upper(const int* end, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > x)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPtThreads) k_update_page_table(PtArgs a) {
  extern __shared__ __align__(16) unsigned char pt_smem[];
  PtSmem& sm = *reinterpret_cast<PtSmem*>(pt_smem);
  int* old_len = reinterpret_cast<int*>(pt_smem + sizeof(PtSmem));
  int* new_len = old_len + a.B;
  int* tok_end = new_len + a.B;
  int* give_end = tok_end + a.B;
  int* take_end = give_end + a.B;
  const int tid = threadIdx.x;
  const int nth = blockDim.x, nt = (int)cluster_size() * nth, gt = (int)cluster_rank() * nth + tid;
  const int room = a.W * kPage;
  auto pages = [&](int n) { return max((n + kPage - 1) / kPage, a.keep); };

  const int F = max(0, min(*a.num_free, a.cap));
  // thread t owns the per consecutive sequences from t * per
  const int per = (a.B + nth - 1) / nth;
  int64_t tok[kPtPer], tok_sum = 0, tok_all;
  int give[kPtPer], give_sum = 0, give_all;
#pragma unroll
  for (int j = 0; j < kPtPer; ++j) {
    const int b = tid * per + j;
    tok[j] = give[j] = 0;
    if (j < per && b < a.B) {
      const int o = max(0, min(a.seq_lens[b], room)), n = max(0, a.new_lens[b]);
      old_len[b] = o;
      new_len[b] = n;
      tok[j] = max(0, n - o);
      give[j] = n < o ? pages(o) - pages(n) : 0;
    }
    tok_sum += tok[j];
    give_sum += give[j];
  }
  int64_t tok_at = block_scan(tok_sum, sm.scan64, &tok_all) - tok_sum;
  int give_at = block_scan(give_sum, sm.scan32, &give_all) - give_sum;
  int take[kPtPer], take_sum = 0, take_all;
#pragma unroll
  for (int j = 0; j < kPtPer; ++j) {
    const int b = tid * per + j;
    take[j] = 0;
    if (j < per && b < a.B) {
      tok_at += tok[j];
      give_at += give[j];
      const int n = new_len[b], o = old_len[b];
      const bool fits = n <= room && (!a.slots || tok_at <= a.num_slots);
      if (!fits && n > o) new_len[b] = -1;   // growth refused: no room for it
      if (fits && n > o) take[j] = pages(n) - pages(o);
      tok_end[b] = (int)min(tok_at, (int64_t)0x7FFFFFFF);
      give_end[b] = give_at;
    }
    take_sum += take[j];
  }
  int take_at = block_scan(take_sum, sm.scan32, &take_all) - take_sum;
#pragma unroll
  for (int j = 0; j < kPtPer; ++j) {
    const int b = tid * per + j;
    if (j < per && b < a.B) {
      take_at += take[j];
      take_end[b] = take_at;
    }
  }
  __syncthreads();
  // pages given back, in order of sequence and page, onto the stack (a stack
  // that would pass its capacity, which only a page held twice can cause,
  // drops what does not fit)
  const int avail = min(F + give_all, a.cap);
  for (int i = gt; i < give_all; i += nt) {
    const int b = upper(give_end, a.B, i);
    const int at = i - (b ? give_end[b - 1] : 0);
    if (F + i < a.cap)
      a.free_pages[F + i] = a.page_table[(int64_t)b * a.W + pages(new_len[b]) + at];
  }
  cluster_sync();

  // a growth is served when the stack holds its pages and all before them
  auto served = [&](int b) {
    const int before = b ? take_end[b - 1] : 0;
    return new_len[b] > old_len[b] && (take_end[b] == before || take_end[b] <= avail);
  };
  const int last = upper(take_end, a.B, avail);   // first sequence whose takes pass the stack
  const int used = last ? take_end[last - 1] : 0;
  for (int i = gt; i < used; i += nt) {
    const int b = upper(take_end, a.B, i);
    const int at = i - (b ? take_end[b - 1] : 0);
    a.page_table[(int64_t)b * a.W + pages(old_len[b]) + at] = __ldcg(a.free_pages + avail - 1 - i);
  }
  for (int b = gt; b < a.B; b += nt) {
    const int n = new_len[b], o = old_len[b];
    a.out_lens[b] = n >= 0 && (n < o || served(b)) ? n : o;
    a.offsets[b + 1] = tok_end[b];
  }
  if (gt == 0) {
    a.offsets[0] = 0;
    *a.num_free_out = avail - used;
  }
  // a slot per new token; the page of a token past the old ones is read from
  // the stack, not from the table entry that another thread may be writing
  if (a.slots) {
    // runs of four places per thread: one search for the sequence of the first
    for (int i0 = 4 * gt; i0 < a.num_slots; i0 += 4 * nt) {
      int b = upper(tok_end, a.B, i0);
      const int n = min(4, a.num_slots - i0);
      int out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int i = i0 + j;
        int slot = -1;
        if (j < n) {
          if (b < a.B && tok_end[b] <= i) b = upper(tok_end, a.B, i);
          if (b < a.B && served(b)) {
            const int o = old_len[b], pos = o + i - (b ? tok_end[b - 1] : 0);
            const int pg = pos / kPage, have = pages(o);
            if (pg >= a.keep) {
              const int p = pg < have
                                ? a.page_table[(int64_t)b * a.W + pg]
                                : __ldcg(a.free_pages + avail - 1 -
                                         ((b ? take_end[b - 1] : 0) + pg - have));
              if ((unsigned)p < (unsigned)a.cap) slot = p * kPage + pos % kPage;
            }
          }
        }
        out[j] = slot;
      }
      if (n == 4 && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
        *reinterpret_cast<int4*>(a.slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          if (j < n) a.slots[i0 + j] = out[j];
      }
    }
  }
}

cudaError_t launch_update_page_table(const PtArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(PtSmem) + (size_t)a.B * 5 * sizeof(int);
  static std::atomic<int> done[kMaxDevices];
  const cudaError_t e = once_per_device(done, [] {
    return cudaFuncSetAttribute(k_update_page_table, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)(sizeof(PtSmem) + kPtMaxBatch * 5 * sizeof(int)));
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // a small batch on one small block: its barriers cost least; a large one on
  // a cluster of eight
  const int64_t work = a.B + (int64_t)a.num_slots;
  const int ctas = work > 4 * kPtThreads ? 8 : 1;
  cfg.gridDim = dim3(ctas);
  cfg.blockDim = dim3(work > 1024 ? kPtThreads : 256);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_update_page_table, a);
}

}  // namespace tw
