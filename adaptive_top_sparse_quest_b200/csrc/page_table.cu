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
// stack.  (2999 sequences, 94,000 tokens: DRAM idle, issue slots 0.6 on the SMs that
// work, the longest stalls instructions that wait for the one before and for shared
// memory.)  One launch does all: every CTA of one thread-block cluster forms the
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

// Pages that a stack of `height` (at most cap) takes of `give`.  The sum of the
// two may pass 32 bits: up to 2^31 - 1 table entries, 2^27 pages of a pool.
__host__ __device__ constexpr int pushed(int height, int give, int cap) {
  return give < cap - height ? give : cap - height;
}
constexpr int kPtMaxPool = INT32_MAX / kPage;
static_assert(pushed(kPtMaxPool, INT32_MAX, kPtMaxPool) == 0, "full stack");
static_assert(pushed(1, INT32_MAX, kPtMaxPool) == kPtMaxPool - 1, "32-bit sums");
static_assert(pushed(0, 7, 8) == 7 && pushed(3, 7, 8) == 5 && pushed(3, 0, 8) == 0, "stack room");
// strides of the loops over them stay in range as well
static_assert(kPtMaxPool <= INT32_MAX - 16 * kPtThreads, "loop index");

struct PtSmem {
  int64_t scan64[32];
  int scan32[32];
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

// The same by a whole warp, 32 probes at a time.
__device__ __forceinline__ int upper_warp(const int* end, int n, int x) {
  int lo = 0;
  while (n > 0) {   // the answer lies in [lo, lo + n]
    const int step = (n + 31) / 32, at = (threadIdx.x & 31) * step + step - 1;
    const unsigned above = __ballot_sync(0xffffffffu, at < n && end[lo + at] > x);
    // the first group whose last end is above x, or what is left past the last whole group
    const int grp = above ? __ffs(above) - 1 : n / step;
    lo += grp * step;
    n = above ? step - 1 : n - grp * step;
    if (!above && n == 0) break;
  }
  return lo;
}

__global__ void __launch_bounds__(kPtThreads) k_update_page_table(PtArgs a) {
  extern __shared__ __align__(16) unsigned char pt_smem[];
  PtSmem& sm = *reinterpret_cast<PtSmem*>(pt_smem);
  // four words per sequence, which later hold its record; then its last place + 1
  int* old_len = reinterpret_cast<int*>(pt_smem + sizeof(PtSmem));
  int* new_len = old_len + a.B;
  int* give_end = new_len + a.B;
  int* take_end = give_end + a.B;
  int* tok_end = take_end + a.B;
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
  // pages given back, in order of sequence and page, onto the stack; what would
  // pass its capacity, which only a page held twice or a length above the real one
  // can cause, is dropped
  const int given = pushed(F, give_all, a.cap), avail = F + given;
  for (int i = gt; i < given; i += nt) {
    const int b = upper(give_end, a.B, i);
    const int at = i - (b ? give_end[b - 1] : 0);
    a.free_pages[F + i] = a.page_table[(int64_t)b * a.W + pages(new_len[b]) + at];
  }
  if (cluster_size() > 1)
    cluster_sync();
  else
    __syncthreads();

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
  if (!a.slots) return;
  // what a place needs of its sequence, as one record: first place, old length
  // (below 0: no growth served), place on the stack of its first new page, old pages
  __syncthreads();
  int4 rec[kPtPer];
#pragma unroll
  for (int j = 0; j < kPtPer; ++j) {
    const int b = tid * per + j;
    if (j < per && b < a.B)
      rec[j] = make_int4(b ? tok_end[b - 1] : 0, served(b) ? old_len[b] : -1,
                         avail - 1 - (b ? take_end[b - 1] : 0), pages(old_len[b]));
  }
  __syncthreads();
  int4* recs = reinterpret_cast<int4*>(old_len);
#pragma unroll
  for (int j = 0; j < kPtPer; ++j) {
    const int b = tid * per + j;
    if (j < per && b < a.B) recs[b] = rec[j];
  }
  __syncthreads();
  // runs of four places per thread, the last threads first (the first ones have
  // the pages to move); a warp's 128 places span few sequences, which its lanes
  // find together
  const int lane = tid & 31;
  for (int64_t w0 = 128 * (int64_t)((nt - 1 - gt) >> 5); w0 < a.num_slots; w0 += 4 * nt) {
    const int b_lo = upper_warp(tok_end, a.B, (int)w0);
    const int last = (int)min(w0 + 127, (int64_t)a.num_slots - 1);
    const int b_hi = b_lo < a.B && tok_end[b_lo] <= last ? upper_warp(tok_end, a.B, last) : b_lo;
    const int i0 = (int)w0 + 4 * lane;
    if (i0 >= a.num_slots) continue;
    int b = b_lo + upper(tok_end + b_lo, b_hi - b_lo, i0);
    const int n = min(4, a.num_slots - i0);
    // where each place's page id stands, then the four loads at once (a page past
    // the old ones from the stack, not from the table entry being written)
    const int32_t* src[4];
    int row[4], out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int i = i0 + j;
      src[j] = nullptr;
      row[j] = 0;
      if (b < b_hi && tok_end[b] <= i) b += upper(tok_end + b, b_hi - b, i);
      if (j < n && b < a.B) {
        const int4 r = recs[b];
        if (i < tok_end[b] && r.y >= 0) {
          const int pos = r.y + i - r.x, pg = pos / kPage;
          row[j] = pos % kPage;
          if (pg >= a.keep)
            src[j] = pg < r.w ? a.page_table + (int64_t)b * a.W + pg : a.free_pages + r.z - (pg - r.w);
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) out[j] = src[j] ? __ldcg(src[j]) : -1;
#pragma unroll
    for (int j = 0; j < 4; ++j)
      out[j] = (unsigned)out[j] < (unsigned)a.cap ? out[j] * kPage + row[j] : -1;
    if (n == 4 && (reinterpret_cast<uintptr_t>(a.slots) & 15) == 0) {
      *reinterpret_cast<int4*>(a.slots + i0) = make_int4(out[0], out[1], out[2], out[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < n) a.slots[i0 + j] = out[j];
    }
  }
}

cudaError_t launch_update_page_table(const PtArgs& a, cudaStream_t st) {
  const size_t smem = sizeof(PtSmem) + (size_t)a.B * 5 * sizeof(int);
  static std::atomic<int> done[kMaxDevices];
  const cudaError_t e = once_per_device(done, [] {
    const cudaError_t e = cudaFuncSetAttribute(
        k_update_page_table, cudaFuncAttributeMaxDynamicSharedMemorySize,
        (int)(sizeof(PtSmem) + kPtMaxBatch * 5 * sizeof(int)));
    return e != cudaSuccess ? e
                            : cudaFuncSetAttribute(k_update_page_table,
                                                   cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // a small batch on one small block, whose barriers cost least (256 sequences of
  // a token each: 7.6 us, 9.0 on 1024 threads); a larger one on a cluster of 8
  // CTAs, or 16 (48 sequences, 48,000 tokens: 8.5 us, 10.3 on 8; 2999 sequences,
  // 94,000 tokens: 15.2 us, 20.4 on 8)
  const int64_t work = a.B + (int64_t)a.num_slots;
  const int ctas = work > 32 * kPtThreads ? 16 : work > 4 * kPtThreads ? 8 : 1;
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
