// Dense decode attention of a batch whose sequences share their first tokens
// (tw_prefix_decode):
//   out_b,hq = sum_{t < len_b} softmax_t(q_b,hq . k_b,t / sqrt(128)) v_b,t,
// tokens t < prefix_len being the same rows for every sequence.
//
// Mathematics.  The rows of K and V of one KV head that all sequences share
// meet the B * G query rows of that head as two matrix products,
//   S = Q K^T (M x keys),  O += P V,  P = 2^(S c - m),  c = log2(e) / sqrt(128),
// so the shared part is read once per 256 query rows instead of once per
// sequence; a sequence's own tokens meet its G rows the same way.  A softmax
// over any subset of the keys is summed up by (m, l = sum P, O); subsets are
// joined by weights 2^(m_i - m).  Each CTA takes an equal share of all key
// tiles (128 keys), writes a record (m, l, O) per row and unit it touched, and
// a second kernel joins a row's records.
//
// Pipeline.  One CTA per SM, twelve warps, two independent streams of tiles:
//   - a producer warp per stream copies K and V (page by page, 16 rows x 64
//     columns per tensor-map copy, 128-byte swizzle) into its 64 KB of buffers;
//   - a warp per stream issues tcgen05: S (128 x 128, fp32) into tensor memory,
//     and O += P V with P read from tensor memory, where it overwrites S;
//   - four warps per stream hold one query row per thread: they read S, keep
//     the running maximum and sum in registers, and write P.  O is rescaled
//     only when a row's maximum has risen by more than 2^8 (its weights still
//     fit fp16: they are scaled to at most 2^15, so that what falls below
//     fp16's normal range is below 2^-21 of the row's largest at least).
// While one stream's softmax runs, the other's products do.  With more than
// 128 query rows per KV head the two streams are two row tiles on the same K / V
// buffers, which halves the traffic; with fewer they take separate tiles of
// keys.  Tensor memory: S0 | S1 | O0 | O1, 128 columns each.
#include <cstring>

#include "tw_common.cuh"
#include "tw_kernels.h"
#include "tw_tcgen05.cuh"

namespace tw {

constexpr int kPdThreads = 384;
constexpr int kPdCtas = kTargetSms;
constexpr int kTile = 128;                      // keys per tile, query rows per stream
constexpr int kTilePages = kTile / kPage;
constexpr uint32_t kBlk = kTile * 128;          // a 64-column block of a tile: 16 KB
constexpr uint32_t kBuf = 2 * kBlk;             // a tile of Q, K or V: 32 KB
constexpr float kPdScale = 1.4426950408889634f * 0.08838834764831845f;   // log2(e) / sqrt(128)
constexpr float kLift = 7.f;                    // weights are 2^(s - m + 7), m within 2^8 of the maximum
constexpr float kSlack = 8.f;

// 2^x of two values by arithmetic, for some of the weights: the special-function
// unit's 16 exponentials per clock and SM are what bounds the softmax (128 x 128
// weights take it the 1024 clocks that the tile's two products take the tensor
// cores).  x = n + f with n the nearest integer, f in [-1/2, 1/2] and 2^f by a
// polynomial of degree 4 fitted to the least relative error, 2.6e-6: a 200th of
// the rounding to fp16 that follows.  Below 2^-125 the result is 2^-125.
__device__ __forceinline__ float2 ex2_poly(uint64_t x) {
  const float2 v = f2_unpack(x);
  x = f2_pack(fmaxf(v.x, -125.f), fmaxf(v.y, -125.f));
  const uint64_t big = f2_pack(12582912.f, 12582912.f), neg = f2_pack(-12582912.f, -12582912.f);
  const uint64_t t = f2_add(x, big);            // n in the low bits (1.5 * 2^23 + n)
  const uint64_t n = f2_add(t, neg);
  const uint64_t f = f2_fma(n, f2_pack(-1.f, -1.f), x);
  uint64_t p = f2_pack(0.00957010187736371f, 0.00957010187736371f);
  p = f2_fma(p, f, f2_pack(0.05591786178285024f, 0.05591786178285024f));
  p = f2_fma(p, f, f2_pack(0.24024744841456852f, 0.24024744841456852f));
  p = f2_fma(p, f, f2_pack(0.6931218145593883f, 0.6931218145593883f));
  p = f2_fma(p, f, f2_pack(0.9999992614376404f, 0.9999992614376404f));
  const float2 pv = f2_unpack(p), tv = f2_unpack(t);
  return make_float2(__uint_as_float(__float_as_uint(pv.x) + (__float_as_uint(tv.x) << 23)),
                     __uint_as_float(__float_as_uint(pv.y) + (__float_as_uint(tv.y) << 23)));
}

// Maxima of 32 scores, four running ones.
__device__ __forceinline__ void max32(const uint32_t* s, float* mx) {
#pragma unroll
  for (int z = 0; z < 32; z += 8)
#pragma unroll
    for (int w = 0; w < 4; ++w)
      mx[w] = max3(mx[w], __uint_as_float(s[z + 2 * w]), __uint_as_float(s[z + 2 * w + 1]));
}

struct PdRange {
  int p0, pm, p1, s0, sm, s1;   // prefix tiles [p0, pm, p1), own tiles [s0, sm, s1): stream 0 | 1
};

struct PdArgs {
  Layout L;
  const __half* q;
  int Hq, G, P, M;              // M = B * G query rows per KV head
  int pair;                     // the two streams are two row tiles (M > 128)
  int KT, RT;                   // key tiles of the prefix, 256-row tiles per KV head
  int rows1;                    // rows of a prefix record
  float* o1;                    // [slot][rows1][128]
  float2* ml1;                  // [slot][rows1] (m, l)
  float* o2;                    // [slot][G][128]
  float2* ml2;
  int* cum;                     // [B + 1] own key tiles before each sequence
  PdRange* ranges;              // [kPdCtas]
  int* status;
  __half* out;
  float* lse;
};

struct PdCtl {
  uint64_t kfull[2], vfull[2], kempty[2], vempty[2], qfull[2], sfull[2], pfull[2], ofull[2], drain;
  uint32_t tmem;
  int red[kPdThreads / 32];
  PdRange range;
  int at_b[2], at_h[2], at_t[2];   // where each stream's own tiles begin
};
constexpr size_t kPdSmem = 6 * kBuf + sizeof(PdCtl) + 1024;

__device__ __forceinline__ int own_tiles(const PdArgs& a, int b) {
  const int n = a.L.len(b) - a.P;
  return n > 0 ? (n + kTile - 1) / kTile : 0;
}

// A run of consecutive key tiles of one unit, on one stream.
struct Seg {
  bool prefix;
  int b, h, rt;        // own part: sequence and KV head; prefix: KV head and row tile
  int t0, n;           // key tiles
  int keys;            // keys of the part: P, or the sequence's own length
  int64_t slot;        // record
};

// The segments of stream i of this CTA, in order: prefix tiles, then own tiles.
struct SegIter {
  int p, pe, s, se, b, h, t;
  __device__ __forceinline__ SegIter(const PdArgs& a, const PdCtl& c, int i) {
    const PdRange& r = c.range;
    p = a.pair || i == 0 ? r.p0 : r.pm;
    pe = a.pair || i == 1 ? r.p1 : r.pm;
    s = i == 0 ? r.s0 : r.sm;
    se = i == 0 ? r.sm : r.s1;
    b = c.at_b[i];
    h = c.at_h[i];
    t = c.at_t[i];
  }
  __device__ __forceinline__ bool next(const PdArgs& a, int i, Seg& g) {
    if (p < pe) {
      const int u = p / a.KT;
      g.prefix = true;
      g.b = 0;
      g.h = u / a.RT;
      g.rt = u % a.RT;
      g.t0 = p - u * a.KT;
      g.n = min(pe - p, a.KT - g.t0);
      g.keys = a.P;
      g.slot = a.pair ? (int)blockIdx.x + u : 2 * (int)blockIdx.x + i + u;
      p += g.n;
      return true;
    }
    if (s < se) {
      // tiles are left, so a sequence with some follows (unless the lengths
      // were changed under the kernel, which ends the list here)
      while (b < a.L.B - 1 && own_tiles(a, b) == 0) ++b;
      const int kt = own_tiles(a, b);
      if (kt <= t) return false;
      g.prefix = false;
      g.b = b;
      g.h = h;
      g.rt = 0;
      g.t0 = t;
      g.n = min(se - s, kt - t);
      g.keys = a.L.len(b) - a.P;
      g.slot = (int64_t)2 * blockIdx.x + i + (int64_t)b * a.L.Hk + h;
      s += g.n;
      t = 0;
      if (++h == a.L.Hk) {
        h = 0;
        ++b;
      }
      return true;
    }
    return false;
  }
};

// Query rows of a segment that stream i holds.
__device__ __forceinline__ int seg_rows(const PdArgs& a, const Seg& g, int i) {
  if (!g.prefix) return a.G;
  const int left = a.M - g.rt * 2 * kTile - (a.pair ? i * kTile : 0);
  return left < 0 ? 0 : min(left, kTile);
}

// Which K / V buffers the k-th tile of a stream uses, and their how-manieth
// fill that is.  Paired streams share the prefix tiles, which alternate
// between the two buffer sets; other tiles use the stream's own.
struct Fill {
  int set, j;
};
__device__ __forceinline__ Fill fill_of(bool shared, int k, int i, int base) {
  return shared ? Fill{k & 1, k >> 1} : Fill{i, base + k};
}

__global__ void __launch_bounds__(kPdThreads, 1)
k_prefix_decode(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                const __grid_constant__ PdArgs a) {
  extern __shared__ unsigned char pd_smem_raw[];
  const uint32_t raw = smem_u32(pd_smem_raw);
  unsigned char* smem = pd_smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  auto q_buf = [&](int i) { return base + i * kBuf; };
  auto k_buf = [&](int i) { return base + (2 + i) * kBuf; };
  auto v_buf = [&](int i) { return base + (4 + i) * kBuf; };
  PdCtl& c = *reinterpret_cast<PdCtl*>(smem + 6 * kBuf);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  griddep_launch();   // the joining kernel waits for this grid's end by itself

  if (warp == 8) tmem_alloc(&c.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.kfull[i], 1);
      mbar_init(&c.vfull[i], 1);
      mbar_init(&c.kempty[i], 2);   // both streams, or one twice
      mbar_init(&c.vempty[i], 2);
      mbar_init(&c.qfull[i], 4);
      mbar_init(&c.sfull[i], 1);
      mbar_init(&c.pfull[i], 4);
      mbar_init(&c.ofull[i], 1);
    }
    mbar_init(&c.drain, 2);
    mbar_fence_init();
  }
  // own key tiles of all sequences, this CTA's share of all tiles
  {
    int sum = 0;
    for (int b = tid; b < a.L.B; b += kPdThreads) sum += own_tiles(a, b);
    sum = warp_sum(sum);
    if (lane == 0) c.red[warp] = sum;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kPdThreads / 32; ++w) total += c.red[w];
    const int64_t S1 = (int64_t)a.L.Hk * a.RT * a.KT, S2 = (int64_t)total * a.L.Hk;
    const int64_t X = S1 + S2;
    if (tid == 0) {
      const int64_t x0 = X * blockIdx.x / gridDim.x, x1 = X * (blockIdx.x + 1) / gridDim.x;
      PdRange r;
      r.p0 = (int)min(x0, S1);
      r.p1 = (int)min(x1, S1);
      r.s0 = (int)(max(x0, S1) - S1);
      r.s1 = (int)(max(x1, S1) - S1);
      // an odd tile goes to stream 0, of both parts to one stream each
      r.pm = r.p0 + (r.p1 - r.p0 + 1) / 2;
      r.sm = r.s0 + (r.s1 - r.s0 + (!a.pair && ((r.p1 - r.p0) & 1) ? 0 : 1)) / 2;
      c.range = r;
      a.ranges[blockIdx.x] = r;
    }
    __syncthreads();
    // sequence, head and tile at which each stream's own tiles begin
    int before = 0;
    for (int b0 = 0; b0 < a.L.B; b0 += kPdThreads) {
      const int b = b0 + tid;
      const int kt = b < a.L.B ? own_tiles(a, b) : 0;
      int incl = kt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int t = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += t;
      }
      __syncthreads();
      if (lane == 31) c.red[warp] = incl;
      __syncthreads();
      int chunk = 0, wbefore = 0;
      for (int w = 0; w < kPdThreads / 32; ++w) {
        if (w < warp) wbefore += c.red[w];
        chunk += c.red[w];
      }
      const int first = before + wbefore + incl - kt;
      if (blockIdx.x == 0 && b < a.L.B) a.cum[b] = first;
      const int64_t lo = (int64_t)first * a.L.Hk;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t s = (i == 0 ? c.range.s0 : c.range.sm) - lo;
        if (kt > 0 && s >= 0 && s < (int64_t)kt * a.L.Hk) {
          c.at_b[i] = b;
          c.at_h[i] = (int)(s / kt);
          c.at_t[i] = (int)(s % kt);
        }
      }
      before += chunk;
    }
    if (blockIdx.x == 0 && tid == 0) a.cum[a.L.B] = before;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
  }
  const uint32_t tmem = c.tmem;
  const int pairs = a.pair ? c.range.p1 - c.range.p0 : 0;   // tiles on shared buffers

  if (warp >= 10) {
    // ---- producer of buffer set i: lane 2 j + half copies that half of page j's rows
    const int i = warp - 10;
    SegIter it(a, c, i);
    Seg g;
    int k = 0;                                // tiles of this stream seen
    const int own0 = (pairs + 1 - i) / 2;     // shared fills of this set
    bool ok = true;
    int kfills = 0, vfills = 0;
    while (ok && it.next(a, i, g)) {
      const bool shared = a.pair && g.prefix;
      for (int t = g.t0; t < g.t0 + g.n; ++t, ++k) {
        if (shared && (k & 1) != i) continue;
        const int j = shared ? k >> 1 : own0 + k - pairs;
        const int np = min(kTilePages, (g.keys - t * kTile + kPage - 1) / kPage);
        const int pg = lane >> 1, half = lane & 1;
        const int lpg = (g.prefix ? 0 : a.P / kPage) + t * kTilePages + pg;
        const int row = pg < np ? (int)a.L.page_row(g.b, g.h, lpg) : 0;
        const uint32_t at = half * kBlk + pg * (kPage * 128);
        if (j > 0 && !mbar_wait(&c.kempty[i], (j - 1) & 1, a.status)) { ok = false; break; }
        if (lane == 0) mbar_arrive_tx(&c.kfull[i], np * kPage * kHeadDim * 2);
        __syncwarp();
        if (pg < np) tma_load_2d(k_buf(i) + at, &map_k, half * 64, row, &c.kfull[i]);
        kfills = j + 1;
        if (j > 0 && !mbar_wait(&c.vempty[i], (j - 1) & 1, a.status)) { ok = false; break; }
        if (lane == 0) mbar_arrive_tx(&c.vfull[i], np * kPage * kHeadDim * 2);
        __syncwarp();
        if (pg < np) tma_load_2d(v_buf(i) + at, &map_v, half * 64, row, &c.vfull[i]);
        vfills = j + 1;
      }
    }
    // copies in flight land before the CTA may end (also after a wait gave up)
    if (kfills > 0) mbar_wait(&c.kfull[i], (kfills - 1) & 1, a.status);
    if (vfills > 0) mbar_wait(&c.vfull[i], (vfills - 1) & 1, a.status);
  } else if (warp >= 8) {
    // ---- tensor-core issue of stream i
    const int i = warp - 8;
    const uint32_t s_col = tmem + i * kTile, o_col = tmem + 2 * kTile + i * kTile;
    const uint64_t q_desc = umma_desc(q_buf(i), 16, 1024);
    const int own0 = (pairs + 1 - i) / 2;
    SegIter it(a, c, i);
    Seg g;
    int k = 0, nt = 0, nseg = 0;   // tiles seen, tiles computed, segments computed
    bool ok = true;
    while (ok && it.next(a, i, g)) {
      const bool shared = a.pair && g.prefix;
      if (seg_rows(a, g, i) == 0) {
        // no rows of this stream: only hand the shared buffers on
        for (int x = 0; x < g.n && ok; ++x, ++k) {
          const Fill f = fill_of(shared, shared ? k : k - pairs, i, own0);
          ok = mbar_wait(&c.kfull[f.set], f.j & 1, a.status);
          if (ok && lane == 0) mbar_arrive(&c.kempty[f.set]);
          ok = ok && mbar_wait(&c.vfull[f.set], f.j & 1, a.status);
          if (ok && lane == 0) mbar_arrive(&c.vempty[f.set]);
          __syncwarp();
        }
        continue;
      }
      ok = mbar_wait(&c.qfull[i], nseg & 1, a.status);
      for (int x = 0; x < g.n && ok; ++x, ++k, ++nt) {
        const Fill f = fill_of(shared, shared ? k : k - pairs, i, own0);
        const int valid = min(kTile, g.keys - (g.t0 + x) * kTile);
        const int np = (valid + kPage - 1) / kPage;
        ok = mbar_wait(&c.kfull[f.set], f.j & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t kd = umma_desc(k_buf(f.set), 16, 1024);
          const uint32_t id = umma_idesc(np * kPage, false);
#pragma unroll
          for (int s = 0; s < 8; ++s) {
            const uint32_t off = (s >> 2) * (kBlk >> 4) + (s & 3) * 2;
            umma_ss(s_col, q_desc + off, kd + off, id, s > 0);
          }
          umma_commit(&c.sfull[i]);
          umma_commit(&c.kempty[f.set]);
          if (!shared) umma_commit(&c.kempty[f.set]);
        }
        __syncwarp();
        ok = mbar_wait(&c.vfull[f.set], f.j & 1, a.status);
        if (!ok) break;
        if (valid & (kPage - 1)) {
          // rows past the sequence's end meet weights of zero, whatever they
          // hold: make them zero
          const int nz = np * kPage - valid;
          for (int y = lane; y < nz * 16; y += 32) {
            const uint32_t at = v_buf(f.set) + (y & 1) * kBlk + (valid + (y >> 4)) * 128 +
                                ((y >> 1) & 7) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
          }
          fence_async_proxy();
          __syncwarp();
        }
        ok = mbar_wait(&c.pfull[i], nt & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint64_t vd = umma_desc(v_buf(f.set), kBlk, 1024);
          const uint32_t id = umma_idesc(kHeadDim, true);
          for (int s = 0; s < np; ++s)
            umma_ts(o_col, s_col + s * 8, vd + s * (2048 >> 4), id, x > 0 || s > 0);
          umma_commit(&c.vempty[f.set]);
          if (!shared) umma_commit(&c.vempty[f.set]);
          if (x == g.n - 1) umma_commit(&c.ofull[i]);
        }
        __syncwarp();
      }
      ++nseg;
    }
    // this warp's products and their arrivals are done before the CTA may end
    if (lane == 0) umma_commit(&c.drain);
    mbar_wait(&c.drain, 0, a.status);
  } else {
    // ---- softmax of stream i, one query row per thread
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                       // row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + i * kTile, o_col = tmem + lanes + 2 * kTile + i * kTile;
    SegIter it(a, c, i);
    Seg g, ng;
    int nt = 0, nseg = 0;
    bool ok = true;
    // next segment with rows on this stream; its query rows into shared memory
    auto next = [&](Seg& s) {
      while (it.next(a, i, s))
        if (seg_rows(a, s, i) > 0) return true;
      return false;
    };
    auto row_of = [&](const Seg& s, int& b, int& hq) {
      const int m = s.prefix ? (a.pair ? s.rt * 2 * kTile + i * kTile : 0) + r : r;
      b = s.prefix ? m / a.G : s.b;
      hq = s.h * a.G + (s.prefix ? m % a.G : m);
    };
    auto load_q = [&](const Seg& s) {
      if (r < seg_rows(a, s, i)) {
        int b, hq;
        row_of(s, b, hq);
        const uint4* src = reinterpret_cast<const uint4*>(a.q + ((int64_t)b * a.Hq + hq) * kHeadDim);
        const uint32_t dst = q_buf(i) + r * 128;
#pragma unroll
        for (int x = 0; x < 16; ++x) {
          const uint4 v = __ldg(src + x);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                           dst + (x >> 3) * kBlk + (((x & 7) ^ (r & 7)) * 16)),
                       "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                       : "memory");
        }
      }
      fence_async_proxy();
      __syncwarp();
      if (lane == 0) mbar_arrive(&c.qfull[i]);
    };
    bool have = next(g);
    if (have) load_q(g);
    while (have && ok) {
      const int rows = seg_rows(a, g, i);
      const bool busy = (warp & 3) * 32 < rows;   // this warp has rows
      int lim = g.keys;                            // keys this row sees
      if (g.prefix && r < rows) {
        int b, hq;
        row_of(g, b, hq);
        lim = min(lim, a.L.len(b));
      }
      float m = -INFINITY, l = 0.f;
      // raise the running maximum (log2 units) to the tile's; past kSlack, or
      // on the first tile, it is taken over and what is summed so far rescaled
      auto raise = [&](const float* mx, bool first) {
        const float top = fmaxf(m, max3(fmaxf(mx[0], mx[1]), mx[2], mx[3]) * kPdScale);
        if (first) {
          m = top;
        } else if (__any_sync(0xffffffffu, r < rows && top > m + kSlack)) {
          // S is there, so the products before it are complete: O may be rescaled
          const float f = top == -INFINITY ? 1.f : ex2(m - top);
          l *= f;
          m = top;
#pragma unroll 1
          for (int y = 0; y < 8; ++y) {
            uint32_t o[16];
            tmem_ld16(o_col + 16 * y, o);
            tmem_wait_ld();
            tmem_use16(o);
#pragma unroll
            for (int z = 0; z < 16; ++z) o[z] = __float_as_uint(__uint_as_float(o[z]) * f);
            tmem_st16(o_col + 16 * y, o);
          }
        }
      };
      // weights of 32 keys: fp16 into tensor memory, their sum to l
      auto weights32 = [&](const uint32_t* s, int y, float lift) {
        const uint64_t c2 = f2_pack(kPdScale, kPdScale), off2 = f2_pack(lift, lift);
        uint64_t sum[2] = {0, 0};
        uint32_t p[16];
#pragma unroll
        for (int z = 0; z < 16; ++z) {
          const uint64_t e = f2_fma(f2_pack(__uint_as_float(s[2 * z]), __uint_as_float(s[2 * z + 1])),
                                    c2, off2);
          float2 w;
          if (z % 4 == 3) {
            w = ex2_poly(e);
          } else {
            w = f2_unpack(e);
            w.x = ex2(w.x);
            w.y = ex2(w.y);
          }
          sum[z & 1] = f2_add(sum[z & 1], f2_pack(w.x, w.y));
          const __half2 hh = __floats2half2_rn(w.x, w.y);
          p[z] = *reinterpret_cast<const uint32_t*>(&hh);
        }
        tmem_st16(s_col + 16 * y, p);
        const float2 t = f2_unpack(f2_add(sum[0], sum[1]));
        l += t.x + t.y;
      };
      for (int x = 0; x < g.n; ++x, ++nt) {
        ok = mbar_wait(&c.sfull[i], nt & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        if (busy) {
          const int ncol = lim - (g.t0 + x) * kTile;   // keys of the tile this row sees
          if (__all_sync(0xffffffffu, ncol >= kTile)) {
            // the scores are read twice, a chunk ahead of their use: holding a
            // row of 128 would cost the registers that the exponentials need
            uint32_t s[2][32];
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            tmem_ld32(s_col, s[0]);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              tmem_wait_ld();
              tmem_use32(s[y & 1]);
              tmem_ld32(s_col + 32 * ((y + 1) & 3), s[(y + 1) & 1]);
              max32(s[y & 1], mx);
            }
            raise(mx, x == 0);
            const float lift = kLift - m;
#pragma unroll
            for (int y = 0; y < 4; ++y) {
              tmem_wait_ld();
              tmem_use32(s[y & 1]);
              if (y < 3) tmem_ld32(s_col + 32 * (y + 1), s[(y + 1) & 1]);
              weights32(s[y & 1], y, lift);   // over scores read already
            }
          } else {
            // a tile that ends early, for some row at least: chunk by chunk,
            // the scores read twice
            const int nch = min(4, (g.keys - (g.t0 + x) * kTile + 31) / 32);
            float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
            uint32_t s[32];
            auto load = [&](int y) {
              tmem_ld32(s_col + 32 * y, s);
              tmem_wait_ld();
              tmem_use32(s);
#pragma unroll
              for (int z = 0; z < 32; ++z)
                if (32 * y + z >= ncol) s[z] = __float_as_uint(-INFINITY);
            };
#pragma unroll 1
            for (int y = 0; y < nch; ++y) {
              load(y);
              max32(s, mx);
            }
            raise(mx, x == 0);
            const float lift = m == -INFINITY ? 0.f : kLift - m;
#pragma unroll 1
            for (int y = 0; y < nch; ++y) {
              load(y);
              weights32(s, y, lift);   // over scores of chunks up to y / 2: read already
            }
          }
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&c.pfull[i]);
      }
      if (!ok) break;
      // the next segment's query rows go in while this one's last product runs
      have = next(ng);
      if (have) load_q(ng);
      ok = mbar_wait(&c.ofull[i], nseg & 1, a.status);
      if (!ok) break;
      ++nseg;
      tc_fence_after();
      if (busy) {
        const int per = g.prefix ? a.rows1 : a.G;
        const int64_t at = g.slot * per + (g.prefix && a.pair ? i * kTile : 0) + r;
        float* o_dst = (g.prefix ? a.o1 : a.o2) + at * kHeadDim;
        if (r < rows) (g.prefix ? a.ml1 : a.ml2)[at] = make_float2(m - kLift, l);
#pragma unroll
        for (int y = 0; y < 4; ++y) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * y, o);
          tmem_wait_ld();
          tmem_use32(o);
          if (r < rows)
#pragma unroll
            for (int z = 0; z < 8; ++z)
              reinterpret_cast<uint4*>(o_dst + 32 * y)[z] =
                  make_uint4(o[4 * z], o[4 * z + 1], o[4 * z + 2], o[4 * z + 3]);
        }
      }
      g = ng;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_free(tmem, 512);
}

// Join a row's records: a warp per output row, four channels per lane.
constexpr int kJoinThreads = 128;

__global__ void __launch_bounds__(kJoinThreads) k_prefix_join(const __grid_constant__ PdArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t bh = (int64_t)blockIdx.x * (kJoinThreads / 32) + (threadIdx.x >> 5);
  griddep_wait();
  if (bh >= (int64_t)a.L.B * a.Hq) return;
  const int b = (int)(bh / a.Hq), hq = (int)(bh % a.Hq), h = hq / a.G, g = hq % a.G;
  const int64_t S1 = (int64_t)a.L.Hk * a.RT * a.KT;
  const int64_t X = S1 + (int64_t)__ldcg(a.cum + a.L.B) * a.L.Hk;
  float M = -INFINITY, Ls = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
  // records of tiles [first, first + n) of the prefix's (part 0) or the own
  // (part 1) list, written to slot worker + u, row `row`
#pragma unroll 1
  for (int part = 0; part < 2; ++part) {
    int64_t first, u;
    int n, per, row;
    if (part == 0) {
      const int m = b * a.G + g;
      u = (int64_t)h * a.RT + (a.pair ? m / (2 * kTile) : 0);
      first = u * a.KT;
      n = a.L.len(b) > 0 ? a.KT : 0;
      per = a.rows1;
      row = a.pair ? m % (2 * kTile) : m;
    } else {
      const int c0 = __ldcg(a.cum + b);
      n = __ldcg(a.cum + b + 1) - c0;
      u = (int64_t)b * a.L.Hk + h;
      first = (int64_t)c0 * a.L.Hk + (int64_t)h * n;
      per = a.G;
      row = g;
    }
    if (n == 0) continue;
    const int split = part == 0 && a.pair ? 1 : 2;   // records per CTA at most
    // tile x of all X lies with CTA c when X c / n_ctas <= x
    const int64_t x0 = first + (part ? S1 : 0), x1 = x0 + n - 1;
    const int c_lo = (int)(((x0 + 1) * kPdCtas + X - 1) / X - 1);
    const int c_hi = (int)(((x1 + 1) * kPdCtas + X - 1) / X - 1);
    const int nw = (c_hi - c_lo + 1) * split;
    const float2* ml = part ? a.ml2 : a.ml1;
    const float* o = part ? a.o2 : a.o1;
    for (int w0 = 0; w0 < nw; w0 += 32) {
      const int w = w0 + lane, cta = c_lo + w / split;
      float2 v = make_float2(-INFINITY, 0.f);
      int64_t at = 0;
      if (w < nw) {
        const PdRange rg = a.ranges[cta];
        int lo = part ? rg.s0 : rg.p0, hi = part ? rg.s1 : rg.p1;
        if (split == 2) {
          const int mid = part ? rg.sm : rg.pm;
          if (w % 2 == 0) hi = mid; else lo = mid;
        }
        if (max((int64_t)lo, first) < min((int64_t)hi, first + n)) {
          const int64_t slot = (split == 2 ? 2 * cta + w % 2 : cta) + u;
          at = slot * per + row;
          v = __ldcg(ml + at);
        }
      }
      const float top = fmaxf(M, warp_max(v.x));
      if (top == -INFINITY) continue;
      const float keep = M == -INFINITY ? 0.f : ex2(M - top);
      const float f = v.x == -INFINITY ? 0.f : ex2(v.x - top);
      M = top;
      Ls = Ls * keep + warp_sum(v.y * f);
      A.x *= keep;
      A.y *= keep;
      A.z *= keep;
      A.w *= keep;
      unsigned todo = __ballot_sync(0xffffffffu, f != 0.f);
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const float fs = __shfl_sync(0xffffffffu, f, src);
        const int64_t as = __shfl_sync(0xffffffffu, at, src);
        const float4 x = __ldcg(reinterpret_cast<const float4*>(o + as * kHeadDim) + lane);
        A.x = __fmaf_rn(fs, x.x, A.x);
        A.y = __fmaf_rn(fs, x.y, A.y);
        A.z = __fmaf_rn(fs, x.z, A.z);
        A.w = __fmaf_rn(fs, x.w, A.w);
      }
    }
  }
  const float inv = Ls > 0.f ? 1.f / Ls : 0.f;
  const __half2 o2[2] = {__floats2half2_rn(A.x * inv, A.y * inv),
                         __floats2half2_rn(A.z * inv, A.w * inv)};
  *reinterpret_cast<uint2*>(a.out + bh * kHeadDim + 4 * lane) = *reinterpret_cast<const uint2*>(o2);
  if (a.lse && lane == 0)
    a.lse[bh] = Ls > 0.f ? (M + log2f(Ls)) * 0.6931471805599453f : -INFINITY;
}

// Workspace: status word | CTA ranges | own tiles before each sequence |
// prefix records | own records.
struct PdPlan {
  int pair, RT, KT, rows1;
  size_t ranges, cum, ml1, o1, ml2, o2, total;
};

static PdPlan pd_plan(int B, int Hq, int Hk, int P) {
  PdPlan p;
  const int G = Hq / Hk;
  const int64_t M = (int64_t)B * G;
  p.pair = M > kTile;
  p.RT = p.pair ? (int)((M + 2 * kTile - 1) / (2 * kTile)) : 1;
  p.KT = (P + kTile - 1) / kTile;
  p.rows1 = p.pair ? 2 * kTile : (int)M;
  auto up = [](size_t x) { return (x + 255) & ~(size_t)255; };
  const size_t slots1 = P == 0 ? 0 : p.pair ? kPdCtas + (size_t)Hk * p.RT : 2 * kPdCtas + (size_t)Hk;
  const size_t slots2 = 2 * kPdCtas + (size_t)B * Hk;
  size_t at = 256;
  p.ranges = at;
  at += up(kPdCtas * sizeof(PdRange));
  p.cum = at;
  at += up(((size_t)B + 1) * sizeof(int));
  p.ml1 = at;
  at += up(slots1 * p.rows1 * sizeof(float2));
  p.o1 = at;
  at += up(slots1 * p.rows1 * kHeadDim * sizeof(float));
  p.ml2 = at;
  at += up(slots2 * G * sizeof(float2));
  p.o2 = at;
  p.total = at + up(slots2 * G * kHeadDim * sizeof(float));
  return p;
}

size_t prefix_decode_ws_bytes(int B, int Hq, int Hk, int prefix_len) {
  return pd_plan(B, Hq, Hk, prefix_len).total;
}

// cuTensorMapEncodeTiled, looked up through the runtime (the library does not
// link libcuda).
using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                 const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                 const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

static cudaError_t encode_rows(CUtensorMap* map, const __half* p, int64_t rows) {
  static std::atomic<void*> fn{nullptr};
  void* f = fn.load(std::memory_order_acquire);
  if (!f) {
    cudaDriverEntryPointQueryResult res;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000,
                                                           cudaEnableDefault, &res);
    if (e != cudaSuccess) return e;
    if (res != cudaDriverEntryPointSuccess || !f) return cudaErrorNotSupported;
    fn.store(f, std::memory_order_release);
  }
  const cuuint64_t dims[2] = {kHeadDim, (cuuint64_t)rows}, strides[1] = {kHeadDim * 2};
  const cuuint32_t box[2] = {64, kPage}, step[2] = {1, 1};
  const CUresult r = reinterpret_cast<EncodeTiled>(f)(
      map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 2, const_cast<__half*>(p), dims, strides, box, step,
      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

cudaError_t launch_prefix_decode(const Layout& L, const __half* q, int Hq, int prefix_len,
                                 const __half* K, const __half* V, __half* out, float* lse,
                                 void* ws, cudaStream_t st) {
  const PdPlan p = pd_plan(L.B, Hq, L.Hk, prefix_len);
  char* w = static_cast<char*>(ws);
  PdArgs a;
  std::memset(&a, 0, sizeof(a));
  a.L = L;
  a.q = q;
  a.Hq = Hq;
  a.G = Hq / L.Hk;
  a.P = prefix_len;
  a.M = L.B * a.G;
  a.pair = p.pair;
  a.KT = p.KT;
  a.RT = p.RT;
  a.rows1 = p.rows1;
  a.o1 = reinterpret_cast<float*>(w + p.o1);
  a.ml1 = reinterpret_cast<float2*>(w + p.ml1);
  a.o2 = reinterpret_cast<float*>(w + p.o2);
  a.ml2 = reinterpret_cast<float2*>(w + p.ml2);
  a.cum = reinterpret_cast<int*>(w + p.cum);
  a.ranges = reinterpret_cast<PdRange*>(w + p.ranges);
  a.status = reinterpret_cast<int*>(w);
  a.out = out;
  a.lse = lse;
  const int64_t rows = L.page_table ? (int64_t)L.pool_pages * L.Hk * kPage
                                    : (int64_t)L.B * L.Hk * L.N;
  cudaError_t e;
  if (rows > 0) {   // a cache without rows has no tiles: no copy uses the maps
    CUtensorMap mk, mv;
    if ((e = encode_rows(&mk, K, rows)) != cudaSuccess) return e;
    if ((e = encode_rows(&mv, V, rows)) != cudaSuccess) return e;
    static std::atomic<int> done[kMaxDevices];
    e = once_per_device(done, [] {
      return cudaFuncSetAttribute(k_prefix_decode, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)kPdSmem);
    });
    if (e != cudaSuccess) return e;
    e = launch_k(k_prefix_decode, dim3(kPdCtas), dim3(kPdThreads), kPdSmem, st, false, mk, mv, a);
    if (e != cudaSuccess) return e;
  } else if ((e = cudaMemsetAsync(a.cum, 0, ((size_t)L.B + 1) * sizeof(int), st)) != cudaSuccess) {
    return e;
  }
  const int64_t out_rows = (int64_t)L.B * Hq;
  constexpr int per = kJoinThreads / 32;
  return launch_k(k_prefix_join, dim3((unsigned)((out_rows + per - 1) / per)), dim3(kJoinThreads),
                  0, st, rows > 0, a);
}

}  // namespace tw
