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
// joined by weights 2^(m_i - m).  Each CTA takes a stretch of the list of key
// tiles (128 keys) that costs as much as any other's, writes a record (m, l, O)
// per row and unit it touched, and a second kernel joins a row's records.
//
// Pipeline.  One CTA per SM, twelve warps, two streams of tiles:
//   - a warp per stream copies its query rows, and K and V (page by page, 16 rows
//     x 64 columns per tensor-map copy, 128-byte swizzle) into 64 KB of buffers;
//   - a warp per stream issues tcgen05: S (128 x 128, fp32) into tensor memory,
//     and O += P V with P read from tensor memory, where it overwrites S;
//   - four warps per stream hold one query row per thread: they read S twice (the
//     maximum, then the weights), and write P, the first half ahead of the second.
//     The running maximum and sum stay in registers, in fp32.  P is rounded to
//     fp16, as the products need it: 2^-11 of each weight.  (The result is off by
//     2.9e-4 of its size, rms; 2.1e-4 is its own rounding to fp16.)  O is rescaled
//     only when a row's maximum has risen by more than 2^8: the weights are lifted to
//     between 2^7 and 2^15 at the maximum, so that they fit fp16, and what falls
//     below its normal range is below 2^-21 of the row's largest.
// Segments of at most eight query rows (a sequence's own tokens, small batches)
// are turned round, keys along the tensor cores' rows: see is_thin().
// With more than 128 query rows per KV head the two streams are two row tiles on
// the same K / V buffers, which halves the traffic, and one stream's softmax runs
// while the other's products do; with fewer they take separate tiles of keys.
// Tensor memory: S0 | S1 | O0 | O1, 128 columns each.
//
// What bounds it (one B200; whole calls, in us, in a loop of them):
//   - few query rows (16 sequences of 1000 .. 9000 tokens, nothing shared): HBM;
//     307 MB take 59, 57.7 of them the tile kernel (0.81 of the measured copy rate);
//   - 512 rows per head (128 sequences behind 128k tokens): a CTA takes 353 thousand
//     clocks, in which the tensor cores are busy for 227 (a tile of 256 rows 2930, its
//     products 2048); K and V are read once per 256 rows, twice here (1.15 GB).  Single
//     launches take 226 at 1.6 GHz; calls 278 in a loop of 50 ms, 325 in one of seconds,
//     where the 1000 W cap holds the clock at 1.2 .. 1.3 GHz: 0.85 PFLOP/s;
//   - 256 rows (64 behind 32k): 64, and 70 in a loop of seconds (power cap, 1.7 GHz).
//     82 CTAs hold prefix tiles only, bound by the products and the softmax, 65 own
//     tiles only, which move 34 bytes per ns each (36 in the first case above), with
//     HBM at two thirds of the copy rate;
//   - many short own parts (16 sequences of a multi-head layer): 47, 31 by bytes; 45 CTAs
//     hold prefix tiles, whose 16 rows take the form of 128, and 102 own tiles;
//   - small calls (15 .. 18): latency: set-up 2, first copies 2, a tile's chain 2,
//     the records and the join 6.
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
constexpr float kNone = -1e38f;                 // running maximum before a finite score
constexpr int kThin = 8;                        // query rows of a thin segment at most
constexpr int kThinCols = 16;                   // columns of its products (the least there are)

// 2^x of two values by arithmetic, for a quarter of the weights: the special-
// function unit gives 16 exponentials per clock and SM, so that 128 x 128 weights
// take it the 1024 clocks that the tile's two products take the tensor cores
// (64 sequences behind 128k tokens: 129 us; 138 with none by arithmetic, 132 with
// half).  x = n + f with n the nearest integer, f in [-1/2, 1/2] and 2^f by a
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
  const __half *q, *K, *V;
  int Hq, G, P, M;              // M = B * G query rows per KV head
  int pair;                     // the two streams are two row tiles (M > 128)
  int KT, RT;                   // key tiles of the prefix, 256-row tiles per KV head
  int rows1;                    // rows of a prefix record
  float* o1;                    // [slot][rows1][128]
  float2* ml1;                  // [slot][rows1] (m, l)
  float* o2;                    // [slot][G][128]
  float2* ml2;
  uint64_t* cum;                // [B + 1] sequences with own tiles (high half) and own tiles before each
  PdRange* ranges;              // [kPdCtas]
  int* status;
  __half* out;
  float* lse;
};

// What the four softmax warps of a stream exchange over a thin segment.
struct PdThin {
  float x[4][kThin];     // a value per warp and row: maxima, at the end sums
  float m[kThin];
  int lim[kThin];        // keys a row sees
  int b;                 // sequence of an own part
};

struct PdCtl {
  uint64_t kfull[2], vfull[2], kempty[2], vempty[2];   // per buffer set
  uint64_t qfull[2], qempty[2];                        // per stream: query rows,
  uint64_t sfull[2], phalf[2], pfull[2], ofull[2];     // S, P's first half, P, a segment's O
  uint64_t shared_done, drain;
  uint32_t tmem;
  uint64_t red[kPdThreads / 32];
  PdRange range;
  int at_b[2], at_h[2], at_t[2];   // where each stream's own tiles begin
  PdThin thin[2];
};
constexpr uint32_t kPdCtlBytes = 1280;
static_assert(sizeof(PdCtl) <= kPdCtlBytes, "control block");
// Q, K, V tiles of both streams | 4 KB per softmax warp to write records through,
// a thin segment's P at the head of each stream's | control block | alignment to 1 KB
constexpr uint32_t kStage = 4096;
constexpr size_t kPdSmem = 6 * kBuf + 8 * kStage + kPdCtlBytes + 1024;
static_assert(kPdSmem <= 227 * 1024, "shared memory");

__device__ __forceinline__ int own_tiles(const PdArgs& a, int b) {
  const int n = a.L.len(b) - a.P;
  return n > 0 ? (n + kTile - 1) / kTile : 0;
}

// The CTAs share the tiles out by cost, on one line: the prefix's units, each a
// start (query rows, record) and KT tiles, then the own parts' units (sequence
// by sequence, head by head) likewise.  Costs are in sixths of the time of a
// tile that only waits for its copy; a pair's tile of 256 query rows takes half
// as long again.  (64 sequences behind 32k tokens: 59 us, 68 with every tile
// alike; 16 of a multi-head layer, many short units: 41 us, 47 without starts.)
constexpr int kOwnCost = 6, kOwnStart = 2, kUnitStart = 12;
__host__ __device__ __forceinline__ int tile_cost(const PdArgs& a) { return a.pair ? 9 : 6; }
__host__ __device__ __forceinline__ int unit_span(const PdArgs& a) {
  return a.KT * tile_cost(a) + kUnitStart;
}
__device__ __forceinline__ int64_t prefix_span(const PdArgs& a) {
  return a.KT > 0 ? (int64_t)a.L.Hk * a.RT * unit_span(a) : 0;
}
// Cost per KV head of (sequences, own tiles).
__device__ __forceinline__ int64_t own_cost(uint64_t v) {
  return (int64_t)(v >> 32) * kOwnStart + (int64_t)(uint32_t)v * kOwnCost;
}
// First prefix tile that lies at x or after it.
__device__ __forceinline__ int prefix_tile_at(const PdArgs& a, int64_t x) {
  if (x <= 0) return 0;
  const uint32_t span = unit_span(a);
  const int64_t u = (uint64_t)x >> 32 ? x / span : (uint32_t)x / span;
  const int in = (int)(x - u * span) - kUnitStart, cost = tile_cost(a);
  return (int)(u * a.KT) + (in <= 0 ? 0 : (in + cost - 1) / cost);
}

// A value that is the same in all lanes, in a form that lets the compiler know:
// it then keeps operand descriptors in uniform registers.
__device__ __forceinline__ uint32_t uni(uint32_t x) { return __shfl_sync(0xffffffffu, x, 0); }

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
    return s < se && take(a, i, find(a), g);
  }
  // Keys of the next own sequence that has some (0: none is left, although tiles
  // are: the lengths were changed under the kernel, which ends the list).
  __device__ __forceinline__ int find(const PdArgs& a) {
    for (; b < a.L.B; ++b) {
      const int keys = (int)uni(a.L.len(b)) - a.P;
      if (keys > 0) return keys;
    }
    return 0;
  }
  // Its tiles from here.  They follow from that one reading of its length, so that a
  // segment's tiles and keys agree whatever happens to it.
  __device__ __forceinline__ bool take(const PdArgs& a, int i, int keys, Seg& g) {
    const int kt = (keys + kTile - 1) / kTile;
    if (kt <= t) return false;
    g.prefix = false;
    g.b = b;
    g.h = h;
    g.rt = 0;
    g.t0 = t;
    g.n = min(se - s, kt - t);
    g.keys = keys;
    g.slot = (int64_t)2 * blockIdx.x + i + (int64_t)b * a.L.Hk + h;
    s += g.n;
    t = 0;
    if (++h == a.L.Hk) {
      h = 0;
      ++b;
    }
    return true;
  }
};

// First of the M = B * G query rows of a KV head that stream i holds (prefix).
__device__ __forceinline__ int first_row(const PdArgs& a, const Seg& g, int i) {
  return a.pair ? g.rt * 2 * kTile + i * kTile : 0;
}

// Query rows of a segment that stream i holds.
__device__ __forceinline__ int seg_rows(const PdArgs& a, const Seg& g, int i) {
  if (!g.prefix) return a.G;
  const int left = a.M - g.rt * 2 * kTile - (a.pair ? i * kTile : 0);
  return left < 0 ? 0 : min(left, kTile);
}

// Segments of at most kThin query rows are turned round: S^T = K Q^T and
// O^T += V^T P^T, keys and then channels along the tensor cores' 128 rows and the
// query rows along 16 columns.  A product then costs a quarter or less (it is
// bound by reading K or V from shared memory, 256 clocks a tile) and the softmax
// has a key per thread instead of a row of 128 keys.  Eight covers every own part
// (G <= 8) in registers a thread has left.  (16 sequences, nothing shared: 58.2 us,
// 61.5 with one form for all; 64 behind 32k tokens: 71.5, 76.)
__device__ __forceinline__ bool is_thin(const PdArgs& a, const Seg& g) {
  return !g.prefix || (!a.pair && a.M <= kThin);
}

// A record's maximum, of the weights without their lift; minus infinity: no record.
__device__ __forceinline__ float record_max(float m) { return m == kNone ? -INFINITY : m - kLift; }

__global__ void __launch_bounds__(kPdThreads, 1)
k_prefix_decode(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_q1,
                const __grid_constant__ PdArgs a) {
  extern __shared__ unsigned char pd_smem_raw[];
  const uint32_t raw = smem_u32(pd_smem_raw);
  unsigned char* smem = pd_smem_raw + ((1024 - (raw & 1023)) & 1023);
  const uint32_t base = smem_u32(smem);
  auto q_buf = [&](int i) { return base + i * kBuf; };
  auto k_buf = [&](int i) { return base + (2 + i) * kBuf; };
  auto v_buf = [&](int i) { return base + (4 + i) * kBuf; };
  auto p_buf = [&](int i) { return base + 6 * kBuf + 4 * i * kStage; };
  PdCtl& c = *reinterpret_cast<PdCtl*>(smem + 6 * kBuf + 8 * kStage);
  const int tid = threadIdx.x, lane = tid & 31, warp = (int)uni(tid >> 5);
  griddep_launch();   // the joining kernel waits for this grid's end by itself

  if (warp == 8) tmem_alloc(&c.tmem, 512);
  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&c.kfull[i], 1);
      mbar_init(&c.vfull[i], 1);
      mbar_init(&c.kempty[i], 2);   // both streams, or one twice
      mbar_init(&c.vempty[i], 2);
      mbar_init(&c.qfull[i], 1);
      mbar_init(&c.qempty[i], 1);
      mbar_init(&c.sfull[i], 1);
      mbar_init(&c.pfull[i], 4);
      mbar_init(&c.phalf[i], 4);
      mbar_init(&c.ofull[i], 1);
    }
    mbar_init(&c.shared_done, 1);
    mbar_init(&c.drain, 2);
    mbar_fence_init();
  }
  griddep_wait();   // what follows reads and writes memory
  // own key tiles of all sequences, this CTA's stretch of the line of costs, and
  // the tiles at its ends and its middle
  {
    // inclusive sum over the block of (sequences with own tiles, own tiles), 32 bits each
    auto block_incl = [&](uint64_t v, uint64_t* all) {
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint64_t t = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += t;
      }
      if (lane == 31) c.red[warp] = v;
      __syncthreads();
      *all = 0;
#pragma unroll
      for (int w = 0; w < kPdThreads / 32; ++w) {
        const uint64_t x = c.red[w];
        if (w < warp) v += x;
        *all += x;
      }
      return v;
    };
    auto tiles_of = [&](int b) {
      const int kt = own_tiles(a, b);
      return kt > 0 ? (1ull << 32) | (uint64_t)kt : 0ull;
    };
    uint64_t sum = 0, total;
    for (int b = tid; b < a.L.B; b += kPdThreads) sum += tiles_of(b);
    const uint64_t incl0 = block_incl(sum, &total);
    const int64_t X1 = prefix_span(a), X = X1 + own_cost(total) * a.L.Hk;
    const int64_t x0 = X * blockIdx.x / kPdCtas, x1 = X * (blockIdx.x + 1) / kPdCtas;
    // paired streams share the prefix's tiles and halve the own ones; others halve
    // the whole stretch
    const int64_t xm = a.pair ? (max(x0, X1) + max(x1, X1)) / 2 : (x0 + x1) / 2;
    const int64_t at[3] = {max(x0, X1) - X1, max(xm, X1) - X1, max(x1, X1) - X1};
    if (tid == 0) {
      PdRange r;
      r.p0 = prefix_tile_at(a, min(x0, X1));
      r.p1 = prefix_tile_at(a, min(x1, X1));
      r.pm = a.pair ? r.p1 : prefix_tile_at(a, min(xm, X1));
      r.s0 = r.sm = r.s1 = (int)(uint32_t)total * a.L.Hk;   // past the last, unless found below
      c.range = r;
      for (int k = 0; k < 2; ++k) c.at_b[k] = c.at_h[k] = c.at_t[k] = 0;
    }
    __syncthreads();
    uint64_t before = 0;
    for (int b0 = 0; b0 < a.L.B; b0 += kPdThreads) {
      const int b = b0 + tid;
      uint64_t mine = sum, incl = incl0, chunk = total;
      if (a.L.B > kPdThreads) {   // else the sums above are these
        mine = b < a.L.B ? tiles_of(b) : 0;
        __syncthreads();
        incl = block_incl(mine, &chunk);
      }
      const uint64_t first = before + incl - mine;
      if (blockIdx.x == 0 && b < a.L.B) a.cum[b] = first;
      const int kt = (int)(uint32_t)mine, cost = (int)own_cost(mine);
      const int64_t lo = own_cost(first) * a.L.Hk;
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int64_t off = at[k] - lo;
        if (off >= 0 && off < (int64_t)cost * a.L.Hk) {
          int h = (int)off / cost;
          const int in = (int)off - h * cost - kOwnStart;
          int t = in <= 0 ? 0 : (in + kOwnCost - 1) / kOwnCost;
          const int tile = (int)(uint32_t)first * a.L.Hk + h * kt + t;
          if (t == kt) {   // the next unit's start
            t = 0;
            ++h;
          }
          if (k == 0) c.range.s0 = tile;
          if (k == 1) c.range.sm = tile;
          if (k == 2) c.range.s1 = tile;
          if (k < 2) {
            c.at_b[k] = h == a.L.Hk ? b + 1 : b;
            c.at_h[k] = h == a.L.Hk ? 0 : h;
            c.at_t[k] = t;
          }
        }
      }
      before += chunk;
    }
    if (blockIdx.x == 0 && tid == 0) a.cum[a.L.B] = before;
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (tid == 0) a.ranges[blockIdx.x] = c.range;
  }
  const uint32_t tmem = uni(c.tmem);
  const int pairs = a.pair ? c.range.p1 - c.range.p0 : 0;   // tiles on shared buffers

  if (warp >= 10) {
    // ---- producer of stream i's query rows and of buffer set i, which paired
    // streams' shared tiles take in turn: lane 2 j + half copies that half of
    // page j's rows
    const int i = warp - 10;
    SegIter it(a, c, i);
    Seg g;
    int k = 0;                                // tiles of this stream seen
    const int own0 = (pairs + 1 - i) / 2;     // shared fills of this set
    bool ok = true;
    int kfills = 0, vfills = 0, nseg = 0;
    while (ok && it.next(a, i, g)) {
      const bool shared = a.pair && g.prefix;
      if (seg_rows(a, g, i) > 0) {
        // the segment's query rows: 128 of the M of its KV head, or a sequence's G
        const int rows = g.prefix ? kTile : a.G;
        const int b = g.prefix ? first_row(a, g, i) / a.G : g.b;
        if (nseg > 0 && !mbar_wait(&c.qempty[i], (nseg - 1) & 1, a.status)) break;
        if (lane == 0) mbar_arrive_tx(&c.qfull[i], rows * kHeadDim * 2);
        __syncwarp();
        if (lane < 2)
          tma_load_3d(q_buf(i) + lane * kBlk, g.prefix ? &map_q : &map_q1, lane * 64, g.h * a.G, b,
                      &c.qfull[i]);
        ++nseg;
      }
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
    if (nseg > 0) mbar_wait(&c.qfull[i], (nseg - 1) & 1, a.status);
    // copies in flight land before the CTA may end (also after a wait gave up)
    if (kfills > 0) mbar_wait(&c.kfull[i], (kfills - 1) & 1, a.status);
    if (vfills > 0) mbar_wait(&c.vfull[i], (vfills - 1) & 1, a.status);
  } else if (warp >= 8) {
    // ---- tensor-core issue.  Paired streams' shared tiles are issued by the
    // first warp alone: what it issues runs in order, a stream's O += P V and
    // next S as a block, while the other stream's softmax runs.  (Two warps'
    // products take turns one by one, both streams' end late, and their softmax
    // run, and wait, at the same time.)  Other tiles are bound by the copies:
    // a warp per stream, so that neither waits for the other's.
    const int i = warp - 8;
    bool ok = true;
    auto issue_s = [&](const int i, uint32_t set, uint32_t np) {   // S = Q K^T
      const uint32_t s_col = tmem + i * kTile;
      const uint64_t qd = umma_desc(q_buf(i), 16, 1024), kd = umma_desc(k_buf(set), 16, 1024);
      const uint32_t id = umma_idesc(np * kPage, false, false);
      umma_ss4(s_col, qd, kd, id, 0);
      umma_ss4(s_col, qd + (kBlk >> 4), kd + (kBlk >> 4), id, 1);
      umma_commit(&c.sfull[i]);
    };
    // thin: S^T = K Q^T, O^T += V^T P^T
    auto issue_s_thin = [&](const int i) {
      const uint64_t qd = umma_desc(q_buf(i), 16, 1024), kd = umma_desc(k_buf(i), 16, 1024);
      const uint32_t id = umma_idesc(kThinCols, false, false);
      umma_ss4(tmem + i * kTile, kd, qd, id, 0);
      umma_ss4(tmem + i * kTile, kd + (kBlk >> 4), qd + (kBlk >> 4), id, 1);
      umma_commit(&c.sfull[i]);
    };
    auto issue_o_thin = [&](const int i, uint32_t np, uint32_t more) {
      const uint64_t vd = umma_desc(v_buf(i), kBlk, 1024), pd = umma_desc(p_buf(i), 16, 1024);
      const uint32_t id = umma_idesc(kThinCols, true, false);
      // 16 keys at a time: a quarter of P's 64-key blocks of 16 rows
      for (uint32_t y = 0; y < np; ++y)
        umma_ss(tmem + 2 * kTile + i * kTile, vd + y * (2048 >> 4),
                pd + (y >> 2) * (kThinCols * 128 >> 4) + (y & 3) * 2, id, more | y);
    };
    // O += P V, the first or second 64 keys: the first while the softmax is at the others
    auto issue_o = [&](const int i, uint32_t set, uint32_t np, uint32_t more, const int half) {
      const uint32_t s_col = tmem + i * kTile, o_col = tmem + 2 * kTile + i * kTile;
      const uint64_t vd = umma_desc(v_buf(set), kBlk, 1024);
      const uint32_t id = umma_idesc(kHeadDim, false, true);
      const uint32_t y0 = half * (kTilePages / 2), y1 = half ? np : min(np, (uint32_t)kTilePages / 2);
      if (y1 == y0 + kTilePages / 2) {
        umma_ts4(o_col, s_col + half * 32, vd + half * 4 * (2048 >> 4), id, half ? 1 : more);
      } else {
        for (uint32_t y = y0; y < y1; ++y)
          umma_ts(o_col, s_col + y * 8, vd + y * (2048 >> 4), id, more | y);
      }
    };
    SegIter it(a, c, i);
    Seg g;
    int nt = 0, nseg = 0;   // tiles and segments of this stream so far
    if (a.pair) {
      int k = 0, nt1 = 0, nseg1 = 0;
      while (ok && it.p < it.pe && it.next(a, i, g)) {
        const uint32_t two = uni(seg_rows(a, g, 1) > 0);   // the second stream has rows
        if (i == 0) {
          auto pages = [&](int x) {
            return uni(min(kTilePages, (g.keys - (g.t0 + x) * kTile + kPage - 1) / kPage));
          };
          uint32_t set = uni(k & 1), np = pages(0);
          ok = mbar_wait(&c.kfull[set], (k >> 1) & 1, a.status) &&
               mbar_wait(&c.qfull[0], nseg & 1, a.status);
          if (!ok) break;
          tc_fence_after();
          issue_s(0, set, np);
          umma_commit(&c.kempty[set]);
          if (two) {
            ok = mbar_wait(&c.qfull[1], nseg1 & 1, a.status);
            if (!ok) break;
            tc_fence_after();
            issue_s(1, set, np);
          }
          umma_commit(&c.kempty[set]);
          for (int x = 0; x < g.n; ++x, ++k) {
            const uint32_t last = uni(x == g.n - 1), more = uni(x > 0);
            const uint32_t set_n = uni((k + 1) & 1), np_n = last ? 0 : pages(x + 1);
            const int par_n = ((k + 1) >> 1) & 1;
            ok = mbar_wait(&c.vfull[set], (k >> 1) & 1, a.status);
            if (!ok) break;
            for (int j = 0; j < 1 + (int)two; ++j) {
              ok = mbar_wait(&c.phalf[j], (j ? nt1 + x : nt + x) & 1, a.status);
              if (!ok) break;
              tc_fence_after();
              issue_o(j, set, np, more, 0);
              ok = mbar_wait(&c.pfull[j], (j ? nt1 + x : nt + x) & 1, a.status);
              if (!ok) break;
              tc_fence_after();
              issue_o(j, set, np, more, 1);
              umma_commit(&c.vempty[set]);
              if (!two) umma_commit(&c.vempty[set]);
              if (last) {
                umma_commit(&c.qempty[j]);
                umma_commit(&c.ofull[j]);
              } else {
                if (j == 0) ok = mbar_wait(&c.kfull[set_n], par_n, a.status);
                if (!ok) break;
                tc_fence_after();
                issue_s(j, set_n, np_n);
                umma_commit(&c.kempty[set_n]);
                if (!two) umma_commit(&c.kempty[set_n]);
              }
            }
            if (!ok) break;
            set = set_n;
            np = np_n;
          }
        }
        nt += i == 0 || two ? g.n : 0;
        nseg += i == 0 || two ? 1 : 0;
        nt1 += two ? g.n : 0;
        nseg1 += two ? 1 : 0;
      }
      // the second warp goes on with its stream when its shared tiles are done
      if (i == 0)
        umma_commit(&c.shared_done);
      else
        ok = mbar_wait(&c.shared_done, 0, a.status);
    }
    int j = (pairs + 1 - i) / 2;   // fills of this stream's buffers so far
    while (ok && it.next(a, i, g)) {
      const uint32_t thin = uni(is_thin(a, g));
      ok = mbar_wait(&c.qfull[i], nseg & 1, a.status);
      for (int x = 0; x < g.n && ok; ++x, ++j, ++nt) {
        const int valid = min(kTile, g.keys - (g.t0 + x) * kTile);
        const uint32_t np = uni((valid + kPage - 1) / kPage);
        const uint32_t last = uni(x == g.n - 1), more = uni(x > 0);
        ok = mbar_wait(&c.kfull[i], j & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        if (thin)
          issue_s_thin(i);
        else
          issue_s(i, i, np);
        umma_commit(&c.kempty[i]);
        umma_commit(&c.kempty[i]);
        if (last) umma_commit(&c.qempty[i]);
        ok = mbar_wait(&c.vfull[i], j & 1, a.status);
        if (!ok) break;
        if (!thin) {
          ok = mbar_wait(&c.phalf[i], nt & 1, a.status);
          if (!ok) break;
          tc_fence_after();
          issue_o(i, i, np, more, 0);
        } else if (valid & (kPage - 1)) {
          // rows past a sequence's end meet weights of zero, whatever they hold:
          // make them zero (the prefix ends with a page)
          const int nz = (int)np * kPage - valid;
          for (int y = lane; y < nz * 16; y += 32) {
            const uint32_t at = v_buf(i) + (y & 1) * kBlk + (valid + (y >> 4)) * 128 +
                                ((y >> 1) & 7) * 16;
            asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(at), "r"(0) : "memory");
          }
          fence_async_proxy();
          __syncwarp();
        }
        ok = mbar_wait(&c.pfull[i], nt & 1, a.status);
        if (!ok) break;
        tc_fence_after();
        if (thin)
          issue_o_thin(i, np, more);
        else
          issue_o(i, i, np, more, 1);
        umma_commit(&c.vempty[i]);
        umma_commit(&c.vempty[i]);
        if (last) umma_commit(&c.ofull[i]);
      }
      ++nseg;
    }
    // this warp's products and their arrivals are done before the CTA may end
    umma_commit(&c.drain);
    mbar_wait(&c.drain, 0, a.status);
  } else {
    // ---- softmax of stream i, one query row per thread (or, thin, one key).  No
    // step depends on a wait's success: the stream's warps meet at barriers
    const int i = warp >> 2;
    const int r = (warp & 3) * 32 + lane;                       // row of the tile
    const uint32_t lanes = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + i * kTile, o_col = tmem + lanes + 2 * kTile + i * kTile;
    SegIter it(a, c, i);
    Seg g;
    int nt = 0, nseg = 0;
    bool ok = true;
    // a thin segment: thread `key` holds that key's scores (then that channel's O) of
    // all rows, every thread the rows' maxima and its share of their sums
    const int w4 = warp & 3, key = r, meet = 1 + i;   // hardware barrier of the four warps
    PdThin& th = c.thin[i];
    // Next segment with rows on this stream; a thin one's limits.  The four warps meet
    // at barriers in a thin segment, so they have to agree on it whatever happens to
    // the lengths in memory: one of them reads them for all.
    auto next = [&](Seg& s) {
      while (it.p < it.pe) {
        it.next(a, i, s);
        const int rows = seg_rows(a, s, i);
        if (rows == 0) continue;
        if (is_thin(a, s)) {
          if (w4 == 0 && lane < kThin)
            th.lim[lane] = lane < rows ? min(s.keys, a.L.len(lane / a.G)) : s.keys;
          bar_sync(meet, 128);
        }
        return true;
      }
      if (it.s >= it.se) return false;
      if (w4 == 0) {
        const int keys = it.find(a);
        if (lane < kThin) th.lim[lane] = keys;
        if (lane == 0) th.b = it.b;
      }
      bar_sync(meet, 128);   // and P's memory is free of earlier records
      it.b = th.b;
      return it.take(a, i, th.lim[0], s);
    };
    auto thin_seg = [&]() {
      constexpr int NR = kThin;
      const int rows = seg_rows(a, g, i);
      int low = g.keys;      // keys that every row sees
      float m[NR], l[NR];
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        low = min(low, th.lim[n]);
        m[n] = kNone;
        l[n] = 0.f;
      }
      for (int x = 0; x < g.n; ++x, ++nt) {
        ok = ok && mbar_wait(&c.sfull[i], nt & 1, a.status);
        tc_fence_after();
        uint32_t s[16];
        tmem_ld16(s_col, s);
        tmem_wait_ld();
        tmem_use16(s);
        const int at = (g.t0 + x) * kTile + key;
        if ((g.t0 + x + 1) * kTile > low) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
            if (at >= th.lim[n]) s[n] = __float_as_uint(-INFINITY);
        }
        float top[NR];
        bool up = x == 0;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          top[n] = max2(m[n], redux_max(__uint_as_float(s[n])) * kPdScale);
          up |= n < rows && !(top[n] <= m[n] + kSlack);
        }
        // (on the first tile it is true for all, and the barrier free of others' records)
        if (bar_any(meet, 128, up)) {
#pragma unroll
          for (int n = 0; n < NR; ++n)
            if (lane == n) th.x[w4][n] = top[n];
          bar_sync(meet, 128);
          float f[NR];
#pragma unroll
          for (int n = 0; n < NR; ++n) {
            const float t = max2(max3(th.x[0][n], th.x[1][n], th.x[2][n]), th.x[3][n]);
            f[n] = ex2(m[n] - t);
            l[n] *= f[n];
            m[n] = t;
          }
          if (x > 0) {   // S is there, so the products before it are complete
            uint32_t o[16];
            tmem_ld16(o_col, o);
            tmem_wait_ld();
            tmem_use16(o);
#pragma unroll
            for (int n = 0; n < NR; ++n) o[n] = __float_as_uint(__uint_as_float(o[n]) * f[n]);
            tmem_st16(o_col, o);
            tmem_wait_st();
          }
        }
        // this key's weights: fp16, a column of P (rows of 64 keys, swizzled)
        const uint32_t dst = p_buf(i) + (key >> 6) * (kThinCols * 128) + (key & 7) * 2;
#pragma unroll
        for (int n = 0; n < NR; ++n) {
          const float p = ex2(__fmaf_rn(__uint_as_float(s[n]), kPdScale, kLift - m[n]));
          l[n] += p;
          asm volatile("st.shared.u16 [%0], %1;" ::"r"(
                           dst + n * 128 + ((((key & 63) >> 3) ^ (n & 7)) * 16)),
                       "h"(__half_as_ushort(__float2half_rn(p)))
                       : "memory");
        }
        fence_async_proxy();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&c.phalf[i]);
          mbar_arrive(&c.pfull[i]);
        }
      }
      ok = ok && mbar_wait(&c.ofull[i], nseg & 1, a.status);
      ++nseg;
      tc_fence_after();
#pragma unroll
      for (int n = 0; n < NR; ++n) {
        const float sum = warp_sum(l[n]);
        if (lane == n) {
          th.x[w4][n] = sum;
          if (w4 == 0) th.m[n] = m[n];
        }
      }
      bar_sync(meet, 128);
      const int64_t at = g.slot * (g.prefix ? a.rows1 : a.G);
      if (w4 == 0 && lane < rows)
        (g.prefix ? a.ml1 : a.ml2)[at + lane] =
            make_float2(record_max(th.m[lane]),
                        (th.x[0][lane] + th.x[1][lane]) + (th.x[2][lane] + th.x[3][lane]));
      float* o_dst = (g.prefix ? a.o1 : a.o2) + at * kHeadDim + key;
      uint32_t o[16];
      tmem_ld16(o_col, o);
      tmem_wait_ld();
      tmem_use16(o);
#pragma unroll
      for (int n = 0; n < NR; ++n)
        if (n < rows) o_dst[n * kHeadDim] = __uint_as_float(o[n]);
    };
    while (next(g)) {
      if (is_thin(a, g)) {
        thin_seg();
        continue;
      }
      const int rows = seg_rows(a, g, i);
      const bool busy = (warp & 3) * 32 < rows;   // this warp has rows
      int lim = g.keys;                            // keys this row sees (of the prefix)
      if (r < rows) lim = min(lim, a.L.len((first_row(a, g, i) + r) / a.G));
      float m = kNone, l = 0.f;
      // raise the running maximum (log2 units) to the tile's; past kSlack, or
      // on the first tile, it is taken over and what is summed so far rescaled
      auto raise = [&](const float* mx, bool first) {
        const float top = max2(m, max3(max2(mx[0], mx[1]), mx[2], mx[3]) * kPdScale);
        if (first) {
          m = top;
        } else if (__any_sync(0xffffffffu, r < rows && !(top <= m + kSlack))) {
          // S is there, so the products before it are complete: O may be rescaled
          const float f = ex2(m - top);
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
        ok = ok && mbar_wait(&c.sfull[i], nt & 1, a.status);
        tc_fence_after();
        bool half = false;   // the first 64 keys' weights are handed over
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
              if (y == 1) {
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c.phalf[i]);
                half = true;
              }
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
            const float lift = kLift - m;
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
        if (lane == 0) {
          if (!half) mbar_arrive(&c.phalf[i]);
          mbar_arrive(&c.pfull[i]);
        }
      }
      ok = ok && mbar_wait(&c.ofull[i], nseg & 1, a.status);
      ++nseg;
      tc_fence_after();
      if (busy) {
        const int64_t at = g.slot * a.rows1 + (a.pair ? i * kTile : 0);
        if (r < rows) a.ml1[at + r] = make_float2(record_max(m), l);
        // 32 columns of the warp's rows at a time, through shared memory, so that
        // eight lanes write 128 bytes of one row
        const int row0 = (warp & 3) * 32, nrow = min(32, rows - row0);
        float* o_dst = a.o1 + (at + row0) * kHeadDim;
        const uint32_t stage = base + 6 * kBuf + warp * kStage;
#pragma unroll 1
        for (int y = 0; y < 4; ++y) {
          uint32_t o[32];
          tmem_ld32(o_col + 32 * y, o);
          tmem_wait_ld();
          tmem_use32(o);
#pragma unroll
          for (int z = 0; z < 8; ++z)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(
                             stage + lane * 128 + ((z ^ (lane & 7)) * 16)),
                         "r"(o[4 * z]), "r"(o[4 * z + 1]), "r"(o[4 * z + 2]), "r"(o[4 * z + 3])
                         : "memory");
          __syncwarp();
          for (int z = 0; z < (nrow + 3) / 4; ++z) {
            const int w = 4 * z + (lane >> 3);
            uint4 v;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                         : "r"(stage + w * 128 + (((lane & 7) ^ (w & 7)) * 16)));
            if (w < nrow)
              *reinterpret_cast<uint4*>(o_dst + w * kHeadDim + 32 * y + 4 * (lane & 7)) = v;
          }
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 8) tmem_free(tmem, 512);
}

// Join a row's records: W warps per output row.  A warp's lanes look 32 records
// up at a time, of those that may be there; the warp then adds them with four
// channels per lane, four loads in flight; the warps' sums are added in order,
// so that the result does not depend on timing.  W = 4 where a row of the prefix has
// many records, or so many CTAs share its unit that one warp would look them up in
// two turns or more, unless rows are many; else 1, since four are four times the
// warps.  Calls with one warp and with four, in us (medians of ten; 100 shapes), by
// (places looked up, records of them, rows):
//   four: (147, 147, 4) 60.4, 37.4; (112, 112, 132) 45.9, 27.4; (81, 1, 48) 16.3, 14.0;
//         (34, 10, 240) 17.3, 16.2; (32, 32, 1024) 50.5, 44.0; (16, 16, 1280) 50.1, 48.5;
//         (15, 15, 1088) 22.8, 21.8; (21, 12, 128) 17.4, 17.0
//   one:  (15, 15, 2048), own parts of 1000 tokens among them, 64.6, 66.0; (12, 12, 1056)
//         24.8, 25.1; (18, 8, 128) 15.8, 16.1; (16, 3, 80) 13.7, 14.9; (6, 6, 4096) 38.8, 42.2
constexpr int kJoinThreads = 128;
constexpr int kJoinWarps = kJoinThreads / 32;
constexpr int kJoinMany = 12, kJoinRows = 12 * kPdCtas;

// Output row bh (KV head h) by one warp alone, from sequence 0's first len rows:
// a key per lane, then four channels per lane.
__device__ __forceinline__ void row_alone(const PdArgs& a, int h, int64_t bh, int len, float& M,
                                       float& Ls, float4& A) {
  const int lane = threadIdx.x & 31;
  const __half2* q = reinterpret_cast<const __half2*>(a.q + bh * kHeadDim);
  M = -INFINITY;
  Ls = 0.f;
  A = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int t0 = 0; t0 < len; t0 += 32) {
    const int t = min(t0 + lane, len - 1), n = min(32, len - t0);
    const int64_t row = a.L.page_row(0, h, t / kPage) + t % kPage;
    const __half2* k = reinterpret_cast<const __half2*>(a.K + row * kHeadDim);
    float s = 0.f;
#pragma unroll 8
    for (int z = 0; z < kHeadDim / 2; ++z) {
      const float2 x = __half22float2(q[z]), y = __half22float2(k[z]);
      s = __fmaf_rn(x.y, y.y, __fmaf_rn(x.x, y.x, s));
    }
    s = lane < n ? s * kPdScale : -INFINITY;
    const float top = fmaxf(M, warp_max(s));
    const float keep = M == -INFINITY ? 0.f : ex2(M - top);
    const float p = s == -INFINITY ? 0.f : ex2(s - top);
    M = top;
    Ls = Ls * keep + warp_sum(p);
    A.x *= keep;
    A.y *= keep;
    A.z *= keep;
    A.w *= keep;
    for (int j = 0; j < n; ++j) {
      const float f = __shfl_sync(0xffffffffu, p, j);
      const __half2* v = reinterpret_cast<const __half2*>(
          a.V + __shfl_sync(0xffffffffu, row, j) * kHeadDim + 4 * lane);
      const float2 v0 = __half22float2(v[0]), v1 = __half22float2(v[1]);
      A.x = __fmaf_rn(f, v0.x, A.x);
      A.y = __fmaf_rn(f, v0.y, A.y);
      A.z = __fmaf_rn(f, v1.x, A.z);
      A.w = __fmaf_rn(f, v1.y, A.w);
    }
  }
}

template <int W>
__global__ void __launch_bounds__(kJoinThreads) k_prefix_join(const __grid_constant__ PdArgs a) {
  __shared__ float4 acc_s[kJoinWarps][32];
  __shared__ float2 ml_s[kJoinWarps];
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) % W;
  const int bh = (int)blockIdx.x * (kJoinWarps / W) + (threadIdx.x >> 5) / W;   // output row
  const int lgG = 31 - __clz(a.G);   // G is a power of two
  const int b = bh / a.Hq, hq = bh - b * a.Hq, h = hq >> lgG, g = hq & (a.G - 1);
  griddep_wait();
  griddep_launch();   // the next call's tile kernel may set itself up
  if (W < kJoinWarps && bh >= a.L.B * a.Hq) return;
  const int len = a.L.len(b);
  // (through L1: every row's warps read the same few words)
  const uint64_t total = a.cum[a.L.B], c0 = a.cum[b], c1 = a.cum[b + 1];
  const int64_t X1 = prefix_span(a), X = X1 + own_cost(total) * a.L.Hk;
  // what lies at x is CTA floor(x kPdCtas / X)'s or, after rounding, a
  // neighbour's; the CTAs' own ranges decide
  const float per_x = (float)kPdCtas / (float)max(X, (int64_t)1);
  // Records of tiles [first, first + n) of the prefix's (part 0) or the own
  // (part 1) list, written to slot worker + u, row `row` of `per`; the workers
  // nw that may have some
  struct Part {
    int64_t u, first;
    int n, per, row, split, c_lo, nw;
  } p[2];
  const int m = b * a.G + g;
#pragma unroll
  for (int part = 0; part < 2; ++part) {
    Part& q = p[part];
    int64_t x0, x1;
    if (part == 0) {
      q.n = len > 0 ? a.KT : 0;
      q.u = (int64_t)h * a.RT + (a.pair ? m / (2 * kTile) : 0);
      q.first = q.u * a.KT;
      q.per = a.rows1;
      q.row = a.pair ? m % (2 * kTile) : m;
      q.split = a.pair ? 1 : 2;   // records per CTA at most
      x0 = q.u * unit_span(a);
      x1 = x0 + unit_span(a);
    } else {
      q.n = (int)(uint32_t)(c1 - c0);
      q.u = (int64_t)b * a.L.Hk + h;
      q.first = (int64_t)(uint32_t)c0 * a.L.Hk + (int64_t)h * q.n;
      q.per = a.G;
      q.row = g;
      q.split = 2;
      x0 = X1 + own_cost(c0) * a.L.Hk + h * own_cost(c1 - c0);
      x1 = x0 + own_cost(c1 - c0);
    }
    q.c_lo = max(0, (int)((float)x0 * per_x) - 1);
    const int c_hi = min(kPdCtas - 1, (int)((float)x1 * per_x) + 1);
    q.nw = q.n > 0 ? (c_hi - q.c_lo + 1) * q.split : 0;
  }
  float M = -INFINITY, Ls = 0.f;
  float4 A = make_float4(0.f, 0.f, 0.f, 0.f);
  const float4* o1 = reinterpret_cast<const float4*>(a.o1);
  const float4* o2 = reinterpret_cast<const float4*>(a.o2);
  for (int w0 = warp; w0 < p[0].nw + p[1].nw; w0 += 32 * W) {
    int w = w0 + lane * W;
    const bool own = w >= p[0].nw;
    const Part q = own ? p[1] : p[0];
    if (own) w -= p[0].nw;
    float2 v = make_float2(-INFINITY, 0.f);
    const float4* src = o1;
    if (w < q.nw) {
      const int cta = q.c_lo + (w >> (q.split - 1)), i = w & (q.split - 1);
      const PdRange rg = a.ranges[cta];
      int lo = own ? rg.s0 : rg.p0, hi = own ? rg.s1 : rg.p1;
      if (q.split == 2) {
        const int mid = own ? rg.sm : rg.pm;
        if (i == 0) hi = mid; else lo = mid;
      }
      const int64_t at = ((int64_t)q.split * cta + i + q.u) * q.per + q.row;
      src = (own ? o2 : o1) + at * (kHeadDim / 4);
      if (max((int64_t)lo, q.first) < min((int64_t)hi, q.first + q.n))
        v = __ldcg((own ? a.ml2 : a.ml1) + at);
    }
    const float top = fmaxf(M, warp_max(v.x));
    if (!__any_sync(0xffffffffu, v.x != -INFINITY)) continue;
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
      float4 x[4];
      float fs[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int from = todo ? __ffs(todo) - 1 : 0;
        fs[j] = __shfl_sync(0xffffffffu, f, from);
        const float4* s = reinterpret_cast<const float4*>(
            __shfl_sync(0xffffffffu, reinterpret_cast<unsigned long long>(src), from));
        if (!todo) fs[j] = 0.f;
        x[j] = todo ? __ldcg(s + lane) : make_float4(0.f, 0.f, 0.f, 0.f);
        todo &= todo - 1;
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        A.x = __fmaf_rn(fs[j], x[j].x, A.x);
        A.y = __fmaf_rn(fs[j], x[j].y, A.y);
        A.z = __fmaf_rn(fs[j], x[j].z, A.z);
        A.w = __fmaf_rn(fs[j], x[j].w, A.w);
      }
    }
  }
  if (W > 1) {
    acc_s[warp][lane] = A;
    if (lane == 0) ml_s[warp] = make_float2(M, Ls);
    __syncthreads();
    if (warp != 0) return;
#pragma unroll
    for (int w = 1; w < W; ++w) M = fmaxf(M, ml_s[w].x);
    Ls = 0.f;
    A = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < W; ++w) {
      const float2 v = ml_s[w];
      const float f = v.x == -INFINITY ? 0.f : ex2(v.x - M);
      const float4 e = acc_s[w][lane];
      Ls = __fmaf_rn(v.y, f, Ls);
      A.x = __fmaf_rn(e.x, f, A.x);
      A.y = __fmaf_rn(e.y, f, A.y);
      A.z = __fmaf_rn(e.z, f, A.z);
      A.w = __fmaf_rn(e.w, f, A.w);
    }
  }
  // A row that ends inside the prefix has weights of zero for the rows of V past
  // its end, which its tiles hold for other sequences: an infinity or a NaN there
  // would still reach it.  Its result then tells, and it is done again by itself.
  if (len < a.P && !__all_sync(0xffffffffu, fabsf((A.x + A.y) + (A.z + A.w)) < INFINITY))
    row_alone(a, h, bh, len, M, Ls, A);
  const float inv = Ls == 0.f ? 0.f : 1.f / Ls;
  const __half2 r[2] = {__floats2half2_rn(A.x * inv, A.y * inv),
                        __floats2half2_rn(A.z * inv, A.w * inv)};
  *reinterpret_cast<uint2*>(a.out + (int64_t)bh * kHeadDim + 4 * lane) = *reinterpret_cast<const uint2*>(r);
  if (a.lse && lane == 0)
    a.lse[bh] = Ls == 0.f ? -INFINITY : (M + log2f(Ls)) * 0.6931471805599453f;
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
  at += up(((size_t)B + 1) * sizeof(uint64_t));
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

static cudaError_t encode(CUtensorMap* map, const __half* p, int rank, const cuuint64_t* dims,
                          const cuuint64_t* strides, const cuuint32_t* box) {
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
  const cuuint32_t step[3] = {1, 1, 1};
  const CUresult r = reinterpret_cast<EncodeTiled>(f)(
      map, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, const_cast<__half*>(p), dims, strides, box, step,
      CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
      CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// K or V as rows of 128: boxes of 16 rows (a page) by 64 columns.
static cudaError_t encode_rows(CUtensorMap* map, const __half* p, int64_t rows) {
  const cuuint64_t dims[2] = {kHeadDim, (cuuint64_t)rows}, strides[1] = {kHeadDim * 2};
  const cuuint32_t box[2] = {64, kPage};
  return encode(map, p, 2, dims, strides, box);
}

// q [B][Hq][128]: boxes of a KV head's G query heads of `seqs` sequences by 64
// columns; sequences past the batch are filled with zeros.
static cudaError_t encode_q(CUtensorMap* map, const __half* q, int B, int Hq, int G, int seqs) {
  const cuuint64_t dims[3] = {kHeadDim, (cuuint64_t)Hq, (cuuint64_t)B};
  const cuuint64_t strides[2] = {kHeadDim * 2, (cuuint64_t)Hq * kHeadDim * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)G, (cuuint32_t)seqs};
  return encode(map, q, 3, dims, strides, box);
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
  a.K = K;
  a.V = V;
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
  a.cum = reinterpret_cast<uint64_t*>(w + p.cum);
  a.ranges = reinterpret_cast<PdRange*>(w + p.ranges);
  a.status = reinterpret_cast<int*>(w);
  a.out = out;
  a.lse = lse;
  const int64_t rows = L.page_table ? (int64_t)L.pool_pages * L.Hk * kPage
                                    : (int64_t)L.B * L.Hk * L.N;
  cudaError_t e;
  if (rows > 0) {   // a cache without rows has no tiles: no copy uses the maps
    CUtensorMap mk, mv, mq, mq1;
    if ((e = encode_rows(&mk, K, rows)) != cudaSuccess) return e;
    if ((e = encode_rows(&mv, V, rows)) != cudaSuccess) return e;
    if ((e = encode_q(&mq, q, L.B, Hq, a.G, kTile / a.G)) != cudaSuccess) return e;
    if ((e = encode_q(&mq1, q, L.B, Hq, a.G, 1)) != cudaSuccess) return e;
    static std::atomic<int> done[kMaxDevices];
    e = once_per_device(done, [] {
      return cudaFuncSetAttribute(k_prefix_decode, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                  (int)kPdSmem);
    });
    if (e != cudaSuccess) return e;
    e = launch_k(k_prefix_decode, dim3(kPdCtas), dim3(kPdThreads), kPdSmem, st, true, mk, mv, mq, mq1,
                 a);
    if (e != cudaSuccess) return e;
  } else if ((e = cudaMemsetAsync(a.cum, 0, ((size_t)L.B + 1) * sizeof(uint64_t), st)) != cudaSuccess) {
    return e;
  }
  // Places that may hold records of a prefix unit: its stretch of the line of costs,
  // on which every sequence has a tile of its own for each head at least (the lengths
  // are not known here), in CTAs of one or two; records: a tile each at least
  const int64_t units = (int64_t)L.Hk * a.RT, span = unit_span(a);
  const int64_t line = units * span + (int64_t)L.B * L.Hk * (kOwnStart + kOwnCost);
  const int64_t places = a.KT > 0 ? kPdCtas * (a.pair ? 1 : 2) * span / line : 0;
  const int64_t out_rows = (int64_t)L.B * Hq;
  if (out_rows < kJoinRows && (places >= 32 || (places >= kJoinMany && a.KT >= kJoinMany)))
    return launch_k(k_prefix_join<kJoinWarps>, dim3((unsigned)out_rows), dim3(kJoinThreads), 0, st,
                    rows > 0, a);
  return launch_k(k_prefix_join<1>, dim3((unsigned)((out_rows + kJoinWarps - 1) / kJoinWarps)),
                  dim3(kJoinThreads), 0, st, rows > 0, a);
}

}  // namespace tw
