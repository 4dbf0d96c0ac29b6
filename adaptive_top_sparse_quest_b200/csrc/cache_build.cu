// Cache-build kernels (prefill time, once per token): the quantised key cache
// and the Quest page metadata.
//
// Key cache: Twilight estimates attention weights from INT4 keys
// (atlas.scime.ai summary of "Twilight: Adaptive Attention Sparsity with
// Hierarchical Top-p Pruning", "Approach"); the 2-bit width its quantisation
// ablation compares against (table of measured effects) is built by the same
// kernels with 3 levels instead of 15.  Quest page metadata: per-page
// channel-wise key min / max, the layout Quest's page selection works on
// ("Surprising findings").
//
// Both kernels stream K once with 16-byte loads; one half-warp owns one token
// row (or one page), lane l owns channels 8l..8l+7, so a group of 32 channels
// is 4 adjacent lanes and its min / max needs two xor-shuffles.  The decode-
// time append kernel applies the same row quantisation to each sequence's
// newest token and folds that row into its page's min / max.
#include "tw_common.cuh"
#include "tw_kernels.h"

namespace tw {

// h_key of both halves of a word (its own inverse).
__device__ __forceinline__ uint32_t h_key2(uint32_t w) {
  return w ^ (((w >> 15) & 0x00010001u) * 0x7FFFu);
}

// Quantise one token row held by a half-warp (lane l16 holds channels
// 8 l16 .. 8 l16 + 7 in `raw`, their keys (h_key2) in `key`) to BITS-bit codes
// (levels 0 .. 2^BITS - 1) and store its codes, scales and zeros at `row`.  Every
// value equals a fixed sequence of IEEE round-to-nearest operations, so it is
// bit-exact with the CPU definition.  Code j of the lane sits at bits BITS * j of
// its 4 (BITS = 4) or 2 (BITS = 2) bytes: channel c at bits BITS * (c % (8 / BITS))
// of byte c / (8 / BITS).
template <int BITS>
__device__ __forceinline__ void quantize_row(const uint4 raw, const uint32_t (&key)[4], int64_t row,
                                             int lane, unsigned hmask,
                                             uint8_t* __restrict__ codes,
                                             __half* __restrict__ scales,
                                             __half* __restrict__ zeros) {
  static_assert(BITS == 4 || BITS == 2, "key-cache width");
  constexpr int kLevels = (1 << BITS) - 1;
  const int l16 = lane & 15;
  const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
  uint32_t lo = key[0], hi = lo;
#pragma unroll
  for (int j = 1; j < 4; ++j) {
    lo = __vmins2(lo, key[j]);
    hi = __vmaxs2(hi, key[j]);
  }
#pragma unroll
  for (int o = 1; o <= 2; o <<= 1) {
    lo = __vmins2(lo, __shfl_xor_sync(hmask, lo, o));
    hi = __vmaxs2(hi, __shfl_xor_sync(hmask, hi, o));
  }
  const int kmin = min((int)(int16_t)lo, (int)lo >> 16), kmax = max((int)(int16_t)hi, (int)hi >> 16);
  const uint32_t mn_bits = h_from_key(kmin);
  const uint32_t mx_bits = h_from_key(kmax);
  const float mnf = __half2float(__ushort_as_half((unsigned short)mn_bits));
  const float mxf = __half2float(__ushort_as_half((unsigned short)mx_bits));
  const float s32 = __fdiv_rn(__fsub_rn(mxf, mnf), (float)kLevels);
  const __half sc = __float2half_rn(s32);
  const float scf = __half2float(sc);
  // code = min(rint(fl((x - mn) / scale)), levels).  With the approximate
  // reciprocal (off by 2^-23 of itself at most) made 2^-21 smaller and larger, the
  // two products enclose the rounded quotient: where they round to one integer,
  // the quotient does too; a lane with a value that lies between divides.
  // 1.5 * 2^23 + y, fused, rounds y to the nearest integer, ties to even, into its
  // low bits; the sum of those bits' shifts, less that of the constants, packs
  // them.  A lane divides as well where the scale is no normal fp16 number: where
  // a key is infinite or NaN the scale is (finite keys' are below 2^16), and all
  // codes are 0; a subnormal one may be rounded down so far that quotients pass the
  // levels (a normal one is within 2^-11, and 15 (1 + 2^-11) rounds to 15).  Scale
  // 0, all keys alike, gives codes of 0 by a reciprocal of 0.
  float inv;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(scf));
  if (scf == 0.0f) inv = 0.0f;
  const bool plain = scf == 0.0f || (scf >= 0x1p-14f && scf < INFINITY);
  constexpr float kBig = 12582912.0f;
  const float lo1 = inv * (1.0f - 0x1p-21f), hi1 = inv * (1.0f + 0x1p-21f);
  const uint64_t inv_lo = f2_pack(lo1, lo1), inv_hi = f2_pack(hi1, hi1);
  const uint64_t big = f2_pack(kBig, kBig), sub = f2_pack(-mnf, -mnf);
  uint32_t packed = 0, shifts = 0, apart = plain ? 0u : 1u;
  uint64_t d[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
    d[j] = f2_add(f2_pack(x.x, x.y), sub);
    const float2 z = f2_unpack(f2_fma(d[j], inv_lo, big)), y = f2_unpack(f2_fma(d[j], inv_hi, big));
    apart |= __float_as_uint(z.x) ^ __float_as_uint(y.x);
    apart |= __float_as_uint(z.y) ^ __float_as_uint(y.y);
    packed += __float_as_uint(z.x) * (1u << (2 * BITS * j));
    packed += __float_as_uint(z.y) * (1u << (2 * BITS * j + BITS));
    shifts += 0x4B400000u * ((1u << (2 * BITS * j)) + (1u << (2 * BITS * j + BITS)));
  }
  if (apart) {
    packed = 0;
    const bool some = scf > 0.0f && scf < INFINITY;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 x = f2_unpack(d[j]);
      const float y0 = some ? fminf(__fdiv_rn(x.x, scf), (float)kLevels) : 0.0f;
      const float y1 = some ? fminf(__fdiv_rn(x.y, scf), (float)kLevels) : 0.0f;
      packed += __float_as_uint(__fadd_rn(y0, kBig)) * (1u << (2 * BITS * j));
      packed += __float_as_uint(__fadd_rn(y1, kBig)) * (1u << (2 * BITS * j + BITS));
    }
  }
  packed -= shifts;
  if (BITS == 4)
    *reinterpret_cast<uint32_t*>(codes + row * (kHeadDim / 2) + l16 * 4) = packed;
  else
    *reinterpret_cast<uint16_t*>(codes + row * (kHeadDim / 4) + l16 * 2) = (uint16_t)packed;
  if ((l16 & 3) == 0) {   // a group's first lane
    scales[row * kGroups + (l16 >> 2)] = sc;
    zeros[row * kGroups + (l16 >> 2)] = __ushort_as_half((unsigned short)mn_bits);
  }
}

template <int BITS>
__global__ void __launch_bounds__(256)
k_quantize_keys(Layout L, const __half* __restrict__ K, uint8_t* __restrict__ codes,
                __half* __restrict__ scales, __half* __restrict__ zeros) {
  const int lane = threadIdx.x & 31;
  const int l16 = lane & 15;
  const unsigned hmask = 0xFFFFu << (lane & 16);
  const int64_t total = (int64_t)L.B * L.Hk * L.N;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 4);
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 4) + (threadIdx.x >> 4); i < total;
       i += step) {
    const int t = (int)(i % L.N);
    const int64_t bh = i / L.N;
    const int h = (int)(bh % L.Hk);
    const int b = (int)(bh / L.Hk);
    if (t >= L.len(b)) continue;  // uniform across the half-warp
    const int64_t row = L.row(b, h, t);
    const uint4 raw = ld_stream16(K + row * kHeadDim + l16 * 8);
    const uint32_t key[4] = {h_key2(raw.x), h_key2(raw.y), h_key2(raw.z), h_key2(raw.w)};
    quantize_row<BITS>(raw, key, row, lane, hmask, codes, scales, zeros);
  }
}

// Incremental decode append: for every sequence b with len_b >= 1 and every
// KV head, quantise the newest token t = len_b - 1 and fold it into the
// metadata of its page (a page starting at t holds only t).  With the cache
// current for the lengths minus one, the result equals a rebuild for the new
// lengths bit for bit: quantisation is per row, and exact fp16 min / max of
// a page's valid rows may be taken one row at a time.
template <int BITS>
__global__ void __launch_bounds__(256)
k_append_keys(Layout L, const __half* __restrict__ K, uint8_t* __restrict__ codes,
              __half* __restrict__ scales, __half* __restrict__ zeros, __half* __restrict__ meta) {
  const int lane = threadIdx.x & 31;
  const int l16 = lane & 15;
  const unsigned hmask = 0xFFFFu << (lane & 16);
  const int64_t total = (int64_t)L.B * L.Hk;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 4);
  griddep_wait();
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 4) + (threadIdx.x >> 4); i < total;
       i += step) {
    const int h = (int)(i % L.Hk);
    const int b = (int)(i / L.Hk);
    const int t = L.len(b) - 1;
    if (t < 0) continue;  // uniform across the half-warp
    const int64_t row = L.row(b, h, t);
    const uint4 raw = *reinterpret_cast<const uint4*>(K + row * kHeadDim + l16 * 8);
    if (codes) {
      const uint32_t key[4] = {h_key2(raw.x), h_key2(raw.y), h_key2(raw.z), h_key2(raw.w)};
      quantize_row<BITS>(raw, key, row, lane, hmask, codes, scales, zeros);
    }
    if (meta) {
      __half* dst = meta + L.meta_index(b, h, t / kPage) * (2 * kHeadDim) + l16 * 8;
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t mn[4], mx[4];
      if (t % kPage == 0) {   // the page's first row
#pragma unroll
        for (int j = 0; j < 4; ++j) mn[j] = mx[j] = w[j];
      } else {
        const uint4 omn = *reinterpret_cast<const uint4*>(dst);
        const uint4 omx = *reinterpret_cast<const uint4*>(dst + kHeadDim);
        const uint32_t on[4] = {omn.x, omn.y, omn.z, omn.w};
        const uint32_t ox[4] = {omx.x, omx.y, omx.z, omx.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t a = 0, c = 0;
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int kx = h_key((w[j] >> (16 * e)) & 0xFFFFu);
            const int kn = min(h_key((on[j] >> (16 * e)) & 0xFFFFu), kx);
            const int km = max(h_key((ox[j] >> (16 * e)) & 0xFFFFu), kx);
            a |= h_from_key(kn) << (16 * e);
            c |= h_from_key(km) << (16 * e);
          }
          mn[j] = a;
          mx[j] = c;
        }
      }
      *reinterpret_cast<uint4*>(dst) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
      *reinterpret_cast<uint4*>(dst + kHeadDim) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
    }
  }
  griddep_launch();
}

// Write new K/V rows by slot.  Rows t of k_new / v_new go to the cache rows that
// slots[t] names; in the same pass over the key row it is quantised, and the
// page's min / max is folded, so K is read once instead of three times.
//
// A run of list neighbours on consecutive slots of one page is one warp's work
// per KV head, a row per half-warp at a time: it alone touches that page's
// metadata, so no atomics are needed and the result does not depend on an order.
// The run that starts at a page's first row starts its metadata anew; another
// folds what is there (its earlier rows are in it).  A warp looks at `chunk` list
// places, for one head, and takes the runs that start there, to their ends up to
// 15 places further on; it needs no other warp, so a block is only what shares a
// launch slot.
//
// What bounds it (one B200).  8191 tokens x 8 heads at 4 bits, 19.3 us (11 by the bytes
// at the copy rate): no unit is full (issue slots 0.6, DRAM a quarter); the grid is one
// wave, and each warp takes its page in four turns of loads, quantiser and stores that
// wait for one another.  20000 x 32 at 2 bits, 119 us (108): HBM, 0.9 of the copy rate.
// 64 single tokens x 8 heads, 2.8 us: one chain of loads.  Many runs of one to three
// tokens: up to sixteen of those chains in a warp, one after another.
constexpr int kWrThreads = 128;
constexpr int kWrWarps = kWrThreads / 32;
constexpr int kWrRows = 2;   // rows of a run in flight per half-warp

template <int BITS>
__global__ void __launch_bounds__(kWrThreads, 8)
k_write_rows(Layout L, const __half* __restrict__ k_new, const __half* __restrict__ v_new,
             int64_t k_stride, int64_t v_stride, const int32_t* __restrict__ slots, int T,
             int chunk, __half* __restrict__ K, __half* __restrict__ V,
             uint8_t* __restrict__ codes, __half* __restrict__ scales, __half* __restrict__ zeros,
             __half* __restrict__ meta) {
  const int tid = threadIdx.x, lane = tid & 31, l16 = tid & 15, hw = lane >> 4;
  const unsigned hmask = 0xFFFFu << (lane & 16);
  const uint32_t item = blockIdx.x * kWrWarps + (tid >> 5), ck = item / (uint32_t)L.Hk;
  const int h = (int)(item - ck * L.Hk);
  // lane l holds place t0 - 1 + l
  const int64_t t0 = (int64_t)ck * chunk, t = t0 - 1 + lane;
  const int nslot = L.page_table ? L.pool_pages * kPage : L.B * L.N;
  int s = lane <= chunk + kPage - 1 && t >= 0 && t < T ? slots[t] : -1;
  if ((unsigned)s >= (unsigned)nslot) s = -1;
  const int prev = __shfl_up_sync(0xffffffffu, s, 1);
  // a place carries its neighbour's run on unless a page (or sequence) begins there
  const bool first = s < 0 || (L.page_table ? s : s % L.N) % kPage == 0;
  const unsigned on = __ballot_sync(0xffffffffu, lane > 0 && !first && prev == s - 1);
  unsigned starts = __ballot_sync(0xffffffffu, s >= 0 && lane > 0 && lane <= chunk) & ~on;
  for (; starts; starts &= starts - 1) {
    const int at = __ffs(starts) - 1, n = __ffs(~(on >> (at + 1)));
    const int slot = __shfl_sync(0xffffffffu, s, at);
    const int64_t tok = t0 - 1 + at;
    int64_t row, mrec;
    int o;
    if (L.page_table) {
      o = slot % kPage;
      mrec = (int64_t)(slot / kPage) * L.Hk + h;
      row = mrec * kPage + o;
    } else {
      const int pos = slot % L.N;
      o = pos % kPage;
      const int64_t bh = (int64_t)(slot / L.N) * L.Hk + h;
      row = bh * L.N + pos;
      mrec = bh * L.max_pages + pos / kPage;
    }
    const __half* ks = k_new + tok * k_stride + h * kHeadDim + l16 * 8;
    const __half* vs = v_new + tok * v_stride + h * kHeadDim + l16 * 8;
    uint32_t kmin[4], kmax[4];   // keys of the lane's eight channels
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      kmin[j] = 0x7FFF7FFFu;
      kmax[j] = 0x80008000u;
    }
    // (the rows in flight are quantised together, which hides the arithmetic's
    // latency; loads sent ahead of the row before them instead: 21 -> 24 us for a
    // prompt of 8191 tokens and 8 heads)
    for (int c = hw; c < n; c += 2 * kWrRows) {
      uint4 kr[kWrRows], vr[kWrRows];
#pragma unroll
      for (int x = 0; x < kWrRows; ++x)
        if (c + 2 * x < n) {
          kr[x] = ld_stream16(ks + (c + 2 * x) * k_stride);
          vr[x] = ld_stream16(vs + (c + 2 * x) * v_stride);
        }
#pragma unroll
      for (int x = 0; x < kWrRows; ++x)
        if (c + 2 * x < n) {
          const int64_t at = row + c + 2 * x;
          *reinterpret_cast<uint4*>(K + at * kHeadDim + l16 * 8) = kr[x];
          *reinterpret_cast<uint4*>(V + at * kHeadDim + l16 * 8) = vr[x];
          const uint32_t key[4] = {h_key2(kr[x].x), h_key2(kr[x].y), h_key2(kr[x].z),
                                   h_key2(kr[x].w)};
          if (codes) quantize_row<BITS>(kr[x], key, at, lane, hmask, codes, scales, zeros);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            kmin[j] = __vmins2(kmin[j], key[j]);
            kmax[j] = __vmaxs2(kmax[j], key[j]);
          }
        }
    }
    if (!meta) continue;
    // fold the two halves' rows; one half then keeps the minima, the other the maxima
    __syncwarp();
    uint32_t m[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t lo = __vmins2(kmin[j], __shfl_xor_sync(0xffffffffu, kmin[j], 16));
      const uint32_t hi = __vmaxs2(kmax[j], __shfl_xor_sync(0xffffffffu, kmax[j], 16));
      m[j] = hw ? hi : lo;
    }
    __half* dst = meta + (mrec * 2 + hw) * kHeadDim + l16 * 8;
    if (o != 0) {
      const uint4 old = *reinterpret_cast<const uint4*>(dst);
      const uint32_t ow[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
      for (int j = 0; j < 4; ++j)
        m[j] = hw ? __vmaxs2(m[j], h_key2(ow[j])) : __vmins2(m[j], h_key2(ow[j]));
    }
    *reinterpret_cast<uint4*>(dst) =
        make_uint4(h_key2(m[0]), h_key2(m[1]), h_key2(m[2]), h_key2(m[3]));
  }
}

__global__ void __launch_bounds__(256)
k_page_meta(Layout L, const __half* __restrict__ K, __half* __restrict__ meta) {
  const int l16 = threadIdx.x & 15;
  const int64_t total = (int64_t)L.B * L.Hk * L.max_pages;
  const int64_t step = (int64_t)gridDim.x * (blockDim.x >> 4);
  for (int64_t i = (int64_t)blockIdx.x * (blockDim.x >> 4) + (threadIdx.x >> 4); i < total;
       i += step) {
    const int pg = (int)(i % L.max_pages);
    const int64_t bh = i / L.max_pages;
    const int h = (int)(bh % L.Hk);
    const int b = (int)(bh / L.Hk);
    const int n = min(kPage, L.len(b) - pg * kPage);
    if (n <= 0) continue;
    const int64_t row0 = L.page_row(b, h, pg);
    const __half* src = K + row0 * kHeadDim + l16 * 8;
    uint4 raw[kPage];
#pragma unroll
    for (int r = 0; r < kPage; ++r)
      if (r < n) raw[r] = ld_stream16(src + (int64_t)r * kHeadDim);
    int kmin[8], kmax[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      kmin[j] = 0x7FFFFFFF;
      kmax[j] = -0x7FFFFFFF - 1;
    }
#pragma unroll
    for (int r = 0; r < kPage; ++r) {
      if (r < n) {
        const uint32_t w[4] = {raw[r].x, raw[r].y, raw[r].z, raw[r].w};
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int kk = h_key((w[j >> 1] >> (16 * (j & 1))) & 0xFFFFu);
          kmin[j] = min(kmin[j], kk);
          kmax[j] = max(kmax[j], kk);
        }
      }
    }
    uint32_t mn[4], mx[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      mn[j] = h_from_key(kmin[2 * j]) | (h_from_key(kmin[2 * j + 1]) << 16);
      mx[j] = h_from_key(kmax[2 * j]) | (h_from_key(kmax[2 * j + 1]) << 16);
    }
    __half* dst = meta + L.meta_index(b, h, pg) * (2 * kHeadDim) + l16 * 8;
    *reinterpret_cast<uint4*>(dst) = make_uint4(mn[0], mn[1], mn[2], mn[3]);
    *reinterpret_cast<uint4*>(dst + kHeadDim) = make_uint4(mx[0], mx[1], mx[2], mx[3]);
  }
}

void launch_quantize_keys(const Layout& L, const __half* K, uint8_t* codes, __half* scales,
                          __half* zeros, cudaStream_t st, int num_sms) {
  const int64_t rows = (int64_t)L.B * L.Hk * L.N;
  const int64_t want = (rows + 15) / 16;
  const int64_t cap_blocks = (int64_t)num_sms * 8;
  const int blocks = (int)(want < 1 ? 1 : (want < cap_blocks ? want : cap_blocks));
  if (L.kbits == 2)
    k_quantize_keys<2><<<blocks, 256, 0, st>>>(L, K, codes, scales, zeros);
  else
    k_quantize_keys<4><<<blocks, 256, 0, st>>>(L, K, codes, scales, zeros);
}

cudaError_t launch_append_keys(const Layout& L, const __half* K, uint8_t* codes, __half* scales,
                               __half* zeros, __half* meta, cudaStream_t st, int num_sms,
                               bool pdl) {
  const int64_t units = (int64_t)L.B * L.Hk;
  const int64_t want = (units + 15) / 16;
  const int64_t cap_blocks = (int64_t)num_sms * 8;
  const int blocks = (int)(want < 1 ? 1 : (want < cap_blocks ? want : cap_blocks));
  return launch_k(L.kbits == 2 ? k_append_keys<2> : k_append_keys<4>, dim3(blocks), dim3(256), 0,
                  st, pdl, L, K, codes, scales, zeros, meta);
}

void launch_page_meta(const Layout& L, const __half* K, __half* meta, cudaStream_t st,
                      int num_sms) {
  const int64_t pages = (int64_t)L.B * L.Hk * L.max_pages;
  const int64_t want = (pages + 15) / 16;
  const int64_t cap_blocks = (int64_t)num_sms * 8;
  const int blocks = (int)(want < 1 ? 1 : (want < cap_blocks ? want : cap_blocks));
  k_page_meta<<<blocks, 256, 0, st>>>(L, K, meta);
}

cudaError_t launch_write_rows(const Layout& L, const __half* k_new, const __half* v_new,
                              int64_t k_stride, int64_t v_stride, const int32_t* slots, int T,
                              __half* K, __half* V, uint8_t* codes, __half* scales, __half* zeros,
                              __half* meta, cudaStream_t st, int num_sms) {
  // list places per warp: as many as a page has rows, fewer while there would
  // not be 16 warps for every SM: single tokens are a run each (1024 x 8 heads: 7.2
  // us, 14.9 with 4 warps per SM asked for), of a prompt's places only every 16th
  // starts one (2000 x 8 heads: 10.0, 11.9 with 64)
  int chunk = kPage;
  auto items = [&] { return (int64_t)((T + chunk - 1) / chunk) * L.Hk; };
  while (chunk > 1 && items() < 16 * num_sms) chunk /= 2;
  const dim3 grid((unsigned)((items() + kWrWarps - 1) / kWrWarps));
  return launch_k(L.kbits == 2 ? k_write_rows<2> : k_write_rows<4>, grid, dim3(kWrThreads), 0, st,
                  false, L, k_new, v_new, k_stride, v_stride, slots, T, chunk, K, V, codes, scales,
                  zeros, meta);
}

}  // namespace tw
