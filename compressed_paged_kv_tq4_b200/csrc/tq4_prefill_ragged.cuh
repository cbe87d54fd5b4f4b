// Attention of chunks of several requests over their paged TQ4 prefixes, with a sliding
// window and sinks (sm_100a).
//
// Request r brings n_r new tokens (rows cu[r] .. cu[r + 1] - 1 of q, k, v) at positions
// first_r = T_r - n_r .. T_r - 1. The token at position P sees j <= P with j > P - window or
// j < n_sink: positions before first_r from the cache, the rest from the chunk's own k and v.
// The arithmetic is the rotated domain's ([V2] wpnews.pro "JustFit: Run Qwen 27B Fast ...",
// mechanism table row KVExec): o = R^T sum_j p_j R v_j / sum_j p_j, p_j = exp(scale R q . R k_j).
//
// Three launches.
//   prep     every vector that some token sees becomes one f16 row of 512 B (and its norm one
//            float): a cached vector its centroids c[idx] (the norm apart), a chunk vector R x
//            brought to [0.5, 1) by a power of two (its norm). Rows of a request lie tile by
//            tile, those of the sinks, then those of the window. The queries become rows R q,
//            scaled likewise. One CTA also lays out the work: tiles per block of 256 query
//            rows, their running sum, and where each CTA pair's share begins.
//   attend   one persistent CTA pair per two SMs. All tiles of all (KV head, row block) items
//            stand in one line, of which each pair takes an equal part, so lengths, heads and
//            chunk sizes of any mixture keep every SM busy to the end; an item that two pairs
//            share leaves partial rows.
//   combine  merges the rows of shared items.
// Why rows first: the 256-row blocks of a chunk read the same positions, (6 n_r / 256) times
// over, and a row costs 512 B of L2 once against 128 table lookups each time. The tensor
// cores then never wait for a lookup: tiles arrive by TMA, and the CTA is a plain pipeline.
//
// attend, per CTA (rank r of the pair holds query rows 128 r .. of the item's 256):
//   warps 0-3  softmax, one thread per row: scores from TMEM, K norms, mask, running maximum
//              (raised only when it grows by more than 2^4), P = p * n_v written over the
//              scores as f16; the epilogue: O / l, R^T by in-register butterflies, out.
//   warp 4     K tiles (its half of each tile's positions) and the norms
//   warp 5     rank 0: issues every tcgen05.mma of the pair, QK(j) then PV(j - 1);
//              rank 1: tells rank 0 when its own copies have landed
//   warp 6     V tiles (its half of the dims)      warp 7  Q rows
// bf16 results: single f16 operands (queries, centroids, weights: each rounded once, 2^-11
// relative), tiles of 128 positions, two stages. fp32 results (kExact): f16 hi + lo pairs,
// S = Qh Kh + Ql Kh + Qh Kl, O = Ph Vh + Pl Vh + Ph Vl, tiles of 64 positions, one stage.
// TMEM (512 columns): S/P buffers at 0 and 128, O at 256. Every wait is bounded, as in the
// one-request prefill.
#pragma once
#include "tq4_decode_q1.cuh"
#include "tq4_prefill_tc.cuh"
#include "tq4_step.cuh"

namespace tq4 {

constexpr int kRgThreads = 256;
constexpr int kRgSoftWarps = 4, kRgKWarp = 4, kRgMmaWarp = 5, kRgVWarp = 6, kRgQWarp = 7;
constexpr int kRgNormSlots = 4;
constexpr int kRgMinTiles = 256;      // positions: a pair's share is at least this many (a few tiles)
template <bool kExact>
struct RgShape {
  static constexpr int kTile = kExact ? 64 : 128;            // positions per tile
  static constexpr int kStages = kExact ? 1 : 2;
  static constexpr int kParts = kExact ? 2 : 1;              // hi (and lo)
  static constexpr uint32_t kQPanel = kPfRows * 128;          // 64 dims of 128 rows
  static constexpr uint32_t kQPart = 4 * kQPanel;             // 64 KiB
  static constexpr uint32_t kKPanel = (kTile / 2) * 128;      // 64 dims of this CTA's half tile
  static constexpr uint32_t kKPart = 4 * kKPanel;
  static constexpr uint32_t kVPanel = kTile * 128;            // 64 of this CTA's 128 dims, all positions
  static constexpr uint32_t kVPart = 2 * kVPanel;
  static constexpr uint32_t kKOff = kParts * kQPart;
  static constexpr uint32_t kVOff = kKOff + kStages * kParts * kKPart;
  static constexpr uint32_t kNormOff = kVOff + kStages * kParts * kVPart;   // [slots][K, V][kTile] f32
  static constexpr uint32_t kBarOff = kNormOff + kRgNormSlots * 2 * kTile * 4;
  static constexpr uint32_t kMiscOff = kBarOff + 256;         // [0] TMEM base, [1] abort
  static constexpr uint32_t kSmem = kMiscOff + 64 + 1024;     // + alignment slack
  static constexpr float kLazy = kExact ? 0.f : 4.f;           // P = p n_v / 16 <= 2^4 * 65504 / 16; fp32: p <= 1, P = p n_v
  static constexpr float kPScale = kExact ? 1.f : 0.0625f;
};
static_assert(RgShape<false>::kSmem <= 227u * 1024u && RgShape<true>::kSmem <= 227u * 1024u, "shared memory");

// barriers (8 B each)
constexpr int kRgQFull = 0, kRgQPeer = 1, kRgKFull = 2, kRgKPeer = 4, kRgVFull = 6, kRgVPeer = 8, kRgNFull = 10,
              kRgPFull = 14, kRgSFull = 16, kRgVEmpty = 18, kRgEpi = 20, kRgDrain = 21;

struct RgReq {
  int32_t row0, n_new;   // rows of q, k, v; 0 new tokens for a request without work
  int32_t first, len;    // position of its first new token; all positions
  int32_t sink_tiles, skip;   // tiles of sinks, then real tile = row tile + skip
  int32_t tile0, blk0;   // its first row tile and row block
};
struct RgHead {
  int32_t n_blk, n_tiles;   // row blocks; row tiles
  int32_t n_pairs;          // pairs with work
  int32_t pad;
};
struct RgStart { int32_t head, blk, tile, pad; };

struct RaggedParams {
  const uint8_t* pool;
  int32_t num_pages;
  const int32_t* tables;
  int32_t max_pages;
  const int32_t* seq_lens;
  const int32_t* cu;
  int32_t n_req, n_tok;
  int32_t window, n_sink;
  const uint16_t* q;
  const uint16_t* k;
  const uint16_t* v;
  float scale;
  void* out;
  int out_dtype;
  Signs signs;
  int* status;
  uint32_t spin_limit;
  int test_withhold;
  int32_t max_pairs;
  // workspace
  RgHead* head;
  RgReq* req;         // [n_req]
  int32_t* blk_req;   // [blocks]
  int64_t* blk_cum;   // [blocks + 1] tiles before each block
  RgStart* starts;    // [max_pairs]
  __half* qr;         // [parts][4][6 n_tok][256]
  float* qfac;        // [4][6 n_tok]
  __half* rows;       // [parts][K, V][4][store_rows][256]
  float* norms;       // [K, V][4][store_rows]
  int64_t store_rows;
  float* po;          // [2 max_pairs][256][256]
  float2* pml;        // [2 max_pairs][256]
};

// Bounds that the host knows. A request's row tiles number at most sinks / tile + (window +
// new) / tile + 3 and never more than its table's; its row blocks 6 new / 256 + 1.
struct RgLayout {
  int64_t blocks, store_rows;
  size_t head, req, blk_req, blk_cum, starts, qr, qfac, rows, norms, po, pml, total;
};
inline RgLayout ragged_layout(int32_t num_sms, int32_t n_req, int32_t n_tok, int32_t max_pages, int32_t window,
                              int32_t n_sink, bool exact) {
  RgLayout l{};
  const int64_t tile = exact ? 64 : 128, parts = exact ? 2 : 1, busy = std::min(n_req, n_tok);
  const int64_t most = int64_t(max_pages) * (kPage / tile);
  const int64_t some = (int64_t(n_sink) + tile - 1) / tile + int64_t(window) / tile + 3;
  l.blocks = int64_t(6) * n_tok / 256 + busy;
  l.store_rows = tile * (busy * std::min(most, some) + (n_tok + tile - 1) / tile);
  size_t at = 0;
  auto take = [&at](size_t bytes) {
    const size_t p = at;
    at += (bytes + 1023) & ~size_t(1023);
    return p;
  };
  const size_t pairs = size_t(std::max(num_sms / 2, 1));
  l.head = take(sizeof(RgHead));
  l.req = take(size_t(n_req) * sizeof(RgReq));
  l.blk_req = take(size_t(l.blocks) * 4);
  l.blk_cum = take(size_t(l.blocks + 1) * 8);
  l.starts = take(pairs * sizeof(RgStart));
  l.qr = take(size_t(parts) * kHq * n_tok * kD * 2);
  l.qfac = take(size_t(kHq) * n_tok * 4);
  l.rows = take(size_t(parts) * 2 * kHkv * l.store_rows * kD * 2);
  l.norms = take(size_t(2) * kHkv * l.store_rows * 4);
  l.po = take(2 * pairs * 256 * kD * 4);
  l.pml = take(2 * pairs * 256 * 8);
  l.total = at;
  return l;
}

// the last index i of a[0 .. n - 1] (non-decreasing) with a[i] <= x; a[0] <= x
template <typename T>
__device__ __forceinline__ int rg_last_at_most(const T* a, int n, T x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Tiles that a block of query rows visits: those of sinks [0, sinks), then all from the first
// position of its first token's window to its last token; real tile = i < sinks ? i : i + skip.
struct RgSpan { int32_t sinks, skip, n; };
template <int kTile>
__device__ __forceinline__ RgSpan rg_span(int32_t lo, int32_t last, int32_t n_sink) {
  RgSpan s;
  s.sinks = (min(n_sink, lo) + kTile - 1) / kTile;
  s.skip = max(lo / kTile - s.sinks, 0);
  s.n = last / kTile + 1 - s.skip;
  return s;
}
template <int kTile>
__device__ __forceinline__ RgSpan rg_block_span(const RaggedParams& p, const RgReq& r, int rb) {
  const int t0 = 256 * rb / 6, t1 = min((256 * rb + 255) / 6, r.n_new - 1);
  return rg_span<kTile>(max(0, r.first + t0 - p.window + 1), r.first + t1, p.n_sink);
}

// --------------------------------------------------------------------------
// prep. Every CTA scans the requests (as plan_step does); CTA 0 then lays out the work, the
// others make rows: units of one (row tile, K or V, KV head) and of one token's queries.
// --------------------------------------------------------------------------
constexpr int kRgPrepThreads = 256;

// f16 rows of one vector held as 8 coordinates a lane (already times `down`)
template <bool kExact>
__device__ __forceinline__ void rg_store_row(__half* dst, int64_t part_stride, const float v[8]) {
  const int lane = threadIdx.x & 31;
  uint32_t hi[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) hi[i] = pack_half2(v[2 * i], v[2 * i + 1]);
  *reinterpret_cast<uint4*>(dst + lane * 8) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
  if constexpr (kExact) {
    uint32_t lo[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 h = __half22float2(*reinterpret_cast<const __half2*>(&hi[i]));
      lo[i] = pack_half2(v[2 * i] - h.x, v[2 * i + 1] - h.y);
    }
    *reinterpret_cast<uint4*>(dst + part_stride + lane * 8) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}
// R x * 16 of a bf16 vector, brought to [0.5, 1) by 2^-e; returns 2^e (0 for a zero vector). A vector
// with an infinity or a NaN becomes zeros with the factor NaN, so that only those who see it feel it.
__device__ __forceinline__ float rg_rotate(const uint16_t* src, uint32_t sb, float v[8]) {
  const int lane = threadIdx.x & 31;
  const uint4 raw = __ldg(reinterpret_cast<const uint4*>(src + lane * 8));
  const uint32_t ww[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = apply_sign(__uint_as_float(ww[i] << 16), sb, 2 * i);
    v[2 * i + 1] = apply_sign(__uint_as_float(ww[i] & 0xFFFF0000u), sb, 2 * i + 1);
  }
  warp_fwht256(v);
  uint32_t top = 0;   // largest magnitude as bits: orders infinities and NaN above every number
#pragma unroll
  for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(v[i]) & 0x7FFFFFFFu);
  top = __reduce_max_sync(0xffffffffu, top);
  if (top >= 0x7F800000u) {
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = 0.f;
    return __uint_as_float(0x7FC00000u);
  }
  if (top == 0) return 0.f;
  const int e = min(max(int(top >> 23) - 126, -100), 126);
  const float down = __uint_as_float(uint32_t(127 - e) << 23);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] *= down;
  return __uint_as_float(uint32_t(127 + e) << 23);
}

template <bool kExact>
__global__ void __launch_bounds__(kRgPrepThreads) ragged_prep_kernel(const RaggedParams p) {
  using Sh = RgShape<kExact>;
  constexpr int kTile = Sh::kTile;
  extern __shared__ int32_t prep_smem[];
  __shared__ int64_t tot[3][kRgPrepThreads / 32], carry[3];
  __shared__ uint32_t pair_s[256];   // centroid pairs of a byte of codes: f16 hi
  __shared__ uint32_t res_s[kExact ? 256 : 1];   // and lo
  __shared__ int32_t s_blocks, s_tiles;
  int32_t* const row0_s = prep_smem;             // [n_req]
  int32_t* const tile0_s = row0_s + p.n_req;     // [n_req]
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  {
    const uint2 c = lut_row(tid);
    pair_s[tid] = c.x;
    if constexpr (kExact) res_s[tid] = c.y;
  }
  if (tid < 3) carry[tid] = 0;
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();

  // ---- the requests: rows, blocks and row tiles before each. A request's rows are its own when
  // its cu follows from the ones before it, so no two requests with work share a row.
  const int32_t cu0 = p.n_req > 0 ? p.cu[0] : 0;
  for (int base = 0; base < p.n_req; base += kRgPrepThreads) {
    const int r = base + tid;
    RgReq rq{};
    int64_t raw = 0, blocks = 0, tiles = 0;
    int32_t a = 0, b = 0, T = 0;
    if (r < p.n_req) {
      a = p.cu[r];
      b = p.cu[r + 1];
      T = p.seq_lens[r];
      raw = b > a ? int64_t(b) - a : 0;
    }
    const int64_t sum_raw = warp_scan_i64(raw);
    if (lane == 31) tot[0][w] = sum_raw;
    __syncthreads();
    int64_t before = carry[0] + sum_raw - raw;
    for (int x = 0; x < w; ++x) before += tot[0][x];
    if (r < p.n_req) {
      const bool rows_ok = a >= 0 && b >= a && b <= p.n_tok && int64_t(a) == cu0 + before;
      const bool len_ok = T >= 0 && int64_t(T) <= int64_t(p.max_pages) * kPage && (T == 0 || T >= raw);
      if (!rows_ok || !len_ok) {
        if (blockIdx.x == 0) record_error(p.status, TQ4_ERR_SEQ);
      }
      rq.row0 = rows_ok ? a : 0;
      if (rows_ok && len_ok && T > 0 && raw > 0) {
        rq.n_new = int32_t(raw);
        rq.first = T - rq.n_new;
        rq.len = T;
        const RgSpan s = rg_span<kTile>(max(0, rq.first - p.window + 1), T - 1, p.n_sink);
        rq.sink_tiles = s.sinks;
        rq.skip = s.skip;
        tiles = s.n;
        blocks = (int64_t(6) * rq.n_new + 255) / 256;
      }
    }
    const int64_t sum_b = warp_scan_i64(blocks), sum_t = warp_scan_i64(tiles);
    if (lane == 31) {
      tot[1][w] = sum_b;
      tot[2][w] = sum_t;
    }
    __syncthreads();
    int64_t blk0 = carry[1] + sum_b - blocks, tile0 = carry[2] + sum_t - tiles;
    for (int x = 0; x < w; ++x) {
      blk0 += tot[1][x];
      tile0 += tot[2][x];
    }
    if (r < p.n_req) {
      row0_s[r] = int32_t(min(int64_t(cu0) + before, int64_t(INT32_MAX)));
      tile0_s[r] = int32_t(tile0);
      rq.tile0 = int32_t(tile0);
      rq.blk0 = int32_t(blk0);
      if (blockIdx.x == 0) p.req[r] = rq;
    }
    __syncthreads();
    if (tid < 3)
      for (int x = 0; x < kRgPrepThreads / 32; ++x) carry[tid] += tot[tid][x];
    __syncthreads();
  }
  if (tid == 0) {
    s_blocks = int32_t(carry[1]);
    s_tiles = int32_t(carry[2]);
  }
  __syncthreads();

  if (blockIdx.x == 0) {
    // ---- tiles of each row block, their running sum, and the pairs' shares
    if (tid == 0) carry[0] = 0;
    __syncthreads();
    for (int base = 0; base < s_blocks; base += kRgPrepThreads) {
      const int i = base + tid;
      int64_t n = 0;
      if (i < s_blocks) {
        int lo = 0, hi = p.n_req - 1;   // the last request whose first block is at or before i
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (p.req[mid].blk0 <= i) lo = mid;
          else hi = mid - 1;
        }
        p.blk_req[i] = lo;
        const RgReq rq = p.req[lo];
        n = rg_block_span<kTile>(p, rq, i - rq.blk0).n;
      }
      const int64_t sum = warp_scan_i64(n);
      if (lane == 31) tot[0][w] = sum;
      __syncthreads();
      int64_t before = carry[0] + sum - n;
      for (int x = 0; x < w; ++x) before += tot[0][x];
      if (i < s_blocks) p.blk_cum[i] = before;
      __syncthreads();
      if (tid == 0)
        for (int x = 0; x < kRgPrepThreads / 32; ++x) carry[0] += tot[0][x];
      __syncthreads();
    }
    const int64_t per_head = carry[0], all = per_head * kHkv;
    constexpr int64_t kMin = kRgMinTiles / kTile;
    const int pairs = int(min(int64_t(p.max_pairs), all > 0 ? max(all / kMin, int64_t(1)) : int64_t(0)));
    if (tid == 0) {
      p.blk_cum[s_blocks] = per_head;
      *p.head = RgHead{s_blocks, s_tiles, pairs, 0};
    }
    __syncthreads();
    for (int s = tid; s < pairs; s += kRgPrepThreads) {
      const int64_t g = int64_t(s) * all / pairs, head = g / per_head, at = g - head * per_head;
      const int blk = rg_last_at_most<int64_t>(p.blk_cum, s_blocks, at);
      p.starts[s] = RgStart{int32_t(head), blk, int32_t(at - p.blk_cum[blk]), 0};
    }
    return;
  }

  // ---- rows
  const uint32_t sb = lane_sign_bits(p.signs);
  const int64_t kv_units = int64_t(s_tiles) * 2 * kHkv;
  const int32_t live = int32_t(min(max(int64_t(cu0) + carry[0], int64_t(0)), int64_t(p.n_tok)));   // rows of the last request end here
  const int64_t q_part = int64_t(kHq) * p.n_tok * kD, kv_part = int64_t(2) * kHkv * p.store_rows * kD;
  for (int64_t u = int64_t(blockIdx.x) - 1; u < kv_units + live; u += int64_t(gridDim.x) - 1) {
    if (u >= kv_units) {   // one token's 24 queries
      const int tok = int(u - kv_units);
      if (tok < cu0) continue;
      const int r = rg_last_at_most<int32_t>(row0_s, p.n_req, tok);
      const int32_t T = p.seq_lens[r], a = p.cu[r], b = p.cu[r + 1];
      const bool work = a >= 0 && a == row0_s[r] && b <= p.n_tok && tok >= a && tok < b && T > 0 &&
                        int64_t(T) <= int64_t(p.max_pages) * kPage && T >= b - a;
#pragma unroll
      for (int x = 0; x < kHq / 8; ++x) {
        const int hq = w + 8 * x, h = hq / kGroup;
        if (!work) {   // a refused request: zeros
          const int64_t off = (int64_t(tok) * kHq + hq) * kD + lane * 8;
          const uint4 z = make_uint4(0, 0, 0, 0);
          if (p.out_dtype == TQ4_DTYPE_F32) {
            uint4* dst = reinterpret_cast<uint4*>(static_cast<float*>(p.out) + off);
            dst[0] = z;
            dst[1] = z;
          } else {
            *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.out) + off) = z;
          }
          continue;
        }
        float v[8];
        const float up = rg_rotate(p.q + (int64_t(tok) * kHq + hq) * kD, sb, v);
        const int64_t row = int64_t(h) * kGroup * p.n_tok + int64_t(tok) * kGroup + (hq - h * kGroup);
        // the scores' factor is kept positive (the scale's sign goes into the row) and above zero,
        // so that a masked -infinity stays one
        const float sgn = p.scale > 0.f ? 1.f : p.scale < 0.f ? -1.f : 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= sgn;
        rg_store_row<kExact>(p.qr + row * kD, q_part, v);
        // (fmaxf would drop the NaN of a row that holds one)
        const float fac = up * (fabsf(p.scale) * 0.0625f * kLog2e);
        if (lane == 0) p.qfac[row] = fac < 1.17549435e-38f ? 1.17549435e-38f : fac;
      }
      continue;
    }
    // one row tile of one KV head's keys or values
    const int st = int(u >> 3), kv = int(u >> 2) & 1, h = int(u) & 3;
    const int r = rg_last_at_most<int32_t>(tile0_s, p.n_req, st);   // requests without tiles share their next's tile0
    const int32_t T = p.seq_lens[r], row0 = p.cu[r], first = T - (p.cu[r + 1] - row0);
    const int32_t lo = max(0, first - p.window + 1);
    const RgSpan s = rg_span<kTile>(lo, T - 1, p.n_sink);
    const int local = st - tile0_s[r];
    const int32_t pos0 = (local < s.sinks ? local : local + s.skip) * kTile;
    const int32_t page = pos0 < first ? __ldg(p.tables + int64_t(r) * p.max_pages + (pos0 >> 8)) : -1;   // a tile lies in one page
    const bool page_ok = page >= 0 && page < p.num_pages;
    const uint8_t* pg = p.pool + int64_t(page_ok ? page : 0) * kPageBytes;
    __half* dst0 = p.rows + (int64_t(kv * kHkv + h) * p.store_rows + int64_t(st) * kTile) * kD;
    float* nrm0 = p.norms + int64_t(kv * kHkv + h) * p.store_rows + int64_t(st) * kTile;
    const float unit = kv ? Sh::kPScale : 1.f;
    bool bad_page = false;
#pragma unroll 4
    for (int i = w; i < kTile; i += kRgPrepThreads / 32) {
      const int32_t pos = pos0 + i;
      float norm = 0.f;
      if (pos >= first && pos < T) {   // the chunk's own
        float v[8];
        norm = 0.0625f * unit * rg_rotate((kv ? p.v : p.k) + (int64_t(row0 + pos - first) * kHkv + h) * kD, sb, v);
        rg_store_row<kExact>(dst0 + int64_t(i) * kD, kv_part, v);
      } else {
        const bool seen = pos < first && (pos >= lo || pos < p.n_sink);
        uint4 hi = make_uint4(0, 0, 0, 0), lo4 = hi;
        bad_page |= seen && !page_ok;
        if (seen && page_ok) {
          const int slot = h * kPage + (pos & (kPage - 1));
          const uint32_t word = __ldg(reinterpret_cast<const uint32_t*>(pg + (kv ? kVWords : kKWords) + int64_t(slot) * 128) + lane);
          norm = ldg_half(pg + (kv ? kVNorms : kKNorms) + slot * 2) * unit;
          hi = make_uint4(pair_s[word & 255u], pair_s[(word >> 8) & 255u], pair_s[(word >> 16) & 255u], pair_s[word >> 24]);
          if constexpr (kExact)
            lo4 = make_uint4(res_s[word & 255u], res_s[(word >> 8) & 255u], res_s[(word >> 16) & 255u], res_s[word >> 24]);
        }
        *reinterpret_cast<uint4*>(dst0 + int64_t(i) * kD + lane * 8) = hi;
        if constexpr (kExact) *reinterpret_cast<uint4*>(dst0 + kv_part + int64_t(i) * kD + lane * 8) = lo4;
      }
      if (lane == 0) nrm0[i] = norm;
    }
    if (bad_page && lane == 0) record_error(p.status, TQ4_ERR_PAGE_RANGE);
  }
}

// 64 consecutive TMEM columns of this thread's lane (load and wait in one statement, as tm_ld32)
__device__ __forceinline__ void tm_ld64(uint32_t taddr, uint32_t (&r)[64]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {"
      "%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,"
      "%32,%33,%34,%35,%36,%37,%38,%39,%40,%41,%42,%43,%44,%45,%46,%47,"
      "%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,%60,%61,%62,%63"
      "}, [%64];\n"
      "tcgen05.wait::ld.sync.aligned;\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
        "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
        "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31]),
        "=r"(r[32]), "=r"(r[33]), "=r"(r[34]), "=r"(r[35]), "=r"(r[36]), "=r"(r[37]), "=r"(r[38]), "=r"(r[39]),
        "=r"(r[40]), "=r"(r[41]), "=r"(r[42]), "=r"(r[43]), "=r"(r[44]), "=r"(r[45]), "=r"(r[46]), "=r"(r[47]),
        "=r"(r[48]), "=r"(r[49]), "=r"(r[50]), "=r"(r[51]), "=r"(r[52]), "=r"(r[53]), "=r"(r[54]), "=r"(r[55]),
        "=r"(r[56]), "=r"(r[57]), "=r"(r[58]), "=r"(r[59]), "=r"(r[60]), "=r"(r[61]), "=r"(r[62]), "=r"(r[63])
      : "r"(taddr)
      : "memory");
}

// One stretch of a pair's share: tiles [tile, tile + n) of item (head, blk).
struct RgSeg {
  int32_t head, blk, tile, n, all;
  int32_t part;   // partial rows' index, -1: the whole item
};
// The pair's stretches in order; every warp walks them by itself.
struct RgWalk {
  const RaggedParams& p;
  int pair, n_blk;
  int64_t left;
  int32_t head, blk, tile;
  bool first;
  __device__ __forceinline__ RgWalk(const RaggedParams& params, int pr) : p(params), pair(pr) {
    const RgHead hd = *p.head;
    n_blk = hd.n_blk;
    const int64_t all = p.blk_cum[n_blk] * kHkv;
    left = int64_t(pair + 1) * all / hd.n_pairs - int64_t(pair) * all / hd.n_pairs;
    const RgStart s = p.starts[pair];
    head = s.head;
    blk = s.blk;
    tile = s.tile;
    first = true;
  }
  __device__ __forceinline__ bool next(RgSeg& g) {
    if (left <= 0) return false;
    g.head = head;
    g.blk = blk;
    g.tile = tile;
    g.all = int32_t(p.blk_cum[blk + 1] - p.blk_cum[blk]);
    g.n = int32_t(min(int64_t(g.all - tile), left));
    g.part = g.n == g.all ? -1 : 2 * pair + (first ? 0 : 1);
    left -= g.n;
    first = false;
    tile = 0;
    if (++blk == n_blk) {
      blk = 0;
      ++head;
    }
    return true;
  }
};

// 32-point Walsh-Hadamard transform in registers
__device__ __forceinline__ void fwht32(float (&v)[32]) {
#pragma unroll
  for (int s = 1; s < 32; s <<= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if ((i & s) == 0) {
        const float a = v[i], b = v[i + s];
        v[i] = a + b;
        v[i + s] = a - b;
      }
}

template <bool kExact>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kRgThreads, 1)
    ragged_attend_kernel(const RaggedParams p, const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kvmap) {
  using Sh = RgShape<kExact>;
  constexpr int kTile = Sh::kTile, kStages = Sh::kStages;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t sbase = (raw_s + 1023) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw_s);
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const uint32_t rank = cluster_rank();
  const int pair = int(blockIdx.x >> 1);
  auto bar = [sbase](int i) -> uint32_t { return sbase + Sh::kBarOff + 8u * uint32_t(i); };
  volatile uint32_t* misc = reinterpret_cast<volatile uint32_t*>(smem + Sh::kMiscOff);
  const uint32_t lead_bar0 = map_to_rank(bar(0), 0);

  if (tid == 0) {
    mbar_init(bar(kRgQFull), 1);
    mbar_init(bar(kRgQPeer), 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(bar(kRgKFull + b), 1);
      mbar_init(bar(kRgKPeer + b), 1);
      mbar_init(bar(kRgVFull + b), 1);
      mbar_init(bar(kRgVPeer + b), 1);
      mbar_init(bar(kRgPFull + b), 2 * kRgSoftWarps);
      mbar_init(bar(kRgSFull + b), 1);
      mbar_init(bar(kRgVEmpty + b), 1);
    }
    for (int b = 0; b < kRgNormSlots; ++b) mbar_init(bar(kRgNFull + b), 1);
    mbar_init(bar(kRgEpi), kRgSoftWarps);
    mbar_init(bar(kRgDrain), 1);
    misc[1] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
  }
  if (w == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], 512;\n" ::"r"(sbase + Sh::kMiscOff)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;\n" ::: "memory");
  }
  pdl_wait();
  pdl_launch_dependents();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem = misc[0];

  int* const status = p.status;
  const uint32_t spin_limit = p.spin_limit;
  const uint32_t peer_abort = map_to_rank(sbase + Sh::kMiscOff + 4, rank ^ 1u);
  auto bounded_wait = [misc, spin_limit, status, peer_abort](uint32_t b, uint32_t parity) -> bool {
    uint32_t spins = 0;
    while (!mbar_try_wait_cluster(b, parity)) {
      if (misc[1]) return false;
      if (++spins > spin_limit) {
        misc[1] = 1;
        st_cluster_u32(peer_abort, 1u);
        record_error(status, TQ4_ERR_TIMEOUT);
        return false;
      }
    }
    return true;
  };
  auto warp_wait = [&bounded_wait](uint32_t b, uint32_t parity) -> bool {
    return __all_sync(0xffffffffu, bounded_wait(b, parity));
  };
  // copies that an aborted call may have in flight end before the CTA does
  auto drain = [](uint32_t b, uint32_t parity) {
    for (uint32_t spins = 0; !mbar_try_wait_cluster(b, parity) && spins < TQ4_DEFAULT_WAIT_POLLS; ++spins) {
    }
  };

  if (pair < p.head->n_pairs) {
    RgWalk walk(p, pair);
    RgSeg g;
    if (w < kRgSoftWarps) {
      // =========================================================== softmax / epilogue
      const int r_local = 32 * w + lane;
      const uint32_t lane_addr = tmem + (uint32_t(32 * w) << 16);
      uint8_t* const stage = smem + w * 16384;   // this warp's 16 KiB of the Q panels, free once the item's last QK has run
      const float* norms = reinterpret_cast<const float*>(smem + Sh::kNormOff);
      int t = 0;      // tiles of this pair so far
      bool ok = true;
      while (ok && walk.next(g)) {
        const RgReq rq = p.req[p.blk_req[g.blk]];
        const int rb = g.blk - rq.blk0;
        const RgSpan span = rg_block_span<kTile>(p, rq, rb);
        const int n_rows = min(256, 6 * rq.n_new - 256 * rb);       // the item's rows
        const int row = min(int(rank) * kPfRows + r_local, n_rows - 1);   // padding rows repeat the last
        const int P = rq.first + (256 * rb + row) / 6;              // this row's position
        const float fac = p.qfac[int64_t(g.head) * kGroup * p.n_tok + int64_t(rq.row0) * kGroup + 256 * rb + row];
        float m_ref = -INFINITY, l_sum = 0.f;
        for (int j = 0; j < g.n; ++j, ++t) {
          const int b = t & 1;
          const int at = g.tile + j;
          const int pos0 = (at < span.sinks ? at : at + span.skip) * kTile;
          if (!(ok = warp_wait(bar(kRgNFull + (t & 3)), (t >> 2) & 1))) break;
          if (!(ok = warp_wait(bar(kRgSFull + b), (t >> 1) & 1))) break;
          tc_fence_after();
          const float4* kn4 = reinterpret_cast<const float4*>(norms + (t & 3) * 2 * kTile);
          const float4* vn4 = kn4 + kTile / 4;
          uint32_t sr[kTile / 64][64];
          float mx4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
          const bool full = __all_sync(0xffffffffu, pos0 + kTile - 1 <= P && (pos0 > P - p.window || pos0 + kTile <= p.n_sink));
#pragma unroll
          for (int c = 0; c < kTile / 64; ++c) {
            tm_ld64(lane_addr + 128 * b + 64 * c, sr[c]);
            if (full) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float4 k = kn4[16 * c + i];
                const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const float s = __uint_as_float(sr[c][4 * i + e]) * kk[e];
                  sr[c][4 * i + e] = __float_as_uint(s);
                  mx4[e] = fmaxf(mx4[e], s);
                }
              }
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float4 k = kn4[16 * c + i];
                const float kk[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  const int pos = pos0 + 64 * c + 4 * i + e;
                  const bool see = pos <= P && (pos > P - p.window || pos < p.n_sink);
                  const float s = see ? __uint_as_float(sr[c][4 * i + e]) * kk[e] : -INFINITY;
                  sr[c][4 * i + e] = __float_as_uint(s);
                  mx4[e] = fmaxf(mx4[e], s);
                }
              }
            }
          }
          const float mx = fmaxf(fmaxf(mx4[0], mx4[1]), fmaxf(mx4[2], mx4[3])) * fac;   // in log2 units
          const bool raise = mx > m_ref + Sh::kLazy;
          float alpha = 1.f;
          if (raise) {
            alpha = fast_exp2(m_ref - mx);
            m_ref = mx;
            l_sum *= alpha;
          }
          const float mu = m_ref == -INFINITY ? 0.f : m_ref;
          float l4[4] = {0.f, 0.f, 0.f, 0.f};
          // P over the scores: 32 columns per 64 positions (fp32: hi, then lo)
#pragma unroll
          for (int c = 0; c < kTile / 64; ++c) {
            uint32_t pk[32];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float4 v = vn4[16 * c + i];
              const float vv[4] = {v.x, v.y, v.z, v.w};
              float pw[4];
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const float s = __uint_as_float(sr[c][4 * i + e]);
                const float pr = fast_exp2(fmaf(s, fac, -mu));   // +0 when masked
                l4[e] += pr;
                pw[e] = pr * vv[e];
                if (!full) pw[e] = s == -INFINITY ? 0.f : pw[e];   // a masked position's norm may be anything
                if constexpr (kExact) sr[c][4 * i + e] = __float_as_uint(pw[e]);
              }
              pk[2 * i] = pack_half2(pw[0], pw[1]);
              pk[2 * i + 1] = pack_half2(pw[2], pw[3]);
            }
            tm_st32(lane_addr + 128 * b + 32 * c, pk);
            if constexpr (kExact) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float2 hi = __half22float2(*reinterpret_cast<const __half2*>(&pk[i]));
                pk[i] = pack_half2(__uint_as_float(sr[c][2 * i]) - hi.x, __uint_as_float(sr[c][2 * i + 1]) - hi.y);
              }
              tm_st32(lane_addr + 128 * b + 32, pk);
            }
          }
          l_sum += (l4[0] + l4[1]) + (l4[2] + l4[3]);
          tm_wait_st();
          if (j > 0) {   // PV(t - 1) has completed: O may be rescaled
            if (!(ok = warp_wait(bar(kRgVEmpty + ((t - 1) & 1)), ((t - 1) >> 1) & 1))) break;
            tc_fence_after();
            if (__any_sync(0xffffffffu, raise)) {
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                uint32_t ov[32];
                tm_ld32(lane_addr + kTmO + 32 * c, ov);
#pragma unroll
                for (int i = 0; i < 32; ++i) ov[i] = __float_as_uint(__uint_as_float(ov[i]) * alpha);
                tm_st32(lane_addr + kTmO + 32 * c, ov);
              }
              tm_wait_st();
            }
          }
          tc_fence_before();
          __syncwarp();
          // (test hook: the first P signals are withheld, so the issuer's wait for them runs out)
          if (lane == 0 && !(p.test_withhold && t < 2)) mbar_arrive_cluster(lead_bar0 + 8u * uint32_t(kRgPFull + b));
        }
        if (!ok) break;
        // ---- the item's rows: wait for its last PV; R^T; out
        if (!(ok = warp_wait(bar(kRgVEmpty + ((t - 1) & 1)), ((t - 1) >> 1) & 1))) break;
        tc_fence_after();
        const bool whole = g.part < 0;
        const float inv = !whole ? 0.0625f / Sh::kPScale : l_sum == 0.f ? 0.f : (0.0625f / Sh::kPScale) / l_sum;
        const int in_item = int(rank) * kPfRows + 32 * w;   // this warp's first row of the item
        if (!whole) p.pml[int64_t(g.part) * 256 + in_item + lane] = make_float2(m_ref, l_sum);
#pragma unroll
        for (int hp = 0; hp < 2; ++hp) {   // dims 128 hp ..: the transform's top level is a sum or a difference
#pragma unroll 1
          for (int c = 0; c < 4; ++c) {
            uint32_t a[32], d[32];
            tm_ld32(lane_addr + kTmO + 32 * c, a);
            tm_ld32(lane_addr + kTmO + 128 + 32 * c, d);
            float v[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = hp ? __uint_as_float(a[i]) - __uint_as_float(d[i]) : __uint_as_float(a[i]) + __uint_as_float(d[i]);
            fwht32(v);
#pragma unroll
            for (int i = 0; i < 8; ++i)   // row `lane` of [32][128] floats, 16-byte chunks swizzled by the row
              *reinterpret_cast<float4*>(stage + lane * 512 + (((8 * c + i) ^ lane) << 4)) =
                  make_float4(v[4 * i] * inv, v[4 * i + 1] * inv, v[4 * i + 2] * inv, v[4 * i + 3] * inv);
          }
          __syncwarp();
          const int li = lane & 15;
#pragma unroll 2
          for (int it = 0; it < 16; ++it) {   // two rows at a time: the two levels across the 32-dim chunks, signs, store
            const int rr = 2 * it + (lane >> 4);
            float2 x[4];
#pragma unroll
            for (int c = 0; c < 4; ++c)
              x[c] = *reinterpret_cast<const float2*>(stage + rr * 512 + (((8 * c + (li >> 1)) ^ rr) << 4) + (li & 1) * 8);
            if (in_item + rr < n_rows) {
              const float2 s0 = make_float2(x[0].x + x[1].x, x[0].y + x[1].y), d0 = make_float2(x[0].x - x[1].x, x[0].y - x[1].y);
              const float2 s1 = make_float2(x[2].x + x[3].x, x[2].y + x[3].y), d1 = make_float2(x[2].x - x[3].x, x[2].y - x[3].y);
              float2 y[4] = {make_float2(s0.x + s1.x, s0.y + s1.y), make_float2(d0.x + d1.x, d0.y + d1.y),
                             make_float2(s0.x - s1.x, s0.y - s1.y), make_float2(d0.x - d1.x, d0.y - d1.y)};
              const int ir = 256 * rb + in_item + rr, tok = rq.row0 + ir / 6, jh = ir % 6;
              const int64_t off = whole ? (int64_t(tok) * kHq + g.head * kGroup + jh) * kD : (int64_t(g.part) * 256 + in_item + rr) * kD;
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t sw = p.signs.bits[4 * hp + c] >> (2 * li);
                y[c].x = apply_sign(y[c].x, sw, 0);
                y[c].y = apply_sign(y[c].y, sw, 1);
                const int64_t o = off + 128 * hp + 32 * c + 2 * li;
                if (!whole) *reinterpret_cast<float2*>(p.po + o) = y[c];
                else if (kExact) *reinterpret_cast<float2*>(static_cast<float*>(p.out) + o) = y[c];
                else *reinterpret_cast<__nv_bfloat162*>(static_cast<uint16_t*>(p.out) + o) = __floats2bfloat162_rn(y[c].x, y[c].y);
              }
            }
          }
          __syncwarp();
        }
        asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");   // the next Q rows replace what was staged
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_local(bar(kRgEpi));
      }
    } else if (w == kRgKWarp || w == kRgVWarp) {
      // =========================================================== K tiles and norms; V tiles
      if (lane == 0) {
        const bool is_v = w == kRgVWarp;
        const int empty = is_v ? kRgVEmpty : kRgSFull, full0 = is_v ? kRgVFull : kRgKFull;
        int t = 0;
        bool ok = true;
        while (ok && walk.next(g)) {
          const RgReq rq = p.req[p.blk_req[g.blk]];
          const RgSpan span = rg_block_span<kTile>(p, rq, g.blk - rq.blk0);
          for (int j = 0; j < g.n; ++j, ++t) {
            const int at = g.tile + j, real = at < span.sinks ? at : at + span.skip;
            // the sinks' tiles of a block reach at most its request's, or there is no gap to skip
            const int64_t srow = int64_t(rq.tile0 + (real < rq.sink_tiles ? real : real - rq.skip)) * kTile;
            const int o = t - kStages, st = t % kStages;
            if (o >= 0 && !(ok = bounded_wait(bar(empty + (o & 1)), (o >> 1) & 1))) break;
            const uint32_t fb = bar(full0 + st);
            if (is_v) {
              mbar_expect_tx(fb, Sh::kParts * Sh::kVPart);
#pragma unroll
              for (int x = 0; x < Sh::kParts; ++x) {
                const uint32_t dst = sbase + Sh::kVOff + (st * Sh::kParts + x) * Sh::kVPart;
                const int64_t row = ((x * 2 + 1) * kHkv + g.head) * p.store_rows + srow;
#pragma unroll
                for (int d = 0; d < 2; ++d)
#pragma unroll
                  for (int y = 0; y < 2; ++y)
                    tma_load_2d(dst + d * Sh::kVPanel + y * (kTile / 2) * 128, &kvmap, 128 * int(rank) + 64 * d, int(row + y * (kTile / 2)), fb);
              }
            } else {
              mbar_expect_tx(fb, Sh::kParts * Sh::kKPart);
#pragma unroll
              for (int x = 0; x < Sh::kParts; ++x) {
                const uint32_t dst = sbase + Sh::kKOff + (st * Sh::kParts + x) * Sh::kKPart;
                const int64_t row = (x * 2 * kHkv + g.head) * p.store_rows + srow + int(rank) * (kTile / 2);
#pragma unroll
                for (int d = 0; d < 4; ++d) tma_load_2d(dst + d * Sh::kKPanel, &kvmap, 64 * d, int(row), fb);
              }
              // norms: slot t & 3 was read by tile t - 4, whose PV came before the QK just waited for
              const uint32_t nb = bar(kRgNFull + (t & 3)), nd = sbase + Sh::kNormOff + (t & 3) * 2 * kTile * 4;
              mbar_expect_tx(nb, 2 * kTile * 4);
              bulk_load(nd, p.norms + g.head * p.store_rows + srow, kTile * 4, nb);
              bulk_load(nd + kTile * 4, p.norms + (kHkv + g.head) * p.store_rows + srow, kTile * 4, nb);
            }
          }
        }
        if (misc[1]) {
          for (int o = max(t - kStages, 0); o < t; ++o) drain(bar(full0 + o % kStages), (o / kStages) & 1);
          if (!is_v)
            for (int o = max(t - kRgNormSlots, 0); o < t; ++o) drain(bar(kRgNFull + (o & 3)), (o >> 2) & 1);
        }
      }
    } else if (w == kRgQWarp) {
      // =========================================================== Q rows, one item at a time
      if (lane == 0) {
        int s = 0;
        while (walk.next(g)) {
          const RgReq rq = p.req[p.blk_req[g.blk]];
          const int64_t row = int64_t(g.head) * kGroup * p.n_tok + int64_t(rq.row0) * kGroup + 256 * (g.blk - rq.blk0) + int(rank) * kPfRows;
          if (s > 0 && !bounded_wait(bar(kRgEpi), (s - 1) & 1)) break;   // the last item's rows are out
          mbar_expect_tx(bar(kRgQFull), Sh::kParts * Sh::kQPart);
#pragma unroll
          for (int x = 0; x < Sh::kParts; ++x)
#pragma unroll
            for (int d = 0; d < 4; ++d)
              tma_load_2d(sbase + x * Sh::kQPart + d * Sh::kQPanel, &qmap, 64 * d, int(x * int64_t(kHq) * p.n_tok + row), bar(kRgQFull));
          ++s;
        }
        if (misc[1] && s > 0) drain(bar(kRgQFull), (s - 1) & 1);
      }
    } else if (rank == 1) {
      // =========================================================== rank 1: its copies have landed
      if (lane == 0) {
        int t = 0, s = 0;
        bool ok = true;
        while (ok && walk.next(g)) {
          if (!(ok = bounded_wait(bar(kRgQFull), s & 1))) break;
          mbar_arrive_cluster(lead_bar0 + 8u * uint32_t(kRgQPeer));
          ++s;
          for (int j = 0; ok && j <= g.n; ++j) {   // in the order in which rank 0 waits for them
            if (j < g.n) {
              const int u = t + j, st = u % kStages;
              if (!(ok = bounded_wait(bar(kRgKFull + st), (u / kStages) & 1))) break;
              mbar_arrive_cluster(lead_bar0 + 8u * uint32_t(kRgKPeer + st));
            }
            if (j > 0) {
              const int u = t + j - 1, st = u % kStages;
              if (!(ok = bounded_wait(bar(kRgVFull + st), (u / kStages) & 1))) break;
              mbar_arrive_cluster(lead_bar0 + 8u * uint32_t(kRgVPeer + st));
            }
          }
          t += g.n;
        }
      }
    } else {
      // =========================================================== rank 0: MMA issuer (one thread)
      if (lane == 0) {
        constexpr uint32_t idesc_qk = tc_idesc(2 * kPfRows, kTile, 0);
        constexpr uint32_t idesc_pv = tc_idesc(2 * kPfRows, kD, 1);
        const uint64_t q0 = tc_sdesc(sbase, 16, 1024);
        int t = 0, s = 0;
        bool ok = true;
        while (ok && walk.next(g)) {
          if (!(ok = bounded_wait(bar(kRgQFull), s & 1) && bounded_wait(bar(kRgQPeer), s & 1))) break;
          ++s;
          for (int j = 0; j <= g.n; ++j) {
            if (j < g.n) {   // S[u & 1] = Q K^T
              const int u = t + j, st = u % kStages;
              const uint32_t par = (u / kStages) & 1;
              if (!(ok = bounded_wait(bar(kRgKFull + st), par) && bounded_wait(bar(kRgKPeer + st), par))) break;
              tc_fence_after();
              const uint32_t s_t = tmem + 128 * (u & 1);
#pragma unroll
              for (int x = 0; x < (kExact ? 3 : 1); ++x) {   // Qh Kh, Ql Kh, Qh Kl
                const uint64_t qx = q0 + (x == 1 ? (Sh::kQPart >> 4) : 0);
                const uint64_t kx = tc_sdesc(sbase + Sh::kKOff + (st * Sh::kParts + (x == 2 ? 1 : 0)) * Sh::kKPart, 16, 1024);
#pragma unroll
                for (int kk = 0; kk < 16; ++kk)
                  tc2_mma_ss(s_t, qx + (((kk >> 2) * Sh::kQPanel + (kk & 3) * 32) >> 4), kx + (((kk >> 2) * Sh::kKPanel + (kk & 3) * 32) >> 4),
                             idesc_qk, (x > 0 || kk > 0) ? 1u : 0u);
              }
              tc2_commit_both(bar(kRgSFull + (u & 1)));
            }
            if (j > 0) {   // O += P V of tile j - 1
              const int u = t + j - 1, st = u % kStages;
              const uint32_t par = (u / kStages) & 1;
              if (!(ok = bounded_wait(bar(kRgVFull + st), par) && bounded_wait(bar(kRgVPeer + st), par) &&
                         bounded_wait(bar(kRgPFull + (u & 1)), (u >> 1) & 1)))
                break;
              tc_fence_after();
              const uint32_t p_t = tmem + 128 * (u & 1);
#pragma unroll
              for (int x = 0; x < (kExact ? 3 : 1); ++x) {   // Ph Vh, Pl Vh, Ph Vl
                const uint64_t vx = tc_sdesc(sbase + Sh::kVOff + (st * Sh::kParts + (x == 2 ? 1 : 0)) * Sh::kVPart, Sh::kVPanel, 1024);
#pragma unroll
                for (int ks = 0; ks < kTile / 16; ++ks)
                  tc2_mma_ts(tmem + kTmO, p_t + (x == 1 ? 32 : 0) + 8 * ks, vx + ((ks * 16 * 128) >> 4), idesc_pv,
                             (j > 1 || x > 0 || ks > 0) ? 1u : 0u);
              }
              tc2_commit_both(bar(kRgVEmpty + (u & 1)));
            }
          }
          t += g.n;
        }
        // every MMA that this thread issued has completed before TMEM is released
        tc2_commit_own(bar(kRgDrain));
        drain(bar(kRgDrain), 0);
      }
    }
  }
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();   // no MMA of the pair, no copy and no remote access is outstanding past this point
  tc_fence_after();
  if (w == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, 512;\n" ::"r"(tmem) : "memory");
}

// --------------------------------------------------------------------------
// combine: the rows of items that several pairs share. CTA (b, y) looks at the border before
// pair b + 1's share: where it is the first border inside an item, rows 32 y .. of that item
// are merged, o = sum_i 2^(m_i - m) o_i / sum_i 2^(m_i - m) l_i.
// --------------------------------------------------------------------------
template <bool kExact>
__global__ void __launch_bounds__(256) ragged_combine_kernel(const RaggedParams p) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int b = int(blockIdx.x) + 1;
  pdl_wait();
  pdl_launch_dependents();
  const int n_pairs = p.head->n_pairs;
  if (b >= n_pairs) return;
  const RgStart me = p.starts[b], prev = p.starts[b - 1];
  if (me.tile == 0) return;                                                        // no item is cut here
  if (prev.head == me.head && prev.blk == me.blk && prev.tile > 0) return;         // not its first cut
  const int part0 = 2 * (b - 1) + (prev.head == me.head && prev.blk == me.blk ? 0 : 1);
  int last = b;   // pairs b .. last hold the rest of the item, as their first stretch
  while (last + 1 < n_pairs) {
    const RgStart s = p.starts[last + 1];
    if (s.head != me.head || s.blk != me.blk) break;   // (its tile is then past 0)
    ++last;
  }
  const RgReq rq = p.req[p.blk_req[me.blk]];
  const int rb = me.blk - rq.blk0, n_rows = min(256, 6 * rq.n_new - 256 * rb);
#pragma unroll 1
  for (int x = 0; x < 4; ++x) {
    const int row = 32 * int(blockIdx.y) + 8 * x + w;
    if (row >= n_rows) break;
    float M = p.pml[int64_t(part0) * 256 + row].x;
    for (int i = b; i <= last; ++i) M = fmaxf(M, p.pml[int64_t(2 * i) * 256 + row].x);
    float L = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int i = b - 1; i <= last; ++i) {
      const int64_t rec = int64_t(i < b ? part0 : 2 * i) * 256 + row;
      const float2 ml = p.pml[rec];
      if (ml.x == -INFINITY && ml.y == 0.f) continue;   // that stretch showed this row nothing
      const float f = fast_exp2(ml.x - M);
      L = fmaf(f, ml.y, L);
      const float4* src = reinterpret_cast<const float4*>(p.po + rec * kD + lane * 8);
      const float4 a = src[0], c = src[1];
      o[0] = fmaf(f, a.x, o[0]); o[1] = fmaf(f, a.y, o[1]); o[2] = fmaf(f, a.z, o[2]); o[3] = fmaf(f, a.w, o[3]);
      o[4] = fmaf(f, c.x, o[4]); o[5] = fmaf(f, c.y, o[5]); o[6] = fmaf(f, c.z, o[6]); o[7] = fmaf(f, c.w, o[7]);
    }
    const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
    for (int i = 0; i < 8; ++i) o[i] *= inv;
    const int ir = 256 * rb + row;
    const int64_t off = (int64_t(rq.row0 + ir / 6) * kHq + me.head * kGroup + ir % 6) * kD + lane * 8;
    if constexpr (kExact) {
      float4* dst = reinterpret_cast<float4*>(static_cast<float*>(p.out) + off);
      dst[0] = make_float4(o[0], o[1], o[2], o[3]);
      dst[1] = make_float4(o[4], o[5], o[6], o[7]);
    } else {
      store8_bf16(static_cast<uint16_t*>(p.out) + off, o);
    }
  }
}

constexpr int kRgMaxReq = TQ4_RAGGED_MAX_REQUESTS;   // 8 B of the prep's shared memory each
inline cudaError_t ragged_set_attrs() {
  cudaError_t e = cudaSuccess;
  auto set = [&e](const void* k, size_t bytes) {
    if (e == cudaSuccess) e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, int(bytes));
  };
  set(reinterpret_cast<const void*>(ragged_prep_kernel<false>), kRgMaxReq * 8);
  set(reinterpret_cast<const void*>(ragged_prep_kernel<true>), kRgMaxReq * 8);
  set(reinterpret_cast<const void*>(ragged_attend_kernel<false>), RgShape<false>::kSmem);
  set(reinterpret_cast<const void*>(ragged_attend_kernel<true>), RgShape<true>::kSmem);
  return e;
}

template <bool kExact>
cudaError_t launch_ragged_t(RaggedParams& p, const CUtensorMap& qmap, const CUtensorMap& kvmap, const RgLayout& l, int num_sms, cudaStream_t st) {
  // units of the prep: at most 8 per row tile and one per token
  const int64_t units = l.store_rows / RgShape<kExact>::kTile * 8 + p.n_tok;
  const dim3 prep(unsigned(std::min<int64_t>(units, int64_t(num_sms) * 6) + 1));
  cudaError_t e = launch_pdl(ragged_prep_kernel<kExact>, prep, dim3(kRgPrepThreads), size_t(p.n_req) * 8, st, p);
  if (e != cudaSuccess) return e;
  e = launch_pdl(ragged_attend_kernel<kExact>, dim3(unsigned(2 * p.max_pairs)), dim3(kRgThreads), size_t(RgShape<kExact>::kSmem), st, p, qmap, kvmap);
  if (e != cudaSuccess || p.max_pairs < 2) return e;
  return launch_pdl(ragged_combine_kernel<kExact>, dim3(unsigned(p.max_pairs - 1), 8), dim3(256), 0, st, p);
}

}  // namespace tq4
