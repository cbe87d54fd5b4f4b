// The ragged serving step around the paged cache (sm_100a): block tables and slot
// maps from request lengths, rotary positions fused with encode + append by slot,
// and the stored vectors of a list of slots.
//
// A slot is page * 256 + position-in-page (int64); a negative slot means "no
// position" (padding, or a request that was refused). [BUDGET] and [STATE]
// (simpleprog.com "Fitting a 27B-Parameter LLM into 24 GiB of Laptop Memory",
// sections "The Memory Budget Equation" and "StateTrans") give the pages and the
// admission that these maps follow.
#pragma once
#include <algorithm>

#include "tq4_device.cuh"
#include "tq4_encode.cuh"

namespace tq4 {

// --------------------------------------------------------------------------
// plan_step: has = ceil(past / 256), need = ceil((past + new) / 256) pages;
// request r's fresh pages are free[start_r ..), start_r = sum of need - has over
// the requests before it. One launch: every CTA scans all requests (a few thousand
// at most: the scan costs less than a second launch would) and keeps first row,
// past length and first fresh page of each in shared memory; the tokens are then
// dealt out over the CTAs, each thread finding its token's request by bisection.
// Latency bound: launch + two dependent loads + the scan.
// --------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxReq = TQ4_PLAN_MAX_REQUESTS;   // 12 B of shared memory each
constexpr int kPlanTokens = 2048;    // tokens per CTA: two per thread

struct PlanParams {
  const int32_t* past;
  const int32_t* n_new;
  int32_t n_req;
  const int32_t* free_pages;
  int32_t n_free;
  int32_t num_pages;
  int32_t* tables;
  int32_t max_pages;
  int32_t* cu_tok;
  int32_t* seq_lens;
  int32_t* tok_pos;
  int64_t* tok_slot;
  int32_t max_tok;
  int32_t* taken;
  int* status;
};

__device__ __forceinline__ int64_t warp_scan_i64(int64_t v) {   // inclusive
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  return v;
}

__global__ void __launch_bounds__(kPlanThreads) plan_step_kernel(const PlanParams p) {
  extern __shared__ int32_t plan_smem[];
  __shared__ int64_t tot_n[32], tot_d[32];
  __shared__ int64_t carry_n, carry_d;
  __shared__ int32_t s_taken;
  int32_t* const row0 = plan_smem;               // first token row of each request, [n_req + 1]
  int32_t* const past_s = row0 + p.n_req + 1;    // cached positions
  int32_t* const fresh0 = past_s + p.n_req;      // first fresh page in the free list; -1: refused
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  if (tid == 0) {
    carry_n = carry_d = 0;
    s_taken = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  for (int base = 0; base < p.n_req; base += kPlanThreads) {
    const int r = base + tid;
    int64_t past = 0, nn = 0, d = 0;
    bool bad = false;
    if (r < p.n_req) {
      past = p.past[r];
      nn = p.n_new[r];
      bad = past < 0 || nn < 0 || past + nn > int64_t(p.max_pages) * kPage;
      nn = nn < 0 ? 0 : nn > p.max_tok ? int64_t(p.max_tok) + 1 : nn;   // its rows keep their place in the batch
      if (!bad) d = ((past + nn + kPage - 1) >> 8) - ((past + kPage - 1) >> 8);
    }
    int64_t sn = warp_scan_i64(nn), sd = warp_scan_i64(d);
    if (lane == 31) {
      tot_n[w] = sn;
      tot_d[w] = sd;
    }
    __syncthreads();
    if (w == 0) {
      tot_n[lane] = warp_scan_i64(tot_n[lane]);
      tot_d[lane] = warp_scan_i64(tot_d[lane]);
    }
    __syncthreads();
    const int64_t en = carry_n + (w ? tot_n[w - 1] : 0) + sn;   // rows up to and including r
    const int64_t ed = carry_d + (w ? tot_d[w - 1] : 0) + sd;   // fresh pages likewise
    if (r < p.n_req) {
      const bool rows_ok = !bad && en <= p.max_tok;
      const bool fits = rows_ok && (d == 0 || ed <= p.n_free);
      row0[r + 1] = int32_t(en < p.max_tok ? en : p.max_tok);
      past_s[r] = bad ? 0 : int32_t(past);
      fresh0[r] = fits ? int32_t(ed - d < p.n_free ? ed - d : p.n_free) : -1;
      if (blockIdx.x == 0) {
        p.seq_lens[r] = fits ? int32_t(past + nn) : 0;
        if (fits && d > 0) atomicMax(&s_taken, int32_t(ed));
        if (!rows_ok) record_error(p.status, TQ4_ERR_SEQ);
        else if (!fits) record_error(p.status, TQ4_ERR_NO_PAGES);
      }
    }
    __syncthreads();
    if (tid == 0) {
      carry_n += tot_n[31];
      carry_d += tot_d[31];
    }
    __syncthreads();
  }
  if (tid == 0) row0[0] = 0;
  __syncthreads();
  const int total = row0[p.n_req];
  if (blockIdx.x == 0) {
    for (int r = tid; r <= p.n_req; r += kPlanThreads) p.cu_tok[r] = row0[r];
    if (tid == 0) *p.taken = s_taken;
  }
  // fresh table entries: one warp per request, the requests dealt out over all CTAs
  for (int r = int(blockIdx.x) * (kPlanThreads / 32) + w; r < p.n_req; r += int(gridDim.x) * (kPlanThreads / 32)) {
    const int f0 = fresh0[r];
    if (f0 < 0) continue;
    const int has = (past_s[r] + kPage - 1) >> 8, need = (past_s[r] + row0[r + 1] - row0[r] + kPage - 1) >> 8;
    for (int i = has + lane; i < need; i += 32) p.tables[int64_t(r) * p.max_pages + i] = p.free_pages[f0 + i - has];
  }
  // tokens: position and slot; the page comes from the table (cached positions) or straight
  // from the free list, so no CTA reads an entry that another one writes
  const int64_t stride = int64_t(gridDim.x) * kPlanThreads;
  for (int64_t i = int64_t(blockIdx.x) * kPlanThreads + tid; i < p.max_tok; i += stride) {
    int32_t pos = 0;
    int64_t slot = -1;
    if (i < total) {
      int lo = 0, hi = p.n_req - 1;   // the last request whose first row is at or before i and which has rows
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (row0[mid] <= i) lo = mid;
        else hi = mid - 1;
      }
      pos = past_s[lo] + int32_t(i) - row0[lo];
      const int f0 = fresh0[lo];
      if (f0 >= 0) {
        const int has = (past_s[lo] + kPage - 1) >> 8, pg = pos >> 8;
        const int32_t page = pg < has ? p.tables[int64_t(lo) * p.max_pages + pg] : p.free_pages[f0 + pg - has];
        if (page >= 0 && page < p.num_pages) slot = int64_t(page) * kPage + (pos & (kPage - 1));
        else record_error(p.status, TQ4_ERR_PAGE_RANGE);
      }
    }
    p.tok_pos[i] = pos;
    p.tok_slot[i] = slot;
  }
}

inline size_t plan_smem_bytes(int32_t n_req) { return size_t(3 * size_t(n_req) + 1) * sizeof(int32_t); }
inline cudaError_t plan_set_attrs() {
  return cudaFuncSetAttribute(plan_step_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                              int(plan_smem_bytes(kPlanMaxReq)));
}
inline cudaError_t launch_plan_step(const PlanParams& p, int num_sms, cudaStream_t st) {
  const int64_t ctas = std::min<int64_t>(std::max<int64_t>((int64_t(p.max_tok) + kPlanTokens - 1) / kPlanTokens, 1), num_sms);
  return launch_pdl(plan_step_kernel, dim3(unsigned(ctas)), dim3(kPlanThreads), plan_smem_bytes(p.n_req), st, p);
}

// --------------------------------------------------------------------------
// rope_table: {cos, sin}(pos * base^(-2 i / rot)) for pos < len, i < rot / 2. The
// angle is formed and reduced in 64 bits (at position 229,376 a 32-bit angle is off
// by up to 2^-7), then rounded to fp32.
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(256) rope_table_kernel(float2* table, int64_t n, int half, double base) {
  const int64_t e = int64_t(blockIdx.x) * 256 + threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  if (e >= n) return;
  const int64_t pos = e / half;
  const int i = int(e - pos * half);
  double s, c;
  sincos(double(pos) * pow(base, -double(i) / double(half)), &s, &c);
  table[e] = make_float2(float(c), float(s));
}

// --------------------------------------------------------------------------
// rope_append. Per token: 24 query heads and 4 key heads are rotated by position,
// q (and on request k) go out in bf16 rounded once, and the rotated keys and the
// values are encoded into the token's slot.
//
// Quantiser decisions equal the 64-bit definition. The 32-bit path bounds its own
// error: with u = 2^-24 and ||x||_1 <= 16 ||x||_2, the rotation of a pair adds 3 u,
// the norm 9 u (times |y| <= 0.16 next to a boundary), the scaling u and the eight
// Hadamard levels 8 u of ||x||_1 / 16, together under 8e-7 of the unit vector. A
// vector with a coordinate within 1e-6 of a boundary (one in ~40 of Gaussian ones),
// or whose norm lies within 6e-7 (relative) of an fp16 rounding midpoint, is redone
// in 64 bits by the whole warp.
//
// One CTA of 12 warps per token: warps 0-3 six query heads each (their six row loads
// fly together), warps 4-7 the keys, 8-11 the values: an encode costs about as many
// instructions as six rotations, so the three groups end together.
// --------------------------------------------------------------------------
constexpr int kRopeWarps = 12;
constexpr float kRopeNear = 1e-6f;      // coordinates closer to a boundary are decided in 64 bits
constexpr float kRopeNormNear = 6e-7f;  // and norms closer (relative) to an fp16 midpoint
__constant__ double g_boundaries64[15]; // decision boundaries in 64 bits

struct RopeParams {
  uint8_t* pool;
  int32_t num_pages;
  const void* q;       // nullptr: no queries
  const void* k;
  const void* v;
  int64_t q_stride, k_stride, v_stride;   // elements between tokens
  int32_t n_tok;
  const int32_t* pos;  // [n_axes][n_tok]
  int32_t n_axes;
  const float2* table; // [table_len][rot / 2]
  int32_t table_len;
  int32_t rot;
  int32_t adjacent;    // 0: pairs (i, i + rot / 2); 1: pairs (2 i, 2 i + 1)
  uint32_t axis[8];    // two bits per frequency
  const int64_t* slots;
  uint16_t* q_out;
  uint16_t* k_out;     // nullptr: not wanted
  Signs signs;
  int* status;
};

// 8 elements; plain loads, since q_out may be q itself
template <typename T>
__device__ __forceinline__ void load8_rw(const T* src, float v[8]);
template <>
__device__ __forceinline__ void load8_rw<float>(const float* src, float v[8]) {
  const float4 a = reinterpret_cast<const float4*>(src)[0], b = reinterpret_cast<const float4*>(src)[1];
  v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
template <>
__device__ __forceinline__ void load8_rw<uint16_t>(const uint16_t* src, float v[8]) {
  const uint4 a = *reinterpret_cast<const uint4*>(src);
  const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void store8_bf16(uint16_t* dst, const float v[8]) {
  uint32_t pk[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __nv_bfloat162 b2 = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    pk[i] = *reinterpret_cast<const uint32_t*>(&b2);
  }
  *reinterpret_cast<uint4*>(dst) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
}

// The encode of one vector in 64 bits (x: the rotated vector's coordinates 8 lane ..).
__device__ __noinline__ void encode_vector_warp64(const double* x, uint32_t sb, uint32_t& word, uint16_t& norm) {
  const int lane = threadIdx.x & 31;
  double ss = 0.0, y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fma(x[i], x[i], ss);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  const double n = sqrt(ss);
  word = 0;
  norm = __half_as_ushort(__double2half(n));
  if (!(n > 0.0)) return;   // the same in every lane
#pragma unroll
  for (int i = 0; i < 8; ++i) y[i] = ((sb >> i) & 1u) ? -x[i] / n : x[i] / n;
#pragma unroll
  for (int h = 1; h < 8; h <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if ((i & h) == 0) {
        const double a = y[i], b = y[i + h];
        y[i] = a + b;
        y[i + h] = a - b;
      }
#pragma unroll
  for (int m = 1; m < 32; m <<= 1)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double o = __shfl_xor_sync(0xffffffffu, y[i], m);
      y[i] = (lane & m) ? o - y[i] : y[i] + o;
    }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t idx = 0;
#pragma unroll
    for (int j = 0; j < 15; ++j) idx += (y[i] * 0.0625 > g_boundaries64[j]) ? 1u : 0u;
    word |= idx << (4 * i);
  }
}

// Rotation angles of one lane: c[i], s[i] for its coordinates 8 lane + i (halves: one
// frequency per coordinate; adjacent: one per pair, in entries 0-3). partner: the lane
// with the other half of its pairs; sgn: -1 on the first half, +1 on the second.
struct LaneAngles {
  float c[8], s[8];
  int partner;
  bool active;
};
// false: a position outside the table (the same in every lane of the CTA)
__device__ __forceinline__ bool load_angles(const RopeParams& p, int tok, LaneAngles& a) {
  const int lane = threadIdx.x & 31, half = p.rot >> 1;
  int32_t pos[3];
  bool ok = true;
#pragma unroll
  for (int x = 0; x < 3; ++x) {
    pos[x] = x < p.n_axes ? __ldg(p.pos + int64_t(x) * p.n_tok + tok) : 0;
    ok &= pos[x] >= 0 && pos[x] < p.table_len;
  }
  if (!ok) return false;
  a.active = 8 * lane < p.rot;
  const int per = p.adjacent ? 4 : 8;      // frequencies of this lane
  const int m = half >> 3;                 // lanes per half
  const int f0 = p.adjacent ? 4 * lane : 8 * (lane < m ? lane : lane - m);
  a.partner = p.adjacent || !a.active ? lane : lane < m ? lane + m : lane - m;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    a.c[i] = 1.f;
    a.s[i] = 0.f;
    if (a.active && i < per) {
      const int f = f0 + i;
      int32_t at = pos[0];
      if (p.n_axes > 1) {
        uint32_t wa = p.axis[0];
#pragma unroll
        for (int k = 1; k < 8; ++k) wa = (f >> 4) == k ? p.axis[k] : wa;
        const uint32_t ax = (wa >> (2 * (f & 15))) & 3u;
        at = ax == 0 ? pos[0] : ax == 1 ? pos[1] : pos[2];
      }
      const float2 cs = __ldg(p.table + int64_t(at) * half + f);
      a.c[i] = cs.x;
      a.s[i] = !p.adjacent && lane < m ? -cs.y : cs.y;   // first half: x cos - partner sin
    }
  }
  return true;
}
__device__ __forceinline__ void rotate8(const LaneAngles& a, bool adjacent, float x[8]) {
  if (adjacent) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = x[2 * j], w = x[2 * j + 1];
      if (a.active) {
        x[2 * j] = u * a.c[j] - w * a.s[j];
        x[2 * j + 1] = w * a.c[j] + u * a.s[j];
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float o = __shfl_sync(0xffffffffu, x[i], a.partner);
      if (a.active) x[i] = x[i] * a.c[i] + o * a.s[i];   // the other dims pass as they are, infinities too
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kRopeWarps) rope_append_kernel(const RopeParams p) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int tok = blockIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const int64_t slot = __ldg(p.slots + tok);
  if (slot < 0) return;   // padding, or a refused request: every row of it is left as it was
  if (slot >= int64_t(p.num_pages) * kPage) {
    if (threadIdx.x == 0) record_error(p.status, TQ4_ERR_PAGE_RANGE);
    return;
  }
  LaneAngles a;
  if (w < 8 && !load_angles(p, tok, a)) {
    if (threadIdx.x == 0) record_error(p.status, TQ4_ERR_SEQ);
    return;
  }
  const bool adjacent = p.adjacent != 0;
  if (w < 4) {
    if (!p.q) return;
    float x[kGroup][8];
    const T* src = static_cast<const T*>(p.q) + int64_t(tok) * p.q_stride + w * kGroup * kD + lane * 8;
#pragma unroll
    for (int j = 0; j < kGroup; ++j) load8_rw<T>(src + j * kD, x[j]);
#pragma unroll
    for (int j = 0; j < kGroup; ++j) {
      rotate8(a, adjacent, x[j]);
      store8_bf16(p.q_out + (int64_t(tok) * kHq + w * kGroup + j) * kD + lane * 8, x[j]);
    }
    return;
  }
  const int kv = (w - 4) >> 2, head = w & 3;
  if (kv == 1) {   // values are not rotated; their warps check the positions too, so that a
    bool ok = true; // bad one leaves the whole token unwritten
    for (int x = 0; x < p.n_axes; ++x) {
      const int32_t at = __ldg(p.pos + int64_t(x) * p.n_tok + tok);
      ok &= at >= 0 && at < p.table_len;
    }
    if (!ok) return;
  }
  float raw[8], x[8];
  load8_rw<T>(static_cast<const T*>(kv ? p.v : p.k) + int64_t(tok) * (kv ? p.v_stride : p.k_stride) + head * kD + lane * 8, raw);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = raw[i];
  if (kv == 0) {
    rotate8(a, adjacent, x);
    if (p.k_out) store8_bf16(p.k_out + (int64_t(tok) * kHkv + head) * kD + lane * 8, x);
  }
  const uint32_t sb = lane_sign_bits(p.signs);
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, m);
  const float n = sqrtf(ss);
  uint32_t word = 0;
  uint16_t norm = __half_as_ushort(__float2half_rn(n));
  // sums of squares outside [2^-100, 2^126] (and NaN) have lost digits in 32 bits
  bool redo = ss != 0.f && !(ss > 0x1p-100f && ss < 0x1p126f);
  redo |= __half_as_ushort(__float2half_rn(n * (1.f - kRopeNormNear))) != __half_as_ushort(__float2half_rn(n * (1.f + kRopeNormNear)));
  if (!redo && ss > 0.f) {
    const float inv = 1.0f / n;
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = apply_sign(x[i] * inv, sb, i);
    warp_fwht256(y);
    float near = 1.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float yi = y[i] * 0.0625f;
      uint32_t idx = 0;
#pragma unroll
      for (int j = 0; j < 15; ++j) {
        const float d = yi - g_codebook.b[j];
        idx += d > 0.f ? 1u : 0u;
        near = fminf(near, fabsf(d));
      }
      word |= idx << (4 * i);
    }
    redo = __any_sync(0xffffffffu, near < kRopeNear);
  } else if (ss == 0.f) {   // all zeros, or squares below the fp32 range
    bool any = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) any |= x[i] != 0.f;
    redo = __any_sync(0xffffffffu, any);
  }
  if (redo) {   // uniform in the warp
    double xd[8];
    if (kv == 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) xd[i] = raw[i];
    } else if (adjacent) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const double u = raw[2 * j], v = raw[2 * j + 1], c = a.c[j], s = a.s[j];
        xd[2 * j] = a.active ? u * c - v * s : u;
        xd[2 * j + 1] = a.active ? v * c + u * s : v;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float o = __shfl_sync(0xffffffffu, raw[i], a.partner);
        xd[i] = a.active ? double(raw[i]) * double(a.c[i]) + double(o) * double(a.s[i]) : double(raw[i]);
      }
    }
    encode_vector_warp64(xd, sb, word, norm);
  }
  uint8_t* page = p.pool + (slot >> 8) * kPageBytes;
  const int at = head * kPage + int(slot & (kPage - 1));
  reinterpret_cast<uint32_t*>(page + (kv ? kVWords : kKWords))[at * kWords + lane] = word;
  if (lane == 0) reinterpret_cast<uint16_t*>(page + (kv ? kVNorms : kKNorms))[at] = norm;
}

// --------------------------------------------------------------------------
// reconstruct_slots: x_hat = fp16 norm * R^T c[idx] of the vectors in each slot, fp32
// or bf16 (rounded once); a negative slot gives zeros. One warp per vector.
// --------------------------------------------------------------------------
__global__ void __launch_bounds__(256) reconstruct_slots_kernel(const uint8_t* __restrict__ pool, int32_t num_pages,
                                                                const int64_t* __restrict__ slots, int32_t n, void* k_out,
                                                                void* v_out, int out_dtype, Signs signs, int* status) {
  __shared__ float cb[16];
  if (threadIdx.x < 16) cb[threadIdx.x] = g_codebook.c[threadIdx.x];
  __syncthreads();
  const int lane = threadIdx.x & 31;
  const int64_t vec = int64_t(blockIdx.x) * 8 + (threadIdx.x >> 5);
  pdl_wait();
  pdl_launch_dependents();
  const int64_t i = vec >> 3;
  if (i >= n) return;
  const int kv = int(vec >> 2) & 1, head = int(vec) & 3;
  const int64_t slot = __ldg(slots + i);
  float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
  if (slot >= int64_t(num_pages) * kPage) {
    if (lane == 0) record_error(status, TQ4_ERR_PAGE_RANGE);
  } else if (slot >= 0) {
    const uint8_t* page = pool + (slot >> 8) * kPageBytes;
    const int at = head * kPage + int(slot & (kPage - 1));
    const uint32_t word = reinterpret_cast<const uint32_t*>(page + (kv ? kVWords : kKWords))[at * kWords + lane];
    const float nrm = __half2float(reinterpret_cast<const __half*>(page + (kv ? kVNorms : kKNorms))[at]) * 0.0625f;
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = cb[(word >> (4 * j)) & 15u];
    warp_fwht256(y);
    const uint32_t sb = lane_sign_bits(signs);
#pragma unroll
    for (int j = 0; j < 8; ++j) y[j] = apply_sign(y[j] * nrm, sb, j);
  }
  const int64_t off = (i * kHkv + head) * kD + lane * 8;
  if (out_dtype == TQ4_DTYPE_F32) {
    float4* dst = reinterpret_cast<float4*>(static_cast<float*>(kv ? v_out : k_out) + off);
    dst[0] = make_float4(y[0], y[1], y[2], y[3]);
    dst[1] = make_float4(y[4], y[5], y[6], y[7]);
  } else {
    store8_bf16(static_cast<uint16_t*>(kv ? v_out : k_out) + off, y);
  }
}

inline cudaError_t launch_rope_append(const RopeParams& p, int dtype, cudaStream_t st) {
  const dim3 grid(unsigned(p.n_tok)), block(32 * kRopeWarps);
  return dtype == TQ4_DTYPE_F32 ? launch_pdl(rope_append_kernel<float>, grid, block, 0, st, p)
                                : launch_pdl(rope_append_kernel<uint16_t>, grid, block, 0, st, p);
}
inline cudaError_t launch_reconstruct_slots(const uint8_t* pool, int32_t num_pages, const int64_t* slots, int32_t n,
                                            void* k_out, void* v_out, int out_dtype, const Signs& signs, int* status,
                                            cudaStream_t st) {
  return launch_pdl(reconstruct_slots_kernel, dim3(unsigned(n)), dim3(256), 0, st, pool, num_pages, slots, n, k_out,
                    v_out, out_dtype, signs, status);
}
inline cudaError_t launch_rope_table(float2* table, int64_t len, int rot, double base, cudaStream_t st) {
  const int64_t n = len * (rot / 2);
  return launch_pdl(rope_table_kernel, dim3(unsigned((n + 255) / 256)), dim3(256), 0, st, table, n, rot / 2, base);
}

}  // namespace tq4
