// kv_cache.cu — operators around the paged cache for sm_103a: rotary positions with the append of the
// new rows, expansion of 4-bit blocks to bf16, and block copies.
#include <cuda_runtime.h>

#include <algorithm>
#include <climits>
#include <cstring>
#include <new>
#include <vector>

#include "launch.cuh"
#include "pod_internal.h"
#include "ptx.cuh"

namespace pod {

using namespace ptx;

namespace {

// ============================================================================ rotary + append
struct RopeAppendArgs {
  const uint16_t* q;  // NULL: k and v only
  const uint16_t* k;
  const uint16_t* v;
  int64_t q_stride, k_stride, v_stride;
  uint16_t* q_prefill;
  uint16_t* q_decode;
  uint8_t* k_pool;
  uint8_t* v_pool;
  const float* k_scale;
  float* v_scale;
  const int32_t* block_tables;
  const int32_t* new_rows;  // (sequence, position) per token
  int32_t* status;
  int32_t T, Tp, Hq, Hkv, maxb, num_blocks;
  int32_t rows;              // most heads of one warp's work
  int32_t q_parts, kv_parts; // a token's works: q_parts of its q heads, kv_parts of k, kv_parts of v
  int32_t rot;               // rotated channels (0: none)
  int32_t adjacent;          // nonzero: pairs (2i, 2i + 1)
  float mag;
  uint64_t turns[kHeadDim / 2];  // 2^-64 turns per position
};

// How a lane's 8 channels of a head lie, and with it how their partners are reached.
enum RopeLayout {
  kHalf = 0,         // pairs (i, i + rot / 2), rot a multiple of 8: a lane holds 4 pairs
  kInterleaved = 1,  // pairs (2i, 2i + 1), rot a multiple of 8 (0: no rotation): 8 neighbours, 4 pairs
  kAny = 2           // any even rot, either kind: 8 neighbours, partners through shared memory
                     // (16384 tokens of 32 + 2 x 4 heads: 117 us, the others 58 and 55 us)
};

// Eight channels of one head in fp32 and as they were read.
struct Oct {
  uint4 raw;
  float x[8];
  __device__ __forceinline__ void unpack() {
    x[0] = bf16lo(raw.x), x[1] = bf16hi(raw.x), x[2] = bf16lo(raw.y), x[3] = bf16hi(raw.y);
    x[4] = bf16lo(raw.z), x[5] = bf16hi(raw.z), x[6] = bf16lo(raw.w), x[7] = bf16hi(raw.w);
  }
  __device__ __forceinline__ void pack() {
    raw = make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                     pack_bf16x2(x[6], x[7]));
  }
};

// cos and sin, times the attention factor, of one pair's angle at a position. Position times a 64-bit
// fraction of a turn wraps around modulo a turn by itself, so far positions lose only what the 53 bits of
// the frequency's quotient by 2 pi leave. Its top 32 bits split into the nearest quarter turn and a rest x of
// at most pi / 4, exact in the integer; there the Taylor series to x^9 and x^8 are off by 2^-29 and 2^-25,
// and quarter turns swap and negate.
// kFine: the radians are x + e, e being what rounding x left (the integer's two parts are exact in fp32, and
// so are the remainders of the products), and cos has its x^10 term. sin is then good to 0.8 units in the
// last place instead of 1.4, cos to 1.1 instead of 1.4. e4m3 K rows are rotated with it: of a million codes
// 1.1 instead of 1.5 fall on the other side of a tie than in 64 bits, for about 2 % more time (8000 tokens, 8
// kv-heads). q is rotated without it whatever the cache; bf16 rows round it away and e2m1 codes do not
// change with it.
template <bool kFine>
__device__ __forceinline__ void angle(uint64_t turn, int pos, float mag, float& c, float& s) {
  constexpr float kUnit = 1.46291807926715968e-9f;  // 2 pi / 2^32
  constexpr float kRest = -4.07094043e-17f;         // ... less what fp32 holds of it
  const uint32_t f = (uint32_t)(((uint64_t)(uint32_t)pos * turn) >> 32);
  const uint32_t quarter = (f + 0x20000000u) >> 30;
  const int32_t n = (int32_t)(f - (quarter << 30));
  float x, e = 0.f;
  if constexpr (kFine) {
    const float hi = (float)(n & ~0xFF), lo = (float)(n & 0xFF), y = hi * kUnit;
    e = fmaf(lo, kUnit, fmaf(hi, kRest, fmaf(hi, kUnit, -y)));
    x = y + e;
    e -= x - y;
  } else {
    x = (float)n * kUnit;
  }
  const float z = x * x;
  float sn = fmaf(z, 1.f / 362880, -1.f / 5040);
  sn = fmaf(sn, z, 1.f / 120);
  sn = fmaf(sn, z, -1.f / 6);
  sn = (kFine ? x + fmaf(sn * z, x, e) : fmaf(sn * z, x, x)) * mag;
  float cs = fmaf(z, kFine ? fmaf(z, -1.f / 3628800, 1.f / 40320) : 1.f / 40320, -1.f / 720);
  cs = fmaf(cs, z, 1.f / 24);
  cs = fmaf(cs, z, -.5f);
  cs = fmaf(cs, z, 1.f) * mag;
  s = quarter & 1 ? cs : sn;
  c = quarter & 1 ? sn : cs;
  if (quarter & 2) s = -s;
  if ((quarter + 1) & 2) c = -c;
}

// A row of a quantised cache: the lane's 8 neighbouring channels ch .. ch + 7 of kv-head g, of row
// `slot` in unit `unit` of the pool. The lanes of a row are HD / 8 neighbours.
template <int KV, int HD>
__device__ __forceinline__ void store_quantised(const RopeAppendArgs& a, const float (&x)[8], int ch,
                                                bool is_v, int g, size_t unit, int slot, bool live) {
  uint8_t* pool = is_v ? a.v_pool : a.k_pool;
  if constexpr (KV == POD_ATTN_KV_E4M3) {
    const size_t at = unit * kBlockSize + slot;
    float d[8];
    if (is_v) {
      float amax = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) amax = fmaxf(amax, fabsf(x[j]));
#pragma unroll
      for (int off = HD / 16; off > 0; off >>= 1)
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, off));
      const float s = amax > 0.f ? __fdiv_rn(amax, 448.f) : 1.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) d[j] = s;
      if (live && ch == 0) a.v_scale[at] = s;
    } else {
      const float4* ks = reinterpret_cast<const float4*>(a.k_scale + (size_t)g * HD + ch);
      const float4 u = ks[0], w = ks[1];
      d[0] = u.x, d[1] = u.y, d[2] = u.z, d[3] = u.w, d[4] = w.x, d[5] = w.y, d[6] = w.z, d[7] = w.w;
    }
    uint32_t o[2];
#pragma unroll
    for (int j = 0; j < 2; ++j)
      o[j] = (uint32_t)e4m3x2_from_f32(__fdiv_rn(x[4 * j], d[4 * j]), __fdiv_rn(x[4 * j + 1], d[4 * j + 1])) |
             ((uint32_t)e4m3x2_from_f32(__fdiv_rn(x[4 * j + 2], d[4 * j + 2]),
                                        __fdiv_rn(x[4 * j + 3], d[4 * j + 3])) << 16);
    if (live) *reinterpret_cast<uint2*>(pool + at * HD + ch) = make_uint2(o[0], o[1]);
  } else {
    // a group of 16 channels is two neighbouring lanes; magnitudes are compared as integers, so that
    // a NaN (above the infinity's bits) wins
    uint32_t amax = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(x[j]) & 0x7FFFFFFFu);
    amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    const float h = (is_v ? a.v_scale : a.k_scale)[g];
    const bool nan = amax > 0x7F800000u;
    const uint32_t s8 =
        nan ? 0x7Fu : e4m3x2_from_f32(__fdiv_rn(__fdiv_rn(__uint_as_float(amax), h), 6.f), 0.f) & 0xFFu;
    const float div = f16lo(e4m3x2_to_f16x2(s8)) * h;
    uint32_t code = 0;
    if (s8 != 0 && !nan) {
#pragma unroll
      for (int j = 0; j < 8; j += 2)
        code |= e2m1x2_from_f32(__fdiv_rn(x[j], div), __fdiv_rn(x[j + 1], div)) << (4 * j);
    }
    if (!live) return;
    uint8_t* u = pool + unit * (9 * HD);
    *reinterpret_cast<uint32_t*>(u + slot * (HD / 2) + ch / 2) = code;
    if (ch % 16 == 0)
      u[8 * HD + (is_v ? ch : slot) * (is_v ? 1 : HD / 16) + (is_v ? slot : ch / 16)] = (uint8_t)s8;
  }
}

// One warp's work is up to `rows` heads of one token's q, k or v: 256 / HD heads at a time, HD / 8
// lanes each, with the loads of kRopeBatch such steps in flight. The angles of a lane's pairs are
// computed once per work and serve all its heads. Bound by memory on a bf16 cache (16380 tokens of 32 +
// 2 x 32 heads, 64 of 128 channels rotated: 118 us from call to call, the measured copy rate; 16384 of 32 + 2
// x 4: 58 us, 85 %). Bound by instructions on the others: of 16380 tokens of 32 + 2 x 32 heads the e4m3 cache
// takes 207 us (48 %), e2m1 214 us (42 %), with an instruction issued in 72 % of the cycles, the ALU pipe busy in
// 43 to 45 % and the memory at a third (8000 of 32 + 2 x 8 heads in e4m3: 47.7 us, 56 %). More CTAs an SM with
// fewer registers, or fewer steps in flight, were slower (16380 tokens in bf16: 140 to 157 us).
constexpr int kRopeBatch = 4;
constexpr int kRopeWarps = 8;
constexpr int kRopeCtas = 4;  // CTAs an SM holds

template <int KV, int HD, int LAYOUT>
__global__ void __launch_bounds__(kRopeWarps * 32, kRopeCtas)
    rope_append_kernel(const __grid_constant__ RopeAppendArgs a) {
  griddep_wait();
  constexpr int kLanes = HD / 8;        // lanes of a head
  constexpr int kStep = 32 / kLanes;    // heads of a step
  // rotated rows on their way to neighbouring channels (kAny: rows before their rotation, too)
  constexpr bool kStage = LAYOUT == kAny || (LAYOUT == kHalf && KV != POD_ATTN_KV_BF16);
  __shared__ __align__(16) float stage[kStage ? kRopeWarps : 1][kStage ? kStep : 1][HD];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int l = lane % kLanes, sub = lane / kLanes, h = a.rot / 2;
  // channels of the lane: c0 .. + 3 and c1 .. + 3
  const bool on = LAYOUT == kHalf ? l < a.rot / 8 : 8 * l < a.rot;  // kAny: some of them rotate
  const int c0 = LAYOUT == kHalf && on ? 4 * l : 8 * l;
  const int c1 = LAYOUT == kHalf && on ? 4 * l + h : 8 * l + 4;
  constexpr int kAngles = LAYOUT == kAny ? 8 : 4;
  uint64_t turn[kAngles];
#pragma unroll
  for (int j = 0; j < kAngles; ++j) {
    int i = 4 * l + j;
    if constexpr (LAYOUT == kAny) {
      const int ch = 8 * l + j;
      i = a.adjacent ? ch / 2 : ch < h ? ch : ch - h;
      turn[j] = ch < a.rot ? a.turns[i] : 0;
    } else {
      turn[j] = on ? a.turns[i] : 0;
    }
  }
  const int parts = a.q_parts + 2 * a.kv_parts;
  const int64_t works = (int64_t)a.T * parts;
  for (int64_t w = (int64_t)blockIdx.x * kRopeWarps + warp; w < works;
       w += (int64_t)gridDim.x * kRopeWarps) {
    const int tok = (int)(w / parts);
    int part = (int)(w % parts);
    int what = 0;  // 0 q, 1 k, 2 v
    if (part >= a.q_parts) {
      part -= a.q_parts;
      what = part >= a.kv_parts ? 2 : 1;
      if (what == 2) part -= a.kv_parts;
    }
    const int heads = what == 0 ? a.Hq : a.Hkv;
    const int h0 = part * a.rows, h1 = min(heads, h0 + a.rows);
    const uint16_t* src = (what == 0   ? a.q + (int64_t)tok * a.q_stride
                           : what == 1 ? a.k + (int64_t)tok * a.k_stride
                                       : a.v + (int64_t)tok * a.v_stride);
    const int pos = a.new_rows[2 * tok + 1];
    int phys = 0;
    if (what != 0) {
      phys = a.block_tables[(size_t)a.new_rows[2 * tok] * a.maxb + pos / kBlockSize];
      if (phys < 0 || phys >= a.num_blocks) {
        if (lane == 0) record_error(a.status, POD_ATTN_ERR_BAD_INDEX);
        continue;
      }
    }
    const int slot = pos % kBlockSize;
    // v rows are not rotated: 8 neighbours a lane, whatever the layout
    const bool turned = what != 2 && a.rot > 0;
    const int a0 = turned ? c0 : 8 * l, a1 = turned ? c1 : 8 * l + 4;
    float c[kAngles], s[kAngles];
    if (turned) {
      if (KV == POD_ATTN_KV_E4M3 && what == 1) {
#pragma unroll
        for (int j = 0; j < kAngles; ++j) angle<true>(turn[j], pos, a.mag, c[j], s[j]);
      } else {
#pragma unroll
        for (int j = 0; j < kAngles; ++j) angle<false>(turn[j], pos, a.mag, c[j], s[j]);
      }
    }
    uint16_t* dst;       // bf16 rows: head r at dst + r * pitch
    int64_t pitch = HD;
    if (what == 0) {
      dst = tok < a.Tp ? a.q_prefill + (int64_t)tok * a.Hq * HD
                       : a.q_decode + (int64_t)(tok - a.Tp) * a.Hq * HD;
    } else {
      pitch = kBlockSize * HD;
      dst = reinterpret_cast<uint16_t*>(what == 1 ? a.k_pool : a.v_pool) +
            ((int64_t)phys * a.Hkv * kBlockSize + slot) * HD;
    }
    for (int r0 = h0; r0 < h1; r0 += kStep * kRopeBatch) {
      Oct o[kRopeBatch];
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b) {
        const int r = r0 + b * kStep + sub;
        o[b].raw = make_uint4(0u, 0u, 0u, 0u);
        if (r < h1) {
          const uint16_t* p = src + (int64_t)r * HD;
          if constexpr (LAYOUT == kHalf) {
            const uint2 u = *reinterpret_cast<const uint2*>(p + a0);
            const uint2 v = *reinterpret_cast<const uint2*>(p + a1);
            o[b].raw = make_uint4(u.x, u.y, v.x, v.y);
          } else {
            o[b].raw = *reinterpret_cast<const uint4*>(p + a0);
          }
        }
      }
#pragma unroll
      for (int b = 0; b < kRopeBatch; ++b) {
        if (r0 + b * kStep >= h1) break;  // the same for the whole warp
        const int r = r0 + b * kStep + sub;
        const bool live = r < h1;
        if (turned && (LAYOUT == kAny || on)) {
          o[b].unpack();
          float (&x)[8] = o[b].x;
          if constexpr (LAYOUT == kHalf) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float u = x[j], v = x[j + 4];
              x[j] = fmaf(u, c[j], -(v * s[j]));
              x[j + 4] = fmaf(v, c[j], u * s[j]);
            }
          } else if constexpr (LAYOUT == kInterleaved) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float u = x[2 * j], v = x[2 * j + 1];
              x[2 * j] = fmaf(u, c[j], -(v * s[j]));
              x[2 * j + 1] = fmaf(v, c[j], u * s[j]);
            }
          } else {
            float* row = stage[warp][sub];
            __syncwarp();
            *reinterpret_cast<float4*>(row + 8 * l) = make_float4(x[0], x[1], x[2], x[3]);
            *reinterpret_cast<float4*>(row + 8 * l + 4) = make_float4(x[4], x[5], x[6], x[7]);
            __syncwarp();
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const int ch = 8 * l + j;
              if (ch < a.rot) {
                const bool first = a.adjacent ? (ch & 1) == 0 : ch < h;
                const float y = row[a.adjacent ? ch ^ 1 : first ? ch + h : ch - h];
                x[j] = fmaf(x[j], c[j], first ? -(y * s[j]) : y * s[j]);
              }
            }
          }
          if (KV == POD_ATTN_KV_BF16 || what == 0) o[b].pack();
        } else if (KV != POD_ATTN_KV_BF16 && what != 0) {
          o[b].unpack();
        }
        if (KV == POD_ATTN_KV_BF16 || what == 0) {
          if (!live) continue;
          uint16_t* p = dst + r * pitch;
          if constexpr (LAYOUT == kHalf) {
            *reinterpret_cast<uint2*>(p + a0) = make_uint2(o[b].raw.x, o[b].raw.y);
            *reinterpret_cast<uint2*>(p + a1) = make_uint2(o[b].raw.z, o[b].raw.w);
          } else {
            *reinterpret_cast<uint4*>(p + a0) = o[b].raw;
          }
        } else if constexpr (KV != POD_ATTN_KV_BF16) {
          if constexpr (LAYOUT == kHalf) {
            if (turned) {  // to 8 neighbouring channels a lane
              float* row = stage[warp][sub];
              __syncwarp();
              float (&x)[8] = o[b].x;
              *reinterpret_cast<float4*>(row + a0) = make_float4(x[0], x[1], x[2], x[3]);
              *reinterpret_cast<float4*>(row + a1) = make_float4(x[4], x[5], x[6], x[7]);
              __syncwarp();
              const float4 u = *reinterpret_cast<const float4*>(row + 8 * l);
              const float4 v = *reinterpret_cast<const float4*>(row + 8 * l + 4);
              x[0] = u.x, x[1] = u.y, x[2] = u.z, x[3] = u.w;
              x[4] = v.x, x[5] = v.y, x[6] = v.z, x[7] = v.w;
            }
          }
          store_quantised<KV, HD>(a, o[b].x, 8 * l, what == 2, min(r, h1 - 1),
                                  (size_t)phys * a.Hkv + r, slot, live);
        }
      }
    }
  }
}

// ============================================================================ expansion
struct ExpandArgs {
  const uint8_t* k4;
  const uint8_t* v4;
  const float* k_scale;
  const float* v_scale;
  uint16_t* k;
  uint16_t* v;
  const int32_t* tables4;
  const int32_t* tables;
  const int32_t* kv_lens;
  int32_t* status;
  int32_t Hkv, maxb, num_blocks4, num_blocks;
  int32_t wide;  // the bf16 pools are 32-byte aligned
};

// One warp per K or V unit of a sequence's block. A lane takes eight code bytes at a time, which are one
// group of 16 channels, and writes their 32 bytes at once, so that every store is a whole sector. Bound
// by memory: 30720 rows of 4 heads take 15 us (80.6 MB, 79 % of the measured copy rate; 4-byte loads,
// 16-byte stores and K and V in one warp took 9 us more). A grid row per sequence, as wide as the longest
// one asks for: CTAs beyond a sequence's end read its length and leave, which costs most where one long
// sequence stands beside many short ones (30720 rows and 256 times 40: 172 us of a floor of 16).
template <int HD>
__global__ void __launch_bounds__(256) expand_fp4_kernel(const __grid_constant__ ExpandArgs a) {
  constexpr int kSteps = HD / 32;  // groups of a lane
  const int lane = threadIdx.x & 31;
  const int seq = blockIdx.y;
  griddep_wait();
  const int L = a.kv_lens[seq];
  const int nblk = min((L + kBlockSize - 1) / kBlockSize, a.maxb);
  const int64_t units = (int64_t)nblk * a.Hkv * 2;
  for (int64_t u = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * 8) {
    const bool is_v = u & 1;
    const int j = (int)(u / 2 / a.Hkv), g = (int)(u / 2 % a.Hkv);
    const int src = a.tables4[(size_t)seq * a.maxb + j], dst = a.tables[(size_t)seq * a.maxb + j];
    if (src < 0 || src >= a.num_blocks4 || dst < 0 || dst >= a.num_blocks) {
      if (lane == 0) record_error(a.status, POD_ATTN_ERR_BAD_INDEX);
      continue;
    }
    const int nv = min(kBlockSize, L - j * kBlockSize);
    const uint8_t* unit = (is_v ? a.v4 : a.k4) + ((size_t)src * a.Hkv + g) * (9 * HD);
    uint16_t* out = (is_v ? a.v : a.k) + ((size_t)dst * a.Hkv + g) * kBlockSize * HD;
    const float h = (is_v ? a.v_scale : a.k_scale)[g];
    uint2 w[kSteps];
    uint32_t s8[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int at = i * 32 + lane;  // group within the unit: row at / (HD / 16)
      const int row = at / (HD / 16), grp = at % (HD / 16);
      w[i] = *reinterpret_cast<const uint2*>(unit + at * 8);
      s8[i] = unit[8 * HD + (is_v ? grp * kBlockSize + row : at)];
    }
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
      const int at = i * 32 + lane;
      const uint32_t s = e4m3x2_to_f16x2(s8[i] * 0x101u);
      uint32_t f[8];
      e2m1x8_to_f16x2(w[i].x, *reinterpret_cast<uint32_t(*)[4]>(f));
      e2m1x8_to_f16x2(w[i].y, *reinterpret_cast<uint32_t(*)[4]>(f + 4));
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        f[b] = hmul2(f[b], s);  // exact
        f[b] = pack_bf16x2(f16lo(f[b]) * h, f16hi(f[b]) * h);
      }
      if (at / (HD / 16) >= nv) continue;
      if (a.wide) {
        st_global_256(out + at * 16, f);
      } else {
        uint4* o = reinterpret_cast<uint4*>(out + at * 16);
        o[0] = make_uint4(f[0], f[1], f[2], f[3]);
        o[1] = make_uint4(f[4], f[5], f[6], f[7]);
      }
    }
  }
}

// ============================================================================ block copies
// One CTA per pair and pool; the pools and the pairs of one launch are in its parameters (the device has
// nothing to read first, and nothing has to outlive the call). Bound by memory: 1201 blocks of 16 KiB in
// 16 pools take 92 us from call to call, the measured copy rate. Few pairs of very large blocks are bound by
// what one SM moves (four of 1 MiB in two pools: 22 us of a floor of 2.5).
template <int POOLS, int PAIRS>
struct CopyArgs {
  struct {
    uint8_t* base;
    uint64_t bytes;
  } pool[POOLS];
  int32_t pair[PAIRS][2];
};

template <int POOLS, int PAIRS>
__global__ void __launch_bounds__(256) copy_blocks_kernel(const __grid_constant__ CopyArgs<POOLS, PAIRS> a) {
  griddep_wait();
  const auto& pool = a.pool[blockIdx.y];
  const int from = a.pair[blockIdx.x][0], to = a.pair[blockIdx.x][1];
  if (from == to) return;
  const uint4* src = reinterpret_cast<const uint4*>(pool.base + (size_t)from * pool.bytes);
  uint4* dst = reinterpret_cast<uint4*>(pool.base + (size_t)to * pool.bytes);
  const uint32_t vecs = (uint32_t)(pool.bytes / 16);
  uint32_t v = threadIdx.x;
  for (; v + 3 * 256 < vecs; v += 4 * 256) {  // four loads of a thread in flight
    const uint4 a0 = src[v], a1 = src[v + 256], a2 = src[v + 512], a3 = src[v + 768];
    dst[v] = a0;
    dst[v + 256] = a1;
    dst[v + 512] = a2;
    dst[v + 768] = a3;
  }
  for (; v < vecs; v += 256) dst[v] = src[v];
}

template <int POOLS, int PAIRS>
cudaError_t launch_copy(const pod_attn_block_pool* pools, int n_pools, const int32_t* pairs, int n_pairs,
                        cudaStream_t st) {
  CopyArgs<POOLS, PAIRS> a;
  for (int64_t p0 = 0; p0 < n_pools; p0 += POOLS) {
    const int np = (int)std::min<int64_t>(POOLS, n_pools - p0);
    for (int i = 0; i < np; ++i)
      a.pool[i] = {static_cast<uint8_t*>(pools[p0 + i].base), pools[p0 + i].block_bytes};
    for (int64_t j0 = 0; j0 < n_pairs; j0 += PAIRS) {
      const int nj = (int)std::min<int64_t>(PAIRS, n_pairs - j0);
      std::memcpy(a.pair, pairs + 2 * j0, sizeof(int32_t) * 2 * nj);
      const cudaError_t e = launch_early(copy_blocks_kernel<POOLS, PAIRS>, dim3(nj, np), 256, 0, st, a);
      if (e != cudaSuccess) return e;
    }
  }
  return cudaSuccess;
}

// [p, p + n) and [q, q + m) share a byte
bool overlap(const void* p, size_t n, const void* q, size_t m) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
  return n > 0 && m > 0 && a < b + m && b < a + n;
}

template <int KV, int HD>
cudaError_t launch_rope(const RopeAppendArgs& a, bool interleaved, int grid, cudaStream_t st) {
  if (a.rot % 8 != 0)
    return launch_early(rope_append_kernel<KV, HD, kAny>, dim3(grid), kRopeWarps * 32, 0, st, a);
  if (interleaved || a.rot == 0)
    return launch_early(rope_append_kernel<KV, HD, kInterleaved>, dim3(grid), kRopeWarps * 32, 0, st, a);
  return launch_early(rope_append_kernel<KV, HD, kHalf>, dim3(grid), kRopeWarps * 32, 0, st, a);
}

}  // namespace
}  // namespace pod

using namespace pod;

extern "C" {

pod_attn_status pod_attn_rope_append(pod_attn_plan_t plan, pod_attn_rope_t rope, const void* q,
                                     int64_t q_stride, const void* k_new, int64_t k_stride,
                                     const void* v_new, int64_t v_stride,
                                     const pod_attn_kv_cache* cache, const int32_t* d_block_tables,
                                     void* q_prefill, void* q_decode, void* workspace,
                                     size_t workspace_bytes, void* stream) {
  if (!plan || !cache) return POD_ATTN_ERR_INVALID_ARG;
  const pod_attn_status st = check_workspace(plan, workspace, workspace_bytes);
  if (st != POD_ATTN_OK) return st;
  const pod_attn_problem& pr = plan->prob;
  const int64_t Tp = pr.num_prefill_tokens, Nd = pr.num_decode_seqs, T = Tp + Nd;
  const int D = pr.head_dim;
  const int64_t q_row = (int64_t)pr.num_q_heads * D, kv_row = (int64_t)pr.num_kv_heads * D;
  const bool scaled = cache->type != POD_ATTN_KV_BF16;
  if (cache->type != POD_ATTN_KV_BF16 && cache->type != POD_ATTN_KV_E4M3 &&
      cache->type != POD_ATTN_KV_E2M1)
    return POD_ATTN_ERR_INVALID_ARG;
  if (cache->type == POD_ATTN_KV_E4M3 && D != kHeadDim) return POD_ATTN_ERR_UNSUPPORTED;
  if (rope && rope->rot > D) return POD_ATTN_ERR_INVALID_ARG;
  if (T == 0) return POD_ATTN_OK;
  if (!k_new || !v_new || !cache->k_pool || !cache->v_pool || cache->num_blocks < 1 ||
      !d_block_tables || (scaled && (!cache->k_scale || !cache->v_scale)))
    return POD_ATTN_ERR_INVALID_ARG;
  if (q && ((Tp > 0 && !q_prefill) || (Nd > 0 && !q_decode))) return POD_ATTN_ERR_INVALID_ARG;
  if (!aligned16({q, k_new, v_new, q_prefill, q_decode}) || !cache_aligned(*cache))
    return POD_ATTN_ERR_INVALID_ARG;
  if ((q && (q_stride < q_row || q_stride % 8)) || k_stride < kv_row || k_stride % 8 ||
      v_stride < kv_row || v_stride % 8)
    return POD_ATTN_ERR_INVALID_ARG;
  if (q) {
    uint16_t* qp = static_cast<uint16_t*>(q_prefill);
    const auto span = [&](int64_t stride, int64_t row) { return (size_t)((T - 1) * stride + row) * 2; };
    const size_t np = (size_t)(Tp * q_row) * 2, nd = (size_t)(Nd * q_row) * 2;
    const uint16_t* whole = static_cast<const uint16_t*>(q);
    const bool in_place = q_stride == q_row && (Tp == 0 || qp == whole) &&
                          (Nd == 0 || static_cast<uint16_t*>(q_decode) == whole + Tp * q_row);
    if (!in_place && (overlap(q, span(q_stride, q_row), q_prefill, np) ||
                      overlap(q, span(q_stride, q_row), q_decode, nd)))
      return POD_ATTN_ERR_INVALID_ARG;
    if (overlap(q_prefill, np, q_decode, nd)) return POD_ATTN_ERR_INVALID_ARG;
    for (const void* x : {k_new, v_new}) {
      const size_t n = span(x == k_new ? k_stride : v_stride, kv_row);
      if (overlap(x, n, q_prefill, np) || overlap(x, n, q_decode, nd)) return POD_ATTN_ERR_INVALID_ARG;
    }
  }
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  RopeAppendArgs a{};
  a.q = static_cast<const uint16_t*>(q);
  a.k = static_cast<const uint16_t*>(k_new);
  a.v = static_cast<const uint16_t*>(v_new);
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.q_prefill = static_cast<uint16_t*>(q_prefill);
  a.q_decode = static_cast<uint16_t*>(q_decode);
  a.k_pool = static_cast<uint8_t*>(cache->k_pool);
  a.v_pool = static_cast<uint8_t*>(cache->v_pool);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.block_tables = d_block_tables;
  a.new_rows = reinterpret_cast<const int32_t*>(ws + plan->ws.new_rows);
  a.status = reinterpret_cast<int32_t*>(ws + plan->ws.status);
  a.T = (int32_t)T;
  a.Tp = (int32_t)Tp;
  a.Hq = pr.num_q_heads;
  a.Hkv = pr.num_kv_heads;
  a.maxb = pr.max_blocks_per_seq;
  a.num_blocks = cache->num_blocks;
  bool interleaved = false;
  if (rope) {
    a.rot = rope->rot;
    a.mag = rope->attention_factor;
    interleaved = rope->interleaved != 0;
    std::memcpy(a.turns, rope->turns, sizeof(a.turns));
  }
  a.adjacent = interleaved;
  const auto works = [&](int rows) {
    a.rows = rows;
    a.q_parts = q ? (pr.num_q_heads + rows - 1) / rows : 0;
    a.kv_parts = (pr.num_kv_heads + rows - 1) / rows;
    return T * (a.q_parts + 2 * a.kv_parts);
  };
  // Heads per warp. One batch of steps (8 heads of 128 channels, 16 of 64) keeps all of a work's loads
  // in flight at once and serves large batches best (16380 tokens of 96 heads: 13 us less than with
  // two or four batches); up to a few rounds of the resident warps the rounds are whole, and what counts is
  // their number times the length of one (1088 tokens of 48 heads: 8.4 us in one round of two batches,
  // 9.8 us in two of one).
  const int64_t resident = (int64_t)plan->num_sms * kRopeCtas * kRopeWarps;
  const int base = kRopeBatch * 256 / D;
  int rows = base;
  if (works(base) < 4 * resident) {
    int64_t best = INT64_MAX;
    for (int n : {1, 2, 4}) {
      const int64_t cost = (works(n * base) + resident - 1) / resident * (2 * n + 1);
      if (cost < best) best = cost, rows = n * base;
    }
  }
  const int grid = (int)std::min<int64_t>((works(rows) + kRopeWarps - 1) / kRopeWarps,
                                          (int64_t)plan->num_sms * kRopeCtas);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e;
  if (cache->type == POD_ATTN_KV_E4M3)
    e = launch_rope<POD_ATTN_KV_E4M3, 128>(a, interleaved, grid, s);
  else if (cache->type == POD_ATTN_KV_E2M1)
    e = D == 64 ? launch_rope<POD_ATTN_KV_E2M1, 64>(a, interleaved, grid, s)
                : launch_rope<POD_ATTN_KV_E2M1, 128>(a, interleaved, grid, s);
  else
    e = D == 64 ? launch_rope<POD_ATTN_KV_BF16, 64>(a, interleaved, grid, s)
                : launch_rope<POD_ATTN_KV_BF16, 128>(a, interleaved, grid, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return POD_ATTN_ERR_CUDA;
  }
  return POD_ATTN_OK;
}

pod_attn_status pod_attn_expand_fp4(pod_attn_plan_t plan, const pod_attn_kv_cache* cache,
                                    const int32_t* d_block_tables4, void* k_pool, void* v_pool,
                                    const int32_t* d_block_tables, const int32_t* d_kv_lens,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (!plan || !cache) return POD_ATTN_ERR_INVALID_ARG;
  const pod_attn_status st = check_workspace(plan, workspace, workspace_bytes);
  if (st != POD_ATTN_OK) return st;
  const pod_attn_problem& pr = plan->prob;
  if (plan->opt.kv_fp8 || plan->opt.kv_fp4 || cache->type != POD_ATTN_KV_E2M1)
    return POD_ATTN_ERR_UNSUPPORTED;
  const int n = pr.num_prefill_seqs + pr.num_decode_seqs;
  if (n == 0) return POD_ATTN_OK;
  if (!cache->k_pool || !cache->v_pool || !cache->k_scale || !cache->v_scale || cache->num_blocks < 1 ||
      !k_pool || !v_pool || !d_block_tables4 || !d_block_tables || !d_kv_lens)
    return POD_ATTN_ERR_INVALID_ARG;
  if (!aligned16({k_pool, v_pool}) || !cache_aligned(*cache))
    return POD_ATTN_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  ExpandArgs a{};
  a.k4 = static_cast<const uint8_t*>(cache->k_pool);
  a.v4 = static_cast<const uint8_t*>(cache->v_pool);
  a.k_scale = cache->k_scale;
  a.v_scale = cache->v_scale;
  a.k = static_cast<uint16_t*>(k_pool);
  a.v = static_cast<uint16_t*>(v_pool);
  a.tables4 = d_block_tables4;
  a.tables = d_block_tables;
  a.kv_lens = d_kv_lens;
  a.status = reinterpret_cast<int32_t*>(ws + plan->ws.status);
  a.Hkv = pr.num_kv_heads;
  a.maxb = pr.max_blocks_per_seq;
  a.num_blocks4 = cache->num_blocks;
  a.wide = ((reinterpret_cast<uintptr_t>(k_pool) | reinterpret_cast<uintptr_t>(v_pool)) & 31) == 0;
  a.num_blocks = pr.num_blocks;
  const int longest = *std::max_element(plan->kv.begin(), plan->kv.end());
  const int64_t warps = (int64_t)((longest + kBlockSize - 1) / kBlockSize) * pr.num_kv_heads * 2;
  const int grid = (int)std::min<int64_t>((warps + 7) / 8, (int64_t)plan->num_sms * 8);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // one grid row per sequence; the hardware takes at most 65535
  for (int s0 = 0; s0 < n; s0 += 65535) {
    const dim3 g(grid, std::min(65535, n - s0));
    ExpandArgs b = a;
    b.tables4 += (size_t)s0 * a.maxb;
    b.tables += (size_t)s0 * a.maxb;
    b.kv_lens += s0;
    if (launch_early(pr.head_dim == 64 ? expand_fp4_kernel<64> : expand_fp4_kernel<128>, g, 256, 0, s,
                     b) != cudaSuccess) {
      cudaGetLastError();
      return POD_ATTN_ERR_CUDA;
    }
  }
  return POD_ATTN_OK;
}

pod_attn_status pod_attn_copy_blocks(const pod_attn_block_pool* h_pools, int32_t n_pools,
                                     int32_t num_blocks, const int32_t* h_pairs, int32_t n_pairs,
                                     void* stream) {
  const pod_attn_status st = check_copies(h_pools, n_pools, num_blocks, h_pairs, n_pairs);
  if (st != POD_ATTN_OK) return st;
  if (n_pools == 0 || n_pairs == 0) return POD_ATTN_OK;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  // Small lists in a small launch: its 0.8 KB of parameters are quicker to send than the large one's
  // 18 KB (five pairs of two pools 7.2 us from call to call, 7.7 us).
  const cudaError_t e = n_pools <= 16 && n_pairs <= 64
                            ? launch_copy<16, 64>(h_pools, n_pools, h_pairs, n_pairs, s)
                            : launch_copy<128, 2048>(h_pools, n_pools, h_pairs, n_pairs, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return POD_ATTN_ERR_CUDA;
  }
  return POD_ATTN_OK;
}

}  // extern "C"
