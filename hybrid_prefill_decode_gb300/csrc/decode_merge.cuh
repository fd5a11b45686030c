// decode_merge.cuh — what the decode kernels of every cache type share: where a decode item runs, and
// how the states of its warps and of its splits are combined.
#pragma once

#include <cmath>
#include <cstdint>

#include "pod_internal.h"
#include "ptx.cuh"

namespace pod {

using namespace ptx;

// Where a decode item runs: `nw` warps (4; in the 4-bit decode a group's 4 or 16) from absolute warp
// `w0`, the memory in which they are combined, the named barrier of the slot or group that runs it and
// its index in the control block.
struct DecodeCtx {
  int w0, nw;
  uint8_t* ring;        // combine scratch: the warps' rings (nw * kDecodeSlots * kSmemDecodeSlot bytes);
                        // in the 4-bit decode memory of its own beside them
  float* scores;        // nw * kMaxGroup * kBlockSize floats; not used by the 4-bit decode
  int bar_id, bar_threads, first_thread, slot;
};

__device__ __forceinline__ uint16_t f2bf(float f) {
  return static_cast<uint16_t>(pack_bf16x2(f, 0.f) & 0xFFFFu);
}

__device__ __forceinline__ int atomic_inc_acq_rel(int32_t* p) {
  int old;
  asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], 1;" : "=r"(old) : "l"(p) : "memory");
  return old;
}

constexpr int kScr = kHeadDim + 4;  // shared scratch row of one warp and head: o[128], m, l
constexpr int kRow = kHeadDim + 2;  // global partial slot row: o[128], m, l

// Merge of the 4-bit decode: what a group of kGW warps does with its split's partial in place. An output
// of many splits (a unit with bundles, word 3) is merged in two levels: the last split of a bundle to
// arrive sums the bundle up into the bundle's first slot, the last bundle's sum goes with the others'
// into the output. Sums go in the splits' order, whoever makes them. kLevels: plans that have such units;
// the others' kernels leave the second level out, without which their main loop comes out 2 to 3 % faster
// (64 sequences of 8192 to 16384 rows, 8 kv-heads of 4 heads: 155 -> 150 us when it was left out).
// A barrier orders the group's partials before the release of the thread that counts the arrival, its
// acquire (in the last to arrive) the others' before the group's reads.
template <int GT, int HD, int kGW, bool kLevels, class P, class Ctl>
__device__ __forceinline__ void merge_fp4(const P& p, int d, int g, int unit, int split,
                                          const DecodeCtx& dc, Ctl* ctl, float out_scale) {
  constexpr int kPairs = GT * HD / 2, kStep = kGW * 32;
  constexpr int kPer = (kPairs + kStep - 1) / kStep;  // pairs of channels of a thread
  const int G = p.G;
  const int ltid = threadIdx.x - dc.first_thread;
  const int32_t* un = p.units + unit * kUnitWords;
  const int nsplit = un[0], bundle = kLevels ? un[3] : 0;
  const int slot = decode_slot_floats(G);
  float* base = p.partial_d + (size_t)un[1] * slot;
  for (int level = bundle > 0 ? 1 : 0;; level = 0) {
    int n = nsplit, step = slot;  // slots to be merged, and how far apart they lie
    float* part = base;
    int32_t* arrive = p.arrive + unit * kFp4Counters;
    if (level) {
      const int b = split / bundle;
      n = min(bundle, nsplit - b * bundle);
      part += (size_t)b * bundle * slot;
      arrive += 1 + b;
    } else if (bundle > 0) {
      n = (nsplit + bundle - 1) / bundle;
      step *= bundle;
    }
    named_bar_sync(dc.bar_id, dc.bar_threads);
    if (ltid == 0) {
      const bool last = atomic_inc_acq_rel(arrive) == n - 1;
      if (last) *arrive = 0;  // for the next run
      ctl->merge_last[dc.slot] = last;
    }
    named_bar_sync(dc.bar_id, dc.bar_threads);
    if (!ctl->merge_last[dc.slot]) break;
    uint16_t* out = p.o_decode + ((size_t)d * p.Hq + (size_t)g * G) * HD;
    if constexpr (kPer == 1) {
      // One pass over the slots: a thread keeps the running max and sum of its head beside its two
      // channels, with the loads of eight slots in flight. (64 outputs of two to eight splits, MHA of 128
      // channels: 1 to 3 us less than with weights first.)
      constexpr int kAhead = 8;
      const int h = min(ltid / (HD / 2), G - 1), c = 2 * (ltid % (HD / 2));
      const float* at = part + h * kRow;
      float2 num = make_float2(0.f, 0.f);
      float mx = -INFINITY, den = 0.f;
      for (int k0 = 0; k0 < n; k0 += kAhead) {
        float2 v[kAhead], s[kAhead];  // channels; (m, l)
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const float* sl = at + (size_t)min(k0 + j, n - 1) * step;
          v[j] = __ldcg(reinterpret_cast<const float2*>(sl + c));
          s[j] = __ldcg(reinterpret_cast<const float2*>(sl + kHeadDim));
        }
        float top = mx;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (k0 + j >= n) s[j].x = -INFINITY;
          top = fmaxf(top, s[j].x);
        }
        const float f = mx == -INFINITY ? 0.f : ex2(mx - top);
        num.x *= f;
        num.y *= f;
        den *= f;
        mx = top;
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (s[j].x == -INFINITY) continue;  // no split, or one that saw nothing
          const float w = ex2(s[j].x - top);
          num.x += w * v[j].x;
          num.y += w * v[j].y;
          den += w * s[j].y;
        }
      }
      const bool mine = ltid < G * (HD / 2);
      if (level) {
        named_bar_sync(dc.bar_id, dc.bar_threads);  // every thread has read the first slot
        float* dst = part + h * kRow;
        if (mine) *reinterpret_cast<float2*>(dst + c) = num;
        if (mine && c == 0) *reinterpret_cast<float2*>(dst + kHeadDim) = make_float2(mx, den);
      } else if (mine) {
        const float inv = out_scale / den;
        *reinterpret_cast<uint32_t*>(out + h * HD + c) = pack_bf16x2(num.x * inv, num.y * inv);
      }
    } else {
      // the slots' weights into shared memory, 16 lanes a head and a lane per slot, while the first slots'
      // channels are on their way
      static_assert(kMaxGroup * kFp4Bundle == kStep && kFp4Bundle == 16, "a thread per head and slot");
      // 16 loads in flight (with 8, an output of 16 splits takes 2 us more), 8 beside a second level
      // (16 spill registers of the main loop)
      constexpr int kAhead = (kLevels ? 8 : 16) / kPer;
      float* wts = reinterpret_cast<float*>(dc.ring);  // [G][kFp4Bundle]: the scratch is free again
      float* inv = wts + kMaxGroup * kFp4Bundle;       // [G]: out_scale / merged l
      float2 v[kAhead][kPer], num[kPer];
      auto load = [&](int k0) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const int idx = ltid + e * kStep, h = min(idx / (HD / 2), G - 1), c = 2 * (idx % (HD / 2));
            v[j][e] = __ldcg(reinterpret_cast<const float2*>(
                part + (size_t)min(k0 + j, n - 1) * step + h * kRow + c));
          }
      };
      load(0);
      const int hw = ltid / kFp4Bundle, kw = ltid % kFp4Bundle;
      const float2 ml = __ldcg(reinterpret_cast<const float2*>(
          part + (size_t)min(kw, n - 1) * step + min(hw, G - 1) * kRow + kHeadDim));
      const float m = kw < n ? ml.x : -INFINITY;
      float mx = m;
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
      const float f = m == -INFINITY ? 0.f : ex2(m - mx);
      float den = m == -INFINITY ? 0.f : f * ml.y;
#pragma unroll
      for (int off = 8; off > 0; off >>= 1) den += __shfl_xor_sync(0xffffffffu, den, off);
      wts[ltid] = f;
      if (kw == 0) inv[hw] = out_scale / den;
      named_bar_sync(dc.bar_id, dc.bar_threads);
#pragma unroll
      for (int e = 0; e < kPer; ++e) num[e] = make_float2(0.f, 0.f);
      for (int k0 = 0;;) {
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          if (k0 + j >= n) break;
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const float w = wts[min((ltid + e * kStep) / (HD / 2), G - 1) * kFp4Bundle + k0 + j];
            num[e].x += w * v[j][e].x;
            num[e].y += w * v[j][e].y;
          }
        }
        k0 += kAhead;
        if (k0 >= n) break;
        load(k0);
      }
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        const int idx = ltid + e * kStep, h = idx / (HD / 2), c = 2 * (idx % (HD / 2));
        if (h >= G) continue;
        if (level)
          *reinterpret_cast<float2*>(part + h * kRow + c) = num[e];
        else
          *reinterpret_cast<uint32_t*>(out + h * HD + c) =
              pack_bf16x2(num[e].x * inv[h], num[e].y * inv[h]);
      }
      if (level && kw == 0 && hw < G)  // every thread has read the slot's (m, l) before the barrier above
        *reinterpret_cast<float2*>(part + hw * kRow + kHeadDim) = make_float2(mx, den);
    }
    if (!level) break;
  }
}

// Combine the warps' states of a decode item (sequence d, kv-head g, split `split` of unit `unit`;
// in the shared scratch at dc.ring, a row per warp and head), then write the output or the split's
// partial and, for the last split of a unit to arrive, merge all partials. `ctl` is the CTA's control
// block (its abort flag and the slots' merge_last); FP4: the 4-bit cache, in groups of FP4 warps, whose
// output is multiplied by out_scale and may be merged in two levels (0: the other caches).
template <int GT, int HD, int FP4 = 0, bool kLevels = false, class P, class Ctl>
__device__ __forceinline__ void combine_decode(const P& p, int d, int g, int unit, int split,
                                               const DecodeCtx& dc, Ctl* ctl, float out_scale) {
  const int G = p.G;
  const int ltid = threadIdx.x - dc.first_thread;
  named_bar_sync(dc.bar_id, dc.bar_threads);
  const float* scr = reinterpret_cast<const float*>(dc.ring);
  if (!ctl->abort) {
    const int nsplit = unit >= 0 ? p.units[unit * kUnitWords + 0] : 1;
    const int slot0 = unit >= 0 ? p.units[unit * kUnitWords + 1] : 0;
    float* slot = unit >= 0 ? p.partial_d + (size_t)(slot0 + split) * decode_slot_floats(G) : nullptr;
    for (int idx = ltid; idx < G * HD; idx += dc.bar_threads) {
      const int h = idx / HD, c = idx % HD;
      float mx = -INFINITY;
      for (int w = 0; w < dc.nw; ++w) mx = fmaxf(mx, scr[(w * GT + h) * kScr + kHeadDim]);
      float num = 0.f, den = 0.f;
      for (int w = 0; w < dc.nw; ++w) {
        const float* src = scr + (w * GT + h) * kScr;
        const float mw = src[kHeadDim];
        if (mw == -INFINITY) continue;
        const float f = ex2(mw - mx);
        num += f * src[c];
        den += f * src[kHeadDim + 1];
      }
      if (unit < 0) {
        p.o_decode[((size_t)d * p.Hq + (size_t)g * G + h) * HD + c] =
            f2bf(FP4 ? num / den * out_scale : num / den);
      } else {
        slot[h * kRow + c] = num;
        if (c == 0) {
          slot[h * kRow + kHeadDim] = mx;
          slot[h * kRow + kHeadDim + 1] = den;
        }
      }
    }
    if constexpr (FP4 > 0) {
      if (unit >= 0) merge_fp4<GT, HD, FP4, kLevels>(p, d, g, unit, split, dc, ctl, out_scale);
    } else if (unit >= 0) {
      __threadfence();
      named_bar_sync(dc.bar_id, dc.bar_threads);
      if (ltid == 0) ctl->merge_last[dc.slot] = (atomicAdd(&p.arrive[unit], 1) == nsplit - 1);
      named_bar_sync(dc.bar_id, dc.bar_threads);
      if (ctl->merge_last[dc.slot]) {
        __threadfence();
        const size_t stride = (size_t)decode_slot_floats(G);
        const float* part0 = p.partial_d + (size_t)slot0 * stride;
        // the splits' (m, l) once into shared memory (the scratch is free again), one weight
        // per (head, split), then every output element as a weighted sum over the splits with
        // the loads of all of this thread's elements in flight together
        float* wts = reinterpret_cast<float*>(dc.ring);   // [G][nsplit]: m, then the weight
        float* ls = wts + kMaxGroup * kMaxDecodeSplits;    // [G][nsplit]: l
        float* inv = ls + kMaxGroup * kMaxDecodeSplits;    // [G]: 1 / merged l
        for (int idx = ltid; idx < G * nsplit; idx += dc.bar_threads) {
          const int h = idx / nsplit, k = idx - h * nsplit;
          const float* sl = part0 + (size_t)k * stride + h * kRow;
          wts[idx] = __ldcg(sl + kHeadDim);
          ls[idx] = __ldcg(sl + kHeadDim + 1);
        }
        named_bar_sync(dc.bar_id, dc.bar_threads);
        if (ltid < G) {
          float* w = wts + ltid * nsplit;
          const float* l = ls + ltid * nsplit;
          float mx = -INFINITY;
          for (int k = 0; k < nsplit; ++k) mx = fmaxf(mx, w[k]);
          float den = 0.f;
          for (int k = 0; k < nsplit; ++k) {
            const float f = w[k] == -INFINITY ? 0.f : ex2(w[k] - mx);
            w[k] = f;
            den += f * l[k];
          }
          inv[ltid] = 1.f / den;
        }
        named_bar_sync(dc.bar_id, dc.bar_threads);
        constexpr int kPer = (GT * HD + kDecodeWarps * 32 - 1) / (kDecodeWarps * 32);
        float num[kPer];
#pragma unroll
        for (int e = 0; e < kPer; ++e) num[e] = 0.f;
        for (int k = 0; k < nsplit; ++k) {
          const float* sl = part0 + (size_t)k * stride;
#pragma unroll
          for (int e = 0; e < kPer; ++e) {
            const int idx = ltid + e * kDecodeWarps * 32;
            if (idx < G * HD) {
              const int h = idx / HD, c = idx % HD;
              num[e] += wts[h * nsplit + k] * __ldcg(sl + h * kRow + c);
            }
          }
        }
#pragma unroll
        for (int e = 0; e < kPer; ++e) {
          const int idx = ltid + e * kDecodeWarps * 32;
          if (idx < G * HD) {
            const int h = idx / HD, c = idx % HD;
            p.o_decode[((size_t)d * p.Hq + (size_t)g * G + h) * HD + c] =
                f2bf(num[e] * inv[h]);
          }
        }
        if (ltid == 0) p.arrive[unit] = 0;
      }
    }
  }
  named_bar_sync(dc.bar_id, dc.bar_threads);
}

}  // namespace pod
