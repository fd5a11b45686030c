// decode_fp4.cu — decode attention over a 4-bit (e2m1) paged cache for sm_103a.
//
// A cached value is e2m1(code) * e4m3(scale of the row's 16 channels) * fp32(scale of the kv-head).
// The head scale of K joins the softmax scale and that of V the final division, so the tensor cores
// see code * group scale: 2 significant bits times 4, exact in f16.
//
// The work is the plan's shares of decode items (one sequence, one kv-head with its G query heads, a
// range of 16-row blocks; "LLMSO - W4", §"FlashDecoding — decode 단계의 병렬성 확보"), one for each group
// of warps: a persistent CTA per SM holds four groups of four, or one of all 16 where outputs are few
// (the planner chooses). Each warp streams its own (block, kv-head) units into a private ring in shared
// memory, one bulk copy for the K unit and one for the V unit (codes and scales of 16 rows are
// contiguous), and keeps an online softmax per head.
//
// What bounds it (GB300): 9 * D bytes of a (block, kv-head) take as long to arrive as the SM has to
// convert and multiply them, 279 instructions at 128 channels: 64 conversions and 16 interleavings (two
// issue cycles each on the ALU pipe), 64 packed products by the group scales, 16 warp MMAs of 9 cycles.
// With one query head it is 208 (see fp4_item). Long sequences run at 94 % of the measured copy rate (76 of
// 16384 rows, 8 kv-heads: 225 us), with one query head at 98 % (216 us); 64 sequences of 8192 to 16384
// rows take 146 us (89 %), 32 MHA sequences of 2048 to 4096 rows 75.7 us (88 %), one of 2^20 rows of 2
// kv-heads 63 us (70 %), one of 130001 rows of 4 kv-heads and 64 channels 19.8 us (28 %): there 128 CTAs take
// 8 to 11 us over their four rounds each and end 12 us after the first start, then one CTA an output reads
// and merges 32 partials for 5 us while the others are idle.

#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "decode_merge.cuh"
#include "launch.cuh"
#include "pod_internal.h"
#include "ptx.cuh"

namespace pod {

namespace {

constexpr int kFp4Threads = kFp4Warps * 32;
constexpr uint64_t kFp4TimeoutNs = 4000000000ull;    // 4 s: no healthy wait comes close
constexpr uint32_t kFp4SleepNs = 20000;

// The reference m of a head's weights 2^(x - m) is kept kHead below a running max of its scores, which is
// raised only when one passes it by more than kLazy (all in log2 units): most batches need no exchange
// between lanes. Weights stay below 2^(kHead + kLazy), within f16's range: 2^15, and with a single head,
// where they take V's scales (up to 448), 2^7. Those more than 2^(14 + kHead) below the largest are f16
// subnormals.
template <int GT>
struct Fp4Weights {
  static constexpr float kHead = GT == 1 ? 5.f : 7.f;
  static constexpr float kLazy = GT == 1 ? 2.f : 8.f;
};

// A warp takes its blocks a batch of kBatch neighbours at a time (one barrier, one pass over the
// bookkeeping for each batch); a ring slot holds a batch: its K units, then its V units. Two slots of
// 4.5 KiB for each of 16 warps keep 74 to 147 KB of an SM in flight, enough for the memory's latency
// (three measured the same). The combine scratch lies beside the rings, so that the next item's first
// batches are on their way while an item is combined.
template <int HD>
struct Fp4Geom {
  static constexpr int kUnit = 9 * HD;               // bytes of one K or V unit: codes, then scales
  static constexpr int kBatch = fp4_batch_blocks(HD);
  static constexpr int kSlot = 2 * kBatch * kUnit;
  static constexpr int kSlots = 2;                   // batches in flight per warp
  static constexpr int kRing = kSlots * kSlot;
  static_assert(kRing % 128 == 0, "aligned rings");
};

// Bytes of the scratch of four warps: a row per warp and head, and in a merge of four warps the splits'
// weights.
template <int GT>
constexpr int kFp4Rows = kDecodeWarps * GT * kScr;
constexpr int kFp4Weights = kMaxGroup * kFp4Bundle + kMaxGroup;
template <int GT>
constexpr int kFp4Scratch =
    ((kFp4Rows<GT> > kFp4Weights ? kFp4Rows<GT> : kFp4Weights) * 4 + 127) / 128 * 128;

constexpr int kFp4MaxSlots = 2;

// A group's words. `abort`: a wait of one of its warps has given up; set before the barrier behind
// which the whole group reads it, so that its threads always take the same way.
struct Fp4Group {
  int abort;
  int share;
  int merge_last[1];
};

struct Fp4Ctl {
  uint64_t full[kFp4Warps][kFp4MaxSlots];
  Fp4Group group[kFp4Warps / kDecodeWarps];
  int abort;  // of any group: the others' waits end soon
};

template <int GT, int HD>
constexpr int fp4_smem() {
  return kFp4Warps * Fp4Geom<HD>::kRing + kFp4Warps / kDecodeWarps * kFp4Scratch<GT> +
         (int)sizeof(Fp4Ctl);
}
static_assert(fp4_smem<8, 128>() <= 227 * 1024 && fp4_smem<8, 64>() <= 227 * 1024, "one CTA per SM");

struct Fp4Params {
  const uint16_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  const int32_t* block_tables;
  const int32_t* items;
  const int32_t* units;
  uint16_t* o_decode;
  float* partial_d;
  int32_t* counters;
  int32_t* arrive;
  int32_t* status;
  pod_attn_item_record* records;
  int32_t n_shares, Hq, Hkv, G, maxb, num_blocks;
  float scale_log2;
  uint64_t timeout_ns;
};

// Position of a warp in its ring: the next slot to fill and to read, and the parity of its barrier's
// phase. It runs on from item to item.
struct Fp4Ring {
  uint32_t slot = 0, parity = 0;
};

// One warp's share of an item: which blocks, and the copies of them into its ring. The warp's block i
// is block (i / kBatch * 4 + wl) * kBatch + i % kBatch of the item: batches of the four warps alternate.
// Lane 2u copies the K unit of a batch's block u, lane 2u + 1 the V unit; each holds the block-table
// entry of its block in the next batch to be copied, read one batch ahead.
template <int HD, int GW>
struct Fp4Stream {
  using Geo = Fp4Geom<HD>;
  static constexpr int kBatch = Geo::kBatch, kUnit = Geo::kUnit, kSlots = Geo::kSlots;
  int mine, nmine;     // batches, blocks
  int last_rows;       // rows of the warp's last batch that exist
  int left;            // of this lane: the warp's blocks from its own in the next batch on
  int next;            // its entry there
  const int32_t* row;  // where the one behind that stands
  const uint8_t* pool;

  // wl: the warp within its group
  __device__ __forceinline__ Fp4Stream(const Fp4Params& p, const int32_t* it, int wl, int lane) {
    const int d = it[1], g = it[2], kb = it[4], ke = it[5];
    const int nblk = (ke - kb + kBlockSize - 1) / kBlockSize;
    const int n_batches = (nblk + kBatch - 1) / kBatch;
    mine = n_batches > wl ? (n_batches - wl + GW - 1) / GW : 0;
    // the warp that has the item's last batch may have less than a whole one
    const bool has_last = mine > 0 && (mine - 1) * GW + wl == n_batches - 1;
    nmine = mine * kBatch - (has_last ? n_batches * kBatch - nblk : 0);
    last_rows = ke - (kb + ((mine - 1) * GW + wl) * (kBatch * kBlockSize));
    pool = (lane & 1 ? p.v_pool : p.k_pool) + (size_t)g * kUnit;
    row = p.block_tables + (size_t)d * p.maxb + kb / kBlockSize + wl * kBatch + (lane >> 1);
    left = lane < 2 * kBatch ? nmine - (lane >> 1) : 0;
    next = left > 0 ? *row : 0;
  }

  // The next batch, the warp's batch b, into a slot; all lanes call.
  __device__ __forceinline__ void issue(const Fp4Params& p, int b, uint32_t lane_dst, uint32_t bars,
                                        uint32_t slot, int lane, uint64_t policy) {
    if (lane == 0)
      mbar_arrive_expect_tx(bars + 8 * slot, (uint32_t)min(kBatch, nmine - b * kBatch) * 2 * kUnit);
    if (left > 0) {
      int phys = next;
      if ((uint32_t)phys >= (uint32_t)p.num_blocks) {
        record_error(p.status, POD_ATTN_ERR_BAD_INDEX);
        phys = 0;
      }
      bulk_load(lane_dst + slot * Geo::kSlot,
                pool + (uint64_t)(uint32_t)phys * (uint32_t)(p.Hkv * kUnit), kUnit, bars + 8 * slot,
                policy);
    }
    left -= kBatch;
    row += kBatch * GW;
    if (left > 0) next = *row;
  }

  // The first batches, from the ring's position on: every slot is empty between items.
  __device__ __forceinline__ void start(const Fp4Params& p, uint32_t lane_dst, uint32_t bars,
                                        const Fp4Ring& rg, int lane, uint64_t policy) {
    uint32_t slot = rg.slot;
    for (int b = 0; b < kSlots && b < mine; ++b) {
      issue(p, b, lane_dst, bars, slot, lane, policy);
      slot = slot == kSlots - 1 ? 0 : slot + 1;
    }
  }
};

// The attention of one item on this warp's share of its blocks, whose copies have been started; leaves
// (o, m, l) of each head in the group's scratch. Tensor-core operands, with hr = lane / 4 and
// qd = lane % 4:
//  * S = K q': A is the unit's K (16 keys x 16 channels a step), B the queries (n = head), so a lane
//    gets the scores of keys row(hr), row(hr) + 8 for heads 2qd, 2qd + 1. A lane reads the HD / 4
//    channels [qd * HD / 4, ...) of its two rows as one vector and the queries' channels are taken in
//    the same order, so step ks contracts channels qd * HD / 4 + 4 ks .. + 3 of each qd.
//  * Oᵀ += Vᵀ Pᵀ: A is Vᵀ (rows hr, hr + 8 of m-tile mt are channels hr * HD / 8 + 2 mt, + 1), B is Pᵀ,
//    whose layout movmatrix makes from the scores'. The pairs of A run along the keys: the nibbles of
//    two rows are interleaved before they are converted.
// With one query head (GT == 1) the eight columns of B serve the HD / 16 groups of channels instead, and
// the group scales leave the A operands: column n of q' holds only group n's channels, so a lane's scores
// are sums over single groups, scaled in fp32 and added up over the quad; column n of Pᵀ is the weights
// times group n's V scales, and of the columns of Oᵀ a row's own group is kept. That replaces 64 packed
// products a block by some 20 instructions (Llama-2-7B shape: 7 us less).
// Key index i of both products is row i ^ ((i >> 1) & 1) of the unit: with neighbouring rows swapped
// for every other pair the V reads of a half-warp fall on both halves of the banks.
template <int GT, int HD, int GW>
__device__ __forceinline__ void fp4_item(const Fp4Params& p, const int32_t* it, const DecodeCtx& dc,
                                         Fp4Stream<HD, GW>& st, uint32_t ring, uint32_t lane_dst,
                                         uint32_t bars, Fp4Ring& rg, uint64_t policy, Fp4Group* gc,
                                         const WaitCtx& wc) {
  using Geo = Fp4Geom<HD>;
  constexpr int kSteps = HD / 16;  // k-steps of S, m-tiles of O
  constexpr int kSlots = Geo::kSlots, kBatch = Geo::kBatch, kUnit = Geo::kUnit;
  constexpr int kHeads = GT == 1 ? 1 : 2;  // heads a lane has scores of
  const int lane = threadIdx.x & 31;
  const int wl = (threadIdx.x >> 5) - dc.w0;
  const int d = it[1], g = it[2];
  const int G = p.G;
  const int hr = lane >> 2, qd = lane & 3;

  constexpr bool kOne = GT == 1;
  using Wt = Fp4Weights<GT>;
  // B fragments of q: column hr (a head, or a group of the one head), channels qd * HD / 4 + 4 ks +
  // {0, 1} and {2, 3}
  uint32_t qb[kSteps][2];
#pragma unroll
  for (int ks = 0; ks < kSteps; ++ks) qb[ks][0] = qb[ks][1] = 0u;
  if (kOne || hr < G) {
    const uint4* qv = reinterpret_cast<const uint4*>(
        p.q + ((size_t)d * p.Hq + (size_t)g * G + (kOne ? 0 : hr)) * HD + qd * (HD / 4));
    const auto to_f16 = [](uint32_t two) {
      const float a = bf16lo(two), b = bf16hi(two);
      return pack_f16x2(f16_range(a, a), f16_range(b, b));
    };
#pragma unroll
    for (int j = 0; j < kSteps / 2; ++j) {
      const uint4 w = qv[j];
      qb[2 * j][0] = to_f16(w.x);
      qb[2 * j][1] = to_f16(w.y);
      qb[2 * j + 1][0] = to_f16(w.z);
      qb[2 * j + 1][1] = to_f16(w.w);
    }
    if constexpr (kOne) {
#pragma unroll
      for (int ks = 0; ks < kSteps; ++ks)
        if ((qd * (HD / 4) + 4 * ks) / 16 != hr) qb[ks][0] = qb[ks][1] = 0u;
    }
  }
  const float scale = p.scale_log2 * p.k_scale[g], inv_scale = 1.f / scale;

  float ot[kSteps][4];  // Oᵀ: channels hr * HD / 8 + 2 mt (+ 1) x columns 2qd, 2qd + 1
#pragma unroll
  for (int mt = 0; mt < kSteps; ++mt) ot[mt][0] = ot[mt][1] = ot[mt][2] = ot[mt][3] = 0.f;
  // Running max of each head less kHead (log2 units), the weights' reference from it (its negative, 0
  // before there is one) and the raw score past which it is raised. (One head: only [0].)
  float m[2] = {-INFINITY, -INFINITY}, mr[2] = {0.f, 0.f}, over[2] = {-INFINITY, -INFINITY};
  float l[2] = {0.f, 0.f};
  const int r0 = hr ^ ((hr >> 1) & 1);            // this lane's K rows: r0, r0 + 8
  const int k0 = 2 * qd + (qd & 1), k1 = k0 ^ 1;  // its V rows: k0, k1, k0 + 8, k1 + 8
  const uint32_t v_order = qd & 1 ? 0x1032u : 0x3210u;
  // the lane's places in a slot: K codes and scales, V codes (k0, k1) and scales
  const uint32_t k_at = ring + r0 * (HD / 2) + qd * (HD / 8);
  // (one head: of groups 2qd, 2qd + 1; with 64 channels columns 4 to 7 are empty and any group's do)
  const uint32_t ks_at = ring + 8 * HD + r0 * (HD / 16) +
                         (kOne && HD == 64 ? 2 * (qd & 1) : qd * (HD / 64));
  const uint32_t v_at = ring + kBatch * kUnit + k0 * (HD / 2) + hr * (HD / 16);
  const uint32_t v_at1 = ring + kBatch * kUnit + k1 * (HD / 2) + hr * (HD / 16);
  const uint32_t vs_at = ring + kBatch * kUnit + 8 * HD + 2 * qd +
                         (kOne ? hr % (HD / 16) : hr * HD / 128) * kBlockSize;
  const int mine = st.mine, last_rows = st.last_rows;
  const int tail_batch = last_rows < kBatch * kBlockSize ? mine - 1 : -1;

  // One batch. Only the warp's last one can have rows that do not exist: it has code of its own, so that
  // the others carry no masks.
  auto batch = [&](uint32_t off, auto tail) {
    constexpr bool kTail = decltype(tail)::value;
    // ---- scores
    float s[kBatch][4];
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      uint32_t kw[2][kSteps / 2];  // 8 channels a word
      uint32_t ks2[2][2];          // f16 pair (s, s) of row j, group h of the lane's channels
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint32_t src = k_at + off + u * kUnit + 8 * j * (HD / 2);
        const uint32_t sc = ks_at + off + u * kUnit + 8 * j * (HD / 16);
        if constexpr (HD == 128) {
          const uint4 w = lds_v4(src);
          kw[j][0] = w.x, kw[j][1] = w.y, kw[j][2] = w.z, kw[j][3] = w.w;
        } else {
          const uint2 w = lds_v2(src);
          kw[j][0] = w.x, kw[j][1] = w.y;
        }
        const uint32_t f = e4m3x2_to_f16x2(kOne || HD == 128 ? lds_u16(sc) : lds_u8(sc));
        if constexpr (kOne) {
          ks2[j][0] = f;  // groups 2qd, 2qd + 1
        } else {
          ks2[j][0] = __byte_perm(f, f, 0x1010);
          ks2[j][1] = HD == 128 ? __byte_perm(f, f, 0x3232) : ks2[j][0];
        }
      }
#pragma unroll
      for (int w = 0; w < kSteps / 2; ++w) {
        const int h = HD == 128 ? w >> 1 : 0;
        uint32_t f0[4], f1[4];
        e2m1x8_to_f16x2(kw[0][w], f0);
        e2m1x8_to_f16x2(kw[1][w], f1);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          uint32_t a[4] = {f0[2 * j], f1[2 * j], f0[2 * j + 1], f1[2 * j + 1]};
          if constexpr (!kOne) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = hmul2(a[i], ks2[i & 1][h]);
          }
          if (w + j == 0)
            mma_16816_f16_zero(s[u], a, qb[0][0], qb[0][1]);
          else
            mma_16816_f16(s[u], a, qb[2 * w + j][0], qb[2 * w + j][1]);
        }
      }
      if constexpr (kOne) {  // the groups' sums, scaled, over the quad: s[u][0], s[u][2] of rows r0, r0 + 8
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float x = fmaf(s[u][2 * j], f16lo(ks2[j][0]), s[u][2 * j + 1] * f16hi(ks2[j][0]));
          x += __shfl_xor_sync(0xffffffffu, x, 1);
          s[u][2 * j] = x + __shfl_xor_sync(0xffffffffu, x, 2);
        }
      }
    }
    if constexpr (kTail) {
#pragma unroll
      for (int u = 0; u < kBatch; ++u)
#pragma unroll
        for (int e = 0; e < 4; ++e)
          if (r0 + u * kBlockSize + (e >> 1) * 8 >= last_rows) s[u][e] = -INFINITY;
    }
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int u = 0; u < kBatch; ++u)
#pragma unroll
      for (int e = 0; e < kHeads; ++e) mx[e] = fmax3(mx[e], s[u][e], s[u][2 + e]);
    if (__any_sync(0xffffffffu, mx[0] > over[0] || (!kOne && mx[1] > over[1]))) {
#pragma unroll
      for (int e = 0; e < kHeads; ++e) {
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
          mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], o));
        const float m_new = mx[e] * scale - Wt::kHead;
        if (m_new > m[e]) {
          const float alpha = ex2(m[e] - m_new);
          m[e] = m_new;
          mr[e] = -m_new;
          over[e] = mx[e] + Wt::kLazy * inv_scale;
          l[e] *= alpha;
#pragma unroll
          for (int mt = 0; mt < kSteps; ++mt) {
            ot[mt][e] *= alpha;
            ot[mt][2 + e] *= alpha;
            if constexpr (kOne) ot[mt][1] *= alpha, ot[mt][3] *= alpha;
          }
        }
      }
    }
    // ---- output
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      uint32_t pb[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float p0 = ex2(fmaf(s[u][2 * j], scale, mr[0]));
        const float p1 = kOne ? p0 : ex2(fmaf(s[u][2 * j + 1], scale, mr[1]));
        l[0] += p0;
        if constexpr (!kOne) l[1] += p1;
        pb[j] = movmatrix_trans(pack_f16x2(p0, p1));
      }
      uint32_t vw[4][HD / 64];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t src = (j & 1 ? v_at1 : v_at) + off + u * kUnit + (j & 2 ? 8 * (HD / 2) : 0);
        if constexpr (HD == 128) {
          const uint2 w = lds_v2(src);
          vw[j][0] = w.x, vw[j][1] = w.y;
        } else {
          vw[j][0] = lds_u32(src);
        }
      }
      uint32_t vs[2];  // f16 pair of the scales of keys (k0, k1), (k0 + 8, k1 + 8)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        uint32_t f = e4m3x2_to_f16x2(lds_u16(vs_at + off + u * kUnit + 8 * j));
        if constexpr (kTail) {
          // rows behind the sequence's last may hold anything, even a NaN scale: weight 0 times 0
          const int key = u * kBlockSize + 2 * qd + 8 * j;
          if (key >= last_rows) f &= 0xFFFF0000u;
          if (key + 1 >= last_rows) f &= 0x0000FFFFu;
        }
        vs[j] = __byte_perm(f, f, v_order);
        if constexpr (kOne) pb[j] = hmul2(pb[j], vs[j]);
      }
      constexpr uint32_t kLo = 0x0F0F0F0Fu;
#pragma unroll
      for (int w = 0; w < HD / 64; ++w) {
        uint32_t f[4][4];  // channels even, odd of keys (k0, k1), then of (k0 + 8, k1 + 8)
        e2m1x8_to_f16x2((vw[0][w] & kLo) | ((vw[1][w] << 4) & ~kLo), f[0]);
        e2m1x8_to_f16x2(((vw[0][w] >> 4) & kLo) | (vw[1][w] & ~kLo), f[1]);
        e2m1x8_to_f16x2((vw[2][w] & kLo) | ((vw[3][w] << 4) & ~kLo), f[2]);
        e2m1x8_to_f16x2(((vw[2][w] >> 4) & kLo) | (vw[3][w] & ~kLo), f[3]);
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t a[4] = {f[0][c], f[1][c], f[2][c], f[3][c]};
          if constexpr (!kOne) {
#pragma unroll
            for (int i = 0; i < 4; ++i) a[i] = hmul2(a[i], vs[i >> 1]);
          }
          mma_16816_f16(ot[4 * w + c], a, pb[0], pb[1]);
        }
      }
    }
  };
  for (int b = 0; b < mine; ++b) {
    const bool got = mbar_wait(bars + 8 * rg.slot, rg.parity, wc, kFp4SleepNs);
    if (!__all_sync(0xffffffffu, got)) {
      if (lane == 0) *static_cast<volatile int*>(&gc->abort) = 1;
      break;
    }
    const uint32_t off = rg.slot * Geo::kSlot;
    if (b == tail_batch)
      batch(off, std::true_type{});
    else
      batch(off, std::false_type{});
    __syncwarp();  // every lane has read the slot
    if (b + kSlots < mine) st.issue(p, b + kSlots, lane_dst, bars, rg.slot, lane, policy);
    if (++rg.slot == kSlots) {
      rg.slot = 0;
      rg.parity ^= 1;
    }
  }
#pragma unroll
  for (int e = 0; e < kHeads; ++e)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) l[e] += __shfl_xor_sync(0xffffffffu, l[e], off);
  float* scr = reinterpret_cast<float*>(dc.ring) + wl * GT * kScr;
#pragma unroll
  for (int e = 0; e < kHeads; ++e) {
    const int head = kOne ? 0 : 2 * qd + e;
    if (head >= G) continue;
    float* dst = scr + head * kScr;
    const int group = hr * HD / 128;  // one head: the column of this lane's rows
    if (!kOne || qd == group >> 1) {
#pragma unroll
      for (int mt = 0; mt < kSteps; ++mt) {
        const bool second = kOne ? group & 1 : e;
        *reinterpret_cast<float2*>(dst + hr * (HD / 8) + 2 * mt) =
            second ? make_float2(ot[mt][1], ot[mt][3]) : make_float2(ot[mt][0], ot[mt][2]);
      }
    }
    if (hr == 0 && (!kOne || qd == 0)) {
      // scores that are all NaN leave the max at -inf: their weights were taken against 0
      dst[kHeadDim] = m[e] == -INFINITY && l[e] != l[e] ? 0.f : m[e];
      dst[kHeadDim + 1] = l[e];
    }
  }
}

template <int GT, int HD, int GW, bool kLevels>
__global__ void __launch_bounds__(kFp4Threads, 1) decode_fp4_kernel(const __grid_constant__ Fp4Params p) {
  extern __shared__ __align__(1024) uint8_t smem[];
  using Geo = Fp4Geom<HD>;
  constexpr int kGroups = kFp4Warps / GW;
  uint8_t* scratch = smem + kFp4Warps * Geo::kRing;
  Fp4Ctl* ctl = reinterpret_cast<Fp4Ctl*>(scratch + kFp4Warps / kDecodeWarps * kFp4Scratch<GT>);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, grp = warp / GW, wl = warp % GW;
  if (tid < kFp4Warps * kFp4MaxSlots)
    mbar_init(smem_u32(&ctl->full[0][0] + tid), 1);
  if (tid == 0) ctl->abort = 0;
  if (tid < kGroups) ctl->group[tid].abort = 0;
  fence_barrier_init();
  __syncthreads();
  griddep_wait();
  const WaitCtx wc{&ctl->abort, p.status, p.timeout_ns};
  const DecodeCtx dc{grp * GW, GW,      scratch + grp * kFp4Scratch<GT>, nullptr,
                     1 + grp,  GW * 32, grp * GW * 32,                   0};
  Fp4Group* gc = &ctl->group[grp];
  const uint32_t ring = smem_u32(smem + warp * Geo::kRing);
  const uint32_t lane_dst = ring + ((lane & 1) * Geo::kBatch + (lane >> 1)) * Geo::kUnit;
  const uint32_t bars = smem_u32(&ctl->full[warp][0]);
  const uint64_t policy = policy_evict_first();  // the cache is read once
  const bool leader = tid == dc.first_thread;
  Fp4Ring rg;
  // The first shares are dealt out over the CTAs before their groups, so that a few shares spread over
  // all SMs; further ones by ticket.
  int share = grp * (int)gridDim.x + (int)blockIdx.x;
  while (share < p.n_shares) {
    bool bad = false;
    int idx = share;  // the share's first item; word 3 of an item names the next
    const int32_t* it = p.items + (size_t)idx * kItemWords;
    Fp4Stream<HD, GW> st(p, it, wl, lane);
    st.start(p, lane_dst, bars, rg, lane, policy);
    for (;;) {
      const uint64_t t0 = p.records != nullptr && leader ? globaltimer() : 0;
      fp4_item<GT, HD, GW>(p, it, dc, st, ring, lane_dst, bars, rg, policy, gc, wc);
      const int d = it[1], g = it[2], next = it[3], unit = it[6], split = it[7];
      named_bar_sync(dc.bar_id, dc.bar_threads);
      bad = *static_cast<volatile int*>(&gc->abort) != 0;
      if (bad) break;
      if (next != 0) {  // the next item's copies run beside this one's combination
        it = p.items + (size_t)next * kItemWords;
        st = Fp4Stream<HD, GW>(p, it, wl, lane);
        st.start(p, lane_dst, bars, rg, lane, policy);
      }
      combine_decode<GT, HD, GW, kLevels>(p, d, g, unit, split, dc, gc, p.v_scale[g]);
      if (p.records != nullptr && leader) {
        pod_attn_item_record* rec = p.records + idx;
        rec->smid = (int32_t)smid();
        rec->kind = 1;
        rec->item = idx;
        rec->cta = blockIdx.x;
        rec->t_start = t0;
        rec->t_end = globaltimer();
      }
      if (next == 0) break;
      idx = next;
    }
    if (bad) break;
    if (leader) gc->share = atomicAdd(&p.counters[1], 1) + kGroups * (int)gridDim.x;
    named_bar_sync(dc.bar_id, dc.bar_threads);
    share = gc->share;
  }
  __syncthreads();
  if (ctl->abort) {
    // give copies still in flight time to land before this CTA's shared memory is released
    if (tid == 0) {
      const uint64_t t0 = globaltimer();
      while (globaltimer() - t0 < 2000000ull) __nanosleep(1000);
    }
    __syncthreads();
  }
  if (tid == 0) {
    __threadfence();
    if (atomicAdd(&p.counters[2], 1) == (int)gridDim.x - 1) {  // the last CTA resets the counters
      p.counters[1] = 0;
      p.counters[2] = 0;
      __threadfence();
    }
  }
}

template <int GT, int HD, int GW, bool kLevels>
cudaError_t launch_fp4(const Fp4Params& p, int grid, cudaStream_t st) {
  // once per device: the kernel's shared memory is above the default limit
  static std::atomic<uint64_t> ready{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? uint64_t(1) << dev : 0;
  if (!bit || !(ready.load() & bit)) {
    e = cudaFuncSetAttribute(decode_fp4_kernel<GT, HD, GW, kLevels>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             fp4_smem<GT, HD>());
    if (e != cudaSuccess) return e;
    ready.fetch_or(bit);
  }
  return launch_early(decode_fp4_kernel<GT, HD, GW, kLevels>, dim3(grid), kFp4Threads,
                      fp4_smem<GT, HD>(), st, p);
}

// Heads that the kernel of a group of G heads has room for.
constexpr int fp4_group(int G) { return G <= 2 ? G : G <= 4 ? 4 : kMaxGroup; }

template <int HD, int GW, bool kLevels>
cudaError_t launch_fp4(const Fp4Params& p, int grid, cudaStream_t st) {
  switch (fp4_group(p.G)) {
    case 1: return launch_fp4<1, HD, GW, kLevels>(p, grid, st);
    case 2: return launch_fp4<2, HD, GW, kLevels>(p, grid, st);
    case 4: return launch_fp4<4, HD, GW, kLevels>(p, grid, st);
    default: return launch_fp4<kMaxGroup, HD, GW, kLevels>(p, grid, st);
  }
}

}  // namespace

int fp4_smem_bytes(int group, int head_dim) {
  const auto of = [&](auto gt) {
    constexpr int GT = decltype(gt)::value;
    return head_dim == 64 ? fp4_smem<GT, 64>() : fp4_smem<GT, 128>();
  };
  switch (fp4_group(group)) {
    case 1: return of(std::integral_constant<int, 1>{});
    case 2: return of(std::integral_constant<int, 2>{});
    case 4: return of(std::integral_constant<int, 4>{});
    default: return of(std::integral_constant<int, kMaxGroup>{});
  }
}

}  // namespace pod

using namespace pod;

extern "C" pod_attn_status pod_attn_run_decode_fp4(pod_attn_plan_t plan, const void* q_decode,
                                                   const pod_attn_kv_cache* cache,
                                                   const int32_t* d_block_tables,
                                                   const int32_t* d_kv_lens, void* o_decode,
                                                   void* workspace, size_t workspace_bytes,
                                                   void* stream) {
  if (!plan) return POD_ATTN_ERR_INVALID_ARG;
  const pod_attn_status st = check_workspace(plan, workspace, workspace_bytes);
  if (st != POD_ATTN_OK) return st;
  const pod_attn_problem& pr = plan->prob;
  if (!plan->opt.kv_fp4 || pr.num_prefill_seqs != 0) return POD_ATTN_ERR_UNSUPPORTED;
  const int n_d = (int)(plan->items_d.size() / kItemWords);
  if (n_d == 0) return POD_ATTN_OK;
  if (!cache) return POD_ATTN_ERR_INVALID_ARG;
  if (cache->type != POD_ATTN_KV_E2M1) return POD_ATTN_ERR_UNSUPPORTED;
  if (!q_decode || !o_decode || !d_block_tables || !d_kv_lens || !cache->k_pool || !cache->v_pool ||
      !cache->k_scale || !cache->v_scale || cache->num_blocks != pr.num_blocks)
    return POD_ATTN_ERR_INVALID_ARG;
  if (!aligned16({q_decode, o_decode}) || !cache_aligned(*cache))
    return POD_ATTN_ERR_INVALID_ARG;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  const WorkspaceLayout& w = plan->ws;
  Fp4Params p{};
  p.q = static_cast<const uint16_t*>(q_decode);
  p.k_pool = static_cast<const uint8_t*>(cache->k_pool);
  p.v_pool = static_cast<const uint8_t*>(cache->v_pool);
  p.k_scale = cache->k_scale;
  p.v_scale = cache->v_scale;
  p.block_tables = d_block_tables;
  p.items = reinterpret_cast<const int32_t*>(ws + w.items_d);
  p.units = reinterpret_cast<const int32_t*>(ws + w.units);
  p.o_decode = static_cast<uint16_t*>(o_decode);
  p.partial_d = reinterpret_cast<float*>(ws + w.partial_d);
  p.counters = reinterpret_cast<int32_t*>(ws + w.counters);  // the fused launch's block
  p.arrive = reinterpret_cast<int32_t*>(ws + w.arrive);
  p.status = reinterpret_cast<int32_t*>(ws + w.status);
  p.records = plan->opt.instrument ? reinterpret_cast<pod_attn_item_record*>(ws + w.records) : nullptr;
  p.n_shares = plan->num_shares;
  p.Hq = pr.num_q_heads;
  p.Hkv = pr.num_kv_heads;
  p.G = plan->group;
  p.maxb = pr.max_blocks_per_seq;
  p.num_blocks = pr.num_blocks;
  p.scale_log2 = pr.scale * 1.4426950408889634f;
  p.timeout_ns = kFp4TimeoutNs;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const int grid = plan->grid_fused;
  cudaError_t e;
  if (plan->fp4_group_warps == kFp4Warps)
    e = pr.head_dim == 64 ? launch_fp4<64, kFp4Warps, true>(p, grid, s)
                          : launch_fp4<128, kFp4Warps, true>(p, grid, s);
  else if (plan->fp4_levels)
    e = pr.head_dim == 64 ? launch_fp4<64, kDecodeWarps, true>(p, grid, s)
                          : launch_fp4<128, kDecodeWarps, true>(p, grid, s);
  else
    e = pr.head_dim == 64 ? launch_fp4<64, kDecodeWarps, false>(p, grid, s)
                          : launch_fp4<128, kDecodeWarps, false>(p, grid, s);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return POD_ATTN_ERR_CUDA;
  }
  return POD_ATTN_OK;
}
