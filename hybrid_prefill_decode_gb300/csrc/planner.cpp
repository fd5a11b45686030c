// planner.cpp — host planner of the hybrid prefill+decode launch.
//
// "POD-Attention" digest (Silicon & Systems), §"가상 CTA와 SM별 균형": a normal grid of CTAs
// is mapped onto virtual prefill and decode CTAs; the number of CTAs one prefill chunk may
// generate is limited so decode work is not pushed out. §"동시 실행만으로 부족한 이유": a CTA
// count just above a multiple of what the SMs hold at once costs a whole extra wave.
//
// This file turns one hybrid batch into two work lists (virtual CTAs):
//   prefill item = (chunk s, tile t, block of hp query heads, KV split k) — a tile is 128
//                  rows = 128/hp tokens x hp heads of one kv-head group
//   decode item  = (sequence d, kv-head g, KV split k)   — one item serves all G query heads
//                  of the kv-head (GQA grouping, "LLMSO - W4", §"KV 헤드 줄이기")
// and sizes the persistent grid: one CTA per SM, each with a prefill slot and a decode slot
// that pull items from the two lists.
//
// Split planning. Every item gets a cost (decode: 8 per 16-row K/V block, i.e. its bytes in
// KiB; prefill: 57 per 128-key step of its 128 rows, its tensor-core time expressed in the
// same byte-time units at a 6.8 TB/s : 1 PFLOP/s balance). Outputs are split along the keys
// ("LLMSO - W4", §"FlashDecoding — decode 단계의 병렬성 확보"), so no single item can leave a
// long tail after the others finish:
//  * prefill: one chunk size c (steps per item) for all outputs, c = ceil(longest / k) for
//    k = 1..8 (at least 4 steps), the one that minimises the makespan of the items taken
//    longest first by the SMs' prefill slots, each to the slot that frees first, with a fixed
//    per-item overhead. A split count just past a multiple of the SMs costs a whole extra
//    round of items (§"동시 실행만으로 부족한 이유"), which this model sees.
//  * decode: with W the total cost and S the item slots, an output whose cost exceeds
//    W / (4 S) is split into at most 64 parts of at least 12 blocks.
// Items are then ordered longest first. All arithmetic is integer, so the plan is reproducible
// bit for bit.
//
// Decode-only plans (no prefill work; the FP8-cache decode is one) know how many items run at
// once: S = groups x SMs 4-warp decode groups (3 per SM on a bf16 cache, where the prefill
// slot's softmax warps become two groups beside the decode slot; 4 on an e4m3 cache, where its
// producer and issuer warps become a third). There one chunk size c (blocks per item, before
// each output is rebalanced into equal parts) is chosen for all outputs to minimise the makespan of
// the items taken longest first by S groups, modelled wave by wave (each wave of S items lasts
// as long as its longest), each item costing ceil(blocks / 4) + 2 block-times of one warp (its
// four warps share the blocks; the 2 stand for its start and merge). A split count just past a multiple of S costs a whole extra wave
// of items (the wave-quantisation point of §"동시 실행만으로 부족한 이유"), which the
// W / (4 S) rule above cannot see.
//
// Plans for the 4-bit cache (kv_fp4) deal the work out in shares, one for each group of warps of the GPU
// at most, which a group takes whole. A group is four warps, or where it is likely to be sooner done
// (fp4_time) all sixteen of an SM: a sixteenth of an output's blocks for each warp, fewer partials and more
// threads to merge them. That suits a GPU with no more outputs than SMs. (16 sequences of 1024 rows, 8
// kv-heads of 4 heads of 128 channels: 11.1 us in groups of sixteen, 12.9 in groups of four; 20 sequences
// 19 and 15. One of 131072 rows, one kv-head of 8 heads: 17.1 and 21.9 us.) Two ways of cutting are
// compared, in blocks (an item's start and merge count as fp4_item_blocks of them):
//  * apart: every share is a piece of one output, no longer than a size S; the least S, in whole rounds
//    of the group's warps, with which the pieces are no more than the groups. A rest that costs more
//    than it evens out is shared among an output's other pieces.
//  * through: the outputs' blocks, one output after another, are cut into equal shares, whatever
//    outputs they span. All groups finish together, without the waves that whole items come in; a
//    share that spans outputs pays for their starts and merges.
// 512 outputs of 515 to 1015 blocks on 608 groups took 157 us cut through and 167 us as items in waves; 64
// outputs of 256 blocks 17 us apart and 21 us through.
#include <algorithm>
#include <cmath>
#include <cstring>
#include <functional>
#include <numeric>
#include <queue>

#include "pod_internal.h"

namespace pod {
namespace {

constexpr int64_t kDecodeBlockCost = 8;   // 16 rows x (K + V) x 128 x bf16 = 8 KiB
constexpr int64_t kPrefillStepCost = 57;  // 4*128*128*128 FLOPs at the byte-time balance
constexpr int kMinDecodeBlocksPerSplit = 12;
constexpr int kMinPrefillTilesPerSplit = 4;
constexpr int64_t kPrefillItemOverhead = 8;  // per-item start and epilogue, in steps
constexpr int64_t kDecodeItemOverhead = 2;   // per-item start and merge, in warp block-times
constexpr int kDecodeGroupsBf16 = 3;         // 4-warp decode groups per SM, bf16 cache
constexpr int kDecodeGroupsFp8 = 4;          // ... e4m3 cache
constexpr int kFp4Flat = 32;  // most splits of the 4-bit decode that are merged at once
// Start and merge of an item in blocks: 12 of 128-channel heads, 24 of 64. (An output of 32 blocks takes
// 8.8 us whole and 9.3 us in two items, one of 64 blocks 12 and 10.3 us; with 64 channels 64 blocks take
// 8.2 and 10.1 us.)
constexpr int64_t fp4_item_blocks(int64_t round) { return round * 3 / 2; }
// chunk candidates of the decode-only rule: ceil(longest output / k)
constexpr int kChunkDivisors[] = {1, 2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 40, 48, 64};

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

size_t align256(size_t x) { return (x + 255) & ~size_t(255); }

// Split of one output of `nblk` blocks for a chunk of about `c` blocks: ns parts of
// ceil(nblk / ns) blocks (the last one shorter).
inline void rebalanced(int64_t nblk, int64_t c, int64_t* ns, int64_t* chunk) {
  *ns = std::max<int64_t>(1, std::min(ceil_div(nblk, c), nblk));
  *chunk = ceil_div(nblk, *ns);
  *ns = ceil_div(nblk, *chunk);
}

// Modelled makespan (in warp block-times) of the items that chunk size c makes of the outputs
// `nblks` on `slots` decode groups taking them longest first: wave w holds the items ranked
// w*slots .. (w+1)*slots - 1 and lasts as long as its first (longest) one. Item costs are
// counted in `hist` (indexed by cost), so this is linear in the outputs and the largest cost.
int64_t decode_makespan(const std::vector<int64_t>& nblks, int64_t c, int64_t slots,
                        std::vector<int64_t>& hist) {
  std::fill(hist.begin(), hist.end(), 0);
  int64_t top = 0;
  for (int64_t n : nblks) {
    int64_t ns, ch;
    rebalanced(n, c, &ns, &ch);
    const int64_t full = ceil_div(ch, 4) + kDecodeItemOverhead;
    const int64_t last = ceil_div(n - (ns - 1) * ch, 4) + kDecodeItemOverhead;
    hist[full] += ns - 1;
    hist[last] += 1;
    top = std::max(top, full);
  }
  int64_t span = 0, rank = 0, next_head = 0;  // rank of the next item; rank of the next wave head
  for (int64_t x = top; x > 0; --x) {
    const int64_t k = hist[x];
    if (k == 0) continue;
    // wave heads among ranks [rank, rank + k)
    if (next_head < rank + k) {
      const int64_t heads = (rank + k - 1 - next_head) / slots + 1;
      span += heads * x;
      next_head += heads * slots;
    }
    rank += k;
  }
  return span;
}

// Modelled makespan (in steps) of the prefill items that chunk size c makes of the outputs
// `nts` on `slots` prefill slots taking them longest first, each to the slot that frees first
// (list scheduling); an item costs its steps plus kPrefillItemOverhead. The makespan depends
// only on the multiset of slot loads, so the items are counted by cost (`hist`) and the loads
// kept as a histogram (`load`): the least loaded slot's load never decreases, so a cursor
// finds it, and the whole model is linear in the items and the largest load.
int64_t prefill_makespan(const std::vector<int64_t>& nts, int64_t c, int64_t slots,
                         std::vector<int64_t>& hist, std::vector<int64_t>& load) {
  int64_t top = 0, total = 0;
  for (int64_t n : nts) top = std::max(top, std::min(c, n) + kPrefillItemOverhead);
  hist.assign((size_t)top + 1, 0);
  for (int64_t n : nts) {
    int64_t ns, ch;
    rebalanced(n, c, &ns, &ch);
    const int64_t last = n - (ns - 1) * ch + kPrefillItemOverhead;
    hist[(size_t)(ch + kPrefillItemOverhead)] += ns - 1;
    hist[(size_t)last] += 1;
    total += (ns - 1) * (ch + kPrefillItemOverhead) + last;
  }
  // an item starts at the least load, which is at most total / slots
  load.assign((size_t)(total / slots + top + 1), 0);
  load[0] = slots;
  int64_t cur = 0, span = 0;
  for (int64_t x = top; x > 0; --x) {
    // the k items of cost x go to the k least loaded slots, as many at a time as share a load
    for (int64_t k = hist[(size_t)x]; k > 0;) {
      while (load[(size_t)cur] == 0) ++cur;
      const int64_t m = std::min(k, load[(size_t)cur]);
      load[(size_t)cur] -= m;
      load[(size_t)(cur + x)] += m;
      span = std::max(span, cur + x);
      k -= m;
    }
  }
  return span;
}

// Splits of a bundle of the 4-bit decode's merge: as many as there will be bundles. 0: all at once, up to
// kFp4Flat of them where a thread of the group has one pair of the output's channels, and up to kFp4Bundle
// where it has more. (MHA of 128 channels, four sequences of 20000 rows in 18 splits: 23.3 us at once, 24.1
// in bundles; one of 16384 rows in 64: 13.3 and 11.7.)
int fp4_bundle(int64_t nsplit, int pairs, int group_warps) {
  if (nsplit <= (pairs <= 32 * group_warps ? kFp4Flat : kFp4Bundle)) return 0;
  int b = 1;
  while (b * b < nsplit) ++b;
  return b;
}

// One decode item of a plan by shares: blocks [first, end) of output `out`.
struct Piece {
  size_t out;
  int64_t first, end;
};

// The shares of a plan: their pieces in order, share s from starts[s] up to starts[s + 1].
struct Shares {
  std::vector<Piece> pieces;
  std::vector<int32_t> starts;
};

// Cut outputs of nblks blocks each into at most `groups` shares (see the top of the file), in units of
// `round` blocks (what the warps of a group take in one pass).
Shares cut_shares(const std::vector<int64_t>& nblks, int64_t groups, int64_t round) {
  const int64_t outs = (int64_t)nblks.size(), item = fp4_item_blocks(round);
  int64_t total = 0, longest = 0;
  for (int64_t n : nblks) {
    total += n;
    longest = std::max(longest, n);
  }
  // Least pieces: two rounds, and long enough for at most kMaxFp4Splits of an output, of which cuts
  // through may leave one more than whole ones would be.
  const auto least = [&](int splits) {
    return ceil_div(std::max(2 * round, ceil_div(longest, splits)), round) * round;
  };
  Shares cut;
  std::vector<Piece>& out = cut.pieces;
  std::vector<int32_t>& starts = cut.starts;
  int64_t apart = 0;
  if (outs <= groups) {
    int64_t lo = least(kMaxFp4Splits) / round, hi = std::max(lo, ceil_div(longest, round));
    while (lo < hi) {  // the pieces of a longer size are never more
      const int64_t mid = (lo + hi) / 2;
      int64_t n = 0;
      for (int64_t x : nblks) n += ceil_div(x, mid * round);
      if (n <= groups) hi = mid; else lo = mid + 1;
    }
    apart = lo * round;
  }
  const int64_t sum = total + outs * item;
  const int64_t n = std::max<int64_t>(
      1, std::min(groups, sum / (least(kMaxFp4Splits - 1) + item)));
  if (apart > 0 && std::min(apart, longest) <= sum / n + item) {
    for (size_t o = 0; o < nblks.size(); ++o) {
      int64_t k = ceil_div(nblks[o], apart);
      const int64_t rest = nblks[o] - (k - 1) * apart;
      if (k == 2 ? rest < 2 * item : k > 2 && rest < item) --k;  // a single piece needs no merge at all
      const int64_t len = ceil_div(ceil_div(nblks[o], k), round) * round;
      for (int64_t at = 0; at < nblks[o]; at += len) {
        starts.push_back((int32_t)out.size());
        out.push_back({o, at, std::min(nblks[o], at + len)});
      }
    }
  } else {
    // equal shares of blocks and item costs; `at` counts blocks of output o, `done` what is dealt out
    size_t o = 0;
    int64_t at = 0, done = 0;
    for (int64_t i = 0; i < n && o < nblks.size(); ++i) {
      const int64_t end = (i + 1) * sum / n;
      if (end <= done && i < n - 1) continue;  // an output's end has moved past it
      starts.push_back((int32_t)out.size());
      while (o < nblks.size() && (done < end || out.size() == (size_t)starts.back())) {
        const int64_t cost = at == 0 ? item : 0;
        int64_t take = nblks[o] - at;
        if (i < n - 1 && end - done < cost + take) {  // the share ends inside this output
          take = (end - done - cost) / round * round;
          const bool first = out.size() == (size_t)starts.back();
          if (nblks[o] - at - take < item) {
            take = nblks[o] - at;  // a rest that would cost more than it evens out
          } else if (take < item) {
            if (!first) break;  // a beginning that would: it stays with the next share
            take = std::min(nblks[o] - at, ceil_div(item, round) * round);
          }
        }
        out.push_back({o, at, at + take});
        at += take;
        done += cost + take;
        if (at == nblks[o]) {
          ++o;
          at = 0;
        }
      }
    }
  }
  starts.push_back((int32_t)out.size());
  return cut;
}

// About how long shares take (in 1/20 us, without the launch) in groups of `warps` warps, pairs pairs of
// channels an output. A round of four warps takes 0.65 us alone and 0.45 for each of the SM's groups when
// they share it, one of 16 warps 1.9; to this an item's start and the merge. Of 176 batches of 1 to 76
// sequences of 64 to 131072 rows (64 and 128 channels, 1 to 8 heads) the choice between the two groups takes
// 0.7 % more than the better one on average and 12 % at worst, and 5.9 % less than groups of four always.
int64_t fp4_time(const Shares& cut, int64_t num_sms, int64_t round, int warps, int pairs) {
  const bool wide = warps == kFp4Warps;
  const int64_t shares = (int64_t)cut.starts.size() - 1;
  const int64_t busy = std::min<int64_t>(kFp4Warps / kDecodeWarps, ceil_div(shares, num_sms));
  const int64_t per_round = wide ? 38 : std::max<int64_t>(13, 9 * busy), per_item = wide ? 38 : 45;
  int64_t longest = 0;
  for (int64_t s = 0; s < shares; ++s) {
    int64_t at = 0;
    for (int32_t i = cut.starts[s]; i < cut.starts[s + 1]; ++i)
      at += per_item + per_round * ceil_div(cut.pieces[i].end - cut.pieces[i].first, round);
    longest = std::max(longest, at);
  }
  int64_t most = 1, n = 0;
  for (const Piece& x : cut.pieces) {
    n = x.first == 0 ? 1 : n + 1;
    most = std::max(most, n);
  }
  if (most == 1) return longest;
  if (wide) return longest + 54;
  return longest + 10 + (pairs > 32 * warps ? 54 : 0) + (fp4_bundle(most, pairs, warps) > 0 ? 68 : 0);
}

}  // namespace

pod_attn_status build_plan(const pod_attn_problem& prob, const int32_t* cu, const int32_t* kv,
                           const pod_attn_options& opt, int num_sms, pod_attn_plan_s* plan) {
  const int Hq = prob.num_q_heads, Hkv = prob.num_kv_heads;
  const int Np = prob.num_prefill_seqs, Nd = prob.num_decode_seqs;
  if (Hq < 1 || Hkv < 1 || Np < 0 || Nd < 0 || prob.num_prefill_tokens < 0 ||
      prob.num_blocks < 0 || prob.max_blocks_per_seq < 0 || !std::isfinite(prob.scale) ||
      !(prob.scale > 0.f))
    return POD_ATTN_ERR_INVALID_ARG;
  if (Hq % Hkv != 0) return POD_ATTN_ERR_INVALID_ARG;
  if (opt.ctas_per_sm < 0 || opt.max_prefill_ctas < 0) return POD_ATTN_ERR_INVALID_ARG;
  if (opt.kv_fp8 && opt.kv_fp4) return POD_ATTN_ERR_INVALID_ARG;
  // one persistent CTA per SM holds both slots (232 KiB of shared memory, all 512 TMEM columns)
  if (opt.ctas_per_sm > 1) return POD_ATTN_ERR_UNSUPPORTED;
  // head dims 128 and 64 (the layouts are sized for 128; 64 uses their first half)
  if ((prob.head_dim != kHeadDim && prob.head_dim != 64) || prob.block_size != kBlockSize)
    return POD_ATTN_ERR_UNSUPPORTED;
  const int D = prob.head_dim;
  const int G = Hq / Hkv;
  if (G > kMaxGroup) return POD_ATTN_ERR_UNSUPPORTED;
  if ((Np == 0) != (prob.num_prefill_tokens == 0)) return POD_ATTN_ERR_INVALID_ARG;
  if (Np > 0 && cu == nullptr) return POD_ATTN_ERR_INVALID_ARG;
  if (Np + Nd > 0 && (kv == nullptr || prob.num_blocks < 1 || prob.max_blocks_per_seq < 1))
    return POD_ATTN_ERR_INVALID_ARG;
  if (num_sms < 1) return POD_ATTN_ERR_INVALID_ARG;
  // TMA row coordinates of the pools are int32.
  if ((int64_t)prob.num_blocks * Hkv * kBlockSize >= (int64_t(1) << 31))
    return POD_ATTN_ERR_UNSUPPORTED;
  const int64_t max_rows = (int64_t)prob.max_blocks_per_seq * kBlockSize;
  if (Np > 0) {
    if (cu[0] != 0 || cu[Np] != prob.num_prefill_tokens) return POD_ATTN_ERR_INVALID_ARG;
    for (int s = 0; s < Np; ++s) {
      int64_t q = (int64_t)cu[s + 1] - cu[s];
      if (q < 1 || kv[s] < q || kv[s] > max_rows) return POD_ATTN_ERR_INVALID_ARG;
    }
  }
  for (int d = 0; d < Nd; ++d)
    if (kv[Np + d] < 1 || kv[Np + d] > max_rows) return POD_ATTN_ERR_INVALID_ARG;

  plan->prob = prob;
  plan->opt = opt;
  plan->group = G;
  const int hp = G & -G;  // largest power of two dividing G (G <= 8)
  const int tq = kTileM / hp;
  plan->head_pack = hp;
  plan->tile_tokens = tq;
  plan->num_sms = num_sms;
  plan->ctas_per_sm = 1;  // one CTA per SM holds both slots (and all 512 TMEM columns)
  // the cap on CTAs that take prefill items ("POD-Attention" digest, §"가상 CTA와 SM별 균형": the
  // CTAs one prefill may take are limited so decode work is not crowded out); 0 = every CTA
  const int prefill_ctas =
      opt.max_prefill_ctas > 0 ? std::min(opt.max_prefill_ctas, num_sms) : num_sms;
  plan->max_prefill_ctas = prefill_ctas;
  plan->cu.assign(cu ? cu : nullptr, cu ? cu + Np + 1 : nullptr);
  plan->kv.assign(kv ? kv : nullptr, kv ? kv + Np + Nd : nullptr);
  const int64_t slots = (int64_t)num_sms * 2;  // a prefill slot and a decode slot per SM

  // ---- enumerate outputs (before splitting) and their costs --------------------------------
  struct PUnit { int s, t, h; int64_t kend; int64_t ntiles; };
  struct DUnit { int d, g; int64_t L; int64_t nblk; };
  std::vector<PUnit> pu;
  std::vector<DUnit> du;
  int64_t total = 0;
  double pf = 0, pb = 0, db = 0, df = 0;
  const double row_bytes = (double)(Hkv * kv_row_bytes(opt, D));
  const bool causal = opt.non_causal == 0;
  for (int s = 0; s < Np; ++s) {
    const int64_t q = (int64_t)cu[s + 1] - cu[s], L = kv[s], P = L - q;
    pf += 4.0 * D * Hq * (double)(causal ? q * P + q * (q + 1) / 2 : q * L);
    pb += (double)L * row_bytes + 4.0 * q * Hq * D;
    for (int64_t t = 0; t < ceil_div(q, (int64_t)tq); ++t) {
      // causal: the tile's last token sees up to its own position; otherwise every row
      const int64_t kend = causal ? P + std::min(q, (t + 1) * tq) : L;
      const int64_t nt = ceil_div(kend, kTileN);
      for (int h0 = 0; h0 < Hq; h0 += hp) {
        pu.push_back({s, (int)t, h0, kend, nt});
        total += nt * kPrefillStepCost;
      }
    }
  }
  for (int d = 0; d < Nd; ++d) {
    const int64_t L = kv[Np + d];
    db += (double)L * row_bytes + 4.0 * Hq * D;
    df += 4.0 * D * Hq * (double)L;
    for (int g = 0; g < Hkv; ++g) {
      du.push_back({d, g, L, ceil_div(L, kBlockSize)});
      total += ceil_div(L, kBlockSize) * kDecodeBlockCost;
    }
  }
  plan->est_prefill_flops = pf;
  plan->est_prefill_bytes = pb;
  plan->est_decode_bytes = db;
  plan->est_decode_flops = df;
  const int64_t target = std::max<int64_t>(1, total / (slots * 4));

  // ---- split and emit ----------------------------------------------------------------------
  // Items are written in enumeration order into flat arrays (cost, 8 words), then ordered
  // longest first; ties keep enumeration order (the sort key carries the item's index).
  struct Split { int64_t ns, chunk; };
  // prefill: one chunk size (steps per item) for all outputs, the one whose items the SMs'
  // prefill slots finish first in the model above; ties keep the larger chunk
  int64_t chunk_p = 0;
  if (!pu.empty() && opt.prefill_splits <= 0) {
    std::vector<int64_t> nts(pu.size()), hist, load;
    int64_t longest = 0;
    for (size_t i = 0; i < pu.size(); ++i) {
      nts[i] = pu[i].ntiles;
      longest = std::max(longest, pu[i].ntiles);
    }
    int64_t best = -1, prev_c = -1;
    for (int k = 1; k <= kMaxPrefillSplits; ++k) {
      const int64_t c = ceil_div(longest, k);
      if (c == prev_c) continue;
      if (k > 1 && c < kMinPrefillTilesPerSplit) break;
      prev_c = c;
      const int64_t t = prefill_makespan(nts, c, prefill_ctas, hist, load);
      if (best < 0 || t < best) {
        best = t;
        chunk_p = c;
      }
    }
  }
  auto split_p = [&](const PUnit& x) {
    int64_t ns;
    if (chunk_p > 0) {
      int64_t chunk;
      rebalanced(x.ntiles, chunk_p, &ns, &chunk);
      return Split{ns, chunk};
    }
    ns = std::max<int64_t>(1, std::min<int64_t>({opt.prefill_splits, x.ntiles,
                                                  (int64_t)kMaxPrefillSplits}));
    const int64_t chunk = ceil_div(x.ntiles, ns);
    return Split{ceil_div(x.ntiles, chunk), chunk};
  };
  // decode-only plans: one chunk size for all outputs, against the groups that run at once
  int64_t chunk_do = 0;
  const bool by_shares = opt.kv_fp4 && pu.empty() && !du.empty() && opt.decode_splits <= 0;
  if (pu.empty() && !du.empty() && opt.decode_splits <= 0 && !by_shares) {
    const int64_t groups = (int64_t)num_sms * (opt.kv_fp8 ? kDecodeGroupsFp8 : kDecodeGroupsBf16);
    std::vector<int64_t> nblks(du.size());
    int64_t longest = 0;
    for (size_t i = 0; i < du.size(); ++i) {
      nblks[i] = du[i].nblk;
      longest = std::max(longest, du[i].nblk);
    }
    std::vector<int64_t> hist((size_t)(ceil_div(longest, 4) + kDecodeItemOverhead + 1), 0);
    int64_t best = -1, prev_c = -1;
    for (int k : kChunkDivisors) {
      const int64_t c = ceil_div(longest, k);
      if (c == prev_c || (k > 1 && c < kMinDecodeBlocksPerSplit)) continue;
      prev_c = c;
      int64_t n_items = 0;
      for (int64_t n : nblks) {
        int64_t ns, ch;
        rebalanced(n, c, &ns, &ch);
        n_items += ns;
      }
      if (k > 1 && n_items > 4 * groups) break;  // past four waves the tail is already short
      const int64_t t = decode_makespan(nblks, c, groups, hist);
      if (best < 0 || t < best) {  // ties keep the larger chunk (fewer items, fewer merges)
        best = t;
        chunk_do = c;
      }
    }
  }
  auto split_d = [&](const DUnit& x) {
    int64_t ns;
    if (chunk_do > 0) {
      int64_t chunk;
      rebalanced(x.nblk, chunk_do, &ns, &chunk);
      return Split{ns, chunk};
    }
    if (opt.decode_splits > 0) {
      ns = std::min<int64_t>(opt.decode_splits, kMaxDecodeSplits);
    } else {
      ns = ceil_div(x.nblk * kDecodeBlockCost, target);
      ns = std::min<int64_t>(ns, std::max<int64_t>(1, x.nblk / kMinDecodeBlocksPerSplit));
      ns = std::min<int64_t>(ns, kMaxDecodeSplits);
    }
    ns = std::max<int64_t>(1, std::min(ns, x.nblk));
    const int64_t chunk = ceil_div(x.nblk, ns);
    return Split{ceil_div(x.nblk, chunk), chunk};
  };
  std::vector<Split> sp(pu.size()), sd(du.size());
  Shares cut;
  size_t n_p = 0, n_d = 0, n_units = 0;
  for (size_t i = 0; i < pu.size(); ++i) {
    sp[i] = split_p(pu[i]);
    n_p += (size_t)sp[i].ns;
    n_units += sp[i].ns > 1;
  }
  if (by_shares) {
    std::vector<int64_t> nblks(du.size());
    for (size_t i = 0; i < du.size(); ++i) nblks[i] = du[i].nblk;
    const int64_t round = fp4_round_blocks(D, kDecodeWarps), wide = fp4_round_blocks(D, kFp4Warps);
    cut = cut_shares(nblks, (int64_t)num_sms * (kFp4Warps / kDecodeWarps), round);
    if ((int64_t)nblks.size() <= num_sms) {
      Shares other = cut_shares(nblks, num_sms, wide);
      if (fp4_time(other, num_sms, wide, kFp4Warps, G * D / 2) <
          fp4_time(cut, num_sms, round, kDecodeWarps, G * D / 2)) {
        cut = std::move(other);
        plan->fp4_group_warps = kFp4Warps;
      }
    }
    const std::vector<Piece>& pieces = cut.pieces;
    n_d = pieces.size();
    for (size_t i = 0; i < n_d; ++i)
      n_units += pieces[i].first == 0 && pieces[i].end < nblks[pieces[i].out];
  } else {
    for (size_t i = 0; i < du.size(); ++i) {
      sd[i] = split_d(du[i]);
      n_d += (size_t)sd[i].ns;
      n_units += sd[i].ns > 1;
    }
  }
  std::vector<int64_t> cost_p(n_p), cost_d(n_d);
  std::vector<int32_t> words_p(n_p * kItemWords), words_d(n_d * kItemWords);
  plan->units.clear();
  plan->units.reserve(n_units * kUnitWords);
  int p_slots = 0, d_slots = 0;
  auto add_unit = [&](int nsplit, int kind) {
    int u = (int)(plan->units.size() / kUnitWords);
    int first = kind == 0 ? p_slots : d_slots;
    (kind == 0 ? p_slots : d_slots) += nsplit;
    plan->units.push_back(nsplit);
    plan->units.push_back(first);
    plan->units.push_back(kind);
    const int b = opt.kv_fp4 && kind == 1 ? fp4_bundle(nsplit, G * D / 2, plan->fp4_group_warps) : 0;
    plan->units.push_back(b);
    plan->fp4_levels |= b > 0;
    return u;
  };
  size_t ip = 0, id = 0;
  for (size_t i = 0; i < pu.size(); ++i) {
    const PUnit& x = pu[i];
    const int64_t ns = sp[i].ns, chunk = sp[i].chunk;
    const int u = ns > 1 ? add_unit((int)ns, 0) : -1;
    for (int64_t k = 0; k < ns; ++k, ++ip) {
      const int64_t t0 = k * chunk, t1 = std::min(x.ntiles, (k + 1) * chunk);
      cost_p[ip] = (t1 - t0) * kPrefillStepCost;
      const int32_t w[kItemWords] = {0, x.s, x.t, x.h, (int32_t)(t0 * kTileN),
                                     (int32_t)std::min(x.kend, t1 * kTileN), u, (int32_t)k};
      std::memcpy(&words_p[ip * kItemWords], w, sizeof(w));
    }
  }
  auto emit_d = [&](const DUnit& x, int64_t b0, int64_t b1, int u, int64_t k) {
    cost_d[id] = (b1 - b0) * kDecodeBlockCost;
    const int32_t w[kItemWords] = {1, x.d, x.g, 0, (int32_t)(b0 * kBlockSize),
                                   (int32_t)std::min(x.L, b1 * kBlockSize), u, (int32_t)k};
    std::memcpy(&words_d[id * kItemWords], w, sizeof(w));
    ++id;
  };
  if (by_shares) {
    for (size_t i = 0; i < n_d;) {
      size_t j = i;
      while (j < n_d && cut.pieces[j].out == cut.pieces[i].out) ++j;
      const int u = j - i > 1 ? add_unit((int)(j - i), 1) : -1;
      for (int64_t k = 0; i < j; ++i, ++k)
        emit_d(du[cut.pieces[i].out], cut.pieces[i].first, cut.pieces[i].end, u, k);
    }
  } else {
    for (size_t i = 0; i < du.size(); ++i) {
      const DUnit& x = du[i];
      const int64_t ns = sd[i].ns, chunk = sd[i].chunk;
      const int u = ns > 1 ? add_unit((int)ns, 1) : -1;
      for (int64_t k = 0; k < ns; ++k) emit_d(x, k * chunk, std::min(x.nblk, (k + 1) * chunk), u, k);
    }
  }
  // Items are taken longest first. Decode items: by cost, ties in enumeration order (a stable
  // counting sort over the cost in blocks). Prefill items: by cost rounded to a coarse relative
  // bucket (3 significant bits, ~12 % steps), then by split index, then in enumeration order, so
  // that the items running at once share their key ranges (split k of every output reads the
  // same part of its sequence) and keep the K/V rows they read resident in L2, while the order
  // stays longest first to within a bucket.
  auto order = [](const std::vector<int64_t>& key, const std::vector<int32_t>& words,
                  std::vector<int32_t>& out) {  // stable, largest key first
    const size_t n = key.size();
    int64_t top = 0;
    for (int64_t k : key) top = std::max(top, k);
    std::vector<size_t> start((size_t)top + 2, 0);
    for (int64_t k : key) ++start[(size_t)(top - k) + 1];
    for (size_t b = 1; b < start.size(); ++b) start[b] += start[b - 1];
    out.resize(n * kItemWords);
    for (size_t i = 0; i < n; ++i)
      std::memcpy(&out[(start[(size_t)(top - key[i])]++) * kItemWords], &words[i * kItemWords],
                  kItemWords * sizeof(int32_t));
  };
  auto bucket = [](int64_t steps) -> int64_t {  // monotone, 3 significant bits above 15
    if (steps < 16) return steps;
    int bl = 0;
    while ((steps >> bl) != 0) ++bl;
    return 16 + (int64_t)(bl - 5) * 8 + ((steps >> (bl - 4)) & 7);
  };
  for (size_t i = 0; i < n_p; ++i)
    cost_p[i] = bucket(cost_p[i] / kPrefillStepCost) * kMaxPrefillSplits +
                (kMaxPrefillSplits - 1 - words_p[i * kItemWords + 7]);
  for (size_t i = 0; i < n_d; ++i) cost_d[i] /= kDecodeBlockCost;
  order(cost_p, words_p, plan->items_p);
  if (by_shares) {
    // the shares' first items in the shares' order, then the others; word 3 leads from an item to the
    // next of its share
    const size_t n_sh = cut.starts.size() - 1;
    plan->items_d.resize(n_d * kItemWords);
    size_t more = n_sh;
    for (size_t s = 0; s < n_sh; ++s) {
      size_t at = s;
      for (int32_t i = cut.starts[s]; i < cut.starts[s + 1]; ++i) {
        int32_t* w = &plan->items_d[at * kItemWords];
        std::memcpy(w, &words_d[(size_t)i * kItemWords], kItemWords * sizeof(int32_t));
        if (i + 1 < cut.starts[s + 1]) w[3] = (int32_t)(at = more++);
      }
    }
    plan->num_shares = (int)n_sh;
  } else {
    order(cost_d, words_d, plan->items_d);
    plan->num_shares = (int)n_d;  // every item a share of its own
  }
  plan->num_p_slots = p_slots;
  // where each token of this iteration sits in its sequence (the KV append writes its K/V
  // row there): chunk token i of prefill sequence s at kv_len - q_len + i, a decode token at
  // kv_len - 1 ("Week 6: Beyond PyTorch: Custom Kernel과 vLLM", §"한 스텝에 여러 종류의 request
  // 섞기": an extend token follows the cached rows, a decode token is the last row)
  plan->new_rows.resize(2 * ((size_t)prob.num_prefill_tokens + Nd));
  size_t r = 0;
  for (int s = 0; s < Np; ++s) {
    const int32_t q = cu[s + 1] - cu[s], P = kv[s] - q;
    for (int32_t i = 0; i < q; ++i, r += 2) {
      plan->new_rows[r] = s;
      plan->new_rows[r + 1] = P + i;
    }
  }
  for (int d = 0; d < Nd; ++d, r += 2) {
    plan->new_rows[r] = Np + d;
    plan->new_rows[r + 1] = kv[Np + d] - 1;
  }
  plan->num_d_slots = d_slots;

  plan->grid_fused = (int)std::min<int64_t>(num_sms, (int64_t)(n_p + n_d));
  if (by_shares) plan->grid_fused = (int)std::min<int64_t>(num_sms, plan->num_shares);
  plan->grid_prefill = (int)std::min<int64_t>(prefill_ctas, (int64_t)n_p);
  plan->grid_decode = (int)std::min<int64_t>(num_sms, (int64_t)n_d);

  // ---- workspace layout --------------------------------------------------------------------
  WorkspaceLayout& w = plan->ws;
  size_t off = 0;
  w.status = off;
  off += 256;
  w.counters = off;
  w.counter_block_words = kCounterHeader + (size_t)num_sms;
  off = align256(off + kNumModes * w.counter_block_words * 4);
  w.arrive = off;
  off = align256(off + plan->units.size() / kUnitWords * (opt.kv_fp4 ? kFp4Counters : 1) * 4);
  w.zero_bytes = off;
  w.items_p = off;
  off = align256(off + plan->items_p.size() * 4);
  w.items_d = off;
  off = align256(off + plan->items_d.size() * 4);
  w.units = off;
  off = align256(off + plan->units.size() * 4);
  w.new_rows = off;
  off = align256(off + plan->new_rows.size() * 4);
  w.partial_p = off;
  off = align256(off + (size_t)p_slots * kPrefillSlotBytes);
  w.partial_d = off;
  off = align256(off + (size_t)d_slots * decode_slot_floats(G) * 4);
  w.records = off;
  if (opt.instrument) off = align256(off + (size_t)(n_p + n_d) * sizeof(pod_attn_item_record));
  w.total = off;

  // the upload image: zeros up to the work lists, then each list at its workspace offset
  std::vector<uint8_t>& img = plan->upload_image;
  img.assign(w.partial_p, 0);
  auto put = [&](size_t at, const std::vector<int32_t>& v) {
    if (!v.empty()) std::memcpy(img.data() + at, v.data(), v.size() * sizeof(int32_t));
  };
  put(w.items_p, plan->items_p);
  put(w.items_d, plan->items_d);
  put(w.units, plan->units);
  put(w.new_rows, plan->new_rows);
  return POD_ATTN_OK;
}

}  // namespace pod
