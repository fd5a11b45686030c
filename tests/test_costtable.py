"""The plan bucket of the C ABI (bit-exact against a plain restatement of its definition) and
the host logic of the validated-latency table (no GPU: plans are planned on the host only)."""
import json
import random

import pytest

from hybrid_prefill_decode_gb300 import binding as B
from hybrid_prefill_decode_gb300 import costtable as C


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _restated_bucket(Hq, Hkv, q_lens, pkv, dkv, causal=True):
    """prefill FLOPs = 4*128*Hq per visible (query, key) pair (all q*L pairs when non-causal);
    bytes = 512 per (row, kv-head) of every sequence plus 512 per (token, q-head); buckets = bit
    length of ceil(x / unit)."""
    flops = sum(4 * 128 * Hq * ((q * (L - q) + q * (q + 1) // 2) if causal else q * L)
                for q, L in zip(q_lens, pkv))
    by = sum(L * Hkv * 512 + q * Hq * 512 for q, L in zip(q_lens, pkv))
    by += sum(L * Hkv * 512 + Hq * 512 for L in dkv)

    def bucket(x, unit):
        return ((x + unit - 1) // unit).bit_length() if x > 0 else 0
    return flops, by, bucket(flops, 1 << 30), bucket(by, 1 << 20)


@pytest.mark.parametrize("seed", range(12))
def test_plan_bucket_matches_restatement(seed):
    rng = random.Random(seed)
    Hkv = rng.choice([1, 2, 4, 8])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    q_lens = [rng.randint(1, 3000) for _ in range(rng.randint(0, 3))]
    pkv = [q + rng.randint(0, 40000) for q in q_lens]
    dkv = [rng.randint(1, 40000) for _ in range(rng.randint(0, 80))]
    if not q_lens and not dkv:
        dkv = [5]
    causal = rng.random() < 0.7
    cu = [0]
    for q in q_lens:
        cu.append(cu[-1] + q)
    maxb = max(-(-x // 16) for x in pkv + dkv)
    p = B.Plan(Hq, Hkv, cu if q_lens else [], pkv + dkv, len(dkv), 10, maxb, 0.1, num_sms=152,
               non_causal=not causal)
    b = p.bucket()
    flops, by, bf, bb = _restated_bucket(Hq, Hkv, q_lens, pkv, dkv, causal)
    assert (b["prefill_flops"], b["read_bytes"], b["bucket_flops"], b["bucket_bytes"]) == \
        (flops, by, bf, bb)
    inf = p.info()
    assert b["prefill_ctas"] == inf["num_prefill_items"] and b["decode_ctas"] == inf["num_decode_items"]
    assert b["bucket_ctas"] == (b["prefill_ctas"] + b["decode_ctas"]).bit_length()
    assert b["grid"] == inf["grid_fused"] and b["smem_per_cta"] == inf["smem_bytes"]
    assert b["tmem_cols_per_cta"] == (512 if q_lens else 0)


@pytest.mark.parametrize("cache,hd,row", [({}, 128, 512), ({}, 64, 256), (dict(kv_fp8=True), 128, 260),
                                          (dict(kv_fp4=True), 128, 144), (dict(kv_fp4=True), 64, 72)])
def test_bytes_are_those_of_the_plan_s_cache(cache, hd, row):
    """Per row and kv-head: bf16 2 * 2 bytes a channel; e4m3 2 * 1 and the V row's fp32 scale; e2m1
    2 * 1/2 and 2 * 1/16 of e4m3 scales. q and o are bf16 in every plan."""
    lens, hq, hkv = [8192] * 63 + [5], 32, 8
    p = B.Plan(hq, hkv, [], lens, len(lens), 10, 512, 0.1, num_sms=152, head_dim=hd, **cache)
    want = sum(lens) * hkv * row + len(lens) * hq * 4 * hd
    b = p.bucket()
    assert b["read_bytes"] == want == p.info()["est_decode_bytes"]
    assert b["bucket_bytes"] == (-(-want // (1 << 20))).bit_length()


@pytest.mark.parametrize("hd", [64, 128])
@pytest.mark.parametrize("group,room", [(1, 1), (2, 2), (3, 4), (4, 4), (5, 8), (8, 8)])
def test_shared_memory_of_4_bit_plans_is_their_kernel_s(hd, group, room):
    """16 warps with two slots of 2 * blocks units of 9 * hd bytes each; per four warps a row of 132 floats
    for each warp and head that the kernel has room for, or the 8 * 16 + 8 floats of a merge if they are
    more, in 128-byte steps; then barriers and flags, less than 1 KiB."""
    p = B.Plan(2 * group, 2, [], [900], 1, 99, 60, 0.1, num_sms=8, head_dim=hd, kv_fp4=True)
    rings = 16 * 2 * 2 * {128: 2, 64: 4}[hd] * 9 * hd
    scratch = 4 * -(-4 * max(4 * room * 132, 136) // 128) * 128
    inf, b = p.info(), p.bucket()
    assert rings + scratch < inf["smem_bytes"] < rings + scratch + 1024
    assert b["smem_per_cta"] == inf["smem_bytes"] and inf["threads_per_cta"] == 512
    bf16 = B.Plan(2 * group, 2, [], [900], 1, 99, 60, 0.1, num_sms=8, head_dim=hd).info()
    assert inf["smem_bytes"] < bf16["smem_bytes"]


def _table_with(entries):
    t = C.CostTable(32, 8, 152)
    for (q_lens, pkv, dkv), times in entries:
        t.add(t.plan_for(q_lens, pkv, dkv).bucket(), times)
    return t


def test_choose_chunk_takes_the_largest_validated_chunk_within_budget():
    dec = [16384] * 19
    t = _table_with([(([256], [4096 + 256], dec), [300.0] * 10),
                     (([1024], [4096 + 1024], dec), [350.0] * 9 + [420.0]),
                     (([4096], [4096 + 4096], dec), [900.0] * 10)])
    assert t.choose_chunk(4096, [256, 1024, 4096], dec, budget_us=500) == 1024
    assert t.choose_chunk(4096, [256, 1024, 4096], dec, budget_us=410) == 256   # p99 is 420
    assert t.choose_chunk(4096, [256, 1024, 4096], dec, budget_us=100) is None
    assert t.choose_chunk(4096, [4096], dec, budget_us=1000) == 4096
    # a bucket never measured is outside the validated range
    assert t.lookup(t.plan_for([64], [200000], [3] * 500)) is None


def test_buckets_keep_their_worst_figures_and_round_trip_json():
    dec = [2048] * 4
    t = _table_with([(([512], [512 + 1000], dec), [10.0, 11.0, 12.0]),
                     (([512], [512 + 1001], dec), [20.0, 30.0, 40.0])])  # same bucket
    assert len(t.entries) == 1
    e = next(iter(t.entries.values()))
    assert (e.p50_us, e.p99_us, e.samples, e.batches) == (30.0, 40.0, 6, 2)
    t2 = C.CostTable.from_json(t.to_json())
    assert t2.entries == t.entries and (t2.num_q_heads, t2.num_kv_heads, t2.num_sms) == (32, 8, 152)
    json.loads(t.to_json())


def test_other_caches_have_entries_of_their_own():
    """The same batch over three caches: three kernels, three entries, wherever their buckets fall."""
    lens = [8192] * 64
    plans = {n: B.Plan(32, 8, [], lens, 64, 10, 512, 0.1, num_sms=152, **kw)
             for n, kw in (("bf16", {}), ("e4m3", dict(kv_fp8=True)), ("e2m1", dict(kv_fp4=True)))}
    assert [p.bucket()["kv_type"] for p in plans.values()] == \
        [B.KV_TYPES[n] for n in plans] == [0, 1, 2]
    t = C.CostTable(32, 8, 152)
    # a bf16 batch in the bucket of bytes that the 4-bit plan falls in
    small = B.Plan(32, 8, [], [2304] * 64, 64, 10, 512, 0.1, num_sms=152)
    assert small.bucket()["bucket_bytes"] == plans["e2m1"].bucket()["bucket_bytes"]
    for p in (plans["bf16"], small):
        t.add(p.bucket(), [400.0] * 3)
    assert t.lookup(plans["bf16"]).p99_us == 400.0
    assert t.lookup(plans["e4m3"]) is None and t.lookup(plans["e2m1"]) is None
    t.add(plans["e2m1"].bucket(), [90.0] * 3)
    t = C.CostTable.from_json(t.to_json())
    assert t.lookup(plans["e2m1"]).p99_us == 90.0 and t.lookup(small).p99_us == 400.0


def test_tables_without_cache_types_are_of_the_bf16_cache():
    p = B.Plan(32, 8, [], [8192] * 64, 64, 10, 512, 0.1, num_sms=152)
    b, e = p.bucket(), C.Entry(1.0, 2.0, 3, 1, 0, 4, 0.0)
    key = (b["bucket_flops"], b["bucket_bytes"])
    assert C.CostTable(32, 8, 152, {key: e}).lookup(p) == e
    d = json.loads(C.CostTable(32, 8, 152, {key: e}).to_json())
    del d["entries"][0]["kv_type"]
    assert C.CostTable.from_json(json.dumps(d)).lookup(p) == e
    del b["kv_type"]
    t = C.CostTable(32, 8, 152)
    t.add(b, [5.0])
    assert t.lookup(p).p50_us == 5.0
