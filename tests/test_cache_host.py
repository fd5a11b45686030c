"""Host side of the operators around the paged cache, through the C ABI without a GPU: refusals, the
rotary frequencies and the block bookkeeping against a plain model."""
import ctypes
import math
import random

import numpy as np
import pytest
import torch

from hybrid_prefill_decode_gb300 import binding as B
from oracle import cache_ops as C


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build()
    return B.load()


def _desc(kind="bf16", nb=10, k=16, v=32, ks=48, vs=64):
    # addresses that no host check reads through
    return B.KvCacheDesc(B.KV_TYPES[kind], nb, k, v, ks, vs)


def _plan(**kw):
    args = dict(num_q_heads=4, num_kv_heads=2, cu_seqlens=[0, 5], kv_lens=[9, 7],
                num_decode_seqs=1, num_blocks=10, max_blocks_per_seq=4, scale=0.1, num_sms=8)
    args.update(kw)
    return B.Plan(**args)


def _decode_plan(**kw):
    return _plan(cu_seqlens=[], kv_lens=[9], kv_fp4=True, **kw)


# ---------------------------------------------------------------------------------- refusals
def _rope_append(lib, plan=None, rope=None, q=1 << 20, qs=512, k=1 << 24, ks=256, v=1 << 25, vs=256,
                 cache=None, bt=16, qp=1 << 28, qd=1 << 29, ws=1 << 30, nbytes=1 << 30):
    plan = plan or _plan()
    cache = _desc() if cache is None else cache
    return lib.pod_attn_rope_append(plan.handle, rope and rope.handle, q, qs, k, ks, v, vs,
                                    ctypes.byref(cache) if cache else None, bt, qp, qd, ws, nbytes,
                                    None)


def test_rope_append_refusals(lib):
    bad = B.ERR_INVALID_ARG
    assert lib.pod_attn_rope_append(None, None, 16, 512, 16, 256, 16, 256, None, 16, 16, 16, 256, 0,
                                    None) == bad
    p = _plan()
    assert lib.pod_attn_rope_append(p.handle, None, 16, 512, 16, 256, 16, 256, None, 16, 16, 16,
                                    256, 1 << 30, None) == bad          # no cache
    for kw in (dict(k=None), dict(v=None), dict(bt=None), dict(qp=None), dict(qd=None),
               dict(ws=None), dict(q=(1 << 20) + 8), dict(k=(1 << 24) + 2), dict(qp=(1 << 28) + 4),
               dict(qs=504), dict(qs=516), dict(ks=248), dict(vs=260),
               dict(cache=_desc(nb=0)), dict(cache=_desc(k=None)), dict(cache=_desc(v=24)),
               dict(cache=_desc("e2m1", ks=None)), dict(cache=_desc("e4m3", vs=None)),
               dict(cache=B.KvCacheDesc(7, 10, 16, 32, 48, 64))):
        assert _rope_append(lib, p, **kw) == bad, kw
    assert _rope_append(lib, p, ws=(1 << 30) + 16) == B.ERR_WORKSPACE
    assert _rope_append(lib, p, nbytes=16) == B.ERR_WORKSPACE
    p64 = _plan(head_dim=64)
    assert _rope_append(lib, p64, cache=_desc("e4m3")) == B.ERR_UNSUPPORTED
    assert _rope_append(lib, p64, rope=B.Rope(66)) == bad


def test_rope_append_refuses_overlapping_outputs(lib):
    q = 1 << 20
    p = _plan()                                            # 5 chunk tokens, 1 decode, 4 x 128
    row = 4 * 128 * 2
    bad = B.ERR_INVALID_ARG
    assert _rope_append(lib, p, q=q, qp=q + row, qd=q + 6 * row) == bad      # shifted by a row
    assert _rope_append(lib, p, q=q, qp=q, qd=q + 6 * row) == bad            # only half in place
    assert _rope_append(lib, p, q=q, qs=1024, qp=q, qd=q + 5 * row) == bad   # strided in place
    assert _rope_append(lib, p, k=1 << 24, qp=(1 << 24) + 16) == bad
    assert _rope_append(lib, p, v=1 << 25, qd=(1 << 25) + 16) == bad
    assert _rope_append(lib, p, qp=1 << 28, qd=(1 << 28) + 4 * row) == bad   # onto one another


def test_nothing_to_do_is_ok(lib):
    p = _plan(cu_seqlens=[], kv_lens=[], num_decode_seqs=0)
    assert _rope_append(lib, p, k=None, v=None, q=None) == B.OK
    c = _desc("e2m1")
    assert lib.pod_attn_expand_fp4(p.handle, ctypes.byref(c), None, None, None, None, None, 1 << 30,
                                   1 << 30, None) == B.OK
    p = _plan(cu_seqlens=[], kv_lens=[], num_decode_seqs=0, kv_fp4=True)
    assert lib.pod_attn_run_decode_fp4(p.handle, None, None, None, None, None, 1 << 30, 1 << 30,
                                       None) == B.OK
    assert lib.pod_attn_copy_blocks(None, 0, 10, None, 0, None) == B.OK


def test_decode_fp4_refusals(lib):
    def run(p, c=_desc("e2m1"), q=16, bt=16, kv=16, o=16, ws=1 << 30, n=1 << 30):
        return lib.pod_attn_run_decode_fp4(p.handle, q, ctypes.byref(c) if c else None, bt, kv, o,
                                           ws, n, None)
    p = _decode_plan()
    bad = B.ERR_INVALID_ARG
    assert lib.pod_attn_run_decode_fp4(None, 16, None, 16, 16, 16, 256, 256, None) == bad
    for kw in (dict(c=None), dict(q=None), dict(bt=None), dict(kv=None), dict(o=None),
               dict(ws=None), dict(q=8), dict(o=20), dict(c=_desc("e2m1", nb=9)),
               dict(c=_desc("e2m1", k=None)), dict(c=_desc("e2m1", vs=None)),
               dict(c=_desc("e2m1", k=24))):
        assert run(p, **kw) == bad, kw
    assert run(p, ws=128) == B.ERR_WORKSPACE
    assert run(p, n=16) == B.ERR_WORKSPACE
    assert run(p, c=_desc("e4m3")) == B.ERR_UNSUPPORTED
    assert run(p, c=_desc("bf16")) == B.ERR_UNSUPPORTED
    assert run(_plan(kv_fp4=True)) == B.ERR_UNSUPPORTED               # prefill sequences
    assert run(_plan(cu_seqlens=[], kv_lens=[9])) == B.ERR_UNSUPPORTED   # a bf16 plan
    assert run(_plan(cu_seqlens=[], kv_lens=[9], kv_fp8=True)) == B.ERR_UNSUPPORTED


def test_plans_of_the_4_bit_cache_are_refused_elsewhere(lib):
    p = _decode_plan()
    assert lib.pod_attn_run(p.handle, None, 16, 16, 16, 16, None, 16, None, 16, 1 << 30, 1 << 30,
                            None, None) == B.ERR_UNSUPPORTED
    assert lib.pod_attn_run_append(p.handle, None, 16, 16, 16, 16, 16, 16, None, 16, None, 16,
                                   1 << 30, 1 << 30, None, None) == B.ERR_UNSUPPORTED
    assert lib.pod_attn_run_decode_fp8(p.handle, 16, 16, 16, 16, 16, 16, 16, 16, 1 << 30, 1 << 30,
                                       None) == B.ERR_UNSUPPORTED
    assert lib.pod_attn_append_fp8(p.handle, 16, 16, 16, 16, 16, 16, 16, 1 << 30, 1 << 30,
                                   None) == B.ERR_UNSUPPORTED
    f = lib.pod_attn_run_static
    f.restype, f.argtypes = ctypes.c_int32, [ctypes.c_void_p] * 11
    assert f(p.handle, *[None] * 10) == B.ERR_UNSUPPORTED
    with pytest.raises(B.PodAttnError) as e:
        _plan(cu_seqlens=[], kv_lens=[9], kv_fp8=True, kv_fp4=True)
    assert e.value.code == B.ERR_INVALID_ARG


def test_expand_refusals(lib):
    def run(p, c=_desc("e2m1"), b4=16, k=16, v=16, bt=16, kv=16, ws=1 << 30, n=1 << 30):
        return lib.pod_attn_expand_fp4(p.handle, ctypes.byref(c) if c else None, b4, k, v, bt, kv,
                                       ws, n, None)
    p = _plan()
    bad = B.ERR_INVALID_ARG
    for kw in (dict(c=None), dict(b4=None), dict(k=None), dict(v=None), dict(bt=None),
               dict(kv=None), dict(ws=None), dict(k=8), dict(c=_desc("e2m1", nb=0)),
               dict(c=_desc("e2m1", ks=None)), dict(c=_desc("e2m1", v=40))):
        assert run(p, **kw) == bad, kw
    assert run(p, ws=128) == B.ERR_WORKSPACE
    assert run(p, c=_desc("bf16")) == B.ERR_UNSUPPORTED
    assert run(_decode_plan()) == B.ERR_UNSUPPORTED
    assert run(_plan(cu_seqlens=[], kv_lens=[9], kv_fp8=True)) == B.ERR_UNSUPPORTED


def test_scales_that_are_not_aligned_are_refused(lib):
    """A float's alignment for the 4-bit cache's scales (4 bytes), 16 bytes for the e4m3 cache's."""
    bad = B.ERR_INVALID_ARG
    for kw in (dict(ks=50), dict(vs=66)):
        c = _desc("e2m1", **kw)
        assert _rope_append(lib, cache=c) == bad
        assert lib.pod_attn_run_decode_fp4(_decode_plan().handle, 16, ctypes.byref(c), 16, 16, 16,
                                           1 << 30, 1 << 30, None) == bad
        assert lib.pod_attn_expand_fp4(_plan().handle, ctypes.byref(c), 16, 16, 16, 16, 16, 1 << 30,
                                       1 << 30, None) == bad
    for kw in (dict(ks=52), dict(vs=68)):
        assert _rope_append(lib, cache=_desc("e4m3", **kw)) == bad


@pytest.mark.parametrize("pairs,ok", [
    ([(0, 9)], True), ([(0, 9), (0, 8)], True), ([(3, 3)], True), ([(3, 3), (3, 4)], True),
    ([(3, 3), (3, 3)], True), ([(0, 10)], False), ([(-1, 2)], False), ([(10, 2)], False),
    ([(0, -1)], False), ([(0, 5), (1, 5)], False), ([(0, 5), (5, 6)], False),
    ([(5, 6), (0, 5)], False), ([(1, 2), (2, 1)], False), ([(3, 3), (1, 3)], True)])
def test_copy_blocks_checks_its_pairs(lib, pairs, ok):
    """A block written twice, or both written and read, is refused; nothing is launched here (a
    pool count of 0 ends the call after the checks)."""
    a = (ctypes.c_int32 * (2 * len(pairs)))(*[x for p in pairs for x in p])
    code = lib.pod_attn_copy_blocks(None, 0, 10, ctypes.cast(a, ctypes.c_void_p), len(pairs), None)
    assert code == (B.OK if ok else B.ERR_INVALID_ARG)


def test_copy_blocks_checks_its_pools(lib):
    pair = (ctypes.c_int32 * 2)(0, 1)
    ptr = ctypes.cast(pair, ctypes.c_void_p)
    for base, size in ((None, 16), (8, 16), (16, 0), (16, 24), (16, 1 << 32)):
        pool = (B.BlockPool * 1)(B.BlockPool(base, size))
        assert lib.pod_attn_copy_blocks(pool, 1, 4, ptr, 1, None) == B.ERR_INVALID_ARG
    pool = (B.BlockPool * 1)(B.BlockPool(16, 16))
    assert lib.pod_attn_copy_blocks(pool, -1, 4, ptr, 1, None) == B.ERR_INVALID_ARG
    assert lib.pod_attn_copy_blocks(pool, 1, 4, ptr, -1, None) == B.ERR_INVALID_ARG
    assert lib.pod_attn_copy_blocks(pool, 1, 4, None, 1, None) == B.ERR_INVALID_ARG
    assert lib.pod_attn_copy_blocks(None, 1, 4, ptr, 1, None) == B.ERR_INVALID_ARG
    assert lib.pod_attn_copy_blocks(pool, 1, -4, ptr, 1, None) == B.ERR_INVALID_ARG


# ---------------------------------------------------------------------------------- shares
def _restated_shares(nblks, groups, rnd):
    """The plan of the 4-bit cache: (output, first, end) of every piece, share by share."""
    total, longest, outs, item = sum(nblks), max(nblks), len(nblks), rnd * 3 // 2
    up = lambda x: -(-x // rnd) * rnd
    least = lambda splits: up(max(2 * rnd, -(-longest // splits)))
    whole = total + outs * item
    n = max(1, min(groups, whole // (least(255) + item)))
    apart = None
    if outs <= groups:
        apart = least(256)
        while sum(-(-n // apart) for n in nblks) > groups:
            apart += rnd
    if apart and min(apart, longest) <= whole // n + item:
        shares = []
        for o, n in enumerate(nblks):
            k = -(-n // apart)
            rest = n - (k - 1) * apart
            if k > 1 and rest < (2 * item if k == 2 else item):
                k -= 1
            size = up(-(-n // k))
            shares += [[(o, at, min(n, at + size))] for at in range(0, n, size)]
        return shares
    shares, o, at, done = [], 0, 0, 0
    for i in range(n):
        end, last = (i + 1) * whole // n, i == n - 1
        if o == outs or (end <= done and not last):
            continue
        share = []
        while o < outs and (done < end or not share):
            cost, take = 0 if at else item, nblks[o] - at
            if not last and end - done < cost + take:
                cut = int((end - done - cost) / rnd) * rnd            # towards zero, as in C++
                if take - cut < item:
                    pass
                elif cut >= item:
                    take = cut
                elif share:
                    break
                else:
                    take = min(take, up(item))
            share.append((o, at, at + take))
            at, done = at + take, done + cost + take
            if at == nblks[o]:
                o, at = o + 1, 0
        shares.append(share)
    return shares


def _bundle(n, pairs, warps):
    return 0 if n <= (32 if pairs <= 32 * warps else 16) else math.isqrt(n - 1) + 1


def _restated_groups(nblks, sms, dim, pairs):
    """(shares, warps of a group): groups of four warps, or of 16 if they take less time."""
    best = None
    for warps in (4, 16) if len(nblks) <= sms else (4,):
        rnd = warps * (2 if dim == 128 else 4)
        shares = _restated_shares(nblks, 16 // warps * sms, rnd)
        a, r = (38, 38) if warps == 16 else (45, max(13, 9 * min(4, -(-len(shares) // sms))))
        time = max(sum(a + r * -(-(e - b) // rnd) for _, b, e in s) for s in shares)
        pieces = [o for s in shares for o, _, _ in s]
        most = max(pieces.count(o) for o in set(pieces))
        if most > 1:
            time += 54 if warps == 16 else (10 + (54 if pairs > 128 else 0) +
                                            (68 if _bundle(most, pairs, 4) else 0))
        if best is None or time < best[0]:
            best = time, shares, warps
    return best[1:]


@pytest.mark.parametrize("seed", range(120))
def test_plan_by_shares(lib, seed):
    """Every block of every output once and in order, at most 256 pieces of an output, the shares as
    the restated rule cuts them."""
    rng = random.Random(seed)
    hkv, sms = rng.choice([1, 2, 5, 8]), rng.choice([1, 3, 33, 152])
    most = rng.choice([1, 60, 5000, 200000])
    lens = [rng.choice([1, rng.randint(1, 60), rng.randint(1, most), most])
            for _ in range(rng.choice([1, 2, 9, 70]))]
    dim = rng.choice([64, 128])
    if seed == 0:
        lens, hkv, sms = [1 << 20], 1, 152
    if seed == 1:
        lens, hkv, sms = [1] * 8, 8, 152         # short outputs on an idle GPU: a share each
    maxb = -(-max(lens) // 16)
    group = 2 if seed < 60 else rng.choice([1, 2, 4, 8])
    p = B.Plan(group * hkv, hkv, [], lens, len(lens), 10, maxb, .1, num_sms=sms, kv_fp4=True,
               head_dim=dim)
    _, items, units = p.items()
    nblks = [-(-L // 16) for L in lens for _ in range(hkv)]
    shares, warps = _restated_groups(nblks, sms, dim, group * dim // 2)
    assert len(shares) <= 4 * sms and (seed != 1 or len(shares) == 64)
    # items: the shares' first pieces in order, the others behind them, linked by word 3
    got, linked = [], []
    for s in range(len(shares)):
        i, share = s, []
        while True:
            linked.append(i)
            share.append((items[i][1] * hkv + items[i][2], items[i][4] // 16, -(-items[i][5] // 16)))
            i = items[i][3]
            if i == 0:
                break
        got.append(share)
    assert got == shares and sorted(linked) == list(range(len(items)))
    items = [items[i] for i in linked]
    got = [x for s in got for x in s]
    assert all(i[5] == min(e * 16, lens[i[1]]) for i, (_, _, e) in zip(items, got))
    pieces = {}
    for o, first, end in got:
        assert end > first == (pieces[o][-1][1] if o in pieces else 0)
        pieces.setdefault(o, []).append((first, end))
    assert [pieces[o][-1][1] for o in range(len(nblks))] == nblks
    assert max(len(x) for x in pieces.values()) <= 256
    slot = 0
    for o, x in pieces.items():
        own = [i for i, g in zip(items, got) if g[0] == o]
        assert [i[7] for i in own] == list(range(len(x)))
        if len(x) == 1:
            assert own[0][6] == -1
        else:
            assert len({i[6] for i in own}) == 1
            bundle = _bundle(len(x), group * dim // 2, warps)
            assert units[own[0][6]] == [len(x), slot, 1, bundle]
            slot += len(x)
    assert p.info()["grid_fused"] == min(sms, len(shares))


def test_forced_splits_of_the_4_bit_plan_are_as_for_other_caches(lib):
    a, b = (B.Plan(4, 2, [], [900, 33], 2, 99, 60, .1, num_sms=8, decode_splits=5, **kw).items()
            for kw in (dict(kv_fp4=True), dict(kv_fp8=True)))
    assert a == b


# ---------------------------------------------------------------------------------- rotary
@pytest.mark.parametrize("kw", [
    dict(), dict(theta=500000.0), dict(scaling="linear", factor=4.0),
    dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=16.0, original_max_position=4096),
    dict(scaling="yarn", factor=40.0, original_max_position=4096, beta_fast=16.0, beta_slow=2.0),
    dict(scaling="llama3", factor=8.0, original_max_position=8192)])
@pytest.mark.parametrize("rot", [4, 20, 64, 128])
def test_rope_frequencies(lib, rot, kw):
    """Relative to the frequency: a power, a quotient and two products in 64 bits, each off by a few
    2^-53, and the exponent's error times ln theta < 14."""
    freq, mag = B.Rope(rot, **kw).frequencies()
    want, want_mag = C.rope_frequencies(rot, **kw)
    np.testing.assert_allclose(freq, want, rtol=64 * 2.0 ** -53, atol=0)
    assert mag == pytest.approx(want_mag, rel=2.0 ** -23)


def test_rope_custom_and_attention_factor(lib):
    freq = [0.5, -0.25, 7.0, 0.0]
    got, mag = B.Rope(8, scaling="custom", inv_freq=freq, attention_factor=1.5).frequencies()
    assert got == freq and mag == 1.5


@pytest.mark.parametrize("kw", [
    dict(rot_dim=0), dict(rot_dim=3), dict(rot_dim=130), dict(rot_dim=-2), dict(theta=1.0),
    dict(theta=float("nan")), dict(scaling="linear", factor=0.0),
    dict(scaling="linear", factor=float("inf")), dict(rot_dim=2, scaling="ntk", factor=2.0),
    dict(scaling="yarn", factor=2.0), dict(scaling="llama3", factor=2.0),
    dict(scaling="llama3", factor=2.0, original_max_position=8192, low_freq_factor=4.0),
    dict(scaling="custom"), dict(attention_factor=-1.0), dict(attention_factor=float("nan")),
    dict(scaling="yarn", factor=2.0, original_max_position=4096, beta_fast=0.0)])
def test_rope_refusals(lib, kw):
    with pytest.raises(B.PodAttnError) as e:
        B.Rope(**{**dict(rot_dim=8), **kw})
    assert e.value.code == B.ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(), dict(scaling="linear", factor=4.0), dict(scaling="yarn", factor=2.0, original_max_position=64)])
def test_rope_refuses_frequencies_that_it_would_not_use(lib, kw):
    with pytest.raises(ValueError):
        B.Rope(8, inv_freq=[.5, .25, .125, .1], **kw)


def test_rope_custom_refuses_values_that_are_not_finite(lib):
    with pytest.raises(B.PodAttnError):
        B.Rope(4, scaling="custom", inv_freq=[1.0, float("inf")])
    assert lib.pod_attn_rope_create(None, None) == B.ERR_INVALID_ARG
    assert lib.pod_attn_rope_frequencies(None, None, None) == B.ERR_INVALID_ARG
    lib.pod_attn_rope_destroy(None)


# ---------------------------------------------------------------------------------- pages
class Model:
    """Sequences as lists of (row values); blocks are shared by content through copies."""

    def __init__(self, seqs):
        self.rows = [[] for _ in range(seqs)]


@pytest.mark.parametrize("seed", range(12))
def test_pages_against_a_model(lib, seed):
    """Random grows, forks, frees and compactions. A host array stands for the pool: rows are
    written where the tables say after the pairs have been copied, and every sequence must read
    back its own rows after each step; reference counts never leak blocks."""
    rng = random.Random(seed)
    nb, seqs, maxb = rng.choice([(40, 6, 12), (17, 4, 30), (200, 20, 9)])
    pages, model = B.Pages(nb, seqs, maxb), Model(seqs)
    pool = np.full((nb, 16), -1, dtype=np.int64)
    stamp = 0

    def copy(pairs):
        pairs = [tuple(int(x) for x in p) for p in pairs]
        assert len({d for _, d in pairs}) == len(pairs)
        assert not {s for s, _ in pairs} & {d for _, d in pairs}
        for s, d in pairs:
            pool[d] = pool[s]

    for _ in range(300):
        s = rng.randrange(seqs)
        op = rng.choice(["grow", "grow", "grow", "fork", "free", "compact"])
        if op == "grow":
            old = len(model.rows[s])
            new = old + rng.choice([0, 1, 1, 3, 16, 40])
            free = pages.free_blocks
            before = pages.tables(range(seqs))
            try:
                copy(pages.grow(s, new))
            except B.PodAttnError as e:
                after = pages.tables(range(seqs))
                assert pages.free_blocks == free
                assert torch.equal(before[0], after[0]) and torch.equal(before[1], after[1])
                if e.code == B.ERR_INVALID_ARG:
                    assert new > maxb * 16
                else:
                    assert e.code == B.ERR_NO_BLOCKS
                    assert -(-new // 16) - -(-old // 16) + 1 > free
                continue
            bt, lens = pages.tables([s])
            assert int(lens[0]) == new
            for p in range(old, new):
                stamp += 1
                pool[bt[0, p // 16], p % 16] = stamp
                model.rows[s].append(stamp)
        elif op == "fork":
            to = rng.randrange(seqs)
            n = rng.randint(0, len(model.rows[s]))
            if to == s or model.rows[to]:
                with pytest.raises(B.PodAttnError):
                    pages.fork(s, to, n)
            else:
                pages.fork(s, to, n)
                model.rows[to] = model.rows[s][:n]
        elif op == "free":
            pages.free(s)
            model.rows[s] = []
        else:
            copy(pages.compact())
            used = nb - pages.free_blocks
            bt, lens = pages.tables(range(seqs))
            for i in range(seqs):
                assert all(b < used for b in bt[i, :-(-int(lens[i]) // 16)].tolist())
            assert len(pages.compact()) == 0
        bt, lens = pages.tables(range(seqs))
        live = set()
        for i, want in enumerate(model.rows):
            assert int(lens[i]) == len(want)
            n = -(-len(want) // 16)
            live |= set(bt[i, :n].tolist())
            assert (bt[i, n:] == 0).all()
            assert [int(pool[bt[i, p // 16], p % 16]) for p in range(len(want))] == want
        assert pages.free_blocks == nb - len(live)
    for i in range(seqs):
        pages.free(i)
    assert pages.free_blocks == nb


def test_pages_copy_on_write_only_of_a_shared_partial_block(lib):
    p = B.Pages(10, 3, 5)
    assert p.grow(0, 20) == []
    p.fork(0, 1, 20)
    assert p.free_blocks == 8
    assert p.grow(1, 20) == []                       # nothing written, nothing copied
    assert p.grow(1, 21) == [(1, 2)]                 # the block of rows 16-19
    assert p.grow(0, 21) == []                       # its block is its own again
    p.fork(0, 2, 16)
    assert p.grow(2, 17) == []                       # whole blocks stay shared
    assert p.tables([0, 1, 2])[0][:, :2].tolist() == [[0, 1], [0, 2], [0, 3]]
    q = B.Pages(2, 2, 5)
    q.grow(0, 20)
    q.fork(0, 1, 20)
    with pytest.raises(B.PodAttnError) as e:
        q.grow(1, 21)                                # no block left to copy into
    assert e.value.code == B.ERR_NO_BLOCKS


def test_pages_refusals(lib):
    h = ctypes.c_void_p()
    for args in ((0, 1, 1), (1, 0, 1), (1, 1, 0), (1, 1, 1 << 28)):
        assert lib.pod_attn_pages_create(*args, ctypes.byref(h)) == B.ERR_INVALID_ARG
        assert h.value is None
    assert lib.pod_attn_pages_create(1, 1, 1, None) == B.ERR_INVALID_ARG
    p = B.Pages(10, 2, 4)
    for f in (lambda: p.grow(2, 1), lambda: p.grow(-1, 1), lambda: p.grow(0, 65),
              lambda: p.fork(0, 0, 0), lambda: p.fork(0, 1, 1), lambda: p.fork(0, 2, 0),
              lambda: p.free(2), lambda: p.tables([2])):
        with pytest.raises(B.PodAttnError) as e:
            f()
        assert e.value.code == B.ERR_INVALID_ARG
    p.grow(0, 20)
    with pytest.raises(B.PodAttnError):
        p.grow(0, 19)
    pair, n = (ctypes.c_int32 * 2)(), ctypes.c_int32()
    ptr = ctypes.cast(pair, ctypes.c_void_p)
    assert lib.pod_attn_pages_grow(None, 0, 1, ptr, ctypes.byref(n)) == B.ERR_INVALID_ARG
    assert lib.pod_attn_pages_grow(p.handle, 0, 30, None, ctypes.byref(n)) == B.ERR_INVALID_ARG
    assert lib.pod_attn_pages_compact(p.handle, None, 0, None) == B.ERR_INVALID_ARG
    p.grow(1, 33)
    p.free(0)                                        # blocks 2, 3, 4 stay: three moves, two holes
    assert lib.pod_attn_pages_compact(p.handle, None, 0, ctypes.byref(n)) == B.OK
    moves = n.value
    before = p.tables([1])[0]
    assert moves == 2
    assert lib.pod_attn_pages_compact(p.handle, ptr, 1, ctypes.byref(n)) == B.ERR_INVALID_ARG
    assert torch.equal(before, p.tables([1])[0])
    assert lib.pod_attn_pages_free_blocks(None) == -1
    lib.pod_attn_pages_destroy(None)


@pytest.mark.parametrize("kw", [dict(kv_lens=[9]), dict(kv_lens=[]), dict(num_decode_seqs=2),
                                dict(cu_seqlens=[0, 2, 5])])
def test_plans_of_more_sequences_than_lengths_are_refused(lib, kw):
    with pytest.raises(ValueError):
        _plan(**kw)


@pytest.mark.parametrize("off", [1 << 32, -(1 << 32), 1 << 40])
def test_numbers_beyond_32_bits_are_refused(lib, off):
    """Not taken modulo 2^32."""
    p = B.Pages(10, 3, 5)
    p.grow(0, 20)
    for f in (lambda: B.Pages(10 + off, 3, 5), lambda: B.Pages(10, 3 + off, 5),
              lambda: B.Pages(10, 3, 5 + off), lambda: p.grow(0 + off, 21), lambda: p.grow(0, 21 + off),
              lambda: p.fork(off, 1, 20), lambda: p.fork(0, 1 + off, 20), lambda: p.fork(0, 1, 20 + off),
              lambda: p.free(off), lambda: p.tables([off]), lambda: B.Rope(64 + off),
              lambda: _decode_plan(num_blocks=10 + off), lambda: _plan(kv_lens=[9, 7 + off]),
              lambda: _plan(num_q_heads=4 + off), lambda: _plan(cu_seqlens=[0, 5 + off])):
        with pytest.raises(ValueError):
            f()
    assert p.free_blocks == 8 and p.tables([0, 1])[1].tolist() == [20, 0]


# ---------------------------------------------------------------------------------- the oracle
def test_oracle_formats():
    """The oracle's own tables: the values of both formats and rounding to them."""
    assert C.E4M3[-1] == 448 and len(C.E4M3) == 127 and C.E4M3[1] == 2.0 ** -9
    t = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(C.E4M3, t)
    x = np.array([0, .25, .75, 1.25, 1.75, 2.5, 3.5, 5.0, 5.01, 100, .26, .74])
    assert C.E2M1[C.nearest(x, C.E2M1)].tolist() == [0, 0, 1, 1, 2, 2, 4, 4, 6, 6, .5, .5]
    r = np.random.default_rng(3).uniform(0, 448, 4096).astype(np.float32)
    want = torch.from_numpy(r).to(torch.float8_e4m3fn).float().numpy()
    assert np.array_equal(C.E4M3[C.nearest(r, C.E4M3)], want)


def test_oracle_pool_layout_round_trip():
    rng = np.random.default_rng(5)
    x = rng.standard_normal((3, 2, 64)).astype(np.float32)
    h = np.array([1.0, 0.5], dtype=np.float32)
    code, s8 = C.quantise_fp4(x, h)
    for is_v in (False, True):
        pool = np.zeros(B.fp4_pool_shape(4, 2, 64), dtype=np.uint8)
        C.put_rows(pool, 64, is_v, [3, 0, 3], [5, 15, 0], code, s8)
        val = C.pool_values(pool, 64, h, is_v)
        sign = np.where(code & 8, -1, 1)
        want = sign * C.E2M1[code & 7] * np.repeat(C.E4M3[s8], 16, -1) * h[:, None]
        assert np.array_equal(val[[3, 0, 3], :, [5, 15, 0]], want)
        # the largest of a group is 6 (or rounds to 4) of its scale: within a quarter of it
        assert (np.abs(val[[3, 0, 3], :, [5, 15, 0]] - x) <= np.abs(x).max() / 4).all()
    assert math.isnan(C.e4m3_values(np.uint8(0x7F)))
