"""Rotary positions with the append, on the GPU through the C ABI, against NumPy in 64 bits."""
import numpy as np
import pytest
import torch

import cache_cases as K
import oracle
from hybrid_prefill_decode_gb300 import binding as B
from oracle import cache_ops as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


SCALINGS = [dict(), dict(scaling="linear", factor=4.0), dict(scaling="ntk", factor=8.0),
            dict(scaling="yarn", factor=16.0, original_max_position=4096),
            dict(scaling="llama3", factor=8.0, original_max_position=8192)]


class Case:
    """New tokens of chunks and decodes, as views of one fused projection, and a cache."""

    def __init__(self, hq, hkv, D, q_lens, pkv, dkv, seed, kind="bf16", pad=0):
        rng = np.random.default_rng(seed)
        self.hq, self.hkv, self.D, self.kind = hq, hkv, D, kind
        self.lens, self.tp, self.nd = pkv + dkv, sum(q_lens), len(dkv)
        self.cu = [sum(q_lens[:i]) for i in range(len(q_lens) + 1)] if q_lens else []
        self.pos = np.array([p for n, L in zip(q_lens, pkv) for p in range(L - n, L)] +
                            [L - 1 for L in dkv], dtype=np.int64)
        seq = [s for s, n in enumerate(q_lens) for _ in range(n)] + \
            [len(q_lens) + i for i in range(len(dkv))]
        # blocks of the new rows only: the others are never touched
        maxb = max(-(-L // 16) for L in self.lens)
        self.bt = np.full((len(self.lens), maxb), -1, dtype=np.int32)
        used = sorted({(s, p // 16) for s, p in zip(seq, self.pos)})
        self.nb = len(used) + 2
        for (s, j), b in zip(used, rng.permutation(self.nb)):
            self.bt[s, j] = b
        self.blk = np.array([self.bt[s, p // 16] for s, p in zip(seq, self.pos)])
        self.row = self.pos % 16
        t = len(self.pos)
        self.qkv = K.bf16(rng.standard_normal((t, hq + 2 * hkv + pad, D))).cuda()
        self.q, self.k = self.qkv[:, :hq], self.qkv[:, hq:hq + hkv]
        self.v = self.qkv[:, hq + hkv:hq + 2 * hkv]
        dev = torch.Generator(device="cuda").manual_seed(seed)
        if kind == "e2m1":
            pools = [torch.randint(0, 256, B.fp4_pool_shape(self.nb, hkv, D), generator=dev,
                                   device="cuda", dtype=torch.uint8) for _ in range(2)]
            scales = [torch.from_numpy(rng.uniform(.1, 2, hkv).astype(np.float32)).cuda()
                      for _ in range(2)]
        else:
            pools = [torch.randn((self.nb, hkv, 16, D), generator=dev, device="cuda",
                                 dtype=torch.bfloat16) for _ in range(2)]
            scales = [None, None]
            if kind == "e4m3":
                pools = [p.to(torch.float8_e4m3fn) for p in pools]
                scales = [torch.from_numpy(rng.uniform(.003, .02, (hkv, D)).astype(np.float32)).cuda(),
                          torch.rand((self.nb, hkv, 16), generator=dev, device="cuda")]
        self.pools, self.scales = pools, scales
        self.cache = B.KvCache(kind, *pools, *scales)
        self.tab = torch.from_numpy(self.bt).cuda()
        self.plan = B.Plan(hq, hkv, self.cu, self.lens, self.nd, max(1, self.nb), maxb, .1,
                           head_dim=D)
        self.ws = self.plan.alloc_workspace()
        self.plan.upload(self.ws)
        self.q_p = torch.full((self.tp, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.q_d = torch.full((self.nd, hq, D), float("nan"), dtype=torch.bfloat16, device="cuda")

    def run(self, rope, q="own", stream=None):
        q = self.q if isinstance(q, str) else q
        self.plan.rope_append(rope, q, self.k, self.v, self.cache, self.tab, self.q_p, self.q_d,
                              self.ws, stream=stream)
        return self.plan.device_status(self.ws)

    def q_out(self):
        return torch.cat((self.q_p, self.q_d))


def _check_rotated(got, x, pos, rot, interleaved, kw, what=""):
    """Angles are exact to 2^-32 turns, then rounded to 24 bits of at most a half turn (2^-23 radians)
    and their sin and cos are good to 2^-22; the two products, their sum and the attention factor add
    2^-22 of |x| + |y|. The result is rounded to bf16, 2^-8 of it; channels behind the rotated ones
    are copied."""
    freq, mag = C.rope_frequencies(rot, **kw)
    want, size = C.rotate(K.f64(x), pos, freq, mag, rot, interleaved)
    err = np.abs(K.f64(got) - want)
    tol = 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size
    assert (err <= tol).all(), (what, float(np.max(err - tol)), np.argwhere(err > tol)[:3].tolist())


@pytest.mark.parametrize("kw", SCALINGS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("D,rot", [(128, 128), (128, 64), (128, 42), (128, 84), (64, 64), (64, 42),
                                   (64, 16), (128, 6), (64, 4)])
def test_rotation_and_append(D, rot, interleaved, kw):
    c = Case(5, 1, D, [1, 37], [700, 40], [1, 5001, 16, 100000], seed=rot + D)
    before = [p.clone() for p in c.pools]
    assert c.run(B.Rope(rot, interleaved=interleaved, **kw)) == B.OK
    _check_rotated(c.q_out(), c.q, c.pos, rot, interleaved, kw, "q")
    k = c.pools[0][torch.from_numpy(c.blk).cuda(), :, torch.from_numpy(c.row).cuda()]
    _check_rotated(k, c.k, c.pos, rot, interleaved, kw, "k")
    b, r = torch.from_numpy(c.blk).cuda(), torch.from_numpy(c.row).cuda()
    assert torch.equal(c.pools[1][b, :, r], c.v)
    for pool, old in zip(c.pools, before):           # no other row has changed
        pool[b, :, r] = old[b, :, r]
        assert torch.equal(pool, old)


def test_rotary_dims_of_two():
    c = Case(2, 2, 64, [3], [9], [5], seed=1)
    for interleaved in (False, True):
        assert c.run(B.Rope(2, interleaved=interleaved)) == B.OK
        _check_rotated(c.q_out(), c.q, c.pos, 2, interleaved, {})


@pytest.mark.parametrize("rot,interleaved", [(64, False), (64, True), (42, False)])
def test_frequencies_of_the_caller_s(rot, interleaved):
    """Negative ones, zero, some beyond a turn per position, and an attention factor."""
    freq = np.random.default_rng(rot).uniform(-9, 9, rot // 2)
    freq[:3] = 0.0, -0.0, 2 * np.pi
    c = Case(3, 1, 64, [40], [300], [1, 70000], seed=16)
    rope = B.Rope(rot, interleaved=interleaved, scaling="custom", inv_freq=freq.tolist(),
                  attention_factor=1.5)
    assert c.run(rope) == B.OK
    want, size = C.rotate(K.f64(c.q), c.pos, freq, 1.5, rot, interleaved)
    # as _check_rotated's; 70000 positions of 1.5 turns each lose 2^-34 turns of their quotient
    err = np.abs(K.f64(c.q_out()) - want)
    assert (err <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * size).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_far_positions(interleaved):
    """Positions around 2^24 (beyond which fp32 does not hold every whole number) and 2^26."""
    c = Case(2, 1, 128, [3], [(1 << 24) + 2], [(1 << 26) - 5, (1 << 26) + 1], seed=2)
    assert c.run(B.Rope(128, interleaved=interleaved)) == B.OK
    # the frequencies' own last bit (2^-53 relative) over 2^26 positions: 2^-27 radians
    _check_rotated(c.q_out(), c.q, c.pos, 128, interleaved, {})


def test_without_rotation_rows_are_copied():
    c = Case(4, 2, 128, [20], [33], [7, 1], seed=3)
    c.q[0, 0, :4] = torch.tensor([float("nan"), float("inf"), -float("inf"), -0.0])
    assert c.run(None) == B.OK
    assert torch.equal(c.q_out().view(torch.int16), c.q.contiguous().view(torch.int16))
    b, r = torch.from_numpy(c.blk).cuda(), torch.from_numpy(c.row).cuda()
    assert torch.equal(c.pools[0][b, :, r], c.k) and torch.equal(c.pools[1][b, :, r], c.v)


def test_channels_behind_the_rotated_ones_pass_through():
    """A NaN or an infinity stays in its pair, and where it is when it is not rotated."""
    for interleaved in (False, True):
        c = Case(2, 1, 128, [4], [400], [], seed=4)
        c.q[:, :, 100], c.q[:, :, 101], c.q[:, 1, 3] = float("nan"), float("inf"), float("inf")
        assert c.run(B.Rope(64, interleaved=interleaved)) == B.OK
        g = c.q_out().float()
        assert torch.isnan(g[:, :, 100]).all() and torch.isinf(g[:, :, 101]).all()
        bad = [100, 101]
        pair = [2, 3] if interleaved else [3, 35]
        ok0 = [i for i in range(128) if i not in bad]
        ok1 = [i for i in ok0 if i not in pair]
        assert torch.isfinite(g[:, 0, ok0]).all() and torch.isfinite(g[:, 1, ok1]).all()
        assert not torch.isfinite(g[:, 1, pair]).any()


@pytest.mark.parametrize("rot", [128, 42])
def test_in_place(rot):
    c = Case(4, 2, 128, [50], [90], [3, 70], seed=5)
    rope = B.Rope(rot)
    assert c.run(rope) == B.OK
    want = c.q_out()
    q = c.q.contiguous()
    c.q_p, c.q_d = q[:c.tp], q[c.tp:]
    assert c.run(rope, q=q) == B.OK
    assert torch.equal(q, want)


def test_strided_and_dense_inputs_agree():
    a = Case(6, 3, 64, [40], [41], [9], seed=6, pad=2)
    rope = B.Rope(64)
    assert a.run(rope) == B.OK
    want, pools = a.q_out(), [p.clone() for p in a.pools]
    for p in a.pools:
        p.zero_()
    a.q, a.k, a.v = (x.contiguous() for x in (a.q, a.k, a.v))
    assert a.run(rope) == B.OK
    b, r = torch.from_numpy(a.blk).cuda(), torch.from_numpy(a.row).cuda()
    assert torch.equal(a.q_out(), want)
    for p, w in zip(a.pools, pools):
        assert torch.equal(p[b, :, r], w[b, :, r])


def test_only_k_and_v():
    c = Case(4, 2, 128, [20], [30], [11], seed=7)
    assert c.run(B.Rope(128), q=None) == B.OK
    assert torch.isnan(c.q_out().float()).all()
    k = c.pools[0][torch.from_numpy(c.blk).cuda(), :, torch.from_numpy(c.row).cuda()]
    _check_rotated(k, c.k, c.pos, 128, False, {})


@pytest.mark.parametrize("heads", [(1, 1), (32, 32), (8, 1), (13, 13)])
@pytest.mark.parametrize("tokens", [1, 700])
def test_head_counts_and_token_counts(heads, tokens):
    c = Case(*heads, 128, [tokens], [tokens + 9], [], seed=8)
    assert c.run(B.Rope(128)) == B.OK
    _check_rotated(c.q_out(), c.q, c.pos, 128, False, {})
    k = c.pools[0][torch.from_numpy(c.blk).cuda(), :, torch.from_numpy(c.row).cuda()]
    _check_rotated(k, c.k, c.pos, 128, False, {})


# ---------------------------------------------------------------------------------- quantised
def test_e4m3_cache_equals_the_existing_append():
    """Without a rotation the e4m3 rows equal pod_attn_append_fp8's, bit for bit, as the oracle
    defines them."""
    from hybrid_prefill_decode_gb300 import workloads as W
    fb, k_new, v_new = W.fp8_append_case(8, 2, [1, 16, 17, 300], seed=9)
    k8, v8, vs = oracle.append_fp8(fb, k_new, v_new)
    d = fb.to("cuda")
    plan = B.Plan(8, 2, [], list(fb.decode_kv_lens), 4, d.num_blocks, d.max_blocks_per_seq, .1,
                  kv_fp8=True)
    ws = plan.alloc_workspace()
    plan.upload(ws)
    cache = B.KvCache("e4m3", d.k8, d.v8, d.k_scale, d.v_scale)
    plan.rope_append(None, None, k_new.cuda(), v_new.cuda(), cache, d.block_tables, None, None, ws)
    assert plan.device_status(ws) == B.OK
    assert np.array_equal(d.k8.cpu().numpy(), k8) and np.array_equal(d.v8.cpu().numpy(), v8)
    assert np.array_equal(d.v_scale.cpu().numpy(), vs, equal_nan=True)


@pytest.mark.parametrize("rot,interleaved", [(128, True), (64, False), (84, False), (42, True)])
def test_e4m3_rotated_rows_in_every_layout(rot, interleaved):
    """As test_e4m3_rotated_rows, K only."""
    c = Case(4, 2, 128, [60], [100], [1, 5000], seed=17, kind="e4m3")
    assert c.run(B.Rope(rot, interleaved=interleaved)) == B.OK
    freq, mag = C.rope_frequencies(rot)
    want, size = C.rotate(K.f64(c.k), c.pos, freq, mag, rot, interleaved)
    ks = c.scales[0].cpu().numpy().astype(np.float64)
    got = K.f64(c.pools[0])[c.blk, :, c.row] * ks
    want = np.clip(want, -448 * ks, 448 * ks)
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + (2.0 ** -10 + 2.0 ** -14) * ks +
            2.0 ** -19 * size).all()


def test_e4m3_rotated_rows():
    c = Case(4, 2, 128, [60], [100], [1, 5000], seed=10, kind="e4m3")
    assert c.run(B.Rope(128)) == B.OK
    freq, mag = C.rope_frequencies(128)
    want, size = C.rotate(K.f64(c.k), c.pos, freq, mag, 128, False)
    ks = c.scales[0].cpu().numpy().astype(np.float64)
    got = K.f64(c.pools[0])[c.blk, :, c.row] * ks
    # e4m3: half a step is 2^-4 of the value, or half the smallest step 2^-9; saturation at 448
    want = np.clip(want, -448 * ks, 448 * ks)
    assert (np.abs(got - want) <= 2.0 ** -4 * np.abs(want) + (2.0 ** -10 + 2.0 ** -14) * ks +
            2.0 ** -19 * size).all()
    v = K.f64(c.v)
    vs = c.scales[1].cpu().numpy()[c.blk, :, c.row].astype(np.float64)
    assert np.array_equal(vs, (np.abs(v).max(-1).astype(np.float32) / np.float32(448)))
    got = K.f64(c.pools[1])[c.blk, :, c.row] * vs[..., None]
    assert (np.abs(got - v) <= 2.0 ** -4 * np.abs(v) + 2.0 ** -9 * vs[..., None]).all()


@pytest.mark.parametrize("D,rot,interleaved", [(128, 128, False), (64, 42, False), (128, 64, True)])
def test_4_bit_rotated_rows(D, rot, interleaved):
    """Rotated K rows are quantised from fp32: a value is off by at most half the widest step of its
    group (1 of the scale, between 4 and 6) and by what the scale's own rounding lets the largest
    value saturate (2^-4 of it; half the smallest step 2^-10 where the scale is subnormal)."""
    c = Case(4, 2, D, [60], [100], [1, 70000], seed=11, kind="e2m1")
    assert c.run(B.Rope(rot, interleaved=interleaved)) == B.OK
    freq, mag = C.rope_frequencies(rot)
    want, size = C.rotate(K.f64(c.k), c.pos, freq, mag, rot, interleaved)
    h = c.scales[0].cpu().numpy().astype(np.float64)
    got = C.pool_values(c.pools[0].cpu().numpy(), D, h, False)[c.blk, :, c.row]
    grp = np.abs(want).reshape(*want.shape[:-1], -1, 16)
    top = np.repeat(grp.max(-1), 16, -1)
    step = top / 6 * (1 + 2.0 ** -4) + 2.0 ** -10 * h[:, None]
    tol = np.maximum(step, top * 2.0 ** -4 + 6 * 2.0 ** -10 * h[:, None]) + 2.0 ** -19 * size
    assert (np.abs(got - want) <= tol).all()
    # values far from any border are the nearest ones of the format, V (not rotated) exactly
    code, s8 = C.quantise_fp4(want.astype(np.float32), h.astype(np.float32))
    sign = np.where(code & 8, -1, 1)
    exact = sign * C.E2M1[code & 7] * np.repeat(C.E4M3[s8], 16, -1) * h[:, None]
    assert (got == exact).mean() > 0.99
    vcode, vs8 = C.quantise_fp4(K.f64(c.v).astype(np.float32), c.scales[1].cpu().numpy())
    pool = np.zeros(tuple(c.pools[1].shape), dtype=np.uint8)
    C.put_rows(pool, D, True, c.blk, c.row, vcode, vs8)
    a, b = (C.pool_values(p, D, np.ones(2), True)[c.blk, :, c.row]
            for p in (pool, c.pools[1].cpu().numpy()))
    assert np.array_equal(a, b)


@pytest.mark.parametrize("rot,interleaved", [(128, False), (64, True), (84, False)])
def test_queries_do_not_depend_on_the_cache(rot, interleaved):
    outs = []
    for kind in ("bf16", "e4m3", "e2m1"):
        c = Case(8, 1, 128, [3000], [50000], [1, 70001], seed=15, kind=kind)
        assert c.run(B.Rope(rot, interleaved=interleaved)) == B.OK
        outs.append(c.q_out())
    assert torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2])


# ---------------------------------------------------------------------------------- calls
@pytest.mark.parametrize("kind", ["bf16", "e4m3", "e2m1"])
def test_bad_block_index_is_reported(kind):
    c = Case(4, 2, 128, [20], [40], [17, 5], seed=12, kind=kind)
    good = c.tab.clone()
    before = [p.clone().view(torch.uint8) for p in c.pools]
    c.tab[1, 1] = c.nb                               # the first decode's block
    assert c.run(B.Rope(128)) == B.ERR_BAD_INDEX
    _check_rotated(c.q_out(), c.q, c.pos, 128, False, {})     # q does not depend on it
    for p, old in zip(c.pools, before):
        assert torch.equal(p.view(torch.uint8)[good[1, 1]], old[good[1, 1]])
    c.tab = good
    assert c.run(B.Rope(128)) == B.OK


def test_captured_and_replayed_on_another_stream():
    c = Case(8, 2, 128, [33], [80], [3, 900], seed=13)
    rope = B.Rope(128)
    assert c.run(rope) == B.OK
    want, pool = c.q_out(), c.pools[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            c.plan.rope_append(rope, c.q, c.k, c.v, c.cache, c.tab, c.q_p, c.q_d, c.ws)
        del rope                                     # the launch needs the handle no longer
        for _ in range(2):
            c.q_p.zero_(), c.q_d.zero_(), c.pools[0].zero_()
            g.replay()
            side.synchronize()
            assert torch.equal(c.q_out(), want)
    b, r = torch.from_numpy(c.blk).cuda(), torch.from_numpy(c.row).cuda()
    assert torch.equal(c.pools[0][b, :, r], pool[b, :, r])


def test_wrong_tensors_are_refused_by_the_binding():
    c = Case(4, 2, 128, [20], [40], [17], seed=14)
    rope = B.Rope(128)
    args = dict(q=c.q, k=c.k, v=c.v, bt=c.tab, qp=c.q_p, qd=c.q_d)
    def call(**kw):
        a = {**args, **kw}
        c.plan.rope_append(rope, a["q"], a["k"], a["v"], c.cache, a["bt"], a["qp"], a["qd"], c.ws)
    for kw in (dict(q=c.q.float()), dict(q=c.q[:5]), dict(k=c.q), dict(v=c.v.transpose(0, 1)),
               dict(q=c.qkv[:, ::2][:, :4]), dict(bt=c.tab.long()), dict(qp=None),
               dict(qp=c.q_p.float()), dict(qd=c.q_d[:0]), dict(k=c.k.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(B.PodAttnError) as e:
        B.Plan(4, 2, [], [3], 1, 4, 1, .1, head_dim=64).rope_append(
            B.Rope(128), None, c.k[:1, :, :64].contiguous(), c.v[:1, :, :64].contiguous(),
            B.KvCache("bf16", *[torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
                                for _ in range(2)]),
            torch.zeros((1, 1), dtype=torch.int32, device="cuda"), None, None, c.ws)
    assert e.value.code in (B.ERR_INVALID_ARG, B.ERR_WORKSPACE)
