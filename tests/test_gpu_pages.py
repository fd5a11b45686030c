"""Block copies on the GPU, and the operators around the cache run together as a server would: prompts
in chunks, decode steps, forks and a compaction over a 4-bit cache."""
import numpy as np
import pytest
import torch

import cache_cases as K
from hybrid_prefill_decode_gb300 import binding as B
from hybrid_prefill_decode_gb300 import workloads as W
from oracle import cache_ops as C

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__
    __graft_entry__.build()


def _pools(nb, shapes, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.randint(0, 256, (nb, n), generator=g, device="cuda", dtype=torch.uint8)
            for n in shapes]


@pytest.mark.parametrize("nb,sizes,n_pairs", [
    (2, [16], 1), (300, [16, 48, 9216, 40960], 100), (5000, [64], 2499), (7000, [16, 32], 3400),
    (64, [1152 * 3] * 17, 5), (40, [512] * 130, 19), (130, [80] * 16, 64), (131, [80] * 16, 65)])
def test_copies(nb, sizes, n_pairs):
    pools = _pools(nb, sizes, nb)
    rng = np.random.default_rng(nb)
    perm = rng.permutation(nb)
    dst = perm[:n_pairs]
    src = rng.choice(perm[n_pairs:], n_pairs)        # a block may be read many times
    pairs = torch.from_numpy(np.stack((src, dst), 1).astype(np.int32))
    want = [p.clone() for p in pools]
    for w in want:
        w[torch.from_numpy(dst).cuda()] = w[torch.from_numpy(src).cuda()]
    B.copy_blocks(pools, pairs)
    for p, w in zip(pools, want):
        assert torch.equal(p, w)


def test_copies_beyond_4_gib():
    nb = 5000
    pool = torch.zeros((nb, 1 << 20), dtype=torch.uint8, device="cuda")
    pool[4999], pool[7] = 3, 9
    B.copy_blocks([pool], [(4999, 0), (7, 4998)])
    assert (pool[0] == 3).all() and (pool[4998] == 9).all() and not pool[4997].any()
    assert not pool[1].any()


def test_copy_of_a_block_onto_itself_and_of_nothing():
    pool = _pools(4, [32])[0]
    before = pool.clone()
    B.copy_blocks([pool], [(2, 2)])
    B.copy_blocks([pool], [])
    B.copy_blocks([pool[:0]], [])
    B.copy_blocks([], [(1, 2)])
    assert torch.equal(pool, before)


def test_copies_are_refused():
    pool = _pools(4, [32])[0]
    before = pool.clone()
    for pairs in ([(0, 4)], [(0, 1), (2, 1)], [(0, 1), (1, 2)], [(-1, 0)]):
        with pytest.raises(B.PodAttnError):
            B.copy_blocks([pool], pairs)
    for pools, pairs in (([pool, _pools(5, [32])[0]], [(0, 1)]), ([pool[:, ::2]], [(0, 1)]),
                         ([pool], torch.tensor([[0, 1]])), ([pool], torch.tensor([0, 1]).int())):
        with pytest.raises(ValueError):
            B.copy_blocks(pools, pairs)
    with pytest.raises(B.PodAttnError):
        B.copy_blocks([torch.zeros((4, 24), dtype=torch.uint8, device="cuda")], [(0, 1)])
    assert torch.equal(pool, before)


def test_copies_captured_keep_their_pairs():
    pools = _pools(50, [64, 4096])
    pairs = torch.tensor([[1, 2], [3, 4]], dtype=torch.int32)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            B.copy_blocks(pools, pairs)
        pairs.fill_(0)                               # the call has taken what it needs
        g.replay()
        side.synchronize()
    for p in pools:
        assert torch.equal(p[1], p[2]) and torch.equal(p[3], p[4])


def test_kv_cache_names_the_pools_to_copy():
    z = lambda *s, **k: torch.zeros(s, device="cuda", **k)
    u8 = dict(dtype=torch.uint8)
    assert len(B.KvCache("bf16", *[z(4, 2, 16, 64, dtype=torch.bfloat16) for _ in "kv"]).pools) == 2
    c = B.KvCache("e4m3", z(2, 2, 16, 128, **u8), z(2, 2, 16, 128, **u8), z(2, 128), z(2, 2, 16))
    assert [tuple(t.shape) for t in c.pools] == [(2, 2, 16, 128)] * 2 + [(2, 2, 16)]
    c = B.KvCache("e2m1", z(2, 2, 576, **u8), z(2, 2, 576, **u8), z(2), z(2))
    assert len(c.pools) == 2


class Server:
    """One layer of a model over a 4-bit cache, with a copy of every sequence's rows in 64 bits."""

    def __init__(self, hq, hkv, D, rot, interleaved, seed, nb=120, seqs=6, maxb=40):
        self.hq, self.hkv, self.D, self.maxb = hq, hkv, D, maxb
        self.rng = np.random.default_rng(seed)
        self.scale = 1.0 / np.sqrt(D)
        self.rope, self.rot, self.inter = B.Rope(rot, interleaved=interleaved), rot, interleaved
        u8 = dict(dtype=torch.uint8, device="cuda")
        shape = B.fp4_pool_shape(nb, hkv, D)
        self.h = [torch.from_numpy(self.rng.uniform(.3, 1, hkv).astype(np.float32)).cuda()
                  for _ in range(2)]
        self.cache = B.KvCache("e2m1", torch.full(shape, 0x7F, **u8), torch.full(shape, 0x7F, **u8),
                               *self.h)
        self.nb = nb
        self.scratch = [torch.full((nb, hkv, 16, D), float("nan"), dtype=torch.bfloat16,
                                   device="cuda") for _ in range(2)]
        self.pages = B.Pages(nb, seqs, maxb)

    def _new(self, t):
        x = K.bf16(self.rng.standard_normal((t, self.hq + 2 * self.hkv, self.D))).cuda()
        return x, x[:, :self.hq], x[:, self.hq:self.hq + self.hkv], x[:, self.hq + self.hkv:]

    def _rows(self, seqs):
        """Each sequence's K and V values as the cache holds them, read on the host."""
        bt, lens = self.pages.tables(seqs)
        vals = [C.pool_values(t.cpu().numpy(), self.D, h.cpu().numpy(), v)
                for t, h, v in zip(self.cache.tensors[:2], self.h, (False, True))]
        return vals, bt.numpy(), lens.tolist()

    def copy(self, pairs):
        B.copy_blocks(self.cache.pools, pairs)

    def prompt(self, seq, n):
        """A chunk of n tokens behind what the sequence holds."""
        old = int(self.pages.tables([seq])[1][0])
        self.copy(self.pages.grow(seq, old + n))
        bt, lens = self.pages.tables([seq])
        x, q, k, v = self._new(n)
        plan = B.Plan(self.hq, self.hkv, [0, n], lens.tolist(), 0, self.nb, self.maxb, self.scale,
                      head_dim=self.D)
        ws = plan.alloc_workspace()
        plan.upload(ws)
        tab, kv = bt.cuda(), lens.cuda()
        qp = torch.empty((n, self.hq, self.D), dtype=torch.bfloat16, device="cuda")
        plan.rope_append(self.rope, q, k, v, self.cache, tab, qp, None, ws)
        plan.expand_fp4(self.cache, tab, *self.scratch, tab, kv, ws)
        o = torch.empty_like(qp)
        plan.run(qp, None, *self.scratch, tab, torch.tensor([0, n], dtype=torch.int32).cuda(), kv,
                 o, None, ws)
        assert plan.device_status(ws) == B.OK
        freq, mag = C.rope_frequencies(self.rot)
        pos = np.arange(old, old + n)
        q_ref, size = C.rotate(K.f64(q), pos, freq, mag, self.rot, self.inter)
        assert (np.abs(K.f64(qp) - q_ref) <= 2.0 ** -8 * np.abs(q_ref) + 2.0 ** -20 * size).all()
        # every token of the chunk is a decode over the rows up to its own
        (kk, vv), t, _ = self._rows([seq])
        pick = sorted({0, n // 2, n - 1})
        ref = C.decode(K.f64(qp)[pick], kk, vv, np.repeat(t, len(pick), 0),
                       [int(pos[i]) + 1 for i in pick], self.scale)[0]
        # the bf16 attention's own tolerance, its rows rounded to bf16
        assert (np.abs(K.f64(o)[pick] - ref) <= 2e-2 + 2e-2 * np.abs(ref)).all()

    def step(self, seqs):
        """One decode token for each sequence."""
        for s in seqs:
            self.copy(self.pages.grow(s, int(self.pages.tables([s])[1][0]) + 1))
        bt, lens = self.pages.tables(seqs)
        x, q, k, v = self._new(len(seqs))
        plan = B.Plan(self.hq, self.hkv, [], lens.tolist(), len(seqs), self.nb, self.maxb,
                      self.scale, head_dim=self.D, kv_fp4=True)
        ws = plan.alloc_workspace()
        plan.upload(ws)
        tab = bt.cuda()
        qd = torch.empty((len(seqs), self.hq, self.D), dtype=torch.bfloat16, device="cuda")
        o = torch.empty_like(qd)
        plan.rope_append(self.rope, q, k, v, self.cache, tab, None, qd, ws)
        plan.run_decode_fp4(qd, self.cache, tab, lens.cuda(), o, ws)
        assert plan.device_status(ws) == B.OK
        (kk, vv), t, n = self._rows(seqs)
        with np.errstate(invalid="ignore"):
            K.check_decode(o, *C.decode(K.f64(qd), kk, vv, t, n, self.scale), "step")
        return qd, o, tab, lens


@pytest.mark.parametrize("hq,hkv,D,rot,interleaved", [
    (8, 2, 128, 128, False), (4, 4, 64, 32, True), (7, 1, 128, 64, False)])
def test_serving_over_a_4_bit_cache(hq, hkv, D, rot, interleaved):
    s = Server(hq, hkv, D, rot, interleaved, seed=hq + D)
    s.prompt(0, 70)
    s.prompt(0, 129)                                 # a second chunk behind the first
    s.prompt(1, 33)
    for _ in range(2):
        s.step([0, 1])
    n = int(s.pages.tables([0])[1][0])
    s.pages.fork(0, 2, n)                            # the whole sequence, its last page shared
    s.pages.fork(0, 3, 40)                           # a prefix that ends inside a page
    before = s._rows([0])
    for _ in range(3):
        s.step([3, 2, 0, 1])
    after = s._rows([0])                             # what was shared reads the same
    for a, b in zip(before[0], after[0]):
        ra, rb = (v[t[0, np.arange(n) // 16], :, np.arange(n) % 16]
                  for v, t in ((a, before[1]), (b, after[1])))
        assert np.array_equal(ra, rb)
    s.pages.free(1)
    s.prompt(4, 50)
    s.pages.free(4)
    # a decode over the same rows before and after a compaction: the same bits
    qd, o, tab, lens = s.step([0, 2, 3])
    s.copy(s.pages.compact())
    assert int(s.pages.tables([0, 2, 3])[0].max()) < s.nb - s.pages.free_blocks
    plan = B.Plan(hq, hkv, [], lens.tolist(), 3, s.nb, s.maxb, s.scale, head_dim=D, kv_fp4=True)
    ws = plan.alloc_workspace()
    plan.upload(ws)
    again = torch.empty_like(o)
    plan.run_decode_fp4(qd, s.cache, s.pages.tables([0, 2, 3])[0].cuda(), lens.cuda(), again, ws)
    assert plan.device_status(ws) == B.OK and torch.equal(o, again)
    s.step([2, 3, 0])


@pytest.mark.parametrize("hkv,layer", [(1, 1), (1, 3), (2, 1), (5, 2)])
def test_head_scales_in_a_table_of_all_layers(hkv, layer):
    """A layer's head scales as a row of fp32 [layers][Hkv], at whatever multiple of 4 bytes it starts,
    give the bits of the same scales in tensors of their own."""
    c = K.Fp4Case(2 * hkv, hkv, 64, [40, 300], seed=hkv).to()
    table = torch.full((2, 4, hkv), float("nan"), device="cuda")
    table[0, layer], table[1, layer] = c.cache.tensors[2], c.cache.tensors[3]
    rows = torch.randn((2, 4 * hkv, 64), generator=torch.Generator().manual_seed(1))
    rows = rows.to(torch.bfloat16).cuda()
    plan = c.plan()
    wide = B.Plan(2 * hkv, hkv, [], c.lens, 2, c.nb, c.bt.shape[1], .1, head_dim=64)
    ws, ws16 = plan.alloc_workspace(), wide.alloc_workspace()
    plan.upload(ws)
    wide.upload(ws16)
    got = []
    for scales in (c.cache.tensors[2:], table[:, layer]):
        pools = [t.clone() for t in (c.k, c.v)]
        cache = B.KvCache("e2m1", *pools, *scales)
        o, q = torch.empty_like(c.qd), torch.empty_like(c.qd)
        out = [torch.zeros((c.nb, hkv, 16, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
        plan.rope_append(B.Rope(64), rows[:, :2 * hkv], rows[:, 2 * hkv:3 * hkv], rows[:, 3 * hkv:],
                         cache, c.tab, None, q, ws)
        plan.run_decode_fp4(q, cache, c.tab, c.kv, o, ws)
        wide.expand_fp4(cache, c.tab, *out, c.tab, c.kv, ws16)
        assert plan.device_status(ws) == B.OK and wide.device_status(ws16) == B.OK
        got.append(pools + [q, o] + out)
    assert torch.isfinite(got[0][3]).all()
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("hq,hkv,D,lens", [
    (32, 8, 128, [700, 31, 2000, 90]), (8, 8, 64, [300] * 20), (8, 1, 128, [30000])])
def test_launches_one_behind_another_see_each_others_writes(hq, hkv, D, lens, graph):
    """Launches may start while the one in front of them ends: a run of them gives the bits of the same
    run with a wait for the device behind each."""
    c = K.Fp4Case(hq, hkv, D, lens, seed=hq + D).to()
    n, steps = len(lens), 6
    plan = c.plan()
    big = B.Plan(hq, hkv, [], lens, n, c.nb, c.bt.shape[1], c.scale, head_dim=D)   # of the bf16 pools
    ws, ws16 = plan.alloc_workspace(), big.alloc_workspace()
    rope = B.Rope(D)
    spare = sorted(set(range(c.nb)) - set(int(b) for b in c.bt.ravel()))[0]
    first, last = int(c.bt[0, 0]), int(c.bt[0, (lens[0] - 1) // 16])
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((steps, n, hq + 2 * hkv, D), generator=g, device="cuda").to(torch.bfloat16)
    clean = [t.clone() for t in c.cache.tensors]
    buf, qd = torch.empty_like(rows[0]), torch.empty_like(c.qd)
    pools = [torch.empty((c.nb, hkv, 16, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    outs = [torch.empty((steps,) + qd.shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def run(out, wait):
        for t, v in zip(c.cache.tensors, clean):
            t.copy_(v)
        for p in pools:
            p.zero_()
        for i in range(steps):
            buf.copy_(rows[i])
            wait()
            c.cache.tensors[2].mul_(1.25)            # the head scales, just before they are read
            wait()
            plan.rope_append(rope, buf[:, :hq], buf[:, hq:hq + hkv], buf[:, hq + hkv:], c.cache,
                             c.tab, None, qd, ws)
            wait()
            plan.run_decode_fp4(qd, c.cache, c.tab, c.kv, out[i], ws)
            wait()
            B.copy_blocks(c.cache.pools, [(last, spare)])
            wait()
            B.copy_blocks(c.cache.pools, [(spare, first)])
            wait()
            big.expand_fp4(c.cache, c.tab, *pools, c.tab, c.kv, ws16)
            wait()

    for p, w in ((plan, ws), (big, ws16)):
        p.upload(w)
    run(outs[0], torch.cuda.synchronize)
    want = [t.clone() for t in c.cache.tensors + pools]
    if graph:
        torch.cuda.synchronize()
        with torch.cuda.graph(gr := torch.cuda.CUDAGraph()):
            run(outs[1], lambda: None)
    for _ in range(10):
        outs[1].zero_()
        gr.replay() if graph else run(outs[1], lambda: None)
        torch.cuda.synchronize()
        assert plan.device_status(ws) == B.OK and big.device_status(ws16) == B.OK
        assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
        for a, b in zip(c.cache.tensors + pools, want):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("variant", ["fused", "serial", "streams"])
def test_launches_among_those_of_the_attention(variant, graph):
    """The attention's launches (with the append in front one that needs all its CTAs at once, or several
    on two streams) between the cache operators': the bits of the same run with a wait behind each."""
    b = W.make_batch(8, 2, [60, 7], [200, 300], [900, 31], seed=5, device="cuda")
    plan = B.Plan.for_batch(b, variant=variant)
    ws = plan.alloc_workspace()
    plan.upload(ws)
    rope, cache = B.Rope(128), B.KvCache("bf16", b.k_pool, b.v_pool)
    used = set()
    for i, n in enumerate([200, 300, 900, 31]):
        used |= set(b.block_tables[i, :-(-n // 16)].tolist())
    spare = sorted(set(range(b.num_blocks)) - used)[0]
    move = [(int(b.block_tables[2, 3]), spare), (spare, int(b.block_tables[3, 0]))]
    g = torch.Generator(device="cuda").manual_seed(1)
    rows = torch.randn((5, 69, 12, 128), generator=g, device="cuda").to(torch.bfloat16)
    buf, k_new = torch.empty_like(rows[0]), torch.empty((2, 69, 2, 128), dtype=torch.bfloat16,
                                                        device="cuda")
    qp, qd = torch.empty_like(b.q_prefill), torch.empty_like(b.q_decode)
    outs = [[torch.empty((5, 2) + t.shape, dtype=t.dtype, device="cuda") for t in (qp, qd)]
            for _ in range(2)]
    clean, side = [b.k_pool.clone(), b.v_pool.clone()], torch.cuda.Stream()

    def run(out, wait):
        b.k_pool.copy_(clean[0])
        b.v_pool.copy_(clean[1])
        for i in range(5):
            buf.copy_(rows[i])
            k_new[0].copy_(rows[i, :, 8:10])
            k_new[1].copy_(rows[i, :, 10:])
            wait()
            plan.rope_append(rope, buf[:, :8], buf[:, 8:10], buf[:, 10:], cache, b.block_tables, qp, qd,
                             ws)
            wait()
            plan.run(qp, qd, b.k_pool, b.v_pool, b.block_tables, b.cu_seqlens_q, b.kv_lens,
                     out[0][i, 0], out[1][i, 0], ws, stream2=side)
            wait()
            B.copy_blocks([b.k_pool, b.v_pool], move[:1])
            wait()
            plan.run_append(qp, qd, k_new[0], k_new[1], b.k_pool, b.v_pool, b.block_tables,
                            b.cu_seqlens_q, b.kv_lens, out[0][i, 1], out[1][i, 1], ws, stream2=side)
            wait()
            B.copy_blocks([b.k_pool, b.v_pool], move[1:])
            wait()

    main = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        run(outs[0], torch.cuda.synchronize)
        want = [b.k_pool.clone(), b.v_pool.clone()]
        torch.cuda.synchronize()
        if graph:
            with torch.cuda.graph(gr := torch.cuda.CUDAGraph(), stream=main):
                run(outs[1], lambda: None)
        for _ in range(10):
            for t in outs[1]:
                t.zero_()
            gr.replay() if graph else run(outs[1], lambda: None)
            torch.cuda.synchronize()
            assert plan.device_status(ws) == B.OK
            assert all(torch.isfinite(t).all() for t in outs[0])
            for x, y in zip(outs[0] + want, outs[1] + [b.k_pool, b.v_pool]):
                assert torch.equal(x.view(torch.int16), y.view(torch.int16))   # rows of no one: NaN


@pytest.mark.parametrize("graph", [False, True])
def test_a_launch_behind_an_event_of_another_stream_waits_for_it(graph):
    c = K.Fp4Case(32, 8, 128, [900, 3000], seed=3).to()
    plan = c.plan()
    ws = plan.alloc_workspace()
    plan.upload(ws)
    rope = B.Rope(128)
    g = torch.Generator(device="cuda").manual_seed(2)
    rows = torch.randn((2, 48, 128), generator=g, device="cuda").to(torch.bfloat16)
    buf, qd, o = torch.zeros_like(rows), torch.empty_like(c.qd), torch.empty_like(c.qd)
    slow, quick = torch.zeros(1 << 26, device="cuda"), torch.zeros(64, device="cuda")
    side, main = torch.cuda.Stream(), torch.cuda.Stream()

    def run():
        side.wait_stream(main)
        with torch.cuda.stream(side):
            for _ in range(4):
                slow.add_(1)                         # some hundreds of us
            buf.copy_(rows)
        quick.add_(1)
        main.wait_stream(side)                       # the kernel in front in this stream is done long before
        plan.rope_append(rope, buf[:, :32], buf[:, 32:40], buf[:, 40:], c.cache, c.tab, None, qd, ws)
        plan.run_decode_fp4(qd, c.cache, c.tab, c.kv, o, ws)

    clean = [t.clone() for t in c.cache.tensors]
    torch.cuda.synchronize()
    with torch.cuda.stream(main):
        run()
        torch.cuda.synchronize()
        want, qw = o.clone(), qd.clone()
        assert qw.any()
        if graph:
            torch.cuda.synchronize()
            with torch.cuda.graph(gr := torch.cuda.CUDAGraph(), stream=main):
                run()
        for _ in range(10):
            for t in (buf, qd, o):
                t.zero_()
            for t, v in zip(c.cache.tensors, clean):
                t.copy_(v)
            gr.replay() if graph else run()
            torch.cuda.synchronize()
            assert torch.equal(qd, qw) and torch.equal(o, want)
    assert plan.device_status(ws) == B.OK
