"""How the calls that hold a paged cache to a budget are made: on streams of
their own, captured and replayed, again on the same workspace, over shared
pages, over pools past 4 GB, with many conversations and with none."""
import numpy as np
import pytest
import torch

from tests.test_budget_gpu import (_bf16, _f32, _i32, check_evict, check_step, check_weigh,
                                   make_evict, make_step, make_weigh, run_step)
from tests.test_call_streams_gpu import busy  # noqa: F401
from trained_kv_prefix_gb300 import cartattn as ca

pytestmark = pytest.mark.gpu


class Cache:
    """One layer of a batch and a run of the four calls over it."""

    B, n, Hq, Hkv, d, p, P, M, T, budget = 5, 70, 8, 2, 128, 300, 16, 8, 9, 40

    def __init__(self, seed=1):
        rng = np.random.default_rng(seed)
        B, n, Hq, Hkv, d, N = self.B, self.n, self.Hq, self.Hkv, self.d, self.B * self.M + 3
        self.k, self.v = (_bf16(rng, (B, n, Hkv, d)).cuda() for _ in range(2))
        self.q = _bf16(rng, (B, self.T, Hq, d), 1.5).cuda()
        self.lse = _f32(rng.standard_normal((B, Hq, self.T)) + 4)
        self.kc, self.vc = (_bf16(rng, (self.p, Hkv, d)).cuda() for _ in range(2))
        self.q1 = _bf16(rng, (B, Hq, d), 1.5).cuda()
        self.k1, self.v1 = (_bf16(rng, (B, Hkv, d)).cuda() for _ in range(2))
        used = -(-(n + 1) // self.P)
        table = np.full((B, self.M), -1, np.int32)
        table[:, :used] = rng.permutation(N)[:B * used].reshape(B, used)
        self.table0, self.refs0 = _i32(table), _i32(np.bincount(table[table >= 0], minlength=N))
        self.start, self.held = _i32([0] * B), _i32([n] * B)
        self.keep = _i32([self.budget] * B)
        self.pos = _i32([self.p + n] * B)
        self.kp, self.vp = (torch.zeros(N, self.P, Hkv, d, dtype=torch.bfloat16, device="cuda")
                            for _ in range(2))
        self.w = torch.zeros(B, Hkv, self.M * self.P, device="cuda")
        self.table, self.refs, self.lens = (x.clone() for x in (self.table0, self.refs0, self.held))
        N = self.kp.shape[0]
        sizes = (ca.weights_workspace_size(B, self.T, Hq, Hkv, d, self.p, self.P, self.M),
                 ca.evict_workspace_size(B, self.M, N),
                 ca.decode_paged_workspace_size(B, Hq, Hkv, d, self.p, self.P, self.M, True))
        self.sizes = sizes
        self.own = [torch.empty(s, dtype=torch.uint8, device="cuda") for s in sizes]

    def run(self, own=False, **kw):
        """Everything from the start; the outputs."""
        a, b, c = ({"workspace": x} if own else {} for x in self.own)
        self.kp.zero_(), self.vp.zero_(), self.w.zero_()
        self.table.copy_(self.table0), self.refs.copy_(self.refs0), self.lens.copy_(self.held)
        return self.calls(a, b, c, **kw)

    def calls(self, a, b, c, **kw):
        ca.cart_pages_append(self.k, self.v, self.kp, self.vp, self.table, self.start, p=self.p, **kw)
        _, cart = ca.cart_attn_weights(self.q, self.lse, self.kc, self.kp, self.table, self.lens,
                                       self.w, **a, **kw)
        done = ca.cart_pages_evict(self.kp, self.vp, self.table, self.lens, self.refs, self.w,
                                   self.keep, first=3, recent=10, **b, **kw)
        o = ca.cart_attn_decode_paged(self.q1, self.k1, self.v1, self.kc, self.vc, self.kp, self.vp,
                                      self.table, self.lens, pos=self.pos, weights=self.w, **c, **kw)
        return o, done, cart

    def state(self, out):
        torch.cuda.synchronize()
        return [x.clone() for x in (*out, self.kp, self.vp, self.w, self.table, self.refs, self.lens)]


def same(a, b):
    return all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


def test_calls_beside_a_busy_stream(busy):  # noqa: F811
    c = Cache()
    want = c.state(c.run())
    side = torch.cuda.Stream()
    c.kp.zero_(), c.vp.zero_(), c.w.zero_()
    c.table.copy_(c.table0), c.refs.copy_(c.refs0), c.lens.copy_(c.held)
    busy(*c.sizes, want[0].numel() * 2)
    out = c.calls({}, {}, {}, stream=side)      # one after the other on a stream of their own
    assert same(c.state(out), want)
    assert ca.device_status(clear=True) == 0


def test_captured_calls_replay():
    """Captured from the start of the state on; replayed, each run is the
    eager one, beside another graph with workspaces of its own."""
    caches = [Cache(1), Cache(2)]
    want = [c.state(c.run(own=True)) for c in caches]
    graphs, outs = [], []
    for c in caches:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run(own=True))
        graphs.append(g)
    sides = [torch.cuda.Stream() for _ in caches]
    for _ in range(3):
        for c, out in zip(caches, outs):
            for x in (*out, *c.own):
                x.fill_(77)
        torch.cuda.synchronize()
        for _ in range(4):
            for g, s in zip(graphs, sides):
                with torch.cuda.stream(s):
                    g.replay()
        for c, out, w in zip(caches, outs, want):
            assert same(c.state(out), w)
    assert ca.device_status(clear=True) == 0


def test_workspaces_hold_anything():
    c = Cache(3)
    want = c.state(c.run())
    for fill in (0, 255, 127):
        for x in c.own:
            x.fill_(fill)
        assert same(c.state(c.run(own=True)), want)
    # ... and are as large as asked for: what lies behind is left alone
    big = [torch.full((s + 4096,), 93, dtype=torch.uint8, device="cuda") for s in c.sizes]
    c.own = [x[:s] for x, s in zip(big, c.sizes)]
    assert same(c.state(c.run(own=True)), want)
    assert all((x[s:] == 93).all() for x, s in zip(big, c.sizes))


@pytest.mark.parametrize("window,sinks", [(0, 0), (200, 9)])
def test_calls_repeat_bit_for_bit(window, sinks):
    s = make_step(21, 30, 28, 4, 128, 900, tuple(range(3, 1203, 40)), 64)
    t, lse, table, lens, _ = make_weigh(22, 4, 90, 16, 4, 64, 500, (300, 90, 700, 64), 32)
    seen = []
    for _ in range(4):
        w = torch.zeros(30, 4, s[1].shape[1] * 64, device="cuda")
        o, g = run_step(*s, weights=w, window=window, sinks=sinks)
        gw = torch.zeros(4, 4, table.shape[1] * 32, device="cuda")
        x = ca.cart_attn_weights(t["q"].cuda(), _f32(lse), t["kc"].cuda(), t["k_pages"].cuda(),
                                 _i32(table), _i32(lens), gw, window=window, sinks=sinks)
        seen.append((o, w, g["k_pages"], *x))
    assert all(same(x, seen[0]) for x in seen[1:])


def test_shared_pages_are_read_by_all():
    """Branches over one history: the same pages in several tables."""
    t, table, lens, _ = make_step(23, 4, 8, 2, 64, 40, (70, 75, 64, 3), 16)
    table[1:3, :4] = table[0, :4]
    check_step(t, table, lens)
    w, lse, table, lens, _ = make_weigh(24, 3, 7, 4, 2, 64, 20, (70, 75, 64), 16)
    table[1:, :4] = table[0, :4]
    check_weigh(w, lse, table, lens, None)


def test_weights_rows_may_be_wider_or_odd():
    """Rows of weights at any distance: the same numbers."""
    s = make_step(25, 3, 8, 2, 64, 40, (70, 75, 0), 16)
    rows = s[1].shape[1] * 16
    got = []
    for W in (rows, rows + 1, rows + 4):
        w = torch.full((3, 2, W), 0.25, device="cuda")
        run_step(*s, weights=w)
        assert (w[:, :, rows:] == 0.25).all()
        got.append(w[:, :, :rows].clone())
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_queries_without_a_finite_logit_give_no_weight():
    t, lse, table, lens, _ = make_weigh(26, 2, 12, 4, 2, 64, 30, (70, 5), 16)
    got = []
    for x in (-np.inf, np.inf):         # exp(s - inf) = 0
        l = lse.copy()
        l[:, 1, 3:9] = x
        got.append(ca.cart_attn_weights(t["q"].cuda(), _f32(l), t["kc"].cuda(), t["k_pages"].cuda(),
                                        _i32(table), _i32(lens), torch.zeros(2, 2, 96, device="cuda")))
    assert same(*got)


@pytest.mark.parametrize("lens", ["none", "idle", "mixed"])
def test_many_conversations(lens):
    """More conversations than threads that schedule them; with nothing cached,
    or nothing at all."""
    B = 700
    rng = np.random.default_rng(27)
    n = {"none": np.zeros(B, int), "idle": np.full(B, -1),
         "mixed": np.where(rng.random(B) < 0.2, -1, rng.integers(0, 60, B))}[lens]
    check_step(*make_step(28, B, 2, 1, 64, 20, n, 16))
    if lens == "mixed":
        check_weigh(*make_weigh(29, B, 2, 2, 1, 64, 20, n, 16))
    elif lens == "idle":
        t, lse, table, lens, _ = make_weigh(29, B, 2, 2, 1, 64, 20, n, 16)
        w, cart = ca.cart_attn_weights(t["q"].cuda(), _f32(lse), t["kc"].cuda(), t["k_pages"].cuda(),
                                       _i32(table), _i32(lens),
                                       torch.ones(B, 1, table.shape[1] * 16, device="cuda"))
        assert (w == 1).all() and (cart == 0).all()


EVICTS = [
    # id, B, layers, Hkv, d, P, lens, keep, first, recent, share, ties: more blocks
    # than fit at once, more rows than are listed or whose weights are held at once
    ("many_blocks", 2, 20, 8, 16, 16, (1300, 90), (1100, 33), 4, 90, 1, False),
    ("many_blocks_shared", 4, 10, 8, 16, 16, (190, 190, 120, 33), (40, 41, 90, 30), 4, 9, 2, True),
    ("many_blocks_long", 1, 39, 8, 8, 64, (6300,), (150,), 4, 90, 1, False),
    ("long_unheld", 1, 1, 1, 64, 128, (23000,), (5000,), 4, 1000, 1, False),
    ("long_unheld_ties", 1, 1, 1, 64, 128, (21600,), (2500,), 0, 0, 1, True),
    ("wide_rows", 2, 1, 1, 2048, 16, (90, 40), (33, 39), 1, 3, 1, False),
    ("wider_rows", 2, 1, 1, 8192, 16, (40, 30), (33, 11), 1, 3, 1, False),
]


@pytest.mark.parametrize("case", EVICTS, ids=[c[0] for c in EVICTS])
def test_evict_sizes(case):
    _, B, layers, Hkv, d, P, lens, keep, first, recent, share, ties = case
    check_evict(*make_evict(B + layers, B, layers, Hkv, d, P, lens, share, ties=ties), keep, first,
                recent)


def test_pools_past_4_gb():
    """Pages whose bytes and elements lie past 2^32: the calls over the last
    pages of such pools are those over small ones."""
    c = Cache(4)
    want = c.state(c.run())
    n = c.kp.shape[0]
    N = (1 << 32) // c.kp[0].numel() + n + 7       # elements past 2^32
    big = [torch.zeros(N, *c.kp.shape[1:], dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    c.kp, c.vp = big
    c.table0 = torch.where(c.table0 >= 0, c.table0 + (N - n), -1).int()
    c.refs0 = torch.cat([torch.ones(N - n, dtype=torch.int32, device="cuda"), c.refs0])
    c.refs = c.refs0.clone()
    got = c.state(c.run())
    got[3], got[4], got[7] = got[3][N - n:], got[4][N - n:], got[7][N - n:]
    got[6] = torch.where(got[6] >= 0, got[6] - (N - n), -1).int()
    assert same(got, want)
    assert all((x[i:i + 4096] == 0).all() for x in big for i in range(0, N - n, 4096)
               if i + 4096 <= N - n)
    assert ca.device_status(clear=True) == 0


def test_logits_far_apart_across_runs():
    """A conversation's rows over many CTAs, the largest logits in the last, the
    first, or one piece: joined, they are the plain form's."""
    for seed, at in ((31, 4900), (32, 5), (33, 2500)):
        t, table, lens, _ = make_step(seed, 1, 4, 1, 64, 0, (5000,), 64)
        for r in range(at, at + 40):
            t["k_pages"][table[0, r // 64], r % 64] *= 12
        check_step(t, table, lens)
