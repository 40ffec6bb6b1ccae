"""How exact the weights and outputs over a paged cache are: bounds that leave no
room for a term of a query, or of a softmax weight, fewer than the calls state;
each bound against forms with a term fewer first, on the CPU."""
import numpy as np
import pytest
import torch

from tests.paged_reference import HALF_BF16, rope
from trained_kv_prefix_gb300 import cartattn as ca
from trained_kv_prefix_gb300 import synth

F24 = 2.0 ** -24
ANGLE = 2e-7        # of a sine or cosine by sincospif on the reduced angle


def bf16(x):
    return torch.from_numpy(np.asarray(x, np.float64)).to(torch.bfloat16)


def f64(x):
    return synth.f64(x)


def terms(x, n):
    """x as n bf16 terms, each what those before leave, rounded."""
    out, left = np.zeros_like(x), x
    for _ in range(n):
        t = f64(bf16(left))
        out, left = out + t, left - t
    return out


# ------------------------------------------------- queries in three terms ----
# Keys of one element, a power of two, so that a logit is one element of the
# rotated query times it: products and sums are exact but for the query itself.
KEY, SCALE, CONVERSATIONS = 32.0, 0.125, 12


def make_keys(rng, n, d):
    k = np.zeros((n, d))
    k[np.arange(n), rng.permutation(np.arange(n) % d)] = KEY * rng.choice([-1, 1], size=n)
    return k


def logit_error(q, x, base):
    """Of the logits x = SCALE * k . R(pos) q, taken relative to `base`: the
    angles' error and the two roundings of a rotation on both elements of a pair
    (2 * 2^-24), three terms (2^-24 of them), the product's three sums and the
    scaling, and those of the exponent (eight roundings or cuts, 2^-23 of its
    parts).  The exponential's own error, 2^-22, is the caller's."""
    h = q.shape[-1] // 2
    pair = np.abs(q[..., :h]) + np.abs(q[..., h:])
    worst = SCALE * KEY * np.concatenate([pair, pair], -1) * (ANGLE + 3 * F24)
    return worst, (np.abs(x) + np.abs(base)) * 8 * 2 * F24


def weigh_case(seed, d):
    rng = np.random.default_rng(seed)
    B, H, p, rows = CONVERSATIONS, 2, d, 2 * d
    t = dict(q=bf16(rng.standard_normal((B, 1, H, d)) * 1.5),
             kc=bf16(np.stack([make_keys(rng, p, d) for _ in range(H)], 1)),
             k_pages=bf16(np.stack([make_keys(rng, B * rows, d) for _ in range(H)], 1)
                          .reshape(B * rows // 32, 32, H, d)))
    lse = (rng.standard_normal((B, H, 1)) + 3).astype(np.float32)
    return t, lse, rng.integers(0, 5000, size=B), rows


def weigh_plain(t, lse, pos, rows, cut=lambda q: q):
    """(weights of the cartridge's and the private rows, their bound), one query."""
    q, kc, kp = (f64(t[n]) for n in ("q", "kc", "k_pages"))
    B, _, H, d = q.shape
    kp = kp.reshape(B, rows, H, d)
    w, off = np.zeros((B, H, kc.shape[0] + rows)), np.zeros((B, H, kc.shape[0] + rows))
    for b in range(B):
        for h in range(H):
            k = np.concatenate([kc[:, h], kp[b, :, h]])
            x = SCALE * k @ cut(rope(q[b, 0, h], int(pos[b])))
            w[b, h] = np.exp(x - lse[b, h, 0])
            of_q, of_sums = logit_error(q[b, 0, h], x, lse[b, h, 0])
            off[b, h] = w[b, h] * (np.expm1((np.abs(k) / KEY) @ of_q + of_sums) + 2.0 ** -22)
    return w, off


@pytest.mark.parametrize("d", [64, 128])
def test_bound_of_weights_tells_two_terms_from_three(d):
    c = weigh_case(d, d)
    w, off = weigh_plain(*c)
    assert (np.abs(weigh_plain(*c, cut=lambda q: terms(q, 3))[0] - w) <= off).all()
    assert (np.abs(weigh_plain(*c, cut=lambda q: terms(q, 2))[0] - w) > 2 * off).any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_weights_have_all_bits_of_their_queries(d):
    t, lse, pos, rows = weigh_case(d, d)
    B, H = CONVERSATIONS, 2
    table = torch.arange(B * rows // 32, dtype=torch.int32, device="cuda").view(B, -1)
    gw, gc = ca.cart_attn_weights(
        t["q"].cuda(), torch.from_numpy(lse).cuda(), t["kc"].cuda(), t["k_pages"].cuda(), table,
        torch.full((B,), rows, dtype=torch.int32, device="cuda"), torch.zeros(B, H, rows, device="cuda"),
        pos=torch.tensor(pos, dtype=torch.int32, device="cuda"), scale=SCALE)
    assert ca.device_status(clear=True) == 0
    w, off = weigh_plain(t, lse, pos, rows)
    assert (np.abs(np.concatenate([f64(gc), f64(gw)], -1) - w) <= off).all()


def step_weights_plain(t, pos, rows, cut=lambda q: q):
    """Weights of cached rows whose new token's key is 0, and their bound."""
    q, kp = f64(t["q"])[:, 0], f64(t["k_pages"])
    B, H, d = q.shape
    kp = kp.reshape(B, rows, H, d)
    w, off = np.zeros((B, H, rows)), np.zeros((B, H, rows))
    for b in range(B):
        for h in range(H):
            x = np.append(SCALE * kp[b, :, h] @ cut(rope(q[b, h], int(pos[b]))), 0.0)
            top = x.max()
            e = np.exp(x - top)
            total = top + np.log(e.sum())
            of_q, of_sums = logit_error(q[b, h], x, total)
            each = np.append((np.abs(kp[b, :, h]) / KEY) @ of_q, 0.0) + of_sums
            # the log-sum-exp is off by its logits' errors, weighed, and by the
            # roundings of a few joins (16 * 2^-23)
            rel = np.expm1(each + (e * each).sum() / e.sum() + 32 * F24) + 2.0 ** -22
            w[b, h], off[b, h] = (e / e.sum())[:-1], (e / e.sum() * rel)[:-1]
    return w, off


def step_case(d):
    t, _, pos, rows = weigh_case(d + 7, d)
    return t, pos, rows


@pytest.mark.parametrize("d", [64, 128])
def test_bound_of_step_weights_tells_two_terms_from_three(d):
    c = step_case(d)
    w, off = step_weights_plain(*c)
    assert (np.abs(step_weights_plain(*c, cut=lambda q: terms(q, 3))[0] - w) <= off).all()
    assert (np.abs(step_weights_plain(*c, cut=lambda q: terms(q, 2))[0] - w) > 1.5 * off).any()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_step_weights_have_all_bits_of_their_queries(d):
    t, pos, rows = step_case(d)
    B, H, pages = CONVERSATIONS, 2, CONVERSATIONS * rows // 32
    own = rows // 32
    table = torch.full((B, own + 1), -1, dtype=torch.int32)
    table[:, :own] = torch.arange(pages, dtype=torch.int32).view(B, own)
    table[:, own] = torch.arange(pages, pages + B, dtype=torch.int32)   # the new rows'
    kp = torch.cat([t["k_pages"], torch.zeros(B, 32, H, d, dtype=torch.bfloat16)]).cuda()
    none = torch.zeros(0, H, d, dtype=torch.bfloat16, device="cuda")
    new = torch.zeros(B, H, d, dtype=torch.bfloat16, device="cuda")
    w = torch.zeros(B, H, rows + 32, device="cuda")
    ca.cart_attn_decode_paged(t["q"][:, 0].contiguous().cuda(), new, new, none, none, kp,
                              torch.zeros_like(kp), table.cuda(),
                              torch.full((B,), rows, dtype=torch.int32, device="cuda"),
                              pos=torch.tensor(pos, dtype=torch.int32, device="cuda"), weights=w,
                              scale=SCALE)
    assert ca.device_status(clear=True) == 0
    want, off = step_weights_plain(t, pos, rows)
    assert (np.abs(f64(w)[..., :rows] - want) <= off).all()


# ---------------------------------------------- softmax weights in two terms ----
# Small logits, so that outputs are means of values, many near 0, and what is left
# is the rounding of the weights and of the output.
OUTPUTS = [
    # id, B, Hq, Hkv, d, p, lens
    ("rows", 4, 8, 2, 64, 0, (2, 7, 40, 130)),
    ("rows_d128_g8", 3, 16, 2, 128, 0, (3, 33, 70)),
    ("rows_h4", 3, 16, 4, 128, 0, (3, 33, 70)),
    ("rows_one_head", 3, 5, 1, 64, 0, (9, 33, 150)),
    ("cartridge", 3, 8, 2, 64, 40, (0, 0, 0)),
    ("cartridge_d128", 3, 8, 2, 128, 130, (0, 0, 0)),
    ("both", 3, 14, 2, 128, 70, (0, 20, 64)),
]


def output_case(case):
    _, B, Hq, Hkv, d, p, lens = case
    rng = np.random.default_rng(B + d + p)
    make = lambda *shape, std=1.0: f64(bf16(rng.standard_normal(shape) * std))  # noqa: E731
    n = max(lens)
    return dict(q=make(B, Hq, d, std=0.1), k_new=make(B, Hkv, d, std=0.1), v_new=make(B, Hkv, d),
                kc=make(p, Hkv, d, std=0.1), vc=make(p, Hkv, d), k=make(B, n, Hkv, d, std=0.1),
                v=make(B, n, Hkv, d))


def output_plain(case, t, cut=lambda e: e):
    """(o, its bound): `cut` is how the weights of cached rows enter, relative to
    the largest.  The bound: a weight's error from the logits' (queries in two
    terms, 2^-16, angles and f32 sums), the new key's rounding, the weight's two
    terms (2^-15 of it: what the first leaves, at most 2^-7 of it, rounded) and
    f32 sums of so many products, then the output's rounding."""
    _, B, Hq, Hkv, d, p, lens = case
    G, o, off = Hq // Hkv, np.zeros((B, Hq, d)), np.zeros((B, Hq, d))
    for b, n in enumerate(lens):
        for h in range(Hq):
            g = h // G
            kn, qr = rope(t["k_new"][b, g], p + n), rope(t["q"][b, h], p + n)
            k = np.concatenate([t["kc"][:, g], t["k"][b, :n, g], kn[None]])
            v = np.concatenate([t["vc"][:, g], t["v"][b, :n, g], t["v_new"][b, g][None]])
            x = k @ qr / np.sqrt(d)
            e = np.exp(x - x.max())
            each = np.abs(k) @ np.abs(qr) / np.sqrt(d) * (HALF_BF16 ** 2 + 5e-6)
            each[-1] += np.abs(kn) @ np.abs(qr) / np.sqrt(d) * HALF_BF16
            rel = np.expm1(each + (e * each).sum() / e.sum()) + 2.0 ** -15 + (len(x) + 16) * 2 * F24
            o[b, h] = np.append(cut(e[:-1]), e[-1]) @ v / e.sum()
            s = (e * rel) @ np.abs(v) / e.sum()
            off[b, h] = s + HALF_BF16 * (np.abs(e @ v / e.sum()) + s)
    return o, off


def two_terms(e):
    y = torch.from_numpy((e * (1 - F24)).astype(np.float32))
    first = f64((y.view(torch.int32) & -65536).view(torch.float32))
    return first + f64(bf16(e - first))


@pytest.mark.parametrize("case", OUTPUTS, ids=[c[0] for c in OUTPUTS])
def test_bound_of_outputs_tells_one_term_from_two(case):
    t = output_case(case)
    o, off = output_plain(case, t)
    two = f64(bf16(output_plain(case, t, two_terms)[0]))
    assert (np.abs(two - o) <= off).all()
    one = f64(bf16(output_plain(case, t, lambda e: f64(bf16(e)))[0]))
    assert (np.abs(one - o) > 1.5 * off).any()


@pytest.mark.gpu
@pytest.mark.parametrize("case", OUTPUTS, ids=[c[0] for c in OUTPUTS])
def test_outputs_have_the_bits_of_their_weights(case):
    _, B, Hq, Hkv, d, p, lens = case
    t = output_case(case)
    P, pages = 16, max(lens) // 16 + 1
    pool = lambda x: torch.cat([bf16(x), torch.zeros(B, pages * P - x.shape[1], Hkv, d,  # noqa: E731
                                                     dtype=torch.bfloat16)], 1) \
        .view(B * pages, P, Hkv, d).contiguous().cuda()
    g = {n: bf16(t[n]).cuda() for n in ("q", "k_new", "v_new", "kc", "vc")}
    o = ca.cart_attn_decode_paged(
        g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], pool(t["k"]), pool(t["v"]),
        torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages),
        torch.tensor(lens, dtype=torch.int32, device="cuda"))
    assert ca.device_status(clear=True) == 0
    want, off = output_plain(case, t)
    assert (np.abs(f64(o) - want) <= off).all()


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
def test_infinite_values_stay_infinite(d):
    """Weights that one bf16 holds (all keys equal) and others: neither term of a
    weight is 0, so that an infinite value, of a row or the cartridge, is what
    every query that sees it gets."""
    rng = np.random.default_rng(3)
    for std in (0.0, 0.5):
        case = ("", 2, 4, 2, d, 9, (5, 5))
        t = output_case(case)
        t["q"] = t["q"] * std * 10
        g = {n: bf16(t[n]).cuda() for n in ("q", "k_new", "v_new", "kc", "vc")}
        kp, vp = (bf16(rng.standard_normal((2, 16, 2, d))).cuda() for _ in range(2))
        vp[0, 2, 1, 7] = float("inf")
        g["vc"][4, 0, 3] = float("-inf")
        o = ca.cart_attn_decode_paged(g["q"], g["k_new"], g["v_new"], g["kc"], g["vc"], kp, vp,
                                      torch.tensor([[0], [1]], dtype=torch.int32, device="cuda"),
                                      torch.tensor([5, 5], dtype=torch.int32, device="cuda"))
        o = f64(o)
        assert (o[0, 2:, 7] == np.inf).all() and (o[:, :2, 3] == -np.inf).all()
        o[0, 2:, 7] = o[:, :2, 3] = 0
        assert np.isfinite(o).all()
