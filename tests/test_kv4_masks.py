"""Which tokens the 4-bit cache's attention sees: lengths, windows and sinks,
under bounds narrow enough that one token more or less is outside them.

Queries are small, so every visible token has a weight of about 1 / n, and rows
have one size.  Bounds, from the scales of the groups themselves:

* a logit: the codes of a group enter two MMAs as fp16 subnormals of nominal
  exponent 2^-14, of which a code is 2^-8; 16 products and a running sum are 17
  cuts below 2^-23 of the largest, 17 * 2^-15 units of the group's scale times
  its largest |q|, twice a group; and 2^-18 of sum |q||k| / sqrt d for its fp32
  sums (four groups, scale, exponent: under 2^6 roundings of 2^-24);
* lse: a logit's, and 2^-20 (1 + |lse|) for fp32 logarithms and sums;
* out: its rounding to bf16, 2^-8 |o|; weight and weight times scale in fp16,
  2^-11 each, and fp32 sums, 2^-9 of sum p|v|; twice a logit's bound (the weight
  and the sum of weights) of sum p|v|; 17 cuts a tile as above of sum p scale,
  and 17 * 2^-18 for the running sum over at most two tiles a warp (see
  test_gpu_kv4); what the weights' fp16 grid ends at, n * 3.1 * 2^-33 of max p|v|.
"""
import numpy as np
import pytest
import torch

from oracle import serving as S

# (longest lane, sinks, window): none; inside a page, at its ends, past it; sinks
# that meet the window, that pass the lane; windows of one, of all, of more
CASES = [(1, 0, 0), (2, 1, 1), (15, 0, 0), (16, 0, 0), (17, 0, 0), (33, 0, 1), (33, 1, 16), (48, 16, 16), (64, 15, 17),
         (100, 3, 97), (100, 4, 96), (100, 4, 95), (100, 300, 5), (100, 3, 1000), (300, 0, 0), (300, 4, 33), (300, 0, 16),
         (300, 17, 1), (300, 0, 272), (290, 33, 129)]
HEADS = [(1, 1, 1), (2, 3, 1), (1, 16, 2), (1, 16, 1)]       # batch, query heads, KV heads


def visible(n, sinks, window):
    i = np.arange(n)
    return (i < sinks) | (i >= n - window) if window else np.ones(n, bool)


def make(d, batch, hq, hkv, top):
    rng = np.random.default_rng(1000 * top + 10 * hq + d)
    lanes = batch * hkv
    K, V = (S.bf16(rng.normal(size=(lanes, top, d)).astype(np.float32)) for _ in (0, 1))
    q = S.bf16((0.3 * rng.normal(size=(batch, hq, d))).astype(np.float32))
    lens = rng.integers(max(0, top - 20), top + 1, lanes)
    lens[-1] = top
    return K, V, q, [int(n) for n in lens]


def scales(x):
    return S.bf16((np.abs(x.reshape(x.shape[:-1] + (-1, 32))).max(-1)).astype(np.float32) / np.float32(7))


def expected(q, K, V, see):
    """Values and bounds of heads q [g, d] over the rows of K and V that `see`
    marks: out, its bound, lse, its bound."""
    d = q.shape[1]
    hk, hv = S.quantise(K, False)[see], S.quantise(V, True)[see]
    o, lse, mag, _ = S.attend_rows(q, hk, hv)
    if not see.any():
        return o, np.zeros_like(o), lse, np.zeros_like(lse)
    ks, vs = scales(K[see]), scales(V[see])
    qmax = np.abs(q.reshape(q.shape[0], -1, 32)).max(-1)
    logit = 34 * 2.0 ** -15 * (qmax @ ks.T) / np.sqrt(d) + 2.0 ** -18 * (np.abs(q) @ np.abs(hk).T) / np.sqrt(d)
    cut = logit.max(1)
    p = np.exp(q @ hk.T / np.sqrt(d) - lse[:, None])
    unit = 17 * (2.0 ** -15 + 2.0 ** -18) * np.repeat(p @ vs, 32, axis=1)
    floor = 2.0 ** -134 + len(hk) * 3.1 * 2.0 ** -33 * (p * np.abs(hv).max(1)).max(1, keepdims=True)
    return (o, 2.0 ** -8 * np.abs(o) + (2.0 ** -9 + 2 * cut[:, None]) * mag + unit + floor,
            lse, cut + 2.0 ** -20 * (1 + np.abs(lse)))


def inside(got, ref, bound):
    with np.errstate(invalid="ignore"):
        return bool((np.abs(got - ref) <= bound).all())


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch, hq, hkv", HEADS)
@pytest.mark.parametrize("top, sinks, window", CASES)
def test_one_token_more_or_less_is_outside_the_bounds(d, batch, hq, hkv, top, sinks, window):
    """The bounds themselves, on the host: any visible token left out, and any
    token next to the visible ones let in, is seen in every head's lse or out."""
    K, V, q, lens = make(d, batch, hq, hkv, top)
    g = hq // hkv
    for l in range(batch * hkv):
        b, h = divmod(l, hkv)
        n, qh = lens[l], q[b, h * g:(h + 1) * g]
        see = np.zeros(top, bool)
        see[:n] = visible(n, sinks, window)
        o, ob, lse, lb = expected(qh, K[l], V[l], see)
        edges = [i for i in range(top) if not see[i] and (see[max(0, i - 1)] or see[min(top - 1, i + 1)])]
        some = np.flatnonzero(see)
        for i in edges + list(some if len(some) < 40 else some[[0, 1, -1, -2, *range(2, len(some) - 2, 7)]]):
            other = see.copy()
            other[i] = not other[i]
            if not other.any() or not see.any():
                continue
            o2, _, lse2, _ = expected(qh, K[l], V[l], other)
            for e in range(g):
                assert not (inside(o2[e], o[e], ob[e]) and inside(lse2[e], lse[e], lb[e])), (l, i, e)


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("batch, hq, hkv", HEADS)
@pytest.mark.parametrize("top, sinks, window", CASES)
def test_attend_sees_just_the_visible_tokens(d, batch, hq, hkv, top, sinks, window):
    from tests import test_gpu_kv4 as T4
    K, V, q, lens = make(d, batch, hq, hkv, top)
    eng = T4.engine(batch, hq, hkv, d)
    c = T4.shuffled(eng, (top + 15) // 16 + 1, seed=top)
    bf = lambda x: torch.from_numpy(x).to("cuda", torch.bfloat16)
    # every lane holds `top` tokens: those past its length are as fit to be seen as its own
    eng.kv4_write(c, None, T4.shape4(eng, bf(K)), T4.shape4(eng, bf(V)))
    out, lse = eng.kv4_attend(c, T4.ints(eng, lens), bf(q), sinks=sinks, window=window)
    out, lse = T4.host(out), T4.host(lse)
    g = hq // hkv
    for l in range(eng.lanes):
        b, h = divmod(l, hkv)
        hs = slice(h * g, (h + 1) * g)
        see = np.zeros(top, bool)
        see[:lens[l]] = visible(lens[l], sinks, window)
        o, ob, ls, lb = expected(q[b, hs], K[l], V[l], see)
        assert inside(out[b, hs], o, ob), (l, np.abs(out[b, hs] - o).max(), ob.max())
        if see.any():
            assert inside(lse[b, hs], ls, lb), (l, lse[b, hs], ls, lb)
        else:
            assert (lse[b, hs] == -np.inf).all()
    assert eng.last_error()[0] == 0
