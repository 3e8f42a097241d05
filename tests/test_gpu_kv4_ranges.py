"""The 4-bit cache and its attention at the ends of their inputs' ranges."""
import numpy as np
import pytest
import torch

from oracle import serving as S
from tests import test_gpu_kv4 as T4

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("top", [99, 101, 103, 104, 110, 117, 118, 121, 124, 126, 127])
def test_attend_queries_up_to_the_largest_number(d, top):
    """Queries of 2^top against keys as small: logits of ordinary size, exact
    in every step (one element of a head is not zero, keys are whole steps of
    their scale), so out and lse follow the general bound without its cuts:
    half a bf16 step, 2^-9 of sum p|v| for weights in fp16, 2^-20 (1 + |lse|)."""
    eng = T4.engine(1, 4, 2, d)
    n = 90
    g = torch.Generator(device="cuda").manual_seed(top)
    step = 2.0 ** (2 - top)
    k = torch.zeros((2, n, d), device="cuda")
    k[..., 5] = torch.randint(-7, 8, (2, n), generator=g, device="cuda").float() * step
    k[..., 6] = 7 * step                                 # the group's scale is one step
    v = torch.randn((2, n, d), generator=g, device="cuda")
    q = torch.zeros((1, 4, d), device="cuda")
    q[..., 5] = torch.tensor([1.0, -1.0, 1.5, -0.25], device="cuda") * 2.0 ** top
    k, v, q = k.bfloat16(), v.bfloat16(), q.bfloat16()
    assert torch.isfinite(q).all() and (k[..., 6] == 7 * step).all()
    c = T4.shuffled(eng, 6)
    eng.kv4_write(c, None, T4.shape4(eng, k), T4.shape4(eng, v))
    hk, hv = T4.held(k, v)
    out, lse = eng.kv4_attend(c, T4.ints(eng, [n, n - 7]), q)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    for l, m in enumerate((n, n - 7)):
        hs = slice(2 * l, 2 * l + 2)
        o, ls, mag, _ = S.attend_rows(T4.host(q)[0, hs], hk[l, :m], hv[l, :m])
        assert np.abs(ls).max() < 60
        # codes as subnormals cut the value products: 17 * (2^-15 + 2^-18) units of p * scale (see test_gpu_kv4)
        unit = 17 * (2.0 ** -15 + 2.0 ** -18) / 6.97 * np.abs(hv[l, :m]).max()
        assert (np.abs(T4.host(out)[0, hs] - o) <= 2.0 ** -8 * np.abs(o) + 2.0 ** -9 * mag + unit).all()
        assert (np.abs(T4.host(lse)[0, hs] - ls) <= 2.0 ** -20 * (1 + np.abs(ls))).all()
    assert eng.last_error()[0] == 0


@pytest.mark.parametrize("d", [64, 128])
def test_pack_stores_no_other_tokens_row_for_a_slot_out_of_range(d):
    """Table entries outside the pool: those tokens hold NaN and are reported;
    the others, and lanes without such entries, are as always."""
    n = 70
    eng = T4.engine(2, 4, 2, d, blocks_per_pool=30, max_tokens=100, budget=90, recent_window=8)
    k, v = T4.rows(4, n, d, 1), T4.rows(4, n, d, 2)
    eng.prefill(0, T4.shape4(eng, k), T4.shape4(eng, v))
    bad = {0: [0, 17, 69], 2: [31, 32, 33]}
    rows = eng.cfg.blocks_per_pool * 16
    for lane, at in bad.items():
        eng.slots[0, lane, at] = torch.tensor([-1, rows, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    c = T4.shuffled(eng, 6)
    eng.kv4_pack(0, c)
    assert eng.last_error()[0] == 9
    got = eng.kv4_read(c, None, n, lens=eng.counts[0])
    for g, ref in zip(got, T4.held(k, v)):
        g = T4.host(g).reshape(4, n, d)
        for lane in range(4):
            gone = np.zeros(n, bool)
            gone[bad.get(lane, [])] = True
            assert np.isnan(g[lane, gone]).all()
            np.testing.assert_array_equal(g[lane, ~gone], S.bf16(ref[lane, ~gone]))
    q = torch.randn((2, 4, d), device="cuda").bfloat16()
    out, lse = eng.kv4_attend(c, eng.counts[0], q)
    assert out[:, :2].isnan().all() and lse[:, :2].isnan().all()          # lanes 0 and 2
    assert torch.isfinite(out[:, 2:]).all() and torch.isfinite(lse[:, 2:]).all()
    # a count out of range leaves its lane
    before = c.pages.clone()
    eng.counts[0] = torch.tensor([-1, 101, n, 0], dtype=torch.int32)
    eng.kv4_pack(0, c)
    assert eng.last_error()[0] == 9
    changed = set((c.pages != before).any(1).nonzero().flatten().tolist())
    assert changed <= set(c.table[2, :5].tolist())
