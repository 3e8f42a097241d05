"""The rotation's angles at any int32 position, from rows that show them.

A pair (1, 0) turns into (cos t, sin t) without another rounding in fp32, so the
bound is that of the sine or cosine, an ulp of at most 2^-24, and of the angle:
2^-28 turn for its rounding, 2^-32 for the bits cut off, 2^-30 for the
frequency's at position 2^31 (see rope_turns.h): 2 pi (2^-28 + 2^-32 + 2^-30)
rad = 0.52 * 2^-24.  The reference is in long double (its angle is off by
2^31 * 2^-63 rad at most)."""
import numpy as np
import pytest
import torch

from tests.test_gpu_norm_rope import engine
from kv_cache_token_gb300 import F32

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("base, r", [(1e4, 128), (5e5, 128), (1e6, 96), (1.0, 16)])
def test_angles(base, r, interleaved):
    eng = engine(1, 1, 1, 128, F32)
    rng = np.random.default_rng(r)
    far = np.exp2(rng.uniform(0, 31, 4000)).astype(np.int64) * rng.choice([-1, 1], 4000)
    pos = np.clip(np.r_[0, 1, -1, 2 ** 31 - 1, -2 ** 31, far], -2 ** 31, 2 ** 31 - 1)
    n = len(pos)
    x = torch.zeros((1, n, 3 * 128), device="cuda")
    first = slice(0, r, 2) if interleaved else slice(0, r // 2)
    second = slice(1, r, 2) if interleaved else slice(r // 2, r)
    x[0, :, :128][:, first] = 1.0
    q, _, _ = eng.norm_rope(x, pos=torch.from_numpy(pos.astype(np.int32)).cuda(), rotary_dim=r, base=base,
                            interleaved=interleaved)
    got = q[0, 0].double().cpu().numpy()
    i = np.arange(r // 2).astype(np.longdouble)
    t = pos.astype(np.longdouble)[:, None] * np.longdouble(base) ** (-2 * i / r)
    bound = (1 + 0.52) * 2.0 ** -24
    for cols, ref in ((first, np.cos(t)), (second, np.sin(t))):
        err = np.abs(got[:, cols] - ref).max()
        assert err <= bound, err * 2.0 ** 24
