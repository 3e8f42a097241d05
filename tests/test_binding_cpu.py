"""What the Python binding refuses before an address reaches the library.
Engines and caches here have no device memory: a refused call touches none."""
import shutil
import os

import pytest
import torch

pytestmark = pytest.mark.skipif(not (shutil.which("nvcc") or os.path.exists("/usr/local/cuda/bin/nvcc")),
                                reason="nvcc not available")


@pytest.fixture(scope="module")
def B():
    from kv_cache_token_gb300 import build
    build.build()
    from kv_cache_token_gb300 import binding
    return binding


def config(B, **kw):
    f = dict(policy=B.H2O, num_layers=1, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, kv_dtype=B.BF16,
             blocks_per_pool=8, max_tokens=16, budget=8, recent_window=2, obs_window=1, pool_kernel=1)
    f.update(kw)
    return B.config_from(**f)


def bare_engine(B, **kw):
    """An engine without buffers: enough for argument checks."""
    import ctypes
    e = B.Engine.__new__(B.Engine)
    e.cfg, e.device, e.h = config(B, **kw), torch.device("cuda", 0), None
    e.lanes = e.cfg.batch * e.cfg.num_kv_heads
    e.kv_dtype = torch.bfloat16
    e.kv4_geometry = B.kv4_geometry(e.cfg, e.device)
    e.kv4_scratch_bytes = B.lib().kvevict_kv4_scratch_bytes(ctypes.byref(e.cfg))
    return e


def bare_cache(B, eng):
    c = B.Kv4Cache.__new__(B.Kv4Cache)
    c.geometry, c.scratch_bytes, c.ref = eng.kv4_geometry, eng.kv4_scratch_bytes, "ref"
    return c


@pytest.mark.parametrize("other", [dict(batch=3), dict(batch=1), dict(num_kv_heads=4), dict(head_dim=64),
                                   dict(batch=16, num_q_heads=16, num_kv_heads=8)])
def test_a_cache_of_another_engine_is_refused(B, other):
    mine, their = bare_engine(B), bare_engine(B, **other)
    c = bare_cache(B, their)
    assert their._cache_ref(c, their.kv4_scratch_bytes) == "ref"
    k = torch.zeros((2, 2, 4, 128), dtype=torch.bfloat16)
    q, lens = torch.zeros((2, 8, 128), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: mine.kv4_write(c, None, k, k), lambda: mine.kv4_pack(0, c), lambda: mine.kv4_read(c, None, 4, k=k, v=k),
                 lambda: mine.kv4_attend(c, lens, q)):
        with pytest.raises(ValueError, match="cache was made for"):
            call()


def test_a_larger_group_may_not_attend_on_a_smaller_scratch(B):
    small, large = bare_engine(B, num_q_heads=4), bare_engine(B, num_q_heads=16)
    assert small.kv4_geometry == large.kv4_geometry and small.kv4_scratch_bytes < large.kv4_scratch_bytes
    c = bare_cache(B, small)
    q, lens = torch.zeros((2, 16, 128), dtype=torch.bfloat16), torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="scratch"):
        large.kv4_attend(c, lens, q)
    # storing and reading need no scratch, and a smaller group fits a larger one's
    assert large._cache_ref(c) == "ref"
    assert small._cache_ref(bare_cache(B, large), small.kv4_scratch_bytes) == "ref"


def test_a_cache_on_another_device_is_refused(B):
    a, b = bare_engine(B), bare_engine(B)
    b.device = torch.device("cuda", 1)
    b.kv4_geometry = B.kv4_geometry(b.cfg, b.device)
    with pytest.raises(ValueError, match="cache was made for"):
        a.kv4_pack(0, bare_cache(B, b))


class _Recorder:
    """Stands in for torch in the binding: allocations are real (on the CPU)
    and noted with the stream that was current."""

    def __init__(self):
        self.current, self.made, self.users = "main", [], []
        self.cuda = self

    def __getattr__(self, name):
        return getattr(torch, name)

    def stream(self, s):
        import contextlib

        @contextlib.contextmanager
        def on():
            before, self.current = self.current, s
            yield
            self.current = before
        return on()

    def current_stream(self, device=None):
        return self.current

    def _make(self, t):
        self.made.append((self.current, t))
        t.record_stream = self.users.append
        return t

    def empty(self, shape, dtype=None, device=None):
        return self._make(torch.empty(shape, dtype=dtype))

    def zeros(self, shape, dtype=None, device=None):
        return self._make(torch.zeros(shape, dtype=dtype))

    def full(self, shape, value, dtype=None, device=None):
        return self._make(torch.full(shape, value, dtype=dtype))


class _Stream:
    cuda_stream = 7


@pytest.mark.parametrize("call, outputs", [
    (lambda e, c, t, s: e.norm_rope(t(2, 3, 12 * 128), stream=s), 3),
    (lambda e, c, t, s: e.attend_prompt(t(2, 8, 3, 128), t(2, 2, 3, 128), t(2, 2, 3, 128), stream=s), 2),
    (lambda e, c, t, s: e.kv4_read(c, None, 4, stream=s), 2),
    (lambda e, c, t, s: e.kv4_attend(c, torch.zeros(4, dtype=torch.int32), t(2, 8, 128), stream=s), 2),
    (lambda e, c, t, s: e.decode_step(0, t(2, 8, 128), t(2, 2, 128), t(2, 2, 128), 0, stream=s), 2),
    (lambda e, c, t, s: e.finish_step(0, t(2, 8, 128), t(2, 2, 128), t(2, 2, 128), 0, stream=s), 2),
    (lambda e, c, t, s: e.attend_static(0, t(2, 8, 128), t(2, 2, 128), t(2, 2, 128), stream=s), 2),
    (lambda e, c, t, s: e.score(0, t(2, 8, 4, 128), torch.zeros(4, dtype=torch.int32), stream=s), 3),
    (lambda e, c, t, s: e.score_mass(0, t(2, 8, 4, 128), torch.zeros(4, dtype=torch.int32), 0, stream=s), 2),
    (lambda e, c, t, s: e.select(torch.zeros(4, 16), torch.zeros((4, 16), dtype=torch.int32),
                                 torch.zeros(4, dtype=torch.int32), 8, 2, stream=s), 2),
    (lambda e, c, t, s: e.compact(0, None, None, stream=s), 4),
    (lambda e, c, t, s: e.relocate(0, stream=s), 4),
    (lambda e, c, t, s: e.stats(0, stream=s), 1)])
def test_default_outputs_belong_to_the_calls_stream(B, monkeypatch, call, outputs):
    """Outputs that a call makes itself are allocated and filled on the stream
    its kernel runs on: a fill on another one may land after the kernel."""
    import types
    e = bare_engine(B)
    c = bare_cache(B, e)
    e.device = types.SimpleNamespace(index=-1)          # tensors of this test are the CPU's
    e.victims = e.n_victims = torch.zeros(4, dtype=torch.int32)
    rec, s = _Recorder(), _Stream()

    class Lib:
        def __getattr__(self, name):
            return lambda *a: 0
    monkeypatch.setattr(B, "torch", rec)
    monkeypatch.setattr(B, "lib", lambda: Lib())
    call(e, c, lambda *shape: torch.zeros(shape, dtype=torch.bfloat16), s)
    assert len(rec.made) == outputs
    assert all(on is s for on, _ in rec.made)
    assert rec.users == ["main"] * outputs              # and kept while the current stream may read them


@pytest.mark.parametrize("big", [2 ** 31, 2 ** 32, 2 ** 32 + 5, -2 ** 31 - 1, 2 ** 63])
def test_integers_past_int32_are_refused(B, monkeypatch, big):
    """ctypes passes the low 32 bits of an integer: a window of 2^32 + 5 would
    have been 5."""
    import types
    e = bare_engine(B)
    c = bare_cache(B, e)
    e.device = types.SimpleNamespace(index=-1)
    seen = []

    class Lib:
        def __getattr__(self, name):
            return lambda *a: seen.append(name) or 0
    monkeypatch.setattr(B, "lib", lambda: Lib())
    t = lambda *shape: torch.zeros(shape, dtype=torch.bfloat16)
    x, q, k, lens = t(2, 3, 12 * 128), t(2, 8, 3, 128), t(2, 2, 3, 128), torch.zeros(4, dtype=torch.int32)
    out, lse = t(2, 3, 8, 128), torch.zeros(2, 8, 3)
    ro, ao, al, s = dict(q=t(2, 8, 3, 128), k=t(2, 2, 3, 128), v=t(2, 2, 3, 128)), t(2, 8, 128), torch.zeros(2, 8), _Stream()
    calls = [lambda v: e.norm_rope(x, pos0=v, stream=s, **ro), lambda v: e.norm_rope(x, rotary_dim=v, stream=s, **ro),
             lambda v: e.attend_prompt(q, k, k, sinks=v, out=out, lse=lse, stream=s),
             lambda v: e.attend_prompt(q, k, k, window=v, out=out, lse=lse, stream=s),
             lambda v: e.kv4_attend(c, lens, t(2, 8, 128), sinks=v, out=ao, lse=al, stream=s),
             lambda v: e.kv4_attend(c, lens, t(2, 8, 128), window=v, out=ao, lse=al, stream=s),
             lambda v: e.kv4_pack(v, c, stream=s)]
    for call in calls:
        with pytest.raises(ValueError, match="int32"):
            call(big)
    assert seen == []
    for call in calls:
        call(2 ** 31 - 1)
        call(-2 ** 31)
    assert len(seen) == 2 * len(calls)      # the library's own checks see these
