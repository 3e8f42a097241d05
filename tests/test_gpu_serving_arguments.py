"""Arguments of the calls around the eviction that a kernel must never see."""
import ctypes

import pytest
import torch

from kv_cache_token_gb300 import BF16, Engine, H2O, config_from, lib

pytestmark = pytest.mark.gpu


def engine(**kw):
    f = dict(policy=H2O, num_layers=1, batch=2, num_q_heads=4, num_kv_heads=2, head_dim=64, kv_dtype=BF16,
             blocks_per_pool=4, max_tokens=8, budget=4, recent_window=2, obs_window=1, pool_kernel=1)
    f.update(kw)
    eng = Engine(config_from(**f))
    eng.reset()
    return eng


def test_misaligned_arrays_of_words_are_refused():
    """Positions, starts, lengths and log-sum-exps off a 4-byte boundary."""
    eng = engine()
    L = lib()
    P = lambda t, off=0: ctypes.c_void_p(t.data_ptr() + off)
    rows = lambda h, n: torch.zeros((2, h, n, 64), dtype=torch.bfloat16, device="cuda")
    q, k, v, out = rows(4, 3), rows(2, 3), rows(2, 3), torch.empty((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    ints = torch.zeros((64,), dtype=torch.int32, device="cuda")
    f = torch.zeros((64,), dtype=torch.float32, device="cuda")
    qkv = torch.zeros((2, 3, 8 * 64), dtype=torch.bfloat16, device="cuda")
    c = eng.kv4_cache(4, 1)
    rope = lambda pos: L.kvevict_norm_rope(eng.h, P(qkv), 3 * 512, 512, 3, None, None, 1e-6, pos, 0, 64, 1e4, 0, P(q), P(k),
                                           P(v), None)
    prompt = lambda lse: L.kvevict_attend_prompt(eng.h, P(q), P(k), P(v), 3, 0, 0, P(out), lse, None)
    write = lambda st: L.kvevict_kv4_write(eng.h, c.ref, st, 3, P(k), P(v), None)
    read = lambda st, ln: L.kvevict_kv4_read(eng.h, c.ref, st, ln, 3, P(k), P(v), None)
    attend = lambda ln, lse: L.kvevict_kv4_attend(eng.h, c.ref, ln, P(q), 0, 0, P(out), lse, None)
    torch.cuda.synchronize()
    for off in (1, 2, 3):
        assert rope(P(ints, off)) == 1
        assert prompt(P(f, off)) == 1
        assert write(P(ints, off)) == 1
        assert read(P(ints, off), None) == 1 and read(None, P(ints, off)) == 1
        assert attend(P(ints, off), None) == 1 and attend(P(ints), P(f, off)) == 1
    for ok in (rope(P(ints, 4)), prompt(P(f, 4)), write(P(ints, 4)), read(P(ints, 4), P(ints, 8)), attend(P(ints, 4), P(f, 4))):
        assert ok == 0
    assert eng.last_error()[0] == 0
