"""Calls on several streams: results are those of the same calls one after
another."""
import pytest
import torch

from kv_cache_token_gb300 import BF16, Engine, H2O, config_from, lib

pytestmark = pytest.mark.gpu


def decode_engine(B, Hq, Hkv, d, n, L):
    eng = Engine(config_from(policy=H2O, num_layers=L, batch=B, num_q_heads=Hq, num_kv_heads=Hkv, head_dim=d, kv_dtype=BF16,
                             blocks_per_pool=B * Hkv * ((n + 12) // 16 + 2), max_tokens=n + 12, budget=128, recent_window=32,
                             obs_window=1, pool_kernel=1))
    eng.reset()
    return eng


def test_a_cache_call_on_a_second_stream_between_projection_and_decode_step():
    """norm_rope on one stream, kv4_write of its new row on a second, the
    decode step on the first: the step reads the finished rows."""
    B, Hq, Hkv, d, n, L = 2, 16, 2, 128, 200, 2
    a, b = decode_engine(B, Hq, Hkv, d, n, L), decode_engine(B, Hq, Hkv, d, n, L)
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    for l in range(L):
        k, v = rnd(B, Hkv, n, d), rnd(B, Hkv, n, d)
        a.prefill(l, k, v)
        b.prefill(l, k, v)
    c = a.kv4_cache(B * Hkv * 2, 2)
    starts = torch.zeros((B * Hkv,), dtype=torch.int32, device="cuda")
    sq = [torch.empty((B, h, 1, d), dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for t in range(6):
        for l in range(L):
            x = rnd(B, 1, (Hq + 2 * Hkv) * d)
            q, k, v = b.norm_rope(x, pos0=n + t)
            torch.cuda.synchronize()
            ref = [r.clone() for r in b.decode_step(l, q.view(B, Hq, d), k.view(B, Hkv, d), v.view(B, Hkv, d), n + t)]
            for o in sq:
                o.zero_()
            torch.cuda.synchronize()
            a.norm_rope(x, pos0=n + t, q=sq[0], k=sq[1], v=sq[2])
            side.wait_stream(torch.cuda.current_stream())
            a.kv4_write(c, starts, sq[1], sq[2], stream=side)
            got = a.decode_step(l, sq[0].view(B, Hq, d), sq[1].view(B, Hkv, d), sq[2].view(B, Hkv, d), n + t)
            torch.cuda.synchronize()
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
            gk, gv = a.kv4_read(c, starts, 1)
            b_c = b.kv4_cache(B * Hkv * 2, 2)
            b.kv4_write(b_c, starts, k, v)
            rk, rv = b.kv4_read(b_c, starts, 1)
            assert torch.equal(gk, rk) and torch.equal(gv, rv)
    assert a.last_error()[0] == 0 and b.last_error()[0] == 0


def test_a_row_read_back_feeds_the_decode_step():
    """kv4_read's row is the new row of the decode step launched right after
    it, layer after layer."""
    B, Hq, Hkv, d, n, L = 2, 16, 2, 128, 200, 3
    a, b = decode_engine(B, Hq, Hkv, d, n, L), decode_engine(B, Hq, Hkv, d, n, L)
    g = torch.Generator(device="cuda").manual_seed(6)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    for l in range(L):
        k, v = rnd(B, Hkv, n, d), rnd(B, Hkv, n, d)
        a.prefill(l, k, v)
        b.prefill(l, k, v)
    c = a.kv4_cache(B * Hkv * 2, 2)
    k, v = rnd(B, Hkv, 24, d), rnd(B, Hkv, 24, d)
    a.kv4_write(c, None, k, v)
    kn, vn = [torch.empty((B, Hkv, 1, d), dtype=torch.bfloat16, device="cuda") for _ in (0, 1)]
    for t in range(8):
        for l in range(L):
            at = torch.full((B * Hkv,), 3 * t + l, dtype=torch.int32, device="cuda")
            q = rnd(B, Hq, d)
            rk, rv = a.kv4_read(c, at, 1)
            torch.cuda.synchronize()
            ref = [r.clone() for r in b.decode_step(l, q, rk.view(B, Hkv, d), rv.view(B, Hkv, d), n + t)]
            kn.zero_()
            vn.zero_()
            torch.cuda.synchronize()
            a.kv4_read(c, at, 1, k=kn, v=vn)
            got = a.decode_step(l, q, kn.view(B, Hkv, d), vn.view(B, Hkv, d), n + t)
            torch.cuda.synchronize()
            assert torch.equal(got[0], ref[0]) and torch.equal(got[1], ref[1])
    assert a.last_error()[0] == 0 and b.last_error()[0] == 0


def test_outputs_made_by_a_call_on_a_second_stream():
    """While the current stream is busy, calls on a second stream make their
    own outputs: nothing queued on the current one lands in them later."""
    eng = Engine(config_from(policy=H2O, num_layers=1, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, kv_dtype=BF16,
                             blocks_per_pool=4, max_tokens=8, budget=4, recent_window=2, obs_window=1, pool_kernel=1))
    eng.reset()
    g = torch.Generator(device="cuda").manual_seed(9)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    c = eng.kv4_cache(4 * 8, 8)
    k, v, q, lens = rnd(2, 2, 100, 128), rnd(2, 2, 100, 128), rnd(2, 8, 128), torch.full((4,), 100, dtype=torch.int32).cuda()
    x, pq = rnd(2, 100, 12 * 128), rnd(2, 8, 100, 128)
    eng.kv4_write(c, None, k, v)
    calls = [lambda **kw: eng.kv4_read(c, None, 100, **kw), lambda **kw: eng.kv4_attend(c, lens, q, **kw),
             lambda **kw: eng.norm_rope(x, **kw), lambda **kw: eng.attend_prompt(pq, k, v, **kw)]
    ref = [f() for f in calls]
    a = torch.randn((8192, 8192), device="cuda").bfloat16()
    side = torch.cuda.Stream()
    # blocks the allocator would hand out again while the current stream still writes them
    torch.cuda.synchronize()
    for _ in range(2):
        for _ in range(20):
            a = (a @ a).clamp_(-1, 1)
        old = [[torch.empty_like(t) for t in r] for r in ref]
        for r in old:
            for t in r:
                t.fill_(9.0)
        del old, r, t
        got = [f(stream=side) for f in calls]
        side.synchronize()
        for r, o in zip(ref, got):
            for s, t in zip(r, o):
                assert torch.equal(s, t)
        torch.cuda.synchronize()
        for r, o in zip(ref, got):
            for s, t in zip(r, o):
                assert torch.equal(s, t)
    assert eng.last_error()[0] == 0


def test_host_threads_with_bases_of_their_own():
    """Projections of several models' layers, a host thread and a stream each,
    on one engine: every call turns by its own base."""
    import ctypes
    import threading
    eng = Engine(config_from(policy=H2O, num_layers=1, batch=1, num_q_heads=4, num_kv_heads=2, head_dim=128, kv_dtype=BF16,
                             blocks_per_pool=4, max_tokens=8, budget=4, recent_window=2, obs_window=1, pool_kernel=1))
    eng.reset()
    x = torch.randn((1, 1, 8 * 128), device="cuda").bfloat16()
    bases = [(1e4, 128), (5e5, 96), (1e6, 112), (2e4, 64)]
    ref = [eng.norm_rope(x, pos0=1000, base=b, rotary_dim=r)[0].clone() for b, r in bases]
    torch.cuda.synchronize()
    assert all(not torch.equal(ref[i], ref[j]) for i in range(4) for j in range(i))
    wrong, codes, gate, call = [0] * 4, [0] * 4, threading.Barrier(4), lib().kvevict_norm_rope
    P = lambda t: ctypes.c_void_p(t.data_ptr())

    def work(i):
        s = torch.cuda.Stream()
        outs = [[torch.empty((1, h, 1, 128), dtype=torch.bfloat16, device="cuda") for h in (4, 2, 2)] for _ in range(200)]
        torch.cuda.synchronize()
        args = [(eng.h, P(x), 0, 1024, 1, None, None, 1e-6, None, 1000, bases[i][1], bases[i][0], 0, P(q), P(k), P(v),
                 ctypes.c_void_p(s.cuda_stream)) for q, k, v in outs]
        gate.wait()
        for _ in range(40):
            for a in args:
                codes[i] |= call(*a)
            s.synchronize()
            wrong[i] += sum(not torch.equal(o[0], ref[i]) for o in outs)

    t = [threading.Thread(target=work, args=(i,)) for i in range(4)]
    for th in t:
        th.start()
    for th in t:
        th.join()
    assert codes == [0] * 4 and wrong == [0] * 4, (codes, wrong)
    assert eng.last_error()[0] == 0


def test_captured_calls_on_a_forked_stream():
    """A captured graph whose calls run on a forked stream and make their own
    outputs: replays follow the inputs."""
    eng = Engine(config_from(policy=H2O, num_layers=1, batch=2, num_q_heads=8, num_kv_heads=2, head_dim=128, kv_dtype=BF16,
                             blocks_per_pool=4, max_tokens=8, budget=4, recent_window=2, obs_window=1, pool_kernel=1))
    eng.reset()
    g = torch.Generator(device="cuda").manual_seed(2)
    rnd = lambda *s: torch.randn(s, generator=g, device="cuda").bfloat16()
    c = eng.kv4_cache(4 * 5, 5)
    x, lens = rnd(2, 1, 12 * 128), torch.full((4,), 70, dtype=torch.int32, device="cuda")
    eng.kv4_write(c, None, rnd(2, 2, 80, 128), rnd(2, 2, 80, 128))

    def step(stream=None):
        q, k, v = eng.norm_rope(x, pos0=70, stream=stream)
        eng.kv4_write(c, lens, k, v, stream=stream)
        out = eng.kv4_attend(c, lens, q.view(2, 8, 128), sinks=2, window=40, stream=stream)
        return [q, k, v, *out, *eng.kv4_read(c, lens, 4, stream=stream)]

    step()
    side, cap = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=cap):
        side.wait_stream(cap)
        outs = step(side)
        cap.wait_stream(side)
    for _ in range(3):
        x.copy_(rnd(2, 1, 12 * 128))
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        ref = step()
        assert all(torch.equal(a, b) for a, b in zip(got, ref))
    assert eng.last_error()[0] == 0
