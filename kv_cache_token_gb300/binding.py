"""ctypes binding of libkvevict.so: argument marshalling only.

Every method has the name of the C entry point it calls (kvevict_<name>) and
passes raw device pointers and the current torch CUDA stream.  Device memory
for the engine state is owned by the Engine object (torch tensors sized by
kvevict_buffer_size); the library never allocates.
"""
import ctypes
import os

import torch

H2O, SNAPKV, DROPKV = 0, 1, 2
BF16, F32 = 0, 1
KEY_F32, KEY_F64 = 0, 1

STATUS = {0: "OK", 1: "E_INVALID_ARG", 2: "E_POOL_KERNEL_EVEN", 3: "E_RECENT_GE_BUDGET",
          4: "E_OBS_WINDOW_ZERO", 5: "E_NO_BLOCKS", 6: "E_DTYPE", 7: "E_CUDA", 8: "E_TIMEOUT",
          9: "E_DEVICE", 10: "E_SCRATCH_LIMIT"}
STAT_NAMES = ["steps", "victims", "admit_new_block", "freed_dead", "freed_reloc", "moved", "plans",
              "deferred", "nan_keys", "blocks", "live", "half_empty", "lanes"]
NSTATS = len(STAT_NAMES)
(BUF_K_POOL, BUF_V_POOL, BUF_POSITIONS, BUF_SLOTS, BUF_COUNTS, BUF_SCORES, BUF_RING, BUF_RING_SLOT,
 BUF_BLOCK_OWNER, BUF_BLOCK_MASK, BUF_LANE_BLOCKS, BUF_LANE_NBLOCKS, BUF_STATS, BUF_WORKSPACE) = range(14)

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "libkvevict.so")


class KvevictError(RuntimeError):
    def __init__(self, code, what):
        super().__init__("%s: %s" % (what, STATUS.get(code, code)))
        self.code = code


class Config(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in (
        "policy", "num_layers", "batch", "num_q_heads", "num_kv_heads", "head_dim", "kv_dtype",
        "block_size", "blocks_per_pool", "max_tokens", "budget", "recent_window", "obs_window",
        "pool_kernel")] + [("theta_f", ctypes.c_float), ("max_window", ctypes.c_int32)]


class Buffers(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in (
        "k_pool", "v_pool", "positions", "slots", "counts", "scores", "ring", "ring_slot",
        "block_owner", "block_mask", "lane_blocks", "lane_nblocks", "stats", "workspace")]


class Kv4(ctypes.Structure):
    _fields_ = [("pages", ctypes.c_void_p), ("table", ctypes.c_void_p), ("scratch", ctypes.c_void_p),
                ("num_pages", ctypes.c_int32), ("max_pages", ctypes.c_int32)]


_LIB = None


def lib():
    """The loaded library; raises if it has not been built."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError("libkvevict.so is missing: build it with __graft_entry__.build()")
        L = ctypes.CDLL(LIB_PATH)
        P, I, V = ctypes.POINTER, ctypes.c_int32, ctypes.c_void_p
        L.kvevict_validate.argtypes = [P(Config)]
        L.kvevict_buffer_size.argtypes = [P(Config), ctypes.c_int]
        L.kvevict_buffer_size.restype = ctypes.c_size_t
        L.kvevict_workspace_size.argtypes = [P(Config)]
        L.kvevict_workspace_size.restype = ctypes.c_size_t
        L.kvevict_create.argtypes = [P(Config), P(Buffers), P(V)]
        L.kvevict_destroy.argtypes = [V]
        L.kvevict_destroy.restype = None
        L.kvevict_reset.argtypes = [V, V]
        L.kvevict_set_layer_budget.argtypes = [V, ctypes.c_int, I, I]
        L.kvevict_prefill.argtypes = [V, ctypes.c_int, V, V, I, V]
        L.kvevict_decode_step.argtypes = [V, ctypes.c_int, V, V, V, I, V, V, V, V, V]
        L.kvevict_attend.argtypes = [V, ctypes.c_int, V, V, V, V]
        L.kvevict_finish_step.argtypes = [V, ctypes.c_int, V, V, V, I, V, V, V, V, V]
        L.kvevict_score.argtypes = [V, ctypes.c_int, V, I, V, V, V, V, V]
        L.kvevict_score_mass.argtypes = [V, ctypes.c_int, V, I, V, I, V, V, V]
        L.kvevict_attend_static.argtypes = [V, ctypes.c_int, V, V, V, V, V, V]
        L.kvevict_select.argtypes = [V, V, I, V, V, I, I, I, I, V, V, V]
        L.kvevict_compact.argtypes = [V, ctypes.c_int, V, V, V, V, V, V, V]
        L.kvevict_defer_relocation.argtypes = [V, I]
        L.kvevict_relocate.argtypes = [V, ctypes.c_int, V, V, V, V, V]
        L.kvevict_norm_rope.argtypes = [V, V, ctypes.c_int64, ctypes.c_int64, I, V, V, ctypes.c_float, V, I, I,
                                        ctypes.c_double, I, V, V, V, V]
        L.kvevict_attend_prompt.argtypes = [V, V, V, V, I, I, I, V, V, V]
        L.kvevict_kv4_page_bytes.argtypes = [P(Config)]
        L.kvevict_kv4_page_bytes.restype = ctypes.c_size_t
        L.kvevict_kv4_scratch_bytes.argtypes = [P(Config)]
        L.kvevict_kv4_scratch_bytes.restype = ctypes.c_size_t
        L.kvevict_kv4_validate.argtypes = [P(Config), P(Kv4)]
        L.kvevict_kv4_write.argtypes = [V, P(Kv4), V, I, V, V, V]
        L.kvevict_kv4_pack.argtypes = [V, ctypes.c_int, P(Kv4), V]
        L.kvevict_kv4_read.argtypes = [V, P(Kv4), V, V, I, V, V, V]
        L.kvevict_kv4_attend.argtypes = [V, P(Kv4), V, V, I, I, V, V, V]
        L.kvevict_stats.argtypes = [V, ctypes.c_int, V, V]
        L.kvevict_last_error.argtypes = [V, ctypes.c_char_p, ctypes.c_size_t]
        L.kvevict_check_wait_timeout.argtypes = [V, I, V]
        L.kvevict_kernels_per_decode_step.argtypes = [V]
        L.kvevict_kernels_per_decode_step.restype = I
        for f in ("validate", "create", "reset", "set_layer_budget", "prefill", "decode_step", "attend", "finish_step",
                  "attend_static",
                  "score", "score_mass", "select",
                  "norm_rope", "attend_prompt", "kv4_validate", "kv4_write", "kv4_pack", "kv4_read", "kv4_attend",
                  "compact", "defer_relocation", "relocate", "stats", "check_wait_timeout", "last_error"):
            getattr(L, "kvevict_" + f).restype = ctypes.c_int
        _LIB = L
    return _LIB


def config_from(shape=None, **kw):
    """A Config from a workloads Shape (or keyword fields)."""
    f = {}
    if shape is not None:
        f = dict(policy=shape.policy, num_layers=shape.num_layers, batch=shape.batch,
                 num_q_heads=shape.num_q_heads, num_kv_heads=shape.num_kv_heads,
                 head_dim=shape.head_dim, kv_dtype=BF16 if shape.kv_dtype == "bf16" else F32,
                 block_size=16, blocks_per_pool=shape.blocks_per_pool,
                 max_tokens=shape.max_tokens, budget=shape.budget,
                 recent_window=shape.recent_window, obs_window=shape.obs_window,
                 pool_kernel=shape.pool_kernel, theta_f=shape.theta_f, max_window=shape.window)
    f.update(kw)
    f.setdefault("block_size", 16)
    f.setdefault("theta_f", 0.25)
    f.setdefault("max_window", 0)
    return Config(**f)


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _raw(t):
    return None if t is None else t.data_ptr()


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _check(code, what):
    if code != 0:
        raise KvevictError(code, what)


def _need(ok, what):
    """Refuses a tensor argument before its address reaches the library."""
    if not ok:
        raise ValueError(what)


def _dense(t, shape, dtype, device, what):
    # one test, no message built when it holds: this runs several times a call
    if not (t.shape == shape and t.dtype is dtype and t.is_contiguous() and t.get_device() == device.index):
        raise ValueError("%s must be a contiguous %s tensor of shape %s on %s" % (what, dtype, tuple(shape), device))


def kv4_geometry(cfg, device):
    """What a 4-bit cache of this configuration is sized by: lanes, bytes of a
    page (0: the configuration has no such cache), device."""
    return cfg.batch * cfg.num_kv_heads, lib().kvevict_kv4_page_bytes(ctypes.byref(cfg)), device


def _int32(what, a, b=0):
    # ctypes would pass the low 32 bits on
    if not (-0x80000000 <= a <= 0x7FFFFFFF and -0x80000000 <= b <= 0x7FFFFFFF):
        raise ValueError("%s must be in int32's range, not %d, %d" % (what, a, b))


class Kv4Cache:
    """Device buffers of one 4-bit cache (kvevict_kv4): pages, the lanes' page
    table and the attention's scratch.  Caches of several layers may share one
    pool of pages: pass `pages`, and a table per layer.  Other engines of the
    same lanes, head_dim and device may use the cache (to attend, no larger
    a group); any other engine's calls refuse it.  Pages and scratch start at
    zero on the stream that is current here: another stream waits for it."""

    def __init__(self, eng, num_pages, max_pages, table=None, pages=None):
        L, c = lib(), ctypes.byref(eng.cfg)
        self.geometry = eng.kv4_geometry
        page = self.geometry[1]
        if page == 0:
            raise KvevictError(6, "kvevict_kv4_page_bytes")
        self.num_pages, self.max_pages, self.page_bytes = int(num_pages), int(max_pages), page
        if pages is None:
            pages = torch.zeros((num_pages, page), dtype=torch.uint8, device=eng.device)
        if table is None:
            # every lane its own run of pages
            _need(num_pages >= eng.lanes * max_pages, "a default table needs lanes * max_pages pages")
            table = torch.arange(eng.lanes * max_pages, dtype=torch.int32, device=eng.device).view(eng.lanes, max_pages)
        _dense(pages, (num_pages, page), torch.uint8, eng.device, "pages")
        _dense(table, (eng.lanes, max_pages), torch.int32, eng.device, "table")
        self.pages, self.table = pages, table
        self.scratch_bytes = L.kvevict_kv4_scratch_bytes(c)
        self.scratch = torch.zeros((self.scratch_bytes,), dtype=torch.uint8, device=eng.device)
        self.c = Kv4(pages.data_ptr(), table.data_ptr(), self.scratch.data_ptr(), self.num_pages, self.max_pages)
        self.ref = ctypes.byref(self.c)
        _check(L.kvevict_kv4_validate(c, self.ref), "kvevict_kv4_validate")


def validate(cfg):
    return lib().kvevict_validate(ctypes.byref(cfg))


class Engine:
    """Device state of one engine plus the C-ABI calls on it."""

    def __init__(self, cfg, device="cuda"):
        L = lib()
        self.cfg = cfg
        _check(L.kvevict_validate(ctypes.byref(cfg)), "kvevict_validate")
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self.kv4_geometry = kv4_geometry(cfg, self.device)
        self.kv4_scratch_bytes = L.kvevict_kv4_scratch_bytes(ctypes.byref(cfg))
        c = cfg
        lanes = c.batch * c.num_kv_heads
        self.lanes = lanes
        self.g = c.num_q_heads // c.num_kv_heads
        kvdt = torch.bfloat16 if c.kv_dtype == BF16 else torch.float32
        self.kv_dtype = kvdt
        dev = self.device

        def buf(which, shape, dtype):
            nbytes = L.kvevict_buffer_size(ctypes.byref(cfg), which)
            t = torch.empty(shape, dtype=dtype, device=dev)
            assert t.numel() * t.element_size() == nbytes, (which, nbytes, t.numel() * t.element_size())
            return t

        Lr, P, C, d = c.num_layers, c.blocks_per_pool, c.max_tokens, c.head_dim
        self.k_pool = buf(BUF_K_POOL, (Lr, P, 16, d), kvdt)
        self.v_pool = buf(BUF_V_POOL, (Lr, P, 16, d), kvdt)
        self.positions = buf(BUF_POSITIONS, (Lr, lanes, C), torch.int32)
        self.slots = buf(BUF_SLOTS, (Lr, lanes, C), torch.int32)
        self.counts = buf(BUF_COUNTS, (Lr, lanes), torch.int32)
        self.scores = buf(BUF_SCORES, (Lr, lanes, C), torch.float32)
        # history rows sit at the tokens' slots: ring[layer][slot] (slot = block * 16 + offset)
        self.ring = (buf(BUF_RING, (Lr, P * 16, c.obs_window), torch.float32)
                     if c.policy == SNAPKV or (c.policy == DROPKV and c.obs_window >= 1) else None)
        self.ring_slot = buf(BUF_RING_SLOT, (Lr, lanes), torch.int32)
        self.block_owner = buf(BUF_BLOCK_OWNER, (Lr, P), torch.int32)
        self.block_mask = buf(BUF_BLOCK_MASK, (Lr, P), torch.int32)
        self.lane_blocks = buf(BUF_LANE_BLOCKS, (Lr, lanes, C), torch.int32)
        self.lane_nblocks = buf(BUF_LANE_NBLOCKS, (Lr, lanes), torch.int32)
        self.stats_buf = buf(BUF_STATS, (Lr, NSTATS), torch.int64)
        ws = L.kvevict_workspace_size(ctypes.byref(cfg))
        self.workspace = torch.empty(ws + 256, dtype=torch.uint8, device=dev)
        off = (-self.workspace.data_ptr()) % 256
        self.workspace_aligned = self.workspace[off:off + ws]
        b = Buffers(*[_ptr(t) for t in (
            self.k_pool, self.v_pool, self.positions, self.slots, self.counts, self.scores,
            self.ring, self.ring_slot, self.block_owner, self.block_mask, self.lane_blocks,
            self.lane_nblocks, self.stats_buf, self.workspace_aligned)])
        self._bufs = b
        h = ctypes.c_void_p()
        with torch.cuda.device(dev):
            _check(L.kvevict_create(ctypes.byref(cfg), ctypes.byref(b), ctypes.byref(h)), "kvevict_create")
        self.h = h
        # per-call outputs reused by default
        self.victims = torch.zeros((lanes, C), dtype=torch.int32, device=dev)
        self.n_victims = torch.zeros((lanes,), dtype=torch.int32, device=dev)

    def __del__(self):
        h = getattr(self, "h", None)
        if h is not None and _LIB is not None:
            _LIB.kvevict_destroy(h)
            self.h = None

    def _new(self, stream, shape, dtype, make=None):
        """A default output of a call on `stream` (None: the current one).  Its
        memory and its fill are that stream's, as the kernel that writes it is;
        the current stream, where the caller may read it, is noted as a user."""
        make = make or torch.empty
        if stream is None:
            return make(shape, dtype=dtype, device=self.device)
        with torch.cuda.stream(stream):
            t = make(shape, dtype=dtype, device=self.device)
        t.record_stream(torch.cuda.current_stream(self.device))
        return t

    # ---- C-ABI calls ----------------------------------------------------------
    def reset(self, stream=None):
        _check(lib().kvevict_reset(self.h, _stream(stream)), "kvevict_reset")

    def set_layer_budget(self, layer, budget, recent_window):
        """kvevict_set_layer_budget: later decode steps of `layer` keep `budget` tokens."""
        _check(lib().kvevict_set_layer_budget(self.h, layer, budget, recent_window), "kvevict_set_layer_budget")

    def prefill(self, layer, k_ctx, v_ctx, stream=None):
        assert k_ctx.is_contiguous() and v_ctx.is_contiguous() and k_ctx.dtype == self.kv_dtype
        n = k_ctx.shape[2]
        _check(lib().kvevict_prefill(self.h, layer, _ptr(k_ctx), _ptr(v_ctx), n, _stream(stream)),
               "kvevict_prefill")

    def decode_step(self, layer, q, k_new, v_new, new_pos, out=None, lse=None, victims=None,
                    n_victims=None, stream=None):
        c = self.cfg
        if q is not None and out is None:
            out = self._new(stream, (c.batch, c.num_q_heads, c.head_dim), torch.float32)
        if q is not None and lse is None:
            lse = self._new(stream, (c.batch, c.num_q_heads), torch.float32)
        victims = self.victims if victims is None else victims
        n_victims = self.n_victims if n_victims is None else n_victims
        for t in (q, k_new, v_new):
            assert t is None or (t.is_contiguous() and t.dtype == self.kv_dtype)
        _check(lib().kvevict_decode_step(self.h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), int(new_pos),
                                         _ptr(out), _ptr(lse), _ptr(victims), _ptr(n_victims),
                                         _stream(stream)), "kvevict_decode_step")
        return out, lse, victims, n_victims

    def attend(self, layer, q, k_new, v_new, stream=None):
        _check(lib().kvevict_attend(self.h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), _stream(stream)),
               "kvevict_attend")

    def finish_step(self, layer, q, k_new, v_new, new_pos, out=None, lse=None, victims=None, n_victims=None,
                    stream=None):
        c = self.cfg
        if q is not None and out is None:
            out = self._new(stream, (c.batch, c.num_q_heads, c.head_dim), torch.float32)
        if q is not None and lse is None:
            lse = self._new(stream, (c.batch, c.num_q_heads), torch.float32)
        victims = self.victims if victims is None else victims
        n_victims = self.n_victims if n_victims is None else n_victims
        _check(lib().kvevict_finish_step(self.h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), int(new_pos),
                                         _ptr(out), _ptr(lse), _ptr(victims), _ptr(n_victims),
                                         _stream(stream)), "kvevict_finish_step")
        return out, lse, victims, n_victims

    def attend_static(self, layer, q, k_new, v_new, out=None, lse=None, stream=None):
        """kvevict_attend_static: attention output and LSE of one layer using the
        library's built-in scratch array (no workspace, no allocation inside)."""
        c = self.cfg
        if out is None:
            out = self._new(stream, (c.batch, c.num_q_heads, c.head_dim), torch.float32)
        if lse is None:
            lse = self._new(stream, (c.batch, c.num_q_heads), torch.float32)
        _check(lib().kvevict_attend_static(self.h, layer, _ptr(q), _ptr(k_new), _ptr(v_new), _ptr(out), _ptr(lse),
                                           _stream(stream)), "kvevict_attend_static")
        return out, lse

    def score(self, layer, q_win, q_pos, lse=None, a_out=None, scores=None, stream=None):
        c = self.cfg
        if q_win is None:
            _check(lib().kvevict_score(self.h, layer, None, 0, None, None, None, None, _stream(stream)),
                   "kvevict_score")
            return None
        w = q_win.shape[2]
        if lse is None:
            lse = self._new(stream, (c.batch, c.num_q_heads, w), torch.float32)
        if a_out is None:
            a_out = self._new(stream, (c.batch, c.num_q_heads, w, c.head_dim), torch.float32)
        if scores is None:
            scores = self._new(stream, (self.lanes, c.max_tokens), torch.float32, torch.zeros)
        assert q_win.is_contiguous() and q_pos.dtype == torch.int32
        _check(lib().kvevict_score(self.h, layer, _ptr(q_win), w, _ptr(q_pos), _ptr(lse), _ptr(a_out),
                                   _ptr(scores), _stream(stream)), "kvevict_score")
        return lse, a_out, scores

    def score_mass(self, layer, q_win, q_pos, kind, lse=None, scores=None, stream=None):
        """kvevict_score_mass; kind 0 = SnapKV prefill keys, 1 = H2O
        causal-prefill scores.  Returns (lse, scores) or None for q_win None."""
        c = self.cfg
        if q_win is None:
            _check(lib().kvevict_score_mass(self.h, layer, None, 0, None, kind, None, None, _stream(stream)),
                   "kvevict_score_mass")
            return None
        w = q_win.shape[2]
        if lse is None:
            lse = self._new(stream, (c.batch, c.num_q_heads, w), torch.float32)
        if scores is None:
            scores = self._new(stream, (self.lanes, c.max_tokens), torch.float32, torch.zeros)
        assert q_win.is_contiguous() and q_pos.dtype == torch.int32
        _check(lib().kvevict_score_mass(self.h, layer, _ptr(q_win), w, _ptr(q_pos), kind, _ptr(lse),
                                        _ptr(scores), _stream(stream)), "kvevict_score_mass")
        return lse, scores

    def select(self, keys, positions, counts, budget, recent_window, victims=None, n_victims=None,
               stream=None):
        n_lanes, stride = keys.shape
        kd = KEY_F64 if keys.dtype == torch.float64 else KEY_F32
        if victims is None:
            victims = self._new(stream, (n_lanes, stride), torch.int32, lambda *a, **kw: torch.full(*a, -1, **kw))
        if n_victims is None:
            n_victims = self._new(stream, (n_lanes,), torch.int32, torch.zeros)
        assert keys.is_contiguous() and positions.is_contiguous() and positions.shape == keys.shape
        _check(lib().kvevict_select(self.h, _ptr(keys), kd, _ptr(positions), _ptr(counts), n_lanes, stride,
                                    budget, recent_window, _ptr(victims), _ptr(n_victims), _stream(stream)),
               "kvevict_select")
        return victims, n_victims

    def compact(self, layer, victims, n_victims, freed=None, n_freed=None, moves=None, n_moves=None,
                stream=None):
        c = self.cfg
        # the library writes freed[0..n_freed) and moves[0..n_moves) and both counts
        if freed is None:
            freed = self._new(stream, (c.blocks_per_pool,), torch.int32)
        if n_freed is None:
            n_freed = self._new(stream, (1,), torch.int32)
        if moves is None:
            moves = self._new(stream, (self.lanes * c.max_tokens, 6), torch.int32)
        if n_moves is None:
            n_moves = self._new(stream, (1,), torch.int32)
        _check(lib().kvevict_compact(self.h, layer, _ptr(victims), _ptr(n_victims), _ptr(freed), _ptr(n_freed),
                                     _ptr(moves), _ptr(n_moves), _stream(stream)), "kvevict_compact")
        return freed, n_freed, moves, n_moves

    def defer_relocation(self, deferred=True):
        """kvevict_defer_relocation: decode steps plan no relocation while set."""
        _check(lib().kvevict_defer_relocation(self.h, 1 if deferred else 0), "kvevict_defer_relocation")

    def relocate(self, layer, freed=None, n_freed=None, moves=None, n_moves=None, stream=None):
        """kvevict_relocate on `stream`; returns (freed, n_freed, moves, n_moves)."""
        c = self.cfg
        if freed is None:
            freed = self._new(stream, (c.blocks_per_pool,), torch.int32)
        if n_freed is None:
            n_freed = self._new(stream, (1,), torch.int32)
        if moves is None:
            moves = self._new(stream, (self.lanes * c.max_tokens, 6), torch.int32)
        if n_moves is None:
            n_moves = self._new(stream, (1,), torch.int32)
        _check(lib().kvevict_relocate(self.h, layer, _ptr(freed), _ptr(n_freed), _ptr(moves), _ptr(n_moves),
                                      _stream(stream)), "kvevict_relocate")
        return freed, n_freed, moves, n_moves

    # ---- around the eviction --------------------------------------------------
    def _on(self, stream):
        return torch._C._cuda_getCurrentRawStream(self.device.index) if stream is None else stream.cuda_stream

    def norm_rope(self, qkv, wq=None, wk=None, eps=1e-6, pos=None, pos0=0, rotary_dim=None, base=10000.0,
                  interleaved=False, q=None, k=None, v=None, stream=None):
        """kvevict_norm_rope: (q, k, v) in the engine's layouts from projection
        rows qkv [B][n][(Hq + 2 Hkv) d], any batch and row stride."""
        c, dev, dt = self.cfg, self.device, self.kv_dtype
        B, Hq, Hkv, d = c.batch, c.num_q_heads, c.num_kv_heads, c.head_dim
        _need(qkv.dim() == 3 and qkv.shape[0] == B and qkv.shape[2] == (Hq + 2 * Hkv) * d and qkv.dtype is dt and
              qkv.get_device() == dev.index and qkv.stride(2) == 1, "qkv must be [batch][n][(Hq + 2 Hkv) d] of the engine's dtype")
        n = qkv.shape[1]
        r = d if rotary_dim is None else rotary_dim
        _int32("pos0 and rotary_dim", pos0, r)
        # one token has no next row: its row stride is whatever the tensor says
        row = qkv.stride(1) if n > 1 else (Hq + 2 * Hkv) * d
        for w in (wq, wk):
            if w is not None:
                _dense(w, (d,), dt, dev, "a norm weight")
        if pos is not None:
            _dense(pos, (n,), torch.int32, dev, "pos")
        out = lambda t, h: self._new(stream, (B, h, n, d), dt) if t is None else t
        q, k, v = out(q, Hq), out(k, Hkv), out(v, Hkv)
        _dense(q, (B, Hq, n, d), dt, dev, "q")
        _dense(k, (B, Hkv, n, d), dt, dev, "k")
        _dense(v, (B, Hkv, n, d), dt, dev, "v")
        _check(lib().kvevict_norm_rope(self.h, qkv.data_ptr(), qkv.stride(0), row, n, _raw(wq), _raw(wk), eps,
                                       _raw(pos), pos0, r, base,
                                       1 if interleaved else 0, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                                       self._on(stream)), "kvevict_norm_rope")
        return q, k, v

    def attend_prompt(self, q, k, v, sinks=0, window=0, out=None, lse=None, stream=None):
        """kvevict_attend_prompt: (out [B][n][Hq][d], lse [B][Hq][n])."""
        c, dev, bf = self.cfg, self.device, torch.bfloat16
        B, Hq, Hkv, d = c.batch, c.num_q_heads, c.num_kv_heads, c.head_dim
        _need(q.dim() == 4, "q must be [batch][Hq][n][d]")
        _int32("sinks and window", sinks, window)
        n = q.shape[2]
        _dense(q, (B, Hq, n, d), bf, dev, "q")
        _dense(k, (B, Hkv, n, d), bf, dev, "k")
        _dense(v, (B, Hkv, n, d), bf, dev, "v")
        if out is None:
            out = self._new(stream, (B, n, Hq, d), bf)
        if lse is None:
            lse = self._new(stream, (B, Hq, n), torch.float32)
        _dense(out, (B, n, Hq, d), bf, dev, "out")
        _dense(lse, (B, Hq, n), torch.float32, dev, "lse")
        _check(lib().kvevict_attend_prompt(self.h, q.data_ptr(), k.data_ptr(), v.data_ptr(), n, sinks, window,
                                           out.data_ptr(), lse.data_ptr(), self._on(stream)),
               "kvevict_attend_prompt")
        return out, lse

    def kv4_cache(self, num_pages, max_pages, table=None, pages=None):
        """A 4-bit cache for this engine's lanes (Kv4Cache)."""
        return Kv4Cache(self, num_pages, max_pages, table=table, pages=pages)

    def _cache_ref(self, cache, scratch=0):
        # the library sees addresses only: a cache sized for other lanes or rows would be overrun
        if not ((cache.geometry is self.kv4_geometry or cache.geometry == self.kv4_geometry) and cache.scratch_bytes >= scratch):
            raise ValueError("the cache was made for %s (lanes, page bytes, device) and %d bytes of scratch; this engine needs %s and %d"
                             % (cache.geometry, cache.scratch_bytes, self.kv4_geometry, scratch))
        return cache.ref

    def _lane_ints(self, t, what):
        if t is not None:
            _dense(t, (self.lanes,), torch.int32, self.device, what)
        return _raw(t)

    def kv4_write(self, cache, starts, k, v, stream=None):
        """kvevict_kv4_write: k, v [B][Hkv][n][d] at indices starts[lane] and after."""
        c, ref = self.cfg, self._cache_ref(cache)
        _need(k.dim() == 4, "k must be [batch][Hkv][n][d]")
        n = k.shape[2]
        for t, w in ((k, "k"), (v, "v")):
            _dense(t, (c.batch, c.num_kv_heads, n, c.head_dim), torch.bfloat16, self.device, w)
        _check(lib().kvevict_kv4_write(self.h, ref, self._lane_ints(starts, "starts"), n,
                                       k.data_ptr(), v.data_ptr(), self._on(stream)), "kvevict_kv4_write")

    def kv4_pack(self, layer, cache, stream=None):
        """kvevict_kv4_pack: every kept token of an engine layer, from index 0."""
        _int32("layer", layer)
        _check(lib().kvevict_kv4_pack(self.h, layer, self._cache_ref(cache), self._on(stream)), "kvevict_kv4_pack")

    def kv4_read(self, cache, starts, n, lens=None, k=None, v=None, stream=None):
        """kvevict_kv4_read: the values of n tokens a lane, [B][Hkv][n][d]."""
        c, ref = self.cfg, self._cache_ref(cache)
        shp = (c.batch, c.num_kv_heads, n, c.head_dim)
        # rows past a lane's end are not written
        k = self._new(stream, shp, torch.bfloat16, torch.zeros) if k is None else k
        v = self._new(stream, shp, torch.bfloat16, torch.zeros) if v is None else v
        _dense(k, shp, torch.bfloat16, self.device, "k")
        _dense(v, shp, torch.bfloat16, self.device, "v")
        _check(lib().kvevict_kv4_read(self.h, ref, self._lane_ints(starts, "starts"),
                                      self._lane_ints(lens, "lens"), n, k.data_ptr(), v.data_ptr(),
                                      self._on(stream)), "kvevict_kv4_read")
        return k, v

    def kv4_attend(self, cache, lens, q, sinks=0, window=0, out=None, lse=None, stream=None):
        """kvevict_kv4_attend: (out [B][Hq][d], lse [B][Hq])."""
        c, dev, ref = self.cfg, self.device, self._cache_ref(cache, self.kv4_scratch_bytes)
        shp = (c.batch, c.num_q_heads, c.head_dim)
        _int32("sinks and window", sinks, window)
        _dense(q, shp, torch.bfloat16, dev, "q")
        if out is None:
            out = self._new(stream, shp, torch.bfloat16)
        if lse is None:
            lse = self._new(stream, shp[:2], torch.float32)
        _dense(out, shp, torch.bfloat16, dev, "out")
        _dense(lse, shp[:2], torch.float32, dev, "lse")
        _need(lens is not None, "lens")
        _check(lib().kvevict_kv4_attend(self.h, ref, self._lane_ints(lens, "lens"), q.data_ptr(),
                                        sinks, window, out.data_ptr(), lse.data_ptr(), self._on(stream)),
               "kvevict_kv4_attend")
        return out, lse

    def stats(self, layer, stream=None):
        out = self._new(stream, (NSTATS,), torch.int64, torch.zeros)
        _check(lib().kvevict_stats(self.h, layer, _ptr(out), _stream(stream)), "kvevict_stats")
        return out

    def kernels_per_decode_step(self):
        """kvevict_kernels_per_decode_step (2 or 3)."""
        return int(lib().kvevict_kernels_per_decode_step(self.h))

    def check_wait_timeout(self, polls, stream=None):
        """kvevict_check_wait_timeout: the next last_error() reports a timeout."""
        _check(lib().kvevict_check_wait_timeout(self.h, polls, _stream(stream)), "kvevict_check_wait_timeout")

    def last_error(self):
        buf = ctypes.create_string_buffer(256)
        code = lib().kvevict_last_error(self.h, buf, 256)
        return code, buf.value.decode()
