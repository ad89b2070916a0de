"""The Python binding marshals every entry point with the arity and argument
types its ctypes signature declares.

No GPU is involved: the library is replaced by a recorder that checks each
call against the signature table (which test_abi.py ties to the header), and
CPU tensors stand in for device ones. This catches a wrapper that drops,
duplicates or reorders an argument before any kernel runs.
"""
import ctypes

import pytest

import synth
import w8a8_quantized_decode_gb300 as a8w8

torch = pytest.importorskip("torch")


class _Recorder:
    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        res, argtypes = a8w8._SIGNATURES[name]

        def f(*args):
            assert len(args) == len(argtypes), (name, len(args), len(argtypes))
            for i, (a, t) in enumerate(zip(args, argtypes)):
                if t in (ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64):
                    assert isinstance(a, int) and not isinstance(a, bool), (name, i, a)
                elif t in (ctypes.c_float, ctypes.c_double):
                    assert isinstance(a, (int, float)), (name, i, a)
                elif t is ctypes.c_void_p:
                    assert (a is None or isinstance(a, (int, ctypes.Array))
                            or type(a).__name__ == "CArgObject"), (name, i, type(a))
            self.calls.append(name)
            return 0
        return f


@pytest.fixture
def rec(monkeypatch):
    r = _Recorder()
    monkeypatch.setattr(a8w8, "lib", lambda: r)
    monkeypatch.setattr(a8w8, "_ptr", lambda t: None if t is None else t.data_ptr())
    monkeypatch.setattr(a8w8, "_stream", lambda s=None: None)
    return r


CFG = dict(synth.TINY, num_layers=2, vocab=64)


def _t(shape, dtype=torch.bfloat16):
    return torch.zeros(shape, dtype=dtype)


def _caches(n=4):
    page, Hkv, D = CFG["page_size"], CFG["num_kv_heads"], CFG["head_dim"]
    return _t((n * page, Hkv, D))


def _i8_cache(n=4):
    page, Hkv, D = CFG["page_size"], CFG["num_kv_heads"], CFG["head_dim"]
    return _t((n * page, Hkv, D), torch.int8), _t((n * page, Hkv), torch.float32)


def _weights():
    return {k: torch.from_numpy(v.view("int16") if v.dtype.name == "uint16" else v)
            for k, v in synth.layer_weights(CFG, 1).items()}


def _bf16_weights():
    return {k: torch.from_numpy(v.view("int16")) for k, v in synth.bf16_layer_weights(CFG, 1).items()}


def _rows(B):
    i32 = torch.int32
    return _t((B,), i32), _t((B,), i32), _t((B, 2), i32), _t((B,), i32)


def test_int8_kv_wrappers(rec):
    kc, ks = _i8_cache()
    vc, vs = _i8_cache()
    Hkv, D = CFG["num_kv_heads"], CFG["head_dim"]
    a8w8.paged_kv_write_i8(_t((3, Hkv, D)), _t((3, Hkv, D)), _t((3,), torch.int32), kc, vc, ks, vs,
                           CFG["page_size"])
    q = _t((2, CFG["num_q_heads"], D))
    a8w8.paged_decode_attention_i8kv(q, kc, vc, ks, vs, _t((2, 2), torch.int32),
                                     _t((2,), torch.int32), CFG["page_size"], ws=_t((16,), torch.uint8))
    tok, slot, bt, ctx = _rows(2)
    rope, ws = _t((32, 2 * D), torch.float32), _t((64,), torch.uint8)
    hidden = _t((2, CFG["hidden"]))
    a8w8.a8w8_decode_layer_i8kv(_weights(), CFG, hidden, slot, bt, ctx, kc, vc, ks, vs, rope, ws,
                                taps={"xn": _t((2, CFG["hidden"]))})
    a8w8.a8w8_prefill_layer_i8kv(_weights(), CFG, hidden, slot, bt, ctx, kc, vc, ks, vs, rope, ws)
    model = {"embed": _t((64, CFG["hidden"])), "final_norm_w": _t((CFG["hidden"],)),
             "lm_head": _t((64, CFG["hidden"])), "layers": [_weights(), _weights()]}
    a8w8.a8w8_decode_step_i8kv(model, CFG, tok, slot, bt, ctx, [kc, kc], [vc, vc], [ks, ks],
                               [vs, vs], rope, ws, _t((2,), torch.int32))
    assert rec.calls == ["paged_kv_write_i8", "a8w8_attention_workspace_bytes",
                         "paged_decode_attention_i8kv",
                         "a8w8_decode_layer_i8kv", "a8w8_prefill_layer_i8kv",
                         "a8w8_decode_step_i8kv"]


def test_bf16_layer_and_prefill_step_wrappers(rec):
    H, I, D = CFG["hidden"], CFG["intermediate"], CFG["head_dim"]
    x = _t((3, H))
    a8w8.bf16_linear(x, _t((5, H)), residual=_t((3, 5)))
    a8w8.bf16_gate_up_swiglu(x, _t((2 * I, H)))
    tok, slot, bt, ctx = _rows(2)
    rope, ws = _t((32, 2 * D), torch.float32), _t((64,), torch.uint8)
    a8w8.bf16_decode_layer(_bf16_weights(), CFG, _t((2, H)), slot, bt, ctx, _caches(), _caches(),
                           rope, ws)
    model = {"embed": _t((64, H)), "final_norm_w": _t((H,)), "lm_head": _t((64, H)),
             "layers": [_weights(), _weights()]}
    a8w8.a8w8_prefill_step(model, CFG, tok, slot, bt, ctx, [_caches()] * 2, [_caches()] * 2, rope,
                           ws, _t((1,), torch.int32), _t((1,), torch.int32))
    assert rec.calls == ["bf16_linear", "bf16_gate_up_swiglu", "bf16_decode_layer",
                         "a8w8_prefill_step"]


def test_measured_path_wrappers(rec):
    D, H, I = CFG["head_dim"], CFG["hidden"], CFG["intermediate"]
    a8w8.a8w8_rmsnorm_gate_up_swiglu(_t((2, H)), _t((H,)), 1e-6, _t((2 * I, H), torch.int8),
                                     _t((2 * I,), torch.float32))
    a8w8.a8w8_matmul_i8(_t((3, H), torch.int8), _t((5, H), torch.int8), 0, H)
    tok, slot, bt, ctx = _rows(2)
    rope, ws = _t((32, 2 * D), torch.float32), _t((64,), torch.uint8)
    a8w8.a8w8_decode_layer(_weights(), CFG, _t((2, CFG["hidden"])), slot, bt, ctx, _caches(),
                           _caches(), rope, ws)
    a8w8.a8w8_prefill_layer(_weights(), CFG, _t((2, CFG["hidden"])), slot, bt, ctx, _caches(),
                            _caches(), rope, ws)
    model = {"embed": _t((64, CFG["hidden"])), "final_norm_w": _t((CFG["hidden"],)),
             "lm_head": _t((64, CFG["hidden"])), "layers": [_weights(), _weights()]}
    a8w8.a8w8_decode_step(model, CFG, tok, slot, bt, ctx, [_caches()] * 2, [_caches()] * 2, rope,
                          ws, _t((2,), torch.int32))
    assert rec.calls == ["a8w8_rmsnorm_gate_up_swiglu", "a8w8_matmul_i8", "a8w8_decode_layer",
                         "a8w8_prefill_layer", "a8w8_decode_step"]


@pytest.mark.parametrize("what", ["absent", "changed", "raises", "there"])
def test_private_torch_entries_have_public_stand_ins(what):
    """torch's private entries change with any release: whatever is there in their place, the calls
    get the current stream and rows of the shape they ask for."""
    from types import SimpleNamespace as NS
    public, calls = object(), []

    def fail(*a):
        raise TypeError("another signature")

    def private(shape, strides, dtype):
        calls.append(shape)
        t = torch.empty_strided(shape, strides, dtype=dtype)
        return NS(dtype=t.dtype, shape=t.shape, is_contiguous=t.is_contiguous,
                  get_device=lambda: 3 if there else 0)

    there = what == "there"
    own = {"absent": NS(), "raises": NS(_dynamo=NS(guards=NS(_empty_strided_cuda=fail)),
                                        _cuda_getCurrentRawStream=fail, _cuda_getDevice=fail)}.get(
        what, NS(_dynamo=NS(guards=NS(_empty_strided_cuda=private)),
                 _cuda_getCurrentRawStream=lambda dev: 77 if there else 0,
                 _cuda_getDevice=lambda: 3 if there else None))
    fake = NS(_C=own, bfloat16=torch.bfloat16, empty_strided=lambda *a, **k: public,
              cuda=NS(current_device=lambda: 3, current_stream=lambda *a: NS(cuda_stream=77)))
    h = a8w8._HostPath(fake)
    assert h.stream(3) == 77 and h.device() == 3
    rows = h.rows(5, 6, 7, None)
    assert (rows is public) == (what != "there")
    assert calls[1:] == ([(5, 6, 7)] if what == "there" else [])


class _FakeStreams:
    """What _alloc uses of torch: streams, one of them current, and tensors that note the stream
    they were allocated on and those recorded as users."""

    class Stream:
        def __init__(self, n):
            self.cuda_stream = n

    def __init__(self):
        self.now, self.cuda = self.Stream(1), self

    def current_stream(self):
        return self.now

    def stream(self, s):
        import contextlib

        @contextlib.contextmanager
        def switch():
            before, self.now = self.now, s
            yield
            self.now = before
        return switch()

    def tensor(self):
        t = type("T", (), {})()
        t.home, t.users = self.now, []
        t.record_stream = t.users.append
        return t


def test_memory_of_a_call_belongs_to_its_stream(monkeypatch):
    fake = _FakeStreams()
    monkeypatch.setattr(a8w8, "_torch", lambda: fake)
    here, side = fake.now, fake.Stream(2)
    t = a8w8._alloc(fake.tensor, side)
    assert t.home is side and t.users == [here] and fake.now is here
    for s in (None, here, fake.Stream(1)):
        t = a8w8._alloc(fake.tensor, s)
        assert t.home is here and not t.users


def _bare_allocations(names):
    """(function, line) of tensors that the named functions allocate outside of _alloc."""
    import ast
    tree = ast.parse(open(a8w8.__file__).read())
    found = []
    for f in tree.body:
        if not isinstance(f, ast.FunctionDef) or not names(f):
            continue
        inside = {id(n) for c in ast.walk(f) if isinstance(c, ast.Call)
                  and getattr(c.func, "id", "") == "_alloc" for n in ast.walk(c)}
        found += [(f.name, n.lineno) for n in ast.walk(f) if isinstance(n, ast.Call)
                  and getattr(n.func, "attr", "").startswith(("empty", "new_empty", "zeros", "full"))
                  and id(n) not in inside]
    return found


def _takes_stream(f):
    return "stream" in [a.arg for a in f.args.args]


def test_4_bit_and_page_entries_allocate_on_their_stream():
    new = lambda f: _takes_stream(f) and ("i4" in f.name or "page" in f.name)  # noqa: E731
    assert _bare_allocations(lambda f: new(f) and f.name != "paged_decode_attention_i8kv"
                             and not f.name.startswith("paged_decode_attention_bf16")) == []


def test_every_entry_allocates_on_its_stream():
    assert _bare_allocations(_takes_stream) == []
