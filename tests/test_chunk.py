"""A chunk of new tokens and the paged cache: the QKV rows' norm, rotation and placing in each cache
form (paged_kv_append*), and the chunk's attention over it (paged_chunk_attention_*).

On the CPU: the float64 oracle (oracle/chunk.py) against the C oracle and by hand, and the refusals.
On the GPU: rows bit for bit, attention within bounds derived from its arithmetic.
"""
import numpy as np
import pytest

import oracle
import synth
import w8a8_quantized_decode_gb300 as a8w8
from gpu_util import to_dev, to_host
from oracle import chunk, kv_i4

gpu = pytest.mark.gpu
FAKE = 0x10000
KINDS = ("bf16", "i8", "i4")
THETA = 1e6


@pytest.fixture(scope="module")
def lib():
    a8w8.build()
    return a8w8.lib()


def _bf(x):
    return kv_i4.f32_to_bf16(np.asarray(x, np.float32))


# ---------------------------------------------------------------------------
# oracle pins (CPU)
# ---------------------------------------------------------------------------

def test_append_oracle_by_hand_and_against_the_layers_rope():
    x = _bf([[3.0, 0.0, 4.0, 0.0] * 16])
    w = _bf(np.ones(64))
    # position 0 turns nothing; mean square 6.25, so the norm divides by 2.5
    got = oracle.bf16_to_f64(chunk.rotated_heads(x, w, 0.0, 0, THETA))
    assert np.array_equal(got, oracle.bf16_to_f64(_bf([[1.2, 0.0, 1.6, 0.0] * 16])))
    for D in (64, 128):
        x = synth.bf16_normal(D, (3, D))
        want = oracle.rope(x[None], np.array([1234], np.int32), THETA)[0]
        got = chunk.rotated_heads(x, None, 0.0, 1234, THETA)
        d = np.abs(oracle.bf16_to_f64(got) - oracle.bf16_to_f64(want))
        assert d.max() <= 2.0 ** -8 * np.abs(oracle.bf16_to_f64(x)).max() * 2


def test_attention_oracle_equals_the_decode_oracle_row_by_row():
    B, Hq, Hkv, D, page = 2, 4, 2, 64, 16
    n, ctx = np.array([3, 5]), np.array([20, 5], np.int32)
    bt, nblk = synth.paged_layout(3, ctx, page, spare_blocks=1)
    K = synth.bf16_normal(1, (nblk * page, Hkv, D))
    V = synth.bf16_normal(2, (nblk * page, Hkv, D))
    q = synth.bf16_normal(4, (8, Hq, D))
    starts = np.array([0, 3, 8], np.int32)
    out, bound, owned = chunk.attention(q, oracle.bf16_to_f64(K), oracle.bf16_to_f64(V), bt, ctx, starts, page)
    assert owned.all() and (bound > 0).all()
    for b in range(B):
        for i in range(n[b]):
            c = np.array([ctx[b] - n[b] + i + 1], np.int32)
            ref, rc = oracle.paged_attention(q[starts[b] + i][None], K, V, bt[b][None], c, page)
            ref = oracle.bf16_to_f64(ref)[0]
            assert rc == 0
            assert (np.abs(out[starts[b] + i] - ref) <= np.abs(ref) * 2.0 ** -8 + 1e-12).all()


def test_plan_covers_every_block_once(tmp_path):
    """The attention's division into parts, compiled for the host (chunk_plan_check.cpp)."""
    import os
    import subprocess
    exe = str(tmp_path / "check")
    src = os.path.join(os.path.dirname(os.path.abspath(__file__)), "chunk_plan_check.cpp")
    subprocess.run(["g++", "-O2", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-o", exe, src],
                   check=True)
    r = subprocess.run([exe], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr


# ---------------------------------------------------------------------------
# refusals (CPU)
# ---------------------------------------------------------------------------

def _append_call(lib, kind, qkv=FAKE, T=2, Hq=8, Hkv=2, D=128, ld=None, qw=None, kw=None, eps=1e-6, pos=FAKE,
                 rope=FAKE, max_pos=64, slots=FAKE, q=FAKE, k=FAKE, s=FAKE, nb=4, page=16):
    ld = (Hq + 2 * Hkv) * D if ld is None else ld
    f = {"bf16": lib.paged_kv_append, "i8": lib.paged_kv_append_i8, "i4": lib.paged_kv_append_i4}[kind]
    scales = () if kind == "bf16" else (s, FAKE)
    return f(qkv, T, Hq, Hkv, D, ld, qw, kw, eps, pos, rope, max_pos, slots, q, k, FAKE, *scales, nb, page, None)


@pytest.mark.parametrize("kind", KINDS)
def test_append_refusals(lib, kind):
    f = lambda **a: _append_call(lib, kind, **a)  # noqa: E731
    inv, uns = a8w8.ERR_INVALID_ARG, a8w8.ERR_UNSUPPORTED_SHAPE
    assert f(T=-1) == f(Hkv=0) == f(Hq=-1) == f(max_pos=0) == f(nb=0) == f(page=0) == inv
    assert f(D=96) == f(ld=12 * 128 - 8) == f(ld=12 * 128 + 4) == f(T=(1 << 24) + 1) == uns
    assert f(nb=1 << 20, page=1 << 12) == uns
    assert f(qkv=None) == f(pos=None) == f(rope=None) == f(slots=None) == f(k=None) == inv
    assert f(qkv=FAKE + 8) == f(qw=FAKE + 2) == f(q=FAKE + 8) == inv
    assert f(qw=FAKE, eps=-1.0) == f(kw=FAKE, eps=float("nan")) == inv
    if kind != "bf16":
        assert f(s=None) == f(s=FAKE + 4) == inv
    assert f(T=0, qkv=None) == a8w8.OK
    assert "paged_kv_append" in a8w8.last_error()


def _attention_call(lib, kind, q=FAKE, k=FAKE, s=FAKE, bt=FAKE, ctx=FAKE, st=FAKE, T=10, B=2, Hq=16, Hkv=2, D=128,
                    page=16, max_blocks=40, nb=100, out=FAKE, ws=FAKE, wsb=1 << 40):
    f = {"bf16": lib.paged_chunk_attention_bf16, "i8": lib.paged_chunk_attention_i8kv,
         "i4": lib.paged_chunk_attention_i4kv}[kind]
    scales = () if kind == "bf16" else (s, FAKE)
    return f(q, k, FAKE, *scales, bt, ctx, st, T, B, Hq, Hkv, D, page, max_blocks, nb, 0.1, out, ws, wsb, None)


@pytest.mark.parametrize("kind", KINDS)
def test_attention_refusals(lib, kind):
    f = lambda **a: _attention_call(lib, kind, **a)  # noqa: E731
    inv, uns = a8w8.ERR_INVALID_ARG, a8w8.ERR_UNSUPPORTED_SHAPE
    assert f(T=-1) == f(B=-1) == f(Hq=0) == f(Hkv=0) == f(page=0) == f(max_blocks=0) == f(nb=0) == inv
    assert f(D=96) == f(Hq=18) == f(Hq=15) == f(max_blocks=1 << 21) == f(B=65536) == uns
    assert f(T=(1 << 24) + 1) == f(nb=1 << 20, page=1 << 12, max_blocks=1) == uns
    assert f(q=None) == f(k=None) == f(bt=None) == f(ctx=None) == f(st=None) == f(out=None) == inv
    assert f(q=FAKE + 8) == inv
    if kind != "bf16":
        assert f(s=None) == inv
    need = lib.a8w8_chunk_attention_workspace_bytes(10, 2, 16, 2, 128, 640)
    assert need > 0
    assert f(ws=None) == f(wsb=need - 1) == f(ws=FAKE + 8) == a8w8.ERR_WORKSPACE
    assert f(T=0, q=None) == f(B=0, q=None) == a8w8.OK


def test_workspace_sizes(lib):
    f = lib.a8w8_chunk_attention_workspace_bytes
    assert f(0, 1, 8, 2, 128, 64) == f(1, 0, 8, 2, 128, 64) == f(1, 1, 9, 2, 128, 64) == f(1, 1, 32, 2, 128, 64) == 0
    assert f(1, 1, 8, 2, 128, 64) <= f(64, 4, 8, 2, 128, 4096) <= f(4096, 4, 8, 2, 128, 4096)


def test_binding_refuses_wrong_tensors():
    import torch
    z = torch.zeros((32, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(a8w8.A8W8Error, match="caches"):
        a8w8._cache_rows((z, z[:16]), torch.bfloat16, 2, 64, 16, "x", -1)
    with pytest.raises(a8w8.A8W8Error, match="bfloat16"):
        a8w8._cache_rows((z, z.half()), torch.bfloat16, 2, 64, 16, "x", -1)
    with pytest.raises(a8w8.A8W8Error, match="float32"):
        c = torch.zeros((32, 2, 64), dtype=torch.int8)
        a8w8._cache_i8(c, c, torch.zeros(64), torch.zeros(63), 2, 64, 16, "x", -1)
    for qkv in (z, torch.zeros((3, 8 * 64 + 8), dtype=torch.bfloat16), torch.zeros((3, 2 * 64), dtype=torch.bfloat16),
                torch.zeros((8 * 64, 3), dtype=torch.bfloat16).t(), torch.zeros((3, 8 * 64))):
        with pytest.raises(a8w8.A8W8Error):
            a8w8._kv_append("paged_kv_append", qkv, None, None, torch.zeros((4, 128)), [], 2, 16, 2, 64, None, None,
                            1e-6, None, None, -1)


def test_binding_refuses_heads_of_another_size_and_rows_too_far_apart():
    import torch
    for dtype in (torch.bfloat16, torch.int8):      # queries of 64 over a cache of 128: whole pages all the same
        z = torch.zeros((32, 2, 128), dtype=dtype)
        with pytest.raises(a8w8.A8W8Error, match=r"\[slots, 2, 64\]"):
            a8w8._cache_rows((z, z), dtype, 2, 64, 16, "x", -1)
        with pytest.raises(a8w8.A8W8Error, match=r"\[slots, 2, 128\]"):
            a8w8._cache_rows((z, z.view(64, 2, 64)), dtype, 2, 128, 16, "x", -1)
    far = torch.empty_strided((2, 6 * 64), (2 ** 32 + 6 * 64, 1), dtype=torch.bfloat16, device="meta")
    assert far.stride(0) % 2 ** 32 == 6 * 64                 # what a 32-bit stride would pass for
    with pytest.raises(a8w8.A8W8Error, match="apart"):
        a8w8._kv_append("paged_kv_append", far, None, None, torch.zeros((4, 128)), [], 2, 16, 2, 64, None, None,
                        1e-6, None, None, far.get_device())


@pytest.mark.parametrize("name", ["kv_append.cu", "attn_chunk.cu", "quant_i4.cuh"])
def test_no_read_only_loads_beside_the_producer(name):
    """These kernels start beside the one before them, which may write what they read: no load of
    theirs goes through the read-only path."""
    import os
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    src = open(os.path.join(root, "w8a8_quantized_decode_gb300", "csrc", name)).read()
    for word in ("__restrict__", "__ldg(", "ld_nc_v4", "ld_stream_v4", ".nc."):
        assert word not in src, f"{name} uses {word}"


# ---------------------------------------------------------------------------
# append (GPU)
# ---------------------------------------------------------------------------

def _empty_cache(kind, n, Hkv, D):
    if kind == "bf16":
        return [np.full((n, Hkv, D), 0x1234, np.uint16) for _ in "kv"]
    if kind == "i8":
        return [np.full((n, Hkv, D), 77, np.int8) for _ in "kv"] + [np.full((n, Hkv), 5, np.float32) for _ in "kv"]
    return [np.full((n, Hkv, D // 2), 0x77, np.uint8) for _ in "kv"] + \
           [np.full((n, Hkv, 2), 0x1234, np.uint16) for _ in "kv"]


def _fill(kind, cache, k, v, slots, live):
    """The oracle's write of rows k, v (BF16 bits) at the live tokens' slots."""
    s = np.where(live, slots, -1).astype(np.int32)
    if kind == "bf16":
        return oracle.kv_write(k, v, s, *cache)
    if kind == "i8":
        return oracle.kv_write_i8(k, v, s, *cache)
    return kv_i4.kv_write(k, v, s, *cache)


def _entry(kind, what):
    names = {"append": ("paged_kv_append", "paged_kv_append_i8", "paged_kv_append_i4"),
             "attention": ("paged_chunk_attention_bf16", "paged_chunk_attention_i8kv", "paged_chunk_attention_i4kv")}
    return getattr(a8w8, names[what][KINDS.index(kind)])


def _same_rows(got, want):
    """Bit for bit, BF16 as values (a zero may carry either sign)."""
    for g, w in zip(got, want):
        g = to_host(g)
        if w.dtype == np.uint16:
            assert np.array_equal(oracle.bf16_to_f64(g), oracle.bf16_to_f64(w), equal_nan=True)
        else:
            assert np.array_equal(g, w)


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T,Hq,Hkv,D,page,norms,extra", [
    (1, 4, 2, 64, 16, "qk", 0), (5, 40, 8, 128, 128, "qk", 0), (7, 3, 1, 128, 5, "k", 16), (33, 5, 5, 64, 24, "", 8),
    (64, 1, 1, 64, 7, "q", 0), (130, 7, 1, 128, 16, "qk", 24), (3, 0, 2, 64, 16, "k", 0)])
def test_append_rows(kind, T, Hq, Hkv, D, page, norms, extra):
    rng = np.random.default_rng(T + D)
    cols = (Hq + 2 * Hkv) * D
    qkv = synth.bf16_normal(T + 7, (T, cols + extra), std=2.0)
    if T > 4:
        qkv[2, :D] = 0                                             # a head of zeros
        qkv[3] = _bf(rng.normal(size=cols + extra) * 2.0 ** -60)   # tiny and huge heads
        qkv[4] = _bf(rng.normal(size=cols + extra) * 2.0 ** 40)
    nblk = -(-T // page) + 2
    n = nblk * page
    slots = rng.permutation(n)[:T].astype(np.int32)
    max_pos = 4000
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    pos[0] = 0
    if T > 6:
        pos[1], slots[5] = -1, -1                                  # a padded row, a row without a place
        pos[6] = max_pos - 1
    w = {c: _bf(rng.normal(1, 0.3, D)) for c in "qk"}
    qw, kw = (w[c] if c in norms else None for c in "qk")
    host = _empty_cache(kind, n, Hkv, D)
    dev = [to_dev(a) for a in host]
    d = to_dev(qkv)[:, :cols]
    a8w8.read_device_errors()
    rope = a8w8.a8w8_rope_table(max_pos, D, THETA)
    q = _entry(kind, "append")(d, to_dev(pos), to_dev(slots), rope, *dev, page,
                               q_norm_w=None if qw is None else to_dev(qw),
                               k_norm_w=None if kw is None else to_dev(kw), eps=1e-6)
    wq, wk, wv, live = chunk.append(qkv, Hq, Hkv, D, pos, max_pos, THETA, qw, kw, 1e-6)
    assert _fill(kind, host, wk, wv, slots, live) == 0
    _same_rows([q] + dev, [wq] + host)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_append_many_rows_have_the_exact_values_rounding(D):
    """Some 10^6 elements, positions to 2^14: every BF16 rounding is the exact value's, also where the
    float32 evaluation cannot tell."""
    T, Hq, Hkv, max_pos = 700, 16, 4, 1 << 14
    rng = np.random.default_rng(D)
    qkv = synth.bf16_normal(D + 1, (T, (Hq + 2 * Hkv) * D), std=3.0)
    pos = rng.integers(0, max_pos, T).astype(np.int32)
    w = _bf(rng.normal(1, 0.2, D))
    cache = [to_dev(np.zeros((T, Hkv, D), np.uint16)) for _ in "kv"]
    rope = a8w8.a8w8_rope_table(max_pos, D, THETA)
    q = a8w8.paged_kv_append(to_dev(qkv), to_dev(pos), to_dev(np.arange(T, dtype=np.int32)), rope, *cache, 1,
                             q_norm_w=to_dev(w), k_norm_w=to_dev(w))
    wq, wk, wv, _ = chunk.append(qkv, Hq, Hkv, D, pos, max_pos, THETA, w, w, 1e-6)
    _same_rows([q] + cache, [wq, wk, wv])


FAR = [
    # (name, exponents of the rows' values, of the weights (None: no norm), eps, position)
    ("norm of large heads", 70, 0, 1e-6, 5), ("norm of the largest heads", 125, 0, 1e-6, 5),
    ("norm of heads of all sizes", (-60, 120), 0, 1e-6, 5), ("norm of tiny heads, no eps", -100, 0, 0.0, 5),
    ("norm of tiny heads, tiny eps", -90, 0, 1e-36, 5), ("large weights", 55, 100, 1e-6, 5),
    ("the largest weights", 0, 126, 1e-6, 5), ("tiny weights", 0, -90, 1e-6, 5),
    ("large eps", 0, 0, 1e30, 5), ("sums past the largest", 126.5, None, 1e-6, 5)]


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("name,size,wsize,eps,at", FAR, ids=[f[0] for f in FAR])
def test_append_of_far_values(kind, D, name, size, wsize, eps, at):
    """Heads whose squares, products with the weight or rotations leave float32's range have the exact
    values' roundings as others (below 2^-100 to the last bit: such values count as equal here)."""
    T, Hq, Hkv = 9, 3, 2
    rng = np.random.default_rng(D)
    shape = (T, (Hq + 2 * Hkv) * D)
    e = rng.integers(*size, shape) if isinstance(size, tuple) else size
    qkv = rng.normal(size=shape) * 2.0 ** e
    qkv[:, (Hq + Hkv) * D:] = rng.normal(size=(T, Hkv * D))
    qkv = _bf(np.clip(qkv, -3e38, 3e38))
    w = None if wsize is None else _bf(np.clip(rng.normal(1, 0.1, D) * 2.0 ** wsize, -3e38, 3e38))
    pos = np.full(T, at, np.int32)
    slots = np.arange(T, dtype=np.int32)
    host = _empty_cache(kind, T, Hkv, D)
    dev = [to_dev(a) for a in host]
    rope = a8w8.a8w8_rope_table(16, D, THETA)
    dw = None if w is None else to_dev(w)
    q = _entry(kind, "append")(to_dev(qkv), to_dev(pos), to_dev(slots), rope, *dev, 1, q_norm_w=dw, k_norm_w=dw,
                               eps=eps)
    with np.errstate(all="ignore"):
        wq, wk, wv, live = chunk.append(qkv, Hq, Hkv, D, pos, 16, THETA, w, w, eps)
    rows, exact = [(q, wq)], []
    if kind == "bf16":
        rows += zip(dev, (wk, wv))
    elif np.isfinite(oracle.bf16_to_f64(wk)).all():
        _fill(kind, host, wk, wv, slots, live)
        exact = [dev, host]
    for g, x in rows:
        g, x = oracle.bf16_to_f64(to_host(g)), oracle.bf16_to_f64(x)
        same = (g == x) | (np.isnan(g) & np.isnan(x)) | (np.maximum(np.abs(g), np.abs(x)) < 2.0 ** -100)
        assert same.all(), (g[~same][:4], x[~same][:4])
    _same_rows(*exact or ([], []))


@gpu
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("at", [0, 5])
def test_append_of_infinities_and_nan(D, norm, at):
    """An infinity or NaN in a head is where the formulas have it: the other values of its pair by the
    rotation alone; of a normed head itself, beside zeros, and all of them with a NaN."""
    T, Hq, Hkv = 6, 3, 2
    qkv = synth.bf16_normal(D, (T, (Hq + 2 * Hkv) * D))
    for t, d, x in ((0, 3, np.inf), (1, D + 40, -np.inf), (2, Hq * D + D // 2, np.inf), (3, Hq * D + 1, np.nan),
                    (4, 0, np.inf), (4, D // 2, np.inf), (5, 7, np.inf), (5, 8, np.nan)):
        qkv[t, d] = _bf(x)
    w = to_dev(_bf(np.random.default_rng(D).normal(1, 0.1, D))) if norm else None
    pos, slots = np.full(T, at, np.int32), np.arange(T, dtype=np.int32)
    cache = [to_dev(a) for a in _empty_cache("bf16", T, Hkv, D)]
    rope = a8w8.a8w8_rope_table(16, D, THETA)
    q = a8w8.paged_kv_append(to_dev(qkv), to_dev(pos), to_dev(slots), rope, *cache, 1, q_norm_w=w, k_norm_w=w)
    hw = None if w is None else to_host(w)
    with np.errstate(all="ignore"):
        wq, wk, wv, _ = chunk.append(qkv, Hq, Hkv, D, pos, 16, THETA, hw, hw, 1e-6)
    assert not np.isfinite(oracle.bf16_to_f64(wq)).all() and not np.isfinite(oracle.bf16_to_f64(wk)).all()
    _same_rows([q] + cache, [wq, wk, wv])


@gpu
def test_append_equals_the_layers_own_rows():
    """The decode layer's taps of its rotated queries and keys, and the cache it wrote, bit for bit."""
    case = synth.decode_layer_case(synth.TINY, 3, np.array([5, 17, 1], np.int32))
    cfg, w = synth.TINY, case["weights"]
    Hq, Hkv, D, page = cfg["num_q_heads"], cfg["num_kv_heads"], cfg["head_dim"], cfg["page_size"]
    rope = a8w8.a8w8_rope_table(64, D, cfg["rope_theta"])
    dw = {k: to_dev(v) for k, v in w.items()}
    kc, vc = to_dev(case["k_cache"]), to_dev(case["v_cache"])
    mine = [kc.clone(), vc.clone()]
    taps = a8w8.make_taps(cfg, 3)
    ws = a8w8.alloc_workspace(cfg, 3, case["block_table"].shape[1])
    slots = to_dev(case["slot_mapping"])
    a8w8.a8w8_decode_layer(dw, cfg, to_dev(case["hidden"]), slots, to_dev(case["block_table"]),
                           to_dev(case["ctx_lens"]), kc, vc, rope, ws, taps=taps)
    q = a8w8.paged_kv_append(taps["qkv"], to_dev(case["ctx_lens"] - 1), slots, rope, *mine, page,
                             q_norm_w=dw["q_norm_w"], k_norm_w=dw["k_norm_w"], eps=cfg["rms_eps"])
    _same_rows([q] + mine, [to_host(taps["q_rot"]), to_host(kc), to_host(vc)])


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_append_flags_and_skips(kind):
    Hq, Hkv, D, page, nblk, max_pos = 2, 1, 64, 16, 2, 32
    qkv = synth.bf16_normal(5, (4, (Hq + 2 * Hkv) * D))
    host = _empty_cache(kind, nblk * page, Hkv, D)
    dev = [to_dev(a) for a in host]
    rope = a8w8.a8w8_rope_table(max_pos, D, THETA)
    a8w8.read_device_errors()
    slots = np.array([nblk * page, 4, 2 ** 31 - 1, 6], np.int32)
    pos = np.array([3, 4, 5, max_pos], np.int32)
    q = _entry(kind, "append")(to_dev(qkv), to_dev(pos), to_dev(slots), rope, *dev, page)
    assert a8w8.read_device_errors() == a8w8.DEVERR_SLOT | a8w8.DEVERR_POS
    wq, wk, wv, live = chunk.append(qkv, Hq, Hkv, D, pos, max_pos, THETA)
    _fill(kind, host, wk, wv, np.where(slots < nblk * page, slots, -1), live)
    _same_rows([q] + dev, [wq] + host)
    assert not to_host(q)[3].any()
    # queries left out; no tokens
    out = _entry(kind, "append")(to_dev(qkv[:0]), to_dev(pos[:0]), to_dev(slots[:0]), rope, *dev, page)
    assert tuple(out.shape) == (0, Hq, D)
    assert a8w8.read_device_errors() == 0


# ---------------------------------------------------------------------------
# attention (GPU)
# ---------------------------------------------------------------------------

def _cache(kind, rng, n, Hkv, D, v_scale=1.0):
    """A cache of random rows, as arrays and as the float64 values that they stand for; v_scale may
    be an array of one factor per slot."""
    if kind == "bf16":
        k = _bf(rng.normal(size=(n, Hkv, D)))
        v = _bf(rng.normal(size=(n, Hkv, D)) * np.reshape(v_scale, (-1, 1, 1)))
        return [k, v], [oracle.bf16_to_f64(k), oracle.bf16_to_f64(v)]
    arrays, values = [], []
    for sc in (1.0, v_scale):
        s = np.reshape(sc, (-1, 1)) * rng.uniform(0.7, 1.3, (n, Hkv))
        if kind == "i8":
            c = np.clip(np.rint(rng.normal(size=(n, Hkv, D)) * 47), -127, 127).astype(np.int8)
            s = (s * 2.7 / 127).astype(np.float32)
            arrays.append((c, s))
            values.append(c * s.astype(np.float64)[..., None])
        else:
            c = rng.integers(0, 256, (n, Hkv, D // 2)).astype(np.uint8)
            m = np.stack((_bf(0.2 * s), _bf(-1.5 * s * rng.uniform(0.8, 1.2, (n, Hkv)))), axis=-1)
            arrays.append((c, m))
            values.append(kv_i4.dequant_rows(c, m))
    return [arrays[0][0], arrays[1][0], arrays[0][1], arrays[1][1]], values


def _case(kind, seed, reqs, Hq, Hkv, D, page, gain=1.5, before=0, behind=0, **cache):
    """reqs: (new tokens, context) of each request; rows of no request before and behind."""
    rng = np.random.default_rng(seed)
    ctx = np.array([c for _, c in reqs], np.int32)
    bt, nblk = synth.paged_layout(seed, np.maximum(ctx, 1), page, spare_blocks=2)
    arrays, values = _cache(kind, rng, nblk * page, Hkv, D, **cache)
    starts = (before + np.concatenate(([0], np.cumsum([n for n, _ in reqs])))).astype(np.int32)
    q = synth.bf16_normal(seed + 1, (int(starts[-1]) + behind, Hq, D), std=gain)
    return q, arrays, values, bt, ctx, starts


def _run(kind, q, arrays, bt, ctx, starts, page, **kw):
    return _entry(kind, "attention")(to_dev(q), *[to_dev(a) for a in arrays], to_dev(bt), to_dev(ctx),
                                     to_dev(starts), page, **kw)


def _check(got, want, bound, owned=None):
    """Within the derived bound plus the BF16 rounding of the result (half a step: 2^-8)."""
    g = oracle.bf16_to_f64(to_host(got))
    if owned is not None:
        g, want, bound = g[owned], want[owned], bound[owned]
    same = (np.isnan(g) & np.isnan(want)) | (g == want)
    odd = ~same & ~(np.isfinite(g) & np.isfinite(want))
    assert not odd.any(), f"not finite in one alone at {np.argwhere(odd)[:4].tolist()}"
    f = np.isfinite(want)                 # (elsewhere the two agree)
    g, want, bound = g[f], want[f], bound[f]
    d = np.abs(g - want)
    tol = bound + (np.abs(want) + bound) * 2.0 ** -8
    bad = ~(d <= tol)
    if bad.any():
        raise AssertionError(f"{bad.sum()} of {d.size} off, worst {np.max(d / np.maximum(tol, 1e-300)):.3g} of the bound")


SHAPES = [
    # (new tokens, context) of the requests, Hq, Hkv, D, page
    ([(5, 37)], 4, 2, 64, 16),
    ([(1, 1)], 8, 8, 128, 128),
    ([(1, 1), (2, 2), (3, 130), (0, 0), (1, 128), (1, 129), (0, 50), (4, 4)], 4, 2, 64, 16),
    ([(25, 25), (26, 26), (51, 51), (52, 300), (103, 103)], 10, 2, 128, 5),
    ([(1, 500), (200, 650), (7, 7), (64, 1000)], 40, 8, 128, 128),
    ([(300, 300)], 8, 1, 128, 48),
    ([(1, 2111), (301, 1700), (17, 18)], 7, 1, 64, 24),
    ([(256, 257), (255, 700)], 12, 12, 64, 1),
    ([(1, c) for c in range(1, 900, 61)], 10, 5, 128, 32),
    ([(4, 200 + 40 * i) for i in range(30)], 16, 2, 128, 64),
    ([(512, 512)] * 2, 6, 2, 128, 96),
    ([(200, 6500), (90, 300)], 5, 1, 128, 128),
    ([(300, 7000), (256, 6200)], 2, 1, 64, 64),
]


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("reqs,Hq,Hkv,D,page", SHAPES)
def test_attention(kind, reqs, Hq, Hkv, D, page):
    import torch
    q, arrays, values, bt, ctx, starts = _case(kind, len(reqs) * 7 + Hq, reqs, Hq, Hkv, D, page)
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, kind=kind)
    a8w8.read_device_errors()
    # a workspace that holds nothing sensible
    need = a8w8.chunk_attention_workspace_bytes(q.shape[0], len(reqs), Hq, Hkv, D, bt.shape[1] * page)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    got = _run(kind, q, arrays, bt, ctx, starts, page, ws=ws)
    _check(got, want, bound, owned)
    assert a8w8.read_device_errors() == 0
    again = _run(kind, q, arrays, bt, ctx, starts, page)
    assert np.array_equal(to_host(got), to_host(again))           # the same bits every time


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_attention_groups(kind, G):
    reqs = [(2, 70), (90, 200), (1, 3)]
    q, arrays, values, bt, ctx, starts = _case(kind, G, reqs, 2 * G, 2, 128, 16)
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, 16, kind=kind)
    _check(_run(kind, q, arrays, bt, ctx, starts, 16), want, bound, owned)


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("what", ["peaked", "scale 0", "negative scale", "tiny v", "huge v", "rising v", "falling v",
                                  "mixed v", "rising scores", "tiny q"])
def test_attention_ranges(kind, what):
    """One token that takes all, scales of either sign and zero, values over wide ranges in any order
    (the INT8 and 4-bit forms' unit of O grows on the way), scores that rise along the context."""
    reqs, Hq, Hkv, D, page = [(60, 700), (1, 300), (9, 9)], 10, 2, 128, 16
    n = sum(-(-c // page) for _, c in reqs) * page + 2 * page
    gain = {"peaked": 30.0, "tiny q": 1e-20}.get(what, 1.5)
    sc = {"scale 0": 0.0, "negative scale": -0.2}.get(what)
    ramp = 10.0 ** np.linspace(-6, 6, n)
    vs = {"tiny v": 1e-25, "huge v": 1e25, "rising v": ramp, "falling v": ramp[::-1],
          "mixed v": 10.0 ** np.random.default_rng(1).uniform(-2, 2, n)}.get(what, 1.0)
    q, arrays, values, bt, ctx, starts = _case(kind, 9, reqs, Hq, Hkv, D, page, gain=gain, v_scale=vs)
    if what in ("rising v", "falling v"):       # pages in order, so that the ramp runs along the contexts
        at = 0
        for b, (_, c) in enumerate(reqs):
            u = -(-c // page)
            bt[b, :u] = np.arange(at, at + u)
            at += u
    if what == "rising scores":
        # keys along the (positive) query, longer and longer: every block's maximum is a new one
        q[:] = _bf(np.abs(oracle.bf16_to_f64(q)))
        t = np.zeros(values[0].shape[0])
        for b, (_, c) in enumerate(reqs):
            p = np.arange(c)
            t[bt[b][p // page] * page + p % page] = p
        if kind == "bf16":
            arrays[0] = _bf(np.broadcast_to((t * 0.02)[:, None, None], values[0].shape))
            values[0] = oracle.bf16_to_f64(arrays[0])
        elif kind == "i8":
            arrays[0][:] = 100
            arrays[2] = np.broadcast_to((t * 0.0002)[:, None], arrays[2].shape).astype(np.float32).copy()
            values[0] = arrays[0] * arrays[2].astype(np.float64)[..., None]
        else:
            arrays[2] = np.stack((_bf(np.zeros(arrays[2].shape[:2])),
                                  _bf(np.broadcast_to((t * 0.02)[:, None], arrays[2].shape[:2]))), axis=-1)
            values[0] = kv_i4.dequant_rows(arrays[0], arrays[2])
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, scale=sc, kind=kind)
    got = _run(kind, q, arrays, bt, ctx, starts, page, softmax_scale=sc)
    _check(got, want, bound, owned)


@gpu
@pytest.mark.parametrize("kind", ["i8", "i4"])
@pytest.mark.parametrize("step", [8, 11, 14, 16, 18, 20])
@pytest.mark.parametrize("which", [0, 1])
def test_small_rows_beside_large_ones(kind, step, which):
    """The second half of each context is 2^step times the first in its keys or its values; the rows
    of the first half see small ones only, which FP16 holds to the stated part of the large ones in
    the same run of 128, their scales and pairs, too."""
    reqs, Hq, Hkv, D, page = [(7, 7), (120, 120), (200, 200), (80, 90)], 10, 2, 128, 16
    q, arrays, values, bt, ctx, starts = _case(kind, 300 + step, reqs, Hq, Hkv, D, page)
    for b, (_, c) in enumerate(reqs):
        t = np.arange(c // 2, c)
        at = bt[b][t // page] * page + t % page
        if kind == "i8":
            arrays[2 + which][at] *= np.float32(2.0 ** step)
        else:
            arrays[2 + which][at] = _bf(oracle.bf16_to_f64(arrays[2 + which][at]) * 2.0 ** step)
    values[which] = (kv_i4.dequant_rows(arrays[which], arrays[2 + which]) if kind == "i4" else
                     arrays[which] * arrays[2 + which].astype(np.float64)[..., None])
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, kind=kind)
    _check(_run(kind, q, arrays, bt, ctx, starts, page), want, bound, owned)


def _poison(kind, arrays, values, which, slot, h, d, x):
    """Value x (an infinity or NaN) into row (slot, h): at dimension d (BF16), or the whole row by its
    scale or pair."""
    if kind == "bf16":
        arrays[which][slot, h, d] = _bf(x)
        values[which][slot, h, d] = x
    elif kind == "i8":
        arrays[2 + which][slot, h] = x
        with np.errstate(invalid="ignore"):
            values[which][slot, h] = arrays[which][slot, h] * np.float64(x)
    else:
        arrays[2 + which][slot, h] = _bf([x, x])
        with np.errstate(invalid="ignore"):
            values[which][slot, h] = kv_i4.dequant_rows(arrays[which], arrays[2 + which])[slot, h]


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("which", [0, 1])
@pytest.mark.parametrize("x", [np.nan, np.inf, -np.inf])
def test_attention_keeps_infinities_and_nan_to_the_rows_that_see_them(kind, which, x):
    """In tokens that a chunk's first rows do not see, of several segments, two in one tile, in the
    cache behind the context, and in the rest of a page."""
    reqs, Hq, Hkv, D, page = [(60, 90), (300, 300), (1, 40), (20, 20)], 10, 2, 128, 16
    q, arrays, values, bt, ctx, starts = _case(kind, 21, reqs, Hq, Hkv, D, page)
    if which == 0 and not np.isnan(x):
        q = _bf(np.abs(oracle.bf16_to_f64(q)))   # an infinite score of one sign
    slot = lambda b, t: bt[b][t // page] * page + t % page  # noqa: E731
    used = {slot(b, t) for b, (_, c) in enumerate(reqs) for t in range(c)}
    for free in set(range(values[0].shape[0])) - used:
        for w in (0, 1):
            _poison(kind, arrays, values, w, free, 0, 3, np.nan)
    for b, t, h, d in ((0, 50, 0, 7), (0, 70, 0, 7), (0, 71, 0, 100), (1, 20, 1, 0), (1, 280, 0, 127), (3, 19, 1, 64)):
        _poison(kind, arrays, values, which, slot(b, t), h, d, x)
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, kind=kind)
    assert np.isfinite(want).mean() > 0.5
    if which == 1 and kind == "bf16":
        assert not np.isfinite(want[20, 0, 7]) and np.isfinite(want[19]).all()
    _check(_run(kind, q, arrays, bt, ctx, starts, page), want, bound, owned)


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_tables_for_long_contexts(D):
    """A table with room for 6144 keys and more takes the longer code over BF16: ragged requests,
    rows that see nothing, values that are not finite, in the same bounds."""
    reqs, Hq, Hkv, page = [(60, 90), (300, 300), (200, 700), (1, 40), (20, 20), (5, 2)], 10, 2, 16
    q, arrays, values, bt, ctx, starts = _case("bf16", 23, reqs, Hq, Hkv, D, page, gain=3.0)
    slot = lambda b, t: bt[b][t // page] * page + t % page  # noqa: E731
    wide = np.pad(bt, ((0, 0), (0, 400 - bt.shape[1])))
    for poisoned in (False, True):
        if poisoned:
            for b, t, h, d, x in ((0, 50, 0, 7, np.nan), (1, 20, 1, 0, np.inf), (1, 280, 0, 63, -np.inf),
                                  (2, 600, 0, 5, np.inf), (2, 601, 0, 5, -np.inf), (4, 19, 1, 33, np.nan)):
                _poison("bf16", arrays, values, 1, slot(b, t), h, d, x)
        want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page)
        _check(_run("bf16", q, arrays, wide, ctx, starts, page), want, bound, owned)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_leaves_other_rows_alone_and_gives_zeros_for_rows_before_the_context(kind):
    import torch
    reqs = [(3, 3), (5, 2), (0, 7), (4, 0), (130, 100)]          # rows before position 0 see nothing
    q, arrays, values, bt, ctx, starts = _case(kind, 31, reqs, 8, 2, 64, 16, before=2, behind=9)
    out = torch.full((q.shape[0], 8, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    got = _run(kind, q, arrays, bt, ctx, starts, 16, out=out)
    assert got is out
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, 16, kind=kind)
    _check(got, want, bound, owned)
    g = oracle.bf16_to_f64(to_host(got))
    assert (g[~owned] == 3.0).all() and (~owned).sum() == 11
    assert not g[5:8].any() and not g[10:14].any() and not g[14:44].any()
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("B", [513, 1300])
def test_attention_of_many_requests(kind, B):
    """More requests than threads: several a thread in the search for a part."""
    reqs = [(i * 7 % 4, 4 + i * 37 % 290) for i in range(B)]
    q, arrays, values, bt, ctx, starts = _case(kind, B, reqs, 4, 2, 64, 16)
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, 16, kind=kind)
    _check(_run(kind, q, arrays, bt, ctx, starts, 16), want, bound, owned)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_of_nothing(kind):
    """Requests without a row, no request, no row: out stays as it is."""
    import torch
    q, arrays, values, bt, ctx, starts = _case(kind, 3, [(0, 5), (0, 0), (0, 200)], 4, 2, 64, 16, behind=3)
    out = torch.full((3, 4, 64), 2.0, dtype=torch.bfloat16, device="cuda")
    _run(kind, q, arrays, bt, ctx, starts, 16, out=out)
    assert (out == 2.0).all()
    _run(kind, q, arrays, bt[:0], ctx[:0], starts[:1], 16, out=out)
    assert (out == 2.0).all()
    assert tuple(_run(kind, q[:0], arrays, bt, ctx, starts, 16).shape) == (0, 4, 64)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_two_calls_at_once(kind):
    """On two streams, each with its own workspace, and again on one behind the other."""
    import torch
    cases = [_case(kind, 11, [(90, 700), (3, 1500)], 10, 2, 128, 16), _case(kind, 12, [(1, 900)] * 9, 8, 8, 128, 128)]
    wants = [chunk.attention(c[0], *c[2], *c[3:], page, kind=kind) for c, page in zip(cases, (16, 128))]
    devs = [[to_dev(a) for a in (c[0], *c[1], *c[3:])] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(3):
        outs = [_entry(kind, "attention")(*d, page, stream=s) for d, page, s in zip(devs, (16, 128), streams)]
        torch.cuda.synchronize()
        one = [_entry(kind, "attention")(*d, page) for d, page in zip(devs, (16, 128))]
        for got in (outs, one):
            for g, w in zip(got, wants):
                _check(g, *w)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_flags_bad_tables(kind):
    reqs = [(40, 100), (3, 60), (6, 30)]
    q, arrays, values, bt, ctx, starts = _case(kind, 41, reqs, 4, 2, 64, 16)
    a8w8.read_device_errors()
    bad = bt.copy()
    bad[0, 2], bad[1, 0] = 10 ** 6, -1            # rows of zeros
    want, bound, owned = chunk.attention(q, *values, bad, ctx, starts, 16, kind=kind)
    _check(_run(kind, q, arrays, bad, ctx, starts, 16), want, bound, owned)
    assert a8w8.read_device_errors() == a8w8.DEVERR_BLOCK
    for c in (-3, bt.shape[1] * 16 + 1, 2 ** 31 - 1):
        odd = ctx.copy()
        odd[1] = c
        want, bound, owned = chunk.attention(q, *values, bt, odd, starts, 16, kind=kind)
        _check(_run(kind, q, arrays, bt, odd, starts, 16), want, bound, owned)
        assert a8w8.read_device_errors() == a8w8.DEVERR_CTX
    for st in ([0, 40, 43, 60], [-5, 35, 38, 44], [0, 40, 30, 36], [0, 40, 2 ** 31 - 1, -(2 ** 31)]):
        _run(kind, q, arrays, bt, ctx, np.array(st, np.int32), 16)
        assert a8w8.read_device_errors() == a8w8.DEVERR_ROW
    # bad entries beyond the context are nobody's
    bad = bt.copy()
    bad[2, 2:] = 10 ** 6
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, 16, kind=kind)
    _check(_run(kind, q, arrays, bad, ctx, starts, 16), want, bound, owned)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_as_a_replayed_graph_on_another_stream(kind):
    """Captured once, replayed with other rows, contexts and starts in the same buffers; two graphs
    with workspaces of their own in turn."""
    import torch
    Hq, Hkv, D, page = 10, 2, 128, 16
    shapes = [[(30, 200), (1, 77), (9, 40)], [(1, 150), (38, 60), (1, 1)]]
    cases = [_case(kind, 50 + i, r, Hq, Hkv, D, page) for i, r in enumerate(shapes)]
    T, M = 40, 13
    pool = max(c[3].max() + 1 for c in cases) + 2
    dev = None
    graphs = []
    st = torch.cuda.Stream()
    for rep in (0, 1, 0, 1):
        q, arrays, values, bt, ctx, starts = cases[rep]
        full = np.zeros((3, M), np.int32)
        full[:, :bt.shape[1]] = bt[:, :M]
        host = [q] + [np.concatenate((a, np.zeros((pool * page - a.shape[0],) + a.shape[1:], a.dtype)))
                      if a.shape[0] < pool * page else a[:pool * page] for a in arrays] + [full, ctx, starts]
        if dev is None:
            dev = [to_dev(a) for a in host]
            with torch.cuda.stream(st):
                for _ in range(2):
                    need = a8w8.chunk_attention_workspace_bytes(T, 3, Hq, Hkv, D, M * page)
                    ws = torch.empty(need, dtype=torch.uint8, device="cuda")
                    out = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
                    call = lambda: _entry(kind, "attention")(*dev, page, ws=ws, out=out)  # noqa: E731
                    call()
                    torch.cuda.synchronize()
                    g = torch.cuda.CUDAGraph()
                    with torch.cuda.graph(g, stream=st):
                        call()
                    graphs.append((g, out, ws))
        for d, a in zip(dev, host):
            d.copy_(to_dev(a))
        torch.cuda.synchronize()
        want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, kind=kind)
        for g, out, _ in graphs:
            out.zero_()
            torch.cuda.synchronize()
            with torch.cuda.stream(st):
                g.replay()
            st.synchronize()
            _check(out, want, bound, owned)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_on_a_given_stream(kind):
    import torch
    q, arrays, values, bt, ctx, starts = _case(kind, 61, [(20, 100), (1, 30)], 4, 2, 64, 16)
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, 16, kind=kind)
    dev = [to_dev(a) for a in (q, *arrays, bt, ctx, starts)]
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = _entry(kind, "attention")(*dev, 16, stream=st)
    st.synchronize()
    _check(got, want, bound, owned)


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_attention_long_prompt(kind):
    """4096 tokens past 300 at 40 / 8 heads of 128, in one call and in two: some rows against the
    oracle, each as a single token with the context that it sees."""
    import torch
    n, prior, Hq, Hkv, D, page = 4096, 300, 40, 8, 128, 128
    q, arrays, values, bt, ctx, starts = _case(kind, 91, [(n, n + prior)], Hq, Hkv, D, page)
    rows = np.array([0, 1, 50, 51, 127, 128, 1000, 2047, 2048, 3333, n - 2, n - 1])
    want, bound, _ = chunk.attention(q[rows], *values, np.repeat(bt, len(rows), 0), prior + 1 + rows,
                                     np.arange(len(rows) + 1), page, kind=kind)
    pick = torch.from_numpy(rows).cuda()
    got = _run(kind, q, arrays, bt, ctx, starts, page)
    _check(got[pick], want, bound)
    cut = 1999
    parts = [_run(kind, q[a:b], arrays, bt, np.array([prior + b], np.int32), np.array([0, b - a], np.int32), page)
             for a, b in ((0, cut), (cut, n))]
    _check(torch.cat(parts)[pick], want, bound)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("D", [64, 128])
def test_attention_prompt_of_8192_tokens(D):
    """A BF16 prompt long enough for the longer code, whole: some rows against the oracle."""
    import torch
    n, Hq, Hkv, page = 8192, 40, 8, 128
    q, arrays, values, bt, ctx, starts = _case("bf16", 92, [(n, n)], Hq, Hkv, D, page)
    rows = np.array([0, 1, 51, 127, 128, 4095, 4096, 6143, n - 2, n - 1])
    want, bound, _ = chunk.attention(q[rows], *values, np.repeat(bt, len(rows), 0), 1 + rows,
                                     np.arange(len(rows) + 1), page)
    got = _run("bf16", q, arrays, bt, ctx, starts, page)
    _check(got[torch.from_numpy(rows).cuda()], want, bound)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_append_of_a_long_chunk(kind):
    """8192 tokens of 40 / 8 heads, a warp all heads of a token: some rows bit for bit, pages in any
    order."""
    import torch
    T, Hq, Hkv, D, page, first = 8192, 40, 8, 128, 128, 1234
    rng = np.random.default_rng(93)
    qkv = synth.bf16_normal(93, (T, (Hq + 2 * Hkv) * D), std=2.0)
    slots = (rng.permutation(T // page)[:, None] * page + np.arange(page)).reshape(-1).astype(np.int32)
    pos = np.arange(first, first + T, dtype=np.int32)
    w = _bf(rng.normal(1, 0.2, D))
    dev = [to_dev(a) for a in _empty_cache(kind, T, Hkv, D)]
    rope = a8w8.a8w8_rope_table(first + T, D, THETA)
    q = _entry(kind, "append")(to_dev(qkv), to_dev(pos), to_dev(slots), rope, *dev, page, q_norm_w=to_dev(w),
                               k_norm_w=to_dev(w))
    rows = np.concatenate(([0, 1, T - 1], rng.permutation(T)[:60]))
    wq, wk, wv, live = chunk.append(qkv[rows], Hq, Hkv, D, pos[rows], first + T, THETA, w, w)
    small = _empty_cache(kind, len(rows), Hkv, D)
    _fill(kind, small, wk, wv, np.arange(len(rows)), live)
    at = torch.from_numpy(slots[rows]).long().cuda()
    _same_rows([q[torch.from_numpy(rows).cuda()]] + [c[at] for c in dev], [wq] + small)


@gpu
@pytest.mark.slow
@pytest.mark.parametrize("kind", KINDS)
def test_offsets_past_32_bits(kind):
    """Pages at the end of a pool whose rows lie past 2^32 bytes (and 2^31 elements)."""
    import torch
    Hq, Hkv, D, page = 10, 5, 128, 128
    slots = {"bf16": 3_600_000, "i8": 7_000_000, "i4": 14_000_000}[kind] // page * page
    u, w = {"bf16": (torch.int16, D), "i8": (torch.int8, D), "i4": (torch.uint8, D // 2)}[kind]
    dev = [torch.zeros((slots, Hkv, w), dtype=u, device="cuda") for _ in "kv"]
    assert dev[0].numel() * dev[0].element_size() > 2 ** 32
    if kind == "i8":
        dev += [torch.zeros((slots, Hkv), device="cuda") for _ in "kv"]
    elif kind == "i4":
        dev += [torch.zeros((slots, Hkv, 2), dtype=torch.int16, device="cuda") for _ in "kv"]
    reqs = [(70, 300), (1, 129)]
    q, arrays, values, bt, ctx, starts = _case(kind, 71, reqs, Hq, Hkv, D, page)
    far = bt + slots // page - 1 - bt.max()
    for d, a in zip(dev, arrays):
        t = to_dev(a)
        n = (bt.max() + 1) * page
        d[-n:].copy_(t[:n].view(d.dtype))
    bf = torch.bfloat16
    cache = [d.view(bf) if d.dtype == torch.int16 else d for d in dev]
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, kind=kind)
    got = _entry(kind, "attention")(to_dev(q), *cache, to_dev(far.astype(np.int32)), to_dev(ctx), to_dev(starts), page)
    _check(got, want, bound, owned)
    # and the rows of an append land there
    qkv = synth.bf16_normal(72, (3, (Hq + 2 * Hkv) * D))
    at = np.array([slots - 1, slots - 5, slots // 2 + 7], np.int32)
    pos = np.arange(3, dtype=np.int32)
    rope = a8w8.a8w8_rope_table(16, D, THETA)
    _entry(kind, "append")(to_dev(qkv), to_dev(pos), to_dev(at), rope, *cache, page)
    _, wk, wv, live = chunk.append(qkv, Hq, Hkv, D, pos, 16, THETA)
    small = _empty_cache(kind, 3, Hkv, D)
    _fill(kind, small, wk, wv, np.arange(3), live)
    _same_rows([c[torch.from_numpy(at).long().cuda()] for c in cache], small)


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,G", [(64, 2), (128, 5)])
def test_neighbouring_narrow_tiles_keep_their_own_statistics(kind, D, G):
    """Tiles of 128 rows and fewer, of one and two blocks of keys, several to a CTA one behind the
    other, whose scores and values are of very different sizes: each row is joined with its own
    tile's statistics, in every call."""
    rng = np.random.default_rng(D)
    reqs = [(int(rng.integers(1, 5)), int(rng.integers(5, 250))) for _ in range(100)]
    Hkv, page = 8, 16
    n = sum(-(-c // page) for _, c in reqs) * page + 2 * page
    q, arrays, values, bt, ctx, starts = _case(kind, 17, reqs, Hkv * G, Hkv, D, page,
                                               v_scale=10.0 ** rng.uniform(-3, 3, n))
    size = np.repeat(2.0 ** rng.integers(-4, 4, len(reqs)), [m for m, _ in reqs])
    q = _bf(oracle.bf16_to_f64(q) * size[:, None, None])
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, kind=kind)
    a8w8.read_device_errors()
    dev = [to_dev(a) for a in (q, *arrays, bt, ctx, starts)]
    first = _entry(kind, "attention")(*dev, page)
    _check(first, want, bound, owned)
    for _ in range(100):
        assert (_entry(kind, "attention")(*dev, page) == first).all()
    assert a8w8.read_device_errors() == 0


def _poison_tokens(kind, arrays, values, bt, page, tokens):
    """(request, token, kind of value) of `tokens`: infinities and NaN there in every KV head's values."""
    for b, t, x in tokens:
        at = slice(bt[b][t // page] * page + t % page, None)
        a, v = [c[at][:1] for c in arrays], [c[at][:1] for c in values]      # (views of the one slot)
        for h in range(values[1].shape[1]):
            _poison(kind, a, v, 1, 0, h, (7 * t + 3 * h) % values[1].shape[2], x)


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("D,G", [(64, 2), (128, 5)])
def test_values_that_are_not_finite_in_neighbouring_tiles(kind, D, G):
    """Every tile of a CTA holds some that only part of its rows see, in rows that different warps
    bring: no tile waits for a later one."""
    rng = np.random.default_rng(D + 1)
    reqs = [(n, int(rng.integers(n, 129))) for n in rng.integers(2, 60, 72).tolist()]
    Hkv, page = 8, 16
    q, arrays, values, bt, ctx, starts = _case(kind, 19, reqs, Hkv * G, Hkv, D, page)
    odd = [(b, int(rng.integers(c - n + 1, c)), rng.choice([np.nan, np.inf, -np.inf]))
           for b, (n, c) in enumerate(reqs) for _ in range(3) if b % 9]
    _poison_tokens(kind, arrays, values, bt, page, odd)
    want, bound, owned = chunk.attention(q, *values, bt, ctx, starts, page, kind=kind)
    assert 0.2 < np.isfinite(want).mean() < 0.99
    a8w8.read_device_errors()
    dev = [to_dev(a) for a in (q, *arrays, bt, ctx, starts)]
    for _ in range(20):
        got = _entry(kind, "attention")(*dev, page)
    _check(got, want, bound, owned)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("n,prior,G,D", [(8, 122, 2, 128), (4, 126, 5, 64), (60, 100, 2, 64), (3, 126, 4, 128),
                                         (30, 230, 1, 128)])
def test_values_that_are_not_finite_in_narrow_tiles_across_a_block(kind, n, prior, G, D):
    """Neighbouring tiles of two and three blocks of keys whose first block with unseen tokens holds
    such values, in every KV head: what a tile notes of them waits for the last one's notes to be
    read, and for nothing behind it."""
    B, Hkv, page = 48, 8, 16
    ctx = n + prior
    q, arrays, values, bt, ctxs, starts = _case(kind, 29, [(n, ctx)] * B, Hkv * G, Hkv, D, page)
    last = prior + 1 | 1                    # in the block of the first unseen token, behind it
    odd = [(b, t, x) for b in range(B) if b % 8 for t, x in ((last, np.nan if b % 2 else np.inf), (ctx - 1, -np.inf))]
    _poison_tokens(kind, arrays, values, bt, page, odd)
    want, bound, owned = chunk.attention(q, *values, bt, ctxs, starts, page, kind=kind)
    assert prior < last < ctx and 0.1 < np.isfinite(want).mean() < 1
    a8w8.read_device_errors()
    dev = [to_dev(a) for a in (q, *arrays, bt, ctxs, starts)]
    for _ in range(20):
        got = _entry(kind, "attention")(*dev, page)
    _check(got, want, bound, owned)
    assert a8w8.read_device_errors() == 0


# ---------------------------------------------------------------------------
# together (GPU)
# ---------------------------------------------------------------------------

@gpu
@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_in_chunks_then_decoded_tokens(kind):
    """Two sequences grow chunk by chunk through append and attention, the last tokens one at a time:
    every row is the oracle's on the whole sequence, and the decode attention agrees on the last."""
    Hq, Hkv, D, page, max_pos = 10, 2, 128, 16, 512
    rng = np.random.default_rng(81)
    plan = [(70, 0), (130, 33), (1, 64), (1, 1), (3, 1)]         # new tokens of the two sequences, turn by turn
    total = np.array([sum(p[b] for p in plan) for b in (0, 1)], np.int32)
    bt, nblk = synth.paged_layout(82, total, page, spare_blocks=1)
    qkv = [synth.bf16_normal(83 + b, (int(total[b]), (Hq + 2 * Hkv) * D), std=1.3) for b in (0, 1)]
    w = _bf(rng.normal(1, 0.1, D))
    host = _empty_cache(kind, nblk * page, Hkv, D)
    dev = [to_dev(a) for a in host]
    rope = a8w8.a8w8_rope_table(max_pos, D, THETA)
    ctx = np.zeros(2, np.int32)
    a8w8.read_device_errors()
    for new in plan:
        pos = [np.arange(ctx[b], ctx[b] + new[b]) for b in (0, 1)]
        slots = np.concatenate([synth.slots_for(np.repeat(bt[b][None], max(len(pos[b]), 1), 0), pos[b], page)
                                if len(pos[b]) else np.zeros(0, np.int32) for b in (0, 1)]).astype(np.int32)
        rows = np.concatenate([qkv[b][pos[b]] for b in (0, 1)])
        flat = np.concatenate(pos).astype(np.int32)
        ctx = ctx + np.array(new, np.int32)
        starts = np.array([0, new[0], new[0] + new[1]], np.int32)
        q = _entry(kind, "append")(to_dev(rows), to_dev(flat), to_dev(slots), rope, *dev, page,
                                   q_norm_w=to_dev(w), k_norm_w=to_dev(w))
        got = _entry(kind, "attention")(q, *dev, to_dev(bt), to_dev(ctx), to_dev(starts), page)
        wq, wk, wv, live = chunk.append(rows, Hq, Hkv, D, flat, max_pos, THETA, w, w, 1e-6)
        assert _fill(kind, host, wk, wv, slots, live) == 0
        _same_rows([q] + dev, [wq] + host)
        if kind == "bf16":
            values = [oracle.bf16_to_f64(a) for a in host]
        elif kind == "i8":
            values = [host[i] * host[2 + i].astype(np.float64)[..., None] for i in (0, 1)]
        else:
            values = [kv_i4.dequant_rows(host[i], host[2 + i]) for i in (0, 1)]
        want, bound, owned = chunk.attention(wq, *values, bt, ctx, starts, page, kind=kind)
        _check(got, want, bound, owned)
    # the decode attention of the last tokens' queries: the same values within both bounds
    decode = {"bf16": a8w8.paged_decode_attention_bf16, "i8": a8w8.paged_decode_attention_i8kv,
              "i4": a8w8.paged_decode_attention_i4kv}[kind]
    last = starts[1:] - 1
    one = decode(q[to_dev(last).long()].contiguous(), *dev, to_dev(bt), to_dev(ctx), page)
    a, b = (oracle.bf16_to_f64(to_host(x)) for x in (one, got[to_dev(last).long()]))
    assert (np.abs(a - b) <= 2 * bound[last] + 2.0 ** -7 * np.abs(want[last]) + 2.0 ** -9 * np.abs(want[last]).max()).all()
    assert a8w8.read_device_errors() == 0
