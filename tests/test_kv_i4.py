"""The 4-bit KV cache: quantise-on-write, read-back and decode attention.

On the CPU: the float64 oracle (oracle/kv_i4.py) against hand-computed rows,
the C oracle's BF16 attention and its own invariants, and the refusals of the
entry points. On the GPU: written codes and pairs bit for bit, read-back bit
for bit, and attention within bounds derived from its arithmetic.
"""
import numpy as np
import pytest

import oracle
import synth
import w8a8_quantized_decode_gb300 as a8w8
from gpu_util import to_dev, to_host
from oracle import kv_i4

gpu = pytest.mark.gpu
FAKE = 0x10000


@pytest.fixture(scope="module")
def lib():
    a8w8.build()
    return a8w8.lib()


def _bf(x):
    return kv_i4.f32_to_bf16(np.asarray(x, np.float32))


# ---------------------------------------------------------------------------
# oracle pins (CPU)
# ---------------------------------------------------------------------------

def test_rows_by_hand():
    codes, meta = kv_i4.quant_rows(_bf(np.arange(16)))           # s = 1, m = 0: the codes themselves
    assert kv_i4.unpack(codes).tolist() == list(range(16))
    assert kv_i4.bf16_to_f64(meta).tolist() == [1.0, 0.0]
    assert codes[0] == 0x10 and codes[7] == 0xFE                 # element 2j in the low nibble
    # ties to even: s = 1, values k + 1/2 between the ends -2 and 13
    row = np.array([-2, 13, -1.5, -0.5, 0.5, 1.5, 2.5, 3.5], np.float32)
    codes, meta = kv_i4.quant_rows(_bf(row))
    assert kv_i4.bf16_to_f64(meta).tolist() == [1.0, -2.0]
    assert kv_i4.unpack(codes).tolist() == [0, 15, 0, 2, 2, 4, 4, 6]
    # a constant row has s = 0 and reads back exactly
    codes, meta = kv_i4.quant_rows(_bf(np.full(8, 2.71875)))
    assert not codes.any() and (kv_i4.dequant_rows(codes, meta) == 2.71875).all()


@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_rows_that_hold_no_finite_range(bad):
    row = np.ones(8, np.float32)
    row[3] = bad
    codes, meta = kv_i4.quant_rows(_bf(row))
    assert not codes.any() and np.isnan(kv_i4.dequant_rows(codes, meta)).all()
    row = np.array([3e38, -3e38] * 4, np.float32)                # the range overflows float32
    assert np.isnan(kv_i4.dequant_rows(*kv_i4.quant_rows(_bf(row)))).all()


def test_quantisation_error_is_half_a_step():
    """|x^ - x| <= s / 2 + 15 s 2^-8 (s is a BF16 rounding of range / 15, so the top code may
    stand up to 15 s 2^-8 off), plus the float32 roundings of the quotient."""
    for seed, std in ((1, 1.0), (2, 1e-3), (3, 300.0)):
        x = synth.bf16_normal(seed, (200, 128), std=std)
        codes, meta = kv_i4.quant_rows(x)
        s = kv_i4.bf16_to_f64(meta)[:, :1]
        err = np.abs(kv_i4.dequant_rows(codes, meta) - kv_i4.bf16_to_f64(x))
        assert (err <= s * (0.5 + 15 * 2.0 ** -8 + 2.0 ** -18)).all()
        assert (kv_i4.unpack(codes).max(1) >= 14).all() and (kv_i4.unpack(codes).min(1) == 0).all()


def test_attention_oracle_equals_the_bf16_oracle_on_exact_rows():
    """Pairs with s = 2^e and m a small multiple of it give values that BF16 holds, so the C
    oracle's attention over a BF16 cache of those values must agree to its one rounding."""
    rng = np.random.default_rng(5)
    B, Hq, Hkv, D, page = 3, 6, 2, 64, 16
    ctx = np.array([37, 1, 0], np.int32)
    bt, nblk = synth.paged_layout(6, np.maximum(ctx, 1), page, spare_blocks=1)
    n = nblk * page
    kc, vc = (rng.integers(0, 256, (n, Hkv, D // 2)).astype(np.uint8) for _ in range(2))
    km, vm = (np.stack((_bf(2.0 ** rng.integers(-3, 1, (n, Hkv))),
                        _bf(-rng.integers(0, 8, (n, Hkv)))), axis=-1) for _ in range(2))
    q = synth.bf16_normal(7, (B, Hq, D))
    out, bound = kv_i4.attention(q, kc, vc, km, vm, bt, ctx, page)
    kb, vb = (_bf(kv_i4.dequant_rows(c, m)) for c, m in ((kc, km), (vc, vm)))
    assert (kv_i4.bf16_to_f64(kb) == kv_i4.dequant_rows(kc, km)).all()
    ref, rc = oracle.paged_attention(q, kb, vb, bt, ctx, page)
    ref = kv_i4.bf16_to_f64(ref)
    assert rc == 0 and (np.abs(out - ref) <= np.abs(out) * 2.0 ** -8 + 1e-12).all()
    assert not out[2].any() and (bound[:2] > 0).all()


# ---------------------------------------------------------------------------
# refusals (CPU)
# ---------------------------------------------------------------------------

def test_write_and_read_validation(lib):
    w = lambda k=FAKE, D=128, T=2, Hkv=8, km=FAKE, page=16: lib.paged_kv_write_i4(  # noqa: E731
        k, FAKE, T, Hkv, D, FAKE, FAKE, FAKE, km, FAKE, 4, page, None)
    r = lambda k=FAKE, D=128, T=2, Hkv=8, km=FAKE, page=16: lib.paged_kv_read_i4(  # noqa: E731
        FAKE, FAKE, km, FAKE, 4, page, FAKE, T, Hkv, D, k, FAKE, None)
    for f in (w, r):
        assert f(D=96) == a8w8.ERR_UNSUPPORTED_SHAPE
        assert f(T=1 << 30, Hkv=8) == a8w8.ERR_UNSUPPORTED_SHAPE
        assert f(T=-1) == a8w8.ERR_INVALID_ARG
        assert f(Hkv=0) == a8w8.ERR_INVALID_ARG
        assert f(page=0) == a8w8.ERR_INVALID_ARG
        assert f(k=None) == a8w8.ERR_INVALID_ARG
        assert f(km=FAKE + 4) == a8w8.ERR_INVALID_ARG
        assert f(T=0, k=None) == a8w8.OK


def test_attention_validation(lib):
    def f(D=128, Hq=16, Hkv=2, ws=FAKE, wsb=1 << 30, km=FAKE, B=2, page=128, max_blocks=40):
        return lib.paged_decode_attention_i4kv(FAKE, FAKE, FAKE, km, FAKE, FAKE, FAKE, B, Hq, Hkv,
                                               D, page, max_blocks, 100, 0.1, FAKE, ws, wsb, None)
    assert f(D=96) == a8w8.ERR_UNSUPPORTED_SHAPE
    assert f(Hq=18) == a8w8.ERR_UNSUPPORTED_SHAPE      # more than 8 heads a group
    assert f(Hq=15) == a8w8.ERR_UNSUPPORTED_SHAPE
    assert f(max_blocks=1 << 18) == a8w8.ERR_UNSUPPORTED_SHAPE
    assert f(B=65536) == a8w8.ERR_UNSUPPORTED_SHAPE
    assert f(km=None) == a8w8.ERR_INVALID_ARG
    assert f(B=-1) == a8w8.ERR_INVALID_ARG
    assert f(page=0) == a8w8.ERR_INVALID_ARG
    assert f(B=0, km=None) == a8w8.OK
    need = lib.a8w8_attention_i4_workspace_bytes(2, 16, 2, 128, 40 * 128)
    if need:
        assert f(ws=None) == a8w8.ERR_WORKSPACE
        assert f(wsb=need - 1) == a8w8.ERR_WORKSPACE
        assert f(ws=FAKE + 8) == a8w8.ERR_WORKSPACE
    assert lib.a8w8_attention_i4_workspace_bytes(0, 16, 2, 128, 4096) == 0
    assert lib.a8w8_attention_i4_workspace_bytes(1, 16, 3, 128, 4096) == 0


def test_binding_refuses_wrong_tensors():
    import torch
    t = torch.zeros(4, dtype=torch.int64)
    with pytest.raises(a8w8.A8W8Error, match="int32"):
        a8w8._typed(t, torch.int32, "x", -1)
    with pytest.raises(a8w8.A8W8Error, match="codes"):
        z = torch.zeros((32, 2, 32), dtype=torch.uint8)
        m = torch.zeros((32, 2, 2), dtype=torch.bfloat16)
        a8w8._cache_i4(z, z, m, m[:31], 2, 64, 16, "x", -1)


def test_binding_refuses_a_cache_of_no_heads():
    import torch
    z = torch.zeros((32, 0, 32), dtype=torch.uint8)
    m = torch.zeros((32, 0, 2), dtype=torch.bfloat16)
    with pytest.raises(a8w8.A8W8Error, match="codes"):
        a8w8._cache_i4(z, z, m, m, 0, 64, 16, "x", -1)


# ---------------------------------------------------------------------------
# write and read (GPU)
# ---------------------------------------------------------------------------

def _cache(rng, n, Hkv, D, k_scale=0.35, v_scale=0.35):
    """Random codes and pairs; a scale may be an array of one value per slot."""
    out = []
    for sc in (k_scale, v_scale):
        out.append(rng.integers(0, 256, (n, Hkv, D // 2)).astype(np.uint8))
        s = np.reshape(sc, (-1, 1)) * rng.uniform(0.7, 1.3, (n, Hkv))
        out.append(np.stack((_bf(s), _bf(-7.5 * s * rng.uniform(0.85, 1.15, (n, Hkv)))), axis=-1))
    kc, km, vc, vm = out
    return kc, vc, km, vm


@gpu
@pytest.mark.parametrize("T,Hkv,D,page", [(1, 2, 64, 16), (7, 8, 128, 128), (5, 1, 128, 5),
                                          (33, 3, 64, 24), (257, 5, 128, 16)])
def test_write_and_read_exact(T, Hkv, D, page):
    rng = np.random.default_rng(T)
    nblk = -(-T // page) + 2
    n = nblk * page
    k = synth.bf16_normal(T + 1, (T, Hkv, D))
    v = synth.bf16_normal(T + 2, (T, Hkv, D), std=3.0)
    slots = rng.permutation(n)[:T].astype(np.int32)
    if T > 4:
        slots[1] = -1
        k[0, 0] = 0                                        # constant rows: s = 0
        v[2, 0] = _bf(np.full(D, -1.75))
        k[3, 0] = _bf(np.where(np.arange(D) % 3 == 0, 1e-39, 0))       # subnormal range
        v[3, 0] = _bf(np.linspace(-3e38, 2.9e37, D))       # range near the end of float32
        k[4, 0] = _bf(rng.normal(size=D) * 2.0 ** -120)    # quotients by the division
        v[4, 0, 1] = _bf(np.nan)
    host = list(_cache(rng, n, Hkv, D))
    dev = [to_dev(a) for a in host]
    a8w8.read_device_errors()
    a8w8.paged_kv_write_i4(to_dev(k), to_dev(v), to_dev(slots), *dev, page)
    want = [a.copy() for a in host]
    assert kv_i4.kv_write(k, v, slots, *want) == 0
    got = [to_host(d) for d in dev]
    for g, w in zip(got[:2], want[:2]):
        assert np.array_equal(g, w)
    for g, w in zip(got[2:], want[2:]):      # as values: a minimum of zero may carry either sign
        assert np.array_equal(kv_i4.bf16_to_f64(g), kv_i4.bf16_to_f64(w), equal_nan=True)
    # read back, a slot twice and a padded one
    at = np.concatenate((slots, slots[:1], [-1])).astype(np.int32)
    gk, gv = (to_host(x) for x in a8w8.paged_kv_read_i4(*dev, to_dev(at), page))
    for g, c, m in ((gk, got[0], got[2]), (gv, got[1], got[3])):
        with np.errstate(over="ignore"):
            x = kv_i4.dequant_rows(c[np.maximum(at, 0)], m[np.maximum(at, 0)]).astype(np.float32)
        x[at < 0] = 0
        assert np.array_equal(kv_i4.bf16_to_f64(g), kv_i4.bf16_to_f64(_bf(x)), equal_nan=True)
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("exponent", [0, -60, 50])
def test_write_many_rows_exact(exponent):
    """200,000 rows: every code at or next to a rounding boundary as the definition has it."""
    T, Hkv, D, page = 25000, 4, 64, 50
    rng, std = np.random.default_rng(exponent + 100), 2.0 ** exponent
    k = synth.bf16_normal(1, (T, Hkv, D), std=std)
    # rows of small integers times a power of two: quotients that are exact halves
    v = _bf(rng.integers(-30, 31, (T, Hkv, D)) * std)
    host = [np.zeros((T, Hkv, w), t) for w, t in
            ((D // 2, np.uint8), (D // 2, np.uint8), (2, np.uint16), (2, np.uint16))]
    dev = [to_dev(a) for a in host]
    a8w8.paged_kv_write_i4(to_dev(k), to_dev(v), to_dev(np.arange(T, dtype=np.int32)), *dev, page)
    for x, c, m in ((k, dev[0], dev[2]), (v, dev[1], dev[3])):
        wc, wm = kv_i4.quant_rows(x)
        assert np.array_equal(to_host(c), wc)
        assert np.array_equal(kv_i4.bf16_to_f64(to_host(m)), kv_i4.bf16_to_f64(wm))


@gpu
def test_slots_out_of_range_are_flagged_and_skipped():
    Hkv, D, page, nblk = 2, 64, 16, 2
    k = synth.bf16_normal(5, (3, Hkv, D))
    host = list(_cache(np.random.default_rng(1), nblk * page, Hkv, D))
    dev = [to_dev(a) for a in host]
    slots = np.array([nblk * page, 4, 2 ** 31 - 1], np.int32)
    a8w8.read_device_errors()
    a8w8.paged_kv_write_i4(to_dev(k), to_dev(k), to_dev(slots), *dev, page)
    assert a8w8.read_device_errors() == a8w8.DEVERR_SLOT
    want = [a.copy() for a in host]
    assert kv_i4.kv_write(k, k, slots, *want) == 2
    for d, w in zip(dev, want):
        assert np.array_equal(to_host(d), w)
    gk, gv = a8w8.paged_kv_read_i4(*dev, to_dev(slots), page)
    assert a8w8.read_device_errors() == a8w8.DEVERR_SLOT
    assert not to_host(gk)[[0, 2]].any() and to_host(gk)[1].any()
    # no tokens: nothing happens
    a8w8.paged_kv_write_i4(to_dev(k[:0]), to_dev(k[:0]), to_dev(slots[:0]), *dev, page)
    assert a8w8.paged_kv_read_i4(*dev, to_dev(slots[:0]), page)[0].shape == (0, Hkv, D)
    assert a8w8.read_device_errors() == 0


# ---------------------------------------------------------------------------
# attention (GPU)
# ---------------------------------------------------------------------------

def _check(got, want, bound):
    """Within the derived bound plus the BF16 rounding of the result (half a step: 2^-8)."""
    g = kv_i4.bf16_to_f64(to_host(got))
    tol = bound + (np.abs(want) + bound) * 2.0 ** -8
    odd = np.argwhere(np.isnan(g) != np.isnan(want))
    assert not odd.size, f"NaN in one alone at {odd[:4].tolist()}"
    ok = np.isnan(want) | (np.abs(g - want) <= tol)
    worst = np.nanmax(np.abs(g - want) / np.maximum(tol, 1e-300))
    assert ok.all(), f"{(~ok).sum()} of {ok.size} elements off, worst {worst:.3g} of the bound"
    # the error as a whole is that of the one rounding (2^-8 / sqrt(3) at most, relative)
    f = ~np.isnan(want)
    if np.linalg.norm(want[f]) > 0:
        rel = np.linalg.norm((g - want)[f]) / np.linalg.norm(want[f])
        assert rel <= 2.0 ** -8 / np.sqrt(3) + np.linalg.norm(bound[f]) / np.linalg.norm(want[f])


def _case(seed, ctx, Hq, Hkv, D, page, gain=1.5, **scales):
    rng = np.random.default_rng(seed)
    ctx = np.asarray(ctx, np.int32)
    bt, nblk = synth.paged_layout(seed, np.maximum(ctx, 1), page, spare_blocks=2)
    cache = _cache(rng, nblk * page, Hkv, D, **scales)
    q = synth.bf16_normal(seed + 1, (len(ctx), Hq, D), std=gain)
    return q, cache, bt, ctx


SHAPES = [
    # contexts, Hq, Hkv, D, page
    ([255], 40, 8, 128, 128),
    ([1], 8, 8, 128, 128),
    ([16, 17, 15, 31, 32, 33, 63, 64, 65, 0], 4, 2, 64, 16),
    ([1, 2, 3, 5, 7, 8, 9], 6, 2, 128, 5),
    ([4096, 300, 0, 2049], 40, 8, 128, 128),
    ([777, 1300], 8, 1, 128, 48),
    ([129, 1, 3000], 7, 1, 64, 24),
    ([500, 501], 12, 4, 64, 1),
    (list(range(0, 1200, 37)), 10, 5, 128, 32),
    ([128, 256, 384, 512] * 5, 16, 2, 128, 64),
]


@gpu
@pytest.mark.parametrize("ctx,Hq,Hkv,D,page", SHAPES)
def test_attention(ctx, Hq, Hkv, D, page):
    q, cache, bt, ctx = _case(len(ctx) * 7 + Hq, ctx, Hq, Hkv, D, page)
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page)
    a8w8.read_device_errors()
    dev = [to_dev(a) for a in (q, *cache, bt, ctx)]
    got = a8w8.paged_decode_attention_i4kv(*dev, page)
    _check(got, want, bound)
    assert not to_host(got)[ctx == 0].any()
    assert a8w8.read_device_errors() == 0
    again = a8w8.paged_decode_attention_i4kv(*dev, page)
    assert np.array_equal(to_host(got), to_host(again))       # the same bits every time


@gpu
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8])
def test_attention_groups(G):
    q, cache, bt, ctx = _case(G, [70, 200, 3], 2 * G, 2, 128, 16)
    want, bound = kv_i4.attention(q, *cache, bt, ctx, 16)
    _check(a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, *cache, bt, ctx)], 16), want,
           bound)


@gpu
@pytest.mark.parametrize("what", ["peaked", "tiny v", "tiniest v", "mixed v", "zero s", "huge v",
                                  "constant v", "rising", "falling", "scale 0", "negative scale"])
def test_attention_ranges(what):
    """Weights, scales and maxima over wide ranges: one token that takes all, V rows of tiny,
    mixed (10 decades) or zero s, scores that rise along the context."""
    n, page = 600, 16
    rng = np.random.default_rng(3)
    gain = 30.0 if what == "peaked" else 1.5
    sc = {"scale 0": 0.0, "negative scale": -0.2}.get(what)
    v_scale = {"tiny v": 1e-9, "tiniest v": 2.0 ** -70, "huge v": 1e30}.get(what, 0.35)
    q, cache, bt, ctx = _case(9, [n, 1, 77], 10, 2, 128, page, gain=gain, v_scale=v_scale)
    kc, vc, km, vm = cache
    if what == "mixed v":
        s = kv_i4.bf16_to_f64(vm) * (10.0 ** rng.uniform(-5, 5, vm.shape[:2]))[..., None]
        vm = _bf(s)
    if what == "zero s":
        vm[::2, :, 0] = 0                                  # constant rows, every other slot
        km[1::3, :, 0] = 0
    if what == "constant v":                               # s = 0 throughout, up to 2^36
        vm[..., 0] = 0
        vm[..., 1] = _bf(rng.choice([-1.0, 1.0], vm.shape[:2]) * 2.0 ** rng.integers(-60, 37, vm.shape[:2]))
    if what in ("rising", "falling"):
        for t in range(n):                                 # K grows (falls) with the position
            slot = bt[0][t // page] * page + t % page
            f = t / 60.0 if what == "rising" else (n - t) / 60.0
            km[slot] = _bf(kv_i4.bf16_to_f64(km[slot]) * f)
    cache = (kc, vc, km, vm)
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page, scale=sc)
    got = a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, *cache, bt, ctx)], page,
                                           softmax_scale=sc)
    _check(got, want, bound)


@gpu
def test_attention_bad_tables_and_nan_rows():
    page, Hq, Hkv, D = 16, 4, 2, 64
    q, cache, bt, ctx = _case(4, [100, 40, 90, 33], Hq, Hkv, D, page)
    bt[0, 2], bt[1, 0] = 10 ** 6, -5                       # rows of zeros
    ctx[2] = bt.shape[1] * page + 1                        # out of range: no tokens
    cache[2][bt[3, 1] * page + 3, 1] = _bf(np.nan)         # head 1 of request 3
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page)
    a8w8.read_device_errors()
    got = a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, *cache, bt, ctx)], page)
    assert a8w8.read_device_errors() == a8w8.DEVERR_BLOCK | a8w8.DEVERR_CTX
    _check(got, want, bound)
    assert np.isnan(want[3, 2:]).all() and not np.isnan(want[3, :2]).any()
    assert not to_host(got)[2].any()
    # past the context nothing counts: a bad id, a NaN row
    q, cache, bt, ctx = _case(5, [17, 30], Hq, Hkv, D, page)
    cache[2][bt[0, 1] * page + 1:bt[0, 1] * page + page] = _bf(np.nan)
    cache[3][bt[1, 1] * page + 14:bt[1, 1] * page + page] = _bf(np.nan)
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page)
    _check(a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, *cache, bt, ctx)], page), want,
           bound)
    assert a8w8.read_device_errors() == 0 and not np.isnan(want).any()


@gpu
@pytest.mark.parametrize("B,lo,hi,Hq,Hkv,D,page", [
    (300, 0, 40, 6, 6, 64, 16),          # more requests than threads, many in one run
    (140, 0, 700, 12, 3, 64, 32),
    (1, 20011, 20011, 8, 1, 128, 24),    # one request in as many parts as there are runs
    (2, 9000, 9001, 14, 2, 64, 128),
    (5, 250, 258, 40, 8, 128, 129),      # tables just past what one CTA takes whole
    (2, 290, 310, 1900, 1900, 64, 16),   # more KV heads than CTAs at once: one run
    (3, 700, 900, 130, 26, 128, 64),
])
def test_attention_runs(B, lo, hi, Hq, Hkv, D, page):
    ctx = np.random.default_rng(B).integers(lo, hi + 1, B)
    q, cache, bt, ctx = _case(B, ctx, Hq, Hkv, D, page)
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page)
    got = a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, *cache, bt, ctx)], page)
    _check(got, want, bound)
    assert not to_host(got)[ctx == 0].any()


@gpu
def test_attention_wide_tables_and_no_tokens_at_all():
    """A table far wider than the contexts; then every request empty."""
    page, Hq, Hkv, D = 16, 20, 4, 128
    q, cache, bt, ctx = _case(11, [5, 0, 33, 17], Hq, Hkv, D, page)
    wide = np.full((4, 4000), -1, np.int32)
    wide[:, :bt.shape[1]] = bt
    want, bound = kv_i4.attention(q, *cache, wide, ctx, page)
    a8w8.read_device_errors()
    dev = [to_dev(a) for a in (q, *cache, wide, ctx)]
    _check(a8w8.paged_decode_attention_i4kv(*dev, page), want, bound)
    dev[6].zero_()
    assert not to_host(a8w8.paged_decode_attention_i4kv(*dev, page)).any()
    dev[5] = dev[5][:, :4].contiguous()
    assert not to_host(a8w8.paged_decode_attention_i4kv(*dev, page)).any()
    assert a8w8.read_device_errors() == 0


@gpu
def test_attention_queries_out_of_range():
    """A query head with a NaN, an infinity or 2^118 and more gives NaN, its neighbours none of
    it; the largest and smallest queries below that are exact."""
    page, Hq, Hkv, D = 16, 8, 2, 64
    q, cache, bt, ctx = _case(12, [40], Hq, Hkv, D, page)
    q[0, 1, 3], q[0, 2, 0], q[0, 5, 63] = _bf(np.nan), _bf(np.inf), _bf(2.0 ** 118)
    q[0, 3] = _bf(kv_i4.bf16_to_f64(q[0, 3]) * 2.0 ** -120)
    q[0, 6] = 0
    q[0, 7, 0] = _bf(2.0 ** 117)
    q[0, 7, 1:] = 0
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page, scale=2.0 ** -118)
    want[0, [1, 2, 5]] = np.nan
    got = a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, *cache, bt, ctx)], page,
                                           softmax_scale=2.0 ** -118)
    _check(got, want, bound)


@gpu
def test_attention_calls_at_once_on_two_streams():
    import torch
    page, Hq, Hkv, D = 32, 40, 8, 128
    cases, outs, streams = [], [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for k in range(2):
        q, cache, bt, ctx = _case(20 + k, [3000, 17, 900 + k], Hq, Hkv, D, page)
        cases.append(([to_dev(a) for a in (q, *cache, bt, ctx)],
                      kv_i4.attention(q, *cache, bt, ctx, page)))
    torch.cuda.synchronize()
    for _ in range(5):
        outs = []
        for (dev, _w), st in zip(cases, streams):
            outs.append(a8w8.paged_decode_attention_i4kv(*dev, page, stream=st))
        torch.cuda.synchronize()
        for got, (_d, (want, bound)) in zip(outs, cases):
            _check(got, want, bound)


@gpu
def test_attention_captured_on_another_stream():
    """A captured call replays on new queries, tables and contexts; the workspace starts with
    arbitrary contents."""
    import torch
    page, Hq, Hkv, D = 32, 10, 2, 128
    q, cache, bt, ctx = _case(6, [900, 1, 64, 333], Hq, Hkv, D, page)
    dev = [to_dev(a) for a in (q, *cache, bt, ctx)]
    need = max(a8w8.attention_i4_workspace_bytes(4, Hq, Hkv, D, bt.shape[1] * page), 16)
    ws = torch.full((need,), 0xFF, dtype=torch.uint8, device="cuda")
    out = torch.empty_like(dev[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        a8w8.paged_decode_attention_i4kv(*dev, page, ws=ws, out=out)
    side.synchronize()
    first = to_host(out)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        a8w8.paged_decode_attention_i4kv(*dev, page, ws=ws, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert np.array_equal(first, to_host(out))
    q2 = synth.bf16_normal(99, q.shape)
    ctx2 = np.array([17, 0, 50, 900 if bt.shape[1] * page >= 900 else 1], np.int32)
    bt2 = bt[[3, 2, 1, 0]].copy()
    dev[0].copy_(to_dev(q2))
    dev[5].copy_(to_dev(bt2))
    dev[6].copy_(to_dev(ctx2))
    g.replay()
    torch.cuda.synchronize()
    want, bound = kv_i4.attention(q2, *cache, bt2, ctx2, page)
    _check(out, want, bound)


@gpu
def test_offsets_past_32_bits():
    """Pages whose codes lie more than 4 GiB into the cache (write, read, attention)."""
    import torch
    Hkv, D, page = 8, 128, 128
    nblk = (1 << 32) // (page * Hkv * D // 2) + 40
    dev = [torch.zeros((nblk * page, Hkv, D // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    dev += [torch.zeros((nblk * page, Hkv, 2), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    T = 300
    k, v = synth.bf16_normal(1, (T, Hkv, D)), synth.bf16_normal(2, (T, Hkv, D))
    bt = np.array([[nblk - 1, 3, nblk - 7]], np.int32)
    t = np.arange(T)
    slots = (bt[0][t // page] * page + t % page).astype(np.int32)
    a8w8.paged_kv_write_i4(to_dev(k), to_dev(v), to_dev(slots), *dev, page)
    q = synth.bf16_normal(3, (1, 40, D))
    got = a8w8.paged_decode_attention_i4kv(to_dev(q), *dev, to_dev(bt), to_dev(np.array([T], np.int32)),
                                           page)
    small = [np.zeros((3 * page, *d.shape[1:]), np.uint8 if i < 2 else np.uint16)
             for i, d in enumerate(dev)]
    kv_i4.kv_write(k, v, t.astype(np.int32), *small)
    want, bound = kv_i4.attention(q, *small, np.array([[0, 1, 2]]), [T], page)
    _check(got, want, bound)
    gk, _ = a8w8.paged_kv_read_i4(*dev, to_dev(slots), page)
    x = kv_i4.dequant_rows(small[0][:T], small[2][:T]).astype(np.float32)
    assert np.array_equal(to_host(gk), _bf(x))


@gpu
def test_attention_full_server():
    """64 requests of up to 16384 tokens (some 570 MB of rows) over pages in random order; five of
    them against the oracle, and a second call bit for bit."""
    import torch
    B, Hq, Hkv, D, page = 64, 40, 8, 128, 128
    rng = np.random.default_rng(8)
    ctx = rng.integers(64, 16385, B).astype(np.int32)
    ctx[[3, 40]] = 16384, 0
    bt, nblk = synth.paged_layout(8, np.maximum(ctx, 1), page, spare_blocks=3)
    g = torch.Generator(device="cuda").manual_seed(3)
    kc, vc = (torch.randint(0, 256, (nblk * page, Hkv, D // 2), dtype=torch.uint8, device="cuda",
                            generator=g) for _ in range(2))
    meta = []
    for _ in range(2):
        s = 0.25 + 0.2 * torch.rand((nblk * page, Hkv), device="cuda", generator=g)
        meta.append(torch.stack((s, -7.5 * s), dim=-1).to(torch.bfloat16))
    q = synth.bf16_normal(9, (B, Hq, D), std=1.5)
    dev = [to_dev(q), kc, vc, *meta, to_dev(bt), to_dev(ctx)]
    got = a8w8.paged_decode_attention_i4kv(*dev, page)
    assert torch.equal(got, a8w8.paged_decode_attention_i4kv(*dev, page))
    for b in (3, 40, int(ctx.argsort()[1]), 17, 63):
        n = -(-int(ctx[b]) // page)
        rows = (to_dev(bt[b, :n].astype(np.int64))[:, None] * page
                + torch.arange(page, device="cuda")).reshape(-1)
        own = [to_host(c[rows]) for c in (kc, vc, *meta)] if n else [to_host(c[:page]) for c in
                                                                     (kc, vc, *meta)]
        want, bound = kv_i4.attention(q[b:b + 1], *own, np.arange(max(n, 1))[None], ctx[b:b + 1], page)
        _check(got[b:b + 1], want, bound)


@gpu
def test_calls_on_another_stream_with_work_pending_on_the_current_one():
    """The current stream gives back blocks of just the sizes that the calls allocate, with a kernel
    still queued that writes them; the calls on another stream must not be handed those."""
    import torch
    page, Hq, Hkv, D, T = 32, 40, 8, 128, 6000
    q, cache, bt, ctx = _case(41, [3000, 17, 900, 2500] * 8, Hq, Hkv, D, page)
    want, bound = kv_i4.attention(q[:4], *cache, bt[:4], ctx[:4], page)
    dev = [to_dev(a) for a in (q, *cache, bt, ctx)]
    slots = to_dev(np.random.default_rng(2).integers(0, cache[0].shape[0], T).astype(np.int32))
    ref = a8w8.paged_kv_read_i4(*dev[1:5], slots, page)
    need = a8w8.attention_i4_workspace_bytes(len(ctx), Hq, Hkv, D, bt.shape[1] * page)
    a = torch.randn((8192, 8192), device="cuda", dtype=torch.bfloat16)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        left = [torch.empty_like(dev[0]), torch.empty(need, dtype=torch.uint8, device="cuda"),
                torch.empty_like(ref[0]), torch.empty_like(ref[1])]
        for _k in range(20):                               # some 10 ms on the current stream
            a @ a
        for x in left:
            x.fill_(0)
        del left, x
        got = a8w8.paged_decode_attention_i4kv(*dev, page, stream=side)
        k, v = a8w8.paged_kv_read_i4(*dev[1:5], slots, page, stream=side)
        torch.cuda.synchronize()
        _check(got[:4], want, bound)
        assert torch.equal(k, ref[0]) and torch.equal(v, ref[1])
        del got, k, v


@pytest.mark.parametrize("name", ["kv_i4.cu", "attn_i4.cu", "pages.cu"])
def test_kernels_that_start_early_read_nothing_through_the_read_only_path(name):
    """These grids may stand beside the kernel that writes their inputs (programmatic launch); a
    read-only (non-coherent) load is for data that stays as it is for the grid's whole time. The
    compiler takes one for a `const __restrict__` argument."""
    import os
    import re
    src = open(os.path.join(os.path.dirname(a8w8.__file__), "csrc", name)).read()
    code = re.sub(r"//[^\n]*|/\*.*?\*/", "", src, flags=re.S)
    for word in ("__restrict__", "__ldg(", "ld_nc_v4", "ld_stream_v4", ".nc."):
        assert word not in code, word


@gpu
def test_rows_written_by_the_kernel_just_before():
    """Rows read back from one cache into two buffers that are used again and again, and from there
    into another cache, with nothing between the calls."""
    import torch
    T, Hkv, D, page, rounds = 700, 4, 128, 32, 40
    rng = np.random.default_rng(12)
    n = 40 * page
    host = _cache(rng, n, Hkv, D)
    src = [to_dev(a) for a in host]
    dst = [torch.zeros((rounds * T + 32, *a.shape[1:]), dtype=a.dtype, device="cuda") for a in src]
    dst = [d[:(d.shape[0] // page) * page] for d in dst]
    kv = [torch.empty((T, Hkv, D), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    at = rng.integers(0, n, (rounds, T)).astype(np.int32)
    to = rng.permutation(rounds * T).reshape(rounds, T).astype(np.int32)
    at_d, to_d = to_dev(at), to_dev(to)
    torch.cuda.synchronize()
    for i in range(rounds):
        a8w8.paged_kv_read_i4(*src, at_d[i], page, out=kv)
        a8w8.paged_kv_write_i4(*kv, to_d[i], *dst, page)
    assert a8w8.read_device_errors() == 0
    for c, m, gc, gm in ((host[0], host[2], dst[0], dst[2]), (host[1], host[3], dst[1], dst[3])):
        x = _bf(kv_i4.dequant_rows(c, m).astype(np.float32))
        wc, wm = kv_i4.quant_rows(x)
        assert np.array_equal(to_host(gc)[to], wc[at])
        assert np.array_equal(kv_i4.bf16_to_f64(to_host(gm)[to]), kv_i4.bf16_to_f64(wm[at]))


@gpu
def test_attention_largest_query():
    """The largest BF16 below 2^118 is a query value like any other."""
    page, Hq, Hkv, D = 16, 4, 2, 64
    q, cache, bt, ctx = _case(13, [40, 300], Hq, Hkv, D, page)
    q[:, 1] = 0
    q[0, 1, 5] = q[1, 1, 60] = 0x7A7F                      # 1.9921875 * 2^117
    assert kv_i4.bf16_to_f64(q[0, 1, 5]) == 2.0 ** 118 - 2.0 ** 110
    q[0, 2, 7], q[1, 3, 0] = _bf(2.0 ** 118), _bf(-(2.0 ** 118))
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page, scale=2.0 ** -118)
    want[0, 2] = want[1, 3] = np.nan
    got = a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, *cache, bt, ctx)], page,
                                           softmax_scale=2.0 ** -118)
    _check(got, want, bound)


@gpu
@pytest.mark.parametrize("ctx", [[1, 40], [250], [5000, 33, 700]])
@pytest.mark.parametrize("sign", [-1, 1])
def test_attention_scores_far_from_zero(ctx, sign):
    """Scores near +-2^113: equal ones share the weight, one above the others takes all of it."""
    page, Hq, Hkv, D = 16, 4, 2, 64
    q, cache, bt, ctx = _case(32, ctx, Hq, Hkv, D, page)
    kc, vc, km, vm = cache
    q[:] = _bf(2.0 ** 60)
    km[..., 0], km[..., 1] = 0, _bf(sign * 2.0 ** 50)      # constant rows
    want, bound = kv_i4.attention(q, kc, vc, km, vm, bt, ctx, page, scale=0.0)
    dev = [to_dev(a) for a in (q, kc, vc, km, vm, bt, ctx)]
    _check(a8w8.paged_decode_attention_i4kv(*dev, page), want, bound)
    top = ctx // 2                                         # this token's score is 1/8 higher
    for b, t in enumerate(top):
        slot = bt[b][t // page] * page + t % page
        km[slot, :, 1] = _bf(sign * 2.0 ** 50 + 2.0 ** 47)
        for h in range(Hkv):
            v = kv_i4.dequant_rows(vc[slot, h], vm[slot, h])
            want[b, 2 * h:2 * h + 2] = v
            bound[b, 2 * h:2 * h + 2] = 2.0 ** -10 * (15 * abs(kv_i4.bf16_to_f64(vm[slot, h, 0]))
                                                      + abs(kv_i4.bf16_to_f64(vm[slot, h, 1])))
    dev[3] = to_dev(km)
    _check(a8w8.paged_decode_attention_i4kv(*dev, page), want, bound)


@gpu
@pytest.mark.parametrize("ctx", [[64], [192, 33], [3000, 100, 700]])
@pytest.mark.parametrize("Hkv", [1, 2, 4])
@pytest.mark.parametrize("order", ["rising", "falling", "mixed"])
def test_attention_scales_far_apart(ctx, Hkv, order):
    """V rows of ordinary size beside rows near the end of float32's range: their weights in the
    softmax's sum count alike, whichever tile, warp or run they are in."""
    page, D = 16, 64
    q, cache, bt, ctx = _case(31, ctx, 2 * Hkv, Hkv, D, page, gain=0.3)
    kc, vc, km, vm = cache
    rng = np.random.default_rng(5)
    for b, n in enumerate(ctx):
        t = np.arange(n)
        big = {"rising": t >= n // 2, "falling": t < n // 2, "mixed": rng.random(n) < 0.1}[order]
        slot = bt[b][t // page] * page + t % page
        f = np.where(big, 2.0 ** 120, 2.0 ** -12)[:, None, None]
        vm[slot] = _bf(kv_i4.bf16_to_f64(vm[slot]) * f)
    want, bound = kv_i4.attention(q, *cache, bt, ctx, page)
    got = a8w8.paged_decode_attention_i4kv(*[to_dev(a) for a in (q, kc, vc, km, vm, bt, ctx)], page)
    _check(got, want, bound)


@gpu
def test_attention_sums_of_long_runs():
    """64 requests of 2^24 tokens, equal scores and constant V rows c s of one code: 2^30 equal
    weights in 456 runs. The sums' roundings stay below a quarter of BF16's half step, so the
    result is c s itself (a BF16 value: c is a power of two). In one chain a lane adds 294,000
    weights of which each is 2^-18 of the sum at last, and loses (a float32 model of that chain)
    0.41 to 0.43 % for the scales taken here."""
    page, B, Hkv, D = 4096, 64, 4, 64
    scale = np.array([145, 129, 226, 156]) / 128.0
    n = 2 * page
    code = np.array([8, 4, 2, 1], np.uint8)
    vc = np.broadcast_to((code | code << 4)[None, :, None], (n, Hkv, D // 2)).copy()
    vm = np.broadcast_to(np.stack((_bf(scale), _bf(0 * scale)), -1)[None], (n, Hkv, 2)).copy()
    q = np.zeros((B, Hkv, D), np.uint16)
    bt = np.tile(np.array([0, 1], np.int32), (B, 2048))
    ctx = np.full(B, 1 << 24, np.int32)
    dev = [to_dev(a) for a in (q, np.zeros_like(vc), vc, np.zeros_like(vm), vm, bt, ctx)]
    got = kv_i4.bf16_to_f64(to_host(a8w8.paged_decode_attention_i4kv(*dev, page)))
    assert (got == (code * scale)[None, :, None]).all()
    assert a8w8.read_device_errors() == 0


@gpu
@pytest.mark.parametrize("Hkv,D,heads", [(457, 64, (0, 228, 456)), (458, 64, (0, 1, 457)),
                                         (1828, 64, (0, 3, 1827)), (201, 64, (0, 200)),
                                         (402, 128, (1, 400)), (912, 128, (2, 911))])
def test_attention_long_runs(Hkv, D, heads):
    """So many KV heads that one run, or two, takes all tiles: segments of thousands of tiles,
    summed piece by piece, that end with their request or inside it, against the oracle for some
    of the heads; the same bits every time."""
    page = 64
    ctx = np.array([70001, 0, 140000, 90, 66000], np.int32)
    nblk = 9
    cache = _cache(np.random.default_rng(Hkv), nblk * page, Hkv, D)
    bt = np.random.default_rng(1).integers(0, nblk, (len(ctx), 2200)).astype(np.int32)
    q = synth.bf16_normal(Hkv, (len(ctx), 2 * Hkv, D), std=1.5)
    dev = [to_dev(a) for a in (q, *cache, bt, ctx)]
    a8w8.read_device_errors()
    got = a8w8.paged_decode_attention_i4kv(*dev, page)
    assert np.array_equal(to_host(got), to_host(a8w8.paged_decode_attention_i4kv(*dev, page)))
    at = [2 * h + g for h in heads for g in (0, 1)]
    want, bound = kv_i4.attention(q[:, at], *[c[:, list(heads)] for c in cache], bt, ctx, page)
    _check(got[:, at], want, bound)
    assert not to_host(got)[1].any() and a8w8.read_device_errors() == 0


def test_attention_refuses_runs_that_are_too_long(lib):
    """A run's sums are joined piece by piece: 2^27 tokens a run, of which there are as many as the
    KV heads leave room for."""
    def f(B, Hkv, max_blocks=4096, page=4096):
        return lib.paged_decode_attention_i4kv(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, B, Hkv, Hkv,
                                               64, page, max_blocks, 100, 0.1, FAKE, FAKE, 0, None)
    for B, Hkv, ok in ((8, 1901, True), (9, 1901, False), (8, 1824, True), (9, 1824, False),
                       (16, 912, True), (17, 912, False), (2048, 4, True), (2049, 4, False)):
        assert f(B, Hkv) == (a8w8.ERR_WORKSPACE if ok else a8w8.ERR_UNSUPPORTED_SHAPE), (B, Hkv)


@gpu
def test_longest_chunk():
    """16384 tokens of 8 heads of 128, pages in random order: codes, pairs and rows read back, bit
    for bit."""
    import torch
    T, Hkv, D, page = 16384, 8, 128, 128
    rng = np.random.default_rng(77)
    k, v = synth.bf16_normal(78, (T, Hkv, D)), synth.bf16_normal(79, (T, Hkv, D), std=2.0)
    blocks = rng.permutation(T // page + 3)
    t = np.arange(T)
    slots = (blocks[t // page] * page + t % page).astype(np.int32)
    n = len(blocks) * page
    dev = [torch.zeros((n, Hkv, w), dtype=dt, device="cuda") for w, dt in
           ((D // 2, torch.uint8), (D // 2, torch.uint8), (2, torch.bfloat16), (2, torch.bfloat16))]
    a8w8.read_device_errors()
    a8w8.paged_kv_write_i4(to_dev(k), to_dev(v), to_dev(slots), *dev, page)
    got = a8w8.paged_kv_read_i4(*dev, to_dev(slots), page)
    assert a8w8.read_device_errors() == 0
    for x, c, m, g in ((k, dev[0], dev[2], got[0]), (v, dev[1], dev[3], got[1])):
        wc, wm = kv_i4.quant_rows(x)
        assert np.array_equal(to_host(c)[slots], wc)
        assert np.array_equal(kv_i4.bf16_to_f64(to_host(m)[slots]), kv_i4.bf16_to_f64(wm))
        assert np.array_equal(to_host(g), _bf(kv_i4.dequant_rows(wc, wm).astype(np.float32)))
