"""Pins of the 8-bit cache's oracle (oracle/q8.py) and the refusals of its
entry points, without a GPU."""
import ctypes
import itertools

import numpy as np
import pytest
import torch

import oracle
from oracle import q8
import pa_workloads as wl

N_Q, N_KV, D = 32, 8, 64


def test_every_byte_and_every_tie():
    """The 256 bytes decode as torch's e4m3, encode to themselves, and every
    midpoint of two neighbours goes to the even byte."""
    b = np.arange(256, dtype=np.uint8)
    t = torch.from_numpy(b.copy()).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(t, q8.VALUES, equal_nan=True)
    fin = np.isfinite(q8.VALUES)
    assert np.array_equal(q8.encode(q8.VALUES[fin]), b[fin])
    mid = (q8.VALUES[:126] + q8.VALUES[1:127]) / 2
    even = np.where(b[:126] % 2 == 0, b[:126], b[1:127])
    for sign, bit in ((1.0, 0), (-1.0, 128)):
        assert np.array_equal(q8.encode(sign * mid), even | bit)
        assert np.array_equal(q8.encode(sign * np.nextafter(mid, 0)), b[:126] | bit)
        assert np.array_equal(q8.encode(sign * np.nextafter(mid, 999)), b[1:127] | bit)
    assert q8.encode(1e9) == 0x7E and q8.encode(-1e9) == 0xFE
    assert q8.encode(np.nan) == q8.encode(np.inf) == q8.encode(-np.inf) == 0x7F


def test_encode_matches_torch():
    x = np.random.default_rng(1).standard_normal(20000) * np.exp2(
        np.random.default_rng(2).uniform(-12, 8, 20000))
    x = np.clip(x, -448, 448).astype(np.float32)
    t = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(q8.encode(x), t)


def test_exponent_at_its_borders():
    for limit, e in itertools.product((316.0, 448.0), (-117, -3, 0, 7, 119)):
        edge = limit * 2.0 ** e
        assert q8.exponent(np.array([edge, -edge / 2]), limit) == e
        assert q8.exponent(np.array([-edge * (1 + 2.0 ** -8)]), limit) == e + 1
    assert q8.exponent(np.zeros(3), 448.0) == -117
    assert q8.exponent(np.array([np.nan, np.inf, 1.0]), 448.0) == q8.exponent(np.ones(1), 448.0)


@pytest.mark.parametrize("page", [8, 16, 32])
def test_chunk_equals_single_tokens_up_to_subnormal_bytes(page):
    """A chunk appended at once and token by token give the same tables and
    scales; a value differs only where a byte became subnormal on the way and
    was rounded more than once: at most one subnormal step (2^-9 scale)."""
    rng = np.random.default_rng(page)
    n, blocks = 2 * page + 5, 6
    k, v = wl.normal_bf16(rng, (n, N_KV, D)), wl.normal_bf16(rng, (n, N_KV, D))
    k[n // 2] = wl.normal_bf16(rng, (N_KV, D), scale=40.0)       # the scale grows inside a page
    pool, scales = q8.random_pool(rng, blocks, page)
    table = np.full((1, 1, 4), -1, dtype=np.int32)
    fl = np.arange(blocks, dtype=np.int32)
    _, p1, s1, t1, c1, e1 = q8.append(k, v, None, [0, n], pool, scales, table, [0], 0, fl, blocks)
    p2, s2, t2, c2 = pool, scales, table, blocks
    for i in range(n):
        _, p2, s2, t2, c2, e2 = q8.append(k[i:i + 1], v[i:i + 1], None, [0, 1], p2, s2, t2, [i], 0, fl, c2)
        assert e2 == 0
    assert e1 == 0 and c1 == c2 and np.array_equal(t1, t2) and np.array_equal(s1, s2)
    d = np.abs(q8.decode(p1, s1) - q8.decode(p2, s2))
    assert np.all(d <= 2.0 ** -9 * s1[:, :, None, :, None])
    # and every stored value lies within half a step of what the bf16 cache holds
    pos = np.arange(n)
    kr = oracle.bf16_to_f64(q8.to_bf16(q8.rotate(oracle.bf16_to_f64(k), pos)))
    got = q8.decode(p1, s1)[t1[0, 0, pos // page], 0, pos % page]
    sc = s1[t1[0, 0, pos // page], 0][:, :, None].astype(np.float64)
    assert np.all(np.abs(got - kr) <= np.maximum(2.0 ** -4 * np.abs(kr), 2.0 ** -10 * sc))


def test_appended_cache_matches_the_bf16_oracle():
    """Tables, free list and the rotation agree with the bf16 append's."""
    rng = np.random.default_rng(5)
    ctx, lens = [3, 16, 0, 31], [20, 1, 17, 2]
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    k, v = (wl.normal_bf16(rng, (cu[-1], N_KV, D)) for _ in range(2))
    q = wl.normal_bf16(rng, (cu[-1], N_Q, D))
    table = np.full((4, 1, 4), -1, dtype=np.int32)
    table[0, 0, 0], table[1, 0, 0], table[3, 0, :2] = 9, 8, [7, 6]
    fl = np.arange(6, dtype=np.int32)
    pool, scales = q8.random_pool(rng, 10)
    got = q8.append(k, v, q, cu, pool, scales, table, ctx, 0, fl, 6)
    ref = oracle.prefill_append_rope(k, v, q, cu, np.zeros((10, 2, 16, N_KV, D), np.uint16), table, ctx, 0, fl, 6)
    assert np.array_equal(got[3], ref[2]) and got[4] == ref[4] and got[5] == ref[5] == 0
    assert np.array_equal(got[0], ref[0])


# ------------------------------------------------------------------ refusals
def _lib():
    import paged_kv_cache_205_gb300 as pk
    return pk.library()


def _call(fn, **over):
    """The C call with valid host-side arguments (pointers are never followed
    before the checks) and `over` in their place."""
    P = ctypes.c_void_p
    a = dict(k=P(16), v=P(16), q=P(16), qo=P(16), out=P(16), total=4, cu=P(16), kv=P(16), sc=P(16), nb=4, bt=16,
             table=P(16), L=1, mb=4, ctx=P(16), n=2, layer=0, fl=P(16), fc=P(16), scale=0.125, ws=P(16),
             wsb=1 << 40, err=P(16))
    a.update(over)
    g = lambda *names: [a[x] for x in names]  # noqa: E731
    tail = ("table", "L", "mb", "ctx", "n", "layer")
    args = {
        "pa_kv_append_rope_q8": g("k", "v", "q", "qo", "kv", "sc", "nb", "bt", *tail, "fl", "fc", "err"),
        "pa_prefill_append_rope_q8": g("k", "v", "q", "qo", "total", "cu", "kv", "sc", "nb", "bt", *tail, "fl", "fc",
                                       "err"),
        "pa_decode_attention_q8": g("out", "q", "kv", "sc", "nb", "bt", *tail, "scale", "ws", "wsb", "err"),
        "pa_prefill_attention_q8": g("out", "q", "total", "cu", "kv", "sc", "nb", "bt", *tail, "scale", "err"),
    }[fn]
    return getattr(_lib(), fn)(*args, P(0))


ALL = ["pa_kv_append_rope_q8", "pa_prefill_append_rope_q8", "pa_decode_attention_q8", "pa_prefill_attention_q8"]
APPENDS, PREFILLS = ALL[:2], ALL[1::2]


@pytest.mark.parametrize("fn", ALL)
def test_refusals(fn):
    P = ctypes.c_void_p
    for bt in (0, 4, 12, 64, -8):
        assert _call(fn, bt=bt) == -2
    for name, bad in (("nb", 0), ("nb", -1), ("L", 0), ("mb", 0), ("n", -1), ("mb", 1 << 28)):
        assert _call(fn, **{name: bad}) == -2, (name, bad)
    assert _call(fn, layer=1) == _call(fn, layer=-1) == -3
    for name in ("kv", "sc", "table", "ctx", "err"):
        assert _call(fn, **{name: P(0)}) == -1, name
    for name in ("kv", "sc"):
        assert _call(fn, **{name: P(24)}) == -5, name
    assert _call(fn, n=0) == 0
    if fn in APPENDS:
        for name in ("k", "v", "fl", "fc", "qo"):
            assert _call(fn, **{name: P(0)}) == -1, name
        for name in ("k", "v", "q", "qo"):
            assert _call(fn, **{name: P(20)}) == -5, name
    else:
        for name in ("out", "q"):
            assert _call(fn, **{name: P(0)}) == -1
            assert _call(fn, **{name: P(20)}) == -5
        assert _call(fn, n=2049) == -2
    if fn in PREFILLS:
        assert _call(fn, total=-1) == -2 and _call(fn, total=0) == 0
        assert _call(fn, cu=P(0)) == -1
    if fn == "pa_decode_attention_q8":
        assert _call(fn, ws=P(0)) == -4 and _call(fn, ws=P(8)) == -5
    if fn == "pa_prefill_attention_q8":
        for scale in (0.0, -1.0, float("inf"), float("nan")):
            assert _call(fn, scale=scale) == -2


def test_workspace_size():
    import paged_kv_cache_205_gb300 as pk
    assert pk.pa_decode_workspace_size_q8(0, 4) == 0 == pk.pa_decode_workspace_size_q8(4, 4, 12)
    assert 0 < pk.pa_decode_workspace_size_q8(1, 1) <= pk.pa_decode_workspace_size_q8(256, 512, 32)


def test_prompt_append_refuses_more_sequences_than_its_grid_holds():
    assert _call("pa_prefill_append_rope_q8", n=(1 << 29) + 1) == -2


def test_binding_refuses_before_the_library():
    """Tensors off the device, of other types or shapes do not reach the library."""
    import paged_kv_cache_205_gb300 as pk
    z = torch.zeros
    table = z((2, 1, 4), dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        pk.pa_decode_attention_q8(z(2, 32, 64, dtype=torch.bfloat16), z(2, 32, 64, dtype=torch.bfloat16),
                                  z((4, 2, 16, 8, 64), dtype=torch.uint8), z(4, 2, 8), table,
                                  z(2, dtype=torch.int32), 0, 0.125, z(64, dtype=torch.uint8),
                                  z(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        pk.kv_cache_q8(4, block_tokens=12)
    with pytest.raises(ValueError, match="exceeds"):
        pk.pa_decode_attention_q8(None, None, z((4, 2, 16, 8, 64), dtype=torch.uint8), z(4, 2, 8), table, None, 0,
                                  0.125, None, None, num_seqs=3)
