"""GPU parity of the 8-bit cache's operators against the fp64 oracle
(oracle/q8.py for the cache, oracle.decode_attention / prefill_attention on
its values, which are exact in bf16), through the binding.

Tolerances of attention outputs, by arithmetic (V = the largest |value|, T =
the context, S = the largest sum of |q_i k_i| times the scale):
  the output's own bf16 rounding, half an ulp;
  a weight enters the MMA in f16, rounded by at most half a step: 2^-12 of it,
  or 2^-25 absolute below 2^-14; the sum of weights is taken before that, so the
  output moves by at most that times V (+ T 2^-25 V);
  a score is an fp32 sum of 64 products: with a last bit lost at each of up to
  64 additions and the factor's own roundings its error is below 2^-17 S, and
  the weights and their sum each move by at most that, relatively: 2^-16 S V.
"""
import numpy as np
import pytest

import oracle
from oracle import q8
import pa_workloads as wl
from helpers import bf16_half_ulp, dev_bf16, dev_i32, host_bits, host_f64, ulp_diff

pytestmark = pytest.mark.gpu

N_Q, N_KV, D = 32, 8, 64
PAGES = [8, 16, 32]


def _pk():
    import paged_kv_cache_205_gb300 as pk
    return pk


def _dev_pool(pool, scales):
    import torch
    return (torch.from_numpy(pool).cuda().view(torch.float8_e4m3fn), torch.from_numpy(np.asarray(scales)).cuda())


def _cache(seed, lens, page, layers=1, layer=0, extra=6, poison=True):
    """Pages scattered over a pool whose unused slots hold NaN bytes."""
    rng = np.random.default_rng(seed)
    lens = np.asarray(lens, dtype=np.int64)
    pages = (lens + page - 1) // page
    nb = int(pages.sum()) + extra
    mb = int(max(1, pages.max())) + 1
    pool, scales = q8.random_pool(rng, nb, page)
    table = np.full((len(lens), layers, mb), -1, dtype=np.int32)
    ids = rng.permutation(nb).astype(np.int32)
    live = np.zeros((nb, page), dtype=bool)
    at = 0
    for s, t in enumerate(lens):
        table[s, layer, :pages[s]] = ids[at:at + pages[s]]
        for j in range(pages[s]):
            live[ids[at + j], :min(page, int(t) - j * page)] = True
        at += pages[s]
    if poison:
        pool[np.broadcast_to(~live[:, None, :, None, None], pool.shape)] = 0x7F
    return rng, pool, scales, table, ids[at:]


def _assert_close(got, ref, q, pool, scales, tokens, scale, weight_step, what=""):
    v = np.abs(q8.decode(pool, scales))
    big = np.nanmax(v[:, 1], initial=0.0)
    s = scale * np.abs(oracle.bf16_to_f64(q)).sum(-1).max(initial=0.0) * np.nanmax(v[:, 0], initial=0.0)
    tol = bf16_half_ulp(ref) + big * (weight_step + tokens * 2.0 ** -25 + s * 2.0 ** -16)
    assert np.all(np.isfinite(got)), what
    d = np.abs(got - ref)
    i = np.unravel_index(int(np.argmax(d - tol)), d.shape)
    assert np.all(d <= tol), f"{what}: {got[i]} against {ref[i]} at {i}, allowed {tol[i]}"


def _decode(q, pool, scales, table, ctx, layer=0, scale=0.125, ws=None, num_seqs=None):
    import torch
    pk = _pk()
    kv, sc = _dev_pool(pool, scales)
    out = torch.full((len(q), N_Q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = pk.decode_workspace_q8(table.shape[0], table.shape[2], block_tokens=pool.shape[2])
    pk.pa_decode_attention_q8(out, dev_bf16(q), kv, sc, dev_i32(table), dev_i32(ctx), layer, scale, ws, err,
                              num_seqs=num_seqs)
    torch.cuda.synchronize()
    return host_f64(out), int(err.item())


EDGE = [0, 1, 2, 7, 8, 9, 15, 16, 17, 23, 24, 25, 31, 32, 33, 47, 48, 64, 65, 127, 128, 129, 700, 2047]


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("q_scale", [1.0, 8.0])
def test_decode_edge_contexts(page, q_scale):
    rng, pool, scales, table, _ = _cache(page, EDGE, page)
    q = wl.normal_bf16(rng, (len(EDGE), N_Q, D), scale=q_scale)
    ref, e = oracle.decode_attention(q, q8.pool_bf16(pool, scales), table, EDGE, 0, block_tokens=page)
    got, err = _decode(q, pool, scales, table, EDGE)
    assert err == e == 0
    assert np.all(got[0] == 0)
    _assert_close(got, ref, q, pool, scales, max(EDGE), 0.125, 2.0 ** -12, f"page {page}")


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("lens", [[1], [5000], [17, 14], [0, 0, 0], [3] * 40, list(range(0, 1200, 13)),
                                  [4000] + [5] * 30], ids=["one", "long", "two", "none", "forty", "ragged", "tail"])
def test_decode_batches(page, lens):
    """Batches that split long contexts, hold many per chunk, or are empty;
    the second of two layers; a scale of its own."""
    rng, pool, scales, table, _ = _cache(50 + page, lens, page, layers=2, layer=1)
    q = wl.normal_bf16(rng, (len(lens), N_Q, D))
    ref, e = oracle.decode_attention(q, q8.pool_bf16(pool, scales), table, lens, 1, scale=0.3, block_tokens=page)
    got, err = _decode(q, pool, scales, table, lens, layer=1, scale=0.3)
    assert err == e == 0
    _assert_close(got, ref, q, pool, scales, max(lens), 0.3, 2.0 ** -12)


@pytest.mark.parametrize("page", PAGES)
def test_decode_scales_far_apart(page):
    """Neighbouring pages whose scales differ by up to 2^40, tiny and huge q
    heads: each element within the bound relative to what it sums."""
    lens = [40, 300]
    rng, pool, scales, table, _ = _cache(77, lens, page)
    scales[:, 1] = np.ldexp(1.0, rng.integers(-30, 11, size=scales[:, 1].shape)).astype(np.float32)
    q = wl.normal_bf16(rng, (2, N_Q, D))
    q[:, ::3] = wl.to_bf16_bits(oracle.bf16_to_f64(q[:, ::3]).astype(np.float32) * np.float32(2.0 ** -40))
    q[1, 1] = wl.to_bf16_bits(oracle.bf16_to_f64(q[1, 1]).astype(np.float32) * np.float32(2.0 ** 30))
    ref, e = oracle.decode_attention(q, q8.pool_bf16(pool, scales), table, lens, 0, block_tokens=page)
    got, err = _decode(q, pool, scales, table, lens)
    assert err == e == 0
    keep = np.ones(ref.shape[:2], bool)
    keep[1, 1] = False           # its softmax is one key, unless two scores tie
    mag, _ = oracle.decode_attention(q, q8.pool_bf16(pool & 0x7F, scales), table, lens, 0, block_tokens=page)
    kabs = np.nanmax(np.abs(q8.decode(pool, scales)[:, 0]))
    s = 0.125 * np.abs(oracle.bf16_to_f64(q)).sum(-1)[..., None] * kabs
    tol = bf16_half_ulp(ref) + np.nanmax(np.abs(q8.decode(pool, scales)[:, 1])) * (2.0 ** -12 + 2.0 ** -16 * s)
    assert np.all((np.abs(got - ref) <= tol)[keep])
    assert np.all(np.isfinite(got))


def test_decode_nan_and_zero_scores():
    """A NaN key reaches the outputs of its kv head and no other; a query of
    zeros gives the mean of the values; values beyond the context are not
    read (NaN bytes there)."""
    lens = [20, 33]
    rng, pool, scales, table, _ = _cache(5, lens, 16)
    q = wl.normal_bf16(rng, (2, N_Q, D))
    q[1] = 0
    pool[table[0, 0, 1], 0, 2, 3, 5] = 0x7F
    got, err = _decode(q, pool, scales, table, lens)
    assert err == 0
    assert np.all(np.isnan(got[0, 12:16])) and np.all(np.isfinite(np.delete(got[0], range(12, 16), 0)))
    v = q8.decode(pool, scales)[table[1, 0, :3], 1].reshape(48, N_KV, D)[:33]
    mean = np.repeat(v.mean(0), 4, axis=0)
    assert np.all(np.abs(got[1] - mean) <= bf16_half_ulp(mean) + np.abs(v).max() * 2.0 ** -12)


@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0])
@pytest.mark.parametrize("lens", [[20, 1, 9], [2000, 40, 700]], ids=["short", "long"])
def test_decode_q_head_not_finite(bad, lens):
    """An infinity or NaN in a q head makes that head's output NaN and changes no other."""
    rng, pool, scales, table, _ = _cache(9, lens, 16)
    q = wl.normal_bf16(rng, (3, N_Q, D))
    want, _ = _decode(q, pool, scales, table, lens)
    q = q.copy()
    q[0, 9, 3] = q[1, 31, 63] = bad
    got, err = _decode(q, pool, scales, table, lens)
    assert err == 0
    heads = np.zeros((3, N_Q), bool)
    heads[0, 9] = heads[1, 31] = True
    assert np.isnan(got[heads]).all()
    assert np.array_equal(got[~heads], want[~heads])


@pytest.mark.parametrize("page", PAGES)
def test_decode_bad_pages_and_contexts(page):
    """A page id out of range drops its tokens and is reported; a sequence
    with no valid page gives zeros; a context beyond the table is clamped."""
    lens = [70, 2 * page, 40]
    rng, pool, scales, table, _ = _cache(9 + page, lens, page)
    table[0, 0, 1] = pool.shape[0] + 5
    table[1, 0, :2] = [-1, pool.shape[0]]
    q = wl.normal_bf16(rng, (3, N_Q, D))
    bits = q8.pool_bf16(pool, scales)
    ref, e = oracle.decode_attention(q, bits, table, lens, 0, block_tokens=page)
    got, err = _decode(q, pool, scales, table, lens)
    assert err == e == oracle.ERR_BAD_BLOCK
    assert np.all(got[1] == 0)
    _assert_close(got[[0, 2]], ref[[0, 2]], q, pool, scales, 70, 0.125, 2.0 ** -12)
    got, err = _decode(q, pool, scales, table, [-3, 0, 100000])
    assert err & oracle.ERR_CTX_RANGE and np.all(got[:2] == 0)


def test_decode_rows_behind_the_batch_and_workspace_reuse():
    """num_seqs below the table's rows leaves the other outputs as they were;
    one workspace serves calls of other sizes one after another."""
    import torch
    pk = _pk()
    lens = [900, 33, 5, 1700]
    rng, pool, scales, table, _ = _cache(3, lens, 16)
    q = wl.normal_bf16(rng, (4, N_Q, D))
    ws = pk.decode_workspace_q8(300, table.shape[2])
    ref, _ = oracle.decode_attention(q, q8.pool_bf16(pool, scales), table, lens, 0)
    for n in (2, 4, 1, 4):
        got, err = _decode(q, pool, scales, table, lens, ws=ws, num_seqs=n)
        assert err == 0 and np.all(np.isnan(got[n:]))
        _assert_close(got[:n], ref[:n], q, pool, scales, 1700, 0.125, 2.0 ** -12)
    with pytest.raises(pk.PagedKVError) as e:
        _decode(q, pool, scales, table, lens, ws=torch.zeros(512, dtype=torch.uint8, device="cuda"))
    assert e.value.code == -4


def test_decode_graph_stream_and_repeat():
    """Captured on a side stream and replayed with other lengths and inputs:
    the same bits as a direct call, twice."""
    import torch
    pk = _pk()
    lens = [1200, 64, 17, 0, 333]
    rng, pool, scales, table, _ = _cache(21, lens, 16)
    kv, sc = _dev_pool(pool, scales)
    bt, ctx, err = dev_i32(table), dev_i32(lens), dev_i32([0])
    q = dev_bf16(wl.normal_bf16(rng, (5, N_Q, D)))
    out = torch.empty_like(q)
    ws = pk.decode_workspace_q8(5, table.shape[2])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    call = lambda o: pk.pa_decode_attention_q8(o, q, kv, sc, bt, ctx, 0, 0.125, ws, err)  # noqa: E731
    with torch.cuda.stream(side):
        call(out)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call(out)
    torch.cuda.current_stream().wait_stream(side)
    for new in (lens, [5, 1000, 0, 16, 100]):
        ctx.copy_(dev_i32(np.minimum(new, lens)))
        q.copy_(dev_bf16(wl.normal_bf16(rng, (5, N_Q, D))))
        direct = torch.empty_like(q)
        call(direct)
        torch.cuda.synchronize()
        for _ in range(2):
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, direct)
    assert int(err.item()) == 0


def test_decode_wait_that_runs_out():
    """A tile announced but never copied (the library's test hook): the call
    reports the time-out, and the next one on the workspace is right.  (Stage
    0: the only tile that CTA 0 takes whatever the others do.)"""
    pk = _pk()
    lens = [900, 33, 700]
    rng, pool, scales, table, _ = _cache(31, lens, 16)
    q = wl.normal_bf16(rng, (3, N_Q, D))
    ws = pk.decode_workspace_q8(3, table.shape[2])
    pk.pa_decode_set_test_fault(0, 50_000)
    try:
        _, err = _decode(q, pool, scales, table, lens, ws=ws)
    finally:
        pk.pa_decode_set_test_fault(-1)
    assert err & 16
    ref, _ = oracle.decode_attention(q, q8.pool_bf16(pool, scales), table, lens, 0)
    got, err = _decode(q, pool, scales, table, lens, ws=ws)
    assert err == 0
    _assert_close(got, ref, q, pool, scales, 900, 0.125, 2.0 ** -12)


# ------------------------------------------------------------------- append
class _State:
    def __init__(self, pool, scales, table, fl, fc):
        self.kv, self.sc = _dev_pool(pool, scales)
        self.bt, self.fl, self.fc, self.err = dev_i32(table), dev_i32(fl), dev_i32([fc]), dev_i32([0])

    def host(self):
        import torch
        torch.cuda.synchronize()
        return (self.kv.view(torch.uint8).cpu().numpy(), self.sc.cpu().numpy(), self.bt.cpu().numpy(),
                int(self.fc.item()), int(self.err.item()))


def _compare(st, ref, live_only=None):
    """Tables, scales, counts, errors and untouched bytes equal; a K byte may
    lie one step off where the fp32 rotation crosses a rounding border: the
    rotation is off by at most 2^-22 (|a| + |b|), a step is at least 2^-4 of
    the value or a subnormal step above that error, so one step at most, and
    below 1 in 1000 bytes."""
    qr, pool, scales, table, count, err = ref
    gp, gs, gt, gc, ge = st.host()
    assert ge == err and gc == count
    assert np.array_equal(gt, table)
    assert np.array_equal(gs, scales)
    assert np.array_equal(gp[:, 1], pool[:, 1])
    # order of the bytes along the number line; -0 and 0 are one value
    o = lambda b: np.where(b & 128, -(b & 127).astype(int), (b & 127).astype(int))  # noqa: E731
    d = np.abs(o(gp[:, 0]) - o(pool[:, 0]))
    assert d.max(initial=0) <= 1 and (d > 0).mean() <= 1e-3, (d.max(), (d > 0).mean())


def _append_case(seed, ctx, lens, page, k_scale=1.0, layers=2, layer=1):
    rng, pool, scales, table, free = _cache(seed, ctx, page, layers=layers, layer=layer, poison=False,
                                            extra=2 + sum(-(-(c + n) // page) for c, n in zip(ctx, lens)))
    mb = max(-(-(c + n) // page) for c, n in zip(ctx, lens)) + 1
    table = np.concatenate([table, np.full((len(ctx), layers, max(0, mb - table.shape[2])), -1, np.int32)], -1)
    rows = int(sum(lens))
    k, v = (wl.normal_bf16(rng, (rows, N_KV, D), scale=k_scale) for _ in range(2))
    q = wl.normal_bf16(rng, (rows, N_Q, D))
    fl = np.concatenate([free, np.full(len(pool) - len(free), -1, np.int32)]).astype(np.int32)
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    return k, v, q, cu, pool, scales, table, fl, len(free)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("k_scale", [1.0, 300.0, 1e-30], ids=["", "grows", "tiny"])
def test_decode_append(page, k_scale):
    """New and held pages, scales that grow, with and without q, in place and not."""
    ctx = [0, 1, page - 1, page, page + 1, 3 * page - 1, 1000, 31999, 5, 64]
    k, v, q, cu, pool, scales, table, fl, fc = _append_case(page, ctx, [1] * 10, page, k_scale)
    ref = q8.append(k, v, q, cu, pool, scales, table, ctx, 1, fl, fc)
    import torch
    for mode in ("in place", "out", "none"):
        st = _State(pool, scales, table, fl, fc)
        qd = None if mode == "none" else dev_bf16(q)
        qo = torch.full_like(qd, float("nan")) if mode == "out" else None
        _pk().pa_kv_append_rope_q8(dev_bf16(k), dev_bf16(v), qd, st.kv, st.sc, st.bt, dev_i32(ctx), 1, st.fl, st.fc,
                                   st.err, q_out=qo)
        _compare(st, ref)
        if qd is not None:
            got = host_bits(qo if qo is not None else qd)
            close = (ulp_diff(got, ref[0]) <= 1) | (np.abs(oracle.bf16_to_f64(got) - oracle.bf16_to_f64(ref[0])) <= 1.5e-5)
            assert np.all(close)
        if mode == "out":
            assert np.array_equal(host_bits(qd), q)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("ctx,lens,k_scale", [
    ([0, 0], [17, 14], 1.0), ([5, 0, 16, 33], [40, 0, 16, 1], 1.0), ([0], [700], 1.0),
    ([3, 7, 30, 31], [60, 2, 1, 35], 500.0), ([100] * 20, list(range(1, 21)), 1.0), ([31990], [70], 1e-34)],
    ids=["prompts", "empty", "long", "grows", "many", "far"])
def test_prefill_append(page, ctx, lens, k_scale):
    import torch
    k, v, q, cu, pool, scales, table, fl, fc = _append_case(30 + page, ctx, lens, page, k_scale)
    ref = q8.append(k, v, q, cu, pool, scales, table, ctx, 1, fl, fc)
    for q_out in (False, True):
        st = _State(pool, scales, table, fl, fc)
        qd = dev_bf16(q)
        qo = torch.full_like(qd, float("nan")) if q_out else None
        _pk().pa_prefill_append_rope_q8(dev_bf16(k), dev_bf16(v), qd, dev_i32(cu), st.kv, st.sc, st.bt, dev_i32(ctx),
                                        1, st.fl, st.fc, st.err, q_out=qo)
        _compare(st, ref)
        got = host_bits(qo if q_out else qd)
        assert np.all((ulp_diff(got, ref[0]) <= 1) |
                      (np.abs(oracle.bf16_to_f64(got) - oracle.bf16_to_f64(ref[0])) <= 1.5e-5))


@pytest.mark.parametrize("page", PAGES)
def test_appends_quantise_what_the_bf16_append_stores(page):
    """Bit for bit: the bytes are the oracle's rounding of the values that the
    framework's own bf16 append puts in its pool."""
    import torch
    pk = _pk()
    ctx, lens = [0, 5, 2 * page], [3 * page + 2, page, 7]
    k, v, q, cu, pool, scales, table, fl, fc = _append_case(60 + page, ctx, lens, page, layers=1, layer=0)
    st = _State(pool, scales, table, fl, fc)
    wide = torch.zeros((len(pool), 2, page, N_KV, D), dtype=torch.bfloat16, device="cuda")
    bt, f, c = dev_i32(table), dev_i32(fl), dev_i32([fc])
    pk.pa_prefill_append_rope(dev_bf16(k), dev_bf16(v), None, dev_i32(cu), wide, bt, dev_i32(ctx), 0, f, c, st.err)
    pk.pa_prefill_append_rope_q8(dev_bf16(k), dev_bf16(v), None, dev_i32(cu), st.kv, st.sc, st.bt, dev_i32(ctx), 0,
                                 st.fl, st.fc, st.err)
    gp, gs, gt, gc, ge = st.host()
    assert ge == 0 and np.array_equal(gt, bt.cpu().numpy()) and gc == int(c.item())
    w = oracle.bf16_to_f64(host_bits(wide))
    for s, (a, n) in enumerate(zip(ctx, lens)):
        for t in range(a, a + n):
            blk = gt[s, 0, t // page]
            assert np.array_equal(gp[blk, :, t % page], q8.encode(w[blk, :, t % page] / gs[blk][:, :, None]))


def test_append_infinities_and_nan():
    """NaN and infinities become NaN bytes and leave the scale to the rest."""
    ctx, lens = [0, 3], [4, 4]
    k, v, q, cu, pool, scales, table, fl, fc = _append_case(8, ctx, lens, 16, layers=1, layer=0)
    v[1, 2, 7], v[2, 2, 9], v[5, 0, 0] = 0x7F80, 0xFF80, 0x7FC0
    k[6, 4, 10] = 0x7F80
    ref = q8.append(k, v, None, cu, pool, scales, table, ctx, 0, fl, fc)
    st = _State(pool, scales, table, fl, fc)
    _pk().pa_prefill_append_rope_q8(dev_bf16(k), dev_bf16(v), None, dev_i32(cu), st.kv, st.sc, st.bt, dev_i32(ctx), 0,
                                    st.fl, st.fc, st.err)
    gp, gs, *_ = st.host()
    assert np.array_equal(gs, ref[2]) and np.array_equal(gp[:, 1], ref[1][:, 1])
    assert np.array_equal(np.isnan(q8.VALUES[gp[:, 0]]), np.isnan(q8.VALUES[ref[1][:, 0]]))


def test_append_errors():
    """Underflow, chunks out of range, bad table entries and scales that are
    no powers of two: reported, the rest stored."""
    page = 16
    ctx, lens = [0, 20, 5, 40, 8], [33, 4, 3, 5, 2]
    k, v, q, cu, pool, scales, table, fl, fc = _append_case(14, ctx, lens, page, layers=1, layer=0)
    table[1, 0, 1] = len(pool) + 1            # held page out of range
    scales[table[2, 0, 0], 0, 3] = 0.3        # no power of two
    scales[table[2, 0, 0], 1, 5] = 0.0
    scales[table[4, 0, 0], 1, 1] = np.inf
    ctx[3] = table.shape[2] * page            # does not fit the table
    ref = q8.append(k, v, q, cu, pool, scales, table, ctx, 0, fl, 2)
    st = _State(pool, scales, table, fl, 2)
    qd = dev_bf16(q)
    _pk().pa_prefill_append_rope_q8(dev_bf16(k), dev_bf16(v), qd, dev_i32(cu), st.kv, st.sc, st.bt, dev_i32(ctx), 0,
                                    st.fl, st.fc, st.err)
    assert ref[5] == 1 + 2 + 4 + 32
    _compare(st, ref)
    assert np.array_equal(host_bits(qd)[cu[3]:cu[4]], q[cu[3]:cu[4]])
    # the decode append on the same state
    one = np.arange(len(ctx))
    ctx2 = [0, 20, 5, -1, 8]
    ref = q8.append(k[one], v[one], None, np.arange(6), pool, scales, table, ctx2, 0, fl, 0)
    st = _State(pool, scales, table, fl, 0)
    _pk().pa_kv_append_rope_q8(dev_bf16(k[one]), dev_bf16(v[one]), None, st.kv, st.sc, st.bt, dev_i32(ctx2), 0, st.fl,
                               st.fc, st.err)
    _compare(st, ref)


def test_binding_refuses_wrong_tensors():
    import torch
    pk = _pk()
    kv, sc = pk.kv_cache_q8(4)
    t, i = dev_i32(np.zeros((2, 1, 4))), dev_i32([0, 0])
    q = torch.zeros((2, N_Q, D), dtype=torch.bfloat16, device="cuda")
    kn = torch.zeros((2, N_KV, D), dtype=torch.bfloat16, device="cuda")
    ws = pk.decode_workspace_q8(2, 4)
    dec = lambda **o: pk.pa_decode_attention_q8(*[o.get(n, d) for n, d in (  # noqa: E731
        ("out", q), ("q", q), ("kv", kv), ("sc", sc), ("t", t), ("ctx", i))], 0, 0.125, ws, i)
    for over in (dict(q=q.float()), dict(q=q[:1]), dict(q=q.transpose(1, 2)), dict(kv=kv.float()), dict(kv=kv[:, :1]),
                 dict(sc=sc[:3]), dict(sc=sc.double()), dict(ctx=i.long()), dict(ctx=i[:1]), dict(kv=kv.cpu()),
                 dict(kv=kv[..., :32].contiguous())):
        with pytest.raises((ValueError, TypeError)):
            dec(**over)
    app = lambda **o: pk.pa_kv_append_rope_q8(*[o.get(n, d) for n, d in (  # noqa: E731
        ("k", kn), ("v", kn), ("q", q), ("kv", kv), ("sc", sc), ("t", t), ("ctx", i))], 0, o.get("fl", dev_i32([0] * 4)),
        i, i, q_out=o.get("qo"))
    for over in (dict(k=kn[:1]), dict(v=kn.float()), dict(q=q[:1]), dict(qo=q[:1]), dict(fl=i)):
        with pytest.raises((ValueError, TypeError)):
            app(**over)


# --------------------------------------------------------- prefill attention
def _prefill(q, cu, pool, scales, table, ctx, layer=0, scale=0.125, out=None):
    import torch
    kv, sc = _dev_pool(pool, scales)
    if out is None:
        out = torch.full((len(q), N_Q, D), float("nan"), dtype=torch.bfloat16, device="cuda")
    err = dev_i32([0])
    _pk().pa_prefill_attention_q8(out, dev_bf16(q), dev_i32(cu), kv, sc, dev_i32(table), dev_i32(ctx), layer, scale,
                                  err)
    torch.cuda.synchronize()
    return host_f64(out), int(err.item())


def _cu(lens):
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("ctx,lens,q_scale", [
    ([0, 0], [17, 14], 1.0), ([0] * 8, [1, 2, 31, 32, 33, 63, 64, 65], 1.0), ([0, 0, 0], [127, 128, 129], 4.0),
    ([5, 100, 0, 255, 31], [40, 1, 0, 70, 64], 1.0), ([1000], [200], 8.0), ([7] * 30, [3] * 30, 1.0)],
    ids=["prompts", "tiles", "chunks", "cached", "peaked", "many"])
def test_prefill_attention(page, ctx, lens, q_scale):
    total = [a + b for a, b in zip(ctx, lens)]
    rng, pool, scales, table, _ = _cache(200 + page, total, page, layers=2, layer=1)
    cu = _cu(lens)
    q = wl.normal_bf16(rng, (cu[-1], N_Q, D), scale=q_scale)
    ref, e = oracle.prefill_attention(q, cu, q8.pool_bf16(pool, scales), table, ctx, 1, scale=0.2, block_tokens=page)
    got, err = _prefill(q, cu, pool, scales, table, ctx, layer=1, scale=0.2)
    assert err == e == 0
    _assert_close(got, ref, q, pool, scales, max(total), 0.2, 2.0 ** -12, f"page {page}")


@pytest.mark.parametrize("page", PAGES)
def test_prefill_scales_far_apart(page):
    """Values whose pages' scales lie up to 2^40 apart."""
    rng, pool, scales, table, _ = _cache(88, [150, 260], page)
    scales[:, 1] = np.ldexp(1.0, rng.integers(-30, 11, size=scales[:, 1].shape)).astype(np.float32)
    cu = _cu([150, 60])
    q = wl.normal_bf16(rng, (210, N_Q, D))
    q[:, ::5] = wl.to_bf16_bits(oracle.bf16_to_f64(q[:, ::5]).astype(np.float32) * np.float32(2.0 ** -60))
    bits = q8.pool_bf16(pool, scales)
    ref, e = oracle.prefill_attention(q, cu, bits, table, [0, 200], 0, block_tokens=page)
    got, err = _prefill(q, cu, pool, scales, table, [0, 200])
    assert err == e == 0
    # relative to what a row sums: the same weights w over the values'
    # magnitudes.  The kernel rounds P_t = w_t s_t / u (s_t: the scale of t's page;
    # u within [max w s / 2^8, max w s] of the row, so the largest P_t lies in [1,
    # 2^8]) to f16 and sums P_t times t's bytes (<= 448): half a step is 2^-12 of
    # P_t, or 2^-25 below 2^-14, so besides 2^-12 of the magnitudes the output is
    # off by at most T 2^-25 448 u <= T 2^-25 times the output for bytes of 448.
    mag, _ = oracle.prefill_attention(q, cu, np.where(np.arange(2)[None, :, None, None, None] == 1, bits & 0x7FFF, bits),
                                      table, [0, 200], 0, block_tokens=page)
    s = 0.125 * np.abs(oracle.bf16_to_f64(q)).sum(-1)[..., None] * np.nanmax(np.abs(q8.decode(pool, scales)[:, 0]))
    top = pool.copy()
    top[:, 1] = 0x7E
    cap, _ = oracle.prefill_attention(q, cu, q8.pool_bf16(top, scales), table, [0, 200], 0, block_tokens=page)
    tol = bf16_half_ulp(ref) + mag * (2.0 ** -12 + 2.0 ** -16 * s) + cap * 260 * 2.0 ** -25
    assert np.all(np.abs(got - ref) <= tol), (np.abs(got - ref) / tol).max()


@pytest.mark.parametrize("page", PAGES)
def test_prefill_bad_pages_and_refused_chunks(page):
    """A bad page's tokens are dropped and reported; a refused chunk's rows
    stay as they were; NaN bytes in dropped and unused places reach nothing."""
    ctx, lens = [100, 0, 20], [50, 40, 3]
    rng, pool, scales, table, _ = _cache(300 + page, [150, 40, 23], page)
    pool[table[0, 0, 2]] = 0x7F
    table[0, 0, 2] = pool.shape[0] + 7
    cu = _cu(lens)
    q = wl.normal_bf16(rng, (cu[-1], N_Q, D))
    ref, e = oracle.prefill_attention(q, cu, q8.pool_bf16(pool, scales), table, ctx, 0, block_tokens=page)
    got, err = _prefill(q, cu, pool, scales, table, ctx)
    assert err == e == oracle.ERR_BAD_BLOCK
    _assert_close(got, ref, q, pool, scales, 150, 0.125, 2.0 ** -12)
    ctx[1] = table.shape[2] * page
    got, err = _prefill(q, cu, pool, scales, table, ctx)
    assert err == oracle.ERR_BAD_BLOCK | oracle.ERR_CTX_RANGE
    assert np.all(np.isnan(got[50:90]))
    _assert_close(got[:50], ref[:50], q, pool, scales, 150, 0.125, 2.0 ** -12)
    _assert_close(got[90:], ref[90:], q, pool, scales, 150, 0.125, 2.0 ** -12)


def test_prefill_nan_key_and_value():
    """A NaN key or value makes the rows of its kv head that see it NaN, and no others."""
    rng, pool, scales, table, _ = _cache(6, [90], 16)
    pool[table[0, 0, 1], 0, 4, 2, 9] = 0x7F        # key 20, kv head 2
    pool[table[0, 0, 3], 1, 2, 5, 1] = 0xFF        # value 50, kv head 5, dim 1
    q = wl.normal_bf16(rng, (90, N_Q, D))
    got, err = _prefill(q, _cu([90]), pool, scales, table, [0])
    assert err == 0
    bad = np.zeros(got.shape, bool)
    bad[20:, 8:12] = True
    bad[50:, 20:24, 1] = True
    assert np.array_equal(np.isnan(got), bad)


@pytest.mark.parametrize("bad", [0x7F80, 0xFF80, 0x7FC0])
def test_prefill_q_row_not_finite(bad):
    """An infinity or NaN in a row of q makes that row's output NaN and changes no other row."""
    rng, pool, scales, table, _ = _cache(8, [200], 16)
    q = wl.normal_bf16(rng, (150, N_Q, D))
    want, _ = _prefill(q, _cu([150]), pool, scales, table, [50])
    q = q.copy()
    q[40, 9, 3] = bad
    q[100, 31, 63] = bad
    got, err = _prefill(q, _cu([150]), pool, scales, table, [50])
    assert err == 0
    rows = np.zeros((150, N_Q), bool)
    rows[40, 9] = rows[100, 31] = True
    assert np.isnan(got[rows]).all()
    assert np.array_equal(got[~rows], want[~rows])


def test_prefill_wait_that_runs_out():
    """A chunk announced but never copied (the library's test hook): the call
    reports the time-out, and the next one is right."""
    import torch
    pk = _pk()
    rng, pool, scales, table, _ = _cache(7, [700], 16)
    q = wl.normal_bf16(rng, (300, N_Q, D))
    pk.pa_prefill_set_test_fault(1, 50_000)
    try:
        _, err = _prefill(q, _cu([300]), pool, scales, table, [400])
    finally:
        pk.pa_prefill_set_test_fault(-1)
    assert err & 16
    ref, _ = oracle.prefill_attention(q, _cu([300]), q8.pool_bf16(pool, scales), table, [400], 0)
    got, err = _prefill(q, _cu([300]), pool, scales, table, [400])
    assert err == 0
    _assert_close(got, ref, q, pool, scales, 700, 0.125, 2.0 ** -12)


# ---------------------------------------------------------- all of them at once
@pytest.mark.parametrize("page", PAGES)
def test_prompts_then_decode_steps_then_free(page):
    """As a server runs them, over two layers: prompts appended and attended,
    a second chunk, decode steps captured as one graph, pages returned.  The
    attention is compared with the oracle over the values in the cache, the
    cache with the oracle's."""
    import torch
    pk = _pk()
    rng = np.random.default_rng(page)
    lens, more, steps, layers = [17, 3, 40], [5, 33, 0], 2 * page + 3, 2
    n, blocks = 3, 64
    mb = -(-(max(lens) + max(more) + steps) // page) + 1
    pool, scales = q8.random_pool(rng, blocks, page)
    table = np.full((n, layers, mb), -1, np.int32)
    fl = rng.permutation(blocks).astype(np.int32)
    st = _State(pool, scales, table, fl, blocks)
    p, sc, t, c = pool, scales, table, blocks
    ctx = np.zeros(n, np.int32)
    for chunk in (lens, more):
        cu = _cu(chunk)
        for layer in range(layers):
            k, v = (wl.normal_bf16(rng, (cu[-1], N_KV, D)) for _ in range(2))
            q = wl.normal_bf16(rng, (cu[-1], N_Q, D))
            _, p, sc, t, c, e = q8.append(k, v, None, cu, p, sc, t, ctx, layer, fl, c)
            qd = dev_bf16(q)
            pk.pa_prefill_append_rope_q8(dev_bf16(k), dev_bf16(v), qd, dev_i32(cu), st.kv, st.sc, st.bt, dev_i32(ctx),
                                         layer, st.fl, st.fc, st.err)
            out = torch.full_like(qd, float("nan"))
            pk.pa_prefill_attention_q8(out, qd, dev_i32(cu), st.kv, st.sc, st.bt, dev_i32(ctx), layer, 0.125, st.err)
            _compare(st, (None, p, sc, t, c, e))
            gp = st.host()[0]
            ref, _ = oracle.prefill_attention(host_bits(qd), cu, q8.pool_bf16(gp, sc), t, ctx, layer, block_tokens=page)
            _assert_close(host_f64(out), ref, q, gp, sc, 100, 0.125, 2.0 ** -12)
            p = gp
        ctx = ctx + np.asarray(chunk, np.int32)
    # decode: one graph of both layers, its inputs refilled
    kd, vd = (torch.empty((layers, n, N_KV, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    qd = torch.empty((layers, n, N_Q, D), dtype=torch.bfloat16, device="cuda")
    od = torch.empty_like(qd)
    ctx_d, ctx1_d = dev_i32(ctx), dev_i32(ctx + 1)
    ws = pk.decode_workspace_q8(n, mb, block_tokens=page)

    def step():
        for layer in range(layers):
            pk.pa_kv_append_rope_q8(kd[layer], vd[layer], qd[layer], st.kv, st.sc, st.bt, ctx_d, layer, st.fl, st.fc,
                                    st.err)
            pk.pa_decode_attention_q8(od[layer], qd[layer], st.kv, st.sc, st.bt, ctx1_d, layer, 0.125, ws, st.err)
        ctx_d.add_(1)
        ctx1_d.add_(1)

    graph = None
    for i in range(steps):
        k, v = (wl.normal_bf16(rng, (layers, n, N_KV, D)) for _ in range(2))
        q = wl.normal_bf16(rng, (layers, n, N_Q, D))
        kd.copy_(dev_bf16(k)), vd.copy_(dev_bf16(v)), qd.copy_(dev_bf16(q))
        if i == 0:
            step()
            torch.cuda.synchronize()
        elif graph is None:
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph):
                step()
            graph.replay()
        else:
            graph.replay()
        for layer in range(layers):
            _, p, sc, t, c, e = q8.append(k[layer], v[layer], None, np.arange(n + 1), p, sc, t, ctx, layer, fl, c)
        ctx = ctx + 1
        _compare(st, (None, p, sc, t, c, 0))
        p = st.host()[0]
        for layer in range(layers):
            ref, _ = oracle.decode_attention(host_bits(qd[layer]), q8.pool_bf16(p, sc), t, ctx, layer, block_tokens=page)
            _assert_close(host_f64(od[layer]), ref, q, p, sc, 100, 0.125, 2.0 ** -12)
    pk.pa_free(dev_i32([0, 1, 2]), st.bt, dev_i32(ctx), st.fl, st.fc, blocks, st.err, block_tokens=page)
    _, _, bt, count, err = st.host()
    assert err == 0 and count == blocks and np.all(bt == -1)
    assert np.array_equal(np.sort(st.fl.cpu().numpy()), np.arange(blocks))


@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("far", [False, True], ids=["", "far"])
def test_smallest_value_scales(page, far):
    """Values of 2^-110 (the smallest scale), alone and beside pages of 2^-90.
    The prefill kernel holds what lies below 2^-94 of a scale in f16 values whose
    last step is 2^-24: half of it, 2^-25 2^-94, comes to the bound."""
    lens = [300, 20]
    rng, pool, scales, table, _ = _cache(55 + page, lens, page)
    scales[:, 1] = 2.0 ** -117
    if far:
        scales[::3, 1] = 2.0 ** -97
    q = wl.normal_bf16(rng, (sum(lens), N_Q, D))
    ref, _ = oracle.prefill_attention(q, _cu(lens), q8.pool_bf16(pool, scales), table, [0, 0], 0, block_tokens=page)
    got, err = _prefill(q, _cu(lens), pool, scales, table, [0, 0])
    assert err == 0 and np.abs(ref).max() < 2.0 ** -85 and np.all(np.abs(ref).max(-1) > 0)
    v = np.abs(q8.decode(pool, scales))
    s = 0.125 * np.abs(oracle.bf16_to_f64(q)).sum(-1).max() * np.nanmax(v[:, 0])
    tol = bf16_half_ulp(ref) + np.nanmax(v[:, 1]) * (2.0 ** -12 + 300 * 2.0 ** -25 + s * 2.0 ** -16) + 2.0 ** -119
    assert np.all(np.abs(got - ref) <= tol)
    last = [lens[0] - 1, sum(lens) - 1]
    dec, err = _decode(q[last], pool, scales, table, lens)
    assert err == 0 and np.all(np.abs(dec - ref[last]) <= tol[last])


# ------------------------------------------------------------ scores of any size
@pytest.mark.parametrize("page", PAGES)
@pytest.mark.parametrize("exponent", [30, 60, 110], ids=["2^30", "2^60", "2^110"])
@pytest.mark.parametrize("negative", [False, True], ids=["", "negative"])
def test_scores_beyond_the_exponential(page, exponent, negative):
    """Scores of about 2^exponent, all negative in one case: a row's weight is all
    on its largest score (the next lies 2^-9 of it below, 2^21 and more: its weight
    is 0 in fp64 too), however coarse fp32's steps are there.  Rows whose two
    largest scores are closer (fp32 sums of 64 products are off by up to 2^-17 of
    the largest) are not looked at."""
    lens = [50, 137]
    rng, pool, scales, table, _ = _cache(101 + page, lens, page, poison=False)
    scales[:, 0] = 2.0 ** (exponent // 2)
    if negative:
        pool[:, 0] &= 0x7F
    q = np.abs(rng.standard_normal((sum(lens), N_Q, D))) if negative else rng.standard_normal((sum(lens), N_Q, D))
    q = oracle.f64_to_bf16((-1 if negative else 1) * q * 2.0 ** (exponent - exponent // 2 - 8))
    vals, qf = q8.decode(pool, scales), oracle.bf16_to_f64(q)
    got, err = _prefill(q, _cu(lens), pool, scales, table, [0, 0])
    last = [lens[0] - 1, sum(lens) - 1]
    dec, err2 = _decode(q[last], pool, scales, table, lens)
    assert err == err2 == 0
    looked = 0
    for s, (r0, n) in enumerate(zip([0, lens[0]], lens)):
        kv = vals[table[s, 0, :-(-n // page)]]
        keys, values = (kv[:, j].reshape(-1, N_KV, D)[:n] for j in (0, 1))
        for h in range(N_Q):
            z = qf[r0:r0 + n, h] @ keys[:, h // 4].T * 0.125
            z[np.triu_indices(n, 1)] = -np.inf
            order = np.sort(z, -1)
            rows = np.arange(n)
            apart = rows[(rows == 0) | (order[:, -1] - order[:, -2] > 2.0 ** -9 * np.abs(z[z > -np.inf]).max())]
            want = values[z[apart].argmax(-1), h // 4]
            tol = bf16_half_ulp(want)
            assert np.all(np.abs(got[r0 + apart, h] - want) <= tol)
            if n - 1 in apart:
                assert np.all(np.abs(dec[s, h] - want[-1]) <= tol[-1])
            looked += len(apart)
    assert looked > N_Q * sum(lens) // 4


# ------------------------------------------------------------ ways to call them
def test_default_explicit_and_side_stream_agree():
    """The current stream by default, a stream given, a side stream made current:
    the same bits from each of the four calls."""
    import torch
    pk = _pk()
    lens = [40, 0, 129, 7]
    k, v, q, cu, pool, scales, table, fl, fc = _append_case(91, lens, [3, 1, 20, 0], 16)
    side = torch.cuda.Stream()

    def run(stream, current):
        st = _State(pool, scales, table, fl, fc)
        n, ctx = len(lens), dev_i32(lens)
        kd, vd, qd, cud = dev_bf16(k), dev_bf16(v), dev_bf16(q), dev_i32(cu)
        turned, out, dec = torch.zeros_like(qd), torch.zeros_like(qd), torch.zeros_like(qd[:n])
        ws = pk.decode_workspace_q8(n, table.shape[2])
        torch.cuda.synchronize()
        with torch.cuda.stream(current):
            pk.pa_prefill_append_rope_q8(kd, vd, qd, cud, st.kv, st.sc, st.bt, ctx, 1, st.fl, st.fc, st.err,
                                         stream=stream, q_out=turned)
            pk.pa_prefill_attention_q8(out, turned, cud, st.kv, st.sc, st.bt, ctx, 1, 0.125, st.err, stream=stream)
            after = ctx + (cud[1:] - cud[:-1]) if stream is None else dev_i32(np.add(lens, np.diff(cu)))
            pk.pa_kv_append_rope_q8(kd[:n], vd[:n], qd[:n], st.kv, st.sc, st.bt, after, 1, st.fl, st.fc, st.err,
                                    stream=stream)
            pk.pa_decode_attention_q8(dec, qd[:n], st.kv, st.sc, st.bt, dev_i32(np.add(lens, np.diff(cu)) + 1), 1,
                                      0.125, ws, st.err, stream=stream)
        torch.cuda.synchronize()
        return [turned, out, dec, qd, *map(torch.from_numpy, st.host()[:3]), *st.host()[3:]]

    main = torch.cuda.current_stream()
    want = run(None, main)
    assert want[-1] == 0
    for got in (run(main, main), run(None, side)):
        for a, b in zip(got, want):
            assert torch.equal(a, b) if isinstance(a, torch.Tensor) else a == b


def test_two_graphs_share_a_workspace():
    """Graphs of different batches captured over one workspace, replayed one after
    the other in either order, with an eager call between."""
    import torch
    pk = _pk()
    batches, ws = [], None
    for seed, lens in ((71, [3000, 20, 900]), (72, [64] * 40)):
        rng, pool, scales, table, _ = _cache(seed, lens, 16)
        kv, sc = _dev_pool(pool, scales)
        q, err = dev_bf16(wl.normal_bf16(rng, (len(lens), N_Q, D))), dev_i32([0])
        if ws is None:
            ws = pk.decode_workspace_q8(40, 200)
        args = (q, kv, sc, dev_i32(table), dev_i32(lens), 0, 0.125, ws, err)
        want, out = torch.empty_like(q), torch.empty_like(q)
        pk.pa_decode_attention_q8(want, *args)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            pk.pa_decode_attention_q8(out, *args)
        batches.append((g, out, want, args))
    for order in ((0, 1), (1, 0), (0, 0, 1)):
        for i in order:
            g, out, want, args = batches[i]
            out.fill_(float("nan"))
            g.replay()
            other = torch.empty_like(batches[1 - i][1])
            pk.pa_decode_attention_q8(other, *batches[1 - i][3])
            torch.cuda.synchronize()
            assert torch.equal(out, want) and torch.equal(other, batches[1 - i][2])


def test_prefill_graph_replayed_with_other_lengths():
    """Captured once; replayed with other contexts, splits and inputs: a direct call's bits."""
    import torch
    pk = _pk()
    rng, pool, scales, table, _ = _cache(61, [500, 300, 200], 16)
    kv, sc = _dev_pool(pool, scales)
    rows = 180
    q, out = (torch.zeros((rows, N_Q, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    cu, ctx, err = dev_i32(_cu([100, 50, 30])), dev_i32([400, 0, 0]), dev_i32([0])
    args = (q, cu, kv, sc, dev_i32(table), ctx, 0, 0.125, err)
    g = torch.cuda.CUDAGraph()
    pk.pa_prefill_attention_q8(out, *args)
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        pk.pa_prefill_attention_q8(out, *args)
    for lens, c in (([100, 50, 30], [400, 0, 0]), ([0, 179, 1], [0, 121, 199]), ([64, 0, 116], [1, 5, 0])):
        cu.copy_(dev_i32(_cu(lens))), ctx.copy_(dev_i32(c))
        q.copy_(dev_bf16(wl.normal_bf16(rng, (rows, N_Q, D))))
        direct = torch.full_like(q, float("nan"))
        pk.pa_prefill_attention_q8(direct, *args)
        out.fill_(float("nan"))
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, direct) and bool(torch.isfinite(direct).all())
    assert int(err.item()) == 0


@pytest.mark.parametrize("tiles", [2047, 2048, 2049])
def test_prefill_as_many_tiles_as_are_sorted(tiles):
    """One more tile than the work order holds, and up to it: sequences of one
    token, and one of as many tiles as are left."""
    lens = [1] * 1900 + [64 * (tiles - 1900) - 63]
    page = 16
    ctx = [3] * 1900 + [0]
    rng, pool, scales, table, _ = _cache(tiles, [c + n for c, n in zip(ctx, lens)], page, poison=False)
    q = wl.normal_bf16(rng, (sum(lens), N_Q, D))
    got, err = _prefill(q, _cu(lens), pool, scales, table, ctx)
    assert err == 0 and np.all(np.isfinite(got))
    # the single tokens, and the long one's first and last rows (as decode rows)
    n = 1900
    rows = list(range(n)) + [n, n + 63, n + 64, sum(lens) - 1]
    t = np.concatenate([table[:n], np.repeat(table[n:], 4, 0)])
    seen = [4] * n + [r - n + 1 for r in rows[n:]]
    ref, _ = oracle.decode_attention(q[rows], q8.pool_bf16(pool, scales), t, seen, 0, block_tokens=page)
    _assert_close(got[rows], ref, q[rows], pool, scales, max(seen), 0.125, 2.0 ** -12)


@pytest.mark.parametrize("page", PAGES)
def test_prefill_append_of_many_short_chunks(page):
    """More sequences than the CTA has threads, most of a token or three, some
    empty, some refused (past the table's end, or a negative context)."""
    _many_short_chunks(page, 1100)


def test_prefill_append_of_a_great_many_empty_chunks():
    """More sequences than the threads squared, 49 in 50 empty."""
    _many_short_chunks(16, 70000, 0.98)


def _many_short_chunks(page, n, empty=0.0):
    rng = np.random.default_rng(page)
    lens = rng.integers(0, 4, n)
    lens[[5, 700]] = [2 * page + 1, page]
    ctx = rng.integers(0, 3 * page, n)
    if empty:
        gone = rng.random(n) < empty
        lens[gone] = ctx[gone] = 0
    k, v, q, cu, pool, scales, table, fl, fc = _append_case(40 + page, ctx.tolist(), lens.tolist(), page, layers=1,
                                                            layer=0)
    ctx[[9, 900]] = [-1, table.shape[2] * page]
    ref = q8.append(k, v, q, cu, pool, scales, table, ctx.tolist(), 0, fl, fc)
    st = _State(pool, scales, table, fl, fc)
    qd = dev_bf16(q)
    _pk().pa_prefill_append_rope_q8(dev_bf16(k), dev_bf16(v), qd, dev_i32(cu), st.kv, st.sc, st.bt, dev_i32(ctx), 0,
                                    st.fl, st.fc, st.err)
    _compare(st, ref)
    # the rotation is off by at most 2^-22 (|a| + |b|), below 3e-6 for |q| < 6: one
    # step of the result, or, where the two products cancel and steps are smaller
    # than that, less than 1.5e-5
    got = host_bits(qd)
    assert np.all((ulp_diff(got, ref[0]) <= 1) |
                  (np.abs(oracle.bf16_to_f64(got) - oracle.bf16_to_f64(ref[0])) <= 1.5e-5))
