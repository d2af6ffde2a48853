"""The operators over a paged cache held in 8 bits, as cases to measure.

A cache page holds its keys and values as e4m3 numbers with one scale, a
power of two, for each page, kv head and K or V:

  kv_cache   [num_blocks][2][page][8][64] e4m3 (0 = K, 1 = V)
  kv_scales  [num_blocks][2][8] fp32; a value is byte * scale

Four operators work on it:

  append           one new token a sequence: rotate k and q, quantise k and v
                   into the page that the table names
  prompt_append    the same for a prompt chunk a sequence
  decode           one query token a sequence attends over its pages
  prompt_attention causal attention of a prompt chunk over its pages

A scale is 2^e with the smallest e (at least -117) for which the largest
magnitude of the head's values in the page is at most 448 * 2^e (V) or
316 * 2^e (K, taken before the rotation: 316 sqrt(2) < 448, so that it holds
at any position).  An append to a page that holds tokens keeps the larger of
its scale and the new token's, and brings the tokens it holds to it.
"""
import math
import random

import numpy as np
import torch

own = False

N_Q, N_KV, DIM, GROUP = 32, 8, 64, 4
TOP_K, TOP_V, E_MIN, E_MAX = 316.0, 448.0, -117, 120


# ------------------------------------------------------------------- cases
def listed():
    """Lengths: "fixed:a", "uniform:a:b" or "log:a:b" (whole numbers, drawn from lens_seed)."""
    def case(name, op, seqs, ctx, page=16, chunk="fixed:0", layers=1, layer=0, q_scale=1.0):
        return {"name": name, "op": op, "seqs": seqs, "ctx": ctx, "chunk": chunk, "page": page,
                "layers": layers, "layer": layer, "q_scale": q_scale, "lens_seed": 11}
    return [
        # a serving step of 16 rows: bound by the latency of its launches
        case("append 16", "append", 16, "uniform:256:2048", layers=2, layer=1),
        # the full batch with lengths of every size, many pages opened at once
        case("append 256", "append", 256, "log:1:8192"),
        # two short prompts: the smallest call a server makes
        case("prompt_append 31", "prompt_append", 2, "fixed:0", chunk="uniform:14:17"),
        # a batch of fresh long prompts
        case("prompt_append 8x2048", "prompt_append", 8, "fixed:0", chunk="fixed:2048"),
        # chunked prompts whose chunks start and end inside a 32-token page
        case("prompt_append ragged", "prompt_append", 32, "uniform:3900:4100", chunk="uniform:300:512",
             page=32, layers=2, layer=0),
        # the smallest decode call: two rows of a few tokens
        case("decode 2", "decode", 2, "uniform:14:17"),
        # a serving step of 16 rows
        case("decode 16", "decode", 16, "uniform:256:2048", layers=2, layer=1),
        # the full batch, lengths from one token to 8192: bound by memory
        case("decode 256", "decode", 256, "log:1:8192"),
        # few rows of long contexts, a peaked softmax, pages of 32 tokens
        case("decode 4x32768", "decode", 4, "fixed:32768", page=32, q_scale=4.0),
        # two short prompts
        case("prompt_attention 31", "prompt_attention", 2, "fixed:0", chunk="uniform:14:17"),
        # a batch of fresh long prompts: bound by arithmetic
        case("prompt_attention 8x2048", "prompt_attention", 8, "fixed:0", chunk="fixed:2048"),
        # chunks after long cached contexts, the largest call
        case("prompt_attention 32x512", "prompt_attention", 32, "fixed:4096", chunk="fixed:512"),
    ]


def _log_int(rng, a, b):
    return max(a, min(b, int(math.exp(rng.uniform(math.log(a), math.log(b + 1))))))


def draw(rng):
    """Batches of 1 to 256 rows, contexts of 1 to 32768 tokens, chunks of 1 to 2048, pages of 8, 16
    and 32 tokens; no case larger than the listed ones of its operator."""
    op = rng.choice(["append", "prompt_append", "decode", "prompt_attention"])
    c = {"op": op, "page": rng.choice([8, 16, 16, 32]), "layers": rng.choice([1, 2]), "q_scale": 1.0,
         "lens_seed": rng.randrange(1 << 30), "chunk": "fixed:0"}
    c["layer"] = rng.randrange(c["layers"])
    if op in ("append", "decode"):
        c["seqs"] = _log_int(rng, 1, 256)
        top = _log_int(rng, 1, min(32768, (1 << 21) // c["seqs"]))
        low = _log_int(rng, 1, top)
        c["ctx"] = "%s:%d:%d" % (rng.choice(["uniform", "log"]), low, top)
        if op == "decode":
            c["q_scale"] = rng.choice([1.0, 1.0, 4.0])
    else:
        c["seqs"] = _log_int(rng, 1, 32)
        long = _log_int(rng, 1, min(2048, 16384 // c["seqs"]))
        room = (32 * 512 * 4608) // (c["seqs"] * long) - long
        top = _log_int(rng, 1, max(1, min(16384, room)))
        c["chunk"] = "uniform:%d:%d" % (max(1, long // 2), long)
        c["ctx"] = rng.choice(["fixed:0", "uniform:%d:%d" % (top // 2, top)])
    return c


def _lengths(law, rng, n):
    kind, *ab = law.split(":")
    a, b = int(ab[0]), int(ab[-1])
    if kind == "fixed":
        return [a] * n
    if kind == "uniform":
        return [rng.randint(a, b) for _ in range(n)]
    return [_log_int(rng, a, b) for _ in range(n)]


def _plan(case):
    """(tokens cached before the call, chunk tokens) of every sequence."""
    rng = random.Random(case["lens_seed"])
    ctx = _lengths(case["ctx"], rng, case["seqs"])
    return ctx, _lengths(case["chunk"], rng, case["seqs"])


def work(case):
    ctx, chunk = _plan(case)
    n, page, op = case["seqs"], case["page"], case["op"]
    per_q, per_kv8, per_scale = N_Q * DIM * 2, 2 * N_KV * DIM, 2 * N_KV * 4
    if op in ("append", "prompt_append"):
        rows = n if op == "append" else sum(chunk)
        added = [1] * n if op == "append" else chunk
        pages = sum((a + b - 1) // page - a // page + 1 for a, b in zip(ctx, added))
        # k, v in; q in and out; bytes, scales and table entries out; lengths
        size = rows * (2 * per_kv8 + 2 * per_q + per_kv8) + pages * (per_scale + 4) + 4 * n
        return {"bytes": size, "flops": rows * (N_Q + N_KV) * DIM * 3}
    if op == "decode":
        pages = sum(-(-t // page) for t in ctx)
        size = sum(ctx) * per_kv8 + pages * (per_scale + 4) + n * (2 * per_q + 4)
        return {"bytes": size, "flops": 4 * DIM * N_Q * sum(ctx)}
    pages = sum(-(-(a + b) // page) for a, b in zip(ctx, chunk))
    pairs = sum(a * b + b * (b + 1) // 2 for a, b in zip(ctx, chunk))
    size = (sum(ctx) + sum(chunk)) * per_kv8 + pages * (per_scale + 4) + sum(chunk) * 2 * per_q + 8 * n
    return {"bytes": size, "flops": 4 * DIM * N_Q * pairs}


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    ctx, chunk = _plan(case)
    n, page, layers, layer, op = case["seqs"], case["page"], case["layers"], case["layer"], case["op"]
    # attention reads pages that hold the chunk too; an append opens them
    held = [a + b for a, b in zip(ctx, chunk)] if op == "prompt_attention" else ctx
    after = [a + b + (op == "append") for a, b in zip(ctx, chunk)]
    columns = max(-(-t // page) for t in after) + 1
    opened = sum(-(-a // page) - -(-h // page) for a, h in zip(after, held))
    have = torch.tensor([-(-t // page) for t in held], device=dev)
    filled = (torch.arange(columns, device=dev)[None, :] < have[:, None])[:, None, :].expand(n, layers, columns)
    used = int(sum(-(-t // page) for t in held)) * layers
    blocks = used + opened + used // 8 + 16
    ids = torch.randperm(blocks, generator=g, device=dev).to(torch.int32)
    table = torch.full((n, layers, columns), -1, dtype=torch.int32, device=dev)
    table[filled] = ids[:used]
    # keys and values about N(0, 1) to N(0, 3), as a cache in use holds them
    pool = torch.empty((blocks, 2, page, N_KV, DIM), dtype=torch.float8_e4m3fn, device=dev)
    flat = pool.view(-1)
    for i in range(0, flat.numel(), 1 << 28):
        part = flat[i:i + (1 << 28)]
        part.copy_((torch.randn(part.numel(), generator=g, device=dev) * 90.0).clamp_(-448.0, 448.0))
    scales = torch.exp2(torch.randint(-7, -4, (blocks, 2, N_KV), generator=g, device=dev).float())
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=dev)  # noqa: E731
    normal = lambda *s: torch.randn(*s, generator=g, device=dev).to(torch.bfloat16)  # noqa: E731
    rows = n if op in ("append", "decode") else sum(chunk)
    s = {"op": op, "page": page, "layer": layer, "scale": 0.125, "pool": pool, "scales": scales, "table": table,
         "ctx": i32(ctx), "err": i32([0]), "longest": max(after), "longest_chunk": max(chunk),
         "q": (torch.randn(rows, N_Q, DIM, generator=g, device=dev) * case["q_scale"]).to(torch.bfloat16)}
    s["out"] = torch.empty_like(s["q"])
    if op in ("append", "prompt_append"):
        s["k"], s["v"] = normal(rows, N_KV, DIM), normal(rows, N_KV, DIM)
        s["free_list"] = torch.cat([ids[used:], ids.new_full((used,), -1)])
        s["free_count"] = i32([blocks - used])
    if op in ("prompt_append", "prompt_attention"):
        s["cu"] = i32([0] + np.cumsum(chunk).tolist())
        # the scheduler's plan of the step: each packed row's sequence
        s["row_seq"] = torch.repeat_interleave(torch.arange(n, device=dev), torch.tensor(chunk, device=dev))
    if own and op == "decode":
        import paged_kv_cache_205_gb300 as pk
        s["workspace"] = pk.decode_workspace_q8(n, columns, block_tokens=page)
    return s


# --------------------------------------------------------------------- run
def run(s):
    if own:
        return _own(s)
    return {"append": _append, "prompt_append": _prompt_append, "decode": _decode,
            "prompt_attention": _prompt_attention}[s["op"]](s)


def _own(s):
    import paged_kv_cache_205_gb300 as pk
    op = s["op"]
    if op == "decode":
        pk.pa_decode_attention_q8(s["out"], s["q"], s["pool"], s["scales"], s["table"], s["ctx"], s["layer"],
                                  s["scale"], s["workspace"], s["err"])
        return s["out"]
    if op == "prompt_attention":
        pk.pa_prefill_attention_q8(s["out"], s["q"], s["cu"], s["pool"], s["scales"], s["table"], s["ctx"],
                                   s["layer"], s["scale"], s["err"])
        return s["out"]
    # the count as it stands before the step, so that the pass can be made again
    count = s["free_count"].clone()
    if op == "append":
        pk.pa_kv_append_rope_q8(s["k"], s["v"], s["q"], s["pool"], s["scales"], s["table"], s["ctx"], s["layer"],
                                s["free_list"], count, s["err"], q_out=s["out"])
    else:
        pk.pa_prefill_append_rope_q8(s["k"], s["v"], s["q"], s["cu"], s["pool"], s["scales"], s["table"], s["ctx"],
                                     s["layer"], s["free_list"], count, s["err"], q_out=s["out"])
    return {"pool": s["pool"], "scales": s["scales"], "table": s["table"], "count": count, "q": s["out"]}


def _frequencies():
    """Inverse frequencies of the 32 pairs: theta 500000, rescaled by 32 beyond 8192 tokens."""
    f = []
    for i in range(DIM // 2):
        x = 500000.0 ** (-2.0 * i / DIM)
        ratio = 8192.0 * x / (2.0 * math.pi)
        w = min(1.0, max(0.0, (ratio - 1.0) / 3.0))
        f.append(w * x + (1.0 - w) * x / 32.0)
    return f


def _rotate(x, pos):
    """Rotate-half rotation in 64 bits (far angles, values next to a rounding border)."""
    f = torch.tensor(_frequencies(), dtype=torch.float64, device=x.device)
    angle = (pos.double()[:, None] * f)[:, None, :]
    c, n = torch.cos(angle), torch.sin(angle)
    a, b = x[..., :DIM // 2].double(), x[..., DIM // 2:].double()
    return torch.cat([a * c - b * n, b * c + a * n], -1).to(torch.bfloat16)


def _exponent(top, limit):
    """The smallest e >= E_MIN with top <= limit * 2^e."""
    m, e = torch.frexp(top)
    lm, le = math.frexp(limit)
    e = e - le + (m > lm).to(e.dtype)
    return torch.where(top > 0, e, E_MIN).clamp(E_MIN, E_MAX)


def _to_e4m3(x):
    return x.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _store(s, k, v, blk, slot, fresh, first_blk, first_slot):
    """Rows (k rotated, v) into slot `slot` of pages `blk`; `fresh` rows lie in pages opened by this call.
    first_blk / first_slot: the page and slot of every sequence's first row (rows before it are held)."""
    pool, scales = s["pool"].view(torch.uint8), s["scales"]
    top = torch.stack([s["k"].float().abs().amax(-1), s["v"].float().abs().amax(-1)], 1)      # [rows][2][8]
    of_page = torch.zeros_like(scales)
    of_page.scatter_reduce_(0, blk[:, None, None].expand_as(top), top, "amax")
    top = of_page[blk]
    need = torch.stack([_exponent(top[:, 0], TOP_K), _exponent(top[:, 1], TOP_V)], 1)
    held = torch.frexp(scales[blk])[1] - 1
    e = torch.where(fresh[:, None, None], need, torch.maximum(need, held))
    before = scales[first_blk]
    scales[blk] = torch.exp2(e.float())
    # tokens that a page holds already are brought to its new scale
    ratio = (before / scales[first_blk])[:, :, None, :, None]
    old = pool[first_blk]
    moved = _to_e4m3(old.view(torch.float8_e4m3fn).float() * ratio)
    is_held = torch.arange(pool.shape[2], device=pool.device)[None, :] < first_slot[:, None]
    pool[first_blk] = torch.where(is_held[:, None, :, None, None], moved, old)
    inv = torch.exp2(-e.float())
    pool[blk, 0, slot] = _to_e4m3(k.float() * inv[:, 0, :, None])
    pool[blk, 1, slot] = _to_e4m3(v.float() * inv[:, 1, :, None])


def _append(s):
    pos, page = s["ctx"].long(), s["page"]
    row = s["table"][:, s["layer"]]
    slot = pos % page
    opens = slot == 0
    taken = s["free_list"][(s["free_count"] - torch.cumsum(opens, 0)).clamp(min=0).long()]
    column = (pos // page)[:, None]
    blk = torch.where(opens, taken, row.gather(1, column)[:, 0])
    row.scatter_(1, column, blk[:, None])
    blk = blk.long()
    _store(s, _rotate(s["k"], pos), s["v"], blk, slot, opens, blk, slot)
    count = (s["free_count"] - opens.sum()).to(torch.int32)
    return {"pool": s["pool"], "scales": s["scales"], "table": s["table"], "count": count, "q": _rotate(s["q"], pos)}


def _prompt_append(s):
    page, seq, ctx, cu = s["page"], s["row_seq"], s["ctx"].long(), s["cu"].long()
    pos = ctx[seq] + torch.arange(seq.numel(), device=seq.device) - cu[seq]
    slot, column = pos % page, pos // page
    opens = slot == 0
    taken = s["free_list"][(s["free_count"] - torch.cumsum(opens, 0)).clamp(min=0).long()]
    # the rows that open a page write its entry; the others write it again
    row = s["table"][:, s["layer"]]
    last_open = torch.cummax(torch.where(opens, torch.arange(seq.numel(), device=seq.device), -1), 0)[0]
    fresh = column * page >= ctx[seq]
    blk = torch.where(fresh, taken[last_open.clamp(min=0)], row[seq, column])
    row[seq, column] = blk
    blk = blk.long()
    _store(s, _rotate(s["k"], pos), s["v"], blk, slot, fresh, blk[cu[:-1]], slot[cu[:-1]])
    count = (s["free_count"] - opens.sum()).to(torch.int32)
    return {"pool": s["pool"], "scales": s["scales"], "table": s["table"], "count": count, "q": _rotate(s["q"], pos)}


def _cached(s, longest):
    """Keys and values [n][8][tokens][64] of every sequence's first `longest` positions."""
    page = s["page"]
    ids = s["table"][:, s["layer"], :-(-longest // page)].clamp(min=0).long()
    x = s["pool"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).float()      # [n][pages][2][page][8][64]
    x *= s["scales"][ids][:, :, :, None, :, None]
    x = x.permute(2, 0, 4, 1, 3, 5).reshape(2, ids.shape[0], N_KV, -1, DIM)[:, :, :, :longest]
    return x[0], x[1]


def _attend(score, seen, v):
    """softmax(score) v over the positions seen; a row that sees none gives zeros."""
    score = score.masked_fill(~seen, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = torch.exp(score - torch.where(top == -math.inf, torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    return torch.matmul(p, v) / torch.where(total > 0, total, torch.ones_like(total))


def _decode(s):
    n = s["ctx"].numel()
    k, v = _cached(s, s["longest"])
    q = s["q"].float().view(n, N_KV, GROUP, DIM)
    seen = (torch.arange(k.shape[2], device=k.device)[None, :] < s["ctx"][:, None])[:, None, None, :]
    v = torch.where(seen[:, 0, :, :, None], v, 0.0)
    score = torch.matmul(q, k.transpose(-1, -2)) * s["scale"]
    return _attend(score, seen, v).reshape(n, N_Q, DIM).to(torch.bfloat16)


def _prompt_attention(s):
    n, seq = s["ctx"].numel(), s["row_seq"]
    place = torch.arange(seq.numel(), device=seq.device) - s["cu"].long()[seq]
    long = s["longest_chunk"]
    q = torch.zeros(n, long, N_Q, DIM, device=seq.device)
    q[seq, place] = s["q"].float()
    q = q.view(n, long, N_KV, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(n, N_KV, long * GROUP, DIM)
    k, v = _cached(s, s["longest"])
    t = torch.arange(k.shape[2], device=k.device)
    at = s["ctx"][:, None] + torch.arange(long, device=k.device)[None, :]        # positions of the rows
    seen = (t[None, None, :] <= at[:, :, None]).repeat_interleave(GROUP, 1)[:, None]
    length = s["ctx"].long() + torch.diff(s["cu"].long())
    v = torch.where((t[None, :] < length[:, None])[:, None, :, None], v, 0.0)
    score = torch.matmul(q, k.transpose(-1, -2)).mul_(s["scale"])
    o = _attend(score, seen, v)
    o = o.view(n, N_KV, long, GROUP, DIM).permute(0, 2, 1, 3, 4).reshape(n, long, N_Q, DIM)
    return o[seq, place].to(torch.bfloat16)


# ------------------------------------------------------------------- exact
def _step_round(x, bits, low, high):
    """x to the nearest number of `bits` significant bits (ties to even); spacing no finer than at 2^low."""
    a = np.abs(x)
    e = np.maximum(np.frexp(a)[1] - 1, low)
    step = np.ldexp(1.0, e - (bits - 1))
    return np.sign(x) * np.minimum(np.rint(a / step) * step, high)


def _fits(top, limit):
    """Smallest exponent with top <= limit 2^e, from the definition."""
    e = E_MIN
    if top > 0:
        e = max(E_MIN, int(math.floor(math.log2(top / limit))) - 1)
        while top > math.ldexp(limit, e):
            e += 1
    return e


def _turned(x, pos):
    out = np.empty_like(x)
    for i in range(DIM // 2):
        f = 500000.0 ** (-i / 32.0)
        wave = 2.0 * math.pi / f
        if wave > 8192.0:
            f /= 32.0
        elif wave > 2048.0:
            t = (8192.0 / wave - 1.0) / 3.0
            f = (1.0 - t) * f / 32.0 + t * f
        c, n = np.cos(pos * f)[:, None], np.sin(pos * f)[:, None]
        out[..., i] = x[..., i] * c - x[..., i + 32] * n
        out[..., i + 32] = x[..., i + 32] * c + x[..., i] * n
    return out


def exact(case, seed):
    s = prepare(case, seed)
    ctx, chunk = _plan(case)
    page, layer, op = case["page"], case["layer"], case["op"]
    table = s["table"].cpu().numpy().copy()
    if op in ("decode", "prompt_attention"):
        outs = []
        at = 0
        for i, a in enumerate(ctx):
            rows, length = (1, a) if op == "decode" else (chunk[i], a + chunk[i])
            ids = torch.from_numpy(table[i, layer, :-(-length // page)].astype(np.int64)).cuda()
            x = s["pool"].view(torch.uint8)[ids].view(torch.float8_e4m3fn).double()
            x = x * s["scales"][ids].double()[:, :, None, :, None]
            kv = [x[:, j].reshape(-1, N_KV, DIM)[:length].transpose(0, 1) for j in (0, 1)]
            q = s["q"][at:at + rows].double()
            at += rows
            heads = []
            for h in range(N_KV):
                z = q[:, GROUP * h:GROUP * (h + 1)].reshape(-1, DIM) @ kv[0][h].T * s["scale"]
                if op == "prompt_attention":
                    sees = a + torch.arange(rows, device=z.device).repeat_interleave(GROUP)
                    z[torch.arange(length, device=z.device)[None, :] > sees[:, None]] = -math.inf
                heads.append((torch.softmax(z, -1) @ kv[1][h]).view(rows, GROUP, DIM))
            outs.append(torch.cat(heads, 1))
        return torch.cat(outs, 0)
    added = [1] * len(ctx) if op == "append" else chunk
    k, v, q = (s[x].double().cpu().numpy() for x in ("k", "v", "q"))
    pool = s["pool"].view(torch.uint8).cpu().view(torch.float8_e4m3fn).double().numpy()
    scales = s["scales"].double().cpu().numpy()
    free, count = s["free_list"].cpu().numpy(), int(s["free_count"])
    pos = np.concatenate([np.arange(a, a + b) for a, b in zip(ctx, added)])
    k8 = _step_round(_turned(k, pos), 8, -126, math.inf)
    at = 0
    for i, (a, b) in enumerate(zip(ctx, added)):
        t = a
        while t < a + b:
            end = min(a + b, (t // page + 1) * page)
            first = t % page
            if first == 0:
                count -= 1
                table[i, layer, t // page] = free[count]
            blk = table[i, layer, t // page]
            rows = slice(at + t - a, at + end - a)
            for h in range(N_KV):
                for j, (raw, x, limit) in enumerate(((k, k8, TOP_K), (v, v, TOP_V))):
                    e = _fits(np.abs(raw[rows, h]).max(), limit)
                    if first:
                        old = scales[blk, j, h]
                        e = max(e, int(math.log2(old)))
                        moved = pool[blk, j, :first, h] * (old / 2.0 ** e)
                        pool[blk, j, :first, h] = _step_round(moved, 4, -6, 448.0)
                    scales[blk, j, h] = 2.0 ** e
                    pool[blk, j, first:first + end - t, h] = _step_round(x[rows, h] / 2.0 ** e, 4, -6, 448.0)
            t = end
        at += b
    f64 = torch.from_numpy
    return {"pool": f64(pool), "scales": f64(scales), "table": None, "count": None, "q": f64(_turned(q, pos))}
