"""Measured cases of the operators around the products and the 4-bit cache in a decoder layer.

Four operators: the root-mean-square norm with the residual's addition (`wq_rms_norm`), rotary positions with one or
several axes (`wq_rotary`), low-rank adapters of many requests beside a shared projection (`wq_lora`), and the page
tables, lengths and row maps of the paged cache, built on the GPU (`wq_kv_resize`).

Norm: h = x + r, y = w h / sqrt(mean h^2 + eps).  Rotary: pair i of a head turns by p f_i, p the row's position on the
pair's axis.  Adapters: out = y + scale_a (x A_a^T) B_a^T with a the adapter of the row's sequence, slice s of the
columns from its own rows A_a[s]; only the first rank_a rows of A_a[s] and columns of B_a count.  Pages: a sequence
whose length changes from len to want holds ceil(want / P) pages; pages in the order (sequence, index), the f-th page
taken is the f-th one given back, and beyond those stack[c + back - 1 - f], where the f-th page given back beyond the
taken ones goes too (c: pages on the stack before, back: given back).
"""
import math
import random

import torch

own = False

_DT = {"f16": torch.float16, "bf16": torch.bfloat16}


# ----------------------------------------------------------------------------
# Cases
# ----------------------------------------------------------------------------
def _case(name, op, **more):
    d = dict(op=op, **more)
    if name:
        d["name"] = name
    return d


def _norm(name, dtype, rows, dim, residual, heads=0, eps=1e-5):
    """heads > 0: `heads` heads of a fused projection's rows, each normalised over its `dim` channels."""
    return _case(name, "norm", dtype=dtype, rows=rows, dim=dim, residual=residual, heads=heads, eps=eps)


def _rotary(name, dtype, batch, q_len, far, q_heads, kv_heads, head_dim, rotary_dim, axes=1, adjacent=False,
            ragged=False, base=10000.0):
    """q_len: rows of the longest sequence; far: length of the longest one, these rows included."""
    return _case(name, "rotary", dtype=dtype, batch=batch, q_len=q_len, far=far, q_heads=q_heads, kv_heads=kv_heads,
                 head_dim=head_dim, rotary_dim=rotary_dim, axes=axes, adjacent=adjacent, ragged=ragged, base=base)


def _lora(name, dtype, batch, q_len, K, widths, rank, adapters, mixed=False, ragged=False):
    """widths: columns of each slice, comma separated; mixed: ranks differ from adapter to adapter."""
    return _case(name, "lora", dtype=dtype, batch=batch, q_len=q_len, K=K, widths=widths, rank=rank, adapters=adapters,
                 mixed=mixed, ragged=ragged)


def _pages(name, batch, page, max_len, grow, turnover):
    """Each running sequence grows by up to `grow` tokens and is cut back again; turnover: instead, one half of the
    sequences ends while the other half's prompts come in, and the other way round."""
    return _case(name, "pages", batch=batch, page=page, max_len=max_len, grow=grow, turnover=turnover)


def listed():
    return [
        # one token's row before a product, the last block's output added (4096 wide)
        _norm("norm_token", "f16", 1, 4096, True),
        # a long prompt's rows (8192 wide)
        _norm("norm_prompt", "bf16", 4099, 8192, True),
        # the query heads of a chunk, normalised head by head in the fused projection's output
        _norm("norm_heads", "f16", 2001, 128, False, heads=32, eps=1e-6),
        # one new token of each of 64 sequences of long contexts
        _rotary("rotary_tokens", "bf16", 64, 1, 131071, 64, 8, 128, 128, base=500000.0),
        # ragged prompts of a model that turns a part of each head, neighbouring channels
        _rotary("rotary_prompts", "bf16", 5, 901, 901, 16, 4, 256, 64, adjacent=True, ragged=True),
        # a video's rows: time, height and width (4096 wide)
        _rotary("rotary_video", "f16", 1, 7001, 9000, 32, 8, 128, 128, axes=3, base=1000000.0),
        # a single chat with its own adapter
        _lora("lora_token", "f16", 1, 1, 4096, "4096", 16, 8),
        # a decode batch of many adapters of several ranks beside fused QKV (8192 wide, 8 kv heads)
        _lora("lora_tokens", "bf16", 64, 1, 8192, "8192,1024,1024", 32, 40, mixed=True),
        # a decode batch of few adapters beside the down projection
        _lora("lora_down", "bf16", 16, 1, 11008, "4096", 8, 3),
        # ragged prompts of one prefill batch beside fused QKV (4096 wide)
        _lora("lora_prompts", "f16", 6, 1499, 4096, "4096,4096,4096", 64, 4, ragged=True),
        # a step of 64 sequences with a few guessed tokens, cut back to those that held
        _pages("pages_step", 64, 16, 8000, 5, False),
        # prompts come in while other sequences end
        _pages("pages_turnover", 300, 16, 5003, 0, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rotary", "rotary", "lora", "lora", "pages"])
    dtype = rng.choice(["f16", "bf16"])
    if op == "norm":
        eps = rng.choice([1e-5, 1e-6])
        if rng.random() < 0.4:
            return _norm(None, dtype, _log(rng, 1, 3000), 8 * rng.choice([8, 8, 10, 12, 16, 16, 24, 32]), False,
                         heads=rng.choice([1, 4, 8, 32, 40]), eps=eps)
        dim = 8 * _log(rng, 8, 2048)
        return _norm(None, dtype, max(1, _log(rng, 1, 4000) * 4096 // max(4096, dim)), dim, rng.random() < 0.6, eps=eps)
    if op == "rotary":
        head_dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rotary_dim = rng.choice([head_dim, head_dim, 32, 64])
        axes = rng.choice([1, 1, 2, 3, 4])
        kv_heads = rng.choice([1, 2, 4, 8, 8, 16])
        q_heads = kv_heads * rng.choice([1, 4, 5, 8])
        if rng.random() < 0.5:
            batch, q_len = _log(rng, 1, 300), 1
        else:
            batch = rng.randint(1, 8)
            q_len = _log(rng, 2, min(5000, 50000000 // ((q_heads + kv_heads) * head_dim * batch)))
        return _rotary(None, dtype, batch, q_len, q_len + _log(rng, 1, 130000), q_heads, kv_heads, head_dim, rotary_dim,
                       axes, rng.random() < 0.4, rng.random() < 0.5, rng.choice([10000.0, 500000.0, 1000000.0]))
    if op == "lora":
        K = 128 * rng.randint(4, 86)
        widths = [16 * _log(rng, 16, 512)]
        if rng.random() < 0.5:
            widths += [16 * _log(rng, 4, 128)] * 2
        if rng.random() < 0.6:
            batch, q_len = _log(rng, 1, 150), 1
        else:
            batch, q_len = rng.randint(1, 8), _log(rng, 2, 500)
        return _lora(None, dtype, batch, q_len, K, ",".join(str(w) for w in widths),
                     rng.choice([8, 16, 16, 24, 32, 64, 128]), rng.randint(1, 30), rng.random() < 0.5,
                     rng.random() < 0.5)
    page = rng.choice([16, 16, 32, 64, 256])
    batch = _log(rng, 1, 400)
    max_len = _log(rng, 2, 1000000 // batch)
    return _pages(None, batch, page, min(max_len, 60000), rng.randint(1, 9), rng.random() < 0.4)


def _plan(case):
    """What a program knows on the host: the sizes that differ from sequence to sequence (from the case alone)."""
    c = {k: case[k] for k in sorted(case) if k != "name"}
    rng = random.Random(repr(c))
    if case["op"] == "pages":
        rest, other = [], []
        for b in range(case["batch"]):
            n = case["max_len"] if b == 0 else rng.randint(1, case["max_len"])
            if case["turnover"]:
                rest.append(n if b % 2 else 0)
                other.append(0 if b % 2 else n)
            else:
                rest.append(n)
                other.append(n + rng.randint(0 if b else 1, case["grow"]))
        return rest, other
    new = [case["q_len"] if b == 0 or not case["ragged"] else rng.randint(1, case["q_len"])
           for b in range(case["batch"])]
    if case["op"] == "rotary":
        return new, [case["far"] if b == 0 else rng.randint(new[b], case["far"]) for b in range(case["batch"])]
    n = case["adapters"]
    # every sixth sequence or so has no adapter, the first one has
    ids = [0 if b == 0 else rng.randint(0, n - 1) if rng.random() < 0.85 else -1 for b in range(case["batch"])]
    sizes = [8, 16, 32, 64, 128]
    ranks = [case["rank"] if a == 0 or not case["mixed"]
             else rng.choice([r for r in sizes + [case["rank"]] if r <= case["rank"]]) for a in range(n)]
    return new, ids, ranks


def _widths(case):
    return [int(w) for w in case["widths"].split(",")]


def work(case):
    if case["op"] == "norm":
        n = case["rows"] * max(1, case["heads"]) * case["dim"]
        return {"bytes": 2 * n * (4 if case["residual"] else 2) + 2 * case["dim"],
                "flops": n * (5 if case["residual"] else 4)}
    if case["op"] == "rotary":
        T = sum(_plan(case)[0])
        heads = case["q_heads"] + case["kv_heads"]
        positions = 4 * T * case["axes"] if case["axes"] > 1 else 4 * case["batch"]
        return {"bytes": 4 * T * heads * case["head_dim"] + positions, "flops": 3 * T * heads * case["rotary_dim"]}
    if case["op"] == "lora":
        new, ids, ranks = _plan(case)
        K, w = case["K"], _widths(case)
        n, S = sum(w), len(w)
        T = sum(new)
        with_one = sum(q for q, a in zip(new, ids) if a >= 0)
        bytes_ = 2 * with_one * K + 4 * T * n + sum(2 * ranks[a] * (S * K + n) for a in set(ids) if a >= 0)
        return {"bytes": bytes_, "flops": sum(2 * q * ranks[a] * (S * K + n) for q, a in zip(new, ids) if a >= 0)}
    rest, other = _plan(case)
    P = case["page"]
    moved = sum(abs(-(-a // P) + (b // -P)) for a, b in zip(rest, other))
    rows = sum(abs(a - b) for a, b in zip(rest, other))
    # both changes of a pass: lengths read and written, wanted lengths, offsets; pages from one place to another;
    # position and slot of every new row
    return {"bytes": 2 * 16 * case["batch"] + 2 * 8 * moved + 12 * rows, "flops": 8 * case["batch"] + 4 * rows}


# ----------------------------------------------------------------------------
# Inputs
# ----------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(1 + 7919 * seed)
    return {"norm": _prepare_norm, "rotary": _prepare_rotary, "lora": _prepare_lora,
            "pages": _prepare_pages}[case["op"]](case, g)


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _offsets(new):
    cu = [0]
    for q in new:
        cu.append(cu[-1] + q)
    return cu


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _prepare_norm(case, g):
    dt, rows, dim = _DT[case["dtype"]], case["rows"], case["dim"]
    st = dict(case=case, dt=dt, residual=None)
    st["weight"] = (1 + 0.2 * _randn(g, dim)).to(dt)
    if case["heads"]:
        # queries within a fused projection's rows (keys and values behind them)
        st["x"] = _randn(g, rows, case["heads"] + 2, dim).mul(2).to(dt)[:, :case["heads"]]
        return st
    # a residual stream: a few channels far larger than the rest
    big = 1 + 30 * (torch.rand((dim,), generator=g, device="cuda") < 0.01)
    st["x"] = (_randn(g, rows, dim) * big).to(dt)
    if case["residual"]:
        st["residual"] = (3 * _randn(g, rows, dim) * big).to(dt)
    return st


def _axis_of_pairs(case):
    """Contiguous sections of the pairs, the first axis with what is left over."""
    half, axes = case["rotary_dim"] // 2, case["axes"]
    each = half // axes
    return [0] * (half - each * (axes - 1)) + [a for a in range(1, axes) for _ in range(each)]


def _frequencies(case):
    R = case["rotary_dim"]
    return [case["base"] ** (-2.0 * i / R) for i in range(R // 2)]


def _prepare_rotary(case, g):
    dt, Hq, Hk, D = _DT[case["dtype"]], case["q_heads"], case["kv_heads"], case["head_dim"]
    new, total = _plan(case)
    cu = _offsets(new)
    T = cu[-1]
    st = dict(case=case, dt=dt, T=T, new=new, total=total, lens=_i32(total), positions=None,
              cu=_i32(cu) if case["ragged"] else None)
    # one projection gave queries, keys and values
    qkv = _randn(g, T, Hq + 2 * Hk, D).mul(2).to(dt)
    st["q"], st["k"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hk]
    if case["axes"] > 1:
        # a grid in time, height and width; further axes count on
        last = _i32([n for n, q in zip(total, new) for _ in range(q)])
        t = torch.arange(T, device="cuda", dtype=torch.int32)
        grid = [last - 1 - (t % 977) // 64, (t // 13) % 64, t % 53, (7 * t) % 4099]
        st["positions"] = torch.stack(grid[:case["axes"]]).to(torch.int32).contiguous()
    st["axis"] = torch.tensor(_axis_of_pairs(case), device="cuda")
    st["freq"] = torch.tensor(_frequencies(case), dtype=torch.float64, device="cuda")
    if own:
        import weight_only_quantized_w4a16_amd as wq
        st["plan"] = wq.wq_rotary_plan(D, case["rotary_dim"], base=case["base"],
                                       axes=_axis_of_pairs(case) if case["axes"] > 1 else None,
                                       adjacent=case["adjacent"], device="cuda")
    return st


def _prepare_lora(case, g):
    dt, K, w, r, n = _DT[case["dtype"]], case["K"], _widths(case), case["rank"], case["adapters"]
    new, ids, ranks = _plan(case)
    cu = _offsets(new)
    T, S, N = cu[-1], len(w), sum(w)
    st = dict(case=case, dt=dt, T=T, cu_host=cu, ids=ids, ranks=ranks, cu=_i32(cu) if case["ragged"] else None)
    st["x"] = _randn(g, T, K).to(dt)
    st["y"] = _randn(g, T, N).mul(2).to(dt)
    st["a"] = torch.stack([(_randn(g, S, r, K) / math.sqrt(K)).to(dt) for _ in range(n)])
    st["b"] = torch.stack([(_randn(g, N, r) * 0.3).to(dt) for _ in range(n)])
    st["scales"] = torch.tensor([16.0 / k for k in ranks], device="cuda")
    st["out"] = torch.empty_like(st["y"])
    if own:
        import weight_only_quantized_w4a16_amd as wq
        st["bank"] = wq.LoraBank(st["a"], st["b"], st["scales"], _i32(ranks) if case["mixed"] else None,
                                 tuple(w) if S > 1 else None)
        st["adapters"] = _i32(ids)
    return st


def _prepare_pages(case, g):
    rest, other = _plan(case)
    P = case["page"]
    used = [-(-n // P) for n in rest]
    most = [-(-max(a, b) // P) for a, b in zip(rest, other)]
    num_pages = sum(most) + 7
    width = max(most) + 1
    order = torch.randperm(num_pages, generator=g, device="cuda").to(torch.int32)
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    # pages on the stack, the next one to be taken last; behind them whatever was there
    free = torch.cat([order[at:], order[:at]])
    st = dict(case=case, want=(_i32(other), _i32(rest)), num_pages=num_pages,
              rows=tuple(sum(max(0, q - p) for p, q in zip(x, y)) for x, y in ((rest, other), (other, rest))),
              table=table, lens=_i32(rest), free=free, counts=_i32([num_pages - at, 0]))
    if own:
        import weight_only_quantized_w4a16_amd as wq
        st["pages"] = wq.KVPages(table, st["lens"], free, st["counts"], num_pages, P)
    return st


# ----------------------------------------------------------------------------
# One pass
# ----------------------------------------------------------------------------
def run(state):
    return {"norm": _run_norm, "rotary": _run_rotary, "lora": _run_lora, "pages": _run_pages}[state["case"]["op"]](state)


def _run_norm(st):
    eps = st["case"]["eps"]
    if own:
        import weight_only_quantized_w4a16_amd as wq
        return wq.wq_rms_norm(st["x"], st["weight"], eps, residual=st["residual"])
    h = st["x"].float()
    if st["residual"] is not None:
        h = h + st["residual"].float()
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + eps) * st["weight"].float()
    return y.to(st["dt"]) if st["residual"] is None else (y.to(st["dt"]), h.to(st["dt"]))


def _row_positions(st):
    """[axes][T] (from the lengths where the program gives none: a sequence's rows are its last ones)."""
    if st["positions"] is not None:
        return st["positions"]
    c = st["case"]
    if st["cu"] is None:
        n = c["q_len"]
        p = st["lens"][:, None] - n + torch.arange(n, device="cuda")
        return p.reshape(1, -1)
    t = torch.arange(st["T"], device="cuda")
    seq = torch.searchsorted(st["cu"][1:].long(), t, right=True)
    return (st["lens"].long()[seq] - st["cu"].long()[seq + 1] + t)[None]


def _run_rotary(st):
    c = st["case"]
    if own:
        import weight_only_quantized_w4a16_amd as wq
        if st["positions"] is not None:
            return wq.wq_rotary(st["q"], st["k"], st["plan"], positions=st["positions"])
        return wq.wq_rotary(st["q"], st["k"], st["plan"], kv_lens=st["lens"], cu_q=st["cu"])
    R = c["rotary_dim"]
    p = _row_positions(st).double()[st["axis"]]           # [R / 2][T]
    angle = (p * st["freq"][:, None]).t()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    out = []
    for x in (st["q"], st["k"]):
        v = x.float()
        if c["adjacent"]:
            a, b = v[..., 0:R:2], v[..., 1:R:2]
            turned = torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
        else:
            a, b = v[..., :R // 2], v[..., R // 2:R]
            turned = torch.cat([a * cos - b * sin, a * sin + b * cos], -1)
        out.append(torch.cat([turned, v[..., R:]], -1).to(st["dt"]))
    return tuple(out)


def _run_lora(st):
    if own:
        import weight_only_quantized_w4a16_amd as wq
        return wq.wq_lora(st["x"], st["bank"], st["adapters"], st["y"], cu_q=st["cu"], out=st["out"])
    c = st["case"]
    out = st["out"]
    out.copy_(st["y"])
    cu, w = st["cu_host"], _widths(c)
    for a in sorted(set(st["ids"])):
        if a < 0:
            continue
        spans = [(cu[b], cu[b + 1]) for b, i in enumerate(st["ids"]) if i == a]
        rows = torch.cat([torch.arange(p, q, device="cuda") for p, q in spans])
        x, r, at = st["x"][rows].float(), st["ranks"][a], 0
        parts = []
        for s, n in enumerate(w):
            v = x @ st["a"][a, s, :r].float().t()
            parts.append(v @ st["b"][a, at:at + n, :r].float().t())
            at += n
        out[rows] = (st["y"][rows].float() + st["scales"][a] * torch.cat(parts, 1)).to(st["dt"])
    return out


def _run_pages(st):
    results = []
    for want, rows in zip(st["want"], st["rows"]):
        if own:
            import weight_only_quantized_w4a16_amd as wq
            results += wq.wq_kv_resize(st["pages"], want, rows)
        else:
            results += _resize(st, want, rows)
    return results + [st["table"], st["lens"], st["free"], st["counts"]]


def _resize(st, want, rows):
    P, table, free, counts = st["case"]["page"], st["table"], st["free"], st["counts"]
    B, width = table.shape
    old = st["lens"].clone()
    have, need = (old + P - 1) // P, (want + P - 1) // P
    i = torch.arange(width, device="cuda")
    back = ((i >= need[:, None]) & (i < have[:, None])).flatten().nonzero().flatten()
    take = ((i >= have[:, None]) & (i < need[:, None])).flatten().nonzero().flatten()
    flat = table.view(-1)
    c = counts[0].long()
    given = flat[back].clone()
    flat[back] = -1
    n, m = back.numel(), take.numel()
    both = min(n, m)
    flat[take[:both]] = given[:both]
    f = torch.arange(both, max(n, m), device="cuda")
    if n > m:
        free[c + n - 1 - f] = given[both:]
    else:
        flat[take[both:]] = free[c + n - 1 - f]
    counts[0] += n - m
    counts[1] = 0
    st["lens"].copy_(want)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = (want - old).clamp(min=0).cumsum(0)
    t = torch.arange(rows, device="cuda")
    seq = torch.searchsorted(cu[1:].long(), t, right=True)
    pos = want.long()[seq] - cu.long()[seq + 1] + t
    slots = table[seq, pos // P].long() * P + pos % P
    return cu, pos.to(torch.int32), slots


# ----------------------------------------------------------------------------
# The definition in 64 bits, written apart from the plain forms
# ----------------------------------------------------------------------------
def exact(case, seed):
    global own
    before, own = own, False  # inputs only: nothing of the repository's own code
    try:
        st = prepare(case, seed)
    finally:
        own = before
    return {"norm": _exact_norm, "rotary": _exact_rotary, "lora": _exact_lora, "pages": _exact_pages}[case["op"]](st)


def _exact_norm(st):
    h = st["x"].double()
    if st["residual"] is not None:
        h = h + st["residual"].double()
    size = torch.sqrt(h.pow(2).sum(-1) / h.shape[-1] + st["case"]["eps"])
    y = (st["weight"].double() * (h / size.unsqueeze(-1))).cpu()
    return y if st["residual"] is None else (y, h.cpu())


def _exact_rotary(st):
    """A pair as a complex number, times e^(i angle)."""
    c = st["case"]
    R = c["rotary_dim"]
    at = []
    for q, n in zip(st["new"], st["total"]):
        at += range(n - q, n)
    one = torch.tensor(at, dtype=torch.float64, device="cuda")
    where = [one if st["positions"] is None else st["positions"][a].double() for a in range(c["axes"])]
    out = []
    for x in (st["q"], st["k"]):
        v = x.double()
        for i, (a, f) in enumerate(zip(_axis_of_pairs(c), _frequencies(c))):
            first, second = (2 * i, 2 * i + 1) if c["adjacent"] else (i, i + R // 2)
            turn = torch.polar(torch.ones_like(where[a]), where[a] * f)
            z = torch.complex(v[:, :, first].contiguous(), v[:, :, second].contiguous()) * turn[:, None]
            v[:, :, first], v[:, :, second] = z.real, z.imag
        out.append(v.cpu())
    return tuple(out)


def _exact_lora(st):
    c = st["case"]
    out = st["y"].double()
    ends = _offsets(_widths(c))
    for b, a in enumerate(st["ids"]):
        if a < 0:
            continue
        r, p, q = st["ranks"][a], st["cu_host"][b], st["cu_host"][b + 1]
        B = st["b"][a].double()[:, :r] * float(st["scales"][a].double())
        for s in range(len(ends) - 1):
            v = torch.matmul(st["x"][p:q].double(), st["a"][a][s].double()[:r].t().contiguous())
            out[p:q, ends[s]:ends[s + 1]] += torch.matmul(v, B[ends[s]:ends[s + 1]].t().contiguous())
    return out.cpu()


def _exact_pages(st):
    """Page by page on the host."""
    P = st["case"]["page"]
    table, lens, free = st["table"].tolist(), st["lens"].tolist(), st["free"].tolist()
    count = st["counts"].tolist()[0]
    results = []
    for want, rows in zip(st["want"], st["rows"]):
        want = want.tolist()
        given, places = [], []
        for b, (n, m) in enumerate(zip(lens, want)):
            for i in range(len(table[b])):
                held, wanted = i * P < n, i * P < m
                if held and not wanted:
                    given.append(table[b][i])
                    table[b][i] = -1
                elif wanted and not held:
                    places.append((b, i))
        top = count + len(given)
        for f in range(max(len(given), len(places))):
            page = given[f] if f < len(given) else free[top - 1 - f]
            if f < len(places):
                table[places[f][0]][places[f][1]] = page
            else:
                free[top - 1 - f] = page
        count = top - len(places)
        cu, positions, slots = [0], [], []
        for b, (n, m) in enumerate(zip(lens, want)):
            for p in range(n, m):
                positions.append(p)
                slots.append(table[b][p // P] * P + p % P)
            cu.append(len(positions))
        assert len(positions) == rows
        lens = want
        results += [torch.tensor(cu, dtype=torch.int32), torch.tensor(positions, dtype=torch.int32),
                    torch.tensor(slots, dtype=torch.int64)]
    return results + [torch.tensor(table, dtype=torch.int32), torch.tensor(lens, dtype=torch.int32),
                      torch.tensor(free, dtype=torch.int32), torch.tensor([count, 0], dtype=torch.int32)]
