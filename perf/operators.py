"""Cases that measure the operators between a decoder layer's quantised products.

norm   residual + gated, scaled block output, normed before and after, and
       quantised into the next product's operand
write  rotary positions on queries and keys, keys and values quantised into the
       pages of the cache
trip   the same write followed by the read of the same slots (a prefix that is
       attended to in bf16)
read   slots of the cache read back as bf16
attend attention of drafted token trees (a single token is a tree of one) over
       the quantised cache

`run` computes the plain form with elementary torch operations where `own` is
false, and makes the package's calls where it is true.
"""
import math

import torch

own = False
DEV = "cuda"


def listed():
    return [
        # a single sequence's decode step between two layers of hidden size 5120: latency alone
        dict(name="norm-1x5120-fp8", op="norm", fmt="fp8", rows=1, width=5120, kind="rms", post=False, gate="none"),
        # a decode batch, post-normed block output with a channel gate, block scales
        dict(name="norm-33x7168-block", op="norm", fmt="block", rows=33, width=7168, kind="rms", post=True, gate="row"),
        # a mid-size batch with LayerNorm and a gate per element, int8
        dict(name="norm-517x4096-int8", op="norm", fmt="int8", rows=517, width=4096, kind="layer", post=False, gate="full"),
        # a long prefill: the bandwidth of the path
        dict(name="norm-16384x5120-fp8", op="norm", fmt="fp8", rows=16384, width=5120, kind="rms", post=True, gate="none"),
        # a decode batch's new keys and values, whole head rotated by halves
        dict(name="write-32-fp8", op="write", fmt="fp8", tokens=32, q_heads=40, kv_heads=8, dim=128, rope=128,
             pairs=False, page=64, far=131072),
        # a prefill chunk, a quarter of the head rotated in neighbouring pairs, read back
        dict(name="trip-8191-int8", op="trip", fmt="int8", tokens=8191, q_heads=32, kv_heads=8, dim=128, rope=32,
             pairs=True, page=16, far=1000000),
        # a long prefix read back
        dict(name="read-100000-fp8", op="read", fmt="fp8", tokens=100000, kv_heads=8, dim=128, page=64),
        # one user's token over a short context: latency
        dict(name="attend-1-fp8", op="attend", fmt="fp8", batch=1, draft=1, tree=False, longest=1000, q_heads=40,
             kv_heads=8, dim=128, page=64),
        # a serving batch's decode step, ragged contexts
        dict(name="attend-64-fp8", op="attend", fmt="fp8", batch=64, draft=1, tree=False, longest=16384, q_heads=64,
             kv_heads=8, dim=128, page=64),
        # one long context, single token: the split over the long axis
        dict(name="attend-long-int8", op="attend", fmt="int8", batch=1, draft=1, tree=False, longest=131072, q_heads=32,
             kv_heads=8, dim=128, page=128),
        # trees of up to 64 drafted tokens over medium contexts
        dict(name="attend-tree-fp8", op="attend", fmt="fp8", batch=8, draft=64, tree=True, longest=8192, q_heads=64,
             kv_heads=8, dim=128, page=64),
        # small trees, narrow heads, small pages
        dict(name="attend-tree-d64-int8", op="attend", fmt="int8", batch=13, draft=7, tree=True, longest=5000,
             q_heads=15, kv_heads=5, dim=64, page=16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "write", "trip", "read", "attend", "attend", "attend"])
    if op == "norm":
        fmt = rng.choice(["fp8", "block", "int8", "bf16"])
        step = {"fp8": 16, "int8": 16, "block": 128, "bf16": 8}[fmt]
        width = max(1, _log_int(rng, 256, 16384) // step) * step
        return dict(op=op, fmt=fmt, rows=min(_log_int(rng, 1, 16384), 16384 * 5120 // width), width=width,
                    kind=rng.choice(["rms", "rms", "layer"]), post=rng.random() < 0.5,
                    gate=rng.choice(["none", "row", "full"]))
    dim = rng.choice([64, 128])
    fmt = rng.choice(["fp8", "int8"])
    page = rng.choice([16, 32, 64, 128])
    kv_heads = rng.choice([1, 2, 4, 5, 8])
    q_heads = kv_heads * rng.choice([1, 3, 4, 5, 7, 8])
    if op in ("write", "trip"):
        return dict(op=op, fmt="fp8" if op == "write" else fmt, tokens=_log_int(rng, 1, 8192), q_heads=q_heads,
                    kv_heads=kv_heads, dim=dim, rope=rng.choice([0, 16, 32, dim // 2, dim]), pairs=rng.random() < 0.5,
                    page=page, far=_log_int(rng, 10000, 1000000))
    if op == "read":
        return dict(op=op, fmt=fmt, tokens=_log_int(rng, 1, 100000), kv_heads=kv_heads, dim=dim, page=page)
    tree = rng.random() < 0.6
    draft = _log_int(rng, 2, 128) if tree else 1
    batch = _log_int(rng, 1, 64)
    longest = _log_int(rng, 300, 32768)
    # no more than the largest listed case reads or multiplies
    longest = max(200, min(longest, 64 * 16384 * 8 // (batch * kv_heads), 8 * 8192 * 64 * 64 // (batch * draft * q_heads)))
    return dict(op=op, fmt=fmt, batch=batch, draft=draft, tree=tree, longest=longest, q_heads=q_heads,
                kv_heads=kv_heads, dim=dim, page=page)


# ------------------------------------------------------------- sizes and work --
def _spread(n, lo, hi):
    """n whole numbers between lo and hi, spread evenly without a period; the last is hi."""
    v = [lo + int(((i + 1) * 0.6180339887498949 % 1.0) * (hi - lo + 1)) for i in range(n)]
    v[-1] = hi
    return v


def _lengths(case):
    """(cached positions, query tokens) of each sequence: the sizes of a case do not depend on the seed."""
    n = _spread(case["batch"], max(1, case["draft"] // 2), case["draft"])
    return [max(a, b) for a, b in zip(_spread(case["batch"], max(1, case["longest"] // 4), case["longest"]), n)], n


def work(case):
    op = case["op"]
    if op == "norm":
        m, n = case["rows"], case["width"]
        b = 2 * m * n * 2                                   # residual and block output
        b += {"none": 0, "row": 2 * n, "full": 2 * m * n}[case["gate"]]
        vectors = (1 + case["post"]) * (2 if case["kind"] == "layer" else 1)
        b += 2 * n * vectors + 2 * m * n                    # weights; the new residual
        b += {"bf16": 2 * m * n, "block": m * n + 4 * m * (n // 128)}.get(case["fmt"], m * n + 4 * m)
        return {"bytes": b, "flops": 12 * m * n}
    row = case["kv_heads"] * case["dim"]
    if op in ("write", "trip"):
        t, q = case["tokens"], case["q_heads"] * case["dim"]
        codes = t * (2 * row + 8 * case["kv_heads"])
        b = t * (2 * q * 2 + 2 * row * 2) + codes + 8 * t + 8 * (case["rope"] // 2)
        if op == "trip":
            b += codes + t * 2 * row * 2
        return {"bytes": b, "flops": t * (6 * (q + row) + 4 * row)}
    if op == "read":
        return {"bytes": case["tokens"] * (2 * row + 8 * case["kv_heads"] + 4 * row + 4), "flops": 2 * case["tokens"] * row}
    length, n = _lengths(case)
    q = case["q_heads"] * case["dim"]
    b = sum(length) * (2 * row + 8 * case["kv_heads"]) + sum(n) * (4 * q + 4 * case["q_heads"])
    return {"bytes": b, "flops": sum(4 * a * c for a, c in zip(length, n)) * q}


# --------------------------------------------------------- plain quantisation --
def _top(fmt):
    return 127.0 if fmt == "int8" else 448.0


def _quantised(y, fmt, group=None):
    """Codes (numbers, in y's type) and scale of y's rows, or of each row's groups: scale = amax / top, 1 for a zero row."""
    shape = y.shape
    if group is not None:
        y = y.reshape(*shape[:-1], shape[-1] // group, group)
    amax = y.abs().amax(-1, keepdim=True)
    scale = torch.where(amax > 0, amax.float() / _top(fmt), torch.ones_like(amax, dtype=torch.float32))
    code = y / scale
    code = code.round().clamp(-127, 127) if fmt == "int8" else code.clamp(-448, 448).to(torch.float8_e4m3fn).to(y.dtype)
    return code.reshape(shape), scale.squeeze(-1)


def _bytes_of(code, fmt):
    return code.to(torch.int8).view(torch.uint8) if fmt == "int8" else code.to(torch.float8_e4m3fn).view(torch.uint8)


def _values_of(codes, fmt, dtype=torch.float32):
    return codes.view(torch.int8).to(dtype) if fmt == "int8" else codes.view(torch.float8_e4m3fn).to(dtype)


# -------------------------------------------------------------------- prepare --
def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _activations(g, rows, width):
    """bf16 rows with a few strong channels, as a residual stream has them."""
    x = torch.randn(rows, width, generator=g, device=DEV)
    strong = torch.randint(0, width, (max(1, width // 512),), generator=g, device=DEV)
    x[:, strong] *= 12.0
    return x.to(torch.bfloat16)


def _empty_pool(case, pages):
    shape = (pages, case["kv_heads"], case["page"])
    return {"k": torch.zeros(*shape, case["dim"], dtype=torch.uint8, device=DEV),
            "v": torch.zeros(*shape, case["dim"], dtype=torch.uint8, device=DEV),
            "k_scale": torch.zeros(*shape, device=DEV), "v_scale": torch.zeros(*shape, device=DEV)}


def _filled_pool(case, pages, g):
    pool = _empty_pool(case, pages)
    for part in ("k", "v"):
        bias = torch.randn(case["kv_heads"], 1, case["dim"], generator=g, device=DEV)
        bias[..., ::16] *= 3.0 if part == "k" else 1.0
        for at in range(0, pages, 4096):
            n = min(4096, pages - at)
            x = torch.randn(n, case["kv_heads"], case["page"], case["dim"], generator=g, device=DEV) + 0.5 * bias
            code, scale = _quantised(x, case["fmt"])
            pool[part][at:at + n] = _bytes_of(code, case["fmt"])
            pool[part + "_scale"][at:at + n] = scale
    return pool


def _ancestors(n, limit, g):
    """[B, limit, limit] truth values: which drafted tokens each drafted token sees in a random tree, itself among them."""
    batch = len(n)
    parent = (torch.rand(batch, limit, generator=g, device=DEV) * torch.arange(limit, device=DEV)).long()
    see = torch.zeros(batch, limit, limit, dtype=torch.bool, device=DEV)
    each = torch.arange(batch, device=DEV)
    for j in range(limit):
        if j:
            see[:, j] = see[each, parent[:, j]]
        see[:, j, j] = True
    return see


def _words(see):
    """Truth values [..., n] as 64-bit words [..., ceil(n / 64)], bit j % 64 of word j // 64."""
    n = see.shape[-1]
    words = -(-n // 64)
    see = torch.nn.functional.pad(see, (0, words * 64 - n)).reshape(*see.shape[:-1], words, 64)
    return (see.long() << torch.arange(64, device=see.device)).sum(-1)


def _package_cache(case, pool):
    import precision_quantized_gemm_b200 as qg
    return qg.Cache(qg.QG_W8A8_INT8 if case["fmt"] == "int8" else qg.QG_FP8_DYNAMIC, k=pool["k"], v=pool["v"],
                    k_scale=pool["k_scale"], v_scale=pool["v_scale"])


def prepare(case, seed):
    g, op = _generator(seed), case["op"]
    s = {"case": case}
    if op == "norm":
        m, n = case["rows"], case["width"]
        s["residual"], s["x"] = _activations(g, m, n), _activations(g, m, n)
        rows = {"none": 0, "row": 1, "full": m}[case["gate"]]
        s["gate"] = (1 + 0.3 * torch.randn(rows, n, generator=g, device=DEV)).to(torch.bfloat16) if rows else None
        s["gate"] = s["gate"][0] if case["gate"] == "row" else s["gate"]
        for name, kept in (("weight", True), ("bias", case["kind"] == "layer"), ("post_weight", case["post"]),
                           ("post_bias", case["post"] and case["kind"] == "layer")):
            v = torch.randn(n, generator=g, device=DEV) * 0.2 + (0.0 if "bias" in name else 1.0)
            s[name] = v.to(torch.bfloat16) if kept else None
        return s
    if op in ("write", "trip"):
        t, d = case["tokens"], case["dim"]
        heads = case["q_heads"] + 2 * case["kv_heads"]
        # one fused projection's output: queries, keys and values of a token side by side
        s["qkv"] = _activations(g, t, heads * d).view(t, heads, d)
        pages = -(-t // case["page"]) + 3
        s["pool"] = _empty_pool(case, pages)
        s["slots"] = torch.randperm(pages * case["page"], generator=g, device=DEV)[:t].int()
        s["positions"] = torch.randint(0, case["far"], (t,), generator=g, device=DEV).int()
        j = torch.arange(case["rope"] // 2, dtype=torch.float64, device=DEV)
        s["frequency"] = 500000.0 ** (-2.0 * j / max(1, case["rope"]))
    elif op == "read":
        pages = -(-case["tokens"] // case["page"]) + 3
        s["pool"] = _filled_pool(case, pages, g)
        s["slots"] = torch.randperm(pages * case["page"], generator=g, device=DEV)[:case["tokens"]].int()
    else:
        length, n = _lengths(case)
        order = torch.randperm(case["batch"], generator=g, device=DEV).tolist()
        length, n = [length[i] for i in order], [n[i] for i in order]
        each = [-(-a // case["page"]) for a in length]
        pages = sum(each) + 1
        s["pool"] = _filled_pool(case, pages, g)
        s["table"] = torch.zeros(case["batch"], max(each), dtype=torch.int32, device=DEV)
        own_pages, at = torch.randperm(pages, generator=g, device=DEV).int(), 0
        for b, e in enumerate(each):
            s["table"][b, :e] = own_pages[at:at + e]
            at += e
        s["length"] = torch.tensor(length, dtype=torch.int32, device=DEV)
        starts = [0]
        for a in n:
            starts.append(starts[-1] + a)
        s["starts"] = torch.tensor(starts, dtype=torch.int32, device=DEV)
        s["tokens"], s["most"] = starts[-1], case["draft"]
        s["q"] = _activations(g, starts[-1], case["q_heads"] * case["dim"]).view(starts[-1], case["q_heads"], case["dim"])
        s["mask"] = None
        if case["tree"]:
            see = _ancestors(n, case["draft"], g)
            s["mask"] = torch.cat([_words(see[b, :a]) for b, a in enumerate(n)]).contiguous()
    if own:
        import precision_quantized_gemm_b200 as qg
        s["cache"] = _package_cache(case, s["pool"])
        if op in ("write", "trip"):
            s["rope"] = qg.Rope(s["frequency"], interleaved=case["pairs"]) if case["rope"] else None
        if op == "attend":
            s["workspace"] = qg.Workspace(DEV)
    return s


# ----------------------------------------------------------------- definitions --
EPS, BLOCK_SCALE, RESIDUAL_SCALE = 1e-6, 0.8, 1.1


def _normed(x, weight, bias, kind):
    if kind == "layer":
        x = x - x.mean(-1, keepdim=True)
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * weight
    return x if bias is None else x + bias


def _norm_plain(s, dtype):
    """h and y of the definition, in `dtype`."""
    up = lambda t: None if t is None else t.to(dtype)  # noqa: E731
    x = up(s["x"])
    if s["case"]["post"]:
        x = _normed(x, up(s["post_weight"]), up(s["post_bias"]), s["case"]["kind"])
    if s["gate"] is not None:
        x = x * up(s["gate"])
    h = RESIDUAL_SCALE * up(s["residual"]) + BLOCK_SCALE * x
    return h, _normed(h, up(s["weight"]), up(s["bias"]), s["case"]["kind"])


def _rotated(x, angle, pairs, dtype):
    """x [T, H, D] with its first 2 * angle.shape[-1] channels rotated by angle [T, R / 2] (64 bits)."""
    half = angle.shape[-1]
    if not half:
        return x
    cos, sin = angle.cos().to(dtype)[:, None], angle.sin().to(dtype)[:, None]
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs else (x[..., :half], x[..., half:2 * half])
    out = x.clone()
    c, d = a * cos - b * sin, b * cos + a * sin
    if pairs:
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = c, d
    else:
        out[..., :half], out[..., half:2 * half] = c, d
    return out


def _qkv_plain(s, dtype):
    """Rotated queries and keys, and values."""
    c, x = s["case"], s["qkv"].to(dtype)
    angle = s["positions"].double()[:, None] * s["frequency"]
    q, k, v = x.split([c["q_heads"], c["kv_heads"], c["kv_heads"]], 1)
    return _rotated(q, angle, c["pairs"], dtype), _rotated(k, angle, c["pairs"], dtype), v


def _at(pool, slots, page):
    slots = slots.long()
    return pool[slots // page, :, slots % page]


def _attend_plain(s, dtype):
    c = s["case"]
    d, most, group, page = c["dim"], s["most"], c["q_heads"] // c["kv_heads"], c["page"]
    starts, length = s["starts"].long(), s["length"].long()
    n = starts[1:] - starts[:-1]
    place = torch.arange(s["table"].shape[1] * page, device=DEV)
    slots = s["table"].long()[:, place // page] * page + place % page                     # [B, L]
    k = _values_of(_at(s["pool"]["k"], slots, page), c["fmt"], dtype) * _at(s["pool"]["k_scale"], slots, page).to(dtype)[..., None]
    i = torch.arange(most, device=DEV)
    row = (starts[:-1, None] + i).clamp(max=s["tokens"] - 1)                              # [B, most]
    q = s["q"].to(dtype)[row].view(-1, most, c["kv_heads"], group, d).transpose(1, 2)
    score = q.reshape(-1, c["kv_heads"], most * group, d) @ k.permute(0, 2, 3, 1) / math.sqrt(d)
    del k
    j = place - (length - n)[:, None]                                                     # drafted token at a place
    if s["mask"] is None:
        sees = (j[:, None] <= i[:, None]) & (place < length[:, None])[:, None]
    else:
        word = (j.clamp(0, 64 * s["mask"].shape[1] - 1) // 64)[:, None].expand(-1, most, -1)
        bit = s["mask"][row].gather(2, word) >> (j.clamp(min=0) % 64)[:, None]
        sees = (j < 0)[:, None] | ((bit & 1).bool() & (place < length[:, None])[:, None])
    sees = sees[:, None, :, None].expand(-1, 1, most, group, -1).reshape(-1, 1, most * group, place.numel())
    score = score.masked_fill(~sees, -math.inf)
    top = score.amax(-1, keepdim=True)
    p = (score - top.clamp(min=-1e30)).exp()
    total = p.sum(-1, keepdim=True)
    del score
    v = _values_of(_at(s["pool"]["v"], slots, page), c["fmt"], dtype) * _at(s["pool"]["v_scale"], slots, page).to(dtype)[..., None]
    out = (p @ v.transpose(1, 2)) / total.clamp(min=1e-30)
    lse = (top + total.log()).squeeze(-1)
    real = (i < n[:, None])
    out = out.view(-1, c["kv_heads"], most, group, d).transpose(1, 2).reshape(-1, most, c["q_heads"], d)[real]
    lse = lse.view(-1, c["kv_heads"], most, group).transpose(1, 2).reshape(-1, most, c["q_heads"])[real]
    return out, lse


# ------------------------------------------------------------------------- run --
def _own(s):
    import precision_quantized_gemm_b200 as qg
    c, op = s["case"], s["case"]["op"]
    if op == "norm":
        fmt = {"fp8": qg.QG_FP8_DYNAMIC, "int8": qg.QG_W8A8_INT8, "block": qg.QG_BLOCK_FP8, "bf16": None}[c["fmt"]]
        r = qg.norm(s["residual"], s["weight"], s["x"], bias=s["bias"], kind=c["kind"], post_weight=s["post_weight"],
                    post_bias=s["post_bias"], gate=s["gate"], block_scale=BLOCK_SCALE, residual_scale=RESIDUAL_SCALE,
                    eps=EPS, fmt=fmt)
        if fmt is None:
            return {"h": r.h, "y": r.y}
        scale = r.operand.scale.view(torch.float32)
        codes = r.operand.q.view(c["rows"], c["width"])
        if c["fmt"] == "int8":
            return {"h": r.h, "scale": scale, "y": (codes.view(torch.int8) * scale[:, None]).to(torch.bfloat16)}
        return {"h": r.h, "scale": scale, "code": codes.view(torch.float8_e4m3fn)}
    if op in ("write", "trip"):
        q, k, v = s["qkv"].split([c["q_heads"], c["kv_heads"], c["kv_heads"]], 1)
        out = {"q": qg.cache_write(s["cache"], k, v, s["slots"], q=q, rope=s["rope"], positions=s["positions"])}
        if op == "trip":
            out["k"], out["v"] = qg.cache_read(s["cache"], s["slots"])
            return out
        return {**out, **_pool_out(s)}
    if op == "read":
        k, v = qg.cache_read(s["cache"], s["slots"])
        return {"k": k, "v": v}
    lse = torch.empty(s["tokens"], c["q_heads"], device=DEV)
    out = qg.attend(s["cache"], s["q"], s["starts"], s["length"], s["table"], tree_mask=s["mask"], max_q=s["most"],
                    lse=lse, workspace=s["workspace"])
    return {"out": out, "lse": lse}


def _pool_out(s):
    p = s["pool"]
    return {"k": p["k"].view(torch.float8_e4m3fn), "v": p["v"].view(torch.float8_e4m3fn), "k_scale": p["k_scale"],
            "v_scale": p["v_scale"]}


def _read_plain(s):
    p, c = s["pool"], s["case"]
    return {x: (_values_of(_at(p[x], s["slots"], c["page"]), c["fmt"])
                * _at(p[x + "_scale"], s["slots"], c["page"])[..., None]).to(torch.bfloat16) for x in ("k", "v")}


def run(state):
    if own:
        return _own(state)
    s, c, op = state, state["case"], state["case"]["op"]
    if op == "norm":
        h, y = _norm_plain(s, torch.float32)
        out = {"h": h.to(torch.bfloat16)}
        if c["fmt"] == "bf16":
            return {**out, "y": y.to(torch.bfloat16)}
        code, scale = _quantised(y, c["fmt"], 128 if c["fmt"] == "block" else None)
        if c["fmt"] == "int8":
            return {**out, "scale": scale, "y": (code * scale[:, None]).to(torch.bfloat16)}
        return {**out, "scale": scale.reshape(-1), "code": code.to(torch.float8_e4m3fn)}
    if op in ("write", "trip"):
        q, k, v = _qkv_plain(s, torch.float32)
        page, slots = c["page"], s["slots"].long()
        for part, x in (("k", k), ("v", v)):
            code, scale = _quantised(x, c["fmt"])
            s["pool"][part][slots // page, :, slots % page] = _bytes_of(code, c["fmt"])
            s["pool"][part + "_scale"][slots // page, :, slots % page] = scale
        out = {"q": q.to(torch.bfloat16)}
        return {**out, **(_pool_out(s) if op == "write" else _read_plain(s))}
    if op == "read":
        return _read_plain(s)
    out, lse = _attend_plain(s, torch.float32)
    return {"out": out.to(torch.bfloat16), "lse": lse}


# ----------------------------------------------------------------------- exact --
def _exact_quantised(y, fmt, group=None):
    """(what the code stands for, scale) of rows in 64 bits.  An e4m3 code is given as the quotient before its
    rounding: a code's own step is both sides' alike, and next to a border either neighbour is right."""
    code, scale = _quantised(y, fmt, group)
    if fmt == "int8":
        return code, scale.double()
    wide = scale.double().repeat_interleave(group, -1) if group else scale.double()[..., None]
    return y / wide, scale.double()


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    x = {name: v.double() for name, v in s.items() if torch.is_tensor(v) and v.is_floating_point()}
    if op == "norm":
        centre = (lambda t: t - t.mean(-1, keepdim=True)) if case["kind"] == "layer" else (lambda t: t)

        def unit(t):
            t = centre(t)
            return t / (t.pow(2).mean(-1, keepdim=True) + EPS).sqrt()

        b = x["x"]
        if case["post"]:
            b = unit(b) * x["post_weight"] + x.get("post_bias", 0.0)
        h = RESIDUAL_SCALE * x["residual"] + BLOCK_SCALE * b * x.get("gate", 1.0)
        del b
        y = unit(h) * x["weight"] + x.get("bias", 0.0)
        if case["fmt"] == "bf16":
            return {"h": h, "y": y}
        code, scale = _exact_quantised(y, case["fmt"], 128 if case["fmt"] == "block" else None)
        if case["fmt"] == "int8":
            return {"h": h, "scale": scale, "y": code * scale[:, None]}
        return {"h": h, "scale": scale.reshape(-1), "code": code}
    page = case["page"]
    if op in ("write", "trip"):
        hq, hk, r = case["q_heads"], case["kv_heads"], case["rope"]
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None] * x["frequency"])[:, None] if r else None

        def rotate(t):
            if not r:
                return t
            order = torch.arange(r, device=DEV)
            order = order if case["pairs"] else order.view(2, -1).t().reshape(-1)      # neighbours first
            z = torch.view_as_complex(t[..., order].reshape(*t.shape[:-1], r // 2, 2).contiguous()) * turn
            t = t.clone()
            t[..., order] = torch.view_as_real(z).flatten(-2)
            return t

        qkv = x["qkv"]
        q, k, v = rotate(qkv[:, :hq]), rotate(qkv[:, hq:hq + hk]), qkv[:, hq + hk:]
        out = {"q": q}
        slots = s["slots"].long()
        for part, t in (("k", k), ("v", v)):
            code, scale = _exact_quantised(t, case["fmt"])
            if op == "trip":
                full, _ = _quantised(t, case["fmt"])
                out[part] = full * scale[..., None]
                continue
            full = torch.zeros(s["pool"][part].shape, dtype=torch.float64, device=DEV)
            full[slots // page, :, slots % page] = code
            wide = torch.zeros(s["pool"][part + "_scale"].shape, dtype=torch.float64, device=DEV)
            wide[slots // page, :, slots % page] = scale
            out[part], out[part + "_scale"] = full, wide
        return out
    value = lambda t: (t.view(torch.int8) if case["fmt"] == "int8" else t.view(torch.float8_e4m3fn)).double()  # noqa: E731
    pool = s["pool"]
    if op == "read":
        a, b = s["slots"].long() // page, s["slots"].long() % page
        return {p: value(pool[p][a, :, b]) * pool[p + "_scale"][a, :, b].double()[..., None] for p in ("k", "v")}
    # attention, one sequence at a time
    group, outs, sums = case["q_heads"] // case["kv_heads"], [], []
    starts, length = s["starts"].tolist(), s["length"].tolist()
    for b in range(case["batch"]):
        n, past = starts[b + 1] - starts[b], length[b]
        pages = s["table"][b, :-(-past // page)].long()
        k, v = (((value(pool[p][pages]) * pool[p + "_scale"][pages].double()[..., None])
                 .transpose(1, 2).reshape(-1, case["kv_heads"], case["dim"])[:past]).transpose(0, 1) for p in ("k", "v"))
        q = x["q"][starts[b]:starts[b + 1]].view(n, case["kv_heads"], group, case["dim"]).permute(1, 0, 2, 3)
        z = torch.einsum("hngd,hld->hngl", q, k) * case["dim"] ** -0.5
        see = torch.ones(n, past, dtype=torch.bool, device=DEV)
        if s["mask"] is None:
            see[:, past - n:] = torch.ones(n, n, dtype=torch.bool, device=DEV).tril()
        else:
            bits = s["mask"][starts[b]:starts[b + 1], :, None] >> torch.arange(64, device=DEV)
            see[:, past - n:] = (bits & 1).bool().flatten(1)[:, :n]
        z = z.masked_fill(~see[None, :, None], -math.inf)
        lse = z.logsumexp(-1)
        w = (z - lse[..., None]).exp()
        outs.append(torch.einsum("hngl,hld->nhgd", w, v).reshape(n, case["q_heads"], case["dim"]))
        sums.append(lse.permute(1, 0, 2).reshape(n, case["q_heads"]))
    return {"out": torch.cat(outs), "lse": torch.cat(sums)}
