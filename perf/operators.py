"""Cases of the attention sublayer's query/key and cache operators, for measurement.

Four operators, as a program calls them that trains the attention sublayer and then
answers with it:

* ``rope``     norms of queries and keys for each head and the position rotation, in one
               pass over the packed projection rows (forward);
* ``rope_bwd`` its backward pass: the rows' gradient and the two norm weights' gradients;
* ``append``   the same for new tokens, with the keys and values stored into a paged cache
               (bf16 or E4M3) on the way;
* ``decode``   attention of one new token per sequence over that cache.

``run`` computes them in elementary torch operations where ``own`` is false, and through
the package's entry points where it is true.
"""
import math

import torch

own = False

BF16, F32, E4M3 = "bf16", "f32", "e4m3"
EPS = 1e-6
E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases


def _rope(name, op, rows, nq, nkv, d, rot, dtype, norm, interleaved, seq, far):
    return {"name": name, "op": op, "rows": rows, "nq": nq, "nkv": nkv, "d": d, "rot": rot, "dtype": dtype,
            "norm": norm, "interleaved": interleaved, "seq": seq, "far": far}


def _append(name, batch, rows, ragged, past, nq, nkv, d, rot, cache, norm, interleaved, page):
    return {"name": name, "op": "append", "batch": batch, "rows": rows, "ragged": ragged, "past": past, "nq": nq,
            "nkv": nkv, "d": d, "rot": rot, "cache": cache, "norm": norm, "interleaved": interleaved, "page": page}


def _decode(name, batch, longest, ragged, nq, nkv, d, cache, page, window, sinks):
    return {"name": name, "op": "decode", "batch": batch, "longest": longest, "ragged": ragged, "nq": nq, "nkv": nkv,
            "d": d, "cache": cache, "page": page, "window": window, "sinks": sinks}


def listed():
    return [
        # one long training sequence of the attention benchmark's heads
        _rope("rope 1x32768", "rope", 32768, 32, 8, 128, 128, BF16, True, False, 32768, False),
        # an fp32 model with partial rotation of neighbouring pairs, positions given, far ones among them
        _rope("rope f32 1017 far", "rope", 1017, 6, 2, 64, 32, F32, False, True, 0, True),
        # the attention benchmark's training step, 4 x 2048 tokens
        _rope("rope backward 4x2048", "rope_bwd", 8192, 32, 8, 128, 128, BF16, True, False, 2048, False),
        # a short odd batch in fp32, one key head
        _rope("rope backward f32 333", "rope_bwd", 333, 5, 1, 192, 192, F32, True, False, 0, False),
        # the smallest call: one new token of one sequence
        _append("append one token", 1, 1, False, 700, 32, 8, 128, 128, BF16, True, False, 16),
        # one new token of each of many sequences, cache in 8 bits
        _append("append 256 tokens e4m3", 256, 256, False, 4000, 32, 8, 128, 128, E4M3, True, False, 64),
        # prompts of different lengths, packed one behind the other
        _append("append 13 prompts", 13, 16000, True, 300, 32, 8, 128, 128, BF16, True, False, 64),
        # the smallest call: a short sequence answered alone
        _decode("decode 1x500", 1, 500, False, 32, 8, 128, BF16, 16, 0, 0),
        # one long document answered alone
        _decode("decode 1x131072", 1, 131072, False, 32, 8, 128, BF16, 64, 0, 0),
        # a serving batch of sequences of very different lengths
        _decode("decode 64 ragged", 64, 8192, True, 32, 8, 128, BF16, 64, 0, 0),
        # the same with twice the sequences and the cache in 8 bits
        _decode("decode 128 ragged e4m3", 128, 8192, True, 32, 8, 128, E4M3, 32, 0, 0),
        # multi-head attention with a sliding window and the first tokens kept
        _decode("decode 48 window", 48, 12000, True, 16, 16, 64, BF16, 48, 1024, 4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["rope", "rope_bwd", "append", "decode"])
    d = rng.choice([64, 128, 128, 192, 256])
    nkv = rng.choice([1, 2, 4, 8])
    nq = nkv * rng.choice([1, 2, 3, 4, 7, 8, 16])
    rot = rng.choice([d, d, d // 2, 16])
    norm, interleaved = rng.random() < 0.6, rng.random() < 0.4
    if op in ("rope", "rope_bwd"):
        dtype = rng.choice([BF16, BF16, F32])
        most = 32768 * 40 * 128 * 2 // (2 if op == "rope_bwd" else 1)
        rows = min(_log_int(rng, 1, 32768), most // ((nq + nkv) * d * (2 if dtype == BF16 else 4)))
        seq = rng.choice([0, 0, 128 * rng.randint(1, 32)])
        c = _rope("", op, max(1, rows), nq, nkv, d, rot, dtype, norm, interleaved, seq, seq == 0 and rng.random() < 0.3)
    elif op == "append":
        most = 16000 * 48 * 128 // ((nq + 2 * nkv) * d)
        rows = max(1, min(_log_int(rng, 1, 16000), most))
        ragged = rng.random() < 0.5
        batch = rng.randint(1, min(rows, 300)) if ragged else rows
        if not ragged and rows > 512:
            batch = rng.randint(1, 40)
            rows -= rows % batch
        past = _log_int(rng, 1, 4000)
        c = _append("", batch, rows, ragged, past, nq, nkv, d, rot, rng.choice([BF16, E4M3]), norm, interleaved,
                    rng.choice([16, 32, 48, 64, 128]))
    else:
        cache = rng.choice([BF16, E4M3])
        batch = _log_int(rng, 1, 128)
        most = 2 ** 18 * 8 * 128 // (batch * nkv * d)  # tokens of the longest sequence
        longest = _log_int(rng, 1, max(2, min(131072, most)))
        window = rng.choice([0, 0, rng.randint(1, 2048)])
        c = _decode("", batch, longest, rng.random() < 0.7, nq, nkv, d, cache, rng.choice([16, 32, 48, 64, 128]), window,
                    rng.choice([0, 4, 70]) if window else 0)
    del c["name"]
    return c


# ------------------------------------------------------------------ inputs


def _inv_freq(rot):
    """Radians per position of each rotated pair, in 64 bits."""
    return torch.tensor([10000.0 ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float64)


def _randn(g, shape, dtype=torch.bfloat16, scale=1.0, shift=0.0):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(scale).add_(shift).to(dtype)


def _table(g, lens, page, total):
    """A block table [batch, pages of the longest + 1]: pages in random order, -1 behind each sequence's last page."""
    need = (lens + page - 1) // page
    width = int(need.max()) + 1
    perm = torch.randperm(total, generator=g, device="cuda").to(torch.int32)
    col = torch.arange(width, device="cuda")[None, :]
    start = torch.cumsum(need, 0) - need
    at = (start[:, None] + col).clamp(max=total - 1)
    return torch.where(col < need[:, None], perm[at], torch.full_like(perm[at], -1))


def _new_cache(g, pages, nkv, page, d, kind):
    """Key or value pages [pages, nkv, page, d]; E4M3 codes stand for values of about unit size."""
    if kind == BF16:
        return _randn(g, (pages, nkv, page, d))
    return _randn(g, (pages, nkv, page, d), torch.bfloat16, 32.0).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    op, nq, nkv, d = case["op"], case["nq"], case["nkv"], case["d"]
    s = {"case": dict(case)}
    if op in ("rope", "rope_bwd"):
        dtype = torch.bfloat16 if case["dtype"] == BF16 else torch.float32
        rows, qk = case["rows"], (nq + nkv) * d
        s["x"] = _randn(g, (rows, qk + nkv * d), dtype, 1.5)  # packed projection rows: queries, keys, values
        if case["seq"] == 0:
            s["pos"] = torch.randint(0, 1 << 20 if case["far"] else 4096, (rows,), generator=g, device="cuda",
                                     dtype=torch.int32)
        if op == "rope_bwd":
            s["dout"] = _randn(g, (rows, qk), dtype, 0.02)
    elif op == "append":
        batch, rows = case["batch"], case["rows"]
        past = torch.randint(case["past"] // 2, case["past"] + 1, (batch,), generator=g, device="cuda",
                             dtype=torch.int32)
        if case["ragged"]:
            cuts = torch.randint(0, rows + 1, (batch - 1,), generator=g, device="cuda").sort().values
            ends = torch.tensor([0, rows], device="cuda")
            cu = torch.cat([ends[:1], cuts, ends[1:]])
            s["cu"] = cu.to(torch.int32)
            new = cu[1:] - cu[:-1]
        else:
            new = torch.full((batch,), rows // batch, device="cuda")
        s["past"], s["x"] = past, _randn(g, (rows, (nq + 2 * nkv) * d), torch.bfloat16, 1.5)
        pages = rows // case["page"] + batch * (case["past"] // case["page"] + 2) + 3
        s["table"] = _table(g, past + new, case["page"], pages)
    else:
        batch = case["batch"]
        if case["ragged"]:
            lens = torch.randint(0, case["longest"] + 1, (batch,), generator=g, device="cuda")
            lens[0] = case["longest"]
        else:
            lens = torch.full((batch,), case["longest"], device="cuda")
        s["lens"], s["q"] = lens.to(torch.int32), _randn(g, (batch, nq * d), torch.bfloat16, 1.5)
        pages = int(((lens + case["page"] - 1) // case["page"]).sum()) + 3
        s["table"] = _table(g, lens, case["page"], pages)
    if op in ("append", "decode"):
        s["k"] = _new_cache(g, pages, nkv, case["page"], d, case["cache"])
        s["v"] = _new_cache(g, pages, nkv, case["page"], d, case["cache"])
        if case["cache"] == E4M3:  # what one code unit stands for, for each key head
            s["ks"] = torch.rand(nkv, generator=g, device="cuda").mul_(0.02).add_(0.02)
            s["vs"] = torch.rand(nkv, generator=g, device="cuda").mul_(0.02).add_(0.02)
    if op != "decode":
        s["freq"] = _inv_freq(case["rot"]).cuda()
        if case["norm"]:
            s["qw"], s["kw"] = (_randn(g, (d,), s["x"].dtype, 0.1, 1.0) for _ in range(2))
    if own:  # the handles that a program keeps: host structures and the context's scratch
        import tensor_transformer_mlp_rmsnorm_gb300 as tp
        if op != "decode":
            s["rot"] = tp.Rotary(case["rot"], inv_freq=_inv_freq(case["rot"]).tolist(),
                                 interleaved=case["interleaved"])
        if op in ("append", "decode"):
            s["kv"] = tp.TPKV(s["k"], s["v"], nq, max_batch=case["batch"], k_inv_scale=s.get("ks"),
                              v_inv_scale=s.get("vs"))
        if op == "append":
            s["kv"].set_rotary(s["rot"], s.get("qw"), s.get("kw"), EPS)
    return s


# ------------------------------------------------------------------ plain forms


def _positions(s):
    rows = s["x"].shape[0]
    return s["pos"] if "pos" in s else torch.arange(rows, device="cuda") % s["case"]["seq"]


def _angles(s, pos):
    """cos and sin [rows, 1, rot / 2] in 32 bits, of angles taken in 64."""
    a = (pos.double()[:, None] * s["freq"][None, :])[:, None, :]
    return a.cos().float(), a.sin().float()


def _turn(h, cos, sin, rot, interleaved):
    """Rotates the first rot values of each head of h [rows, heads, d]."""
    if interleaved:
        a, b = h[..., 0:rot:2], h[..., 1:rot:2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = h[..., : rot // 2], h[..., rot // 2: rot]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, h[..., rot:]], -1)


def _normed(h, w):
    """x / rms(x) of each head, its reciprocal rms, and the weighted norm."""
    rstd = (h.square().mean(-1, keepdim=True) + EPS).rsqrt()
    return h * rstd, rstd, h * rstd * w.float()


def _heads(s, x, lo, n):
    d = s["case"]["d"]
    return x[:, lo * d: (lo + n) * d].float().unflatten(1, (n, d))


def _rope_plain(s, pos):
    c = s["case"]
    cos, sin = _angles(s, pos)
    q, k = _heads(s, s["x"], 0, c["nq"]), _heads(s, s["x"], c["nq"], c["nkv"])
    if c["norm"]:
        q, k = _normed(q, s["qw"])[2], _normed(k, s["kw"])[2]
    return _turn(q, cos, sin, c["rot"], c["interleaved"]), _turn(k, cos, sin, c["rot"], c["interleaved"])


def _head_bwd(h, g, w):
    """Gradients of the weighted norm's input and of its weight, g the gradient of its output."""
    xhat, rstd, _ = _normed(h, w)
    gw = g * w.float()
    dx = rstd * (gw - xhat * (gw * xhat).mean(-1, keepdim=True))
    return dx, (g * xhat).sum((0, 1), dtype=torch.float64).float()


def _rope_bwd_plain(s):
    c, x = s["case"], s["x"]
    cos, sin = _angles(s, _positions(s))
    gq = _turn(_heads(s, s["dout"], 0, c["nq"]), cos, -sin, c["rot"], c["interleaved"])
    gk = _turn(_heads(s, s["dout"], c["nq"], c["nkv"]), cos, -sin, c["rot"], c["interleaved"])
    if not c["norm"]:
        return {"dx": torch.cat([gq, gk], 1).flatten(1).to(x.dtype)}
    dq, dqw = _head_bwd(_heads(s, x, 0, c["nq"]), gq, s["qw"])
    dk, dkw = _head_bwd(_heads(s, x, c["nq"], c["nkv"]), gk, s["kw"])
    return {"dx": torch.cat([dq, dk], 1).flatten(1).to(x.dtype), "dqw": dqw, "dkw": dkw}


def _row_places(s):
    """Each row's position, page and slot in the page."""
    c, rows = s["case"], torch.arange(s["x"].shape[0], device="cuda")
    if c["ragged"]:
        seq = (rows[:, None] >= s["cu"][None, 1:]).sum(1)
        at = rows - s["cu"][seq]
    else:
        per = c["rows"] // c["batch"]
        seq, at = rows // per, rows % per
    pos = s["past"][seq] + at
    return pos, s["table"][seq, pos // c["page"]].long(), pos % c["page"]


def _stored(h, s, scale):
    """What the cache holds of heads h [rows, nkv, d]."""
    if s["case"]["cache"] == BF16:
        return h.to(torch.bfloat16)
    return (h / s[scale][None, :, None]).clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _put(cache, page, slot, h):
    """cache[page, :, slot] = h; codes of 8 bits are moved as bytes."""
    if cache.dtype == torch.float8_e4m3fn:
        cache, h = cache.view(torch.uint8), h.view(torch.uint8)
    cache[page, :, slot] = h


def _append_plain(s):
    c = s["case"]
    pos, page, slot = _row_places(s)
    q, k = _rope_plain(s, pos)
    _put(s["k"], page, slot, _stored(k, s, "ks"))
    _put(s["v"], page, slot, _stored(_heads(s, s["x"], c["nq"] + c["nkv"], c["nkv"]), s, "vs"))
    return {"q": q.flatten(1).to(torch.bfloat16), "k": s["k"], "v": s["v"]}


def _gathered(s, name, scale):
    """The pages of every sequence in order, [batch, nkv, tokens, d] in 32 bits."""
    cache, batch = s[name], s["table"].shape[0]
    raw = cache.view(torch.uint8) if cache.dtype == torch.float8_e4m3fn else cache
    t = raw[s["table"].clamp(min=0).long()].view(cache.dtype).float()
    t = t * s[scale][:, None, None] if scale in s else t
    return t.transpose(1, 2).reshape(batch, cache.shape[1], -1, cache.shape[3])


def _decode_plain(s):
    c = s["case"]
    k, lens = _gathered(s, "k", "ks"), s["lens"][:, None]
    q = s["q"].float().unflatten(1, (c["nkv"], c["nq"] // c["nkv"], c["d"]))
    sc = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(c["d"]))  # [batch, nkv, heads, tokens]
    del k
    at = torch.arange(sc.shape[3], device="cuda")[None, :]
    seen = at < lens
    if c["window"]:
        seen = seen & ((at >= lens - c["window"]) | (at < c["sinks"]))
    seen = seen[:, None, None, :]
    sc = torch.where(seen, sc, float("-inf"))
    top = sc.amax(-1, keepdim=True).clamp(min=-3.0e38)
    p = torch.where(seen, (sc - top).exp(), 0.0)
    total = p.sum(-1, keepdim=True)
    v = torch.where(seen[:, :, 0, :, None], _gathered(s, "v", "vs"), 0.0)
    out = torch.matmul(p, v) / torch.where(total > 0, total, 1.0)
    lse = torch.where(total > 0, top + total.log(), float("-inf"))
    return {"out": out.flatten(1).to(torch.bfloat16), "lse": lse.flatten(1)}


def run(state):
    s, c = state, state["case"]
    op = c["op"]
    if not own:
        if op == "rope":
            q, k = _rope_plain(s, _positions(s))
            return {"out": torch.cat([q, k], 1).flatten(1).to(s["x"].dtype)}
        return _rope_bwd_plain(s) if op == "rope_bwd" else _append_plain(s) if op == "append" else _decode_plain(s)
    import tensor_transformer_mlp_rmsnorm_gb300 as tp
    if op == "rope":
        out = tp.qk_norm_rope(s["x"], c["nq"], c["nkv"], c["d"], s["rot"], positions=s.get("pos"), seq=c["seq"],
                              q_norm_w=s.get("qw"), k_norm_w=s.get("kw"), eps=EPS)
        return {"out": out}
    if op == "rope_bwd":
        dx, dqw, dkw = tp.qk_norm_rope_backward(s["dout"], s["x"], c["nq"], c["nkv"], c["d"], s["rot"],
                                                positions=s.get("pos"), seq=c["seq"], q_norm_w=s.get("qw"),
                                                k_norm_w=s.get("kw"), eps=EPS)
        return {"dx": dx, "dqw": dqw, "dkw": dkw} if c["norm"] else {"dx": dx}
    if op == "append":
        q = s["kv"].append(s["x"], s["past"], s["table"], cu_rows=s.get("cu"))
        return {"q": q, "k": s["k"], "v": s["v"]}
    out, lse = s["kv"].decode(s["q"], s["lens"], s["table"], window=c["window"], sinks=c["sinks"], return_lse=True)
    return {"out": out, "lse": lse}


# ------------------------------------------------------------------ work


def work(case):
    nq, nkv, d, op = case["nq"], case["nkv"], case["d"], case["op"]
    if op in ("rope", "rope_bwd"):
        e = 2 if case["dtype"] == BF16 else 4
        values = case["rows"] * (nq + nkv) * d
        passes = 2 if op == "rope" else 3 if case["norm"] else 2
        return {"bytes": values * e * passes, "flops": values * (8 if op == "rope" else 16)}
    e = 2 if case["cache"] == BF16 else 1
    if op == "append":
        rows = case["rows"]
        return {"bytes": rows * d * ((nq + 2 * nkv) * 2 + nq * 2 + 2 * nkv * e), "flops": rows * (nq + nkv) * d * 8}
    longest, batch = case["longest"], case["batch"]
    most = case["window"] + case["sinks"] if case["window"] else longest
    if case["ragged"] and most < longest:  # lengths are uniform up to the longest: the mean of min(length, most)
        mean = most - most * most / (2.0 * longest)
    else:
        mean = longest / 2.0 if case["ragged"] else float(min(longest, most))
    tokens = (batch - 1) * mean + min(longest, most)  # the first sequence has the longest length
    return {"bytes": tokens * nkv * d * 2 * e + batch * nq * d * 4, "flops": tokens * nq * d * 4}


# ------------------------------------------------------------------ the definition in 64 bits


def _exact_rotate(h, pos, freq, rot, interleaved):
    """h [rows, heads, d] as complex pairs times exp(i pos freq)."""
    first = torch.arange(0, rot, 2, device="cuda") if interleaved else torch.arange(rot // 2, device="cuda")
    second = first + (1 if interleaved else rot // 2)
    z = torch.complex(h[:, :, first], h[:, :, second])
    angle = torch.outer(pos.to(torch.float64), freq)
    z = z * torch.polar(torch.ones_like(angle), angle)[:, None, :]
    out = h.clone()
    out[:, :, first], out[:, :, second] = z.real, z.imag
    return out


def _exact_norm(h, w):
    return h if w is None else h / torch.sqrt((h * h).sum(-1, keepdim=True) / h.shape[-1] + EPS) * w.double()


def _exact_rows(s, c):
    if "pos" in s:
        return s["pos"]
    return torch.arange(c["rows"], device="cuda").remainder(c["seq"])


def _exact_rope(c, s, pos):
    nq, nkv, d = c["nq"], c["nkv"], c["d"]
    h = s["x"][:, : (nq + nkv) * d].double().reshape(-1, nq + nkv, d)
    h = torch.cat([_exact_norm(h[:, :nq], s.get("qw")), _exact_norm(h[:, nq:], s.get("kw"))], 1)
    return _exact_rotate(h, pos, s["freq"], c["rot"], c["interleaved"])


def _exact_rope_bwd(c, s):
    nq, nkv, d, rows = c["nq"], c["nkv"], c["d"], c["rows"]
    x = s["x"][:, : (nq + nkv) * d].double().reshape(rows, nq + nkv, d)
    g = s["dout"].double().reshape(rows, nq + nkv, d)
    g = _exact_rotate(g, -_exact_rows(s, c).long(), s["freq"], c["rot"], c["interleaved"])
    if not c["norm"]:
        return {"dx": g.reshape(rows, -1)}
    w = torch.cat([s["qw"].double().expand(nq, d), s["kw"].double().expand(nkv, d)], 0)
    rms = torch.sqrt((x * x).sum(-1, keepdim=True) / d + EPS)
    # y = w x / rms, so dL/dx = w g / rms - x (sum_j w_j g_j x_j) / (d rms^3)
    dx = w * g / rms - x * (w * g * x).sum(-1, keepdim=True) / (d * rms ** 3)
    per_head = (g * x / rms).sum(0)
    return {"dx": dx.reshape(rows, -1), "dqw": per_head[:nq].sum(0), "dkw": per_head[nq:].sum(0)}


def _exact_append(c, s):
    nq, nkv, d, page = c["nq"], c["nkv"], c["d"], c["page"]
    past, table, batch = s["past"].tolist(), s["table"], c["batch"]
    cu = s["cu"].tolist() if c["ragged"] else [b * (c["rows"] // batch) for b in range(batch + 1)]
    counts = torch.tensor([b - a for a, b in zip(cu, cu[1:])], device="cuda")
    seq = torch.repeat_interleave(torch.arange(batch, device="cuda"), counts)
    pos = torch.cat([torch.arange(p, p + b - a, device="cuda") for p, a, b in zip(past, cu, cu[1:])])
    h = _exact_rope(c, s, pos)
    k, v = h[:, nq:], s["x"][:, (nq + nkv) * d:].double().reshape(-1, nkv, d)
    if c["cache"] == E4M3:
        k = (k / s["ks"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        v = (v / s["vs"].double()[:, None]).clamp(-E4M3_MAX, E4M3_MAX)
    out = {"q": h[:, :nq].reshape(-1, nq * d)}
    where = table[seq, pos // page].long()
    for name, new in (("k", k), ("v", v)):
        full = s[name].double()
        full[where, :, pos % page] = new
        out[name] = full
    return out


def _exact_decode(c, s):
    nq, nkv, d, page = c["nq"], c["nkv"], c["d"], c["page"]
    outs, lses = [], []
    for b, n in enumerate(s["lens"].tolist()):
        q = s["q"][b].double().reshape(nkv, nq // nkv, d)
        at = torch.arange(n, device="cuda")
        if c["window"]:
            at = at[(at >= n - c["window"]) | (at < c["sinks"])]
        if n == 0:
            outs.append(torch.zeros(nq * d, dtype=torch.float64, device="cuda"))
            lses.append(torch.full((nq,), -math.inf, dtype=torch.float64, device="cuda"))
            continue
        pages = s["table"][b][at // page].long()
        kv = {}
        for name in ("k", "v"):
            if c["cache"] == E4M3:
                kv[name] = s[name].view(torch.uint8)[pages, :, at % page].view(torch.float8_e4m3fn).double()
                kv[name] = kv[name] * s[name + "s"].double()[:, None]
            else:
                kv[name] = s[name][pages, :, at % page].double()
        sc = torch.einsum("ghd,tgd->ght", q, kv["k"]) / math.sqrt(d)
        lse = torch.logsumexp(sc, -1)
        outs.append(torch.einsum("ght,tgd->ghd", torch.exp(sc - lse[..., None]), kv["v"]).reshape(-1))
        lses.append(lse.reshape(-1))
    return {"out": torch.stack(outs), "lse": torch.stack(lses)}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "rope":
        return {"out": _exact_rope(case, s, _exact_rows(s, case)).reshape(case["rows"], -1)}
    if op == "rope_bwd":
        return _exact_rope_bwd(case, s)
    return _exact_append(case, s) if op == "append" else _exact_decode(case, s)
