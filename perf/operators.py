"""Cases, plain forms and 64-bit values of the prompt operators.

A prompt passes through four operators before and between decode steps:
  qk_rotary         per-head RMS norms of queries and keys and the rotary
                    position rotation, in one pass (also for the new token
                    of every decode step)
  prompt_attention  causal attention of packed prompts of different lengths
                    with grouped heads, also of a chunk (down to one token)
                    against a longer history
  cache_write       one layer's packed K/V into the mixed FP16/INT8 cache
                    (Cache.prefill_begin / prefill_layer), returned as read
                    back
  cache_read        one layer's resident entries as packed K/V
                    (Cache.read_layer)
run() computes them with elementary torch operations, or through the package
when `own` is true.
"""
import math

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _lens(text):
    return [int(x) for x in str(text).split(",")]


# ---------------------------------------------------------------- the cases

def _rotary_case(tokens, Hq, Hkv, d, rot, dtype, norm=True, interleaved=False, scaling="none", factor=1.0,
                 far=40000, **kw):
    return dict(op="qk_rotary", tokens=tokens, Hq=Hq, Hkv=Hkv, d=d, rot=rot, dtype=dtype, norm=norm,
                interleaved=interleaved, scaling=scaling, factor=factor, far=far, **kw)


def _attention_case(lens_q, lens_k, Hq, Hkv, d, dtype, causal=True, lse=False, **kw):
    return dict(op="prompt_attention", lens_q=lens_q, lens_k=lens_k, Hq=Hq, Hkv=Hkv, d=d, dtype=dtype,
                causal=causal, lse=lse, **kw)


def _cache_case(op, lens, Hkv, d, W, dtype, **kw):
    return dict(op=op, lens=lens, Hkv=Hkv, d=d, W=W, dtype=dtype, **kw)


def listed():
    return [
        # one new token of one sequence, 32B-shaped layer: a decode step's latency
        _rotary_case(1, 40, 8, 128, 128, "bf16", name="rotary_token"),
        # a whole layer's prompt of the 14B-shaped workload
        _rotary_case(8192, 40, 8, 128, 128, "bf16", name="rotary_prompt_8192"),
        # odd count, equal head counts, half of each head rotated in adjacent
        # pairs, positions far beyond the trained length
        _rotary_case(1373, 12, 12, 64, 32, "f16", norm=False, interleaved=True, scaling="yarn", factor=32.0,
                     far=1000000, name="rotary_partial_far"),
        # the small-model workload's prompt
        _attention_case("600", "600", 12, 12, 64, "f16", lse=True, name="attention_600"),
        # the next token of eight sequences with histories of unlike lengths
        _attention_case("1,1,1,1,1,1,1,1", "4096,37,2500,4095,1025,129,3333,1", 40, 8, 128, "bf16",
                        name="attention_tokens"),
        # packed prompts of a mixed batch: one token to a few thousand
        _attention_case("2047,1,511,130,1280,77,333,1536", "2047,1,511,130,1280,77,333,1536", 40, 8, 128, "bf16",
                        lse=True, name="attention_ragged"),
        # a chunk of a long prompt against all of its history
        _attention_case("1000", "15000", 40, 8, 128, "f16", name="attention_chunk"),
        # one long prompt
        _attention_case("16384", "16384", 40, 8, 128, "bf16", name="attention_16384"),
        # the small-model workload's layer
        _cache_case("cache_write", "600", 12, 64, 64, "f16", name="cache_write_600"),
        # the 32B-shaped workload's layer, eight prompts
        _cache_case("cache_write", "4096,4096,4096,4096,4096,4096,4096,4096", 8, 128, 256, "bf16",
                    name="cache_write_8x4096"),
        _cache_case("cache_read", "600", 12, 64, 64, "f16", name="cache_read_600"),
        # unlike lengths, one shorter than the window
        _cache_case("cache_read", "8191,100,2048,5000,1,4097,8192,6001", 8, 128, 256, "bf16",
                    name="cache_read_ragged"),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["qk_rotary", "prompt_attention", "prompt_attention", "cache_write", "cache_read"])
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4, 8, 12])
    dtype = rng.choice(["f16", "bf16"])
    if op == "qk_rotary":
        G = rng.randint(1, 8)
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        return _rotary_case(_log(rng, 1, 8192), Hkv * G if Hkv * G <= 40 else Hkv, Hkv, d,
                            rng.choice([d, d, d // 2, d // 4, 24]), dtype, norm=rng.random() < 0.6,
                            interleaved=rng.random() < 0.5, scaling=scaling,
                            factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                            far=_log(rng, 1000, 1000000))
    if op == "prompt_attention":
        G = rng.randint(1, 8)
        Hq = Hkv * G if Hkv * G <= 40 else Hkv
        B = rng.randint(1, 8)
        kind = rng.choice(["prompt", "prompt", "chunk", "token"])
        top = int(math.sqrt(4e9 / (B * Hq)))          # padded scores of the plain form
        lk = [_log(rng, 1, min(8192, top)) for _ in range(B)]
        if kind == "prompt":
            lq = list(lk)
        elif kind == "chunk":
            lq = [_log(rng, 1, x) for x in lk]
        else:
            lq = [1] * B
        return _attention_case(",".join(map(str, lq)), ",".join(map(str, lk)), Hq, Hkv, d, dtype,
                               causal=rng.random() < 0.8, lse=rng.random() < 0.5)
    lens = ",".join(str(_log(rng, 1, 8192)) for _ in range(rng.randint(1, 8)))
    return _cache_case(op, lens, min(Hkv, 8), d, rng.choice([16, 64, 100, 256]), dtype)


# ---------------------------------------------------------------- inputs

def _normal(g, shape, dtype):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _padded(lens):
    """Row of each (sequence, token) in the packed tensor, [B, Tmax], clamped
    to the sequence, and each packed row's place in the padded form."""
    n = torch.tensor(lens, device="cuda")
    start = torch.cumsum(n, 0) - n
    t = torch.arange(max(lens), device="cuda")
    rows = start[:, None] + torch.minimum(t[None, :], (n - 1).clamp(min=0)[:, None])
    seg = torch.repeat_interleave(torch.arange(len(lens), device="cuda"), n)
    at = torch.arange(sum(lens), device="cuda") - start[seg]
    return n, rows, seg, at


def _keys(g, lens, H, d, dtype):
    """Packed keys, one in 200 of them three times as long (heavy tokens)."""
    k = torch.randn((sum(lens), H, d), generator=g, device="cuda")
    heavy = torch.rand((sum(lens), 1, 1), generator=g, device="cuda") < 0.005
    return torch.where(heavy, 3.0 * k, k).to(dtype)


def _inv_freq(case):
    """Rotation of each pair per position, in 64 bits (python floats)."""
    rot, base, f, L0 = case["rot"], 10000.0, case["factor"], 4096.0
    if case["scaling"] == "ntk":
        base = base * f ** (rot / (rot - 2.0))
    inv = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if case["scaling"] == "linear":
        inv = [x / f for x in inv]
    if case["scaling"] == "yarn":
        keep = [min(1.0, max(0.0, (L0 * x / (2.0 * math.pi) - 1.0) / 31.0)) for x in inv]
        inv = [x * w + x / f * (1.0 - w) for x, w in zip(inv, keep)]
    return inv, (0.1 * math.log(f) + 1.0 if case["scaling"] == "yarn" else 1.0)


def _cache(case, lens):
    import confidence_gated_kv_gb300 as ck
    W = case["W"]
    cap = max(16, max(lens))
    return ck.Cache(ck.make_config(L=1, Hq=case["Hkv"], Hkv=case["Hkv"], d=case["d"], V=1000, B=len(lens), cap=cap,
                                   W=W, P=1, n_high=[cap], n_low=[cap]))


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    op, dt = case["op"], DTYPES[case["dtype"]]
    s = {"case": case}
    if op == "qk_rotary":
        n, d = case["tokens"], case["d"]
        s["q"], s["k"] = _normal(g, (n, case["Hq"], d), dt), _normal(g, (n, case["Hkv"], d), dt)
        first = int(torch.randint(0, case["far"], (1,), generator=g, device="cuda"))
        s["pos"] = (first + torch.arange(n, device="cuda")).to(torch.int32)
        s["qw"] = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt) if case["norm"] else None
        s["kw"] = (1.0 + 0.1 * torch.randn(d, generator=g, device="cuda")).to(dt) if case["norm"] else None
        inv, s["mscale"] = _inv_freq(case)
        s["inv_freq"] = torch.tensor(inv, dtype=torch.float64, device="cuda")
        if own:   # the table that a model keeps
            import confidence_gated_kv_gb300 as ck
            s["rotary"] = ck.Rotary(case["rot"], base=10000.0, scaling=case["scaling"], factor=case["factor"],
                                    original_length=4096, interleaved=case["interleaved"])
        return s
    if op == "prompt_attention":
        lq, lk, d = _lens(case["lens_q"]), _lens(case["lens_k"]), case["d"]
        s["q"] = _normal(g, (sum(lq), case["Hq"], d), dt)
        s["k"], s["v"] = _keys(g, lk, case["Hkv"], d, dt), _normal(g, (sum(lk), case["Hkv"], d), dt)
        s["pad_q"], s["pad_k"] = _padded(lq), _padded(lk)
        s["cu_q"] = torch.tensor([sum(lq[:i]) for i in range(len(lq) + 1)], dtype=torch.int32, device="cuda")
        s["cu_k"] = torch.tensor([sum(lk[:i]) for i in range(len(lk) + 1)], dtype=torch.int32, device="cuda")
        return s
    lens = _lens(case["lens"])
    k = _keys(g, lens, case["Hkv"], case["d"], dt)
    v = _normal(g, (sum(lens), case["Hkv"], case["d"]), dt)
    s["lens"] = lens
    if own:       # the cache that a decode loop keeps
        s["cache"] = _cache(case, lens)
    if op == "cache_write":
        s["k"], s["v"], s["pad"] = k, v, _padded(lens)
        return s
    n, _, seg, at = s["pad"] = _padded(lens)
    s["old"] = at < (n - case["W"])[seg]
    for name, x in (("k", k), ("v", v)):
        s[name + "_scale"], s[name + "_codes"] = _quantise(x.half().float(), s["pad"])
        s[name + "_codes"], s[name + "16"] = s[name + "_codes"].to(torch.int8), x.half()
    if own:
        s["cache"].prefill_begin(lens)
        s["cache"].prefill_layer(0, k, v)
    return s


# ---------------------------------------------------------------- plain forms

def _rotate(x, w, cos, sin, case):
    x = x.float()
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w.float()
    rot, h = case["rot"], case["rot"] // 2
    y = x.clone()
    a, b = (slice(0, rot, 2), slice(1, rot, 2)) if case["interleaved"] else (slice(0, h), slice(h, rot))
    y[..., a] = x[..., a] * cos - x[..., b] * sin
    y[..., b] = x[..., b] * cos + x[..., a] * sin
    return y


def _plain_rotary(s):
    case, dt = s["case"], s["q"].dtype
    angle = s["pos"].double()[:, None, None] * s["inv_freq"]
    cos, sin = (angle.cos() * s["mscale"]).float(), (angle.sin() * s["mscale"]).float()
    return [_rotate(s["q"], s["qw"], cos, sin, case).to(dt), _rotate(s["k"], s["kw"], cos, sin, case).to(dt)]


def _plain_attention(s):
    case, dt = s["case"], s["q"].dtype
    nq, rows_q, seg_q, at_q = s["pad_q"]
    nk, rows_k, _, _ = s["pad_k"]
    (B, Tq), Tk, Hkv, d = rows_q.shape, rows_k.shape[1], case["Hkv"], case["d"]
    G = case["Hq"] // Hkv
    q = s["q"].float()[rows_q].view(B, Tq, Hkv, G, d).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * Tq, d)
    k, v = (s[x].float()[rows_k].transpose(1, 2) for x in ("k", "v"))
    score = (q * (1.0 / math.sqrt(d))) @ k.transpose(-1, -2)
    i, j = torch.arange(Tq, device="cuda")[:, None], torch.arange(Tk, device="cuda")[None, :]
    hidden = j >= nk[:, None, None]
    if case["causal"]:
        hidden = hidden | (j > i + (nk - nq)[:, None, None])
    score.view(B, Hkv, G, Tq, Tk).masked_fill_(hidden[:, None, None], -math.inf)
    top = score.amax(-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = score.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.where(total > 0, (p @ v) / total, 0.0)
    out = out.view(B, Hkv, G, Tq, d).permute(0, 3, 1, 2, 4)[seg_q, at_q].reshape(-1, case["Hq"], d).to(dt)
    if not case["lse"]:
        return [out]
    lse = (top + total.log()).view(B, Hkv, G, Tq).permute(0, 3, 1, 2)[seg_q, at_q].reshape(-1, case["Hq"])
    return [out, lse]


def _quantise(x, pad):
    """Scale of each (sequence, head, channel) and the code of each value."""
    n, rows, seg, _ = pad
    inside = torch.arange(rows.shape[1], device="cuda")[None, :] < n[:, None]
    top = torch.where(inside[:, :, None, None], x[rows].abs(), 0.0).amax(1)
    scale = torch.where(top > 0, top / 127.0, 1.0)
    return scale, torch.round(x / scale[seg]).clamp(-127.0, 127.0)


def _plain_write(s):
    n, _, seg, at = s["pad"]
    old = (at < (n - s["case"]["W"])[seg])[:, None, None]
    got = []
    for name in ("k", "v"):
        x = s[name].half().float()
        scale, code = _quantise(x, s["pad"])
        got.append(torch.where(old, code * scale[seg], x).half())
    return got + [at.to(torch.int32)]


def _plain_read(s):
    n, _, seg, at = s["pad"]
    dt, old = DTYPES[s["case"]["dtype"]], s["old"][:, None, None]
    got = [torch.where(old, s[x + "_codes"].float() * s[x + "_scale"][seg], s[x + "16"].float()).to(dt)
           for x in ("k", "v")]
    return got + [at.to(torch.int32)]


# ---------------------------------------------------------------- the calls

def _own(s):
    import confidence_gated_kv_gb300 as ck
    case, op = s["case"], s["case"]["op"]
    if op == "qk_rotary":
        return list(ck.qk_rotary(s["q"], s["k"], s["pos"], s["rotary"], s["qw"], s["kw"], eps=1e-6))
    if op == "prompt_attention":
        if case["lse"]:
            return list(ck.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"],
                                            return_lse=True))
        return [ck.prompt_attention(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], causal=case["causal"])]
    cache = s["cache"]
    if op == "cache_write":
        cache.prefill_begin(s["lens"])
        cache.prefill_layer(0, s["k"], s["v"])
        r = cache.read_layer(0)
    else:
        r = cache.read_layer(0, dtype=DTYPES[case["dtype"]])
    return [r["k"], r["v"], r["positions"]]


def run(state):
    if own:
        return _own(state)
    return {"qk_rotary": _plain_rotary, "prompt_attention": _plain_attention, "cache_write": _plain_write,
            "cache_read": _plain_read}[state["case"]["op"]](state)


# ---------------------------------------------------------------- work

def _pairs(lq, lk, causal):
    """(query, key) pairs that the mask leaves."""
    total = 0
    for a, b in zip(lq, lk):
        if not causal:
            total += a * b
            continue
        first = max(1, b - a + 1)                  # keys of the first query that has any
        rows = min(a, b)
        total += rows * (first + b) // 2
    return total


def work(case):
    op, d = case["op"], case["d"]
    if op == "qk_rotary":
        n, H = case["tokens"], case["Hq"] + case["Hkv"]
        return {"bytes": 2 * 2 * n * H * d + 4 * n + 4 * case["rot"] + (4 * d if case["norm"] else 0),
                "flops": n * H * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    if op == "prompt_attention":
        lq, lk = _lens(case["lens_q"]), _lens(case["lens_k"])
        nbytes = 2 * 2 * sum(lq) * case["Hq"] * d + 2 * 2 * sum(lk) * case["Hkv"] * d
        nbytes += 4 * sum(lq) * case["Hq"] if case["lse"] else 0
        return {"bytes": nbytes, "flops": 4 * d * case["Hq"] * _pairs(lq, lk, case["causal"])}
    lens = _lens(case["lens"])
    row = 2 * case["Hkv"] * d                      # values of one token, K and V
    stored = sum(max(0, n - case["W"]) + 2 * min(n, case["W"]) for n in lens) * row
    both = 2 * sum(lens) * row
    nbytes = stored + both + 4 * sum(lens)         # cache read, packed K/V written
    flops = sum(lens) * row
    if op == "cache_write":                        # packed K/V read, cache written, both once more
        nbytes, flops = nbytes + stored + both, 4 * flops
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------- 64 bits

def _exact_rotary(case, s):
    rot, out, f = case["rot"], [], float(case["factor"])
    pair = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    log_base = math.log(10000.0) + (rot / (rot - 2.0) * math.log(f) if case["scaling"] == "ntk" else 0.0)
    freq, mscale = torch.exp(-log_base * 2.0 * pair / rot), 1.0
    if case["scaling"] == "linear":
        freq = freq / f
    elif case["scaling"] == "yarn":
        # turns within the trained length: below 1 interpolated, above 32 kept, between them a ramp
        ramp = ((4096.0 / (2.0 * math.pi) * freq - 1.0) / 31.0).clamp(0.0, 1.0)
        freq, mscale = freq * (ramp + (1.0 - ramp) / f), 1.0 + math.log(f) / 10.0
    angle = torch.outer(s["pos"].to(torch.float64), freq)
    turn = torch.polar(torch.full_like(angle, mscale), angle)[:, None, :]
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.to(torch.float64)
        if w is not None:
            x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * w.to(torch.float64)
        head, rest = x[..., :rot], x[..., rot:]
        if case["interleaved"]:
            z = torch.view_as_complex(head.reshape(*head.shape[:-1], rot // 2, 2).contiguous()) * turn
            head = torch.view_as_real(z).reshape(head.shape)
        else:
            z = torch.complex(head[..., : rot // 2].contiguous(), head[..., rot // 2:].contiguous()) * turn
            head = torch.cat([z.real, z.imag], -1)
        out.append(torch.cat([head, rest], -1))
    return out


def _exact_attention(case, s):
    lq, lk, G = _lens(case["lens_q"]), _lens(case["lens_k"]), case["Hq"] // case["Hkv"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    q0 = k0 = 0
    for a, b in zip(lq, lk):
        for h in range(case["Hq"]):
            k, v = (s[x][k0:k0 + b, h // G].to(torch.float64) for x in ("k", "v"))
            for i in range(0, a, 2048):
                e = min(a, i + 2048)
                z = s["q"][q0 + i:q0 + e, h].to(torch.float64) @ k.T / math.sqrt(case["d"])
                if case["causal"]:
                    r = torch.arange(i, e, device="cuda")[:, None] + (b - a)
                    z = torch.where(torch.arange(b, device="cuda")[None, :] > r, -math.inf, z)
                w = torch.logsumexp(z, -1) if b else torch.full((e - i,), -math.inf, dtype=torch.float64, device="cuda")
                some = (w > -math.inf)[:, None]
                out[q0 + i:q0 + e, h] = torch.where(some, torch.exp(z - torch.where(some, w[:, None], 0.0)) @ v, 0.0)
                lse[q0 + i:q0 + e, h] = w
        q0, k0 = q0 + a, k0 + b
    return [out, lse] if case["lse"] else [out]


def _exact_cache(case, s):
    got, W, at, t = [], case["W"], [], 0
    for name in ("k", "v"):
        rows, t = [], 0
        for b, n in enumerate(s["lens"]):
            if case["op"] == "cache_write":
                x = s[name][t:t + n].to(torch.float16).to(torch.float64)
                scale = (x.abs().amax(0).to(torch.float32) / 127).to(torch.float64)
                scale = torch.where(scale > 0, scale, 1.0)
                old = torch.clamp(torch.round(x / scale), -127, 127) * scale
            else:
                x = s[name + "16"][t:t + n].to(torch.float64)
                old = s[name + "_codes"][t:t + n].to(torch.float64) * s[name + "_scale"][b].to(torch.float64)
            cut = max(0, n - W)
            rows.append(torch.cat([old[:cut], x[cut:]]))
            t += n
        got.append(torch.cat(rows))
    for n in s["lens"]:
        at.append(torch.arange(n, dtype=torch.int32, device="cuda"))
    return got + [torch.cat(at)]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "qk_rotary":
        return _exact_rotary(case, s)
    if case["op"] == "prompt_attention":
        return _exact_attention(case, s)
    return _exact_cache(case, s)
