"""Cases of the position rotation, the per-head norm of queries and keys, the paged
key/value cache and the attention that reads it: inputs, plain forms in elementary
torch operations, the framework's own calls, and the definitions in 64 bits.

Operators (names of the cases' "op"):
  rotary           positions rotated into q and k (interleaved or half layout, part of
                   the head, scaled for long contexts), optionally after an RMS norm of
                   every head ("norm")
  rotary_backward  the gradients of that with respect to q, k and the norm's weights
  append           new keys and values written into a paged cache, the rotation (and the
                   norm) applied on the way, the queries rotated in the same call
  attend           queries of one or many new tokens a sequence over the paged cache:
                   causal, sliding window or none, grouped heads, capped scores
"""
import math

import torch

own = False

INT = torch.int32
DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------ cases
def listed():
    return [
        # One decoding step's rotation of eight sequences far into a long context: latency.
        dict(name="rotary_token", op="rotary", dtype="bf16", batch=8, seq=1, q_heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=True, scaling="linear", factor=4.0, norm=False, far=131071),
        # The prompt of the causal 512-key window layer (32 query, 8 KV heads), read from the
        # projection's token-major layout and written head-major for the attention.
        dict(name="rotary_prompt", op="rotary", dtype="bf16", batch=1, seq=32768, q_heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=True, scaling="none", factor=1.0, norm=False, far=0),
        # A training prompt with normed heads, half layout, ragged length.
        dict(name="norm_prompt", op="rotary", dtype="bf16", batch=2, seq=8191, q_heads=32, kv_heads=8, dim=128,
             rotary=128, interleaved=False, scaling="yarn", factor=8.0, norm=True, far=0),
        # 32-bit check runs of a small encoder, a quarter of the head rotated.
        dict(name="norm_fp32", op="rotary", dtype="fp32", batch=2, seq=1021, q_heads=12, kv_heads=12, dim=64,
             rotary=16, interleaved=False, scaling="ntk", factor=2.0, norm=True, far=0),
        # Training step of a 12-head encoder: the gradient back through the rotation alone.
        dict(name="rotary_backward", op="rotary_backward", dtype="bf16", batch=2, seq=4099, q_heads=12, kv_heads=12,
             dim=64, rotary=32, interleaved=False, scaling="yarn", factor=4.0, norm=False, far=0),
        # Training step of the 32/8-head decoder layer: through rotation and norm, the weights'
        # gradients included; the upstream gradients are the attention backward's 32-bit ones.
        dict(name="norm_backward", op="rotary_backward", dtype="bf16", batch=1, seq=16384, q_heads=32, kv_heads=8,
             dim=128, rotary=128, interleaved=True, scaling="none", factor=1.0, norm=True, far=0),
        # One decoding step of 64 sequences: one token each into pages of 64.
        dict(name="append_token", op="append", dtype="bf16", batch=64, tokens=1, ragged=False, q_heads=32, kv_heads=8,
             dim=128, rotary=128, interleaved=True, scaling="none", factor=1.0, norm=False, page=64, length=4000),
        # Prompts of different lengths into pages of 48, normed heads.
        dict(name="append_prompt", op="append", dtype="bf16", batch=7, tokens=2500, ragged=True, q_heads=32, kv_heads=8,
             dim=128, rotary=64, interleaved=False, scaling="linear", factor=2.0, norm=True, page=48, length=4096),
        # One decoding step of four sequences in a 512-key window layer: latency.
        dict(name="attend_token_window", op="attend", dtype="bf16", batch=4, tokens=1, ragged=False, q_heads=32,
             kv_heads=8, dim=128, window=511, softcap=0.0, page=64, length=20000),
        # One decoding step of 32 sequences of very different lengths in a layer without a
        # window, scores capped.
        dict(name="attend_token_long", op="attend", dtype="bf16", batch=32, tokens=1, ragged=True, q_heads=32,
             kv_heads=8, dim=128, window=-1, softcap=30.0, page=16, length=32000),
        # Prompt chunks of different lengths in a 512-key window layer.
        dict(name="attend_chunk_window", op="attend", dtype="bf16", batch=6, tokens=2048, ragged=True, q_heads=32,
             kv_heads=8, dim=128, window=511, softcap=0.0, page=64, length=6000),
        # A 4096-token chunk of one long prompt in a layer without a window.
        dict(name="attend_chunk_long", op="attend", dtype="bf16", batch=1, tokens=4096, ragged=False, q_heads=32,
             kv_heads=8, dim=128, window=-1, softcap=0.0, page=128, length=16384),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rotary", "rotary_backward", "append", "attend", "attend"])
    dtype = "fp32" if rng.random() < 0.2 else "bf16"
    kv = rng.choice([1, 2, 4, 8, 12])
    group = rng.choice([1, 2, 3, 4, 5, 8])
    while kv * group > 40:
        group = rng.choice([1, 2, 3, 4])
    dim = rng.choice([64, 128])
    if op in ("rotary", "rotary_backward", "append"):
        scaling = rng.choice(["none", "linear", "ntk", "yarn"])
        base = dict(op=op, dtype=dtype, q_heads=kv * group, kv_heads=kv, dim=dim,
                    rotary=rng.choice([dim, dim, dim // 2, 16, 48]), interleaved=rng.random() < 0.5,
                    scaling=scaling, factor=1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0, 32.0]),
                    norm=rng.random() < 0.5)
        if op == "append":
            batch = _log_int(rng, 1, 128)
            tokens = rng.choice([1, 1, _log_int(rng, 1, max(1, 16384 // batch))])
            base.update(batch=batch, tokens=tokens, ragged=tokens > 1 and rng.random() < 0.5,
                        page=rng.choice([16, 32, 48, 64, 128]), length=tokens + _log_int(rng, 1, 4096))
        else:
            batch = _log_int(rng, 1, 8)
            base.update(batch=batch, seq=_log_int(rng, 1, 16384 // batch),
                        far=rng.choice([0, 0, _log_int(rng, 1, 1000000)]))
        return base
    batch = _log_int(rng, 1, 48)
    if rng.random() < 0.5:                                # single tokens, or a few for a check of guesses
        tokens = rng.choice([1, 1, 1, rng.randint(2, 8)])
        length = _log_int(rng, 1, min(32000, 1000000 // (batch * kv // 4 + 1)))
    else:
        tokens = _log_int(rng, 9, max(9, 4096 // batch))
        length = _log_int(rng, 1, 8192)
    if dtype == "fp32":                                   # check runs
        batch, tokens, length = min(batch, 8), min(tokens, 256), min(length, 4096)
    return dict(op="attend", dtype=dtype, batch=batch, tokens=tokens, ragged=rng.random() < 0.5, q_heads=kv * group,
                kv_heads=kv, dim=dim, window=rng.choice([-1, _log_int(rng, 1, 4096) - 1]),
                softcap=rng.choice([0.0, 0.0, 30.0, 50.0]), page=rng.choice([16, 32, 48, 64, 128]),
                length=tokens + length)


# ------------------------------------------------------------------ inputs
def _frequencies(case):
    """Radians a position for each rotated pair, and the amplitude, in 64 bits."""
    half = case["rotary"] // 2
    j = torch.arange(half, dtype=torch.float64)
    base, f = 10000.0, case["factor"]
    if case["scaling"] == "ntk":
        base = base * f ** (case["rotary"] / (case["rotary"] - 2))
    freq = base ** (-2.0 * j / case["rotary"])
    if case["scaling"] == "linear":
        return freq / f, 1.0
    if case["scaling"] == "yarn":
        turns = 4096 * freq / (2 * math.pi)               # full turns over the original length
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
        return freq * keep + freq / f * (1 - keep), 0.1 * math.log(f) + 1.0
    return freq, 1.0


def _ragged(case):
    """New tokens and lengths (new tokens included) of every sequence: the case's own, so
    that outputs of every seed have one shape (the seed gives their order)."""
    B, m, length = case["batch"], case["tokens"], case["length"]
    if not case["ragged"]:
        return [m] * B, [length] * B
    u = [(i * 0.6180339887498949 + 0.31) % 1.0 for i in range(B)]
    w = [(i * 0.4142135623730951 + 0.17) % 1.0 for i in range(B)]
    new = [m] + [max(1, math.ceil(m * x)) for x in u[1:]]
    old = [length - m] + [int((length - m) * x * x) for x in w[1:]]
    return new, [a + b for a, b in zip(old, new)]


def _paged(case, g, fill):
    B, Hkv, D, ps = case["batch"], case["kv_heads"], case["dim"], case["page"]
    new, lens = (torch.tensor(x) for x in _ragged(case))
    order = torch.randperm(B, generator=g)
    new, lens = new[order], lens[order]
    per = (case["length"] + ps - 1) // ps
    used = (lens + ps - 1) // ps
    pages = int(used.sum()) + 3
    order = torch.randperm(pages, generator=g)            # pages lie anywhere in the pool
    first = torch.cumsum(used, 0) - used
    col = torch.arange(per)
    at = first[:, None] + col[None, :]
    table = torch.where(col[None, :] < used[:, None], order[at.clamp(max=pages - 1)], torch.full((), -1))
    dt = DTYPES[case["dtype"]]
    shape = (pages, Hkv, ps, D)
    k_pages = fill(shape).to(dt) if fill else torch.zeros(shape, dtype=dt, device="cuda")
    v_pages = fill(shape).to(dt) if fill else torch.zeros(shape, dtype=dt, device="cuda")
    cu = torch.zeros(B + 1, dtype=torch.int64)
    cu[1:] = torch.cumsum(new, 0)
    return dict(k_pages=k_pages, v_pages=v_pages, table=table.to(INT).cuda(), lens=lens.to(INT).cuda(),
                cu=cu.to(INT).cuda(), total=int(cu[-1]), max_new=int(new.max()))


def prepare(case, seed):
    g = torch.Generator("cpu").manual_seed(seed * 7919 + 17)
    gpu = torch.Generator("cuda").manual_seed(seed * 7919 + 18)

    def normal(shape):
        return torch.randn(shape, generator=gpu, device="cuda")

    dt = DTYPES[case["dtype"]]
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["dim"]
    s = dict(case=case)
    if case["op"] != "attend":
        freq, amp = _frequencies(case)
        s.update(freq=freq, amp=amp, freq_gpu=freq.cuda(), eps=1e-6 if case["norm"] else None,
                 q_weight=None, k_weight=None)
        if case["norm"]:
            s["q_weight"] = 1 + 0.1 * normal((D,))
            s["k_weight"] = 1 + 0.1 * normal((D,))
    if case["op"] in ("rotary", "rotary_backward"):
        B, n = case["batch"], case["seq"]
        # the projection's output, token-major: q, k and v of a token side by side
        qkv = (normal((B, n, Hq + 2 * Hkv, D)) * 1.5).to(dt)
        s["q"] = qkv[:, :, :Hq].transpose(1, 2)
        s["k"] = qkv[:, :, Hq:Hq + Hkv].transpose(1, 2)
        start = torch.randint(case["far"] // 2, case["far"] + 1, (B, 1), generator=g) if case["far"] else None
        s["positions"] = (start + torch.arange(n)[None, :]).to(INT).cuda() if case["far"] else None
        if case["op"] == "rotary_backward":
            s["dq_out"] = normal((B, Hq, n, D))
            s["dk_out"] = normal((B, Hkv, n, D))
    elif case["op"] == "append":
        s.update(_paged(case, g, None))
        qkv = (normal((s["total"], Hq + 2 * Hkv, D)) * 1.5).to(dt)
        s["q"], s["k"], s["v"] = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    else:
        s.update(_paged(case, g, normal))
        s["q"] = (normal((s["total"], Hq, D)) * 1.5).to(dt)
    if own:
        from sliding_window_global_b200 import PagedCache, Rotary
        if case["op"] != "attend":
            s["rotary"] = Rotary(D, rotary_dim=case["rotary"], interleaved=case["interleaved"], frequencies=s["freq"],
                                 amplitude=s["amp"])
        if case["op"] in ("append", "attend"):
            s["cache"] = PagedCache(s["k_pages"], s["v_pages"])
    return s


# ------------------------------------------------------------------ plain forms
def _angles(s, positions):
    a = positions.double()[..., None] * s["freq_gpu"]
    return (a.cos() * s["amp"]).float(), (a.sin() * s["amp"]).float()


def _rotate(case, x, c, sn):
    """x [..., D] in 32 bits; c, sn broadcast against [..., rotary / 2]."""
    R = case["rotary"]
    y = x.clone()
    if case["interleaved"]:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        y[..., 0:R:2] = a * c - b * sn
        y[..., 1:R:2] = a * sn + b * c
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        y[..., :R // 2] = a * c - b * sn
        y[..., R // 2:R] = a * sn + b * c
    return y


def _unit(s, x):
    """RMS norm of the last axis: the normed rows and 1 / rms."""
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"])
    return x * r, r


def _forward_one(s, x, w, c, sn):
    y = x.float()
    if s["eps"] is not None:
        y = _unit(s, y)[0] * w
    return _rotate(s["case"], y, c, sn).to(x.dtype)


def _backward_one(s, dy, x, w, c, sn):
    h = _rotate(s["case"], dy.float(), c, -sn)
    if s["eps"] is None:
        return h.to(x.dtype), None
    u, r = _unit(s, x.float())
    dw = (h.double() * u.double()).sum((0, 1, 2)).float()
    h = h * w
    return (r * (h - u * (h * u).mean(-1, keepdim=True))).to(x.dtype), dw


def _token_positions(s):
    t = torch.arange(s["total"], device="cuda", dtype=INT)
    b = torch.searchsorted(s["cu"][1:], t, right=True)
    return b, s["lens"][b] - s["cu"][b + 1] + t


def _plain_attend(s):
    case = s["case"]
    B, Hkv, D, ps = case["batch"], case["kv_heads"], case["dim"], case["page"]
    G, m, T = case["q_heads"] // Hkv, s["max_new"], s["total"]
    length = case["length"] if case["window"] < 0 else min(case["length"], case["window"] + m)
    b, pos = _token_positions(s)
    i = torch.arange(T, device="cuda") - s["cu"][b]
    q = torch.zeros((B, m, Hkv * G, D), device="cuda")
    q[b, i] = s["q"].float()
    q = q.view(B, m, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * m, D)
    # the last `length` positions of every sequence, in order
    j = s["lens"][:, None] - length + torch.arange(length, device="cuda")[None, :]
    page = torch.gather(s["table"], 1, j.clamp(min=0).long() // ps).clamp(min=0)
    slot = j.clamp(min=0).long() % ps
    k = s["k_pages"][page.long(), :, slot].float().transpose(1, 2)         # [B, Hkv, length, D]
    scores = torch.matmul(q, k.transpose(2, 3)).mul_(1.0 / math.sqrt(D))
    del k
    if case["softcap"] > 0:
        scores = scores.div_(case["softcap"]).tanh_().mul_(case["softcap"])
    at = s["lens"][:, None] - (s["cu"][1:] - s["cu"][:-1])[:, None] + torch.arange(m, device="cuda")[None, :]
    hide = (j[:, None, :] < 0) | (j[:, None, :] > at[:, :, None])           # [B, m, length]
    if case["window"] >= 0:
        hide |= j[:, None, :] < at[:, :, None] - case["window"]
    scores = scores.view(B, Hkv, G, m, length).masked_fill_(hide[:, None, None], -math.inf).view(B, Hkv, G * m, length)
    top = scores.amax(-1, keepdim=True)
    top = torch.where(torch.isfinite(top), top, torch.zeros_like(top))      # padded rows see nothing
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    v = s["v_pages"][page.long(), :, slot].float().transpose(1, 2)
    out = torch.matmul(p, v) / total.clamp(min=1e-30)
    lse = top + total.log()
    out = out.view(B, Hkv, G, m, D).permute(0, 3, 1, 2, 4).reshape(B, m, Hkv * G, D)
    lse = lse.view(B, Hkv, G, m).permute(0, 3, 1, 2).reshape(B, m, Hkv * G)
    return out[b, i].to(s["q"].dtype), lse[b, i]


# ------------------------------------------------------------------ one pass
def run(s):
    case = s["case"]
    op = case["op"]
    if own:
        if op == "rotary":
            return s["rotary"].forward(s["q"], s["k"], positions=s["positions"], norm_eps=s["eps"],
                                       q_weight=s["q_weight"], k_weight=s["k_weight"])
        if op == "rotary_backward":
            return s["rotary"].backward(s["dq_out"], s["dk_out"], s["q"], s["k"], positions=s["positions"],
                                        norm_eps=s["eps"], q_weight=s["q_weight"], k_weight=s["k_weight"])
        cu = s["cu"] if case["ragged"] else None
        if op == "append":
            q = s["cache"].append(s["k"], s["v"], s["lens"], s["table"], q=s["q"], cu_tokens=cu, rotary=s["rotary"],
                                  norm_eps=s["eps"], q_weight=s["q_weight"], k_weight=s["k_weight"])
            return q, s["k_pages"], s["v_pages"]
        return s["cache"].attend(s["q"], s["lens"], s["table"], cu_tokens=cu, max_tokens=s["max_new"],
                                 max_len=case["length"], window=None if case["window"] < 0 else case["window"],
                                 softcap=case["softcap"])
    if op in ("rotary", "rotary_backward"):
        n = case["seq"]
        positions = s["positions"] if s["positions"] is not None else torch.arange(n, device="cuda")[None, :]
        c, sn = _angles(s, positions)
        c, sn = c[:, None], sn[:, None]                                     # [B, 1, n, rotary / 2]
        if op == "rotary":
            return (_forward_one(s, s["q"], s["q_weight"], c, sn).contiguous(),
                    _forward_one(s, s["k"], s["k_weight"], c, sn).contiguous())
        dq, dwq = _backward_one(s, s["dq_out"], s["q"], s["q_weight"], c, sn)
        dk, dwk = _backward_one(s, s["dk_out"], s["k"], s["k_weight"], c, sn)
        return (dq, dk) if s["eps"] is None else (dq, dk, dwq, dwk)
    if op == "append":
        b, pos = _token_positions(s)
        c, sn = _angles(s, pos)
        c, sn = c[:, None], sn[:, None]
        page = s["table"][b, (pos // case["page"]).long()].long()
        slot = (pos % case["page"]).long()
        s["k_pages"][page, :, slot] = _forward_one(s, s["k"], s["k_weight"], c, sn)
        s["v_pages"][page, :, slot] = s["v"]
        return _forward_one(s, s["q"], s["q_weight"], c, sn), s["k_pages"], s["v_pages"]
    return _plain_attend(s)


# ------------------------------------------------------------------ the definitions in 64 bits
def _exact_rotary(case, x, positions, freq, amp):
    """x [..., T, D] in 64 bits rotated at positions [T], as complex numbers."""
    R = case["rotary"]
    turn = torch.polar(torch.full_like(positions[:, None] * freq, amp), positions[:, None] * freq)
    part = x[..., :R]
    z = (torch.view_as_complex(part.unflatten(-1, (R // 2, 2)).contiguous()) if case["interleaved"]
         else torch.complex(part[..., :R // 2].contiguous(), part[..., R // 2:].contiguous()))
    z = z * turn
    part = torch.view_as_real(z).flatten(-2) if case["interleaved"] else torch.cat([z.real, z.imag], -1)
    return torch.cat([part, x[..., R:]], -1)


def _exact_heads(case, s, x, w, positions):
    x = x.double()
    if case["norm"]:
        x = x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / case["dim"] + s["eps"]) * w.double()
    return _exact_rotary(case, x, positions, s["freq_gpu"], s["amp"])


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op in ("rotary", "rotary_backward"):
        outs, weights = [], []
        for name in ("q", "k"):
            x, w = s[name], s[name + "_weight"]
            if op == "rotary_backward":
                x = x.double().requires_grad_(True)
                w = None if w is None else w.double().requires_grad_(True)
            ys = []
            for b in range(case["batch"]):
                pos = (torch.arange(case["seq"], device="cuda") if s["positions"] is None else s["positions"][b])
                ys.append(_exact_heads(case, s, x[b], w, pos.double()))
            y = torch.stack(ys)
            if op == "rotary":
                outs.append(y)
                continue
            grads = torch.autograd.grad(y, [x] if w is None else [x, w], s["d" + name + "_out"].double())
            outs.append(grads[0])
            weights += grads[1:]
        return tuple(outs + weights)
    lens, cu, table = s["lens"].tolist(), s["cu"].tolist(), s["table"].long()
    if op == "append":
        k_pages, v_pages, q_out = s["k_pages"].double(), s["v_pages"].double(), []
        for b in range(case["batch"]):
            rows = slice(cu[b], cu[b + 1])
            pos = torch.arange(lens[b] - (cu[b + 1] - cu[b]), lens[b], device="cuda")
            page, slot = table[b, pos // case["page"]], pos % case["page"]
            k = _exact_heads(case, s, s["k"][rows].transpose(0, 1), s["k_weight"], pos.double())
            k_pages[page, :, slot] = k.transpose(0, 1)
            v_pages[page, :, slot] = s["v"][rows].double()
            q_out.append(_exact_heads(case, s, s["q"][rows].transpose(0, 1), s["q_weight"], pos.double()).transpose(0, 1))
        return torch.cat(q_out), k_pages, v_pages
    outs, lses = [], []
    G, D = case["q_heads"] // case["kv_heads"], case["dim"]
    for b in range(case["batch"]):
        L, new = lens[b], cu[b + 1] - cu[b]
        lo = 0 if case["window"] < 0 else max(0, L - new - case["window"])
        j = torch.arange(lo, L, device="cuda")
        page, slot = table[b, j // case["page"]], j % case["page"]
        out = torch.empty((new, case["q_heads"], D), dtype=torch.float64, device="cuda")
        lse = torch.empty((new, case["q_heads"]), dtype=torch.float64, device="cuda")
        i = torch.arange(L - new, L, device="cuda")
        seen = j[None, :] <= i[:, None]
        if case["window"] >= 0:
            seen &= i[:, None] - j[None, :] <= case["window"]
        for h in range(case["q_heads"]):
            k = s["k_pages"][page, h // G, slot].double()
            v = s["v_pages"][page, h // G, slot].double()
            x = s["q"][cu[b]:cu[b + 1], h].double() @ k.T / D ** 0.5
            if case["softcap"] > 0:
                x = case["softcap"] * torch.tanh(x / case["softcap"])
            x = x.masked_fill(~seen, -math.inf)
            lse[:, h] = torch.logsumexp(x, -1)
            out[:, h] = torch.softmax(x, -1) @ v
        outs.append(out)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses)


# ------------------------------------------------------------------ work
def work(case):
    e = 2 if case["dtype"] == "bf16" else 4
    Hq, Hkv, D = case["q_heads"], case["kv_heads"], case["dim"]
    if case["op"] == "rotary":
        rows = case["batch"] * case["seq"] * (Hq + Hkv)
        return {"bytes": rows * D * e * 2, "flops": rows * (3 * case["rotary"] + (4 * D if case["norm"] else 0))}
    if case["op"] == "rotary_backward":
        rows = case["batch"] * case["seq"] * (Hq + Hkv)
        # the upstream gradient in 32 bits, the gradient out, with a norm also its input
        moved = rows * D * (4 + e + (e if case["norm"] else 0))
        return {"bytes": moved, "flops": rows * (3 * case["rotary"] + (14 * D if case["norm"] else 0))}
    new, lens = _ragged(case)
    T = sum(new)
    if case["op"] == "append":
        rows = T * (Hq + 2 * Hkv)
        return {"bytes": rows * D * e * 2,
                "flops": T * (Hq + Hkv) * (3 * case["rotary"] + (4 * D if case["norm"] else 0))}
    keys, pairs = 0.0, 0.0
    for a, t in zip(lens, new):
        w = a if case["window"] < 0 else case["window"] + 1
        keys += min(a, w - 1 + t)
        first = a - t + 1                                 # keys that the first new token could see
        full = max(0.0, min(t, a - w))                    # tokens whose window is full
        rest = t - full
        pairs += full * w + rest * (first + (rest - 1) / 2) if first < w else t * w
    return {"bytes": keys * Hkv * D * 2 * e + T * Hq * (D * e * 2 + 4), "flops": 4 * D * Hq * pairs}
