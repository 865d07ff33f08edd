"""Rotation and head norm of queries and keys, and their gradients: against the
definition in 64 bits and against differences of it (GPU), the frequencies and the
refusals (CPU)."""
import ctypes
import math

import pytest
import torch

from sliding_window_global_b200 import Rotary, SwaError, load_library, rotary_frequencies
from sliding_window_global_b200.rotary import HeadNorm, RotaryArgs, RotaryBackwardArgs, Rotation

INVALID, UNSUPPORTED = 1, 2
BF16, FP32 = torch.bfloat16, torch.float32


# ------------------------------------------------------------------ the definition
def rotated(x, pos, freq, amp, interleaved):
    """x [B, H, n, D] fp64 rotated at positions [B, n]."""
    R = 2 * freq.numel()
    ang = pos.double()[:, None, :, None] * freq
    c, s = amp * ang.cos(), amp * ang.sin()
    if interleaved:
        a, b = x[..., 0:R:2], x[..., 1:R:2]
        part = torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    else:
        a, b = x[..., :R // 2], x[..., R // 2:R]
        part = torch.cat([a * c - b * s, a * s + b * c], -1)
    return torch.cat([part, x[..., R:]], -1)


def normed(x, eps, w):
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w.double()


def definition(x, pos, freq, amp, interleaved, eps, w):
    return rotated(x if eps is None else normed(x, eps, w), pos, freq, amp, interleaved)


# ------------------------------------------------------------------ CPU
def test_frequencies():
    f, a = rotary_frequencies(128)
    assert a == 1.0 and f.dtype == torch.float64 and f.shape == (64,)
    assert f[0] == 1.0 and torch.allclose(f, 10000.0 ** (-torch.arange(64).double() / 64), rtol=1e-14, atol=0)
    lin, a = rotary_frequencies(128, scaling="linear", factor=4.0)
    assert a == 1.0 and torch.equal(lin, f / 4)
    ntk, a = rotary_frequencies(64, scaling="ntk", factor=8.0)
    plain = rotary_frequencies(64)[0]
    assert a == 1.0 and ntk[0] == 1.0 and abs(ntk[-1] / (plain[-1] / 8) - 1) < 1e-12   # the slowest is interpolated
    yarn, a = rotary_frequencies(128, scaling="yarn", factor=8.0, original_length=4096)
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(yarn[turns >= 32], f[turns >= 32])
    assert torch.allclose(yarn[turns <= 1], f[turns <= 1] / 8, rtol=1e-14, atol=0)
    assert abs(a - (0.1 * math.log(8.0) + 1)) < 1e-15
    for bad in (dict(rotary_dim=3), dict(rotary_dim=0), dict(rotary_dim=2, scaling="ntk"), dict(rotary_dim=16, factor=0),
                dict(rotary_dim=16, scaling="other")):
        with pytest.raises(ValueError):
            rotary_frequencies(**bad)


def test_constructor_refusals():
    for bad in (dict(head_dim=96), dict(head_dim=64, rotary_dim=24), dict(head_dim=64, rotary_dim=128),
                dict(head_dim=64, rotary_dim=-16), dict(head_dim=64, amplitude=math.inf),
                dict(head_dim=64, amplitude=0.0), dict(head_dim=64, frequencies=torch.ones(31)),
                dict(head_dim=64, frequencies=torch.full((32,), math.nan))):
        with pytest.raises(ValueError):
            Rotary(**bad)
    assert Rotary(64, rotary_dim=0).rotary_dim == 0


def test_cpu_tensors_are_refused():
    r = Rotary(64)
    with pytest.raises(ValueError):
        r.forward(torch.zeros(1, 2, 3, 64))
    with pytest.raises(ValueError):
        r.backward(torch.zeros(1, 2, 3, 64))


_FREQ = (ctypes.c_double * 32)(*([0.5] * 32))
_BUF = ctypes.create_string_buffer(8192)
_PTR = (ctypes.addressof(_BUF) + 255) & ~255          # never read: every call below is refused on the host


def _args(cls, **kw):
    base = dict(batch=1, seq_len=2, num_q_heads=2, num_kv_heads=1, head_dim=64, dtype=0,
                rotation=Rotation(64, 0, ctypes.addressof(_FREQ), 1.0), head_norm=HeadNorm(0, 0, None, None, 0))
    names = ("q", "k", "q_out", "k_out") if cls is RotaryArgs else ("q", "k", "dq_out", "dk_out", "dq", "dk")
    for n in names:
        base[n] = _PTR
        base[n + "_stride0"], base[n + "_stride1"], base[n + "_stride2"] = 256, 128, 64
    base.update(kw)
    return cls(**base)


def _rot(dim=64, inter=0, freq=ctypes.addressof(_FREQ), amp=1.0):
    return Rotation(dim, inter, freq, amp)


COMMON = [
    (dict(batch=-1), INVALID), (dict(seq_len=-1), INVALID), (dict(num_q_heads=0), INVALID),
    (dict(num_kv_heads=-1), INVALID), (dict(head_dim=0), INVALID), (dict(head_dim=96), UNSUPPORTED),
    (dict(dtype=5), INVALID), (dict(positions=_PTR + 2), INVALID),
    (dict(batch=2 ** 20, seq_len=2 ** 20), UNSUPPORTED),
    (dict(rotation=_rot(dim=24)), UNSUPPORTED), (dict(rotation=_rot(dim=80)), INVALID),
    (dict(rotation=_rot(dim=-16)), INVALID), (dict(rotation=_rot(inter=2)), INVALID),
    (dict(rotation=_rot(freq=None)), INVALID), (dict(rotation=_rot(amp=math.inf)), INVALID),
    (dict(head_norm=HeadNorm(2, 0, None, None, 0)), INVALID), (dict(head_norm=HeadNorm(1, -1.0, None, None, 0)), INVALID),
    (dict(head_norm=HeadNorm(1, math.nan, None, None, 0)), INVALID),
    (dict(head_norm=HeadNorm(1, 0, _PTR + 4, None, 0)), INVALID), (dict(head_norm=HeadNorm(1, 0, None, None, 9)), INVALID),
]


@pytest.mark.parametrize("bad,status", COMMON + [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(q_out=None), INVALID), (dict(k_out=_PTR + 8), INVALID),
    (dict(q_stride1=4), INVALID), (dict(k_stride2=-64), INVALID),
    (dict(q_out_stride2=0), INVALID), (dict(q_out_stride1=64), INVALID),     # an output that overlaps itself
])
def test_forward_refusals(bad, status):
    assert load_library().swa_rotary_forward(ctypes.byref(_args(RotaryArgs, **bad)), None) == status


@pytest.mark.parametrize("bad,status", COMMON + [
    (dict(dq_out=None), INVALID), (dict(dk=None), INVALID), (dict(dq=_PTR + 4), INVALID),
    (dict(dtype=1, grad_dtype=0, out_dtype=1), INVALID), (dict(dtype=1, grad_dtype=1, out_dtype=0), INVALID),
    (dict(grad_dtype=3), INVALID), (dict(dq_stride1=64), INVALID), (dict(dq_out_stride2=-8), INVALID),
    (dict(head_norm=HeadNorm(1, 0, None, None, 0), q=None), INVALID),
    (dict(head_norm=HeadNorm(1, 0, None, None, 0), k=None), INVALID),
    (dict(head_norm=HeadNorm(1, 0, _PTR, None, 0), dq_weight=_PTR), INVALID),         # no workspace
    (dict(head_norm=HeadNorm(1, 0, _PTR, None, 0), dq_weight=_PTR, workspace=_PTR, workspace_bytes=256), INVALID),
])
def test_backward_refusals(bad, status):
    assert load_library().swa_rotary_backward(ctypes.byref(_args(RotaryBackwardArgs, **bad)), None) == status


def test_null_and_empty_calls():
    lib = load_library()
    assert lib.swa_rotary_forward(None, None) == INVALID
    assert lib.swa_rotary_backward(None, None) == INVALID
    assert lib.swa_rotary_workspace_bytes(None) == 0
    empty = _args(RotaryArgs, seq_len=0, q=None, k=None, q_out=None, k_out=None)
    assert lib.swa_rotary_forward(ctypes.byref(empty), None) == 0
    a = _args(RotaryBackwardArgs)
    assert lib.swa_rotary_workspace_bytes(ctypes.byref(a)) == 0              # no norm, nothing to add up
    a = _args(RotaryBackwardArgs, head_norm=HeadNorm(1, 0, _PTR, _PTR, 0), dq_weight=_PTR, dk_weight=_PTR)
    assert lib.swa_rotary_workspace_bytes(ctypes.byref(a)) >= 2 * 64 * 4


# ------------------------------------------------------------------ GPU
def _heads(B, H, n, D, dtype, layout, g):
    """Random head rows [B, H, n, D]: contiguous, or a slice of a token-major projection."""
    x = torch.randn((B, n, H + 3, D) if layout == "tokens" else (B, H, n, D), generator=g) * 1.5
    x = x.to(dtype).cuda()
    return x[:, :, 2:2 + H].transpose(1, 2) if layout == "tokens" else x


# name, dtype, B, Hq, Hkv, n, D, R, interleaved, norm, layout, scaling, far
CASES = [
    ("one_token", BF16, 1, 1, 1, 1, 128, 128, True, False, "heads", "none", 0),
    ("half_ragged", BF16, 2, 5, 1, 37, 64, 64, False, False, "tokens", "linear", 1000000),
    ("inter_part", BF16, 3, 7, 7, 19, 128, 48, True, True, "tokens", "yarn", 131072),
    ("half_part", BF16, 1, 32, 8, 130, 128, 16, False, True, "heads", "ntk", 0),
    ("half_48", BF16, 2, 3, 2, 65, 64, 48, False, True, "tokens", "none", 5000),
    ("inter_16", FP32, 2, 4, 2, 33, 64, 16, True, True, "tokens", "yarn", 1 << 24),
    ("fp32_half", FP32, 1, 12, 12, 257, 64, 64, False, False, "heads", "ntk", 0),
    ("fp32_full", FP32, 1, 2, 1, 100, 128, 128, False, True, "tokens", "linear", 100000),
    ("norm_only", BF16, 2, 6, 3, 21, 128, 0, False, True, "tokens", "none", 0),
    ("many_heads", BF16, 1, 40, 1, 5, 64, 32, True, True, "heads", "none", -50),
    ("long", BF16, 1, 9, 3, 6001, 128, 128, True, True, "tokens", "none", 0),
]
IDS = [c[0] for c in CASES]


def _setup(case, seed=3):
    name, dtype, B, Hq, Hkv, n, D, R, inter, norm, layout, scaling, far = case
    g = torch.Generator().manual_seed(seed)
    q, k = _heads(B, Hq, n, D, dtype, layout, g), _heads(B, Hkv, n, D, dtype, layout, g)
    freq, amp = rotary_frequencies(R, scaling=scaling, factor=4.0) if R else (torch.empty(0).double(), 1.0)
    r = Rotary(D, rotary_dim=R, interleaved=inter, frequencies=freq, amplitude=amp)
    pos = None
    if far:
        pos = torch.randint(min(far, 0), max(far, 1), (B, n), generator=g).to(torch.int32)
    eps, qw, kw = None, None, None
    if norm:
        eps = 1e-5
        qw = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
        kw = (1 + 0.2 * torch.randn(D, generator=g)).cuda()
        if name == "half_48":
            qw, kw = qw.bfloat16(), kw.bfloat16()
        if name == "norm_only":
            kw = None
    ref_pos = pos if pos is not None else torch.arange(n)[None].expand(B, n)
    return dict(q=q, k=k, r=r, freq=freq, amp=amp, inter=inter, eps=eps, qw=qw, kw=kw, g=g,
                pos=None if pos is None else pos.cuda(), ref_pos=ref_pos, R=R, D=D)


def _cpu(x):
    return None if x is None else x.cpu()


def _close(got, want, scale, dtype):
    """One rounding to dtype, and fp32 arithmetic: cosines and sines to 2^-22, sums of 128
    squares in a tree (20 roundings), a handful of products -- below 2^-18 of the
    magnitudes that enter, `scale`."""
    tol = torch.finfo(dtype).eps / 2 * want.abs() + 2.0 ** -18 * scale + 1e-30
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


def _pair_scale(x, R, inter):
    """|a| + |b| of each element's pair."""
    m = x.abs().clone()
    if inter:
        t = m[..., 0:R:2] + m[..., 1:R:2]
        m[..., 0:R:2] = t
        m[..., 1:R:2] = t
    else:
        t = m[..., :R // 2] + m[..., R // 2:R]
        m[..., :R // 2] = t
        m[..., R // 2:R] = t
    return m


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_forward_matches_the_definition(case):
    s = _setup(case)
    q, k = s["r"].forward(s["q"], s["k"], positions=s["pos"], norm_eps=s["eps"], q_weight=s["qw"], k_weight=s["kw"])
    for x, w, y in ((s["q"], s["qw"], q), (s["k"], s["kw"], k)):
        assert y.is_contiguous() and y.dtype == x.dtype
        u = x.double().cpu()
        if s["eps"] is not None:
            u = normed(u, s["eps"], _cpu(w))
        want = rotated(u, s["ref_pos"], s["freq"], s["amp"], s["inter"])
        _close(y, want, s["amp"] * _pair_scale(u, s["R"], s["inter"]), x.dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("grad", [FP32, BF16])
@pytest.mark.parametrize("case", CASES, ids=IDS)
def test_backward_matches_the_formula(case, grad):
    s = _setup(case)
    if s["q"].dtype == FP32 and grad == BF16:
        grad = FP32
    gq = torch.randn(s["q"].shape, generator=s["g"]).to(grad).cuda()
    gk = torch.randn(s["k"].shape, generator=s["g"]).to(grad).cuda()
    args = dict(positions=s["pos"], norm_eps=s["eps"], q_weight=s["qw"], k_weight=s["kw"])
    res = s["r"].backward(gq, gk, s["q"], s["k"], **args)
    assert len(res) == (2 if s["eps"] is None else 4)
    for i, (x, w, g) in enumerate(((s["q"], s["qw"], gq), (s["k"], s["kw"], gk))):
        assert res[i].dtype == x.dtype
        xd = x.double().cpu().requires_grad_(True)
        wd = None if w is None else w.double().cpu().requires_grad_(True)
        y = definition(xd, s["ref_pos"], s["freq"], s["amp"], s["inter"], s["eps"], wd)
        want = torch.autograd.grad(y, [xd] if wd is None else [xd, wd], g.double().cpu())
        gd = g.double().cpu()
        h = s["amp"] * _pair_scale(gd, s["R"], s["inter"])
        if s["eps"] is not None:
            xc = x.double().cpu()
            rms = 1 / torch.sqrt((xc * xc).mean(-1, keepdim=True) + s["eps"])
            u = xc * rms
            hw = h if w is None else h * w.double().cpu().abs()
            scale = rms * (hw + u.abs() * (hw * u.abs()).mean(-1, keepdim=True))
            if w is not None:
                # per column: terms of at most 2^-18 relative error each, added up in runs
                # of at most 2^8 terms by a thread and in trees above that
                tol = 2.0 ** -15 * (h * u.abs()).sum((0, 1, 2))
                err = (res[2 + i].double().cpu() - want[1]).abs()
                assert bool((err <= tol).all()), float((err / tol).max())
            else:
                assert res[2 + i] is None
        else:
            scale = h
        _close(res[i], want[0], scale, x.dtype)


@pytest.mark.gpu
def test_backward_matches_differences():
    """The kernel's gradients along random directions against central differences of the
    64-bit definition (step 1e-4: an error of order 1e-8)."""
    s = _setup(CASES[7])
    gq = torch.randn(s["q"].shape, generator=s["g"])
    gk = torch.randn(s["k"].shape, generator=s["g"])
    dq, dk, dqw, dkw = s["r"].backward(gq.cuda(), gk.cuda(), s["q"], s["k"], positions=s["pos"], norm_eps=s["eps"],
                                       q_weight=s["qw"], k_weight=s["kw"])

    def loss(x, w, g):
        y = definition(x, s["ref_pos"], s["freq"], s["amp"], s["inter"], s["eps"], w)
        return (y * g.double()).sum()

    for x, w, g, dx, dw in ((s["q"], s["qw"], gq, dq, dqw), (s["k"], s["kw"], gk, dk, dkw)):
        x, w = x.double().cpu(), w.double().cpu()
        ex = torch.randn(x.shape, generator=s["g"]).double()
        ew = torch.randn(w.shape, generator=s["g"]).double()
        step = 1e-4
        num = (loss(x + step * ex, w + step * ew, g) - loss(x - step * ex, w - step * ew, g)) / (2 * step)
        ana = (dx.double().cpu() * ex).sum() + (dw.double().cpu() * ew).sum()
        mag = (dx.double().cpu() * ex).abs().sum() + (dw.double().cpu() * ew).abs().sum()
        assert abs(num - ana) <= 2.0 ** -16 * mag             # fp32 arithmetic of the kernel, see _close


@pytest.mark.gpu
def test_in_place_broadcast_and_start():
    g = torch.Generator().manual_seed(1)
    r = Rotary(128)
    x = torch.randn((2, 4, 50, 128), generator=g).bfloat16().cuda()
    want, _ = r.forward(x, start=77)
    y = x.clone()
    out, _ = r.forward(y, start=77, q_out=y)                       # in place
    assert out is y and torch.equal(y, want)
    pos = (77 + torch.arange(50))[None].expand(2, 50).contiguous().to(torch.int32).cuda()
    assert torch.equal(r.forward(x, positions=pos)[0], want)
    one = x[:, :1].expand(2, 4, 50, 128)                           # one head broadcast to four
    assert torch.equal(r.forward(one)[0], r.forward(one.contiguous())[0])
    dq, none = r.backward(one, start=3)                            # broadcast upstream, no k
    assert none is None and torch.equal(dq, r.backward(one.contiguous(), start=3)[0])
    back, _ = r.backward(want.float(), start=77)                   # a rotation turned back
    assert float((back - x.float()).abs().max()) <= 2.0 ** -7 * float(x.float().abs().max()) * 1.5


@pytest.mark.gpu
def test_values_outside_a_pair_stay_apart():
    """Infinities and NaN in elements that do not rotate reach no other element."""
    r = Rotary(64, rotary_dim=32, interleaved=False)
    x = torch.ones((1, 1, 4, 64), dtype=BF16, device="cuda")
    x[..., 40] = math.inf
    x[..., 41] = math.nan
    y, _ = r.forward(x, start=5)
    bad = ~torch.isfinite(y)
    assert bool(bad[..., 40].all()) and bool(bad[..., 41].all()) and int(bad.sum()) == 8


@pytest.mark.gpu
def test_same_bits_every_time_and_empty():
    s = _setup(CASES[10])
    gq, gk = torch.randn_like(s["q"], dtype=FP32), torch.randn_like(s["k"], dtype=FP32)
    args = dict(positions=s["pos"], norm_eps=s["eps"], q_weight=s["qw"], k_weight=s["kw"])
    a = s["r"].backward(gq, gk, s["q"], s["k"], **args)
    b = s["r"].backward(gq, gk, s["q"], s["k"], **args)
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    e = torch.empty((1, 2, 0, 128), dtype=BF16, device="cuda")
    q, k = s["r"].forward(e, e)
    assert q.shape == e.shape and k.shape == e.shape
    res = s["r"].backward(e, e, e, e, norm_eps=1e-6, q_weight=s["qw"], k_weight=s["kw"])
    assert res[0].shape == e.shape and not res[2].any() and not res[3].any()


@pytest.mark.gpu
def test_capture_and_streams():
    """Captured and replayed, on another stream, with an eager call in between."""
    s = _setup(CASES[8])
    args = dict(positions=s["pos"], norm_eps=s["eps"], q_weight=s["qw"])
    g = torch.randn_like(s["q"], dtype=FP32), torch.randn_like(s["k"], dtype=FP32)
    want = s["r"].forward(s["q"], s["k"], **args) + s["r"].backward(*g, s["q"], s["k"], **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = s["r"].forward(s["q"], s["k"], **args) + s["r"].backward(*g, s["q"], s["k"], **args)
    for t in got:
        if t is not None:
            t.zero_()
    graph.replay()
    eager = s["r"].forward(s["q"], s["k"], stream=side, **args)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert (a is None and b is None) or torch.equal(a, b)
    assert torch.equal(eager[0], want[0])


@pytest.mark.gpu
def test_gpu_refusals():
    r = Rotary(64)
    q = torch.zeros((1, 2, 3, 64), dtype=BF16, device="cuda")
    w = torch.ones(64, device="cuda")
    for call in (lambda: r.forward(q[..., ::2]), lambda: r.forward(q.transpose(2, 3)),
                 lambda: r.forward(q, q[:, :, :2]), lambda: r.forward(q[0]),
                 lambda: r.forward(q, q_weight=w), lambda: r.forward(q, norm_eps=1e-6, q_weight=w[:32]),
                 lambda: r.forward(q, positions=torch.zeros((1, 2), dtype=torch.int32, device="cuda")),
                 lambda: r.forward(q, q_out=q[:, :1]), lambda: r.forward(q, start=2 ** 31), lambda: r.backward(q, norm_eps=1e-6),
                 lambda: r.backward(q, None, q, q), lambda: r.backward(q, q, q, q[:, :1])):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: r.forward(q.half()), lambda: r.forward(q, q.float()),
                 lambda: r.forward(q, positions=torch.zeros((1, 3), dtype=torch.int64, device="cuda")),
                 lambda: r.forward(q, q, norm_eps=0.0, q_weight=w, k_weight=w.bfloat16())):
        with pytest.raises(TypeError):
            call()
    with pytest.raises(SwaError) as e:
        r.forward(q, q_out=q[:, :, :1].expand(1, 2, 3, 64))         # an output that overlaps itself
    assert e.value.status == INVALID
    with pytest.raises(SwaError):
        r.forward(torch.zeros(1 + q.numel(), dtype=BF16, device="cuda")[1:].view(q.shape))   # misaligned
