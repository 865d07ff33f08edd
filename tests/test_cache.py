"""Paged cache: appending with rotation and norm, and the attention over it, against the
definition in 64 bits (GPU); refusals (CPU)."""
import ctypes
import math

import pytest
import torch

from sliding_window_global_b200 import Plan, PagedCache, Rotary, SwaError, load_library, rotary_frequencies
from sliding_window_global_b200.cache import Cache, CacheAppendArgs, CacheAttendArgs, CacheBatch
from sliding_window_global_b200.rotary import HeadNorm, Rotation
from tests.test_rotary import normed, rotated

INVALID, UNSUPPORTED, DEVICE_CHECK = 1, 2, 6
BF16, FP32 = torch.bfloat16, torch.float32

# ------------------------------------------------------------------ CPU: refusals
_FREQ = (ctypes.c_double * 32)(*([0.5] * 32))
_BUF = ctypes.create_string_buffer(8192)
_PTR = (ctypes.addressof(_BUF) + 255) & ~255          # never read: every call below is refused on the host


def _cache(**kw):
    base = dict(k_pages=_PTR, v_pages=_PTR, num_pages=4, num_kv_heads=2, page_size=16, head_dim=64, dtype=0,
                error_word=_PTR)
    base.update(kw)
    return Cache(**base)


def _batch(**kw):
    base = dict(batch=2, num_tokens=4, block_table=_PTR, max_pages=3, seq_lens=_PTR, cu_tokens=None)
    base.update(kw)
    return CacheBatch(**base)


def _append(**kw):
    base = dict(num_q_heads=4, q=_PTR, k=_PTR, v=_PTR, q_out=_PTR, q_stride0=256, q_stride1=64, k_stride0=128,
                k_stride1=64, v_stride0=128, v_stride1=64, q_out_stride0=256, q_out_stride1=64,
                rotation=Rotation(64, 0, ctypes.addressof(_FREQ), 1.0), head_norm=HeadNorm(0, 0, None, None, 0))
    base.update(kw)
    return CacheAppendArgs(**base)


def _attend(**kw):
    base = dict(num_q_heads=4, q=_PTR, q_stride0=256, q_stride1=64, max_tokens=0, max_len=48, window=-1, softcap=0.0,
                scale=0.0, out=_PTR, lse=_PTR)
    base.update(kw)
    return CacheAttendArgs(**base)


CACHE_BAD = [(dict(k_pages=None), INVALID), (dict(v_pages=_PTR + 8), INVALID), (dict(error_word=None), INVALID),
             (dict(num_pages=0), INVALID), (dict(num_kv_heads=0), INVALID), (dict(page_size=0), INVALID),
             (dict(page_size=24), UNSUPPORTED), (dict(head_dim=96), UNSUPPORTED), (dict(head_dim=0), INVALID),
             (dict(dtype=2), INVALID), (dict(num_pages=2 ** 30, num_kv_heads=4), UNSUPPORTED)]
BATCH_BAD = [(dict(batch=-1), INVALID), (dict(num_tokens=-1), INVALID), (dict(max_pages=0), INVALID),
             (dict(block_table=None), INVALID), (dict(seq_lens=None), INVALID), (dict(seq_lens=_PTR + 2), INVALID),
             (dict(num_tokens=5), INVALID)]
APPEND_BAD = [(dict(num_q_heads=-1), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
              (dict(v=_PTR + 8), INVALID), (dict(q_out=None), INVALID), (dict(k_stride0=4), INVALID),
              (dict(v_stride1=-64), INVALID), (dict(q_out_stride0=64), INVALID), (dict(q_out_stride1=0), INVALID),
              (dict(rotation=Rotation(128, 0, ctypes.addressof(_FREQ), 1.0)), INVALID),
              (dict(rotation=Rotation(8, 0, ctypes.addressof(_FREQ), 1.0)), UNSUPPORTED),
              (dict(head_norm=HeadNorm(1, -1.0, None, None, 0)), INVALID)]
ATTEND_BAD = [(dict(num_q_heads=3), INVALID), (dict(num_q_heads=0), INVALID), (dict(num_q_heads=130), UNSUPPORTED),
              (dict(q=None), INVALID), (dict(out=_PTR + 4), INVALID), (dict(lse=_PTR + 1), INVALID),
              (dict(window=-2), INVALID), (dict(softcap=-1.0), INVALID), (dict(softcap=math.nan), INVALID),
              (dict(scale=math.inf), INVALID), (dict(max_len=-1), INVALID), (dict(q_stride0=4), INVALID),
              (dict(q_stride1=-8), INVALID), (dict(q_stride0=0), INVALID)]


@pytest.mark.parametrize("which,bad,status",
                         [("cache", b, s) for b, s in CACHE_BAD] + [("batch", b, s) for b, s in BATCH_BAD] +
                         [("append", b, s) for b, s in APPEND_BAD] + [("attend", b, s) for b, s in ATTEND_BAD])
def test_refusals(which, bad, status):
    lib = load_library()
    c = _cache(**(bad if which == "cache" else {}))
    b = _batch(**(bad if which == "batch" else {}))
    if which != "attend":
        a = _append(**(bad if which == "append" else {}))
        assert lib.swa_cache_append(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), None) == status
    if which != "append":
        a = _attend(**(bad if which == "attend" else {}))
        assert lib.swa_cache_attend(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), None) == status


def test_null_empty_and_workspace():
    lib = load_library()
    assert lib.swa_cache_append(None, None, None, None) == INVALID
    assert lib.swa_cache_attend(None, None, None, None) == INVALID
    assert lib.swa_cache_attend_workspace_bytes(None, None, None) == 0
    assert lib.swa_cache_check(None, None) == INVALID
    c, e = _cache(), _batch(batch=0, num_tokens=0, block_table=None, seq_lens=None)
    assert lib.swa_cache_append(ctypes.byref(c), ctypes.byref(e), ctypes.byref(_append()), None) == 0
    assert lib.swa_cache_attend(ctypes.byref(c), ctypes.byref(e), ctypes.byref(_attend()), None) == 0
    # few rows over a long cache are split, and a workspace too small is refused
    b = _batch(batch=1, num_tokens=1, max_pages=8192)
    a = _attend(max_len=100000)
    refs = ctypes.byref(c), ctypes.byref(b), ctypes.byref(a)
    need = lib.swa_cache_attend_workspace_bytes(*refs)
    assert need > 0 and lib.swa_cache_attend(*refs, None) == INVALID
    a.workspace, a.workspace_bytes = _PTR, need - 1
    assert lib.swa_cache_attend(*refs, None) == INVALID


def test_cpu_pages_are_refused():
    p = torch.zeros((2, 1, 16, 64))
    with pytest.raises(ValueError):
        PagedCache(p, p)
    with pytest.raises(ValueError):
        PagedCache(p, p[:1])


# ------------------------------------------------------------------ GPU: append
def _problem(dtype, Hkv, D, page, new, lens, seed, spare=3, fill=True):
    """A pool whose pages lie in random order; unused table entries are -1."""
    g = torch.Generator().manual_seed(seed)
    B = len(new)
    used = [(n + page - 1) // page for n in lens]
    pages = sum(used) + spare
    order = torch.randperm(pages, generator=g)
    table = torch.full((B, max(used + [1]) + 1), -1, dtype=torch.int32)
    at = 0
    for b in range(B):
        table[b, :used[b]] = order[at:at + used[b]]
        at += used[b]
    shape = (pages, Hkv, page, D)
    k = (torch.randn(shape, generator=g) if fill else torch.zeros(shape)).to(dtype).cuda()
    v = (torch.randn(shape, generator=g) if fill else torch.zeros(shape)).to(dtype).cuda()
    cu = torch.tensor([0] + list(torch.tensor(new).cumsum(0)), dtype=torch.int32)
    return dict(g=g, k=k, v=v, table=table, lens=torch.tensor(lens, dtype=torch.int32), cu=cu, total=int(cu[-1]),
                new=list(new), page=page, cache=PagedCache(k, v))


APPENDS = [
    # dtype, Hq, Hkv, D, R, interleaved, norm, page, new tokens, lengths
    ("tokens", BF16, 32, 8, 128, 128, True, False, 64, [1] * 9, [1, 64, 65, 128, 4000, 17, 63, 200, 129]),
    ("ragged", BF16, 6, 2, 64, 48, False, True, 48, [5, 0, 100, 1, 0], [5, 10, 147, 49, 0]),
    ("fp32", FP32, 3, 3, 64, 16, True, True, 16, [33, 2], [40, 1000]),
    ("one", BF16, 1, 1, 128, 0, False, False, 16, [1], [1]),
    ("no_queries", BF16, 0, 12, 128, 64, False, True, 32, [7, 300], [7, 310]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", APPENDS, ids=[c[0] for c in APPENDS])
def test_append(case):
    name, dtype, Hq, Hkv, D, R, inter, norm, page, new, lens = case
    s = _problem(dtype, Hkv, D, page, new, lens, 5)
    g, T, behind = s["g"], s["total"], 3
    ragged = len(set(new)) > 1
    rows = T + (behind if ragged else 0)                   # rows behind the last sequence belong to nobody
    qkv = (torch.randn((rows, Hq + 2 * Hkv, D), generator=g) * 1.5).to(dtype).cuda()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    freq, amp = rotary_frequencies(R, scaling="yarn", factor=2.0) if R else (torch.empty(0).double(), 1.0)
    rot = Rotary(D, rotary_dim=R, interleaved=inter, frequencies=freq, amplitude=amp) if R else None
    eps = 1e-6 if norm else None
    qw = (1 + 0.1 * torch.randn(D, generator=g)).cuda() if norm and Hq else None
    kw = (1 + 0.1 * torch.randn(D, generator=g)).cuda() if norm else None
    before_k, before_v = s["k"].clone(), s["v"].clone()
    q_out = torch.full((rows, Hq, D), 7.0, dtype=dtype, device="cuda") if Hq else None
    out = s["cache"].append(k, v, s["lens"].cuda(), s["table"].cuda(), q=q if Hq else None,
                            cu_tokens=s["cu"].cuda() if ragged else None, rotary=rot, norm_eps=eps, q_weight=qw,
                            k_weight=kw, q_out=q_out)
    assert s["cache"].check() == 0
    assert out is q_out
    want_k, want_v = before_k.double().cpu(), before_v.cpu()
    written = torch.zeros(want_k.shape[:3], dtype=torch.bool)
    tol = torch.finfo(dtype).eps / 2

    def heads(x, w, pos):                                   # [t, H, D] -> rotated [t, H, D], and its magnitudes
        u = x.double().cpu().transpose(0, 1)[None]
        if eps is not None:
            u = normed(u, eps, None if w is None else w.cpu())
        m = u.abs()
        top = m.amax(-1, keepdim=True) * 2 * amp
        return rotated(u, pos[None], freq, amp, inter)[0].transpose(0, 1), top[0].transpose(0, 1)

    for b in range(len(new)):
        c0, c1 = int(s["cu"][b]), int(s["cu"][b + 1])
        pos = torch.arange(lens[b] - new[b], lens[b])
        if not len(pos):
            continue
        pg, slot = s["table"][b].long()[pos // page], pos % page
        want, top = heads(k[c0:c1], kw, pos)
        got = s["k"].cpu().double()[pg, :, slot]
        assert bool(((got - want).abs() <= tol * want.abs() + 2.0 ** -18 * top).all())
        want_v[pg, :, slot] = v[c0:c1].cpu()
        written[pg, :, slot] = True
        if Hq:
            want, top = heads(q[c0:c1], qw, pos)
            got = out[c0:c1].cpu().double()
            assert bool(((got - want).abs() <= tol * want.abs() + 2.0 ** -18 * top).all())
    assert torch.equal(s["v"].cpu(), want_v)                # values as they came, everything else untouched
    assert torch.equal(s["k"].cpu()[~written], before_k.cpu()[~written])
    if Hq and ragged:
        assert bool((out[T:] == 7.0).all())


@pytest.mark.gpu
def test_append_in_place_matches():
    s = _problem(BF16, 2, 64, 16, [3, 3], [3, 40], 9)
    q = torch.randn((6, 4, 64), generator=s["g"]).bfloat16().cuda()
    k = torch.randn((6, 2, 64), generator=s["g"]).bfloat16().cuda()
    r = Rotary(64)
    args = (k, k, s["lens"].cuda(), s["table"].cuda())
    want = s["cache"].append(*args, q=q, rotary=r)
    same = q.clone()
    assert s["cache"].append(*args, q=same, rotary=r, q_out=same) is same
    assert torch.equal(same, want)


@pytest.mark.gpu
def test_append_leaves_out_what_does_not_exist():
    """Pages outside the pool, positions before 0 and beyond the table, cu_tokens that pass
    T or decrease: those rows write nothing, the others are written, the check reports it."""
    page, D = 16, 64
    pages = torch.zeros((4, 1, page, D), dtype=BF16, device="cuda")
    cache = PagedCache(pages, pages.clone())
    k = torch.ones((4, 1, D), dtype=BF16, device="cuda")

    def run(lens, table, cu=None):
        pages.zero_()
        cache.append(k, k, torch.tensor(lens, dtype=torch.int32, device="cuda"),
                     torch.tensor(table, dtype=torch.int32, device="cuda"),
                     cu_tokens=None if cu is None else torch.tensor(cu, dtype=torch.int32, device="cuda"))
        return cache.check(), int(pages[:, 0, :, 0].sum())

    assert run([4], [[0, 1]]) == (0, 4)
    assert run([4], [[4, 1]]) == (DEVICE_CHECK, 0)
    assert run([4], [[-1, 1]]) == (DEVICE_CHECK, 0)
    assert run([18], [[0, 9]]) == (DEVICE_CHECK, 2)         # two of four rows lie in the bad page
    assert run([2], [[0, 1]]) == (DEVICE_CHECK, 2)          # two rows before position 0
    assert run([33], [[0, 1]]) == (DEVICE_CHECK, 3)         # one row beyond the table
    assert run([2 ** 31 - 1], [[0, 1]]) == (DEVICE_CHECK, 0)
    assert run([2, 2], [[0, 1], [2, 3]], [0, 2, 9]) == (DEVICE_CHECK, 2)
    assert run([2, 2], [[0, 1], [2, 3]], [0, 2, 4]) == (0, 4)
    assert run([2, 2, 2], [[0, 1], [2, 3], [3, 1]], [0, 2, 1, 4])[0] == DEVICE_CHECK
    assert run([2], [[0, 1]], [2, 4])[0] == DEVICE_CHECK    # does not start at 0
    assert run([2, 0], [[0, 1], [2, 3]], [0, 2, 2]) == (0, 2)


# ------------------------------------------------------------------ GPU: attention
def reference(s, q, window, softcap, scale, Hq):
    """(out, lse, sum p |v|, largest |s|) per row in 64 bits; rows without a key: 0, -inf."""
    Hkv, D = s["k"].shape[1], s["k"].shape[3]
    G, T = Hq // Hkv, s["total"]
    kp, vp, qd = s["k"].double().cpu(), s["v"].double().cpu(), q.double().cpu()
    out, mag = torch.zeros((T, Hq, D)).double(), torch.zeros((T, Hq, D)).double()
    lse, top = torch.full((T, Hq), -math.inf).double(), torch.zeros((T, Hq)).double()
    scale = scale or 1 / math.sqrt(D)
    for b, c in enumerate(s["new"]):
        L = int(s["lens"][b])
        for i in range(c):
            t = L - c + i
            lo = 0 if window is None else max(0, t - window)
            j = torch.arange(lo, t + 1)
            pg = s["table"][b].long()[j // s["page"]]
            keep = (pg >= 0) & (pg < kp.shape[0])
            if not bool(keep.any()):
                continue
            pg, slot = pg[keep], (j % s["page"])[keep]
            k = kp[pg, :, slot].repeat_interleave(G, 1)             # [keys, Hq, D]
            v = vp[pg, :, slot].repeat_interleave(G, 1)
            row = int(s["cu"][b]) + i
            x = (qd[row][None] * k).sum(-1) * scale
            top[row] = (qd[row][None] * k).abs().sum(-1).amax(0) * scale
            if softcap > 0:
                x = softcap * torch.tanh(x / softcap)
            p = torch.softmax(x, 0)
            out[row] = (p[..., None] * v).sum(0)
            mag[row] = (p[..., None] * v.abs()).sum(0)
            lse[row] = torch.logsumexp(x, 0)
    return out, lse, mag, top


def check_attention(out, lse, ref, dtype):
    """Scores: products summed in fp32 over D <= 128 elements, at most 2^-17 of their
    absolute sum; exponentials within 2^-13 (bf16 kernels, whose polynomial is off by at most
    1.02e-4) or 2^-20 (fp32).  Outputs: twice that of sum p |v|, in bf16 another half step
    for the rounded p, and the rounding of the result."""
    want, want_lse, mag, top = ref
    empty = torch.isneginf(want_lse)
    assert bool((out.cpu()[empty] == 0).all()) and bool(torch.isneginf(lse.cpu()[empty]).all())
    e = 2.0 ** -13 if dtype == BF16 else 2.0 ** -20
    d = 2.0 ** -17 * top + e
    half = torch.finfo(dtype).eps / 2
    tol = (2 * d[..., None] + (half if dtype == BF16 else 0)) * mag + half * want.abs() + 1e-30
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())
    err = (lse.double().cpu() - want_lse).abs()[~empty]
    tol = (d + 2.0 ** -22 * want_lse.abs())[~empty]
    assert bool((err <= tol).all()), float((err / tol).max())


# name, dtype, Hq, Hkv, D, page, window, softcap, new tokens, lengths
ATTENDS = [
    ("first_token", BF16, 4, 2, 128, 16, None, 0.0, [1], [1]),
    ("tokens", BF16, 32, 8, 128, 64, None, 0.0, [1] * 5, [1, 64, 65, 700, 16]),
    ("tokens_window", BF16, 8, 2, 64, 48, 130, 0.0, [1] * 4, [5, 131, 132, 1000]),
    ("tokens_cap", BF16, 16, 2, 128, 16, None, 5.0, [1] * 3, [33, 300, 1]),
    ("long_split", BF16, 8, 1, 64, 128, None, 0.0, [1], [9001]),
    ("long_split_cap", BF16, 3, 1, 128, 32, 6000, 30.0, [1, 1], [7001, 40]),
    ("many_short", BF16, 8, 4, 64, 16, None, 0.0, [1] * 50, [1 + 37 * i % 211 for i in range(50)]),
    ("many_uneven", BF16, 4, 1, 128, 64, None, 30.0, [1] * 40, [1 + 977 * i % 2999 for i in range(39)] + [12000]),
    ("cluster", BF16, 6, 1, 128, 16, 900, 0.0, [2, 1], [700, 2000]),
    ("cluster_of_8", BF16, 8, 1, 128, 64, None, 0.0, [1], [1900]),
    ("one_block_each", BF16, 12, 12, 64, 32, None, 0.0, [1] * 13, [1 + 31 * i for i in range(13)]),
    ("guesses", BF16, 10, 2, 128, 16, None, 0.0, [3] * 3, [3, 50, 517]),
    ("guesses_window", BF16, 40, 8, 64, 16, 17, 0.0, [8, 1, 5, 0], [8, 20, 300, 77]),
    ("wide_group", BF16, 24, 1, 64, 32, None, 0.0, [1, 2], [100, 400]),
    ("chunk", BF16, 8, 2, 128, 64, None, 0.0, [150, 33], [150, 400]),
    ("chunk_window", BF16, 6, 2, 128, 48, 100, 0.0, [200, 1, 0, 77], [333, 12, 5, 500]),
    ("chunk_window_64", BF16, 5, 1, 64, 16, 31, 50.0, [129, 70], [200, 70]),
    ("chunk_cap", BF16, 12, 12, 64, 128, None, 20.0, [140], [290]),
    ("chunk_self", BF16, 3, 1, 128, 32, 0, 0.0, [64, 65], [64, 100]),
    ("chunk_long", BF16, 4, 1, 128, 128, None, 0.0, [260], [3001]),
    ("chunk_few", BF16, 8, 2, 64, 32, None, 20.0, [70, 33], [1900, 1500]),
    ("chunk_many_parts", BF16, 8, 1, 128, 64, None, 0.0, [9], [9001]),
    ("one_tile", BF16, 32, 8, 128, 16, None, 0.0, [1 + 7 * i % 32 for i in range(40)], [33 + 29 * i % 300 for i in range(40)]),
    ("one_tile_window", BF16, 15, 5, 64, 48, 70, 20.0, [11 + i % 31 for i in range(60)], [41 + 17 * i % 400 for i in range(60)]),
    ("one_tile_long", BF16, 36, 12, 64, 64, None, 0.0, [12, 1, 42, 0, 5, 12, 12, 30], [4800, 300, 42, 0, 5, 999, 2000, 31]),
    ("one_tile_long_cap", BF16, 24, 8, 128, 32, 5000, 9.0, [20, 40] + [3] * 9, [6000, 700] + [40] * 9),
    ("sequences_600", BF16, 2, 1, 64, 16, None, 0.0, [1] * 600, [1 + 7 * i % 41 for i in range(600)]),
    ("sequences_600_rows_40", BF16, 8, 1, 64, 16, 20, 0.0, [5] * 599 + [6], [6 + 7 * i % 41 for i in range(600)]),
    ("heads_128", BF16, 128, 1, 64, 32, None, 0.0, [3], [77]),
    ("fp32_tokens", FP32, 12, 12, 64, 16, None, 0.0, [1, 1], [300, 7]),
    ("fp32_long", FP32, 4, 1, 128, 64, None, 30.0, [2], [3000]),
    ("fp32_group", FP32, 32, 8, 128, 64, None, 0.0, [1] * 6, [1, 7, 8, 9, 64, 2900]),
    ("fp32_window", FP32, 7, 1, 64, 16, 130, 0.0, [1] * 4, [5, 131, 132, 1003]),
    ("fp32_guesses", FP32, 6, 2, 128, 48, 33, 0.0, [5, 1, 0, 3], [5, 20, 9, 517]),
    ("fp32_guesses_cap", FP32, 10, 2, 64, 32, None, 5.0, [6, 2], [70, 700]),
    ("fp32_rows_32", FP32, 8, 1, 128, 16, None, 0.0, [4, 4], [4, 333]),
    ("fp32_rows_33", FP32, 11, 1, 64, 16, None, 0.0, [3, 3], [3, 333]),
    ("fp32_many_parts", FP32, 2, 1, 64, 128, None, 0.0, [1], [9001]),
    ("fp32_waves", FP32, 4, 4, 128, 16, 2500, 0.0, [1] * 30, [1 + 977 * i % 2999 for i in range(30)]),
    ("fp32_chunk", FP32, 6, 2, 64, 48, 50, 0.0, [100, 1, 0, 13], [170, 3, 9, 13]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", ATTENDS, ids=[c[0] for c in ATTENDS])
def test_attend(case):
    name, dtype, Hq, Hkv, D, page, window, cap, new, lens = case
    s = _problem(dtype, Hkv, D, page, new, lens, 11)
    T, ragged = s["total"], len(set(new)) > 1
    wide = (torch.randn((T + 2, Hq + 3, D), generator=s["g"]) * 1.5).to(dtype).cuda()
    q = wide[:T + (2 if ragged else 0), 1:1 + Hq]                     # rows of a wider projection
    out = torch.full((q.shape[0], Hq, D), 7.0, dtype=dtype, device="cuda")
    lse = torch.full((q.shape[0], Hq), 7.0, device="cuda")
    # positions that nobody attends hold NaN: behind every sequence, and before the windows
    for b, c in enumerate(new):
        L, first = lens[b], lens[b] - c
        seen = torch.zeros(s["table"].shape[1] * page, dtype=torch.bool)
        if c:
            seen[0 if window is None else max(0, first - window):L] = True
        for t in range(int((s["table"][b] >= 0).sum()) * page):
            if not seen[t]:
                s["k"][s["table"][b, t // page], :, t % page] = math.nan
                s["v"][s["table"][b, t // page], :, t % page] = math.nan
    s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda() if ragged else None,
                      max_tokens=max(new), max_len=max(lens), window=window, softcap=cap, out=out, lse=lse)
    assert s["cache"].check() == 0
    check_attention(out[:T], lse[:T], reference(s, q, window, cap, 0.0, Hq), dtype)
    assert bool((out[T:] == 7.0).all()) and bool((lse[T:] == 7.0).all())
    # the same without bounds on lengths and tokens, and without lse
    again, none = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda() if ragged else None,
                                    window=window, softcap=cap, return_lse=False)
    assert none is None
    check_attention(again[:T], lse[:T], reference(s, q, window, cap, 0.0, Hq), dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,new,G", [(BF16, [1, 1], 4), (BF16, [40, 3], 4), (FP32, [40, 3], 2), (BF16, [6, 5], 8),
                                         (FP32, [1, 1], 4), (FP32, [6, 5], 4)])
def test_pages_that_do_not_exist_are_left_out(dtype, new, G):
    s = _problem(dtype, 2, 128, 16, new, [100, 50], 13)
    s["table"][0, 2] = -5                                   # keys 32-47
    s["table"][0, 4] = 1 << 30                              # keys 64-79
    s["table"][1, :] = 10 ** 6                              # every key: no row has one
    Hq = 2 * G
    q = torch.randn((s["total"], Hq, 128), generator=s["g"]).to(dtype).cuda()
    out, lse = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda(), max_tokens=max(new))
    assert s["cache"].check() == DEVICE_CHECK and s["cache"].check() == 0
    ref = reference(s, q, None, 0.0, 0.0, Hq)
    assert bool(torch.isneginf(ref[1][new[0]:]).all())
    check_attention(out, lse, ref, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,new,G", [(BF16, 1, 4), (BF16, 70, 2), (FP32, 1, 4), (FP32, 40, 2)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
@pytest.mark.parametrize("at", [3, 30])
def test_a_nan_among_the_keys_is_not_lost(dtype, new, G, cap, at):
    s = _problem(dtype, 2, 128, 16, [new, new], [120, 90], 17)
    page, slot = int(s["table"][0, at // 16]), at % 16
    s["k"][page, 0, slot, 5] = math.nan                     # sequence 0, KV head 0
    q = torch.randn((s["total"], 2 * G, 128), generator=s["g"]).to(dtype).cuda()
    out, lse = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda(), max_tokens=new,
                                 softcap=cap)
    assert bool(out[:new, :G].isnan().all()) and bool(lse[:new, :G].isnan().all())
    assert bool(out[:new, G:].isfinite().all()) and bool(out[new:].isfinite().all())
    assert s["cache"].check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,new,G,length", [(BF16, 1, 4, 9), (BF16, 1, 4, 9000), (BF16, 2, 12, 700), (BF16, 70, 2, 90),
                                                (BF16, 200, 1, 5000), (FP32, 1, 4, 9), (FP32, 3, 4, 3000),
                                                (FP32, 40, 2, 90)])
@pytest.mark.parametrize("cap", [0.0, 20.0])
def test_a_nan_query_is_not_lost(dtype, new, G, length, cap):
    """Every score of its row is NaN; the rows beside it are as without it."""
    s = _problem(dtype, 1, 64, 16, [new], [length], 19)
    q = torch.randn((new, G, 64), generator=s["g"]).to(dtype).cuda()
    bad = q.clone()
    bad[new // 2, G // 2, 7] = math.nan
    run = lambda x: s["cache"].attend(x, s["lens"].cuda(), s["table"].cuda(), softcap=cap)
    (out, lse), (want, want_lse) = run(bad), run(q)
    hit = torch.zeros((new, G), dtype=torch.bool)
    hit[new // 2, G // 2] = True
    assert bool(out[hit].isnan().all()) and bool(lse[hit].isnan().all())
    assert torch.equal(out[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[2, 2], [70, 70]])
def test_broken_bounds_stay_in_bounds(new):
    """Lengths and tokens beyond what the call states, negative lengths, cu_tokens that
    decrease or pass T: reported, the rest is computed, rows of no sequence untouched."""
    s = _problem(BF16, 1, 64, 16, new, [200, 90], 17)
    T, c = s["total"], new[0]
    q = torch.randn((T, 4, 64), generator=s["g"]).bfloat16().cuda()
    lens, table, cu = s["lens"].cuda(), s["table"].cuda(), s["cu"].cuda()

    def run(lens=lens, cu=cu, **kw):
        out = torch.full((T, 4, 64), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((T, 4), 7.0, device="cuda")
        s["cache"].attend(q, lens, table, cu_tokens=cu, out=out, lse=lse, **{**dict(max_tokens=c), **kw})
        return s["cache"].check(), out, lse

    st, good, good_lse = run()
    assert st == 0
    ref = reference(s, q, None, 0.0, 0.0, 4)

    def first_holds(out, lse):
        # Not bit for bit: where the keys of a sequence are parted depends on all lengths,
        # and parts are joined in fp32.  Every parting meets the definition's own bound.
        check_attention(out[:c], lse[:c], [x[:c] for x in ref], BF16)
        return True

    i32 = dict(dtype=torch.int32, device="cuda")
    st, out, lse = run(lens=torch.tensor([200, -3], **i32))
    assert st == DEVICE_CHECK and first_holds(out, lse)
    assert not out[c:].any() and bool(torch.isneginf(lse[c:]).all())
    st, out, lse = run(cu=torch.tensor([0, c, T + 5], **i32))
    assert st == DEVICE_CHECK and first_holds(out, lse) and bool((out[c:] == 7.0).all())
    st, out, lse = run(cu=torch.tensor([0, c, c - 1], **i32))
    assert st == DEVICE_CHECK and first_holds(out, lse) and bool((out[c:] == 7.0).all())
    st, out, lse = run(max_tokens=c - 1)                   # the last token of each is left out
    assert st == DEVICE_CHECK and bool((out[c - 1] == 7.0).all()) and bool((out[T - 1] == 7.0).all())
    assert bool(((out[0].float() - good[0].float()).abs() <= 2.0 ** -6 * (1 + good[0].float().abs())).all())
    st, out, lse = run(max_len=100)                        # the first sequence is longer: its later keys are left out
    assert st == DEVICE_CHECK and bool(torch.isfinite(out).all())
    assert bool(((out[c:].float() - good[c:].float()).abs() <= 2.0 ** -6 * (1 + good[c:].float().abs())).all())
    st, out, lse = run(lens=torch.tensor([2 ** 31 - 1, 90], **i32))
    assert st == DEVICE_CHECK and bool(torch.isfinite(out[:c].float()).all())


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,T,G", [(BF16, 6, 4), (BF16, 140, 4), (FP32, 20, 1), (FP32, 60, 1)])
def test_sequences_that_claim_the_same_rows(dtype, T, G):
    """cu_tokens that go back to 0 name more rows than there are: in bounds, and reported."""
    s = _problem(dtype, 2, 64, 16, [T, 0, T], [200, 10, 160], 37)
    q = torch.randn((T, 2 * G, 64), generator=s["g"]).to(dtype).cuda()
    cu = torch.tensor([0, T, 0, T], dtype=torch.int32, device="cuda")
    out, lse = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=cu, max_tokens=T)
    assert s["cache"].check() == DEVICE_CHECK
    k = torch.randn((T, 2, 64), generator=s["g"]).to(dtype).cuda()
    s["cache"].append(k, k, s["lens"].cuda(), s["table"].cuda(), cu_tokens=cu)
    s["cache"].check()


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 1, 1], [200, 90, 3]])
def test_capture_streams_and_repeats(new):
    """The same bits from every run: eager, on another stream, captured twice with a shared
    pool and replayed in turn, with changed lengths between replays."""
    s = _problem(BF16, 2, 128, 32, new, [3000, 2500, 700], 19)
    q = torch.randn((s["total"], 8, 128), generator=s["g"]).bfloat16().cuda()
    lens, table, cu = s["lens"].cuda(), s["table"].cuda(), s["cu"].cuda()
    args = dict(cu_tokens=cu, max_tokens=max(new), max_len=3000)
    want, want_lse = s["cache"].attend(q, lens, table, **args)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a, al = s["cache"].attend(q, lens, table, stream=side, **args)
    torch.cuda.synchronize()
    assert torch.equal(a, want) and torch.equal(al, want_lse)
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, pool=graphs[0].pool() if graphs else None):
            outs.append(s["cache"].attend(q, lens, table, **args))
        graphs.append(g)
    shorter = s["lens"] - 300
    for k in (0, 1, 0, 1):
        lens.copy_(s["lens"])
        graphs[k].replay()
        assert torch.equal(outs[k][0], want) and torch.equal(outs[k][1], want_lse)
        lens.copy_(shorter)
        graphs[k].replay()
        again, _ = s["cache"].attend(q, lens, table, **args)
        assert torch.equal(outs[k][0], again)
    assert s["cache"].check() == 0


@pytest.mark.gpu
def test_offsets_beyond_32_bits():
    """Pages whose element offsets pass 2^31: the last ones of two pools of 4.3 GB."""
    page, Hkv, D = 128, 8, 128
    pages = (1 << 31) // (page * Hkv * D) + 64
    g = torch.Generator().manual_seed(3)
    k = torch.zeros((pages, Hkv, page, D), dtype=BF16, device="cuda")
    v = torch.zeros_like(k)
    for x in (k, v):
        x[-3:] = torch.randn((3, Hkv, page, D), generator=g).bfloat16().cuda()
    table = torch.tensor([[pages - 1, pages - 3, pages - 2]], dtype=torch.int32)
    s = dict(k=k[-3:], v=v[-3:], table=table - (pages - 3), lens=torch.tensor([300], dtype=torch.int32), page=page)
    for c in (1, 130):
        s.update(new=[c], cu=torch.tensor([0, c]), total=c)
        cache = PagedCache(k, v)
        q = torch.randn((c, 16, D), generator=g).bfloat16().cuda()
        new = torch.randn((c, Hkv, D), generator=g).bfloat16().cuda()
        cache.append(new, new, s["lens"].cuda(), table.cuda())
        out, lse = cache.attend(q, s["lens"].cuda(), table.cuda())
        assert cache.check() == 0
        at = s["lens"] - 1
        assert torch.equal(v[table[0, int(at) // page], :, int(at) % page], new[-1])
        check_attention(out, lse, reference(s, q, None, 0.0, 0.0, 16), BF16)


@pytest.mark.gpu
@pytest.mark.parametrize("new", [[1, 2], [60, 3]])
def test_bounds_beyond_int32(new):
    """Windows, lengths and token bounds that no int32 length can reach bound nothing."""
    s = _problem(BF16, 1, 64, 16, new, [90, 70], 27)
    q = torch.randn((s["total"], 4, 64), generator=s["g"]).bfloat16().cuda()
    args = (q, s["lens"].cuda(), s["table"].cuda())
    want, _ = s["cache"].attend(*args, cu_tokens=s["cu"].cuda())
    for big in (2 ** 31 - 1, 2 ** 31, 2 ** 32, 2 ** 40):
        out, lse = s["cache"].attend(*args, cu_tokens=s["cu"].cuda(), window=big, max_len=big, max_tokens=big)
        assert s["cache"].check() == 0
        check_attention(out, lse, reference(s, q, None, 0.0, 0.0, 4), BF16)


@pytest.mark.gpu
def test_nothing_to_do():
    """No sequences, no new tokens, sequences without any: nothing is written, nothing fails."""
    s = _problem(BF16, 2, 64, 16, [0, 3, 0], [0, 3, 40], 31)
    q, k = (torch.randn((3, h, 64), generator=s["g"]).bfloat16().cuda() for h in (4, 2))
    lens, table, cu = s["lens"].cuda(), s["table"].cuda(), s["cu"].cuda()
    before = s["k"].clone()
    none = dict(cu_tokens=torch.zeros(4, dtype=torch.int32, device="cuda"))
    assert s["cache"].append(k[:0], k[:0], lens, table, q=q[:0], **none).shape == (0, 4, 64)
    assert s["cache"].attend(q[:0], lens, table, **none)[0].shape == (0, 4, 64)
    s["cache"].append(k[:0], k[:0], lens[:0], table[:0])
    assert s["cache"].attend(q[:0], lens[:0], table[:0])[1].shape == (0, 4)
    assert torch.equal(s["k"], before)
    out, lse = s["cache"].attend(q, lens, table, cu_tokens=cu, max_tokens=0)      # the call's own bound: no row
    s["cache"].check()
    out, lse = s["cache"].attend(q, lens, table, cu_tokens=cu, max_tokens=3)
    assert s["cache"].check() == 0
    check_attention(out, lse, reference(s, q, None, 0.0, 0.0, 4), BF16)


@pytest.mark.gpu
def test_shared_prefix_pages_and_scale():
    s = _problem(BF16, 2, 64, 16, [1, 1], [90, 90], 23)
    s["table"][1, :5] = s["table"][0, :5]                  # 80 shared positions
    q = torch.randn((2, 4, 64), generator=s["g"]).bfloat16().cuda()
    out, lse = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), scale=0.3)
    check_attention(out, lse, reference(s, q, None, 0.0, 0.3, 4), BF16)


@pytest.mark.gpu
def test_a_layer_from_prompt_to_tokens():
    """As a decoder layer runs: a training forward of rotated q and k through the banded
    attention, the same tokens appended in chunks and one by one and attended from the
    cache -- one result -- and the gradients back through attention and rotation."""
    Hq, Hkv, D, n, page, r = 8, 2, 128, 400, 48, 127
    g = torch.Generator().manual_seed(29)
    qkv = torch.randn((1, n, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()
    q, k, v = (x.transpose(1, 2) for x in (qkv[:, :, :Hq], qkv[:, :, Hq:Hq + Hkv], qkv[:, :, Hq + Hkv:]))
    qw, kw = ((1 + 0.1 * torch.randn(D, generator=g)).cuda() for _ in range(2))
    rot = Rotary(D)
    norm = dict(norm_eps=1e-6, q_weight=qw, k_weight=kw)
    plan = Plan(1, n, Hq, Hkv, D, BF16)
    band = dict(window=[r] * Hq, causal=True)
    qr, kr = rot.forward(q, k, **norm)
    out, lse = plan.forward(qr, kr, v.contiguous(), **band)
    pages = torch.zeros((n // page + 3, Hkv, page, D), dtype=BF16, device="cuda")
    cache = PagedCache(pages, torch.zeros_like(pages))
    table = torch.randperm(n // page + 1, generator=g).to(torch.int32)[None].cuda()
    rows, start = qkv[0], 0
    for c in (150, 1, 1, 7, 41, 200):
        new = rows[start:start + c]
        start += c
        lens = torch.tensor([start], dtype=torch.int32, device="cuda")
        qn = cache.append(new[:, Hq:Hq + Hkv], new[:, Hq + Hkv:], lens, table, q=new[:, :Hq], rotary=rot, **norm)
        o, l = cache.attend(qn, lens, table, window=r)
        assert torch.equal(qn, qr[0, :, start - c:start].transpose(0, 1))
        # both round p and the result to bf16: two half steps each of at most max |v|
        want = out[0, :, start - c:start].transpose(0, 1).float()
        assert float((o.float() - want).abs().max()) <= 4 * 2.0 ** -8 * float(v.float().abs().max())
        assert float((l - lse[0, :, start - c:start].transpose(0, 1)).abs().max()) <= 2.0 ** -11
    assert cache.check() == 0 and plan.check() == 0 and start == n
    dout = torch.randn(out.shape, generator=g).bfloat16().cuda()
    dq, dk, dv = plan.backward(qr, kr, v.contiguous(), out, lse, dout, **band)
    gq, gk, gqw, gkw = rot.backward(dq, dk, q, k, **norm)
    # the whole layer's gradient by differentiating its definition in 64 bits
    x, y, z = (t.double().cpu().requires_grad_(True) for t in (q, k, v))
    wq, wk = (t.double().cpu().requires_grad_(True) for t in (qw, kw))
    freq = rotary_frequencies(D)[0]
    pos = torch.arange(n)[None]
    a = rotated(normed(x, 1e-6, wq), pos, freq, 1.0, True)
    b = rotated(normed(y, 1e-6, wk), pos, freq, 1.0, True).repeat_interleave(Hq // Hkv, 1)
    sc = a @ b.transpose(2, 3) / math.sqrt(D)
    i = torch.arange(n)
    see = (i[None] <= i[:, None]) & (i[:, None] - i[None] <= r)
    o = torch.softmax(sc.masked_fill(~see, -math.inf), -1) @ z.repeat_interleave(Hq // Hkv, 1)
    want = torch.autograd.grad(o, (x, y, wq, wk), dout.double().cpu())
    for got, ref in zip((gq, gk, gqw, gkw), want):
        # the attention backward's own bound: 2e-2 of the largest gradient
        assert float((got.double().cpu() - ref).abs().max()) <= 2e-2 * float(ref.abs().max())


@pytest.mark.gpu
@pytest.mark.parametrize("window", [None, 40])
def test_decoding_loop_in_a_graph(window):
    """One captured step (append, attend, lengths moved on) replayed token after token, against
    the attention of the whole sequences in 64 bits."""
    B, Hq, Hkv, D, page, n = 3, 8, 2, 64, 16, 37
    g = torch.Generator().manual_seed(43)
    pages = torch.zeros((B * 6, Hkv, page, D), dtype=BF16, device="cuda")
    cache = PagedCache(pages, torch.zeros_like(pages))
    table = torch.randperm(B * 6, generator=g).view(B, 6).to(torch.int32)
    start = torch.tensor([0, 11, 50], dtype=torch.int32)
    qkv = torch.randn((B, int(start.max()) + n, Hq + 2 * Hkv, D), generator=g).bfloat16().cuda()
    rot, dev = Rotary(D), table.cuda()
    for b in range(B):                                     # what came before the loop
        c = int(start[b])
        if c:
            rows = qkv[b, :c]
            cache.append(rows[:, Hq:Hq + Hkv], rows[:, Hq + Hkv:], start[b:b + 1].cuda(), dev[b:b + 1], rotary=rot)
    lens = start.cuda()
    new = torch.empty((B, Hq + 2 * Hkv, D), dtype=BF16, device="cuda")

    def step():
        lens.add_(1)
        q = cache.append(new[:, Hq:Hq + Hkv], new[:, Hq + Hkv:], lens, dev, q=new[:, :Hq], rotary=rot)
        return (q,) + cache.attend(q, lens, dev, window=window)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            q, out, lse = step()
        got = []
        for t in range(n):
            new.copy_(torch.stack([qkv[b, int(start[b]) + t] for b in range(B)]))
            graph.replay()
            got.append((q.clone(), out.clone(), lse.clone()))
    torch.cuda.synchronize()
    assert cache.check() == 0 and torch.equal(lens.cpu(), start + n)
    for t in (0, 1, n // 2, n - 1):
        s = dict(k=cache.k_pages, v=cache.v_pages, page=page, table=table, lens=start + t + 1, new=[1] * B,
                 cu=torch.arange(B + 1), total=B)
        check_attention(got[t][1], got[t][2], reference(s, got[t][0], window, 0.0, 0.0, Hq), BF16)


@pytest.mark.gpu
def test_two_streams_at_once():
    """Calls that overlap on the GPU share nothing: each has its own workspace."""
    cases = []
    for new, lens, seed in (([1, 1], [9000, 4000], 47), ([300, 20], [2500, 20], 53)):
        s = _problem(BF16, 2, 128, 64, new, lens, seed)
        q = torch.randn((s["total"], 8, 128), generator=s["g"]).bfloat16().cuda()
        args = (q, s["lens"].cuda(), s["table"].cuda())
        kw = dict(cu_tokens=s["cu"].cuda(), max_tokens=max(new))
        cases.append((s["cache"], args, kw, s["cache"].attend(*args, **kw), torch.cuda.Stream()))
    torch.cuda.synchronize()
    res = [[], []]
    for _ in range(20):
        for i, (cache, args, kw, _, stream) in enumerate(cases):
            res[i].append(cache.attend(*args, stream=stream, **kw))
    torch.cuda.synchronize()
    for i, (cache, _, _, want, _) in enumerate(cases):
        assert cache.check() == 0
        for out, lse in res[i]:
            assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


@pytest.mark.gpu
def test_gpu_refusals():
    p = torch.zeros((2, 2, 16, 64), dtype=BF16, device="cuda")
    cache = PagedCache(p, p.clone())
    lens = torch.ones(2, dtype=torch.int32, device="cuda")
    table = torch.zeros((2, 1), dtype=torch.int32, device="cuda")
    q, k = torch.zeros((2, 4, 64), dtype=BF16, device="cuda"), torch.zeros((2, 2, 64), dtype=BF16, device="cuda")
    for call in (lambda: PagedCache(p[:, :, :8].contiguous(), p[:, :, :8].contiguous()),
                 lambda: PagedCache(p.transpose(1, 2), p.transpose(1, 2)),
                 lambda: cache.attend(q[0], lens, table), lambda: cache.attend(q[:, :, ::2], lens, table),
                 lambda: cache.attend(q, lens, table[:1]), lambda: cache.attend(q[:1], lens, table),
                 lambda: cache.attend(q, lens, table, window=-1), lambda: cache.attend(q, lens.cpu(), table),
                 lambda: cache.attend(q, lens, table, out=q.transpose(0, 1)),
                 lambda: cache.attend(q, lens, table, cu_tokens=lens),
                 lambda: cache.append(k[:, :1], k, lens, table), lambda: cache.append(k, k[:1], lens, table),
                 lambda: cache.append(k, k, lens, table, q=q[:1]),
                 lambda: cache.append(k, k, lens, table, rotary=Rotary(128)),
                 lambda: cache.append(k, k, lens, table, k_weight=torch.ones(64, device="cuda"))):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: cache.attend(q.float(), lens, table), lambda: cache.attend(q, lens.long(), table),
                 lambda: cache.append(k, k.float(), lens, table), lambda: PagedCache(p, p.float())):
        with pytest.raises(TypeError):
            call()
    for call in (lambda: cache.attend(q[:, :3], lens, table), lambda: cache.attend(q, lens, table, softcap=-1.0)):
        with pytest.raises(SwaError) as e:
            call()
        assert e.value.status == INVALID
