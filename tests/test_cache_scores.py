"""Scores of the cache attention: capped ones for every cap, against the definition in 64
bits, on products that fp32 holds exactly, so that what is left is the scores' own error."""
import math

import pytest
import torch

from tests.test_cache import BF16, FP32, _problem

# name, dtype, Hq, Hkv, D, page, window, new tokens, lengths: every kernel of the attention
KERNELS = [
    ("cluster", BF16, 4, 1, 64, 16, None, [1, 2, 1], [300, 200, 77]),
    ("cluster_rows_32", BF16, 16, 2, 128, 32, 90, [3, 4], [300, 200]),
    ("runs", BF16, 4, 1, 128, 64, None, [1] * 40, [1 + 97 * i % 299 for i in range(39)] + [9000]),
    ("runs_rows_32", BF16, 30, 1, 64, 64, None, [1] * 40, [1 + 97 * i % 299 for i in range(39)] + [9000]),
    ("chunks", BF16, 4, 2, 128, 48, 100, [200, 90, 1], [300, 200, 177]),
    ("chunks_64", BF16, 3, 3, 64, 16, None, [150, 90], [300, 200]),
    ("one_tile", BF16, 32, 8, 128, 16, None, [1 + 7 * i % 32 for i in range(40)], [33 + 29 * i % 200 for i in range(40)]),
    ("fp32_tokens", FP32, 4, 1, 128, 16, 100, [1, 2, 1], [300, 200, 77]),
    ("fp32_chunks", FP32, 2, 2, 64, 48, None, [70, 3], [200, 133]),
]
CAPS = [0.0, 1e-3, 5.0, 128.0, 129.0, 1e3, 1e4, 1e6, 1e12, 1e30]


def exact_scores(s, Hq):
    """Queries and keys of the problem replaced by halves of whole numbers up to 3: products
    are whole quarters, and so are their sums, far below 2^24 of them."""
    D = s["k"].shape[3]
    q = torch.randint(-3, 4, (s["total"], Hq, D), generator=s["g"]).double() / 2
    s["k"].copy_((torch.randint(-3, 4, s["k"].shape, generator=s["g"]).double() / 2).cuda())
    return q.to(s["k"].dtype).cuda()


def definition(s, q, window, cap):
    """Per row: lse, out, sum p |v|, the largest |score| (before the cap), the number of keys."""
    Hkv, D = s["k"].shape[1], s["k"].shape[3]
    T, Hq = q.shape[:2]
    lse, top, count = (torch.zeros((T, Hq)).double() for _ in range(3))
    out, mag = torch.zeros((T, Hq, D)).double(), torch.zeros((T, Hq, D)).double()
    for b, c in enumerate(s["new"]):
        L, rows = int(s["lens"][b]), slice(int(s["cu"][b]), int(s["cu"][b]) + c)
        j, t = torch.arange(L), torch.arange(L - c, L)
        at = (s["table"][b].long()[j // s["page"]].cuda(), slice(None), (j % s["page"]).cuda())
        k, v = (x[at].double().repeat_interleave(Hq // Hkv, 1).permute(1, 0, 2) for x in (s["k"], s["v"]))
        x = q[rows].double().permute(1, 0, 2) @ k.transpose(1, 2) / math.sqrt(D)     # [Hq, c, L]
        seen = j[None] <= t[:, None]
        if window is not None:
            seen &= j[None] >= t[:, None] - window
        top[rows] = x.abs().masked_fill(~seen.cuda(), 0).amax(-1).T.cpu()
        if cap > 0:
            x = cap * torch.tanh(x / cap)
        x = x.masked_fill(~seen.cuda(), -math.inf)
        lse[rows] = torch.logsumexp(x, -1).T.cpu()
        p = torch.softmax(x, -1)
        out[rows] = (p @ v).permute(1, 0, 2).cpu()
        mag[rows] = (p @ v.abs()).permute(1, 0, 2).cpu()
        count[rows] = seen.sum(-1)[:, None].double()
    return lse, out, mag, top, count


def score_error(dtype, cap, top):
    """Half steps of fp32 in a score |s| <= top, absolute, beside the product's sum (exact here).

    Always: the scale, its product with log2(e) and the product with the sum are rounded, four
    half steps (the constant's too), 2^-22 |s|; the exponent's argument s - max is rounded
    again, another 2^-24 of at most twice the largest: below 2^-22 |s| together with the first
    for all but the largest scores, so 2^-21 in all.
    Capped, fp32: the quotient, tanh within two steps and the product, 2^-21 |s|.
    Capped, bf16: up to a cap of 128, 1 / (1 + 2^u) with ex2 within 2^-22 (a quarter of which
    reaches the quotient, at most half a unit of it), the sum within 2^-24, the reciprocal within
    2^-23 and the argument u within 2^-22 |u|, where it moves the result by |s| 2^-22: 2 cap
    (2^-25 + 2^-25 + 2^-24) + the last rounding of 2^-24 cap, below 2^-21.5 cap. Above, the
    same where |s| >= cap / 8, so 2^-18.5 |s|, and the series below, cut at 2^-22 and of five roundings:
    2^-21 |s|."""
    e = 2.0 ** -21 * top
    if cap > 0 and dtype == FP32:
        e = e + 2.0 ** -21 * top
    elif cap > 0:
        top = torch.minimum(top, torch.tensor(cap, dtype=torch.float64))
        e = e + 2.0 ** -22 * top + (2.0 ** -21.5 * cap if cap <= 128 else 2.0 ** -18.5 * top)
    return e


@pytest.mark.gpu
@pytest.mark.parametrize("case", KERNELS, ids=[c[0] for c in KERNELS])
@pytest.mark.parametrize("cap", CAPS)
def test_capped_scores(case, cap):
    """The error of the log sum: the scores', exponentials within 2^-22 (their approximation's
    stated bound), the fp32 sum of at most a quarter of the row's keys in one accumulator and
    the join of at most 1200 parts, each rounding once on either side, and the logarithm with
    its products, 2^-21 of the parts' own lse. Of the output: twice that of sum p |v| (numerator
    and denominator) and the product's sum, as long as the row; in bf16 half a step for the rounded
    p; the rounding of the result."""
    name, dtype, Hq, Hkv, D, page, window, new, lens = case
    s = _problem(dtype, Hkv, D, page, new, lens, 47)
    q = exact_scores(s, Hq)
    out, lse = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda(), max_tokens=max(new),
                                 max_len=max(lens), window=window, softcap=cap)
    assert s["cache"].check() == 0
    want_lse, want, mag, top, count = definition(s, q, window, cap)
    parts = 1200 if max(lens) > 1000 else 64
    d = (score_error(dtype, cap, top) + 2.0 ** -22 + (count / 4 + 8) * 2.0 ** -24 + 2.0 ** -22 * want_lse.abs() +
         2.0 ** -21 * (1 + top) + parts * 2.0 ** -24)
    err = (lse.double().cpu() - want_lse).abs()
    assert bool((err <= d).all()), float((err / d).max())
    half = torch.finfo(dtype).eps / 2
    tol = (2 * d + count * 2.0 ** -24)[..., None] * mag + (half * mag if dtype == BF16 else 0) + half * want.abs() + 1e-30
    err = (out.double().cpu() - want).abs()
    assert bool((err <= tol).all()), float((err / tol).max())


@pytest.mark.gpu
@pytest.mark.parametrize("case", KERNELS, ids=[c[0] for c in KERNELS])
@pytest.mark.parametrize("cap", [1e-40, 3e38])
def test_caps_at_the_ends_of_fp32(case, cap):
    """The smallest caps leave every key the same weight, the largest bend no score: finite, and
    within 1e-3 of that."""
    name, dtype, Hq, Hkv, D, page, window, new, lens = case
    s = _problem(dtype, Hkv, D, page, new, lens, 53)
    q = exact_scores(s, Hq)
    q[0, 0] = 0                                            # scores of 0
    out, lse = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda(), window=window,
                                 softcap=cap)
    want_lse, want, mag, _, count = definition(s, q, window, 0.0 if cap > 1 else cap)
    assert bool(((lse.double().cpu() - want_lse).abs() <= 1e-3).all())
    assert bool(((out.double().cpu() - want).abs() <= (1e-3 + torch.finfo(dtype).eps) * mag + 1e-30).all())


@pytest.mark.gpu
@pytest.mark.parametrize("case", KERNELS, ids=[c[0] for c in KERNELS])
@pytest.mark.parametrize("cap", [20.0, 500.0])
def test_infinite_and_nan_scores_under_a_cap(case, cap):
    """A score of +inf or -inf is the cap or its negative, a NaN makes its row NaN, and the
    other sequences keep their bits."""
    name, dtype, Hq, Hkv, D, page, window, new, lens = case
    s = _problem(dtype, Hkv, D, page, new, lens, 59)
    q = exact_scores(s, Hq)
    last, keys, row = lens[0] - 1, s["k"], new[0] - 1      # its own key is one that the last token sees
    run = lambda x: s["cache"].attend(x, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda(), window=window,
                                      softcap=cap)
    q[row, :2] = 0
    want, want_lse = run(q)
    at = (int(s["table"][0, last // page]), 0, last % page)
    keys[at] = 0
    keys[at + (0,)] = 1e30
    bad = q.clone()
    bad[row, 0, 0], bad[row, 1, 0] = 1e30, -1e30
    out, lse = run(bad)
    exact = definition(s, bad, window, cap)[0]             # 64 bits hold the products: 1e60
    assert bool(((lse[row, :2].double().cpu() - exact[row, :2]).abs() <= 2e-4 * max(1.0, cap / 128)).all())
    assert bool(out[row, :2].isfinite().all())
    bad[row, 0, 0] = math.nan
    out, lse = run(bad)
    assert bool(out[row, 0].isnan().all()) and bool(lse[row, 0].isnan())
    c = new[0]
    assert torch.equal(out[c:], want[c:]) and torch.equal(lse[c:], want_lse[c:])
    assert bool(out[row, 1].isfinite().all())
