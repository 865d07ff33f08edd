"""Bounds of the paged cache's calls: which block-table entries the kernels read, lengths
and capacities at the edge of what an int32 holds."""
import ctypes
import random

import pytest
import torch

from sliding_window_global_b200 import PagedCache, load_library
from sliding_window_global_b200.cache import Cache, CacheAttendArgs, CacheBatch
from tests.test_cache import _problem, check_attention, reference

DEVICE_CHECK = 6
BF16, FP32 = torch.bfloat16, torch.float32

_BUF = ctypes.create_string_buffer(512)
_PTR = (ctypes.addressof(_BUF) + 255) & ~255          # stands for device memory that no host call reads


def looked_up(D, page, max_pages, lens, new, window, max_len, max_tokens):
    """First and last block-table column that the few-token kernel reads of each sequence."""
    B, cu = len(lens), [0]
    for c in new:
        cu.append(cu[-1] + c)
    lens, cu = (ctypes.c_int32 * B)(*lens), (ctypes.c_int32 * (B + 1))(*cu)
    c = Cache(_PTR, _PTR, 8, 1, page, D, 0, _PTR)
    b = CacheBatch(B, cu[B], _PTR, max_pages, ctypes.addressof(lens), ctypes.addressof(cu))
    a = CacheAttendArgs(num_q_heads=4, q=_PTR, q_stride0=256, q_stride1=64, max_tokens=max_tokens, max_len=max_len,
                        window=window, out=_PTR)
    columns = (ctypes.c_int32 * (2 * B))()
    lib = load_library()
    assert lib.swa_selftest_token_columns(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a), columns) == 0
    return [(columns[2 * i], columns[2 * i + 1]) for i in range(B)]


@pytest.mark.parametrize("D", [64, 128])
def test_no_length_leads_outside_the_table(D):
    """seq_lens is device memory that nobody has checked: whatever it holds, only columns of
    the table are read, and none for a window that lies behind the bound on lengths."""
    assert looked_up(D, 16, 64, [5001], [1], 511, 1024, 1) == [(-1, -1)]
    assert looked_up(D, 16, 64, [2 ** 31 - 1], [1], 511, 0, 1) == [(-1, -1)]
    assert looked_up(D, 16, 64, [1030], [2], 511, 0, 2)[0] == ((1028 - 511) // 16, 63)
    rng = random.Random(D)
    for _ in range(3000):
        page, columns = rng.choice([16, 48, 64]), rng.randint(1, 40)
        capacity = page * columns
        max_len = rng.choice([0, rng.randint(1, capacity), capacity, 4 * capacity])
        new = [rng.randint(0, 9) for _ in range(3)]
        lens = [rng.choice([rng.randint(-20, 2 * capacity), rng.randint(0, capacity), 2 ** 31 - 1 - rng.randint(0, 40),
                            -2 ** 31 + rng.randint(0, 40), rng.randint(-2 ** 31, 2 ** 31 - 1)]) for _ in range(3)]
        window = rng.choice([-1, 0, rng.randint(1, 2 * capacity), 2 ** 31 - 1])
        for first, last in looked_up(D, page, columns, lens, new, window, max_len, rng.randint(1, 9)):
            assert -1 <= first <= last < columns and (first >= 0) == (last >= 0)


@pytest.mark.parametrize("D", [64, 128])
def test_only_pages_in_reach_are_looked_up(D):
    """Entries of pages that no key of the call lies in may hold anything: a window that
    begins in the second half of a step of 32 keys, in another page than its first half."""
    assert looked_up(D, 16, 64, [1011], [1], 130, 0, 1) == [(55, 63)]
    rng = random.Random(D + 1)
    for _ in range(3000):
        page, c, window = rng.choice([16, 32, 48, 80, 128]), rng.randint(1, 8), rng.randint(0, 400)
        length = rng.randint(c, 2000)
        keys = range(max(0, length - c - window), length)
        assert looked_up(D, page, 2000 // page + 1, [length], [c], window, 0, c) == [(keys[0] // page, keys[-1] // page)]


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("page,columns", [(16, 2 ** 27), (65536, 2 ** 15), (65536, 2 ** 15 + 1), (65536, 2 ** 20)])
def test_capacities_beyond_int32_bound_nothing(dtype, page, columns):
    """A table of 2^31 positions or more: split as for the longest length that an int32 holds."""
    lib = load_library()

    def workspace(columns, max_len=0):
        c = Cache(_PTR, _PTR, 8, 1, page, 64, dtype, _PTR)
        b = CacheBatch(1, 1, _PTR, columns, _PTR, None)
        a = CacheAttendArgs(num_q_heads=4, q=_PTR, q_stride0=256, q_stride1=64, max_len=max_len, window=-1, out=_PTR)
        return lib.swa_cache_attend_workspace_bytes(ctypes.byref(c), ctypes.byref(b), ctypes.byref(a))

    assert workspace(columns) == workspace(columns, 2 ** 31 - 1) == workspace(columns, 2 ** 31 - 256) > 0
    if dtype == 0:
        assert looked_up(64, page, columns, [2000], [1], 100, 0, 1) == [(1899 // page, 1999 // page)]
        top = 2 ** 31 - 256
        assert looked_up(64, page, columns, [top], [1], 100, 0, 1) == [((top - 101) // page, (top - 1) // page)]


# kernels: few tokens (clusters, runs), many tokens (with a list of units, without), fp32 few and many
KERNELS = [
    ("cluster", BF16, 4, 1, 64, 16, 100, [1, 2, 1], [300, 200, 77]),
    ("runs", BF16, 4, 1, 128, 64, 5000, [1] * 40, [1 + 977 * i % 2999 for i in range(39)] + [12000]),
    ("chunks", BF16, 4, 2, 128, 48, 100, [200, 90, 1], [900, 500, 333]),
    ("one_chunk", BF16, 8, 1, 64, 16, 50, [20, 30], [300, 200]),
    ("fp32_tokens", FP32, 4, 1, 128, 16, 100, [1, 2, 1], [300, 200, 77]),
    ("fp32_chunks", FP32, 2, 2, 64, 48, 100, [70, 3], [400, 333]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", KERNELS, ids=[c[0] for c in KERNELS])
@pytest.mark.parametrize("beyond", [1, 4000, 2 ** 30, None])
def test_windows_behind_the_bound_on_lengths(case, beyond):
    """A length beyond the table, whose windows lie partly or wholly behind its last page:
    reported; rows without a key are 0 and -inf, the other sequences as ever."""
    name, dtype, Hq, Hkv, D, page, window, new, lens = case
    s = _problem(dtype, Hkv, D, page, new, lens, 41)
    q = torch.randn((s["total"], Hq, D), generator=s["g"]).to(dtype).cuda()
    ref = reference(s, q, window, 0.0, 0.0, Hq)
    max_len = max(lens)
    bad = 2 ** 31 - 1 if beyond is None else max_len + window + new[0] + beyond
    given = s["lens"].clone()
    given[0] = bad                                        # the first of its windows begins behind max_len
    out, lse = s["cache"].attend(q, given.cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda(), max_tokens=max(new),
                                 max_len=max_len, window=window)
    assert s["cache"].check() == DEVICE_CHECK and s["cache"].check() == 0
    c = new[0]
    assert not out[:c].any() and bool(torch.isneginf(lse[:c]).all())
    check_attention(out[c:], lse[c:], [x[c:] for x in ref], dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("page", [16, 48])
@pytest.mark.parametrize("dtype,G,new", [(BF16, 4, [1] * 40), (BF16, 4, [1, 3, 2]), (BF16, 8, [20, 33]),
                                         (BF16, 2, [150, 1, 70]), (FP32, 2, [1, 1, 2]), (FP32, 2, [40, 3])])
@pytest.mark.parametrize("D", [64, 128])
def test_entries_before_the_windows_may_hold_anything(D, dtype, G, new, page):
    """Pages behind a sliding window given back, their entries -1 or another sequence's."""
    B, window = len(new), 130
    lens = [400 + 83 * i % 1201 + new[i] for i in range(B)]
    lens[0] = 1010 + new[0]
    s = _problem(dtype, 2, D, page, new, lens, 43)
    q = torch.randn((s["total"], 2 * G, D), generator=s["g"]).to(dtype).cuda()
    ref = reference(s, q, window, 0.0, 0.0, 2 * G)
    for b in range(B):
        gone = (lens[b] - new[b] - window) // page         # whole pages before the first window
        s["table"][b, :gone] = -1
        s["table"][b, :gone:3] = 2 ** 31 - 1
    for bounds in (dict(max_tokens=max(new), max_len=max(lens)), {}):
        out, lse = s["cache"].attend(q, s["lens"].cuda(), s["table"].cuda(), cu_tokens=s["cu"].cuda(), window=window,
                                     **bounds)
        assert s["cache"].check() == 0
        check_attention(out, lse, ref, dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype,new,G", [(BF16, 1, 4), (BF16, 200, 2), (BF16, 20, 8), (FP32, 1, 4), (FP32, 90, 2)])
def test_a_table_of_two_billion_positions(dtype, new, G):
    """Two pages of 65536 positions, named in turn by a table that passes 2^31: short lengths
    without a bound on them, and the longest ones, behind a window."""
    page, D = 65536, 64
    g = torch.Generator().manual_seed(61)
    k, v = (torch.randn((2, 1, page, D), generator=g).to(dtype).cuda() for _ in range(2))
    table = (torch.arange(2 ** 15 + 1, dtype=torch.int32) % 2)[None]
    cache = PagedCache(k, v)
    q = torch.randn((new, G, D), generator=g).to(dtype).cuda()
    s = dict(k=k, v=v, table=table, page=page, new=[new], cu=torch.tensor([0, new]), total=new)
    for length, window in ((1000, None), (1000, 70), (2 ** 31 - 256, 70), (2 ** 31 - 65536 + 30, 70)):
        s["lens"] = torch.tensor([length], dtype=torch.int32)
        out, lse = cache.attend(q, s["lens"].cuda(), table.cuda(), window=window)
        assert cache.check() == 0
        check_attention(out, lse, reference(s, q, window, 0.0, 0.0, G), dtype)
    # positions from 2^31 - 256 on are beyond every bound of the attention
    cache.attend(q, torch.tensor([2 ** 31 - 255], dtype=torch.int32, device="cuda"), table.cuda(), window=70)
    assert cache.check() == DEVICE_CHECK
    at = 2 ** 31 - 256 - new
    rows = torch.randn((new, 1, D), generator=g).to(dtype).cuda()
    cache.append(rows, rows, torch.tensor([at + new], dtype=torch.int32, device="cuda"), table.cuda())
    assert cache.check() == 0
    assert torch.equal(v[int(table[0, at // page]), 0, at % page:at % page + new], rows[:, 0])


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["scale", "softcap"])
def test_numbers_that_fp32_does_not_hold_are_refused(name):
    """Rounded to 0 a scale would stand for the default, a cap for none."""
    p = torch.randn((2, 1, 16, 64), device="cuda")
    cache = PagedCache(p, p.clone())
    lens, table = torch.full((1,), 20, dtype=torch.int32, device="cuda"), torch.tensor([[0, 1]], dtype=torch.int32).cuda()
    q = torch.randn((1, 2, 64), device="cuda")
    for value in (1e-50, 1e-46, 1e39):
        with pytest.raises(ValueError):
            cache.attend(q, lens, table, **{name: value})
    out, _ = cache.attend(q, lens, table, **{name: 1e-40})           # every score alike
    assert float((out - out[:, :1]).abs().max()) <= 2.0 ** -20 * float(p.abs().max())
    assert cache.check() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_a_bound_of_no_tokens_is_reported_where_it_does_not_hold(dtype):
    s = _problem(dtype, 2, 64, 16, [0, 3, 0], [0, 30, 40], 71)
    q = torch.randn((3, 4, 64), generator=s["g"]).to(dtype).cuda()
    out, lse = torch.full_like(q, 7.0), torch.full((3, 4), 7.0, device="cuda")
    args = (q, s["lens"].cuda(), s["table"].cuda())
    s["cache"].attend(*args, cu_tokens=s["cu"].cuda(), max_tokens=0, out=out, lse=lse)
    assert s["cache"].check() == DEVICE_CHECK
    s["cache"].attend(*args, cu_tokens=torch.zeros(4, dtype=torch.int32, device="cuda"), max_tokens=0, out=out, lse=lse)
    assert s["cache"].check() == 0                         # rows of no sequence only
    assert bool((out == 7.0).all()) and bool((lse == 7.0).all())


def test_a_cache_keeps_its_pages():
    """The kernels use the addresses of the pages that the cache was made of."""
    cache = object.__new__(PagedCache)
    for name in ("k_pages", "v_pages"):
        with pytest.raises(AttributeError):
            setattr(cache, name, torch.zeros(1))


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["k_pages", "v_pages"])
def test_pages_that_moved_are_refused(name):
    p = torch.zeros((2, 1, 16, 64), device="cuda")
    cache = PagedCache(p, p.clone())
    lens, table = torch.ones(1, dtype=torch.int32, device="cuda"), torch.zeros((1, 1), dtype=torch.int32, device="cuda")
    k = torch.ones((1, 1, 64), device="cuda")
    cache.append(k, k, lens, table)
    old = getattr(cache, name).clone()
    assert float(old.sum()) == 64
    getattr(cache, name).data = old                        # the same tensor in other memory
    for call in (lambda: cache.append(k, k, lens, table), lambda: cache.attend(k, lens, table)):
        with pytest.raises(ValueError):
            call()
    assert cache.check() == 0
