"""fp_cache_write, fp_cache_read and fp_cache_commit against their definitions, bit for bit."""
import numpy as np
import pytest
import torch

from block_sparse_long_blocks_b200 import binding as fb
from tests._cache_helpers import E4M3_MAX, Case, bits8, quantise

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "e4m3_head", "e4m3_token"]


def same(a, b):
    """Equal bits (NaN positions included)."""
    a, b = a.cpu().contiguous(), b.cpu().contiguous()
    return a.shape == b.shape and a.dtype == b.dtype and torch.equal(a.view(torch.uint8), b.view(torch.uint8))


def packed_rows(case, seed=1, spread=True):
    g = torch.Generator().manual_seed(seed)
    out = []
    for _ in "kv":
        x = torch.randn(case.total, case.hkv, case.d, generator=g)
        if spread:
            x = x * torch.exp2(torch.randint(-12, 9, (case.total, case.hkv, 1), generator=g).float())
        out.append(x.bfloat16())
    return out


def written(case, rows, skip=()):
    """The pools and scales that a write of `rows` leaves, from the definition."""
    pool = {n: case.pool[n].clone() for n in "kv"}
    scale = {n: None if case.scale[n] is None else case.scale[n].clone() for n in "kv"}
    for r in range(case.R):
        a, b = int(case.cu[r]), int(case.cu[r + 1])
        if a == b or r in skip:
            continue
        at = case.new_slots(r)
        for name, x in zip("kv", rows):
            x = x[a:b].float()
            if case.fmt == "bf16":
                pool[name].flatten(0, 1)[at] = x.bfloat16()
                continue
            if case.fmt == "e4m3_head":
                sc = case.scale[name].expand(b - a, case.hkv)
            else:
                sc = x.abs().amax(-1) / torch.full((), E4M3_MAX)
                scale[name][at // case.page, :, at % case.page] = sc
            codes = quantise(x, torch.where(sc == 0, 1.0, sc)[..., None])
            bits8(pool[name]).flatten(0, 1)[at] = bits8(codes)
    return pool, scale


def check_cache(case, want):
    for name in "kv":
        assert same(case.gpu[name], want[0][name]), name
        if want[1][name] is not None:
            assert same(case.gpu[name + "s"], want[1][name]), name + " scale"
    assert fb.fp_get_device_status() == 0


SHAPES = [
    dict(kv=[1], n=[1], hkv=1, page=16),
    dict(kv=[17, 40, 3], n=[1, 1, 1], hkv=8, page=64),
    dict(kv=[33, 1, 200, 64], n=[20, 0, 129, 64], hkv=3, page=32),
    dict(kv=[700], n=[700], hkv=4, page=256),
    dict(kv=[3] * 70, n=[2] * 70, hkv=2, page=16),                 # more requests than a warp
    dict(kv=[2000, 5], n=[1999, 5], hkv=8, page=1024),
]


@pytest.mark.parametrize("fmt", FORMATS + ["bf16_64"])
@pytest.mark.parametrize("shape", SHAPES)
def test_write(shape, fmt):
    c = Case(**shape, fmt=fmt.replace("_64", ""), d=64 if fmt.endswith("_64") else 128, seed=3).cuda()
    rows = packed_rows(c)
    want = written(c, rows)
    fb.fp_cache_write(c.cache, c.gpu["cu"], rows[0].cuda(), rows[1].cuda())
    check_cache(c, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_takes_slices_of_a_fused_projection(fmt):
    c = Case([50, 9], [13, 9], hkv=3, page=16, fmt=fmt).cuda()
    qkv = torch.randn(c.total, 7, c.d).bfloat16()
    rows = [qkv[:, 1:4], qkv[:, 4:7]]
    want = written(c, rows)
    dev = qkv.cuda()
    fb.fp_cache_write(c.cache, c.gpu["cu"], dev[:, 1:4], dev[:, 4:7])
    check_cache(c, want)


@pytest.mark.parametrize("fmt", ["e4m3_head", "e4m3_token"])
def test_write_values_where_quantising_can_go_wrong(fmt):
    """Zero rows, a row of one tiny value, values past +-448 of a head's scale, subnormal codes, midpoints."""
    c = Case([12], [12], hkv=2, page=16, fmt=fmt)
    if fmt == "e4m3_head":
        for name in "kv":
            c.scale[name] = torch.tensor([2.0 ** -4, 0.0])  # (0: taken as 1)
    c.cuda()
    rows = packed_rows(c, spread=False)
    for x in rows:
        x[0] = 0
        x[1] = 0
        x[1, :, 5] = 2.0 ** -130
        x[2] = 1e4
        x[3] = -3e38
        x[4] = (torch.arange(128) * 2.0 ** -10).bfloat16()              # subnormal codes and their midpoints
        x[5, :, :] = ((torch.arange(128) * 2 + 1) * 2.0 ** -9).bfloat16()
        x[6, :, 0] = 448
        x[6, :, 1:] = (torch.arange(127) / 4 + 16.5).bfloat16()         # midpoints at scale 1
    want = written(c, rows)
    fb.fp_cache_write(c.cache, c.gpu["cu"], rows[0].cuda(), rows[1].cuda())
    check_cache(c, want)


@pytest.mark.parametrize("fmt", ["e4m3_head", "e4m3_token"])
def test_write_keeps_the_sign_of_zero(fmt):
    """-0.0 alone, beside ordinary values, and values so small that they become -0: codes 0x80, whatever the scale."""
    c = Case([6], [6], hkv=3, page=16, fmt=fmt)
    if fmt == "e4m3_head":
        for name in "kv":
            c.scale[name] = torch.tensor([0.37, 2.0 ** -100, 0.0])  # in and out of the correction's range; 0: taken as 1
    c.cuda()
    rows = packed_rows(c, spread=False)
    for x in rows:
        x[0] = -0.0
        x[1, :, ::3] = -0.0
        x[2] = x[2].abs() * 2.0 ** -120
        x[2, :, 1::2] = -0.0
        x[3, :, 5:] *= 2.0 ** -60
        x[4] = 0.0
    want = written(c, rows)
    fb.fp_cache_write(c.cache, c.gpu["cu"], rows[0].cuda(), rows[1].cuda())
    check_cache(c, want)
    assert (bits8(want[0]["k"]).flatten(0, 1)[c.new_slots(0)[:1]] == 0x80).all()


def test_write_keeps_nan_where_it_is():
    c = Case([4], [4], hkv=1, page=16, fmt="e4m3_token").cuda()
    rows = packed_rows(c, spread=False)
    rows[0][1, 0, 7] = float("nan")
    fb.fp_cache_write(c.cache, c.gpu["cu"], rows[0].cuda(), rows[1].cuda())
    codes = c.gpu["k"].cpu().float().flatten(0, 1)[c.new_slots(0)]
    assert torch.isnan(codes[1, 0, 7]) and int(torch.isnan(codes).sum()) == 1
    others = rows[0][1, 0].float()
    others[7] = 0
    s = c.gpu["ks"].cpu()[c.new_slots(0)[1] // 16, 0, c.new_slots(0)[1] % 16]
    assert s == others.abs().max() / torch.full((), E4M3_MAX)


@pytest.mark.parametrize("fmt", FORMATS + ["bf16_64"])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("with_starts", [False, True])
def test_read(shape, fmt, with_starts):
    c = Case(**shape, fmt=fmt.replace("_64", ""), d=64 if fmt.endswith("_64") else 128, seed=4).cuda()
    width = c.hkv + 2  # the destination's token rows are wider than what is written
    out = [torch.full((c.total, width, c.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    starts = [int(c.rng.integers(0, kv - n + 1)) for kv, n in zip(c.kv, c.n)]
    dev = torch.tensor(starts, dtype=torch.int32).cuda() if with_starts else None
    fb.fp_cache_read(c.cache, c.gpu["cu"], out[0][:, :c.hkv], out[1][:, :c.hkv], starts=dev)
    for name, x in zip("kv", out):
        want = torch.full((c.total, width, c.d), 7.0, dtype=torch.bfloat16)
        for r in range(c.R):
            a, b = int(c.cu[r]), int(c.cu[r + 1])
            first = starts[r] if with_starts else c.kv[r] - c.n[r]
            at = c.flat(r, np.arange(first, first + b - a))
            y = bits8(c.pool[name]).flatten(0, 1)[at].view(c.pool[name].dtype).float()
            if c.fmt == "e4m3_head":
                y = y * c.scale[name][:, None]
            elif c.fmt == "e4m3_token":
                y = y * c.scale[name][at // c.page, :, at % c.page][..., None]
            want[a:b, :c.hkv] = y.bfloat16()
        assert same(x, want), name
    assert fb.fp_get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("in_place", [False, True])
def test_commit(fmt, in_place):
    c = Case([40, 17, 300, 16, 9, 1], [12, 17, 64, 1, 0, 1], hkv=3, page=16, fmt=fmt, seed=5).cuda()
    lists = [[0, 3, 4, 11], list(range(17)), sorted(c.rng.choice(64, 21, replace=False).tolist()), [], [], [0]]
    accept = torch.full((c.R, 24), -9, dtype=torch.int32)
    for r, l in enumerate(lists):
        accept[r, :len(l)] = torch.tensor(l, dtype=torch.int32)
    pool = {n: c.pool[n].clone() for n in "kv"}
    scale = {n: None if c.scale[n] is None else c.scale[n].clone() for n in "kv"}
    for r, l in enumerate(lists):
        base = c.kv[r] - c.n[r]
        if not l:
            continue
        src, dst = c.flat(r, base + np.array(l)), c.flat(r, base + np.arange(len(l)))
        for n in "kv":
            bits8(pool[n]).flatten(0, 1)[dst] = bits8(c.pool[n]).flatten(0, 1)[src]
            if fmt == "e4m3_token":
                scale[n][dst // 16, :, dst % 16] = c.scale[n][src // 16, :, src % 16]
    lens = c.gpu["kv_lens"] if in_place else torch.full((c.R,), -1, dtype=torch.int32, device="cuda")
    fb.fp_cache_commit(c.cache, c.gpu["cu"], c.total, accept.cuda(),
                       torch.tensor([len(l) for l in lists], dtype=torch.int32).cuda(), lens)
    check_cache(c, (pool, scale))
    assert lens.tolist() == [kv - n + len(l) for kv, n, l in zip(c.kv, c.n, lists)]


@pytest.mark.parametrize("bad", [[1, 1], [2, 1], [-1, 0], [0, 5], [0, 1, 2, 3]])
def test_commit_leaves_a_request_with_a_bad_list_alone(bad):
    c = Case([20, 30], [5, 5], hkv=1, page=16, fmt="e4m3_token").cuda()
    accept = torch.tensor([(bad + [0, 0])[:3], [1, 3, 4]], dtype=torch.int32).cuda()
    num = torch.tensor([len(bad), 3], dtype=torch.int32).cuda()
    before = c.gpu["k"].view(torch.uint8).clone()
    lens = torch.zeros(2, dtype=torch.int32, device="cuda")
    fb.fp_cache_commit(c.cache, c.gpu["cu"], c.total, accept, num, lens)
    assert fb.fp_get_device_status() == fb.DEV_BAD_LIST
    assert lens.tolist() == [20, 28]
    after = c.gpu["k"].view(torch.uint8)
    mine = c.flat(0, np.arange(20)).cuda()
    assert torch.equal(after.flatten(0, 1)[mine], before.flatten(0, 1)[mine])
    assert not torch.equal(after, before)  # the other request moved


def bad_requests(c):
    """Request 0: more new tokens than cached; 1: longer than its table; 2: a bad page; 3: fine."""
    c.gpu["kv_lens"][0] = c.n[0] - 1
    c.gpu["kv_lens"][1] = c.table.shape[1] * c.page + 1
    c.gpu["table"][2, (c.kv[2] - 1) // c.page] = 10 ** 6
    return fb.DEV_BAD_SEQLENS | fb.DEV_BAD_PAGE


@pytest.mark.parametrize("fmt", FORMATS)
def test_bad_lengths_and_pages_are_skipped_and_reported(fmt):
    c = Case([8, 40, 33, 20], [4, 5, 3, 6], hkv=2, page=16, fmt=fmt).cuda()
    rows = packed_rows(c)
    status = bad_requests(c)
    last = int(c.cu[2]) + 2  # request 2's only row on the bad page
    want = written(c, rows, skip=(0, 1, 2))
    at = c.new_slots(2)[:2]
    full = written(c, rows, skip=(0, 1, 3))
    for n in "kv":  # its rows on good pages are written
        bits8(want[0][n]).flatten(0, 1)[at] = bits8(full[0][n]).flatten(0, 1)[at]
        if fmt == "e4m3_token":
            want[1][n][at // 16, :, at % 16] = full[1][n][at // 16, :, at % 16]
    fb.fp_cache_write(c.cache, c.gpu["cu"], rows[0].cuda(), rows[1].cuda())
    assert fb.fp_get_device_status() == status
    check_cache(c, want)
    out = [torch.full((c.total, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fb.fp_cache_read(c.cache, c.gpu["cu"], *out)
    assert fb.fp_get_device_status() == status
    for x in out:
        assert (x[:9] == 5).all()                       # rejected requests' rows stay
        assert (x[last] == 0).all()                     # a bad page reads as zeros
        assert not (x[9:last] == 5).all() and torch.isfinite(x.float()).all()
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    accept = torch.tensor([[1, 2]] * 4, dtype=torch.int32, device="cuda")
    fb.fp_cache_commit(c.cache, c.gpu["cu"], c.total, accept, torch.full((4,), 2, dtype=torch.int32, device="cuda"),
                       lens)
    assert fb.fp_get_device_status() == status
    assert lens.tolist() == [3, c.table.shape[1] * 16 + 1, 33, 16]


def test_bad_cu_tokens_and_starts():
    c = Case([8, 8, 8], [2, 2, 2], hkv=1).cuda()
    out = [torch.full((6, 1, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    for cu in ([0, 4, 2, 6], [-1, 2, 4, 6], [0, 2, 4, 7]):
        fb.fp_cache_read(c.cache, torch.tensor(cu, dtype=torch.int32).cuda(), *out)
        assert fb.fp_get_device_status() == fb.DEV_BAD_SEQLENS
    out = [torch.full((6, 1, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fb.fp_cache_read(c.cache, c.gpu["cu"], *out, starts=torch.tensor([0, -1, 7], dtype=torch.int32).cuda())
    assert fb.fp_get_device_status() == fb.DEV_BAD_SEQLENS
    for x in out:
        assert (x[2:] == 5).all() and not (x[:2] == 5).any()


def test_rows_outside_every_request_are_left():
    """A padded batch: cu_tokens covers rows 3 .. 7 of ten."""
    c = Case([9, 30], [2, 3], hkv=2, page=16, fmt="e4m3_token").cuda()
    cu = (c.cu + 3).cuda()
    rows = [torch.cat([torch.full((3, 2, 128), float("nan")), x.float(), torch.full((2, 2, 128), float("nan"))]).bfloat16()
            for x in packed_rows(c)]
    want = written(c, [x[3:8] for x in rows])
    fb.fp_cache_write(c.cache, cu, rows[0].cuda(), rows[1].cuda())
    check_cache(c, want)
    out = [torch.full((10, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fb.fp_cache_read(c.cache, cu, *out)
    for x in out:
        assert (x[:3] == 5).all() and (x[8:] == 5).all() and not (x[3:8] == 5).all()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements; the request's page is its last one."""
    pages, page, hkv = 2 ** 15 + 3, 1024, 1
    k = torch.zeros(pages, page, hkv, 128, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.zeros(pages, hkv, page, device="cuda") for _ in "kv")
    table = torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda")
    lens = torch.tensor([1000], dtype=torch.int32, device="cuda")
    cache = fb.Cache(k, v, table, lens, ks, vs)
    cu = torch.tensor([0, 300], dtype=torch.int32, device="cuda")
    x = [torch.randn(300, hkv, 128, device="cuda").bfloat16() for _ in "kv"]
    fb.fp_cache_write(cache, cu, *x)
    for pool, scale, y in ((k, ks, x[0]), (v, vs, x[1])):
        s = y.float().abs().amax(-1) / torch.full((), E4M3_MAX, device="cuda")
        assert torch.equal(scale[-1, :, 700:1000].t(), s) and int((scale != 0).sum()) == 300
        assert torch.equal(pool[-1, 700:1000].view(torch.uint8), quantise(y.float(), s[..., None]).view(torch.uint8))
    out = [torch.empty_like(y) for y in x]
    fb.fp_cache_read(cache, cu, *out)
    assert torch.equal(out[0], (k[-1, 700:1000].float() * ks[-1, :, 700:1000].t()[..., None]).bfloat16())
    fb.fp_cache_commit(cache, cu, 300, torch.tensor([[5, 299]], dtype=torch.int32, device="cuda"),
                       torch.tensor([2], dtype=torch.int32, device="cuda"), lens)
    assert lens.item() == 702 and torch.equal(ks[-1, 0, 701], ks[-1, 0, 999]) and fb.fp_get_device_status() == 0


@pytest.mark.parametrize("seed", [0, 1])
def test_quotients_are_ieee_division(seed):
    """Four million random bf16 values of every exponent, by scales with full mantissas (and some out of the
    correction's range): the codes are those of float32 division."""
    c = Case([2048, 2100], [2048, 2048], hkv=8, G=1, page=128, fmt="e4m3_head", seed=seed, poison=False)
    g = torch.Generator().manual_seed(seed)
    lo, hi = ((-10, 6), (-126, 126))[seed]
    c.scale = {n: torch.exp2(torch.rand(8, generator=g) * (hi - lo) + lo) for n in "kv"}
    rows = []
    for n in "kv":
        x = torch.randn(c.total, 8, 128, generator=g).double()
        # values whose quotients spread over e4m3's range and beyond, many next to its rounding borders
        x = x * c.scale[n][:, None].double() * torch.exp2(torch.randint(-12, 12, x.shape, generator=g).double())
        rows.append(x.clamp(-3e38, 3e38).bfloat16())
    want = written(c, rows)
    c.cuda()
    fb.fp_cache_write(c.cache, c.gpu["cu"], *(x.cuda() for x in rows))
    check_cache(c, want)


@pytest.mark.parametrize("fmt", FORMATS)
def test_many_requests(fmt):
    """More requests than one search step separates, many of them empty: write, read back, keep the first ones."""
    rng = np.random.default_rng(3)
    n = rng.integers(0, 4, 1030)
    c = Case((n + rng.integers(0, 40, 1030)).tolist(), n.tolist(), hkv=2, G=1, fmt=fmt, seed=3)
    rows = packed_rows(c)
    want = written(c, rows)
    c.cuda()
    fb.fp_cache_write(c.cache, c.gpu["cu"], *(x.cuda() for x in rows))
    check_cache(c, want)
    out = [torch.full((c.total, 2, 128), 7.0, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    fb.fp_cache_read(c.cache, c.gpu["cu"], *out)
    for name, x in zip("kv", out):
        at = torch.cat([c.new_slots(r) for r in range(c.R)])
        vals = want[0][name].float().flatten(0, 1)[at]
        if fmt == "e4m3_head":
            vals = vals * c.scale[name][:, None]
        elif fmt == "e4m3_token":
            vals = vals * want[1][name][at // c.page, :, at % c.page][..., None]
        assert same(x, vals.bfloat16())
    num = torch.from_numpy((n > 1).astype(np.int32)).cuda()
    new = torch.empty(c.R, dtype=torch.int32, device="cuda")
    fb.fp_cache_commit(c.cache, c.gpu["cu"], c.total, torch.ones(c.R, 1, dtype=torch.int32, device="cuda"), num, new)
    assert torch.equal(new.cpu(), c.kv_lens - torch.from_numpy(n).int() + num.cpu())
    first = torch.from_numpy(np.concatenate([c.flat(r, [c.kv[r] - c.n[r]]).numpy() for r in range(c.R) if n[r] > 1]))
    second = torch.from_numpy(np.concatenate([c.flat(r, [c.kv[r] - c.n[r] + 1]).numpy() for r in range(c.R) if n[r] > 1]))
    for name in "kv":
        want[0][name].view(torch.uint8).flatten(0, 1)[first] = want[0][name].view(torch.uint8).flatten(0, 1)[second]
        if want[1][name] is not None and fmt == "e4m3_token":
            want[1][name][first // c.page, :, first % c.page] = want[1][name][second // c.page, :, second % c.page]
    check_cache(c, want)
