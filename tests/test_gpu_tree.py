"""fp_tree_attention against the float64 reference, and what must not reach its results."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_long_blocks_b200 import binding as fb
from block_sparse_long_blocks_b200 import build
from tests._cache_helpers import Case, check_tree

pytestmark = pytest.mark.gpu
FORMATS = ["bf16", "e4m3_head", "e4m3_token"]


def run_and_check(c, **kw):
    o, lse = c.cuda().attend(**kw)
    assert fb.fp_get_device_status() == 0
    worst = check_tree(c, o, lse)
    print(f"of the bound: O {worst[0]:.3f}, lse {worst[1]:.3f}")
    return o, lse


@pytest.mark.parametrize("fmt", FORMATS + ["bf16_64"])
@pytest.mark.parametrize("kv", [1, 2, 15, 16, 17, 127, 128, 129, 256, 1000])
def test_single_token(fmt, kv):
    run_and_check(Case([kv], [1], fmt=fmt.replace("_64", ""), d=64 if fmt.endswith("_64") else 128, seed=kv))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G", [1, 2, 3, 4, 5, 6, 7, 8, 16])
@pytest.mark.parametrize("n", [1, 2, 5])
def test_group_sizes(fmt, G, n):
    run_and_check(Case([140, 31], [n, n], hkv=2, G=G, fmt=fmt, seed=G * 10 + n).trees())


@pytest.mark.parametrize("fmt", FORMATS + ["bf16_64"])
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256, 1024])
def test_pages_and_ragged_batches(fmt, page):
    c = Case([5, 700, 129, 64, 1, 333], [5, 1, 0, 9, 1, 13], hkv=3, G=4, page=page, fmt=fmt.replace("_64", ""),
             d=64 if fmt.endswith("_64") else 128, seed=page)
    run_and_check(c.trees())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n,base", [(1, 0), (7, 0), (33, 100), (64, 64), (127, 1), (128, 0), (200, 56)])
@pytest.mark.parametrize("causal", [False, True])
def test_many_new_tokens(fmt, n, base, causal):
    c = Case([base + n], [n], hkv=1, G=4, fmt=fmt, seed=n)
    run_and_check(c if causal else c.trees())


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_that_see_little_or_nothing(fmt):
    """Empty masks, with and without a cached prefix, and rows without their own token."""
    c = Case([6, 40, 1, 130], [6, 10, 1, 2], hkv=2, G=4, fmt=fmt, seed=9).trees(empty_rows=True, self_bit=False)
    o, lse = run_and_check(c)
    first = torch.from_numpy(~c.see[:6].any(1))
    assert first.any() and (o[:6][first.cuda()] == 0).all() and torch.isneginf(lse[:, :6][:, first.cuda()]).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("what", ["k", "v", "both"])
@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_values_behind_the_mask_do_not_reach_a_row(fmt, what, value):
    """New tokens that hold infinities or NaN: rows that do not see them are what they are without them."""
    if fmt != "bf16" and np.isinf(value):
        value = float("nan")  # (e4m3 has no infinities)
    c = Case([50, 9, 140], [12, 9, 20], hkv=2, G=3, fmt=fmt, seed=12).trees()
    clean, clean_lse = c.cuda().attend()
    bad = [3, 7]  # new tokens of every request
    at = torch.cat([c.new_slots(r)[bad] for r in range(c.R)])
    for name in "kv" if what == "both" else what:
        c.fill(name, at, value, scale=value if fmt == "e4m3_token" else None)
    o, lse = c.cuda().attend()
    sees = torch.from_numpy(np.concatenate([c.see[int(c.cu[r]):int(c.cu[r + 1]), bad].any(1) for r in range(c.R)])).cuda()
    assert sees.any() and (~sees).any()
    assert torch.isfinite(o[~sees].float()).all() and torch.isfinite(lse[:, ~sees]).all()
    # the same keys in the same order: only a token scale's common reference may differ in its last bits
    assert (o[~sees].float() - clean[~sees].float()).abs().max() <= 2.0 ** -7 * clean.float().abs().max()
    assert torch.equal(lse[:, ~sees], clean_lse[:, ~sees])
    if what == "v":
        assert not torch.isfinite(o[sees].float()).all(-1).any()
    assert fb.fp_get_device_status() == 0


def test_infinities_of_seen_values_arrive():
    c = Case([20, 70], [6, 6], hkv=1, G=2, fmt="bf16", seed=2).trees()
    pools = c.pool["v"].flatten(0, 1)
    pools[c.new_slots(0)[2], 0, 5] = float("inf")
    pools[c.new_slots(0)[2], 0, 77] = float("-inf")
    pools[c.new_slots(1)[0], 0, 8] = float("nan")
    run_and_check(c)  # (the reference has them in the same places)


@pytest.mark.parametrize("fmt", FORMATS)
def test_nan_of_cached_tokens_reaches_every_row(fmt):
    c = Case([40], [3], hkv=1, G=4, fmt=fmt, seed=3)
    c.fill("v", c.flat(0, np.array([10])), float("nan"))
    o, _ = c.cuda().attend()
    assert torch.isnan(o.float()).all()
    c = Case([40], [3], hkv=1, G=4, fmt=fmt, seed=3)
    c.fill("k", c.flat(0, np.array([10])), float("nan"))
    o, lse = c.cuda().attend()
    assert torch.isnan(o.float()).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("factor", [1e-30, 1e-6, 1e4, 1e30])
def test_scores_and_values_of_any_size(fmt, factor):
    """Queries and values scaled by a factor: small ones keep their precision, large ones do not overflow."""
    c = Case([150], [4], hkv=1, G=4, fmt=fmt, seed=6)
    c.q = (c.q.float() * min(factor, 1e4)).bfloat16()
    if fmt == "bf16":
        c.pool["v"] = torch.where(torch.isnan(c.pool["v"]), c.pool["v"], (c.pool["v"].float() * factor).bfloat16())
    else:
        c.scale["v"] = c.scale["v"] * factor
    o, lse = c.cuda().attend()
    # float64 of the definition times the factor: the bound is relative to W
    check_tree(c, o, lse)


def test_uneven_token_scales():
    """V of one barely weighted token is 2^20 times the others'."""
    c = Case([300], [2], hkv=1, G=4, fmt="e4m3_token", seed=8)
    flat = c.flat(0, np.array([77]))
    c.scale["v"][flat // c.page, :, flat % c.page] *= 2.0 ** 20
    c.pool["k"].view(torch.uint8).flatten(0, 1)[flat] = torch.zeros((), dtype=torch.uint8)
    run_and_check(c)


@pytest.mark.parametrize("fmt", FORMATS)
def test_long_keys_split_over_the_whole_gpu(fmt):
    c = Case([9001, 4100], [3, 1], hkv=2, G=8, page=64, fmt=fmt, seed=1).trees()
    run_and_check(c)


def test_scale_and_query_stride():
    c = Case([90, 20], [4, 4], hkv=2, G=2, seed=4).trees().cuda()
    plan = c.plan(softmax_scale=0.3)
    o, lse = c.attend(plan)
    check_tree(c, o, lse, scale=float(np.float32(0.3)))
    wide = torch.randn(c.total, c.hq + 3, c.d, device="cuda").bfloat16()
    wide[:, :c.hq] = c.gpu["q"]
    o2, lse2 = c.attend(plan, q=wide[:, :c.hq])
    assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_equal_calls_give_equal_bits():
    c = Case([5000, 900, 64], [7, 1, 20], hkv=4, G=7, fmt="e4m3_token", seed=5).trees().cuda()
    plan = c.plan()
    o, lse = c.attend(plan)
    for _ in range(5):
        plan.workspace.random_(0, 255)
        o2, lse2 = c.attend(plan)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_rows_outside_every_request_are_left():
    c = Case([30, 200], [2, 3], hkv=1, G=4, seed=7).cuda()
    want, want_lse = c.attend()
    cu = (c.cu + 2).cuda()
    q = torch.full((9, 4, 128), float("nan"), dtype=torch.bfloat16, device="cuda")
    q[2:7] = c.gpu["q"]
    plan = fb.Tree(c.cache, hq=4, total_tokens=9, max_tokens=3)
    o = torch.full_like(q, 5.0)
    lse = torch.full((4, 9), 5.0, device="cuda")
    fb.fp_tree_attention(plan, cu, q, o, lse=lse)
    assert torch.equal(o[2:7], want) and torch.equal(lse[:, 2:7], want_lse)
    assert (o[:2] == 5).all() and (o[7:] == 5).all() and (lse[:, :2] == 5).all() and (lse[:, 7:] == 5).all()


def test_bad_lengths_and_pages():
    c = Case([8, 40, 33, 20, 9], [4, 5, 3, 6, 9], hkv=2, G=2).cuda()
    # request 4 has more new tokens than the plan allows. One plan for both calls: another
    # max_tokens may take another tile height, and with it another order of the sums.
    plan = fb.Tree(c.cache, hq=c.hq, total_tokens=c.total, max_tokens=6)
    want, _ = c.attend(plan)
    assert fb.fp_get_device_status() == fb.DEV_BAD_SEQLENS
    c.gpu["kv_lens"][0] = 3
    c.gpu["kv_lens"][1] = c.table.shape[1] * c.page + 1
    c.gpu["table"][2, 0] = -5  # reads as zeros
    o, lse = c.attend(plan)
    assert fb.fp_get_device_status() == fb.DEV_BAD_SEQLENS | fb.DEV_BAD_PAGE
    assert torch.isnan(o[:9].float()).all() and torch.isnan(o[18:].float()).all()
    assert torch.equal(o[12:18], want[12:18]) and torch.isfinite(o[9:12].float()).all()


def test_no_request_has_new_tokens():
    c = Case([8, 40], [0, 0], hkv=1, G=2).cuda()
    plan = fb.Tree(c.cache, hq=2, total_tokens=3, max_tokens=1)
    o = torch.full((3, 2, 128), 5.0, dtype=torch.bfloat16, device="cuda")
    fb.fp_tree_attention(plan, c.gpu["cu"], torch.zeros_like(o), o)
    assert (o == 5).all() and fb.fp_get_device_status() == 0


def test_captured_replayed_with_new_lengths_and_on_another_stream():
    """A graph reads lengths, masks and the cache at replay; two plans run on two streams at once."""
    c = Case([4000, 300], [4, 4], hkv=2, G=4, page=32, fmt="e4m3_token", seed=11, poison=False).trees().cuda()
    plan = c.plan()
    o, lse = c.attend(plan)
    g = torch.cuda.CUDAGraph()
    go, glse = torch.zeros_like(o), torch.zeros_like(lse)
    with torch.cuda.graph(g):
        fb.fp_tree_attention(plan, c.gpu["cu"], c.gpu["q"], go, mask=c.gpu["mask"], lse=glse)
    g.replay()
    assert torch.equal(go, o) and torch.equal(glse, lse)
    c.gpu["kv_lens"].copy_(torch.tensor([77, 290], dtype=torch.int32))
    g.replay()
    o2, lse2 = c.attend(plan)
    assert torch.equal(go, o2) and not torch.equal(o2, o)
    c.kv, c.kv_lens = [77, 290], torch.tensor([77, 290], dtype=torch.int32)
    check_tree(c, o2, lse2)
    streams, plans, outs = [torch.cuda.Stream() for _ in range(2)], [c.plan() for _ in range(2)], []
    torch.cuda.synchronize()
    for _ in range(20):
        for s, p in zip(streams, plans):
            x = torch.empty_like(o)
            with torch.cuda.stream(s):
                fb.fp_tree_attention(p, c.gpu["cu"], c.gpu["q"], x, mask=c.gpu["mask"])
            outs.append(x)
    torch.cuda.synchronize()
    assert all(torch.equal(x, o2) for x in outs)


def test_binding_refuses_what_does_not_fit():
    c = Case([8], [2], hkv=1, G=2).trees().cuda()
    plan = c.plan()
    o = torch.empty_like(c.gpu["q"])
    call = lambda **kw: fb.fp_tree_attention(**(dict(plan=plan, cu_tokens=c.gpu["cu"], q=c.gpu["q"], o=o) | kw))  # noqa: E731
    for bad in (dict(q=c.gpu["q"].float()), dict(q=c.gpu["q"][:1]), dict(o=o.cpu()), dict(o=o.transpose(0, 1)),
                dict(cu_tokens=c.gpu["cu"].long()), dict(mask=c.gpu["mask"].long()), dict(mask=c.gpu["mask"][:1]),
                dict(lse=torch.zeros(2, 2))):
        with pytest.raises(ValueError):
            call(**bad)
    with pytest.raises(fb.FPError):
        fb.Tree(c.cache, hq=9, total_tokens=2, max_tokens=2)


def test_waits_that_run_out_are_reported_and_the_next_call_is_exact():
    """The build whose pipeline waits end after 500 ns returns, with FP_DEV_TIMEOUT."""
    short = fb.load_library(build.build_variant("short_wait"))
    # long enough that HBM, not the first tiles' latency, sets the pace: 64 KB per SM and wait
    c = Case([131072], [2], hkv=4, G=4, page=64, fmt="bf16").trees().cuda()
    o, lse = c.attend()
    plan, out = c.plan(), torch.empty_like(o)
    p = plan.p
    p.cu_tokens, p.mask, p.mask_words = c.gpu["cu"].data_ptr(), c.gpu["mask"].data_ptr(), c.gpu["mask"].shape[1]
    s = torch.cuda.current_stream().cuda_stream
    assert short.fp_tree_attention(c.cache.ref, plan.ref, c.gpu["q"].data_ptr(), out.data_ptr(), None,
                                   plan.workspace.data_ptr(), plan.ws_bytes, s) == 0
    bits = ctypes.c_uint32(0)
    assert short.fp_get_device_status(ctypes.byref(bits), s) == -6 and bits.value == fb.DEV_TIMEOUT
    o2, lse2 = c.attend()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and fb.fp_get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
def test_a_decoding_run_over_a_prefilled_cache(fmt):
    """Prompt written -> drafted trees written, attended, the accepted path kept -> the next token attends to it."""
    n, keep = [10, 7], [[0, 2, 5], [0, 1, 3, 6]]
    c = Case([150, 40], n, hkv=2, G=4, page=16, fmt=fmt, seed=21).trees().cuda()
    g = torch.Generator().manual_seed(5)
    kv_rows = [torch.randn(190, 2, 128, generator=g).bfloat16() for _ in "kv"]
    dev = [x.cuda() for x in kv_rows]
    # the prompts, then the drafted tokens, as a serving loop writes them
    base = [kv - m for kv, m in zip(c.kv, n)]
    pick = lambda spans: [torch.cat([x[a:b] for a, b in spans]) for x in dev]  # noqa: E731
    start = [0, 150]
    c.gpu["kv_lens"].copy_(torch.tensor(base, dtype=torch.int32))
    cu = torch.tensor([0, base[0], sum(base)], dtype=torch.int32).cuda()
    fb.fp_cache_write(c.cache, cu, *pick([(s, s + b) for s, b in zip(start, base)]))
    c.gpu["kv_lens"].copy_(c.kv_lens)
    fb.fp_cache_write(c.cache, c.gpu["cu"], *pick([(s + b, s + b + m) for s, b, m in zip(start, base, n)]))
    for name, pool, sc in (("k", "k", "ks"), ("v", "v", "vs")):  # the reference takes what was stored
        c.pool[name] = c.gpu[pool].cpu()
        c.scale[name] = None if c.gpu[sc] is None else c.gpu[sc].cpu()
    o, lse = c.attend()
    check_tree(c, o, lse)
    accept = torch.tensor([keep[0] + [0], keep[1]], dtype=torch.int32).cuda()
    num = torch.tensor([len(x) for x in keep], dtype=torch.int32).cuda()
    fb.fp_cache_commit(c.cache, c.gpu["cu"], c.total, accept, num, c.gpu["kv_lens"])
    # one more token per request behind the kept ones
    c.gpu["kv_lens"].add_(1)
    step = torch.arange(3, dtype=torch.int32).cuda()
    last = [torch.randn(2, 2, 128, generator=g).bfloat16() for _ in "kv"]
    fb.fp_cache_write(c.cache, step, last[0].cuda(), last[1].cuda())
    # the same history written once, in order, into a fresh cache
    hist = [[torch.cat([x[s:s + b], x[s + b:s + b + m][k], y[r:r + 1]]) for r, (s, b, m, k) in
             enumerate(zip(start, base, n, keep))] for x, y in zip(kv_rows, last)]
    lens = [len(x) for x in hist[0]]
    assert c.gpu["kv_lens"].tolist() == lens
    f = Case(lens, [1, 1], hkv=2, G=4, page=64, fmt=fmt, seed=22)
    if fmt == "e4m3_head":
        f.scale = dict(c.scale)
    f.cuda()
    cu = torch.tensor([0, lens[0], sum(lens)], dtype=torch.int32).cuda()
    fb.fp_cache_write(f.cache, cu, *(torch.cat(x).cuda() for x in hist))
    back = [torch.empty(sum(lens), 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    fb.fp_cache_read(f.cache, cu, *back[:2])
    fb.fp_cache_read(c.cache, cu, *back[2:])
    assert torch.equal(back[0], back[2]) and torch.equal(back[1], back[3])
    q = torch.randn(2, 8, 128, generator=g).bfloat16().cuda()
    outs = []
    for cache in (c.cache, f.cache):
        plan = fb.Tree(cache, hq=8, total_tokens=2, max_tokens=1)
        outs.append(torch.empty_like(q))
        fb.fp_tree_attention(plan, step, q, outs[-1])
    assert torch.equal(outs[0], outs[1])  # the same tiles of the same keys, whatever the pages
    assert fb.fp_get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS + ["bf16_64"])
@pytest.mark.parametrize("G,n", [(8, 1), (3, 5), (4, 9), (8, 16), (8, 17), (16, 40)])
def test_every_kernel_over_keys_split_between_ctas(fmt, G, n):
    """8, 16, 128 and 256 rows per unit, each over keys that many CTAs share, with short requests between long ones."""
    c = Case([6000, 17 + n, 2500, n, 900], [n, 1, n, n, 0], hkv=2, G=G, page=32, fmt=fmt.replace("_64", ""),
             d=64 if fmt.endswith("_64") else 128, seed=G + n)
    run_and_check(c.trees())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("R", [33, 1030])
@pytest.mark.parametrize("G", [4, 8, 16])
def test_many_requests(fmt, R, G):
    """More requests than a warp has lanes, and than the spans that shared memory holds; few and many rows."""
    rng = np.random.default_rng(R + G)
    n = rng.integers(0, 4, R)
    kv = n + rng.integers(0, 90, R)
    kv[R // 2], n[R // 2] = 2000, 3
    run_and_check(Case(kv.tolist(), n.tolist(), hkv=1, G=G, fmt=fmt, seed=R).trees())


@pytest.mark.parametrize("fmt", FORMATS)
def test_rows_combined_by_warps(fmt):
    """More (token, head) rows than get a CTA each in the combining kernel, of split and of whole units."""
    c = Case([3000] + [70] * 9, [64] * 10, hkv=4, G=1, page=64, fmt=fmt, seed=4)
    assert c.total * c.hq > 2 * 148 * 8
    run_and_check(c.trees())


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G,n", [(2, 3), (2, 7), (4, 9), (8, 20)])
def test_unseen_values_in_every_kernel(fmt, G, n):
    """NaN in V (and its scale) of a new token: rows that see it become NaN, others do not notice."""
    kv = [n + 40, n + 131]
    c = Case(kv, [n, n], hkv=2, G=G, fmt=fmt, seed=n).trees()
    clean, clean_lse = c.cuda().attend()
    at = torch.cat([c.new_slots(r)[[1]] for r in range(c.R)])
    c.fill("v", at, float("nan"), scale=float("nan") if fmt == "e4m3_token" else None)
    o, lse = c.cuda().attend()
    sees = torch.from_numpy(np.concatenate([c.see[int(c.cu[r]):int(c.cu[r + 1]), 1] for r in range(c.R)])).cuda()
    assert sees.any() and (~sees).any()
    assert torch.isnan(o[sees].float()).all() and torch.isfinite(o[~sees].float()).all()
    assert (o[~sees].float() - clean[~sees].float()).abs().max() <= 2.0 ** -7 * clean.float().abs().max()
    assert torch.equal(lse, clean_lse) and fb.fp_get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [3, 12, 40])
def test_infinite_and_huge_queries(fmt, n):
    """A query row of infinities gives NaN and leaves the others; one outlier element dominates a row."""
    c = Case([90 + n], [n], hkv=1, G=4, fmt=fmt, seed=n)
    clean, _ = c.cuda().attend()
    c.q[1, 2] = float("inf")
    c.q[0, 1, 7] = 300.0
    o, lse = c.cuda().attend()
    rest = torch.ones(c.total, c.hq, dtype=torch.bool, device="cuda")
    rest[1, 2] = rest[0, 1] = False
    assert torch.isnan(o[1, 2].float()).all() and torch.equal(o[rest], clean[rest])
    assert torch.isfinite(o[0, 1].float()).all() and fb.fp_get_device_status() == 0


@pytest.mark.parametrize("fmt,n", [("bf16", 16), ("bf16", 64), ("e4m3_token", 16), ("e4m3_head", 64)])
def test_waits_that_run_out_with_many_rows(fmt, n):
    """As above for the kernels of 128 and 256 rows."""
    short = fb.load_library(build.build_variant("short_wait"))
    c = Case([60000], [n], hkv=4, G=4, page=64, fmt=fmt).trees().cuda()
    o, lse = c.attend()
    plan, out = c.plan(), torch.empty_like(o)
    p = plan.p
    p.cu_tokens, p.mask, p.mask_words = c.gpu["cu"].data_ptr(), c.gpu["mask"].data_ptr(), c.gpu["mask"].shape[1]
    s = torch.cuda.current_stream().cuda_stream
    assert short.fp_tree_attention(c.cache.ref, plan.ref, c.gpu["q"].data_ptr(), out.data_ptr(), None,
                                   plan.workspace.data_ptr(), plan.ws_bytes, s) == 0
    bits = ctypes.c_uint32(0)
    assert short.fp_get_device_status(ctypes.byref(bits), s) == -6 and bits.value == fb.DEV_TIMEOUT
    o2, lse2 = c.attend()
    assert torch.equal(o, o2) and torch.equal(lse, lse2) and fb.fp_get_device_status() == 0


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("n", [1, 3, 9, 40])
def test_what_an_earlier_call_left_in_shared_memory(fmt, n):
    """The ring's slots hold another cache's keys, values and scales, as large as they get, behind a short request's last
    token."""
    big = Case([90000], [n], hkv=8, G=4, page=64, fmt=fmt, seed=1)
    for name in "kv":
        if fmt == "bf16":
            big.pool[name].fill_(3e38)
        else:
            big.scale[name] = torch.full_like(big.scale[name], 3e38)
    big.cuda().attend()
    c = Case([17 + n, n, 300], [n, n, n], hkv=8, G=4, page=16, fmt=fmt, seed=2).trees().cuda()
    for _ in range(3):
        big.attend()
        o, lse = c.attend()
        check_tree(c, o, lse)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("G,n", [(4, 1), (4, 3), (4, 9), (8, 20)])
def test_a_bad_page_reads_as_zeros_whatever_other_pages_hold(fmt, G, n):
    """Equal bits with a table that names a page of zeros instead, page 0 and its scales being NaN."""
    outs = []
    for bad in (False, True):
        c = Case([330, 60], [n, 1], hkv=2, G=G, page=32, fmt=fmt, seed=6, extra_pages=4).trees()
        used = set(c.table[0, :11].tolist()) | set(c.table[1, :2].tolist())
        zeros = next(p for p in range(1, 17) if p not in used)
        if 0 in used:  # page 0 changes places with a free one
            other = next(p for p in range(zeros + 1, 17) if p not in used)
            c.table[c.table == 0] = other
            for name in "kv":
                bits = c.pool[name].view(torch.uint8)
                bits[other] = bits[0]
                if fmt == "e4m3_token":
                    c.scale[name][other] = c.scale[name][0]
        for name in "kv":
            c.pool[name].view(torch.uint8)[0] = 0xFF  # NaN
            c.pool[name].view(torch.uint8)[zeros] = 0
            if fmt == "e4m3_token":
                c.scale[name][0] = float("nan")
                c.scale[name][zeros] = 0
        c.table[0, 4] = -3 if bad else zeros
        outs.append(c.cuda().attend())
        assert fb.fp_get_device_status() == (fb.DEV_BAD_PAGE if bad else 0)
    assert torch.isfinite(outs[0][0].float()).all()
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
