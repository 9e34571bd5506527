"""fp_tree_attention where V's token scales differ by many orders of magnitude between the keys of a row, and where V
holds infinities and NaN."""
import numpy as np
import pytest
import torch

from block_sparse_long_blocks_b200 import binding as fb
from oracle import paged_cache as pc
from tests._cache_helpers import E4M3_MAX, Case, check_tree

pytestmark = pytest.mark.gpu
# (G, n): 8, 16, 128 and 256 rows per unit
KERNELS = [(2, 3), (2, 7), (4, 9), (8, 20)]


def reference(c):
    """The float64 reference, and per row and head the largest p_j v_scale_j / sum p (token scales)."""
    see = c.see if c.mask is not None else None
    O, L, W, A = pc.tree_attention(c.oracle(), c.cu.numpy(), c.q.double().numpy(), see, 1 / np.sqrt(c.d))
    cache, M = c.oracle(), np.zeros((c.total, c.hq))
    for r in range(c.R):
        a, n, kv = int(c.cu[r]), c.n[r], c.kv[r]
        flat = c.flat(r, np.arange(kv)).numpy()
        K, vs = pc.tokens(cache, "k", flat), pc.scales(cache, "v", flat)
        for t in range(n):
            on = np.ones(kv, dtype=bool)
            on[kv - n:] = see[a + t, :n] if see is not None else np.arange(n) <= t
            for h in range(c.hq if on.any() else 0):
                s = K[on, h // c.G] @ c.q[a + t, h].double().numpy() / np.sqrt(c.d)
                M[a + t, h] = (np.exp(s - L[h, a + t]) * vs[on, h // c.G]).max()
    return O, L, W, A, M


def check_rows(c, o, lse):
    """O and lse against float64, within what e4m3 caches with token scales may be off by.

    The exponents, the float32 sums and ex2 give a weight off by delta relative, as in `check_tree`; the two factors that
    bring it to its row's reference are ex2.approx of differences below 2^8 (off by 2^-17 in log2, each side rounding
    once) and three products: 2^-15 more. The product p v_scale goes to f16: 2^-11 of it, or, below f16's normal range, half of
    its step 2^-24, where the row's own largest product is at least 2^8: 2^-33 of that, times a code of at most 448, for each
    key. lse does not depend on V."""
    O, L, W, A, M = reference(c)
    o, lse, kv = o.double().cpu().numpy(), lse.double().cpu().numpy(), max(c.kv)
    delta = 2 * (c.d + 8) * 2.0 ** -23 * A + 2.0 ** -21 + (kv / 16 + 16) * 2.0 ** -23
    tol = 2.0 ** -8 * np.abs(O) + (2 * delta + 2.0 ** -15 + 2.0 ** -11)[..., None] * W * 1.01 \
        + kv * 2.0 ** -33 * E4M3_MAX * M[..., None]
    err = np.abs(o - O)
    worst = (err / np.maximum(tol, 1e-300)).max()
    assert worst <= 1.0, f"O off by {worst:.2f} of its bound"
    assert (np.abs(lse - L) <= delta.T + 2.0 ** -22 * (np.abs(L) + 4)).all()
    return worst


@pytest.mark.parametrize("fmt", ["bf16", "e4m3_head", "e4m3_token"])
@pytest.mark.parametrize("factor", [1e6, 1e12, 1e30])
@pytest.mark.parametrize("G,n", KERNELS)
def test_large_values_behind_the_mask_do_not_reach_a_row(fmt, G, n, factor):
    """A new token with large finite V: rows that do not see it have the bits they have without it."""
    c = Case([n + 40, n + 131, n], [n, n, n], hkv=2, G=G, fmt=fmt, seed=n).trees()
    clean, clean_lse = c.cuda().attend()
    at = torch.cat([c.new_slots(r)[[1]] for r in range(c.R)])
    if fmt == "e4m3_token":
        c.scale["v"][at // c.page, :, at % c.page] *= factor
    else:
        c.fill("v", at, 448.0 if fmt == "e4m3_head" else factor)
    o, lse = c.cuda().attend()
    sees = torch.from_numpy(np.concatenate([c.see[int(c.cu[r]):int(c.cu[r + 1]), 1] for r in range(c.R)])).cuda()
    assert sees.any() and (~sees).any()
    assert torch.equal(o[~sees], clean[~sees]) and torch.equal(lse, clean_lse)
    if fmt == "e4m3_token":
        check_rows(c, o, lse)
    assert fb.fp_get_device_status() == 0


@pytest.mark.parametrize("bits", [20, 40, 64])
@pytest.mark.parametrize("where", ["cached", "new"])
@pytest.mark.parametrize("G,n", KERNELS)
def test_a_large_scale_with_a_small_weight(G, n, where, bits):
    """A seen key whose v_scale is 2^bits times the others' and whose weight is near 2^-bits, or far below it: it adds
    what it adds, and the other keys keep their weights."""
    for far in (False, True):
        c = Case([n + 60, n + 300], [n, n], hkv=2, G=G, fmt="e4m3_token", seed=n + bits).trees()
        c.see[:, 0] = True  # (every row sees the first new token of its request)
        words = c.mask.numpy()
        words[:, 0] |= 1
        at = torch.cat([c.new_slots(r)[[0]] if where == "new" else c.flat(r, np.array([21])) for r in range(c.R)])
        # k = -t u / |u|^2 puts q . k near -t, as q = u + noise: log2 of the weight near -t / (sqrt(d) ln 2)
        t = bits * (2 if far else 1) * np.sqrt(c.d) * np.log(2.0)
        k = (-t * c.u / c.u.square().sum()).expand(c.hkv, c.d)
        sc = k.abs().amax(-1) / E4M3_MAX
        for i in at.tolist():
            c.pool["k"].view(torch.uint8).flatten(0, 1)[i] = (k / sc[:, None]).to(torch.float8_e4m3fn).view(torch.uint8)
            c.scale["k"][i // c.page, :, i % c.page] = sc
        c.scale["v"][at // c.page, :, at % c.page] *= 2.0 ** bits
        o, lse = c.cuda().attend()
        print("of the bound", check_rows(c, o, lse))
    assert fb.fp_get_device_status() == 0


@pytest.mark.parametrize("factor", [2.0 ** -60, 2.0 ** 100])
@pytest.mark.parametrize("G,n", KERNELS)
def test_token_scales_of_any_size_and_zero(G, n, factor):
    """All scales far from one, some keys' V zero (a scale of zero), single rows that see nothing else."""
    c = Case([n + 150, n], [n, n], hkv=2, G=G, fmt="e4m3_token", seed=n).trees()
    c.scale["v"] *= factor
    zero = torch.cat([c.flat(0, np.arange(5, 90, 7)), c.new_slots(1)[[0, n - 1]]])
    c.scale["v"][zero // c.page, :, zero % c.page] = 0
    o, lse = c.cuda().attend()
    print("of the bound", check_rows(c, o, lse))
    assert (o[int(c.cu[1])] == 0).all()  # (the second request's first token sees itself alone)
    assert fb.fp_get_device_status() == 0


@pytest.mark.parametrize("G,n", KERNELS)
def test_a_scale_of_minus_zero_is_zero(G, n):
    """Bits with scales of -0.0 are those with 0.0, whatever else the tile holds."""
    outs = []
    for zero in (0.0, -0.0):
        c = Case([n + 400, n], [n, n], hkv=2, G=G, fmt="e4m3_token", seed=n).trees()
        big = c.flat(0, np.arange(150, 390, 5))
        c.scale["v"][big // c.page, :, big % c.page] *= 2.0 ** 30  # (references rise there)
        at = torch.cat([c.flat(0, np.arange(5, 400, 17)), c.new_slots(1)[[1]]])
        c.scale["v"][at // c.page, :, at % c.page] = zero
        outs.append(c.cuda().attend())
        check_rows(c, *outs[-1])
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])


@pytest.mark.parametrize("G,n", KERNELS)
def test_uneven_scales_over_keys_split_between_ctas(G, n):
    """Keys over many CTAs, their scales spread over 2^60: the partial rows' references differ as much."""
    c = Case([6000, 17 + n, 2500], [n, 1, n], hkv=2, G=G, page=32, fmt="e4m3_token", seed=G + n).trees()
    c.scale["v"] *= torch.exp2(torch.randint(-40, 20, c.scale["v"].shape, generator=torch.Generator().manual_seed(n)).float())
    o, lse = c.cuda().attend()
    print("of the bound", check_rows(c, o, lse))
    again = c.attend()
    assert torch.equal(o, again[0]) and torch.equal(lse, again[1]) and fb.fp_get_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("page", [16, 256])
@pytest.mark.parametrize("G,n", KERNELS)
def test_infinities_of_cached_values_arrive(G, n, page, d):
    """Infinities of either sign in cached rows, alone and both in a column, beside NaN, and in a new token as well."""
    c = Case([n + 500, n + 20, n + 70], [n, n, n], hkv=2, G=G, d=d, page=page, fmt="bf16", seed=n).trees()
    v = c.pool["v"].flatten(0, 1)
    at = c.flat(0, np.array([3, 130, 131, 400]))
    v[at[0], :, 5] = float("inf")
    v[at[1], :, 6] = float("-inf")
    v[at[[1, 3]], :, 9] = float("inf")
    v[at[2], 0, 20], v[at[3], 0, 20] = float("inf"), float("-inf")
    v[at[0], 1, 33], v[at[2], 1, 33] = float("inf"), float("nan")
    v[c.flat(1, np.array([7])), :, 40] = float("-inf")
    v[c.new_slots(1)[[1]], :, 40] = float("inf")   # NaN for the rows that see it
    v[c.new_slots(1)[[1]], :, 41] = float("inf")
    o, lse = c.cuda().attend()
    check_tree(c, o, lse)
    assert torch.isinf(o[:n].float()).any() and fb.fp_get_device_status() == 0


def test_infinities_over_keys_split_between_ctas_and_a_query_of_nan():
    c = Case([9000, 40], [3, 2], hkv=2, G=2, page=64, fmt="bf16", seed=3).trees()
    v = c.pool["v"].flatten(0, 1)
    for pos, col, x in ((5, 1, "inf"), (8000, 1, "inf"), (4000, 2, "-inf"), (100, 3, "inf"), (8900, 3, "-inf"), (77, 4, "nan")):
        v[c.flat(0, np.array([pos])), :, col] = float(x)
    c.q[1, 3] = float("nan")
    o, lse = c.cuda().attend()
    check_tree(c, o, lse)
    assert fb.fp_get_device_status() == 0


@pytest.mark.parametrize("fmt", ["bf16", "e4m3_head", "e4m3_token"])
@pytest.mark.parametrize("kv", [300, 9000])
@pytest.mark.parametrize("G,n", KERNELS)
def test_nan_of_a_value_reaches_a_row_that_hardly_weighs_it(G, n, kv, fmt):
    """NaN in cached V where the last new token's weight is 2^200 times the others', within a CTA and over many."""
    c = Case([n + kv], [n], hkv=1, G=G, page=64, fmt=fmt, seed=n)
    see = np.tril(np.ones((n, n), dtype=bool))
    see[:, 0] = True
    c.trees()
    c.see = see
    c.mask = torch.from_numpy(np.packbits(np.pad(see, ((0, 0), (0, 64 - n))).reshape(n, 2, 32), axis=-1,
                                          bitorder="little").view(np.int32).reshape(n, 2).copy())
    t = 200 * np.sqrt(c.d) * np.log(2.0)
    k = (t * c.u / c.u.square().sum()).expand(1, c.d)
    i = c.new_slots(0)[:1]
    if fmt == "bf16":
        c.pool["k"].flatten(0, 1)[i] = k.bfloat16()
    else:
        sc = k.abs().amax() / E4M3_MAX
        if fmt == "e4m3_token":
            c.scale["k"][i // c.page, :, i % c.page] = sc
        else:
            c.scale["k"] = torch.maximum(c.scale["k"], sc)  # (the other keys' scores just grow a little)
            sc = c.scale["k"][0]
        c.pool["k"].view(torch.uint8).flatten(0, 1)[i] = (k / sc).to(torch.float8_e4m3fn).view(torch.uint8)
    c.fill("v", c.flat(0, np.array([3])), float("nan"))
    o, lse = c.cuda().attend()
    assert torch.isnan(o.float()).all() and torch.isfinite(lse).all() and fb.fp_get_device_status() == 0
    c.pool["v"].view(torch.uint8).flatten(0, 1)[c.flat(0, np.array([3]))] = 0
    o, lse = c.cuda().attend()
    check_tree(c, o, lse)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3_head", "e4m3_token"])
@pytest.mark.parametrize("outlier", [300.0, -1e4])
@pytest.mark.parametrize("G,n", KERNELS)
def test_a_query_with_an_outlier_element(G, n, outlier, fmt):
    """One element of a query is far above the others; K is small in its channel, as a model's would be.

    q of e4m3 caches is the sum of two e4m3 values, off by at most eps = 2^-22 (more than 16 rows: 2^-17) of the row's
    largest element, which puts an exponent off by at most B = eps max|q| scale sum|k|, a weight by e^B - 1 relative, lse by
    as much and O, a quotient, by twice that of W."""
    c = Case([n + 200], [n], hkv=2, G=G, fmt=fmt, seed=n).trees()
    shrink = 2.0 ** -6 if abs(outlier) < 1000 else 2.0 ** -11
    k = c.pool["k"].float()
    k[..., 7] *= shrink
    c.pool["k"] = k.to(c.pool["k"].dtype)
    c.q[0, 1, 7] = c.q[n - 1, c.hq - 1, 7] = outlier
    o, lse = c.cuda().attend()
    O, L, W, A = pc.tree_attention(c.oracle(), c.cu.numpy(), c.q.double().numpy(), c.see, 1 / np.sqrt(c.d))
    eps = 0.0 if fmt == "bf16" else 2.0 ** -22 if n * G <= 16 else 2.0 ** -17
    flat = c.flat(0, np.arange(c.kv[0])).numpy()
    K = np.repeat(np.abs(pc.tokens(c.oracle(), "k", flat)).sum(-1).max(0), G)  # [hq]: the largest sum|k|
    B = eps * c.q.double().abs().amax(-1).numpy() * K / np.sqrt(c.d)
    delta = 2 * (c.d + 8) * 2.0 ** -23 * A + 2.0 ** -21 + (c.kv[0] / 16 + 16) * 2.0 ** -23 + np.expm1(B)
    p_round = 2.0 ** -11 if fmt != "bf16" else 2.0 ** -7 if n * G > 16 else 2.0 ** -16
    # f16 below its normal range: 2^-33 of the row's largest product a key (see check_rows), V's rows being within 2^6
    tol = 2.0 ** -8 * np.abs(O) + (2 * delta + 2.0 ** -15 + p_round)[..., None] * W * 1.01 \
        + c.kv[0] * 2.0 ** -33 * 64 * W.max(-1)[..., None]
    o, lse = o.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (np.abs(o - O) <= tol).all(), f"O off by {(np.abs(o - O) / tol).max():.2f} of its bound"
    assert (np.abs(lse - L) <= delta.T + 2.0 ** -22 * (np.abs(L) + 4)).all()
    assert fb.fp_get_device_status() == 0
