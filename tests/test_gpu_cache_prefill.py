"""The prefill over a cache that fp_cache_write filled, chunk by chunk, and a token decoded behind it."""
import numpy as np
import pytest
import torch

from block_sparse_long_blocks_b200 import binding as fb
from oracle import paged_cache as pc
from tests._cache_helpers import Case, check_tree, quantise

pytestmark = pytest.mark.gpu
HQ, HKV = 8, 2


def prefill(c, q, q_scale, n):
    """fp_prefill of the last n[r] tokens of every request, every causal block kept."""
    fp8 = q.dtype is torch.float8_e4m3fn
    cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
    cfg = fb.Config(batch=c.R, max_seqlen=c.table.shape[1] * c.page, hq=HQ, hkv=HKV, block=128, alpha=0.0, fp8=fp8,
                    total_tokens=sum(n), page_size=c.page, max_pages_per_req=c.table.shape[1],
                    num_pages=c.gpu["k"].shape[0])
    p = fb.make_params(cfg, q_scale, c.gpu["ks"], c.gpu["vs"], cu, c.gpu["table"], c.gpu["kv_lens"])
    b = fb.Buffers(p, lse_rows=sum(n), o_shape=tuple(q.shape), hq=HQ)
    fb.fp_prefill(p, q, c.gpu["k"], c.gpu["v"], None, b.idx, b.cnt, b.o, b.workspace, b.lse)
    return b.o, b.lse, cu


@pytest.mark.parametrize("fmt", ["bf16", "e4m3_head"])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_prefill_and_decode_of_written_chunks(fmt, page):
    """Bits of the prefill over written chunks are those over a cache filled by the definition, its values those of dense
    causal attention in float64, and the decoded token attends to the same cache.

    As in `check_tree`; the prefill's weights enter the product rounded to bf16 (e4m3 inputs: f16, and below 2^-24 of the
    row's largest not at all), and lse is the logarithm of the sum of the rounded ones: 2^-8 (2^-11) relative."""
    kv, chunk = [300, 717], [[300, 400], [0, 317]]  # (the second chunk: nothing new of request 0)
    c = Case(kv, chunk[1], hkv=HKV, G=HQ // HKV, page=page, fmt=fmt, seed=page, poison=False)
    g = torch.Generator().manual_seed(page)
    rows = [torch.randn(1017, HKV, 128, generator=g).bfloat16() for _ in "kv"]
    q = (torch.randn(1017, HQ, 128, generator=g) + c.u).bfloat16()
    q_scale = None
    if fmt == "e4m3_head":
        c.scale = {name: x.float().abs().amax((0, 2)) / 448 for name, x in zip("kv", rows)}
        q_scale = (q.float().abs().amax((0, 2)) / 448).cuda()
        q = quantise(q.float(), q_scale.cpu()[:, None])
    c.cuda()
    first = [0, 300]
    done = [0, 0]
    for n in chunk:
        pick = torch.cat([torch.arange(f + d, f + d + m) for f, d, m in zip(first, done, n)])
        done = [d + m for d, m in zip(done, n)]
        c.gpu["kv_lens"].copy_(torch.tensor(done, dtype=torch.int32))
        cu = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32).cuda()
        fb.fp_cache_write(c.cache, cu, *(x[pick].cuda() for x in rows))
        # the same cache from the definition
        for r in range(2):
            at = c.flat(r, np.arange(done[r] - n[r], done[r]))
            for name, x in zip("kv", rows):
                x = x[first[r] + done[r] - n[r]:first[r] + done[r]]
                x = x if fmt == "bf16" else quantise(x.float(), c.scale[name][:, None])
                c.pool[name].view(torch.uint8).flatten(0, 1)[at] = x.view(torch.uint8)
        d = Case(done, n, hkv=HKV, G=HQ // HKV, page=page, fmt=fmt, seed=page, poison=False)
        d.table, d.pool, d.scale = c.table, c.pool, c.scale
        d.cuda()
        if max(n) == 0:
            continue
        o, lse, cu = prefill(c, q[pick].cuda(), q_scale, n)
        want, want_lse, _ = prefill(d, q[pick].cuda(), q_scale, n)
        assert fb.fp_get_device_status() == 0
        assert torch.equal(o, want) and torch.equal(lse, want_lse)
        Q = q[pick].double() if q_scale is None else q[pick].double() * q_scale.cpu().double()[:, None]
        O, L, W, A = pc.tree_attention(d.oracle(), cu.cpu().numpy(), Q.numpy(), None, 128 ** -0.5)
        delta = 2 * (128 + 8) * 2.0 ** -23 * A + 2.0 ** -21 + (max(done) / 16 + 16) * 2.0 ** -23
        p_round = 2.0 ** -7 if fmt == "bf16" else 2.0 ** -10
        tol = 2.0 ** -8 * np.abs(O) + (2 * delta + p_round)[..., None] * W * 1.01 + max(done) * 2.0 ** -24 * W.max()
        assert (np.abs(o.double().cpu().numpy() - O) <= tol).all()
        assert (np.abs(lse.double().cpu().numpy() - L) <= delta.T + p_round + 2.0 ** -22 * (np.abs(L) + 4)).all()
    # one more token per request, decoded
    c.gpu["kv_lens"].add_(1)
    step = torch.arange(3, dtype=torch.int32).cuda()
    last = [torch.randn(2, HKV, 128, generator=g).bfloat16() for _ in "kv"]
    if c.table.shape[1] * page >= max(kv) + 1:
        t = Case([x + 1 for x in kv], [1, 1], hkv=HKV, G=HQ // HKV, page=page, fmt=fmt, seed=page, poison=False)
        fresh = [i for i in range(c.gpu["k"].shape[0]) if i not in set(c.table.flatten().tolist())]
        for r in range(2):  # (a page that begins with this token)
            if kv[r] % page == 0:
                c.table[r, kv[r] // page] = fresh.pop()
        c.gpu["table"].copy_(c.table)
        fb.fp_cache_write(c.cache, step, *(x.cuda() for x in last))
        t.table, t.scale, t.q = c.table, c.scale, torch.randn(2, HQ, 128, generator=g).bfloat16()
        t.pool = {"k": c.gpu["k"].cpu(), "v": c.gpu["v"].cpu()}
        o, lse = t.cuda().attend()
        check_tree(t, o, lse)
    assert fb.fp_get_device_status() == 0
