"""The paged-cache entry points without a GPU: what they refuse before any CUDA call, the
binding's own checks, and the float64 reference the GPU tests use."""
import ctypes
import subprocess

import numpy as np
import pytest
import torch

from block_sparse_long_blocks_b200 import binding as fb
from block_sparse_long_blocks_b200 import build
from oracle import paged_cache as pc
from tests._cache_helpers import Case

OK, INVALID, UNSUPPORTED, ALIGNMENT, WORKSPACE = 0, -1, -2, -3, -4
P = 1 << 20  # a pointer that is never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    build.build()
    return fb.load()


def cache(**kw):
    p = dict(dtype=fb.FP_E4M3, scale=fb.FP_SCALE_TOKEN, batch=3, hkv=4, head_dim=128, page_size=64, num_pages=10,
             max_pages_per_req=5, k_pool=P, v_pool=P, k_scale=P, v_scale=P, page_table=P, kv_lens=P)
    return fb.CacheParams(**(p | kw))


def tree(**kw):
    return fb.TreeParams(**(dict(hq=32, total_tokens=6, max_tokens=4, cu_tokens=P) | kw))


BAD_CACHE = [
    (dict(dtype=2), INVALID), (dict(scale=3), INVALID), (dict(scale=fb.FP_SCALE_NONE), INVALID),
    (dict(dtype=fb.FP_BF16), INVALID), (dict(batch=0), INVALID), (dict(batch=4097), UNSUPPORTED),
    (dict(hkv=0), INVALID), (dict(hkv=257), UNSUPPORTED), (dict(head_dim=64), UNSUPPORTED),
    (dict(head_dim=96), UNSUPPORTED), (dict(page_size=8), UNSUPPORTED), (dict(page_size=48), UNSUPPORTED),
    (dict(page_size=131072), UNSUPPORTED), (dict(num_pages=0), INVALID), (dict(max_pages_per_req=0), INVALID),
    (dict(max_pages_per_req=1 << 26), UNSUPPORTED), (dict(k_pool=None), INVALID), (dict(v_pool=None), INVALID),
    (dict(k_scale=None), INVALID), (dict(v_scale=None), INVALID), (dict(page_table=None), INVALID),
    (dict(kv_lens=None), INVALID), (dict(k_pool=P + 8), ALIGNMENT), (dict(v_scale=P + 4), ALIGNMENT),
    (dict(page_table=P + 2), ALIGNMENT),
]


@pytest.mark.parametrize("bad,code", BAD_CACHE)
def test_bad_caches_are_refused_by_every_call(lib, bad, code):
    c = ctypes.byref(cache(**bad))
    t = ctypes.byref(tree(hq=4 * bad.get("hkv", 4) or 4))
    assert lib.fp_cache_write(c, P, 6, P, 512, P, 512, None) == code
    assert lib.fp_cache_read(c, P, 6, None, P, 512, P, 512, None) == code
    assert lib.fp_cache_commit(c, P, 6, P, P, 4, P, None) == code
    assert lib.fp_tree_workspace_size(c, t) == 0
    assert lib.fp_tree_attention(c, t, P, P, None, P, 1 << 40, None) == code


def test_null_structs(lib):
    c, t = ctypes.byref(cache()), ctypes.byref(tree())
    assert lib.fp_cache_write(None, P, 6, P, 512, P, 512, None) == INVALID
    assert lib.fp_tree_attention(c, None, P, P, None, P, 1 << 40, None) == INVALID
    assert lib.fp_tree_attention(None, t, P, P, None, P, 1 << 40, None) == INVALID
    assert lib.fp_tree_workspace_size(None, t) == 0 and lib.fp_tree_workspace_size(c, None) == 0


@pytest.mark.parametrize("call", ["fp_cache_write", "fp_cache_read"])
def test_rows_of_write_and_read(lib, call):
    c = ctypes.byref(cache())

    def f(cu=P, total=6, k=P, ks=512, v=P, vs=512):
        extra = (None,) if call == "fp_cache_read" else ()
        return getattr(lib, call)(c, cu, total, *extra, k, ks, v, vs, None)

    assert f(cu=None) == INVALID and f(total=-1) == INVALID and f(cu=P + 2) == ALIGNMENT
    assert f(k=None) == INVALID and f(v=None) == INVALID and f(ks=504) == INVALID and f(vs=511) == INVALID
    assert f(k=P + 8) == ALIGNMENT and f(ks=516) == ALIGNMENT and f(vs=520 + 1) == ALIGNMENT
    assert f(total=0) == OK  # nothing to do, nothing launched
    if call == "fp_cache_read":
        assert lib.fp_cache_read(c, P, 6, P + 1, P, 512, P, 512, None) == ALIGNMENT


def test_commit_arguments(lib):
    c = ctypes.byref(cache())

    def f(cu=P, total=6, accept=P, num=P, most=4, out=P):
        return lib.fp_cache_commit(c, cu, total, accept, num, most, out, None)

    assert f(cu=None) == INVALID and f(num=None) == INVALID and f(out=None) == INVALID and f(most=-1) == INVALID
    assert f(accept=None) == INVALID and f(most=1025) == UNSUPPORTED
    assert f(accept=P + 1) == ALIGNMENT and f(num=P + 2) == ALIGNMENT and f(out=P + 3) == ALIGNMENT


@pytest.mark.parametrize("bad,code", [
    (dict(hq=0), INVALID), (dict(hq=30), INVALID), (dict(hq=36), UNSUPPORTED), (dict(hq=128), UNSUPPORTED),
    (dict(total_tokens=-1), INVALID), (dict(max_tokens=0), INVALID), (dict(max_tokens=1025), UNSUPPORTED),
    (dict(softmax_scale=-1.0), INVALID), (dict(softmax_scale=float("nan")), INVALID),
    (dict(q_stride=4088), INVALID), (dict(q_stride=4100), ALIGNMENT), (dict(mask=P, mask_words=0), INVALID),
    (dict(mask=P, mask_words=1, max_tokens=33), INVALID), (dict(total_tokens=1 << 27), UNSUPPORTED),
])
def test_bad_trees(lib, bad, code):
    c, t = ctypes.byref(cache()), ctypes.byref(tree(**bad))
    assert lib.fp_tree_attention(c, t, P, P, None, P, 1 << 40, None) == code
    assert lib.fp_tree_workspace_size(c, t) == 0


def test_tree_pointers_and_workspace(lib):
    c, t = ctypes.byref(cache()), ctypes.byref(tree())
    ws = lib.fp_tree_workspace_size(c, t)
    assert ws > 0 and ws % 256 == 0

    def f(t=t, q=P, o=P, lse=None, w=P, n=ws):
        return lib.fp_tree_attention(c, t, q, o, lse, w, n, None)

    assert f(q=None) == INVALID and f(o=None) == INVALID
    assert f(q=P + 8) == ALIGNMENT and f(o=P + 4) == ALIGNMENT and f(lse=P + 2) == ALIGNMENT
    assert f(w=None) == WORKSPACE and f(w=P + 16) == WORKSPACE and f(n=ws - 1) == WORKSPACE
    assert f(t=ctypes.byref(tree(cu_tokens=None))) == INVALID
    assert f(t=ctypes.byref(tree(total_tokens=0)), q=None) == OK
    # the count of all tiles has to fit an int
    big = ctypes.byref(cache(batch=4096, hkv=256, max_pages_per_req=32768))
    assert lib.fp_tree_attention(big, ctypes.byref(tree(hq=256)), P, P, None, P, 1 << 40, None) == UNSUPPORTED


def test_binding_checks_tensors():
    c = Case([5], [2], fmt="e4m3_token")
    k, v, s = c.pool["k"], c.pool["v"], c.scale
    fb.Cache(k, v, c.table, c.kv_lens, s["k"], s["v"])
    for bad in [(k, v.bfloat16(), c.table, c.kv_lens, s["k"], s["v"]), (k, v, c.table.long(), c.kv_lens, s["k"], s["v"]),
                (k, v, c.table, c.kv_lens[:0], s["k"], s["v"]), (k, v, c.table, c.kv_lens),
                (k, v, c.table, c.kv_lens, s["k"], s["v"][:, :1]), (k[0], v[0], c.table, c.kv_lens, s["k"], s["v"]),
                (k.transpose(0, 1), v.transpose(0, 1), c.table, c.kv_lens, s["k"], s["v"]),
                (k.bfloat16(), v.bfloat16(), c.table, c.kv_lens, s["k"], s["v"])]:
        with pytest.raises(ValueError):
            fb.Cache(*bad)


# ---------------------------------------------------------------- the reference's own pins

def test_reference_e4m3_rounding_is_torchs():
    x = torch.arange(-2 ** 15, 2 ** 15, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double()
    x = x[torch.isfinite(x)]
    for scale in (1.0, 0.37, 3.1e-3):
        y = (x * scale).float()  # float32 values, midpoints among them
        want = y.clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
        assert np.array_equal(pc.e4m3_round(y.double().numpy()), want)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3_head", "e4m3_token"])
def test_reference_attention_is_masked_sdpa(fmt):
    c = Case([37, 5, 64], [6, 5, 1], hkv=2, G=3, d=128, page=16, fmt=fmt).trees()
    O, lse, _, _ = pc.tree_attention(c.oracle(), c.cu.numpy(), c.q.double().numpy(), c.see, 128 ** -0.5)
    for r in range(c.R):
        a, b, kv, n = int(c.cu[r]), int(c.cu[r + 1]), c.kv[r], c.n[r]
        flat = c.flat(r, np.arange(kv))
        K, V = [], []
        for name, out in (("k", K), ("v", V)):
            x = c.pool[name].double().flatten(0, 1)[flat]
            if fmt == "e4m3_head":
                x = x * c.scale[name].double()[:, None]
            elif fmt == "e4m3_token":
                x = x * c.scale[name].double().transpose(1, 2).flatten(0, 1)[flat][..., None]
            out.append(x.repeat_interleave(3, dim=1).transpose(0, 1))
        m = torch.ones(n, kv, dtype=torch.bool)
        m[:, kv - n:] = torch.from_numpy(c.see[a:b, :n])
        want = torch.nn.functional.scaled_dot_product_attention(c.q[a:b].double().transpose(0, 1), K[0], V[0], m)
        assert np.allclose(O[a:b].transpose(1, 0, 2), want.numpy(), rtol=1e-10, atol=1e-12)


def test_reference_rows_that_see_nothing():
    c = Case([3], [3], hkv=1, G=2).trees()
    c.see[:] = False
    O, lse, _, _ = pc.tree_attention(c.oracle(), c.cu.numpy(), c.q.double().numpy(), c.see, 1.0)
    assert (O == 0).all() and np.isneginf(lse).all()


def test_native_calls_check_before_any_cuda_call(lib):
    """The per-step calls refuse CPU tensors of the wrong kind by ValueError, other objects by TypeError."""
    c = Case([5, 9], [1, 2], hkv=2, G=2, seed=3)
    cache = fb.Cache(c.pool["k"], c.pool["v"], c.table, c.kv_lens)
    k = torch.zeros(3, 2, 128, dtype=torch.bfloat16)
    for cu, a, b in ((c.cu.long(), k, k), (c.cu[:-1], k, k), (c.cu, k.float(), k), (c.cu, k, k[:2]), (c.cu, k[0], k[0]),
                     (c.cu, k[:, :1], k[:, :1]), (c.cu, k.transpose(1, 2).contiguous().transpose(1, 2), k)):
        with pytest.raises(ValueError):
            fb.fp_cache_write(cache, cu, a, b)
        with pytest.raises(ValueError):
            fb.fp_cache_read(cache, cu, a, b)
    with pytest.raises(ValueError):
        fb.fp_cache_read(cache, c.cu, k, k, starts=torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        fb.fp_cache_commit(cache, c.cu, 3, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32),
                           torch.zeros(2, dtype=torch.int32))
    with pytest.raises(TypeError):
        fb.fp_cache_write(cache, [0, 1, 3], k, k)
    with pytest.raises(TypeError):
        fb.fp_cache_write(cache, c.cu, k, None)


def test_build_includes_the_per_step_calls(monkeypatch, tmp_path):
    """`build()` brings the module that the binding loads beside the library, and again for another torch."""
    made = []

    def compiler(cmd, **kw):
        made.append(cmd[cmd.index("-o") + 1])
        open(made[-1], "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "CALLS_STAMP", str(tmp_path / "stamp"))
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "up_to_date", lambda lib: True)  # (the library itself)
    monkeypatch.setattr(build.subprocess, "run", compiler)
    build.build()
    assert made == [build.CALLS + ".tmp"]
    build.build()
    assert len(made) == 1
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    build.build()
    assert len(made) == 2


def test_calls_of_another_torch_are_refused(lib, monkeypatch):
    monkeypatch.setattr(fb, "_calls", None)
    fb._native()
    monkeypatch.setattr(fb, "_calls", None)
    monkeypatch.setattr(torch, "__version__", "0.0.0")
    with pytest.raises(RuntimeError, match="was built for torch"):
        fb._native()


def test_native_tree_refuses_rows_repeated_by_a_zero_stride(lib):
    """A token stride of 0 means "packed" to the C call, so an expanded q must not reach it."""
    c = Case([5, 9], [1, 2], hkv=2, G=2, seed=3)
    cache = fb.Cache(c.pool["k"], c.pool["v"], c.table, c.kv_lens)
    t = tree(hq=4, total_tokens=3, max_tokens=2)
    q = torch.zeros(1, 4, 128, dtype=torch.bfloat16).expand(3, 4, 128)
    o = torch.zeros(3, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="q must be"):
        fb._native().tree_attention(cache.addr, -1, ctypes.addressof(t), 0, 0, c.cu, q, o, None, None, None)
    with pytest.raises(ValueError, match="o must be"):
        fb._native().tree_attention(cache.addr, -1, ctypes.addressof(t), 0, 0, c.cu, o, q, None, None, None)


@pytest.mark.parametrize("total,stride,off,code", [
    (6, 0, 0, INVALID), (6, 0, 6 * 32 * 128 * 2 - 16, INVALID), (6, 0, 16 - 6 * 32 * 128 * 2, INVALID),
    (6, 6144, 32 * 128 * 2, INVALID), (6, 0, 6 * 32 * 128 * 2, None), (6, 0, -6 * 32 * 128 * 2, None),
    (1, 6144, 32 * 128 * 2, None)])
def test_tree_output_does_not_overlap_q(lib, total, stride, off, code):
    c, t = ctypes.byref(cache()), ctypes.byref(tree(hq=32, total_tokens=total, q_stride=stride))
    ws = lib.fp_tree_workspace_size(c, t)
    Q = P + (1 << 24)
    # (no workspace where the call would be let through: nothing is launched either way)
    got = lib.fp_tree_attention(c, t, Q, Q + off, None, P if code else None, ws, None)
    assert got == (code if code else WORKSPACE)
